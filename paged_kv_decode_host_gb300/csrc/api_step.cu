// C ABI of the calls around a step with drafted tokens: argument checks of
// pkd_rotate_append_kv and pkd_accept_kv (kernels: rotate_kernel.cu,
// accept_kernel.cu).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "pkd_internal.h"
#include "step.h"

using namespace pkd;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Strides of [n][heads][dim] rows of 16-byte pieces; `written`: no two rows may
// share memory, as far as one stride shows it.
bool good_strides(int64_t token, int64_t head, int32_t n, int32_t heads, int32_t dim, bool written) {
  const int64_t most = (int64_t)1 << 40, least = written ? dim : 0;
  return (n <= 1 || (token % 8 == 0 && token >= least && token <= most)) &&
         (heads <= 1 || (head % 8 == 0 && head >= least && head <= most));
}

RotateArgs::Divisor divisor(float scale) {
  int e;
  std::frexp(scale, &e);
  const float lift = std::ldexp(1.f, e < -126 ? 127 : 1 - e), by = scale * lift;
  return {lift, by, 1.f / by};
}

bool good_scale(float s) { return std::isfinite(s) && s > 0.f && std::isfinite(1.f / s); }

}  // namespace

extern "C" {

int pkd_rotate_append_kv(const void* q, int64_t q_token, int64_t q_head, void* q_out,
                         int64_t out_token, int64_t out_head, const void* k, int64_t k_token,
                         int64_t k_head, const void* v, int64_t v_token, int64_t v_head,
                         const void* q_norm, const void* k_norm, int32_t norms_f32, float eps,
                         const uint64_t* turns, const int32_t* axes, int32_t rotary_dim,
                         int32_t interleaved, float rope_scale, const int32_t* rope_positions,
                         int32_t num_axes, const int32_t* batch_indices,
                         const int32_t* positions, int32_t n, const int32_t* indptr,
                         const int32_t* indices, int32_t num_indices,
                         const int32_t* last_page_len, int32_t batch, void* kv,
                         int32_t num_pages, int32_t page_size, int32_t num_qo_heads,
                         int32_t num_kv_heads, int32_t head_dim, float k_scale, float v_scale,
                         uint32_t flags, int32_t* err, void* stream) {
  if ((flags & ~(PKD_FLAG_HND | PKD_FLAG_KV_FP8)) != 0) return PKD_E_INVALID_ARG;
  const bool fp8 = (flags & PKD_FLAG_KV_FP8) != 0, hnd = (flags & PKD_FLAG_HND) != 0;
  if (n < 0 || batch < 0 || num_indices < 0 || num_pages < 1 || page_size < 1 ||
      num_qo_heads < 0 || num_qo_heads > 65536 || num_kv_heads < 1 || num_kv_heads > 65536 ||
      num_axes < 1 || num_axes > kMaxAxes || !std::isfinite(eps) || eps < 0.f ||
      !std::isfinite(rope_scale) || (norms_f32 & ~1) != 0 || (interleaved & ~1) != 0)
    return PKD_E_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return PKD_E_UNSUPPORTED_SHAPE;
  if (rotary_dim < 0 || rotary_dim > head_dim || rotary_dim % (interleaved ? 8 : 16) != 0)
    return PKD_E_INVALID_ARG;
  if (!good_scale(k_scale) || !good_scale(v_scale) || (!fp8 && (k_scale != 1.f || v_scale != 1.f)))
    return PKD_E_INVALID_ARG;
  if (n == 0) return PKD_OK;
  if (!k || !v || !batch_indices || !positions || !indptr || !indices || !last_page_len || !kv ||
      (rotary_dim > 0 && (!turns || !axes || !rope_positions)) ||
      (num_qo_heads > 0 && (!q || !q_out)))
    return PKD_E_INVALID_ARG;
  const int norm_align = norms_f32 ? 4 : 2;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(kv, 16) || !aligned(turns, 8) ||
      !aligned(axes, 4) || !aligned(rope_positions, 4) || !aligned(err, 4) ||
      !aligned(q_norm, norm_align) || !aligned(k_norm, norm_align) ||
      (num_qo_heads > 0 && (!aligned(q, 16) || !aligned(q_out, 16))))
    return PKD_E_INVALID_ARG;
  if (!good_strides(k_token, k_head, n, num_kv_heads, head_dim, false) ||
      !good_strides(v_token, v_head, n, num_kv_heads, head_dim, false) ||
      (num_qo_heads > 0 && (!good_strides(q_token, q_head, n, num_qo_heads, head_dim, false) ||
                            !good_strides(out_token, out_head, n, num_qo_heads, head_dim, true))))
    return PKD_E_INVALID_ARG;
  RotateArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_out = static_cast<uint16_t*>(q_out);
  // (a stride that no second row uses may be anything)
  a.q_token = n > 1 ? q_token : 0;
  a.out_token = n > 1 ? out_token : 0;
  a.k_token = n > 1 ? k_token : 0;
  a.v_token = n > 1 ? v_token : 0;
  a.q_head = num_qo_heads > 1 ? q_head : 0;
  a.out_head = num_qo_heads > 1 ? out_head : 0;
  a.k_head = num_kv_heads > 1 ? k_head : 0;
  a.v_head = num_kv_heads > 1 ? v_head : 0;
  a.q_norm = q_norm;
  a.k_norm = k_norm;
  a.eps = eps;
  a.norms_f32 = norms_f32;
  a.turns = turns;
  a.axes = axes;
  a.rotary_dim = rotary_dim;
  a.pairs = interleaved;
  a.rope_scale = rope_scale;
  a.rope_positions = rope_positions;
  a.num_axes = num_axes;
  a.batch_indices = batch_indices;
  a.positions = positions;
  a.n = n;
  a.indptr = indptr;
  a.indices = indices;
  a.last = last_page_len;
  a.num_indices = num_indices;
  a.batch = batch;
  a.kv = static_cast<uint8_t*>(kv);
  const int64_t head = (int64_t)head_dim * (fp8 ? 1 : 2);
  a.v_bytes = (int64_t)page_size * num_kv_heads * head;
  a.page_bytes = 2 * a.v_bytes;
  a.token_bytes = hnd ? head : head * num_kv_heads;
  a.head_bytes = hnd ? head * page_size : head;
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.hq = num_qo_heads;
  a.hkv = num_kv_heads;
  a.k_div = divisor(k_scale);
  a.v_div = divisor(v_scale);
  a.fp8 = fp8 ? 1 : 0;
  a.err = err;
  return launch_rotate_append(a, head_dim, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PKD_OK
             : PKD_E_CUDA;
}

int pkd_accept_kv(int32_t layers, void* const* kv, const int32_t* accepted, int32_t width,
                  const int32_t* drafted, const int32_t* indptr, const int32_t* indices,
                  int32_t num_indices, const int32_t* last_page_len, int32_t batch,
                  int32_t num_pages, int32_t page_size, int32_t num_kv_heads, int32_t head_dim,
                  uint32_t flags, int32_t* err, void* stream) {
  if ((flags & ~(PKD_FLAG_HND | PKD_FLAG_KV_FP8)) != 0) return PKD_E_INVALID_ARG;
  const int elem = (flags & PKD_FLAG_KV_FP8) ? 1 : 2;
  if (layers < 1 || layers > kMaxAcceptLayers || !kv || width < 0 || width > kMaxAccepted ||
      batch < 0 || num_indices < 0 || num_pages < 1 || page_size < 1 || num_kv_heads < 1 ||
      head_dim < 1 || ((int64_t)head_dim * elem) % 16 != 0 ||
      (int64_t)head_dim * elem * num_kv_heads > (1 << 24))
    return PKD_E_INVALID_ARG;
  AcceptArgs a{};
  uintptr_t order[kMaxAcceptLayers];
  for (int32_t l = 0; l < layers; ++l) {
    if (!kv[l] || !aligned(kv[l], 16)) return PKD_E_INVALID_ARG;
    a.kv[l] = kv[l];
    order[l] = (uintptr_t)kv[l];
  }
  std::sort(order, order + layers);
  if (std::adjacent_find(order, order + layers) != order + layers) return PKD_E_INVALID_ARG;
  if (batch == 0 || width == 0) return PKD_OK;
  const int64_t head = (int64_t)head_dim * elem;
  a.v_bytes = (int64_t)page_size * num_kv_heads * head;
  a.page_bytes = 2 * a.v_bytes;
  // two layers in one place would race (and a pool past the address space wraps around)
  if (a.page_bytes > ((int64_t)1 << 56) / num_pages) return PKD_E_INVALID_ARG;
  for (int32_t l = 1; l < layers; ++l)
    if (order[l] - order[l - 1] < (uintptr_t)(num_pages * a.page_bytes)) return PKD_E_INVALID_ARG;
  if (!accepted || !drafted || !indptr || !indices || !last_page_len || !aligned(accepted, 4) ||
      !aligned(drafted, 4) || !aligned(err, 4))
    return PKD_E_INVALID_ARG;
  a.accepted = accepted;
  a.drafted = drafted;
  a.width = width;
  a.indptr = indptr;
  a.indices = indices;
  a.last = last_page_len;
  a.num_indices = num_indices;
  a.batch = batch;
  a.num_pages = num_pages;
  a.page_size = page_size;
  const bool hnd = (flags & PKD_FLAG_HND) != 0;
  a.token_bytes = hnd ? head : head * num_kv_heads;
  a.head_bytes = hnd ? head * page_size : head;
  a.hkv = num_kv_heads;
  a.pieces = (int32_t)(head / 16);
  a.err = err;
  return launch_accept(a, layers, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PKD_OK
                                                                                    : PKD_E_CUDA;
}

}  // extern "C"
