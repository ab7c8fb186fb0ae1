// Kernels around a step with drafted tokens: the append with norms and rotation
// (rotate_kernel.cu) and the move of accepted drafts (accept_kernel.cu).
#pragma once

#include <stdint.h>

#include <cuda_runtime_api.h>

namespace pkd {

constexpr int kMaxAxes = 4;

struct RotateArgs {
  const uint16_t *q, *k, *v;       // bf16 rows of heads
  uint16_t* q_out;
  int64_t q_token, q_head, out_token, out_head;   // strides in elements
  int64_t k_token, k_head, v_token, v_head;
  const void *q_norm, *k_norm;     // [D] bf16 or fp32, or null
  float eps;
  int32_t norms_f32;
  const uint64_t* turns;           // [rotary_dim / 2] turns per position, times 2^64
  const int32_t* axes;             // [rotary_dim / 2]
  int32_t rotary_dim, pairs;
  float rope_scale;
  const int32_t* rope_positions;   // [n][num_axes]
  int32_t num_axes;
  const int32_t *batch_indices, *positions;
  int32_t n;
  const int32_t *indptr, *indices, *last;
  int32_t num_indices, batch;
  uint8_t* kv;
  int64_t page_bytes, v_bytes, token_bytes, head_bytes;   // strides in the cache
  int32_t num_pages, page_size, hq, hkv;
  // an e4m3 cache's scales: a power of two (lift), scale * lift in [0.5, 2) and its inverse
  struct Divisor {
    float lift, by, inv;
  } k_div, v_div;
  int32_t fp8;
  int32_t* err;
  int32_t segments;                // blocks that share a token's heads (the launcher's)
};
cudaError_t launch_rotate_append(RotateArgs& a, int head_dim, cudaStream_t stream);

constexpr int kMaxAcceptLayers = 128;
constexpr int kMaxAccepted = 1024;
struct AcceptArgs {
  const int32_t *accepted, *drafted;   // [batch][width], [batch]
  int32_t width;
  const int32_t *indptr, *indices, *last;
  int32_t num_indices, batch, num_pages, page_size;
  int64_t page_bytes, v_bytes, token_bytes, head_bytes;
  int32_t hkv, pieces;                 // 16-byte pieces of a head's row
  int32_t* err;
  void* kv[kMaxAcceptLayers];
};
cudaError_t launch_accept(const AcceptArgs& a, int layers, cudaStream_t stream);

}  // namespace pkd
