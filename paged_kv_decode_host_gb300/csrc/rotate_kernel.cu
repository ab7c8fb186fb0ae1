// New tokens' queries and keys normed per head and rotated by their positions,
// keys and values written into their page slots, in one pass (sm_103a).
//
// For a head's values x (queries and keys, each with or without a norm):
//     y = x / sqrt(mean(x^2) + eps) * w
// then, for every pair (a, b) of the first R dims (a = i, b = i + R / 2, or a =
// 2 i, b = 2 i + 1) with its frequency f_i and its axis' position p,
//     (y_a cos - y_b sin, y_b cos + y_a sin) * scale,  angle p f_i.
// Queries go to q_out (bf16), keys and values to the cache (bf16, or e4m3 of
// x / k_scale and x / v_scale, saturated), each rounded once, from fp32.
//
// Angles: a frequency is held as turns per position times 2^64, so p times it
// in 64-bit integers is the angle modulo one turn, off by at most p 2^-65
// turns, at any position and sign; its upper 32 bits become the fraction of a
// turn.  Sine and cosine of an angle in [-pi, pi] are the hardware's, absolute
// error under 2^-20: a result is then rounded to 2^-9 of itself or coarser.
//
// The work is moving bytes (24 KB a token of 32 + 2 x 8 heads).  A head is D /
// 8 lanes of 16 bytes, so a warp holds 256 / D heads at a time and walks the
// heads of one token; its lanes' sines and cosines stay in registers for all of
// them.  Partners of the half-split form are R / 16 lanes away.  Few tokens are
// spread over more warps, down to one group of heads each (a lane's 8 sincos
// pairs are then computed once per group): measured at the entry of the launch.
// The table is looked up by every warp that writes a key or a value, behind the
// loads of its first heads.  A token without a slot is flagged and its key and
// value skipped; its query is rotated all the same.
#include <cuda_runtime.h>
#include <stdint.h>

#include "pkd_internal.h"
#include "step.h"
#include "sm103_ptx.cuh"

namespace pkd {
namespace {

using namespace dev;

constexpr int kWarps = 4;     // per block
constexpr int kAhead = 4;     // groups of heads whose loads are in flight per warp

__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ uint32_t pair_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// two floats to e4m3 (lo in the low byte), to nearest even, at most 448
__device__ __forceinline__ uint32_t pair_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The slot of token i in the cache, in bytes, or -1.
__device__ __forceinline__ int64_t slot_of(const RotateArgs& a, int64_t i) {
  const int b = a.batch_indices[i], pos = a.positions[i];
  if (b < 0 || b >= a.batch) return -1;
  const int p0 = a.indptr[b], p1 = a.indptr[b + 1], last = a.last[b];
  const int64_t len = (int64_t)a.page_size * ((int64_t)p1 - p0 - 1) + last;
  if (p0 < 0 || p1 <= p0 || p1 > a.num_indices || last < 1 || last > a.page_size || pos < 0 ||
      pos >= len)
    return -1;
  const int page = a.indices[p0 + pos / a.page_size];
  if (page < 0 || page >= a.num_pages) return -1;
  return page * a.page_bytes + (pos % a.page_size) * a.token_bytes;
}

template <int D, bool kNorm, bool kPairs>
__global__ void __launch_bounds__(kWarps * 32) rotate_kernel(const __grid_constant__ RotateArgs a) {
  constexpr int kLanes = D / 8, kHeads = 32 / kLanes;   // lanes of a head, heads of a warp
  const int lane = threadIdx.x & 31, sub = lane % kLanes;
  const int heads = a.hq + 2 * a.hkv;
  const int groups = (heads + kHeads - 1) / kHeads;
  const int segments = (groups + a.segment - 1) / a.segment;
  const int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t i = task / segments;
  pdl_wait();   // (the launch alone overlaps the kernel before)
  if (i >= a.n) return;
  const int g0 = (int)(task % segments) * a.segment, g1 = min(groups, g0 + a.segment);

  // this lane's 16 bytes of head h
  auto source = [&](int h) -> const uint4* {
    const uint16_t* p = h < a.hq ? a.q + i * a.q_token + h * a.q_head
                        : h < a.hq + a.hkv ? a.k + i * a.k_token + (h - a.hq) * a.k_head
                                           : a.v + i * a.v_token + (h - a.hq - a.hkv) * a.v_head;
    return reinterpret_cast<const uint4*>(p + 8 * sub);
  };
  uint4 x[kAhead];
  auto load = [&](int g) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int h = (g + u) * kHeads + lane / kLanes;
      x[u] = make_uint4(0, 0, 0, 0);
      if (g + u < g1 && h < heads) x[u] = __ldcs(source(h));
    }
  };
  load(g0);
  const bool writes = g1 * kHeads > a.hq;   // a key or value in this segment
  const int64_t slot = writes ? slot_of(a, i) : -1;
  if (writes && slot < 0 && lane == 0 && a.err != nullptr) atomicOr(a.err, PKD_DEV_ERR_BOUNDS);

  // cosines, and sines with the sign that this lane's values take them with
  float c[8], s[8];
  const bool turns = 8 * sub < a.rotary_dim;
  const int half = a.rotary_dim >> 1;
  const int partner = kPairs ? lane : 8 * sub < half ? lane + half / 8 : lane - half / 8;
#pragma unroll
  for (int e = 0; e < (kPairs ? 4 : 8); ++e) {
    const int f = kPairs ? 4 * sub + e : 8 * sub < half ? 8 * sub + e : 8 * sub - half + e;
    float cs = 1.f, sn = 0.f;
    if (turns) {
      const int axis = min(max(__ldg(a.axes + f), 0), a.num_axes - 1);
      const int64_t p = __ldg(a.rope_positions + i * a.num_axes + axis);
      const int32_t part = (int32_t)(((uint64_t)p * __ldg(a.turns + f)) >> 32);
      __sincosf((float)part * (float)(6.283185307179586 / 4294967296.0), &sn, &cs);
      cs *= a.rope_scale;
      sn *= a.rope_scale;
    }
    if (kPairs) {
      c[2 * e] = c[2 * e + 1] = cs;
      s[2 * e] = -sn;
      s[2 * e + 1] = sn;
    } else {
      c[e] = cs;
      s[e] = 8 * sub < half ? -sn : sn;
    }
  }
  float wq[8], wk[8];
  if constexpr (kNorm) {
    auto weights = [&](const void* p, float (&w)[8]) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        w[e] = p == nullptr ? 1.f
               : a.norms_f32 ? __ldg(static_cast<const float*>(p) + 8 * sub + e)
                             : lo_f32(__ldg(static_cast<const uint16_t*>(p) + 8 * sub + e));
    };
    weights(a.q_norm, wq);
    weights(a.k_norm, wk);
  }

  for (int g = g0; g < g1; g += kAhead) {
    if (g > g0) load(g);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (g + u >= g1) break;
      const int h = (g + u) * kHeads + lane / kLanes;   // (past the last head: nothing is written)
      const bool is_q = h < a.hq, is_k = !is_q && h < a.hq + a.hkv;
      const uint32_t raw[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      float y[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[2 * e] = lo_f32(raw[e]);
        y[2 * e + 1] = hi_f32(raw[e]);
      }
      if constexpr (kNorm) {
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(y[e], y[e], sum);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
        if (is_q ? a.q_norm != nullptr : is_k && a.k_norm != nullptr) {
          const float r = rsqrtf(sum * (1.f / D) + a.eps);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = y[e] * r * (is_q ? wq[e] : wk[e]);
        }
      }
      float other[8];
      if constexpr (kPairs) {
#pragma unroll
        for (int e = 0; e < 8; ++e) other[e] = y[e ^ 1];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) other[e] = __shfl_sync(kFull, y[e], partner & 31);
      }
      if ((is_q || is_k) && turns) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = fmaf(other[e], s[e], y[e] * c[e]);
      }
      if (is_q) {
        __stcs(reinterpret_cast<uint4*>(a.q_out + i * a.out_token + h * a.out_head + 8 * sub),
               make_uint4(pair_bf16(y[0], y[1]), pair_bf16(y[2], y[3]), pair_bf16(y[4], y[5]),
                          pair_bf16(y[6], y[7])));
      } else if (h < heads && slot >= 0) {
        uint8_t* dst = a.kv + slot + (is_k ? 0 : a.v_bytes) +
                       (int64_t)(h - a.hq - (is_k ? 0 : a.hkv)) * a.head_bytes;
        if (a.fp8) {
          const float m = is_k ? a.k_mul : a.v_mul;
          *reinterpret_cast<uint2*>(dst + 8 * sub) =
              make_uint2(pair_e4m3(y[0] * m, y[1] * m) | (pair_e4m3(y[2] * m, y[3] * m) << 16),
                         pair_e4m3(y[4] * m, y[5] * m) | (pair_e4m3(y[6] * m, y[7] * m) << 16));
        } else {
          // (a value's bits as they are, a NaN's too)
          *reinterpret_cast<uint4*>(dst + 16 * sub) =
              is_k ? make_uint4(pair_bf16(y[0], y[1]), pair_bf16(y[2], y[3]),
                                pair_bf16(y[4], y[5]), pair_bf16(y[6], y[7]))
                   : x[u];
        }
      }
    }
  }
}

template <int D>
const void* kernel_of(bool norm, bool pairs) {
  if (norm)
    return pairs ? reinterpret_cast<const void*>(&rotate_kernel<D, true, true>)
                 : reinterpret_cast<const void*>(&rotate_kernel<D, true, false>);
  return pairs ? reinterpret_cast<const void*>(&rotate_kernel<D, false, true>)
               : reinterpret_cast<const void*>(&rotate_kernel<D, false, false>);
}

}  // namespace

cudaError_t launch_rotate_append(RotateArgs& a, int head_dim, cudaStream_t stream) {
  const bool norm = a.q_norm != nullptr || a.k_norm != nullptr, pairs = a.pairs != 0;
  const void* f = head_dim == 64    ? kernel_of<64>(norm, pairs)
                  : head_dim == 128 ? kernel_of<128>(norm, pairs)
                                    : kernel_of<256>(norm, pairs);
  // as few segments a token as still make kWarpsWanted warps
  constexpr int kWarpsWanted = 152 * 16;
  const int groups = (a.hq + 2 * a.hkv + 256 / head_dim - 1) / (256 / head_dim);
  const int wanted = (kWarpsWanted + a.n - 1) / a.n;
  const int parts = wanted < groups ? wanted : groups;
  a.segment = (groups + parts - 1) / parts;
  const int64_t warps = (int64_t)a.n * ((groups + a.segment - 1) / a.segment);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((warps + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {&a};
  return cudaLaunchKernelExC(&cfg, f, args);
}

}  // namespace pkd
