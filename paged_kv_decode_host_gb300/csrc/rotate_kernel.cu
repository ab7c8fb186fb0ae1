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
// Angles: a frequency is held as turns per position times 2^64, rounded to
// nearest, so p times it in 64-bit integers is the angle modulo one turn, off by
// at most p 2^-65 turns, at any position and sign; its upper 32 bits become the
// fraction of a turn.  Sine and cosine of an angle in [-pi, pi] are the hardware's, absolute
// error under 2^-20: a result is then rounded to 2^-9 of itself or coarser.
//
// The work is moving bytes (24 KB a token of 32 + 2 x 8 heads).  A head is D /
// 16 lanes, each with the two 16-byte pieces that turn together (the half-split
// form needs no exchange between lanes then), so a warp holds 512 / D heads at a
// time and a block's warps share the heads of one token.  The block looks the
// token's slot up and computes its sines and cosines once, into shared memory,
// behind the loads of its first heads; they, and the norms' weights, are read
// from there for every head, so that registers leave room for 32 warps an SM.
// 16,088 tokens of 32 + 2 x 8 heads: 64.8 us, 6.1 TB/s; one piece a lane with
// shuffles between partners took 78.8 (bound by instructions), sines in
// registers 72 (too few warps).
// A token without a slot is flagged and its key and value skipped; its query is
// rotated all the same.
#include <cuda_runtime.h>
#include <stdint.h>

#include "pkd_internal.h"
#include "step.h"
#include "sm103_ptx.cuh"

namespace pkd {
namespace {

using namespace dev;

constexpr int kMostWarps = 4;   // per block
constexpr int kAhead = 2;       // groups of heads whose loads a warp has in flight

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

// Four floats of shared memory, read where they are used: held in registers
// for a whole token they cost half of the warps that an SM can have.
__device__ __forceinline__ float4 lds4(const float* p) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(smem_u32(p)));
  return v;
}

// The two pieces of 8 values that a lane holds of a head.
struct Pieces {
  uint4 a, b;
};

__device__ __forceinline__ void unpack(const uint4& x, float* y) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    y[2 * e] = lo_f32(w[e]);
    y[2 * e + 1] = hi_f32(w[e]);
  }
}
__device__ __forceinline__ uint4 pack(const float* y) {
  return make_uint4(pair_bf16(y[0], y[1]), pair_bf16(y[2], y[3]), pair_bf16(y[4], y[5]),
                    pair_bf16(y[6], y[7]));
}
// y / scale, rounded as the division is (times a rounded 1 / scale alone, a quotient
// between two codes takes the other one): a product, and its rest by the same inverse,
// after Markstein's theorem (IBM J. Res. Dev. 34, 1990).  The power of two that takes
// the scale near 1 is exact wherever the quotient is a code's; one past them all may be
// infinite, and has no rest.
__device__ __forceinline__ float quotient(float y, const RotateArgs::Divisor& d) {
  const float x = y * d.lift, q = x * d.inv;
  return fabsf(q) < 1024.f ? fmaf(-fmaf(q, d.by, -x), d.inv, q) : q;   // (-0 stays -0)
}
__device__ __forceinline__ uint2 pack_e4m3(const float* y, const RotateArgs::Divisor& d) {
  uint32_t two[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) two[e] = pair_e4m3(quotient(y[2 * e], d), quotient(y[2 * e + 1], d));
  return make_uint2(two[0] | (two[1] << 16), two[2] | (two[3] << 16));
}

template <int D, bool kNorm, bool kPairs>
__global__ void __launch_bounds__(kMostWarps * 32, 8)
    rotate_kernel(const __grid_constant__ RotateArgs a) {
  constexpr int kLanes = D / 16, kHeads = 32 / kLanes;   // lanes of a head, heads of a warp
  __shared__ __align__(16) float cosines[D / 2], sines[D / 2];
  __shared__ __align__(16) float norms[kNorm ? 2 : 1][kNorm ? D : 1];   // weights of queries, keys
  __shared__ int64_t slot_shared;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % kLanes, own = lane / kLanes;
  const int q_groups = (a.hq + kHeads - 1) / kHeads;
  const int groups = q_groups + (2 * a.hkv + kHeads - 1) / kHeads;
  const int64_t i = blockIdx.x / a.segments;
  const int warps = blockDim.x >> 5;
  // this warp's groups of heads: g0, g0 + stride, ...
  const int stride = warps * a.segments, g0 = (int)(blockIdx.x % a.segments) * warps + warp;
  pdl_wait();   // (the launch alone overlaps the kernel before)

  // This lane's pieces: in the half-split form those of the dims 8 p and 8 p +
  // R / 2, the lanes behind R share what does not turn; else piece p and D / 16
  // behind it.
  const int half = a.rotary_dim >> 1;
  int pa = sub, pb = sub + kLanes;
  bool ta = 8 * pa < a.rotary_dim, tb = 8 * pb < a.rotary_dim;
  if (!kPairs) {
    ta = tb = 8 * sub < half;
    pa = ta ? sub : half / 8 + sub;
    pb = ta ? sub + half / 8 : sub + kLanes;
  }
  const int ea = 8 * pa, eb = 8 * pb;   // first dims

  Pieces x[kAhead];
  auto load = [&](int g, Pieces& to) {
    to.a = to.b = make_uint4(0, 0, 0, 0);
    const uint16_t* p = nullptr;
    if (g < q_groups) {
      const int h = g * kHeads + own;
      if (h < a.hq) p = a.q + i * a.q_token + h * a.q_head;
    } else {
      const int h = (g - q_groups) * kHeads + own;
      if (h < a.hkv)
        p = a.k + i * a.k_token + h * a.k_head;
      else if (h < 2 * a.hkv)
        p = a.v + i * a.v_token + (h - a.hkv) * a.v_head;
    }
    if (p != nullptr) {
      to.a = __ldcs(reinterpret_cast<const uint4*>(p + ea));
      to.b = __ldcs(reinterpret_cast<const uint4*>(p + eb));
    }
  };
#pragma unroll
  for (int u = 0; u < kAhead; ++u) load(g0 + u * stride, x[u]);
  // the token's slot, cosines and sines, once per block
  if (threadIdx.x == blockDim.x - 1) {
    const int64_t at = slot_of(a, i);
    if (at < 0 && a.err != nullptr) atomicOr(a.err, PKD_DEV_ERR_BOUNDS);
    slot_shared = at;
  }
  for (int f = threadIdx.x; f < a.rotary_dim >> 1; f += blockDim.x) {
    const int axis = min(max(__ldg(a.axes + f), 0), a.num_axes - 1);
    const int64_t p = __ldg(a.rope_positions + i * a.num_axes + axis);
    const int32_t part = (int32_t)(((uint64_t)p * __ldg(a.turns + f)) >> 32);
    float sn, cs;
    __sincosf((float)part * (float)(6.283185307179586 / 4294967296.0), &sn, &cs);
    cosines[f] = cs * a.rope_scale;
    sines[f] = sn * a.rope_scale;
  }
  if constexpr (kNorm) {
    for (int d = threadIdx.x; d < 2 * D; d += blockDim.x) {
      const void* p = d < D ? a.q_norm : a.k_norm;
      const int e = d < D ? d : d - D;
      norms[d / D][e] = p == nullptr  ? 1.f
                        : a.norms_f32 ? __ldg(static_cast<const float*>(p) + e)
                                      : lo_f32(__ldg(static_cast<const uint16_t*>(p) + e));
    }
  }
  __syncthreads();
  const int64_t slot = slot_shared;
  // the norm (`on`: this lane's head has one) and the rotation of a head's values
  auto norm = [&](float (&y)[16], bool on, const float* weights) {
    if constexpr (kNorm) {
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) sum = fmaf(y[e], y[e], sum);
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
      if (on) {
        const float r = rsqrtf(sum * (1.f / D) + a.eps);
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const float4 w = lds4(weights + (e < 8 ? ea + e : eb + e - 8));
          y[e] *= r * w.x;
          y[e + 1] *= r * w.y;
          y[e + 2] *= r * w.z;
          y[e + 3] *= r * w.w;
        }
      }
    }
  };
  auto turn = [&](float (&y)[16]) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {   // pairs (ea + e, eb + e), or (2 e', 2 e' + 1) of either piece
      if (!(kPairs && q == 1 ? tb : ta)) continue;
      const int f = kPairs ? (q == 0 ? 4 * pa : 4 * pb) : ea + 4 * q;
      const float4 c4 = lds4(cosines + f), s4 = lds4(sines + f);
      const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int lo = kPairs ? 8 * q + 2 * e : 4 * q + e, hi = kPairs ? lo + 1 : lo + 8;
        const float u = y[lo], v = y[hi];
        y[lo] = fmaf(-v, s[e], u * c[e]);
        y[hi] = fmaf(u, s[e], v * c[e]);
      }
    }
  };

  for (int g = g0; g < groups; g += kAhead * stride) {
    if (g > g0) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) load(g + u * stride, x[u]);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int at = g + u * stride;
      if (at >= groups) break;
      float y[16];
      unpack(x[u].a, y);
      unpack(x[u].b, y + 8);
      const bool queries = at < q_groups;
      const int h = (queries ? at : at - q_groups) * kHeads + own;
      const bool is_k = !queries && h < a.hkv;
      norm(y, queries ? a.q_norm != nullptr : is_k && a.k_norm != nullptr, norms[kNorm && !queries]);
      if (queries) {
        turn(y);
        if (h < a.hq) {
          uint16_t* p = a.q_out + i * a.out_token + h * a.out_head;
          __stcs(reinterpret_cast<uint4*>(p + ea), pack(y));
          __stcs(reinterpret_cast<uint4*>(p + eb), pack(y + 8));
        }
        continue;
      }
      if (is_k) turn(y);
      if (h >= 2 * a.hkv || slot < 0) continue;
      uint8_t* dst = a.kv + slot + (is_k ? h * a.head_bytes : a.v_bytes + (h - a.hkv) * a.head_bytes);
      if (a.fp8) {
        const RotateArgs::Divisor div = is_k ? a.k_div : a.v_div;
        *reinterpret_cast<uint2*>(dst + ea) = pack_e4m3(y, div);
        *reinterpret_cast<uint2*>(dst + eb) = pack_e4m3(y + 8, div);
      } else {
        // (a value's bits as they are, a NaN's too)
        *reinterpret_cast<uint4*>(dst + 2 * ea) = is_k ? pack(y) : x[u].a;
        *reinterpret_cast<uint4*>(dst + 2 * eb) = is_k ? pack(y + 8) : x[u].b;
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
  // A block per token: 4 warps, and 2 where the tokens are many times the blocks
  // that are resident anyway (16,088 tokens of 32 + 2 x 8 heads: 64.8 us with 2
  // warps, 70.1 with 4; 1,152 of 64 + 2 x 8 with norms: 12.9 and 11.1; 64 of 32
  // + 2 x 8: 3.1 and 2.6).  Tokens fewer than two per SM are shared by more
  // blocks, down to a group of heads per warp.
  constexpr int kManyTokens = 4096, kBlocksWanted = 304;
  const int warps = a.n >= kManyTokens ? 2 : kMostWarps;
  const int heads = 512 / head_dim;   // of a warp
  const int groups = (a.hq + heads - 1) / heads + (2 * a.hkv + heads - 1) / heads;
  const int most = (groups + warps - 1) / warps, wanted = (kBlocksWanted + a.n - 1) / a.n;
  a.segments = wanted < most ? wanted : most;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)a.n * a.segments));
  cfg.blockDim = dim3(warps * 32);
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
