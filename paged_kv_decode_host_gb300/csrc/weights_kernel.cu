// The attention weight each cached token receives in a decode step, added to
// a running sum kept beside the cache, for sm_103a.
//
// For a token t of request b and KV head h, with the g query heads of h and
// the lse that the step's attention returned:
//     w_t = sum_{j < g} exp(k_scale * q_j . k_t / sqrt(128) - lse_j)
//     weights[page][h][slot] = (t is new ? 0 : weights[page][h][slot]) + w_t
// The softmax statistics are known, so no maximum, no sum and no V are
// needed: K is read once and nothing else of that size, and a token's sum is
// written by the one warp that owns it -- no atomics, the same bits every
// run.
//
// HBM bound (2 x 256 flop per 256-byte row and query head).  One block per
// SM walks the planner's items; a warp takes 16 tokens of one KV head at a
// time.  The scores are mma.sync m16n8k16 products with the tokens as the 16
// rows and the group's heads as the 8 columns: K goes from global memory
// straight into the A fragments, with no shared memory and for any layout or
// page size, because the order of the contraction is free -- a lane takes 16
// contiguous bytes of a row for two (bf16) or four (E4M3) steps and the
// queries are permuted alike.  (A tcgen05 product would have to stage K in
// shared memory to use 8 of its columns.)
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "evict.h"
#include "pkd_internal.h"
#include "sm103_ptx.cuh"

namespace pkd {
namespace {

using namespace dev;

constexpr int kWarps = 24;   // a multiple of 1, 2, 4 and 8 heads: a warp keeps its head
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load_stream(const uint8_t* p, uint64_t policy) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::cache_hint.v4.u32 {%0,%1,%2,%3}, [%4], %5;"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p), "l"(policy));
  return v;
}

// four E4M3 bytes to two f16 pairs (exact)
__device__ __forceinline__ void e4m3x4(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b;}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// kTiles: the page size is a multiple of 16, so that a tile lies in one page.
template <bool kFp8, bool kTiles>
__global__ void __launch_bounds__(kWarps * 32, 1) weights_kernel(const __grid_constant__ WeightsArgs a) {
  if (!schedule_ready(a.sched + H_EPOCH, a.wait_epoch, a.err)) return;
  constexpr int kPieces = kFp8 ? 2 : 4;      // 16-byte pieces of a row per lane
  constexpr int kSteps = kFp8 ? 4 : 2;       // products fed by a piece
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r8 = lane >> 2, c4 = lane & 3;   // row (token, or head of the queries) and quad lane
  const int per = kWarps / a.hkv;            // warps of one head
  const int h = warp % a.hkv, sub = warp / a.hkv;
  if (sub >= per) return;                    // 24 is not a multiple of 5 or 7 heads
  const uint64_t policy = l2_evict_first_policy();
  const int g = a.hq / a.hkv;
  const int P = a.page_size;
  const int nnz = a.sched[H_NNZ];
  const int it0 = a.sched[a.off_cta + blockIdx.x];
  const int it1 = a.sched[a.off_cta + blockIdx.x + 1];
  for (int it = it0; it < it1; ++it) {
    const int32_t* item = a.sched + a.off_items + (int64_t)it * kItemWords;
    const int req = item[0], tb = item[1], n = item[2] - item[1];
    const int32_t* pages = a.sched + a.off_pages + item[4];
    const int len = a.sched[a.off_pages + nnz + req];
    const int fresh =   // the first new token, from tb
        (a.new_tokens ? len - min(max(a.new_tokens[req], 0), len) : len) - tb;
    const int age0 = a.positions ? a.seen[req] - len + tb : 0;
    // queries of this KV head: lane's row is query head r8, in the pieces'
    // permuted order.  For E4M3 they become f16, scaled by a power of two
    // (exact down to 2^-29 of the head's largest value).
    uint32_t qf[kPieces][kSteps][2];
    float qs = 1.f;
    {
      const uint16_t* qr = a.q + ((int64_t)req * a.hq + h * g + (r8 < g ? r8 : 0)) * kHeadDim;
      if constexpr (kFp8) {
        float top = 0.f;
        uint4 v[kPieces][2];
#pragma unroll
        for (int p = 0; p < kPieces; ++p)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            v[p][i] = *reinterpret_cast<const uint4*>(qr + 64 * p + 16 * c4 + 8 * i);
            const uint32_t w[4] = {v[p][i].x, v[p][i].y, v[p][i].z, v[p][i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              top = fmaxf(top, fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
          }
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
        // 2^(14 - exponent of top), as two factors that stay normal
        const int ex = top > 0.f && top < CUDART_INF_F ? 14 - ilogbf(top) : 0;
        qs = r8 < g ? ldexpf(1.f, ex < 100 ? ex : 100) : 0.f;
#pragma unroll
        for (int p = 0; p < kPieces; ++p)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w[4] = {v[p][i].x, v[p][i].y, v[p][i].z, v[p][i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __half2 x = r8 < g ? __floats2half2_rn(bf16_lo(w[e]) * qs, bf16_hi(w[e]) * qs)
                                       : __floats2half2_rn(0.f, 0.f);
              qf[p][2 * i + (e >> 1)][e & 1] = *reinterpret_cast<const uint32_t*>(&x);
            }
          }
      } else {
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
          const uint4 v = *reinterpret_cast<const uint4*>(qr + 32 * p + 8 * c4);
          qf[p][0][0] = r8 < g ? v.x : 0u;
          qf[p][0][1] = r8 < g ? v.y : 0u;
          qf[p][1][0] = r8 < g ? v.z : 0u;
          qf[p][1][1] = r8 < g ? v.w : 0u;
        }
      }
    }
    // this lane's two columns of the products: heads 2 c4 and 2 c4 + 1
    float sc[2], base[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int j = 2 * c4 + e;
      const float s = __shfl_sync(kFull, qs, 4 * j);   // the scale of that head's queries
      sc[e] = kFp8 ? a.scale_log2 / (s > 0.f ? s : 1.f) : a.scale_log2;
      const float l = j < g ? a.lse[(int64_t)req * a.hq + h * g + j] : 0.f;
      base[e] = l * kLog2e;
      // an empty state (lse -inf) gives its tokens nothing
      if (j >= g || l == -CUDART_INF_F) base[e] = CUDART_INF_F;
    }
    const int tiles = (n + 15) >> 4;
    // a tile's pages, looked up a tile before they are used: one with kTiles,
    // else the lane's two tokens'
    int pg[2] = {0, 0};
    auto look_up = [&](int tile) {
      const int t = 16 * tile;
      if constexpr (kTiles) {
        pg[0] = t < n ? pages[t / P] : 0;
      } else {
        pg[0] = t + r8 < n ? pages[(t + r8) / P] : 0;
        pg[1] = t + r8 + 8 < n ? pages[(t + r8 + 8) / P] : 0;
      }
    };
    // one tile on its way: K, the lane's own sum (lanes 0 and 1 of a quad own
    // its two tokens), and where that lies
    struct Tile {
      uint4 k[2][kPieces];
      float old;
      int64_t at;
    };
    const int64_t lane_at = h * a.head_bytes + 16 * c4;
    auto fetch = [&](int tile, Tile& x) {
      int64_t slot_at[2];
      if constexpr (kTiles) {
        const bool in = (unsigned)pg[0] < (unsigned)a.num_pages;   // (the tile has a token)
        if (!in && lane == 0) atomicOr(a.err, PKD_DEV_ERR_BOUNDS);
        const int64_t page = in ? pg[0] : 0;
        const int slot = 16 * tile % P, left = in ? n - 16 * tile : 0;
        const uint8_t* row = a.kv + page * a.page_bytes + (slot + r8) * a.token_bytes + lane_at;
        const int64_t first = (page * a.hkv + h) * P + slot + r8;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bool live = r8 + 8 * i < left;
          slot_at[i] = live ? first + 8 * i : -1;
#pragma unroll
          for (int p = 0; p < kPieces; ++p)
            x.k[i][p] = live ? load_stream(row + 8 * i * a.token_bytes + 64 * p, policy)
                             : make_uint4(0, 0, 0, 0);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int t = 16 * tile + r8 + 8 * i;
          const bool in = t < n && (unsigned)pg[i] < (unsigned)a.num_pages;
          if (t < n && !in) atomicOr(a.err, PKD_DEV_ERR_BOUNDS);
          const int64_t page = in ? pg[i] : 0;
          const int slot = t % P;
          slot_at[i] = in ? (page * a.hkv + h) * P + slot : -1;
          const uint8_t* row = a.kv + page * a.page_bytes + slot * a.token_bytes + lane_at;
#pragma unroll
          for (int p = 0; p < kPieces; ++p)
            x.k[i][p] = in ? load_stream(row + 64 * p, policy) : make_uint4(0, 0, 0, 0);
        }
      }
      x.at = c4 == 0 ? slot_at[0] : c4 == 1 ? slot_at[1] : -1;
      x.old = x.at >= 0 && 16 * tile + r8 + 8 * c4 < fresh ? a.weights[x.at] : 0.f;
    };
    auto finish = [&](int tile, const Tile& x) {
      float c[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        const uint32_t lo[4] = {x.k[0][p].x, x.k[0][p].y, x.k[0][p].z, x.k[0][p].w};
        const uint32_t hi[4] = {x.k[1][p].x, x.k[1][p].y, x.k[1][p].z, x.k[1][p].w};
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          uint32_t af[4];
          if constexpr (kFp8) {
            e4m3x4(lo[s], af[0], af[2]);
            e4m3x4(hi[s], af[1], af[3]);
            mma_f16(c[s & 1], af, qf[p][s][0], qf[p][s][1]);
          } else {
            af[0] = lo[2 * s];
            af[1] = hi[2 * s];
            af[2] = lo[2 * s + 1];
            af[3] = hi[2 * s + 1];
            mma_bf16(c[s & 1], af, qf[p][s][0], qf[p][s][1]);
          }
        }
      }
      // c: (token r8, heads 2 c4, 2 c4 + 1), (token r8 + 8, the same heads)
      float w[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w[i] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float z = fmaf(c[0][2 * i + e] + c[1][2 * i + e], sc[e], -base[e]);
          w[i] += base[e] == CUDART_INF_F ? 0.f : exp2f(z);
        }
        w[i] += __shfl_xor_sync(kFull, w[i], 1);
        w[i] += __shfl_xor_sync(kFull, w[i], 2);
      }
      if (x.at >= 0) {
        const int mine = 16 * tile + r8 + 8 * c4;
        a.weights[x.at] = x.old + (c4 == 0 ? w[0] : w[1]);
        if (a.positions && mine >= fresh) a.positions[x.at] = age0 + mine;
      }
    };
    // Two E4M3 tiles are on their way per warp (a bf16 tile has twice the
    // bytes; two of them do not fit the registers of 24 warps).
    int tile = sub;
    look_up(tile);
    if constexpr (kFp8) {
      Tile x[2];
      if (tile < tiles) {
        fetch(tile, x[0]);
        look_up(tile + per);
      }
      while (tile < tiles) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (tile >= tiles) break;
          if (tile + per < tiles) {
            fetch(tile + per, x[i ^ 1]);
            look_up(tile + 2 * per);
          }
          finish(tile, x[i]);
          tile += per;
        }
      }
    } else {
      for (; tile < tiles; tile += per) {
        Tile x;
        fetch(tile, x);
        look_up(tile + per);
        finish(tile, x);
      }
    }
  }
}

}  // namespace

cudaError_t launch_weights(const WeightsArgs& a, bool fp8, int grid, cudaStream_t stream) {
  const bool tiles = a.page_size % 16 == 0;
  if (fp8)
    (tiles ? weights_kernel<true, true> : weights_kernel<true, false>)<<<grid, kWarps * 32, 0, stream>>>(a);
  else
    (tiles ? weights_kernel<false, true> : weights_kernel<false, false>)<<<grid, kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pkd
