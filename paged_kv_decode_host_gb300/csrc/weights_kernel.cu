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
// SM takes an even share of the 16-token tiles of all requests, laid end to
// end (nothing is merged afterwards, so cutting costs nothing; the planner's
// items, which the decode kernel walks, left a block up to half more than
// the mean beside one long request, and most blocks idle for a few short
// ones); a warp takes 16 tokens of one KV head at a time.  The scores are
// mma.sync m16n8k16 products with the tokens as the 16 rows and the group's
// heads as the 8 columns: K goes from global memory straight into the A
// fragments, with no shared memory and for any layout or page size, because
// the order of the contraction is free -- a lane takes 32 contiguous bytes of
// a row for four (bf16) or eight (E4M3) steps and the queries are permuted
// alike.  (A tcgen05 product would have to stage K in
// shared memory to use 8 of its columns.)
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "evict.h"
#include "pkd_internal.h"
#include "plan_layout.h"
#include "sm103_ptx.cuh"

namespace pkd {
namespace {

using namespace dev;

// Warps of a block: a multiple of 1, 2, 4 and 8 heads (a warp keeps its head),
// each with one 16-token tile under way.  Fewer warps with two to four tiles
// each were no faster for bf16 (16 x 2: 79 against 76 us, 64 requests of up
// to 8,192 tokens) and slower for E4M3 (16 x 3: 37 against 33 us, 64 of
// 2,048); 24 with two E4M3 tiles spill (25 against 20 us, 50,021 tokens and 16
// short requests).
constexpr int kWarps = 24;
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

// 32 bytes that are read once: one load where the cache lies on 32 bytes, so
// that a quad's four lanes ask for one whole 128-byte line, else two.
template <bool kWide>
__device__ __forceinline__ void load_stream(const uint8_t* p, uint32_t* v) {
  if constexpr (kWide) {
    asm volatile("ld.global.nc.L1::no_allocate.L2::evict_first.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                   "=r"(v[6]), "=r"(v[7])
                 : "l"(p));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(v[4 * i]), "=r"(v[4 * i + 1]), "=r"(v[4 * i + 2]), "=r"(v[4 * i + 3])
                   : "l"(p + 16 * i));
  }
}

// four E4M3 bytes to two f16 pairs (exact)
__device__ __forceinline__ void e4m3x4(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b;}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}

__device__ __forceinline__ float exp2_of(float x) {   // relative error 2^-22
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// kTiles: the page size is a multiple of 16, so that a tile lies in one page.
// kWide: the cache lies on a 32-byte boundary.
template <bool kFp8, bool kTiles, bool kWide>
__global__ void __launch_bounds__(kWarps * 32, 1) weights_kernel(const __grid_constant__ WeightsArgs a) {
  // Up to its first request a block reads the schedule alone, beside the end
  // of the kernel before (3 requests of up to 37 tokens 6.2 -> 3.4 us, 50,021
  // E4M3 tokens and 16 short requests 20.4 -> 17.5).  Every way out waits for
  // that kernel, so that this one is complete after it.
  if (!schedule_ready(a.sched + H_EPOCH, a.wait_epoch, a.err)) {
    pdl_wait();
    return;
  }
  constexpr int kPieces = kFp8 ? 1 : 2;      // 32-byte pieces of a row per lane
  constexpr int kSteps = kFp8 ? 8 : 4;       // products fed by a piece, four columns a lane each
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r8 = lane >> 2, c4 = lane & 3;   // row (token, or head of the queries) and quad lane
  const int per = kWarps / a.hkv;            // warps of one head
  const int h = warp % a.hkv, sub = warp / a.hkv;
  if (sub >= per) {                          // 24 is not a multiple of 5 or 7 heads
    pdl_wait();
    return;
  }
  const int g = a.hq / a.hkv;
  const int P = a.page_size, shift = a.page_shift;   // most sizes are powers of two
  auto page_div = [&](int t) { return shift >= 0 ? t >> shift : t / P; };
  auto in_page = [&](int t) { return shift >= 0 ? t & (P - 1) : t % P; };
  // this block's tiles of all requests', end to end: [lo, hi), even shares
  const int batch = a.sched[H_BATCH], nnz = a.sched[H_NNZ];
  if (batch > a.batch) {   // a captured call, under a later plan of more requests
    if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(a.err, PKD_DEV_ERR_BOUNDS);
    pdl_wait();
    return;
  }
  const int4* requests = reinterpret_cast<const int4*>(a.sched + request_words(a.off_pages, nnz));
  const int64_t total = requests[batch].x;
  const int lo = (int)(total * blockIdx.x / gridDim.x), hi = (int)(total * (blockIdx.x + 1) / gridDim.x);
  if (lo >= hi) {
    pdl_wait();
    return;
  }
  // the request that holds tile lo: a lane per candidate, 32 times finer each time
  int req = 0;
  for (int span = batch + 1; span > 1;) {
    const int step = (span + 31) / 32;
    const int before = requests[min(req + lane * step, batch)].x;
    const uint32_t not_past = __ballot_sync(kFull, before <= lo);   // lane 0 always
    req += (31 - __clz(not_past)) * step;
    span = step;
  }
  pdl_wait();   // lse, the cache, sums and positions may be that kernel's
  for (int at = lo; at < hi; ++req) {
    const int4 entry = requests[req];
    const int tiles = min(hi, requests[req + 1].x) - entry.x;   // this block's end, in the request
    const int tile0 = at - entry.x;
    at = entry.x + tiles;
    const int n = entry.z;
    const int32_t* pages = a.sched + a.off_pages + entry.y;
    const int fresh = a.new_tokens ? n - min(max(a.new_tokens[req], 0), n) : n;   // first new token
    const int age0 = a.positions ? a.seen[req] - n : 0;
    // queries of this KV head: lane's row is query head r8, in the pieces'
    // permuted order.  For E4M3 they become f16, scaled by a power of two
    // (exact down to 2^-29 of the head's largest value).
    uint32_t qf[kPieces][kSteps][2];
    float qs = 1.f;
    {
      const uint16_t* qr = a.q + ((int64_t)req * a.hq + h * g + (r8 < g ? r8 : 0)) * kHeadDim;
      // columns of piece p: 16 (bf16) or 32 (E4M3) from 4 times that many p + c4 of them
      constexpr int kCols = kSteps * 4;
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
#pragma unroll
        for (int i = 0; i < kSteps / 2; ++i) {
          const uint4 v = *reinterpret_cast<const uint4*>(qr + 4 * kCols * p + kCols * c4 + 8 * i);
          qf[p][2 * i][0] = r8 < g ? v.x : 0u;
          qf[p][2 * i][1] = r8 < g ? v.y : 0u;
          qf[p][2 * i + 1][0] = r8 < g ? v.z : 0u;
          qf[p][2 * i + 1][1] = r8 < g ? v.w : 0u;
        }
      if constexpr (kFp8) {
        float top = 0.f;
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            top = fmaxf(top, fmaxf(fabsf(bf16_lo(qf[0][s][e])), fabsf(bf16_hi(qf[0][s][e]))));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
        const int ex = top > 0.f && top < CUDART_INF_F ? 14 - ilogbf(top) : 0;
        qs = ldexpf(1.f, ex < 100 ? ex : 100);
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const __half2 x = __floats2half2_rn(bf16_lo(qf[0][s][e]) * qs, bf16_hi(qf[0][s][e]) * qs);
            qf[0][s][e] = *reinterpret_cast<const uint32_t*>(&x);
          }
      }
    }
    // this lane's two columns of the products: heads 2 c4 and 2 c4 + 1
    float sc[2], base[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int j = 2 * c4 + e;
      const float s = __shfl_sync(kFull, qs, 4 * j);   // the scale of that head's queries
      sc[e] = kFp8 ? a.scale_log2 / s : a.scale_log2;
      const float l = j < g ? a.lse[(int64_t)req * a.hq + h * g + j] : 0.f;
      base[e] = l * kLog2e;
      // an empty state (lse -inf) gives its tokens nothing
      if (j >= g || l == -CUDART_INF_F) base[e] = CUDART_INF_F;
    }
    // a tile's pages, looked up a tile before they are used: one with kTiles,
    // else the lane's two tokens'
    int pg[2] = {0, 0};
    auto look_up = [&](int tile) {
      const int t = 16 * tile;
      if constexpr (kTiles) {
        pg[0] = t < n ? pages[page_div(t)] : 0;
      } else {
        pg[0] = t + r8 < n ? pages[page_div(t + r8)] : 0;
        pg[1] = t + r8 + 8 < n ? pages[page_div(t + r8 + 8)] : 0;
      }
    };
    // one tile on its way: K, the lane's own sum (lanes 0 and 1 of a quad own
    // its two tokens), and where that lies
    struct Tile {
      uint32_t k[2][8 * kPieces];
      float old;
      int64_t at;
    };
    const int64_t lane_at = h * a.head_bytes + 32 * c4;
    auto fetch = [&](int tile, Tile& x) {
      int64_t slot_at[2];
      if constexpr (kTiles) {
        const bool in = (unsigned)pg[0] < (unsigned)a.num_pages;   // (the tile has a token)
        if (!in && lane == 0) atomicOr(a.err, PKD_DEV_ERR_BOUNDS);
        const int64_t page = in ? pg[0] : 0;
        const int slot = in_page(16 * tile), left = in ? n - 16 * tile : 0;
        const uint8_t* row = a.kv + page * a.page_bytes + (slot + r8) * a.token_bytes + lane_at;
        const int64_t first = (page * a.hkv + h) * P + slot + r8;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bool live = r8 + 8 * i < left;
          slot_at[i] = live ? first + 8 * i : -1;
#pragma unroll
          for (int p = 0; p < kPieces; ++p) {
#pragma unroll
            for (int w = 0; w < 8; ++w) x.k[i][8 * p + w] = 0u;
            if (live)
              load_stream<kWide>(row + 8 * i * a.token_bytes + 128 * p, &x.k[i][8 * p]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int t = 16 * tile + r8 + 8 * i;
          const bool in = t < n && (unsigned)pg[i] < (unsigned)a.num_pages;
          if (t < n && !in) atomicOr(a.err, PKD_DEV_ERR_BOUNDS);
          const int64_t page = in ? pg[i] : 0;
          const int slot = in_page(t);
          slot_at[i] = in ? (page * a.hkv + h) * P + slot : -1;
          const uint8_t* row = a.kv + page * a.page_bytes + slot * a.token_bytes + lane_at;
#pragma unroll
          for (int p = 0; p < kPieces; ++p) {
#pragma unroll
            for (int w = 0; w < 8; ++w) x.k[i][8 * p + w] = 0u;
            if (in) load_stream<kWide>(row + 128 * p, &x.k[i][8 * p]);
          }
        }
      }
      x.at = c4 == 0 ? slot_at[0] : c4 == 1 ? slot_at[1] : -1;
      x.old = x.at >= 0 && 16 * tile + r8 + 8 * c4 < fresh ? a.weights[x.at] : 0.f;
    };
    auto finish = [&](int tile, const Tile& x) {
      float c[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        const uint32_t* lo = &x.k[0][8 * p];
        const uint32_t* hi = &x.k[1][8 * p];
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
          w[i] += base[e] == CUDART_INF_F ? 0.f : exp2_of(z);
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
    look_up(tile0 + sub);
    for (int tile = tile0 + sub; tile < tiles; tile += per) {
      Tile x;
      fetch(tile, x);
      look_up(tile + per);
      finish(tile, x);
    }
  }
}

}  // namespace

cudaError_t launch_weights(const WeightsArgs& a, bool fp8, int grid, cudaStream_t stream) {
  const bool tiles = a.page_size % 16 == 0, wide = (uintptr_t)a.kv % 32 == 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaSuccess;
  auto go = [&](auto f) { e = cudaLaunchKernelEx(&cfg, f, a); };
  if (fp8) {
    if (tiles)
      wide ? go(weights_kernel<true, true, true>) : go(weights_kernel<true, true, false>);
    else
      wide ? go(weights_kernel<true, false, true>) : go(weights_kernel<true, false, false>);
  } else {
    if (tiles)
      wide ? go(weights_kernel<false, true, true>) : go(weights_kernel<false, true, false>);
    else
      wide ? go(weights_kernel<false, false, true>) : go(weights_kernel<false, false, false>);
  }
  return e;
}

}  // namespace pkd
