// Decode attention over a paged cache of latent vectors (contexts with
// PKD_FLAG_LATENT), the merge of its split requests, and the append of new
// latent rows, for sm_103a.
//
// The cache holds one row per token, shared by every query head: kLatentDim
// latent columns and kLatentRope columns of the rotary key.  With the
// up-projections absorbed into the queries and the output projection, head h
// of request i computes
//     s_t   = scale * q[i][h] . c_t                 (all 576 columns)
//     out   = sum_t softmax(s)_t * c_t[0 .. 511]    (the latent columns)
// so one read of a row serves as key and value of up to 128 heads: 4 * 544
// flop per head and 1,152 bytes per token.
//
// GB300 design: one CTA per SM walks its queue of (request, 64-head block,
// token range) items from the planner's schedule.  Both products put the
// long axis on the tensor core's 128 rows and the heads on its columns, so a
// CTA's tensor-memory use follows the number of heads (the transposed
// orientation would need all 512 columns for the 512-wide output alone) and
// short head counts cost narrow instructions:
//     S^T [tokens x heads]  = C [tokens x 576]  Q^T    A = C, B = Q, K-major
//     O^T [dims x heads]   += C^T [dims x tokens] P^T  A = C, B = P, MN-major
// The same shared-memory tile of C feeds both: blocks of 8 tokens x 64 columns
// (1 KB, 128-byte swizzle), the 9 column chunks in two regions: 4-8 (with the
// rotary key) and 0-3.  (Four regions shorten the wait for the last scores but
// lengthen the producer's way more: 78 -> 79 us for 128 heads.)
//  * a warp streams C: one TMA tensor copy per region and 16 tokens (10 and 8
//    KB; a 5-D map of the cache gives the blocked order, so page tiles join
//    to one operand however the pages are scattered; 36 copies of 2 KB a tile
//    were bound by their issue, about 110 cycles a copy);
//  * one issues the score products of a region as it lands, one the P.V
//    products, whose regions are refilled one after the other; the whole warp
//    runs the loop and one elected lane issues, with unrolled constant
//    descriptor steps: 29 / 38 cycles per 64 x 16 / 64 x 64 product and 45 /
//    54 with 128 rows, where a lone thread that forms descriptors in the loop
//    takes 135 for any;
//  * warps 0-7 (0-15 from 32 heads on) are the softmax: a thread holds one
//    token and 4 or 8 of the block's heads.  The maxima run over tokens, that
//    is, across lanes and warps, so they are not formed per tile: every tile
//    is only compared with the running base, and the exact maxima are taken
//    when some score exceeds its head's base by more than 2^8 (always in an
//    item's first tile), from the scores read again.  P is written as bf16,
//    for up to 32 heads with the rounding's rest beside it, into shared
//    memory; the sums that divide it are kept unrounded in fp32.
// Every wait is bounded; on timeout the kernel sets the device error word,
// stops, waits (bounded) for its copies and products, frees tensor memory
// and returns.
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "latent.h"
#include "pkd_internal.h"
#include "prefix_tc_body.cuh"
#include "sm103_ptx.cuh"
#include "tensor_map.h"

namespace pkd {
namespace {

using namespace dev;
using tc::fast_exp2;
using tc::mma_commit;
using tc::mma_ss;
using tc::pack_bf16;
using tc::smem_desc;
using tc::tc_fence_after;
using tc::tc_fence_before;
using tc::tc_wait;

constexpr int kChunks = kLatentRow / 64;        // 9 column chunks: 8 latent, 1 rotary
constexpr int kPairs = kLatentDim / 128;        // 4 O^T products of 128 dims
constexpr int kRegions = 2;
// first chunk and chunks of a region; the products (128 dims) whose values it
// holds
__host__ __device__ constexpr int region_first(int g) { return g == 0 ? 4 : 0; }
__host__ __device__ constexpr int region_chunks(int g) { return g == 0 ? 5 : 4; }
constexpr int kRegionPairs = kPairs / kRegions;
constexpr float kRaiseLog2 = 8.f;
constexpr float kLowest = -3.0e38f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994530942f;

// Tokens of a tile: the 64 rows of a score product.  (128-row products take
// 45 to 54 cycles against 28 to 38, and two tiles of 128 tokens do not fit
// shared memory beside the queries.)
constexpr int kTile = 64, kBoxes = kTile / 16;
static_assert(32 % kBoxes == 0, "a warp's 32 page ids are whole tiles'");
constexpr int kStages = 2;
// 8 tokens of a region: the stride of the products' 8-row groups
__host__ __device__ constexpr int group_bytes(int g) { return region_chunks(g) * 1024; }
__host__ __device__ constexpr int region_at(int g) { return g == 0 ? 0 : kTile / 8 * group_bytes(0); }
constexpr int kStage = kTile / 8 * kChunks * 1024;
constexpr int kP = kTile * 128;   // [token][64 heads] bf16, 128-byte rows

// NH: heads (instruction columns) of a block.
template <int NH_>
struct LatentShape {
  static constexpr int NH = NH_;
  // Softmax teams of four warps (a warp per 16 tokens), a team's heads and a
  // thread's (half a warp each); the warps behind them load, score and
  // multiply.  Four teams where a thread keeps four heads or more: the softmax
  // is part of a 64-head tile's round (128 heads, 32 requests: 77.9 -> 72.6 us;
  // 32 heads, 64 requests of 2,000 tokens: 38.2 -> 37.2).
  static constexpr int kTeams = NH >= 32 ? 4 : 2, HH = NH / kTeams, QH = HH / 2;
  static constexpr int kSoft = 4 * kTeams;
  static constexpr int kLoad = kSoft, kScore = kSoft + 1, kOut = kSoft + 2;
  static constexpr int kThreads = (kSoft + 3) * 32;
  static constexpr int kQChunk = NH * 128;
  static constexpr int kQ = kChunks * kQChunk;
  // P is kept as two bf16 values, the rounded weight and what the rounding
  // left (16 bits in all), where that is free: their products share the
  // instruction, as columns h and NH + h, and 32 columns take the time of 16,
  // 64 of 32 nearly so (45, 46 and 54 cycles).  For 64 heads the second half
  // fits neither tensor memory nor shared memory: there P is one bf16, and a
  // result's error that of two roundings instead of one.
  static constexpr bool kSplit = NH <= 32;
  static constexpr int NP = kSplit ? 2 * NH : NH;   // columns of an O^T product
  // A tile's copies leave when the products of the tile two before are done,
  // and the way from there to its scores is the longest part of a 64-head
  // tile's round.  Where two blocks of heads read the same rows, fetching them
  // into L2 a tile earlier pays (128 heads, 32 requests: 75.5 -> 71.4 us); one
  // block is nearer HBM's rate, which the extra requests disturb (64 heads, 32
  // requests: 46.3 -> 47.7; 16 heads, 64 requests: 50 -> 53; but 40 heads,
  // 100,003 tokens: 34.2 -> 33.8).
  static constexpr bool kPrefetch = NH == 64;
  // What a round of products of one CTA cannot go below is the shared memory's
  // rate: they read their operands at about 110 bytes a cycle (of 128), 147 KB
  // for a 64-head tile's scores and 98 KB for its P.V, beside 74 KB of copies:
  // 2,550 cycles of some 3,250.
  static constexpr uint32_t kColO = 0, kColS = kPairs * NP;
  static_assert(NH % 16 == 0 && NH <= 64 && kColS + 2 * NH <= 512, "shape");
};

template <class C>
struct LatentSmem {
  uint64_t full[kStages][kRegions];    // region landed
  uint64_t empty[kStages][kRegions];   // its P.V products done
  uint64_t qfull, qfree;
  uint64_t sfull[2], sfree[2];
  uint64_t pfull, pvdone, ofree;
  uint64_t xch[C::kTeams];           // a team's four warps' exchanges
  uint64_t fin;
  uint32_t tmem_base;
  int abort_flag;
  int raise[2][C::kTeams][4];                      // [phase parity][team][quadrant]
  float top[2][C::kTeams][4][C::HH];               // column maxima / sums, likewise
};

template <class C>
constexpr int latent_smem() {
  return kStages * kStage + C::kQ + kP + (int)sizeof(LatentSmem<C>);
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ uint64_t l2_evict_normal_policy() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// 4-D tensor-map copy global -> shared, as tensor_copy_g2s.
__device__ __forceinline__ void tensor_copy4_g2s(void* dst, const CUtensorMap* map, int c0, int c1,
                                                 int c2, int c3, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar)),
      "l"(policy)
      : "memory");
}

// A 64-row product keeps row 16 q + i in lane 32 q + i, i < 16.  Lanes 0-15
// of the warp get N columns of the quadrant's 16 rows from column t on, lanes
// 16-31 the same rows' N columns from t + N on.
template <int N>
__device__ __forceinline__ void tmem_ld_rows16(uint32_t t, uint32_t (&r)[N]) {
  static_assert(N == 4 || N == 8 || N == 16, "columns");
  if constexpr (N == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15}, [%16], 16;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(t)
        : "memory");
  } else if constexpr (N == 8) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8], 8;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(t)
        : "memory");
  } else {
    asm volatile("tcgen05.ld.sync.aligned.16x32bx2.x4.b32 {%0,%1,%2,%3}, [%4], 4;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(t)
                 : "memory");
  }
}

// The same box of a 5-D map (first two coordinates 0) into L2 only.
__device__ __forceinline__ void tensor_prefetch(const CUtensorMap* map, int c2, int c3, int c4) {
  asm volatile("cp.async.bulk.prefetch.tensor.5d.L2.global.tile [%0, {%1, %1, %2, %3, %4}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(0), "r"(c2), "r"(c3), "r"(c4)
               : "memory");
}

// N columns of this warp's 32 lanes
template <int N>
__device__ __forceinline__ void tmem_ldn(uint32_t t, uint32_t (&r)[N]) {
  static_assert(N == 8 || N == 16 || N == 32, "columns");
  if constexpr (N == 32) {
    tc::tmem_ld32(t, r);
  } else if constexpr (N == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(t)
        : "memory");
  } else {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "r"(t)
                 : "memory");
  }
}
template <int N>
__device__ __forceinline__ void tmem_stn(uint32_t t, const uint32_t (&r)[N]) {
  if constexpr (N == 32) {
    tc::tmem_st32(t, r);
  } else if constexpr (N == 16) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
        "%13,%14,%15,%16};" ::"r"(t),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
  } else {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                 "r"(r[7])
                 : "memory");
  }
}

// Column-wise reduction over 16 lanes (both halves of the warp at once) of N
// <= 16 values per lane: a butterfly that halves the columns a lane still
// holds with every exchange (N - 1 shuffles and the rest of the log; a
// reduction per column would take 4 N).  Lane j (mod N) of a half returns its
// column j.
template <int N, class Op>
__device__ __forceinline__ float columns_over_lanes(const float (&x)[N], int lane, Op op) {
  float v[N];
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = x[j];
#pragma unroll
  for (int w = N / 2; w >= 1; w >>= 1) {   // lanes with bit w keep the upper w columns
    const bool upper = (lane & w) != 0;
#pragma unroll
    for (int j = 0; j < w; ++j) {
      const float send = upper ? v[j] : v[j + w];
      const float keep = upper ? v[j + w] : v[j];
      v[j] = op(keep, __shfl_xor_sync(kFull, send, w));
    }
  }
#pragma unroll
  for (int w = N; w < 16; w <<= 1) v[0] = op(v[0], __shfl_xor_sync(kFull, v[0], w));
  return v[0];
}
// the larger, NaN above all
__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

struct LatentItem {
  int req, tb, te, dst, page0, block;
};
__device__ __forceinline__ LatentItem item_at(const LatentArgs& a, int it) {
  const int4* w = reinterpret_cast<const int4*>(a.sched + a.off_items + (int64_t)it * kItemWords);
  const int4 x = w[0], y = w[1];
  auto same = [](int v) { return __shfl_sync(kFull, v, 0); };
  return LatentItem{same(x.x), same(x.y), same(x.z), same(x.w), same(y.x), same(y.w)};
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1)
    latent_decode_kernel(const __grid_constant__ LatentArgs a) {
  extern __shared__ __align__(1024) uint8_t sC[];   // the swizzle repeats every 1024 bytes
  if (!schedule_ready(a.sched + H_EPOCH, a.wait_epoch, a.err)) return;
  if ((smem_u32(sC) & 1023u) != 0) {   // the compiler's alignment was not honoured
    if (threadIdx.x == 0) atomicOr(a.err, PKD_DEV_ERR_BOUNDS);
    pdl_wait();
    return;
  }
  uint8_t* sQ = sC + kStages * kStage;
  uint8_t* sP = sQ + C::kQ;
  LatentSmem<C>* sh = reinterpret_cast<LatentSmem<C>*>(sP + kP);
  volatile int* abort_flag = &sh->abort_flag;
  // (shuffled from lane 0 so that the compiler knows these as the same in the
  // whole warp: the issuing loops then keep their descriptors in uniform
  // registers)
  const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  pdl_launch_dependents();
  const int it0 = __shfl_sync(kFull, a.sched[a.off_cta + blockIdx.x], 0);
  const int it1 = __shfl_sync(kFull, a.sched[a.off_cta + blockIdx.x + 1], 0);
  // a captured call, under a later plan of more requests than q and out have
  const bool outgrown = __shfl_sync(kFull, a.sched[H_BATCH], 0) > a.batch;
  if (it0 >= it1 || outgrown) {
    if (outgrown && threadIdx.x == 0 && blockIdx.x == 0) atomicOr(a.err, PKD_DEV_ERR_BOUNDS);
    pdl_wait();
    return;
  }
  if (warp == C::kLoad && lane < 3) {   // the first copies would wait for their maps
    const CUtensorMap* map = lane < 2 ? &a.kv_map[lane] : &a.q_map;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s)
      for (int g = 0; g < kRegions; ++g) {
        mbar_init(&sh->full[s][g], 1);
        mbar_init(&sh->empty[s][g], 1);
      }
    mbar_init(&sh->qfull, 1);
    mbar_init(&sh->qfree, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh->sfull[b], 1);
      mbar_init(&sh->sfree[b], C::kSoft);
    }
    for (int b = 0; b < C::kTeams; ++b) mbar_init(&sh->xch[b], 4);
    mbar_init(&sh->pfull, C::kSoft);
    mbar_init(&sh->pvdone, 1);
    mbar_init(&sh->ofree, C::kSoft);
    mbar_init(&sh->fin, 2);
    sh->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sh->tmem_base)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // the producer's first item and its page ids, on their way while the block
  // sets itself up
  LatentItem item0{};
  int page_a = 0, page_b = 0;
  if (warp == C::kLoad) {
    item0 = item_at(a, it0);
    const int boxes = (item0.te - item0.tb + 15) >> 4;
    const int32_t* pages = a.sched + a.off_pages + item0.page0;
    if (lane < boxes) page_a = pages[16 * lane / a.page_size];
    if (32 + lane < boxes) page_b = pages[16 * (32 + lane) / a.page_size];
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(kFull, sh->tmem_base, 0);

  if (warp == C::kLoad) {
    // ------------------------------------------------------------ producer
    // q and the cache are read before the previous kernel is waited for, as
    // the decode kernel does (the contract of pkd_run)
    // a second block of heads reads the rows from L2
    const uint64_t policy = a.blocks > 1 ? l2_evict_normal_policy() : l2_evict_first_policy();
    const int P = a.page_size;
    int r = 0, nq = 0;
    int extra = 0;   // regions issued of a tile that a timeout cut short
    bool ok = true;
    for (int it = it0; it < it1 && ok; ++it) {
      const LatentItem w = it == it0 ? item0 : item_at(a, it);
      if (it > it0 && !tc_wait(&sh->qfree, (uint32_t)((it - it0 - 1) & 1), abort_flag, a.err, lane)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        ++nq;
        mbar_arrive_expect_tx(&sh->qfull, (uint32_t)C::kQ);
        tensor_copy4_g2s(sQ, &a.q_map, 0, C::NH * w.block, 0, w.req, &sh->qfull, policy);
      }
      __syncwarp();
      // page ids of 32 consecutive 16-token boxes, one per lane (items start
      // on page boundaries); the next 32 are fetched while these are copied
      const int boxes = (w.te - w.tb + 15) >> 4;
      const int32_t* pages = a.sched + a.off_pages + w.page0;
      auto page_of = [&](int box) { return box < boxes ? pages[16 * box / P] : 0; };
      int base = 0, my_page = page_a, next_page = page_b;
      if (it > it0) {
        my_page = page_of(lane);
        next_page = page_of(32 + lane);
      }
      for (int t = w.tb, k = 0; t < w.te; t += kTile, ++k, ++r) {
        const int nbox = min(kBoxes, (w.te - t + 15) >> 4);
        const int st = r % kStages;
        const uint32_t use = (uint32_t)(r / kStages);
        // lane j copies box j of the tile; a tile's boxes, and the next
        // tile's once the window has moved on, lie in one window of 32
        int page = __shfl_sync(kFull, my_page, (kBoxes * k + lane % kBoxes) & 31);
        if (kBoxes * (k + 1) >= base + 32) {
          base += 32;
          my_page = next_page;
          next_page = page_of(base + 32 + lane);
        }
        if ((unsigned)page >= (unsigned)a.num_pages) {
          atomicOr(a.err, PKD_DEV_ERR_BOUNDS);
          page = 0;
        }
        const int tok = (t + 16 * lane) % P;
#pragma unroll
        for (int g = 0; g < kRegions; ++g) {
          if (ok && use > 0 && !tc_wait(&sh->empty[st][g], (use - 1) & 1u, abort_flag, a.err, lane))
            ok = false;
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&sh->full[st][g], (uint32_t)(nbox * 2 * group_bytes(g)));
          __syncwarp();
          if (lane < nbox)
            tensor_copy_g2s(sC + st * kStage + region_at(g) + lane * 2 * group_bytes(g),
                            &a.kv_map[g], 0, 0, region_first(g), tok / 8, page, &sh->full[st][g],
                            policy);
          ++extra;
        }
        if (!ok) break;
        extra = 0;
        if (C::kPrefetch && a.blocks > 1) {
          // the next tile into L2 while its slots are in use (a lane per box
          // and region)
          const int next = kBoxes * (k + 1) + lane % kBoxes, g = lane / kBoxes;
          const int np = __shfl_sync(kFull, my_page, next & 31);
          if (g < kRegions && next < boxes && (unsigned)np < (unsigned)a.num_pages)
            tensor_prefetch(&a.kv_map[g], region_first(g), (t + kTile + 16 * (lane % kBoxes)) % P / 8,
                            np);
        }
      }
    }
    // drain: no copy may be in flight when the block ends.  Region g of stage
    // s was copied once per whole tile of the stage, and once more when it
    // was among the first of a tile cut short.
    if (lane == 0) {
      for (int s = 0; s < kStages; ++s)
        for (int g = 0; g < kRegions; ++g) {
          int uses = r > s ? (r - 1 - s) / kStages + 1 : 0;
          if (s == r % kStages && g < extra) ++uses;
          if (uses > 0 && !mbar_wait(&sh->full[s][g], (uint32_t)((uses - 1) & 1), nullptr))
            atomicOr(a.err, PKD_DEV_ERR_TIMEOUT);
        }
      if (nq > 0 && !mbar_wait(&sh->qfull, (uint32_t)((nq - 1) & 1), nullptr))
        atomicOr(a.err, PKD_DEV_ERR_TIMEOUT);
    }
    __syncwarp();
  } else if (warp == C::kScore) {
    // -------------------------------------------------------- S^T products
    const bool me = elect_one();
    const uint32_t idesc = tc::mma_idesc(kTile, C::NH, 0);
    uint64_t c0[kRegions];
#pragma unroll
    for (int g = 0; g < kRegions; ++g)
      c0[g] = smem_desc(smem_u32(sC) + region_at(g), 16, group_bytes(g));
    const uint64_t q0 = smem_desc(smem_u32(sQ), 16, 1024);
    int r = 0;
    bool ok = true;
    for (int it = it0; it < it1 && ok; ++it) {
      const LatentItem w = item_at(a, it);
      if (!tc_wait(&sh->qfull, (uint32_t)((it - it0) & 1), abort_flag, a.err, lane)) break;
      for (int t = w.tb; t < w.te && ok; t += kTile, ++r) {
        const int st = r % kStages, b = r & 1;
        const uint32_t use = (uint32_t)(r / kStages);
        if (r >= 2 && !tc_wait(&sh->sfree[b], (uint32_t)(((r >> 1) - 1) & 1), abort_flag, a.err, lane)) {
          ok = false;
          break;
        }
        const uint32_t d = tmem + C::kColS + C::NH * b;
#pragma unroll
        for (int g = 0; g < kRegions; ++g) {
          if (ok && !tc_wait(&sh->full[st][g], use & 1u, abort_flag, a.err, lane)) ok = false;
          if (ok && me) {
            tc_fence_after();
            const uint64_t cs = c0[g] + (uint64_t)(st * (kStage >> 4));
            const uint64_t qs = q0 + (uint64_t)(region_first(g) * (C::kQChunk >> 4));
#pragma unroll
            for (int i = 0; i < region_chunks(g); ++i)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_ss(d, cs + (uint64_t)(64 * i + 2 * kk),
                       qs + (uint64_t)(i * (C::kQChunk >> 4) + 2 * kk), idesc,
                       g > 0 || i > 0 || kk > 0);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (me) {
          mma_commit(&sh->sfull[b]);
          if (t + kTile >= w.te) mma_commit(&sh->qfree);
        }
        __syncwarp();
      }
    }
    if (me) {
      mma_commit(&sh->fin);
      if (!mbar_wait(&sh->fin, 0, nullptr)) atomicOr(a.err, PKD_DEV_ERR_TIMEOUT);
    }
    __syncwarp();
  } else if (warp == C::kOut) {
    // -------------------------------------------------------- O^T products
    const bool me = elect_one();
    const uint32_t idesc = tc::mma_idesc(128, C::NP, 1) | (1u << 15);   // A and B MN-major
    uint64_t c0[kRegions];   // 64-dim blocks 1 KB apart, 8-token groups a group apart
#pragma unroll
    for (int g = 0; g < kRegions; ++g)
      c0[g] = smem_desc(smem_u32(sC) + region_at(g), 1024, group_bytes(g));
    const uint64_t p0 = smem_desc(smem_u32(sP), 16, 1024);
    int r = 0;
    bool ok = true;
    for (int it = it0; it < it1 && ok; ++it) {
      const LatentItem w = item_at(a, it);
      for (int t = w.tb; t < w.te; t += kTile, ++r) {
        const int st = r % kStages;
        if (!tc_wait(&sh->pfull, (uint32_t)(r & 1), abort_flag, a.err, lane) ||
            (t == w.tb && it > it0 &&
             !tc_wait(&sh->ofree, (uint32_t)((it - it0 - 1) & 1), abort_flag, a.err, lane))) {
          ok = false;
          break;
        }
        const int n = min(kTile, w.te - t);
        const int nbox = (n + 15) >> 4;
        if (n & 15) {
          // rows past the last token: their P is 0, but 0 x NaN would stay
          const int rows = 16 * nbox - n;
          for (int i = lane; i < 2 * kPairs * rows * 8; i += 32) {
            const int c = i / (rows * 8), rem = i % (rows * 8), row = n + rem / 8;
            const int g = c >= region_first(0) ? 0 : 1;
            *reinterpret_cast<uint4*>(sC + st * kStage + region_at(g) + (row >> 3) * group_bytes(g) +
                                      (c - region_first(g)) * 1024 + (row & 7) * 128 +
                                      (rem % 8) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (me) {
          tc_fence_after();
#pragma unroll
          for (int g = 0; g < kRegions; ++g) {
            const uint64_t cs = c0[g] + (uint64_t)(st * (kStage >> 4));
#pragma unroll
            for (int p = 0; p < kRegionPairs; ++p)
#pragma unroll
              for (int kk = 0; kk < kBoxes; ++kk)
                if (kk < nbox)
                  mma_ss(tmem + C::kColO + C::NP * (region_first(g) / 2 + p),
                         cs + (uint64_t)(128 * p + kk * (group_bytes(g) >> 3)),
                         p0 + (uint64_t)(128 * kk), idesc, t > w.tb || kk > 0);
            mma_commit(&sh->empty[st][g]);
          }
          mma_commit(&sh->pvdone);
        }
        __syncwarp();
      }
    }
    if (me) {
      mma_commit(&sh->fin);
      if (!mbar_wait(&sh->fin, 0, nullptr)) atomicOr(a.err, PKD_DEV_ERR_TIMEOUT);
    }
    __syncwarp();
  } else {
    // -------------------------------------------------- softmax + epilogue
    constexpr int HH = C::HH, QH = C::QH;
    const int quad = warp & 3, team = warp >> 2;
    // scores: this thread's token of the tile and its heads of the team
    const int row = 16 * quad + (lane & 15), hq = (lane >> 4) * QH;
    const uint32_t tq = tmem + ((uint32_t)(32 * quad) << 16);   // this quadrant's lanes
    // the column that a column-wise reduction leaves here, and whether this
    // lane speaks for it
    const int col = hq + (lane & (QH - 1));
    const bool speaks = (lane & 15) < QH;
    uint32_t xc = 0;                                            // exchanges so far
    int r = 0;
    bool ok = true, waited = false;
    // the four warps of this team meet (bounded): what each wrote into the
    // exchange arrays of this phase's parity is visible to all afterwards;
    // the other parity's arrays may be rewritten from here on
    auto meet = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->xch[team]);
      if (!tc_wait(&sh->xch[team], xc & 1u, abort_flag, a.err, lane)) return false;
      ++xc;
      return true;
    };
    for (int it = it0; it < it1 && ok; ++it) {
      const LatentItem w = item_at(a, it);
      // l: this token's sums.  base: lane j holds the base (log2 units) of the
      // team's head j; every warp keeps its own copy
      float l[QH], m[QH], base = 0.f;   // m: the bases of this thread's heads
#pragma unroll
      for (int j = 0; j < QH; ++j) l[j] = m[j] = 0.f;
      for (int t = w.tb; t < w.te && ok; t += kTile, ++r) {
        const int b = r & 1;
        // P of the tile before has been read (its buffer is written below,
        // and a raised base rescales O): long so when the scores arrive
        if ((r > 0 && !tc_wait(&sh->pvdone, (uint32_t)((r - 1) & 1), abort_flag, a.err, lane)) ||
            !tc_wait(&sh->sfull[b], (uint32_t)((r >> 1) & 1), abort_flag, a.err, lane)) {
          ok = false;
          break;
        }
        const bool first = t == w.tb;
        const bool live = row < w.te - t;
        tc_fence_after();
        float y[QH];   // scores over the base (log2 units)
        auto read_scores = [&](bool over_base) {
          uint32_t sv[QH];
          tmem_ld_rows16<QH>(tq + C::kColS + C::NH * b + HH * team, sv);
          tc::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < QH; ++j)
            y[j] = live ? fmaf(__uint_as_float(sv[j]), a.scale_log2, over_base ? -m[j] : 0.f)
                        : -CUDART_INF_F;
        };
        read_scores(true);   // (an item's first tile: over 0)
        float over = -CUDART_INF_F;
#pragma unroll
        for (int j = 0; j < QH; ++j) over = fmaxf(over, y[j]);
        // the four warps of this team agree whether to raise their bases; an
        // item's first tile always does, and brings its maxima along
        const int par = (int)(xc & 1u);
        if (first) {
          const float top = columns_over_lanes<QH>(y, lane, max_nan);
          if (speaks) sh->top[par][team][quad][col] = top;
        } else {
          const bool want = __any_sync(kFull, over > kRaiseLog2);
          if (lane == 0) sh->raise[par][team][quad] = want ? 1 : 0;
        }
        if (!meet()) {
          ok = false;
          break;
        }
        const bool up = first || (sh->raise[par][team][0] | sh->raise[par][team][1] |
                                  sh->raise[par][team][2] | sh->raise[par][team][3]) != 0;
        if (up) {
          int at = par;
          if (!first) {
            at = (int)(xc & 1u);
            // maxima of the scores themselves: over a base that lies far
            // below, as after tiles of masked tokens, they are rounded away
            read_scores(false);
            const float top = columns_over_lanes<QH>(y, lane, max_nan);
            if (speaks) sh->top[at][team][quad][col] = top;
            if (!meet()) {
              ok = false;
              break;
            }
          }
          // the new bases, and how far they rise.  A base stays finite, so that
          // scores of -inf weigh 0 (not -inf - -inf).  A lane per head, then
          // all read.
          float rise = 0.f;
          if (lane < HH) {
            const float top = max_nan(max_nan(sh->top[at][team][0][lane], sh->top[at][team][1][lane]),
                                      max_nan(sh->top[at][team][2][lane], sh->top[at][team][3][lane]));
            const float raised = max_nan(top, first ? kLowest : base);
            rise = raised - base;
            base = raised;
          }
          __syncwarp();
          if (!first) {
            // O shrinks by 2^-rise
            tc_fence_after();
            constexpr int kPart = HH < 16 ? HH : 16;   // columns at a time: the registers
#pragma unroll
            for (int p = 0; p < kPairs * (C::kSplit ? 2 : 1); ++p)
#pragma unroll
              for (int c = 0; c < HH; c += kPart) {
                uint32_t o[kPart];
                const uint32_t at_o = tq + C::kColO + C::NH * p + HH * team + c;
                tmem_ldn<kPart>(at_o, o);
                tc::tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < kPart; ++j)
                  o[j] = __float_as_uint(__uint_as_float(o[j]) *
                                         exp2f(-__shfl_sync(kFull, rise, c + j)));
                tmem_stn<kPart>(at_o, o);
              }
            tc::tmem_wait_st();
          }
#pragma unroll
          for (int j = 0; j < QH; ++j) {
            const float now = __shfl_sync(kFull, base, hq + j);
            if (!first) l[j] *= exp2f(m[j] - now);
            m[j] = now;
            y[j] -= now;
          }
        }
        // weights 2^y; this thread's part of a row of P, 16-byte pieces of 8
        // heads swizzled as the products read them
        uint32_t pw[QH / 2], pl[QH / 2];
#pragma unroll
        for (int j = 0; j < QH; j += 2) {
          const float p0 = fast_exp2(y[j]);   // 0 past the last token
          const float p1 = fast_exp2(y[j + 1]);
          l[j] += p0;
          l[j + 1] += p1;
          const uint32_t hi = pack_bf16(p0, p1);
          pw[j / 2] = hi;
          pl[j / 2] = pack_bf16(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xffff0000u));
        }
        const int h8 = HH * team + hq;   // the block's head, a multiple of QH
        uint8_t* prow = sP + row * 128;
        auto put = [&](int h, const uint32_t (&w)[QH / 2]) {
          if constexpr (QH == 4) {
            *reinterpret_cast<uint2*>(prow + (((h >> 3) ^ (row & 7)) << 4) + (h & 4) * 2) =
                make_uint2(w[0], w[1]);
          } else {
#pragma unroll
            for (int i = 0; i < QH / 8; ++i)
              *reinterpret_cast<uint4*>(prow + ((((h >> 3) + i) ^ (row & 7)) << 4)) =
                  make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          }
        };
        put(h8, pw);
        if constexpr (C::kSplit) put(C::NH + h8, pl);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh->pfull);
          // (the scores of the tile after next wait for this tile's P.V anyway)
          mbar_arrive(&sh->sfree[b]);
        }
      }
      if (!ok) break;
      // ---- epilogue: sums over the tokens in a fixed order
      const int par = (int)(xc & 1u);
      {
        const float z = columns_over_lanes<QH>(l, lane, [](float x, float y) { return x + y; });
        if (speaks) sh->top[par][team][quad][col] = z;
      }
      if (!meet() || !tc_wait(&sh->pvdone, (uint32_t)((r - 1) & 1), abort_flag, a.err, lane)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (!waited) {
        pdl_wait();   // outputs and partial states may be in use by the previous kernel
        waited = true;
      }
      const int h0 = C::NH * w.block + HH * team;
      float inv_mine = 0.f;
      if (lane < HH) {
        const float z = (sh->top[par][team][0][lane] + sh->top[par][team][1][lane]) +
                        (sh->top[par][team][2][lane] + sh->top[par][team][3][lane]);
        inv_mine = z == 0.f ? 0.f : a.v_scale / z;   // 0: every score -inf, an empty state
        if (quad == 0 && h0 + lane < a.heads) {
          const float lse = (base + log2f(z)) * kLn2;
          if (w.dst >= 0)
            a.l_part[(int64_t)w.dst * a.heads + h0 + lane] = lse;
          else if (a.lse != nullptr)
            a.lse[(int64_t)w.req * a.heads + h0 + lane] = lse;
        }
      }
      __syncwarp();
      float inv[HH];
#pragma unroll
      for (int j = 0; j < HH; ++j) inv[j] = __shfl_sync(kFull, inv_mine, j);
#pragma unroll
      for (int p = 0; p < kPairs; ++p) {
        uint32_t o[HH];
        tmem_ldn<HH>(tq + C::kColO + C::NP * p + HH * team, o);
        if constexpr (C::kSplit) {
          uint32_t o2[HH];
          tmem_ldn<HH>(tq + C::kColO + C::NP * p + C::NH + HH * team, o2);
          tc::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < HH; ++j)
            o[j] = __float_as_uint(__uint_as_float(o[j]) + __uint_as_float(o2[j]));
        } else {
          tc::tmem_wait_ld();
        }
        const int dim = 128 * p + 32 * quad + lane;
        if (w.dst >= 0) {
          float* to = a.o_part + ((int64_t)w.dst * a.heads + h0) * kLatentDim + dim;
#pragma unroll
          for (int j = 0; j < HH; ++j)
            if (h0 + j < a.heads) to[(int64_t)j * kLatentDim] = __uint_as_float(o[j]) * inv[j];
        } else {
          uint16_t* to = a.out + ((int64_t)w.req * a.heads + h0) * kLatentDim + dim;
#pragma unroll
          for (int j = 0; j < HH; ++j)
            if (h0 + j < a.heads)
              to[(int64_t)j * kLatentDim] =
                  (uint16_t)(pack_bf16(__uint_as_float(o[j]) * inv[j], 0.f) & 0xffffu);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->ofree);
    }
    if (!waited) pdl_wait();
  }
  pdl_wait();   // complete only after the previous kernel
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
}

// Merge of split requests: out = sum_i w_i o_i / sum_i w_i, w_i = exp(L_i -
// max L), over a request's partial states.  A task is 128 dims of one
// (request, head); a lane holds four of them, so a slot is one 512-byte read
// of a warp.  Up to 8 warps share a task (one reads a task's few slots in one
// round trip; a long request's 150 would take it twenty): warp w takes slots w, w + warps, ... eight loads at
// a time, and the warps' sums are added in warp order.
constexpr int kMergeDims = 128, kMergeWarps = 8, kMergeParts = kLatentDim / kMergeDims;
// Warps per task: one per eight slots of the longest request (up to 8) while
// all of them find room at once (three blocks to an SM).  Eight for every
// request of more than 8 slots ran in two waves where tasks are many: 20
// against 11 us (8 requests of 2,000 tokens, 64 heads, 16 slots each).
__host__ __device__ constexpr int merge_team(int most_slots, int64_t tasks) {
  int team = 1;
  while (team < kMergeWarps && most_slots > 8 * team && tasks * team * 2 <= 152 * 3 * kMergeWarps)
    team *= 2;
  return team;
}
template <int kTeam>
__device__ __forceinline__ void merge_tasks(const LatentArgs& a, int units,
                                            float4 (&acc_s)[kMergeWarps][32],
                                            float (&z_s)[kMergeWarps]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kTeams = kMergeWarps / kTeam;
  const int sub = warp % kTeam;
  const int64_t tasks = (int64_t)units * a.heads * kMergeParts;
  bool waited = false;
  for (int64_t t0 = (int64_t)blockIdx.x * kTeams; t0 < tasks; t0 += (int64_t)gridDim.x * kTeams) {
    const int64_t task = t0 + warp / kTeam;
    const bool on = task < tasks;
    int part = 0, h = 0, req = 0, s0 = 0, s1 = 0;
    if (on) {
      part = (int)(task % kMergeParts);
      h = (int)(task / kMergeParts % a.heads);
      const int u = (int)(task / ((int64_t)kMergeParts * a.heads));
      s0 = a.sched[a.off_merge + u];
      s1 = a.sched[a.off_merge + u + 1];
      req = a.sched[a.off_units + 2 * u];
    }
    if (!waited) {
      pdl_wait();   // the partial states belong to the decode kernel
      waited = true;
    }
    float base = 0.f, z = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on) {
      const float* lp = a.l_part + h;
      const float* op = a.o_part + (int64_t)h * kLatentDim + kMergeDims * part + 4 * lane;
      constexpr int kAtOnce = 8;
      float4 o[kAtOnce];
      float lv[kAtOnce];
      auto load = [&](int s) {
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          const int64_t si = min(s + i * kTeam, s1 - 1);
          // volatile: all eight leave before the first is used
          asm volatile("ld.global.v4.f32 {%0,%1,%2,%3}, [%4];"
                       : "=f"(o[i].x), "=f"(o[i].y), "=f"(o[i].z), "=f"(o[i].w)
                       : "l"(op + si * a.heads * kLatentDim));
          lv[i] = lp[si * a.heads];
        }
      };
      load(s0 + sub);   // the first eight travel with the maxima
      float top = -CUDART_INF_F;
      for (int s = s0 + lane; s < s1; s += 32) top = fmaxf(top, lp[(int64_t)s * a.heads]);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, x));
      base = top == -CUDART_INF_F ? 0.f : top;
      for (int s = s0 + sub; s < s1; s += kAtOnce * kTeam) {
        if (s > s0 + sub) load(s);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          if (s + i * kTeam >= s1) break;
          const float w = exp2f((lv[i] - base) * kLog2e);
          z += w;
          acc.x = fmaf(w, o[i].x, acc.x);
          acc.y = fmaf(w, o[i].y, acc.y);
          acc.z = fmaf(w, o[i].z, acc.z);
          acc.w = fmaf(w, o[i].w, acc.w);
        }
      }
    }
    if constexpr (kTeam > 1) {
      acc_s[warp][lane] = acc;
      if (lane == 0) z_s[warp] = z;
      __syncthreads();
      if (sub == 0) {
#pragma unroll
        for (int w = 1; w < kTeam; ++w) {
          const float4 v = acc_s[warp + w][lane];
          acc.x += v.x;
          acc.y += v.y;
          acc.z += v.z;
          acc.w += v.w;
          z += z_s[warp + w];
        }
      }
      __syncthreads();
    }
    if (on && sub == 0) {
      const float inv = z == 0.f ? 0.f : 1.f / z;
      const int64_t qrow = (int64_t)req * a.heads + h;
      *reinterpret_cast<uint2*>(a.out + qrow * kLatentDim + kMergeDims * part + 4 * lane) =
          make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
      if (part == 0 && lane == 0 && a.lse != nullptr) a.lse[qrow] = base + log2f(z) * kLn2;
    }
  }
  if (!waited) pdl_wait();   // complete only after the decode kernel
}

__global__ void __launch_bounds__(kMergeWarps * 32) latent_merge_kernel(const __grid_constant__ LatentArgs a) {
  __shared__ float4 acc_s[kMergeWarps][32];
  __shared__ float z_s[kMergeWarps];
  pdl_launch_dependents();
  if (a.wait_epoch != 0) pdl_wait();   // the schedule came from another stream
  const int units = a.sched[H_BATCH] > a.batch ? 0 : a.sched[H_NUNITS];   // as the decode kernel
  const int team = merge_team(a.sched[H_MAXCHUNKS], (int64_t)units * a.heads * kMergeParts);
  if (team == 1)
    merge_tasks<1>(a, units, acc_s, z_s);
  else if (team == 2)
    merge_tasks<2>(a, units, acc_s, z_s);
  else if (team == 4)
    merge_tasks<4>(a, units, acc_s, z_s);
  else
    merge_tasks<8>(a, units, acc_s, z_s);
}

using Shape16 = LatentShape<16>;
using Shape32 = LatentShape<32>;
using Shape64 = LatentShape<64>;
static_assert(latent_smem<Shape16>() <= 227 * 1024 && latent_smem<Shape32>() <= 227 * 1024 &&
                  latent_smem<Shape64>() <= 227 * 1024,
              "dynamic shared memory of one CTA");

const void* kernel_of(int32_t heads) {
  switch (latent_block_heads(heads)) {
    case 16: return reinterpret_cast<const void*>(&latent_decode_kernel<Shape16>);
    case 32: return reinterpret_cast<const void*>(&latent_decode_kernel<Shape32>);
    default: return reinterpret_cast<const void*>(&latent_decode_kernel<Shape64>);
  }
}

int threads_of(int32_t heads) {
  switch (latent_block_heads(heads)) {
    case 16: return Shape16::kThreads;
    case 32: return Shape32::kThreads;
    default: return Shape64::kThreads;
  }
}

// ---------------------------------------------------------------- append
// A warp makes one cache row of a new token's latent and rotary parts, read
// from rows of any stride (they are often column ranges of one projection's
// output).  Bytes: a row read and written per token.  The rows do not depend
// on the table, so they are fetched while it is read (three dependent
// lookups).  Both sides are marked as streamed: a prompt's rows pass through
// L2 once (32,767 tokens of three states in turn: 14.7 us, 5.1 TB/s, against
// 16.8 us; the reads or the writes alone so marked change nothing; 131,072
// tokens 47.2 us, 6.4 TB/s, against 51.4), and rows that lie in L2 are as fast
// either way.  Two or four tokens a warp are no faster so, and slower for
// some 5,000 tokens (5.5 against 4.2 us).
constexpr int kAppendWarps = 8;
__global__ void __launch_bounds__(kAppendWarps * 32) latent_append_kernel(
    const uint8_t* __restrict__ latent, int64_t latent_stride, const uint8_t* __restrict__ rope,
    int64_t rope_stride, const int32_t* __restrict__ batch_indices,
    const int32_t* __restrict__ positions, int32_t n, const int32_t* __restrict__ indptr,
    const int32_t* __restrict__ indices, int32_t num_indices,
    const int32_t* __restrict__ last_page_len, int32_t batch, uint8_t* __restrict__ cache,
    int32_t num_pages, int32_t page_size, int32_t* err) {
  // the launch alone overlaps the kernel before (64 tokens 4.1 -> 1.8 us, 32,767
  // over two states in turn 14.4 -> 12.4)
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  if (i >= n) return;
  constexpr int kLat16 = kLatentDim * 2 / 16, kRope16 = kLatentRope * 2 / 16;
  const uint4* src = reinterpret_cast<const uint4*>(latent + i * latent_stride);
  const uint4 v0 = __ldcs(src + lane), v1 = __ldcs(src + 32 + lane);
  uint4 vr = make_uint4(0, 0, 0, 0);
  if (lane < kRope16) vr = __ldcs(reinterpret_cast<const uint4*>(rope + i * rope_stride) + lane);
  int64_t row = -1;   // the cache's row: page * page_size + slot
  const int b = batch_indices[i], pos = positions[i];
  if (b >= 0 && b < batch) {
    const int p0 = indptr[b], p1 = indptr[b + 1], last = last_page_len[b];
    const int64_t len = (int64_t)page_size * (p1 - p0 - 1) + last;
    if (p0 >= 0 && p1 > p0 && p1 <= num_indices && last >= 1 && last <= page_size && pos >= 0 &&
        pos < len) {
      const int pg = indices[p0 + pos / page_size];
      if (pg >= 0 && pg < num_pages) row = (int64_t)pg * page_size + pos % page_size;
    }
  }
  if (row < 0) {
    if (lane == 0 && err != nullptr) atomicOr(err, PKD_DEV_ERR_BOUNDS);
    return;
  }
  uint4* dst = reinterpret_cast<uint4*>(cache + row * kLatentRow * 2);
  __stcs(dst + lane, v0);
  __stcs(dst + 32 + lane, v1);
  if (lane < kRope16) __stcs(dst + kLat16 + lane, vr);
}
static_assert(kLatentDim * 2 / 16 == 64 && kLatentRope * 2 / 16 <= 32, "two pieces per lane");

}  // namespace

int latent_smem_bytes(int32_t heads) {
  switch (latent_block_heads(heads)) {
    case 16: return latent_smem<Shape16>();
    case 32: return latent_smem<Shape32>();
    default: return latent_smem<Shape64>();
  }
}

cudaError_t latent_prepare(int32_t heads) {
  return cudaFuncSetAttribute(kernel_of(heads), cudaFuncAttributeMaxDynamicSharedMemorySize,
                              latent_smem_bytes(heads));
}

cudaError_t latent_occupancy(int32_t heads, int* blocks_per_sm) {
  return cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks_per_sm, kernel_of(heads), threads_of(heads),
                                                       (size_t)latent_smem_bytes(heads));
}

int latent_merge_blocks(int32_t heads, int32_t units, int32_t most_slots, int most) {
  const int64_t tasks = (int64_t)units * heads * kMergeParts;
  const int64_t teams = kMergeWarps / merge_team(most_slots, tasks);
  const int64_t blocks = (tasks + teams - 1) / teams;
  return (int)(blocks < most ? blocks : most);
}

cudaError_t launch_latent(const LatentArgs& a, int grid, int merge_grid, cudaEvent_t decode_done,
                          cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads_of(a.heads));
  cfg.dynamicSmemBytes = (size_t)latent_smem_bytes(a.heads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {const_cast<LatentArgs*>(&a)};
  cudaError_t e = cudaLaunchKernelExC(&cfg, kernel_of(a.heads), args);
  if (e != cudaSuccess) return e;
  if (decode_done && (e = cudaEventRecordWithFlags(decode_done, stream, cudaEventRecordExternal)) !=
                         cudaSuccess)
    return e;
  if (merge_grid == 0) return cudaSuccess;
  cfg.gridDim = dim3(merge_grid);
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(&latent_merge_kernel), args);
}

// The cache maps, one per region: {64 columns, token of 8, column chunk, group
// of 8 tokens, page} with byte strides {row, 128, 8 rows, page}; box {64, 8,
// the region's chunks, 2 groups, 1 page}, which lands as [group][chunk][8
// tokens][128 bytes] with the 128-byte swizzle.
cudaError_t encode_latent_map(const void* cache, int32_t num_pages, int32_t page_size, int region,
                              CUtensorMap* map) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = map_encoder();
  if (encode == nullptr) return cudaErrorNotSupported;
  if (cache == nullptr || (uintptr_t)cache % 16 != 0 || page_size % 16 != 0 || num_pages < 1)
    return cudaErrorInvalidValue;
  const cuuint64_t row = (cuuint64_t)kLatentRow * 2;
  const cuuint64_t dims[5] = {64, 8, (cuuint64_t)kChunks, (cuuint64_t)(page_size / 8),
                              (cuuint64_t)num_pages};
  const cuuint64_t strides[4] = {row, 128, 8 * row, row * (cuuint64_t)page_size};
  const cuuint32_t box[5] = {64, 8, (cuuint32_t)region_chunks(region), 2, 1};
  const cuuint32_t elem[5] = {1, 1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(cache), dims, strides,
                box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

// The query map: {64 columns, head, column chunk, request}, box {64, a block's
// heads, every chunk, 1}, which lands as [chunk][head][128 bytes] with the
// 128-byte swizzle; heads past the last read as zeros.
cudaError_t encode_latent_q_map(const void* q, int32_t batch, int32_t heads, CUtensorMap* map) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = map_encoder();
  if (encode == nullptr) return cudaErrorNotSupported;
  if (q == nullptr || (uintptr_t)q % 16 != 0 || batch < 1 || heads < 1) return cudaErrorInvalidValue;
  const cuuint64_t row = (cuuint64_t)kLatentRow * 2;
  const cuuint64_t dims[4] = {64, (cuuint64_t)heads, (cuuint64_t)kChunks, (cuuint64_t)batch};
  const cuuint64_t strides[3] = {row, 128, row * (cuuint64_t)heads};
  const cuuint32_t box[4] = {64, (cuuint32_t)latent_block_heads(heads), (cuuint32_t)kChunks, 1};
  const cuuint32_t elem[4] = {1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(q), dims, strides, box,
                elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

cudaError_t launch_latent_append(const void* latent, int64_t latent_stride, const void* rope,
                                 int64_t rope_stride, const int32_t* batch_indices,
                                 const int32_t* positions, int32_t n, const int32_t* indptr,
                                 const int32_t* indices, int32_t num_indices,
                                 const int32_t* last_page_len, int32_t batch, void* cache,
                                 int32_t num_pages, int32_t page_size, int32_t* err,
                                 cudaStream_t stream) {
  const int64_t blocks = ((int64_t)n + kAppendWarps - 1) / kAppendWarps;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kAppendWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, latent_append_kernel, static_cast<const uint8_t*>(latent),
                            latent_stride, static_cast<const uint8_t*>(rope), rope_stride,
                            batch_indices, positions, n, indptr, indices, num_indices,
                            last_page_len, batch, static_cast<uint8_t*>(cache), num_pages,
                            page_size, err);
}

}  // namespace pkd
