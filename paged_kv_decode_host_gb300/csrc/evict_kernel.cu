// Eviction from a paged KV cache by accumulated attention weight, in place,
// for sm_103a.
//
// For a layer, a request of n > budget tokens and a KV head (or, when the
// heads evict together, their sum): the tokens with the `budget` largest
// weights stay -- tokens whose position is below `sinks` or among the last
// `recent` of those seen always, ties the lower slot first, a NaN weight as
// the lowest.  Attention does not depend on the order of cached tokens, so
// the cache is closed up with as few moves as there are holes: the i-th free
// slot below the budget takes the i-th kept token from behind it (its K and V
// rows, weight and position).  Slots behind the budget keep what they held.
// Sources and destinations are disjoint, so the moves need no order.
//
// Choosing is latency bound (weights and positions are read once: 8 bytes a
// token), moving is HBM bound.  A block takes one job (layer, request, head)
// and keeps its tokens' ordered keys in shared memory.  The budget-th largest
// key is found by a radix search of four 8-bit digits; when at most kFew
// tokens go (each step of steady decoding evicts one), by as many block-wide
// minima instead.  The kept tokens become a bitmap, whose running counts pair
// holes and movers.  Jobs with more than 32,768 tokens, and calls of few jobs
// with long requests, take a cluster of up to 8 blocks a job, whose digit
// counts and bitmaps meet through distributed shared memory.  Where a job may
// move 512 tokens or more, however many jobs there are, the moves are left to
// a second kernel over the whole GPU, which reads the bitmaps from the
// workspace.  A job's moves begin only when all its weights are read.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "evict.h"
#include "pkd.h"
#include "sm103_ptx.cuh"

namespace pkd {
namespace {

namespace cg = cooperative_groups;
using dev::kFull;
using dev::pdl_launch_dependents;
using dev::pdl_wait;

// Pairs listed at a time.  128 / 256 / 512: 102 / 98 / 99 us (24 requests of up
// to 4,609 tokens cut to 2,048, four layers), 91 / 92 / 112 (two of 65,539 to
// half, two layers).
constexpr int kWindow = 256;
constexpr int kFew = 8;        // evictions taken by block-wide minima

// fp32 order as unsigned order: NaN lowest, -0 equal to 0; kept-always above all
__device__ __forceinline__ uint32_t key_of(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
constexpr uint32_t kAlways = 0xffffffffu;

// x / d for x < 2^20 and d <= 2^11 by a multiplication: m = ceil(2^32 / d)
// gives x m / 2^32 = x / d + x e / (d 2^32) with e < d, an error below
// 2^20 / 2^32 < 1 / d
struct Div {
  uint32_t d, m;
  __device__ explicit Div(uint32_t v) : d(v), m(v == 1 ? 0 : 0xffffffffu / v + 1) {}
  __device__ uint32_t div(uint32_t x) const { return d == 1 ? x : __umulhi(x, m); }
};

// Tokens of a page: most sizes are powers of two.
struct PageSize {
  int size, shift;
  __device__ explicit PageSize(const EvictArgs& a) : size(a.page_size), shift(a.page_shift) {}
  __device__ int div(int t) const { return shift >= 0 ? t >> shift : t / size; }
};

// The sum of up to a few fp32 values, each addition's rounding error carried
// along (a + b = s + e exactly) and added at the end: as exact as 64-bit
// additions, whose rate here is 1/64 of fp32's.
struct Sum2 {
  float s = 0.f, e = 0.f;
  __device__ void add(float x) {
    const float t = s + x, z = t - s;
    e += (s - (t - z)) + (x - z);
    s = t;
  }
  __device__ float value() const { return fabsf(s) < CUDART_INF_F ? s + e : s; }
};

template <int kThreads>
struct Shared {
  // a pass's digits; three in turn, as a block may still read the last pass's
  // from here while this one zeroes the next
  int hist[3][256];
  int sums[kThreads / 32 + 1];
  unsigned long long low[2][kThreads / 32];
  uint32_t prefix;       // digits found so far
  int need;              // keys still to take among those with the prefix
  int equal;             // this block's keys equal to the threshold
  int eq_before;
  // the tokens of a window's pairs (where to, from), then the same as bytes of
  // head 0's K row and as slots of head 0
  int token[2 * kWindow];
  int64_t row[2 * kWindow], slot[2 * kWindow];
};

// exclusive prefix sum over the block's threads; total in sh.sums[warps]
template <int kThreads>
__device__ __forceinline__ int block_scan(Shared<kThreads>& sh, int v) {
  constexpr int kWarps = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();   // sums may still be read from the call before
  if (lane == 31) sh.sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const int s = lane < kWarps ? sh.sums[lane] : 0;
    int z = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, z, o);
      if (lane >= o) z += y;
    }
    __syncwarp();
    if (lane < kWarps) sh.sums[lane] = z - s;
    if (lane == 31) sh.sums[kWarps] = z;
  }
  __syncthreads();
  return sh.sums[warp] + x - v;
}

// Dynamic shared memory: Shared, bitmap [words], before [words], keys [share].
struct Sizes {
  int share;   // tokens of a block (a multiple of 32)
  int words;   // bitmap words of the longest request
};
__host__ __device__ inline Sizes sizes_for(int max_len, int blocks) {
  const int words = (max_len + 31) / 32;
  return Sizes{(words + blocks - 1) / blocks * 32, words};
}
template <int kThreads>
__host__ __device__ constexpr size_t shared_bytes() {
  return (sizeof(Shared<kThreads>) + 15) & ~(size_t)15;
}

struct Job {
  int layer, req, head, n;
  const int32_t* pages;
};
// false when the job has nothing to do: the table row is wrong (flagged by
// `tell`), or the request is not over the budget
__device__ __forceinline__ bool job_of(const EvictArgs& a, int job, bool tell, Job* j) {
  const int groups = a.per_head ? a.hkv : 1;
  j->head = job % groups;
  job /= groups;
  j->req = job % a.batch;
  j->layer = job / a.batch;
  const int p0 = a.indptr[j->req], p1 = a.indptr[j->req + 1], last = a.last[j->req];
  const int64_t len = p1 > p0 ? (int64_t)a.page_size * (p1 - p0 - 1) + last : 0;
  const bool wrong = p0 < 0 || p1 <= p0 || p1 > a.num_indices || last < 1 ||
                     last > a.page_size || len > a.max_len;
  if (wrong && tell && a.err != nullptr) atomicOr(a.err, PKD_DEV_ERR_BOUNDS);
  j->n = (int)len;
  j->pages = a.indices + p0;
  return !wrong && len > a.budget;
}

// Running counts of the bitmap, then the moves: windows of pairs `first`,
// `first` + `step`, ...
template <int kThreads>
__device__ __forceinline__ void move_pairs(const EvictArgs& a, Shared<kThreads>& sh, const Job& j,
                                           const uint32_t* kept, int* before, int first, int step) {
  const int tid = threadIdx.x;
  const PageSize P(a);
  const int keep = a.budget;
  const int words = (j.n + 31) / 32;
  int run = 0;
  for (int wb = 0; wb < words; wb += kThreads) {
    const int w = wb + tid;
    const int ex = block_scan(sh, w < words ? __popc(kept[w]) : 0);
    if (w < words) before[w] = run + ex;
    run += sh.sums[kThreads / 32];
  }
  __syncthreads();
  // kept tokens below the budget, and so the number of holes there
  const int kw = keep / 32, kb = keep % 32;
  const int below = before[kw] + __popc(kept[kw] & ((1u << kb) - 1u));   // keep < n: kw < words
  const int moves = keep - below;
  const int nh = a.per_head ? 1 : a.hkv;
  uint8_t* kv = static_cast<uint8_t*>(a.kv[j.layer]);
  float* weights = a.weights[j.layer];
  int32_t* positions = a.positions[j.layer];
  const Div by_row((uint32_t)(2 * a.pieces)), by_heads((uint32_t)nh);
  for (int m0 = first * kWindow; m0 < moves; m0 += step * kWindow) {
    const int m1 = min(moves, m0 + kWindow);
    __syncthreads();
    for (int w = tid; w < words; w += kThreads) {
      const int tw = 32 * w;
      if (tw < keep) {   // holes: tokens below the budget that go
        const uint32_t in = tw + 32 <= keep ? kFull : (1u << kb) - 1u;
        uint32_t bits = ~kept[w] & in;
        int r = tw - before[w];
        if (r < m1 && r + __popc(bits) > m0)
          for (; bits; bits &= bits - 1, ++r)
            if (r >= m0 && r < m1) sh.token[r - m0] = tw + __ffs(bits) - 1;
      }
      if (tw + 32 > keep) {   // movers: kept tokens behind it
        const uint32_t in = tw >= keep ? kFull : ~((1u << kb) - 1u);
        uint32_t bits = kept[w] & in;
        int r = tw >= keep ? before[w] - below : 0;
        if (r < m1 && r + __popc(bits) > m0)
          for (; bits; bits &= bits - 1, ++r)
            if (r >= m0 && r < m1) sh.token[kWindow + r - m0] = tw + __ffs(bits) - 1;
      }
    }
    __syncthreads();
    for (int i = tid; i < 2 * kWindow; i += kThreads)
      if ((i & (kWindow - 1)) < m1 - m0) {
        const int t = sh.token[i], pi = P.div(t), ps = t - pi * P.size;
        const int64_t page = j.pages[pi];
        sh.row[i] = page * a.page_bytes + ps * a.token_bytes;
        sh.slot[i] = page * a.hkv * P.size + ps;
      }
    __syncthreads();
    // 16 bytes of a row a thread, four in flight: scattered rows of 256 bytes
    // read and written at once come to 4.5 TB/s (24 requests of up to 4,609
    // tokens cut to 2,048, four layers), and more in flight are slower (eight
    // 107 against 100 us a call, sixteen 144)
    const int rows = (m1 - m0) * nh;
    const int total = rows * 2 * a.pieces;
    constexpr int kUnroll = 4;
    for (int p = tid; p < total; p += kUnroll * kThreads) {
      uint4 v[kUnroll];
      uint8_t* to[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int q = p + u * kThreads;
        to[u] = nullptr;
        if (q < total) {
          const int row = (int)by_row.div((uint32_t)q), piece = q - row * 2 * a.pieces;
          const int pair = (int)by_heads.div((uint32_t)row);
          const int h = a.per_head ? j.head : row - pair * nh;
          const int64_t in_row = h * a.head_bytes + (piece >= a.pieces
                                                         ? a.v_bytes + 16 * (piece - a.pieces)
                                                         : 16 * piece);
          v[u] = __ldcs(reinterpret_cast<const uint4*>(kv + sh.row[kWindow + pair] + in_row));
          to[u] = kv + sh.row[pair] + in_row;
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (to[u] != nullptr) __stcs(reinterpret_cast<uint4*>(to[u]), v[u]);
    }
    for (int row = tid; row < rows; row += kThreads) {
      const int pair = (int)by_heads.div((uint32_t)row);
      const int64_t h = (int64_t)(a.per_head ? j.head : row - pair * nh) * P.size;
      const float w = weights[sh.slot[kWindow + pair] + h];
      const int32_t pos = positions[sh.slot[kWindow + pair] + h];
      weights[sh.slot[pair] + h] = w;
      positions[sh.slot[pair] + h] = pos;
    }
  }
}

// kCluster: a cluster per job (of one block or more); kMove: the job's moves
// follow, else the bitmap is left in the workspace for evict_move_kernel.
template <int kThreads, bool kCluster, bool kMove>
__global__ void __launch_bounds__(kThreads) evict_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  constexpr int kWarps = kThreads / 32;
  pdl_wait();   // the launch alone overlaps the kernel before (98.1 -> 96.2 us, 92.2 -> 90.3)
  if (!kMove) pdl_launch_dependents();
  int blocks = 1, rank = 0;
  if constexpr (kCluster) {
    blocks = (int)cg::this_cluster().num_blocks();
    rank = (int)cg::this_cluster().block_rank();
  }
  auto meet = [&] {   // every block of the job
    if constexpr (kCluster)
      cg::this_cluster().sync();
    else
      __syncthreads();
  };
  auto theirs = [&](auto* p, int r) {
    if constexpr (kCluster)
      return cg::this_cluster().map_shared_rank(p, r);
    else
      return p;
  };
  const Sizes z = sizes_for(a.max_len, blocks);
  Shared<kThreads>& sh = *reinterpret_cast<Shared<kThreads>*>(raw);
  uint32_t* kept = reinterpret_cast<uint32_t*>(raw + shared_bytes<kThreads>());
  int* before = reinterpret_cast<int*>(kept + z.words);
  uint32_t* keys = reinterpret_cast<uint32_t*>(before + z.words);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  Job j;
  const int job = (int)blockIdx.x / blocks;
  if (!job_of(a, job, tid == 0, &j)) return;   // the same for every block of the cluster
  const PageSize P(a);
  const int keep = a.budget, n = j.n;
  // a page outside the pool: the request is left as it is (every block of
  // the cluster sees the same pages)
  int bad = 0;
  for (int i = tid; i <= P.div(n - 1); i += kThreads)
    bad |= (unsigned)j.pages[i] >= (unsigned)a.num_pages ? 1 : 0;
  const int words = (n + 31) / 32;
  if (__syncthreads_or(bad)) {
    if (tid == 0 && a.err != nullptr) atomicOr(a.err, PKD_DEV_ERR_BOUNDS);
    if (!kMove && rank == 0)   // nothing to move: the slots below the budget stay
      for (int w = tid; w < words; w += kThreads)
        a.bitmaps[(int64_t)job * z.words + w] =
            32 * w + 32 <= keep ? kFull : 32 * w < keep ? (1u << (keep - 32 * w)) - 1u : 0u;
    return;
  }
  const float* weights = a.weights[j.layer];
  const int32_t* positions = a.positions[j.layer];
  const int seen = a.seen[j.req];
  const int w0 = min(words, rank * (z.share / 32)), w1 = min(words, w0 + z.share / 32);
  const int t0 = 32 * w0, t1 = min(n, 32 * w1);

  // ---- keys of this block's tokens, several tokens' loads in flight
  auto key_with = [&](float w, int pos) {
    return (pos < a.sinks || pos >= seen - a.recent) ? kAlways : key_of(w);
  };
  if (a.per_head) {
    constexpr int kAtOnce = 8;
    for (int tb = t0 + tid; tb < t1; tb += kAtOnce * kThreads) {
      float w[kAtOnce];
      int pos[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int t = min(tb + i * kThreads, t1 - 1), pi = P.div(t);
        const int64_t at = ((int64_t)j.pages[pi] * a.hkv + j.head) * P.size + (t - pi * P.size);
        w[i] = weights[at];
        pos[i] = positions[at];
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        if (tb + i * kThreads < t1) keys[tb + i * kThreads - t0] = key_with(w[i], pos[i]);
    }
  } else {
    // by the heads' sum, in head order
    constexpr int kAtOnce = 4, kHeads = 4;
    for (int tb = t0 + tid; tb < t1; tb += kAtOnce * kThreads) {
      Sum2 sum[kAtOnce];
      int64_t at[kAtOnce];
      int pos[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int t = min(tb + i * kThreads, t1 - 1), pi = P.div(t);
        at[i] = (int64_t)j.pages[pi] * a.hkv * P.size + (t - pi * P.size);
        pos[i] = positions[at[i]];
      }
      for (int h = 0; h < a.hkv; h += kHeads) {
        float w[kAtOnce][kHeads];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
          for (int k = 0; k < kHeads; ++k)
            w[i][k] = h + k < a.hkv ? weights[at[i] + (int64_t)(h + k) * P.size] : 0.f;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
          for (int k = 0; k < kHeads; ++k)
            if (h + k < a.hkv) sum[i].add(w[i][k]);
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        if (tb + i * kThreads < t1) keys[tb + i * kThreads - t0] = key_with(sum[i].value(), pos[i]);
    }
  }

  if (!kCluster && n - keep <= kFew) {
    // ---- few go: the lowest key, of equal ones the highest slot, so often
    for (int w = tid; w < words; w += kThreads)
      kept[w] = n - 32 * w >= 32 ? kFull : (1u << (n - 32 * w)) - 1u;
    auto lowest = [&] {   // of this thread's tokens that are still kept
      unsigned long long low = ~0ull;
      for (int t = tid; t < n; t += kThreads)
        if (kept[t >> 5] >> (t & 31) & 1u) {
          const unsigned long long k = (unsigned long long)keys[t] << 32 | (0xffffffffu - (uint32_t)t);
          low = k < low ? k : low;
        }
      return low;
    };
    __syncthreads();
    unsigned long long mine = lowest();
    for (int e = 0; e < n - keep; ++e) {
      unsigned long long low = mine;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long x = __shfl_xor_sync(kFull, low, o);
        low = x < low ? x : low;
      }
      if (lane == 0) sh.low[e & 1][warp] = low;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWarps; ++w) low = sh.low[e & 1][w] < low ? sh.low[e & 1][w] : low;
      const int t = (int)(0xffffffffu - (uint32_t)low);
      if (mine == low) {   // the token's owner; others of its word wait for the next barrier
        atomicAnd(&kept[t >> 5], ~(1u << (t & 31)));
        mine = lowest();
      }
    }
    __syncthreads();
  } else {
    for (int i = tid; i < 256; i += kThreads) sh.hist[0][i] = 0;
    if (tid == 0) {
      sh.prefix = 0;
      sh.need = keep;
      sh.equal = 0;
    }
    __syncthreads();
    // ---- the keep-th largest key, digit by digit
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = 24 - 8 * pass, cur = pass % 3;
      const uint32_t prefix = sh.prefix;
      const int need = sh.need;
      for (int i = tid; i < t1 - t0; i += kThreads) {
        const uint32_t k = keys[i];
        if (pass == 0 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
          atomicAdd(&sh.hist[cur][(k >> shift) & 255], 1);
      }
      for (int i = tid; i < 256; i += kThreads) sh.hist[(pass + 1) % 3][i] = 0;
      meet();
      // bins from the largest down, 256 / kThreads or one to a thread
      constexpr int kBins = kThreads >= 256 ? 1 : 256 / kThreads;
      int c[kBins], all = 0;
#pragma unroll
      for (int b = 0; b < kBins; ++b) {
        c[b] = 0;
        const int bin = 255 - (tid * kBins + b);
        if (bin >= 0)
          for (int r = 0; r < blocks; ++r) c[b] += theirs(&sh.hist[cur][0], r)[bin];
        all += c[b];
      }
      int above = block_scan(sh, all);
#pragma unroll
      for (int b = 0; b < kBins; ++b) {
        if (above < need && above + c[b] >= need) {
          sh.prefix = prefix | ((uint32_t)(255 - (tid * kBins + b)) << shift);
          sh.need = need - above;
        }
        above += c[b];
      }
      __syncthreads();
    }
    const uint32_t limit = sh.prefix;
    const int need = sh.need;   // keys equal to the limit that stay, lowest slots first

    // ---- kept bits of this block's words: above the limit, then the first
    // `need` equal ones of the whole request
    int eq_before = 0;
    if constexpr (kCluster) {
      int mine = 0;
      for (int i = tid; i < t1 - t0; i += kThreads) mine += keys[i] == limit ? 1 : 0;
      mine = __reduce_add_sync(kFull, mine);
      if (lane == 0) atomicAdd(&sh.equal, mine);
      meet();
      if (tid == 0) {
        int b = 0;
        for (int r = 0; r < rank; ++r) b += *theirs(&sh.equal, r);
        sh.eq_before = b;
      }
      __syncthreads();
      eq_before = sh.eq_before;
    }
    for (int wb = w0; wb < w1; wb += kThreads) {   // a word a thread
      uint32_t gt = 0, eq = 0;
      // a warp's 32 words, whose masks come from 32 lanes at a time
      const int wn = min(32, w1 - wb - 32 * warp);
      for (int i = 0; i < wn; ++i) {
        const int t = 32 * (wb + 32 * warp + i) + lane;
        const uint32_t k = t < t1 ? keys[t - t0] : 0u;
        const uint32_t g = __ballot_sync(kFull, t < t1 && k > limit);
        const uint32_t e = __ballot_sync(kFull, t < t1 && k == limit);
        if (lane == i) {
          gt = g;
          eq = e;
        }
      }
      const int first = eq_before + block_scan(sh, __popc(eq));
      if (wb + tid < w1) {
        int left = need - first;
        uint32_t take = 0;
        if (left >= __popc(eq)) {
          take = eq;
        } else {
          for (; left > 0; --left) {
            take |= eq & (0u - eq);
            eq &= eq - 1;
          }
        }
        kept[wb + tid] = gt | take;
      }
      eq_before += sh.sums[kWarps];
    }
  }
  if constexpr (!kMove) {
    // the words of this block; a job that has nothing to do leaves none
    __syncthreads();
    uint32_t* out = a.bitmaps + (int64_t)job * z.words;
    for (int w = w0 + tid; w < w1; w += kThreads) out[w] = kept[w];
    meet();   // no block ends while others read its shared memory
    return;
  }
  meet();
  if constexpr (kCluster) {
    // ---- every block gathers the whole bitmap
    for (int w = tid; w < words; w += kThreads) {
      const int owner = w / (z.share / 32);
      if (owner != rank) kept[w] = theirs(kept, owner)[w];
    }
    meet();   // no block's shared memory is read by others from here on
  }
  move_pairs(a, sh, j, kept, before, rank, blocks);
}

// The moves of a call whose jobs may move 512 tokens or more: a.splits blocks
// per job.
constexpr int kMoveThreads = 512;
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  const Sizes z = sizes_for(a.max_len, 1);
  Shared<kMoveThreads>& sh = *reinterpret_cast<Shared<kMoveThreads>*>(raw);
  uint32_t* kept = reinterpret_cast<uint32_t*>(raw + shared_bytes<kMoveThreads>());
  int* before = reinterpret_cast<int*>(kept + z.words);
  // neighbouring blocks: the heads of a request in the same window, whose
  // rows lie near each other
  const int groups = a.per_head ? a.hkv : 1;
  const int split = (int)blockIdx.x / groups % a.splits;
  const int job = (int)blockIdx.x / (groups * a.splits) * groups + (int)blockIdx.x % groups;
  // the table is older than the kernel before, which only reads it
  Job j;
  const bool idle = !job_of(a, job, false, &j);
  pdl_wait();   // the bitmaps
  if (idle) return;
  const uint32_t* in = a.bitmaps + (int64_t)job * z.words;
  for (int w = threadIdx.x; 32 * w < j.n; w += kMoveThreads) kept[w] = in[w];
  __syncthreads();
  move_pairs(a, sh, j, kept, before, split, a.splits);
}

// Where max_len is at most the budget nothing is cut; what is wrong is flagged
// all the same, a thread per request.
constexpr int kCheckThreads = 128;
__global__ void __launch_bounds__(kCheckThreads) evict_check_kernel(const __grid_constant__ EvictArgs a) {
  pdl_wait();
  const int req = (int)(blockIdx.x * kCheckThreads + threadIdx.x);
  Job j;
  if (req < a.batch) job_of(a, req, true, &j);
}

constexpr int kSms = 152;

struct EvictPlan {
  int64_t jobs;
  int blocks;    // of a job
  bool cluster, split;
  int threads, splits;
};

EvictPlan plan_for(int layers, int batch, int hkv, int per_head, int max_len, int budget) {
  EvictPlan p{};
  p.jobs = (int64_t)layers * batch * (per_head ? hkv : 1);
  // Where a job may move more than two windows, a kernel of its own moves
  // them, in blocks of a window or a few: within the choosing blocks the
  // longest jobs' moves would run alone at the end.  Few jobs choose with a
  // cluster each (while a block keeps 4,096 tokens or more).
  const int most = (max_len - budget < budget ? max_len - budget : budget);
  p.split = most >= 2 * kWindow;
  p.blocks = 1;
  while (p.blocks < 8 && (max_len > p.blocks * kEvictBlockTokens ||
                          (p.split && p.jobs * p.blocks * 2 <= kSms && max_len > p.blocks * 4096)))
    p.blocks *= 2;
  p.cluster = p.blocks > 1;
  // a block per 2,048 tokens of four warps: more blocks per SM hide each
  // other's barriers
  const int share = (max_len + p.blocks - 1) / p.blocks;
  p.threads = p.cluster ? 512 : share <= 2048 ? 128 : share <= 8192 ? 256 : 512;
  const int64_t windows = (most + kWindow - 1) / kWindow, want = (8 * kSms + p.jobs - 1) / p.jobs;
  p.splits = (int)(windows < 4 ? windows : want < 4 ? 4 : want < windows ? want : windows);
  return p;
}

template <int kThreads, bool kCluster, bool kMove>
cudaError_t launch_choose(const EvictArgs& a, const EvictPlan& p, cudaStream_t stream) {
  const Sizes z = sizes_for(a.max_len, p.blocks);
  const size_t smem = shared_bytes<kThreads>() + ((size_t)z.share + 2 * (size_t)z.words) * 4;
  auto f = &evict_kernel<kThreads, kCluster, kMove>;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.jobs * p.blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.blocks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kCluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, f, a);
}

cudaError_t launch_check(EvictArgs& a, cudaStream_t stream) {
  a.layers = a.per_head = 0;   // jobs are requests
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.batch + kCheckThreads - 1) / kCheckThreads));
  cfg.blockDim = dim3(kCheckThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_check_kernel, a);
}

}  // namespace

size_t evict_workspace_bytes(int layers, int batch, int hkv, int per_head, int max_len, int budget) {
  const EvictPlan p = plan_for(layers, batch, hkv, per_head, max_len, budget);
  return p.split ? (size_t)p.jobs * (size_t)sizes_for(max_len, 1).words * 4 : 0;
}

cudaError_t launch_evict(EvictArgs& a, cudaStream_t stream) {
  if (a.max_len <= a.budget) return launch_check(a, stream);
  const EvictPlan p = plan_for(a.layers, a.batch, a.hkv, a.per_head, a.max_len, a.budget);
  a.splits = p.splits;
  a.page_shift = page_shift_of(a.page_size);
  if (!p.split) {
    if (p.cluster) return launch_choose<512, true, true>(a, p, stream);
    if (p.threads == 128) return launch_choose<128, false, true>(a, p, stream);
    if (p.threads == 256) return launch_choose<256, false, true>(a, p, stream);
    return launch_choose<512, false, true>(a, p, stream);
  }
  cudaError_t e = p.cluster          ? launch_choose<512, true, false>(a, p, stream)
                  : p.threads == 128 ? launch_choose<128, false, false>(a, p, stream)
                  : p.threads == 256 ? launch_choose<256, false, false>(a, p, stream)
                                     : launch_choose<512, false, false>(a, p, stream);
  if (e != cudaSuccess) return e;
  const size_t smem = shared_bytes<kMoveThreads>() + 2 * (size_t)sizes_for(a.max_len, 1).words * 4;
  if (smem > 48 * 1024) {
    e = cudaFuncSetAttribute(evict_move_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.jobs * p.splits));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_move_kernel, a);
}

}  // namespace pkd
