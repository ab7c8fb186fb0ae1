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
// HBM bound where many rows move, latency bound where one does.  A cluster
// of 1 to 8 blocks takes one (layer, request, head): each block keeps the
// ordered keys of its share of the tokens in shared memory (weights and
// positions are read once), the budget-th largest key is found by a radix
// search of four 8-bit digits whose histograms the blocks add up through
// distributed shared memory, the bitmap of kept tokens is gathered by every
// block, and the blocks then move disjoint windows of the pairs.  The moves
// begin only after every block of the cluster has read its weights.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "evict.h"
#include "pkd.h"

namespace pkd {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kWindow = 512;   // pairs whose slots are listed at a time
constexpr uint32_t kFull = 0xffffffffu;

// fp32 order as unsigned order: NaN lowest, -0 equal to 0; kept-always above all
__device__ __forceinline__ uint32_t key_of(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
constexpr uint32_t kAlways = 0xffffffffu;

struct Shared {
  // a pass's digits; three in turn, as a block may still read the last pass's
  // from here while this one zeroes the next
  int hist[3][256];
  int sums[kWarps + 1];
  uint32_t prefix;       // digits found so far
  int need;              // keys still to take among those with the prefix
  int equal;             // this block's keys equal to the threshold
  int eq_before;
};

// exclusive prefix sum over the block's threads; total in sh.sums[kWarps]
__device__ __forceinline__ int block_scan(Shared& sh, int v) {
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

// Dynamic shared memory: Shared, keys [share], bitmap [words], before
// [words], lists [2][kWindow].
struct Sizes {
  int share;   // tokens of a block (a multiple of 32)
  int words;   // bitmap words of the longest request
};
__host__ __device__ inline Sizes sizes_for(int max_len, int blocks) {
  const int words = (max_len + 31) / 32;
  return Sizes{(words + blocks - 1) / blocks * 32, words};
}
inline size_t smem_for(const Sizes& z) {
  return sizeof(Shared) + 16 + ((size_t)z.share + 2 * (size_t)z.words + 2 * kWindow) * 4;
}

__global__ void __launch_bounds__(kThreads) evict_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  cg::cluster_group cluster = cg::this_cluster();
  const int blocks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const Sizes z = sizes_for(a.max_len, blocks);
  Shared& sh = *reinterpret_cast<Shared*>(raw);
  uint32_t* keys = reinterpret_cast<uint32_t*>(raw + ((sizeof(Shared) + 15) & ~(size_t)15));
  uint32_t* kept = keys + z.share;
  int* before = reinterpret_cast<int*>(kept + z.words);
  int* holes = before + z.words;
  int* movers = holes + kWindow;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  const int groups = a.per_head ? a.hkv : 1;
  int job = (int)(blockIdx.x / blocks);
  const int head = job % groups;
  job /= groups;
  const int req = job % a.batch, layer = job / a.batch;
  const int P = a.page_size, keep = a.budget;
  const int p0 = a.indptr[req], p1 = a.indptr[req + 1], last = a.last[req];
  const int64_t len = p1 > p0 ? (int64_t)P * (p1 - p0 - 1) + last : 0;
  const bool wrong = p0 < 0 || p1 <= p0 || last < 1 || last > P || len > a.max_len;
  if (wrong || len <= keep) {   // the same for every block of the cluster
    if (wrong && tid == 0 && a.err != nullptr) atomicOr(a.err, PKD_DEV_ERR_BOUNDS);
    return;
  }
  const int n = (int)len;
  const int32_t* pages = a.indices + p0;
  // a page outside the pool: the request is left as it is
  int bad = 0;
  for (int i = tid; i < p1 - p0; i += kThreads)
    bad |= (unsigned)pages[i] >= (unsigned)a.num_pages ? 1 : 0;
  if (__syncthreads_or(bad)) {
    if (tid == 0 && a.err != nullptr) atomicOr(a.err, PKD_DEV_ERR_BOUNDS);
    return;   // every block of the cluster saw the same pages
  }
  float* weights = a.weights[layer];
  int32_t* positions = a.positions[layer];
  const int seen = a.seen[req];
  const int words = (n + 31) / 32;
  const int w0 = min(words, rank * (z.share / 32)), w1 = min(words, w0 + z.share / 32);
  const int t0 = 32 * w0, t1 = min(n, 32 * w1);

  // ---- keys of this block's tokens
  for (int t = t0 + tid; t < t1; t += kThreads) {
    const int64_t at = (int64_t)pages[t / P] * a.hkv * P + t % P;
    float w;
    int pos;
    if (a.per_head) {
      w = weights[at + (int64_t)head * P];
      pos = positions[at + (int64_t)head * P];
    } else {
      // the heads' sum in head order, 64 bits, rounded once
      double s = 0.0;
      for (int h = 0; h < a.hkv; ++h) s += (double)weights[at + (int64_t)h * P];
      w = (float)s;
      pos = positions[at];
    }
    keys[t - t0] = (pos < a.sinks || pos >= seen - a.recent) ? kAlways : key_of(w);
  }
  if (tid < 256) sh.hist[0][tid] = 0;
  if (tid == 0) {
    sh.prefix = 0;
    sh.need = keep;
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
    if (tid < 256) sh.hist[(pass + 1) % 3][tid] = 0;
    cluster.sync();
    // thread i holds bin 255 - i, so the scan counts from the largest down
    int c = 0;
    if (tid < 256)
      for (int r = 0; r < blocks; ++r)
        c += cluster.map_shared_rank(&sh.hist[cur][0], r)[255 - tid];
    const int above = block_scan(sh, c);
    if (tid < 256 && above < need && above + c >= need) {
      sh.prefix = prefix | ((uint32_t)(255 - tid) << shift);
      sh.need = need - above;
    }
    __syncthreads();
  }
  const uint32_t limit = sh.prefix;
  const int need = sh.need;   // keys equal to the limit that stay, lowest slots first

  // ---- kept bits of this block's words: above the limit, then the first
  // `need` equal ones of the whole request
  int mine = 0;
  for (int i = tid; i < t1 - t0; i += kThreads) mine += keys[i] == limit ? 1 : 0;
  mine = __reduce_add_sync(kFull, mine);
  __syncthreads();
  if (tid == 0) sh.equal = 0;
  __syncthreads();
  if (lane == 0) atomicAdd(&sh.equal, mine);
  cluster.sync();
  if (tid == 0) {
    int b = 0;
    for (int r = 0; r < rank; ++r) b += *cluster.map_shared_rank(&sh.equal, r);
    sh.eq_before = b;
  }
  __syncthreads();
  int eq_before = sh.eq_before;
  for (int wb = w0; wb < w1; wb += kThreads) {   // a chunk of up to 512 words, a thread each
    const int w = wb + tid;
    uint32_t gt = 0, eq = 0;
    // warps form the words' masks: word wb + 32 warp + i from 32 lanes
    for (int i = 0; i < 32; ++i) {
      const int ww = wb + 32 * warp + i;
      if (ww >= w1) break;
      const int t = 32 * ww + lane;
      const uint32_t k = t < t1 ? keys[t - t0] : 0u;
      const uint32_t g = __ballot_sync(kFull, t < t1 && k > limit);
      const uint32_t e = __ballot_sync(kFull, t < t1 && k == limit);
      if (lane == i) {
        gt = g;
        eq = e;
      }
    }
    const int first = eq_before + block_scan(sh, __popc(eq));
    if (w < w1) {
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
      kept[w] = gt | take;
    }
    eq_before += sh.sums[kWarps];
  }
  cluster.sync();
  // ---- every block gathers the whole bitmap and its running counts
  for (int w = tid; w < words; w += kThreads) {
    const int owner = w / (z.share / 32);
    if (owner != rank) kept[w] = cluster.map_shared_rank(kept, owner)[w];
  }
  cluster.sync();   // no block's shared memory is read by others from here on
  int run = 0;
  for (int wb = 0; wb < words; wb += kThreads) {
    const int w = wb + tid;
    const int c = w < words ? __popc(kept[w]) : 0;
    const int ex = block_scan(sh, c);
    if (w < words) before[w] = run + ex;
    run += sh.sums[kWarps];
  }
  __syncthreads();
  // kept tokens below the budget, and so the number of holes there
  const int kw = keep / 32, kb = keep % 32;
  const int below = before[kw] + __popc(kept[kw] & ((1u << kb) - 1u));   // keep < n: kw < words
  const int moves = keep - below;

  // ---- the moves, a window of pairs at a time; windows go round the blocks
  const int nh = a.per_head ? 1 : a.hkv;
  uint8_t* kv = static_cast<uint8_t*>(a.kv[layer]);
  const int pieces = 2 * a.pieces;   // K and V
  for (int m0 = rank * kWindow; m0 < moves; m0 += blocks * kWindow) {
    const int m1 = min(moves, m0 + kWindow);
    __syncthreads();
    for (int w = tid; w < words; w += kThreads) {
      const int tw = 32 * w;
      if (tw < keep) {   // holes: tokens below the budget that go
        const uint32_t in = tw + 32 <= keep ? kFull : (1u << kb) - 1u;
        uint32_t free_bits = ~kept[w] & in;
        int r = tw - before[w];
        if (r < m1 && r + __popc(free_bits) > m0)
          for (; free_bits; free_bits &= free_bits - 1, ++r)
            if (r >= m0 && r < m1) holes[r - m0] = tw + __ffs(free_bits) - 1;
      }
      if (tw + 32 > keep) {   // movers: kept tokens behind it
        const uint32_t in = tw >= keep ? kFull : ~((1u << kb) - 1u);
        uint32_t bits = kept[w] & in;
        int r = tw >= keep ? before[w] - below : 0;
        if (r < m1 && r + __popc(bits) > m0)
          for (; bits; bits &= bits - 1, ++r)
            if (r >= m0 && r < m1) movers[r - m0] = tw + __ffs(bits) - 1;
      }
    }
    __syncthreads();
    const int rows = (m1 - m0) * nh;
    const int total = rows * pieces;
    constexpr int kUnroll = 4;
    for (int p = tid; p < total; p += kUnroll * kThreads) {
      uint4 v[kUnroll];
      uint8_t* to[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int q = p + u * kThreads;
        to[u] = nullptr;
        if (q < total) {
          const int row = q / pieces, piece = q % pieces;
          const int pair = row / nh, h = a.per_head ? head : row % nh;
          const int64_t in_row = (int64_t)h * a.head_bytes +
                                 (piece >= a.pieces ? a.v_bytes + 16 * (piece - a.pieces) : 16 * piece);
          const int src = movers[pair], dst = holes[pair];
          v[u] = *reinterpret_cast<const uint4*>(kv + pages[src / P] * a.page_bytes +
                                                 (src % P) * a.token_bytes + in_row);
          to[u] = kv + pages[dst / P] * a.page_bytes + (dst % P) * a.token_bytes + in_row;
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (to[u] != nullptr) *reinterpret_cast<uint4*>(to[u]) = v[u];
    }
    for (int row = tid; row < rows; row += kThreads) {
      const int pair = row / nh, h = a.per_head ? head : row % nh;
      const int src = movers[pair], dst = holes[pair];
      const int64_t from = ((int64_t)pages[src / P] * a.hkv + h) * P + src % P;
      const int64_t to = ((int64_t)pages[dst / P] * a.hkv + h) * P + dst % P;
      const float w = weights[from];
      const int32_t pos = positions[from];
      weights[to] = w;
      positions[to] = pos;
    }
  }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
  const int groups = a.per_head ? a.hkv : 1;
  const int64_t jobs = (int64_t)a.layers * a.batch * groups;
  // blocks per job: enough for the longest request's keys, then more while
  // the grid leaves SMs idle and a block keeps 512 tokens or more
  int blocks = 1;
  while (blocks < 8 && (a.max_len > blocks * kEvictBlockTokens ||
                        (jobs * blocks * 2 <= 304 && a.max_len >= blocks * 1024)))
    blocks *= 2;
  const size_t smem = smem_for(sizes_for(a.max_len, blocks));
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(jobs * blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)blocks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_kernel, a);
}

}  // namespace pkd
