// Attention of drafted tokens over a paged cache for sm_103a.
//
// Request b has l_b cached tokens, the last n_b of which are drafted in this
// step: a tree, or a chain.  With c_b = l_b - n_b, query token i (n_b of them)
// stands at position c_b + depth_i, cached token t < c_b at t, draft j at c_b
// + depth_j.  Per query head
//     s = scale q.k;  s = cap tanh(s / cap);  s -= slope (pos_q - pos_k)
// over the tokens t < c_b and the drafts whose bit is set in the query's mask
// (a chain: j <= i), in a window only where pos_q - pos_k < window;
//     out = softmax(s) V,  lse = log sum exp(s);  nothing seen: 0 and -inf.
//
// A work item is one KV head of up to 128 / g query tokens of a request over a
// range of its cached tokens: the 128 query rows of a tile share every key and
// value, so both products run on the tensor cores, in rounds of 128 tokens.  Per
// CTA: warps 8 and 10 copy queries and K, and V, into rings of three rounds;
// warp 9 issues S = Q K^T, two S buffers ahead of the softmax; warps 0-7 (two per
// lane quadrant of tensor memory, a row per lane) turn S into P, in tensor memory;
// warp 11 issues O += P V, whose accumulator stays there for the whole item.
//  * S and P have two buffers each and O one: 512 columns of tensor memory.  Q
//    (32 KB) and the rings (192 KB) fill the shared memory.
//  * rounds that some row does not see whole (drafts, a window's edge, the
//    range's end) get a 64-bit word per row of the columns that it sees, from
//    the context's length, the window and 64 bits of the mask; other rounds
//    (nearly all of a long context) pay for none of it;
//  * masked scores are replaced, never added to, so what K holds there plays
//    no part.  P is 0 there, and 0 x V is 0 only for finite V: a result that
//    is not finite while some token that its row does not see has a value
//    that is not is summed again over the tokens seen (redo_rows);
//  * rows that have seen nothing keep the base -inf and a sum of 0;
//  * tanh(x) is a polynomial up to 0.4, within 2^-23 of itself; past that 1 - 2
//    / (1 + e^2x), an exponential and a reciprocal, within about 2^-22; the
//    hardware's tanh (2^-11) would show in the lse;
//  * distances are subtracted as whole numbers before they meet the slope;
//  * P is rounded to bf16 for the product (V's type, which the tensor cores
//    want for both); the row's sum, and with it the lse, is that of the weights
//    before it.  Beside the output's own rounding that makes errors up to 1.41
//    times those of an fp32 P (measured 0.0019 to 0.0024 against 0.0017); a second
//    product with the rest of P would want 128 more columns of tensor memory, whose
//    512 are taken.  Sums, bases and states between parts are fp32;
//  * lane quadrants without a query row (fewer than 97 rows) only keep the
//    barriers' count.
// What bounds it: with few rows per KV head memory (64 ragged requests up to 8,192
// tokens x 16 drafts, 32 heads on 8: 1.06 GB in 157 to 160 us, 6.6 TB/s); with full tiles
// the round, about 1,750 cycles for 1,024 of tensor products (16 requests x 61 drafts
// of 64 heads: 155 GFLOP in 123 us, 1.26 PFLOP/s; 140 in a long row of calls, where
// the power limit takes the clock from 2,070 to 1,680 MHz), in which the tensor cores
// wait for the softmax; a capped score's polynomial adds 700.  On the way there: one
// copy instead of two per 16 tokens 159 -> 141 us; descriptors stepped by constants,
// by an elected thread, 900 cycles of issue a round less; waits whose first tries do
// not look at the clock 139 -> 131.  Tried and
// slower: an O of its own for each stream of rounds; two tiles per item; weights
// under the last base before the round's largest score is known (they mend too
// often what they save); releasing S before its scores are capped.
// Every wait is bounded, as in the dense shared-prefix role (prefix_tc_body.cuh),
// whose instructions and barriers these are (but see slow_wait).
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <type_traits>

#include "plan_layout.h"
#include "prefix_tc_body.cuh"
#include "tensor_map.h"
#include "tree.h"

namespace pkd {
namespace {

using namespace dev;
using namespace tc;
static_assert(kTreeRows == kDenseRows && kTreeRound == kRoundTok, "the dense role's tile");

// Caps up to here (in units of log2) keep the base 0: weights within 2^-90 ..
// 2^90, sums of 2^31 of them below 2^122.
constexpr float kFixedBase = 90.f;
// Tokens that every row of the warp sees, from which on a base of 0 costs no
// precision (errors against 64 bits: 1.41 times those of a plain fp32 form from
// some hundred tokens on, with either base; 1.51 for 6 to 15 with 0).
constexpr int kFixedTokens = 384;
// Staged K and V: tiles of 16 tokens, [2 x 8 tokens][half of the dims][8][128 B],
// each one copy: a copy costs its warp 50 to 90 cycles, and two (one per half)
// were what bounded rounds of wide trees (2,300 cycles: 1,400 of copies).
constexpr int kTileBytes = 2 * kBoxBytes;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.4426950408889634f;

// the lowest x bits of 64
__device__ __forceinline__ uint64_t low_bits(int x) {
  return x <= 0 ? 0ull : x >= 64 ? ~0ull : (1ull << x) - 1;
}

__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}

// tc_wait whose first tries are the whole warp's, with a vote at once: a branch
// that the compiler knows to be uniform, and no look at the clock.  Behind the
// abort flag stands a count that a recomputation (redo_rows) raises as it goes: a
// wait that runs out while it rises is for that, however long it takes, and
// starts over (the recomputation is a loop over its item's tokens, which ends).
__device__ __noinline__ bool slow_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* err,
                                       int lane) {
  for (;;) {
    const int before = abort_flag[1];
    if (__all_sync(kFull, mbar_wait(bar, parity, abort_flag))) return true;
    if (__any_sync(kFull, *abort_flag != 0 || abort_flag[1] == before)) break;
  }
  if (lane == 0) raise_error(err, abort_flag, PKD_DEV_ERR_TIMEOUT);
  return false;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* err,
                                          int lane) {
#pragma unroll 1
  for (int n = 0; n < 64; ++n)
    if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
  return slow_wait(bar, parity, abort_flag, err, lane);
}

__device__ __forceinline__ uint64_t l2_evict_normal_policy() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// One query row of an item.
struct Row {
  const uint32_t* mask;   // its words, null in a chain
  int words;
  const int32_t* depths;  // of its request's drafts, or null: their numbers
  int ctx, drafts;        // cached tokens before the drafts, drafts
  int i, depth;           // its token's number and depth
  int window;             // 0: none
  int first_seen;         // the window's first context token (or below 0)
};

__device__ __forceinline__ int depth_of(const Row& r, int j) {
  return r.depths != nullptr ? max(__ldg(r.depths + j), 0) : j;
}

// Bits j0 .. j0 + 63 of the row's mask (j0 > -64), those outside it 0.
__device__ __forceinline__ uint64_t mask_bits(const Row& r, int j0) {
  const int w = j0 >> 5, s = j0 & 31;   // w may be -1 or -2
  auto word = [&](int k) -> uint64_t { return k >= 0 && k < r.words ? __ldg(r.mask + k) : 0u; };
  const uint64_t lo = word(w) | (word(w + 1) << 32);
  return s == 0 ? lo : (lo >> s) | (word(w + 2) << (64 - s));
}

// The columns c of 64 whose token t0 + c, below te, the row sees.
__device__ __forceinline__ uint64_t visible(const Row& r, int t0, int te) {
  uint64_t vis = low_bits(r.ctx - t0) & ~low_bits(r.first_seen - t0);
  const int j0 = t0 - r.ctx;
  if (j0 > -64 && j0 < r.drafts) {
    uint64_t own = r.mask != nullptr ? mask_bits(r, j0)
                                     : low_bits(r.i + 1 - j0) & ~low_bits(-j0);
    own &= low_bits(r.drafts - j0);
    if (r.window > 0 && r.depth >= r.window) {
      if (r.depths == nullptr)   // draft j stands j behind the context
        own &= ~low_bits(r.depth - r.window + 1 - j0);
      else   // (a tree deeper than the window: rare)
        for (uint64_t m = own; m != 0; m &= m - 1) {
          const int c = __ffsll((long long)m) - 1;
          if (r.depth - depth_of(r, j0 + c) >= r.window) own &= ~(1ull << c);
        }
    }
    vis |= own;
  }
  return vis & low_bits(te - t0);
}

// cap tanh(s scale ln 2 / 2), scale = 2 log2(e) scale_of_the_scores / cap: the
// exponential's error is 2^-22 of the cap, so small ones take the polynomial.
__device__ __forceinline__ float capped(float s, float scale, float cap) {
  const float u = s * scale, x = u * (0.5f * kLn2), y = x * x;
  const float small =
      cap * x * fmaf(fmaf(fmaf(kTanhFit3, y, kTanhFit2), y, kTanhFit1), y, kTanhFit0);
  const float any = fmaf(-2.f * cap, fast_rcp(1.f + fast_exp2(u)), cap);
  return y <= kTanhFitTo ? small : any;   // (NaN: any, a NaN)
}

__device__ __forceinline__ int64_t token_offset(const TreeArgs& a, int first_page, int head, int t) {
  int page = a.sched[a.off_pages + first_page + t / a.page_size];
  if ((unsigned)page >= (unsigned)a.num_pages) page = 0;   // (as the copies do)
  return page * a.page_elems + (t % a.page_size) * a.token_elems + head * a.head_elems;
}

// Two e4m3 values (in 16 bits) to bf16 pairs, exact; a NaN stays one.
__device__ __forceinline__ uint32_t widen2(uint32_t two) {
  uint32_t h, r;
  float lo, hi;
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\t}" : "=r"(h) : "r"(two));
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.f32.f16 %0, x;\n\tcvt.f32.f16 %1, y;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 8 values from element `at` on.
template <bool kFp8>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&f)[8]) {
  uint32_t w[4];
  if (kFp8) {
    const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p) + at);
    w[0] = widen2(x.x);
    w[1] = widen2(x.x >> 16);
    w[2] = widen2(x.y);
    w[3] = widen2(x.y >> 16);
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    f[2 * u] = __uint_as_float(w[u] << 16);
    f[2 * u + 1] = __uint_as_float(w[u] & 0xffff0000u);
  }
}

// Are the 64 values from element `at` on finite?
template <bool kFp8>
__device__ __forceinline__ bool finite64(const void* p, int64_t at) {
  float bad = 0.f;
#pragma unroll
  for (int d = 0; d < 64; d += 8) {
    float v[8];
    load8<kFp8>(p, at + d, v);
#pragma unroll
    for (int u = 0; u < 8; ++u) bad = fmaf(v[u], 0.f, bad);
  }
  return bad == 0.f;
}

// What redo_rows takes and gives, in memory: its registers are the round's as well
// (held there, sums and arguments took 2 to 3 % of wide trees).
struct Redo {
  Row row;
  bool mine;              // this lane's row is one
  const uint16_t* q;      // its query (any, where it is none)
  int first_page, head, tb, te, dim0, lane;
  float total, slope2;
  volatile int* beats;    // slow_wait's count
  float o[64];
};

// 64 dims (from dim0) of the warp's rows, one a lane, summed over the tokens that a row
// sees with weights 2^(s - total), where a token that it does not see has a value that
// is not finite in these dims, or where all that it sees are finite (weights above 1,
// whose sums pass fp32's range); false for rows whose result stands.  Tokens go by 8
// (on one page): all lanes read the same K and V.  (A look at V before each product
// took 5 to 10 % of a step of short requests; this is for caches that hold such values,
// and takes 1.4 us a token: 16 requests of 8,192 tokens x 16 drafts 10 ms, and 29 where
// every token read the rows' queries anew.)
template <bool kFp8>
__device__ __noinline__ bool redo_rows(const TreeArgs& a, Redo& in) {
  const Row& r = in.row;
  const int tb = in.tb, te = in.te, lane = in.lane, head = in.head, first_page = in.first_page;
  bool mine = in.mine;
  const auto beat = [&](int t0) {
    if (lane == 0 && (t0 - tb) % 1024 == 0) atomicAdd(const_cast<int*>(in.beats), 1);
  };
  bool hidden = false, shown = false;   // a value that is not finite: of a token not seen, of one that is
  for (int t0 = tb; t0 < te; t0 += 32) {
    beat(t0);
    const int t = t0 + lane;
    const uint32_t odd = __ballot_sync(
        kFull, t < te && !finite64<kFp8>(a.kv, token_offset(a, first_page, head, t) + a.v_elems + in.dim0));
    if (odd == 0) continue;
    const uint32_t see = mine ? (uint32_t)visible(r, t0, te) : 0u;
    hidden = hidden || (odd & ~see) != 0;
    shown = shown || (odd & see) != 0;
  }
  mine = mine && (hidden || !shown);
  if (!__any_sync(kFull, mine)) return false;
  for (int d = 0; d < 64; ++d) in.o[d] = 0.f;
  for (int t0 = tb; t0 < te; t0 += 8) {
    beat(t0);
    const uint32_t see = mine ? (uint32_t)visible(r, t0, te) & 0xffu : 0u;
    if (!__any_sync(kFull, see != 0)) continue;
    // (of 8 tokens the last may lie behind the range, on its last page: read, not used)
    const int64_t at = token_offset(a, first_page, head, t0);
    float s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = 0.f;
#pragma unroll 1
    for (int d = 0; d < kHeadDim; d += 8) {
      float y[8];
      load8<false>(in.q, d, y);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float x[8];
        load8<kFp8>(a.kv, at + j * a.token_elems + d, x);
#pragma unroll
        for (int u = 0; u < 8; ++u) s[j] = fmaf(x[u], y[u], s[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int t = t0 + j;
      const float x = a.cap_log2 != 0.f ? capped(s[j], a.scale_log2, a.cap_log2) : s[j] * a.scale_log2;
      const int64_t away = t < r.ctx              ? (int64_t)r.ctx + r.depth - t
                           : (see >> j & 1u) != 0 ? (int64_t)r.depth - depth_of(r, t - r.ctx)
                                                  : 0;
      s[j] = fast_exp2(fmaf(-in.slope2, (float)away, x) - in.total);
    }
    const int64_t v = at + a.v_elems + in.dim0;
#pragma unroll 1
    for (int d = 0; d < 64; d += 8) {
      float sum[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) sum[u] = in.o[d + u];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float x[8];
        load8<kFp8>(a.kv, v + j * a.token_elems + d, x);
        if ((see >> j & 1u) != 0) {
#pragma unroll
          for (int u = 0; u < 8; ++u) sum[u] = fmaf(s[j], x[u], sum[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) in.o[d + u] = sum[u];
    }
  }
  for (int d = 0; d < 64; ++d) in.o[d] *= a.v_scale;
  return mine;
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// 32 bytes (a whole sector: the lanes of a warp write rows far apart)
__device__ __forceinline__ void store32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// What the softmax of a round needs of its row and item.
struct Span {
  int ctx, te;            // tokens before the drafts; the item's end
  int reach;              // rounds that start below it need the window's mask in some row of the warp
  float slope2;           // log2(e) * the head's slope
  bool steep;             // some row's slope is too steep for the estimate of 32 biased scores' largest
};

// The largest of 32 biased scores is taken as the largest score's plus the
// largest bias: up to 31 slopes above what it is, so that weights of 2^-62 at
// worst stand for 1.  (Models' slopes are at most 1, 1.44 in log2.)
constexpr float kSteepest = 2.f;

// The order of an item's nr rounds: with slopes from the newest tokens to the
// oldest, whose biases only fall (the other way the base was raised, and O
// rescaled, in every round: 700 cycles of 3,000).
template <bool kSlopes>
__device__ __forceinline__ int round_at(int k, int nr) {
  return kSlopes ? nr - 1 - k : k;
}

// Two fp32 operations an instruction: these softmaxes are bound by instruction
// issue, and packed ones count once.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 f2(uint32_t lo, uint32_t hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void split(F2 x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x.v));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

// Largest of 32 values and `most`.
__device__ __forceinline__ float max32(const uint32_t (&v)[32], float most) {
  float m[4] = {most, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
  for (int j = 0; j < 32; j += 8)
#pragma unroll
    for (int u = 0; u < 4; ++u)
      m[u] = fmaxf(fmaxf(m[u], __uint_as_float(v[j + 2 * u])), __uint_as_float(v[j + 2 * u + 1]));
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// 64 products of a row (columns s_addr .. of its S) to capped scores, in units
// of log2.  At most 0.4 of the cap in magnitude, as nearly all are, they take
// tanh's polynomial on the FMA units; where any in the warp is larger, all are
// read again and take the exponential and the reciprocal, three times as long.
__device__ __noinline__ void cap64_any(float scale, float cap, uint32_t s_addr, uint32_t (&v)[64]) {
#pragma unroll 1
  for (int c = 0; c < 64; c += 16) {
    uint32_t x[16];
    tmem_ld16(s_addr + c, x);
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 16; ++j) v[c + j] = __float_as_uint(capped(__uint_as_float(x[j]), scale, cap));
  }
}
// (counts: this row is one, and what no row of the run sees is 0 here: columns that
// no product wrote hold what was there before, and would decide otherwise every run.)
__device__ __forceinline__ void cap64(const TreeArgs& a, bool counts, uint32_t s_addr, uint32_t (&v)[2][32]) {
  F2 c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) c[k] = f2(a.cap_poly[k], a.cap_poly[k]);
  float most[2] = {0.f, 0.f};   // of the squares
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const F2 x = f2(v[q][j], v[q][j + 1]), y = mul2(x, x);
      float lo, hi;
      split(y, lo, hi);
      most[q] = fmaxf(fmaxf(most[q], lo), hi);
      split(mul2(x, fma2(fma2(fma2(c[3], y, c[2]), y, c[1]), y, c[0])), lo, hi);
      v[q][j] = __float_as_uint(lo);
      v[q][j + 1] = __float_as_uint(hi);
    }
  if (__any_sync(kFull, counts && fmaxf(most[0], most[1]) > a.cap_bound)) {
    uint32_t w[64];
    cap64_any(a.scale_log2, a.cap_log2, s_addr, w);
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      v[0][j] = w[j];
      v[1][j] = w[32 + j];
    }
  }
}

// `value` for those of 32 scores that the row does not see.
__device__ __forceinline__ void hide32(uint32_t vis, float value, uint32_t (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (!(vis & (1u << j))) v[j] = __float_as_uint(value);
}

// 32 scores of tokens t0 .. t0 + 31 where some are biased by other distances
// than the place in the cache says (drafts), or masked: in units of log2 where
// there is a cap or a slope, else as they are.  (v: capped already)
template <bool kCap, bool kSlopes>
__device__ __forceinline__ void shape32(const TreeArgs& a, const Row& me, const Span& sp, int t0, uint32_t vis,
                                        uint32_t (&v)[32]) {
  if constexpr (kSlopes) {
    const float d0 = (float)((int64_t)sp.ctx + me.depth - t0);   // distance to the first one's token
    const float sc = kCap ? 1.f : a.scale_log2;
    const bool drafts = me.depths != nullptr && t0 + 32 > sp.ctx;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const int t = t0 + j;
      const float d = drafts && t >= sp.ctx && t < sp.te ? (float)(me.depth - depth_of(me, t - sp.ctx))
                                                         : d0 - (float)j;
      v[j] = __float_as_uint(fmaf(-sp.slope2, d, __uint_as_float(v[j]) * sc));
    }
  }
  hide32(vis, -CUDART_INF_F, v);
}

// Weights 2^(v sc + b + j step) of 32 scores (plain: 2^v): P in 16 words at
// p_addr, their sum into ps.
template <bool kStep, bool kPlain = false>
__device__ __forceinline__ void weights32(const uint32_t (&v)[32], float sc, float b, float step, uint32_t p_addr,
                                          F2 (&ps)[2]) {
  uint32_t pw[16];
  const F2 sc2 = f2(sc, sc), b2 = f2(b, b), st2 = f2(step, step);
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const F2 at = kStep ? fma2(st2, f2((float)(2 * j), (float)(2 * j + 1)), b2) : b2;
    float x0, x1;
    split(kPlain ? f2(v[2 * j], v[2 * j + 1]) : fma2(f2(v[2 * j], v[2 * j + 1]), sc2, at), x0, x1);
    const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
    pw[j] = pack_bf16(p0, p1);
    ps[j & 1] = add2(ps[j & 1], f2(p0, p1));
  }
  tmem_st16(p_addr, pw);
}

// How the softmax warps share the rounds.  Where a CTA has many: four warps take
// the even ones, four the odd ones, so that the two of a scheduler are at
// different places and one's exponentials run beside the other's copies and waits
// (16 x 61 drafts of 64 heads 133 -> 124 us, capped pieces of prompts 128 -> 118).
// Where it has few (kHalves): all eight take every round, a half of its columns
// each, which is over sooner (a request of one round a CTA 9.7 -> 9.1 us).  With
// slopes always so: the base moves on with every round of a start (39.5 -> 35.6).
constexpr int kStreamRounds = 4;

// An e4m3 cache: K and V arrive as they are, in tiles of 16 tokens [16][128 B] and
// two rounds of each, and the producers' warps widen them to bf16 (exact) into rings
// of two rounds: the same 192 KB.
constexpr int kNarrowBytes = kRoundTok * kHeadDim;   // K or V of a round
// Three warps widen K, three V: the producer and two of a fourth warpgroup (64 ragged
// requests x 16 drafts 324 us with the producers alone, 175 so; 157 over bf16, 145 if
// nothing were widened).  128 registers each then, which spills a few words.
constexpr int kWideners = 3;
constexpr int kThreadsFp8 = kTcThreads + 128;

__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ void sts16(uint32_t at, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// Tiles first, first + step, ... of a round from e4m3 (chunk c of 16 bytes of token t
// holds dims 16 (c ^ (t & 7)) on, as the copy swizzles them) to bf16 as the products
// want them.  8 lanes take a token; those of one half of its dims write their second
// piece first, so that the 8 pieces written at a time lie in different banks.  Bound by
// the conversions, so the tiles are dealt out such that each scheduler's warps have as
// many.  (Integer operations and a product by 2^120 were slower the more values they
// took: 181 us with none, 193, 200, 207 and 212 with a quarter, half, three quarters and
// all.)  Not inlined: unrolled in two places, the whole kernel waited for instructions.
__device__ __noinline__ void widen_round(const uint8_t* narrow, uint8_t* wide, int tiles, int first, int step,
                                         int lane) {
  uint32_t from[2], to[2][2];   // of tokens x and x + 4 of 8
  bool turn[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int x = (lane >> 3) + 4 * u, q = (lane & 7) ^ x, piece = (q & 3) * 2;
    turn[u] = q >= 4;
    from[u] = smem_u32(narrow) + x * kHeadDim + (lane & 7) * 16;
    const uint32_t row = smem_u32(wide) + (q >> 2) * 1024 + x * 128;
    to[u][0] = row + ((piece + (q >> 2)) ^ x) * 16;
    to[u][1] = row + ((piece + 1 - (q >> 2)) ^ x) * 16;
  }
#pragma unroll 1
  for (int tile = first; tile < tiles; tile += step) {
    uint4 v[4];   // tokens x, x + 4, x + 8, x + 12
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = lds16(from[u & 1] + tile * 16 * kHeadDim + (u >> 1) * 8 * kHeadDim);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool t = turn[u & 1];   // the piece to write first
      const uint4 x = t ? make_uint4(v[u].z, v[u].w, v[u].x, v[u].y) : v[u];
      const uint32_t at = tile * kTileBytes + (u >> 1) * 2048;
      sts16(to[u & 1][0] + at, make_uint4(widen2(x.x), widen2(x.x >> 16), widen2(x.y), widen2(x.y >> 16)));
      sts16(to[u & 1][1] + at, make_uint4(widen2(x.z), widen2(x.z >> 16), widen2(x.w), widen2(x.w >> 16)));
    }
  }
}

struct TreeSmem {
  float base[kTreeRows];      // a row's exponent base, as the last round left it
  float swap[2][2][kTreeRows];   // exchanges of the warps of a quadrant: place, half, row
  uint64_t ready[2][4];       // base written by the stream's warp of a quadrant
  uint64_t narrow[2][2];      // K's, V's two rounds of an e4m3 cache landed,
  uint64_t widened[2][2];     // and read by the wideners beside the producer
  int stop[2];                // the abort flag, and the count of slow_wait
};
constexpr int kSmemBytes = kQBytes + kTcStages * kStageBytes + (int)sizeof(TcSmem) + (int)sizeof(TreeSmem);
static_assert(kSmemBytes <= 227 * 1024 && sizeof(TcSmem) % 4 == 0, "dynamic shared memory of one CTA");

template <bool kCap, bool kSlopes, bool kHalves, bool kFp8>
__global__ void __launch_bounds__(kFp8 ? kThreadsFp8 : kTcThreads, 1) tree_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int kStages = kFp8 ? 2 : kTcStages;   // rounds of K, and of V, that the products read
  extern __shared__ __align__(1024) uint8_t smem[];
  if (!schedule_ready(a.sched + H_EPOCH, a.wait_epoch, a.err)) return;
  pdl_launch_dependents();
  const bool chain = a.sched[H_CAUSAL] != 0;
  // a captured launch under a later plan that its tensors do not fit (and, never
  // seen, shared memory that the swizzle could not use)
  if (a.sched[H_BATCH] > a.tokens || (!chain && a.sched[H_MAXQ] > 32 * (int64_t)a.mask_words) ||
      (smem_u32(smem) & 1023) != 0) {
    if (threadIdx.x == 0) atomicOr(a.err, PKD_DEV_ERR_BOUNDS);
    pdl_wait();
    return;
  }
  uint8_t* sQ = smem;
  uint8_t* stages = smem + kQBytes;
  TcSmem* sh = reinterpret_cast<TcSmem*>(stages + kTcStages * kStageBytes);
  TreeSmem* more = reinterpret_cast<TreeSmem*>(sh + 1);
  volatile int* abort_flag = more->stop;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int it0 = a.sched[a.off_cta + blockIdx.x];
  const int it1 = a.sched[a.off_cta + blockIdx.x + 1];
  if (it0 >= it1) {
    pdl_wait();
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sh->fullk[s], kFp8 ? kWideners : 1);
      mbar_init(&sh->emptyk[s], 1);
      mbar_init(&sh->fullv[s], kFp8 ? kWideners : 1);
      mbar_init(&sh->emptyv[s], 1);
    }
    mbar_init(&sh->qfull, 1);
    mbar_init(&sh->qfree, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh->sfull[b], 1);
      mbar_init(&sh->sfree[b], kHalves ? kSoftmaxWarps : kSoftmaxWarps / 2);
      mbar_init(&sh->pfull[b], kHalves ? kSoftmaxWarps : kSoftmaxWarps / 2);
      mbar_init(&sh->pfree[b], 1);
      for (int q = 0; q < 4; ++q) mbar_init(&more->ready[b][q], 1);
      for (int c = 0; c < 2; ++c) {
        mbar_init(&more->narrow[c][b], 1);
        mbar_init(&more->widened[c][b], kWideners - 1);
      }
    }
    mbar_init(&sh->ofree, kSoftmaxWarps);
    mbar_init(&sh->fin, 2);
    more->stop[0] = more->stop[1] = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == 32) {
    prefetch_map(&a.q_map);
    prefetch_map(&a.kv_map);
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sh->tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  const int P = a.page_size;
  const int g = a.hq / a.hkv;
  const int tile_tokens = kTreeRows / g;
  const int32_t* requests = a.sched + request_words(a.off_pages, a.sched[H_NNZ]);

  if (warp == kWarpK || warp == kWarpV) {
    // ------------------------------------------- producers (queries, K; V)
    const int c = warp == kWarpK ? 0 : 1;
    uint64_t* full = c ? sh->fullv : sh->fullk;
    uint64_t* empty = c ? sh->emptyv : sh->emptyk;
    uint8_t* ring = stages + (size_t)c * kStages * kKvBytes;
    const bool me = elect_one();
    const int step_pages = kRoundTok / P, step_at = kRoundTok % P;
    const uint64_t first = l2_evict_first_policy(), normal = l2_evict_normal_policy();
    // The queue's rounds, one after the other: `next_it`, round `next_k` of it.  Lane j
    // < 8 copies the round's tile j (its first token is a multiple of 16), which lies on
    // page `at_page` of the request, from token `next_at` of it on; they move on by one
    // round each time (a division takes as long as two copies), and the page ids
    // (`next`) are on their way a round ahead.
    int next_it = it0, next_k = 0, nr = 0, from = 0, to = 0, head = 0, q_row = 0;
    int tile = 0, ntiles = 0, at_page = 0, next_at = 0, next = 0;
    const int32_t* pages = nullptr;
    uint64_t policy = first;
    auto enter = [&]() {
      const int32_t* item = a.sched + a.off_items + (int64_t)next_it * kItemWords;
      const int32_t* entry = requests + item[0] * kRequestWords;
      from = item[1];
      to = item[2];
      head = item[7];
      q_row = entry[0] + item[5];
      // (more than one row block reads these tokens: they may stay in L2)
      policy = entry[1] > tile_tokens ? normal : first;
      pages = a.sched + a.off_pages + entry[3];
      nr = rounds_of(from, to);
      ntiles = (to - from + 15) >> 4;
      tile = kRoundTiles * round_at<kSlopes>(0, nr) + (lane & (kRoundTiles - 1));
      at_page = (from + 16 * tile) / P;
      next_at = (from + 16 * tile) % P;
      next = tile < ntiles ? pages[at_page] : 0;
    };
    auto issue = [&](uint8_t* dst, uint64_t* bar) {
      int page = next;
      const int at = next_at;
      const int nbox = (min(kRoundTok, to - from - kRoundTok * round_at<kSlopes>(next_k, nr)) + 15) >> 4;
      if (next_k + 1 < nr) {
        tile += kSlopes ? -kRoundTiles : kRoundTiles;
        at_page += kSlopes ? -step_pages : step_pages;
        next_at += kSlopes ? -step_at : step_at;
        if (!kSlopes && next_at >= P) {
          next_at -= P;
          ++at_page;
        }
        if (kSlopes && next_at < 0) {
          next_at += P;
          --at_page;
        }
        next = tile < ntiles ? pages[at_page] : 0;
      }
      if ((unsigned)page >= (unsigned)a.num_pages) {
        atomicOr(a.err, PKD_DEV_ERR_BOUNDS);
        page = 0;
      }
      const int place = kFp8 ? at : head * a.head_group + (at >> 3), row = 2 * page + c;
      int places[kRoundTiles], rows[kRoundTiles];
#pragma unroll
      for (int u = 0; u < kRoundTiles; ++u) {
        places[u] = __shfl_sync(kFull, place, u);
        rows[u] = __shfl_sync(kFull, row, u);
      }
      constexpr int kBytes = kFp8 ? 16 * kHeadDim : kTileBytes;
      if (me) {
        mbar_arrive_expect_tx(bar, (uint32_t)(nbox * kBytes));
#pragma unroll
        for (int u = 0; u < kRoundTiles; ++u)
          if (u < nbox) {
            if (kFp8)
              tensor_copy_g2s(dst + u * kBytes, &a.kv_map, 0, places[u], 0, head, rows[u], bar, policy);
            else
              tensor_copy_g2s(dst + u * kBytes, &a.kv_map, 0, 0, head * a.head_half, places[u], rows[u], bar, policy);
          }
      }
      __syncwarp();
      if (++next_k == nr) {
        next_k = 0;
        if (++next_it < it1) enter();
      }
    };
    int st = 0, nq = 0, issued = 0;
    bool ok = true;
    uint8_t* narrow = stages + 2 * kStages * kKvBytes + c * 2 * kNarrowBytes;   // (an e4m3 cache's)
    enter();
    pdl_wait();   // q and the cache may come from the previous kernel
    for (; kFp8 && issued < 2 && next_it < it1; ++issued)
      issue(narrow + issued * kNarrowBytes, &more->narrow[c][issued]);
    for (int it = it0; it < it1 && ok; ++it) {
      const int32_t* item = a.sched + a.off_items + (int64_t)it * kItemWords;
      // (without narrow rounds ahead, the queue's next round is this item's first)
      const int tb = kFp8 ? item[1] : from, te = kFp8 ? item[2] : to, rounds = rounds_of(tb, te);
      // the item's queries (the previous item's score MMAs must be done)
      if (c == 0 && it > it0 &&
          !warp_wait(&sh->qfree, (uint32_t)((it - it0 - 1) & 1), abort_flag, a.err, lane)) {
        ok = false;
        break;
      }
      if (c == 0) ++nq;
      if (c == 0 && me) {
        const int row0 = kFp8 ? requests[item[0] * kRequestWords] + item[5] : q_row;
        mbar_arrive_expect_tx(&sh->qfull, (uint32_t)kQBytes);
        for (int h = 0; h < 2; ++h)
          tensor_copy_g2s(sQ + h * (kQBytes / 2), &a.q_map, 0, h, 0, kFp8 ? item[7] : head, row0, &sh->qfull,
                          first);
      }
      __syncwarp();
      for (int k = 0; k < rounds; ++k, ++st) {
        const int slot = st % kStages;
        const uint32_t round = (uint32_t)(st / kStages);
        uint8_t* dst = ring + (size_t)slot * kKvBytes;
        if (round > 0 && !warp_wait(&empty[slot], (round - 1) & 1u, abort_flag, a.err, lane)) {
          ok = false;
          break;
        }
        if constexpr (kFp8) {
          const int buf = st & 1;
          if (!warp_wait(&more->narrow[c][buf], (uint32_t)((st >> 1) & 1), abort_flag, a.err, lane)) {
            ok = false;
            break;
          }
          const int tiles = (min(kRoundTok, te - tb - kRoundTok * round_at<kSlopes>(k, rounds)) + 15) >> 4;
          widen_round(narrow + buf * kNarrowBytes, dst, tiles, 1, 4, lane);
          fence_proxy_async_smem();   // before the products' reads, and the next copy here
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[slot]);
          if (next_it < it1) {
            if (!warp_wait(&more->widened[c][buf], (uint32_t)((st >> 1) & 1), abort_flag, a.err, lane)) {
              ok = false;
              break;
            }
            issue(narrow + buf * kNarrowBytes, &more->narrow[c][buf]);
            ++issued;
          }
        } else {
          issue(dst, &full[slot]);
        }
      }
    }
    // drain: the last phase of every slot, and the last queries
    if (lane == 0) {
      for (int s = 0; !kFp8 && s < kStages; ++s)
        if (st > s && !mbar_wait(&full[s], (uint32_t)(((st - 1 - s) / kStages) & 1), nullptr))
          atomicOr(a.err, PKD_DEV_ERR_TIMEOUT);
      for (int s = st; kFp8 && s < issued; ++s)
        if (!mbar_wait(&more->narrow[c][s & 1], (uint32_t)((s >> 1) & 1), nullptr))
          atomicOr(a.err, PKD_DEV_ERR_TIMEOUT);
      if (nq > 0 && !mbar_wait(&sh->qfull, (uint32_t)((nq - 1) & 1), nullptr))
        atomicOr(a.err, PKD_DEV_ERR_TIMEOUT);
    }
  } else if (kFp8 && warp >= kTcThreads / 32) {
    // ------------------------------------- more wideners (two of K, two of V)
    // (odd warps have no producer beside them: half of the tiles, the others a quarter)
    const int c = (warp - kTcThreads / 32) >> 1, tile0 = warp & 1 ? 0 : 3, step = warp & 1 ? 2 : 4;
    uint64_t* full = c ? sh->fullv : sh->fullk;
    uint64_t* empty = c ? sh->emptyv : sh->emptyk;
    uint8_t* ring = stages + (size_t)c * kStages * kKvBytes;
    const uint8_t* narrow = stages + 2 * kStages * kKvBytes + c * 2 * kNarrowBytes;
    int st = 0;
    bool ok = true;
    for (int it = it0; it < it1 && ok; ++it) {
      const int32_t* item = a.sched + a.off_items + (int64_t)it * kItemWords;
      const int tb = item[1], te = item[2], rounds = rounds_of(tb, te);
      for (int k = 0; k < rounds; ++k, ++st) {
        const int slot = st % kStages, buf = st & 1;
        const uint32_t round = (uint32_t)(st / kStages);
        if ((round > 0 && !warp_wait(&empty[slot], (round - 1) & 1u, abort_flag, a.err, lane)) ||
            !warp_wait(&more->narrow[c][buf], (uint32_t)((st >> 1) & 1), abort_flag, a.err, lane)) {
          ok = false;
          break;
        }
        const int tiles = (min(kRoundTok, te - tb - kRoundTok * round_at<kSlopes>(k, rounds)) + 15) >> 4;
        widen_round(narrow + buf * kNarrowBytes, ring + (size_t)slot * kKvBytes, tiles, tile0, step, lane);
        fence_proxy_async_smem();   // before the products' reads, and the next copy there
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[slot]);
        if (lane == 0) mbar_arrive(&more->widened[c][buf]);
      }
    }
  } else if (warp == kWarpS) {
    // ------------------------------------------- S = Q K^T (lane 0 issues)
    const bool me = elect_one();
    const uint64_t q0 = smem_desc(smem_u32(sQ), 16, 1024), k0 = smem_desc(smem_u32(stages), 16, 2048);
    int r = 0;
    bool ok = true;
    for (int it = it0; it < it1 && ok; ++it) {
      const int32_t* item = a.sched + a.off_items + (int64_t)it * kItemWords;
      const int tb = item[1], te = item[2];
      const int nr = rounds_of(tb, te);
      if (!warp_wait(&sh->qfull, (uint32_t)((it - it0) & 1), abort_flag, a.err, lane)) {
        ok = false;
        break;
      }
      for (int k = 0; k < nr; ++k, ++r) {
        const int slot = r % kStages, b = r & 1;
        // (the wait that is over first, first: one that is over still takes its time)
        if (!warp_wait(&sh->fullk[slot], (uint32_t)((r / kStages) & 1), abort_flag, a.err, lane) ||
            (r >= 2 &&
             !warp_wait(&sh->sfree[b], (uint32_t)(((r >> 1) - 1) & 1), abort_flag, a.err, lane))) {
          ok = false;
          break;
        }
        const int n = min(kRoundTok, te - (tb + round_at<kSlopes>(k, nr) * kRoundTok));
        const uint32_t idesc_s = mma_idesc(kDenseRows, 16 * ((n + 15) >> 4), 0);
        if (me) {
          tc_fence_after();
          const uint64_t ks = k0 + (uint64_t)(slot * (kKvBytes >> 4));
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ss(tmem + kColS + kSCols * b, q0 + (uint64_t)((kk >> 2) * (kQBytes / 2 >> 4) + (kk & 3) * 2),
                   ks + (uint64_t)((kk >> 2) * (1024 >> 4) + (kk & 3) * 2), idesc_s, kk > 0);
          mma_commit(&sh->sfull[b]);
          mma_commit(&sh->emptyk[slot]);
          if (k == nr - 1) mma_commit(&sh->qfree);   // the item's last score MMA
        }
        __syncwarp();
      }
    }
    if (me) {
      mma_commit(&sh->fin);
      if (!mbar_wait(&sh->fin, 0, nullptr)) atomicOr(a.err, PKD_DEV_ERR_TIMEOUT);
    }
    __syncwarp();
  } else if (warp == kWarpPV) {
    // --------------------------------------------- O += P V (lane 0 issues)
    const bool me = elect_one();
    const uint32_t idesc_o = mma_idesc(kDenseRows, kHeadDim, 1);
    const uint64_t v0 = smem_desc(smem_u32(stages) + kStages * kKvBytes, 1024, 2048);
    int r = 0;
    bool ok = true;
    for (int it = it0; it < it1 && ok; ++it) {
      const int32_t* item = a.sched + a.off_items + (int64_t)it * kItemWords;
      const int tb = item[1], te = item[2];
      const int nr = rounds_of(tb, te);
      for (int k = 0; k < nr; ++k, ++r) {
        const int slot = r % kStages, b = r & 1;
        if (!warp_wait(&sh->fullv[slot], (uint32_t)((r / kStages) & 1), abort_flag, a.err, lane) ||
            (k == 0 && it > it0 &&
             !warp_wait(&sh->ofree, (uint32_t)((it - it0 - 1) & 1), abort_flag, a.err, lane))) {
          ok = false;
          break;
        }
        const int n = min(kRoundTok, te - (tb + round_at<kSlopes>(k, nr) * kRoundTok));
        const int nbox = (n + 15) >> 4;
        uint8_t* vbase = stages + (size_t)(kStages + slot) * kKvBytes;
        if (n & 15) {
          // slots past the range's end in the last tile: P is 0 there, but
          // 0 x NaN would poison O, so zero those V rows (both halves)
          const int past = n & 15;
          uint8_t* tile = vbase + (nbox - 1) * kTileBytes;
          for (int i = lane; i < 2 * (16 - past) * 8; i += 32) {
            const int h = i / ((16 - past) * 8), rem = i % ((16 - past) * 8);
            const int row = past + rem / 8, chunk = rem % 8;
            *reinterpret_cast<uint4*>(tile + (row >> 3) * 2048 + h * 1024 + (row & 7) * 128 + chunk * 16) =
                make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (!warp_wait(&sh->pfull[b], (uint32_t)((r >> 1) & 1), abort_flag, a.err, lane)) {
          ok = false;
          break;
        }
        if (me) {
          tc_fence_after();
          const uint64_t vs = v0 + (uint64_t)(slot * (kKvBytes >> 4));
#pragma unroll
          for (int j = 0; j < kRoundTiles; ++j)
            if (j < nbox)
              mma_ts(tmem + kColO, tmem + kColP + kPCols * b + 8 * j, vs + (uint64_t)(j * (kTileBytes >> 4)),
                     idesc_o, k > 0 || j > 0);
          mma_commit(&sh->pfree[b]);
          mma_commit(&sh->emptyv[slot]);
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
    // ------------------------------------------------- softmax + epilogue
    const int quad = warp & 3, stream = warp >> 2;   // lane quadrant; parity of its rounds
    const int row = quad * 32 + lane;               // tile row = tensor-memory lane
    const uint32_t tq = tmem + ((uint32_t)(quad * 32) << 16);   // this quadrant's lanes
    const int window = a.sched[H_WINDOW];
    pdl_wait();   // outputs, mask and depths may belong to the previous kernel
    int rho = 0;
    uint32_t swaps = 0;   // exchanges with the partner warp so far
    uint32_t seen = 0;    // bases that the partner warp has handed over in the items before
    bool ok = true;
    auto pv_wait = [&](int r) -> bool {
      if (r < 0) return true;
      return warp_wait(&sh->pfree[r & 1], (uint32_t)((r >> 1) & 1), abort_flag, a.err, lane);
    };
    // One float per row with the partner warp of this quadrant, through shared
    // memory: two places in turn (the partner has read one before it comes to the
    // next exchange, and that is over before this warp writes there again).  The
    // two warps meet at a barrier of their own, in a third of an mbarrier's time.
    // A warp whose wait ran out has raised the abort flag and arrives there once
    // more (below): a partner that waits goes on, and stops at the flag.
    auto exchange = [&](float v, float* other) -> bool {
      if (*abort_flag) return false;
      more->swap[swaps & 1u][stream][row] = v;
      asm volatile("barrier.sync %0, 64;" ::"r"(1 + quad) : "memory");
      *other = more->swap[swaps & 1u][stream ^ 1][row];
      ++swaps;
      return true;
    };
    for (int it = it0; it < it1 && ok; ++it) {
      const int32_t* item = a.sched + a.off_items + (int64_t)it * kItemWords;
      const int tb = item[1], te = item[2], dst = item[3], n_tok = item[4], i0 = item[5];
      const int stride = item[6], head = item[7];
      const int32_t* entry = requests + item[0] * kRequestWords;
      const int q_first = entry[0], drafts = entry[1], ctx = entry[2], first_page = entry[3];
      const int nr = rounds_of(tb, te);
      const int r0 = rho;
      rho = r0 + nr;
      // this warp's rounds k0, k0 + kBy, ... of the item
      constexpr int kBy = kHalves ? 1 : 2;
      const int k0 = kHalves ? 0 : (r0 ^ stream) & 1;
      if (quad * 32 >= n_tok * g) {
        // no row of this quadrant: keep the barriers' count, in their order
        for (int r = r0 + k0; r < rho && ok; r += kBy) {
          ok = warp_wait(&sh->sfull[r & 1], (uint32_t)((r >> 1) & 1), abort_flag, a.err, lane);
          if (!ok) break;
          if (lane == 0) mbar_arrive(&sh->sfree[r & 1]);
          ok = pv_wait(r - 2);
          if (ok && lane == 0) mbar_arrive(&sh->pfull[r & 1]);
        }
        ok = ok && pv_wait(rho - 2) && pv_wait(rho - 1);
        if (ok && lane == 0) mbar_arrive(&sh->ofree);
        continue;
      }
      const int i = row / g, hq = head * g + row % g;
      const bool valid = i < n_tok;
      Row me;
      me.ctx = ctx;
      me.drafts = drafts;
      me.i = i0 + i;
      me.words = a.mask_words;
      me.mask = chain || !valid ? nullptr : a.mask + (int64_t)(q_first + me.i) * a.mask_words;
      me.depths = chain || a.depths == nullptr ? nullptr : a.depths + q_first;
      me.depth = valid ? depth_of(me, me.i) : 0;
      me.window = window;
      // (64 bits: a depth may be any int32)
      me.first_seen = window > 0 ? (int)max((int64_t)-1, min((int64_t)0x7fffffff,
                                            (int64_t)ctx + me.depth - window + 1))
                                 : -1;
      Span sp;
      sp.ctx = ctx;
      sp.te = te;
      sp.reach = valid ? me.first_seen : -1;
      if (window > 0) sp.reach = __reduce_max_sync(kFull, sp.reach);
      sp.slope2 = kSlopes && valid ? a.slopes[hq] * kLog2e : 0.f;
      sp.steep = kSlopes && __any_sync(kFull, fabsf(sp.slope2) > kSteepest);
      // Capped scores lie between -cap and cap: with the base 0 no weight or sum
      // leaves fp32's (and bf16's) range, and the largest need not be known.  Not
      // for rows that see few tokens: with their largest as the base the weights
      // that count most are powers of 2, or near them, and lose little as P.
      const bool fixed = kCap && !kSlopes && a.cap_log2 <= kFixedBase &&
                         min(te, ctx) - max(tb, sp.reach) >= kFixedTokens;
      // the row's base when this warp last saw it, and the sum of its weights under it
      float m_used = fixed ? 0.f : -CUDART_INF_F, l = 0.f;
      for (int k = k0; k < nr && ok; k += kBy) {
        const int r = r0 + k, b = kHalves ? r & 1 : stream;
        const uint32_t s_col = tq + kColS + kSCols * b, p_col = tq + kColP + kPCols * b;
        if (!warp_wait(&sh->sfull[b], (uint32_t)((r >> 1) & 1), abort_flag, a.err, lane)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // Halves: this warp's 64 columns, once.  Else 0-63 for their largest score,
        // 64-127 for theirs and, once the base is known, their weights, then 0-63
        // again for theirs: a lane's 128 scores do not fit its registers.  (A fixed
        // base: 64-127, 0-63.)
        const int last = kHalves ? 1 : 2;
        float mx = -CUDART_INF_F;
        F2 ps[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll 1
        for (int pass = fixed || kHalves ? 1 : 0; pass <= last; ++pass) {
          const int h = kHalves ? stream : pass & 1;
          const int t0 = tb + round_at<kSlopes>(k, nr) * kRoundTok + 64 * h;   // token of the first column
          // does some row of the warp not see all of the 64 columns (or want each
          // score's own bias)?
          const bool special = t0 + 64 > ctx || t0 < sp.reach || te - t0 < 64 || (kSlopes && sp.steep);
          uint32_t sv[2][32];
          tmem_ld32(s_col + 64 * h, sv[0]);
          tmem_ld32(s_col + 64 * h + 32, sv[1]);
          tmem_wait_ld();
          float sc = a.scale_log2, step = 0.f;
          if constexpr (kCap) {
            // (where some columns hold no token of this run, or one that no row sees;
            // a draft that some rows do not see is this run's all the same)
            if (te - t0 < 64 || t0 < sp.reach) {
              const uint64_t live = valid ? visible(me, t0, te) : 0u;
              hide32((uint32_t)live, 0.f, sv[0]);
              hide32((uint32_t)(live >> 32), 0.f, sv[1]);
            }
            cap64(a, valid, s_col + 64 * h, sv);
            sc = 1.f;
          }
          if (pass == last) {   // S is read: the buffer may be refilled
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->sfree[b]);
          }
          if (special) {
            const uint64_t vis = valid ? visible(me, t0, te) : 0u;
            shape32<kCap, kSlopes>(a, me, sp, t0, (uint32_t)vis, sv[0]);
            shape32<kCap, kSlopes>(a, me, sp, t0 + 32, (uint32_t)(vis >> 32), sv[1]);
            if (kSlopes) sc = 1.f;
          } else if (kSlopes) {
            step = sp.slope2;
          }
          const float far = kSlopes && !special ? -step * (float)((int64_t)ctx + me.depth - t0) : 0.f;
          if (!fixed && pass < 2) {
            if (kSlopes && !special) {
              // the largest product of 32 and their largest bias bound their scores
              for (int q = 0; q < 2; ++q)
                mx = fmaxf(mx, fmaf(max32(sv[q], -CUDART_INF_F), sc,
                                    far + fmaxf(step * (32 * q), step * (32 * q + 31))));
            } else {
              mx = fmaxf(mx, fmaxf(max32(sv[0], -CUDART_INF_F), max32(sv[1], -CUDART_INF_F)) * sc);   // (sc > 0)
            }
          }
          if (pass == 0) continue;
          if (pass == 1) {
            // (P's buffer was read by the P.V products of round r - 2)
            if (!pv_wait(r - 2)) {
              ok = false;
              break;
            }
            if (!fixed) {
              // The base is raised, and O rescaled, only past 2^8 of growth (per row;
              // the waits and tensor-memory accesses are the whole warp's).  Without
              // halves it goes from round to round, that is, from stream to stream.
              float m_old = m_used;
              if (kHalves) {
                float m_other;
                if (!exchange(mx, &m_other)) {
                  ok = false;
                  break;
                }
                mx = fmaxf(mx, m_other);
              } else if (k > 0) {
                if (!warp_wait(&more->ready[stream ^ 1][quad], (seen + ((k - 1) >> 1)) & 1u, abort_flag,
                               a.err, lane)) {
                  ok = false;
                  break;
                }
                m_old = more->base[row];
              }
              const bool need = mx > m_old + kRescaleLog2;
              const float m_new = need ? mx : m_old;
              if (!kHalves) {
                more->base[row] = m_new;
                __syncwarp();
                if (lane == 0) mbar_arrive(&more->ready[stream][quad]);
              }
              if (m_new != m_used) l *= exp2f(m_used - m_new);   // (0 while m_used = -inf)
              m_used = m_new;
              if (k > 0 && __any_sync(kFull, need)) {
                const float alpha = need ? exp2f(m_old - mx) : 1.f;
                if (!pv_wait(r - 1)) {
                  ok = false;
                  break;
                }
                tc_fence_after();
#pragma unroll 1
                for (int cb = kHalves ? 64 * h : 0; cb < (kHalves ? 64 * h + 64 : kHeadDim); cb += 16) {
                  uint32_t o[16];
                  tmem_ld16(tq + kColO + cb, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                  tmem_st16(tq + kColO + cb, o);
                }
                tmem_wait_st();
              }
            }
          }
          if (fixed) {
            weights32<false, true>(sv[0], 1.f, 0.f, 0.f, p_col + 32 * h, ps);
            weights32<false, true>(sv[1], 1.f, 0.f, 0.f, p_col + 32 * h + 16, ps);
          } else {
            const float base = (m_used == -CUDART_INF_F ? 0.f : -m_used) + far;   // nothing seen yet: weights 0
            weights32<kSlopes>(sv[0], sc, base, step, p_col + 32 * h, ps);
            weights32<kSlopes>(sv[1], sc, kSlopes ? fmaf(step, 32.f, base) : base, step, p_col + 32 * h + 16, ps);
          }
        }
        if (!ok) break;
        float l0, l1;
        split(add2(ps[0], ps[1]), l0, l1);
        l += l0 + l1;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->pfull[b]);
      }
      if (!ok) break;
      if (!kHalves && !fixed) seen += (uint32_t)((nr - (k0 ^ 1) + 1) >> 1);   // the partner's rounds
      // ---- epilogue: the item's P.V MMAs done (rounds in order; lag <= 1)
      const int rl = rho - 1;
      if (!pv_wait(rl - 1) || !pv_wait(rl)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // the row's base (it only rises) and its sum, of both warps' in their order
      float m_other = m_used, l_other;
      if (!kHalves && !exchange(m_used, &m_other)) {
        ok = false;
        break;
      }
      if (m_other > m_used) {
        l *= exp2f(m_used - m_other);
        m_used = m_other;
      }
      if (!exchange(l, &l_other)) {
        ok = false;
        break;
      }
      const float lt = stream == 0 ? l + l_other : l_other + l;
      const int64_t q_row = (int64_t)(q_first + i0 + i) * a.hq + hq;
      const int64_t p_row = ((int64_t)dst + (int64_t)i * stride) * a.hq + hq;   // its partial state
      // (not v_scale / lt: with a fixed base the sum may lie near either end of fp32's range)
      const float inv = lt == 0.f ? 0.f : 1.f / lt;
      // 32 dims of the row's result from cb on
      const auto store = [&](int cb, const uint32_t* o) {
        if (dst < 0) {
          uint16_t* op = a.out + q_row * kHeadDim + cb;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
              w[j] = pack_bf16(__uint_as_float(o[16 * q + 2 * j]), __uint_as_float(o[16 * q + 2 * j + 1]));
            store32(op + 16 * q, w);
          }
        } else {
          float* op = a.o_part + p_row * kHeadDim + cb;
#pragma unroll
          for (int q = 0; q < 4; ++q) store32(op + 8 * q, o + 8 * q);
        }
      };
      bool odd = false;   // a value is not finite (a NaN sum: the scores')
#pragma unroll 1
      for (int cb = 64 * stream; cb < 64 * stream + 64; cb += 32) {
        uint32_t o[32];
        tmem_ld32(tq + kColO + cb, o);
        tmem_wait_ld();
        float bad = 0.f;   // NaN if a value is not finite
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float x = lt == 0.f ? 0.f : __uint_as_float(o[j]) * inv * a.v_scale;
          o[j] = __float_as_uint(x);
          bad = fmaf(x, 0.f, bad);
        }
        odd = odd || (bad != bad && lt > 0.f);
        if (valid) store(cb, o);
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->ofree);
      if (__any_sync(kFull, valid && odd)) {
        Redo in;
        in.row = me;
        in.mine = valid && odd;
        in.q = a.q + (valid ? q_row * kHeadDim : 0);
        in.first_page = first_page, in.head = head, in.tb = tb, in.te = te;
        in.dim0 = 64 * stream, in.lane = lane;
        in.total = m_used + log2f(lt), in.slope2 = sp.slope2;
        in.beats = abort_flag + 1;
        if (redo_rows<kFp8>(a, in))
          for (int c = 0; c < 64; c += 32) store(64 * stream + c, reinterpret_cast<const uint32_t*>(in.o + c));
      }
      if (valid && stream == 0) {
        const float lse = lt == 0.f ? -CUDART_INF_F : (m_used + log2f(lt)) * kLn2;
        if (dst >= 0)
          a.l_part[p_row] = lse;
        else if (a.lse != nullptr)
          a.lse[q_row] = lse;
      }
    }
    if (!ok) asm volatile("barrier.arrive %0, 64;" ::"r"(1 + quad) : "memory");
  }
  // all roles done: tensor memory is no longer read or written
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  }
}

template <bool kFp8>
const void* kernel_of(bool cap, bool slopes, bool halves) {
  if (slopes)
    return cap ? reinterpret_cast<const void*>(&tree_kernel<true, true, true, kFp8>)
               : reinterpret_cast<const void*>(&tree_kernel<false, true, true, kFp8>);
  if (halves)
    return cap ? reinterpret_cast<const void*>(&tree_kernel<true, false, true, kFp8>)
               : reinterpret_cast<const void*>(&tree_kernel<false, false, true, kFp8>);
  return cap ? reinterpret_cast<const void*>(&tree_kernel<true, false, false, kFp8>)
             : reinterpret_cast<const void*>(&tree_kernel<false, false, false, kFp8>);
}

}  // namespace

cudaError_t encode_tree_kv_map(const void* kv, int32_t num_pages, int32_t page_size, int32_t hkv,
                               bool hnd, CUtensorMap* map) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = map_encoder();
  if (encode == nullptr) return cudaErrorNotSupported;
  if (kv == nullptr || (uintptr_t)kv % 16 != 0 || page_size % 16 != 0 || num_pages < 1 ||
      hkv < 1 || hkv > kMaxKvHeads)
    return cudaErrorInvalidValue;
  const cuuint64_t head = (cuuint64_t)kHeadDim * 2, row = hkv * head, groups = page_size / 8;
  const cuuint64_t dims[5] = {64, 8, hnd ? 2 : 2 * (cuuint64_t)hkv, hnd ? hkv * groups : groups,
                              2 * (cuuint64_t)num_pages};
  const cuuint64_t token = hnd ? head : row;
  const cuuint64_t strides[4] = {token, 128, 8 * token, (cuuint64_t)page_size * row};
  const cuuint32_t box[5] = {64, 8, 2, 2, 1};
  const cuuint32_t elem_strides[5] = {1, 1, 1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(kv), dims,
                            strides, box, elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

int tree_smem_bytes() { return kSmemBytes; }

cudaError_t tree_prepare(bool fp8) {
  for (int k = 0; k < 8; ++k) {
    const void* f = fp8 ? kernel_of<true>(k & 1, k & 2, k & 4) : kernel_of<false>(k & 1, k & 2, k & 4);
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, tree_smem_bytes());
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t tree_occupancy(bool fp8, int* blocks_per_sm) {
  return cudaOccupancyMaxActiveBlocksPerMultiprocessor(
      blocks_per_sm, fp8 ? kernel_of<true>(false, false, false) : kernel_of<false>(false, false, false),
      fp8 ? kThreadsFp8 : kTcThreads, (size_t)tree_smem_bytes());
}

cudaError_t launch_tree(const TreeArgs& a, int grid, int64_t most_tokens, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(a.fp8 ? kThreadsFp8 : kTcThreads);
  cfg.dynamicSmemBytes = (size_t)tree_smem_bytes();
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {const_cast<TreeArgs*>(&a)};
  const bool cap = a.cap_log2 != 0.f, slopes = a.slopes != nullptr;
  const bool halves = most_tokens < kStreamRounds * kTreeRound;
  return cudaLaunchKernelExC(
      &cfg, a.fp8 ? kernel_of<true>(cap, slopes, halves) : kernel_of<false>(cap, slopes, halves), args);
}

}  // namespace pkd
