// Attention of drafted tokens over a paged cache (tree_kernel.cu): sizes,
// arguments and launchers.
#pragma once

#include <stdint.h>

#include <cuda.h>
#include <cuda_runtime_api.h>

#include "pkd_internal.h"

namespace pkd {

// Header words of tree plans, behind those of all plans (the rest are 0).
enum TreeHeaderWord {
  H_REQUESTS = H_EPOCH + 1,   // requests (H_BATCH counts their query tokens)
  H_CAUSAL,                   // 1: every request's tokens are a chain
  H_WINDOW,                   // the sliding window, 0 without
  H_MAXQ,                     // the most query tokens of a request
};
static_assert(H_MAXQ < H_WORDS, "header words");

constexpr int kTreeRows = 128;       // query rows of a tile: 128 / g tokens x g heads of a KV head
constexpr int kTreeRound = 128;      // tokens per round of the kernel; plans cut at multiples of it
// An item's fixed cost and the split floor, in tokens.  Measured with 512 / 128,
// 256 / 128, 1024 / 128 and 768 / 256: 24 ragged requests x 7 drafts with slopes
// 36.4, 38.3, 36.9 and 36.4 us; 16 x 61 drafts of 64 heads 123.6, 134.1, 123.5 and
// 123.4; one of 517 tokens 9.1, 9.0, 9.0 and 9.8.
constexpr int kTreeAlpha = 512;
constexpr int kTreeMinChunk = 128;
// Tokens that several row blocks read, in bytes, from which on L2 does not hold
// them from one block to the next, and what it is worth, in percent of a plan's
// span, that all such blocks stay together then.  Measured: 256 tokens behind
// 100,000, 64 heads 900 -> 586 us, 32 heads 469 -> 304; 4 x 100 drafts behind
// 30,000 302 -> 185; 2 x 200 behind 50,000 of 4 KV heads (184 MB) 224 as it is.
constexpr int64_t kTreeSharedBytes = 192ll << 20;
constexpr int kTreeSharedGain = 60;

// tanh(x) / x for |x| <= 0.4 as a polynomial of x^2, fitted for the least largest
// error (tanh within 7e-8, in fp32).
constexpr float kTanhFit0 = 0.9999999043749117f, kTanhFit1 = -0.33331390193300425f,
                kTanhFit2 = 0.13271438197786756f, kTanhFit3 = -0.04757281035736614f;
constexpr float kTanhFitTo = 0.16f;   // of x^2

struct TreeArgs {
  const int32_t* sched;
  float* o_part;            // fp32 [slot][Hq][128]
  float* l_part;            // fp32 [slot][Hq] (natural log)
  int32_t* err;
  const uint16_t* q;        // bf16 [tokens][Hq][128]
  const void* kv;           // the cache, bf16 or (fp8) e4m3
  uint16_t* out;            // bf16 [tokens][Hq][128]
  float* lse;               // fp32 [tokens][Hq] or null
  const uint32_t* mask;     // [tokens][mask_words] or null
  const int32_t* depths;    // [tokens] or null: the tokens' numbers in their request
  const float* slopes;      // [Hq] or null
  int64_t off_cta, off_items, off_pages;
  int64_t page_elems, token_elems, head_elems, v_elems;   // strides in the cache
  int32_t hq, hkv, page_size, num_pages, mask_words;
  int32_t tokens;           // rows of q, out and lse
  float scale_log2;         // scale * log2(e); with a cap: 2 scale / cap * log2(e)
  float cap_log2;           // cap * log2(e), 0 without
  // for products whose square is up to cap_bound: cap_log2 * tanh(scale / cap * x)
  // = x times this polynomial of x^2
  float cap_bound, cap_poly[4];
  float v_scale;            // of the values (that of the keys is in scale_log2)
  int32_t fp8;
  int32_t wait_epoch;
  int32_t head_half, head_group;   // where a head starts in kv_map
  CUtensorMap kv_map;       // boxes of 16 tokens of a KV head: [2 x 8 tokens][half][8][128 B]
  CUtensorMap q_map;        // boxes of a KV head's 128 query rows and one half
};

// The merge of a tree run, whose states may be empty (lse -inf).  A plan of more
// query tokens than out has rows, or of more in a request than the run's masks
// cover, is not merged.
struct TreeMergeArgs : MergeArgs {
  int32_t rows = 0;
  int64_t most = 0;
};
cudaError_t launch_merge_tree(const TreeMergeArgs& a, int grid, int32_t max_chunks, cudaStream_t stream);

// The map of a bf16 cache: boxes of 16 tokens of one KV head as [2 groups of 8
// tokens][half][8][128 bytes], so that both matrix products find a fixed stride
// between groups (2 KB) and between halves (1 KB).
cudaError_t encode_tree_kv_map(const void* kv, int32_t num_pages, int32_t page_size, int32_t hkv,
                               bool hnd, CUtensorMap* map);

int tree_smem_bytes();
cudaError_t tree_prepare(bool fp8);
cudaError_t tree_occupancy(bool fp8, int* blocks_per_sm);
// most_tokens: of a CTA, as planned (any plan may run under either choice of kernel)
cudaError_t launch_tree(const TreeArgs& a, int grid, int64_t most_tokens, cudaStream_t stream);

}  // namespace pkd
