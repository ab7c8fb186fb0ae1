// The latent cache's decode and append (latent_kernel.cu): sizes, arguments
// and launchers.
#pragma once

#include <stdint.h>

#include <cuda.h>
#include <cuda_runtime_api.h>

namespace pkd {

constexpr int kLatentDim = 512;   // latent columns: the output's width
constexpr int kLatentRope = 64;   // rotary key columns behind them
constexpr int kLatentRow = kLatentDim + kLatentRope;
constexpr int kLatentMaxHeads = 128;

// Query heads that one work item covers: the products' columns, 16, 32 or
// 64 (the output of 64 heads, 512 dims each, fills half of tensor memory).
// More heads make ceil(heads / 64) blocks, each an item of its own.
__host__ __device__ constexpr int32_t latent_block_heads(int32_t heads) {
  return heads <= 16 ? 16 : heads <= 32 ? 32 : 64;
}
__host__ __device__ constexpr int32_t latent_blocks(int32_t heads) {
  return (heads + latent_block_heads(heads) - 1) / latent_block_heads(heads);
}

// Latent plans: an item's fixed cost (its queries, its first tile, its
// epilogue) in tokens, and the split floor: a part's state is 2 KB per head,
// written and read back, so many heads pay for finer parts.  Measured with
// floors of 128 / 256: one request of 517 tokens, 16 heads 5.0 / 5.8 us; one of
// 8,000, 128 heads 15.8 / 11.8; 8 of up to 2,000, 64 heads 11.1 / 10.1.
constexpr int kLatentAlpha = 128;
inline int64_t latent_min_chunk(int32_t heads) { return heads <= 32 ? 128 : 256; }

struct LatentArgs {
  const int32_t* sched;
  float* o_part;         // fp32 [slot][heads][512]
  float* l_part;         // fp32 [slot][heads] (natural log)
  int32_t* err;
  uint16_t* out;         // bf16 [batch][heads][512]
  float* lse;            // fp32 [batch][heads] or null
  int64_t off_cta, off_items, off_pages, off_units, off_merge;
  int32_t heads, blocks, page_size, num_pages;
  int32_t batch;         // requests of q, out and lse
  float scale_log2, v_scale;
  int32_t wait_epoch;
  CUtensorMap kv_map[2]; // the cache, 16-token boxes of either column region
  CUtensorMap q_map;     // the queries, a block's heads of 64 columns
};

int latent_smem_bytes(int32_t heads);
cudaError_t latent_prepare(int32_t heads);
cudaError_t latent_occupancy(int32_t heads, int* blocks_per_sm);
// Merge blocks for a plan of `units` split requests, at most `most`: blocks
// without a task would only keep the next kernel off their SMs.
int latent_merge_blocks(int32_t heads, int32_t units, int32_t most_slots, int most);
// The decode kernel and, with a merge grid, the merge of split requests (its
// tasks are the plan's, read on the device; any grid does them all).
// decode_done (or null) is recorded between the two.
cudaError_t launch_latent(const LatentArgs& a, int grid, int merge_grid, cudaEvent_t decode_done,
                          cudaStream_t stream);
cudaError_t encode_latent_map(const void* cache, int32_t num_pages, int32_t page_size, int region,
                              CUtensorMap* map);
cudaError_t encode_latent_q_map(const void* q, int32_t batch, int32_t heads, CUtensorMap* map);
cudaError_t launch_latent_append(const void* latent, int64_t latent_stride, const void* rope,
                                 int64_t rope_stride, const int32_t* batch_indices,
                                 const int32_t* positions, int32_t n, const int32_t* indptr,
                                 const int32_t* indices, int32_t num_indices,
                                 const int32_t* last_page_len, int32_t batch, void* cache,
                                 int32_t num_pages, int32_t page_size, int32_t* err,
                                 cudaStream_t stream);

}  // namespace pkd
