// Attention weights of cached tokens (weights_kernel.cu) and eviction by them
// (evict_kernel.cu): arguments and launchers.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

namespace pkd {

struct WeightsArgs {
  const int32_t* sched;
  int32_t* err;
  const uint16_t* q;          // bf16 [batch][Hq][128]
  const uint8_t* kv;
  const float* lse;           // fp32 [batch][Hq]
  float* weights;             // fp32 [num_pages][Hkv][P]
  int32_t* positions;         // int32 [num_pages][Hkv][P] or null
  const int32_t* new_tokens;  // [batch] or null
  const int32_t* seen;        // [batch] (with positions)
  int64_t off_pages;
  int64_t page_bytes, token_bytes, head_bytes;   // strides of K in the cache
  int32_t hq, hkv, page_size, page_shift, num_pages;   // page_shift: log2 of the size, or -1
  int32_t batch;              // requests of q, lse, new_tokens and seen
  float scale_log2;
  int32_t wait_epoch;
};
cudaError_t launch_weights(const WeightsArgs& a, bool fp8, int grid, cudaStream_t stream);

// log2 of a page size, -1 when it is no power of two
inline int32_t page_shift_of(int32_t page_size) {
  for (int32_t k = 0; k < 31; ++k)
    if (page_size == 1 << k) return k;
  return -1;
}

constexpr int kMaxEvictLayers = 128;
// Longest request of an eviction: its keys lie in the shared memory of a
// cluster of up to 8 blocks, 32,768 each.
constexpr int kEvictBlockTokens = 32768;
constexpr int kEvictMaxTokens = 8 * kEvictBlockTokens;
struct EvictArgs {
  const int32_t *indptr, *indices, *last, *seen;
  int32_t* err;
  int32_t layers, batch, num_indices, num_pages, page_size, hkv;
  int32_t budget, sinks, recent, per_head;
  int32_t max_len;
  int64_t page_bytes, token_bytes, head_bytes;   // strides in the cache
  int64_t v_bytes;                               // from a page's K block to its V block
  int32_t pieces;                                // 16-byte pieces of one head's row
  int32_t page_shift;                            // log2 of the page size, -1 if it has none
  int32_t splits;                                // blocks of the moving kernel per job
  uint32_t* bitmaps;                             // workspace: kept tokens per job
  void* kv[kMaxEvictLayers];
  float* weights[kMaxEvictLayers];
  int32_t* positions[kMaxEvictLayers];
};
// Workspace of a call: 0 when its blocks choose and move in one kernel.
size_t evict_workspace_bytes(int layers, int batch, int hkv, int per_head, int max_len, int budget);
cudaError_t launch_evict(EvictArgs& a, cudaStream_t stream);

}  // namespace pkd
