// The schedule layout of host plans (make_layout's, with room for the items of
// latent plans) and of contexts (with room for the requests' entries behind
// the page list, where they have them); and the latent planner.
#pragma once

#include "latent.h"
#include "pkd_internal.h"

namespace pkd {

// The entries that pkd_accumulate_weights cuts its work from: behind the page
// list's nnz words (rounded up to 4) one per request, and one more with the
// total: 16-token tiles of the requests before, index of the first page in the
// page list, tokens, 0.  Only contexts that can accumulate hold them; the
// host plans and the other contexts do without.
constexpr int kRequestWords = 4, kRequestTile = 16;
__host__ __device__ inline int64_t request_words(int64_t page_list, int64_t nnz) {
  return page_list + (nnz + 3) / 4 * 4;
}

inline bool is_latent(const pkd_config& c) { return (c.flags & PKD_FLAG_LATENT) != 0; }

inline Layout plan_layout(const pkd_config& c, int64_t n_cta) {
  if (!is_latent(c)) return make_layout(c, n_cta);
  // latent plans: an item per block of heads (plans beyond the clamp are
  // refused for want of items)
  pkd_config room = c;
  const int64_t blocks = latent_blocks(c.num_qo_heads), rows = blocks * c.max_batch;
  room.max_batch = (int32_t)(rows < 0x7fffffff ? rows : 0x7fffffff);
  Layout L = make_layout(room, n_cta);
  // A plan cuts at most once between two neighbouring stretches, of n_cta /
  // blocks in all, and k cuts leave a request in k + 1 <= 2 k parts; a part's
  // slot is one for all blocks of heads.  (Slots by items, as other plans need
  // them, were 2 to 11 times as many: 431 MB instead of 39 for 128 heads and
  // batches of up to 512.)
  const int64_t stretches = n_cta < blocks ? 1 : n_cta / blocks;
  L.max_slots = 2 * (stretches - 1);
  const size_t row = (size_t)L.max_slots * c.num_qo_heads * sizeof(float);
  L.l_part_byte = (size_t)align_up((int64_t)(L.o_part_byte + row * c.head_dim), 256);
  L.total_bytes = (size_t)align_up((int64_t)(L.l_part_byte + row), 256);
  return L;
}

inline bool has_requests(const pkd_config& c) {
  return (c.flags & (PKD_FLAG_SHARED_PREFIX | PKD_FLAG_CASCADE | PKD_FLAG_LATENT)) == 0;
}
// The layout of a context's workspace and staging: plan_layout's offsets, then
// the requests' entries where it has them.
inline Layout context_layout(const pkd_config& c, int64_t n_cta) {
  Layout L = plan_layout(c, n_cta);
  if (!has_requests(c)) return L;
  // what lies behind the schedule words moves along by whole 256 bytes
  L.words = request_words(L.page_list, c.max_num_pages) +
            (int64_t)kRequestWords * ((int64_t)c.max_batch + 1);
  const size_t more = ((size_t)L.words * 4 + 255) / 256 * 256 - L.err_byte;
  L.err_byte += more;
  L.o_part_byte += more;
  L.l_part_byte += more;
  L.total_bytes += more;
  return L;
}

// The entries of a table that a plan has accepted, behind the plan's words;
// returns the words up to their end.
int64_t write_requests(const Layout& L, int32_t page_size, const int32_t* indptr,
                       const int32_t* last, int32_t batch, int32_t* words);

// Plans of latent contexts (planner.cpp; plan_schedule_grouped calls it).
int plan_schedule_latent(const pkd_config& cfg, int32_t n_cta, const Layout& L,
                         const int32_t* indptr, const int32_t* indices, const int32_t* last,
                         int32_t batch, int32_t* words, pkd_plan_info* info);

}  // namespace pkd
