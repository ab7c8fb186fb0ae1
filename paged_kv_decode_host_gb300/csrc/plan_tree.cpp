// Plans of tree contexts: every request has one or more query tokens, the
// last ones of its cached tokens.
//
// A row block is up to 128 / g of a request's query tokens (the 128 rows of a
// tile per KV head) with the range of cached tokens that any of them may see:
// a window leaves the tokens before it out, and in a chain the tokens behind a
// block's last one.  Blocks go, whole or cut, to groups of Hkv CTAs in equal
// shares, the cheaper of two ways: laid end to end and cut into equal stretches,
// or whole ones first (below).  The CTAs of a group walk the same tokens at the
// same time, one KV head each: a token's heads are neighbours in memory.  Cuts fall
// on whole rounds of the kernel.  A block in several parts leaves a partial
// state per query token and part, and each of its tokens is a unit of the
// merge, as the requests of a split shared-prefix block are.
#include <algorithm>
#include <cstring>
#include <functional>
#include <utility>
#include <vector>

#include "pkd_internal.h"
#include "plan_layout.h"
#include "plan_parts.h"

namespace pkd {
namespace {

struct RowBlock {
  int32_t req, begin, tokens, first;   // its tokens in the request; first: of all query tokens
  int64_t lo;                          // first cached token, a multiple of 16
};

// The other way to share the blocks out: whole ones, longest first, where the
// load is least, and those that fit nowhere laid end to end into the room that
// is left, within stretches of cost `span`; false when they do not fit.  Fewer
// blocks are cut (and merged) than where all are laid end to end, and the
// blocks of a request stand side by side, so that their groups read its tokens
// at the same time, all but one of them from L2: 16 requests x 61 drafts of 64
// heads 188 -> 159 us, 8 prompts' pieces of 256 tokens 149 -> 136.
// A group's parts: of requests with several blocks first, in the order they were
// placed (the groups stay together), then the others in the requests' order
// (longest first, all groups came to their short blocks, whose starts leave
// gaps, at the same time: windows of 64 ragged requests 123.7 us, 118.3 so).
//
// Where L2 does not hold the tokens that blocks share, the blocks' staying
// together is worth more than equal loads: then these blocks go in `pieces` of
// equal length (the longest one's), none of them cut otherwise.
struct Placer {
  struct Unit {
    int32_t block, begin;
    int64_t len;
  };
  std::vector<Unit> units, rest;
  std::vector<std::pair<int64_t, int32_t>> load;   // a heap: least load, then least group
  std::vector<int64_t> room;
  std::vector<PlanPart> whole, cut, parts;
  std::vector<char> shared;

  // The blocks, those of a request's several in `pieces` each, longest first.
  void divide(const std::vector<RowBlock>& blocks, const std::vector<int64_t>& lens, int64_t pieces,
              int64_t round) {
    units.clear();
    for (size_t i = 0, end; i < blocks.size(); i = end) {
      int64_t longest = 0;
      for (end = i; end < blocks.size() && blocks[end].req == blocks[i].req; ++end)
        longest = std::max(longest, lens[end]);
      const int64_t by = shared[i] ? ceil_div(ceil_div(longest, pieces), round) * round : longest;
      for (int64_t at = 0; at < longest; at += by)
        for (size_t b = i; b < end; ++b)
          if (at < lens[b]) units.push_back(Unit{(int32_t)b, (int32_t)at, std::min(by, lens[b] - at)});
    }
    std::stable_sort(units.begin(), units.end(), [](const Unit& x, const Unit& y) { return x.len > y.len; });
  }
  bool place(int64_t span, int64_t alpha, int64_t round, int64_t floor_c, int32_t nv, bool cuts) {
    load.clear();
    for (int32_t v = 0; v < nv; ++v) load.emplace_back(0, v);   // (a heap already)
    const auto later = std::greater<std::pair<int64_t, int32_t>>();
    whole.clear();
    cut.clear();
    rest.clear();
    for (const Unit& u : units) {
      if (load.front().first + u.len + alpha > span) {
        if (!cuts) return false;
        rest.push_back(u);
        continue;
      }
      std::pop_heap(load.begin(), load.end(), later);
      std::pair<int64_t, int32_t>& to = load.back();
      whole.push_back(PlanPart{u.block, u.begin, (int32_t)(u.begin + u.len), to.second});
      to.first += u.len + alpha;
      std::push_heap(load.begin(), load.end(), later);
    }
    room.assign((size_t)nv, span);
    for (const auto& l : load) room[l.second] -= l.first;
    int32_t v = 0;
    for (const Unit& u : rest) {
      const int64_t end = u.begin + u.len;
      for (int64_t pos = u.begin; pos < end; ++v) {
        if (v >= nv) return false;
        const int64_t rem = end - pos, fits = (room[v] - alpha) / round * round;
        int64_t take = 0;
        if (rem + alpha <= room[v]) {
          take = rem;
        } else if (room[v] == span) {   // an empty group: as much as fits, but no short rest
          take = fits;
          if (rem - take < floor_c) take = std::min(take, ceil_div(ceil_div(rem, 2), round) * round);
        } else {
          take = std::min(fits, (rem - floor_c) / round * round);
          if (take < floor_c) take = 0;
        }
        if (take > 0) cut.push_back(PlanPart{u.block, (int32_t)pos, (int32_t)(pos + take), v});
        pos += take;
        room[v] -= take + (take > 0 ? alpha : 0);
        if (pos >= end) break;   // (this group may have room for the next one)
      }
    }
    parts = whole;
    parts.insert(parts.end(), cut.begin(), cut.end());
    std::stable_sort(parts.begin(), parts.end(), [&](const PlanPart& x, const PlanPart& y) {
      if (x.cta != y.cta) return x.cta < y.cta;
      const bool sx = shared[x.req], sy = shared[y.req];
      return sx != sy ? sx : !sx && x.req < y.req;
    });
    return true;
  }
};

}  // namespace

int plan_schedule_tree(const pkd_config& cfg, int32_t n_cta, const Layout& L,
                       const int32_t* q_indptr, const int32_t* indptr, const int32_t* indices,
                       const int32_t* last, int32_t batch, int32_t causal, int32_t window,
                       int32_t* words, pkd_plan_info* info, int64_t* end) {
  if (batch < 0 || n_cta < 1 || words == nullptr || window < 0 || (causal != 0 && causal != 1))
    return PKD_E_INVALID_ARG;
  if (batch > 0 && (q_indptr == nullptr || indptr == nullptr || last == nullptr))
    return PKD_E_INVALID_ARG;
  if (batch > cfg.max_batch) return PKD_E_CAPACITY;
  const int64_t P = cfg.page_size;
  const int32_t hkv = cfg.num_kv_heads;
  const int32_t rows = kTreeRows / (cfg.num_qo_heads / hkv);   // tokens of a block
  thread_local std::vector<RowBlock> blocks;
  thread_local std::vector<int64_t> lens;
  thread_local std::vector<PlanPart> parts;
  thread_local std::vector<int32_t> first_slot, n_chunks, chunk_of, by_place, order;
  blocks.clear();
  lens.clear();
  int64_t nnz = 0, total = 0;
  int32_t tokens = 0, most = 0;
  if (batch > 0) {
    if (indptr[0] != 0 || q_indptr[0] != 0) return PKD_E_BAD_TABLE;
    for (int32_t i = 0; i < batch; ++i) {
      const int64_t pages = (int64_t)indptr[i + 1] - indptr[i];
      const int64_t n = (int64_t)q_indptr[i + 1] - q_indptr[i];
      if (pages < 1 || last[i] < 1 || last[i] > P || n < 0) return PKD_E_BAD_TABLE;
      const int64_t len = P * (pages - 1) + last[i];
      // (the kernel counts tokens in 32 bits, up to a round past the end)
      if (len > 0x7fffffffLL - 1024) return PKD_E_CAPACITY;
      if (n > len) return PKD_E_BAD_TABLE;
      if (q_indptr[i + 1] > cfg.max_batch) return PKD_E_CAPACITY;
      const int64_t context = len - n;
      most = std::max(most, (int32_t)n);
      for (int32_t b = 0; (int64_t)b * rows < n; ++b) {
        const int64_t r0 = (int64_t)b * rows, r1 = std::min<int64_t>(n, r0 + rows);
        const int64_t at = context + (causal ? r0 : 0);   // the least position of a row
        const int64_t lo = window > 0 ? std::max<int64_t>(0, at - window + 1) / 16 * 16 : 0;
        const int64_t hi = causal ? context + r1 : len;
        blocks.push_back(RowBlock{i, (int32_t)r0, (int32_t)(r1 - r0), (int32_t)(q_indptr[i] + r0), lo});
        lens.push_back(hi - lo);
        total += hi - lo;
      }
    }
    tokens = q_indptr[batch];
    nnz = indptr[batch];
    if (nnz > cfg.max_num_pages) return PKD_E_CAPACITY;
    if (indices == nullptr) return PKD_E_INVALID_ARG;
    if (!copy_checked(indices, words + L.page_list, nnz, cfg.num_pages)) return PKD_E_BAD_TABLE;
  }
  const int32_t nv = std::max(1, n_cta / hkv);
  const int64_t alpha = cfg.alpha < 0 ? kTreeAlpha : cfg.alpha;
  const int64_t min_chunk = cfg.min_chunk_tokens < 0 ? kTreeMinChunk : cfg.min_chunk_tokens;
  const int64_t floor_c = ceil_div(std::max<int64_t>(min_chunk, 1), kTreeRound) * kTreeRound;
  int64_t span =
      std::max(alpha + floor_c, ceil_div(total + alpha * (int64_t)blocks.size(), nv));
  thread_local Placer placer;
  placer.shared.assign(blocks.size(), 0);
  int64_t together = 0, distinct = 0;   // tokens of blocks that share them; those tokens
  for (size_t i = 0; i < blocks.size(); ++i) {
    placer.shared[i] = q_indptr[blocks[i].req + 1] - q_indptr[blocks[i].req] > rows;
    if (!placer.shared[i]) continue;
    together += lens[i];
    if (blocks[i].begin == 0) distinct += lens[i];
  }
  const auto grow = [](int64_t s) { return s + std::max<int64_t>(kTreeRound, s / 64); };
  const int64_t least = span, token_bytes = 2 * kHeadDim * ((cfg.flags & PKD_FLAG_KV_FP8) ? 1 : 2);
  int64_t even = span;
  while (!cut_even(lens, even, alpha, kTreeRound, floor_c, nv, &parts)) even = grow(even);
  placer.divide(blocks, lens, 1, kTreeRound);
  while (span <= even && !placer.place(span, alpha, kTreeRound, floor_c, nv, true)) span = grow(span);
  int64_t apart = together;   // of these tokens, those of blocks that do not stay together
  if (span <= even) {
    parts = placer.parts;
    apart = 0;
    for (const Placer::Unit& u : placer.rest)
      if (placer.shared[u.block]) apart += u.len;
  } else {
    span = even;
  }
  if (2 * together > total && distinct * hkv * token_bytes > kTreeSharedBytes) {
    int64_t best = span + (int64_t)((double)span * kTreeSharedGain / 100 * apart / together);
    int64_t several = 0, rows_of = 0;   // such blocks, their query tokens
    for (size_t i = 0; i < blocks.size(); ++i)
      if (placer.shared[i]) ++several, rows_of += blocks[i].tokens;
    for (int64_t times = 1; times <= 6; ++times) {   // about so many for each group
      const int64_t pieces = times * std::max<int64_t>(nv, several) / several;
      const int64_t slots = pieces > 1 ? pieces * rows_of : 0;   // (blocks may have a piece less)
      if (slots > L.max_slots) break;
      placer.divide(blocks, lens, pieces, kTreeRound);
      if ((int64_t)placer.units.size() * hkv > L.max_items) break;
      int64_t s = least;
      while (s < best && !placer.place(s, alpha, kTreeRound, floor_c, nv, false)) s = grow(s);
      if (s >= best) continue;
      best = span = s;
      parts = placer.parts;
    }
  }

  // reduction map: the tokens of a block in several parts, blocks of most
  // parts first, a token's slots one after the other in part order
  const int32_t n_blocks = (int32_t)blocks.size();
  n_chunks.assign((size_t)n_blocks, 0);
  first_slot.assign((size_t)n_blocks, -1);
  // (a block's slots in the order of its tokens, whatever groups have its parts)
  chunk_of.assign(parts.size(), 0);
  by_place.resize(parts.size());
  for (size_t k = 0; k < parts.size(); ++k) by_place[k] = (int32_t)k;
  std::sort(by_place.begin(), by_place.end(), [](int32_t x, int32_t y) {
    return parts[x].req != parts[y].req ? parts[x].req < parts[y].req
                                        : parts[x].tok_begin < parts[y].tok_begin;
  });
  for (const int32_t k : by_place) chunk_of[k] = n_chunks[parts[k].req]++;
  order.clear();
  for (int32_t i = 0; i < n_blocks; ++i)
    if (n_chunks[i] > 1) order.push_back(i);
  std::stable_sort(order.begin(), order.end(),
                   [&](int32_t x, int32_t y) { return n_chunks[x] > n_chunks[y]; });
  const int64_t n_items = (int64_t)parts.size() * hkv;
  int64_t n_slots = 0;
  for (int32_t i : order) n_slots += (int64_t)n_chunks[i] * blocks[i].tokens;
  if (n_items > L.max_items || n_slots > L.max_slots) return PKD_E_CAPACITY;
  int32_t* unit_words = words + L.units;
  int32_t* merge_indptr = words + L.merge_indptr;
  int32_t n_units = 0;
  merge_indptr[0] = 0;
  for (int32_t i : order) {
    first_slot[i] = merge_indptr[n_units];
    for (int32_t t = 0; t < blocks[i].tokens; ++t, ++n_units) {
      unit_words[2 * n_units] = blocks[i].first + t;
      unit_words[2 * n_units + 1] = n_chunks[i];
      merge_indptr[n_units + 1] = merge_indptr[n_units] + n_chunks[i];
    }
  }

  // queues: the parts of stretch v, once per KV head, on CTAs v * Hkv + head
  // (all on one CTA when there are fewer CTAs than heads)
  int32_t* cta_indptr = words + L.cta_indptr;
  int32_t* item_words = words + L.items;
  int64_t at = 0, p0 = 0;
  int32_t cta = 0;
  cta_indptr[0] = 0;
  while (p0 < (int64_t)parts.size()) {
    int64_t p1 = p0;
    while (p1 < (int64_t)parts.size() && parts[p1].cta == parts[p0].cta) ++p1;
    const int32_t v = parts[p0].cta;
    for (int32_t h = 0; h < hkv; ++h) {
      const int32_t c = n_cta >= hkv ? v * hkv + h : 0;
      while (cta < c) cta_indptr[++cta] = (int32_t)at;
      for (int64_t k = p0; k < p1; ++k, ++at) {
        const PlanPart& p = parts[k];
        const RowBlock& b = blocks[p.req];
        int32_t* w = item_words + at * kItemWords;
        const int32_t chunk = chunk_of[k];
        w[0] = b.req;
        w[1] = (int32_t)(b.lo + p.tok_begin);
        w[2] = (int32_t)(b.lo + p.tok_end);
        w[3] = first_slot[p.req] >= 0 ? first_slot[p.req] + chunk : -1;
        w[4] = b.tokens;
        w[5] = b.begin;
        w[6] = first_slot[p.req] >= 0 ? n_chunks[p.req] : 0;
        w[7] = h;
      }
    }
    p0 = p1;
  }
  while (cta < n_cta) cta_indptr[++cta] = (int32_t)at;

  // the requests' entries: first query token, query tokens, tokens before
  // them in the cache, first page in the page list
  int32_t* r = words + request_words(L.page_list, nnz);
  for (int32_t i = 0; i < batch; ++i, r += kRequestWords) {
    r[0] = q_indptr[i];
    r[1] = q_indptr[i + 1] - q_indptr[i];
    r[2] = (int32_t)(P * (indptr[i + 1] - indptr[i] - 1) + last[i] - r[1]);
    r[3] = indptr[i];
  }
  *end = r - words;

  int32_t* h = words;
  std::memset(h, 0, sizeof(int32_t) * H_WORDS);
  h[H_MAGIC] = kMagic;
  h[H_BATCH] = tokens;
  h[H_HQ] = cfg.num_qo_heads;
  h[H_HKV] = hkv;
  h[H_D] = cfg.head_dim;
  h[H_P] = cfg.page_size;
  h[H_NCTA] = n_cta;
  h[H_NITEMS] = (int32_t)n_items;
  h[H_NUNITS] = n_units;
  h[H_NSLOTS] = (int32_t)n_slots;
  h[H_CHUNK] = (int32_t)std::min<int64_t>(span - alpha, 0x7fffffff);
  h[H_ALPHA] = (int32_t)std::min<int64_t>(alpha, 0x7fffffff);
  h[H_NNZ] = (int32_t)nnz;
  h[H_MAKESPAN] = (int32_t)std::min<int64_t>(span, 0x7fffffff);
  h[H_MINCHUNK] = (int32_t)std::min<int64_t>(floor_c, 0x7fffffff);
  h[H_BLOCK] = rows;
  h[H_MAXCHUNKS] = order.empty() ? 0 : n_chunks[order[0]];
  h[H_MAXBATCH] = cfg.max_batch;
  h[H_MAXPAGES] = cfg.max_num_pages;
  h[H_REQUESTS] = batch;
  h[H_CAUSAL] = causal;
  h[H_WINDOW] = window;
  h[H_MAXQ] = most;
  if (info) {
    *info = pkd_plan_info{};
    info->batch = tokens;
    info->num_ctas = n_cta;
    info->chunk_tokens = h[H_CHUNK];
    info->num_items = (int32_t)n_items;
    info->num_units = n_units;
    info->num_slots = (int32_t)n_slots;
    info->total_tokens = total;
    info->makespan = span;
    info->nnz = (int32_t)nnz;
    info->schedule_words = (int32_t)*end;
  }
  return PKD_OK;
}

}  // namespace pkd
