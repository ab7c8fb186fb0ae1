// Pieces shared by the planners: division, the checked copy of page ids, and
// the cut of table rows laid end to end into equal stretches.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <vector>

namespace pkd {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Copy n page ids and check 0 <= id < num_pages, in one pass the compiler
// can vectorise (no early exit).
inline bool copy_checked(const int32_t* __restrict__ src, int32_t* __restrict__ dst, int64_t n,
                         int32_t num_pages) {
  int32_t lo = 0, hi = 0;
  for (int64_t k = 0; k < n; ++k) {
    const int32_t v = src[k];
    dst[k] = v;
    lo = v < lo ? v : lo;
    hi = v > hi ? v : hi;
  }
  return lo >= 0 && hi < num_pages;
}

struct PlanPart {
  int32_t req, tok_begin, tok_end, cta;   // cta: of the first block of heads
};

// Cut the requests into stretches of cost `span` for nv CTAs; false when they
// do not fit.
inline bool cut_even(const std::vector<int64_t>& lens, int64_t span, int64_t alpha, int64_t P,
                     int64_t floor_c, int32_t nv, std::vector<PlanPart>* parts) {
  parts->clear();
  int32_t v = 0;
  int64_t cap = span;
  for (size_t i = 0; i < lens.size(); ++i) {
    int64_t pos = 0;
    while (pos < lens[i]) {
      if (v >= nv) return false;
      const int64_t rem = lens[i] - pos;
      int64_t take = 0;
      if (rem + alpha <= cap) {
        take = rem;
      } else if (cap == span) {   // an empty CTA: as much as fits, but no short rest
        take = (span - alpha) / P * P;
        if (rem - take < floor_c) take = std::min(take, ceil_div(ceil_div(rem, 2), P) * P);
      } else {
        take = std::min((cap - alpha) / P * P, (rem - floor_c) / P * P);
        if (take < floor_c) take = 0;
      }
      if (take > 0) parts->push_back(PlanPart{(int32_t)i, (int32_t)pos, (int32_t)(pos + take), v});
      pos += take;
      cap -= take + alpha;
      if (pos < lens[i]) {   // this CTA is full
        ++v;
        cap = span;
      }
    }
  }
  return true;
}

}  // namespace pkd
