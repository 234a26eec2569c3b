// The arithmetic of planning page operations (pages.cu), plain C++ so that it can be checked
// on the host at sizes whose tables fill a GPU: up to 2048 sequences of up to 2^30 pages each.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define QD_PLAN __host__ __device__ inline
#else
#define QD_PLAN inline
#endif

namespace qd {

QD_PLAN int pages_of(int tokens, int ps) { return tokens / ps + (tokens % ps != 0); }

// What an extension takes from the free pages for one sequence: up to 2^30 pages (31 bits), and
// whether the first of them is a copy of its shared last page (the top bit).
struct PageNeed {
  uint32_t bits;
  QD_PLAN int pages() const { return (int)(bits & 0x7fffffffu); }
  QD_PLAN bool copy() const { return bits >> 31 != 0; }
};
// len + n_new <= 2^30
QD_PLAN PageNeed page_need(int len, int n_new, int ps, bool copy) {
  const uint32_t fresh = n_new > 0 ? (uint32_t)(pages_of(len + n_new, ps) - pages_of(len, ps)) : 0u;
  return PageNeed{(fresh + (copy ? 1u : 0u)) | (copy ? 1u << 31 : 0u)};
}

// Sums of needs over the sequences: up to 2^41.
typedef int64_t PageSum;

}  // namespace qd
