// Device view of a paged latent cache (csa_paged_kv in csa.h).
#pragma once
#include "common.cuh"

namespace csa {

// The sequence whose packed rows contain `row`: the largest b with
// cu[b] <= row (every lane of a warp calls it and gets the answer), or -1
// behind the last sequence and before the first.  32-way search: one load
// per lane and step.
CSA_DEV int paged_find_seq(const int32_t* cu, int B, int64_t row, int lane) {
  if (row < cu[0] || row >= cu[B]) return -1;
  int lo = 0, hi = B;                       // cu[lo] <= row < cu[hi]
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = min(lo + lane * step, hi);
    const uint32_t le = __ballot_sync(0xffffffffu, at < hi && cu[at] <= row);
    // lane 0 holds cu[lo] <= row; a table that decreases (outside the
    // contract) still only narrows the range
    const int k = 31 - __clz(le | 1u);
    const int nlo = lo + k * step;
    hi = min(nlo + step, hi);
    lo = nlo;
  }
  return lo;
}

// Entry of position p (>= 0) of sequence b, or nullptr where there is none.
CSA_DEV uint8_t* paged_entry(const csa_paged_kv& kv, int b, int64_t p) {
  if (p < 0 || p >= (int64_t)kv.max_pages * kv.page_size) return nullptr;
  const uint32_t pg = (uint32_t)p / (uint32_t)kv.page_size;
  const int32_t id = kv.block_table[(int64_t)b * kv.table_stride + pg];
  if (id < 0 || id >= kv.n_pages) return nullptr;
  return kv.pages + (int64_t)id * kv.page_stride +
         (int64_t)((uint32_t)p - pg * (uint32_t)kv.page_size) * kv.row_stride;
}

}  // namespace csa
