// What the kernels over a paged cache share: a sequence of the batch, the page
// of a position, and TMA boxes of a page.
//
// Everything that comes from the device's tables is bounded where it is read:
// lengths to [0, capacity], token starts to [0, T] and in order, page numbers
// by page_ok. A malformed table gives wrong rows, never an access outside the
// tensors.
#pragma once
#include "fa2_fwd_common.cuh"
#include "fa2_paged.h"

namespace fa2 {

struct PagedSeq {
  int t0, n;    // tokens [t0, t0 + n)
  int length;   // positions; the tokens are the last n of them (should n be more, the first ones have none)
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedBatch& p, int b) {
  PagedSeq s;
  s.length = min(max(__ldg(p.lengths + b), 0), p.capacity);
  if (p.starts) {
    s.t0 = min(max(__ldg(p.starts + b), 0), p.T);
    s.n = min(max(__ldg(p.starts + b + 1), s.t0), p.T) - s.t0;
  } else {
    s.t0 = b * p.each;
    s.n = p.each;
  }
  return s;
}

// The table's entry for position `pos` (below the capacity) of sequence b.
__device__ __forceinline__ int paged_entry(const PagedBatch& p, int b, int pos) {
  return __ldg(p.table + b * p.table_stride + (pos >> p.page_shift));
}
__device__ __forceinline__ bool page_ok(const PagedBatch& p, int page) {
  return static_cast<unsigned>(page) < static_cast<unsigned>(p.pages);
}

// 4-D tiled bulk tensor load global -> shared of one page's (or part of one's) box.
__device__ __forceinline__ void tma_load_4d_hint(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1,
                                                 int c2, int c3, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "l"(policy)
      : "memory");
}

}  // namespace fa2
