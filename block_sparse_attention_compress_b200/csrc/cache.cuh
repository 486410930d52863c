// The paged cache as the device sees it: where a token's row lies, and the 4-bit format.
#pragma once
#include "common.cuh"
#include "kernels.h"

namespace nsa {
namespace cache {

__device__ __forceinline__ void report(int32_t* status) {
  if (status) atomicCAS(status, 0, kErrCache);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Where row i of an append's or a read's tensors lives: its position in sequence b, and the
// page and place of that position.
struct Row {
  int seq;    // -1: the row belongs to no sequence
  int pos;    // < 0: padding in front of a short sequence
  int page;   // -1: no valid page
  int place;
};

__device__ __forceinline__ Row find_row(const CacheArgs& c, const RowsArgs& r, int i) {
  Row w{-1, -1, -1, 0};
  int end;   // one past sequence w.seq's last row
  if (r.cu) {
    int lo = 0, hi = c.batch;   // the largest b in [0, batch] with cu[b] <= i, if there is one
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(r.cu + mid) <= i) lo = mid; else hi = mid - 1;
    }
    if (lo >= c.batch || __ldg(r.cu + lo) > i) return w;
    end = __ldg(r.cu + lo + 1);
    if (i >= end) return w;
    w.seq = lo;
  } else {
    w.seq = i / r.n_new;
    end = (w.seq + 1) * r.n_new;
  }
  const long long pos = (long long)__ldg(r.seqlens + w.seq) - (end - i);
  const long long cap = (long long)c.max_pages * c.page_size;
  if (pos < 0) return w;
  w.pos = pos < cap ? (int)pos : INT32_MAX;
  if (pos < cap) {
    const int j = (int)pos / c.page_size;
    const int p = __ldg(c.page_table + (size_t)w.seq * c.max_pages + j);
    if (p >= 0 && p < c.n_pages) {
      w.page = p;
      w.place = (int)pos - j * c.page_size;
    }
  }
  return w;
}

}  // namespace cache
}  // namespace nsa
