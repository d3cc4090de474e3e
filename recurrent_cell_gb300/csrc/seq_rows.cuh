// seq_rows.cuh -- rows of sequences that lie one after another: which sequence
// a row belongs to, found on the device from the row offsets.
#pragma once

#include "cfc_internal.cuh"

namespace cfc {
namespace seqs {

struct Seqs {
  const int* off;     // n + 1 row offsets, or NULL: n sequences of rows / n rows
  int n;
  long long rows, per;
};
__host__ __forceinline__ Seqs make_seqs(const int* off, int n, long long rows) { return Seqs{off, n, rows, rows / n}; }

// The same with the rows that belong to a sequence: those behind the last are nobody's,
// neither read nor written.
__device__ __forceinline__ Seqs trim(Seqs s) {
  if (s.off) {
    const long long end = __ldg(s.off + s.n);
    s.rows = end < 0 ? 0 : (end < s.rows ? end : s.rows);
  }
  return s;
}

// Rows [begin, end) of sequence i.  Offsets are held inside [0, rows], so that
// nothing outside the tensors is touched whatever the array holds.
__device__ __forceinline__ void range_of(const Seqs& s, int i, long long* begin, long long* end) {
  if (s.off) {
    const long long a = __ldg(s.off + i), b = __ldg(s.off + i + 1);
    *begin = a < 0 ? 0 : (a > s.rows ? s.rows : a);
    *end = b < *begin ? *begin : (b > s.rows ? s.rows : b);
  } else {
    *begin = i * s.per;
    *end = *begin + s.per;
  }
}

// The sequence of a row in [0, rows), and its rows: begin <= row < end whatever the
// offsets hold.  A binary search, of one step for every doubling of n.
struct Where {
  int i;
  long long begin, end;
};
__device__ __forceinline__ Where find(const Seqs& s, long long row) {
  Where w;
  if (s.off) {
    int lo = 0, hi = s.n;               // off[lo] <= row < off[hi], where they ascend
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(s.off + mid) <= row) lo = mid;
      else hi = mid;
    }
    w.i = lo;
    const long long a = __ldg(s.off + lo), b = __ldg(s.off + lo + 1);
    w.begin = a < 0 ? 0 : (a > row ? row : a);
    w.end = b <= row ? row + 1 : (b > s.rows ? s.rows : b);
  } else {
    w.i = (int)(row / s.per);
    w.begin = w.i * s.per;
    w.end = w.begin + s.per;
  }
  return w;
}

}  // namespace seqs
}  // namespace cfc
