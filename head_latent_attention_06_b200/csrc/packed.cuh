// Packed batches: the sequence a row belongs to, found by a whole warp.
#pragma once

#include "common.cuh"

namespace mla {

// Rows [lo, hi) of the sequence `b` that row t belongs to; b = -1 when it has none.
struct PackedSeq {
  int b, lo, hi;
};

// Counts the entries cu[1 .. B] that are <= t (they do not decrease), 32 at a
// time: every round the lanes test 32 evenly spaced entries, so B < 32 takes one
// round of loads and B < 1024 two, where a binary search would take 10 dependent
// ones.  A warp-collective call with the same t in every lane.
MLA_DEVI PackedSeq packed_find(const int32_t* cu, int B, int n_tok, int t, int lane) {
  int lo = 0, hi = B;
  while (lo < hi) {
    const int step = (hi - lo + 31) >> 5;
    const int64_t e = (int64_t)lo + (int64_t)(lane + 1) * step;
    const bool le = e <= hi && cu[e] <= t;
    const uint32_t m = __ballot_sync(0xffffffffu, le);
    const int n = m == 0xffffffffu ? 32 : __ffs(~m) - 1;  // leading lanes whose entry is <= t
    const int64_t top = (int64_t)lo + (int64_t)(n + 1) * step - 1;
    lo += n * step;
    hi = top < hi ? (int)top : hi;
    if (lo > hi) lo = hi;
  }
  PackedSeq s = {-1, 0, 0};
  if (lo >= B) return s;
  const int a = cu[lo], z = cu[lo + 1];
  if (a < 0 || a > t || t >= z || z > n_tok) return s;
  s.b = lo;
  s.lo = a;
  s.hi = z;
  return s;
}

// Rows [lo, hi) of the sequence that this thread's row t belongs to (lo = hi = 0: none).
struct PackedRow {
  int lo, hi;
};
MLA_DEVI PackedRow packed_own(const int32_t* cu, int B, int n_tok, int t) {
  int a = 0, z = B;  // the count of entries cu[1 .. B] that are <= t
  while (a < z) {
    const int mid = a + (z - a) / 2;
    if (cu[mid + 1] <= t)
      a = mid + 1;
    else
      z = mid;
  }
  if (a >= B) return {0, 0};
  const int lo = cu[a], hi = cu[a + 1];
  if (lo < 0 || lo > t || t >= hi || hi > n_tok) return {0, 0};
  return {lo, hi};
}

// Records offsets that decrease or leave [0, n_tok]; `n` threads of one block.
MLA_DEVI void packed_check(const int32_t* cu, int B, int n_tok, uint32_t* status, int tid, int n) {
  bool bad = false;
  for (int i = tid; i <= B; i += n) {
    const int v = cu[i];
    bad |= v < 0 || v > n_tok || (i > 0 && v < cu[i - 1]);
  }
  if (bad) set_status(status, MLA_ERR_BAD_SEQ_LEN);
}

}  // namespace mla
