// Which tokens stand behind a packed row on the paths through it (gfx950): the
// next token of its segment or, for a segment's last row, the first token of
// every child.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace tg {

// The segment of packed row r: a 64-way search by the whole wave.
__device__ __forceinline__ int seg_of(const int32_t* seg_off, int n_seg, int r, int lane) {
  int lo = 0, hi = n_seg;
  while (hi - lo > 1) {
    const int step = (hi - lo + 63) >> 6, at = lo + lane * step;
    const bool le = at < hi && seg_off[at] <= r;
    lo += (__popcll(__ballot(le)) - 1) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// The tokens behind packed row r.  A holds the trie's tables (seg_off, n_seg,
// parent, kid_off, kid) and its tokens (tokens, token64, vocab).
struct Behind {
  int n, row;         // how many; the only one's row (middle of a segment)
  int seg;            // r's segment
  const int32_t *kid, *seg_off;
  bool root_start;    // r is a root's first token (it has no row in front)
  template <typename A>
  __device__ __forceinline__ Behind(const A& a, int r, int lane) : seg_off(a.seg_off) {
    const int s = seg = seg_of(a.seg_off, a.n_seg, r, lane);
    const bool last = r + 1 == a.seg_off[s + 1];
    kid = last ? a.kid + a.kid_off[s] : nullptr;
    n = last ? a.kid_off[s + 1] - a.kid_off[s] : 1;
    row = r + 1;
    root_start = a.parent[s] < 0 && r == a.seg_off[s];
  }
  __device__ __forceinline__ int at(int j) const { return kid ? seg_off[kid[j]] : row; }
};

// Token id of row t, or -1 where it is outside the vocabulary.
template <typename A>
__device__ __forceinline__ int token(const A& a, int t) {
  if (a.token64) {
    const int64_t x = static_cast<const int64_t*>(a.tokens)[t];
    return x >= 0 && x < a.vocab ? static_cast<int>(x) : -1;
  }
  const int32_t x = static_cast<const int32_t*>(a.tokens)[t];
  return x >= 0 && x < a.vocab ? x : -1;
}

}  // namespace tg
