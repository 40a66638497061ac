// Host-side tables of the tree attention.  See attn_plan.hpp.
#include "attn_plan.hpp"

#include <algorithm>
#include <cstring>

#include "../../include/tree_gdn.h"

namespace tg {

namespace {

struct Range {
  int32_t lo, hi;
};

// Sorts, joins touching ranges, and appends them as runs from position v on.
int32_t emit(std::vector<Range>* r, int32_t v, std::vector<AttnRun>* runs) {
  std::sort(r->begin(), r->end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  int32_t end = -1;
  for (const Range& x : *r) {
    if (x.lo >= x.hi) continue;
    if (x.lo != end) runs->push_back({v, x.lo});
    v += x.hi - x.lo;
    end = x.hi;
  }
  return v;
}

}  // namespace

int build_attn_plan(const Plan& p, AttnPlan* out, std::string* err) {
  const int32_t n_seg = p.n_seg;
  const int32_t n = static_cast<int32_t>(p.n_tokens);
  AttnPlan a;
  a.n_tokens = n;

  // Depth-first numbers: pre[s], and the end pout[s] of s's subtree; the same
  // in tokens.  at[m] is the segment with number m.
  std::vector<int32_t> pre(n_seg), pout(n_seg), at(n_seg), dbeg(n_seg), dend(n_seg);
  {
    std::vector<int32_t> stack, next(n_seg, 0);
    int32_t m = 0, tok = 0;
    for (const int32_t root : p.roots) {
      stack.push_back(root);
      while (!stack.empty()) {
        const int32_t s = stack.back();
        if (next[s] == 0) {
          pre[s] = m;
          at[m++] = s;
          dbeg[s] = tok;
          tok += p.lens[s];
        }
        const int32_t k = p.kid_off[s] + next[s];
        if (k < p.kid_off[s + 1]) {
          next[s] += 1;
          stack.push_back(p.kid[k]);
        } else {
          next[s] = next[s] == 0 ? 1 : next[s];
          pout[s] = m;
          dend[s] = tok;
          stack.pop_back();
        }
      }
    }
  }
  bool dfs = true;
  for (int32_t s = 0; s < n_seg; ++s) dfs = dfs && pre[s] == s;

  // Unbranched stretches: top[s] is the first segment of the run of segments
  // .. s-1, s in which each is the next one's parent (their rows touch).
  std::vector<int32_t> top(n_seg);
  for (int32_t s = 0; s < n_seg; ++s) top[s] = s > 0 && p.parents[s] == s - 1 ? top[s - 1] : s;

  std::vector<AttnRun> runs;
  std::vector<AttnItem> qitems, kitems;
  const auto too_large = [&] {
    *err = "tree_attention_plan: the tiles' run lists exceed 2^26 entries";
    return TREE_ERR_UNSUPPORTED;
  };

  // Query tiles: walk up from every segment of the tile, stopping where an
  // earlier walk of the same tile has been.
  std::vector<int32_t> stamp(n_seg, -1), reach(n_seg, 0), touched;
  std::vector<Range> full, part;
  const int32_t n_qt = (n + kQTile - 1) / kQTile;
  int64_t steps = 0;
  for (int32_t t = 0, s1 = 0; t < n_qt; ++t) {
    const int32_t lo = t * kQTile, hi = std::min<int64_t>(n, int64_t(lo) + kQTile);
    while (p.seg_off[s1 + 1] <= lo) ++s1;
    int32_t min_pre = n_seg, max_pre = -1;
    touched.clear();
    for (int32_t s = s1; s < n_seg && p.seg_off[s] < hi; ++s) {
      min_pre = std::min(min_pre, pre[s]);
      max_pre = std::max(max_pre, pre[s]);
      for (int32_t c = s; c >= 0; c = p.parents[top[c]]) {
        const int32_t tp = top[c];
        ++steps;
        if (stamp[tp] == t) {
          reach[tp] = std::max(reach[tp], c);
          break;
        }
        stamp[tp] = t;
        reach[tp] = c;
        touched.push_back(tp);
      }
    }
    full.clear();
    part.clear();
    for (const int32_t tp : touched) {
      // The deepest segment of the stretch that every row's segment descends
      // from (or is): the first such segments are its ancestors.
      int32_t l = tp - 1, r = reach[tp];
      while (l < r) {
        const int32_t m = l + (r - l + 1) / 2;
        if (pre[m] <= min_pre && max_pre < pout[m]) l = m;
        else r = m - 1;
      }
      const int32_t beg = p.seg_off[tp], end = std::min(p.seg_off[reach[tp] + 1], hi);
      const int32_t cut = l >= tp ? std::max(beg, std::min(p.seg_off[l + 1], lo)) : beg;
      full.push_back({beg, cut});
      part.push_back({cut, end});
    }
    AttnItem it{t, static_cast<int32_t>(runs.size()), 0, 0, 0, 0, 0, 0};
    it.n_full = emit(&full, 0, &runs);
    it.n_total = it.v1 = emit(&part, it.n_full, &runs);
    it.n_runs = static_cast<int32_t>(runs.size()) - it.run_off;
    qitems.push_back(it);
    if (static_cast<int64_t>(runs.size()) > AttnPlan::kMaxRuns || steps > (int64_t(1) << 31)) return too_large();
  }

  // Key tiles: the subtrees of the tile's segments.
  const int32_t n_kt = (n + kKTile - 1) / kKTile;
  std::vector<AttnParts> parts;
  std::vector<Range> pres;
  for (int32_t t = 0, s1 = 0; t < n_kt; ++t) {
    const int32_t lo = t * kKTile, hi = std::min<int64_t>(n, int64_t(lo) + kKTile);
    while (p.seg_off[s1 + 1] <= lo) ++s1;
    int32_t flo = -1, fhi = n_seg;  // depth-first numbers of the segments below all of the tile's
    pres.clear();
    for (int32_t s = s1; s < n_seg && p.seg_off[s] < hi; ++s) {
      flo = std::max(flo, pre[s]);
      fhi = std::min(fhi, pout[s]);
      pres.push_back({pre[s], pout[s]});
    }
    std::sort(pres.begin(), pres.end(), [](const Range& x, const Range& y) { return x.lo < y.lo; });
    full.clear();
    part.clear();
    int32_t done = 0;
    for (const Range& x : pres) {
      const int32_t x0 = std::max(x.lo, done);
      done = std::max(done, x.hi);
      if (x0 >= x.hi) continue;
      if (dfs) {
        const int32_t r0 = std::max(lo, p.seg_off[x0]), r1 = p.seg_off[x.hi];
        int32_t f0 = r1, f1 = r1;  // rows below all of the tile's segments, and after the tile
        if (flo < fhi) {
          f0 = std::min(r1, std::max(r0, std::max(hi, p.seg_off[flo])));
          f1 = std::max(f0, std::min(r1, p.seg_off[fhi]));
        }
        part.push_back({r0, f0});
        full.push_back({f0, f1});
        part.push_back({f1, r1});
        ++steps;
      } else {
        for (int32_t m = x0; m < x.hi; ++m, ++steps) {
          const int32_t s = at[m], r1 = p.seg_off[s + 1];
          if (r1 <= lo) continue;
          const int32_t r0 = std::max(lo, p.seg_off[s]);
          const int32_t f0 = m >= flo && m < fhi ? std::min(r1, std::max(r0, hi)) : r1;
          part.push_back({r0, f0});
          full.push_back({f0, r1});
        }
      }
    }
    AttnItem it{t, static_cast<int32_t>(runs.size()), 0, 0, 0, 0, 0, 0};
    it.n_full = emit(&full, 0, &runs);
    it.n_total = emit(&part, it.n_full, &runs);
    it.n_runs = static_cast<int32_t>(runs.size()) - it.run_off;
    // Equal parts, each a whole number of 64 virtual rows.
    const int32_t n_parts = static_cast<int32_t>((int64_t(it.n_total) + kPart - 1) / kPart);
    const int32_t each = ((it.n_total + n_parts - 1) / n_parts + 63) / 64 * 64;
    parts.push_back({t, static_cast<int32_t>(kitems.size()), 0, 0});
    for (int64_t v = 0; v < it.n_total; v += each) {
      it.v0 = static_cast<int32_t>(v);
      it.v1 = static_cast<int32_t>(std::min<int64_t>(it.n_total, v + each));
      kitems.push_back(it);
      parts.back().n_parts += 1;
    }
    if (static_cast<int64_t>(runs.size()) > AttnPlan::kMaxRuns || steps > (int64_t(1) << 31)) return too_large();
  }
  // Part numbers: key tiles with several parts first.
  std::vector<AttnParts> ordered;
  int32_t next = 0;
  for (int pass = 0; pass < 2; ++pass) {
    for (AttnParts x : parts) {
      if ((x.n_parts > 1) != (pass == 0)) continue;
      for (int32_t i = 0; i < x.n_parts; ++i) kitems[x.part0 + i].part = next + i;
      x.part0 = next;
      next += x.n_parts;
      ordered.push_back(x);
    }
    if (pass == 0) {
      a.n_multi = static_cast<int32_t>(ordered.size());
      a.n_multi_parts = next;
    }
  }
  // Longest work first.
  const auto longer = [](const AttnItem& x, const AttnItem& y) { return x.v1 - x.v0 > y.v1 - y.v0; };
  std::stable_sort(qitems.begin(), qitems.end(), longer);
  std::stable_sort(kitems.begin(), kitems.end(), longer);

  a.n_qtiles = n_qt;
  a.n_ktiles = n_kt;
  a.n_kitems = static_cast<int32_t>(kitems.size());
  const auto up = [](size_t x) { return (x + 7) / 8 * 8; };
  a.m_d = 0;
  a.m_e = up(size_t(n) + 1);
  a.m_q = a.m_e + up(size_t(n) + 1);
  a.m_k = a.m_q + qitems.size() * 8;
  a.m_parts = a.m_k + kitems.size() * 8;
  a.m_runs = up(a.m_parts + ordered.size() * 4);
  a.mirror.assign(a.m_runs + runs.size() * 2, 0);
  for (int32_t s = 0; s < n_seg; ++s)
    for (int32_t j = 0; j < p.lens[s]; ++j) {
      a.mirror[a.m_d + p.seg_off[s] + j] = dbeg[s] + j;
      a.mirror[a.m_e + p.seg_off[s] + j] = dend[s];
    }
  a.mirror[a.m_d + n] = -1;  // the position of no token: sees nothing,
  a.mirror[a.m_e + n] = 0;   // and nothing sees it
  static_assert(sizeof(AttnItem) == 32 && sizeof(AttnRun) == 8 && sizeof(AttnParts) == 16, "device layout");
  std::memcpy(a.mirror.data() + a.m_q, qitems.data(), qitems.size() * sizeof(AttnItem));
  std::memcpy(a.mirror.data() + a.m_k, kitems.data(), kitems.size() * sizeof(AttnItem));
  std::memcpy(a.mirror.data() + a.m_parts, ordered.data(), ordered.size() * sizeof(AttnParts));
  std::memcpy(a.mirror.data() + a.m_runs, runs.data(), runs.size() * sizeof(AttnRun));
  *out = std::move(a);
  return TREE_OK;
}

}  // namespace tg
