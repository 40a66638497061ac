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

// Cuts every list into parts of `most` positions and a rest (a whole number of
// 64 but at the list's end); the parts of tiles with several are numbered
// first.  Query tiles' lists begin alike (at the roots) and key tiles' lists end
// alike (at the ends of subtrees; `from_end`: the rest comes first), so that
// equal parts of neighbouring tiles hold the same rows.  They are put next to
// each other and run together, sharing them in L2 (8/2 heads of 128; chain of
// 16383 tokens: backward 1885 -> 1841 us against equal parts in the tiles'
// order, chain of 4096: forward 64.6 -> 61.2 us, backward 197 -> 181 us).
AttnCut cut_lists(const std::vector<AttnItem>& lists, int64_t most, bool from_end, std::vector<AttnItem>* items,
                  std::vector<AttnParts>* parts) {
  AttnCut c;
  c.most = static_cast<int32_t>(most);
  std::vector<AttnParts> all;
  items->clear();
  parts->clear();
  for (AttnItem it : lists) {
    const int64_t n_parts = (it.n_total + most - 1) / most;
    const int64_t rest = from_end ? ((it.n_total - 1) % most + 64) / 64 * 64 : most;
    all.push_back({it.tile, static_cast<int32_t>(items->size()), 0, 0});
    for (int64_t v = 0, e; v < it.n_total; v = e) {
      e = std::min<int64_t>(it.n_total, v + (v ? most : n_parts == 1 ? it.n_total : rest));
      it.v0 = static_cast<int32_t>(v);
      it.v1 = static_cast<int32_t>(e);
      c.longest = std::max(c.longest, it.v1 - it.v0);
      items->push_back(it);
      all.back().n_parts += 1;
    }
  }
  int32_t next = 0;
  for (int pass = 0; pass < 2; ++pass) {
    for (AttnParts x : all) {
      if ((x.n_parts > 1) != (pass == 0)) continue;
      for (int32_t i = 0; i < x.n_parts; ++i) (*items)[x.part0 + i].part = next + i;
      x.part0 = next;
      next += x.n_parts;
      parts->push_back(x);
    }
    if (pass == 0) {
      c.n_multi = static_cast<int32_t>(parts->size());
      c.n_multi_parts = next;
    }
  }
  c.n_items = next;
  // Longest first; with items enough to fill the device many times, only by
  // powers of 2, in the order of the tiles within them: neighbours then read the
  // same keys (32 prompts of 8 completions, 282665 tokens, 16/4 heads of 128: forward
  // 7.09 -> 6.67 ms, backward 21.9 -> 20.8 ms; a trie of 80 tiles loses 3%).
  const bool many = items->size() > 1024;
  const auto rank = [&](const AttnItem& x) {
    int32_t n = x.v1 - x.v0, r = 0;
    if (!many) return n;
    while (n >>= 1) ++r;
    return r;
  };
  std::stable_sort(items->begin(), items->end(),
                   [&](const AttnItem& x, const AttnItem& y) {
                     const int32_t a = rank(x), b = rank(y);
                     if (a != b || many) return a > b;
                     return from_end ? x.n_total - x.v1 < y.n_total - y.v1 : x.v0 < y.v0;
                   });
  return c;
}

// All cuts of one kind of lists, appended to the device copy.
AttnLists cut_all(const std::vector<AttnItem>& lists, bool from_end, std::vector<int32_t>* mirror) {
  AttnLists l;
  l.n_tiles = static_cast<int32_t>(lists.size());
  int64_t longest = 0;
  for (const AttnItem& it : lists) {
    l.total += it.n_total;
    longest = std::max<int64_t>(longest, it.n_total);
  }
  std::vector<AttnItem> items;
  std::vector<AttnParts> parts;
  const auto append = [&](const void* p, size_t ints) {
    const size_t at = (mirror->size() + 7) / 8 * 8;
    mirror->resize(at + ints, 0);
    std::memcpy(mirror->data() + at, p, ints * sizeof(int32_t));
    return at;
  };
  static_assert(sizeof(AttnItem) == 32 && sizeof(AttnRun) == 8 && sizeof(AttnParts) == 16, "device layout");
  for (int64_t most = int64_t(1) << 31; most >= 64; most = most > 8192 ? 8192 : most / 2) {
    const bool whole = most > 8192;
    if (!whole && longest <= most) continue;  // the whole lists again
    if (!whole && l.total / most + l.n_tiles > AttnPlan::kMaxParts) break;
    AttnCut c = cut_lists(lists, whole ? std::max<int64_t>(longest, 1) : most, from_end, &items, &parts);
    c.m_items = append(items.data(), items.size() * 8);
    c.m_parts = append(parts.data(), parts.size() * 4);
    l.cuts.push_back(c);
  }
  return l;
}

}  // namespace

const AttnCut& choose_cut(const AttnLists& l, int32_t heads, int32_t steps, int32_t least, int32_t worth,
                          int32_t* split) {
  if (split) *split = 1;
  const AttnCut& whole = l.cuts.front();
  const double room = double(l.total) * heads * steps / kSlots;  // of a slot
  const auto fits = [&](int64_t len, bool uncut) { return double(len) <= (uncut ? 1.0 : 0.75) * room; };
  for (size_t i = 0; i < l.cuts.size(); ++i) {
    const AttnCut& c = l.cuts[i];
    const bool last = i + 1 == l.cuts.size() || l.cuts[i + 1].most < least;
    const int64_t items = int64_t(c.n_items) * heads;
    const bool enough = items >= kSlots && c.most <= 4 * least;
    if (!fits(int64_t(c.longest) * steps, i == 0) && !enough && !last) continue;
    int32_t s = 1;
    if (split)
      while (s < steps && items * s < kSlots && !fits(int64_t(c.longest) * ((steps + s - 1) / s), false)) ++s;
    const int64_t saved = int64_t(whole.longest) * steps - int64_t(c.longest) * ((steps + s - 1) / s);
    if (saved < worth) return whole;
    if (split) *split = s;
    return c;
  }
  return whole;
}

int build_attn_plan(const Plan& p, AttnPlan* out, std::string* err, int64_t max_runs, int64_t max_steps) {
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
  std::vector<AttnItem> qlists, klists;
  int64_t steps = 0;
  const auto too_large = [&] {
    if (static_cast<int64_t>(runs.size()) > max_runs)
      *err = "tree_attention_plan: the tiles' run lists exceed " + std::to_string(max_runs) + " entries";
    else if (steps > max_steps)
      *err = "tree_attention_plan: the tiles' lists take more than " + std::to_string(max_steps) +
             " steps over their segments (" + (dfs ? "a very deep and branched trie" : "a depth-first numbering takes fewer") +
             ")";
    else
      return false;
    return true;
  };

  // Query tiles: walk up from every segment of the tile, stopping where an
  // earlier walk of the same tile has been.
  std::vector<int32_t> stamp(n_seg, -1), reach(n_seg, 0), touched;
  std::vector<Range> full, part;
  const int32_t n_qt = (n + kQTile - 1) / kQTile;
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
    it.n_total = emit(&part, it.n_full, &runs);
    it.n_runs = static_cast<int32_t>(runs.size()) - it.run_off;
    qlists.push_back(it);
    if (too_large()) return TREE_ERR_UNSUPPORTED;
  }

  // Key tiles: the subtrees of the tile's segments.
  const int32_t n_kt = (n + kKTile - 1) / kKTile;
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
    klists.push_back(it);
    if (too_large()) return TREE_ERR_UNSUPPORTED;
  }
  const auto up = [](size_t x) { return (x + 7) / 8 * 8; };
  a.m_d = 0;
  a.m_e = up(size_t(n) + 1);
  a.m_runs = a.m_e + up(size_t(n) + 1);
  a.mirror.assign(a.m_runs + runs.size() * 2, 0);
  for (int32_t s = 0; s < n_seg; ++s)
    for (int32_t j = 0; j < p.lens[s]; ++j) {
      a.mirror[a.m_d + p.seg_off[s] + j] = dbeg[s] + j;
      a.mirror[a.m_e + p.seg_off[s] + j] = dend[s];
    }
  a.mirror[a.m_d + n] = -1;  // the position of no token: sees nothing,
  a.mirror[a.m_e + n] = 0;   // and nothing sees it
  std::memcpy(a.mirror.data() + a.m_runs, runs.data(), runs.size() * sizeof(AttnRun));
  a.q = cut_all(qlists, false, &a.mirror);
  a.k = cut_all(klists, true, &a.mirror);
  *out = std::move(a);
  return TREE_OK;
}

}  // namespace tg
