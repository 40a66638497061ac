// Checks the tree attention's host tables (csrc/attn_plan.cpp) against the
// definition on random tries: token i sees token j iff j's segment is i's or
// an ancestor of it and j <= i.  Built with the host sanitizers by
// test_attn_plan.py.  Prints one line per group of tries; exit code 1 on the
// first difference.
#include <algorithm>
#include <cstdio>
#include <cstring>
#include <random>
#include <string>
#include <vector>

#include "../prefix_tree_packed_plan_amd/csrc/attn_plan.hpp"

using tg::AttnItem;
using tg::AttnParts;
using tg::AttnRun;

static int failures = 0;
#define CHECK(c, ...)                     \
  do {                                    \
    if (!(c)) {                           \
      std::printf("FAILED %s: ", #c);     \
      std::printf(__VA_ARGS__);           \
      std::printf("\n");                  \
      std::fflush(stdout);                \
      ++failures;                         \
      return;                             \
    }                                     \
  } while (0)

static std::vector<int> rows_of(const AttnItem& it, const AttnRun* runs, int n, int* bad) {
  std::vector<int> rows;
  for (int r = 0; r < it.n_runs; ++r) {
    const AttnRun x = runs[it.run_off + r];
    const int end = r + 1 < it.n_runs ? runs[it.run_off + r + 1].virt : it.n_total;
    if (x.virt != static_cast<int>(rows.size()) || end <= x.virt) *bad = 1;
    for (int v = x.virt; v < end; ++v) rows.push_back(x.row + v - x.virt);
  }
  for (const int r : rows)
    if (r < 0 || r >= n) *bad = 1;
  if (static_cast<int>(rows.size()) != it.n_total) *bad = 1;
  return rows;
}

static void check(const std::vector<int32_t>& parents, const std::vector<int32_t>& lens) {
  tg::Plan p;
  std::string err;
  const int n_seg = static_cast<int>(parents.size());
  CHECK(tg::build_plan(parents.data(), lens.data(), n_seg, 4, &p, &err) == 0, "%s", err.c_str());
  tg::AttnPlan a;
  CHECK(tg::build_attn_plan(p, &a, &err) == 0, "%s", err.c_str());
  const int n = static_cast<int>(p.n_tokens);
  std::vector<int> seg(n);
  for (int s = 0; s < n_seg; ++s)
    for (int j = 0; j < lens[s]; ++j) seg[p.seg_off[s] + j] = s;
  std::vector<std::vector<char>> anc(n_seg, std::vector<char>(n_seg, 0));
  for (int s = 0; s < n_seg; ++s)
    for (int c = s; c >= 0; c = parents[c]) anc[s][c] = 1;
  const auto sees = [&](int i, int j) { return j <= i && anc[seg[i]][seg[j]]; };
  const int32_t* d = a.mirror.data() + a.m_d;
  const int32_t* e = a.mirror.data() + a.m_e;
  for (int i = 0; i < n; ++i) {
    CHECK(d[i] >= 0 && d[i] < n, "token %d", i);
    CHECK(!(d[n] <= d[i] && d[i] < e[n]) && !(d[i] <= d[n] && d[n] < e[i]), "token %d and no token", i);
    for (int j = 0; j < n; ++j) CHECK((d[j] <= d[i] && d[i] < e[j]) == sees(i, j), "tokens %d, %d", i, j);
  }
  const AttnRun* runs = reinterpret_cast<const AttnRun*>(a.mirror.data() + a.m_runs);
  CHECK(a.m_runs % 2 == 0, "alignment");
  for (int side = 0; side < 2; ++side) {
    const tg::AttnLists& l = side ? a.k : a.q;
    CHECK(l.n_tiles == (n + 127) / 128 && !l.cuts.empty(), "tiles");
    for (size_t ci = 0; ci < l.cuts.size(); ++ci) {
      const tg::AttnCut& c = l.cuts[ci];
      CHECK(ci == 0 || c.most < l.cuts[ci - 1].most, "cuts get finer");
      CHECK(c.m_items % 8 == 0 && c.m_parts % 4 == 0, "alignment");
      CHECK(c.m_items + 8 * size_t(c.n_items) <= a.mirror.size() && c.m_parts + 4 * size_t(l.n_tiles) <= a.mirror.size(),
            "size");
      const AttnItem* items = reinterpret_cast<const AttnItem*>(a.mirror.data() + c.m_items);
      const AttnParts* parts = reinterpret_cast<const AttnParts*>(a.mirror.data() + c.m_parts);
      std::vector<std::vector<std::pair<int, int>>> cover(l.n_tiles);
      std::vector<int> part_tile(c.n_items, -1);
      int64_t total = 0;
      int longest = 0;
      for (int t = 0; t < c.n_items; ++t) {
        const AttnItem& it = items[t];
        CHECK(it.tile >= 0 && it.tile < l.n_tiles && it.n_runs > 0, "tile %d", it.tile);
        CHECK(it.part >= 0 && it.part < c.n_items && part_tile[it.part] < 0, "part %d", it.part);
        CHECK(it.v0 >= 0 && it.v0 < it.v1 && it.v1 <= it.n_total, "tile %d", it.tile);
        const auto rank = [&](const AttnItem& x) {  // whole length, or its power of 2 where there are many
          int len = x.v1 - x.v0, r = 0;
          if (c.n_items <= 1024) return len;
          while (len >>= 1) ++r;
          return r;
        };
        CHECK(t == 0 || rank(it) <= rank(items[t - 1]), "longest first");
        CHECK(it.v0 % 64 == 0 && (it.v1 % 64 == 0 || it.v1 == it.n_total) && it.v1 - it.v0 <= c.most, "part of %d",
              it.tile);
        longest = std::max(longest, it.v1 - it.v0);
        total += it.v1 - it.v0;
        cover[it.tile].push_back({it.v0, it.v1});
        part_tile[it.part] = it.tile;
        if (ci > 0 && it.v0 > 0) continue;  // the list itself has been looked at
        int bad = 0;
        std::vector<int> rows = rows_of(it, runs, n, &bad);
        CHECK(!bad, "runs of tile %d", it.tile);
        const int lo = it.tile * 128, hi = std::min(n, lo + 128);
        const auto pair = [&](int mine, int other) { return side ? sees(other, mine) : sees(mine, other); };
        std::vector<int> want;
        for (int j = 0; j < n; ++j) {
          bool any = false;
          for (int i = lo; i < hi; ++i) any = any || pair(i, j);
          if (any) want.push_back(j);
        }
        for (int v = 0; v < it.n_full; ++v)
          for (int i = lo; i < hi; ++i) CHECK(pair(i, rows[v]), "tile %d: %d and %d are not a pair", it.tile, i, rows[v]);
        std::sort(rows.begin(), rows.end());
        CHECK(rows == want, "list of tile %d", it.tile);
      }
      CHECK(total == l.total && longest == c.longest, "totals");
      int next = 0, multi = 0, multi_parts = 0;
      for (int t = 0; t < l.n_tiles; ++t) {
        const AttnParts& x = parts[t];
        auto& r = cover[x.tile];
        CHECK(static_cast<int>(r.size()) == x.n_parts, "parts of %d", x.tile);
        std::sort(r.begin(), r.end());
        int at = 0;
        for (const auto& y : r) {
          CHECK(y.first == at, "part of %d", x.tile);
          at = y.second;
        }
        for (int i = 0; i < x.n_parts; ++i) CHECK(part_tile[x.part0 + i] == x.tile, "part %d", x.part0 + i);
        // Parts are numbered along the list: the order their results are added in.
        for (int i = 0; i < c.n_items; ++i)
          if (items[i].tile == x.tile) {
            const int k = items[i].part - x.part0;
            CHECK(k >= 0 && k < x.n_parts && r[k].first == items[i].v0, "order of parts");
          }
        CHECK(x.part0 == next, "numbers of parts");
        next += x.n_parts;
        if (x.n_parts > 1) {
          CHECK(multi == t, "tiles with several parts come first");
          ++multi;
          multi_parts += x.n_parts;
        }
        r.clear();
      }
      CHECK(next == c.n_items && multi == c.n_multi && multi_parts == c.n_multi_parts, "part counts");
    }
    for (const int heads : {1, 2, 16, 1000})
      for (const int steps : {1, 3, 8}) {
        int32_t split = -1;
        for (const int least : {64, 256}) {
          const tg::AttnCut& c = tg::choose_cut(l, heads, steps, least, least / 2, &split);
          CHECK(split >= 1 && split <= steps, "split %d", split);
          CHECK(&c >= l.cuts.data() && &c < l.cuts.data() + l.cuts.size(), "a cut of these lists");
          CHECK(&c == l.cuts.data() || c.most >= least, "too fine a cut");
          tg::choose_cut(l, heads, steps, least, least / 2, nullptr);
        }
      }
  }
}

int main() {
  std::mt19937 rng(7);
  const auto uni = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); };
  check({-1}, {1});
  check({-1}, {127});
  check({-1}, {128});
  check({-1}, {129});
  check({-1, -1}, {64, 64});
  check({-1}, {4500});              // several parts
  check({-1, 0, 0, 0}, {300, 900, 1000, 1100});
  for (int t = 0; t < 60 && !failures; ++t) {
    const int n_seg = uni(1, 40), most = t % 3 == 0 ? 4 : t % 3 == 1 ? 40 : 150;
    std::vector<int32_t> parents(n_seg), lens(n_seg);
    for (int i = 0; i < n_seg; ++i) {
      // Any numbering with parents first (t even), or depth-first order.
      parents[i] = i == 0 ? -1 : uni(-1, i - 1);
      lens[i] = uni(1, most);
    }
    if (t % 2) {
      for (int i = 1; i < n_seg; ++i) {  // the parent is on the path of the segment before
        int p = i - 1;
        while (p >= 0 && uni(0, 2) == 0) p = parents[p];
        parents[i] = p;
      }
    }
    check(parents, lens);
  }
  std::printf("random tries done\n");
  std::fflush(stdout);
  {  // a deep chain of single tokens, and one with a leaf at every step
    std::vector<int32_t> p, l;
    for (int i = 0; i < 1500; ++i) {
      p.push_back(i - 1);
      l.push_back(1);
    }
    check(p, l);
    p = {-1};
    l = {1};
    for (int i = 0, at = 0; i < 400; ++i) {
      p.push_back(at);
      l.push_back(1);
      p.push_back(at);
      l.push_back(2);
      at = static_cast<int>(p.size()) - 1;
    }
    check(p, l);
  }
  std::printf(failures ? "FAILED\n" : "attention tables hold\n");
  return failures ? 1 : 0;
}
