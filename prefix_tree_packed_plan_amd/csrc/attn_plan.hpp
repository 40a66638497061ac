// Host-side tables of the tree attention (no HIP headers: this file and
// attn_plan.cpp build and run without a GPU).
//
// Token i sees token j iff j lies on i's root-to-token path, i itself
// included ("Tree Training" section 3.1 Eq. 6 applied to attention).  With
// D(i) the token's position in a depth-first walk of the trie and E(j) the
// end of the subtree of j's segment in that walk,
//     i sees j  <=>  D(j) <= D(i) < E(j),
// for any numbering in which parents precede children (in depth-first order
// D(i) = i).  The kernels test exactly that where a tile is not wholly seen.
//
// A query tile is kQTile consecutive packed rows.  The keys any of its rows
// sees are a few runs of packed rows (an unbranched stretch of segments is
// one run), laid end to end as virtual key positions: first the runs every
// row sees (no test needed), then the others.  A key tile (kKTile rows) has
// the rows that see any of its keys in the same form, for the gradients of k
// and v.
//
// A list may be cut into parts, worked on by different work-groups, whose
// results are added in the order of the parts.  The tables hold every list
// whole and cut into parts of at most 8192, 4096, .. 64 positions; a call
// takes the coarsest cut that balances its work-groups (choose_cut).
#pragma once

#include <cstddef>
#include <cstdint>
#include <string>
#include <vector>

#include "plan.hpp"

namespace tg {

constexpr int32_t kQTile = 128;
constexpr int32_t kKTile = 128;

// One tile's list of runs.  Virtual positions [v0, v1) of it are this item's
// work; [0, n_full) need no visibility test; n_total is the list's length.
struct AttnItem {
  int32_t tile;      // packed rows tile * kQTile (or kKTile) ..
  int32_t run_off;   // first run
  int32_t n_runs;
  int32_t n_full;
  int32_t n_total;
  int32_t v0, v1;
  int32_t part;      // number of this part among all parts of the cut
};
struct AttnRun {
  int32_t virt;  // virtual position of the run's first row
  int32_t row;   // its packed row
};
// A tile's parts: part0 .. part0 + n_parts - 1.
struct AttnParts {
  int32_t tile, part0, n_parts, pad;
};

// All lists of one kind, each cut into parts of at most `most` positions.
struct AttnCut {
  int32_t most = 0;
  int32_t n_items = 0;
  int32_t n_multi = 0;        // tiles with more than one part (first in the parts table)
  int32_t n_multi_parts = 0;  // their parts (numbered first)
  int32_t longest = 0;        // positions of the longest part
  size_t m_items = 0, m_parts = 0;  // in the device copy: AttnItem (longest first), AttnParts
};
struct AttnLists {
  int32_t n_tiles = 0;
  int64_t total = 0;          // positions of all lists
  std::vector<AttnCut> cuts;  // whole lists first, then finer and finer
};

struct AttnPlan {
  int32_t n_tokens = 0;
  AttnLists q, k;
  // Entries a trie may need at most: the run lists of all tiles together.
  static constexpr int64_t kMaxRuns = int64_t(1) << 26;
  // Segments looked at for all lists (a few seconds).  A key tile's list costs
  // its stretches in depth-first numbering, every segment below it in others.
  static constexpr int64_t kMaxSteps = int64_t(1) << 31;
  // A cut of more parts is not made (the coarser ones have parts enough).
  static constexpr int64_t kMaxParts = 1 << 12;

  std::vector<int32_t> mirror;  // device copy
  size_t m_d = 0, m_e = 0, m_runs = 0;
  size_t device_bytes() const { return mirror.size() * sizeof(int32_t); }
};

// The cut for `heads` work items per part, each `steps` times as long as the
// part, on a device that runs kSlots work-groups at a time: the coarsest whose
// longest item is at most 3/4 of what a slot gets on average (whole lists: at
// most all of it, as the shorter ones fill the gaps), or that has
// kSlots items of at most 4 `least` positions, or that the next one would cut
// below `least` (whose work is about what a part costs in starting and
// joining); whole lists where that would shorten the longest item by less than
// `worth` positions, what the join launch costs.  *split
// (1..steps, may be null) spreads the steps over further work-groups.
// Measured (bf16, 8/2 heads of 128, least = 256 / 128 / 64): forward on a chain
// of 1024 tokens 21.8 / 24.2 / 36.0 us, backward on 600 tokens of 8/1 heads
// 47.5 / 42.4 / 44.0 us; fp32 (600 tokens, 8/2 heads of 64) 85 / 57 / 46 us.
constexpr int32_t kSlots = 512;
const AttnCut& choose_cut(const AttnLists& l, int32_t heads, int32_t steps, int32_t least, int32_t worth,
                          int32_t* split);

// Returns 0 or a negative TREE_ERR_* code; on failure *err holds a message and
// *out is as it was.
int build_attn_plan(const Plan& p, AttnPlan* out, std::string* err, int64_t max_runs = AttnPlan::kMaxRuns,
                    int64_t max_steps = AttnPlan::kMaxSteps);

}  // namespace tg
