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
// and v; a long list is cut into parts of at most kPart virtual rows, whose
// partial sums are added in the order of the parts.
#pragma once

#include <cstddef>
#include <cstdint>
#include <string>
#include <vector>

#include "plan.hpp"

namespace tg {

constexpr int32_t kQTile = 128;
constexpr int32_t kKTile = 128;
constexpr int32_t kPart = 2048;

// One tile's list of runs.  Virtual positions [v0, v1) of it are this item's
// work; [0, n_full) need no visibility test; n_total is the list's length.
struct AttnItem {
  int32_t tile;      // packed rows tile * kQTile (or kKTile) ..
  int32_t run_off;   // first run
  int32_t n_runs;
  int32_t n_full;
  int32_t n_total;
  int32_t v0, v1;
  int32_t part;      // key tiles: number of this part among all parts
};
struct AttnRun {
  int32_t virt;  // virtual position of the run's first row
  int32_t row;   // its packed row
};
// A key tile's parts: part0 .. part0 + n_parts - 1.
struct AttnParts {
  int32_t tile, part0, n_parts, pad;
};

struct AttnPlan {
  int32_t n_tokens = 0;
  int32_t n_qtiles = 0, n_kitems = 0, n_ktiles = 0;
  int32_t n_multi = 0;        // key tiles with more than one part (first in `parts`)
  int32_t n_multi_parts = 0;  // their parts (numbered first)
  // Entries a trie may need at most: the run lists of all tiles together.
  static constexpr int64_t kMaxRuns = int64_t(1) << 26;

  std::vector<int32_t> mirror;  // device copy
  size_t m_d = 0, m_e = 0, m_q = 0, m_k = 0, m_runs = 0, m_parts = 0;
  size_t device_bytes() const { return mirror.size() * sizeof(int32_t); }
};

// Returns 0 or a negative TREE_ERR_* code; on failure *err holds a message.
int build_attn_plan(const Plan& p, AttnPlan* out, std::string* err);

}  // namespace tg
