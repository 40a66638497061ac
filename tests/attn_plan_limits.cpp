// The refusals of the tree attention's host tables (csrc/attn_plan.cpp), with
// limits small enough for small tries.  Prints "limits hold" if they do.
#include <cstdint>
#include <cstdio>
#include <string>
#include <vector>

#include "../include/tree_gdn.h"
#include "../prefix_tree_packed_plan_amd/csrc/attn_plan.hpp"

static int failures = 0;

static void expect(const char* what, const std::vector<int32_t>& parents, const std::vector<int32_t>& lens,
                   int64_t max_runs, int64_t max_steps, const char* words) {
  tg::Plan p;
  std::string err;
  if (tg::build_plan(parents.data(), lens.data(), static_cast<int>(parents.size()), 4, &p, &err) != 0) {
    std::printf("FAILED %s: plan: %s\n", what, err.c_str());
    ++failures;
    return;
  }
  tg::AttnPlan a;
  a.n_tokens = -7;
  err.clear();
  const int rc = tg::build_attn_plan(p, &a, &err, max_runs, max_steps);
  const bool ok = words ? rc == TREE_ERR_UNSUPPORTED && err.find(words) != std::string::npos && a.n_tokens == -7
                        : rc == 0 && err.empty() && a.n_tokens == p.n_tokens;
  if (!ok) {
    std::printf("FAILED %s: code %d, message '%s'\n", what, rc, err.c_str());
    ++failures;
  }
}

int main() {
  const int64_t big = int64_t(1) << 40;
  // A root of 400 tokens with 300 children of 3: in depth-first order, and with
  // two roots whose children take turns.
  std::vector<int32_t> fan{-1}, fan_lens{400}, turns{-1, -1}, turns_lens{200, 200};
  for (int i = 0; i < 300; ++i) {
    fan.push_back(0);
    fan_lens.push_back(3);
    turns.push_back(i % 2);
    turns_lens.push_back(3);
  }
  expect("depth-first", fan, fan_lens, tg::AttnPlan::kMaxRuns, tg::AttnPlan::kMaxSteps, nullptr);
  expect("taking turns", turns, turns_lens, tg::AttnPlan::kMaxRuns, tg::AttnPlan::kMaxSteps, nullptr);
  expect("runs", turns, turns_lens, 100, big, "run lists exceed 100 entries");
  expect("runs of a chain", {-1}, {1000}, 4, big, "run lists exceed 4 entries");
  // Query tiles walk up from each of their segments: 300 and a few; key tiles
  // of the second numbering look at every segment below as well.
  expect("steps", turns, turns_lens, big, 200, "more than 200 steps over their segments (a depth-first numbering");
  expect("steps of the walk down", turns, turns_lens, big, 800, "more than 800 steps");
  expect("steps, depth-first", fan, fan_lens, big, 200, "more than 200 steps over their segments (a very deep");
  expect("enough steps, depth-first", fan, fan_lens, big, 1200, nullptr);
  if (!failures) std::printf("limits hold\n");
  return failures != 0;
}
