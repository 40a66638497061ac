// C ABI (include/tree_gdn.h): argument checks, the device plan, launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <exception>
#include <memory>
#include <mutex>
#include <new>
#include <string>
#include <vector>

#include "../../include/tree_gdn.h"
#include "attn_plan.hpp"
#include "launch.hpp"
#include "plan.hpp"

struct tree_plan {
  tg::Plan p;
  // Device buffers this plan was uploaded into (tree_plan_upload) and their
  // sizes.  The entry points accept a device plan only from this list, so a
  // stale, short or foreign buffer is rejected on the host before any launch.
  // The plan is otherwise immutable; the list has its own lock so that the
  // plan can be shared across threads.
  mutable std::mutex mu;
  mutable std::vector<std::pair<const void*, size_t>> uploads;
};

// The attention tables and, as for the plan, the buffers they were uploaded into.
struct tree_attention_plan {
  tg::AttnPlan p;
  mutable std::mutex mu;
  mutable std::vector<std::pair<const void*, size_t>> uploads;
};

namespace {

thread_local std::string g_err;

int fail(int code, const char* f, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, f);
  std::vsnprintf(buf, sizeof(buf), f, ap);
  va_end(ap);
  g_err = buf;
  return code;
}

int hip_fail(const char* what, hipError_t e) {
  return fail(TREE_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

bool dtype_ok(int32_t d) { return d == TREE_DTYPE_F32 || d == TREE_DTYPE_BF16; }

// The device plan passed to an entry point must be one tree_plan_upload made
// from this plan, of at least the plan's device size.
int check_dplan(const tree_plan_t* plan, const void* dplan, size_t dplan_bytes, const char* fn) {
  const size_t need = plan->p.device_bytes();
  if (dplan_bytes < need)
    return fail(TREE_ERR_WORKSPACE, "%s: dplan has %zu bytes, the plan needs %zu", fn, dplan_bytes, need);
  std::lock_guard<std::mutex> lock(plan->mu);
  for (const auto& u : plan->uploads)
    if (u.first == dplan) {
      if (dplan_bytes > u.second)
        return fail(TREE_ERR_INVALID_ARG, "%s: dplan_bytes %zu exceeds the %zu bytes it was uploaded with", fn,
                    dplan_bytes, u.second);
      return TREE_OK;
    }
  return fail(TREE_ERR_INVALID_ARG, "%s: dplan %p is not an upload of this plan (tree_plan_upload)", fn, dplan);
}

// The same for the attention tables.
int check_dplan(const tree_attention_plan_t* aplan, const void* dplan, size_t dplan_bytes, const char* fn) {
  const size_t need = aplan->p.device_bytes();
  if (dplan_bytes < need)
    return fail(TREE_ERR_WORKSPACE, "%s: dplan has %zu bytes, the attention plan needs %zu", fn, dplan_bytes, need);
  std::lock_guard<std::mutex> lock(aplan->mu);
  for (const auto& u : aplan->uploads)
    if (u.first == dplan) {
      if (dplan_bytes > u.second)
        return fail(TREE_ERR_INVALID_ARG, "%s: dplan_bytes %zu exceeds the %zu bytes it was uploaded with", fn,
                    dplan_bytes, u.second);
      return TREE_OK;
    }
  return fail(TREE_ERR_INVALID_ARG, "%s: dplan %p is not an upload of this attention plan (tree_attention_plan_upload)",
              fn, dplan);
}

// A factor whose products with log2(e) and with fp32 values of ordinary size
// neither overflow nor vanish.
bool ordinary(float x) { return x >= 1e-30f && x <= 1e30f; }
// Work-groups of 256 a launch may have (its work items are counted in 32 bits).
constexpr int64_t kMaxGroups = (int64_t(1) << 24) - 64;

// Grids: parts x heads; and heads along the join launches' second axis.
bool heads_fit(const tg::AttnPlan& p, int32_t h_q) {
  return h_q <= 65535 && (static_cast<int64_t>(p.q.n_tiles) + tg::AttnPlan::kMaxParts) * h_q <= kMaxGroups;
}
// Sizes, head layout and scale of an attention call.
int check_attention(const tg::AttnPlan& p, int64_t n_tokens, int32_t h_q, int32_t h_kv, int32_t d, float scale,
                    int32_t dtype, const char* fn) {
  if (n_tokens != p.n_tokens)
    return fail(TREE_ERR_SIZE, "%s: n_tokens %lld != plan tokens %lld", fn, static_cast<long long>(n_tokens),
                static_cast<long long>(p.n_tokens));
  if (h_q <= 0 || h_kv <= 0 || d <= 0) return fail(TREE_ERR_INVALID_ARG, "%s: head counts and sizes must be > 0", fn);
  if (!dtype_ok(dtype)) return fail(TREE_ERR_INVALID_ARG, "%s: bad dtype %d", fn, dtype);
  if (h_q % h_kv != 0)
    return fail(TREE_ERR_UNSUPPORTED, "%s: h_q %d is not a multiple of h_kv %d", fn, h_q, h_kv);
  if (!tg::attention_supported(d, dtype))
    return fail(TREE_ERR_UNSUPPORTED, "%s: d=%d dtype=%d not compiled in", fn, d, dtype);
  if (!ordinary(scale)) return fail(TREE_ERR_INVALID_ARG, "%s: scale must be in 1e-30..1e30", fn);
  if (!heads_fit(p, h_q))
    return fail(TREE_ERR_UNSUPPORTED, "%s: too many heads (%d) for %d tiles", fn, h_q, p.q.n_tiles);
  return TREE_OK;
}
// A [n_tokens, heads, d] tensor read 16 bytes at a time: `strides` holds the
// elements between token rows and between heads, or is null for a contiguous
// tensor.
int make_heads(const void* ptr, const int64_t* strides, int32_t heads, int32_t d, int32_t dtype, const char* name,
               const char* fn, tg::Heads* out) {
  const int64_t size = dtype == TREE_DTYPE_F32 ? 4 : 2;
  const int64_t row = (strides ? strides[0] : static_cast<int64_t>(heads) * d) * size;
  const int64_t head = (strides ? strides[1] : d) * size;
  const int64_t most = int64_t(1) << 40;
  if (row < 0 || head < 0 || row > most || head > most)
    return fail(TREE_ERR_INVALID_ARG, "%s: bad strides of %s", fn, name);
  if (reinterpret_cast<uintptr_t>(ptr) % 16 != 0 || row % 16 != 0 || head % 16 != 0)
    return fail(TREE_ERR_INVALID_ARG, "%s: %s is not aligned to 16 bytes in every row and head", fn, name);
  *out = tg::Heads{static_cast<const char*>(ptr), row, head};
  return TREE_OK;
}
int check_aligned(const void* ptr, const char* name, const char* fn) {
  if (reinterpret_cast<uintptr_t>(ptr) % 16 != 0)
    return fail(TREE_ERR_INVALID_ARG, "%s: %s is not aligned to 16 bytes", fn, name);
  return TREE_OK;
}

int check_element_aligned(const void* ptr, int32_t dtype, const char* name, const char* fn) {
  if (reinterpret_cast<uintptr_t>(ptr) % (dtype == TREE_DTYPE_F32 ? 4 : 2) != 0)
    return fail(TREE_ERR_INVALID_ARG, "%s: %s is not aligned to its elements", fn, name);
  return TREE_OK;
}

// How a call's lists are cut, and the parts whose results go to the workspace.
struct Work {
  const tg::AttnCut* cut;
  int32_t split, n_join, n_parts;
};
Work attention_work(const tg::AttnLists& l, int32_t heads, int32_t steps, int32_t d, int32_t dtype) {
  Work w{};
  // Starting and joining a part costs about 4 tiles of bf16, and the join
  // launch 2; fp32 products take 16 times as long (192 tokens in fp32, cut into
  // parts of 64 or not: forward of one head of 32 22.4 / 16.8 us, backward of
  // two heads of 64 34 / 56 us).
  const bool f32 = dtype == TREE_DTYPE_F32;
  w.cut = &tg::choose_cut(l, heads, steps, f32 ? 64 : 256, f32 ? 8192 / d : 128, steps > 1 ? &w.split : nullptr);
  if (w.split < 1) w.split = 1;
  w.n_join = w.split > 1 ? l.n_tiles : w.cut->n_multi;
  w.n_parts = w.split > 1 ? w.cut->n_items : w.cut->n_multi_parts;
  return w;
}
void set_work(const Work& w, const int32_t* base, tg::AttnArgs* a) {
  a->items = reinterpret_cast<const tg::AttnItem*>(base + w.cut->m_items);
  a->parts = reinterpret_cast<const tg::AttnParts*>(base + w.cut->m_parts);
  a->n_items = w.cut->n_items;
  a->n_join = w.n_join;
  a->n_parts = w.n_parts;
  a->split = w.split;
}
size_t attention_delta_bytes(const tg::AttnPlan& p, int32_t h_q) {
  return (2 * static_cast<size_t>(p.n_tokens) * h_q * sizeof(float) + 255) / 256 * 256;
}

// Work-groups a row is spread over: of at least `least` of them, as many as
// bring the grid to `want` work-groups with slices of at least `cols` columns;
// a slice starts on 128 bytes.
struct Spread {
  int32_t split, slice;
};
Spread spread(int32_t n_rows, int32_t vocab, int64_t least, int64_t want, int64_t cols) {
  int64_t s = std::min<int64_t>((want - 1 + n_rows) / n_rows, (static_cast<int64_t>(vocab) + cols - 1) / cols);
  s = std::max<int64_t>({s, least, 1});
  const int64_t slice = ((vocab + s - 1) / s + 63) / 64 * 64;
  return {static_cast<int32_t>((vocab + slice - 1) / slice), static_cast<int32_t>(slice)};
}
// Forward: only where the rows alone leave CUs idle, as the slices' sums cost
// a second launch.
Spread logprob_spread(int32_t n_rows, int32_t vocab) { return spread(n_rows, vocab, 1, n_rows >= 512 ? 1 : 1024, 2048); }
// Backward: nothing to join, so a slice is what a work-group loads at a time
// (16 KB): neighbouring work-groups then stream through neighbouring memory
// (8192 rows of 131072 columns in bf16: 701 us, against 744 and 778 us with two
// and four times that, and 819 us with whole rows).
Spread logprob_backward_spread(int32_t n_rows, int32_t vocab, int32_t dtype) {
  const int32_t round = 16384 / (dtype == TREE_DTYPE_F32 ? 4 : 2);
  const int64_t s = (static_cast<int64_t>(vocab) + round - 1) / round;
  if (s * n_rows >= 4096) return {static_cast<int32_t>(s), round};
  return spread(n_rows, vocab, 1, 4096, 2048);
}

int check_logprobs(const tg::Plan& p, int64_t ld, int64_t n_tokens, int32_t first_row, int32_t n_rows, int32_t vocab,
                   int32_t token_bytes, float temperature, int32_t dtype, const char* fn) {
  if (n_tokens != p.n_tokens)
    return fail(TREE_ERR_SIZE, "%s: n_tokens %lld != plan tokens %lld", fn, static_cast<long long>(n_tokens),
                static_cast<long long>(p.n_tokens));
  if (first_row < 0 || n_rows <= 0 || static_cast<int64_t>(first_row) + n_rows > p.n_tokens)
    return fail(TREE_ERR_INVALID_ARG, "%s: rows %d .. +%d are not rows of the plan's %lld tokens", fn, first_row, n_rows,
                static_cast<long long>(p.n_tokens));
  if (vocab <= 0 || vocab > (1 << 30)) return fail(TREE_ERR_INVALID_ARG, "%s: vocab %d must be in 1..2^30", fn, vocab);
  if (ld < vocab || ld > (int64_t(1) << 40))
    return fail(TREE_ERR_INVALID_ARG, "%s: rows %lld elements apart hold %d", fn, static_cast<long long>(ld), vocab);
  if (token_bytes != 4 && token_bytes != 8)
    return fail(TREE_ERR_INVALID_ARG, "%s: token_bytes must be 4 or 8 (got %d)", fn, token_bytes);
  if (!ordinary(temperature)) return fail(TREE_ERR_INVALID_ARG, "%s: temperature must be in 1e-30..1e30", fn);
  if (!dtype_ok(dtype)) return fail(TREE_ERR_INVALID_ARG, "%s: bad dtype %d", fn, dtype);
  return TREE_OK;
}

// Sizes of an embedding call.  Up to 2^30 tokens and rows of the table: positions
// and rows are counted in 32 bits, with room for what a wave reads past the end.
constexpr int32_t kEmbedVocab = 1 << 30;
// The gradient's: every kEmbedSpan rows of the table look through all tokens.
constexpr int32_t kSortVocab = 1 << 22;
bool embed_sizes_ok(int64_t n_tokens, int32_t vocab, int32_t width, int32_t most) {
  return n_tokens >= 0 && n_tokens <= (int64_t(1) << 30) && vocab > 0 && vocab <= most && width > 0 &&
         width <= (1 << 24);
}
int check_embed(int64_t n_tokens, int32_t vocab, int32_t width, int32_t most, int32_t token_bytes, float scale,
                int32_t dtype, const char* fn) {
  if (!embed_sizes_ok(n_tokens, vocab, width, most))
    return fail(TREE_ERR_INVALID_ARG, "%s: n_tokens %lld must be in 0..2^30, vocab %d in 1..%d, width %d in 1..2^24", fn,
                static_cast<long long>(n_tokens), vocab, most, width);
  if (token_bytes != 4 && token_bytes != 8)
    return fail(TREE_ERR_INVALID_ARG, "%s: token_bytes must be 4 or 8 (got %d)", fn, token_bytes);
  if (!dtype_ok(dtype)) return fail(TREE_ERR_INVALID_ARG, "%s: bad dtype %d", fn, dtype);
  if (!ordinary(scale)) return fail(TREE_ERR_INVALID_ARG, "%s: scale must be in 1e-30..1e30", fn);
  return TREE_OK;
}
// The workspace of the embedding's gradient.
struct EmbedWork {
  size_t order, part, bytes;  // offsets, and all of it
  int32_t n_parts, span;
};
EmbedWork embed_work(int64_t n_tokens, int32_t vocab, int32_t width) {
  const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  EmbedWork w{};
  w.n_parts = n_tokens > tg::kEmbedPart ? static_cast<int32_t>((n_tokens + tg::kEmbedPart - 1) / tg::kEmbedPart) : 0;
  w.order = up((static_cast<size_t>(vocab) + 1) * sizeof(int32_t));
  w.part = w.order + up(static_cast<size_t>(n_tokens) * sizeof(int2));
  w.bytes = w.part + static_cast<size_t>(w.n_parts) * 2 * width * sizeof(float);
  // 512 work-groups (two on each CU) share the table, as long as their rows fit.
  w.span = std::min<int32_t>((vocab + 511) / 512, tg::kEmbedSpan);
  return w;
}

// ---- log probabilities from hidden states -----------------------------------------
constexpr int32_t kLinearVocab = 1 << 22, kLinearWidth = 1 << 16;
size_t up256(size_t x) { return (x + 255) / 256 * 256; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tile sizes and splits of a product of m x n over k.  Up to 64 rows n take 64 of them a
// tile, and a sum as many splits as fill the CUs; so do logits, which cannot be split,
// as long as the 64 x 64 tiles run at once (106 rows x 3135 x 4032 fp32 100 us, with 128 x
// 128 195, bf16 23 and 48; 512 tiles, 256 rows x 8192 x 2048, fp32 80 and 104, bf16 23 and
// 29; but 1024 tiles, 512 x 8192 x 2048, fp32 147 and 105, bf16 39 and 30).  Otherwise the least of: rounds of
// work-groups (256 tiles of 256 x 256, one a CU; 512 of 128 x 128, two) times a round's
// time, in us as measured for a k-step of it, and the parts' way through memory.  Large
// bf16 products so take 256 x 256 (8192 x 131072 x 4096 forward 6480 us, with 128 x 128
// 8350); where those leave CUs idle, 128 x 128 (100 rows x 50000 x 2048: 40.5 us, 61 with
// 256 x 256) or, for sums, splits (gradients of 1100 x 50000 x 4096: 1311 us with 256 x
// 256 in 3 splits, 1815 with 128 x 128).  fp32 takes 128 x 128: one work-group splits
// values while the other's products run (1685 rows x 50001 x 1000 forward as fast as
// with 256 x 256, the gradients of 1526 x 20001 x 1000 1290 -> 1030 us).
struct ProductChoice {
  int32_t size, splits;
};
ProductChoice product_choice(int64_t m, int64_t n, int64_t k, int32_t dtype, bool sum, bool few) {
  const bool f32 = dtype == TREE_DTYPE_F32;
  const int64_t steps = ceil_div(k, f32 ? 32 : 64), most = sum ? std::max<int64_t>(1, steps / 8) : 1;
  if (!sum && ceil_div(m, 64) * ceil_div(n, 64) <= 512) return {0, 1};
  if (few && n <= 64)
    return {0, static_cast<int32_t>(std::max<int64_t>(1, std::min(512 / (ceil_div(m, 128) * ceil_div(n, 64)), most)))};
  ProductChoice best{};
  double least = 0;
  for (int size = f32 ? 1 : 2; size >= 1; --size) {
    const int64_t b = size == 2 ? 256 : 128, at_once = size == 2 ? 256 : 512;
    const double step_us = f32 ? 2.7 : size == 2 ? 1.57 : 1.0;
    const int64_t tiles = ceil_div(m, b) * ceil_div(n, b);
    for (int64_t s = 1; s <= std::min<int64_t>(most, 64); ++s) {
      const double rounds = static_cast<double>(ceil_div(tiles * s, at_once));
      double us = rounds * (static_cast<double>(ceil_div(steps, s)) * step_us + 1.0);
      if (s > 1) us += 5.0 + static_cast<double>(s) * m * n * 8 / 5e6;
      if (best.size == 0 || us < least) {
        best = {size, static_cast<int32_t>(s)};
        least = us;
      }
    }
  }
  return best;
}
bool linear_sizes_ok(int64_t n_rows, int32_t vocab, int32_t width, int32_t dtype) {
  return n_rows > 0 && n_rows < (int64_t(1) << 31) && vocab > 0 && vocab <= kLinearVocab && width > 0 &&
         width <= kLinearWidth && dtype_ok(dtype) && width % (dtype == TREE_DTYPE_F32 ? 4 : 8) == 0;
}
// The forward's: the tiles' sums of up to 32768 rows, 1 GiB of them at most.
tg::LinearWork linear_work(int64_t n_rows, int32_t vocab, int32_t width, int32_t dtype) {
  tg::LinearWork w{};
  w.rows = std::min<int64_t>(n_rows, 32768);
  w.size = product_choice(vocab, w.rows, width, dtype, false, true).size;
  const int64_t slots = ceil_div(vocab, w.size == 2 ? 256 : w.size == 1 ? 128 : 64);
  w.rows = std::min(w.rows, std::max<int64_t>(256, (int64_t(1) << 26) / slots / 256 * 256));
  w.ids = static_cast<size_t>(w.rows) * slots * 16;
  w.bytes = w.ids + static_cast<size_t>(w.rows) * 16;
  return w;
}
// The backward's: D of up to 16384 rows and a piece of the vocabulary, 256 Mi elements
// at most; dhidden and dweight in fp32 where they are added up over several.
tg::LinearWork linear_backward_work(int64_t n_rows, int32_t vocab, int32_t width, int32_t dtype) {
  tg::LinearWork w{};
  const size_t es = dtype == TREE_DTYPE_F32 ? 4 : 2;
  w.rows = std::min<int64_t>(n_rows, 16384);
  const int64_t rows_up = ceil_div(w.rows, 256) * 256;
  w.piece = std::min<int64_t>(vocab, (int64_t(1) << 28) / rows_up / 256 * 256);
  w.ldd = ceil_div(w.piece, 256) * 256;
  w.size = product_choice(w.piece, w.rows, width, dtype, false, true).size;
  // Up to 64 rows in bf16, where memory is the bound, D is two bf16 (its rounding would
  // be as large as the result's): 2 stack rows.
  w.stack = dtype == TREE_DTYPE_BF16 && n_rows <= 64 ? (n_rows <= 32 ? 32 : 64) : 0;
  const int64_t d_rows = w.stack ? 2 * w.stack : w.rows;
  const ProductChoice h = product_choice(width, d_rows, w.piece, dtype, true, true);
  const ProductChoice d = product_choice(width, w.piece, d_rows, dtype, true, false);
  w.size_h = h.size;
  w.splits_h = h.splits;
  w.size_w = d.size;
  w.splits_w = d.splits;
  const size_t fw = static_cast<size_t>(width) * sizeof(float);
  w.ids = up256(w.rows * 16);
  w.d = w.ids + up256(w.rows * 16);
  w.dhidden = w.d + static_cast<size_t>(rows_up) * w.ldd * es;
  w.dweight = w.dhidden + (w.piece < vocab ? up256(w.rows * fw) : 0);
  w.hidden2 = w.dweight + (w.rows < n_rows ? up256(vocab * fw) : 0);
  w.parts = w.hidden2 + up256(2 * w.stack * width * es);
  const size_t ph = w.splits_h > 1 || w.stack ? w.splits_h * d_rows * fw : 0, pw = w.splits_w > 1 ? w.splits_w * w.piece * fw : 0;
  w.bytes = w.parts + std::max(ph, pw);
  return w;
}
// What both directions check (the rows and tokens as check_logprobs does).
int check_linear(const tg::Plan& p, const void* hidden, int64_t ld, const void* weight, int64_t n_tokens,
                 int32_t first_row, int32_t n_rows, int32_t vocab, int32_t width, int32_t token_bytes,
                 float temperature, int32_t dtype, const char* fn) {
  if (const int rc = check_logprobs(p, vocab, n_tokens, first_row, n_rows, vocab, token_bytes, temperature, dtype, fn))
    return rc;
  if (width <= 0) return fail(TREE_ERR_INVALID_ARG, "%s: width must be > 0", fn);
  const int64_t es = dtype == TREE_DTYPE_F32 ? 4 : 2;
  if (!linear_sizes_ok(n_rows, vocab, width, dtype))
    return fail(TREE_ERR_UNSUPPORTED, "%s: width %d must be a multiple of %lld up to %d, vocab %d at most %d", fn, width,
                static_cast<long long>(16 / es), kLinearWidth, vocab, kLinearVocab);
  if (ld < width || ld > (1 << 20))
    return fail(TREE_ERR_INVALID_ARG, "%s: rows of hidden %lld elements apart must hold %d, at most 2^20", fn,
                static_cast<long long>(ld), width);
  if (ld * es % 16 != 0)
    return fail(TREE_ERR_INVALID_ARG, "%s: rows of hidden are not aligned to 16 bytes", fn);
  if (const int rc = check_aligned(hidden, "hidden", fn)) return rc;
  return check_aligned(weight, "weight", fn);
}
void set_linear(const tg::Plan& p, const void* hidden, int64_t ld, const void* weight, const void* tokens,
                int32_t first_row, int32_t n_rows, int32_t vocab, int32_t width, int32_t token_bytes,
                float temperature, const void* dplan, void* ws, tg::LinearArgs* a) {
  const int32_t* base = static_cast<const int32_t*>(dplan);
  a->hidden = hidden;
  a->ld = ld;
  a->weight = weight;
  a->tokens = tokens;
  a->token64 = token_bytes == 8;
  a->first_row = first_row;
  a->n_rows = n_rows;
  a->vocab = vocab;
  a->width = width;
  a->inv_t = 1.f / temperature;
  a->ws = ws;
  a->seg_off = base + p.m_seg_off;
  a->parent = base + p.m_parent;
  a->kid_off = base + p.m_kid_off;
  a->kid = base + p.m_kid;
  a->n_seg = p.n_seg;
}

// Blocks along the tokens of the conv backward (each walks every n-th tile).
int32_t conv_bwd_parts(const tg::Plan& p) {
  const int64_t tiles = (p.n_tokens + 63) / 64;
  return static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(tiles, 512)));
}

}  // namespace

extern "C" {

int tree_plan(const int32_t* parents, const int32_t* seg_lens, int32_t n_seg, int32_t conv_width,
              tree_plan_t** out) {
  if (!out) return fail(TREE_ERR_INVALID_ARG, "tree_plan: out is null");
  *out = nullptr;
  tree_plan_t* plan = new (std::nothrow) tree_plan_t;
  if (!plan) return fail(TREE_ERR_INVALID_ARG, "tree_plan: out of host memory");
  std::string err;
  const int rc = tg::build_plan(parents, seg_lens, n_seg, conv_width, &plan->p, &err);
  if (rc != TREE_OK) {
    delete plan;
    g_err = err;
    return rc;
  }
  *out = plan;
  return TREE_OK;
}

void tree_plan_free(tree_plan_t* plan) { delete plan; }

int tree_plan_query(const tree_plan_t* plan, tree_plan_stats_t* out) {
  if (!plan || !out) return fail(TREE_ERR_INVALID_ARG, "tree_plan_query: null argument");
  const tg::Plan& p = plan->p;
  out->n_tokens = p.n_tokens;
  out->path_tokens = p.path_tokens;
  out->max_path_tokens = p.max_path_tokens;
  out->por = p.path_tokens > 0 ? 1.0 - static_cast<double>(p.n_tokens) / p.path_tokens : 0.0;
  out->n_seg = p.n_seg;
  out->n_roots = p.n_roots;
  out->n_leaves = p.n_leaves;
  out->n_parents = p.n_parents;
  out->n_levels = p.n_levels;
  out->conv_width = p.width;
  out->path_entries = p.paths_ok ? p.path_entries : -1;
  return TREE_OK;
}

int tree_plan_paths(const tree_plan_t* plan, int32_t* path_off, int32_t* path_seg) {
  if (!plan || !path_off || !path_seg) return fail(TREE_ERR_INVALID_ARG, "tree_plan_paths: null argument");
  if (!plan->p.paths_ok)
    return fail(TREE_ERR_UNSUPPORTED, "tree_plan_paths: walk table of %lld entries not built",
                static_cast<long long>(plan->p.path_entries));
  std::copy(plan->p.path_off.begin(), plan->p.path_off.end(), path_off);
  std::copy(plan->p.path_seg.begin(), plan->p.path_seg.end(), path_seg);
  return TREE_OK;
}

int tree_plan_choose_schedule(const tree_plan_t* plan, int64_t fork_min_saved_tokens, int32_t* sched) {
  if (!plan || !sched) return fail(TREE_ERR_INVALID_ARG, "tree_plan_choose_schedule: null argument");
  if (fork_min_saved_tokens < 0)
    return fail(TREE_ERR_INVALID_ARG, "tree_plan_choose_schedule: fork_min_saved_tokens %lld < 0",
                static_cast<long long>(fork_min_saved_tokens));
  *sched = tg::choose_schedule(plan->p, fork_min_saved_tokens);
  return TREE_OK;
}

int tree_plan_conv_history(const tree_plan_t* plan, int32_t* hist) {
  if (!plan || !hist) return fail(TREE_ERR_INVALID_ARG, "tree_plan_conv_history: null argument");
  std::copy(plan->p.hist.begin(), plan->p.hist.end(), hist);
  return TREE_OK;
}

int tree_plan_levels(const tree_plan_t* plan, int32_t* level_start, int32_t* order) {
  if (!plan || !level_start || !order)
    return fail(TREE_ERR_INVALID_ARG, "tree_plan_levels: null argument");
  std::copy(plan->p.level_start.begin(), plan->p.level_start.end(), level_start);
  std::copy(plan->p.order.begin(), plan->p.order.end(), order);
  return TREE_OK;
}

size_t tree_plan_device_bytes(const tree_plan_t* plan) { return plan ? plan->p.device_bytes() : 0; }

int tree_plan_upload(const tree_plan_t* plan, void* dplan, size_t dplan_bytes, void* stream) {
  if (!plan || !dplan) return fail(TREE_ERR_INVALID_ARG, "tree_plan_upload: null argument");
  if (dplan_bytes < plan->p.device_bytes())
    return fail(TREE_ERR_WORKSPACE, "tree_plan_upload: dplan has %zu bytes, needs %zu", dplan_bytes,
                plan->p.device_bytes());
  const hipError_t e = hipMemcpyAsync(dplan, plan->p.mirror.data(), plan->p.device_bytes(),
                                      hipMemcpyHostToDevice, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail("tree_plan_upload: hipMemcpyAsync", e);
  std::lock_guard<std::mutex> lock(plan->mu);
  for (auto& u : plan->uploads)
    if (u.first == dplan) {
      u.second = dplan_bytes;
      return TREE_OK;
    }
  plan->uploads.emplace_back(dplan, dplan_bytes);
  return TREE_OK;
}

int tree_conv(const void* x, const void* w, const void* bias, void* y, const void* init_ctx,
              void* ctx_out, int64_t n_tokens, int32_t channels, int32_t dtype, int32_t act,
              const tree_plan_t* plan, const void* dplan, size_t dplan_bytes, void* stream) {
  if (!plan || !x || !w || !y || !dplan) return fail(TREE_ERR_INVALID_ARG, "tree_conv: null argument");
  const tg::Plan& p = plan->p;
  if (n_tokens != p.n_tokens)
    return fail(TREE_ERR_SIZE, "tree_conv: n_tokens %lld != plan tokens %lld",
                static_cast<long long>(n_tokens), static_cast<long long>(p.n_tokens));
  if (channels <= 0) return fail(TREE_ERR_INVALID_ARG, "tree_conv: channels must be > 0");
  if (!dtype_ok(dtype)) return fail(TREE_ERR_INVALID_ARG, "tree_conv: bad dtype %d", dtype);
  if (act != TREE_ACT_NONE && act != TREE_ACT_SILU)
    return fail(TREE_ERR_INVALID_ARG, "tree_conv: bad activation %d", act);
  if (p.width > 4) return fail(TREE_ERR_UNSUPPORTED, "tree_conv: conv width %d > 4", p.width);
  if (x == y) return fail(TREE_ERR_INVALID_ARG, "tree_conv: y must not alias x");
  if (ctx_out != nullptr && (ctx_out == x || ctx_out == y || ctx_out == init_ctx))
    return fail(TREE_ERR_INVALID_ARG, "tree_conv: ctx_out must not alias x, y or init_ctx");
  if (const int rc = check_dplan(plan, dplan, dplan_bytes, "tree_conv")) return rc;
  const int32_t* base = static_cast<const int32_t*>(dplan);
  tg::ConvArgs a{x, w, bias, y, static_cast<int32_t>(n_tokens), channels, p.width, dtype, act,
                 base + p.m_seg_off, base + p.m_hist, p.n_seg, init_ctx, ctx_out, base + p.m_ctx};
  const hipError_t e = tg::launch_conv(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail("tree_conv: launch", e);
  return TREE_OK;
}

size_t tree_conv_backward_workspace_bytes(const tree_plan_t* plan, int32_t channels) {
  if (!plan || channels <= 0) return 0;
  const tg::Plan& p = plan->p;
  const size_t heads = static_cast<size_t>(p.n_seg) * std::max(p.width - 1, 0) * channels;
  const size_t part = static_cast<size_t>(conv_bwd_parts(p)) * channels * (p.width + 1);
  return (heads + part) * sizeof(float);
}

int tree_conv_backward(const void* x, const void* w, const void* bias, const void* dy, const void* init_ctx,
                       void* dx, float* dw, float* dbias, float* dinit_ctx, int64_t n_tokens, int32_t channels,
                       int32_t dtype, int32_t act, const tree_plan_t* plan, const void* dplan,
                       size_t dplan_bytes, void* ws, size_t ws_bytes, void* stream) {
  if (!plan || !x || !w || !dy || !dx || !dw || !dplan)
    return fail(TREE_ERR_INVALID_ARG, "tree_conv_backward: null argument");
  const tg::Plan& p = plan->p;
  if (n_tokens != p.n_tokens)
    return fail(TREE_ERR_SIZE, "tree_conv_backward: n_tokens %lld != plan tokens %lld",
                static_cast<long long>(n_tokens), static_cast<long long>(p.n_tokens));
  if (channels <= 0) return fail(TREE_ERR_INVALID_ARG, "tree_conv_backward: channels must be > 0");
  if (!dtype_ok(dtype)) return fail(TREE_ERR_INVALID_ARG, "tree_conv_backward: bad dtype %d", dtype);
  if (act != TREE_ACT_NONE && act != TREE_ACT_SILU)
    return fail(TREE_ERR_INVALID_ARG, "tree_conv_backward: bad activation %d", act);
  if (p.width > 4) return fail(TREE_ERR_UNSUPPORTED, "tree_conv_backward: conv width %d > 4", p.width);
  if (dx == x || dx == dy) return fail(TREE_ERR_INVALID_ARG, "tree_conv_backward: dx must not alias x or dy");
  const size_t need = tree_conv_backward_workspace_bytes(plan, channels);
  if (!ws || ws_bytes < need)
    return fail(TREE_ERR_WORKSPACE, "tree_conv_backward: workspace has %zu bytes, needs %zu", ws ? ws_bytes : 0,
                need);
  if (const int rc = check_dplan(plan, dplan, dplan_bytes, "tree_conv_backward")) return rc;
  const int32_t* base = static_cast<const int32_t*>(dplan);
  tg::ConvBwdArgs a{};
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.dy = dy;
  a.init_ctx = init_ctx;
  a.dx = dx;
  a.dw = dw;
  a.dbias = bias ? dbias : nullptr;
  a.dinit_ctx = p.width > 1 ? dinit_ctx : nullptr;
  a.heads = static_cast<float*>(ws);
  a.part = a.heads + static_cast<size_t>(p.n_seg) * std::max(p.width - 1, 0) * channels;
  a.n_part = conv_bwd_parts(p);
  a.n_tok = static_cast<int32_t>(n_tokens);
  a.channels = channels;
  a.width = p.width;
  a.dtype = dtype;
  a.act = act;
  a.n_seg = p.n_seg;
  a.n_roots = p.n_roots;
  a.seg_off = base + p.m_seg_off;
  a.hist = base + p.m_hist;
  a.fut_off = base + p.m_fut_off;
  a.fut = base + p.m_fut;
  a.ent_off = base + p.m_ent_off;
  a.ent = base + p.m_ent;
  a.roots = base + p.m_roots;
  const hipError_t e = tg::launch_conv_backward(a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail("tree_conv_backward: launch", e);
  return TREE_OK;
}

size_t tree_scan_workspace_bytes(const tree_plan_t* plan, int32_t h_v, int32_t d_k, int32_t d_v,
                                 int32_t with_states) {
  if (!plan || h_v <= 0 || d_k <= 0 || d_v <= 0 || with_states) return 0;
  return static_cast<size_t>(plan->p.n_parents) * h_v * d_k * d_v * sizeof(float);
}

size_t tree_workspace_bytes(const tree_plan_t* plan, int32_t h_v, int32_t d_k, int32_t d_v, int32_t sched) {
  if (!plan) return 0;
  if (sched == TREE_SCHED_AUTO) sched = tg::choose_schedule(plan->p, TREE_FORK_MIN_SAVED_TOKENS);
  if (sched != TREE_SCHED_LEVEL) return 0;
  return tree_scan_workspace_bytes(plan, h_v, d_k, d_v, 0);
}

}  // extern "C"

namespace {

// Argument checks shared by tree_gdn_scan and tree_gdn_scan_noalloc (all but
// the device plan and the workspace).  Resolves AUTO into *sched and returns
// in *need the parent-slot bytes the level schedule needs.
int check_scan(const char* fn, const void* q, const void* k, const void* v, const float* g, const float* beta,
               void* o, const float* states, int64_t n_tokens, int32_t h_qk, int32_t h_v, int32_t d_k, int32_t d_v,
               int32_t dtype, int32_t* sched, const tree_plan_t* plan, size_t* need) {
  if (!plan || !q || !k || !v || !g || !beta || !o) return fail(TREE_ERR_INVALID_ARG, "%s: null argument", fn);
  const tg::Plan& p = plan->p;
  if (n_tokens != p.n_tokens)
    return fail(TREE_ERR_SIZE, "%s: n_tokens %lld != plan tokens %lld", fn, static_cast<long long>(n_tokens),
                static_cast<long long>(p.n_tokens));
  if (h_qk <= 0 || h_v <= 0 || d_k <= 0 || d_v <= 0)
    return fail(TREE_ERR_INVALID_ARG, "%s: head counts and sizes must be > 0", fn);
  if (h_v % h_qk != 0)
    return fail(TREE_ERR_UNSUPPORTED, "%s: h_v %d is not a multiple of h_qk %d", fn, h_v, h_qk);
  if (!dtype_ok(dtype)) return fail(TREE_ERR_INVALID_ARG, "%s: bad dtype %d", fn, dtype);
  if (*sched == TREE_SCHED_AUTO) *sched = tg::choose_schedule(p, TREE_FORK_MIN_SAVED_TOKENS);
  if (*sched != TREE_SCHED_LEVEL && *sched != TREE_SCHED_RESCAN)
    return fail(TREE_ERR_INVALID_ARG, "%s: bad schedule %d", fn, *sched);
  if (*sched == TREE_SCHED_RESCAN && !p.paths_ok)
    return fail(TREE_ERR_UNSUPPORTED, "%s: rescan walk table of %lld entries not built", fn,
                static_cast<long long>(p.path_entries));
  if (!tg::scan_supported(d_k, d_v, dtype))
    return fail(TREE_ERR_UNSUPPORTED, "%s: d_k=%d d_v=%d dtype=%d not compiled in", fn, d_k, d_v, dtype);
  *need = *sched == TREE_SCHED_LEVEL ? tree_scan_workspace_bytes(plan, h_v, d_k, d_v, states != nullptr) : 0;
  return TREE_OK;
}

// The scan's launches on a device plan `base` and parent-state slots `slots`.
int launch_scan_levels(const char* fn, const void* q, const void* k, const void* v, const float* g,
                       const float* beta, void* o, const float* init_states, float* states, int32_t h_qk,
                       int32_t h_v, int32_t d_k, int32_t d_v, float scale, int32_t dtype, int32_t sched,
                       const tg::Plan& p, const int32_t* base, float* slots, hipStream_t st) {
  tg::ScanArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.o = o;
  a.init = init_states;
  a.root_idx = base + p.m_root;
  a.states = states;
  a.slots = slots;
  a.seg_off = base + p.m_seg_off;
  a.parent = base + p.m_parent;
  a.slot = base + p.m_slot;
  a.h_qk = h_qk;
  a.h_v = h_v;
  a.scale = scale;
  if (sched == TREE_SCHED_RESCAN) {
    a.walk_off = base + p.m_path_off;
    a.walk = base + p.m_path_seg;
    a.n_items = p.n_leaves;
    const hipError_t e = tg::launch_scan(a, d_k, d_v, dtype, true, st);
    if (e != hipSuccess) return hip_fail(fn, e);
    return TREE_OK;
  }
  for (int32_t l = 0; l < p.n_levels; ++l) {
    a.items = base + p.m_order + p.level_start[l];
    a.n_items = p.level_start[l + 1] - p.level_start[l];
    const hipError_t e = tg::launch_scan(a, d_k, d_v, dtype, false, st);
    if (e != hipSuccess) return hip_fail(fn, e);
  }
  return TREE_OK;
}

// Device scratch of tree_gdn_scan_noalloc: the device plan at offset 0, the
// parent-state slots from the next 256-byte boundary.  Each GPU holds its own
// copy for the life of the process.  In host code `scratch` names a host-side
// stand-in, never the device memory: the device address comes from
// hipGetSymbolAddress, once per device, and only that address is used.
static __device__ __align__(256) unsigned char scratch[TREE_NOALLOC_SCRATCH_BYTES];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices] = {};

int scratch_on_current_device(const char* fn, unsigned char** out) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(fn, e);
  if (dev < 0 || dev >= kMaxDevices) return fail(TREE_ERR_UNSUPPORTED, "%s: device %d out of range", fn, dev);
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* ptr = nullptr;
    e = hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch));
    if (e != hipSuccess) return hip_fail(fn, e);
    if (!ptr) return fail(TREE_ERR_HIP, "%s: no device address for the scratch array", fn);
    g_scratch_ptr[dev] = ptr;
  }
  *out = static_cast<unsigned char*>(g_scratch_ptr[dev]);
  return TREE_OK;
}

}  // namespace

extern "C" {

int tree_gdn_scan(const void* q, const void* k, const void* v, const float* g, const float* beta,
                  void* o, const float* init_states, float* states, int64_t n_tokens, int32_t h_qk,
                  int32_t h_v, int32_t d_k, int32_t d_v, float scale, int32_t dtype, int32_t sched,
                  const tree_plan_t* plan, const void* dplan, size_t dplan_bytes, void* ws, size_t ws_bytes,
                  void* stream) {
  size_t need = 0;
  if (const int rc = check_scan("tree_gdn_scan", q, k, v, g, beta, o, states, n_tokens, h_qk, h_v, d_k, d_v, dtype,
                                &sched, plan, &need))
    return rc;
  if (!dplan) return fail(TREE_ERR_INVALID_ARG, "tree_gdn_scan: null argument");
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(TREE_ERR_WORKSPACE, "tree_gdn_scan: workspace has %zu bytes, needs %zu", ws ? ws_bytes : 0,
                need);
  if (const int rc = check_dplan(plan, dplan, dplan_bytes, "tree_gdn_scan")) return rc;
  return launch_scan_levels("tree_gdn_scan: launch", q, k, v, g, beta, o, init_states, states, h_qk, h_v, d_k, d_v,
                            scale, dtype, sched, plan->p, static_cast<const int32_t*>(dplan),
                            static_cast<float*>(ws), static_cast<hipStream_t>(stream));
}

int tree_gdn_scan_noalloc(const void* q, const void* k, const void* v, const float* g, const float* beta, void* o,
                          const float* init_states, float* states, int64_t n_tokens, int32_t h_qk, int32_t h_v,
                          int32_t d_k, int32_t d_v, float scale, int32_t dtype, int32_t sched,
                          const tree_plan_t* plan, void* stream) {
  const char* fn = "tree_gdn_scan_noalloc";
  size_t need = 0;
  if (const int rc = check_scan(fn, q, k, v, g, beta, o, states, n_tokens, h_qk, h_v, d_k, d_v, dtype, &sched,
                                plan, &need))
    return rc;
  const size_t plan_bytes = plan->p.device_bytes();
  const size_t slot_off = (plan_bytes + 255) / 256 * 256;
  if (slot_off + need > TREE_NOALLOC_SCRATCH_BYTES)
    return fail(TREE_ERR_WORKSPACE,
                "%s: needs %zu bytes of scratch (device plan %zu + parent states %zu), the static maximum is %zu; "
                "pass `states` (then no parent slots are needed) or use tree_gdn_scan with a workspace",
                fn, slot_off + need, plan_bytes, need, static_cast<size_t>(TREE_NOALLOC_SCRATCH_BYTES));
  unsigned char* ptr = nullptr;
  if (const int rc = scratch_on_current_device(fn, &ptr)) return rc;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  // The device plan goes into the scratch on the caller's stream, ahead of
  // the launches that read it.  Nothing in the scratch needs clearing: every
  // parent slot is written by its parent before a child reads it.
  const hipError_t e = hipMemcpyAsync(ptr, plan->p.mirror.data(), plan_bytes, hipMemcpyHostToDevice, st);
  if (e != hipSuccess) return hip_fail("tree_gdn_scan_noalloc: hipMemcpyAsync", e);
  return launch_scan_levels("tree_gdn_scan_noalloc: launch", q, k, v, g, beta, o, init_states, states, h_qk, h_v,
                            d_k, d_v, scale, dtype, sched, plan->p, reinterpret_cast<const int32_t*>(ptr),
                            reinterpret_cast<float*>(ptr + slot_off), st);
}

}  // extern "C"

namespace {

static_assert(tg::kBwdCkpt == tg::Plan::kBwdCkpt, "one checkpoint interval for the plan and the kernels");

// Scan backward workspace, in floats, in this order: checkpoint states (slot
// gck[s] + j for segment s's j-th),
// one start-state gradient per segment, every chunk's T, KK and QK, the
// level work-groups' re-run scratch (kBwdCkpt - 1 states each, for the
// largest level), and per-value-head dq, dk when h_v > 2 h_qk.
struct BwdLayout {
  size_t ck, dsseg, tws, scr, per_head, total;
};

BwdLayout bwd_layout(const tg::Plan& p, int32_t h_qk, int32_t h_v, int32_t d_k, int32_t d_v) {
  const size_t dd = static_cast<size_t>(d_k) * d_v;
  int32_t max_level = 0;
  for (int32_t l = 0; l < p.n_levels; ++l) max_level = std::max(max_level, p.level_start[l + 1] - p.level_start[l]);
  BwdLayout b{};
  b.ck = 0;
  b.dsseg = b.ck + static_cast<size_t>(p.total_ckpts) * h_v * dd;
  b.tws = b.dsseg + static_cast<size_t>(p.n_seg) * h_v * dd;
  b.scr = b.tws + static_cast<size_t>(p.total_chunks) * h_v * 3 * tg::Plan::kBwdChunk * tg::Plan::kBwdChunk;
  b.per_head = b.scr + static_cast<size_t>(max_level) * h_v * (tg::kBwdCkpt - 1) * dd;
  b.total = b.per_head + (h_v > 2 * h_qk ? 2 * static_cast<size_t>(p.n_tokens) * h_v * d_k : 0);
  return b;
}

}  // namespace

extern "C" {

size_t tree_gdn_scan_backward_workspace_bytes(const tree_plan_t* plan, int32_t h_qk, int32_t h_v, int32_t d_k,
                                              int32_t d_v) {
  if (!plan || h_qk <= 0 || h_v <= 0 || d_k <= 0 || d_v <= 0) return 0;
  return bwd_layout(plan->p, h_qk, h_v, d_k, d_v).total * sizeof(float);
}

int tree_gdn_scan_backward(const void* q, const void* k, const void* v, const float* g, const float* beta,
                           const void* dout, const float* dstates, const float* init_states,
                           const float* states, float* dq, float* dk, float* dv, float* dg, float* dbeta,
                           float* dinit_states, int64_t n_tokens, int32_t h_qk, int32_t h_v, int32_t d_k,
                           int32_t d_v, float scale, int32_t dtype, const tree_plan_t* plan, const void* dplan,
                           size_t dplan_bytes, void* ws, size_t ws_bytes, void* stream) {
  if (!plan || !q || !k || !v || !g || !beta || !dout || !states || !dq || !dk || !dv || !dg || !dbeta || !dplan)
    return fail(TREE_ERR_INVALID_ARG, "tree_gdn_scan_backward: null argument");
  const tg::Plan& p = plan->p;
  if (n_tokens != p.n_tokens)
    return fail(TREE_ERR_SIZE, "tree_gdn_scan_backward: n_tokens %lld != plan tokens %lld",
                static_cast<long long>(n_tokens), static_cast<long long>(p.n_tokens));
  if (h_qk <= 0 || h_v <= 0 || d_k <= 0 || d_v <= 0)
    return fail(TREE_ERR_INVALID_ARG, "tree_gdn_scan_backward: head counts and sizes must be > 0");
  if (h_v % h_qk != 0)
    return fail(TREE_ERR_UNSUPPORTED, "tree_gdn_scan_backward: h_v %d is not a multiple of h_qk %d", h_v, h_qk);
  if (!dtype_ok(dtype)) return fail(TREE_ERR_INVALID_ARG, "tree_gdn_scan_backward: bad dtype %d", dtype);
  if (!tg::scan_backward_supported(d_k, d_v, dtype))
    return fail(TREE_ERR_UNSUPPORTED, "tree_gdn_scan_backward: d_k=%d d_v=%d dtype=%d not compiled in", d_k, d_v,
                dtype);
  const size_t need = tree_gdn_scan_backward_workspace_bytes(plan, h_qk, h_v, d_k, d_v);
  if (!ws || ws_bytes < need)
    return fail(TREE_ERR_WORKSPACE, "tree_gdn_scan_backward: workspace has %zu bytes, needs %zu",
                ws ? ws_bytes : 0, need);
  if (const int rc = check_dplan(plan, dplan, dplan_bytes, "tree_gdn_scan_backward")) return rc;
  const int32_t* base = static_cast<const int32_t*>(dplan);
  const size_t dd = static_cast<size_t>(d_k) * d_v;
  tg::ScanBwdArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.dout = dout;
  a.dstates = dstates;
  a.init = init_states;
  a.states = states;
  a.dv = dv;
  a.dg = dg;
  a.dbeta = dbeta;
  a.dinit = dinit_states;
  const BwdLayout lay = bwd_layout(p, h_qk, h_v, d_k, d_v);
  float* const wsf = static_cast<float*>(ws);
  a.hws = wsf + lay.ck;
  a.dsseg = wsf + lay.dsseg;
  a.tws = wsf + lay.tws;
  a.scr = wsf + lay.scr;
  float* per_head = wsf + lay.per_head;
  // One value head per q/k head: dq, dk written directly.  Two: the prep
  // launch clears dq, dk and both heads add into them.  More: per-value-head
  // parts, summed in head order.
  const bool pairwise = h_v == 2 * h_qk;
  const bool grouped = h_v > 2 * h_qk;
  a.dq = grouped ? per_head : dq;
  a.dk = grouped ? per_head + static_cast<size_t>(n_tokens) * h_v * d_k : dk;
  a.dq_heads = grouped ? h_v : h_qk;
  // Pairwise: the first value head of every pair stores its part of dq, dk
  // and the second, in a later launch, adds to it (a + b either way round),
  // so nothing needs clearing.  Level l's first heads run in the launch
  // after level l + 1's first heads, together with level l + 1's second.
  a.dq_accum = 0;
  a.dq_accum2 = 0;
  a.head_step = 1;
  a.head_off = 0;
  a.head_off2 = 0;
  a.items2 = nullptr;
  a.n_items2 = 0;
  a.seg_off = base + p.m_seg_off;
  a.parent = base + p.m_parent;
  a.root_idx = base + p.m_root;
  a.kid_off = base + p.m_kid_off;
  a.kid = base + p.m_kid;
  a.gchunk = base + p.m_gchunk;
  a.chunk_seg = base + p.m_chunk_seg;
  a.gck = base + p.m_gck;
  a.n_chunks = static_cast<int32_t>(p.total_chunks);
  a.n_seg = p.n_seg;
  a.h_qk = h_qk;
  a.h_v = h_v;
  a.scale = scale;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  // Checkpoints and the chunk tables: at bf16 d = 128 from the forward scan
  // kernel (32-token chunks, all segments in one launch from the given final
  // states; prep then only clears dq, dk), else from the prep and states
  // kernels.
  const bool ck_fwd = d_k == 128 && d_v == 128 && dtype == TREE_DTYPE_BF16;
  {
    hipError_t e = tg::launch_scan_backward_prep(a, d_k, dtype, !ck_fwd, !ck_fwd, st);
    if (e == hipSuccess && ck_fwd) {
      tg::ScanArgs c{};
      c.q = q;
      c.k = k;
      c.v = v;
      c.g = g;
      c.beta = beta;
      c.init = init_states;
      c.root_idx = a.root_idx;
      c.states = const_cast<float*>(states);  // read only in this pass
      c.seg_off = a.seg_off;
      c.parent = a.parent;
      c.items = base + p.m_order;  // every segment, level by level
      c.n_items = p.n_seg;
      c.h_qk = h_qk;
      c.h_v = h_v;
      c.scale = scale;
      c.ckpt = a.hws;
      c.gck = a.gck;
      c.tws = a.tws;
      c.gchunk = a.gchunk;
      e = tg::launch_scan_d128_checkpoints(c, st);
    }
    if (e != hipSuccess) return hip_fail("tree_gdn_scan_backward: launch", e);
  }
  // Deepest level first: a parent sums its children's start-state gradients.
  for (int32_t l = p.n_levels - 1; l >= (pairwise ? -1 : 0); --l) {
    const int32_t ld = l + 1;  // the level below, whose second heads run now
    a.items = l >= 0 ? base + p.m_order + p.level_start[l] : nullptr;
    a.n_items = l >= 0 ? p.level_start[l + 1] - p.level_start[l] : 0;
    a.head_step = pairwise ? 2 : 1;
    a.head_off = 0;
    a.dq_accum = 0;
    a.items2 = nullptr;
    a.n_items2 = 0;
    if (pairwise && ld < p.n_levels) {
      a.items2 = base + p.m_order + p.level_start[ld];
      a.n_items2 = p.level_start[ld + 1] - p.level_start[ld];
      a.head_off2 = 1;
      a.dq_accum2 = 1;
    }
    const hipError_t e = tg::launch_scan_backward_level(a, d_k, dtype, st);
    if (e != hipSuccess) return hip_fail("tree_gdn_scan_backward: launch", e);
  }
  if (grouped) {
    const int group = h_v / h_qk;
    hipError_t e = tg::launch_head_group_sum(a.dq, dq, n_tokens, h_qk, group, d_k, st);
    if (e == hipSuccess) e = tg::launch_head_group_sum(a.dk, dk, n_tokens, h_qk, group, d_k, st);
    if (e != hipSuccess) return hip_fail("tree_gdn_scan_backward: launch", e);
  }
  return TREE_OK;
}

int tree_ssd_scan(const void* x, const float* dt, const float* A, const void* B, const void* C, const float* D,
                  void* y, const float* init_states, float* states, int64_t n_tokens, int32_t n_groups,
                  int32_t n_heads, int32_t d_state, int32_t head_dim, int32_t dtype, const tree_plan_t* plan,
                  const void* dplan, size_t dplan_bytes, void* ws, size_t ws_bytes, void* stream) {
  if (!plan || !x || !dt || !A || !B || !C || !y || !dplan)
    return fail(TREE_ERR_INVALID_ARG, "tree_ssd_scan: null argument");
  const tg::Plan& p = plan->p;
  if (n_tokens != p.n_tokens)
    return fail(TREE_ERR_SIZE, "tree_ssd_scan: n_tokens %lld != plan tokens %lld", static_cast<long long>(n_tokens),
                static_cast<long long>(p.n_tokens));
  if (n_groups <= 0 || n_heads <= 0 || d_state <= 0 || head_dim <= 0)
    return fail(TREE_ERR_INVALID_ARG, "tree_ssd_scan: head counts and sizes must be > 0");
  if (n_heads % n_groups != 0)
    return fail(TREE_ERR_UNSUPPORTED, "tree_ssd_scan: n_heads %d is not a multiple of n_groups %d", n_heads, n_groups);
  if (!dtype_ok(dtype)) return fail(TREE_ERR_INVALID_ARG, "tree_ssd_scan: bad dtype %d", dtype);
  if (!tg::ssd_supported(d_state, head_dim, dtype))
    return fail(TREE_ERR_UNSUPPORTED, "tree_ssd_scan: d_state=%d head_dim=%d dtype=%d not compiled in", d_state,
                head_dim, dtype);
  const size_t need = tree_scan_workspace_bytes(plan, n_heads, d_state, head_dim, states != nullptr);
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(TREE_ERR_WORKSPACE, "tree_ssd_scan: workspace has %zu bytes, needs %zu", ws ? ws_bytes : 0, need);
  if (const int rc = check_dplan(plan, dplan, dplan_bytes, "tree_ssd_scan")) return rc;
  const int32_t* base = static_cast<const int32_t*>(dplan);
  tg::SsdArgs a{};
  a.x = x;
  a.dt = dt;
  a.A = A;
  a.B = B;
  a.C = C;
  a.D = D;
  a.y = y;
  a.init = init_states;
  a.states = states;
  a.slots = static_cast<float*>(ws);
  a.seg_off = base + p.m_seg_off;
  a.parent = base + p.m_parent;
  a.slot = base + p.m_slot;
  a.root_idx = base + p.m_root;
  a.n_groups = n_groups;
  a.n_heads = n_heads;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  for (int32_t l = 0; l < p.n_levels; ++l) {
    a.items = base + p.m_order + p.level_start[l];
    a.n_items = p.level_start[l + 1] - p.level_start[l];
    const hipError_t e = tg::launch_ssd_scan(a, d_state, head_dim, dtype, st);
    if (e != hipSuccess) return hip_fail("tree_ssd_scan: launch", e);
  }
  return TREE_OK;
}

int tree_attention_plan(const tree_plan_t* plan, tree_attention_plan_t** out) {
  if (!plan || !out) return fail(TREE_ERR_INVALID_ARG, "tree_attention_plan: null argument");
  *out = nullptr;
  try {
    std::unique_ptr<tree_attention_plan_t> a(new tree_attention_plan_t);
    std::string err;
    const int rc = tg::build_attn_plan(plan->p, &a->p, &err);
    if (rc != TREE_OK) {
      g_err = err;
      return rc;
    }
    *out = a.release();
    return TREE_OK;
  } catch (const std::exception&) {
    return fail(TREE_ERR_INVALID_ARG, "tree_attention_plan: out of host memory");
  }
}

void tree_attention_plan_free(tree_attention_plan_t* aplan) { delete aplan; }

size_t tree_attention_plan_device_bytes(const tree_attention_plan_t* aplan) {
  return aplan ? aplan->p.device_bytes() : 0;
}

int tree_attention_plan_upload(const tree_attention_plan_t* aplan, void* dplan, size_t dplan_bytes, void* stream) {
  if (!aplan || !dplan) return fail(TREE_ERR_INVALID_ARG, "tree_attention_plan_upload: null argument");
  const size_t need = aplan->p.device_bytes();
  if (dplan_bytes < need)
    return fail(TREE_ERR_WORKSPACE, "tree_attention_plan_upload: dplan has %zu bytes, needs %zu", dplan_bytes, need);
  if (reinterpret_cast<uintptr_t>(dplan) % 32 != 0)
    return fail(TREE_ERR_INVALID_ARG, "tree_attention_plan_upload: dplan is not aligned to 32 bytes");
  const hipError_t e = hipMemcpyAsync(dplan, aplan->p.mirror.data(), need, hipMemcpyHostToDevice,
                                      static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail("tree_attention_plan_upload: hipMemcpyAsync", e);
  try {
    std::lock_guard<std::mutex> lock(aplan->mu);
    for (auto& u : aplan->uploads)
      if (u.first == dplan) {
        u.second = dplan_bytes;
        return TREE_OK;
      }
    aplan->uploads.emplace_back(dplan, dplan_bytes);
  } catch (const std::exception&) {
    return fail(TREE_ERR_INVALID_ARG, "tree_attention_plan_upload: out of host memory");
  }
  return TREE_OK;
}

size_t tree_attention_workspace_bytes(const tree_attention_plan_t* aplan, int32_t h_q, int32_t d, int32_t dtype) {
  if (!aplan || h_q <= 0 || !tg::attention_supported(d, dtype) || !heads_fit(aplan->p, h_q)) return 0;
  const Work w = attention_work(aplan->p.q, h_q, 1, d, dtype);
  return static_cast<size_t>(w.n_parts) * h_q * tg::attention_part_floats(d) * sizeof(float);
}

int tree_attention(const void* q, const void* k, const void* v, void* o, float* lse, const int64_t* strides,
                   int64_t n_tokens, int32_t h_q, int32_t h_kv, int32_t d, float scale, int32_t dtype,
                   const tree_attention_plan_t* aplan, const void* dplan, size_t dplan_bytes, void* ws,
                   size_t ws_bytes, void* stream) {
  const char* fn = "tree_attention";
  if (!aplan || !q || !k || !v || !o || !dplan) return fail(TREE_ERR_INVALID_ARG, "%s: null argument", fn);
  const tg::AttnPlan& p = aplan->p;
  if (const int rc = check_attention(p, n_tokens, h_q, h_kv, d, scale, dtype, fn)) return rc;
  tg::AttnArgs a{};
  const auto st_of = [&](int i) { return strides ? strides + 2 * i : nullptr; };
  if (const int rc = make_heads(q, st_of(0), h_q, d, dtype, "q", fn, &a.q)) return rc;
  if (const int rc = make_heads(k, st_of(1), h_kv, d, dtype, "k", fn, &a.k)) return rc;
  if (const int rc = make_heads(v, st_of(2), h_kv, d, dtype, "v", fn, &a.v)) return rc;
  if (const int rc = check_aligned(o, "o", fn)) return rc;
  if (o == q || o == k || o == v) return fail(TREE_ERR_INVALID_ARG, "%s: o must not alias q, k or v", fn);
  const size_t need = tree_attention_workspace_bytes(aplan, h_q, d, dtype);
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(TREE_ERR_WORKSPACE, "%s: workspace has %zu bytes, needs %zu", fn, ws ? ws_bytes : 0, need);
  if (need > 0)
    if (const int rc = check_aligned(ws, "the workspace", fn)) return rc;
  if (const int rc = check_dplan(aplan, dplan, dplan_bytes, fn)) return rc;
  const int32_t* base = static_cast<const int32_t*>(dplan);
  a.out = o;
  a.lse = lse;
  a.part = static_cast<float*>(ws);
  a.tok_d = base + p.m_d;
  a.tok_e = base + p.m_e;
  a.runs = reinterpret_cast<const tg::AttnRun*>(base + p.m_runs);
  set_work(attention_work(p.q, h_q, 1, d, dtype), base, &a);
  a.n_tok = p.n_tokens;
  a.h_q = h_q;
  a.h_kv = h_kv;
  a.scale = scale;
  const hipError_t e = tg::launch_attention(a, d, dtype, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail("tree_attention: launch", e);
  return TREE_OK;
}

size_t tree_attention_backward_workspace_bytes(const tree_attention_plan_t* aplan, int32_t h_q, int32_t h_kv,
                                               int32_t d, int32_t dtype) {
  if (!aplan || h_q <= 0 || h_kv <= 0 || h_q % h_kv != 0 || !tg::attention_supported(d, dtype)) return 0;
  const tg::AttnPlan& p = aplan->p;
  if (!heads_fit(p, h_q)) return 0;
  const Work wq = attention_work(p.q, h_q, 1, d, dtype), wk = attention_work(p.k, h_kv, h_q / h_kv, d, dtype);
  const size_t dq = static_cast<size_t>(wq.n_parts) * h_q * tg::attention_dq_part_floats(d);
  const size_t dkv = static_cast<size_t>(wk.n_parts) * wk.split * h_kv * tg::attention_dkv_part_floats(d);
  return attention_delta_bytes(p, h_q) + std::max(dq, dkv) * sizeof(float);
}

int tree_attention_backward(const void* q, const void* k, const void* v, const void* o, const float* lse,
                            const void* dout, void* dq, void* dk, void* dv, const int64_t* strides,
                            int64_t n_tokens, int32_t h_q, int32_t h_kv, int32_t d,
                            float scale, int32_t dtype, const tree_attention_plan_t* aplan, const void* dplan,
                            size_t dplan_bytes, void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "tree_attention_backward";
  if (!aplan || !q || !k || !v || !o || !lse || !dout || !dq || !dk || !dv || !dplan)
    return fail(TREE_ERR_INVALID_ARG, "%s: null argument", fn);
  const tg::AttnPlan& p = aplan->p;
  if (const int rc = check_attention(p, n_tokens, h_q, h_kv, d, scale, dtype, fn)) return rc;
  tg::AttnArgs a{};
  const auto st_of = [&](int i) { return strides ? strides + 2 * i : nullptr; };
  if (const int rc = make_heads(q, st_of(0), h_q, d, dtype, "q", fn, &a.q)) return rc;
  if (const int rc = make_heads(k, st_of(1), h_kv, d, dtype, "k", fn, &a.k)) return rc;
  if (const int rc = make_heads(v, st_of(2), h_kv, d, dtype, "v", fn, &a.v)) return rc;
  if (const int rc = make_heads(o, st_of(3), h_q, d, dtype, "o", fn, &a.o)) return rc;
  if (const int rc = make_heads(dout, st_of(4), h_q, d, dtype, "dout", fn, &a.dout)) return rc;
  if (const int rc = check_aligned(dq, "dq", fn)) return rc;
  if (const int rc = check_aligned(dk, "dk", fn)) return rc;
  if (const int rc = check_aligned(dv, "dv", fn)) return rc;
  const void* outs[3] = {dq, dk, dv};
  const void* ins[5] = {q, k, v, o, dout};
  for (const void* x : outs)
    for (const void* y : ins)
      if (x == y) return fail(TREE_ERR_INVALID_ARG, "%s: gradients must not alias the inputs", fn);
  if (dq == dk || dq == dv || dk == dv) return fail(TREE_ERR_INVALID_ARG, "%s: gradients must not alias", fn);
  const size_t need = tree_attention_backward_workspace_bytes(aplan, h_q, h_kv, d, dtype);
  if (!ws || ws_bytes < need)
    return fail(TREE_ERR_WORKSPACE, "%s: workspace has %zu bytes, needs %zu", fn, ws ? ws_bytes : 0, need);
  if (const int rc = check_aligned(ws, "the workspace", fn)) return rc;
  if (const int rc = check_dplan(aplan, dplan, dplan_bytes, fn)) return rc;
  const int32_t* base = static_cast<const int32_t*>(dplan);
  a.out = dq;
  a.dk = dk;
  a.dv = dv;
  a.lse = const_cast<float*>(lse);
  a.delta = static_cast<float*>(ws);
  a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + attention_delta_bytes(p, h_q));
  a.tok_d = base + p.m_d;
  a.tok_e = base + p.m_e;
  a.runs = reinterpret_cast<const tg::AttnRun*>(base + p.m_runs);
  a.n_tok = p.n_tokens;
  a.h_q = h_q;
  a.h_kv = h_kv;
  a.scale = scale;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  set_work(attention_work(p.q, h_q, 1, d, dtype), base, &a);
  hipError_t e = tg::launch_attention_dq(a, d, dtype, st);  // also delta
  if (e == hipSuccess) {
    set_work(attention_work(p.k, h_kv, h_q / h_kv, d, dtype), base, &a);
    e = tg::launch_attention_dkv(a, d, dtype, st);  // its parts take dq's place in the workspace
  }
  if (e != hipSuccess) return hip_fail("tree_attention_backward: launch", e);
  return TREE_OK;
}

size_t tree_logprobs_workspace_bytes(int32_t n_rows, int32_t vocab, int32_t top_k) {
  if (n_rows <= 0 || vocab <= 0 || vocab > (1 << 30) || top_k < 0 || top_k > TREE_MAX_TOP_K) return 0;
  const Spread s = logprob_spread(n_rows, vocab);
  return s.split == 1 ? 0 : static_cast<size_t>(n_rows) * s.split * (16 + 8 * top_k);
}

int tree_logprobs(const void* logits, const void* tokens, float* logp, float* entropy, float* lse, float* top_logp,
                  int32_t* top_id, int64_t ld, int64_t n_tokens, int32_t first_row, int32_t n_rows, int32_t vocab,
                  int32_t token_bytes, float temperature, int32_t top_k, int32_t dtype, const tree_plan_t* plan,
                  const void* dplan, size_t dplan_bytes, void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "tree_logprobs";
  if (!plan || !logits || !tokens || !logp || !entropy || !lse || !dplan)
    return fail(TREE_ERR_INVALID_ARG, "%s: null argument", fn);
  const tg::Plan& p = plan->p;
  if (const int rc = check_logprobs(p, ld, n_tokens, first_row, n_rows, vocab, token_bytes, temperature, dtype, fn))
    return rc;
  if (top_k < 0 || top_k > TREE_MAX_TOP_K || top_k > vocab)
    return fail(TREE_ERR_INVALID_ARG, "%s: top_k %d must be in 0..min(%d, vocab)", fn, top_k, TREE_MAX_TOP_K);
  if (top_k > 0 && (!top_logp || !top_id)) return fail(TREE_ERR_INVALID_ARG, "%s: top_logp or top_id is null", fn);
  const size_t need = tree_logprobs_workspace_bytes(n_rows, vocab, top_k);
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(TREE_ERR_WORKSPACE, "%s: workspace has %zu bytes, needs %zu", fn, ws ? ws_bytes : 0, need);
  if (need > 0 && reinterpret_cast<uintptr_t>(ws) % 16 != 0)
    return fail(TREE_ERR_INVALID_ARG, "%s: the workspace is not aligned to 16 bytes", fn);
  if (const int rc = check_dplan(plan, dplan, dplan_bytes, fn)) return rc;
  const int32_t* base = static_cast<const int32_t*>(dplan);
  const Spread s = logprob_spread(n_rows, vocab);
  tg::LogprobArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.tokens = tokens;
  a.token64 = token_bytes == 8;
  a.first_row = first_row;
  a.n_rows = n_rows;
  a.vocab = vocab;
  a.inv_t = 1.f / temperature;
  a.top_k = top_k;
  a.split = s.split;
  a.slice = s.slice;
  a.logp = logp;
  a.entropy = entropy;
  a.lse = lse;
  a.top_logp = top_logp;
  a.top_id = top_id;
  a.part = static_cast<float*>(ws);
  a.seg_off = base + p.m_seg_off;
  a.parent = base + p.m_parent;
  a.kid_off = base + p.m_kid_off;
  a.kid = base + p.m_kid;
  a.n_seg = p.n_seg;
  const hipError_t e = tg::launch_logprobs(a, dtype, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail("tree_logprobs: launch", e);
  return TREE_OK;
}

int tree_logprobs_backward(const void* logits, const void* tokens, const float* lse, const float* entropy,
                           const float* dlogp, const float* dentropy, void* dlogits, int64_t ld, int64_t ldd,
                           int64_t n_tokens, int32_t first_row, int32_t n_rows, int32_t vocab, int32_t token_bytes,
                           float temperature, int32_t dtype, const tree_plan_t* plan, const void* dplan,
                           size_t dplan_bytes, void* stream) {
  const char* fn = "tree_logprobs_backward";
  if (!plan || !logits || !tokens || !lse || !dlogp || !dlogits || !dplan || (dentropy && !entropy))
    return fail(TREE_ERR_INVALID_ARG, "%s: null argument", fn);
  const tg::Plan& p = plan->p;
  if (const int rc = check_logprobs(p, ld, n_tokens, first_row, n_rows, vocab, token_bytes, temperature, dtype, fn))
    return rc;
  if (const int rc = check_logprobs(p, ldd, n_tokens, first_row, n_rows, vocab, token_bytes, temperature, dtype, fn))
    return rc;
  if (dlogits == logits && ldd != ld)
    return fail(TREE_ERR_INVALID_ARG, "%s: dlogits over logits needs ldd = ld", fn);
  if (const int rc = check_dplan(plan, dplan, dplan_bytes, fn)) return rc;
  const int32_t* base = static_cast<const int32_t*>(dplan);
  const Spread s = logprob_backward_spread(n_rows, vocab, dtype);
  tg::LogprobArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.tokens = tokens;
  a.token64 = token_bytes == 8;
  a.first_row = first_row;
  a.n_rows = n_rows;
  a.vocab = vocab;
  a.inv_t = 1.f / temperature;
  a.split = s.split;
  a.slice = s.slice;
  a.dlogp = dlogp;
  a.dentropy = dentropy;
  a.lse_in = lse;
  a.entropy_in = entropy;
  a.dlogits = dlogits;
  a.ldd = ldd;
  a.seg_off = base + p.m_seg_off;
  a.parent = base + p.m_parent;
  a.kid_off = base + p.m_kid_off;
  a.kid = base + p.m_kid;
  a.n_seg = p.n_seg;
  const hipError_t e = tg::launch_logprobs_backward(a, dtype, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail("tree_logprobs_backward: launch", e);
  return TREE_OK;
}

size_t tree_linear_logprobs_workspace_bytes(int32_t n_rows, int32_t vocab, int32_t width, int32_t dtype) {
  return linear_sizes_ok(n_rows, vocab, width, dtype) ? linear_work(n_rows, vocab, width, dtype).bytes : 0;
}

int tree_linear_logprobs(const void* hidden, const void* weight, const void* tokens, float* logp, float* entropy,
                         float* lse, int64_t ld, int64_t n_tokens, int32_t first_row, int32_t n_rows, int32_t vocab,
                         int32_t width, int32_t token_bytes, float temperature, int32_t dtype, const tree_plan_t* plan,
                         const void* dplan, size_t dplan_bytes, void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "tree_linear_logprobs";
  if (!plan || !hidden || !weight || !tokens || !logp || !entropy || !lse || !dplan)
    return fail(TREE_ERR_INVALID_ARG, "%s: null argument", fn);
  const tg::Plan& p = plan->p;
  if (const int rc = check_linear(p, hidden, ld, weight, n_tokens, first_row, n_rows, vocab, width, token_bytes,
                                  temperature, dtype, fn))
    return rc;
  const tg::LinearWork w = linear_work(n_rows, vocab, width, dtype);
  if (!ws || ws_bytes < w.bytes)
    return fail(TREE_ERR_WORKSPACE, "%s: workspace has %zu bytes, needs %zu", fn, ws ? ws_bytes : 0, w.bytes);
  if (const int rc = check_aligned(ws, "the workspace", fn)) return rc;
  if (const int rc = check_dplan(plan, dplan, dplan_bytes, fn)) return rc;
  tg::LinearArgs a{};
  set_linear(p, hidden, ld, weight, tokens, first_row, n_rows, vocab, width, token_bytes, temperature, dplan, ws, &a);
  a.logp = logp;
  a.entropy = entropy;
  a.lse = lse;
  const hipError_t e = tg::launch_linear(a, w, dtype, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail("tree_linear_logprobs: launch", e);
  return TREE_OK;
}

size_t tree_linear_logprobs_backward_workspace_bytes(int32_t n_rows, int32_t vocab, int32_t width, int32_t dtype) {
  return linear_sizes_ok(n_rows, vocab, width, dtype) ? linear_backward_work(n_rows, vocab, width, dtype).bytes : 0;
}

int tree_linear_logprobs_backward(const void* hidden, const void* weight, const void* tokens, const float* lse,
                                  const float* entropy, const float* dlogp, const float* dentropy, void* dhidden,
                                  void* dweight, int64_t ld, int64_t n_tokens, int32_t first_row, int32_t n_rows,
                                  int32_t vocab, int32_t width, int32_t token_bytes, float temperature, int32_t dtype,
                                  const tree_plan_t* plan, const void* dplan, size_t dplan_bytes, void* ws,
                                  size_t ws_bytes, void* stream) {
  const char* fn = "tree_linear_logprobs_backward";
  if (!plan || !hidden || !weight || !tokens || !lse || !dlogp || !dhidden || !dweight || !dplan ||
      (dentropy && !entropy))
    return fail(TREE_ERR_INVALID_ARG, "%s: null argument", fn);
  const tg::Plan& p = plan->p;
  if (const int rc = check_linear(p, hidden, ld, weight, n_tokens, first_row, n_rows, vocab, width, token_bytes,
                                  temperature, dtype, fn))
    return rc;
  if (const int rc = check_aligned(dhidden, "dhidden", fn)) return rc;
  if (const int rc = check_aligned(dweight, "dweight", fn)) return rc;
  for (const void* x : {hidden, weight})
    if (x == dhidden || x == dweight) return fail(TREE_ERR_INVALID_ARG, "%s: gradients must not alias the inputs", fn);
  if (dhidden == dweight) return fail(TREE_ERR_INVALID_ARG, "%s: gradients must not alias", fn);
  const tg::LinearWork w = linear_backward_work(n_rows, vocab, width, dtype);
  if (!ws || ws_bytes < w.bytes)
    return fail(TREE_ERR_WORKSPACE, "%s: workspace has %zu bytes, needs %zu", fn, ws ? ws_bytes : 0, w.bytes);
  if (const int rc = check_aligned(ws, "the workspace", fn)) return rc;
  if (const int rc = check_dplan(plan, dplan, dplan_bytes, fn)) return rc;
  tg::LinearArgs a{};
  set_linear(p, hidden, ld, weight, tokens, first_row, n_rows, vocab, width, token_bytes, temperature, dplan, ws, &a);
  a.dlogp = dlogp;
  a.dentropy = dentropy;
  a.lse_in = lse;
  a.entropy_in = entropy;
  a.dhidden = dhidden;
  a.dweight = dweight;
  const hipError_t e = tg::launch_linear_backward(a, w, dtype, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail("tree_linear_logprobs_backward: launch", e);
  return TREE_OK;
}

int tree_embedding(const void* tokens, const void* table, void* out, int64_t n_tokens, int32_t vocab, int32_t width,
                   int32_t token_bytes, float scale, int32_t dtype, void* stream) {
  const char* fn = "tree_embedding";
  if (const int rc = check_embed(n_tokens, vocab, width, kEmbedVocab, token_bytes, scale, dtype, fn)) return rc;
  if (!table || (n_tokens > 0 && (!tokens || !out))) return fail(TREE_ERR_INVALID_ARG, "%s: null argument", fn);
  if (out == table) return fail(TREE_ERR_INVALID_ARG, "%s: out must not alias the table", fn);
  if (const int rc = check_element_aligned(table, dtype, "table", fn)) return rc;
  if (const int rc = check_element_aligned(out, dtype, "out", fn)) return rc;
  if (n_tokens == 0) return TREE_OK;
  tg::EmbedArgs a{};
  a.tokens = tokens;
  a.table = table;
  a.out = out;
  a.n_tokens = n_tokens;
  a.vocab = vocab;
  a.width = width;
  a.scale = scale;
  a.lanes_log2 = tg::embed_lanes_log2(width, dtype, 0);
  const hipError_t e = tg::launch_embed(a, dtype, token_bytes == 8, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail("tree_embedding: launch", e);
  return TREE_OK;
}

size_t tree_embedding_backward_workspace_bytes(int64_t n_tokens, int32_t vocab, int32_t width) {
  return embed_sizes_ok(n_tokens, vocab, width, kSortVocab) ? embed_work(n_tokens, vocab, width).bytes : 0;
}

int tree_embedding_backward(const void* tokens, const void* dout, void* dtable, int64_t n_tokens, int32_t vocab,
                            int32_t width, int32_t token_bytes, float scale, int32_t dtype, void* ws, size_t ws_bytes,
                            void* stream) {
  const char* fn = "tree_embedding_backward";
  if (const int rc = check_embed(n_tokens, vocab, width, kSortVocab, token_bytes, scale, dtype, fn)) return rc;
  if (!dtable || (n_tokens > 0 && (!tokens || !dout))) return fail(TREE_ERR_INVALID_ARG, "%s: null argument", fn);
  if (dtable == dout) return fail(TREE_ERR_INVALID_ARG, "%s: dtable must not alias dout", fn);
  if (const int rc = check_element_aligned(dout, dtype, "dout", fn)) return rc;
  if (const int rc = check_element_aligned(dtable, dtype, "dtable", fn)) return rc;
  const EmbedWork w = embed_work(n_tokens, vocab, width);
  if (!ws || ws_bytes < w.bytes)
    return fail(TREE_ERR_WORKSPACE, "%s: workspace has %zu bytes, needs %zu", fn, ws ? ws_bytes : 0, w.bytes);
  if (const int rc = check_aligned(ws, "the workspace", fn)) return rc;
  char* base = static_cast<char*>(ws);
  tg::EmbedArgs a{};
  a.tokens = tokens;
  a.dout = dout;
  a.out = dtable;
  a.n_tokens = n_tokens;
  a.vocab = vocab;
  a.width = width;
  a.scale = scale;
  a.lanes_log2 = tg::embed_lanes_log2(width, dtype, 6);  // whole waves
  a.span = w.span;
  a.n_parts = w.n_parts;
  a.start = reinterpret_cast<int32_t*>(base);
  a.order = reinterpret_cast<int2*>(base + w.order);
  a.part = reinterpret_cast<float*>(base + w.part);
  const hipError_t e = tg::launch_embed_backward(a, dtype, token_bytes == 8, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail("tree_embedding_backward: launch", e);
  return TREE_OK;
}

const char* tree_last_error(void) { return g_err.c_str(); }

}  // extern "C"
