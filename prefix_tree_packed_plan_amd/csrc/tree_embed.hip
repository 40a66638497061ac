// Token embedding and its gradient (gfx950):
//     out_n = scale * table[tok n],   dtable[v] = scale * sum over n with tok n = v of dout_n.
// A token outside the table has no row: its output is 0 and its gradient goes nowhere.
//
// Both are bound by memory: rows are read and written once, 16 bytes a lane
// (rows need not be aligned to 16 bytes: the hardware reads and writes such
// pieces at any address).
//
// The gradient takes the tokens sorted by their row of the table.  sort_kernel
// makes that order: every work-group owns `span` rows and looks through all tokens,
// which come from L2, counts its own and places them.  It needs no pass over global
// memory and no atomic whose order shows: each wave keeps counters of its own
// for its share of the tokens, and within 64 tokens a lane's place among its
// equals comes from comparing the ids bit by bit.  A row's list is therefore
// in ascending order of the tokens, and the sums are the same in every run.  Rows
// without a token, most of a large table, are cleared on the way.
//
// sum_kernel then writes the rows that have tokens, one for every position of the order at
// which a row begins.  Rows of more than kPart tokens would keep one work-group busy
// long after the others (a token that is a fifth of all of them); their lists are
// cut into parts at multiples of kPart, and join_kernel adds the parts in order.
//
// Measured (us; inputs that change from call to call; a copy reaches 4.9 TB/s here, a fill
// 6.9): 10240 tokens of 131072 x 4096 bf16, forward 25 (5.1 TB/s of distinct rows read and
// all written; 22 where those rows stay in the last-level cache); gradient 245: the sort with
// its clearing 173 (5.8 TB/s of zeros), the sums 49, the join, without work, 5.  65536
// tokens, a fifth of them equal, of 32000 x 2048: 173: the sort 80 (one work-group's
// long row: vector issue), the sums 79 (3.4 TB/s of dout), the join 12.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "../../include/tree_gdn.h"
#include "chunk_mfma.hpp"
#include "launch.hpp"

namespace tg {

namespace {

using chunk::pk2;

constexpr int kThreads = 256;
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kPart = kEmbedPart;
static_assert(kPart == 64, "a part's tokens are held by the lanes of a wave");
constexpr int kKept = 256;  // tokens in range a sorting wave keeps at hand
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// 16 bytes at any address.
typedef u32x4 any_u32x4 __attribute__((aligned(2)));

template <typename T>
struct Vec;
template <>
struct Vec<uint16_t> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const u32x4 w, float* x) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = chunk::lo_f(w[j]);
      x[2 * j + 1] = chunk::hi_f(w[j]);
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float* x) {
    return u32x4{pk2(x[0], x[1]), pk2(x[2], x[3]), pk2(x[4], x[5]), pk2(x[6], x[7])};
  }
  static __device__ __forceinline__ float one(const uint16_t* p) { return __uint_as_float(uint32_t(*p) << 16); }
  static __device__ __forceinline__ void put(uint16_t* p, float x) { *p = static_cast<uint16_t>(pk2(x, x)); }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const u32x4 w, float* x) {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = __uint_as_float(w[j]);
  }
  static __device__ __forceinline__ u32x4 pack(const float* x) {
    return u32x4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ void put(float* p, float x) { *p = x; }
};

// Row of the table of token n, or -1.
template <typename I>
__device__ __forceinline__ int token(const EmbedArgs& a, int64_t n) {
  const I x = static_cast<const I*>(a.tokens)[n];
  return x >= 0 && x < a.vocab ? static_cast<int>(x) : -1;
}

// The items (rows) of this thread, one after another: an item has 2^lanes_log2
// threads of a work-group, this one is its j0-th.
struct Item {
  int64_t i, step;
  int j0, lanes;
  __device__ __forceinline__ explicit Item(const EmbedArgs& a)
      : i(int64_t(blockIdx.x) * (kThreads >> a.lanes_log2) + (threadIdx.x >> a.lanes_log2)),
        step(int64_t(gridDim.x) * (kThreads >> a.lanes_log2)), j0(threadIdx.x & ((1 << a.lanes_log2) - 1)),
        lanes(1 << a.lanes_log2) {}
  __device__ __forceinline__ void next() { i += step; }
};

// ---- forward ----------------------------------------------------------------------
template <typename T, typename I>
__global__ __launch_bounds__(kThreads) void embed_kernel(EmbedArgs a) {
  constexpr int N = Vec<T>::N;
  const int vecs = a.width / N;
  for (Item it(a); it.i < a.n_tokens; it.next()) {
    const int id = token<I>(a, it.i);
    const T* src = static_cast<const T*>(a.table) + int64_t(id) * a.width;
    T* dst = static_cast<T*>(a.out) + it.i * a.width;
#pragma unroll 4
    for (int j = it.j0; j < vecs; j += it.lanes) {
      float x[N];
      u32x4 w = {0, 0, 0, 0};
      if (id >= 0) w = *reinterpret_cast<const any_u32x4*>(src + j * N);
      Vec<T>::unpack(w, x);
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] *= a.scale;
      *reinterpret_cast<any_u32x4*>(dst + j * N) = Vec<T>::pack(x);
    }
    for (int c = vecs * N + it.j0; c < a.width; c += it.lanes)
      Vec<T>::put(dst + c, id >= 0 ? Vec<T>::one(src + c) * a.scale : 0.f);
  }
}

// ---- the tokens in order of their rows ----------------------------------------------
// Token n as an unsigned row of the table; one without a row is above all of them.
template <typename I>
__device__ __forceinline__ uint32_t row_of(const EmbedArgs& a, int n);
template <>
__device__ __forceinline__ uint32_t row_of<int32_t>(const EmbedArgs& a, int n) {
  const uint32_t x = static_cast<const uint32_t*>(a.tokens)[n];
  return x < static_cast<uint32_t>(a.vocab) ? x : ~0u;
}
template <>
__device__ __forceinline__ uint32_t row_of<int64_t>(const EmbedArgs& a, int n) {
  const uint2 x = static_cast<const uint2*>(a.tokens)[n];
  return x.y == 0 && x.x < static_cast<uint32_t>(a.vocab) ? x.x : ~0u;
}

// This work-group's rows: lo .. lo + span - 1.  cnt[w][r]: tokens of row lo + r in
// wave w's share; then where its next one goes.  Rows without a token are cleared here,
// where their number is known early and clearing overlaps others' sorting (in
// sum_kernel, one item a row of the table, 131072 x 4096 took 354 us instead of 291).
// 16 waves, so that a share is short: the longest row's work-group sets the time.
template <typename T, typename I>
__global__ __launch_bounds__(kSortThreads) void sort_kernel(EmbedArgs a) {
  constexpr int U = 8;
  __shared__ int cnt[kSortWaves * kEmbedSpan];
  __shared__ int2 kept[kSortWaves * kKept];
  __shared__ int wave_total[kSortWaves];
  __shared__ int wave_less[kSortWaves];
  __shared__ uint64_t empty[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lo = blockIdx.x * a.span, span = min(a.span, a.vocab - lo);
  const int n = static_cast<int>(a.n_tokens);
  const int share = ((n + kSortThreads - 1) / kSortThreads) * 64;
  const int t0 = min(n, wave * share), t1 = min(n, t0 + share);
  const uint64_t lower = (uint64_t(1) << lane) - 1;
  int* mine = cnt + wave * kEmbedSpan;
  for (int i = tid; i < kSortWaves * kEmbedSpan; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  // Calls f(rows, t) for U times 64 tokens from t on of this wave's share, in order; the
  // next ones are on their way meanwhile.
  const auto each = [&](auto f) {
    uint32_t id[U];
    const auto load = [&](int t) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = t + 64 * u + lane;
        id[u] = at < t1 ? row_of<I>(a, at) : ~0u;
      }
    };
    load(t0);
    for (int t = t0; t < t1; t += 64 * U) {
      uint32_t now[U];
#pragma unroll
      for (int u = 0; u < U; ++u) now[u] = id[u];
      load(t + 64 * U);
      f(now, t);
    }
  };
  int less = 0;  // tokens of rows below lo
  int held = 0;  // tokens in range so far: the first kKept are kept in LDS
  each([&](const uint32_t (&id)[U], int t) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      less += id[u] < static_cast<uint32_t>(lo);
      const uint32_t r = id[u] - lo;
      const bool in = r < static_cast<uint32_t>(span);
      const uint64_t who = __ballot(in);
      if (who == 0) continue;
      const int at = held + __popcll(who & lower);
      if (in) atomicAdd(&mine[r], 1);
      if (in && at < kKept) kept[wave * kKept + at] = make_int2(r, t + 64 * u + lane);
      held += __popcll(who);
    }
  });
#pragma unroll
  for (int o = 32; o; o >>= 1) less += __shfl_xor(less, o, 64);
  if (lane == 0) wave_less[wave] = less;
  __syncthreads();
  int base = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) base += wave_less[w];
  // Thread r: row lo + r.
  int total = 0;
  if (tid < span)
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) total += cnt[w * kEmbedSpan + tid];
  const uint64_t none = __ballot(total == 0);
  if (lane == 0) empty[wave] = none;
  int sum = total;  // of this lane and those below
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(sum, o, 64);
    if (lane >= o) sum += y;
  }
  if (lane == 63) wave_total[wave] = sum;
  __syncthreads();
  int at = base + sum - total;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) at += w < wave ? wave_total[w] : 0;
  if (tid < span) {
    a.start[lo + tid] = at;
    if (lo + tid + 1 == a.vocab) a.start[a.vocab] = at + total;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = cnt[w * kEmbedSpan + tid];
      cnt[w * kEmbedSpan + tid] = at;
      at += c;
    }
  }
  __syncthreads();
  // K times 64 tokens: all of one kind of step, then all of the next, so that LDS is
  // waited for once; as many bits are compared as the rows need (65536 tokens of 32000
  // rows, a fifth equal: 173 us, 184 with 9 bits).
  const auto place = [&](auto count, const uint32_t* r, const int* t) {
    constexpr int K = decltype(count)::value;
    uint64_t same[K];
    int first[K];
#pragma unroll
    for (int u = 0; u < K; ++u) {
      same[u] = __ballot(r[u] < static_cast<uint32_t>(span));
      for (uint32_t bit = 1; bit < static_cast<uint32_t>(span); bit += bit) {
        const bool set = r[u] & bit;
        const uint64_t ones = __ballot(set);
        same[u] &= set ? ones : ~ones;
      }
      // The first of its equals moves their counter on; waves share none.
      first[u] = 0;
      if (r[u] < static_cast<uint32_t>(span) && (same[u] & lower) == 0)
        first[u] = atomicAdd(&mine[r[u]], static_cast<int>(__popcll(same[u])));
    }
#pragma unroll
    for (int u = 0; u < K; ++u)
      first[u] = __shfl(first[u], r[u] < static_cast<uint32_t>(span) ? __builtin_ctzll(same[u]) : lane, 64);
#pragma unroll
    for (int u = 0; u < K; ++u)
      if (r[u] < static_cast<uint32_t>(span))
        a.order[first[u] + __popcll(same[u] & lower)] = make_int2(t[u], lo + static_cast<int>(r[u]));
  };
  if (held <= kKept) {
    for (int i = 0; i < held; i += 64) {
      const int2 x = i + lane < held ? kept[wave * kKept + i + lane] : make_int2(-1, 0);
      const uint32_t r = x.x;
      place(std::integral_constant<int, 1>{}, &r, &x.y);
    }
  } else {
    constexpr int K = 4;
    each([&](const uint32_t (&id)[U], int t) {
#pragma unroll
      for (int h = 0; h < U; h += K) {
        uint32_t r[K];
        int at[K];
#pragma unroll
        for (int u = 0; u < K; ++u) {
          r[u] = id[h + u] - lo;  // without a row: 2^32 - 1 - lo, out of range
          at[u] = t + 64 * (h + u) + lane;
        }
        place(std::integral_constant<int, K>{}, r, at);
      }
    });
  }
  // A wave a row: zeros where there is no token.
  constexpr int N = Vec<T>::N;
  const int vecs = a.width / N;
  for (int r = wave; r < span; r += kSortWaves) {
    if (!((empty[r >> 6] >> (r & 63)) & 1)) continue;
    T* out = static_cast<T*>(a.out) + int64_t(lo + r) * a.width;
#pragma unroll 4
    for (int j = lane; j < vecs; j += 64) *reinterpret_cast<any_u32x4*>(out + j * N) = u32x4{0, 0, 0, 0};
    for (int c = vecs * N + lane; c < a.width; c += 64) Vec<T>::put(out + c, 0.f);
  }
}

// ---- sums ----------------------------------------------------------------------------
// Calls f(whether it is a single column, column) for this thread's pieces of a row.
template <typename T, typename F>
__device__ __forceinline__ void columns(const EmbedArgs& a, int j0, int lanes, F f) {
  constexpr int N = Vec<T>::N;
  const int vecs = a.width / N;
  for (int j = j0; j < vecs; j += lanes) f(std::false_type{}, j * N);
  for (int c = vecs * N + j0; c < a.width; c += lanes) f(std::true_type{}, c);
}

// x += the gradients, at a column (TAIL) or piece from `col` on, of the tokens that lanes
// p .. p + U - 1 hold (REST: of those below i1), in order and with all loads in flight
// (one after another: 291 us instead of 249 for 10240 tokens of 131072 x 4096).
template <typename T, bool TAIL, int U, bool REST>
__device__ __forceinline__ void add_some(const EmbedArgs& a, int held, int p, int i1, int col, float* x) {
  constexpr int N = TAIL ? 1 : Vec<T>::N;
  const T* row[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    row[u] = static_cast<const T*>(a.dout) + col +
             int64_t(__builtin_amdgcn_readlane(held, REST ? min(p + u, i1 - 1) : p + u)) * a.width;
  if constexpr (TAIL) {
    float y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) y[u] = Vec<T>::one(row[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) x[0] += !REST || p + u < i1 ? y[u] : 0.f;
  } else {
    u32x4 w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = *reinterpret_cast<const any_u32x4*>(row[u]);
    __builtin_amdgcn_sched_barrier(0);  // all loads, then one row's values at a time
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float y[N];
      Vec<T>::unpack(w[u], y);
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] += !REST || p + u < i1 ? y[i] : 0.f;
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}
// The same of lanes i0 .. i1 - 1, from 0 on.
template <typename T, bool TAIL>
__device__ __forceinline__ void add_rows(const EmbedArgs& a, int held, int i0, int i1, int col, float* x) {
  constexpr int U = 8;
#pragma unroll
  for (int i = 0; i < (TAIL ? 1 : Vec<T>::N); ++i) x[i] = 0.f;
  int p = i0;
  for (; p + U <= i1; p += U) add_some<T, TAIL, U, false>(a, held, p, i1, col, x);
  if (i1 - p > 4) add_some<T, TAIL, U, true>(a, held, p, i1, col, x);
  else if (i1 > p) add_some<T, TAIL, 4, true>(a, held, p, i1, col, x);
}

template <typename T, bool TAIL>
__device__ __forceinline__ void put_row(const EmbedArgs& a, int64_t v, int col, float* x) {
  T* o = static_cast<T*>(a.out) + v * a.width + col;
  constexpr int N = TAIL ? 1 : Vec<T>::N;
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] *= a.scale;
  if constexpr (TAIL) Vec<T>::put(o, x[0]);
  else *reinterpret_cast<any_u32x4*>(o) = Vec<T>::pack(x);
}

// Position p of the order: the row that begins there, if one does and it has at most
// kPart tokens.  Every wave of the item reads the whole list, an entry a lane.
template <typename T>
__device__ __forceinline__ void sum_row(const EmbedArgs& a, int p, int n, const Item& it, int lane) {
  const int2 e = p + lane < n ? a.order[p + lane] : make_int2(0, -1);
  const int before = p > 0 ? a.order[p - 1].y : -1, after = p + kPart < n ? a.order[p + kPart].y : -1;
  const int v = __builtin_amdgcn_readfirstlane(e.y);
  if (v == before || v == after) return;
  const int count = __popcll(__ballot(e.y == v));
  columns<T>(a, it.j0, it.lanes, [&](auto tail, int col) {
    constexpr bool TAIL = decltype(tail)::value;
    float x[Vec<T>::N];
    add_rows<T, TAIL>(a, e.x, 0, count, col, x);
    put_row<T, TAIL>(a, v, col, x);
  });
}

// Part q, positions kPart q .. kPart (q + 1) - 1: at most its first and its last row have
// more than kPart tokens, and their sums are part[q][0] and part[q][1].
template <typename T>
__device__ __forceinline__ void sum_part(const EmbedArgs& a, int q, int n, const Item& it, int lane) {
  const int p0 = q * kPart, p1 = min(n, p0 + kPart);
  if (p0 >= p1) return;
  const int2 e = a.order[min(p0 + lane, p1 - 1)];
  const int first = __builtin_amdgcn_readfirstlane(e.y), last = __builtin_amdgcn_readlane(e.y, p1 - 1 - p0);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int v = s ? last : first;
    if (s && last == first) break;
    const int r0 = a.start[v], r1 = a.start[v + 1];
    if (r1 - r0 <= kPart) continue;
    float* out = a.part + (int64_t(q) * 2 + s) * a.width;
    columns<T>(a, it.j0, it.lanes, [&](auto tail, int col) {
      constexpr bool TAIL = decltype(tail)::value;
      float x[Vec<T>::N];
      add_rows<T, TAIL>(a, e.x, max(p0, r0) - p0, min(p1, r1) - p0, col, x);
#pragma unroll
      for (int i = 0; i < (TAIL ? 1 : Vec<T>::N); ++i) out[col + i] = x[i];
    });
  }
}

// Items: the parts of long lists, which take longest, then the positions.
template <typename T>
__global__ __launch_bounds__(kThreads) void sum_kernel(EmbedArgs a) {
  const int lane = threadIdx.x & 63, n = a.start[a.vocab];
  const Item all(a);
  for (Item it = all; it.i < a.n_parts + a.n_tokens; it.next()) {
    const int i = __builtin_amdgcn_readfirstlane(static_cast<int>(it.i));
    if (i < a.n_parts) sum_part<T>(a, i, n, it, lane);
    else if (i - a.n_parts < n) sum_row<T>(a, i - a.n_parts, n, it, lane);
  }
}

// Item q: the row of more than kPart tokens whose list begins in part q, if there is
// one (it reaches past the part's end, so there is at most one).  A work-group takes
// kJoinColumns columns of it; each wave adds a quarter of the parts, and the
// quarters are added in order (13 us for 205 parts of 2048 columns).
constexpr int kJoinColumns = 256;
template <typename T>
__global__ __launch_bounds__(kThreads) void join_kernel(EmbedArgs a) {
  constexpr int U = 16, W = kThreads / 64;
  __shared__ float4 sums[W][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int q = blockIdx.x; q < a.n_parts; q += gridDim.x) {
    const int end = (q + 1) * kPart;
    // The row goes on behind the part.
    if (end >= a.n_tokens) return;
    const int n = a.start[a.vocab], v = a.order[end - 1].y, next = a.order[end].y;
    if (end >= n) return;
    if (next != v) continue;
    const int r0 = a.start[v], r1 = a.start[v + 1];
    if (r1 - r0 <= kPart || r0 < q * kPart) continue;
    const int q1 = (r1 - 1) / kPart + 1, each = (q1 - q + W - 1) / W;
    const int s0 = r0 == q * kPart ? 0 : 1;  // other parts begin with this row
    const int b = q + wave * each, e = min(q1, b + each);
    for (int c0 = blockIdx.y * kJoinColumns; c0 < a.width; c0 += gridDim.y * kJoinColumns) {
      const int col = c0 + 4 * lane, left = a.width - col;
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      if (left >= 4) {
        for (int p = b; p < e; p += U) {
          u32x4 y[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int pu = min(p + u, e - 1);
            y[u] = *reinterpret_cast<const any_u32x4*>(a.part + (int64_t(pu) * 2 + (pu == q ? s0 : 0)) * a.width + col);
          }
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] += p + u < e ? __uint_as_float(y[u][i]) : 0.f;
        }
      } else if (left > 0) {
        for (int p = b; p < e; ++p)
          for (int i = 0; i < left; ++i) x[i] += a.part[(int64_t(p) * 2 + (p == q ? s0 : 0)) * a.width + col + i];
      }
      sums[wave][lane] = make_float4(x[0], x[1], x[2], x[3]);
      __syncthreads();
      if (wave == 0) {
#pragma unroll
        for (int w = 1; w < W; ++w) {
          const float4 y = sums[w][lane];
          x[0] += y.x, x[1] += y.y, x[2] += y.z, x[3] += y.w;
        }
        T* o = static_cast<T*>(a.out) + int64_t(v) * a.width + col;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < left) Vec<T>::put(o + i, x[i] * a.scale);
      }
      __syncthreads();
    }
  }
}

template <typename F>
hipError_t by_type(int dtype, bool token64, F f) {
  if (dtype == TREE_DTYPE_BF16) return token64 ? f(uint16_t{}, int64_t{}) : f(uint16_t{}, int32_t{});
  return token64 ? f(float{}, int64_t{}) : f(float{}, int32_t{});
}

uint32_t groups(int64_t items, int lanes_log2) {
  // A launch's work items are counted in 32 bits; past that an item's threads
  // take several.
  const int64_t each = kThreads >> lanes_log2, most = (int64_t(1) << 24) - 64;
  return static_cast<uint32_t>(std::min((items + each - 1) / each, most));
}

}  // namespace

// Threads of one row: a power of two that covers it, `least` at least and 256 at most.
int embed_lanes_log2(int32_t width, int dtype, int least) {
  const int n = dtype == TREE_DTYPE_BF16 ? 8 : 4;
  int l = least;
  while (l < 8 && (int64_t(n) << l) < width) ++l;
  return l;
}

hipError_t launch_embed(const EmbedArgs& a, int dtype, bool token64, hipStream_t stream) {
  return by_type(dtype, token64, [&](auto t, auto i) {
    embed_kernel<decltype(t), decltype(i)><<<groups(a.n_tokens, a.lanes_log2), kThreads, 0, stream>>>(a);
    return hipGetLastError();
  });
}

hipError_t launch_embed_backward(const EmbedArgs& a, int dtype, bool token64, hipStream_t stream) {
  return by_type(dtype, token64, [&](auto t, auto i) {
    using T = decltype(t);
    sort_kernel<T, decltype(i)><<<(a.vocab + a.span - 1) / a.span, kSortThreads, 0, stream>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.n_tokens == 0) return e;
    sum_kernel<T><<<groups(a.n_tokens + a.n_parts, a.lanes_log2), kThreads, 0, stream>>>(a);
    e = hipGetLastError();
    if (e != hipSuccess || a.n_parts == 0) return e;
    const int columns = (a.width + kJoinColumns - 1) / kJoinColumns;
    const dim3 grid(std::min(a.n_parts, 65536), std::min(columns, 64));
    join_kernel<T><<<grid, kThreads, 0, stream>>>(a);
    return hipGetLastError();
  });
}

}  // namespace tg
