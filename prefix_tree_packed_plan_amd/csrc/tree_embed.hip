// Token embedding and its gradient (gfx950):
//     out_n = scale * table[tok n],   dtable[v] = scale * sum over n with tok n = v of dout_n.
// A token outside the table has no row: its output is 0 and its gradient goes nowhere.
//
// Both are bound by memory: rows are read and written once, 16 bytes a lane
// (rows need not be aligned to 16 bytes: the hardware reads and writes such
// pieces at any address).
//
// The gradient takes the tokens sorted by their row of the table.  sort_kernel
// makes that order: every work-group owns `span` rows and looks through all
// tokens twice (they come from L2: 512 work-groups read 10240 tokens of 8 bytes
// in 3 us), first to count, then to place.  It needs no pass over global
// memory and no atomic whose order shows: each wave keeps counters of its own
// for its share of the tokens, and within 64 tokens a lane's place among its
// equals comes from comparing the ids bit by bit.  A row's list is therefore
// in ascending order of the tokens, and the sums are the same in every run.
//
// sum_kernel then writes every row of the gradient, also those without a
// token.  Rows of more than kPart tokens would keep one work-group busy long
// after the others (a token that is a fifth of all of them); their lists are cut
// into parts at multiples of kPart, and join_kernel adds the parts in order.
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
// This work-group's rows: lo .. lo + span - 1.  cnt[w][r]: tokens of row lo + r in
// wave w's share; then where its next one goes.
template <typename I>
__global__ __launch_bounds__(kSortThreads) void sort_kernel(EmbedArgs a) {
  constexpr int U = 8;
  __shared__ int cnt[kSortWaves * kEmbedSpan];
  __shared__ int wave_total[kSortWaves];
  __shared__ int wave_less[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lo = blockIdx.x * a.span, span = min(a.span, a.vocab - lo);
  const int n = static_cast<int>(a.n_tokens);
  const int share = ((n + kSortThreads - 1) / kSortThreads) * 64;
  const int t0 = min(n, wave * share), t1 = min(n, t0 + share);
  int* mine = cnt + wave * kEmbedSpan;
  for (int i = tid; i < kSortWaves * kEmbedSpan; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  // Calls f(token's row minus lo, n) for 64 tokens at a time, in order; -1 past
  // the end or without a row.
  const auto each = [&](auto f) {
    for (int t = t0; t < t1; t += 64 * U) {
      int id[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = t + 64 * u + lane;
        id[u] = at < t1 ? token<I>(a, at) : -1;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) f(id[u], t + 64 * u + lane);
    }
  };
  int less = 0;
  each([&](int id, int) {
    less += id >= 0 && id < lo;
    const int r = id - lo;
    if (id >= lo && r < span) atomicAdd(&mine[r], 1);
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
  each([&](int id, int t) {
    const int r = id - lo;
    const bool in = id >= lo && r < span;
    uint64_t same = __ballot(in);
    if (same == 0) return;
#pragma unroll
    for (int b = 0; b < kEmbedSpanLog2; ++b) {
      const uint64_t ones = __ballot((r >> b) & 1);
      same &= (r >> b) & 1 ? ones : ~ones;
    }
    const uint64_t below = same & ((uint64_t(1) << lane) - 1);
    int first = 0;
    // The first of its equals moves their counter on; waves share none.
    if (in && below == 0) first = atomicAdd(&mine[r], static_cast<int>(__popcll(same)));
    const int leader = in ? __builtin_ctzll(same) : lane;
    first = __shfl(first, leader, 64);
    if (in) a.order[first + __popcll(below)] = t;
  });
}

// ---- sums ----------------------------------------------------------------------------
// Positions p0 .. p1 - 1 of the order, this lane's piece j (or, TAIL, column j),
// added in ascending order with U rows' loads in flight.
template <typename T, bool TAIL>
__device__ __forceinline__ void add_rows(const EmbedArgs& a, int p0, int p1, int64_t col, float* x) {
  constexpr int N = TAIL ? 1 : Vec<T>::N, U = 8;
  const T* d = static_cast<const T*>(a.dout) + col;
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = 0.f;
  for (int p = p0; p < p1; p += U) {
    int64_t row[U];
#pragma unroll
    for (int u = 0; u < U; ++u) row[u] = a.order[min(p + u, p1 - 1)];
    if constexpr (TAIL) {
      float w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) w[u] = Vec<T>::one(d + row[u] * a.width);
#pragma unroll
      for (int u = 0; u < U; ++u) x[0] += p + u < p1 ? w[u] : 0.f;
    } else {
      u32x4 w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) w[u] = *reinterpret_cast<const any_u32x4*>(d + row[u] * a.width);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (p + u >= p1) break;
        float y[N];
        Vec<T>::unpack(w[u], y);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += y[i];
      }
    }
  }
}

// Calls f(whether it is a single column, column) for this thread's pieces of a row.
template <typename T, typename F>
__device__ __forceinline__ void columns(const EmbedArgs& a, const Item& it, F f) {
  constexpr int N = Vec<T>::N;
  const int vecs = a.width / N;
  for (int j = it.j0; j < vecs; j += it.lanes) f(std::false_type{}, j * N);
  for (int c = vecs * N + it.j0; c < a.width; c += it.lanes) f(std::true_type{}, c);
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

// Items 0 .. vocab - 1: rows of the table; then the parts of long lists.  Part q
// is positions kPart q .. kPart (q + 1) - 1; at most its first and its last row have
// more than kPart tokens, and their sums are part[q][0] and part[q][1].
template <typename T, typename I>
__device__ __forceinline__ void sum_part(const EmbedArgs& a, const Item& it) {
  const int q = static_cast<int>(it.i - a.vocab);
  const int p0 = q * kPart, p1 = min(a.start[a.vocab], p0 + kPart);
  if (p0 >= p1) return;
  const int first = token<I>(a, a.order[p0]), last = token<I>(a, a.order[p1 - 1]);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int v = s ? last : first;
    if (s && last == first) break;
    const int r0 = a.start[v], r1 = a.start[v + 1];
    if (r1 - r0 <= kPart) continue;
    float* out = a.part + (int64_t(q) * 2 + s) * a.width;
    columns<T>(a, it, [&](auto tail, int col) {
      constexpr bool TAIL = decltype(tail)::value;
      float x[Vec<T>::N];
      add_rows<T, TAIL>(a, max(p0, r0), min(p1, r1), col, x);
#pragma unroll
      for (int i = 0; i < (TAIL ? 1 : Vec<T>::N); ++i) out[col + i] = x[i];
    });
  }
}

template <typename T, typename I>
__global__ __launch_bounds__(kThreads) void sum_kernel(EmbedArgs a) {
  Item it(a);
  for (; it.i < a.vocab; it.next()) {
    const int p0 = a.start[it.i], p1 = a.start[it.i + 1];
    if (p1 - p0 > kPart) continue;
    columns<T>(a, it, [&](auto tail, int col) {
      constexpr bool TAIL = decltype(tail)::value;
      float x[Vec<T>::N];
      add_rows<T, TAIL>(a, p0, p1, col, x);
      put_row<T, TAIL>(a, it.i, col, x);
    });
  }
  for (; it.i < int64_t(a.vocab) + a.n_parts; it.next()) sum_part<T, I>(a, it);
}

// Item q: the row of more than kPart tokens whose list begins in part q, if there is
// one (it reaches past the part's end, so there is at most one).
template <typename T, typename I>
__global__ __launch_bounds__(kThreads) void join_kernel(EmbedArgs a) {
  constexpr int U = 16;
  for (Item it(a); it.i < a.n_parts; it.next()) {
    const int q = static_cast<int>(it.i), end = (q + 1) * kPart;
    if (end > a.start[a.vocab]) continue;
    const int v = token<I>(a, a.order[end - 1]);
    const int r0 = a.start[v], r1 = a.start[v + 1];
    if (r1 - r0 <= kPart || r0 < q * kPart) continue;
    const int q1 = (r1 - 1) / kPart;
    const int s0 = r0 == q * kPart ? 0 : 1;  // other parts begin with this row
    columns<T>(a, it, [&](auto tail, int col) {
      constexpr bool TAIL = decltype(tail)::value;
      constexpr int N = TAIL ? 1 : Vec<T>::N;
      float x[Vec<T>::N] = {};
      for (int p = q; p <= q1; p += U) {
        float y[U][N];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int pu = min(p + u, q1);
          const float* src = a.part + (int64_t(pu) * 2 + (pu == q ? s0 : 0)) * a.width + col;
#pragma unroll
          for (int i = 0; i < N; ++i) y[u][i] = src[i];
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (p + u <= q1)
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] += y[u][i];
      }
      put_row<T, TAIL>(a, v, col, x);
    });
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

// Threads of one row: a power of two that covers it, 256 at most.
int embed_lanes_log2(int32_t width, int dtype) {
  const int n = dtype == TREE_DTYPE_BF16 ? 8 : 4;
  int l = 0;
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
    using I = decltype(i);
    sort_kernel<I><<<(a.vocab + a.span - 1) / a.span, kSortThreads, 0, stream>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    sum_kernel<T, I><<<groups(int64_t(a.vocab) + a.n_parts, a.lanes_log2), kThreads, 0, stream>>>(a);
    e = hipGetLastError();
    if (e != hipSuccess || a.n_parts == 0) return e;
    join_kernel<T, I><<<groups(a.n_parts, a.lanes_log2), kThreads, 0, stream>>>(a);
    return hipGetLastError();
  });
}

}  // namespace tg
