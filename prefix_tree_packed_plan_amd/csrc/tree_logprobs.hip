// Log probabilities of a trie's tokens, and their gradient (gfx950).
//
// With z = logits / T of one row, lse = log sum_i exp(z_i), p_i = exp(z_i -
// lse) and H = -sum_i p_i log p_i = lse - sum_i p_i z_i:
//   token t behind the row:  logp_t = z_{tok t} - lse,
//   dz_i = sum_t g_t ([i = tok t] - p_i) - h p_i (log p_i + H)
// for gradients g_t of logp_t and h of H.  A row in the middle of a segment
// has one token behind it; the last row of a segment has the first token of
// every child ("Tree Training" section 3.1 Eq. 6: each token's value is the
// one of its own root-to-leaf path), whose gradients add up in that row.
//
// Both kernels read the logits once.  The forward works in powers of 2: with c
// = log2(e) / T and a whole number M per lane (raised only when a value passes
// 2^(M + 10), so nearly never), y = c x - M in one rounding, s = sum exp2(y)
// and t = sum exp2(y) y; then lse = (M + log2 s) / log2(e), logp = (c x - M -
// log2 s) / log2(e), H = (log2 s - t / s) / log2(e).  M being whole, changing it
// is exact, and c's own rounding cancels in logp and H.  M stays within +-2^22,
// where c x rounded to fp32 still tells whole numbers apart: masked values far
// below add 0.  A row whose largest c x lies outside (nothing but masked values,
// or values of millions) is read a second time, relative to its largest x.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/tree_gdn.h"
#include "chunk_mfma.hpp"
#include "launch.hpp"

namespace tg {

namespace {

using chunk::ex2;
using chunk::kLog2e;
using chunk::pk2;

constexpr int kThreads = 256;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kFltMax = 3.40282347e38f;
constexpr int kNoId = 0x7FFFFFFF;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

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
  static __device__ __forceinline__ u32x4 none() { return u32x4{0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u}; }
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
  static __device__ __forceinline__ u32x4 none() { return u32x4{0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u}; }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ void put(float* p, float x) { *p = x; }
};

// A slice of a row: columns [0, head) and [tail, n) element by element (they
// are not part of an aligned 16-byte piece), the rest in `vecs` pieces.
template <typename T>
struct Slice {
  const T* p;
  int n, head, vecs, tail;
  __device__ __forceinline__ Slice(const T* base, int count) : p(base), n(count) {
    constexpr int N = Vec<T>::N;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    head = min(n, off ? N - off : 0);
    vecs = (n - head) / N;
    tail = head + vecs * N;
  }
  // Element-wise column of thread i (i < ends()).
  __device__ __forceinline__ int ends() const { return head + n - tail; }
  __device__ __forceinline__ int end_col(int i) const { return i < head ? i : tail + i - head; }
};

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

// The tokens behind packed row r.
struct Behind {
  int n, row;         // how many; the only one's row (middle of a segment)
  const int32_t *kid, *seg_off;
  bool root_start;    // r is a root's first token (it has no row in front)
  __device__ __forceinline__ Behind(const LogprobArgs& a, int r, int lane) : seg_off(a.seg_off) {
    const int s = seg_of(a.seg_off, a.n_seg, r, lane);
    const bool last = r + 1 == a.seg_off[s + 1];
    kid = last ? a.kid + a.kid_off[s] : nullptr;
    n = last ? a.kid_off[s + 1] - a.kid_off[s] : 1;
    row = r + 1;
    root_start = a.parent[s] < 0 && r == a.seg_off[s];
  }
  __device__ __forceinline__ int at(int j) const { return kid ? seg_off[kid[j]] : row; }
};

// Token id of row t, or -1 where it is outside the vocabulary.
__device__ __forceinline__ int token(const LogprobArgs& a, int t) {
  if (a.token64) {
    const int64_t x = static_cast<const int64_t*>(a.tokens)[t];
    return x >= 0 && x < a.vocab ? static_cast<int>(x) : -1;
  }
  const int32_t x = static_cast<const int32_t*>(a.tokens)[t];
  return x >= 0 && x < a.vocab ? x : -1;
}

// Thread j's token behind the row, if there is one, and its logit: half a dozen
// dependent loads.
template <typename T>
struct Ahead {
  int t = -1, id = -1;
  float x = 0.f;
  __device__ __forceinline__ Ahead(const LogprobArgs& a, int lr, const Behind& b, int j) {
    if (j < b.n) {
      t = b.at(j);
      id = token(a, t);
      if (id >= 0) x = Vec<T>::one(static_cast<const T*>(a.logits) + int64_t(lr) * a.ld + id);
    }
  }
};

// ---- the largest values of a row ------------------------------------------------
// The k-th largest of the wave's 64 values, none of them NaN (a bitonic sort, in
// which fmaxf and fminf would replace a NaN by a second copy of its partner).
__device__ __forceinline__ float kth_largest(float x, int k, int lane) {
#pragma unroll
  for (int size = 2; size <= 64; size *= 2)
#pragma unroll
    for (int o = size / 2; o; o /= 2) {
      const float y = __shfl_xor(x, o, 64);
      const bool down = (lane & size) == 0;  // this run is sorted downwards
      x = ((lane & o) == 0) == down ? fmaxf(x, y) : fminf(x, y);
    }
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), k - 1));
}

// A wave's list, best first: lane j < k holds entry j.  Ties go to the lowest
// index.  (tv, ti) is the last entry, which a new one has to beat.
struct TopList {
  float v = kNegInf, tv = kNegInf;
  int id = kNoId, ti = kNoId, k;
  __device__ __forceinline__ explicit TopList(int k_) : k(k_) {}
  static __device__ __forceinline__ bool better(float x, int i, float y, int j) { return x > y || (x == y && i < j); }
  // One candidate per lane (index kNoId: none), if it is at least `floor`.
  __device__ __forceinline__ void offer(float x, int i, int lane, float floor = kNegInf) {
    uint64_t m = __ballot(x >= floor && better(x, i, tv, ti));
    while (m) {
      const int src = __builtin_ctzll(m);
      const float nx = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), src));
      const int ni = __builtin_amdgcn_readlane(i, src);
      const int pos = __popcll(__ballot(lane < k && better(v, id, nx, ni)));
      // The entries from pos on move up by one lane.
      const float up = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x138, 0xf, 0xf, false));
      const int upi = __builtin_amdgcn_update_dpp(0, id, 0x138, 0xf, 0xf, false);
      v = lane > pos ? up : lane == pos ? nx : v;
      id = lane > pos ? upi : lane == pos ? ni : id;
      tv = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), k - 1));
      ti = __builtin_amdgcn_readlane(id, k - 1);
      m &= m - 1;
      m &= __ballot(better(x, i, tv, ti));
    }
  }
  // What a value has to reach to be worth offering, given each lane's largest
  // of those at hand: while the list is not full, the k-th largest of these
  // (at least k values reach it), which spares most of the first insertions.  A
  // lane with nothing but NaN has none.
  __device__ __forceinline__ float floor_of(float big, int lane) const {
    return ti == kNoId ? kth_largest(big == big ? big : kNegInf, k, lane) : tv;
  }
};

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int o = 32; o; o >>= 1) x += __shfl_xor(x, o, 64);
  return x;
}

// ---- forward --------------------------------------------------------------------
struct Sums {
  float m, s, t;  // M (-inf: nothing yet), sum of e = exp2(y), sum of e y
  float top;      // the largest value
};
// The sums of both, over the larger M.
__device__ __forceinline__ Sums join(const Sums a, const Sums b) {
  const float m = fmaxf(a.m, b.m);
  const float top = fmaxf(a.top, b.top);
  if (m == kNegInf) return Sums{m, a.s + b.s, a.t + b.t, top};
  Sums r{m, 0.f, 0.f, top};
  // A factor of 0 (that side is empty, or far below) drops t, whose shift may
  // overflow; a NaN stays in s.
  const float da = a.m - m, db = b.m - m;
  const float fa = ex2(da), fb = ex2(db);
  r.s = a.s * fa + b.s * fb;
  r.t = (fa == 0.f ? 0.f : fmaf(da, a.s, a.t) * fa) + (fb == 0.f ? 0.f : fmaf(db, b.s, b.t) * fb);
  return r;
}

// The M for values up to x: c x rounded to a whole number, within +-kMostM.
// Past 2^23 or so a rounded c x is off by more than exp2 allows.
constexpr float kMostM = 4194304.f;
__device__ __forceinline__ float whole(float x, float c) {
  return x == kNegInf ? kNegInf : rintf(fminf(fmaxf(x * c, -kMostM), kMostM));
}
// Whether a row's sums by M are none, because its largest value is outside
// what M covers (+inf too: its row becomes NaN).
__device__ __forceinline__ bool far(float top, float c) { return top != kNegInf && fabsf(top * c) > kMostM; }

// The sums of such a row, y = c (x - top): this thread's share, columns tid,
// tid + nt, ..
template <typename T>
__device__ __forceinline__ Sums far_sums(const T* x, int n, float top, float c, int tid, int nt) {
  Sums z{0.f, 0.f, 0.f, top};
#pragma unroll 4
  for (int i = tid; i < n; i += nt) {
    const float y = (Vec<T>::one(x + i) - top) * c, e = ex2(y);
    z.s += e;
    z.t = fmaf(e, fmaxf(y, -3.4e38f), z.t);  // e = 0 where y = -inf
  }
  return z;
}
template <typename T>
struct Scan {
  static constexpr int N = Vec<T>::N;
  float c;
  float limit = kNegInf;  // a value above this raises M
  float m = kNegInf, mr = 0.f, s = 0.f, t = 0.f, top = kNegInf;
  __device__ __forceinline__ explicit Scan(float c_) : c(c_) {}
  // n values (the others -inf).
  template <int n>
  __device__ __forceinline__ float add(const float* x) {
    float big = x[0];
#pragma unroll
    for (int j = 1; j < n; ++j) big = fmaxf(big, x[j]);
    top = fmaxf(top, big);
    if (__any(big > limit)) {
      const float mn = fmaxf(m, whole(big, c));
      const float d = m == kNegInf ? 0.f : m - mn, f = ex2(d);
      t = f == 0.f ? 0.f : fmaf(d, s, t) * f;
      s *= f;
      m = mn;
      mr = m == kNegInf ? 0.f : m;
      limit = m == kNegInf ? kNegInf : (m + 10.f) / c;
    }
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const float y = fmaf(x[j], c, -mr), e = ex2(y);
      s += e;
      t = fmaf(e, fmaxf(y, -3.4e38f), t);  // e = 0 where y = -inf
    }
    return big;
  }
};

// Log probabilities of one row, from its sums (far_sums where `away`).
template <typename T>
struct Row {
  float c, m, top, ls;  // ls: log2 of the sum of exponentials
  float entropy, lse;
  bool empty;           // every logit is -inf
  bool away;
  __device__ __forceinline__ Row(const LogprobArgs& a, const Sums z, bool away_)
      : c(a.inv_t * kLog2e), m(z.m), top(z.top), away(away_) {
    empty = z.s == 0.f && top == kNegInf;
    ls = __log2f(z.s);
    lse = (m + ls) * kLn2;
    if (away) {  // held at the type's largest value; a NaN stays one
      lse = fmaf(top, a.inv_t, ls * kLn2);
      lse = lse < -kFltMax ? -kFltMax : lse > kFltMax ? kFltMax : lse;
    }
    entropy = (ls - z.t / z.s) * kLn2;
    if (empty) {
      lse = kNegInf;
      entropy = 0.f;
    }
  }
  __device__ __forceinline__ float logp(float v) const {
    if (empty) return kNegInf;
    return ((away ? (v - top) * c : fmaf(v, c, -m)) - ls) * kLn2;
  }
};

// Everything a row's sums decide but the list, by the threads tid, tid + nt, ...
template <typename T>
__device__ __forceinline__ void finish_row(const LogprobArgs& a, int lr, const Row<T>& row, const Behind& b,
                                           const Ahead<T>& first, int tid, int nt) {
  if (tid == 0) {
    a.lse[lr] = row.lse;
    a.entropy[lr] = row.entropy;
    if (b.root_start) a.logp[a.first_row + lr] = 0.f;
  }
  if (first.t >= 0) a.logp[first.t] = first.id < 0 ? 0.f : row.logp(first.x);
  for (int j = tid + nt; j < b.n; j += nt) {
    const Ahead<T> next(a, lr, b, j);
    a.logp[next.t] = next.id < 0 ? 0.f : row.logp(next.x);
  }
}
template <typename T>
__device__ __forceinline__ void put_top(const LogprobArgs& a, int lr, const Row<T>& row, const TopList& l, int lane) {
  if (lane >= a.top_k) return;
  const int64_t o = int64_t(lr) * a.top_k + lane;
  a.top_id[o] = l.id == kNoId ? -1 : l.id;
  a.top_logp[o] = row.logp(l.v);
}
__device__ __forceinline__ float* part_lists(const LogprobArgs& a) {
  return a.part + int64_t(a.n_rows) * a.split * 4;
}

// One work-group a row, or a slice of one (SPLIT: `split` slices a row, where
// rows alone do not fill the card), U 16-byte non-temporal loads in flight a
// thread.  8192 x 131072 bf16: 324 us, 6.6 TB/s of reads, with the vector units
// 82% busy (about 8 instructions an element): memory and issue are near their
// ends together, which is why the sums take y from one fma and no maximum is
// exchanged between lanes.  With 5 alternatives the insertions are what is left:
// 4283 x 50001 bf16, 98 us against 73 without.
template <typename T, bool TOP, bool SPLIT>
__global__ __launch_bounds__(kThreads) void logprobs_kernel(LogprobArgs a) {
  constexpr int N = Vec<T>::N, U = 4;
  __shared__ Sums sums[kThreads / 64];
  __shared__ float tv[TOP ? kThreads : 1];
  __shared__ int ti[TOP ? kThreads : 1];
  __shared__ float last[kThreads / 64];  // each wave's last entry
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = blockIdx.x / a.split, part = blockIdx.x % a.split;
  const int c0 = part * a.slice;
  const Slice<T> sl(static_cast<const T*>(a.logits) + int64_t(lr) * a.ld + c0, min(a.slice, a.vocab - c0));
  Scan<T> sc(a.inv_t * kLog2e);
  TopList top(a.top_k);

  // A value below another wave's last entry is not among the row's top_k
  // either.  The waves read these whenever they come by: that decides how many
  // values are offered in vain, not which stay.
  volatile float* const lasts = last;
  float others = kNegInf;
  if constexpr (TOP) {
    if (tid < kThreads / 64) last[tid] = kNegInf;
    __syncthreads();
  }
  const auto* pv = reinterpret_cast<const u32x4*>(sl.p + sl.head);
  // A piece of N columns from col on (kNoId: none, all -inf).
  auto one = [&](const float* x, int col) {
    const float big = sc.template add<N>(x);
    if constexpr (TOP) {
      if (__any(big >= fmaxf(top.tv, others))) {
        const float floor = fmaxf(top.floor_of(col == kNoId ? kNegInf : big, lane), others);
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (__any(x[j] >= floor)) top.offer(x[j], col == kNoId ? kNoId : col + j, lane, floor);
        if (lane == 0) lasts[wave] = top.tv;
      }
    }
  };
  int v = tid;
  for (int i = 0; i < sl.vecs / (U * kThreads); ++i, v += U * kThreads) {
    u32x4 w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = __builtin_nontemporal_load(pv + v + u * kThreads);
    if constexpr (TOP) others = fmaxf(fmaxf(lasts[0], lasts[1]), fmaxf(lasts[2], lasts[3]));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float x[N];
      Vec<T>::unpack(w[u], x);
      one(x, c0 + sl.head + (v + u * kThreads) * N);
    }
  }
  // The last pieces, loaded together, and the columns outside of them; lanes
  // without one add -inf, which changes nothing.
  const int turns = (sl.vecs - (v - tid) + kThreads - 1) / kThreads;
  {
    u32x4 w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      w[u] = Vec<T>::none();
      if (v + u * kThreads < sl.vecs) w[u] = __builtin_nontemporal_load(pv + v + u * kThreads);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u >= turns) break;
      float x[N];
      Vec<T>::unpack(w[u], x);
      one(x, v + u * kThreads < sl.vecs ? c0 + sl.head + (v + u * kThreads) * N : kNoId);
    }
  }
  if (wave == 0) {
    const int i = lane;
    const bool has = i < sl.ends();
    const float x = has ? Vec<T>::one(sl.p + sl.end_col(i)) : kNegInf;
    sc.template add<1>(&x);
    if constexpr (TOP) top.offer(x, has ? c0 + sl.end_col(i) : kNoId, lane);
  }

  Sums z{sc.m, sc.s, sc.t, sc.top};
#pragma unroll
  for (int o = 32; o; o >>= 1)
    z = join(z, Sums{__shfl_xor(z.m, o, 64), __shfl_xor(z.s, o, 64), __shfl_xor(z.t, o, 64), __shfl_xor(z.top, o, 64)});
  if (lane == 0) sums[wave] = z;
  if constexpr (TOP) {
    tv[tid] = top.v;
    ti[tid] = top.id;
  }
  __syncthreads();
  z = sums[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) z = join(z, sums[w]);
  if constexpr (TOP) {
    if (wave == 0) {
#pragma unroll
      for (int w = 1; w < kThreads / 64; ++w) {
        const bool has = lane < a.top_k;
        top.offer(has ? tv[64 * w + lane] : kNegInf, has ? ti[64 * w + lane] : kNoId, lane);
      }
    }
  }
  if (!SPLIT) {
    const Behind b(a, a.first_row + lr, lane);
    const Ahead<T> first(a, lr, b, tid);
    const bool away = far(z.top, sc.c);
    if (away) {  // uniform over the work-group
      z = far_sums<T>(static_cast<const T*>(a.logits) + int64_t(lr) * a.ld, a.vocab, z.top, sc.c, tid, kThreads);
      z.s = wave_sum(z.s);
      z.t = wave_sum(z.t);
      __syncthreads();  // sums has been read
      if (lane == 0) sums[wave] = z;
      __syncthreads();
      z = sums[0];
#pragma unroll
      for (int w = 1; w < kThreads / 64; ++w) {
        z.s += sums[w].s;
        z.t += sums[w].t;
      }
    }
    const Row<T> row(a, z, away);
    finish_row<T>(a, lr, row, b, first, tid, kThreads);
    if (TOP && wave == 0) put_top<T>(a, lr, row, top, lane);
  } else {
    if (tid == 0) *reinterpret_cast<float4*>(a.part + int64_t(blockIdx.x) * 4) = make_float4(z.m, z.s, z.t, z.top);
    if (TOP && wave == 0 && lane < a.top_k)
      *reinterpret_cast<float2*>(part_lists(a) + (int64_t(blockIdx.x) * a.top_k + lane) * 2) =
          make_float2(top.v, __int_as_float(top.id));
  }
}

// A row spread over several work-groups: its sums and lists joined by one wave.
template <typename T, bool TOP>
__global__ __launch_bounds__(64) void logprobs_join_kernel(LogprobArgs a) {
  const int lane = threadIdx.x, lr = blockIdx.x;
  const Behind b(a, a.first_row + lr, lane);
  const Ahead<T> first(a, lr, b, lane);
  Sums z{kNegInf, 0.f, 0.f, kNegInf};
  for (int i = lane; i < a.split; i += 64) {
    const float4 y = *reinterpret_cast<const float4*>(a.part + (int64_t(lr) * a.split + i) * 4);
    z = join(z, Sums{y.x, y.y, y.z, y.w});
  }
#pragma unroll
  for (int o = 32; o; o >>= 1)
    z = join(z, Sums{__shfl_xor(z.m, o, 64), __shfl_xor(z.s, o, 64), __shfl_xor(z.t, o, 64), __shfl_xor(z.top, o, 64)});
  const float c = a.inv_t * kLog2e;
  const bool away = far(z.top, c);
  if (away) {
    z = far_sums<T>(static_cast<const T*>(a.logits) + int64_t(lr) * a.ld, a.vocab, z.top, c, lane, 64);
    z.s = wave_sum(z.s);
    z.t = wave_sum(z.t);
  }
  const Row<T> row(a, z, away);
  finish_row<T>(a, lr, row, b, first, lane, 64);
  if constexpr (TOP) {
    TopList top(a.top_k);
    const float2* l = reinterpret_cast<const float2*>(part_lists(a)) + int64_t(lr) * a.split * a.top_k;
    const int n = a.split * a.top_k;
    for (int i = lane; i < n + lane; i += 64) {
      const float2 y = i < n ? l[i] : make_float2(kNegInf, __int_as_float(kNoId));
      top.offer(y.x, __float_as_int(y.y), lane, top.floor_of(y.x, lane));
    }
    put_top<T>(a, lr, row, top, lane);
  }
}

// ---- backward ---------------------------------------------------------------------
constexpr int kListed = 512;  // tokens behind a row that are kept in LDS

// One slice of a row a work-group, read and written once: 8192 x 131072 bf16 in
// 704 us, 1685 x 50001 fp32 in 113 us (6.1 and 5.9 TB/s).  Slices of 16 KB, so
// that work-groups that run together stream through neighbouring memory: whole
// rows took 819 us, 64 KB 778, 32 KB 744.  The pieces that hold a token behind
// the row are marked in a bitmap, so that the others cost nothing for it.
//
// p = exp(x / T - lse) is off by 2^-24 |lse|, half a unit of lse.  From kFarLse on
// (a row of nothing but masked values, logits of tens of thousands) one of the
// row's work-groups therefore takes all of it, reading it once for its largest
// value and once for its sum relative to that; the others leave, so that the
// gradient may still be written over the logits.  Which one changes with the
// row, or one XCD had them all (8192 x 131072 bf16, all rows such: 2.1 ms against
// 9.7).
constexpr float kFarLse = 16384.f;
template <typename T>
__global__ __launch_bounds__(kThreads) void logprobs_backward_kernel(LogprobArgs a) {
  constexpr int N = Vec<T>::N, U = 4;
  __shared__ uint32_t flag[kMaxSlice / N / 32];  // pieces of the slice with a token behind the row
  __shared__ int ids[kListed];
  __shared__ float gs[kListed];
  __shared__ float wsum[kThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = blockIdx.x / a.split, part = blockIdx.x % a.split;
  const int c0 = part * a.slice;
  const Slice<T> sl(static_cast<const T*>(a.logits) + int64_t(lr) * a.ld + c0, min(a.slice, a.vocab - c0));
  T* out = static_cast<T*>(a.dlogits) + int64_t(lr) * a.ldd + c0;
  // The first pieces are on their way while the tokens behind the row are
  // looked up.
  const auto* pv = reinterpret_cast<const u32x4*>(sl.p + sl.head);
  const int rounds = sl.vecs / (U * kThreads);
  u32x4 w[U] = {};
  if (rounds > 0) {
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = __builtin_nontemporal_load(pv + tid + u * kThreads);
  }
  const Behind b(a, a.first_row + lr, lane);
  for (int i = tid; i < (sl.vecs + 31) / 32; i += kThreads) flag[i] = 0;
  __syncthreads();
  const auto mark = [&](const Slice<T>& sl, int c0, int id) {
    const int at = id - c0 - sl.head;
    if (id >= 0 && at >= 0 && at < sl.vecs * N) atomicOr(&flag[at / N >> 5], 1u << (at / N & 31));
  };
  // The gradients behind the row: their sum, and which pieces they touch.
  float g = 0.f;
  for (int j = tid; j < b.n; j += kThreads) {
    const int t = b.at(j), id = token(a, t);
    const float gj = id < 0 ? 0.f : a.dlogp[t];
    g += gj;
    if (j < kListed) {
      ids[j] = id;
      gs[j] = gj;
    }
    mark(sl, c0, id);
  }
  g = wave_sum(g);
  if (lane == 0) wsum[wave] = g;
  __syncthreads();
  g = 0.f;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) g += wsum[w];

  const float lse = a.lse_in[lr], dh = a.dentropy ? a.dentropy[lr] : 0.f;
  const bool empty = lse == kNegInf;
  const float ca = empty ? 0.f : -(g + dh * (a.dentropy ? a.entropy_in[lr] : 0.f)) * a.inv_t, cb = empty ? 0.f : -dh * a.inv_t;
  // What the tokens behind the row that equal `id` add, in their order.
  auto direct = [&](int id) {
    float s = 0.f;
    for (int j = 0; j < b.n; ++j) {
      if (j < kListed) {
        s += ids[j] == id ? gs[j] : 0.f;
      } else {
        const int t = b.at(j);
        if (token(a, t) == id) s += a.dlogp[t];
      }
    }
    return s * a.inv_t;
  };
  // The 16-byte pieces of a slice (the first ones are in w if `loaded`).
  auto pieces = [&](const Slice<T>& sl, bool loaded, auto use) {
    const auto* pv = reinterpret_cast<const u32x4*>(sl.p + sl.head);
    const int rounds = sl.vecs / (U * kThreads);
    int v = tid;
    for (int i = 0; i < rounds; ++i, v += U * kThreads) {
      if (i > 0 || !loaded) {
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] = __builtin_nontemporal_load(pv + v + u * kThreads);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) use(w[u], v + u * kThreads);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (v + u * kThreads < sl.vecs) w[u] = __builtin_nontemporal_load(pv + v + u * kThreads);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (v + u * kThreads < sl.vecs) use(w[u], v + u * kThreads);
  };
  // The gradients of a slice from column c0 on, to `out`.
  auto stream = [&](const Slice<T>& sl, T* out, int c0, bool loaded, auto grad) {
    const bool aligned = (reinterpret_cast<uintptr_t>(out + sl.head) & 15) == 0;
    pieces(sl, loaded, [&](const u32x4 w, int v) {
      float x[N];
      Vec<T>::unpack(w, x);
#pragma unroll
      for (int j = 0; j < N; ++j) x[j] = empty ? 0.f : grad(x[j]);
      if ((flag[v >> 5] >> (v & 31)) & 1 && !empty) {
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] += direct(c0 + sl.head + v * N + j);
      }
      T* o = out + sl.head + v * N;
      if (aligned) {
        __builtin_nontemporal_store(Vec<T>::pack(x), reinterpret_cast<u32x4*>(o));
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) Vec<T>::put(o + j, x[j]);
      }
    });
    if (tid < sl.ends()) {
      const int col = sl.end_col(tid);
      const float x = Vec<T>::one(sl.p + col);
      Vec<T>::put(out + col, empty ? 0.f : grad(x) + direct(c0 + col));
    }
  };

  if (fabsf(lse) < kFarLse || empty || lse != lse) {
    // The gradient of a value whose token is not behind the row.
    stream(sl, out, c0, rounds > 0, [&](float x) {
      const float lp = fmaf(x, a.inv_t, -lse);
      return ex2(lp * kLog2e) * fmaf(cb, fmaxf(lp, -1e4f), ca);  // exp is 0 below -104
    });
    return;
  }
  if (part != lr % a.split) return;  // uniform, as the branch above
  const Slice<T> all(static_cast<const T*>(a.logits) + int64_t(lr) * a.ld, a.vocab);
  const float c = a.inv_t * kLog2e;
  auto each = [&](auto use) {
    pieces(all, false, [&](const u32x4 w, int) {
      float x[N];
      Vec<T>::unpack(w, x);
#pragma unroll
      for (int j = 0; j < N; ++j) use(x[j]);
    });
    if (tid < all.ends()) use(Vec<T>::one(all.p + all.end_col(tid)));
  };
  float top = kNegInf, s = 0.f;
  each([&](float x) { top = fmaxf(top, x); });
#pragma unroll
  for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
  __syncthreads();  // wsum has been read
  if (lane == 0) wsum[wave] = top;
  __syncthreads();
  top = fmaxf(fmaxf(wsum[0], wsum[1]), fmaxf(wsum[2], wsum[3]));
  each([&](float x) { s += ex2((x - top) * c); });
  s = wave_sum(s);
  __syncthreads();
  if (lane == 0) wsum[wave] = s;
  __syncthreads();
  const float ls = __log2f(wsum[0] + wsum[1] + wsum[2] + wsum[3]);
  for (int q0 = 0; q0 < a.vocab; q0 += kMaxSlice) {
    const Slice<T> cur(all.p + q0, min(kMaxSlice, a.vocab - q0));
    __syncthreads();  // flag has been read
    for (int i = tid; i < (cur.vecs + 31) / 32; i += kThreads) flag[i] = 0;
    __syncthreads();
    for (int j = tid; j < b.n; j += kThreads) mark(cur, q0, j < kListed ? ids[j] : token(a, b.at(j)));
    __syncthreads();
    stream(cur, static_cast<T*>(a.dlogits) + int64_t(lr) * a.ldd + q0, q0, false, [&](float x) {
      const float y = (x - top) * c - ls;
      return ex2(y) * fmaf(cb, fmaxf(y * kLn2, -1e4f), ca);
    });
  }
}

}  // namespace

namespace {

// Calls f on as many rows at a time as one launch may have work-groups (its
// work items are counted in 32 bits).
template <typename F>
hipError_t by_rows(const LogprobArgs& a, int dtype, F f) {
  const int64_t size = dtype == TREE_DTYPE_BF16 ? 2 : 4, most = ((int64_t(1) << 24) - 64) / a.split;
  for (int64_t r = 0; r < a.n_rows; r += most) {
    LogprobArgs b = a;
    const int64_t n = a.n_rows - r < most ? a.n_rows - r : most;
    b.n_rows = static_cast<int32_t>(n);
    b.first_row = static_cast<int32_t>(a.first_row + r);
    b.logits = static_cast<const char*>(a.logits) + r * a.ld * size;
    b.entropy = a.entropy ? a.entropy + r : nullptr;
    b.lse = a.lse ? a.lse + r : nullptr;
    b.top_logp = a.top_logp ? a.top_logp + r * a.top_k : nullptr;
    b.top_id = a.top_id ? a.top_id + r * a.top_k : nullptr;
    b.dentropy = a.dentropy ? a.dentropy + r : nullptr;
    b.lse_in = a.lse_in ? a.lse_in + r : nullptr;
    b.entropy_in = a.entropy_in ? a.entropy_in + r : nullptr;
    b.dlogits = a.dlogits ? static_cast<char*>(a.dlogits) + r * a.ldd * size : nullptr;
    const hipError_t e = f(b);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_logprobs(const LogprobArgs& args, int dtype, hipStream_t stream) {
  return by_rows(args, dtype, [&](const LogprobArgs& a) {
    const dim3 grid(static_cast<uint32_t>(a.n_rows) * a.split), block(kThreads);
    const bool top = a.top_k > 0, split = a.split > 1;
    const auto kernel =
        dtype == TREE_DTYPE_BF16
            ? (top ? (split ? logprobs_kernel<uint16_t, true, true> : logprobs_kernel<uint16_t, true, false>)
                   : (split ? logprobs_kernel<uint16_t, false, true> : logprobs_kernel<uint16_t, false, false>))
            : (top ? (split ? logprobs_kernel<float, true, true> : logprobs_kernel<float, true, false>)
                   : (split ? logprobs_kernel<float, false, true> : logprobs_kernel<float, false, false>));
    kernel<<<grid, block, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !split) return e;
    const auto join = dtype == TREE_DTYPE_BF16
                          ? (top ? logprobs_join_kernel<uint16_t, true> : logprobs_join_kernel<uint16_t, false>)
                          : (top ? logprobs_join_kernel<float, true> : logprobs_join_kernel<float, false>);
    join<<<dim3(a.n_rows), 64, 0, stream>>>(a);
    return hipGetLastError();
  });
}

hipError_t launch_logprobs_backward(const LogprobArgs& args, int dtype, hipStream_t stream) {
  return by_rows(args, dtype, [&](const LogprobArgs& a) {
    const dim3 grid(static_cast<uint32_t>(a.n_rows) * a.split), block(kThreads);
    if (dtype == TREE_DTYPE_BF16) logprobs_backward_kernel<uint16_t><<<grid, block, 0, stream>>>(a);
    else logprobs_backward_kernel<float><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
  });
}

}  // namespace tg
