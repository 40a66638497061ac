// Log probabilities of a trie's tokens from hidden states and the output weight,
// and the gradients of both (gfx950).  With z = hidden weight^T / T, of row r and
// vocabulary entry v:
//     lse_r = log sum_v exp(z_rv),  p_rv = exp(z_rv - lse_r),
//     H_r = lse_r - sum_v p_rv z_rv,  logp_t = z_{r, tok t} - lse_r
// for every token t behind row r, and, for gradients g_t and h_r,
//     D_rv = (1 / T) (sum_t g_t [tok t = v] - G_r p_rv - h_r p_rv (log p_rv + H_r)),
//     dhidden = D weight,  dweight = D^T hidden,   G_r = sum_t g_t.
//
// The logits are never stored.  The forward computes them a tile of vocabulary x
// rows at a time (product_tile.hpp, vocabulary along m, so that a lane holds
// values of one row) and keeps each tile's largest value, sum of exponentials and
// sum of exponentials times exponent; a wave a row joins these and takes the dot
// products of the tokens behind it.  The backward goes through the vocabulary in
// pieces: a piece's D is computed from the same products, stored (rounded to the
// inputs' type, as the operand of the two products that follow; for few rows in bf16 as
// two bf16, a row of the largest parts and one of what they leave), and multiplied
// into dhidden, in fp32 over the pieces, and the piece's dweight.
//
// Measured (us; inputs that change from call to call): 8192 rows x 131072 x 4096 bf16 6460
// (1360 TFLOP/s; a library product of that shape alone reaches 1496), gradients of 8192 x
// 131072 x 2048 10340 (1280), fp32 1685 x 50001 x 1000 920 (183), gradients of 1526 x
// 20001 x 1000 1000 (183; a library fp32 product 155); 33 rows x 32000 x 2048 39 (the
// product 30: 131 MB of weight at 4.4 TB/s) and 126.  Where those 131 MB stay in the
// last-level cache these take 30 (22: 5.9 TB/s) and 105.  Large ones are bound by the matrix units at two thirds of their
// cycles, with DMA and LDS reads between, and by the clock under load.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/tree_gdn.h"
#include "launch.hpp"
#include "product_tile.hpp"
#include "trie_rows.hpp"

namespace tg {

namespace {

using chunk::ex2;
using chunk::kLog2e;
using chunk::f32x4;

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2eRest = 1.92596299e-8f;  // log2(e) - kLog2e
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kFltMax = 3.402823466e38f;

// Of some products x, whose logits are x / T: m (the largest; -inf: nothing yet), sum of e =
// exp2(y) with y = (x - m) c, c = log2(e) / T, and sum of e y.  The difference comes
// before the scale, so that m c may be too large for fp32 (entries masked by the
// lowest number) and y is off by roundings of its own size alone.
struct LinearSums {
  float m, s, t;
};
__device__ __forceinline__ LinearSums join(const LinearSums a, const LinearSums b, float c) {
  const float m = fmaxf(a.m, b.m);
  if (m == kNegInf) return LinearSums{m, a.s + b.s, a.t + b.t};
  LinearSums r;
  r.m = m;
  // A factor of 0 (that side is empty, or far below) drops t, whose shift may
  // overflow; a NaN stays in s.
  const float da = (a.m - m) * c, db = (b.m - m) * c;
  const float fa = ex2(da), fb = ex2(db);
  r.s = a.s * fa + b.s * fb;
  r.t = (fa == 0.f ? 0.f : fmaf(da, a.s, a.t) * fa) + (fb == 0.f ? 0.f : fmaf(db, b.s, b.t) * fb);
  return r;
}

// Four neighbouring values to a row of T.
template <typename T>
__device__ __forceinline__ void put4(void* p, int64_t i, float a, float b, float c, float d);
template <>
__device__ __forceinline__ void put4<uint16_t>(void* p, int64_t i, float a, float b, float c, float d) {
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = make_uint2(chunk::pk2(a, b), chunk::pk2(c, d));
}
template <>
__device__ __forceinline__ void put4<float>(void* p, int64_t i, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(a, b, c, d);
}

// Neighbouring blocks x and y, from m on, to a row of T; the row ends at `end`.
template <typename T>
__device__ __forceinline__ void put_blocks(T* row, int m, int g4, int end, const f32x4 x, const f32x4 y) {
  if constexpr (sizeof(T) == 2) {
    const uint4 w = product::pair_up(x, y);
    m += 16 * (g4 & 1) + 8 * (g4 >> 1);
    if (m < end) *reinterpret_cast<uint4*>(row + m) = w;
  } else {
    m += 4 * g4;
    if (m < end) *reinterpret_cast<f32x4*>(row + m) = x;
    if (m + 16 < end) *reinterpret_cast<f32x4*>(row + m + 16) = y;
  }
}

enum Use { kStats, kGrad, kSum };

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int o = 32; o; o >>= 1) x += __shfl_xor(x, o, 64);
  return x;
}

// hidden row lr x weight row id, to all lanes of a wave: by the matrix instructions of a
// tile in the tile's order, so that it is bitwise what the row's maximum and sum are made of
// (summed by 64 lanes, a log probability near 0 came out as up to 4e-5, width 4096; those
// of unlikely tokens are off by 1.9e-7 of their size instead of 0.5e-7, logits in torch's
// fp32 3.4e-7, 8192 rows x 131072 x 4096).
// Lane 16 g + i loads piece g of the i-th 32 k; of an instruction's 256 sums the i-th on
// the diagonal is the one wanted, and all start from the last one.
template <typename T>
__device__ __forceinline__ float logit(const LinearArgs& a, int lr, int id) {
  constexpr int E16 = 16 / sizeof(T), P = 8 / E16;  // pieces of 16 bytes a lane has of 32 k
  constexpr int U = sizeof(T) == 2 ? 4 : 1;         // 512 k, loaded at once
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const char* hrow = reinterpret_cast<const char*>(static_cast<const T*>(a.hidden) + int64_t(lr) * a.ld);
  const char* wrow = reinterpret_cast<const char*>(static_cast<const T*>(a.weight) + int64_t(id) * a.width);
  float x = 0.f, rest = 0.f;
  for (int k0 = 0; k0 < a.width; k0 += 512 * U) {
    uint4 w[U][P], h[U][P];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int k = k0 + 512 * u + 32 * i + 8 * g + E16 * p;
        const bool in = k < a.width;  // zeros past the end
        w[u][p] = in ? *reinterpret_cast<const uint4*>(wrow + k * sizeof(T)) : make_uint4(0, 0, 0, 0);
        h[u][p] = in ? *reinterpret_cast<const uint4*>(hrow + k * sizeof(T)) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      product::Split ws, hs;
      if constexpr (sizeof(T) == 4) {
        ws = product::split3(w[u]);
        hs = product::split3(h[u]);
      }
      product::unrolled<16>([&](auto step) {
        constexpr int j = decltype(step)::value, from = 16 * (j / 4) + j;
        if (k0 + 512 * u + 32 * j >= a.width) return;
        const auto diagonal = [&](const f32x4 c) {
          return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(c[j % 4]), from));
        };
        if constexpr (sizeof(T) == 2) {
          x = diagonal(product::mma(w[u][0], h[u][0], f32x4{x, x, x, x}));
        } else {
          rest = diagonal(product::mma_rest(ws, hs, f32x4{rest, rest, rest, rest}));
          x = diagonal(product::mma(ws.part(0), hs.part(0), f32x4{x, x, x, x}));
        }
      });
    }
  }
  return x + rest;
}

// Tokens and their logits, by work-groups beside those of the product, which they take
// no longer than: a wave a row, for the first token behind it, and a wave a segment
// that is not its parent's first child, for its first token (a row with 1024 children
// would keep one wave longer than the product takes).
//   found: (logit of the first token, that token, the row's segment, flags)
// The logits of further tokens go to their logp.
constexpr int kAny = 1, kOutside = 2, kMore = 4, kRootStart = 8;
template <typename T>
__device__ __forceinline__ void find_row(const LinearArgs& a, int lr, int4* found) {
  const int lane = threadIdx.x & 63;
  const Behind b(a, a.first_row + lr, lane);
  int flags = (b.n > 0 ? kAny : 0) | (b.n > 1 ? kMore : 0) | (b.root_start ? kRootStart : 0);
  const int t = b.n > 0 ? b.at(0) : 0, id = b.n > 0 ? token(a, t) : -1;
  if (id < 0) flags |= kOutside;
  const float x = id >= 0 ? logit<T>(a, lr, id) : 0.f;
  if (lane == 0) found[lr] = make_int4(__float_as_int(x), t, b.seg, flags);
}
template <typename T>
__device__ __forceinline__ void find_segment(const LinearArgs& a, int s) {
  const int p = a.parent[s];
  if (p < 0 || a.kid[a.kid_off[p]] == s) return;
  const int lr = a.seg_off[p + 1] - 1 - a.first_row, t = a.seg_off[s];
  if (lr < 0 || lr >= a.n_rows) return;
  const int id = token(a, t);
  const float x = id >= 0 ? logit<T>(a, lr, id) : 0.f;
  if ((threadIdx.x & 63) == 0) a.logp[t] = x;
}

// A product's operands and where its tiles stand.
struct Job {
  const char *a, *b;
  int64_t lda, ldb;         // bytes between stored rows
  int32_t m, n, k;
  int32_t m_tiles, n_tiles, band;  // tiles run through `band` n for each m
  int32_t splits, k_split;  // k is cut into `splits` of k_split (a multiple of a step)
  // kStats
  float c;                  // log2(e) / T
  float4* part;             // [n, m_tiles]: LinearSums of a tile's entries
  int4* found;              // [n]: find_row
  // kGrad: entry v0 + m
  const float4* row;        // RowGrad of each row
  const int4* ids;
  float inv_t;
  int32_t v0;
  void* d;                  // [padded n, ldd]
  int64_t ldd;
  int32_t stack;            // LinearWork's: rows `stack` .. have what rounding row 0 .. left
  // kSum: out[n][m], or fp32 sums (of a split) in acc
  void* out;
  float* acc;
  const float* add;         // or null: what `acc` or `out` starts from
  int64_t acc_split;        // elements between splits' sums
};

// The gradient's coefficients of a row: D = exp(z - lse) (cb log p + ca), plus g /
// T at the entries that stand behind it.
//   row: (lse, ca, cb, g of the first token)
//   ids: (the first token's entry or -1, tokens behind, first of them in kid or -1, a
//        product x0; lse is then that of the products less x0: 0 but for far rows)
template <typename T, typename C, bool BIG, Use USE>
__global__ __launch_bounds__(C::THREADS, C::OCC) void product_kernel(Job j, LinearArgs la) {
  constexpr int BM = C::BM, BN = C::BN, WM = C::WM;
  __shared__ __attribute__((aligned(1024))) char lds[C::LDS];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int tiles = j.m_tiles * j.n_tiles;
  if constexpr (USE == kStats) {
    // The work-groups behind the tiles'.
    if (static_cast<int>(blockIdx.x) >= tiles) {
      constexpr int W = C::THREADS / 64;
      const int64_t step = int64_t(gridDim.x - tiles) * W, end = int64_t(la.n_rows) + la.n_seg;
      for (int64_t i = int64_t(blockIdx.x - tiles) * W + wave; i < end; i += step) {
        if (i < la.n_rows) find_row<T>(la, static_cast<int>(i), j.found);
        else find_segment<T>(la, static_cast<int>(i - la.n_rows));
      }
      return;
    }
  }
  const int id = product::of_xcd(blockIdx.x, tiles * j.splits);
  const int split = id / tiles, tile = id % tiles;
  // Bands of `band` n tiles; within one, all n of an m.
  const int in_band = j.band * j.m_tiles, band = tile / in_band, at = tile % in_band;
  const int width = min(j.band, j.n_tiles - band * j.band);
  const int mt = at / width, nt = band * j.band + at % width;
  const int m0 = mt * BM, n0 = nt * BN;
  const int k0 = split * j.k_split, k = min(j.k - k0, j.k_split);

  f32x4 acc[C::MB][C::NB];
  if constexpr (BIG) {
    typename C::OpA A[2];
    typename C::OpB B[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // A second half past the end repeats the first (its results are not used).
      const int ma = m0 + 128 * i < j.m ? m0 + 128 * i : m0, nb = n0 + 128 * i < j.n ? n0 + 128 * i : n0;
      A[i].init(j.a, j.lda, ma, j.m - ma, k0, wave, lane);
      B[i].init(j.b, j.ldb, nb, j.n - nb, k0, wave, lane);
    }
    const typename C::RdA ra(4 * wm, lane);
    const typename C::RdB rb(C::NH * wn, lane);
    product::run_big<C>(acc, A, B, ra, rb, k, lds);
  } else {
    typename C::OpA A;
    typename C::OpB B;
    A.init(j.a, j.lda, m0, j.m - m0, k0, wave, lane);
    B.init(j.b, j.ldb, n0, j.n - n0, k0, wave, lane);
    const typename C::RdA ra(wm * C::MB, lane);
    const typename C::RdB rb(wn * C::NB, lane);
    product::run<C>(acc, A, B, ra, rb, k, lds);
  }
  // Blocks mb, nb begin at m0 + am(mb), n0 + an(nb).
  const auto am = [&](int mb) {
    return BIG ? 128 * (mb / 4) + 64 * wm + 16 * (mb % 4) : 16 * (wm * C::MB + mb);
  };
  constexpr int NH = C::NB / 2;
  const auto an = [&](int nb) { return BIG ? 128 * (nb / NH) + 16 * (NH * wn + nb % NH) : 16 * (wn * C::NB + nb); };

  const int l16 = lane & 15, g4 = lane >> 4;
  const int mw = m0 + 4 * g4, nw = n0 + l16;  // this lane's first m of block 0, and its n
  if constexpr (USE == kStats) {
    if (m0 + BM > j.m) {  // past the vocabulary
#pragma unroll
      for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (mw + am(mb) + i >= j.m)
#pragma unroll
            for (int nb = 0; nb < C::NB; ++nb) acc[mb][nb][i] = kNegInf;
    }
    float* red = reinterpret_cast<float*>(lds);  // [3][WM][BN]
    product::barrier();                          // the last step has been read
#pragma unroll
    for (int nb = 0; nb < C::NB; ++nb) {
      float top = kNegInf;
#pragma unroll
      for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, acc[mb][nb][i]);
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const float m = top == kNegInf ? 0.f : top;
      float s = 0.f, t = 0.f;
#pragma unroll
      for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float y = (acc[mb][nb][i] - m) * j.c, e = ex2(y);
          s += e;
          t = fmaf(e, fmaxf(y, -3.4e38f), t);  // e = 0 where y = -inf
        }
      s += __shfl_xor(s, 16, 64);
      t += __shfl_xor(t, 16, 64);
      s += __shfl_xor(s, 32, 64);
      t += __shfl_xor(t, 32, 64);
      if (g4 == 0) {
        const int o = wm * BN + an(nb) + l16;
        red[o] = top;
        red[o + WM * BN] = s;
        red[o + 2 * WM * BN] = t;
      }
    }
    __syncthreads();
    for (int n = tid; n < BN && n0 + n < j.n; n += C::THREADS) {
      LinearSums z{red[n], red[n + WM * BN], red[n + 2 * WM * BN]};
#pragma unroll
      for (int w = 1; w < WM; ++w)
        z = join(z, LinearSums{red[n + w * BN], red[n + (WM + w) * BN], red[n + (2 * WM + w) * BN]}, j.c);
      j.part[int64_t(n0 + n) * j.m_tiles + mt] = make_float4(z.m, z.s, z.t, 0.f);
    }
  } else if constexpr (USE == kGrad) {
#pragma unroll
    for (int nb = 0; nb < C::NB; ++nb) {
      const int n = nw + an(nb);
      const bool valid = n < j.n;
      const float4 rc = j.row[valid ? n : 0];
      const int4 who = j.ids[valid ? n : 0];
      const bool live = valid && rc.x != kNegInf;
      const float x0 = __int_as_float(who.w);
#pragma unroll
      for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float lp = fmaf(acc[mb][nb][i] - x0, j.inv_t, -rc.x), held = fmaxf(lp, -1e4f);  // exp is 0 below -104
          float e = ex2(lp * kLog2e);
          // That product's rounding, 2^-24 of up to 20 or more, is too much for fp32, and so
          // is its constant's, 2^-26 of as much and the same way in all entries.
          if (sizeof(T) == 4)
            e = fmaf(e, fmaf(held, kLog2eRest, fmaf(held, kLog2e, -(held * kLog2e))) * kLn2, e);
          acc[mb][nb][i] = e * fmaf(rc.z, held, rc.y);
        }
      if (!__all(live) || m0 + BM > j.m) {
#pragma unroll
        for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!live || mw + am(mb) + i >= j.m) acc[mb][nb][i] = 0.f;
      }
      // The tokens behind the row: the first here, further ones (a branch point's) below.
      const int o = live && who.y > 0 && who.x >= 0 ? who.x - j.v0 - mw : -1;
      if (__any(o >= 0 && o < BM)) {
#pragma unroll
        for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (o >= 0 && o == am(mb) + i) acc[mb][nb][i] += rc.w;
      }
      // A lane a token, and those in this tile one after another.
      uint64_t branch = __ballot(live && who.y > 1 && g4 == 0);
      while (branch) {
        const int c = __builtin_ctzll(branch), kids = __builtin_amdgcn_readlane(who.y, c);
        const int32_t* kid = la.kid + __builtin_amdgcn_readlane(who.z, c);
        branch &= branch - 1;
        for (int t = 1; t < kids; t += 64) {
          int v = -1;
          float g = 0.f;
          if (t + lane < kids) {
            const int at = la.seg_off[kid[t + lane]];
            v = token(la, at);
            g = v >= 0 ? la.dlogp[at] * j.inv_t : 0.f;
          }
          const int from = v < 0 ? -1 : v - j.v0 - m0;
          uint64_t hit = __ballot(from >= 0 && from < BM);
          while (hit) {
            const int l = __builtin_ctzll(hit);
            hit &= hit - 1;
            const int at = __builtin_amdgcn_readlane(from, l) - 4 * g4;
            const float add = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(g), l));
#pragma unroll
            for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (l16 == c && at == am(mb) + i) acc[mb][nb][i] += add;
          }
        }
      }
      if constexpr (sizeof(T) == 2 && C::BN == 64)
        if (j.stack) {
          if (n0 + an(nb) >= j.stack) continue;
          f32x4 rest[C::MB];
#pragma unroll
          for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
              const uint32_t w = chunk::pk2(acc[mb][nb][i], acc[mb][nb][i + 1]);
              rest[mb][i] = acc[mb][nb][i] - chunk::lo_f(w);
              rest[mb][i + 1] = acc[mb][nb][i + 1] - chunk::hi_f(w);
            }
#pragma unroll
          for (int mb = 0; mb < C::MB; mb += 2)
            put_blocks<T>(static_cast<T*>(j.d) + int64_t(n + j.stack) * j.ldd, m0 + am(mb), g4, j.m_tiles * BM, rest[mb],
                          rest[mb + 1]);
        }
#pragma unroll
      for (int mb = 0; mb < C::MB; mb += 2)
        put_blocks<T>(static_cast<T*>(j.d) + int64_t(n) * j.ldd, m0 + am(mb), g4, j.m_tiles * BM, acc[mb][nb], acc[mb + 1][nb]);
    }
  } else {
#pragma unroll
    for (int nb = 0; nb < C::NB; ++nb) {
      const int n = nw + an(nb);
      if (n >= j.n) continue;
#pragma unroll
      for (int mb = 0; mb < C::MB; mb += 2) {
        f32x4 x[2] = {acc[mb][nb], acc[mb + 1][nb]};
        const int64_t row = int64_t(n) * j.m;
        if (j.add)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int m = mw + am(mb + i);
            if (m < j.m) x[i] += *reinterpret_cast<const f32x4*>(j.add + row + m);
          }
        if (j.out) put_blocks<T>(static_cast<T*>(j.out) + row, m0 + am(mb), g4, j.m, x[0], x[1]);
        else put_blocks<float>(j.acc + split * j.acc_split + row, m0 + am(mb), g4, j.m, x[0], x[1]);
      }
    }
  }
}

// The sums of splits (and of `add`), to fp32 or the gradient itself; quads of
// elements, n of them.
template <typename T>
__global__ __launch_bounds__(256) void split_sum_kernel(const float* part, int64_t acc_split, int splits,
                                                        const float* add, float* acc, void* out, int64_t quads) {
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < quads; i += int64_t(gridDim.x) * 256) {
    float4 x = add ? reinterpret_cast<const float4*>(add)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      const float4 y = reinterpret_cast<const float4*>(part + s * acc_split)[i];
      x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
    }
    if (out) put4<T>(out, 4 * i, x.x, x.y, x.z, x.w);
    else reinterpret_cast<float4*>(acc)[i] = x;
  }
}

// A wave a row: joins the tiles' sums; log probabilities of the tokens behind it.
__global__ __launch_bounds__(256) void finish_kernel(LinearArgs a, const float4* part, int slots, const int4* found) {
  const int lane = threadIdx.x & 63;
  const int lr = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  if (lr >= a.n_rows) return;
  const int4 f = found[lr];
  const float c = a.inv_t * kLog2e;
  LinearSums z{kNegInf, 0.f, 0.f};
#pragma unroll 4
  for (int i = lane; i < slots; i += 64) {
    const float4 y = part[int64_t(lr) * slots + i];
    z = join(z, LinearSums{y.x, y.y, y.z}, c);
  }
#pragma unroll
  for (int o = 32; o; o >>= 1)
    z = join(z, LinearSums{__shfl_xor(z.m, o, 64), __shfl_xor(z.s, o, 64), __shfl_xor(z.t, o, 64)}, c);
  const bool empty = z.m == kNegInf && z.s == 0.f;  // every logit is -inf
  const float ls = __log2f(z.s);
  if (lane == 0) {
    float lse = fmaf(z.m, a.inv_t, ls * kLn2);  // held at the largest fp32 value; a NaN stays one
    lse = lse < -kFltMax ? -kFltMax : lse > kFltMax ? kFltMax : lse;
    a.lse[lr] = empty ? kNegInf : lse;
    a.entropy[lr] = empty ? 0.f : (ls - z.t / z.s) * kLn2;
    if (f.w & kRootStart) a.logp[a.first_row + lr] = 0.f;
  }
  // Halves, whose difference is in range.
  const auto logp = [&](float x) { return empty ? kNegInf : fmaf(0.5f * x - 0.5f * z.m, 2.f * a.inv_t, -(ls * kLn2)); };
  if (lane == 0 && f.w & kAny) a.logp[f.y] = f.w & kOutside ? 0.f : logp(__int_as_float(f.x));
  // The other children's first tokens: their logits wait in logp.
  if (f.w & kMore)
    for (int j = 1 + lane; j < a.kid_off[f.z + 1] - a.kid_off[f.z]; j += 64) {
      const int t = a.seg_off[a.kid[a.kid_off[f.z] + j]];
      a.logp[t] = token(a, t) < 0 ? 0.f : logp(a.logp[t]);
    }
}

// Products of 16 rows of the weight (this lane's: wrow) and 16 of hidden (hrow), as a
// tile's, bitwise.
template <typename T>
__device__ __forceinline__ f32x4 products16(const T* wrow, const T* hrow, int width) {
  constexpr int E16 = 16 / sizeof(T), P = 8 / E16;  // pieces of 16 bytes a lane has of 32 k
  constexpr int U = 4 / P;                          // 32 k each, loaded at once
  const int g8 = 8 * ((threadIdx.x & 63) >> 4);
  f32x4 x = {0.f, 0.f, 0.f, 0.f}, rest = x;
  for (int k0 = 0; k0 < width; k0 += 32 * U) {
    uint4 w[U][P], h[U][P];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int k = k0 + 32 * u + g8 + E16 * p;
        const bool in = k < width;  // zeros past the end
        w[u][p] = in ? *reinterpret_cast<const uint4*>(wrow + k) : make_uint4(0, 0, 0, 0);
        h[u][p] = in ? *reinterpret_cast<const uint4*>(hrow + k) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + 32 * u >= width) break;
      if constexpr (sizeof(T) == 2) {
        x = product::mma(w[u][0], h[u][0], x);
      } else {
        const product::Split ws = product::split3(w[u]), hs = product::split3(h[u]);
        rest = product::mma_rest(ws, hs, rest);
        x = product::mma(ws.part(0), hs.part(0), x);
      }
    }
  }
  return x + rest;
}

// The largest of some products, and the sum of exp2((x - m) c).
__device__ __forceinline__ float2 join(const float2 a, const float2 b, float c) {
  const float m = fmaxf(a.x, b.x);
  if (m == kNegInf) return make_float2(m, 0.f);
  return make_float2(m, a.y * ex2((a.x - m) * c) + b.y * ex2((b.x - m) * c));
}

// A wave a row: the coefficients of its gradient; and, with `stack`, the row's hidden
// states (bf16; zeros past the last row) at rows lr and stack + lr of hidden2.
//
// Where |lse| is kFarLse or more, its rounding would show in the probabilities, up to
// infinity (rows whose logits are masked throughout by large finite numbers).  A
// work-group with such a row finds the largest product and the sum of its 8 rows
// again, a wave 16 entries at a time: one work-group's pass over the weight (32000 x
// 2048 bf16 7 ms, 131072 x 2048 30, and 115 for 8192 such rows; 58 by 16 waves, but then
// calls without such a row, nearly all, take 1.5 us more; so registers are kept few too).
constexpr int kRowWaves = 8;
constexpr float kFarLse = 16384.f;
template <typename T>
__global__ __launch_bounds__(64 * kRowWaves, sizeof(T) == 2 ? 8 : 4) void row_kernel(LinearArgs a, float4* row, int4* ids, int stack,
                                                             uint4* hidden2) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = blockIdx.x * kRowWaves + wave;
  if (lr < stack) {
    const int n = a.width / 8;
    const uint4* from = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.hidden) + int64_t(lr) * a.ld);
#pragma unroll 4
    for (int i = lane; i < n; i += 64) {
      const uint4 x = lr < a.n_rows ? from[i] : make_uint4(0, 0, 0, 0);
      hidden2[lr * n + i] = x;
      hidden2[(stack + lr) * n + i] = x;
    }
  }
  const float lse = lr < a.n_rows ? a.lse_in[lr] : 0.f;
  const bool far = fabsf(lse) >= kFarLse && fabsf(lse) <= kFltMax;
  if (lr < a.n_rows) {
    const Behind b(a, a.first_row + lr, lane);
    float g = 0.f, g0 = 0.f;
    int id0 = -1;
    for (int j = lane; j < b.n; j += 64) {
      const int t = b.at(j), id = token(a, t);
      const float gj = id < 0 ? 0.f : a.dlogp[t];
      g += gj;
      if (j == 0) {
        g0 = gj;
        id0 = id;
      }
    }
    g = wave_sum(g);
    if (lane == 0) {
      const float dh = a.dentropy ? a.dentropy[lr] : 0.f;
      row[lr] = make_float4(lse, -(g + (a.dentropy ? dh * a.entropy_in[lr] : 0.f)) * a.inv_t, -dh * a.inv_t,
                            g0 * a.inv_t);
      ids[lr] = make_int4(id0, b.n, b.kid ? static_cast<int>(b.kid - a.kid) : -1, 0);
    }
  }
  if (!__syncthreads_or(far)) return;

  __shared__ float2 sums[kRowWaves][16];
  const int i = lane & 15, g4 = lane >> 4;
  const float c = a.inv_t * kLog2e;
  const T* hrow = static_cast<const T*>(a.hidden) +
                  int64_t(min(static_cast<int>(blockIdx.x) * kRowWaves + i, a.n_rows - 1)) * a.ld;
  float2 z = make_float2(kNegInf, 0.f);
  for (int v0 = 16 * wave; v0 < a.vocab; v0 += 16 * kRowWaves) {
    const T* wrow = static_cast<const T*>(a.weight) + int64_t(min(v0 + i, a.vocab - 1)) * a.width;
    const f32x4 x = products16<T>(wrow, hrow, a.width);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (v0 + 4 * g4 + e < a.vocab) z = join(z, make_float2(x[e], 1.f), c);
  }
#pragma unroll
  for (int o = 16; o < 64; o += o) z = join(z, make_float2(__shfl_xor(z.x, o, 64), __shfl_xor(z.y, o, 64)), c);
  if (g4 == 0) sums[wave][i] = z;
  __syncthreads();
  if (!far) return;
  z = i < kRowWaves ? sums[i][wave] : make_float2(kNegInf, 0.f);
#pragma unroll
  for (int o = 1; o < 16; o += o) z = join(z, make_float2(__shfl_xor(z.x, o, 64), __shfl_xor(z.y, o, 64)), c);
  if (lane == 0) {
    row[lr].x = __log2f(z.y) * kLn2;
    ids[lr].w = __float_as_int(z.x);
  }
}

// ---- launches -----------------------------------------------------------------------
int32_t ceil_div(int64_t a, int64_t b) { return static_cast<int32_t>((a + b - 1) / b); }

// Work-groups of `waves` that look for tokens, a wave a row or segment.  A launch's
// work items are counted in 32 bits: past 2^16 work-groups a wave takes several.
int32_t find_groups(int32_t n_rows, int32_t n_seg, int32_t waves) {
  const int64_t groups = ceil_div(int64_t(n_rows) + n_seg, waves), most = 1 << 16;
  return static_cast<int32_t>(groups < most ? groups : most);
}

template <typename T, typename C, bool BIG, Use USE>
hipError_t launch_product(Job j, const LinearArgs& a, hipStream_t stream) {
  constexpr int BK = product::kStep / int(sizeof(T));
  j.m_tiles = ceil_div(j.m, C::BM);
  j.n_tiles = ceil_div(j.n, C::BN);
  if (j.splits <= 1) {
    j.splits = 1;
    j.k_split = j.k;
  } else {
    j.k_split = ceil_div(ceil_div(j.k, j.splits), BK) * BK;
    j.splits = ceil_div(j.k, j.k_split);
  }
  // 8 x 4 tiles run on an XCD's 32 CUs at a time: operands of 12 tiles for 32 products.
  j.band = j.n_tiles < 4 ? j.n_tiles : 4;
  int64_t groups = int64_t(j.m_tiles) * j.n_tiles * j.splits;
  if (USE == kStats) groups += find_groups(j.n, a.n_seg, C::THREADS / 64);
  product_kernel<T, C, BIG, USE><<<static_cast<uint32_t>(groups), C::THREADS, 0, stream>>>(j, a);
  return hipGetLastError();
}

// By the tile sizes of `size`: 0: 64 x 64, of a sum product 128 x 64, 1: 128 x
// 128, 2 (bf16): 256 x 256.
template <typename T, bool TA, bool TB, Use USE>
hipError_t launch_sized(int size, const Job& j, const LinearArgs& a, hipStream_t stream) {
  using product::Tile;
  if constexpr (sizeof(T) == 2)
    if (size == 2) return launch_product<T, product::Big<TA, TB>, true, USE>(j, a, stream);
  if constexpr (!TA) {
    if (size == 0) return launch_product<T, Tile<T, TA, TB, 64, 64, 2, 2, 5>, false, USE>(j, a, stream);
  } else if constexpr (!TB) {
    if (size == 0) return launch_product<T, Tile<T, TA, TB, 128, 64, 4, 1, 3>, false, USE>(j, a, stream);
  }
  return launch_product<T, Tile<T, TA, TB, 128, 128, 2, 2, 2>, false, USE>(j, a, stream);
}

template <typename T>
hipError_t forward(const LinearArgs& a, const LinearWork& w, hipStream_t stream) {
  for (int64_t r0 = 0; r0 < a.n_rows; r0 += w.rows) {
    LinearArgs b = a;
    b.n_rows = static_cast<int32_t>(a.n_rows - r0 < w.rows ? a.n_rows - r0 : w.rows);
    b.first_row = static_cast<int32_t>(a.first_row + r0);
    b.hidden = static_cast<const char*>(a.hidden) + r0 * a.ld * sizeof(T);
    b.entropy = a.entropy + r0;
    b.lse = a.lse + r0;
    Job j{};
    j.a = static_cast<const char*>(a.weight);
    j.b = static_cast<const char*>(b.hidden);
    j.lda = int64_t(a.width) * sizeof(T);
    j.ldb = a.ld * sizeof(T);
    j.m = a.vocab;
    j.n = b.n_rows;
    j.k = a.width;
    j.c = a.inv_t * kLog2e;
    j.part = static_cast<float4*>(a.ws);
    j.found = reinterpret_cast<int4*>(static_cast<char*>(a.ws) + w.ids);
    hipError_t e = launch_sized<T, false, false, kStats>(w.size, j, b, stream);
    if (e != hipSuccess) return e;
    const int slots = ceil_div(a.vocab, w.size == 2 ? 256 : w.size == 1 ? 128 : 64);
    finish_kernel<<<ceil_div(b.n_rows, 4), 256, 0, stream>>>(b, j.part, slots, j.found);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// out (or acc) = add + the product, over splits where there are several; with `stack`,
// rows n and stack + n of it are added up for the n_rows first.
template <typename T, bool TB>
hipError_t sum_product(int size, int splits, float* parts, int stack, Job j, float* acc, const float* add, void* out,
                       const LinearArgs& a, hipStream_t stream) {
  j.splits = splits;
  if (splits <= 1 && !stack) {
    j.acc = acc;
    j.add = add;
    j.out = out;
    return launch_sized<T, true, TB, kSum>(size, j, a, stream);
  }
  j.acc = parts;
  j.acc_split = int64_t(j.m) * j.n;
  hipError_t e = launch_sized<T, true, TB, kSum>(size, j, a, stream);
  if (e != hipSuccess) return e;
  constexpr int BK = product::kStep / int(sizeof(T));
  const int k_split = ceil_div(ceil_div(j.k, splits), BK) * BK;
  const int64_t each = stack ? int64_t(stack) * j.m : j.acc_split;
  const int64_t quads = (stack ? int64_t(a.n_rows) * j.m : each) / 4;
  const int64_t groups = (quads + 255) / 256;
  split_sum_kernel<T><<<static_cast<uint32_t>(groups < 8192 ? groups : 8192), 256, 0, stream>>>(
      parts, each, ceil_div(j.k, k_split) * static_cast<int>(j.acc_split / each), add, acc, out, quads);
  return hipGetLastError();
}

template <typename T>
hipError_t backward(const LinearArgs& a, const LinearWork& w, hipStream_t stream) {
  char* base = static_cast<char*>(a.ws);
  float4* row = reinterpret_cast<float4*>(base);
  int4* ids = reinterpret_cast<int4*>(base + w.ids);
  float* dh = reinterpret_cast<float*>(base + w.dhidden);
  float* dw = reinterpret_cast<float*>(base + w.dweight);
  uint4* hidden2 = reinterpret_cast<uint4*>(base + w.hidden2);
  float* parts = reinterpret_cast<float*>(base + w.parts);
  const int64_t es = sizeof(T);
  for (int64_t r0 = 0; r0 < a.n_rows; r0 += w.rows) {
    LinearArgs b = a;
    b.n_rows = static_cast<int32_t>(a.n_rows - r0 < w.rows ? a.n_rows - r0 : w.rows);
    b.first_row = static_cast<int32_t>(a.first_row + r0);
    b.hidden = static_cast<const char*>(a.hidden) + r0 * a.ld * es;
    b.lse_in = a.lse_in + r0;
    b.entropy_in = a.entropy_in ? a.entropy_in + r0 : nullptr;
    b.dentropy = a.dentropy ? a.dentropy + r0 : nullptr;
    row_kernel<T><<<ceil_div(w.stack ? w.stack : b.n_rows, kRowWaves), 64 * kRowWaves, 0, stream>>>(b, row, ids, w.stack,
                                                                                                  hidden2);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const bool first_rows = r0 == 0, last_rows = r0 + w.rows >= a.n_rows;
    for (int64_t v0 = 0; v0 < a.vocab; v0 += w.piece) {
      const int32_t nv = static_cast<int32_t>(a.vocab - v0 < w.piece ? a.vocab - v0 : w.piece);
      const bool first = v0 == 0, last = v0 + w.piece >= a.vocab;
      const char* weight = static_cast<const char*>(a.weight) + v0 * a.width * es;
      Job j{};  // D of this piece
      j.a = weight;
      j.b = static_cast<const char*>(b.hidden);
      j.lda = a.width * es;
      j.ldb = a.ld * es;
      j.m = nv;
      j.n = b.n_rows;
      j.k = a.width;
      j.row = row;
      j.ids = ids;
      j.inv_t = a.inv_t;
      j.v0 = static_cast<int32_t>(v0);
      j.d = base + w.d;
      j.ldd = w.ldd;
      j.stack = w.stack;
      e = launch_sized<T, false, false, kGrad>(w.size, j, b, stream);
      if (e != hipSuccess) return e;
      j = Job{};  // dhidden [rows, width] += D weight
      j.a = weight;
      j.b = base + w.d;
      j.lda = a.width * es;
      j.ldb = w.ldd * es;
      j.m = a.width;
      j.n = w.stack ? 2 * w.stack : b.n_rows;
      j.k = nv;
      e = sum_product<T, false>(w.size_h, w.splits_h, parts, w.stack, j, dh, first ? nullptr : dh,
                                last ? static_cast<char*>(a.dhidden) + r0 * a.width * es : nullptr, b, stream);
      if (e != hipSuccess) return e;
      j.a = w.stack ? base + w.hidden2 : static_cast<const char*>(b.hidden);  // dweight [nv, width] += D^T hidden
      j.lda = (w.stack ? a.width : a.ld) * es;
      j.k = j.n;
      j.n = nv;
      float* acc = dw + v0 * a.width;
      e = sum_product<T, true>(w.size_w, w.splits_w, parts, 0, j, acc, first_rows ? nullptr : acc,
                               last_rows ? static_cast<char*>(a.dweight) + v0 * a.width * es : nullptr, b, stream);
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_linear(const LinearArgs& a, const LinearWork& w, int dtype, hipStream_t stream) {
  return dtype == TREE_DTYPE_BF16 ? forward<uint16_t>(a, w, stream) : forward<float>(a, w, stream);
}

hipError_t launch_linear_backward(const LinearArgs& a, const LinearWork& w, int dtype, hipStream_t stream) {
  return dtype == TREE_DTYPE_BF16 ? backward<uint16_t>(a, w, stream) : backward<float>(a, w, stream);
}

}  // namespace tg
