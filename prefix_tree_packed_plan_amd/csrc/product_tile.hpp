// One tile of a matrix product out[n][m] = sum_k A[m][k] B[n][k] (gfx950), bf16
// or fp32, in the accumulators of a work-group's waves.
//
// Either operand is stored with k contiguous (rows m or n) or, TR, with m or n
// contiguous (rows k), so that one kernel serves a product and both of its
// gradients without a transposed copy of anything.  A k-step of 128 bytes (64
// bf16, 32 fp32) of both goes to LDS by DMA, S steps in a ring; waves read
// their 16x16x32 MFMA fragments from there, rows by 16-byte reads, TR tiles by
// the transposing read (bf16) or by words (fp32).
//
// A wave owns MB x NB blocks of 16 x 16.  Lane l of a block holds column n = l %
// 16 and rows m = 4 (l / 16) + i of register i: four neighbouring m of one n,
// which is 8 or 16 bytes of a row of `out`; pair_up() makes it 16 for bf16.
//
// fp32: a value is the sum of three bf16 (its first 8 bits, the rest rounded, the rest of
// that, which is exact; the second is below 2^-7 of it, the third up to 2^-16), and a
// product of two the six largest of the nine partial products; those left out are up to
// 2^-22 of it, 2^-24 in the mean.  Six bf16 MFMA do 2.7 times the work of fp32 MFMA in
// the same time.  (First parts rounded to the nearest leave out a quarter of that, which
// does not show in a gradient's error, but round the largest fp32 numbers, the usual
// masks, to infinity; held in range they cost 5% of the time.)
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>
#include <utility>

#include "chunk_mfma.hpp"

namespace tg {
namespace product {

using chunk::bf16x8;
using chunk::pk2;

using chunk::f32x4;
typedef __attribute__((address_space(3))) const chunk::u32x4 lds_u4;
typedef __attribute__((address_space(3))) const uint32_t lds_u1;

constexpr int kStep = 128;  // bytes of a k-step of a row

// What is read past the last k: zeros.
static __device__ const uint4 kZeros = {0, 0, 0, 0};

__device__ __forceinline__ uint4 lds16(const char* p) {
  const chunk::u32x4 w = *(lds_u4*)p;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 bytes a lane to LDS at lds + IMM + 16 lane, from src + off (src the same for
// all lanes) or from a lane's own address.  In inline asm, because the compiler
// would otherwise wait for all DMA in flight before any read of LDS; it has no
// output registers, and wait_step() is the wait.  Nothing else here needs m0 (LDS
// instructions of gfx9 on do not), so it is not put back.
template <int IMM>
__device__ __forceinline__ void dma16(uint64_t src, uint32_t off, uint32_t lds) {
  asm volatile("s_add_u32 m0, %0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %3"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "i"(IMM), "v"(off), "s"(src)
               : "memory", "m0", "scc");
}
__device__ __forceinline__ void dma16(const void* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(src)
               : "memory", "m0");
}
__device__ __forceinline__ uint32_t lds_at(const char* lds) {
  return __builtin_amdgcn_readfirstlane(
      static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) void*)lds)));
}

// An operand of R rows (m or n) a tile, staged by W waves.
template <typename T, bool TR, int R, int W>
struct Operand {
  static constexpr int ES = sizeof(T);
  static constexpr int BK = kStep / ES;          // k of a step
  static constexpr int E16 = 16 / ES;            // elements of 16 bytes
  static constexpr int RB = TR ? R * ES : kStep; // bytes of a row in LDS
  static constexpr int BYTES = R * kStep;
  static constexpr int NI = BYTES / 1024 / W;    // DMA instructions of a wave
  static_assert(NI * 1024 * W == BYTES, "whole DMA instructions");
  static_assert(!TR || RB >= 256, "transposing reads spread 4 rows over 256 bytes");

  uint64_t src;      // the tile's first row at this step
  int64_t ld;        // bytes between stored rows
  uint32_t off[NI];  // this lane's pieces
  int wave, lane;

  // The 16-byte piece c of row r sits at slot c ^ swz(r): operand reads (16 rows,
  // one piece each), transposing reads (4 rows x 64 bytes) and reads by words (4
  // rows 8 apart x 64 bytes) then touch every bank once.
  static __device__ __forceinline__ int swz(int r) {
    if (!TR) return 4 * ((r >> 1) & 1) + ((r >> 2) & 3);
    return ES == 2 ? 4 * (r & 3) + ((r >> 2) & 3) : 4 * ((r >> 3) & 3);
  }
  __device__ __forceinline__ static int slot_row(int q, int lane) { return (q * 1024 + lane * 16) / RB; }
  __device__ __forceinline__ static int slot_chunk(int q, int lane) {
    const int at = q * 1024 + lane * 16;
    return ((at % RB) / 16) ^ swz(at / RB);
  }
  // `rows` (m or n) of `base` are left from the tile's first on; those past
  // them repeat one of them (their results are not used).
  __device__ __forceinline__ void init(const char* base, int64_t ld_, int64_t first, int64_t rows, int64_t k0, int wave_,
                                       int lane_) {
    ld = ld_;
    wave = wave_;
    lane = lane_;
    src = reinterpret_cast<uint64_t>(base) + (TR ? k0 * ld + first * ES : first * ld + k0 * ES);
    const int most = static_cast<int>(rows < R ? rows : R);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int q = wave + W * i, r = slot_row(q, lane), c = slot_chunk(q, lane);
      if (TR) off[i] = static_cast<uint32_t>(r * ld) + 16u * (c * E16 < most ? c : 0);
      else off[i] = static_cast<uint32_t>(min(r, most - 1) * ld) + 16u * c;
    }
  }
  // The I-th DMA instruction of a whole step.  `lds` is where this wave's first one
  // goes.
  template <int I>
  __device__ __forceinline__ void issue(uint32_t lds) {
    if constexpr (I < NI) dma16<I * W * 1024>(src, off[I], lds);
  }
  template <int I = 0>
  __device__ __forceinline__ void issue_all(uint32_t lds) {
    if constexpr (I < NI) {
      issue<I>(lds);
      issue_all<I + 1>(lds);
    }
  }
  __device__ __forceinline__ void advance() { src += TR ? BK * ld : kStep; }
  // Starts the DMA of a step of `k` valid k, and moves on.
  __device__ __forceinline__ void stage(uint32_t lds, int k) {
    if (k >= BK) {
      issue_all(lds);
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int q = wave + W * i, r = slot_row(q, lane), c = slot_chunk(q, lane);
        const char* p = reinterpret_cast<const char*>(src + off[i]);
        // Rows k past the end repeat the last (the other operand is zero there).
        if (TR) p -= r >= k ? static_cast<int64_t>(r - (k - 1)) * ld : 0;
        else if (c * E16 >= k) p = reinterpret_cast<const char*>(&kZeros);
        dma16(p, lds + W * i * 1024);
      }
    }
    advance();
  }
};

// Fragment reads of blocks of 16 rows (m or n) from block `blk0` on, 32 k each: lane l
// has row l % 16 and k = 8 (l / 16) .. + 7.
template <typename T, bool TR, int R>
struct Reader {
  static constexpr int ES = sizeof(T);
  static constexpr int RB = TR ? R * ES : kStep;
  int base;
  __device__ __forceinline__ Reader(int blk0, int lane) {
    const int i = lane & 15, g = lane >> 4;
    if (!TR) {
      const int sw = 4 * ((i >> 1) & 1) + ((i >> 2) & 3);
      base = (16 * blk0 + i) * RB + 16 * ((ES == 2 ? g : 2 * g) ^ sw);
    } else if (ES == 2) {
      const int sw = 4 * (i >> 2) + ((2 * g) & 3);
      base = (8 * g + (i >> 2)) * RB + 16 * ((2 * blk0 + ((i & 3) >> 1)) ^ sw) + 8 * (i & 1);
    } else {
      base = 8 * g * RB + 16 * ((4 * blk0 + (i >> 2)) ^ (4 * g)) + 4 * (i & 3);
    }
  }
  // bf16: the fragment of block b (a multiple of its count below blk0), k from 32 ks on.
  __device__ __forceinline__ uint4 bf16(const char* t, int b, int ks) const {
    if constexpr (!TR) {
      return lds16(t + ((base ^ (64 * ks)) + b * 16 * RB));
    } else {
      const int o = (base ^ (32 * b)) + 32 * ks * RB;
      const int o4 = (base ^ (32 * b) ^ 16) + (32 * ks + 4) * RB;
      return chunk::cat(chunk::tile_tr(t, o), chunk::tile_tr(t, o4));
    }
  }
  // fp32: its 8 values.
  __device__ __forceinline__ void f32(const char* t, int b, float (&x)[8]) const {
    if constexpr (!TR) {
      const int o = base + b * 16 * RB;
      const uint4 lo = lds16(t + o), hi = lds16(t + (o ^ 16));
      x[0] = __uint_as_float(lo.x), x[1] = __uint_as_float(lo.y), x[2] = __uint_as_float(lo.z),
      x[3] = __uint_as_float(lo.w);
      x[4] = __uint_as_float(hi.x), x[5] = __uint_as_float(hi.y), x[6] = __uint_as_float(hi.z),
      x[7] = __uint_as_float(hi.w);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(*(lds_u1*)(t + ((base ^ (64 * b)) + e * RB)));
    }
  }
};

// Three bf16 whose sum is x, of 8 values; pair j of them.
struct Split {
  uint32_t w[3][4];
  __device__ __forceinline__ uint4 part(int q) const { return make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]); }
};
__device__ __forceinline__ void split_pair(Split& s, int j, float a, float b) {
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    s.w[q][j] = q ? pk2(a, b) : __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302);
    a -= chunk::lo_f(s.w[q][j]);
    b -= chunk::hi_f(s.w[q][j]);
  }
}
__device__ __forceinline__ Split split3(const float (&x)[8]) {
  Split s;
#pragma unroll
  for (int j = 0; j < 4; ++j) split_pair(s, j, x[2 * j], x[2 * j + 1]);
  return s;
}

__device__ __forceinline__ Split split3(const uint4 (&w)[2]) {
  const float x[8] = {__uint_as_float(w[0].x), __uint_as_float(w[0].y), __uint_as_float(w[0].z), __uint_as_float(w[0].w),
                      __uint_as_float(w[1].x), __uint_as_float(w[1].y), __uint_as_float(w[1].z), __uint_as_float(w[1].w)};
  return split3(x);
}

__device__ __forceinline__ f32x4 mma(const uint4 a, const uint4 b, const f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}
// The five smaller ones of the six largest partial products, the smallest first.
__device__ __forceinline__ f32x4 mma_rest(const Split& a, const Split& b, f32x4 c) {
  c = mma(a.part(1), b.part(1), c);
  c = mma(a.part(2), b.part(0), c);
  c = mma(a.part(0), b.part(2), c);
  c = mma(a.part(1), b.part(0), c);
  return mma(a.part(0), b.part(1), c);
}

// Blocks x and y, y behind x along m, as 8 neighbouring bf16 a lane: of block x (lanes of
// even l / 16) or y, from its row 8 (l / 32) on.
__device__ __forceinline__ uint4 pair_up(const f32x4 x, const f32x4 y) {
  // Swaps the odd 16 lanes of the first with the even ones of the second.
  const auto lo = __builtin_amdgcn_permlane16_swap(pk2(x[0], x[1]), pk2(y[0], y[1]), false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap(pk2(x[2], x[3]), pk2(y[2], y[3]), false, false);
  return make_uint4(lo[0], hi[0], lo[1], hi[1]);
}

// Waits until all but the youngest N of this wave's loads have landed, and its
// reads of LDS have ended.
template <int N>
__device__ __forceinline__ void wait_step() {
  // vmcnt bits 3:0 and 15:14, expcnt 6:4 (no wait), lgkmcnt 11:8 (0).
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x70);
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Sizes of a work-group's tile: BM x BN by WM x WN waves, S steps in the ring.
template <typename T_, bool TA, bool TB, int BM_, int BN_, int WM_, int WN_, int S_>
struct Tile {
  using T = T_;
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, S = S_, W = WM * WN;
  static constexpr int MB = BM / WM / 16, NB = BN / WN / 16;
  static constexpr int THREADS = 64 * W, OCC = 2;
  static constexpr int BK = kStep / int(sizeof(T));
  static constexpr int KS = BK / 32;  // fragments along a step
  // B stored by k: rows of zeros follow its last, up to a whole step (A's repeat
  // its last there).
  static constexpr bool B_PADDED = TB, A_BY_K = TA;
  using OpA = Operand<T, TA, BM, W>;
  using OpB = Operand<T, TB, BN, W>;
  using RdA = Reader<T, TA, BM>;
  using RdB = Reader<T, TB, BN>;
  static constexpr int STEP = OpA::BYTES + OpB::BYTES;
  static constexpr int LDS = S * STEP;
  static constexpr int LOADS = OpA::NI + OpB::NI;
};

// f(std::integral_constant<int, 0>) .. f(.. N - 1).
template <typename F, int... I>
__device__ __forceinline__ void unrolled_(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void unrolled(F f) {
  unrolled_(f, std::make_integer_sequence<int, N>{});
}
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

// When the next fragments are read: the MFMA (of MB x NB, all n of an m one after
// another) behind which the i-th is, and which it is: b[n] as n, a[m] as NB + m.
// b[0], a[0], the other b, the other a; a[m] is read over the one in use, so not before
// its last MFMA; and none before `START`.
template <int MB, int NB>
struct Order {
  static constexpr int N = MB + NB, START = MB * NB / 4;
  int at[N] = {}, what[N] = {};
  constexpr Order() {
    int s = START - 1;
    for (int i = 0; i < N; ++i) {
      what[i] = i == 0 ? 0 : i == 1 ? NB : i <= NB ? i - 1 : i;
      const int m = what[i] - NB, free = m < 0 ? 0 : NB * (m + 1) - 1;
      s = s + 1 > free ? s + 1 : free;
      if (s > MB * NB - 1) s = MB * NB - 1;
      at[i] = s;
    }
  }
};

// acc = the tile's products over the k (>= 1) elements from where A and B stand.
//
// bf16: while the matrix units work on the fragments of 32 k, the next ones' reads
// are issued between the MFMAs, across the barrier into the next k-step too; fences
// keep that order.  The barrier stands a quarter into the last fragments of a
// k-step: by then those have been read, so the step's place in the ring can be
// staged anew, and the next k-step has had S - 1 steps' time to land.
template <typename C>
__device__ __forceinline__ void run(f32x4 (&acc)[C::MB][C::NB], typename C::OpA& A, typename C::OpB& B,
                                    const typename C::RdA& ra, const typename C::RdB& rb, int k, char* lds) {
  using T = typename C::T;
  constexpr int MB = C::MB, NB = C::NB, KS = C::KS, S = C::S;
  const uint32_t at = lds_at(lds) + A.wave * 1024;
  const int steps = (k + C::BK - 1) / C::BK;
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n) acc[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  const auto stage = [&](int t, int buf) {
    A.stage(at + buf * C::STEP, k - t * C::BK);
    B.stage(at + buf * C::STEP + C::OpA::BYTES, C::B_PADDED ? C::BK : k - t * C::BK);
  };
  if constexpr (sizeof(T) == 2) {
    constexpr Order<MB, NB> order;
    static_assert(KS % 2 == 0, "b alternates");
#pragma unroll
    for (int t = 0; t < S; ++t)
      if (t < steps) stage(t, t);
    if (steps >= S) wait_step<C::LOADS * (S - 1)>();
    else wait_step<0>();
    barrier();
    uint4 a[MB], b[2][NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) b[0][n] = rb.bf16(lds + C::OpA::BYTES, n, 0);
#pragma unroll
    for (int m = 0; m < MB; ++m) a[m] = ra.bf16(lds, m, 0);
    int cur = 0;
    for (int t = 0; t < steps; ++t) {
      const int next = cur + 1 == S ? 0 : cur + 1;
      const uint32_t into = at + cur * C::STEP;
      unrolled<KS>([&](auto ks_) {
        constexpr int ks = decltype(ks_)::value;
        constexpr bool turn = ks == KS - 1;
        const char* ta = lds + (turn ? next : cur) * C::STEP;
        const char* tb = ta + C::OpA::BYTES;
        bool whole = false;
        unrolled<MB * NB>([&](auto slot) {
          constexpr int i = decltype(slot)::value;
          acc[i / NB][i % NB] = mma(a[i / NB], b[ks & 1][i % NB], acc[i / NB][i % NB]);
          if constexpr (turn && i == order.START - 1) {
            // Step t + 1 has landed for every wave, and step t has been read by every wave.
            if (t + S <= steps) wait_step<C::LOADS * (S - 2)>();
            else wait_step<0>();
            barrier();
            whole = k - (t + S) * C::BK >= C::BK;
            if (!whole && t + S < steps) stage(t + S, cur);
          }
#pragma unroll
          for (int j = 0; j < order.N; ++j)
            if (order.at[j] == i) {
              const int w = order.what[j];
              if (w < NB) b[(ks + 1) & 1][w] = rb.bf16(tb, w, (ks + 1) % KS);
              else a[w - NB] = ra.bf16(ta, w - NB, (ks + 1) % KS);
            }
          if constexpr (turn && i >= order.START) {
            constexpr int SLOTS = MB * NB - order.START, D = (C::LOADS + SLOTS - 1) / SLOTS;
            if (whole)
              unrolled<D>([&](auto d) {
                constexpr int q = (i - order.START) * D + decltype(d)::value;
                if constexpr (q < C::OpA::NI) A.template issue<q>(into);
                else if constexpr (q < C::LOADS) B.template issue<q - C::OpA::NI>(into + C::OpA::BYTES);
              });
          }
          fence();
        });
        if (turn && whole) {
          A.advance();
          B.advance();
        }
      });
      cur = next;
    }
  } else {
#pragma unroll
    for (int t = 0; t < S - 1; ++t)
      if (t < steps) stage(t, t);
    // Logits: the five smaller partial products, up to 2^-6 of the terms' sizes, are added
    // up by themselves, so that the sum is rounded once for 32 k instead of six times (the
    // largest error of an fp32 gradient is that of a probability near 1).
    constexpr bool APART = !C::B_PADDED && !C::A_BY_K;
    f32x4 rest[APART ? MB : 1][APART ? NB : 1] = {};
    int cur = 0, into = S - 1;
    for (int t = 0; t < steps; ++t) {
      // Step t has landed for every wave, and step t - 1 has been read by every wave.
      if (t + S - 1 <= steps) wait_step<C::LOADS * (S - 2)>();
      else wait_step<0>();
      barrier();
      if (t + S - 1 < steps) stage(t + S - 1, into);
      const char* ta = lds + cur * C::STEP;
      const char* tb = ta + C::OpA::BYTES;
      // All of the step's values are read first; those of the next a are split between the
      // MFMAs of the one before.
      float xa[MB][8], xb[NB][8];
#pragma unroll
      for (int n = 0; n < NB; ++n) rb.f32(tb, n, xb[n]);
#pragma unroll
      for (int m = 0; m < MB; ++m) ra.f32(ta, m, xa[m]);
      Split b[NB], a[2];
#pragma unroll
      for (int n = 0; n < NB; ++n) b[n] = split3(xb[n]);
      a[0] = split3(xa[0]);
      fence();
#pragma unroll
      for (int m = 0; m < MB; ++m) {
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          if constexpr (APART) rest[m][n] = mma_rest(a[m & 1], b[n], rest[m][n]);
          else acc[m][n] = mma_rest(a[m & 1], b[n], acc[m][n]);
          acc[m][n] = mma(a[m & 1].part(0), b[n].part(0), acc[m][n]);
          if (m + 1 < MB)
#pragma unroll
            for (int j = n * 4 / NB; j < (n + 1) * 4 / NB; ++j) split_pair(a[(m + 1) & 1], j, xa[m + 1][2 * j], xa[m + 1][2 * j + 1]);
          fence();
        }
      }
      cur = cur + 1 == S ? 0 : cur + 1;
      into = into + 1 == S ? 0 : into + 1;
    }
    if constexpr (APART)
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int n = 0; n < NB; ++n) acc[m][n] += rest[m][n];
  }
}

// A 256 x 256 tile of bf16 by 8 waves (2 along m), staged as four 128-row halves A0, A1,
// B0, B1 of a 128-byte k-step, two steps in LDS.  A wave has 64 rows of each A half and
// 32 of each B half, and takes the halves' products one after another: A0 B0, A0 B1,
// A1 B1, A1 B0.  So each half is read in one go (over the fragments just used), and
// its place in LDS is staged anew, two steps on, as soon as all waves have read it:
// a DMA has one and a half steps' time to land, and DMA is spread over the step,
// where staging whole steps (run()) gives one and a burst: 8192 x 131072 x 4096, 1350
// TFLOP/s against 1190 with whole steps of 256 x 256 tiles.  128 x 128 tiles, two a CU,
// read twice the bytes for a product: 1080.
template <bool TA, bool TB>
struct Big {
  using T = uint16_t;
  static constexpr bool TRA = TA, TRB = TB;
  static constexpr int W = 8, BM = 256, BN = 256, WM = 2, WN = 4, MB = 8, NB = 4, NH = NB / 2;
  static constexpr int THREADS = 64 * W, OCC = 2, BK = 64;
  using OpA = Operand<T, TA, 128, W>;
  using OpB = Operand<T, TB, 128, W>;
  using RdA = Reader<T, TA, 128>;
  using RdB = Reader<T, TB, 128>;
  static constexpr int HALF = OpA::BYTES, STEP = 4 * HALF, LDS = 2 * STEP;
  static constexpr int NI = OpA::NI;
  static_assert(NI == OpB::NI, "what is counted as in flight");
};

template <typename C>
__device__ __forceinline__ void run_big(f32x4 (&acc)[C::MB][C::NB], typename C::OpA (&A)[2], typename C::OpB (&B)[2],
                                        const typename C::RdA& ra, const typename C::RdB& rb, int k, char* lds) {
  constexpr int HALF = C::HALF, BK = C::BK, NI = C::NI, NH = C::NH;
  constexpr bool TB = C::TRB;
  const uint32_t at = lds_at(lds) + A[0].wave * 1024;
  const int steps = (k + BK - 1) / BK;
#pragma unroll
  for (int m = 0; m < C::MB; ++m)
#pragma unroll
    for (int n = 0; n < C::NB; ++n) acc[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  // Groups of halves of step t: A0, B0, B1; and A1.
  const auto stage0 = [&](int t) {
    const uint32_t to = at + (t & 1) * C::STEP;
    const int left = k - t * BK, left_b = TB ? BK : left;
    A[0].stage(to, left);
    B[0].stage(to + 2 * HALF, left_b);
    B[1].stage(to + 3 * HALF, left_b);
  };
  const auto stage1 = [&](int t) { A[1].stage(at + (t & 1) * C::STEP + HALF, k - t * BK); };
  stage0(0);
  stage1(0);
  if (steps > 1) {
    stage0(1);
    stage1(1);
    wait_step<5 * NI>();
  } else {
    wait_step<NI>();
  }
  barrier();
  uint4 a[2][4], b[2][2][NH];  // [ks][m], [half][ks][n]
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
    for (int m = 0; m < 4; ++m) a[ks][m] = ra.bf16(lds, m, ks);
#pragma unroll
    for (int n = 0; n < NH; ++n) b[0][ks][n] = rb.bf16(lds + 2 * HALF, n, ks);
  }
  constexpr int P = 8 * NH;                        // MFMA of a product of halves
  constexpr int Y = 2 * NH + 10, X = 2 * P + 12;   // behind which the barriers stand
  // The q-th DMA instruction of a step is behind MFMA D0 + EVERY q, the last ones in the
  // next turn of the loop: evenly spread, since a burst of them fills the queue to the
  // address units and then holds up the waves' MFMA too.
  constexpr int D0 = Y + 2, EVERY = P / NI, BEFORE_X = (X - D0 + EVERY - 1) / EVERY;
  static_assert(D0 + EVERY * (4 * NI - 1) - 4 * P < Y && D0 + EVERY * 3 * NI > X, "halves are staged once read");
  const auto issue = [&](auto index, uint32_t to) {
    constexpr int q = decltype(index)::value;
    if constexpr (q < NI) A[0].template issue<q>(to);
    else if constexpr (q < 2 * NI) B[0].template issue<q - NI>(to + 2 * HALF);
    else if constexpr (q < 3 * NI) B[1].template issue<q - 2 * NI>(to + 3 * HALF);
    else A[1].template issue<q - 3 * NI>(to + HALF);
  };
  bool whole = false, was_whole = false;
  for (int t = 0; t < steps; ++t) {
    const char* now = lds + (t & 1) * C::STEP;
    const char* next = lds + ((t + 1) & 1) * C::STEP;
    const uint32_t to = at + (t & 1) * C::STEP, was_to = at + ((t + 1) & 1) * C::STEP;
    was_whole = whole;
    whole = k - (t + 2) * BK >= BK;  // step t + 2 is there, and whole
    unrolled<4 * P>([&](auto slot) {
      constexpr int s = decltype(slot)::value;
      constexpr int p = s / P, ks = s % P / (4 * NH), m = s / NH % 4, n = s % NH;
      constexpr int ah = p >= 2, bh = p == 1 || p == 2;
      acc[4 * ah + m][NH * bh + n] = mma(a[ks][m], b[bh][ks][n], acc[4 * ah + m][NH * bh + n]);
      // Reads, each behind the last use of what it overwrites.
      if constexpr (s >= 2 && s < 2 + 2 * NH)
        b[1][(s - 2) / NH][(s - 2) % NH] = rb.bf16(now + 3 * HALF, (s - 2) % NH, (s - 2) / NH);
      if constexpr (p == 1 && n == NH - 1) a[ks][m] = ra.bf16(now + HALF, m, ks);
      if constexpr (p == 3 && n == NH - 1) a[ks][m] = ra.bf16(next, m, ks);
      if constexpr (p == 3 && m == 3) b[0][ks][n] = rb.bf16(next + 2 * HALF, n, ks);
      if constexpr (s == Y) {
        // A1 of this step has landed for every wave; every wave has read A0, B0 and B1.
        if (t + 1 < steps) wait_step<4 * NI>();
        else wait_step<0>();
        barrier();
        if (!whole && t + 2 < steps) stage0(t + 2);
      }
      if constexpr (s == X) {
        // A0, B0 and B1 of the next step have landed; every wave has read A1.
        if (t + 2 < steps) wait_step<NI + BEFORE_X>();
        else wait_step<0>();
        barrier();
        if (!whole && t + 2 < steps) stage1(t + 2);
      }
      constexpr int q = (s - D0) / EVERY, last = (s + 4 * P - D0) / EVERY;
      if constexpr (s >= D0 && (s - D0) % EVERY == 0 && q < 4 * NI) {
        if (whole) issue(std::integral_constant<int, q>{}, to);
      } else if constexpr (s < D0 && (s + 4 * P - D0) % EVERY == 0 && last < 4 * NI) {
        if (was_whole) {
          issue(std::integral_constant<int, last>{}, was_to);
          if constexpr (last == 4 * NI - 1) A[1].advance();
        }
      }
      fence();
    });
    if (whole) {
      A[0].advance();
      B[0].advance();
      B[1].advance();
    }
  }
}

// The tile that work-group `id` of `total` computes: neighbouring ids go to the 8
// XCDs in turn, and each XCD is given a contiguous share of the tiles, so that
// what its work-groups read together comes from its own L2.
__device__ __forceinline__ int of_xcd(int id, int total) {
  const int x = id & 7, q = total >> 3, rest = total & 7;
  return x * q + min(x, rest) + (id >> 3);
}

}  // namespace product
}  // namespace tg
