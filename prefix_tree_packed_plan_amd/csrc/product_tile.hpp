// One tile of a matrix product out[n][m] = sum_k A[m][k] B[n][k] (gfx950), bf16
// or fp32, in the accumulators of a work-group's waves.
//
// Either operand is stored with k contiguous (rows m or n) or, TR, with m or n
// contiguous (rows k), so that one kernel serves a product and both of its
// gradients without a transposed copy of anything.  A k-step of 128 bytes (64
// bf16, 32 fp32) of both goes to LDS by DMA, S steps in a ring; waves read
// their 32x32x16 MFMA fragments from there, rows by 16-byte reads, TR tiles by
// the transposing read (bf16) or by words (fp32).
//
// A wave owns MB x NB blocks of 32 x 32.  Lane l of a block holds column n = l %
// 32 and rows m = 8 (i / 4) + 4 (l / 32) + i % 4 of register i: four neighbouring
// m of one n, which is 8 or 16 bytes of a row of `out`.
//
// fp32: a value is the sum of three bf16 (rounded, the rest rounded, the rest of
// that: exact to 2^-26 of it), and a product of two the six largest of the nine
// partial products; those left out are below 2^-26 of it.  Six bf16 MFMA do 2.7
// times the work of fp32 MFMA in the same time.  Values within a factor of 2^-8
// of the largest fp32 may round to infinity.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "chunk_mfma.hpp"

namespace tg {
namespace product {

using chunk::bf16x8;
using chunk::pk2;

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) const chunk::u32x4 lds_u4;
typedef __attribute__((address_space(3))) const uint32_t lds_u1;

constexpr int kStep = 128;  // bytes of a k-step of a row

// What is read past the last k: zeros.
static __device__ const uint4 kZeros = {0, 0, 0, 0};

__device__ __forceinline__ uint4 lds16(const char* p) {
  const chunk::u32x4 w = *(lds_u4*)p;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 bytes a lane to LDS at lds + 16 lane, from src + off (src the same for all
// lanes) or from a lane's own address.  In inline asm, because the compiler
// would otherwise wait for all DMA in flight before any read of LDS; it has no
// output registers, and wait_step() is the wait.
__device__ __forceinline__ void dma16(uint64_t src, uint32_t off, uint32_t lds) {
  int m0;
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %3\n\ts_mov_b32 m0, %0"
               : "=&s"(m0)
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(src)
               : "memory");
}
__device__ __forceinline__ void dma16(const void* src, uint32_t lds) {
  int m0;
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, off\n\ts_mov_b32 m0, %0"
               : "=&s"(m0)
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(src)
               : "memory");
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

  // The 16-byte piece c of row r sits at slot c ^ swz(r): operand reads (32 rows,
  // one piece each) and transposing reads (4 rows x 64 bytes) then spread
  // evenly over the banks.
  static __device__ __forceinline__ int swz(int r) {
    if (!TR) return 4 * ((r >> 1) & 1) + ((r >> 2) & 3);
    return ES == 2 ? 4 * (r & 3) + ((r >> 2) & 3) : 8 * ((r >> 3) & 1);
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
  // Starts the DMA of a step of `k` (<= BK) valid k, and moves on.
  __device__ __forceinline__ void stage(uint32_t lds, int k) {
    if (k >= BK) {
#pragma unroll
      for (int i = 0; i < NI; ++i) dma16(src, off[i], lds + (wave + W * i) * 1024);
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int q = wave + W * i, r = slot_row(q, lane), c = slot_chunk(q, lane);
        const char* p = reinterpret_cast<const char*>(src + off[i]);
        // Rows k past the end repeat the last (the other operand is zero there).
        if (TR) p -= r >= k ? static_cast<int64_t>(r - (k - 1)) * ld : 0;
        else if (c * E16 >= k) p = reinterpret_cast<const char*>(&kZeros);
        dma16(p, lds + q * 1024);
      }
    }
    src += TR ? BK * ld : kStep;
  }
};

// Fragment reads of `NBLK` blocks of 32 rows from block `blk0` on.
template <typename T, bool TR, int R>
struct Reader {
  static constexpr int ES = sizeof(T);
  static constexpr int RB = TR ? R * ES : kStep;
  int base;
  __device__ __forceinline__ Reader(int blk0, int lane) {
    const int r = lane & 31, h = lane >> 5, i = lane & 15;
    if (!TR) {
      const int sw = 4 * ((r >> 1) & 1) + ((r >> 2) & 3);
      base = (32 * blk0 + r) * RB + 16 * ((ES == 2 ? h : 2 * h) ^ sw);
    } else if (ES == 2) {
      const int sw = 4 * (i >> 2) + 2 * h;
      base = (8 * h + (i >> 2)) * RB + 16 * ((4 * blk0 + 2 * ((lane >> 4) & 1) + ((i & 3) >> 1)) ^ sw) + 8 * (i & 1);
    } else {
      base = 8 * h * RB + 16 * ((8 * blk0 + (r >> 2)) ^ (8 * h)) + 4 * (r & 3);
    }
  }
  // bf16: fragment of 16 k from 16 ks on, block b.
  __device__ __forceinline__ uint4 bf16(const char* t, int b, int ks) const {
    if constexpr (!TR) {
      return lds16(t + ((base ^ (32 * ks)) + b * 32 * RB));
    } else {
      const int o = (base ^ (64 * b)) + 16 * ks * RB;
      const int o4 = (base ^ (64 * b) ^ 16) + (16 * ks + 4) * RB;
      return chunk::cat(chunk::tile_tr(t, o), chunk::tile_tr(t, o4));
    }
  }
  // fp32: its 8 values.
  __device__ __forceinline__ void f32(const char* t, int b, int ks, float (&x)[8]) const {
    if constexpr (!TR) {
      const int o = (base ^ (64 * ks)) + b * 32 * RB;
      const uint4 lo = lds16(t + o), hi = lds16(t + (o ^ 16));
      x[0] = __uint_as_float(lo.x), x[1] = __uint_as_float(lo.y), x[2] = __uint_as_float(lo.z),
      x[3] = __uint_as_float(lo.w);
      x[4] = __uint_as_float(hi.x), x[5] = __uint_as_float(hi.y), x[6] = __uint_as_float(hi.z),
      x[7] = __uint_as_float(hi.w);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = __uint_as_float(*(lds_u1*)(t + ((base ^ (128 * b)) + (16 * ks + e) * RB)));
    }
  }
};

// Three bf16 whose sum is x, of 8 values.
struct Split {
  uint4 p[3];
};
__device__ __forceinline__ Split split3(const float (&x)[8]) {
  Split s;
  uint32_t w[3][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a = x[2 * j], b = x[2 * j + 1];
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      w[q][j] = pk2(a, b);
      a -= chunk::lo_f(w[q][j]);
      b -= chunk::hi_f(w[q][j]);
    }
  }
#pragma unroll
  for (int q = 0; q < 3; ++q) s.p[q] = make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
  return s;
}

__device__ __forceinline__ f32x16 mma(const uint4 a, const uint4 b, const f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}
// The six largest partial products, the smallest first.
__device__ __forceinline__ f32x16 mma(const Split& a, const Split& b, f32x16 c) {
  c = mma(a.p[1], b.p[1], c);
  c = mma(a.p[2], b.p[0], c);
  c = mma(a.p[0], b.p[2], c);
  c = mma(a.p[1], b.p[0], c);
  c = mma(a.p[0], b.p[1], c);
  return mma(a.p[0], b.p[0], c);
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
  static constexpr int MB = BM / WM / 32, NB = BN / WN / 32;
  static constexpr int THREADS = 64 * W;
  static constexpr int BK = kStep / int(sizeof(T));
  static constexpr int KS = BK / 16;  // fragments along a step
  // B stored by k: rows of zeros follow its last, up to a whole step (A's repeat
  // its last there).
  static constexpr bool B_PADDED = TB;
  using OpA = Operand<T, TA, BM, W>;
  using OpB = Operand<T, TB, BN, W>;
  using RdA = Reader<T, TA, BM>;
  using RdB = Reader<T, TB, BN>;
  static constexpr int STEP = OpA::BYTES + OpB::BYTES;
  static constexpr int LDS = S * STEP;
  static constexpr int LOADS = OpA::NI + OpB::NI;
};

__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

// The fragments of 16 k of a wave's blocks.
template <typename C>
struct Frags {
  uint4 a[C::MB], b[C::NB];
  static constexpr int N = C::MB + C::NB;
  // Loads the i-th of them, in the order in which the products use them.
  __device__ __forceinline__ void load(int i, const typename C::RdA& ra, const typename C::RdB& rb, const char* ta,
                                       const char* tb, int ks) {
    if (i == 0) a[0] = ra.bf16(ta, 0, ks);
    else if (i <= C::NB) b[i - 1] = rb.bf16(tb, i - 1, ks);
    else a[i - C::NB] = ra.bf16(ta, i - C::NB, ks);
  }
};

// acc = the tile's products over the k (>= 1) elements from where A and B stand.
//
// bf16: while the matrix units work on one fragment step, the next one's reads are
// issued between its MFMAs, across the barrier into the next k-step too; fences
// keep that order.  The barrier stands before the last fragment step of a k-step:
// by then its last fragments have been read, so its place in the ring can be
// staged anew, and the next k-step has had S - 1 steps' time to land.
template <typename C>
__device__ __forceinline__ void run(f32x16 (&acc)[C::MB][C::NB], typename C::OpA& A, typename C::OpB& B,
                                    const typename C::RdA& ra, const typename C::RdB& rb, int k, char* lds) {
  using T = typename C::T;
  constexpr int MB = C::MB, NB = C::NB, KS = C::KS, S = C::S;
  const uint32_t at = lds_at(lds);
  const int steps = (k + C::BK - 1) / C::BK;
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[m][n][i] = 0.f;
  const auto stage = [&](int t, int buf) {
    A.stage(at + buf * C::STEP, k - t * C::BK);
    B.stage(at + buf * C::STEP + C::OpA::BYTES, C::B_PADDED ? C::BK : k - t * C::BK);
  };
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int t = 0; t < S; ++t)
      if (t < steps) stage(t, t);
    if (steps >= S) wait_step<C::LOADS * (S - 1)>();
    else wait_step<0>();
    barrier();
    Frags<C> f[2];
#pragma unroll
    for (int i = 0; i < Frags<C>::N; ++i) f[0].load(i, ra, rb, lds, lds + C::OpA::BYTES, 0);
    int cur = 0;
    for (int t = 0; t < steps; ++t) {
      const int next = cur + 1 == S ? 0 : cur + 1;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const bool turn = ks == KS - 1;
        if (turn) {
          // Step t + 1 has landed for every wave, and step t has been read by every wave.
          if (t + S <= steps) wait_step<C::LOADS * (S - 2)>();
          else wait_step<0>();
          barrier();
          if (t + S < steps) stage(t + S, cur);
        }
        const char* ta = lds + (turn ? next : cur) * C::STEP;
        const char* tb = ta + C::OpA::BYTES;
        Frags<C>& x = f[ks & 1];
        Frags<C>& y = f[(ks + 1) & 1];
        constexpr int PER = (Frags<C>::N + MB * NB - 1) / (MB * NB);
#pragma unroll
        for (int i = 0; i < MB * NB; ++i) {
          acc[i / NB][i % NB] = mma(x.a[i / NB], x.b[i % NB], acc[i / NB][i % NB]);
#pragma unroll
          for (int j = 0; j < PER; ++j)
            if (i * PER + j < Frags<C>::N) y.load(i * PER + j, ra, rb, ta, tb, (ks + 1) % KS);
          fence();
        }
      }
      cur = next;
    }
    return;
  }
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int t = 0; t < S - 1; ++t)
      if (t < steps) stage(t, t);
    int cur = 0, into = S - 1;
    for (int t = 0; t < steps; ++t) {
      // Step t has landed for every wave, and step t - 1 has been read by every wave.
      if (t + S - 1 <= steps) wait_step<C::LOADS * (S - 2)>();
      else wait_step<0>();
      barrier();
      if (t + S - 1 < steps) stage(t + S - 1, into);
      const char* ta = lds + cur * C::STEP;
      const char* tb = ta + C::OpA::BYTES;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        Split b[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          float x[8];
          rb.f32(tb, n, ks, x);
          b[n] = split3(x);
        }
#pragma unroll
        for (int m = 0; m < MB; ++m) {
          float x[8];
          ra.f32(ta, m, ks, x);
          const Split a = split3(x);
#pragma unroll
          for (int n = 0; n < NB; ++n) acc[m][n] = mma(a, b[n], acc[m][n]);
        }
      }
      cur = cur + 1 == S ? 0 : cur + 1;
      into = into + 1 == S ? 0 : into + 1;
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
