// Tree attention, forward and backward (gfx950).  Per query head and token i,
// over the tokens j on i's root-to-token path (attn_plan.hpp):
//     s_ij = scale q_i . k_j,  p_ij = exp(s_ij) / sum_j exp(s_ij),
//     o_i = sum_j p_ij v_j,    lse_i = log sum_j exp(s_ij),
// and, for given dO, with delta_i = dO_i . o_i and p recomputed from lse:
//     dv_j = sum_i p_ij dO_i,  ds_ij = p_ij (dO_i . v_j - delta_i),
//     dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i.
//
// All products run on 32x32 MFMA tiles whose accumulator keeps one row of
// the softmax in one lane column: the scores are computed transposed
// (keys x queries), lane l holds 16 keys of query l % 32, and row sums and
// maxima need one exchange between lanes l and l ^ 32.  The accumulator is
// then the B operand of the next product as it stands, because an MFMA's
// contraction index may be permuted if both operands agree: contraction slot
// (h = l / 32, e) is row 4h + e % 4 + 8 (e / 4) of the block, which is where
// the accumulator has its rows, and the A operand (V, K, Q or dO transposed)
// is read from LDS in that order by the transposing read.
//
// fp32 inputs run the same code on fp32 MFMA (32x32x2), four per 16-byte
// fragment, with exact products.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/tree_gdn.h"
#include "attn_plan.hpp"
#include "chunk_mfma.hpp"
#include "launch.hpp"

namespace tg {

namespace {

using chunk::bf16x8;
using chunk::ex2;
using chunk::kLog2e;
using chunk::lds_void;
using chunk::pk2;

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) const chunk::u32x4 lds_u4;
typedef __attribute__((address_space(3))) chunk::u32x4 lds_mu4;

// A copy of x the compiler knows nothing of: what is computed from it is
// computed where it stands, and not kept in registers across a loop.
__device__ __forceinline__ int opaque(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// This lane's number, made anew at every use.
__device__ __forceinline__ int lane_id() {
  int x;
  asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(x));
  return x;
}

// 16 bytes from LDS.
__device__ __forceinline__ uint4 lds16(const char* p) {
  const chunk::u32x4 w = *(lds_u4*)p;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kRows = 64;  // rows of a staged tile
constexpr float kNegInf = -__builtin_huge_valf();

// ---- LDS tiles --------------------------------------------------------------
// Rows of RB bytes; the 16-byte chunk c of row r sits at slot c ^ swz(r), so
// that operand reads (32 rows, one chunk each) and transposing reads (4 rows
// x 64 bytes) touch every bank once per half wave.
template <int RB>
__device__ __forceinline__ constexpr int swz(int r) {
  return RB >= 256 ? 4 * (r & 3) + ((r >> 2) & 3) : RB == 128 ? 4 * ((r >> 1) & 1) + ((r >> 2) & 3) : (r >> 2) & 3;
}

template <typename T>
__device__ __forceinline__ f32x16 mm(const uint4 a, const uint4 b, const f32x16 c);
template <>
__device__ __forceinline__ f32x16 mm<uint16_t>(const uint4 a, const uint4 b, const f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                 0, 0);
}
template <>
__device__ __forceinline__ f32x16 mm<float>(const uint4 a, const uint4 b, f32x16 c) {
  c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.x), __uint_as_float(b.x), c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.y), __uint_as_float(b.y), c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.z), __uint_as_float(b.z), c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.w), __uint_as_float(b.w), c, 0, 0, 0);
}

// Compile-time sizes of element type T and head size D.  A fragment is 16
// bytes a lane: contraction depth KD (16 in bf16, 8 in fp32).
template <typename T, int D>
struct Cfg {
  static constexpr int RB = D * int(sizeof(T));  // bytes of a row
  static constexpr int NC = RB / 16;             // 16-byte chunks of a row
  static constexpr int NK = RB / 32;             // fragments along a row
  static constexpr int NDB = D / 32;             // 32-wide blocks of a row
  static constexpr int KD = 32 / int(sizeof(T));
  static constexpr int NS = 32 / KD;             // fragments along 32 rows
  static constexpr int TILE = kRows * RB;        // bytes of a staged tile
  static constexpr int NI = TILE / 1024 / 4;     // DMA instructions of each of 4 waves
};

// Fragment s of 32 accumulator rows as the B operand of the next product.  bf16
// inputs: rounded to nearest even, by 2^-8 of the value at most, as the MFMA with
// the other operand's bf16 takes it (fp32 operands would take 16 times as long);
// sums stay in fp32.  Errors against 64 bits are 0.0021 (o) and 0.0024 (dq, dk,
// dv) of the result's norm, 0.0015 and 0.0018 with fp32 operands.
template <typename T>
__device__ __forceinline__ uint4 frag(const f32x16& p, int s);
template <>
__device__ __forceinline__ uint4 frag<uint16_t>(const f32x16& p, int s) {
  return make_uint4(pk2(p[8 * s], p[8 * s + 1]), pk2(p[8 * s + 2], p[8 * s + 3]), pk2(p[8 * s + 4], p[8 * s + 5]),
                    pk2(p[8 * s + 6], p[8 * s + 7]));
}
template <>
__device__ __forceinline__ uint4 frag<float>(const f32x16& p, int s) {
  return make_uint4(__float_as_uint(p[4 * s]), __float_as_uint(p[4 * s + 1]), __float_as_uint(p[4 * s + 2]),
                    __float_as_uint(p[4 * s + 3]));
}

// Byte offsets of this lane's operand reads in a tile.
template <typename T, int D>
struct Reader {
  using C = Cfg<T, D>;
  int row;  // operand reads: row lane % 32, chunk lane / 32
  int tr;   // transposing reads
  __device__ __forceinline__ explicit Reader(int lane) {
    const int r = lane & 31, h = lane >> 5, i = lane & 15;
    row = r * C::RB + 16 * (h ^ swz<C::RB>(r));
    if (sizeof(T) == 2) {
      const int k = 4 * h + (i >> 2);
      tr = k * C::RB + 16 * ((2 * ((lane >> 4) & 1) + ((i & 3) >> 1)) ^ swz<C::RB>(k)) + 8 * (i & 1);
    } else {
      tr = 4 * h * C::RB + 16 * ((r >> 2) ^ h) + 4 * (r & 3);
    }
  }
  // Rows 32 kb + lane % 32, fragment ks of the row.
  __device__ __forceinline__ uint4 rows(const char* t, int kb, int ks) const {
    return lds16(t + ((row ^ (32 * ks)) + kb * 32 * C::RB));
  }
  // The same lane's reads 32 rows further on (the offsets' low bits, which
  // the reads change, are not touched).
  __device__ __forceinline__ Reader block(int kb) const {
    Reader r = *this;
    r.row = opaque(row + kb * 32 * C::RB);
    r.tr = opaque(tr + kb * 32 * C::RB);
    return r;
  }
  // Fragment s of rows 32 kb .. 32 kb + 31 of the transposed tile: column 32
  // db + lane % 32.
  __device__ __forceinline__ uint4 cols(const char* t, int kb, int s, int db) const;
};
template <typename T, int D>
__device__ __forceinline__ uint4 Reader<T, D>::cols(const char* t, int kb, int s, int db) const {
  if constexpr (sizeof(T) == 2) {
    const int o = (tr ^ (64 * db)) + (32 * kb + 16 * s) * C::RB;
    const int o8 = (tr ^ (64 * db) ^ 32) + (32 * kb + 16 * s + 8) * C::RB;
    return chunk::cat(chunk::tile_tr(t, o), chunk::tile_tr(t, o8));
  } else {
    uint4 r;
    uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int sj = (C::RB >= 256 ? 4 * j : 4 * (j >> 1)) ^ (2 * (s & 1));
      const int o = (tr ^ (16 * sj) ^ (128 * db)) + (32 * kb + 8 * s + j) * C::RB;
      w[j] = *(__attribute__((address_space(3))) const uint32_t*)(t + o);
    }
    return r;
  }
}

// ---- values that are not finite ----------------------------------------------
// A masked pair's probability is 0, but 0 times an infinity or a NaN of a row
// the token does not see would still reach it through the MFMA.  Tiles with
// masked pairs that hold such elements therefore take them out first.  In the
// forward (rows of v) they are added one row at a time, where the probability
// is not 0, and cleared in LDS.  In the backward the whole row is cleared, and
// the gradients of every token that sees it (of dq) or that it sees (dk, dv)
// become NaN; a row with such a value in q, dO or o has a delta that is not
// finite.
template <typename T>
__device__ __forceinline__ uint32_t nonfinite(uint32_t w) {  // nonzero iff one of the word's elements is not finite
  if (sizeof(T) == 4) return (w & 0x7F800000u) == 0x7F800000u;
  return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}
template <typename T>
__device__ __forceinline__ uint32_t finite(uint32_t w) {  // elements that are not finite replaced by 0
  if (sizeof(T) == 4) return nonfinite<T>(w) ? 0u : w;
  const uint32_t f = nonfinite<T>(w) >> 15;  // bit 0, bit 16
  return w & ~(f * 0xFFFFu);
}
// Whether this thread's share (a quarter of a wave's tile) has one.
template <typename T, int D>
__device__ __forceinline__ bool any_nonfinite(const char* t, int tid) {
  using C = Cfg<T, D>;
  uint32_t f = 0;
#pragma unroll
  for (int i = 0; i < C::TILE / 4096; ++i) {
    const uint4 w = lds16(t + 16 * (tid + 256 * i));
    f |= nonfinite<T>(w.x) | nonfinite<T>(w.y) | nonfinite<T>(w.z) | nonfinite<T>(w.w);
  }
  return f != 0;
}
// Clears this thread's share.
template <typename T, int D>
__device__ __forceinline__ void clear_nonfinite(char* t, int tid) {
#pragma unroll 1
  for (int i = 0; i < Cfg<T, D>::TILE / 4096; ++i) {
    const uint4 w = lds16(t + 16 * (tid + 256 * i));
    *(lds_mu4*)(t + 16 * (tid + 256 * i)) =
        chunk::u32x4{finite<T>(w.x), finite<T>(w.y), finite<T>(w.z), finite<T>(w.w)};
  }
}
// Which of the tile's rows hold one (bit r: row r).
template <typename T, int D>
__device__ __forceinline__ uint64_t nonfinite_rows(const char* t, int lane) {
  using C = Cfg<T, D>;
  uint32_t f = 0;
#pragma unroll 1
  for (int c = 0; c < C::NC; ++c) {
    const uint4 x = lds16(t + lane * C::RB + 16 * c);
    f |= nonfinite<T>(x.x) | nonfinite<T>(x.y) | nonfinite<T>(x.z) | nonfinite<T>(x.w);
  }
  return __ballot(f != 0);
}
// Clears this thread's share of the rows of set `rows`.
template <typename T, int D>
__device__ __forceinline__ void clear_rows(char* t, uint64_t rows, int tid) {
  using C = Cfg<T, D>;
#pragma unroll 1
  for (int i = tid; i < kRows * C::NC; i += 256)
    if ((rows >> (i / C::NC)) & 1) *(lds_mu4*)(t + 16 * i) = chunk::u32x4{0u, 0u, 0u, 0u};
}
// acc[db] (columns 32 db + accumulator row, of the tile's rows weighted by w)
// += the elements that are not finite.
template <typename T, int D>
__device__ __forceinline__ void add_nonfinite(f32x16 (&acc)[D / 32], const f32x16 (&w)[2], const char* t, int lane) {
  using C = Cfg<T, D>;
  const int h = lane >> 5;
#pragma unroll 1
  for (uint64_t m = nonfinite_rows<T, D>(t, lane); m; m &= m - 1) {
    const int c = __builtin_ctzll(m), kb = c >> 5, cc = c & 31;
    const int reg = 4 * (cc >> 3) + (cc & 3), half = (cc >> 2) & 1;
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x = kb == 0 && i == reg ? w[0][i] : x;
      x = kb == 1 && i == reg ? w[1][i] : x;
    }
    const float y = __shfl_xor(x, 32, 64);
    x = h == half ? x : y;
#pragma unroll
    for (int db = 0; db < C::NDB; ++db)
#pragma unroll
      for (int i4 = 0; i4 < 4; ++i4) {
        const int by = (32 * db + 8 * i4 + 4 * h) * int(sizeof(T));
        const char* p = t + c * C::RB + 16 * ((by >> 4) ^ swz<C::RB>(c)) + (by & 15);
        float e[4];
        if (sizeof(T) == 4) {
          const uint4 z = lds16(p);
          e[0] = __uint_as_float(z.x), e[1] = __uint_as_float(z.y);
          e[2] = __uint_as_float(z.z), e[3] = __uint_as_float(z.w);
        } else {
          const chunk::u32x2 z = *(chunk::lds_cu2*)p;
          e[0] = chunk::lo_f(z[0]), e[1] = chunk::hi_f(z[0]);
          e[2] = chunk::lo_f(z[1]), e[3] = chunk::hi_f(z[1]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool lost = (__float_as_uint(e[j]) & 0x7F800000u) == 0x7F800000u;
          acc[db][4 * i4 + j] += lost && x != 0.f ? x * e[j] : 0.f;
        }
        asm volatile("" ::: "memory");  // one read at a time: this path must not cost the others registers
      }
  }
}

// acc[db] += (rows 32 kb .. 32 kb + 31 of the tile, transposed) times w: they
// are contracted with w's accumulator rows.
template <typename T, int D>
__device__ __forceinline__ void contract(f32x16 (&acc)[D / 32], const f32x16& w, const char* t, int kb,
                                         const Reader<T, D>& rd) {
  using C = Cfg<T, D>;
#pragma unroll
  for (int s = 0; s < C::NS; ++s) {
    const uint4 b = frag<T>(w, s);
#pragma unroll
    for (int db = 0; db < C::NDB; ++db) acc[db] = mm<T>(rd.cols(t, kb, s, db), b, acc[db]);
  }
}

// use(i, load(i)) for i < N with the next F loads in flight, in exactly this
// order: left to itself the compiler takes either one operand at a time (of the
// forward's scores; three: chain of 16383 tokens 554 -> 535 us) or more than the
// registers hold.
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }
template <int N, int F, typename Load, typename Use>
__device__ __forceinline__ void pipe(Load load, Use use) {
  constexpr int P = N < F ? N : F;
  uint4 x[P];
#pragma unroll
  for (int i = 0; i < P; ++i) x[i] = load(i);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    use(i, x[i % P]);
    if (i + P < N) x[i % P] = load(i + P);
    fence();
  }
}
// Accumulator rows 8 (i / 4) + i % 4 of 32 values (p already points at the
// lane's half).
__device__ __forceinline__ f32x16 rows16(const float* p) {
  f32x16 r;
#pragma unroll
  for (int i4 = 0; i4 < 4; ++i4) {
    const float4 x = *reinterpret_cast<const float4*>(p + 8 * i4);
    r[4 * i4] = x.x, r[4 * i4 + 1] = x.y, r[4 * i4 + 2] = x.z, r[4 * i4 + 3] = x.w;
  }
  return r;
}

// ---- run lists ----------------------------------------------------------------
// The packed row of virtual position v, for tiles of kRows positions taken in
// order (uniform over the wave but for `row`'s argument).
struct Cursor {
  const AttnRun* runs;
  int n, end;  // runs; positions of this item end here
  int cur, virt, row0, next;
  __device__ __forceinline__ Cursor(const AttnRun* r, const AttnItem& it) : runs(r + it.run_off), n(it.n_runs), end(it.v1) {
    cur = 0;
    load();
    seek(it.v0);
  }
  __device__ __forceinline__ void load() {
    virt = __builtin_amdgcn_readfirstlane(runs[cur].virt);
    row0 = __builtin_amdgcn_readfirstlane(runs[cur].row);
    next = cur + 1 < n ? __builtin_amdgcn_readfirstlane(runs[cur + 1].virt) : 0x7FFFFFFF;
  }
  __device__ __forceinline__ void seek(int v) {
    while (next <= v) {
      ++cur;
      load();
    }
  }
  // Whether the tile at v0 (in run `cur`) is kRows rows of one run.
  __device__ __forceinline__ bool whole(int v0) const { return v0 + kRows <= min(next, end); }
  // The row of position v0 + x (x < kRows, v0 in run `cur`); positions past
  // the end repeat the last.
  __device__ __forceinline__ int row(int v0, int x) const {
    const int v = min(v0 + x, end - 1);
    if (min(v0 + kRows, end) <= next) return row0 + (v - virt);
    int c = cur, lo = virt, r = row0;
    while (c + 1 < n) {
      const int nv = runs[c + 1].virt;
      if (nv > v) break;
      ++c;
      lo = nv;
      r = runs[c].row;
    }
    return r + (v - lo);
  }
};

// 16 (4) bytes a lane from `src` to LDS at lds + 16 (4) * lane.  In inline asm,
// because the compiler would otherwise wait for all DMA in flight before any
// read of LDS; it has no output registers, and wait_dma() is the wait.
__device__ __forceinline__ uint32_t lds_at(const char* lds) {
  return __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void*)lds)));
}
__device__ __forceinline__ void dma16(const void* src, char* lds) {
  int m0;
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, off\n\ts_mov_b32 m0, %0"
               : "=&s"(m0)
               : "s"(lds_at(lds)), "v"(src)
               : "memory");
}
// From src + off, src the same for all lanes; lds as an LDS address.
__device__ __forceinline__ void dma16(uint64_t src, int off, uint32_t lds) {
  int m0;
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %3\n\ts_mov_b32 m0, %0"
               : "=&s"(m0)
               : "s"(lds), "v"(off), "s"(src)
               : "memory");
}
// The same of four sources, to LDS 4096 bytes apart.
__device__ __forceinline__ void dma16x4(uint64_t s0, uint64_t s1, uint64_t s2, uint64_t s3, int off, uint32_t lds) {
  int m0;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %3\n\t"
      "s_add_u32 m0, m0, 0x1000\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %4\n\t"
      "s_add_u32 m0, m0, 0x1000\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %5\n\t"
      "s_add_u32 m0, m0, 0x1000\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %6\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(m0)
      : "s"(lds), "v"(off), "s"(s0), "s"(s1), "s"(s2), "s"(s3)
      : "memory", "scc");
}
__device__ __forceinline__ void dma4(const void* src, char* lds) {
  int m0;
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %2, off\n\ts_mov_b32 m0, %0"
               : "=&s"(m0)
               : "s"(lds_at(lds)), "v"(src)
               : "memory");
}
// All of this wave's loads and DMA have landed: vmcnt(0), the other counters
// as they are.  The builtin, unlike inline asm, lets the compiler know that its
// own loads have, so that it adds no wait behind the next tile's DMA.
__device__ __forceinline__ void wait_dma() {
  __builtin_amdgcn_s_waitcnt(0x0F70);
  asm volatile("" ::: "memory");
}

// Whether rows so many bytes apart can be staged from one address (stage_run: a
// lane's offset from it is below 16 of them, and a product in 32 bits).
__device__ __forceinline__ bool one_base(int64_t lda, int64_t ldb) {
  return uint64_t(lda) < (1 << 24) && uint64_t(ldb) < (1 << 24);
}

// The kRows rows from `first` on (lda bytes apart, one_base) into LDS tile ta,
// this wave's groups of them: one base for all lanes, a group apart.  Every
// instruction in front of a tile's products counts: with each load's address
// made by itself, the forward took 535 us instead of 519 (chain of 16383 tokens,
// 8/2 heads of 128), and 217 instead of 201 (10240 tokens, 16/4 heads).
template <typename T, int D>
__device__ __forceinline__ void stage_run(int64_t first, const char* a, int64_t lda, char* ta, int wave, int lane) {
  using C = Cfg<T, D>;
  constexpr int PER = 1024 / C::RB;  // rows of a group
  const uint32_t ld = uint32_t(lda), lds = lds_at(ta + 1024 * wave);
  const uint64_t src = reinterpret_cast<uint64_t>(a) + uint64_t(uint32_t(first) + uint32_t(wave * PER)) * ld;
  const uint64_t step = uint64_t(4 * PER) * ld;
  const int r = wave * PER + lane / C::NC;
  const auto off = [&](int i) {
    return (lane / C::NC) * int(ld) + 16 * ((lane % C::NC) ^ swz<C::RB>(4 * PER % 16 ? r + 4 * PER * i : r));
  };
  if constexpr (C::NI == 4) {
    dma16x4(src, src + step, src + 2 * step, src + 3 * step, off(0), lds);
  } else {
#pragma unroll
    for (int i = 0; i < C::NI; ++i) dma16(src + i * step, off(i), lds + 4096 * i);
  }
}

// The 64 rows at virtual position v0 of two tensors (a head's first row at a,
// b; bytes lda, ldb between rows) into LDS tiles ta, tb, by 4 waves (wave w:
// every fourth group of 1024 bytes).  Where `run` (kRows rows of one run, and
// one_base) no address arithmetic in the vector unit is needed: all lanes share
// a base.  `row` is this lane's row of the tile (lane l: row l), used otherwise.
template <typename T, int D>
__device__ __forceinline__ void stage(bool run, const Cursor& cs, int v0, int row, const char* a, int64_t lda,
                                      char* ta, const char* b, int64_t ldb, char* tb, int wave, int lane) {
  using C = Cfg<T, D>;
  constexpr int PER = 1024 / C::RB;  // rows of a group
  if (run) {
    const int64_t first = cs.row0 + (v0 - cs.virt);
    stage_run<T, D>(first, a, lda, ta, wave, lane);
    stage_run<T, D>(first, b, ldb, tb, wave, lane);
  } else {
#pragma unroll 1
    for (int i = 0; i < C::NI; ++i) {
      const int g = 4 * i + wave, r = g * PER + lane / C::NC;
      const int64_t from = __shfl(row, r, 64);
      const int c = 16 * ((lane % C::NC) ^ swz<C::RB>(r));
      dma16(a + from * lda + c, ta + 1024 * g);
      dma16(b + from * ldb + c, tb + 1024 * g);
    }
  }
}

// The sum or maximum of a lane and the lane 32 away.
__device__ __forceinline__ float half_swap(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

// A wave in its matrix products goes before one in its exponentials: the two
// waves of a SIMD then take turns, and the matrix unit waits less (chain of
// 16383 tokens, 8/2 heads of 128: 566 -> 536 us).
__device__ __forceinline__ void matrix_first(bool on) {
  if (on) __builtin_amdgcn_s_setprio(1);
  else __builtin_amdgcn_s_setprio(0);
}

__device__ __forceinline__ f32x16 zero16() {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}

// Fragments of row `p` (D elements): the B operand whose column is this lane.
template <typename T, int D>
__device__ __forceinline__ void load_frags(uint4* f, const char* p, int half) {
#pragma unroll
  for (int ks = 0; ks < Cfg<T, D>::NK; ++ks) f[ks] = *reinterpret_cast<const uint4*>(p + 32 * ks + 16 * half);
}

// Stores the accumulator's column (this lane's row of the result, D values
// times f) in 16-byte pieces: lanes l and l ^ 32 hold 4 columns each of every
// 8, and exchange so that each writes 8 (bf16).
template <typename T, int D>
__device__ __forceinline__ void store_row(T* p, const f32x16* acc, float f, int half, bool on) {
#pragma unroll
  for (int db = 0; db < D / 32; ++db) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (on)
          *reinterpret_cast<float4*>(p + 32 * db + 8 * c + 4 * half) =
              make_float4(acc[db][4 * c] * f, acc[db][4 * c + 1] * f, acc[db][4 * c + 2] * f, acc[db][4 * c + 3] * f);
    } else {
#pragma unroll
      for (int c = 0; c < 4; c += 2) {
        const uint32_t x0 = pk2(acc[db][4 * c] * f, acc[db][4 * c + 1] * f);
        const uint32_t x1 = pk2(acc[db][4 * c + 2] * f, acc[db][4 * c + 3] * f);
        const uint32_t y0 = pk2(acc[db][4 * c + 4] * f, acc[db][4 * c + 5] * f);
        const uint32_t y1 = pk2(acc[db][4 * c + 6] * f, acc[db][4 * c + 7] * f);
        const auto r0 = __builtin_amdgcn_permlane32_swap(x0, y0, false, false);
        const auto r1 = __builtin_amdgcn_permlane32_swap(x1, y1, false, false);
        if (on) *reinterpret_cast<uint4*>(p + 32 * db + 8 * (c + half)) = make_uint4(r0[0], r1[0], r0[1], r1[1]);
      }
    }
  }
}

// ---- work-groups to XCDs ---------------------------------------------------------
// Consecutive work-groups go to the 8 XCDs in turn, each with an L2 of its own.
// The query heads of one key/value head and tile, which read the same keys and
// values, are therefore 8 apart.
constexpr int kXcds = 8;
__device__ __forceinline__ bool work_of(const AttnArgs& a, int block, int* item, int* h, int* hk) {
  const int group = a.h_q / a.h_kv, slot = block / kXcds;
  const int u = slot / group * kXcds + block % kXcds;  // tile part and key/value head
  *item = u / a.h_kv;
  *hk = u % a.h_kv;
  *h = *hk * group + slot % group;
  return *item < a.n_items;
}
inline dim3 work_grid(const AttnArgs& a) {
  return dim3((a.n_items * a.h_kv + kXcds - 1) / kXcds * kXcds * (a.h_q / a.h_kv));
}

// ---- parts of a list --------------------------------------------------------------
// What a work-group leaves of its part (floats): the forward's unnormalised
// output rows, then every row's maximum and sum; rows of dq; rows of dk, then
// of dv.
__host__ __device__ constexpr int64_t fwd_part(int d) { return int64_t(kQTile) * (d + 2); }
__host__ __device__ constexpr int64_t dq_part(int d) { return int64_t(kQTile) * d; }
__host__ __device__ constexpr int64_t dkv_part(int d) { return int64_t(kKTile) * d * 2; }
constexpr int kJoinRows = 16;

// ---- forward --------------------------------------------------------------------
// The exponent c s - c m takes one fma with c m rounded, which is off by the same
// for all of a row's keys and cancels, but may be more than exp2 holds where c m
// is past 2^30.  From here on it is c (s - m).
constexpr float kWide = 16777216.f;

template <typename T, int D>
struct FwdSmem {
  alignas(16) char k[2][Cfg<T, D>::TILE];
  alignas(16) char v[2][Cfg<T, D>::TILE];
  alignas(16) int d[2][kRows];
  alignas(16) int e[2][kRows];
};

// Visibility of one staged tile of keys to the queries of one lane column
// (position dq): bit i of the result, accumulator row i of block kb.
__device__ __forceinline__ uint32_t visible(const int* d, const int* e, int kb, int half, int dq) {
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int4 x = *reinterpret_cast<const int4*>(d + 32 * kb + 8 * c + 4 * half);
    const int4 y = *reinterpret_cast<const int4*>(e + 32 * kb + 8 * c + 4 * half);
    m |= (x.x <= dq && dq < y.x ? 1u : 0u) << (4 * c);
    m |= (x.y <= dq && dq < y.y ? 1u : 0u) << (4 * c + 1);
    m |= (x.z <= dq && dq < y.z ? 1u : 0u) << (4 * c + 2);
    m |= (x.w <= dq && dq < y.w ? 1u : 0u) << (4 * c + 3);
  }
  return m;
}

// Least and greatest position of the wave's rows (lane l: row l % 32).
__device__ __forceinline__ void span(int dq, int& lo, int& hi) {
  lo = hi = dq;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    lo = min(lo, __shfl_xor(lo, o, 64));
    hi = max(hi, __shfl_xor(hi, o, 64));
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  hi = __builtin_amdgcn_readfirstlane(hi);
}

// One work-group of four waves: kQTile rows of one query head, 32 a wave; two
// work-groups a CU (96 registers of queries and sums at d = 128, 65 KB of LDS).
// What bounds it is issue: 64 keys are 32 MFMA (1024 cycles of a SIMD) and
// about 150 vector instructions, 32 of them exponentials (600 and more), of
// which the SIMD's other wave covers a part: matrix units are busy 58%, vector
// units 48% of the time, at 1.8 GHz, the clock that the load leaves (20% fewer
// cycles in the last steps took 7% less time); LDS reads have no conflicts and
// the keys come out of L2.  Tried: the exponentials of a tile between the products of the next one's
// scores, instruction by instruction, takes 15% longer (every wave then waits
// in turn for each operand, product and exponential); so do blocks of 32 keys
// (3%); the first values read before the exponentials, 1%.  More rows a wave
// would halve the LDS reads and need twice the registers.
// bf16, d = 128: chain of 16383 tokens, 8/2 heads, 499 us (1103 TFLOP/s; a large
// matrix product reaches 1380 there); 10240 tokens of 8 responses, 16/4 heads,
// 203 us; d = 64, 13941 tokens, 12/4 heads: 56 us.
template <typename T, int D>
__global__ __launch_bounds__(256, D * sizeof(T) <= 256 ? 2 : 1) void attn_fwd_kernel(AttnArgs a) {
  using C = Cfg<T, D>;
  __shared__ FwdSmem<T, D> sm;
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int item, h, hk;
  if (!work_of(a, blockIdx.x, &item, &h, &hk)) return;
  const AttnItem it = a.items[item];
  const int64_t row = int64_t(it.tile) * kQTile + 32 * wave + (lane & 31);
  const bool on = row < a.n_tok;
  const int64_t r = on ? row : a.n_tok - 1;
  const char* kp = a.k.at(0, hk);
  const char* vp = a.v.at(0, hk);

  const bool fast = one_base(a.k.row, a.v.row);
  Cursor cs(a.runs, it);
  auto fetch = [&](int v0, int buf) {
    cs.seek(v0);
    const bool part = v0 + kRows > it.n_full, run = fast && cs.whole(v0);
    const int row = part || !run ? cs.row(v0, lane) : 0;
    stage<T, D>(run, cs, v0, row, kp, a.k.row, sm.k[buf], vp, a.v.row, sm.v[buf], wave, lane);
    if (part && wave < 2) {
      const int x = v0 + lane < cs.end ? row : a.n_tok;
      if (wave == 0) dma4(a.tok_d + x, reinterpret_cast<char*>(sm.d[buf]));
      else dma4(a.tok_e + x, reinterpret_cast<char*>(sm.e[buf]));
    }
  };
  fetch(it.v0, 0);

  uint4 q[C::NK];
  load_frags<T, D>(q, a.q.at(r, h), half);
  const int dq = a.tok_d[r];
  int dlo, dhi;
  span(dq, dlo, dhi);

  const Reader<T, D> rd(lane);
  const float c = a.scale * kLog2e;
  f32x16 acc[C::NDB];
#pragma unroll
  for (int db = 0; db < C::NDB; ++db) acc[db] = zero16();
  float m = kNegInf, l = 0.f;  // running maximum of q.k (both halves of the wave agree), this lane's part of the sum
  bool wide = false;           // a row of this wave has scores past kWide

  // The tile at v0 is in buffer `buf`, a constant: LDS addresses then are a
  // lane's offset plus an immediate.
  const auto tile = [&](int v0, auto buffer) {
    constexpr int buf = decltype(buffer)::value;
    wait_dma();
    __syncthreads();
    // Where the next tile is seen whole (so this one is, too) and goes on in the
    // same run, it is staged behind this one's scores, whose products then start
    // at once (chain of 16383 tokens, 8/2 heads of 128: 532 -> 504 us).  Any tile
    // behind the scores: chain 513, but tiles with masked pairs then wait for their
    // keys (220 short segments, 12/4 heads of 64: 56 -> 67 us).
    const bool late = fast && v0 + 2 * kRows <= min(min(it.n_full, it.v1), cs.next);
    if (!late && v0 + kRows < it.v1) fetch(v0 + kRows, buf ^ 1);
    const char* kt = sm.k[buf];
    char* vt = sm.v[buf];
    bool masked = v0 + kRows > it.n_full, bad = false, skip = false;
    if (masked) {
      bad = __syncthreads_or(any_nonfinite<T, D>(vt, threadIdx.x));
      const int kd = sm.d[buf][lane], ke = sm.e[buf][lane];
      skip = __ballot(kd <= dhi && dlo < ke) == 0;        // no row of this wave sees a key of this tile
      masked = __ballot(kd <= dlo && dhi < ke) != ~0ull;  // every row sees every key
    }
    f32x16 p[2];
    if (!skip) {
      matrix_first(true);
      pipe<2 * C::NK, 3>([&](int i) { return rd.rows(kt, i & 1, i >> 1); },
                       [&](int i, const uint4 x) { p[i & 1] = mm<T>(x, q[i >> 1], i < 2 ? zero16() : p[i & 1]); });
      matrix_first(false);
      if (late) {
        const int64_t first = cs.row0 + (v0 + kRows - cs.virt);
        stage_run<T, D>(first, kp, a.k.row, sm.k[buf ^ 1], wave, lane);
        stage_run<T, D>(first, vp, a.v.row, sm.v[buf ^ 1], wave, lane);
      }
      if (masked) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          const uint32_t see = visible(sm.d[buf], sm.e[buf], kb, half, dq);
#pragma unroll
          for (int i = 0; i < 16; ++i) p[kb][i] = (see >> i) & 1 ? p[kb][i] : kNegInf;
        }
      }
      float mt = p[0][0];
#pragma unroll
      for (int i = 1; i < 16; ++i) mt = fmaxf(mt, p[0][i]);
#pragma unroll
      for (int i = 0; i < 16; ++i) mt = fmaxf(mt, p[1][i]);
      mt = fmaxf(mt, half_swap(mt));
      // A row's accumulators follow its maximum only when that has grown by
      // more than 2^8: until then the probabilities stay below 2^8, harmless
      // in fp32 and no less exact in bf16.
      const bool grown = (mt - m) * c > 8.f;
      if (__any(grown)) {
        const float mn = grown ? mt : m;
        const float al = m == kNegInf ? 0.f : ex2((m - mn) * c);
        m = mn;
        wide = __any(m != kNegInf && fabsf(m * c) > kWide);
        l *= al;
#pragma unroll
        for (int db = 0; db < C::NDB; ++db)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[db][i] *= al;
      }
      const float m0 = m == kNegInf ? 0.f : m;  // -inf: this row has seen no key yet
      float mc = m0 * c;
      if (wide) {
        const float by = fabsf(mc) > kWide ? m0 : 0.f;  // other rows keep their bits
        mc = by != 0.f ? 0.f : mc;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int i = 0; i < 16; ++i) p[kb][i] -= by;
      }
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          p[kb][i] = ex2(fmaf(p[kb][i], c, -mc));
          l += p[kb][i];
        }
    }
    if (bad) {
      if (!skip) add_nonfinite<T, D>(acc, p, vt, lane);
      __syncthreads();
      clear_nonfinite<T, D>(vt, threadIdx.x);
      __syncthreads();
    }
    if (!skip) {
      matrix_first(true);
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) contract<T, D>(acc, p[kb], vt, kb, rd);
      matrix_first(false);
    }
  };
  for (int v0 = it.v0;;) {
    tile(v0, std::integral_constant<int, 0>{});
    if ((v0 += kRows) >= it.v1) break;
    tile(v0, std::integral_constant<int, 1>{});
    if ((v0 += kRows) >= it.v1) break;
  }
  l += half_swap(l);
  if (it.part < a.n_parts) {
    // Part of the list: the sums as they are, with the maximum (in powers of
    // 2) and the sum of exponentials they go by.
    float* w = a.part + (int64_t(it.part) * a.h_q + h) * fwd_part(D);
    const int key = 32 * wave + (lane & 31);
    store_row<float, D>(w + key * D, acc, 1.f, half, true);
    if (half == 0) *reinterpret_cast<float2*>(w + kQTile * D + 2 * key) = make_float2(m * c, l);
    return;
  }
  const float inv = 1.f / l;
  store_row<T, D>(static_cast<T*>(a.out) + (r * a.h_q + h) * D, acc, inv, half, on);
  if (a.lse && on && half == 0) a.lse[r * a.h_q + h] = (m * c + __log2f(l)) * kLn2;
}

// The output of a query tile from its parts, in their order: 16 rows a
// work-group, bound by memory (the parts are written and read once, in fp32).
template <typename T, int D>
__global__ __launch_bounds__(kJoinRows * D / 4) void attn_fwd_join_kernel(AttnArgs a) {
  const int h = blockIdx.y, key = kJoinRows * blockIdx.z + threadIdx.x / (D / 4), col = 4 * (threadIdx.x % (D / 4));
  const AttnParts pt = a.parts[blockIdx.x];
  const int64_t row = int64_t(pt.tile) * kQTile + key;
  if (row >= a.n_tok) return;
  const int64_t step = int64_t(a.h_q) * fwd_part(D);
  const float* w = a.part + (int64_t(pt.part0) * a.h_q + h) * fwd_part(D);
  const float* st = w + kQTile * D + 2 * key;
  float m = kNegInf;
  for (int j = 0; j < pt.n_parts; ++j) m = fmaxf(m, st[j * step]);
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
#pragma unroll 2
  for (int j = 0; j < pt.n_parts; ++j) {
    const float2 x = *reinterpret_cast<const float2*>(st + j * step);
    const float4 y = *reinterpret_cast<const float4*>(w + j * step + key * D + col);
    const float f = x.x == kNegInf ? 0.f : ex2(x.x - m);  // -inf: the row sees nothing of this part
    l = fmaf(f, x.y, l);
    s.x = fmaf(f, y.x, s.x);
    s.y = fmaf(f, y.y, s.y);
    s.z = fmaf(f, y.z, s.z);
    s.w = fmaf(f, y.w, s.w);
  }
  const float inv = 1.f / l;
  T* out = static_cast<T*>(a.out) + (row * a.h_q + h) * D + col;
  if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(out) = make_float4(s.x * inv, s.y * inv, s.z * inv, s.w * inv);
  else *reinterpret_cast<uint2*>(out) = make_uint2(pk2(s.x * inv, s.y * inv), pk2(s.z * inv, s.w * inv));
  if (a.lse && col == 0) a.lse[row * a.h_q + h] = (m + __log2f(l)) * kLn2;
}

// ---- gradient of q -----------------------------------------------------------------
// Same tiles as the forward; also leaves -delta and -lse / scale, which the
// other gradients' sums start from.  Three products and one exponential a pair:
// the matrix units are busy 58% of the time (chain of 16383 tokens, 8/2 heads of
// 128: 740 us).  S and dP are computed here and again for dk and dv, seven
// products in all: a single pass of five would add to dq from every key tile,
// by atomics in an order that changes, or keep a part per tile.
template <typename T, int D>
__global__ __launch_bounds__(256, D * sizeof(T) <= 256 ? 2 : 1) void attn_dq_kernel(AttnArgs a) {
  using C = Cfg<T, D>;
  __shared__ FwdSmem<T, D> sm;
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int item, h, hk;
  if (!work_of(a, blockIdx.x, &item, &h, &hk)) return;
  const AttnItem it = a.items[item];
  const int64_t row = int64_t(it.tile) * kQTile + 32 * wave + (lane & 31);
  const bool on = row < a.n_tok;
  const int64_t r = on ? row : a.n_tok - 1;
  const char* kp = a.k.at(0, hk);
  const char* vp = a.v.at(0, hk);

  const bool fast = one_base(a.k.row, a.v.row);
  Cursor cs(a.runs, it);
  auto fetch = [&](int v0, int buf) {
    cs.seek(v0);
    const bool part = v0 + kRows > it.n_full, run = fast && cs.whole(v0);
    const int row = part || !run ? cs.row(v0, lane) : 0;
    stage<T, D>(run, cs, v0, row, kp, a.k.row, sm.k[buf], vp, a.v.row, sm.v[buf], wave, lane_id());
    if (part && wave < 2) {
      const int x = v0 + lane < cs.end ? row : a.n_tok;
      if (wave == 0) dma4(a.tok_d + x, reinterpret_cast<char*>(sm.d[buf]));
      else dma4(a.tok_e + x, reinterpret_cast<char*>(sm.e[buf]));
    }
  };
  fetch(it.v0, 0);

  uint4 q[C::NK], g[C::NK];
  load_frags<T, D>(q, a.q.at(r, h), half);
  load_frags<T, D>(g, a.dout.at(r, h), half);
  float delta = 0.f;
  {
    const char* op = a.o.at(r, h);
#pragma unroll
    for (int ks = 0; ks < C::NK; ++ks) {
      const uint4 o = *reinterpret_cast<const uint4*>(op + 32 * ks + 16 * half);
      const uint32_t x[4] = {o.x, o.y, o.z, o.w}, y[4] = {g[ks].x, g[ks].y, g[ks].z, g[ks].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (sizeof(T) == 4) {
          delta = fmaf(__uint_as_float(x[j]), __uint_as_float(y[j]), delta);
        } else {
          delta = fmaf(chunk::lo_f(x[j]), chunk::lo_f(y[j]), delta);
          delta = fmaf(chunk::hi_f(x[j]), chunk::hi_f(y[j]), delta);
        }
      }
    }
    delta += half_swap(delta);
  }
  const float lse = a.lse[r * a.h_q + h], lse2 = lse * kLog2e;
  if (on && half == 0) {
    a.delta[r * a.h_q + h] = -delta;
    a.delta[(int64_t(a.n_tok) + r) * a.h_q + h] = -lse / a.scale;
  }
  const int dq = a.tok_d[r];
  int dlo, dhi;
  span(dq, dlo, dhi);

  const Reader<T, D> rd(lane);
  const float c = a.scale * kLog2e;
  f32x16 acc[C::NDB];
#pragma unroll
  for (int db = 0; db < C::NDB; ++db) acc[db] = zero16();

  // The tile at v0 is in buffer `buf`, a constant: LDS addresses then are a
  // lane's offset plus an immediate.
  const auto tile = [&](int v0, auto buffer) {
    constexpr int buf = decltype(buffer)::value;
    wait_dma();
    __syncthreads();
    if (v0 + kRows < it.v1) fetch(v0 + kRows, buf ^ 1);
    char* kt = sm.k[buf];
    const char* vt = sm.v[buf];
    bool masked = v0 + kRows > it.n_full, skip = false;
    if (masked) {
      const bool bad = __syncthreads_or(any_nonfinite<T, D>(kt, threadIdx.x));
      const int kd = sm.d[buf][lane], ke = sm.e[buf][lane];
      skip = __ballot(kd <= dhi && dlo < ke) == 0;
      masked = __ballot(kd <= dlo && dhi < ke) != ~0ull;
      if (bad) {
        const uint64_t rows = nonfinite_rows<T, D>(kt, lane);
        float x = 0.f;
        for (uint64_t m = rows; m; m &= m - 1) {
          const int r = __builtin_ctzll(m);
          x = sm.d[buf][r] <= dq && dq < sm.e[buf][r] ? __builtin_nanf("") : x;
        }
#pragma unroll
        for (int db = 0; db < C::NDB; ++db)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[db][i] += x;
        __syncthreads();
        clear_rows<T, D>(kt, rows, threadIdx.x);
        __syncthreads();
      }
    }
    if (skip) return;
    f32x16 ds[2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      f32x16 s = zero16(), dp = zero16();
      matrix_first(true);
      pipe<C::NK, 2>([&](int ks) { return rd.rows(kt, kb, ks); },
                  [&](int ks, const uint4 x) { s = mm<T>(x, q[ks], s); });
      pipe<C::NK, 2>([&](int ks) { return rd.rows(vt, kb, ks); },
                  [&](int ks, const uint4 x) {
                    dp = mm<T>(x, g[ks], dp);
#pragma unroll
                    for (int i = 16 * ks / C::NK; i < 16 * (ks + 1) / C::NK; ++i) s[i] = ex2(fmaf(s[i], c, -lse2));
                  });
      matrix_first(false);
#pragma unroll
      for (int i = 0; i < 16; ++i) ds[kb][i] = s[i] * (dp[i] - delta);
      if (masked) {
        const uint32_t see = visible(sm.d[buf], sm.e[buf], kb, half, dq);
#pragma unroll
        for (int i = 0; i < 16; ++i) ds[kb][i] = (see >> i) & 1 ? ds[kb][i] : 0.f;
      }
    }
    matrix_first(true);
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
      pipe<C::NS * C::NDB, 2>([&](int i) { return rd.cols(kt, kb, i / C::NDB, i % C::NDB); },
                           [&](int i, const uint4 x) {
                             acc[i % C::NDB] = mm<T>(x, frag<T>(ds[kb], i / C::NDB), acc[i % C::NDB]);
                           });
    matrix_first(false);
  };
  for (int v0 = it.v0;;) {
    tile(v0, std::integral_constant<int, 0>{});
    if ((v0 += kRows) >= it.v1) break;
    tile(v0, std::integral_constant<int, 1>{});
    if ((v0 += kRows) >= it.v1) break;
  }
  {
    const int lane = lane_id(), key = 32 * wave + (lane & 31);
    const int64_t row = int64_t(it.tile) * kQTile + key;
    if (it.part < a.n_parts)
      store_row<float, D>(a.part + (int64_t(it.part) * a.h_q + h) * dq_part(D) + key * D, acc, a.scale, lane >> 5, true);
    else
      store_row<T, D>(static_cast<T*>(a.out) + (row * a.h_q + h) * D, acc, a.scale, lane >> 5, row < a.n_tok);
  }
}

// ---- gradients of k and v ------------------------------------------------------------
template <typename T, int D>
struct BwdSmem {
  alignas(16) char q[2][Cfg<T, D>::TILE];
  alignas(16) char g[2][Cfg<T, D>::TILE];
  alignas(16) float lse[2][kRows];    // -lse / scale
  alignas(16) float delta[2][kRows];  // -delta
  alignas(16) int d[2][kRows];
};

// One work-group of four waves: kKTile keys of one key/value head, 32 a wave,
// over this item's part of the rows that see them and every split-th query
// head of the group.  K and V of a wave's keys and both sums stay in registers
// (192 of 256 at d = 128); rows of q and dO pass through LDS, each read twice:
// by rows for S and dP, transposed for dv and dk.  What bounds it are those reads
// between the products, two or three in flight being all that the registers
// leave: matrix units 56% busy, chain of 16383 tokens, 8/2 heads of 128: 1005 us.
// 64 keys a wave at one wave a SIMD spilled (7.6 ms); an order left to the
// compiler took 1849 us.
template <typename T, int D>
__global__ __launch_bounds__(256, D * sizeof(T) <= 256 ? 2 : 1) void attn_dkv_kernel(AttnArgs a) {
  using C = Cfg<T, D>;
  __shared__ BwdSmem<T, D> sm;
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sub = blockIdx.x % a.split, hk = (blockIdx.x / a.split) % a.h_kv;
  const AttnItem it = a.items[blockIdx.x / (a.split * a.h_kv)];
  const int group = a.h_q / a.h_kv;
  const int64_t r = min(int64_t(it.tile) * kKTile + 32 * wave + (lane & 31), int64_t(a.n_tok) - 1);

  const bool fast = one_base(a.q.row, a.dout.row);
  Cursor cs(a.runs, it);
  auto fetch = [&](int v0, int h, int buf) {
    cs.seek(v0);
    const int lane = lane_id();
    const int row = cs.row(v0, lane);
    stage<T, D>(fast && cs.whole(v0), cs, v0, row, a.q.at(0, h), a.q.row, sm.q[buf], a.dout.at(0, h), a.dout.row,
                sm.g[buf], wave, lane_id());
    const int64_t x = int64_t(row) * a.h_q + h;
    if (wave == 0) dma4(a.delta + int64_t(a.n_tok) * a.h_q + x, reinterpret_cast<char*>(sm.lse[buf]));
    else if (wave == 1) dma4(a.delta + x, reinterpret_cast<char*>(sm.delta[buf]));
    else if (wave == 2) dma4(a.tok_d + (v0 + lane < cs.end ? row : a.n_tok), reinterpret_cast<char*>(sm.d[buf]));
  };
  int h = hk * group + sub;
  fetch(it.v0, h, 0);

  uint4 kf[C::NK], vf[C::NK];
  load_frags<T, D>(kf, a.k.at(r, hk), half);
  load_frags<T, D>(vf, a.v.at(r, hk), half);
  const int kd = a.tok_d[r], ke = a.tok_e[r];
  int kdlo, kdhi, kelo, kehi;
  span(kd, kdlo, kdhi);
  span(ke, kelo, kehi);

  const float c = a.scale * kLog2e;
  f32x16 dk[C::NDB], dv[C::NDB];
#pragma unroll
  for (int db = 0; db < C::NDB; ++db) dk[db] = dv[db] = zero16();

  int v0 = it.v0;
  const auto tile = [&](auto buffer) {
    constexpr int buf = decltype(buffer)::value;
    wait_dma();
    __syncthreads();
    int nv = v0 + kRows, nh = h;
    if (nv >= it.v1) {
      nv = it.v0;
      nh += a.split;
      cs.cur = 0;
      cs.load();
    }
    if (nh < (hk + 1) * group) fetch(nv, nh, buf ^ 1);
    char* qt = sm.q[buf];
    char* gt = sm.g[buf];
    bool masked = min(v0 + kRows, it.v1) > it.n_full || v0 + kRows > it.v1, skip = false;
    uint64_t bad = 0;  // rows of a tile with masked pairs whose delta is not finite
    v0 = nv;
    h = nh;
    if (masked) {
      const int lane = lane_id();
      bad = __ballot(nonfinite<float>(__float_as_uint(sm.delta[buf][lane])));
      const int qd = sm.d[buf][lane];
      skip = __ballot(kdlo <= qd && qd < kehi) == 0;
      masked = __ballot(kdhi <= qd && qd < kelo) != ~0ull;
    }
    if (bad) {  // uniform over the work-group
      float x = 0.f;
      for (uint64_t m = bad; m; m &= m - 1) {
        const int rd = sm.d[buf][__builtin_ctzll(m)];
        x = kd <= rd && rd < ke ? __builtin_nanf("") : x;
      }
#pragma unroll
      for (int db = 0; db < C::NDB; ++db)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          dk[db][i] += x;
          dv[db][i] += x;
        }
      __syncthreads();
      const int r = lane_id();
      clear_rows<T, D>(qt, bad, 64 * wave + r);
      clear_rows<T, D>(gt, bad, 64 * wave + r);
      if (wave == 0 && (bad >> r) & 1) {
        sm.lse[buf][r] = kNegInf;  // p = 0
        sm.delta[buf][r] = 0.f;
      }
      __syncthreads();
    }
    if (skip) return;
    const int ln = lane_id(), half = ln >> 5;
    const Reader<T, D> all(ln);
#pragma unroll 1
    for (int kb = 0; kb < 2; ++kb) {
      const Reader<T, D> rd = all.block(kb);
      // The sums start at -lse / scale and -delta: p = exp2(c s), ds = p dp.
      f32x16 p = rows16(sm.lse[buf] + 32 * kb + 4 * half);
      matrix_first(true);
      pipe<C::NK, 3>([&](int ks) { return rd.rows(qt, 0, ks); },
                  [&](int ks, const uint4 x) { p = mm<T>(x, kf[ks], p); });
      f32x16 ds = rows16(sm.delta[buf] + 32 * kb + 4 * half);
      pipe<C::NK, 3>([&](int ks) { return rd.rows(gt, 0, ks); },
                  [&](int ks, const uint4 x) {
                    ds = mm<T>(x, vf[ks], ds);
#pragma unroll
                    for (int i = 16 * ks / C::NK; i < 16 * (ks + 1) / C::NK; ++i) p[i] = ex2(p[i] * c);
                  });
      matrix_first(false);
      if (masked) {  // an unseen row's dO . v may be anything
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4) {
          const int4 dd = *reinterpret_cast<const int4*>(&sm.d[buf][32 * kb + 8 * i4 + 4 * half]);
          const int x4[4] = {dd.x, dd.y, dd.z, dd.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bool see = kd <= x4[j] && x4[j] < ke;
            p[4 * i4 + j] = see ? p[4 * i4 + j] : 0.f;
            ds[4 * i4 + j] = see ? ds[4 * i4 + j] : 0.f;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) ds[i] *= p[i];
      uint4 pb[C::NS], db[C::NS];
#pragma unroll
      for (int s = 0; s < C::NS; ++s) {
        pb[s] = frag<T>(p, s);
        db[s] = frag<T>(ds, s);
      }
      matrix_first(true);
      pipe<C::NS * C::NDB, 3>([&](int i) { return rd.cols(gt, 0, i / C::NDB, i % C::NDB); },
                           [&](int i, const uint4 x) { dv[i % C::NDB] = mm<T>(x, pb[i / C::NDB], dv[i % C::NDB]); });
      pipe<C::NS * C::NDB, 3>([&](int i) { return rd.cols(qt, 0, i / C::NDB, i % C::NDB); },
                           [&](int i, const uint4 x) { dk[i % C::NDB] = mm<T>(x, db[i / C::NDB], dk[i % C::NDB]); });
      matrix_first(false);
    }
  };
  while (true) {
    tile(std::integral_constant<int, 0>{});
    if (h >= (hk + 1) * group) break;
    tile(std::integral_constant<int, 1>{});
    if (h >= (hk + 1) * group) break;
  }
  const int ln = lane_id(), hl = ln >> 5, key = 32 * wave + (ln & 31);
  if (it.part >= a.n_parts) {
    const int64_t row = int64_t(it.tile) * kKTile + key;
    store_row<T, D>(static_cast<T*>(a.dk) + (row * a.h_kv + hk) * D, dk, a.scale, hl, row < a.n_tok);
    store_row<T, D>(static_cast<T*>(a.dv) + (row * a.h_kv + hk) * D, dv, 1.f, hl, row < a.n_tok);
  } else {
    float* w = a.part + ((int64_t(it.part) * a.split + sub) * a.h_kv + hk) * dkv_part(D) + key * D;
    store_row<float, D>(w, dk, a.scale, hl, true);
    store_row<float, D>(w + kKTile * D, dv, 1.f, hl, true);
  }
}

// A tile's gradients (dq, or dk and dv) from its parts, in their order: 16 rows
// a work-group, bound by memory (25 us on a chain of 16383 tokens, 8/2 heads of
// 128).
template <typename T, int D, bool DQ>
__global__ __launch_bounds__(kJoinRows * D / 4) void attn_grad_join_kernel(AttnArgs a) {
  const int heads = DQ ? a.h_q : a.h_kv, h = blockIdx.y;
  const int which = DQ ? 0 : blockIdx.z & 1, row0 = kJoinRows * (DQ ? blockIdx.z : blockIdx.z >> 1);
  const AttnParts pt = a.parts[blockIdx.x];
  const int64_t split = DQ ? 1 : a.split, slots = pt.n_parts * split;
  const int64_t floats = DQ ? dq_part(D) : dkv_part(D), step = heads * floats / 4;
  const int key = row0 + threadIdx.x / (D / 4);
  const int64_t row = int64_t(pt.tile) * kKTile + key;
  if (row >= a.n_tok) return;
  const float4* p = reinterpret_cast<const float4*>(a.part + (pt.part0 * split * heads + h) * floats +
                                                    which * kKTile * D) +
                    key * (D / 4) + threadIdx.x % (D / 4);
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int64_t j = 0; j < slots; ++j) {
    const float4 x = p[j * step];
    s.x += x.x;
    s.y += x.y;
    s.z += x.z;
    s.w += x.w;
  }
  T* out = static_cast<T*>(DQ ? a.out : which ? a.dv : a.dk) + (row * heads + h) * D + 4 * (threadIdx.x % (D / 4));
  if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(out) = s;
  else *reinterpret_cast<uint2*>(out) = make_uint2(pk2(s.x, s.y), pk2(s.z, s.w));
}

template <typename F>
hipError_t dispatch(int d, int dtype, F f) {
  if (dtype == TREE_DTYPE_BF16) {
    if (d == 32) return f(uint16_t{}, std::integral_constant<int, 32>{});
    if (d == 64) return f(uint16_t{}, std::integral_constant<int, 64>{});
    if (d == 128) return f(uint16_t{}, std::integral_constant<int, 128>{});
  } else if (dtype == TREE_DTYPE_F32) {
    if (d == 32) return f(float{}, std::integral_constant<int, 32>{});
    if (d == 64) return f(float{}, std::integral_constant<int, 64>{});
    if (d == 128) return f(float{}, std::integral_constant<int, 128>{});
  }
  return hipErrorInvalidValue;
}

}  // namespace

bool attention_supported(int d, int dtype) {
  return (d == 32 || d == 64 || d == 128) && (dtype == TREE_DTYPE_BF16 || dtype == TREE_DTYPE_F32);
}

int64_t attention_part_floats(int d) { return fwd_part(d); }
int64_t attention_dq_part_floats(int d) { return dq_part(d); }
int64_t attention_dkv_part_floats(int d) { return dkv_part(d); }

hipError_t launch_attention(const AttnArgs& a, int d, int dtype, hipStream_t stream) {
  return dispatch(d, dtype, [&](auto t, auto dd) {
    using T = decltype(t);
    constexpr int D = decltype(dd)::value;
    attn_fwd_kernel<T, D><<<work_grid(a), 256, 0, stream>>>(a);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && a.n_join > 0) {
      attn_fwd_join_kernel<T, D><<<dim3(a.n_join, a.h_q, kQTile / kJoinRows), kJoinRows * D / 4, 0, stream>>>(a);
      e = hipGetLastError();
    }
    return e;
  });
}

hipError_t launch_attention_dq(const AttnArgs& a, int d, int dtype, hipStream_t stream) {
  return dispatch(d, dtype, [&](auto t, auto dd) {
    using T = decltype(t);
    constexpr int D = decltype(dd)::value;
    attn_dq_kernel<T, D><<<work_grid(a), 256, 0, stream>>>(a);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && a.n_join > 0) {
      attn_grad_join_kernel<T, D, true>
          <<<dim3(a.n_join, a.h_q, kQTile / kJoinRows), kJoinRows * D / 4, 0, stream>>>(a);
      e = hipGetLastError();
    }
    return e;
  });
}

hipError_t launch_attention_dkv(const AttnArgs& a, int d, int dtype, hipStream_t stream) {
  return dispatch(d, dtype, [&](auto t, auto dd) {
    using T = decltype(t);
    constexpr int D = decltype(dd)::value;
    attn_dkv_kernel<T, D><<<dim3(a.n_items * a.h_kv * a.split), 256, 0, stream>>>(a);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && a.n_join > 0) {
      attn_grad_join_kernel<T, D, false>
          <<<dim3(a.n_join, a.h_kv, 2 * kKTile / kJoinRows), kJoinRows * D / 4, 0, stream>>>(a);
      e = hipGetLastError();
    }
    return e;
  });
}

}  // namespace tg
