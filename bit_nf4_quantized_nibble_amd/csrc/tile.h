// tile.h -- the tiled contraction that the 8-bit floating-point product (fp8.hip), the 16-bit GEMMs
// (gemm16.hip) and the products of planes (planes.hip) share, on gfx950.
//
// A workgroup forms a TM x TN tile: NWM x NWN waves, each with WMB x WNB blocks of a 32 x 32 matrix
// instruction.  The contraction advances 128 bytes per stage (128 codes of 8 bits, 64 16-bit
// elements); a stage's operands lie in LDS as rows of 128 bytes [TM rows of A | TN rows of B],
// 16-byte chunk c of row r at chunk c ^ swz(r) (one chunk of 16 consecutive rows then touches every
// bank group once), copied from global memory without passing through registers.  NS stages are
// in flight or in use.
//
// A stage is KIND::SUB sub-steps.  The fragments of a sub-step are read while the one before
// multiplies, across stages too: one barrier per stage, in its last sub-step, is where the next stage
// has landed and every wave has its last fragments of this one, so that from there on the wave reads
// the first fragments of the next stage and the copies into this stage's buffer run.
// 16-bit fragments have two sets of registers.  8-bit ones are twice as long, and two sets would
// take the 256 x 256 tile past the 256 registers that two waves on a SIMD leave each: there a
// fragment is replaced as soon as the products that need it are issued (columns of blocks in the
// outer loop: four or more products of 64 cycles lie between a fragment's read and its use).
#pragma once

#include <type_traits>

#include "common.h"

namespace qnf4 {
namespace tile {

typedef int i32x4_t __attribute__((__vector_size__(16)));
typedef int i32x8_t __attribute__((__vector_size__(32)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef __attribute__((address_space(3))) void lds_void;

__device__ __forceinline__ rsrc_t make_rsrc(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ i32x4_t ld128(rsrc_t r, uint32_t voff, uint32_t soff) {
  return __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)voff, (int)soff, 0));
}
// A copy of 64 x 16 bytes into LDS (lane l's to dst + 16 l); offsets past the buffer bring zeros.
__device__ __forceinline__ void copy16(rsrc_t r, char* dst, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)dst, 16, (int)voff, (int)soff, 0, 0);
}
__device__ __forceinline__ int swz(int row) { return (row & 7) ^ ((row >> 3) & 1); }
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
__device__ __forceinline__ void wait_lgkm0() { __builtin_amdgcn_s_waitcnt(0x3f | (7 << 4) | (0 << 8) | (3 << 14)); }
__device__ __forceinline__ void barrier_only() { asm volatile("s_barrier" ::: "memory"); }

// 16-bit operands: a sub-step is 16 elements, 16 bytes of a row to a lane.
template <int CD>
struct Half16 {
  static constexpr int SUB = 4, SETS = 2;
  typedef i32x4_t frag_t;
  __device__ static __forceinline__ frag_t read(const char* row, int ks, int h, int xr) {
    return *(const i32x4_t*)(row + (((2 * ks + h) ^ xr) << 4));
  }
  // acc += b a^T (the W-side fragment is the row operand: the block is accumulated transposed)
  __device__ static __forceinline__ void mma(f32x16_t& acc, const frag_t& b, const frag_t& a, int, int) {
    if constexpr (CD == CD_BF16)
      acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, b), __builtin_bit_cast(bf16x8_t, a), acc,
                                                    0, 0, 0);
    else
      acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, b), __builtin_bit_cast(f16x8_t, a), acc, 0,
                                                   0, 0);
  }
};

// Eight e4m3 codes as bf16.
__device__ __forceinline__ bf16x8_t e4m3_to_bf16(int lo, int hi) {
  bf16x8_t o;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int w = h ? hi : lo;
    const bf16x2_t p = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, false);
    const bf16x2_t q = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, true);
    o[4 * h] = p[0];
    o[4 * h + 1] = p[1];
    o[4 * h + 2] = q[0];
    o[4 * h + 3] = q[1];
  }
  return o;
}

// 8-bit floats: a sub-step is 64 codes, 32 bytes of a row to a lane, with the exponents of the
// rows' scales (sb, sa: their low bytes).
// The matrix instruction that scales each operand row aligns its products to the largest before it
// adds them and loses what lies about 2^-19 below it: sums are 1e-5 to 8e-5 (of their norm) off, far
// below the step of a 16-bit result but not of an fp32 one.  There (EXACT) codes are brought to
// bf16, which holds every e4m3 value, the bf16 instruction adds their products as fp32 sums do, and
// each sum takes both scales at once (their product alone may leave fp32's range).
template <bool EXACT>
struct Float8 {
  static constexpr int SUB = 2, SETS = 1;
  typedef i32x8_t frag_t;
  __device__ static __forceinline__ frag_t read(const char* row, int ks, int h, int xr) {
    const i32x4_t lo = *(const i32x4_t*)(row + (((4 * ks + 2 * h) ^ xr) << 4));
    const i32x4_t hi = *(const i32x4_t*)(row + (((4 * ks + 2 * h + 1) ^ xr) << 4));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  __device__ static __forceinline__ void mma(f32x16_t& acc, const frag_t& b, const frag_t& a, int sb, int sa) {
    if constexpr (!EXACT) {
      acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, acc, 0, 0, 0, sb, 0, sa);
    } else {
      f32x16_t part;
#pragma unroll
      for (int v = 0; v < 16; ++v) part[v] = 0.f;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        part = __builtin_amdgcn_mfma_f32_32x32x16_bf16(e4m3_to_bf16(b[2 * q], b[2 * q + 1]),
                                                       e4m3_to_bf16(a[2 * q], a[2 * q + 1]), part, 0, 0, 0);
      const int e = (sa & 255) + (sb & 255) - 254;
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[v] += __builtin_amdgcn_ldexpf(part[v], e);
    }
  }
};

template <int WMB_, int WNB_, int NWM_, int NWN_, int NS_>
struct Tile {
  static constexpr int WMB = WMB_, WNB = WNB_, NWM = NWM_, NWN = NWN_, NS = NS_;
  static constexpr int NW = NWM * NWN, TM = 32 * WMB * NWM, TN = 32 * WNB * NWN;
  static constexpr int STAGE = (TM + TN) * 128;  // LDS bytes of a stage
  static constexpr int PER_A = TM / 8 / NW;      // copies (8 rows each) of A rows per wave and stage (all waves copying)
  static constexpr int PER = (TM + TN) / 8 / NW;
  static_assert((TM / 8) % NW == 0 && (TN / 8) % NW == 0 && NW % 2 == 0, "copies split evenly");
  static constexpr int LDS = NS * STAGE;
};

template <class T>
using Acc = f32x16_t[T::WMB][T::WNB];

template <class T>
__device__ __forceinline__ void zero(Acc<T>& acc) {
#pragma unroll
  for (int i = 0; i < T::WMB; ++i)
#pragma unroll
    for (int j = 0; j < T::WNB; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
}

// The contraction over cp's KT stages.  cp.one(buffer, stage, i) issues copy i of a stage (past the
// last stage it brings zeros or nothing anyone reads); cp.begin(stage) is called when a stage's
// copies begin, cp.scales(stage, ..) when its first fragments are read and cp.shift(stage, ..) once the
// stage before is done (what scales() has read becomes the scales in use: no product waits for the
// read).  On entry stage 0 lies in LDS for every wave and the copies of stages 1 .. NS - 1 are requested;
// on return the LDS is free.
// Where fewer waves copy than multiply (C::WAVES: the largest tiles, one wave of each SIMD's two), the others keep the
// matrix pipe busy while the copies go out (all waves copying: the 8-bit product of 4096 x 14336 x 4096 222 us in
// place of 208; copies spread into the next stage's first products 211: they arrive later).
template <class T, class KIND, bool COPY, class C>
__device__ __forceinline__ void stages(Acc<T>& acc, char* lds, C& cp, int wave, int lane) {
  constexpr int WMB = T::WMB, WNB = T::WNB, NMF = WMB * WNB, SUB = KIND::SUB, SETS = KIND::SETS;
  // where in the last sub-step the barrier stands: before the first read of the next stage
  constexpr int BAR = SETS == 2 ? (C::WAVES < T::NW ? 2 : 0) : NMF < 4 ? 0 : NMF < 8 ? 1 : 2;
  static_assert(SETS == 2 || BAR < WMB, "the first fragment is replaced after the barrier");
  const int h = lane >> 5, r32 = lane & 31;
  const int wm = (wave / T::NWN) * 32 * WMB, wn = (wave % T::NWN) * 32 * WNB;
  const int xr = swz(r32);
  const int arow = (wm + r32) * 128, brow = (T::TM + wn + r32) * 128;
  typename KIND::frag_t fa[SETS][WMB], fb[SETS][WNB];
  int sa[2][WMB], sb[2];
  // fragment t of a sub-step: the b's, then the a's
  auto frag = [&](int set, const char* st, int ks, int t) {
    if (t < WNB) fb[set][t] = KIND::read(st + brow + t * 32 * 128, ks, h, xr);
    else fa[set][t - WNB] = KIND::read(st + arow + (t - WNB) * 32 * 128, ks, h, xr);
  };
#pragma unroll
  for (int t = 0; t < WMB + WNB; ++t) frag(0, lds, 0, t);
  cp.scales(0, sa[1], sb[1]);
  cp.shift(0, sa, sb);
  int buf = 0;
  for (int u = 0; u < cp.KT; ++u) {
    char* st = lds + buf * T::STAGE;
    const int nbuf = buf + 1 == T::NS ? 0 : buf + 1;
    char* nx = lds + nbuf * T::STAGE;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int ks = 0; ks < SUB; ++ks) {
      const int set = SETS == 2 ? ks & 1 : 0, next = SETS == 2 ? set ^ 1 : 0;
      const bool last = ks == SUB - 1;
      const char* from = last ? nx : st;
      const int nks = last ? 0 : ks + 1;
#pragma unroll
      for (int t = 0; t < NMF; ++t) {
        if (last && t == BAR) {
          wait_lgkm0();
          wait_vmcnt<(T::NS - 2) * C::PER>();  // this wave's copies of stage u + 1
          barrier_only();
          if (COPY) cp.begin(u + T::NS);
        }
        const int i = t % WMB, j = t / WMB;
        KIND::mma(acc[i][j], fb[set][j], fa[set][i], sb[0], sa[0][i]);
        if constexpr (SETS == 2) {
#pragma unroll
          for (int q = 0; q < WMB + WNB; ++q)
            if ((last ? BAR + q * (NMF - BAR) / (WMB + WNB) : q * NMF / (WMB + WNB)) == t) frag(next, from, nks, q);
        } else {
          if (i == WMB - 1) frag(0, from, nks, j);
          if (j == WNB - 1) frag(0, from, nks, WNB + i);
        }
        if (last && t == BAR) cp.scales(u + 1, sa[1], sb[1]);
        if (COPY && last && t >= BAR) {
#pragma unroll
          for (int q = 0; q < C::PER; ++q)
            if (BAR + q * (NMF - BAR) / C::PER == t) cp.one(st, u + T::NS, q);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    cp.shift(u + 1, sa, sb);
    buf = nbuf;
  }
}
template <class T, class KIND, class C>
__device__ __forceinline__ void contract(Acc<T>& acc, char* lds, C& cp, int wave, int lane) {
  if constexpr (C::WAVES < T::NW) {
    if (wave < C::WAVES) stages<T, KIND, true>(acc, lds, cp, wave, lane);
    else stages<T, KIND, false>(acc, lds, cp, wave, lane);
  } else {
    stages<T, KIND, true>(acc, lds, cp, wave, lane);
  }
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();  // every copy has ended and every wave is past its reads
}

// Position of workgroup b among n when each XCD (workgroups b, b + 8, ...) takes a
// contiguous run of positions, so that its L2 serves neighbouring tiles.
__device__ __forceinline__ int xcd_run(int b, int n) {
  const int q = n >> 3, rem = n & 7, x = b & 7;
  return x * q + min(x, rem) + (b >> 3);
}
// Tile t of an order that walks groups of four tile rows column by column.
__device__ __forceinline__ void grouped_tile(int t, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int per = 4 * tiles_n, g = t / per, u = t % per, gm = min(4, tiles_m - g * 4);
  tm = g * 4 + u % gm;
  tn = u / gm;
}

}  // namespace tile
}  // namespace qnf4
