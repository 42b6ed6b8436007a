// int8.hip -- matrix products in 8-bit integers with a scale per token and per output
// channel, dense and grouped by expert (the serving form of merged weights).
//
//   rows to 8 bits  s = fl32(max |x| / 127), c = round-half-even(fl32(x / s)) in [-127, 127]
//   product         y[i, j] = RNE_cd(s_i t_j sum_k c[i, k] d[j, k] + bias[j])
//
// The integer sum is exact in 32 bits (cols <= QLORA_INT8_MAX_COLS), so the result does
// not depend on how the contraction is cut or in which order its parts are added.
// Codes are stored in rows of QLORA_INT8_LD(cols) bytes, zero past the last column: a
// zero adds nothing, so every kernel reads whole 128-byte rows whatever cols is.
#include <algorithm>

#include "int8_distill.h"

namespace qnf4 {
namespace {

constexpr int kThreads = 256;
typedef int i32x4_t __attribute__((__vector_size__(16)));
typedef int i32x16_t __attribute__((__vector_size__(64)));

// ------------------------------------------------------------------ rows to 8 bits
// Code of x under scale s (s > 0): the quotient is rounded to binary32 first, then to
// the nearest integer, ties to even; the limit only acts where s is subnormal and its
// own rounding makes the largest quotient exceed 127.
__device__ __forceinline__ int code_of(float x, float s) {
  return (int)fminf(fmaxf(rintf(__fdiv_rn(x, s)), -127.f), 127.f);
}

// Scale of a row from the largest |x| as bits (the order of non-negative floats is the
// order of their bits, with infinity and every NaN above all numbers): NaN for a row
// that holds one of those, so that its outputs are NaN.
__device__ __forceinline__ float scale_of_bits(uint32_t amax) {
  return amax >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __fdiv_rn(__uint_as_float(amax), 127.f);
}

// ------------------------------------------------------------------------ routing
// Experts' rows for the product kernels, from the caller's offsets: expert e's rows end at
// the largest of offsets[0 .. e + 1], limited to [0, m], and begin where those of the expert
// before end, so no row belongs to two experts whatever the offsets hold; tiles[t] = {expert,
// first row, rows, 0} for each run of at most tile_m rows of one expert, in order, `count` of
// them (at most cap: m / tile_m whole runs and one partial run for each expert that has a
// row).
struct Route {
  int32_t* count;   // [1]
  int4* tiles;      // [cap]
  const int32_t* offsets;
  int experts, tile_m, cap;
  int64_t m;
};

// Tile i of expert e's n rows from `start` on.
__device__ __forceinline__ void put_tile(const Route& r, int at, int e, int start, int n, int i) {
  if (at < r.cap) r.tiles[at] = make_int4(e, start + i * r.tile_m, min(r.tile_m, n - i * r.tile_m), 0);
}
// By one wave: running maximum and running sum over 64 experts at a time.
__device__ __forceinline__ void route_experts(const Route& r) {
  const int32_t* offsets = r.offsets;
  const int experts = r.experts, tile_m = r.tile_m;
  const int64_t m = r.m;
  const int lane = threadIdx.x;
  int before = 0;  // where the rows of the chunk's first expert begin
  int at = 0;      // tiles so far
  {
    const int o = offsets[0];
    before = (int)min((int64_t)max(o, 0), m);
  }
  for (int e0 = 0; e0 < experts; e0 += 64) {
    const int e = e0 + lane;
    int end = before;
    if (e < experts) end = (int)min((int64_t)max(offsets[e + 1], 0), m);
    end = max(end, before);
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int v = __shfl_up(end, off, 64);
      if (lane >= off) end = max(end, v);
    }
    int start = __shfl_up(end, 1, 64);
    if (lane == 0) start = before;
    const int n = end - start, t = (int)(((uint32_t)n + (uint32_t)tile_m - 1u) / (uint32_t)tile_m);
    int sum = t;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int v = __shfl_up(sum, off, 64);
      if (lane >= off) sum += v;
    }
    if (e < experts) {
      const int first = at + sum - t;
      if (t <= 4)  // most experts have a few tiles: each lane writes its own
        for (int i = 0; i < t; ++i) put_tile(r, first + i, e, start, n, i);
    }
    // the others by the whole wave
    for (uint64_t many = __ballot(e < experts && t > 4); many; many &= many - 1) {
      const int l = (int)__builtin_ctzll(many);
      const int le = e0 + l, ls = __shfl(start, l, 64), ln = __shfl(n, l, 64), lt = __shfl(t, l, 64);
      const int lf = at + __shfl(sum, l, 64) - lt;
      for (int i = lane; i < lt; i += 64) put_tile(r, lf + i, le, ls, ln, i);
    }
    before = __shfl(end, 63, 64);
    at += __shfl(sum, 63, 64);
  }
  if (lane == 0) *r.count = min(at, r.cap);
}

// 16 bytes at any element-aligned address: the memory system takes unaligned vectors (rows of
// odd length start anywhere; element by element a row of 3411 f16 took twice the time).
template <int ES>
struct __attribute__((packed, aligned(ES))) Chunk {
  u32x4_t v;
};

// 8 consecutive elements of a row from column k on.
template <int CD>
__device__ __forceinline__ void load8(const void* x, int64_t at, float (&v)[8]) {
  if constexpr (CD == CD_F32) {
    const u32x4_t a = ((const Chunk<4>*)((const float*)x + at))->v;
    const u32x4_t b = ((const Chunk<4>*)((const float*)x + at + 4))->v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = __uint_as_float(a[e]);
      v[4 + e] = __uint_as_float(b[e]);
    }
  } else {
    const u32x4_t a = ((const Chunk<2>*)((const uint16_t*)x + at))->v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = from_cd16<CD>((uint16_t)(a[e >> 1] >> (16 * (e & 1))));
  }
}

__device__ __forceinline__ uint32_t amax8(const float (&v)[8], uint32_t m) {
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
  return m;
}

// Eight codes without a division: with r = RN(1 / s), two steps q <- q + (x - q s) r, each a
// remainder that is exact in one fused multiply-add, turn x r into the correctly rounded
// quotient (P. Markstein's theorem on division by fused multiply-add, 1990: a correctly rounded
// reciprocal and a quotient within one ulp give it in one step; the first brings the quotient
// there).  The sum with 1.5 * 2^23 then rounds to the nearest integer, ties to even, and
// leaves the code in the low byte.  Ties are common in 16-bit rows (half the largest value has
// the quotient 63.5), so nothing that treats them apart is cheap: 4096 x 4096 bf16 takes
// 18.6 us with divisions, 16.7 with divisions only near ties, 11.5 so.
// A row with a scale below 2^-100, whose remainders might not be exact, is divided (r is NaN).
__device__ __forceinline__ float scale_rcp(float s) {
  return s >= 0x1p-100f ? __fdiv_rn(1.0f, s) : __uint_as_float(0x7fc00000u);
}
__device__ __forceinline__ u32x2_t pack_codes(const uint32_t (&t)[8]) {
  u32x2_t o;
#pragma unroll
  for (int e = 0; e < 8; e += 4)
    o[e >> 2] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(t[e + 3], t[e + 2], 0x0c0c0400u),
                                      __builtin_amdgcn_perm(t[e + 1], t[e], 0x0c0c0400u), 0x05040100u);
  return o;
}
__device__ __forceinline__ u32x2_t codes8(const float (&v)[8], float s, float r) {
  uint32_t t[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float q = v[e] * r;
    q = fmaf(fmaf(-q, s, v[e]), r, q);
    q = fmaf(fmaf(-q, s, v[e]), r, q);
    t[e] = __float_as_uint(q + 12582912.f);
  }
  return pack_codes(t);
}
__device__ __forceinline__ u32x2_t codes8_by_division(const float (&v)[8], float s) {
  uint32_t t[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) t[e] = s > 0.f ? (uint32_t)code_of(v[e], s) : 0u;
  return pack_codes(t);
}

// Codes and scales of rows, TPR threads to a row.  The row stays in registers between the
// maximum and the codes (up to HOLD groups of 8 elements per thread; the rest is read again,
// from the caches).  The columns past the last whole group go one to a thread.  Most threads
// run this code once, so its size counts as its registers do: held groups are unrolled.
// The workgroup after the last row forms the experts' route (r.offsets set), so that it costs
// no launch of its own.
template <int CD, int TPR, int HOLD>
__global__ __launch_bounds__(kThreads) void k_int8_rows(const void* __restrict__ x, int64_t ldx, int64_t rows,
                                                        int cols, int ld, int8_t* __restrict__ codes,
                                                        float* __restrict__ scale, Route r) {
  __shared__ uint32_t red[kThreads / 64];
  const int64_t row = (int64_t)blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
  if (r.offsets && blockIdx.x == gridDim.x - 1) {
    if (threadIdx.x < 64) route_experts(r);
    return;
  }
  const int t = threadIdx.x % TPR;
  const bool live = row < rows;
  const int64_t at = row * ldx;
  const int groups = cols / 8, rest = cols % 8;
  float v[HOLD][8], last = 0.f;
  uint32_t amax = 0;
  if (live) {
#pragma unroll
    for (int i = 0; i < HOLD; ++i)
      if (t + i * TPR < groups) load8<CD>(x, at + 8 * (t + i * TPR), v[i]);
    if (t < rest) last = load_cd<CD>(x, at + 8 * groups + t);
#pragma unroll
    for (int i = 0; i < HOLD; ++i)
      if (t + i * TPR < groups) amax = amax8(v[i], amax);
#pragma unroll 1
    for (int g = t + HOLD * TPR; g < groups; g += TPR) {
      float w[8];
      load8<CD>(x, at + 8 * g, w);
      amax = amax8(w, amax);
    }
    amax = max(amax, __float_as_uint(last) & 0x7fffffffu);
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) amax = max(amax, (uint32_t)__shfl_xor((int)amax, off, 64));
  if constexpr (TPR > 64) {
    static_assert(TPR == kThreads, "one row per wave or per workgroup");
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = amax;
    __syncthreads();
    amax = max(max(red[0], red[1]), max(red[2], red[3]));
  }
  if (!live) return;
  const float s = scale_of_bits(amax), rcp = scale_rcp(s);
  if (t == 0) scale[row] = s;
  int8_t* dst = codes + row * ld;
  if (rcp == rcp) {
#pragma unroll
    for (int i = 0; i < HOLD; ++i)
      if (t + i * TPR < groups) *(u32x2_t*)(dst + 8 * (t + i * TPR)) = codes8(v[i], s, rcp);
  }
  // the groups that were not held; all of them, divided, under a scale near zero (or no number)
#pragma unroll 1
  for (int g = rcp == rcp ? t + HOLD * TPR : t; g < groups; g += TPR) {
    float w[8];
    load8<CD>(x, at + 8 * g, w);
    u32x2_t o;
    if (rcp == rcp) o = codes8(w, s, rcp);
    else o = codes8_by_division(w, s);
    *(u32x2_t*)(dst + 8 * g) = o;
  }
  if (t < 8 && 8 * groups + t < ld) dst[8 * groups + t] = (int8_t)(t < rest && s > 0.f ? code_of(last, s) : 0);
  for (int z = groups + 1 + t; z < ld / 8; z += TPR) *(u32x2_t*)(dst + 8 * z) = u32x2_t{0u, 0u};
}

// ------------------------------------------------------------------------- product
struct I8 {
  const int8_t* a;   // [m][ld] codes of the tokens
  const float* sa;   // [m]
  const int8_t* b;   // [experts][n][ld] codes of the weights
  const float* sb;   // [experts][n]
  const void* bias;  // [experts][n] cd or null
  void* y;           // [m][n] cd
  int64_t m, n, ld;
  const int32_t* count;  // grouped by expert: tiles[0 .. *count), else null
  const int4* tiles;
  int* part;         // contraction cut into `split` slices: their sums, tile by tile
  int split;
};

// y from the sum, before it is rounded into its type: fl32(fl32(fl32(sum) s) t + bias), the second
// product and the bias in one step.  Every kernel forms y by this, and an f16 value is rounded to
// fp32 first in all of them: left alone, the compiler fuses the step with the conversion where a
// value is converted by itself (one rounding) and not where two are packed (two), and a token's y
// would differ by an f16 step from one batch size to another.
// FAR: the token's scale may be so large (2^96: the sum is below 2^31) that its product with the
// sum leaves fp32's range while y need not; such a token's sum takes the channel's scale first.
// (A small sum times a scale near zero loses nothing: the product of an integer and a subnormal
// number is exact as long as it is subnormal.)
constexpr float kFarScale = 0x1p96f;
template <int CD, bool FAR = true>
__device__ __forceinline__ float scaled(int sum, float sa, float sb, float bv) {
  const bool far = FAR && sa >= kFarScale;
  float v = fmaf((float)sum * (far ? sb : sa), far ? sa : sb, bv);
  if constexpr (CD == CD_F16) asm("" : "+v"(v));
  return v;
}
template <int CD>
__device__ __forceinline__ void store_y(const I8& p, int64_t row, int64_t col, int sum, float sa, float sb, float bv) {
  store_cd<CD>(p.y, row * p.n + col, scaled<CD>(sum, sa, sb, bv));
}

// ---------------------------------------------------------------- tiled product
// A workgroup forms a TM x TN tile of y: NWM x NWN waves, each with WMB x WNB blocks of
// the 32 x 32 x 32 matrix instruction.  The contraction advances 128 bytes per stage;
// a stage's operands lie in LDS as rows of 128 bytes [TM token rows | TN weight rows],
// 16-byte chunk c of row r at chunk c ^ swz(r) (one chunk of 16 consecutive rows then
// touches every bank group once), copied from global memory without passing through
// registers.  NS stages are in flight or in use.
//
// Stage u is four sub-steps of 32 contraction elements.  The fragments of a sub-step are
// read while the one before multiplies, across stages too: one barrier per stage, before
// the last sub-step, is where stage u + 1 has landed and every wave has its last
// fragments of stage u, so that during the last sub-step the wave reads the first
// fragments of stage u + 1 and the copies of stage u + NS into stage u's buffer begin.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef __attribute__((address_space(3))) void lds_void;

__device__ __forceinline__ rsrc_t make_rsrc(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ i32x4_t ld128(rsrc_t r, uint32_t voff, uint32_t soff) {
  return __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)voff, (int)soff, 0));
}
__device__ __forceinline__ int swz(int row) { return (row & 7) ^ ((row >> 3) & 1); }
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
__device__ __forceinline__ void wait_lgkm0() { __builtin_amdgcn_s_waitcnt(0x3f | (7 << 4) | (0 << 8) | (3 << 14)); }
__device__ __forceinline__ void barrier_only() { asm volatile("s_barrier" ::: "memory"); }

template <int WMB_, int WNB_, int NWM_, int NWN_, int NS_>
struct Tile {
  static constexpr int WMB = WMB_, WNB = WNB_, NWM = NWM_, NWN = NWN_, NS = NS_;
  static constexpr int NW = NWM * NWN, TM = 32 * WMB * NWM, TN = 32 * WNB * NWN;
  static constexpr int STAGE = (TM + TN) * 128;         // LDS bytes of a stage
  static constexpr int PER = (TM + TN) / 8 / NW;        // copies (8 rows each) per wave and stage
  static constexpr int PER_A = TM / 8 / NW;             // the first of them fetch token rows
  static_assert((TM / 8) % NW == 0 && (TN / 8) % NW == 0 && NW % 2 == 0, "copies split evenly");
  static constexpr int LDS = NS * STAGE;
  static constexpr int COEF = 2 * TN + TM;              // scales and biases of the columns, scales of the rows
};

// Where a tile lies: expert, first token row, token rows, first column.
struct Place {
  int e, rows;
  int64_t m0, n0;
};

// The copies of a tile's stages by one wave: instruction i of wave w fills LDS rows
// 8 (w + NW i) .. + 7 of the stage; lane l lands in chunk l % 8 of row l / 8 and fetches the
// logical chunk that lies there.
template <class T>
struct Copies {
  const int8_t *a, *b;
  int64_t abytes, bbytes;
  uint32_t off, step;
  int KT, wave;
  __device__ __forceinline__ Copies(const I8& p, const Place& t, int wave_, int lane) : wave(wave_) {
    const int ncols = (int)min((int64_t)T::TN, p.n - t.n0), ld = (int)p.ld;
    a = p.a + t.m0 * p.ld;
    b = p.b + ((int64_t)t.e * p.n + t.n0) * p.ld;
    abytes = (int64_t)t.rows * p.ld;
    bbytes = (int64_t)ncols * p.ld;
    const int row = 8 * wave + (lane >> 3);
    off = (uint32_t)(row * ld + (((lane & 7) ^ swz(row)) << 4));
    step = (uint32_t)(8 * T::NW * ld);
    KT = ld >> 7;
  }
  // only stages k0 .. k1 - 1 of the contraction
  __device__ __forceinline__ void cut(int k0, int k1) {
    a += (int64_t)k0 * 128;
    b += (int64_t)k0 * 128;
    abytes -= (int64_t)k0 * 128;
    bbytes -= (int64_t)k0 * 128;
    KT = k1 - k0;
  }
  __device__ __forceinline__ void one(char* stage_lds, int stage, int i) const {
    // past the last stage: an empty buffer, nothing is fetched
    const bool in = stage < KT, a_side = i < T::PER_A;
    const rsrc_t r = a_side ? make_rsrc(a, in ? abytes : 0) : make_rsrc(b, in ? bbytes : 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(stage_lds + (wave + T::NW * i) * 1024), 16,
                                             (int)(off + (a_side ? i : i - T::PER_A) * step), stage * 128, 0, 0);
  }
  __device__ __forceinline__ void all(char* stage_lds, int stage) const {
#pragma unroll
    for (int i = 0; i < T::PER; ++i) one(stage_lds, stage, i);
  }
};

template <class T>
using Acc = i32x16_t[T::WMB][T::WNB];

// The contraction.  On entry stage 0 lies in LDS for every wave and the copies of stages
// 1 .. NS - 1 are requested; on return the LDS is free.
template <class T>
__device__ __forceinline__ void contract(Acc<T>& acc, char* lds, const Copies<T>& cp, int lane) {
  constexpr int WMB = T::WMB, WNB = T::WNB, NMF = WMB * WNB, NRD = WMB + WNB;
  const int h = lane >> 5, r32 = lane & 31;
  const int wm = (cp.wave / T::NWN) * 32 * WMB, wn = (cp.wave % T::NWN) * 32 * WNB;
#pragma unroll
  for (int i = 0; i < WMB; ++i)
#pragma unroll
    for (int j = 0; j < WNB; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
  const int xr = swz(r32);
  const int arow = (wm + r32) * 128, brow = (T::TM + wn + r32) * 128;
  i32x4_t fa[2][WMB], fb[2][WNB];
  // the t-th fragment of a sub-step in the order of first use: a0, the b's, the other a's
  auto frag = [&](int set, const char* st, int ks, int t) {
    const int c = ((2 * ks + h) ^ xr) << 4;
    if (t == 0) fa[set][0] = *(const i32x4_t*)(st + arow + c);
    else if (t <= WNB) fb[set][t - 1] = *(const i32x4_t*)(st + brow + (t - 1) * 32 * 128 + c);
    else fa[set][t - WNB] = *(const i32x4_t*)(st + arow + (t - WNB) * 32 * 128 + c);
  };
#pragma unroll
  for (int t = 0; t < NRD; ++t) frag(0, lds, 0, t);
  int buf = 0;
  for (int u = 0; u < cp.KT; ++u) {
    char* st = lds + buf * T::STAGE;
    const int nbuf = buf + 1 == T::NS ? 0 : buf + 1;
    const char* nx = lds + nbuf * T::STAGE;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      const int set = ks & 1;
      if (ks == 3) {
        wait_lgkm0();
        wait_vmcnt<(T::NS - 2) * T::PER>();  // this wave's copies of stage u + 1
        barrier_only();
      }
#pragma unroll
      for (int t = 0; t < NMF; ++t) {
        const int i = t / WNB, j = t % WNB;
        // the weight fragment is the row operand: the block is accumulated transposed
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[set][j], fa[set][i], acc[i][j], 0, 0, 0);
#pragma unroll
        for (int q = 0; q < NRD; ++q)
          if (q * NMF / NRD == t) frag(set ^ 1, ks == 3 ? nx : st, ks == 3 ? 0 : ks + 1, q);
        if (ks == 3) {
#pragma unroll
          for (int q = 0; q < T::PER; ++q)
            if (q * NMF / T::PER == t) cp.one(st, u + T::NS, q);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    buf = nbuf;
  }
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();  // every copy has ended and every wave is past its reads
}

// The tile's scales and biases, value i of T::COEF.
template <int CD, class T>
__device__ __forceinline__ float coefficient(const I8& p, const Place& t, int i) {
  const int64_t wrow = (int64_t)t.e * p.n + t.n0;
  if (i < T::TN) return t.n0 + i < p.n ? p.sb[wrow + i] : 0.f;
  if (i < 2 * T::TN) return p.bias && t.n0 + i - T::TN < p.n ? load_cd<CD>(p.bias, wrow + i - T::TN) : 0.f;
  return i - 2 * T::TN < t.rows ? p.sa[t.m0 + i - 2 * T::TN] : 0.f;
}

// Lane (r32, h) of block (i, j) holds row 32 i + r32, columns 32 j + 8 q + 4 h + v of the
// wave's part in elements 4 q + v.  32 rows at a time go through the wave's own LDS W (16-byte
// chunk c of a row at chunk c ^ row) and leave as 16-byte chunks of whole rows, at whatever
// address y's rows start (element by element, odd row lengths took three times as long).
// Every wave issues exactly stores() of these (chunks past the tile's rows and whole chunks of
// columns fall outside their buffer), so a caller can count past them; the columns past the
// last whole chunk, and rows too long for a buffer, go element by element, and the wave
// waits for those.
template <int CD, class T>
struct Writer {
  static constexpr int ES = CD == CD_F32 ? 4 : 2, RB = 32 * T::WNB * ES, NC = RB / 16, PC = 16 / ES;
  static constexpr int stores() { return T::WMB * NC / 2; }
  __device__ static __forceinline__ void run(const I8& p, const Place& pl, const Acc<T>& acc, const float* coef, char* W,
                                             int wave, int lane) {
    // far tokens (no f16 value is one) have code of their own: selecting the order for every
    // element would cost the others two instructions each
    bool far = false;
    if constexpr (CD != CD_F16) {
#pragma unroll
      for (int i = 0; i < T::WMB; ++i)
        far |= coef[2 * T::TN + (wave / T::NWN) * 32 * T::WMB + 32 * i + (lane & 31)] >= kFarScale;
      far = __any(far);
    }
    if (far) rows<true>(p, pl, acc, coef, W, wave, lane);
    else rows<false>(p, pl, acc, coef, W, wave, lane);
  }
  template <bool FAR>
  __device__ static __forceinline__ void rows(const I8& p, const Place& pl, const Acc<T>& acc, const float* coef, char* W,
                                              int wave, int lane) {
    constexpr int WMB = T::WMB, WNB = T::WNB;
    const int h = lane >> 5, r32 = lane & 31;
    const int wm = (wave / T::NWN) * 32 * WMB, wn = (wave % T::NWN) * 32 * WNB;
    // the wave's columns that exist, and those of them in whole chunks
    const int ncols = (int)max((int64_t)0, min((int64_t)(32 * WNB), p.n - pl.n0 - wn));
    const int whole = p.n * ES < (1 << 26) ? ncols / PC * PC : 0;
    const bool lines = (p.n * ES) % 128 == 0 && ((uintptr_t)p.y & 127) == 0;  // whole lines are written at once
#pragma unroll
    for (int i = 0; i < WMB; ++i) {
      const float sa = coef[2 * T::TN + wm + 32 * i + r32];
#pragma unroll
      for (int j = 0; j < WNB; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c0 = wn + 32 * j + 8 * q + 4 * h;
          const f32x4_t sb = *(const f32x4_t*)(coef + c0), bv = *(const f32x4_t*)(coef + T::TN + c0);
          float v[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) v[x] = scaled<CD, FAR>(acc[i][j][4 * q + x], sa, sb[x], bv[x]);
          if constexpr (ES == 4) {
            const f32x4_t o = {v[0], v[1], v[2], v[3]};
            *(f32x4_t*)(W + r32 * RB + (((8 * j + 2 * q + h) ^ (r32 & (NC - 1))) << 4)) = o;
          } else {
            const u32x2_t o = {pack2<CD>(v[0], v[1]), pack2<CD>(v[2], v[3])};
            *(u32x2_t*)(W + r32 * RB + (((4 * j + q) ^ (r32 & (NC - 1))) << 4) + 8 * h) = o;
          }
        }
      wait_lgkm0();  // the wave reads back only what it wrote
      asm volatile("" ::: "memory");
      const int row0 = wm + 32 * i, left = min(32, pl.rows - row0);  // rows of the tile in these 32
      const int64_t at0 = (pl.m0 + row0) * p.n + pl.n0 + wn;
      const int c = lane & (NC - 1);
      // up to the end of the last row's whole chunks; other chunks past `whole` are masked
      const rsrc_t r = make_rsrc((char*)p.y + at0 * ES, left > 0 && whole > 0 ? ((left - 1) * p.n + whole) * ES : 0);
      const uint32_t none = c * PC < whole ? 0u : 1u << 31;
#pragma unroll
      for (int it = 0; it < NC / 2; ++it) {
        const int m = (64 / NC) * it + lane / NC;
        const u32x4_t v = *(const u32x4_t*)(W + m * RB + ((c ^ (m & (NC - 1))) << 4));
        const uint32_t off = (uint32_t)(m * (int)p.n * ES + c * 16);
        const int at = (int)((m < left ? off : 1u << 31) | none);
        if (lines) __builtin_amdgcn_raw_buffer_store_b128(v, r, at, 0, 2);
        else __builtin_amdgcn_raw_buffer_store_b128(v, r, at, 0, 0);
      }
      const int rest = ncols - whole;
      for (int q = lane; q < 32 * rest; q += 64) {
        const int m = q / rest, cc = whole + q % rest;
        const int byte = m * RB + (((cc / PC) ^ (m & (NC - 1))) << 4) + (cc % PC) * ES;
        if (m < left) {
          const int64_t at = at0 + (int64_t)m * p.n + cc;
          if constexpr (ES == 4) ((uint32_t*)p.y)[at] = *(const uint32_t*)(W + byte);
          else ((uint16_t*)p.y)[at] = *(const uint16_t*)(W + byte);
        }
      }
      wait_lgkm0();  // the reads are done before the next 32 rows overwrite them
      asm volatile("" ::: "memory");
    }
    if (ncols != whole) wait_vmcnt<0>();
  }
};

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
template <class T>
__device__ __forceinline__ int tile_rows_of(const I8& p) {
  return p.count ? __builtin_amdgcn_readfirstlane(*p.count) : (int)((p.m + T::TM - 1) / T::TM);
}
template <class T>
__device__ __forceinline__ Place place_of(const I8& p, int t, int tiles_m, int tiles_n) {
  int tm, tn;
  grouped_tile(t, tiles_m, tiles_n, tm, tn);
  tm = __builtin_amdgcn_readfirstlane(tm);
  tn = __builtin_amdgcn_readfirstlane(tn);
  Place pl;
  pl.n0 = (int64_t)tn * T::TN;
  if (p.count) {
    const int4 r = p.tiles[tm];
    pl.e = __builtin_amdgcn_readfirstlane(r.x);
    pl.m0 = __builtin_amdgcn_readfirstlane(r.y);
    pl.rows = __builtin_amdgcn_readfirstlane(r.z);
  } else {
    pl.e = 0;
    pl.m0 = (int64_t)tm * T::TM;
    pl.rows = (int)min((int64_t)T::TM, p.m - pl.m0);
  }
  return pl;
}

// One tile to a workgroup; several workgroups share a compute unit.
// SPLIT: p.split workgroups to a tile, each a slice of the contraction; the sums go to p.part
// as [slice][tile][TM][TN] and k_int8_join adds them (exactly, so in any order).
template <int CD, class T, int WGS, bool SPLIT = false>
__global__ __launch_bounds__(64 * T::NW, WGS) void k_int8_tile(I8 p) {
  // One array for everything: with several, the compiler tells them apart and then waits for
  // every copy in flight before each fragment it reads (228 -> 324 us on the long prompt).
  __shared__ __attribute__((aligned(1024))) char lds[T::LDS + T::COEF * 4];
  float* coef = (float*)(lds + T::LDS);
  const int tiles_n = (int)((p.n + T::TN - 1) / T::TN), tiles_m = tile_rows_of<T>(p), total = tiles_m * tiles_n;
  int b = blockIdx.x, slice = 0;
  if (SPLIT) {
    slice = b % p.split;
    b /= p.split;
  }
  if (b >= total) return;
  const int t = SPLIT ? b : xcd_run(b, total);
  const Place pl = place_of<T>(p, t, tiles_m, tiles_n);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  Copies<T> cp(p, pl, wave, lane);
  if (SPLIT) cp.cut(slice * cp.KT / p.split, (slice + 1) * cp.KT / p.split);
  // the coefficients are requested first and stored once the copies are on their way
  constexpr int NC = SPLIT ? 0 : (T::COEF + 64 * T::NW - 1) / (64 * T::NW);
  float c[NC > 0 ? NC : 1];
#pragma unroll
  for (int i = 0; i < NC; ++i)
    c[i] = tid + i * 64 * T::NW < T::COEF ? coefficient<CD, T>(p, pl, tid + i * 64 * T::NW) : 0.f;
#pragma unroll
  for (int s = 0; s < T::NS; ++s) cp.all(lds + s * T::STAGE, s);
#pragma unroll
  for (int i = 0; i < NC; ++i)
    if (tid + i * 64 * T::NW < T::COEF) coef[tid + i * 64 * T::NW] = c[i];
  wait_vmcnt<(T::NS - 1) * T::PER>();
  wait_lgkm0();
  barrier_only();
  Acc<T> acc;
  contract<T>(acc, lds, cp, lane);
  if constexpr (SPLIT) {
    int* dst = p.part + ((int64_t)slice * total + t) * (T::TM * T::TN);
    const int wm = (wave / T::NWN) * 32 * T::WMB, wn = (wave % T::NWN) * 32 * T::WNB;
#pragma unroll
    for (int i = 0; i < T::WMB; ++i)
#pragma unroll
      for (int j = 0; j < T::WNB; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const i32x4_t v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
          *(i32x4_t*)(dst + (wm + 32 * i + (lane & 31)) * T::TN + wn + 32 * j + 8 * q + 4 * (lane >> 5)) = v;
        }
  } else {
    Writer<CD, T>::run(p, pl, acc, coef, lds + wave * 32 * Writer<CD, T>::RB, wave, lane);
  }
}

// y from the slices' sums: four columns of a row to a thread.
template <int CD, class T>
__global__ __launch_bounds__(kThreads) void k_int8_join(I8 p) {
  const int tiles_n = (int)((p.n + T::TN - 1) / T::TN), tiles_m = tile_rows_of<T>(p), total = tiles_m * tiles_n;
  const int t = blockIdx.x;
  if (t >= total) return;
  const Place pl = place_of<T>(p, t, tiles_m, tiles_n);
  const int at = 4 * (blockIdx.y * kThreads + threadIdx.x), row = at / T::TN, col = at % T::TN;
  if (row >= pl.rows || pl.n0 + col >= p.n) return;
  const int* src = p.part + (int64_t)t * (T::TM * T::TN) + at;
  i32x4_t sum = {0, 0, 0, 0};
#pragma unroll 4
  for (int s = 0; s < p.split; ++s) sum = sum + *(const i32x4_t*)(src + (int64_t)s * total * (T::TM * T::TN));
  const int64_t wrow = (int64_t)pl.e * p.n + pl.n0 + col;
  const float sa = p.sa[pl.m0 + row];
#pragma unroll
  for (int x = 0; x < 4; ++x)
    if (pl.n0 + col + x < p.n)
      store_y<CD>(p, pl.m0 + row, pl.n0 + col + x, sum[x], sa, p.sb[wrow + x],
                  p.bias ? load_cd<CD>(p.bias, wrow + x) : 0.f);
}

using Full = Tile<4, 2, 2, 4, 2>;  // 256 x 256, eight waves
using Half = Tile<2, 2, 2, 4, 2>;  // 128 x 256, eight waves
using Wide = Tile<2, 2, 2, 4, 3>;  // 128 x 256, eight waves
using Mid = Tile<2, 2, 2, 2, 4>;   // 128 x 128, four waves
// Two workgroups of these fit a compute unit.  Experts of few rows use that (several rounds); a
// dense call takes them where one round holds all tiles, one to a compute unit.
using Low = Tile<1, 2, 2, 2, 3>;   // 64 x 128, four waves
using Small = Tile<1, 1, 2, 2, 4>;  // 64 x 64, four waves

// Whole rounds of 256 x 256 tiles, a workgroup to a compute unit going through its tiles.
// After a tile's last stage the copies of the next tile's first stage are requested, so
// that they land while the tile's y is scaled and stored (both together took 9 to 14 of 60 us
// per tile of 4096 columns when each tile waited for itself).  A tile of at most 128 rows,
// and a last round of at most half the compute units (cut into halves of 128 rows then, two
// workgroups to a tile), run as 128 x 256.
template <int CD>
__global__ __launch_bounds__(512, 1) void k_int8_full(I8 p) {
  constexpr int kStaging = Full::STAGE;  // y passes through what was stage 1
  static_assert(kStaging + 8 * 32 * Writer<CD, Full>::RB <= Full::LDS, "staging fits");
  __shared__ __attribute__((aligned(1024))) char lds[Full::LDS + 2 * Full::COEF * 4];  // one array, as above
  float* coefs = (float*)(lds + Full::LDS);  // two sets, used in turn
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int b = blockIdx.x, G = gridDim.x;
  const int tiles_n = (int)((p.n + Full::TN - 1) / Full::TN), tiles_m = tile_rows_of<Full>(p);
  const int total = tiles_m * tiles_n;
  // The workgroup's tile in round r; rows 0: none (any more).
  auto item = [&](int r) {
    Place pl = {0, 0, 0, 0};
    const int64_t base = (int64_t)r * G;
    if (base >= total) return pl;
    const int rem = total - (int)base;
    if (rem < G && 2 * rem <= G) {
      if (b >= 2 * rem) return pl;
      const int pos = xcd_run(b, 2 * rem), half = pos & 1;
      pl = place_of<Full>(p, (int)base + (pos >> 1), tiles_m, tiles_n);
      pl.m0 += half * Half::TM;
      pl.rows = half ? max(0, pl.rows - Half::TM) : min(pl.rows, Half::TM);
    } else {
      const int n = min(G, rem);
      if (b < n) pl = place_of<Full>(p, (int)base + xcd_run(b, n), tiles_m, tiles_n);
    }
    return pl;
  };
  // value i (of the thread's) among a tile's coefficients: columns at 0 and 256, rows at 512
  auto coef_of = [&](const Place& pl, int i) {
    return pl.rows > Half::TM ? coefficient<CD, Full>(p, pl, i)
                              : i < Half::COEF ? coefficient<CD, Half>(p, pl, i) : 0.f;
  };
  static_assert(Full::COEF <= 2 * 512 && Half::TN == Full::TN, "two coefficients to a thread");
  auto first_stage = [&](const Place& pl) {
    if (pl.rows > Half::TM) Copies<Full>(p, pl, wave, lane).all(lds, 0);
    else Copies<Half>(p, pl, wave, lane).all(lds, 0);
  };

  Place cur = item(0);
  if (cur.rows == 0) return;
  for (int i = tid; i < Full::COEF; i += 512) coefs[i] = coef_of(cur, i);
  first_stage(cur);
  wait_vmcnt<0>();
  int set = 0;
  for (int r = 1;; ++r) {
    const Place nxt = item(r);
    float c0 = 0.f, c1 = 0.f;  // the next tile's coefficients arrive during this one's contraction
    if (nxt.rows) {
      c0 = coef_of(nxt, tid);
      if (tid + 512 < Full::COEF) c1 = coef_of(nxt, tid + 512);
    }
    wait_lgkm0();
    barrier_only();  // stage 0 and the coefficients are there, the staging of the tile before is free
    // Between here and the next tile's first stage: contract, hand over, write.
    auto work = [&](auto shape) {
      using T = decltype(shape);
      const Copies<T> cp(p, cur, wave, lane);
      cp.all(lds + T::STAGE, 1);
      Acc<T> acc;
      contract<T>(acc, lds, cp, lane);
      if (nxt.rows) {
        float* to = coefs + (set ^ 1) * Full::COEF;
        to[tid] = c0;
        if (tid + 512 < Full::COEF) to[tid + 512] = c1;
        first_stage(nxt);
      }
      Writer<CD, T>::run(p, cur, acc, coefs + set * Full::COEF, lds + kStaging + wave * 32 * Writer<CD, T>::RB, wave, lane);
      asm volatile("" ::: "memory");
      // this wave's copies of the next first stage, older than the stores, have landed
      wait_vmcnt<Writer<CD, T>::stores()>();
    };
    if (cur.rows > Half::TM) work(Full{});
    else work(Half{});
    if (nxt.rows == 0) return;
    cur = nxt;
    set ^= 1;
  }
}

// ------------------------------------------------------------- a few tokens (decode)
// At up to 16 tokens per expert the product reads each weight once and does little else:
// a workgroup of NWV waves takes 16 RB weight rows of one expert over the whole contraction,
// the waves dealing out 128-byte lines of it.  Codes go from global memory straight into the
// 16 x 16 x 64 matrix instruction (lane l: row l % 16, 16 bytes l / 16 of a 64-byte piece),
// weight rows as one operand and tokens as the other; 16 pieces of weights per lane are
// requested before the first product.  The waves' sums meet in LDS.
// More than 16 tokens of an expert: the workgroup goes over its weight rows again for
// each 16 of them (from the caches).
// FUSE (one token of one matrix): the workgroup brings the token to 8 bits itself, which spares
// the call a launch (4096 x 4096: 7.4 against 9.6 us; with two tokens the repeated work already
// costs more than the launch: 11.2 against 9.9).  The first weights are requested before the
// token and loads return in order, so the codes are formed once those weights have arrived.
constexpr int kFuseBytes = 32768;  // codes of the token in LDS at most
constexpr int64_t kFewBlocks = 1 << 22;  // workgroups along x; the weight's other rows along z

// Source of a call's token when it is not in 8 bits yet.
struct Raw {
  const void* x;
  int64_t cols;
};

template <int CD, int RB, int NWV, bool FUSE>
__global__ __launch_bounds__(64 * NWV) void k_int8_few(I8 p, const int32_t* __restrict__ count,
                                                       const int4* __restrict__ runs, Raw raw) {
  constexpr int U = 8 / RB;  // lines per batch of loads and wave
  constexpr int NT = 64 * NWV;
  __shared__ int red[NWV][16][16 * RB + 1];
  __shared__ __attribute__((aligned(16))) char tok[FUSE ? kFuseBytes + 16 : 16];
  __shared__ uint32_t tmax[NWV];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int e = 0;
  int64_t first = 0, end = p.m;
  if (count) {
    // both requested at once: past the count, a run is read (there is room for it) but not used
    const int live = *count;
    const int4 run = runs[blockIdx.y];
    e = __builtin_amdgcn_readfirstlane(run.x);
    first = __builtin_amdgcn_readfirstlane(run.y);
    end = first + __builtin_amdgcn_readfirstlane(run.z);
    if ((int)blockIdx.y >= __builtin_amdgcn_readfirstlane(live)) return;
  }
  const int64_t n0 = (blockIdx.z * kFewBlocks + blockIdx.x) * (16 * RB);
  if (n0 >= p.n) return;
  const int ncols = (int)min((int64_t)(16 * RB), p.n - n0);
  const int64_t wrow = (int64_t)e * p.n + n0;
  const int ld = (int)p.ld, lines = ld >> 7;
  const uint32_t off = (uint32_t)((lane & 15) * ld + (lane >> 4) * 16);
  const char* wbase = (const char*)(p.b + wrow * p.ld);
  i32x4_t w[2 * U * RB];
  // Each workgroup starts at a line of its own (the order of the sum is free): rows a power of
  // two apart would otherwise be read at the same few memory channels by all workgroups at
  // once (16 tokens, 28672 x 4096: 31.4 -> 29.6 us).
  const int rot = (int)((blockIdx.x * 29u) % (unsigned)lines);
  auto line_at = [&](int l) { return l + rot >= lines ? l + rot - lines : l + rot; };
  // the wave's lines l0, l0 + NWV, .. of a batch; past the last line an empty buffer: zeros,
  // nothing is read
  auto load_w = [&](int l0) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int l = l0 + NWV * i;
      const rsrc_t r = make_rsrc(wbase, l < lines ? (int64_t)ncols * ld : 0);
#pragma unroll
      for (int q = 0; q < 2 * RB; ++q)
        w[i * 2 * RB + q] = ld128(r, off + (uint32_t)((q >> 1) * 16 * ld), (uint32_t)(line_at(l) * 128 + (q & 1) * 64));
    }
  };
  float fscale = 0.f;
  if constexpr (FUSE) {
    load_w(wave);
    if (tid < 4) *(uint32_t*)(tok + kFuseBytes + tid * 4) = 0u;  // what the other 15 columns read
    float v[8];
    uint32_t amax = 0;
    const int groups = (int)raw.cols / 8, rest = (int)raw.cols % 8;
    for (int g = tid; g < groups; g += NT) {
      load8<CD>(raw.x, 8 * g, v);
      amax = amax8(v, amax);
    }
    const float last = tid < rest ? load_cd<CD>(raw.x, 8 * groups + tid) : 0.f;
    amax = max(amax, __float_as_uint(last) & 0x7fffffffu);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) amax = max(amax, (uint32_t)__shfl_xor((int)amax, o, 64));
    if (lane == 0) tmax[wave] = amax;
    __syncthreads();
#pragma unroll
    for (int x = 0; x < NWV; ++x) amax = max(amax, tmax[x]);
    fscale = scale_of_bits(amax);
    const float rcp = scale_rcp(fscale);
    for (int g = tid; g < ld / 8; g += NT) {
      u32x2_t c = {0u, 0u};
      if (g < groups) {
        load8<CD>(raw.x, 8 * g, v);
        if (rcp == rcp) c = codes8(v, fscale, rcp);
        else c = codes8_by_division(v, fscale);
      }
      if (g != groups) *(u32x2_t*)(tok + 8 * g) = c;
    }
    if (tid < 8 && 8 * groups + tid < ld)
      tok[8 * groups + tid] = (char)(tid < rest && fscale > 0.f ? code_of(last, fscale) : 0);
    __syncthreads();
  }
  for (int64_t m0 = first; m0 < end; m0 += 16) {
    const int rows = (int)min((int64_t)16, end - m0);
    i32x4_t acc[RB][2];
#pragma unroll
    for (int b = 0; b < RB; ++b) acc[b][0] = acc[b][1] = i32x4_t{0, 0, 0, 0};
    for (int l0 = wave; l0 < lines; l0 += NWV * U) {
      i32x4_t a[2 * U];
      if (!FUSE || l0 != wave) load_w(l0);
#pragma unroll
      for (int i = 0; i < 2 * U; ++i) {
        const int l = l0 + NWV * (i >> 1);
        if constexpr (FUSE) {
          a[i] = *(const i32x4_t*)(tok + ((lane & 15) == 0 && l < lines ? line_at(l) * 128 + (i & 1) * 64 + (lane >> 4) * 16
                                                                        : kFuseBytes));
        } else {
          const rsrc_t r = make_rsrc(p.a + m0 * p.ld, l < lines ? (int64_t)rows * ld : 0);
          a[i] = ld128(r, off, (uint32_t)(line_at(l) * 128 + (i & 1) * 64));
        }
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int q = 0; q < 2 * RB; ++q)
          acc[q >> 1][q & 1] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[i * 2 * RB + q], a[2 * i + (q & 1)],
                                                                    acc[q >> 1][q & 1], 0, 0, 0);
    }
    // lane l: token l % 16, weight rows 4 (l / 16) .. + 3 of each 16
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        red[wave][lane & 15][16 * b + 4 * (lane >> 4) + i] = acc[b][0][i] + acc[b][1][i];
    __syncthreads();
    for (int q = tid; q < (FUSE ? 16 * RB : 256 * RB); q += NT) {
      const int t = q / (16 * RB), c = q % (16 * RB);
      if (t < rows && c < ncols) {
        int sum = red[0][t][c];
#pragma unroll
        for (int x = 1; x < NWV; ++x) sum += red[x][t][c];
        store_y<CD>(p, m0 + t, n0 + c, sum, FUSE ? fscale : p.sa[m0 + t], p.sb[wrow + c],
                    p.bias ? load_cd<CD>(p.bias, wrow + c) : 0.f);
      }
    }
    __syncthreads();
  }
}

size_t al(size_t b) { return (b + 255) & ~(size_t)255; }

// Slices of the contraction for a product of `tiles` tiles of 64 x 64 that leaves most compute
// units idle: as many as give 256 workgroups, of six stages at least.  A stage of a lone
// workgroup takes 0.33 us, the second launch 3 us: 100 x 1000 x 14336 40.1 -> 21.0 us,
// 61 x 1984 x 6212 23.1 -> 16.5, 768 x 64 x 3328 14.4 -> 13.3; below 24 stages or three slices
// it is slower (688 x 128 x 2496 12.9 -> 14.1, 128 x 4096 x 4096 17.3 -> 19.9), two slices gain
// from 40 stages on (500 x 1000 x 14336 42.5 -> 32.4, 1000 x 500 x 5120 21.7 -> 21.1).
constexpr int kSplitItems = 256;
int slices(int64_t tiles, int64_t ld) {
  const int64_t lines = ld >> 7;
  if (lines < 24 || tiles * (lines < 40 ? 3 : 2) > kSplitItems) return 1;
  return (int)std::min<int64_t>(std::min<int64_t>(8, kSplitItems / tiles), lines / 6);
}

// The product's kernels: few tokens, tiles by size.
enum Form { FEW, SMALL, LOW, MID, WIDE, FULL };

// Workspace: the tokens' codes and scales, for the form grouped by expert its route, and the
// sums of a cut contraction.
struct Plan {
  size_t off_codes = 0, off_scale = 0, off_count = 0, off_tiles = 0, off_part = 0, total = 0;
  int cap = 0, split = 1;
  Form cut = SMALL;  // tiles of a cut contraction
};

// Which product kernel takes a call: the few-token kernel, or the smallest tiles that still fit
// the compute units in one round, 256 x 256 beyond.  Larger tiles read each operand less
// often, smaller ones occupy more of the chip (whole calls, weights from memory, us):
//                            few   64 x 64  64 x 128  128 x 128  128 x 256  256 x 256
//   8 x 4096 x 4096          11.1    15.7     21.0
//   16 x 14336 x 4096        19.7    20.2     24.3       26.1
//   24 x 14336 x 4096        29.6    20.7     24.4
//   64 x 14336 x 4096                22.1     26.9       27.8       35.4       47.3
//   128 x 14336 x 4096               29.3     27.2       31.1       38.6       50.4
//   256 x 14336 x 4096               43.8     37.9       31.8       38.5       50.8
//   512 x 14336 x 4096               67.9     60.1       52.2       40.2       52.8
//   1024 x 14336 x 4096               114     89.0       90.2                  63.5
//   512 x 4096 x 4096                26.2     24.2       28.7       36.8       49.1
//   1024 x 4096 x 4096               46.0     40.0       34.8       39.6       52.1
//   2048 x 4096 x 4096               78.9     66.4       57.7       46.7       53.4
// and of experts, by their rows on average:
//   1 of 2 (4096 x 4096)     14.4    18.3     21.8
//   4 of 8 (4096 x 4096)     28.3    34.3     33.7
//   4 of 32 (2048 x 2048)    29.0    30.5     29.3
//   8 of 32 (2048 x 2048)    37.9    31.9     30.8
//   32 of 8 (4096 x 4096)            44.8     49.6       41.9       44.6       54.5
//   64 of 8 (4096 x 4096)            51.3     48.3       44.4       48.5       57.6
//   64 of 64 (1024 x 2048)           49.5     47.5       54.3       55.1       47.6
//   128 of 8 (4096 x 4096)           65.8     64.7       63.5       53.3       63.0
//   192 of 8 (14336 x 4096)           249      203        173        155        174
//   256 of 8 (4096 x 4096)           96.5     86.1       83.2       83.0       74.2
//   28 of 32 (1024 x 4096)           46.0     50.8
//   28 of 16 (4096 x 4096)           75.4     81.6
//   25 of 40 (3000 x 1111)           40.9     37.6
//   160 of 4 (2112 x 1785)           16.5     15.4                  21.0
//   112 of 4 (2048 x 7168)           42.9     37.5                  59.0
// Long rows of few outputs leave the few-token kernel with few workgroups; the smallest tiles
// cut the contraction (16 x 512 x 16384 22.6 -> 16.0 us, 4 x 1024 x 14336 20.3 -> 17.5, 2 x 64 x
// 131072 113 -> 72; but 16 x 256 x 4096 9.0 -> 10.7, 4 x 4096 x 8192 15.4 -> 17.3).
// An uneven routing gives some experts several times the average, and the few-token
// kernel goes over its weights again for each 16 rows, so experts leave it early.
// The rule follows the best column but for two rows of the experts' table: 32 of 8 and 28 of 32
// fill one round of 64 x 128 tiles to the last compute unit and take them (49.6 and 50.8 us), where
// 128 x 128 (41.9) and 64 x 64 (46.0) are faster.
int64_t live_experts(int64_t m, int32_t experts) { return std::max<int64_t>(1, std::min<int64_t>(experts, m)); }
bool few_tokens(int64_t m, int32_t experts) { return m <= (experts == 1 ? 16 : 4 * live_experts(m, experts)); }
bool long_rows_of_few(int64_t n, int64_t ld, int32_t experts) { return experts == 1 && ld > 8192 && n <= 2048; }
// One token of one matrix: one launch does it all.
bool one_launch(int64_t m, int64_t ld, bool grouped) { return !grouped && m == 1 && ld <= kFuseBytes; }

Form form_of(int64_t m, int64_t n, int64_t ld, int32_t experts) {
  const int64_t live = live_experts(m, experts), cus = cu_count();
  if (few_tokens(m, experts)) return long_rows_of_few(n, ld, experts) ? SMALL : FEW;
  // tile rows: each expert's last one is half full on average
  auto one_round = [&](int64_t tm, int64_t tn) {
    return (experts == 1 ? ceil_div(m, tm) : std::max(live, m / tm + (live + 1) / 2)) * ceil_div(n, tn) <= cus;
  };
  if (one_round(64, 64)) return SMALL;
  if (one_round(64, 128)) return LOW;
  if (one_round(128, 128)) return MID;
  if (experts > 1 && m < 96 * live) return m <= 32 * live && ld > 2048 ? SMALL : LOW;
  return one_round(128, 256) || (experts > 1 && m < 256 * live) ? WIDE : FULL;
}
static_assert(Wide::TN == Full::TN && Mid::TN == Low::TN && Wide::TM == Mid::TM && Low::TM == Small::TM &&
                  Mid::NW == Low::NW && Low::NW == Small::NW, "by form");
int tile_rows(Form f) { return f == FULL ? Full::TM : f == WIDE || f == MID ? Mid::TM : Low::TM; }

Plan plan_int8(const qlora_int8_t* w, int64_t m, bool grouped) {
  Plan P;
  const int64_t ld = QLORA_INT8_LD(w->cols);
  size_t off = al((size_t)(m * ld));
  P.off_scale = off;
  off += al((size_t)m * 4);
  if (grouped) {
    // the smallest tiles have the most rows of them: the size does not depend on the device
    P.cap = (int)(m / Low::TM + std::min<int64_t>(w->experts, m));
    P.off_count = off;
    off += al(4);
    P.off_tiles = off;
    off += al((size_t)P.cap * sizeof(int4));
  }
  P.total = off;
  if (one_launch(m, ld, grouped) || (few_tokens(m, w->experts) && !long_rows_of_few(w->rows, ld, w->experts))) return P;
  int64_t tiles = (grouped ? P.cap : ceil_div(m, Small::TM)) * ceil_div(w->rows, Small::TN);
  P.split = tiles > 0 ? slices(tiles, ld) : 1;
  int64_t tile = Small::TM * Small::TN;
  // Where the 64 x 64 tiles are too many for that: 128 x 128 in two to four slices, from 56
  // stages on (300 x 4096 x 14336 62.8 -> 48.0 us, 640 x 800 x 14336 43.9 -> 36.4, 260 x 4096 x
  // 7168 33.9 -> 31.2, 2000 x 500 x 8192 34.7 -> 36.0; 300 x 2048 x 5200 21.0 -> 22.5).
  const int64_t mid = ceil_div(m, Mid::TM) * ceil_div(w->rows, Mid::TN);
  if (P.split == 1 && !grouped && m > 16 && ld >= 56 * 128 && mid > 0 && 2 * mid <= kSplitItems) {
    P.cut = MID;
    P.split = (int)std::min<int64_t>(4, kSplitItems / mid);
    tiles = mid;
    tile = Mid::TM * Mid::TN;
  }
  if (P.split > 1) {
    P.off_part = off;
    off += (size_t)P.split * tiles * tile * 4;
  }
  P.total = off;
  return P;
}

// A launch has fewer than 2^32 threads: more rows than that go in several.
template <int CD, int TPR, int HOLD>
int launch_rows(const void* x, int64_t ldx, int64_t rows, int64_t cols, int8_t* codes, float* scale, const Route& r,
                hipStream_t s) {
  const int ld = (int)QLORA_INT8_LD(cols);
  const int64_t most = (1LL << 31) / TPR;
  for (int64_t r0 = 0; r0 < rows; r0 += most) {
    const int64_t n = std::min(most, rows - r0);
    const Route here = r0 + n == rows ? r : Route{};
    const dim3 g((unsigned)(ceil_div(n, kThreads / TPR) + (here.offsets ? 1 : 0))), b(kThreads);
    k_int8_rows<CD, TPR, HOLD><<<g, b, 0, s>>>((const char*)x + r0 * ldx * cd_bytes(CD), ldx, n, (int)cols, ld,
                                               codes + r0 * ld, scale + r0, here);
    const int rc = check_launch("k_int8_rows");
    if (rc) return rc;
  }
  return QLORA_OK;
}

// A wave per row where rows are short, or enough to fill the chip and not long, else a
// workgroup per row.  Holding two groups to a thread (and reading what exceeds them again)
// beats holding eight for all but long rows: 8192 x 4096 bf16 17.9 against 20.6 us, 16 x 4096
// 3.5 against 3.8, but 4096 x 14336 41.2 against 34.1.
template <int CD>
int rows_cd(const void* x, int64_t ldx, int64_t rows, int64_t cols, int8_t* codes, float* scale, const Route& r,
            hipStream_t s) {
  if (cols <= 512 || (rows >= 4 * cu_count() && cols <= 4096))
    return launch_rows<CD, 64, 2>(x, ldx, rows, cols, codes, scale, r, s);
  if (cols <= 4096) return launch_rows<CD, kThreads, 2>(x, ldx, rows, cols, codes, scale, r, s);
  return launch_rows<CD, kThreads, 8>(x, ldx, rows, cols, codes, scale, r, s);
}

int rows_to_int8(int cd, const void* x, int64_t ldx, int64_t rows, int64_t cols, int8_t* codes, float* scale,
                 const Route& r, hipStream_t s) {
  if (cd == CD_BF16) return rows_cd<CD_BF16>(x, ldx, rows, cols, codes, scale, r, s);
  if (cd == CD_F16) return rows_cd<CD_F16>(x, ldx, rows, cols, codes, scale, r, s);
  return rows_cd<CD_F32>(x, ldx, rows, cols, codes, scale, r, s);
}

// Weight rows per workgroup.  The tokens' codes are read once for each workgroup, so more rows
// spare that traffic, as long as there are workgroups enough: at 16 tokens, 16 / 32 / 64 rows
// take 11.1 / 12.9 / 16.6 us on 4096 x 4096 (256 blocks of 16 rows), 22.2 / 19.0 / 17.3 us on
// 14336 x 4096 (896) and, with more than eight blocks to a compute unit, 50.9 / 47.9 / 51.4 us
// on six experts of 14336 x 4096.
template <int CD, bool FUSE>
int few_rows(const I8& p, int runs, const Raw& raw, hipStream_t s) {
  const int64_t blocks = ceil_div(p.n, 16) * runs, cus = cu_count();
  const int rb = blocks < 2 * cus ? 1 : blocks < 3 * cus || blocks >= 8 * cus ? 2 : 4;
  const int64_t gx = ceil_div(p.n, 16 * rb);
  const dim3 g((unsigned)std::min(gx, kFewBlocks), (unsigned)runs, (unsigned)ceil_div(gx, kFewBlocks));
  // Four waves; eight for one token over a long contraction on few workgroups (4096 x 14336:
  // 19.5 -> 16.3 us; with more tokens or shorter rows the same or worse).
  constexpr int W = FUSE ? 8 : 4;
  if (FUSE && rb == 1 && p.ld >= 8192) k_int8_few<CD, 1, W, FUSE><<<g, dim3(64 * W), 0, s>>>(p, p.count, p.tiles, raw);
  else if (rb == 1) k_int8_few<CD, 1, 4, FUSE><<<g, dim3(256), 0, s>>>(p, p.count, p.tiles, raw);
  else if (rb == 2) k_int8_few<CD, 2, 4, FUSE><<<g, dim3(256), 0, s>>>(p, p.count, p.tiles, raw);
  else k_int8_few<CD, 4, 4, FUSE><<<g, dim3(256), 0, s>>>(p, p.count, p.tiles, raw);
  return check_launch("k_int8_few");
}

// The contraction in p.split slices, and the sum of those.
template <int CD, class T, int WGS>
int cut_product(const I8& p, int cap, hipStream_t s) {
  const int64_t tiles = (p.count ? cap : ceil_div(p.m, T::TM)) * ceil_div(p.n, T::TN);
  k_int8_tile<CD, T, WGS, true><<<dim3((unsigned)(tiles * p.split)), dim3(64 * T::NW), 0, s>>>(p);
  const int rc = check_launch("k_int8_tile");
  if (rc) return rc;
  k_int8_join<CD, T><<<dim3((unsigned)tiles, T::TM * T::TN / (4 * kThreads)), dim3(kThreads), 0, s>>>(p);
  return check_launch("k_int8_join");
}

// Tiles of a form: `cap` rows of them, or (0) of one matrix.
int64_t tiles_of(Form f, int64_t m, int64_t n, int cap) {
  const int tn = f >= WIDE ? Full::TN : f >= LOW ? Low::TN : Small::TN;
  return (cap ? cap : ceil_div(m, tile_rows(f))) * ceil_div(n, tn);
}

template <int CD>
int product(const I8& p, Form f, int cap, Form cut, hipStream_t s) {
  if (p.split > 1 && cut == MID) return cut_product<CD, Mid, 1>(p, cap, s);
  if (p.split > 1 && f == SMALL) return cut_product<CD, Small, 2>(p, cap, s);
  if (f == FEW) return few_rows<CD, false>(p, p.count ? cap : 1, Raw{}, s);
  const int64_t tiles = tiles_of(f, p.m, p.n, p.count ? cap : 0);
  const dim3 g((unsigned)tiles);
  // the large tiles: a workgroup to a compute unit, or to a half tile in an only round
  if (f == FULL)
    k_int8_full<CD><<<dim3((unsigned)std::min<int64_t>(cu_count(), 2 * tiles)), dim3(512), 0, s>>>(p);
  else if (f == WIDE) k_int8_tile<CD, Wide, 1><<<g, dim3(64 * Wide::NW), 0, s>>>(p);
  else if (f == MID) k_int8_tile<CD, Mid, 1><<<g, dim3(64 * Mid::NW), 0, s>>>(p);
  else if (f == LOW) k_int8_tile<CD, Low, 2><<<g, dim3(64 * Low::NW), 0, s>>>(p);
  else k_int8_tile<CD, Small, 2><<<g, dim3(64 * Small::NW), 0, s>>>(p);
  return check_launch(f == FULL ? "k_int8_full" : "k_int8_tile");
}

}  // namespace

int launch_int8_quantize(const void* w, int64_t ldw, int dtype, const qlora_int8_t* q, hipStream_t s) {
  ProfScope prof(QLORA_K_INT8_ROWS, s);
  return rows_to_int8(dtype, w, ldw, q->experts * q->rows, q->cols, q->codes, q->scale, Route{}, s);
}

size_t int8_workspace_bytes(const qlora_int8_t* w, int64_t m, bool grouped) {
  return plan_int8(w, m, grouped).total;
}

int launch_int8_linear(const qlora_int8_t* w, const void* x, int64_t m, int64_t ldx, const int32_t* offsets,
                       const void* bias, int cd, void* y, void* ws, hipStream_t s) {
  const Plan P = plan_int8(w, m, offsets != nullptr);
  char* base = (char*)ws;
  I8 p = {};
  p.a = (const int8_t*)(base + P.off_codes);
  p.sa = (const float*)(base + P.off_scale);
  p.b = w->codes;
  p.sb = w->scale;
  p.bias = bias;
  p.y = y;
  p.m = m;
  p.n = w->rows;
  p.ld = QLORA_INT8_LD(w->cols);
  p.part = (int*)(base + P.off_part);
  p.split = P.split;
  if (one_launch(m, p.ld, offsets != nullptr)) {
    ProfScope prof(QLORA_K_INT8_GEMM, s);
    const Raw raw = {x, w->cols};
    if (cd == CD_BF16) return few_rows<CD_BF16, true>(p, 1, raw, s);
    if (cd == CD_F16) return few_rows<CD_F16, true>(p, 1, raw, s);
    return few_rows<CD_F32, true>(p, 1, raw, s);
  }
  const Form f = form_of(m, w->rows, p.ld, w->experts);
  Route r = {};
  if (offsets) {
    r.count = (int32_t*)(base + P.off_count);
    r.tiles = (int4*)(base + P.off_tiles);
    r.offsets = offsets;
    r.experts = w->experts;
    const int live = (int)std::min<int64_t>(w->experts, m);
    // whole runs of tile_m rows and one partial run for each expert that has a row; for the
    // few-token kernel an expert's rows are one run
    r.tile_m = f == FEW ? (int)m : tile_rows(f);
    r.cap = f == FEW ? live : (int)(m / r.tile_m) + live;
    r.m = m;
    p.count = r.count;
    p.tiles = r.tiles;
  }
  if (f != FEW) {
    // before anything is launched: the kernels count tiles in 31 bits, and the tiles of all forms
    // but the largest (whose workgroups go through theirs) are one launch, of fewer than 2^32 threads
    const int64_t tiles = tiles_of(f, m, p.n, r.cap), threads = f == FULL ? 1 : 64 * (f == WIDE ? Wide::NW : Mid::NW);
    if (tiles >= (1LL << 31) || tiles * threads >= (1LL << 32))
      return set_error(QLORA_ERR_UNSUPPORTED, "int8: %lld tiles in one call", (long long)tiles);
  }
  {
    ProfScope prof(QLORA_K_INT8_ROWS, s);
    const int rc = rows_to_int8(cd, x, ldx, m, w->cols, (int8_t*)p.a, (float*)p.sa, r, s);
    if (rc) return rc;
  }
  ProfScope prof(QLORA_K_INT8_GEMM, s);
  if (cd == CD_BF16) return product<CD_BF16>(p, f, r.cap, P.cut, s);
  if (cd == CD_F16) return product<CD_F16>(p, f, r.cap, P.cut, s);
  return product<CD_F32>(p, f, r.cap, P.cut, s);
}

}  // namespace qnf4
