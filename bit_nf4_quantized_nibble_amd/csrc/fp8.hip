// fp8.hip -- matrix products in 8-bit floating point (e4m3) with a scale for each block of 128:
// the serving form of a merged weight beside the 8-bit integers of int8.hip.
//
//   block      s = 2^e, e the smallest integer >= -127 with max |x| <= 448 s; codes RNE_e4m3(x / s).
//              Tokens: 128 consecutive columns of a row.  Weights: 128 rows by 128 columns.
//   product    y[i, j] = RNE_cd(sum_b s_ib t_jb sum_{k in b} c[i, k] d[j, k] + bias[j])
//
// A scale is a power of two because the values are floating point: another scale moves no code's
// relative step, x / s is exact, and the matrix instruction takes an 8-bit exponent for each
// operand row, so scaling a block costs no instruction of its own.
//
// Codes are stored in rows of QLORA_FP8_LD(cols) bytes, zero past the last column, so every
// kernel reads whole 128-byte blocks.  Scales are stored as exponents e + 127 in a byte: the
// weight's as [row block][column block], the tokens' as one word for four column blocks,
// [column block / 4][token], so that a tile's scales of four blocks are one run of words.
#include <algorithm>

#include "mlp.h"
#include "tile.h"

namespace qnf4 {
namespace {

using namespace tile;
constexpr int kThreads = 256;

// ------------------------------------------------------------------ values to 8 bits
// Exponent byte of a block from its largest |x| as bits: 448 = 1.75 * 2^8.  A block that holds
// an infinity or a NaN has the scale 1 and NaN codes.
__device__ __forceinline__ uint32_t exponent_of(uint32_t amax) {
  const int e = (int)(amax >> 23) - ((amax & 0x7fffffu) <= 0x600000u ? 8 : 7);
  return amax >= 0x7f800000u ? 127u : (uint32_t)max(e, 0);
}
// 1 / s, exactly: 2^(127 - byte), byte at most 247.
__device__ __forceinline__ float inverse_of(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

constexpr uint32_t kNanCodes = 0x7f7f7f7fu;

// 16 bytes at any element-aligned address.
template <int ES>
struct __attribute__((packed, aligned(ES))) Chunk {
  u32x4_t v;
};

// Elements at .. at + 7 of a row with `left` of them (from `at` on) in it; zeros past those.
template <int CD>
__device__ __forceinline__ void load8(const void* x, int64_t at, int left, float (&v)[8]) {
  if (left >= 8) {
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
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < left ? load_cd<CD>(x, at + e) : 0.f;
  }
}
__device__ __forceinline__ uint32_t amax8(const float (&v)[8], uint32_t m) {
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
  return m;
}
__device__ __forceinline__ u32x2_t codes8(const float (&v)[8], uint32_t amax, float inv, int left) {
  u32x2_t o;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * e] * inv, v[4 * e + 1] * inv, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * e + 2] * inv, v[4 * e + 3] * inv, w, true);
    o[e] = (uint32_t)w;
    if (amax >= 0x7f800000u) {
      const int n = max(0, min(4, left - 4 * e));  // columns past the last stay zero
      o[e] = n == 4 ? kNanCodes : kNanCodes & ((1u << (8 * n)) - 1u);
    }
  }
  return o;
}

// Tokens: 16 lanes to a block, four blocks of a row to a wave, whose exponents are one word.
template <int CD>
__global__ __launch_bounds__(kThreads) void k_fp8_rows(const void* __restrict__ x, int64_t ldx, int64_t rows, int cols,
                                                       int ld, int64_t stride, uint8_t* __restrict__ codes,
                                                       uint32_t* __restrict__ scale) {
  const int quads = (ld + 511) / 512, lane = threadIdx.x & 63;
  const int64_t item = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  const int64_t row = item / quads;
  const int quad = (int)(item % quads), col = quad * 512 + lane * 8;
  if (row >= rows) return;
  float v[8];
  load8<CD>(x, row * ldx + col, cols - col, v);
  uint32_t amax = amax8(v, 0u);
#pragma unroll
  for (int off = 8; off >= 1; off >>= 1) amax = max(amax, (uint32_t)__shfl_xor((int)amax, off, 64));
  const uint32_t byte = exponent_of(amax);
  if (col < ld) *(u32x2_t*)(codes + row * ld + col) = codes8(v, amax, inverse_of(byte), cols - col);
  const uint32_t w = byte << (8 * (lane >> 4));
  const uint32_t a = w | (uint32_t)__shfl_xor((int)w, 16, 64);
  const uint32_t word = a | (uint32_t)__shfl_xor((int)a, 32, 64);
  if (lane == 0) scale[quad * stride + row] = word;
}

// The weight: a workgroup to a block of 128 x 128, two threads to a row.  Run once for a weight: 14336 x 4096 bf16 takes 107 to
// 124 us, 34 at a copy's rate; a wave's loads touch 32 rows 16 bytes at a time, and it waits for those (vector pipes busy 7%).
template <int CD>
__global__ __launch_bounds__(kThreads) void k_fp8_weight(const void* __restrict__ w, int64_t ldw, int64_t rows, int cols,
                                                         int ld, int lds, uint8_t* __restrict__ codes,
                                                         uint8_t* __restrict__ scale) {
  __shared__ uint32_t red[kThreads / 64];
  const int64_t rb = blockIdx.x, row = rb * 128 + (threadIdx.x >> 1);
  const int kb = blockIdx.y, k0 = kb * 128 + (threadIdx.x & 1) * 64;
  float v[8][8];
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    load8<CD>(w, row * ldw + k0 + 8 * i, row < rows ? cols - k0 - 8 * i : 0, v[i]);
    amax = amax8(v[i], amax);
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) amax = max(amax, (uint32_t)__shfl_xor((int)amax, off, 64));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = amax;
  __syncthreads();
  amax = max(max(red[0], red[1]), max(red[2], red[3]));
  const uint32_t byte = exponent_of(amax);
  if (threadIdx.x == 0) {
    scale[rb * lds + kb] = (uint8_t)byte;
    if (kb == gridDim.y - 1)
      for (int z = kb + 1; z < lds; ++z) scale[rb * lds + z] = 127;
  }
  if (row >= rows) return;
  const float inv = inverse_of(byte);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *(u32x2_t*)(codes + row * ld + k0 + 8 * i) = codes8(v[i], amax, inv, cols - k0 - 8 * i);
}

// ------------------------------------------------------------------------- product
struct F8 {
  const uint8_t* a;    // [m][ld] codes of the tokens
  const uint32_t* sa;  // [ld / 512 rounded up][stride] their exponents, four column blocks to a word
  int64_t stride;
  const uint8_t* b;    // [n][ld] codes of the weight
  const uint8_t* sb;   // [n / 128 rounded up][lds] its exponents
  const void* bias;    // [n] cd or null
  void* y;             // [m][n] cd
  int64_t m, n, ld, lds;
  float* part;         // contraction cut into `split` slices: their sums, tile by tile
  int split;
};

// Where a tile lies: first token row, token rows, first column.
struct Place {
  int rows;
  int64_t m0, n0;
};

// Beside a tile's stages LDS holds the tokens' exponent words of two groups of four stages (1 KiB
// each, used in turn; a group's copy begins before its first stage's), and a set of coefficients
// that is loaded once: the columns' biases and the exponents of the tile's weight blocks.
constexpr int kRing = 2048;
constexpr int kMaxLds = (int)QLORA_FP8_LDS(QLORA_FP8_MAX_COLS);
template <class T>
struct Coef {
  static constexpr int BLOCKS = T::TN > 128 ? T::TN / 128 : 1, BYTES = T::TN * 4 + BLOCKS * kMaxLds;
};

// The copies of a tile's stages by one wave: instruction i of wave w fills LDS rows
// 8 (w + NW i) .. + 7 of the stage; lane l lands in chunk l % 8 of row l / 8 and fetches the
// logical chunk that lies there.
template <class T>
struct Copies8 {
  // of the eight waves of the 256-column tiles with two buffers, the first four (one to a SIMD) copy
  static constexpr int WAVES = T::NW == 8 && T::NS == 2 ? 4 : T::NW, PER_A = T::TM / 8 / WAVES, PER = (T::TM + T::TN) / 8 / WAVES;
  const uint8_t *a, *b;
  const uint32_t* sa;
  int64_t abytes, bbytes, stride, left;
  const char *ring, *bsc;
  uint32_t off, step;
  int KT, wave, lane, row;
  __device__ __forceinline__ Copies8(const F8& p, const Place& t, char* ring_, const char* coef, int wave_, int lane_)
      : ring(ring_), wave(wave_), lane(lane_) {
    const int ncols = (int)min((int64_t)T::TN, p.n - t.n0), ld = (int)p.ld;
    a = p.a + t.m0 * p.ld;
    b = p.b + t.n0 * p.ld;
    sa = p.sa + t.m0;
    stride = p.stride;
    left = p.stride - t.m0;
    abytes = (int64_t)t.rows * p.ld;
    bbytes = (int64_t)ncols * p.ld;
    const int r = 8 * wave + (lane >> 3);
    off = (uint32_t)(r * ld + (((lane & 7) ^ swz(r)) << 4));
    step = (uint32_t)(8 * WAVES * ld);
    KT = ld >> 7;
    row = (wave / T::NWN) * 32 * T::WMB + (lane & 31);
    const int wn = (wave % T::NWN) * 32 * T::WNB;
    bsc = coef + T::TN * 4 + (T::TN > 128 ? (wn >> 7) * (int)p.lds : 0);
  }
  // only stages k0 .. k1 - 1 of the contraction, k0 a multiple of 4
  __device__ __forceinline__ void cut(int k0, int k1) {
    a += (int64_t)k0 * 128;
    b += (int64_t)k0 * 128;
    abytes -= (int64_t)k0 * 128;
    bbytes -= (int64_t)k0 * 128;
    sa += (k0 >> 2) * stride;
    bsc += k0;
    KT = k1 - k0;
  }
  __device__ __forceinline__ void begin(int stage) const {
    if (wave == 0 && (stage & 3) == 0 && stage < KT)
      copy16(make_rsrc(sa + (stage >> 2) * stride, min(left, (int64_t)256) * 4), (char*)ring + ((stage >> 2) & 1) * 1024,
             (uint32_t)lane * 16, 0);
  }
  __device__ __forceinline__ void one(char* stage_lds, int stage, int i) const {
    // past the last stage: an empty buffer, nothing is fetched
    const bool in = stage < KT, a_side = i < PER_A;
    const rsrc_t r = a_side ? make_rsrc(a, in ? abytes : 0) : make_rsrc(b, in ? bbytes : 0);
    copy16(r, stage_lds + (wave + WAVES * i) * 1024, off + (a_side ? i : i - PER_A) * step, stage * 128);
  }
  __device__ __forceinline__ void all(char* stage_lds, int stage) const {
    if (WAVES < T::NW && wave >= WAVES) return;
    begin(stage);
#pragma unroll
    for (int i = 0; i < PER; ++i) one(stage_lds, stage, i);
  }
  __device__ __forceinline__ void scales(int stage, int (&s)[T::WMB], int& sb) const {
    const char* w = ring + ((stage >> 2) & 1) * 1024 + row * 4;
#pragma unroll
    for (int i = 0; i < T::WMB; ++i) s[i] = *(const int*)(w + 128 * i);
    sb = (int)*(const uint8_t*)(bsc + min(stage, KT - 1));
  }
  __device__ __forceinline__ void shift(int stage, int (&s)[2][T::WMB], int (&sb)[2]) const {
#pragma unroll
    for (int i = 0; i < T::WMB; ++i) s[0][i] = (int)((uint32_t)s[1][i] >> (8 * (stage & 3)));
    sb[0] = sb[1];
  }
};

// Word i (of 4 bytes) of a tile's coefficients: biases as fp32, then the exponents of its blocks.
template <int CD, class T>
__device__ __forceinline__ uint32_t coefficient(const F8& p, const Place& t, int i) {
  if (i < T::TN) return p.bias && t.n0 + i < p.n ? __float_as_uint(load_cd<CD>(p.bias, t.n0 + i)) : 0u;
  const int words = (int)p.lds / 4, blk = (i - T::TN) / words;
  const bool in = blk < Coef<T>::BLOCKS && ((t.n0 >> 7) + blk) * 128 < p.n;
  return in ? ((const uint32_t*)(p.sb + ((t.n0 >> 7) + blk) * p.lds))[(i - T::TN) % words] : 0u;
}
template <class T>
__device__ __forceinline__ int coefficients(const F8& p) { return T::TN + Coef<T>::BLOCKS * (int)p.lds / 4; }

// Lane (r32, h) of block (i, j) holds row 32 i + r32, columns 32 j + 8 q + 4 h + v of the
// wave's part in elements 4 q + v.  32 rows at a time go through the wave's own LDS W (16-byte
// chunk c of a row at chunk c ^ row) and leave as 16-byte chunks of whole rows, at whatever
// address y's rows start.  Every wave issues exactly stores() of these (chunks past the tile's
// rows and whole chunks of columns fall outside their buffer), so a caller can count past them; the
// columns past the last whole chunk, and rows too long for a buffer, go element by element, and
// the wave waits for those.
template <int CD, class T>
struct Writer {
  static constexpr int ES = CD == CD_F32 ? 4 : 2, RB = 32 * T::WNB * ES, NC = RB / 16, PC = 16 / ES;
  static constexpr int stores() { return T::WMB * NC / 2; }
  __device__ static __forceinline__ void run(const F8& p, const Place& pl, const Acc<T>& acc, const char* coef, char* W,
                                             int wave, int lane) {
    constexpr int WMB = T::WMB, WNB = T::WNB;
    const int h = lane >> 5, r32 = lane & 31;
    const int wm = (wave / T::NWN) * 32 * WMB, wn = (wave % T::NWN) * 32 * WNB;
    const int ncols = (int)max((int64_t)0, min((int64_t)(32 * WNB), p.n - pl.n0 - wn));
    const int whole = p.n * ES < (1 << 26) ? ncols / PC * PC : 0;
    const bool lines = (p.n * ES) % 128 == 0 && ((uintptr_t)p.y & 127) == 0;  // whole lines are written at once
#pragma unroll
    for (int i = 0; i < WMB; ++i) {
#pragma unroll
      for (int j = 0; j < WNB; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x4_t bv = *(const f32x4_t*)(coef + (wn + 32 * j + 8 * q + 4 * h) * 4);
          float v[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) v[x] = acc[i][j][4 * q + x] + bv[x];
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

template <class T>
__device__ __forceinline__ Place place_of(const F8& p, int t, int tiles_m, int tiles_n) {
  int tm, tn;
  grouped_tile(t, tiles_m, tiles_n, tm, tn);
  tm = __builtin_amdgcn_readfirstlane(tm);
  tn = __builtin_amdgcn_readfirstlane(tn);
  Place pl;
  pl.n0 = (int64_t)tn * T::TN;
  pl.m0 = (int64_t)tm * T::TM;
  pl.rows = (int)min((int64_t)T::TM, p.m - pl.m0);
  return pl;
}

// One tile to a workgroup; several workgroups share a compute unit.
// SPLIT: p.split workgroups to a tile, each a slice of the contraction (whole groups of four
// stages); the sums go to p.part as [slice][tile][TM][TN] and k_fp8_join adds them in their order.
template <int CD, class T, int WGS, bool SPLIT = false>
__global__ __launch_bounds__(64 * T::NW, WGS) void k_fp8_tile(F8 p) {
  // One array for everything: with several, the compiler tells them apart and then waits for
  // every copy in flight before each fragment it reads.
  __shared__ __attribute__((aligned(1024))) char lds[T::LDS + kRing + Coef<T>::BYTES];
  char *ring = lds + T::LDS, *coef = ring + kRing;
  const int tiles_n = (int)((p.n + T::TN - 1) / T::TN), tiles_m = (int)((p.m + T::TM - 1) / T::TM);
  const int total = tiles_m * tiles_n;
  int b = blockIdx.x, slice = 0;
  if (SPLIT) {
    slice = b % p.split;
    b /= p.split;
  }
  if (b >= total) return;
  const int t = SPLIT ? b : xcd_run(b, total);
  const Place pl = place_of<T>(p, t, tiles_m, tiles_n);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  Copies8<T> cp(p, pl, ring, coef, wave, lane);
  if (SPLIT) {
    const int groups = (cp.KT + 3) >> 2;
    cp.cut(4 * (slice * groups / p.split), min(cp.KT, 4 * ((slice + 1) * groups / p.split)));
  }
  // the coefficients are requested first and stored once the copies are on their way
  constexpr int NC = (Coef<T>::BYTES / 4 + 64 * T::NW - 1) / (64 * T::NW);
  const int nc = coefficients<T>(p);
  uint32_t c[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i)
    if (tid + i * 64 * T::NW < nc) c[i] = coefficient<CD, T>(p, pl, tid + i * 64 * T::NW);
#pragma unroll
  for (int s = 0; s < T::NS; ++s) cp.all(lds + s * T::STAGE, s);
#pragma unroll
  for (int i = 0; i < NC; ++i)
    if (tid + i * 64 * T::NW < nc) ((uint32_t*)coef)[tid + i * 64 * T::NW] = c[i];
  wait_vmcnt<(T::NS - 1) * T::PER>();
  wait_lgkm0();
  barrier_only();
  Acc<T> acc;
  zero<T>(acc);
  contract<T, Float8<CD == CD_F32>>(acc, lds, cp, wave, lane);
  if constexpr (SPLIT) {
    float* dst = p.part + ((int64_t)slice * total + t) * (T::TM * T::TN);
    const int wm = (wave / T::NWN) * 32 * T::WMB, wn = (wave % T::NWN) * 32 * T::WNB;
#pragma unroll
    for (int i = 0; i < T::WMB; ++i)
#pragma unroll
      for (int j = 0; j < T::WNB; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x4_t v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
          *(f32x4_t*)(dst + (wm + 32 * i + (lane & 31)) * T::TN + wn + 32 * j + 8 * q + 4 * (lane >> 5)) = v;
        }
  } else {
    Writer<CD, T>::run(p, pl, acc, coef, lds + wave * 32 * Writer<CD, T>::RB, wave, lane);
  }
}

// y from the slices' sums: four columns of a row to a thread.
template <int CD, class T>
__global__ __launch_bounds__(kThreads) void k_fp8_join(F8 p) {
  const int tiles_n = (int)((p.n + T::TN - 1) / T::TN), tiles_m = (int)((p.m + T::TM - 1) / T::TM);
  const int total = tiles_m * tiles_n, t = blockIdx.x;
  if (t >= total) return;
  const Place pl = place_of<T>(p, t, tiles_m, tiles_n);
  const int at = 4 * (blockIdx.y * kThreads + threadIdx.x), row = at / T::TN, col = at % T::TN;
  if (row >= pl.rows || pl.n0 + col >= p.n) return;
  const float* src = p.part + (int64_t)t * (T::TM * T::TN) + at;
  f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s < p.split; ++s) sum = sum + *(const f32x4_t*)(src + (int64_t)s * total * (T::TM * T::TN));
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int64_t c = pl.n0 + col + x;
    if (c < p.n) store_cd<CD>(p.y, (pl.m0 + row) * p.n + c, sum[x] + (p.bias ? load_cd<CD>(p.bias, c) : 0.f));
  }
}

using Full = Tile<4, 2, 2, 4, 2>;  // 256 x 256, eight waves
using Half = Tile<2, 2, 2, 4, 2>;  // 128 x 256, eight waves
using Wide = Tile<2, 2, 2, 4, 3>;  // 128 x 256, eight waves
using Mid = Tile<2, 2, 2, 2, 4>;   // 128 x 128, four waves
using Low = Tile<1, 2, 2, 2, 3>;   // 64 x 128, four waves; two workgroups fit a compute unit
using Small = Tile<1, 1, 2, 2, 4>;  // 64 x 64, four waves; as well

// Whole rounds of 256 x 256 tiles, a workgroup to a compute unit going through its tiles.
// After a tile's last stage the copies of the next tile's first stage are requested, so that
// they land while the tile's y is stored.  A tile of at most 128 rows, and a last round of at most
// half the compute units (cut into halves of 128 rows then, two workgroups to a tile), run as
// 128 x 256.
template <int CD>
__global__ __launch_bounds__(512, 1) void k_fp8_full(F8 p) {
  constexpr int kStaging = Full::STAGE;  // y passes through what was stage 1
  static_assert(kStaging + 8 * 32 * Writer<CD, Full>::RB <= Full::LDS, "staging fits");
  static_assert(Half::TN == Full::TN && Coef<Full>::BYTES <= 4 * (256 + 512), "one bias and one word of exponents to a thread");
  __shared__ __attribute__((aligned(1024))) char lds[Full::LDS + kRing + 2 * Coef<Full>::BYTES];  // one array, as above
  char *ring = lds + Full::LDS, *coefs = ring + kRing;  // two sets, used in turn
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int b = blockIdx.x, G = gridDim.x;
  const int tiles_n = (int)((p.n + Full::TN - 1) / Full::TN), tiles_m = (int)((p.m + Full::TM - 1) / Full::TM);
  const int total = tiles_m * tiles_n, nc = coefficients<Full>(p);
  // The workgroup's tile in round r; rows 0: none (any more).
  auto item = [&](int r) {
    Place pl = {0, 0, 0};
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
  auto first_stage = [&](const Place& pl) {
    if (pl.rows > Half::TM) Copies8<Full>(p, pl, ring, coefs, wave, lane).all(lds, 0);
    else Copies8<Half>(p, pl, ring, coefs, wave, lane).all(lds, 0);
  };

  Place cur = item(0);
  if (cur.rows == 0) return;
  for (int i = tid; i < nc; i += 512) ((uint32_t*)coefs)[i] = coefficient<CD, Full>(p, cur, i);
  first_stage(cur);
  wait_vmcnt<0>();
  int set = 0;
  for (int r = 1;; ++r) {
    const Place nxt = item(r);
    uint32_t c0 = 0, c1 = 0;  // the next tile's coefficients arrive during this one's contraction
    if (nxt.rows) {
      if (tid < nc) c0 = coefficient<CD, Full>(p, nxt, tid);
      if (tid + 512 < nc) c1 = coefficient<CD, Full>(p, nxt, tid + 512);
    }
    wait_lgkm0();
    barrier_only();  // stage 0 and the coefficients are there, the staging of the tile before is free
    // Between here and the next tile's first stage: contract, hand over, write.
    auto work = [&](auto shape) {
      using T = decltype(shape);
      const char* coef = coefs + set * Coef<Full>::BYTES;
      // the lane counts as unknown here and after the contraction: addresses formed ahead of all tiles would
      // be kept through it and pushed out to memory there
      int ln = lane;
      asm volatile("" : "+v"(ln));
      Copies8<T> cp(p, cur, ring, coef, wave, ln);
      cp.all(lds + T::STAGE, 1);
      Acc<T> acc;
      zero<T>(acc);
      contract<T, Float8<CD == CD_F32>>(acc, lds, cp, wave, ln);
      asm volatile("" : "+v"(ln));
      if (nxt.rows) {
        uint32_t* to = (uint32_t*)(coefs + (set ^ 1) * Coef<Full>::BYTES);
        if (tid < nc) to[tid] = c0;
        if (tid + 512 < nc) to[tid + 512] = c1;
        first_stage(nxt);
      }
      Writer<CD, T>::run(p, cur, acc, coef, lds + kStaging + wave * 32 * Writer<CD, T>::RB, wave, ln);
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
// At up to 16 tokens the product reads each weight once and does little else: a workgroup of NWV
// waves takes 16 RB weight rows over the whole contraction, the waves dealing out groups of four
// 128-byte blocks of it (whose exponents are one word).  Codes go from global memory straight
// into the 16 x 16 x 128 matrix instruction (lane l: row l % 16, bytes 32 (l / 16) .. + 31 of a
// block), weight rows as one operand and tokens as the other; the waves' sums meet in LDS.
// FUSE: each wave brings the tokens' columns of its own groups to 8 bits itself, through LDS of
// its own, which spares the call a launch: no workgroup waits for another wave's columns, since a
// block's scale needs no other block.
constexpr int kFewRow = 544;  // bytes of a token's group in LDS: 512 codes, padded off one bank

template <bool EXACT>
__device__ __forceinline__ void mma16(f32x4_t& acc, const i32x8_t& w, const i32x8_t& a, int sw, int sa) {
  if constexpr (!EXACT) {
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, acc, 0, 0, 0, sw, 0, sa);
  } else {
    f32x4_t part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < 4; ++q)
      part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(e4m3_to_bf16(w[2 * q], w[2 * q + 1]),
                                                     e4m3_to_bf16(a[2 * q], a[2 * q + 1]), part, 0, 0, 0);
    const int e = (sw & 255) + (sa & 255) - 254;
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[v] += __builtin_amdgcn_ldexpf(part[v], e);
  }
}

// Source of a call's tokens when they are not in 8 bits yet.
struct Raw {
  const void* x;
  int64_t ldx;
  int cols;
};

template <int CD, int RB, int NWV, bool FUSE>
__global__ __launch_bounds__(64 * NWV) void k_fp8_few(F8 p, Raw raw) {
  constexpr int NT = 64 * NWV;
  __shared__ float red[NWV][16][16 * RB + 1];
  __shared__ __attribute__((aligned(16))) char tok[FUSE ? NWV * 16 * kFewRow : 16];
  __shared__ uint32_t tsc[FUSE ? NWV * 16 : 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q4 = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * RB);
  const int rows = (int)p.m, ncols = (int)min((int64_t)(16 * RB), p.n - n0);
  const int ld = (int)p.ld, blocks = ld >> 7, groups = (blocks + 3) >> 2;
  const uint32_t off = (uint32_t)(r16 * ld + q4 * 32);
  const uint8_t* wbase = p.b + n0 * p.ld;
  const uint32_t* sw = (const uint32_t*)(p.sb + (n0 >> 7) * p.lds);
  // Each workgroup starts at a group of its own (the order of the sum is fixed by it): rows a
  // power of two apart would otherwise be read at the same few memory channels at once.
  const int rot = (int)((blockIdx.x * 29u) % (unsigned)groups);
  f32x4_t acc[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) acc[b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  char* mine = tok + (FUSE ? wave * 16 * kFewRow : 0);
  for (int g0 = wave; g0 < groups; g0 += NWV) {
    const int g = g0 + rot >= groups ? g0 + rot - groups : g0 + rot;
    i32x8_t w[4][RB];
    // past the last block an empty buffer: zeros, nothing is read
#pragma unroll
    for (int l = 0; l < 4; ++l) {
      const rsrc_t r = make_rsrc(wbase, 4 * g + l < blocks ? (int64_t)ncols * ld : 0);
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        const i32x4_t lo = ld128(r, off + (uint32_t)(16 * b * ld), (uint32_t)((4 * g + l) * 128));
        const i32x4_t hi = ld128(r, off + (uint32_t)(16 * b * ld) + 16, (uint32_t)((4 * g + l) * 128));
        w[l][b] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      }
    }
    const uint32_t wscale = sw[g];
    uint32_t ascale;
    if constexpr (FUSE) {
      const int col = g * 512 + lane * 8;
      for (int t0 = 0; t0 < rows; t0 += 4) {
        float v[4][8];
#pragma unroll
        for (int t = 0; t < 4; ++t)
          if (t0 + t < rows) load8<CD>(raw.x, (t0 + t) * raw.ldx + col, raw.cols - col, v[t]);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          if (t0 + t >= rows) break;
          uint32_t amax = amax8(v[t], 0u);
#pragma unroll
          for (int o = 8; o >= 1; o >>= 1) amax = max(amax, (uint32_t)__shfl_xor((int)amax, o, 64));
          const uint32_t byte = exponent_of(amax);
          *(u32x2_t*)(mine + (t0 + t) * kFewRow + lane * 8) = codes8(v[t], amax, inverse_of(byte), raw.cols - col);
          if (r16 == 0) ((uint8_t*)tsc)[(wave * 16 + t0 + t) * 4 + q4] = (uint8_t)byte;
        }
      }
      wait_lgkm0();  // the wave reads back only what it wrote
      asm volatile("" ::: "memory");
      ascale = tsc[wave * 16 + min(r16, rows - 1)];
    } else {
      ascale = p.sa[g * p.stride + min(r16, rows - 1)];
    }
#pragma unroll
    for (int l = 0; l < 4; ++l) {
      i32x8_t a;
      if constexpr (FUSE) {
        // rows past the last repeat it: their columns of the result are not stored
        const char* src = mine + min(r16, rows - 1) * kFewRow + l * 128 + q4 * 32;
        const i32x4_t lo = *(const i32x4_t*)src, hi = *(const i32x4_t*)(src + 16);
        a = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      } else {
        const rsrc_t r = make_rsrc(p.a, 4 * g + l < blocks ? (int64_t)rows * ld : 0);
        const i32x4_t lo = ld128(r, off, (uint32_t)((4 * g + l) * 128)), hi = ld128(r, off + 16, (uint32_t)((4 * g + l) * 128));
        a = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      }
#pragma unroll
      for (int b = 0; b < RB; ++b)
        mma16<CD == CD_F32>(acc[b], w[l][b], a, (int)(wscale >> (8 * l)), (int)(ascale >> (8 * l)));
    }
    if constexpr (FUSE) {
      wait_lgkm0();  // the reads are done before the next group's codes overwrite them
      asm volatile("" ::: "memory");
    }
  }
  // lane l: token l % 16, weight rows 4 (l / 16) .. + 3 of each 16
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][r16][16 * b + 4 * q4 + i] = acc[b][i];
  __syncthreads();
  for (int q = tid; q < 16 * RB * rows; q += NT) {
    const int t = q / (16 * RB), c = q % (16 * RB);
    if (c < ncols) {
      float sum = red[0][t][c];
#pragma unroll
      for (int x = 1; x < NWV; ++x) sum += red[x][t][c];
      store_cd<CD>(p.y, t * p.n + n0 + c, sum + (p.bias ? load_cd<CD>(p.bias, n0 + c) : 0.f));
    }
  }
}

size_t al(size_t b) { return (b + 255) & ~(size_t)255; }

// Slices of a contraction: where the smallest tiles are few and the rows long, up to eight, of six lines
// of 128 codes or more, as long as the pieces are not more than the compute units (64 x 1024 x 4096 and
// 16 x 4096 x 14336 are as fast in one piece; 64 x 4096 x 14336 18.1 us in four, 23.0 in two; 256 x 1024 x 14336
// 18.7 in four, 24.6 in one).
constexpr int kSplitItems = 256;
int slices(int64_t tiles, int64_t ld) {
  const int64_t lines = ld >> 7;
  if (lines < 24 || tiles * (lines < 40 ? 3 : 2) > kSplitItems) return 1;
  return (int)std::min<int64_t>(std::min<int64_t>(8, kSplitItems / tiles), lines / 6);
}

// The product's kernels: few tokens, tiles by size.
enum Form { FEW, SMALL, LOW, MID, WIDE, FULL };

bool few_tokens(int64_t m) { return m <= 16; }
// Up to four tokens the product brings x to 8 bits itself, every workgroup anew, and saves a launch, until what it
// repeats costs more (us, this way and with the launch: 1 token of 4096 x 4096 9.5 and 12.5, of
// 4096 x 14336 11.8 and 14.9; 4 tokens of 8192 x 4096 10.8 and 12.2, of 14336 x 4096 16.5 and 15.4, of
// 4096 x 14336 18.2 and 15.4; 8 tokens of 4096 x 4096 11.7 and 10.5 without the launch's cost on the host).
bool fused_rows(int64_t m, int64_t n, int64_t ld) { return m <= 4 && m * n * ld <= 1LL << 27; }
// Few tokens on tiles all the same.  Rows so long that the few-token kernel's waves, a row of W each, are too few (us on the
// device, tiles and that kernel, 5 to 16 tokens: bf16 256 x 14336 12.3 and 14 to 17, 2048 x 14336 15.5 and 16 to 19,
// 1024 x 28672 18.4 and 26 to 33; fp32 1024 x 28672 25.5 and 28 to 35, but 2048 x 14336 19.8 and 17.8 to 20.5; bf16
// 4096 x 14336 19.9 and 18 to 21, 1024 x 8192 10.8 and 10 to 12).  And in 16 bits, from 12 tokens on, so many rows that the
// smallest tiles fill the card (12288 x 4096, 5, 8, 12, 16 tokens: 17.3 against 16.7, 17.2, 17.9, 18.8; 14336 x 4096 18.3 against 17.2,
// 17.4, 18.3, 18.9; 28672 x 2048 17.0 against 16.6, 16.9, 17.7, 18.4; but 28672 x 1024 11.5 against 10.6 to 11.6, 8192 x 4096 16.2
// against 13.2 to 13.7, 14336 x 8192 32 against 28 to 32).
bool few_on_tiles(int64_t m, int64_t n, int64_t ld, int cd) {
  return (ld > 8192 && n <= 2048) || (cd != CD_F32 && m >= 12 && ceil_div(n, 64) >= 192 && ld > 1024 && ld <= 4096);
}

// us by form, bf16, m x n x k: 512 x 2048 x 2048 SMALL 10.9, LOW 12.0, MID 15.0; 1024 x 2048 x 2048 14.0, 13.2, 15.9;
// 1024 x 4096 x 4096 37, 28, 25.9, WIDE 31.7, FULL 40.8; 2048 x 4096 x 4096 67, 53, 48, 39.9, 46.0;
// 4096 x 4096 x 4096 123, 97, 90, 74, 69.9: the smallest tiles that take one round.
Form form_of(int64_t m, int64_t n, int64_t ld, int cd) {
  const int64_t cus = cu_count();
  if (few_tokens(m)) return few_on_tiles(m, n, ld, cd) && !fused_rows(m, n, ld) ? SMALL : FEW;
  auto one_round = [&](int64_t tm, int64_t tn) { return ceil_div(m, tm) * ceil_div(n, tn) <= cus; };
  if (one_round(64, 64)) return SMALL;
  if (one_round(64, 128)) return LOW;
  if (one_round(128, 128)) return MID;
  // fp32 results' bf16 fragments and block sums do not fit the registers beside 256 x 256 sums
  return one_round(128, 256) || cd == CD_F32 ? WIDE : FULL;
}
// Workspace: the tokens' codes and exponents, and the sums of a cut contraction.
struct Plan {
  size_t off_scale = 0, off_part = 0, total = 0;
  int64_t stride = 0;
  int split = 1;
  Form cut = SMALL;  // tiles of a cut contraction
};
Plan plan_fp8(const qlora_fp8_t* w, int64_t m, int cd) {
  Plan P;
  const int64_t ld = QLORA_FP8_LD(w->cols);
  P.stride = round_up(m, 64);
  P.off_scale = al((size_t)(m * ld));
  P.off_part = P.total = P.off_scale + al((size_t)(ceil_div(ld, 512) * P.stride * 4));
  if (m == 0 || w->rows == 0 || (few_tokens(m) && (fused_rows(m, w->rows, ld) || !few_on_tiles(m, w->rows, ld, cd)))) return P;
  int64_t tiles = ceil_div(m, Small::TM) * ceil_div(w->rows, Small::TN), tile = Small::TM * Small::TN;
  P.split = slices(tiles, ld);
  const int64_t mid = ceil_div(m, Mid::TM) * ceil_div(w->rows, Mid::TN);
  if (P.split == 1 && m > 16 && ld >= 56 * 128 && 2 * mid <= kSplitItems) {
    P.cut = MID;
    P.split = (int)std::min<int64_t>(4, kSplitItems / mid);
    tiles = mid;
    tile = Mid::TM * Mid::TN;
  }
  if (P.split > 1) P.total += al((size_t)(P.split * tiles * tile * 4));
  return P;
}

// A launch has fewer than 2^32 threads: more rows than that go in several.
template <int CD>
int rows_cd(const void* x, int64_t ldx, int64_t rows, int64_t cols, uint8_t* codes, uint32_t* scale, int64_t stride,
            hipStream_t s) {
  const int64_t ld = QLORA_FP8_LD(cols), quads = ceil_div(ld, 512), most = std::max<int64_t>(1, (1LL << 25) / quads);
  for (int64_t r0 = 0; r0 < rows; r0 += most) {
    const int64_t n = std::min(most, rows - r0);
    k_fp8_rows<CD><<<dim3((unsigned)ceil_div(n * quads, kThreads / 64)), dim3(kThreads), 0, s>>>(
        (const char*)x + r0 * ldx * cd_bytes(CD), ldx, n, (int)cols, (int)ld, stride, codes + r0 * ld, scale + r0);
    const int rc = check_launch("k_fp8_rows");
    if (rc) return rc;
  }
  return QLORA_OK;
}

template <int CD>
int quantize_cd(const void* w, int64_t ldw, const qlora_fp8_t* q, hipStream_t s) {
  const int64_t ld = QLORA_FP8_LD(q->cols), blocks = ceil_div(q->rows, 128);
  k_fp8_weight<CD><<<dim3((unsigned)blocks, (unsigned)(ld / 128)), dim3(kThreads), 0, s>>>(
      w, ldw, q->rows, (int)q->cols, (int)ld, (int)QLORA_FP8_LDS(q->cols), q->codes, q->scale);
  return check_launch("k_fp8_weight");
}

// Weight rows per workgroup, in 16s: the tokens are read once for each workgroup, so more rows spare that
// traffic, as long as there are workgroups enough.
int few_row_blocks(int64_t n) { return ceil_div(n, 16) < 2 * cu_count() ? 1 : 2; }
template <int CD, bool FUSE>
int few_rows(const F8& p, const Raw& raw, hipStream_t s) {
  const int rb = few_row_blocks(p.n);
  const dim3 g((unsigned)ceil_div(p.n, 16 * rb));
  if (rb == 1 && p.ld >= 8192) k_fp8_few<CD, 1, 8, FUSE><<<g, dim3(512), 0, s>>>(p, raw);
  else if (rb == 1) k_fp8_few<CD, 1, 4, FUSE><<<g, dim3(256), 0, s>>>(p, raw);
  else k_fp8_few<CD, 2, 4, FUSE><<<g, dim3(256), 0, s>>>(p, raw);
  return check_launch("k_fp8_few");
}

// The contraction in p.split slices, and the sum of those.
template <int CD, class T, int WGS>
int cut_product(const F8& p, hipStream_t s) {
  const int64_t tiles = ceil_div(p.m, T::TM) * ceil_div(p.n, T::TN);
  k_fp8_tile<CD, T, WGS, true><<<dim3((unsigned)(tiles * p.split)), dim3(64 * T::NW), 0, s>>>(p);
  const int rc = check_launch("k_fp8_tile");
  if (rc) return rc;
  k_fp8_join<CD, T><<<dim3((unsigned)tiles, T::TM * T::TN / (4 * kThreads)), dim3(kThreads), 0, s>>>(p);
  return check_launch("k_fp8_join");
}

int64_t tiles_of(Form f, int64_t m, int64_t n) {
  const int64_t tm = f == FULL ? Full::TM : f >= MID ? Mid::TM : Low::TM;
  const int64_t tn = f >= WIDE ? Full::TN : f >= LOW ? Low::TN : Small::TN;
  return ceil_div(m, tm) * ceil_div(n, tn);
}

template <int CD>
int product(const F8& p, Form f, Form cut, hipStream_t s) {
  if (p.split > 1) return cut == MID ? cut_product<CD, Mid, 1>(p, s) : cut_product<CD, Small, 2>(p, s);
  if (f == FEW) return few_rows<CD, false>(p, Raw{}, s);
  const int64_t tiles = tiles_of(f, p.m, p.n);
  const dim3 g((unsigned)tiles);
  // the large tiles: a workgroup to a compute unit, or to a half tile in an only round
  if constexpr (CD != CD_F32) {
    if (f == FULL) {
      k_fp8_full<CD><<<dim3((unsigned)std::min<int64_t>(cu_count(), 2 * tiles)), dim3(512), 0, s>>>(p);
      return check_launch("k_fp8_full");
    }
  }
  if (f == WIDE) k_fp8_tile<CD, Wide, 1><<<g, dim3(64 * Wide::NW), 0, s>>>(p);
  else if (f == MID) k_fp8_tile<CD, Mid, 1><<<g, dim3(64 * Mid::NW), 0, s>>>(p);
  else if (f == LOW) k_fp8_tile<CD, Low, 2><<<g, dim3(64 * Low::NW), 0, s>>>(p);
  else k_fp8_tile<CD, Small, 2><<<g, dim3(64 * Small::NW), 0, s>>>(p);
  return check_launch("k_fp8_tile");
}

template <int CD>
int linear_cd(const F8& p, const void* x, int64_t ldx, int64_t cols, Form cut, hipStream_t s) {
  if (fused_rows(p.m, p.n, p.ld)) {
    ProfScope prof(QLORA_K_FP8_GEMM, s);
    return few_rows<CD, true>(p, Raw{x, ldx, (int)cols}, s);
  }
  const Form f = form_of(p.m, p.n, p.ld, CD);
  // before anything is launched: the kernels count tiles in 31 bits, and the tiles of all forms but the
  // largest (whose workgroups go through theirs) are one launch, of fewer than 2^32 threads
  const int64_t tiles = f == FEW ? ceil_div(p.n, 16 * few_row_blocks(p.n)) : tiles_of(f, p.m, p.n);
  const int64_t threads = f == FULL ? 1 : f == WIDE ? 512 : 256;
  if (tiles >= (1LL << 31) || tiles * threads >= (1LL << 32))
    return set_error(QLORA_ERR_UNSUPPORTED, "fp8: %lld tiles in one call", (long long)tiles);
  {
    ProfScope prof(QLORA_K_FP8_ROWS, s);
    const int rc = rows_cd<CD>(x, ldx, p.m, cols, (uint8_t*)p.a, (uint32_t*)p.sa, p.stride, s);
    if (rc) return rc;
  }
  ProfScope prof(QLORA_K_FP8_GEMM, s);
  return product<CD>(p, f, cut, s);
}

}  // namespace

int launch_fp8_quantize(const void* w, int64_t ldw, int dtype, const qlora_fp8_t* q, hipStream_t s) {
  ProfScope prof(QLORA_K_FP8_ROWS, s);
  if (dtype == CD_BF16) return quantize_cd<CD_BF16>(w, ldw, q, s);
  if (dtype == CD_F16) return quantize_cd<CD_F16>(w, ldw, q, s);
  return quantize_cd<CD_F32>(w, ldw, q, s);
}

size_t fp8_workspace_bytes(const qlora_fp8_t* w, int64_t m, int cd) { return plan_fp8(w, m, cd).total; }

int launch_fp8_linear(const qlora_fp8_t* w, const void* x, int64_t m, int64_t ldx, const void* bias, int cd, void* y,
                      void* ws, hipStream_t s) {
  const Plan P = plan_fp8(w, m, cd);
  F8 p = {};
  p.a = (const uint8_t*)ws;
  p.sa = (const uint32_t*)((char*)ws + P.off_scale);
  p.stride = P.stride;
  p.b = w->codes;
  p.sb = w->scale;
  p.bias = bias;
  p.y = y;
  p.m = m;
  p.n = w->rows;
  p.ld = QLORA_FP8_LD(w->cols);
  p.lds = QLORA_FP8_LDS(w->cols);
  p.part = (float*)((char*)ws + P.off_part);
  p.split = P.split;
  if (cd == CD_BF16) return linear_cd<CD_BF16>(p, x, ldx, w->cols, P.cut, s);
  if (cd == CD_F16) return linear_cd<CD_F16>(p, x, ldx, w->cols, P.cut, s);
  return linear_cd<CD_F32>(p, x, ldx, w->cols, P.cut, s);
}

}  // namespace qnf4
