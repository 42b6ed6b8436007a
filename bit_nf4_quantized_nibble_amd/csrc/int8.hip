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

#include "common.h"

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

template <int CD>
__global__ __launch_bounds__(kThreads) void k_int8_rows(const void* __restrict__ x, int64_t ldx, int64_t rows,
                                                        int64_t cols, int64_t ld, int8_t* __restrict__ codes,
                                                        float* __restrict__ scale) {
  __shared__ uint32_t red[kThreads / 64];
  const int64_t row = blockIdx.x;
  uint32_t amax = 0;
  for (int64_t k = threadIdx.x; k < cols; k += kThreads)
    amax = max(amax, __float_as_uint(load_cd<CD>(x, row * ldx + k)) & 0x7fffffffu);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) amax = max(amax, (uint32_t)__shfl_xor((int)amax, off, 64));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = amax;
  __syncthreads();
  amax = max(max(red[0], red[1]), max(red[2], red[3]));
  const float s = scale_of_bits(amax);
  if (threadIdx.x == 0) scale[row] = s;
  for (int64_t k = threadIdx.x; k < ld; k += kThreads)
    codes[row * ld + k] = (int8_t)((s > 0.f && k < cols) ? code_of(load_cd<CD>(x, row * ldx + k), s) : 0);
}

// ------------------------------------------------------------------------ routing
// Experts' rows for the product kernels, from the caller's offsets: starts[e] is the
// largest of offsets[0 .. e], limited to [0, m], so no row belongs to two experts
// whatever the offsets hold; tiles[t] = {expert, first row, rows, 0} for each run of at
// most tile_m rows of one expert, in order, `count` of them (at most cap: m / tile_m
// whole runs and one partial run for each expert that has a row).
struct Route {
  int32_t* starts;  // [experts + 1]
  int32_t* count;   // [1]
  int4* tiles;      // [cap]
};

__global__ __launch_bounds__(64) void k_int8_route(const int32_t* __restrict__ offsets, int experts, int64_t m,
                                                   int tile_m, int cap, Route r) {
  const int lane = threadIdx.x;
  int before = 0;  // starts of the chunk's first expert
  int at = 0;      // tiles so far
  {
    const int o = offsets[0];
    before = (int)min((int64_t)max(o, 0), m);
  }
  if (lane == 0) r.starts[0] = before;
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
    const int n = end - start, t = (n + tile_m - 1) / tile_m;
    int sum = t;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int v = __shfl_up(sum, off, 64);
      if (lane >= off) sum += v;
    }
    if (e < experts) {
      r.starts[e + 1] = end;
      const int first = at + sum - t;
      for (int i = 0; i < t; ++i)
        if (first + i < cap) r.tiles[first + i] = make_int4(e, start + i * tile_m, min(tile_m, n - i * tile_m), 0);
    }
    before = __shfl(end, 63, 64);
    at += __shfl(sum, 63, 64);
  }
  if (lane == 0) *r.count = min(at, cap);
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
};

// y from the sum: (sum * s) * t + bias, each product rounded to fp32, then to cd.
template <int CD>
__device__ __forceinline__ void store_y(const I8& p, int64_t row, int64_t col, int sum, float sa, float sb, float bv) {
  store_cd<CD>(p.y, row * p.n + col, (float)sum * sa * sb + bv);
}

constexpr int kT = 64;

template <int CD>
__global__ __launch_bounds__(kThreads) void k_int8_simple(I8 p) {
  __shared__ __attribute__((aligned(16))) int8_t as[kT][128 + 16], bs[kT][128 + 16];
  int e = 0;
  int64_t m0 = (int64_t)blockIdx.y * kT;
  int rows = (int)min((int64_t)kT, p.m - m0);
  if (p.count) {
    if ((int)blockIdx.y >= *p.count) return;
    const int4 t = p.tiles[blockIdx.y];
    e = t.x;
    m0 = t.y;
    rows = t.z;
  }
  const int64_t n0 = (int64_t)blockIdx.x * kT;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int8_t* bp = p.b + (int64_t)e * p.n * p.ld;
  i32x16_t acc;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0;
  for (int64_t k0 = 0; k0 < p.ld; k0 += 128) {
    __syncthreads();
    for (int q = tid; q < kT * 8; q += kThreads) {
      const int r = q >> 3, c = (q & 7) * 16;
      u32x4_t va = {0, 0, 0, 0}, vb = {0, 0, 0, 0};
      if (r < rows) va = *(const u32x4_t*)(p.a + (m0 + r) * p.ld + k0 + c);
      if (n0 + r < p.n) vb = *(const u32x4_t*)(bp + (n0 + r) * p.ld + k0 + c);
      *(u32x4_t*)&as[r][c] = va;
      *(u32x4_t*)&bs[r][c] = vb;
    }
    __syncthreads();
    const int ar = (wave >> 1) * 32 + (lane & 31), br = (wave & 1) * 32 + (lane & 31);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      const int c = (2 * ks + (lane >> 5)) * 16;
      acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(*(const i32x4_t*)&as[ar][c], *(const i32x4_t*)&bs[br][c], acc, 0, 0,
                                                  0);
    }
  }
  const int64_t col = n0 + (wave & 1) * 32 + (lane & 31);
  if (col >= p.n) return;
  const float sb = p.sb[e * p.n + col];
  const float bv = p.bias ? load_cd<CD>(p.bias, e * p.n + col) : 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = (wave >> 1) * 32 + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3);
    if (r < rows) store_y<CD>(p, m0 + r, col, acc[i], p.sa[m0 + r], sb, bv);
  }
}

size_t al(size_t b) { return (b + 255) & ~(size_t)255; }

// Workspace: the tokens' codes and scales, and for the form grouped by expert its route.
struct Plan {
  size_t off_codes = 0, off_scale = 0, off_starts = 0, off_count = 0, off_tiles = 0, total = 0;
  int cap = 0;
};

Plan plan_int8(int64_t m, int64_t cols, int32_t experts, bool grouped) {
  Plan P;
  size_t off = al((size_t)m * QLORA_INT8_LD(cols));
  P.off_scale = off;
  off += al((size_t)m * 4);
  if (grouped) {
    P.cap = (int)(m / kT + std::min<int64_t>(experts, m));
    P.off_starts = off;
    off += al(((size_t)experts + 1) * 4);
    P.off_count = off;
    off += al(4);
    P.off_tiles = off;
    off += al((size_t)P.cap * sizeof(int4));
  }
  P.total = off;
  return P;
}

int rows_to_int8(int cd, const void* x, int64_t ldx, int64_t rows, int64_t cols, int8_t* codes, float* scale,
                 hipStream_t s) {
  const int64_t ld = QLORA_INT8_LD(cols);
  const dim3 g((unsigned)rows), b(kThreads);
  if (cd == CD_BF16) k_int8_rows<CD_BF16><<<g, b, 0, s>>>(x, ldx, rows, cols, ld, codes, scale);
  else if (cd == CD_F16) k_int8_rows<CD_F16><<<g, b, 0, s>>>(x, ldx, rows, cols, ld, codes, scale);
  else k_int8_rows<CD_F32><<<g, b, 0, s>>>(x, ldx, rows, cols, ld, codes, scale);
  return check_launch("k_int8_rows");
}

}  // namespace

int launch_int8_quantize(const void* w, int64_t ldw, int dtype, const qlora_int8_t* q, hipStream_t s) {
  ProfScope prof(QLORA_K_INT8_ROWS, s);
  return rows_to_int8(dtype, w, ldw, q->experts * q->rows, q->cols, q->codes, q->scale, s);
}

size_t int8_workspace_bytes(const qlora_int8_t* w, int64_t m, bool grouped) {
  return plan_int8(m, w->cols, w->experts, grouped).total;
}

int launch_int8_linear(const qlora_int8_t* w, const void* x, int64_t m, int64_t ldx, const int32_t* offsets,
                       const void* bias, int cd, void* y, void* ws, hipStream_t s) {
  const Plan P = plan_int8(m, w->cols, w->experts, offsets != nullptr);
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
  int rc;
  {
    ProfScope prof(QLORA_K_INT8_ROWS, s);
    if ((rc = rows_to_int8(cd, x, ldx, m, w->cols, (int8_t*)p.a, (float*)p.sa, s))) return rc;
    if (offsets) {
      Route r = {(int32_t*)(base + P.off_starts), (int32_t*)(base + P.off_count), (int4*)(base + P.off_tiles)};
      k_int8_route<<<dim3(1), dim3(64), 0, s>>>(offsets, w->experts, m, kT, P.cap, r);
      if ((rc = check_launch("k_int8_route"))) return rc;
      p.count = r.count;
      p.tiles = r.tiles;
    }
  }
  ProfScope prof(QLORA_K_INT8_GEMM, s);
  const dim3 g((unsigned)ceil_div(p.n, kT), (unsigned)(offsets ? P.cap : ceil_div(m, kT))), b(kThreads);
  if (cd == CD_BF16) k_int8_simple<CD_BF16><<<g, b, 0, s>>>(p);
  else if (cd == CD_F16) k_int8_simple<CD_F16><<<g, b, 0, s>>>(p);
  else k_int8_simple<CD_F32><<<g, b, 0, s>>>(p);
  return check_launch("k_int8_simple");
}

}  // namespace qnf4
