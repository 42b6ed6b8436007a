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

namespace qnf4 {
namespace {

constexpr int kThreads = 256;
typedef int i32x4_t __attribute__((__vector_size__(16)));
typedef int i32x8_t __attribute__((__vector_size__(32)));

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

// The weight: a workgroup to a block of 128 x 128, two threads to a row.
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
};

// Eight codes as bf16.
__device__ __forceinline__ bf16x8_t to_bf16(int lo, int hi) {
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

// acc += the scaled products of a block's 128 contraction elements, a[s] and b[s] 64 of them.
// The matrix instruction that scales each operand row aligns its products to the largest before it
// adds them and loses what lies about 2^-19 below it: sums are 1e-5 to 8e-5 (of their norm) off, far
// below the step of a 16-bit result but not of an fp32 one.  There (EXACT) codes are brought to
// bf16, which holds every e4m3 value, the bf16 instruction adds their products as fp32 sums do, and
// the block's sum takes both scales at once (their product alone may leave fp32's range).
template <bool EXACT>
__device__ __forceinline__ void mfma_block(f32x16_t& acc, const i32x8_t (&b)[2], const i32x8_t (&a)[2], int sb, int sa) {
  if constexpr (!EXACT) {
#pragma unroll
    for (int s = 0; s < 2; ++s) acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b[s], a[s], acc, 0, 0, 0, sb, 0, sa);
  } else {
    f32x16_t part;
#pragma unroll
    for (int v = 0; v < 16; ++v) part[v] = 0.f;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        part = __builtin_amdgcn_mfma_f32_32x32x16_bf16(to_bf16(b[s][2 * q], b[s][2 * q + 1]),
                                                       to_bf16(a[s][2 * q], a[s][2 * q + 1]), part, 0, 0, 0);
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[v] += __builtin_amdgcn_ldexpf(part[v], sa + sb - 254);
  }
}

// One wave to 32 x 32 of y, operands from global memory: the plain form of the product.
template <int CD>
__global__ __launch_bounds__(64) void k_fp8_plain(F8 p) {
  const int lane = threadIdx.x, h = lane >> 5, r32 = lane & 31;
  const int64_t n0 = (int64_t)blockIdx.x * 32, m0 = (int64_t)blockIdx.y * 32;
  const int64_t row = min(m0 + r32, p.m - 1), col = min(n0 + r32, p.n - 1);
  f32x16_t acc;
#pragma unroll
  for (int v = 0; v < 16; ++v) acc[v] = 0.f;
  for (int64_t kb = 0; kb < p.ld / 128; ++kb) {
    const int sa = (int)(p.sa[(kb >> 2) * p.stride + row] >> (8 * (kb & 3))) & 255;
    const int sb = p.sb[(n0 >> 7) * p.lds + kb];
    i32x8_t a[2], b[2];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int64_t k = kb * 128 + 64 * s + 32 * h + 16 * q;
        const i32x4_t va = *(const i32x4_t*)(p.a + row * p.ld + k), vb = *(const i32x4_t*)(p.b + col * p.ld + k);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          a[s][4 * q + e] = va[e];
          b[s][4 * q + e] = vb[e];
        }
      }
    mfma_block<CD == CD_F32>(acc, b, a, sb, sa);
  }
  if (m0 + r32 >= p.m) return;
#pragma unroll
  for (int v = 0; v < 16; ++v) {
    const int64_t c = n0 + 8 * (v >> 2) + 4 * h + (v & 3);
    if (c < p.n) store_cd<CD>(p.y, row * p.n + c, acc[v] + (p.bias ? load_cd<CD>(p.bias, c) : 0.f));
  }
}

size_t al(size_t b) { return (b + 255) & ~(size_t)255; }

// Workspace: the tokens' codes and exponents.
struct Plan {
  size_t off_scale = 0, total = 0;
  int64_t stride = 0;
};
Plan plan_fp8(const qlora_fp8_t* w, int64_t m, int cd) {
  Plan P;
  const int64_t ld = QLORA_FP8_LD(w->cols);
  P.stride = round_up(m, 64);
  P.off_scale = al((size_t)(m * ld));
  P.total = P.off_scale + al((size_t)(ceil_div(ld, 512) * P.stride * 4));
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

template <int CD>
int linear_cd(const F8& p, const void* x, int64_t ldx, int64_t cols, hipStream_t s) {
  {
    ProfScope prof(QLORA_K_FP8_ROWS, s);
    const int rc = rows_cd<CD>(x, ldx, p.m, cols, (uint8_t*)p.a, (uint32_t*)p.sa, p.stride, s);
    if (rc) return rc;
  }
  ProfScope prof(QLORA_K_FP8_GEMM, s);
  k_fp8_plain<CD><<<dim3((unsigned)ceil_div(p.n, 32), (unsigned)ceil_div(p.m, 32)), dim3(64), 0, s>>>(p);
  return check_launch("k_fp8_plain");
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
  if (cd == CD_BF16) return linear_cd<CD_BF16>(p, x, ldx, w->cols, s);
  if (cd == CD_F16) return linear_cd<CD_F16>(p, x, ldx, w->cols, s);
  return linear_cd<CD_F32>(p, x, ldx, w->cols, s);
}

}  // namespace qnf4
