// planes.hip -- the layer with seeded dropout and the gated block, forward and backward, for every
// layout and type that the tuned kernels do not take (gfx950): any even block size, rows and columns
// that fill no tile, blocks that run across rows, fp32.
//
// Every product is brought to one form, C[i, j] = sum_k a[i, k] b[j, k] of 16-bit operands with k
// contiguous, rows of whole stages of 64 elements (zeros behind the last), 16-byte aligned:
//
//   pack     one launch writes every operand of a call that is not of that form already: padded copies
//            and transposes of x, dY, A, B, W~ from its codes, x under the drawn mask, dg and du from
//            the saved g and u
//   product  one launch per level of dependence runs all products of that level, each cut into slices
//            of its contraction where its tiles alone would leave compute units idle
//   join     one launch adds the slices in their order and forms what leaves: outputs (bias, gate, mask
//            of the low-rank part), or the rank operands T and dT of the next level
//
// An fp32 operand is three planes of bf16 whose sum it is (24 bits in three times 8): six of the
// nine products of planes, those above 2^-22 of the largest, give the sum to fp32's accuracy at
// a sixth of the bf16 rate, which is still above the rate of the fp32 matrix instruction.  The rank
// operands are sums themselves and are kept in two planes (16 or more bits) of a 16-bit type.
#include <algorithm>

#include "act.h"
#include "mlp.h"
#include "tile.h"

namespace qnf4 {
namespace {

using namespace tile;

constexpr int kThreads = 256;

// ------------------------------------------------------------------------ planes
// v as the sum of `planes` 16-bit values of type KD, each the rounded rest of those before it.
template <int KD>
__device__ __forceinline__ void split(float v, int planes, uint16_t (&o)[3]) {
  o[0] = to_cd16<KD>(v);
  if (planes == 1) return;
  float h = from_cd16<KD>(o[0]);
  if (KD == CD_BF16 && fabsf(h) == INFINITY && fabsf(v) < INFINITY) {  // rounded past the largest value
    o[0] = (o[0] & 0x8000u) | 0x7f7fu;
    h = from_cd16<KD>(o[0]);
  }
  float rest = fabsf(h) < INFINITY ? v - h : 0.f;
  o[1] = to_cd16<KD>(rest);
  if (planes > 2) o[2] = to_cd16<KD>(rest - from_cd16<KD>(o[1]));
}

// A weight as three planes: its first 8 bits, the next 8 and the last (cut off, not rounded: a third of
// the work; x is rounded, so that the products left out stay below 2^-25 of the largest).
__device__ __forceinline__ void cut3(float v, uint32_t (&o)[3]) {
  o[0] = __float_as_uint(v) & 0xffff0000u;
  const float r = v - __uint_as_float(o[0]);
  o[1] = __float_as_uint(r) & 0xffff0000u;
  o[2] = __float_as_uint(r - __uint_as_float(o[1]));
}
// Planes of two weights, the first in the low halves.
template <int CD, int P>
__device__ __forceinline__ void pack_weights(float a, float b, uint32_t (&o)[P]) {
  if constexpr (P == 1) {
    o[0] = pack2<CD>(a, b);
  } else {
    uint32_t x[3], y[3];
    cut3(a, x);
    cut3(b, y);
#pragma unroll
    for (int q = 0; q < 3; ++q) o[q] = __builtin_amdgcn_perm(y[q], x[q], 0x07060302u);
  }
}

// Where a matrix's planes lie: element (i, k) of plane q at p[i ld + q step + k].
struct Planes {
  uint16_t* p = nullptr;
  int64_t ld = 0, step = 0;
  int n = 1;  // planes
};

// -------------------------------------------------------------------------- pack
enum Source { SRC_CD, SRC_F32, SRC_NF4, SRC_GATE, SRC_UP };
struct Pack {
  int src = SRC_CD, w = 0;  // w: which weight (SRC_NF4)
  const void* p = nullptr;
  const void* dh = nullptr;  // SRC_GATE, SRC_UP: p is pre [rows][2 cols], dh [rows][cols]
  int64_t rows = 0, cols = 0;
  bool drawn = false;  // under the drawn mask
  uint8_t* bits = nullptr;  // its bits, rows of wbits bytes
  int64_t wbits = 0;
  Planes rowwise;      // [rows][wide]
  int64_t wide = 0;
  Planes across;       // [cols][tall], the transpose
  int64_t tall = 0;
  uint32_t tiles_x = 0;
};
// The job of a workgroup: job i has those below end[i] that no earlier one has (all ends are read at once).
template <int N>
__device__ __forceinline__ int job_of(const uint32_t (&end)[N], uint32_t b, uint32_t& first) {
  int job = 0;
  first = 0;
#pragma unroll
  for (int i = 0; i < N - 1; ++i)
    if (b >= end[i]) {
      job = i + 1;
      first = end[i];
    }
  return job;
}
constexpr int kPacks = 14;
struct Packs {
  uint32_t end[kPacks];
  Pack j[kPacks];
  Nf4W w[2];
  float lv[16];
  Seeded sd;
  int n, act;
};

// Eight consecutive elements from `at` of which `left` (> 0) are there, zeros behind: vectors need
// no alignment beyond the element's.
template <int CD>
__device__ __forceinline__ void fetch_linear(const void* p, int64_t at, int left, float (&v)[8]) {
  if (left >= 8) {
    if constexpr (CD == CD_F32) {
      __builtin_memcpy(v, (const float*)p + at, 32);
    } else {
      u32x4_t t;
      __builtin_memcpy(&t, (const uint16_t*)p + at, 16);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = from_cd16<CD>((uint16_t)(t[e >> 1] >> (16 * (e & 1))));
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = e < left ? load_cd<CD>(p, at + e) : 0.f;
}

// Eight weights from flat index `at` as they are stored: their codes (element e in nibble e) and the
// scales of the block they begin in and, from element `cut` on, of the next (blocks of eight or more).
struct Eight {
  uint32_t codes, q0, q1;  // q: the scale's bits, or its code
  float t0, t1;            // the second-level scales
  int cut;
};
__device__ __forceinline__ uint32_t nibbles(uint32_t c) {  // the element in the high half of a byte comes first
  return (c >> 4 & 0x0f0f0f0fu) | (c << 4 & 0xf0f0f0f0u);
}
__device__ __forceinline__ Eight load_eight(const Nf4W& w, int64_t at, int left) {
  Eight o = {};
  if (left <= 0) return o;
  const int64_t byte = at >> 1;
  if (byte + 8 <= (w.rows * w.cols) >> 1) {
    u32x2_t c;
    __builtin_memcpy(&c, w.codes + byte, 8);
    o.codes = __builtin_amdgcn_alignbit(nibbles(c[1]), nibbles(c[0]), (uint32_t)(at & 1) * 4);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t b = w.codes[(at + min(e, left - 1)) >> 1];
      o.codes |= ((at + e) & 1 ? b & 15u : b >> 4) << (4 * e);
    }
  }
  if (w.bs_shift >= 3 && (w.cols & 7) == 0) {  // eight that begin at a multiple of eight lie in one block
    const int64_t b = at >> w.bs_shift;
    o.cut = 8;
    if (w.dq) {
      o.q0 = w.absmax_q[b];
      o.t0 = w.scale2[group_of(w, b)];
    } else {
      o.q0 = __float_as_uint(w.absmax[b]);
    }
    return o;
  }
  const int64_t b0 = block_of(w, at);
  o.cut = (int)min((int64_t)8, (b0 + 1) * w.bs - at);
  const int64_t b1 = o.cut < left ? b0 + 1 : b0;
  if (w.dq) {
    o.q0 = w.absmax_q[b0];
    o.q1 = w.absmax_q[b1];
    o.t0 = w.scale2[group_of(w, b0)];
    o.t1 = w.scale2[group_of(w, b1)];
  } else {
    o.q0 = __float_as_uint(w.absmax[b0]);
    o.q1 = __float_as_uint(w.absmax[b1]);
  }
  return o;
}
// Their values in the call's type, zeros from `left` on.
template <int CD>
__device__ __forceinline__ void value_eight(const Nf4W& w, const float* lv, const Eight& c, int64_t at, int left,
                                            float (&v)[8]) {
  const float s0 = w.dq ? (float)c.q0 * c.t0 : __uint_as_float(c.q0), s1 = w.dq ? (float)c.q1 * c.t1 : __uint_as_float(c.q1);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float s = e < c.cut ? s0 : s1;
    if (w.bs < 8 && e < left) s = block_scale(w, block_of(w, at + e));  // up to four blocks
    const float x = fl32_mul(lv[c.codes >> (4 * e) & 15u], s);
    v[e] = e >= left ? 0.f : CD == CD_F32 ? x : from_cd16<CD == CD_F32 ? CD_BF16 : CD>(to_cd16<CD == CD_F32 ? CD_BF16 : CD>(x));
  }
}

// Bound by latency where jobs are small (8 us a launch); W~^T of 5319 x 11200 from its codes takes 59 us, about twice what
// its bytes take.  A workgroup takes 64 x 64 elements of a job; a thread takes eight columns of two neighbouring rows, all
// of whose loads leave before the first is used.  The transpose passes through LDS as words of two rows:
// column k's row of 128 bytes begins 32 banks further for each eight columns, its 16-byte chunk c lies at
// c ^ (k / 8) % 8, so that the lanes of a write (eight columns apart, or four words) touch every bank once.
template <int CD>
__global__ __launch_bounds__(kThreads) void k_pack(Packs ps) {
  constexpr int KD = CD == CD_F32 ? CD_BF16 : CD;
  constexpr int MAX = CD == CD_F32 ? 3 : 2;  // planes
  __shared__ __attribute__((aligned(16))) char tile[MAX][72 * 128];
  auto chunk_at = [](int col, int c) { return (col + (col >> 3)) * 128 + ((c ^ (col >> 3)) << 4); };
  __shared__ float lv[16];
  const int tid = threadIdx.x;
  uint32_t first;
  const int job = job_of(ps.end, blockIdx.x, first);
  const Pack& j = ps.j[job];
  const uint32_t b = blockIdx.x - first;
  const int64_t i0 = (int64_t)(b / j.tiles_x) * 64, k0 = (int64_t)(b % j.tiles_x) * 64;
  if (tid < 16) lv[tid] = ps.lv[tid];
  const int c = tid & 7, r = tid >> 3;
  const int64_t k = k0 + 8 * c, row[2] = {i0 + 2 * r, i0 + 2 * r + 1};
  int left[2];
  float v[2][8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    left[h] = row[h] < j.rows ? (int)max((int64_t)0, min((int64_t)8, j.cols - k)) : 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[h][e] = 0.f;
  }
  if (j.src == SRC_NF4) {
    const Nf4W& w = ps.w[j.w];
    Eight raw[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) raw[h] = load_eight(w, row[h] * j.cols + k, left[h]);
    __syncthreads();  // the levels are there
#pragma unroll
    for (int h = 0; h < 2; ++h) value_eight<CD>(w, lv, raw[h], row[h] * j.cols + k, left[h], v[h]);
  } else if (j.src == SRC_CD) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (left[h] > 0) fetch_linear<CD>(j.p, row[h] * j.cols + k, left[h], v[h]);
  } else if (j.src == SRC_F32) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (left[h] > 0) fetch_linear<CD_F32>(j.p, row[h] * j.cols + k, left[h], v[h]);
  } else {
    float g[2][8], u[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (left[h] > 0) {
        fetch_linear<CD>(j.p, 2 * row[h] * j.cols + k, left[h], g[h]);
        fetch_linear<CD>(j.p, (2 * row[h] + 1) * j.cols + k, left[h], u[h]);
        fetch_linear<CD>(j.dh, row[h] * j.cols + k, left[h], v[h]);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (left[h] > 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float value, slope;
          if (ps.act == QLORA_ACT_SILU) act_grad<QLORA_ACT_SILU>(g[h][e], value, slope);
          else if (ps.act == QLORA_ACT_GELU) act_grad<QLORA_ACT_GELU>(g[h][e], value, slope);
          else act_grad<QLORA_ACT_GELU_TANH>(g[h][e], value, slope);
          v[h][e] = e < left[h] ? v[h][e] * (j.src == SRC_GATE ? u[h][e] * slope : value) : 0.f;
        }
      }
  }
  const int planes = max(j.rowwise.n, j.across.n);
  uint16_t p[2][8][3];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (j.drawn && left[h] > 0) {
      const u32x4_t w = philox(philox_key(ps.sd), (uint32_t)(k >> 3), (uint32_t)row[h]);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[h][e] = keeps(w, e, ps.sd.threshold) ? v[h][e] : 0.f;
      if (j.bits) {
        uint32_t b = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) b |= keeps(w, e, ps.sd.threshold) ? 1u << e : 0u;
        j.bits[row[h] * j.wbits + (k >> 3)] = (uint8_t)b;
      }
    }
    u32x4_t o[MAX];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (CD == CD_F32 && j.src == SRC_NF4) {
        uint32_t w[3];
        cut3(v[h][e], w);
#pragma unroll
        for (int q = 0; q < 3; ++q) p[h][e][q] = (uint16_t)(w[q] >> 16);
      } else {
        split<KD>(v[h][e], planes, p[h][e]);
      }
#pragma unroll
      for (int q = 0; q < MAX; ++q)
        if (q < planes) o[q][e >> 1] = e & 1 ? o[q][e >> 1] | (uint32_t)p[h][e][q] << 16 : p[h][e][q];
    }
    if (j.rowwise.p && row[h] < j.rows && k < j.wide) {
#pragma unroll
      for (int q = 0; q < MAX; ++q)
        if (q < j.rowwise.n) *(u32x4_t*)(j.rowwise.p + row[h] * j.rowwise.ld + q * j.rowwise.step + k) = o[q];
    }
  }
  if (!j.across.p) return;
#pragma unroll
  for (int q = 0; q < MAX; ++q)
    if (q < j.across.n) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        *(uint32_t*)(tile[q] + chunk_at(8 * c + e, r >> 2) + 4 * (r & 3)) = p[0][e][q] | (uint32_t)p[1][e][q] << 16;
    }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int y = r + 32 * h;
    if (k0 + y < j.cols && i0 + 8 * c < j.tall) {
#pragma unroll
      for (int q = 0; q < MAX; ++q)
        if (q < j.across.n)
          *(u32x4_t*)(j.across.p + (k0 + y) * j.across.ld + q * j.across.step + i0 + 8 * c) =
              *(const u32x4_t*)(tile[q] + chunk_at(y, c));
    }
  }
}

// ----------------------------------------------------------------------- product
// One stretch of a contraction: planes of a against planes of b, `seq` the pairs of planes (four bits
// each: plane of a, plane of b << 2) that every 64 elements go through.
struct Seg {
  const uint16_t *a, *b;
  int64_t lda, ldb;
  int32_t stepa, stepb, pairs, KM;
  uint32_t seq;
  int32_t w;  // b is weight w - 1 from its codes (k_decode), w < 0: weight -w - 1 across its rows; 0: planes
};
constexpr int kSegs = 4;
struct Prod {
  Seg s[kSegs];
  int64_t m, n;
  float* part;        // [S][m][ldp] fp32, or null:
  void* out;          // [m][ldo] in the call's type
  int64_t ldp, ldo;
  const void* bias;   // with out
  int32_t nseg, steps, per, S, tiles_m, tiles_n;  // steps in all, and per slice
};
constexpr int kProds = 6;
struct Prods {
  uint32_t end[kProds];
  Prod p[kProds];
};

template <class T>
struct CopiesP {
  static constexpr int NW = T::NW, WAVES = NW, PER = T::PER;
  const Prod& p;
  int KT, left, g, k, q, lane;
  int64_t m0, n0, rows, cols;
  int arow, chunk;
  rsrc_t ra, rb;
  uint32_t oa, ob, sa, sb, soa, sob;
  int wave;
  __device__ __forceinline__ CopiesP(const Prod& p_, int64_t m0_, int64_t n0_, int first, int count, int wave_, int lane_)
      : p(p_), KT(count), left(count), lane(lane_), m0(m0_), n0(n0_), wave(wave_) {
    rows = min((int64_t)T::TM, p.m - m0);
    cols = min((int64_t)T::TN, p.n - n0);
    arow = 8 * wave + (lane >> 3);
    chunk = (lane & 7) ^ swz(arow);
    g = 0;
    while (g + 1 < p.nseg && first >= p.s[g].pairs * p.s[g].KM) first -= p.s[g].pairs * p.s[g].KM, ++g;
    k = first / p.s[g].pairs;
    q = first - k * p.s[g].pairs;
    enter();
  }
  __device__ __forceinline__ void enter() {
    const Seg& e = p.s[g];
    ra = make_rsrc(e.a + m0 * e.lda, rows * e.lda * 2);
    rb = make_rsrc(e.b + n0 * e.ldb, cols * e.ldb * 2);
    oa = (uint32_t)(arow * (int)e.lda * 2 + 16 * chunk);
    ob = (uint32_t)(arow * (int)e.ldb * 2 + 16 * chunk);
    sa = (uint32_t)(8 * NW * (int)e.lda * 2);
    sb = (uint32_t)(8 * NW * (int)e.ldb * 2);
  }
  // the stages come in order
  __device__ __forceinline__ void begin(int) {
    if (left <= 0) {
      ra = rb = make_rsrc(p.s[0].a, 0);
      return;
    }
    const Seg& e = p.s[g];
    const uint32_t pair = e.seq >> (4 * q);
    soa = (uint32_t)(((pair & 3u) * (uint32_t)e.stepa + 64u * (uint32_t)k) * 2u);
    sob = (uint32_t)((((pair >> 2) & 3u) * (uint32_t)e.stepb + 64u * (uint32_t)k) * 2u);
  }
  __device__ __forceinline__ void next() {
    if (--left <= 0) return;
    if (++q == p.s[g].pairs) {
      q = 0;
      if (++k == p.s[g].KM) {
        k = 0;
        ++g;
        enter();
      }
    }
  }
  __device__ __forceinline__ void one(char* dst, int, int i) {
    char* d = dst + (wave + NW * i) * 1024;
    if (i < T::PER_A) copy16(ra, d, oa + i * sa, soa);
    else copy16(rb, d, ob + (i - T::PER_A) * sb, sob);
    if (i == T::PER - 1) next();
  }
  __device__ __forceinline__ void all(char* dst) {
    begin(0);
#pragma unroll
    for (int i = 0; i < T::PER; ++i) one(dst, 0, i);
  }
  __device__ __forceinline__ void scales(int, int (&)[T::WMB], int&) const {}
  __device__ __forceinline__ void shift(int, int (&)[2][T::WMB], int (&)[2]) const {}
};

// A workgroup forms one tile of one slice of one product.  Small calls are launches and waits for memory (6 to 10 us
// a launch); large ones the matrix pipes (fp32, 4000 x 3968 x 4096, seeded forward: 860 us, of which six
// products of planes at 0.9 PFLOP/s).
template <int CD, class T>
__global__ __launch_bounds__(64 * T::NW) void k_product(Prods ps) {
  constexpr int KD = CD == CD_F32 ? CD_BF16 : CD;
  __shared__ __attribute__((aligned(1024))) char lds[T::LDS];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  uint32_t start;
  const Prod& p = ps.p[job_of(ps.end, blockIdx.x, start)];
  const int tiles = p.tiles_m * p.tiles_n, b = (int)(blockIdx.x - start);
  int z = 0, t;
  int tm, tn;
  if (p.S == 1) {
    t = xcd_run(b, tiles);
  } else {
    z = b / tiles;
    t = b - z * tiles;
  }
  grouped_tile(t, p.tiles_m, p.tiles_n, tm, tn);
  const int64_t m0 = (int64_t)__builtin_amdgcn_readfirstlane(tm) * T::TM;
  const int64_t n0 = (int64_t)__builtin_amdgcn_readfirstlane(tn) * T::TN;
  z = __builtin_amdgcn_readfirstlane(z);
  CopiesP<T> cp(p, m0, n0, z * p.per, min(p.per, p.steps - z * p.per), wave, lane);
  Acc<T> acc;
  zero<T>(acc);
#pragma unroll
  for (int s = 0; s < T::NS; ++s) cp.all(lds + s * T::STAGE);
  wait_vmcnt<(T::NS - 1) * T::PER>();
  wait_lgkm0();
  barrier_only();
  contract<T, Half16<KD>>(acc, lds, cp, wave, lane);

  const int h = lane >> 5, r32 = lane & 31;
  const int64_t row0 = m0 + (wave / T::NWN) * 32 * T::WMB + r32, col0 = n0 + (wave % T::NWN) * 32 * T::WNB + 4 * h;
  float* part = p.part ? p.part + (int64_t)z * p.m * p.ldp : nullptr;
#pragma unroll
  for (int i = 0; i < T::WMB; ++i) {
    const int64_t row = row0 + 32 * i;
    if (row >= p.m) continue;
#pragma unroll
    for (int j = 0; j < T::WNB; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t col = col0 + 32 * j + 8 * q;
        if (col >= p.n) continue;
        f32x4_t v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        if (part) {
          *(f32x4_t*)(part + row * p.ldp + col) = v;  // ldp is a multiple of four
          continue;
        }
        const bool whole = col + 4 <= p.n;
        if (p.bias) {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] += whole || col + e < p.n ? load_cd<CD>(p.bias, col + e) : 0.f;
        }
        const int64_t at = row * p.ldo + col;
        if (whole && CD == CD_F32 && (at & 3) == 0) *(f32x4_t*)((float*)p.out + at) = v;
        else if (whole && CD != CD_F32 && (at & 3) == 0)
          *(u32x2_t*)((uint16_t*)p.out + at) = u32x2_t{pack2<KD>(v[0], v[1]), pack2<KD>(v[2], v[3])};
        else
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (col + e < p.n) store_cd<CD>(p.out, at + e, v[e]);
      }
  }
}

// The same where b may be W~ from its codes, which every row of tiles decodes anew: products of few rows,
// weights whose blocks are powers of two of 32 or more within a row.  A stage of such a product is 64
// elements of all planes; of planes it is one pair.  The codes come three stages ahead into registers
// (a stage is shorter than a read from memory), the copies of the other operand one; a stage's codes
// are decoded into the buffer that the products of the stage before do not read.
// 64 tokens of 14336 x 4096, bf16: 31 us; the vector pipe's and the LDS's work are some 10 us each, the rest
// waits that three workgroups to a compute unit do not cover.  64 tokens of 5319 x 11200 across: 38 us, in place of 59 for
// W~^T written and 29 for the product; fp32, 8 tokens of two weights of 10624 x 9728: 263 us in place of 428 and 438.
struct Weights {
  Nf4W w[2];
  float lv[16];
};
template <int CD, class T>
struct Decode {
  static constexpr int KD = CD == CD_F32 ? CD_BF16 : CD, P = CD == CD_F32 ? 3 : 1, THREADS = 64 * T::NW;
  static constexpr int A = T::TM * 128, B = T::TN * 128, STAGE = P * (A + B);
  static constexpr int CA = T::TM / 8 / T::NW, CB = T::TN / 8 / T::NW;  // copies of a plane by a wave
  static constexpr int WORDS = T::TN * 64 / 8 / THREADS;                // of eight codes to a thread and stage
  static constexpr int AHEAD = 3;
  static_assert(T::TN == 128 && CA * 8 * T::NW == T::TM && (WORDS == 2 || WORDS == 4), "whole copies");
  using K = Half16<KD>;
  struct Raw {
    uint32_t word[WORDS], scale[2];
    float second[2];
  };

  // The weights of a word of eight codes: element e is the high half of byte e / 2 first.
  __device__ static __forceinline__ void weights(const char* lv, uint32_t c, float s, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int bit = 4 * (e ^ 1);
      const uint32_t four = bit >= 2 ? c >> (bit - 2) : c << 2;
      const float l = *(const float*)(lv + (four & 60u));
      v[e] = CD == CD_F16 ? fl32_mul(l, s) : l * s;
    }
  }
  // A stage's products: PAIRS of planes (or one).
  template <bool ALL>
  __device__ static __forceinline__ void multiply(Acc<T>& acc, const char* now, int wave, int lane) {
    constexpr int N = ALL ? P : 1;
    const int h = lane >> 5, r32 = lane & 31, xr = swz(r32);
    const char* a = now + ((wave / T::NWN) * 32 * T::WMB + r32) * 128;
    const char* b = now + P * A + ((wave % T::NWN) * 32 * T::WNB + r32) * 128;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      i32x4_t fa[N][T::WMB], fb[N][T::WNB];
#pragma unroll
      for (int s = 0; s < N; ++s) {
#pragma unroll
        for (int i = 0; i < T::WMB; ++i) fa[s][i] = K::read(a + s * A + i * 32 * 128, ks, h, xr);
#pragma unroll
        for (int j = 0; j < T::WNB; ++j) fb[s][j] = K::read(b + s * B + j * 32 * 128, ks, h, xr);
      }
#pragma unroll
      for (int sa = 0; sa < N; ++sa)
#pragma unroll
        for (int sb = 0; sa + sb < N; ++sb)
#pragma unroll
          for (int i = 0; i < T::WMB; ++i)
#pragma unroll
            for (int j = 0; j < T::WNB; ++j) K::mma(acc[i][j], fb[sb][j], fa[sa][i], 0, 0);
    }
  }
  // Copies of 64 elements of rows of `ld` elements, R of them to a wave.
  template <int R>
  __device__ static __forceinline__ void copies(rsrc_t r, char* dst, int64_t ld, uint32_t so, int wave, int lane) {
    const int row = 8 * wave + (lane >> 3), chunk = (lane & 7) ^ swz(row);
    const uint32_t o = (uint32_t)(row * (int)ld * 2 + 16 * chunk), step = (uint32_t)(8 * T::NW * (int)ld * 2);
#pragma unroll
    for (int i = 0; i < R; ++i) copy16(r, dst + (wave + T::NW * i) * 1024, o + i * step, so);
  }

  // Stages first .. first + KT - 1 of planes against planes.
  __device__ static __forceinline__ void plain(Acc<T>& acc, char* lds, const Prod& p, int first, int KT, int64_t m0,
                                               int64_t n0, int wave, int lane) {
    const Seg& e = p.s[0];
    const rsrc_t ra = make_rsrc(e.a + m0 * e.lda, min((int64_t)T::TM, p.m - m0) * e.lda * 2);
    const rsrc_t rb = make_rsrc(e.b + n0 * e.ldb, min((int64_t)T::TN, p.n - n0) * e.ldb * 2);
    auto ask = [&](int u, char* buf) {
      const int k = (first + u) / e.pairs;
      const uint32_t pair = e.seq >> (4 * (first + u - k * e.pairs));
      copies<CA>(ra, buf, e.lda, ((pair & 3u) * (uint32_t)e.stepa + 64u * (uint32_t)k) * 2u, wave, lane);
      copies<CB>(rb, buf + P * A, e.ldb, (((pair >> 2) & 3u) * (uint32_t)e.stepb + 64u * (uint32_t)k) * 2u, wave, lane);
    };
    ask(0, lds);
    for (int u = 0; u < KT; ++u) {
      __builtin_amdgcn_s_waitcnt(0);
      barrier_only();
      if (u + 1 < KT) ask(u + 1, lds + ((u & 1) ^ 1) * STAGE);
      multiply<false>(acc, lds + (u & 1) * STAGE, wave, lane);
    }
  }

  // The same against W~ (ACROSS: W~^T).  A thread takes 8 WORDS codes of a row of W, or (across) 4 WORDS of
  // two neighbouring rows, whose values it stores as words of two.
  template <bool ACROSS>
  __device__ static __forceinline__ void coded(Acc<T>& acc, char* lds, const char* lv, const Prod& p, const Nf4W& w,
                                               int first, int KT, int64_t m0, int64_t n0, int wave, int lane) {
    constexpr int ROWS = ACROSS ? 2 : 1, EACH = WORDS / ROWS;
    const Seg& e = p.s[0];
    const rsrc_t ra = make_rsrc(e.a + m0 * e.lda, min((int64_t)T::TM, p.m - m0) * e.lda * 2);
    const int tid = 64 * wave + lane, t = tid & 31;
    const int64_t r0 = ACROSS ? 64 * (int64_t)first + 2 * t : n0 + tid / (8 / WORDS);
    const int64_t c0 = ACROSS ? n0 + 4 * WORDS * (tid >> 5) : 64 * (int64_t)first + 8 * WORDS * (tid % (8 / WORDS));
    const int64_t at0 = r0 * w.cols + c0, step = ACROSS ? 64 * w.cols : 64;
    // rows of W from here on, counted from r0, are not there
    const int64_t rows = (ACROSS ? c0 < w.cols : r0 < w.rows) ? w.rows - r0 : 0;
    const bool dq = w.dq != 0;
    const uint8_t *codes = w.codes, *absmax_q = w.absmax_q;
    const float *absmax = w.absmax, *scale2 = w.scale2;
    const int bs_shift = w.bs_shift, g_shift = w.g_shift;
    auto load = [&](int u, Raw& o) {
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        const bool ok = u < KT && (ACROSS ? 64 * (int64_t)u + i : 0) < rows;
        const int64_t at = ok ? at0 + i * w.cols + u * step : 0, b = at >> bs_shift;
        if constexpr (EACH == 4) {
          const u32x4_t c = *(const u32x4_t*)(codes + (at >> 1));
#pragma unroll
          for (int x = 0; x < 4; ++x) o.word[x] = c[x];
        } else if constexpr (EACH == 2) {
          const u32x2_t c = *(const u32x2_t*)(codes + (at >> 1));
          o.word[2 * i] = c[0];
          o.word[2 * i + 1] = c[1];
        } else {
          o.word[i] = *(const uint32_t*)(codes + (at >> 1));
        }
        if (dq) {
          o.scale[i] = absmax_q[b];
          o.second[i] = scale2[b >> g_shift];
        } else {
          o.scale[i] = __float_as_uint(absmax[b]);
        }
        if (!ok) o.scale[i] = 0, o.second[i] = 0.f;
      }
    };
    auto decode = [&](const Raw& o, char* buf) {
      char* b = buf + P * A;
      float s[2];
#pragma unroll
      for (int i = 0; i < ROWS; ++i) s[i] = dq ? (float)o.scale[i] * o.second[i] : __uint_as_float(o.scale[i]);
#pragma unroll
      for (int i = 0; i < EACH; ++i) {
        float v[ROWS][8];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) weights(lv, o.word[i + r * EACH], s[r], v[r]);
        if constexpr (!ACROSS) {
          const int row = tid / (8 / WORDS), c = WORDS * (tid % (8 / WORDS)) + i;
          uint32_t w[4][P];
#pragma unroll
          for (int x = 0; x < 4; ++x) pack_weights<CD, P>(v[0][2 * x], v[0][2 * x + 1], w[x]);
#pragma unroll
          for (int u = 0; u < P; ++u)
            *(u32x4_t*)(b + u * B + row * 128 + ((c ^ swz(row)) << 4)) = u32x4_t{w[0][u], w[1][u], w[2][u], w[3][u]};
        } else {
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const int row = 4 * WORDS * (tid >> 5) + 8 * i + x;
            uint32_t w[P];
            pack_weights<CD, P>(v[0][x], v[ROWS - 1][x], w);
#pragma unroll
            for (int u = 0; u < P; ++u)
              *(uint32_t*)(b + u * B + row * 128 + (((t >> 2) ^ swz(row)) << 4) + 4 * (t & 3)) = w[u];
          }
        }
      }
    };
    auto ask = [&](int u, char* buf) {
#pragma unroll
      for (int q = 0; q < P; ++q)
        copies<CA>(ra, buf + q * A, e.lda, ((uint32_t)q * (uint32_t)e.stepa + 64u * (uint32_t)(first + u)) * 2u, wave, lane);
    };
    Raw raw[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) load(i, raw[i]);
    ask(0, lds);
    decode(raw[0], lds);
    for (int u0 = 0; u0 < KT; u0 += AHEAD) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int u = u0 + i;
        if (u >= KT) break;
        char *now = lds + (u & 1) * STAGE, *next = lds + ((u & 1) ^ 1) * STAGE;
        // this wave's copies of the stage (at least 2 ROWS loads of codes and scales left after them) and its
        // decoded rows
        __builtin_amdgcn_sched_barrier(0);
        if (u == 0) wait_vmcnt<0>();
        else wait_vmcnt<2 * ROWS>();
        wait_lgkm0();
        barrier_only();
        if (u + 1 < KT) ask(u + 1, next);
        __builtin_amdgcn_sched_barrier(0);
        load(u + AHEAD, raw[i]);
        __builtin_amdgcn_sched_barrier(0);
        multiply<true>(acc, now, wave, lane);
        decode(raw[(i + 1) % AHEAD], next);
      }
    }
  }
};

template <int CD, class T>
__global__ __launch_bounds__(64 * T::NW) void k_decode(Prods ps, Weights ws) {
  using D = Decode<CD, T>;
  __shared__ __attribute__((aligned(1024))) char lds[2 * D::STAGE];
  __shared__ float lv[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  uint32_t start;
  const Prod& p = ps.p[job_of(ps.end, blockIdx.x, start)];
  const int tiles = p.tiles_m * p.tiles_n, b = (int)(blockIdx.x - start);
  const int z = b / tiles, t = b - z * tiles;
  const int64_t m0 = (int64_t)(t % p.tiles_m) * T::TM, n0 = (int64_t)(t / p.tiles_m) * T::TN;
  const int first = z * p.per, KT = min(p.per, p.steps - first), kind = p.s[0].w;
  if (tid < 16) lv[tid] = ws.lv[tid];
  __syncthreads();
  Acc<T> acc;
  zero<T>(acc);
  if (kind > 0) D::template coded<false>(acc, lds, (const char*)lv, p, ws.w[kind - 1], first, KT, m0, n0, wave, lane);
  else if (kind < 0) D::template coded<true>(acc, lds, (const char*)lv, p, ws.w[-kind - 1], first, KT, m0, n0, wave, lane);
  else D::plain(acc, lds, p, first, KT, m0, n0, wave, lane);

  const int h = lane >> 5, r32 = lane & 31;
  const int64_t row0 = m0 + (wave / T::NWN) * 32 * T::WMB + r32, col0 = n0 + (wave % T::NWN) * 32 * T::WNB + 4 * h;
  float* part = p.part + (int64_t)z * p.m * p.ldp;
#pragma unroll
  for (int i = 0; i < T::WMB; ++i)
#pragma unroll
    for (int j = 0; j < T::WNB; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t row = row0 + 32 * i, col = col0 + 32 * j + 8 * v;
        if (row < p.m && col < p.n)
          *(f32x4_t*)(part + row * p.ldp + col) =
              f32x4_t{acc[i][j][4 * v], acc[i][j][4 * v + 1], acc[i][j][4 * v + 2], acc[i][j][4 * v + 3]};
      }
}

// -------------------------------------------------------------------------- join
enum JoinKind { JOIN_OUT, JOIN_RANK, JOIN_GATE };
struct Join {
  int kind = JOIN_OUT, S = 0;
  const float* part = nullptr;  // [S][m][ldp]
  const float* low = nullptr;   // [m][ldp], JOIN_OUT: added under the drawn mask; JOIN_GATE: the up projection's parts
  int64_t m = 0, n = 0, ldp = 0;
  float scale = 1.f;
  const void* bias = nullptr;
  void* out = nullptr;  // [m][n] of type `type`: scale * sum (+ bias); JOIN_GATE: h
  int type = 0;
  void* pre = nullptr;  // JOIN_GATE: [m][2 n] or null
  float* raw = nullptr;  // JOIN_RANK: the sums [m][n] or null
  Planes rowwise, across;  // JOIN_RANK: scale * sum, [m][wide] and [n][tall]
  int64_t wide = 0, tall = 0;
  uint32_t per = 0;  // groups of four columns to a row
};
constexpr int kJoins = 6;
struct Joins {
  uint32_t end[kJoins];
  Join j[kJoins];
  Seeded sd;
  int act;
};

__device__ __forceinline__ f32x4_t sum_of(const float* part, int S, int64_t stride, int64_t at) {
  f32x4_t s = *(const f32x4_t*)(part + at);
  for (int z = 1; z < S; z += 4) {  // four loads are on their way at once
    f32x4_t v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = *(const f32x4_t*)(part + (z + e < S ? z + e : 0) * stride + at);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (z + e < S) s += v[e];
  }
  return s;
}
__device__ __forceinline__ void store_any(int type, void* p, int64_t at, float v) {
  if (type == CD_F32) store_cd<CD_F32>(p, at, v);
  else if (type == CD_BF16) store_cd<CD_BF16>(p, at, v);
  else store_cd<CD_F16>(p, at, v);
}
__device__ __forceinline__ void store4(int type, void* p, int64_t at, const f32x4_t& v, int left) {
  if (left >= 4 && (at & 3) == 0) {
    if (type == CD_F32) *(f32x4_t*)((float*)p + at) = v;
    else if (type == CD_BF16) *(u32x2_t*)((uint16_t*)p + at) = u32x2_t{pack2<CD_BF16>(v[0], v[1]), pack2<CD_BF16>(v[2], v[3])};
    else *(u32x2_t*)((uint16_t*)p + at) = u32x2_t{pack2<CD_F16>(v[0], v[1]), pack2<CD_F16>(v[2], v[3])};
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < left) store_any(type, p, at + e, v[e]);
}

// A thread takes four columns of a row.
template <int CD>
__global__ __launch_bounds__(kThreads) void k_join(Joins js) {
  constexpr int KD = CD == CD_F32 ? CD_BF16 : CD;
  uint32_t first;
  const Join& j = js.j[job_of(js.end, blockIdx.x, first)];
  const int64_t idx = (int64_t)(blockIdx.x - first) * kThreads + threadIdx.x;
  if (j.kind == JOIN_RANK) {
    // rows next to each other in neighbouring lanes: the transposed planes are written in lines
    const int64_t rows = max(j.m, j.tall), g = idx / rows, i = idx - g * rows, t = 4 * g;
    if (g >= j.per) return;
    f32x4_t s = {0.f, 0.f, 0.f, 0.f};
    if (i < j.m && t < j.n) s = sum_of(j.part, j.S, j.m * j.ldp, i * j.ldp + t);
    uint16_t h[4][3];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (j.raw && i < j.m && t + e < j.n) j.raw[i * j.n + t + e] = s[e];
      split<KD>(t + e < j.n ? j.scale * s[e] : 0.f, max(j.rowwise.n, j.across.n), h[e]);
    }
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      if (j.rowwise.p && q < j.rowwise.n && i < j.m && t < j.wide)
        *(u32x2_t*)(j.rowwise.p + i * j.rowwise.ld + q * j.rowwise.step + t) =
            u32x2_t{h[0][q] | (uint32_t)h[1][q] << 16, h[2][q] | (uint32_t)h[3][q] << 16};
      if (j.across.p && q < j.across.n && i < j.tall) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (t + e < j.n) j.across.p[(t + e) * j.across.ld + q * j.across.step + i] = h[e][q];
      }
    }
    return;
  }
  const int64_t i = idx / j.per, k = 4 * (idx - i * j.per);
  if (i >= j.m) return;
  const int64_t at = i * j.ldp + k;
  const int left = (int)min((int64_t)4, j.n - k);
  f32x4_t s = sum_of(j.part, j.S, j.m * j.ldp, at);
  if (j.kind == JOIN_OUT) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[e] *= j.scale;
      if (j.bias && e < left) s[e] += load_cd<CD>(j.bias, k + e);
    }
    if (j.low) {
      const f32x4_t l = *(const f32x4_t*)(j.low + at);
      const u32x4_t w = philox(philox_key(js.sd), (uint32_t)(k >> 3), (uint32_t)i);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] += keeps(w, (int)(k & 4) + e, js.sd.threshold) ? l[e] : 0.f;
    }
    store4(j.type, j.out, i * j.n + k, s, left);
    return;
  }
  f32x4_t u = sum_of(j.low, j.S, j.m * j.ldp, at), o;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (j.bias && e < left) {
      s[e] += load_cd<CD>(j.bias, k + e);
      u[e] += load_cd<CD>(j.bias, j.n + k + e);
    }
    o[e] = (js.act == QLORA_ACT_SILU ? act_of<QLORA_ACT_SILU>(s[e])
            : js.act == QLORA_ACT_GELU ? act_of<QLORA_ACT_GELU>(s[e])
                                       : act_of<QLORA_ACT_GELU_TANH>(s[e])) * u[e];
  }
  store4(CD, j.out, i * j.n + k, o, left);
  if (j.pre) {
    store4(CD, j.pre, 2 * i * j.n + k, s, left);
    store4(CD, j.pre, (2 * i + 1) * j.n + k, u, left);
  }
}

// -------------------------------------------------------------------------- host
using Low = Tile<1, 2, 2, 2, 3>;   // 64 x 128, four waves; two workgroups fit a compute unit
using Wide = Tile<2, 2, 2, 4, 3>;  // 128 x 256, eight waves
// k_decode's: 64 or 128 x 128, four waves and 48 or 64 KB of LDS; with three planes 64 x 128, eight waves, 144 KB
using FewRows = Tile<1, 2, 2, 2, 2>;
using SomeRows = Tile<2, 2, 2, 2, 2>;
using FewRows3 = Tile<1, 1, 2, 4, 2>;

// One call: its workspace (sizing: only its size is wanted), and its launches' job lists.
template <int CD>
struct Run {
  static constexpr int kPlanes = CD == CD_F32 ? 3 : 1;      // of an operand
  static constexpr int kRankPlanes = CD == CD_F32 ? 3 : 2;  // of T and dT
  char* base;
  bool sizing;
  hipStream_t s;
  int64_t used = 0;
  Packs packs = {};
  Prods prods = {};
  Joins joins = {};
  int np = 0, nj = 0, rc = QLORA_OK;
  bool big = false, decodes = false;

  bool dry() const { return sizing; }
  void* take(int64_t bytes) {
    void* p = sizing ? nullptr : base + used;
    used += round_up(bytes, 256);
    return p;
  }
  Planes planes(int64_t rows, int64_t cols, int n) {
    Planes o;
    o.step = round_up(cols, 64);
    o.ld = o.step * n;
    o.n = n;
    o.p = (uint16_t*)take(rows * o.ld * 2);
    return o;
  }
  // A matrix that lies in the form of an operand already.
  Planes as_is(const void* p, int64_t cols) {
    Planes o;
    o.p = (uint16_t*)p;
    o.ld = o.step = cols;
    return o;
  }

  Pack& pack(int src, const void* p, int64_t rows, int64_t cols) {
    Pack& j = packs.j[packs.n++];
    j = Pack();
    j.src = src;
    j.p = p;
    j.rows = rows;
    j.cols = cols;
    j.rowwise.n = j.across.n = 0;
    return j;
  }
  Planes rowwise(Pack& j, int n = kPlanes) {
    j.wide = round_up(j.cols, 64);
    return j.rowwise = planes(j.rows, j.cols, n);
  }
  Planes across(Pack& j, int n = kPlanes) {
    j.tall = round_up(j.rows, 64);
    return j.across = planes(j.cols, j.rows, n);
  }
  // [rows][cols] of the call's type as a row operand
  Planes operand(const void* p, int64_t rows, int64_t cols, bool drawn = false) {
    if (kPlanes == 1 && cols % 64 == 0 && !drawn) return as_is(p, cols);
    Pack& j = pack(SRC_CD, p, rows, cols);
    j.drawn = drawn;
    return rowwise(j);
  }
  void run_packs(const LayerCall* c, int g, const Seeded* sd, int act) {
    int64_t blocks = 0;
    for (int i = 0; i < packs.n; ++i) {
      Pack& j = packs.j[i];
      const int64_t rows = std::max(j.rows, j.across.n ? j.tall : 0), cols = std::max(j.cols, j.rowwise.n ? j.wide : 0);
      j.tiles_x = (uint32_t)ceil_div(cols, 64);
      blocks += j.tiles_x * ceil_div(rows, 64);
      if (blocks > 0x7fffffff) return fail();
      packs.end[i] = (uint32_t)blocks;
    }
    for (int i = packs.n; i < kPacks; ++i) packs.end[i] = 0xffffffffu;
    if (dry() || rc || blocks == 0) return;
    for (int i = 0; i < g; ++i) packs.w[i] = c[i].w;
    for (int i = 0; i < 16; ++i) packs.lv[i] = host_tables().lv[i];
    if (sd) packs.sd = *sd;
    packs.act = act;
    ProfScope prof(QLORA_K_DEQUANTIZE, s);
    k_pack<CD><<<dim3((unsigned)blocks), dim3(kThreads), 0, s>>>(packs);
    rc = check_launch("k_pack");
  }

  void fail() {
    rc = set_error(QLORA_ERR_UNSUPPORTED, "layer: operand too large");
  }
  static Seg seg(const Planes& a, const Planes& b, int64_t k) {
    Seg e = {};
    e.a = a.p;
    e.b = b.p;
    e.lda = a.ld;
    e.ldb = b.ld;
    e.stepa = (int32_t)a.step;
    e.stepb = (int32_t)b.step;
    e.KM = (int32_t)ceil_div(k, 64);
    // the pairs of planes whose product is not below the last bits kept
    const int deepest = std::max(a.n, b.n);
    for (int i = 0; i < a.n; ++i)
      for (int l = 0; l < b.n && i + l < deepest; ++l) e.seq |= (uint32_t)(i | l << 2) << (4 * e.pairs++);
    return e;
  }
  // a against W~ of weight i (across: W~^T) from its codes
  Seg seg_w(const Planes& a, int i, bool across, int64_t k) {
    decodes = true;
    Seg e = seg(a, Planes(), k);
    e.pairs = 1;
    e.seq = 0;
    e.w = across ? -(i + 1) : i + 1;
    return e;
  }
  Prod& product(int64_t m, int64_t n) {
    Prod& p = prods.p[np++];
    p = Prod{};
    p.m = m;
    p.n = n;
    p.S = 1;
    p.ldp = round_up(n, 4);
    return p;
  }
  static void add(Prod& p, const Seg& e) {
    p.s[p.nseg++] = e;
    p.steps += e.pairs * e.KM;
  }
  static int64_t low_tiles(int64_t m, int64_t n) {
    return std::max<int64_t>(1, ceil_div(m, Low::TM) * ceil_div(n, Low::TN));  // a query may have no tokens
  }
  // Slices of a contraction: workgroups for every compute unit, at least four stages to each (bf16 calls of 16 to 333
  // tokens take 2 to 6 % more at one stage, the same at six; fp32 ones are best at two of the longer stages that
  // decode: 42 tokens of 1472 x 1280, seeded backward, 41, 39.1, 42.0, 47.5 us at 1, 2, 4, 6).
  static int slices(int64_t m, int64_t n, int steps) {
    return (int)std::max<int64_t>(1, std::min<int64_t>({ceil_div(256, low_tiles(m, n)), steps / 4, 32}));
  }
  // The same where the product decodes: as many workgroups as run at once (48 KB of LDS each, 64 KB, 144 KB).
  static int decode_slices(int64_t m, int64_t n, int steps) {
    const int64_t at_once = 256 * (CD == CD_F32 ? 1 : m <= FewRows::TM ? 3 : 2);
    const int64_t tiles = ceil_div(n, 128) * ceil_div(m, CD == CD_F32 || m <= FewRows::TM ? 64 : 128);
    return (int)std::max<int64_t>(1, std::min<int64_t>({at_once / std::max<int64_t>(1, tiles), steps / (CD == CD_F32 ? 2 : 4), 32}));
  }
  // partial sums of p for S slices, and of `more` - 1 products alike and `extra` slices of another behind them
  float* parts(Prod& p, int S, int extra = 0, int more = 1) {
    p.per = std::max(1, (int)ceil_div(p.steps, S));
    p.S = std::max(1, (int)ceil_div(p.steps, p.per));
    return p.part = (float*)take((more * p.S + extra) * p.m * p.ldp * 4);
  }
  template <class T, bool DECODE>
  void launch(int kind, const LayerCall* c, int g) {
    int64_t blocks = 0;
    for (int i = 0; i < np; ++i) {
      Prod& p = prods.p[i];
      if (p.per == 0) p.per = p.steps;
      const int64_t tm = ceil_div(p.m, T::TM), tn = ceil_div(p.n, T::TN);
      blocks += tm * tn * p.S;
      if (blocks > 0x7fffffff) return fail();
      p.tiles_m = (int32_t)tm;
      p.tiles_n = (int32_t)tn;
      prods.end[i] = (uint32_t)blocks;
      for (int e = 0; e < p.nseg; ++e)
        if (std::max(p.s[e].lda, p.s[e].ldb) * 2 * std::max(T::TM, T::TN) >= (1LL << 31)) return fail();
    }
    for (int i = np; i < kProds; ++i) prods.end[i] = 0xffffffffu;
    if (dry() || rc || blocks == 0) return;
    ProfScope prof(kind, s);
    const dim3 grid((unsigned)blocks), threads(64 * T::NW);
    if constexpr (DECODE) {
      Weights w;
      for (int i = 0; i < g; ++i) w.w[i] = c[i].w;
      for (int i = 0; i < 16; ++i) w.lv[i] = host_tables().lv[i];
      k_decode<CD, T><<<grid, threads, 0, s>>>(prods, w);
    } else {
      k_product<CD, T><<<grid, threads, 0, s>>>(prods);
    }
    rc = check_launch(DECODE ? "k_decode" : "k_product");
  }
  void run_products(int kind, const LayerCall* c, int g) {
    if (decodes) {
      if constexpr (CD == CD_F32) launch<FewRows3, true>(kind, c, g);
      else if (c->m <= FewRows::TM) launch<FewRows, true>(kind, c, g);
      else launch<SomeRows, true>(kind, c, g);
    } else if (big) {
      launch<Wide, false>(kind, c, g);
    } else {
      launch<Low, false>(kind, c, g);
    }
    np = 0;
    decodes = false;
  }

  Join& join(int kind, const Prod& p, const float* part) {
    Join& j = joins.j[nj++];
    j = Join();
    j.kind = kind;
    j.S = p.S;
    j.part = part;
    j.m = p.m;
    j.n = p.n;
    j.ldp = p.ldp;
    j.type = CD;
    j.rowwise.n = j.across.n = 0;
    return j;
  }
  void run_joins(const Seeded* sd, int act) {
    int64_t blocks = 0;
    for (int i = 0; i < nj; ++i) {
      Join& j = joins.j[i];
      j.per = (uint32_t)ceil_div(std::max(j.n, j.wide), 4);
      const int64_t rows = std::max(j.m, j.tall);
      blocks += ceil_div(rows * j.per, kThreads);
      if (blocks > 0x7fffffff) return fail();
      joins.end[i] = (uint32_t)blocks;
    }
    for (int i = nj; i < kJoins; ++i) joins.end[i] = 0xffffffffu;
    if (!dry() && !rc && blocks) {
      if (sd) joins.sd = *sd;
      joins.act = act;
      ProfScope prof(QLORA_K_REDUCE, s);
      k_join<CD><<<dim3((unsigned)blocks), dim3(kThreads), 0, s>>>(joins);
      rc = check_launch("k_join");
    }
    nj = 0;
  }
};

// Tiles from which a product is not cut: its output leaves from the product itself (gated backward, us cut
// and not: 600 x 1501 x 960 bf16 53 and 66, fp32 98 and 172; 1000 x 3001 x 1984 bf16 113 and 107, fp32 372 and 329).
constexpr int64_t kDirectTiles = 160;
// Larger tiles from this many on (fp32, us with the small ones and these: seeded forward of 2000 x 2944 x 2048, 192
// of them, 237 and 202, of 4000 x 3968 x 4096, 512, 1115 and 860; gated backward of 2000 x 3001 x 2048, 128, 532 and 605).
constexpr int64_t kWideTiles = 176;
// Rows up to which W~ is decoded by the product that reads it: every 128 rows (64 in fp32) decode it
// again.  Written first and read back, the gated backward of 256 rows takes 122 us against 87 (4096 x 4096),
// 385 against 229 (14336 x 4096).
constexpr int64_t decode_rows(int cd) { return cd == CD_F32 ? 128 : 256; }
bool decodable(const LayerCall* c, int g) {
  for (int i = 0; i < g; ++i)
    if (!fast_layout(c[i].w) || c[i].w.bs_shift < 0 || (c[i].w.dq && c[i].w.g_shift < 0)) return false;
  return c[0].m <= decode_rows(c[0].cd);
}

template <int CD>
int forward(const PlanesFwd& q, char* ws, int64_t* need) {
  const LayerCall& c0 = q.c[0];
  const int64_t m = c0.m, n = c0.w.rows, K = c0.w.cols;
  const bool gated = q.g == 2;
  Run<CD> run;
  run.base = ws;
  run.sizing = need != nullptr;
  run.s = c0.stream;
  const bool decode = decodable(q.c, q.g);
  const bool direct = !decode && Run<CD>::low_tiles(m, n) * q.g >= kDirectTiles;
  // the gated GEMM with its own epilogue
  const bool fused = gated && direct && CD != CD_F32 && c0.r <= 64 && q.c[1].r <= 64 && gemm16_ok(CD, m, n, round_up(K, 64));

  const Planes x = run.operand(c0.x, m, K), xm = q.sd ? run.operand(c0.x, m, K, true) : x;
  Planes a[2], b[2], w[2], t[2];
  for (int i = 0; i < q.g; ++i) {
    const LayerCall& c = q.c[i];
    a[i] = run.operand(c.lora_a, c.r, K);
    b[i] = run.operand(c.lora_b, n, c.r);
    if (decode) continue;
    Pack& j = run.pack(SRC_NF4, nullptr, n, K);
    j.w = i;
    w[i] = run.rowwise(j);
  }
  run.run_packs(q.c, q.g, q.sd, 0);

  Prod rank[2], main[2];
  float* parts[2];
  for (int i = 0; i < q.g; ++i) {
    Prod& p = run.product(m, q.c[i].r);
    run.add(p, run.seg(xm, a[i], K));
    run.parts(p, run.slices(m, p.n, p.steps));
    rank[i] = p;
  }
  if (!direct) {
    int S = 32;
    for (int i = 0; i < q.g; ++i) {
      Prod& p = run.product(m, n);
      run.add(p, decode ? run.seg_w(x, i, false, K) : run.seg(x, w[i], K));
      S = std::min(S, decode ? run.decode_slices(m, q.g * n, p.steps) : run.slices(m, q.g * n, p.steps));
      parts[i] = run.parts(p, S, 1);
      main[i] = p;
    }
  }
  run.run_products(QLORA_K_FWD_GEMM, q.c, q.g);

  uint16_t* both = fused ? (uint16_t*)run.take(m * 128 * 2) : nullptr;
  for (int i = 0; i < q.g; ++i) {
    const LayerCall& c = q.c[i];
    Join& j = run.join(JOIN_RANK, rank[i], rank[i].part);
    j.raw = q.t_save ? q.t_save[i] : nullptr;
    j.scale = c.scale;
    j.wide = round_up(c.r, 64);
    if (fused) {
      j.rowwise.p = both ? both + 64 * i : nullptr;
      j.rowwise.ld = 128;
      j.rowwise.n = 1;
    } else {
      j.rowwise = run.planes(m, c.r, Run<CD>::kRankPlanes);
    }
    t[i] = j.rowwise;
  }
  run.run_joins(nullptr, 0);

  if (fused) {
    if (need) *need = run.used;
    if (run.dry() || run.rc) return run.rc;
    const void* wp[2] = {w[0].p, w[1].p};
    const void* bp[2] = {b[0].p, b[1].p};
    const int64_t ldb[2] = {b[0].ld, b[1].ld};
    return gemm16_gated(CD, x.p, m, n, x.ld, wp, both, bp, ldb, q.bias, q.act, q.out, q.pre, c0.stream);
  }
  // [g | u] where the gate reads it
  void* z = gated && direct ? (q.pre ? q.pre : run.take(m * 2 * n * cd_bytes(CD))) : q.out;
  for (int i = 0; i < q.g; ++i) {
    Prod& p = run.product(m, n);
    if (direct) {
      run.add(p, run.seg(x, w[i], K));
      p.out = (char*)z + i * n * cd_bytes(CD);
      p.ldo = q.g * n;
      p.bias = q.bias ? (const char*)q.bias + i * n * cd_bytes(CD) : nullptr;
    } else {
      p.part = run.dry() ? nullptr : parts[i] + main[i].S * m * p.ldp;
    }
    run.add(p, run.seg(t[i], b[i], q.c[i].r));
  }
  run.big = direct && ceil_div(m, Wide::TM) * ceil_div(n, Wide::TN) * q.g >= kWideTiles;
  run.run_products(QLORA_K_FWD_GEMM, q.c, q.g);
  if (!direct) {
    main[0].S += 1;  // and the low-rank part
    Join& j = run.join(gated ? JOIN_GATE : JOIN_OUT, main[0], parts[0]);
    j.bias = q.bias;
    j.out = q.out;
    j.pre = q.pre;
    if (gated) j.low = parts[1];
    run.run_joins(nullptr, q.act);
  }
  if (need) *need = run.used;
  if (run.dry() || run.rc || !gated || !direct) return run.rc;
  return gate(CD, q.act, z, m, n, q.out, c0.stream);
}

template <int CD>
int backward(const PlanesBwd& q, char* ws, int64_t* need) {
  const LayerCall& c0 = q.c[0];
  const int64_t m = c0.m, n = c0.w.rows, K = c0.w.cols;
  const bool gated = q.g == 2, g32 = q.gd == CD_F32;
  Run<CD> run;
  run.base = ws;
  run.sizing = need != nullptr;
  run.s = c0.stream;
  const bool decode = q.dx && decodable(q.c, q.g);
  const bool direct = q.dx && !decode && Run<CD>::low_tiles(m, K) >= kDirectTiles;
  // the masked GEMM adds the low-rank part itself
  const bool fused = direct && q.sd && CD != CD_F32 && c0.r <= 64 && gemm16_ok(CD, m, K, round_up(n, 64));
  const bool whole = direct && !q.sd;  // dX leaves from one product
  const bool saved = q.t_saved != nullptr;

  Planes d[2], dr[2], dt_[2], wt[2], at[2], bt[2], t0t[2], dtr[2], dtt[2], a[2], xm;
  for (int i = 0; i < q.g; ++i) {
    const LayerCall& c = q.c[i];
    if (gated) {
      Pack& j = run.pack(i ? SRC_UP : SRC_GATE, q.pre, m, n);
      j.dh = q.dy;
      // d B takes what the rounding of d to 16 bits leaves as a second plane: dA is the product of a small sum, whose
      // terms cancel
      dr[i] = run.rowwise(j, Run<CD>::kRankPlanes);
      d[i] = dr[i];
      d[i].n = Run<CD>::kPlanes;
      dt_[i] = run.across(j);
    } else {
      Pack& j = run.pack(SRC_CD, q.dy, m, n);
      d[i] = Run<CD>::kPlanes == 1 && n % 64 == 0 ? run.as_is(q.dy, n) : run.rowwise(j);
      dr[i] = d[i];
      dt_[i] = run.across(j);
    }
    bt[i] = run.across(run.pack(SRC_CD, c.lora_b, n, c.r));
    if (q.dx) {
      if (!decode) {
        Pack& j = run.pack(SRC_NF4, nullptr, n, K);
        j.w = i;
        wt[i] = run.across(j);
      }
      at[i] = run.across(run.pack(SRC_CD, c.lora_a, c.r, K));
    }
    if (saved) t0t[i] = run.across(run.pack(SRC_F32, q.t_saved[i], m, c.r), Run<CD>::kRankPlanes);
    else a[i] = run.operand(c.lora_a, c.r, K);
  }
  Pack& jx = run.pack(SRC_CD, c0.x, m, K);
  jx.drawn = q.sd != nullptr;
  if (fused) {
    jx.wbits = round_up(K, 32) / 8;
    jx.bits = (uint8_t*)run.take(m * jx.wbits);
  }
  const Planes xt = run.across(jx);
  if (!saved) xm = Run<CD>::kPlanes == 1 && K % 64 == 0 && !q.sd ? run.as_is(c0.x, K) : run.rowwise(jx);
  run.run_packs(q.c, q.g, q.sd, q.act);

  Prod rank[2], rank0[2], da[2], db[2], main = {};
  auto grad_b = [&](int i) {
    Prod& p = run.product(n, q.c[i].r);
    run.add(p, run.seg(dt_[i], t0t[i], m));
    run.parts(p, run.slices(n, p.n, p.steps));
    db[i] = p;
  };
  for (int i = 0; i < q.g; ++i) {
    Prod& p = run.product(m, q.c[i].r);
    run.add(p, run.seg(dr[i], bt[i], n));
    run.parts(p, run.slices(m, p.n, p.steps));
    rank[i] = p;
    if (saved) {
      grad_b(i);
    } else {
      Prod& o = run.product(m, q.c[i].r);
      run.add(o, run.seg(xm, a[i], K));
      run.parts(o, run.slices(m, o.n, o.steps));
      rank0[i] = o;
    }
  }
  float* parts = nullptr;
  if (q.dx && !whole && !fused) {
    Prod& p = run.product(m, K);
    for (int i = 0; i < (decode ? 1 : q.g); ++i) run.add(p, decode ? run.seg_w(d[i], i, true, n) : run.seg(d[i], wt[i], n));
    parts = run.parts(p, decode ? run.decode_slices(m, q.g * K, p.steps) : run.slices(m, K, p.steps), 1, decode ? q.g : 1);
    main = p;
    if (decode && gated) {  // one weight to a product: the second's slices behind the first's
      Prod& o = run.product(m, K);
      run.add(o, run.seg_w(d[1], 1, true, n));
      o.per = p.per;
      o.S = p.S;
      o.part = run.dry() ? nullptr : parts + p.S * m * p.ldp;
      main.S = 2 * p.S;
    }
  }
  run.run_products(QLORA_K_BWD_DX, q.c, q.g);

  for (int i = 0; i < q.g; ++i) {
    const LayerCall& c = q.c[i];
    Join& j = run.join(JOIN_RANK, rank[i], rank[i].part);
    j.scale = c.scale;
    j.wide = round_up(c.r, 64);
    j.tall = round_up(m, 64);
    if (q.dx) dtr[i] = j.rowwise = run.planes(m, c.r, fused ? 1 : Run<CD>::kRankPlanes);
    dtt[i] = j.across = run.planes(c.r, m, Run<CD>::kRankPlanes);
    if (!saved) {
      Join& o = run.join(JOIN_RANK, rank0[i], rank0[i].part);
      o.tall = round_up(m, 64);
      t0t[i] = o.across = run.planes(c.r, m, Run<CD>::kRankPlanes);
    }
  }
  run.run_joins(nullptr, 0);

  for (int i = 0; i < q.g; ++i) {
    Prod& p = run.product(q.c[i].r, K);
    run.add(p, run.seg(dtt[i], xt, m));
    run.parts(p, run.slices(p.m, K, p.steps));
    da[i] = p;
    if (!saved) grad_b(i);
  }
  if (parts || (run.dry() && q.dx && !whole && !fused)) {  // the low-rank part of dX, a slice of its own
    Prod& p = run.product(m, K);
    for (int i = 0; i < q.g; ++i) run.add(p, run.seg(dtr[i], at[i], q.c[i].r));
    p.part = run.dry() ? nullptr : parts + main.S * m * p.ldp;
  }
  run.run_products(QLORA_K_BWD_DA, q.c, q.g);
  if (whole) {
    Prod& p = run.product(m, K);
    for (int i = 0; i < q.g; ++i) run.add(p, run.seg(d[i], wt[i], n));
    for (int i = 0; i < q.g; ++i) run.add(p, run.seg(dtr[i], at[i], q.c[i].r));
    p.out = q.dx;
    p.ldo = K;
    run.big = ceil_div(m, Wide::TM) * ceil_div(K, Wide::TN) >= kWideTiles;
    run.run_products(QLORA_K_BWD_DX, q.c, q.g);
  }
  for (int i = 0; i < q.g && !run.dry(); ++i) {
    Join& ja = run.join(JOIN_OUT, da[i], da[i].part);
    ja.out = q.d_a[i];
    Join& jb = run.join(JOIN_OUT, db[i], db[i].part);
    jb.out = q.d_b[i];
    jb.scale = q.c[i].scale;
    ja.type = jb.type = g32 ? CD_F32 : CD;
  }
  if (parts) {
    main.S += q.sd ? 0 : 1;  // the low-rank part is the slice behind the last, under the mask if there is one
    Join& j = run.join(JOIN_OUT, main, parts);
    j.out = q.dx;
    if (q.sd) j.low = parts + main.S * m * main.ldp;
  }
  run.run_joins(q.sd, 0);
  if (need) *need = run.used;
  if (run.dry() || run.rc || !fused) return run.rc;
  return gemm16_masked_dx(CD, d[0].p, m, K, d[0].ld, wt[0].p, dtr[0].p, dtr[0].ld, at[0].p, at[0].ld, jx.bits,
                          jx.wbits / 4, q.dx,
                          c0.stream);
}

}  // namespace

// A call is sized before its first launch, so that one that does not fit, a launch or the workspace, is refused whole.
template <class Q>
int check_size(const Q& q, int (*plan)(const Q&, void*, int64_t*)) {
  int64_t n;
  if (const int rc = plan(q, nullptr, &n)) return rc;
  if ((uint64_t)n > q.c->ws_bytes)
    return set_error(QLORA_ERR_WORKSPACE, "layer: workspace %zu bytes < %lld required", q.c->ws_bytes, (long long)n);
  return QLORA_OK;
}
int planes_forward(const PlanesFwd& q, void* ws, int64_t* need) {
  if (!need)
    if (const int rc = check_size(q, planes_forward)) return rc;
  if (q.c[0].cd == CD_BF16) return forward<CD_BF16>(q, (char*)ws, need);
  if (q.c[0].cd == CD_F16) return forward<CD_F16>(q, (char*)ws, need);
  return forward<CD_F32>(q, (char*)ws, need);
}
int planes_backward(const PlanesBwd& q, void* ws, int64_t* need) {
  if (!need)
    if (const int rc = check_size(q, planes_backward)) return rc;
  if (q.c[0].cd == CD_BF16) return backward<CD_BF16>(q, (char*)ws, need);
  if (q.c[0].cd == CD_F16) return backward<CD_F16>(q, (char*)ws, need);
  return backward<CD_F32>(q, (char*)ws, need);
}

// A backward that wants dX and forms T itself takes every buffer that another does.
int64_t planes_workspace(int op, const LayerCall* c, int g, bool seeded) {
  static const Seeded some = {};
  static char out;
  int64_t need = 0;
  if (op == QLORA_OP_FWD) {
    const PlanesFwd q = {c, g, seeded ? &some : nullptr, 0, nullptr, nullptr, nullptr, nullptr};
    return planes_forward(q, nullptr, &need) ? 0 : need;
  }
  const PlanesBwd q = {c, g, seeded ? &some : nullptr, 0, nullptr, nullptr, nullptr, &out, nullptr, nullptr, CD_F32};
  return planes_backward(q, nullptr, &need) ? 0 : need;
}

}  // namespace qnf4
