// gated.hip -- the gated feed-forward block over two frozen NF4 projections of the same input:
//
//   forward   g = x Wg~^T + s (x Ag^T) Bg^T (+ bias),  u likewise,  h = act(g) u
//   backward  dg = dh u act'(g),  du = dh act(g), then the backward of the two projections as one
//             group: dX, dA, dB
//
// ("LoRA and QLoRA, mathematically", "Rank, alpha, and target modules": the adapted gate and up
// projections of a block's MLP.)  pre [m, 2 rows] = [g | u] in the compute type is what the forward
// saves for the backward.
#include <algorithm>

#include "act.h"
#include "mlp.h"
#include "tile.h"

namespace qnf4 {
namespace {

constexpr int kThreads = 256;

// E consecutive elements of a row (16 bytes where E = 8: rows of whole chunks), as fp32.
template <int CD, int E>
__device__ __forceinline__ void load_n(const void* p, int64_t at, float (&v)[E]) {
  if constexpr (E == 8) {
    const u32x4_t w = *(const u32x4_t*)((const uint16_t*)p + at);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = from_cd16<CD>((uint16_t)(w[e >> 1] >> (16 * (e & 1))));
  } else {
    v[0] = load_cd<CD>(p, at);
  }
}
template <int CD, int E>
__device__ __forceinline__ void store_n(void* p, int64_t at, const float (&v)[E]) {
  if constexpr (E == 8) {
    const u32x4_t w = {pack2<CD>(v[0], v[1]), pack2<CD>(v[2], v[3]), pack2<CD>(v[4], v[5]), pack2<CD>(v[6], v[7])};
    *(u32x4_t*)((uint16_t*)p + at) = w;
  } else {
    store_cd<CD>(p, at, v[0]);
  }
}

// h [m][n] = act(pre[:, :n]) pre[:, n:], E elements of a row to a thread.
template <int CD, int ACT, int E>
__global__ __launch_bounds__(kThreads) void k_gate(const void* __restrict__ pre, int64_t n, int64_t total,
                                                   void* __restrict__ h) {
  const int64_t per = n / E;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
    const int64_t row = i / per, at = 2 * n * row + E * (i - row * per);
    float g[E], u[E];
    load_n<CD, E>(pre, at, g);
    load_n<CD, E>(pre, at + n, u);
#pragma unroll
    for (int e = 0; e < E; ++e) g[e] = act_of<ACT>(g[e]) * u[e];
    store_n<CD, E>(h, E * i, g);
  }
}

// lora_b [n][r] as the operands of 32 x 32 x 16 matrix instructions whose contraction runs over n: operand (q, j) of
// rows 16 q .. and ranks 32 j .., 16 bytes of each lane behind each other (ranks from r on: zeros).
struct RankFrags {
  const uint16_t* b[2];
  u32x4_t* out[2];
  int r[2];
  int64_t n;
};
__global__ __launch_bounds__(kThreads) void k_rank_frags(RankFrags p) {
  const uint16_t* b = blockIdx.y ? p.b[1] : p.b[0];
  u32x4_t* out = blockIdx.y ? p.out[1] : p.out[0];
  const int r = blockIdx.y ? p.r[1] : p.r[0];
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= p.n * 8) return;
  const int lane = (int)(i & 63), rank = 32 * (int)(i >> 6 & 1) + (lane & 31);
  const int64_t row = 16 * (i >> 7) + 8 * (lane >> 5);
  u32x4_t v = {0u, 0u, 0u, 0u};
  if (rank < r) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e >> 1] |= (uint32_t)b[(row + e) * r + rank] << (16 * (e & 1));
  }
  out[i] = v;
}

// [dg | du] (dpre [m][2 n], rounded to the call's type) from dh [m][n] and pre, and slices of the sums dg B_g and
// du B_u over the columns, from the values as they are stored: part[i] [slices][m][64] fp32, b[i] as k_rank_frags
// leaves it.  A wave takes 32 rows of a slice's columns, 64 columns at a time: whole lines in and out, the
// values once through LDS of the wave's own to become operands.  Memory bounds it (4096 tokens, n = 14336:
// 587 MB and 34 MB of sums, 119 us, the rate of a large copy; dpre written first and read back for the sums took 91 and 60).
struct GateRank {
  const void *pre, *dh;
  const u32x4_t* b[2];
  void* dpre;
  float* part[2];
  int64_t m, n, per;  // columns of a slice
};
template <int CD, int ACT>
__global__ __launch_bounds__(kThreads, 2) void k_gate_rank(GateRank p) {
  using namespace tile;
  __shared__ __attribute__((aligned(1024))) char lds[4][2][32 * 128];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r32 = lane & 31, h = lane >> 5;
  const int64_t row0 = 128 * (int64_t)blockIdx.x + 32 * wave, c0 = p.per * blockIdx.y, c1 = min(c0 + p.per, p.n);
  if (row0 >= p.m) return;
  const int chunk = lane & 7, xr = swz(r32);
  const uint16_t* dh = (const uint16_t*)p.dh;
  const uint16_t* pre = (const uint16_t*)p.pre;
  uint16_t* dpre = (uint16_t*)p.dpre;
  char(*mine)[32 * 128] = lds[wave];
  f32x16_t acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  u32x4_t vg[4], vu[4], vd[4];
  auto load = [&](int64_t c) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int64_t row = min(row0 + 8 * t + (lane >> 3), p.m - 1);
      vg[t] = *(const u32x4_t*)(pre + 2 * row * p.n + c + 8 * chunk);
      vu[t] = *(const u32x4_t*)(pre + (2 * row + 1) * p.n + c + 8 * chunk);
      vd[t] = *(const u32x4_t*)(dh + row * p.n + c + 8 * chunk);
    }
  };
  load(c0);
  for (int64_t c = c0; c < c1; c += 64) {
    u32x4_t o[4][2];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        float dg[2], du[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float gv = from_cd16<CD>((uint16_t)(vg[t][e >> 1] >> (16 * x))), uv = from_cd16<CD>((uint16_t)(vu[t][e >> 1] >> (16 * x)));
          const float dv = from_cd16<CD>((uint16_t)(vd[t][e >> 1] >> (16 * x)));
          float value, slope;
          act_grad<ACT>(gv, value, slope);
          dg[x] = dv * uv * slope;
          du[x] = dv * value;
        }
        o[t][0][e >> 1] = pack2<CD>(dg[0], dg[1]);
        o[t][1][e >> 1] = pack2<CD>(du[0], du[1]);
      }
    }
    if (c + 64 < c1) load(c + 64);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int r = 8 * t + (lane >> 3);
      const int64_t row = row0 + r;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (row < p.m) *(u32x4_t*)(dpre + (2 * row + i) * p.n + c + 8 * chunk) = o[t][i];
        *(u32x4_t*)(mine[i] + r * 128 + ((chunk ^ swz(r)) << 4)) = o[t][i];
      }
    }
    wait_lgkm0();  // the wave reads back only what it wrote
    asm volatile("" ::: "memory");
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const i32x4_t a = Half16<CD>::read(mine[i] + r32 * 128, ks, h, xr);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          Half16<CD>::mma(acc[i][j], a, __builtin_bit_cast(i32x4_t, p.b[i][(((c >> 4) + ks) * 2 + j) * 64 + lane]), 0, 0);
      }
    wait_lgkm0();
    asm volatile("" ::: "memory");
  }
  // lane (r32, h) holds rank 32 j + r32 of rows 8 (v / 4) + 4 h + v % 4
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float* part = p.part[i] + (int64_t)blockIdx.y * p.m * 64;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int64_t at = row0 + 8 * (v >> 2) + 4 * h + (v & 3);
        if (at < p.m) part[at * 64 + 32 * j + r32] = acc[i][j][v];
      }
  }
}

int64_t al(int64_t b) { return round_up(b, 256); }
unsigned grid_for(int64_t n) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>(1 << 16, ceil_div(n, kThreads))); }

template <int CD, int ACT>
int gate_t(const void* pre, int64_t n, int64_t total, void* out, hipStream_t s) {
  ProfScope prof(QLORA_K_GATE, s);
  const dim3 b(kThreads);
  if (CD != CD_F32 && n % 8 == 0) k_gate<CD == CD_F32 ? CD_BF16 : CD, ACT, 8><<<dim3(grid_for(total / 8)), b, 0, s>>>(pre, n, total / 8, out);
  else k_gate<CD, ACT, 1><<<dim3(grid_for(total)), b, 0, s>>>(pre, n, total, out);
  return check_launch("k_gate");
}
template <int CD>
int gate_cd(int act, const void* pre, int64_t n, int64_t total, void* out, hipStream_t s) {
  if (act == QLORA_ACT_SILU) return gate_t<CD, QLORA_ACT_SILU>(pre, n, total, out, s);
  if (act == QLORA_ACT_GELU) return gate_t<CD, QLORA_ACT_GELU>(pre, n, total, out, s);
  return gate_t<CD, QLORA_ACT_GELU_TANH>(pre, n, total, out, s);
}

// How a forward runs, and its workspace.
//   DECODE   up to 64 tokens on the split-K GEMV: both projections' partial sums, one epilogue
//   TILED    W~ of both in the workspace, T = s x A^T by the rank-product kernels, then the gated GEMM
//   PLANES   every other layout, fp32, and up to 128 tokens of large weights, which that way decodes in the
//            product (128 tokens, bf16: 89 us against 122 at 14336 x 4096, 103 against 186 at
//            4096 x 14336, but 51 against 48 at 4096 x 4096 and 26 against 17 at 512 x 512)
enum Way { DECODE, TILED, PLANES };
struct FwdPlan {
  Way way;
  int64_t wd, t, bpad[2], part[2], total;
};
FwdPlan plan_fwd(const GroupCall& gc) {
  FwdPlan P = {};
  const LayerCall &c0 = gc.c[0], &c1 = gc.c[1];
  const int64_t m = c0.m, n = c0.w.rows, K = c0.w.cols, es = cd_bytes(c0.cd);
  if (m > 0 && gemv_gated_ok(gc.c)) {
    P.way = DECODE;
    P.total = (int64_t)gemv_gated_workspace_bytes(gc.c);
  } else if (m > 16 && !(m <= 128 && n * K >= 1 << 25) && gemm16_ok(c0.cd, m, n, K) && fast_layout(c0.w) && fast_layout(c1.w) && skinny_ok(c0.cd, c0.r) &&
             skinny_ok(c1.cd, c1.r) && dense256_ok(c0, false) && dense256_ok(c1, false)) {
    P.way = TILED;
    int64_t o = 0;
    P.wd = o; o += al(2 * n * K * es);
    P.t = o; o += al(m * 128 * es);
    for (int i = 0; i < 2; ++i) {
      const int32_t r = gc.c[i].r;
      P.bpad[i] = o; o += r % 8 ? al(n * round_up(r, 8) * es) : 0;
      P.part[i] = o; o += al((int64_t)skinny_part_bytes(m, K));
    }
    P.total = o;
  } else {
    P.way = PLANES;
    P.total = planes_workspace(QLORA_OP_FWD, gc.c, 2, false);
  }
  return P;
}

// dst [n][ld] = src [n][r] with zeros from column r on: rows of lora_b as whole 16-byte chunks.
struct PadRows {
  const uint16_t* src;
  uint16_t* dst;
  int r, ld;
};
__global__ __launch_bounds__(kThreads) void k_pad_rows(PadRows a, PadRows b, int64_t n) {
  const uint16_t* src = blockIdx.y ? b.src : a.src;
  uint16_t* dst = blockIdx.y ? b.dst : a.dst;
  const int r = blockIdx.y ? b.r : a.r, ld = blockIdx.y ? b.ld : a.ld;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n * ld; i += (int64_t)gridDim.x * kThreads) {
    const int64_t row = i / ld;
    const int c = (int)(i - row * ld);
    dst[i] = c < r ? src[row * r + c] : (uint16_t)0;
  }
}

// Whether the group call's tuned kernels take a backward: with few tokens or small weights the other way
// has fewer launches and, up to 256 tokens, no copy of W~ (bf16: 1 token of 14336 x 4096 88 us against 169,
// 128 tokens 138 against 210; 1024 x 512 x 512 37 against 54, 1024 x 2048 x 2048 82 against 90, but
// 2048 x 2048 x 2048 109 against 106, 512 x 4096 x 4096 136 against 113).
bool tuned_bwd(const GroupCall& gc) {
  const LayerCall &c0 = gc.c[0], &c1 = gc.c[1];
  if (c0.m <= 128 || c0.m * c0.w.rows * c0.w.cols <= 1LL << 32) return false;
  if (!skinny_reaches(c0.m, 2 * c0.w.rows) || !skinny_reaches(c0.m, c0.w.cols)) return false;
  return c0.cd != CD_F32 && c0.w.rows % 64 == 0 && fast_layout(c0.w) && fast_layout(c1.w) && skinny_ok(c0.cd, c0.r) &&
         skinny_ok(c1.cd, c1.r) && gemm16_ok(c0.cd, c0.m, c0.w.cols, 2 * c0.w.rows) && dense256_ok(c0, true) &&
         dense256_ok(c1, true);
}

int forward_tiled(const GroupCall& gc, const FwdPlan& P, int act, const void* bias, void* h, void* pre,
                  float* const* t_save, char* ws, hipStream_t s) {
  const LayerCall& c0 = gc.c[0];
  const int64_t m = c0.m, n = c0.w.rows, K = c0.w.cols, es = cd_bytes(c0.cd);
  SkSpec specs[2];
  float* parts[2];
  int S[2], rc;
  for (int i = 0; i < 2; ++i) {
    specs[i].a = c0.x;
    specs[i].lda = K;
    specs[i].arows = m;
    specs[i].b = gc.c[i].lora_a;
    specs[i].ldb = K;
    specs[i].P = m;
    specs[i].R = gc.c[i].r;
    specs[i].Kc = K;
    parts[i] = (float*)(ws + P.part[i]);
  }
  if ((rc = skinny_many(c0.cd, specs, parts, S, 2, s, QLORA_K_LORA_DOWN))) return rc;
  Nf4W w[2];
  void* out[2];
  SkRed red[2];
  const void* b[2];
  int64_t ldb[2];
  PadRows pads[2];
  int np = 0;
  for (int i = 0; i < 2; ++i) {
    const LayerCall& c = gc.c[i];
    w[i] = c.w;
    out[i] = ws + P.wd + i * n * K * es;
    red[i].part = parts[i];
    red[i].S = S[i];
    red[i].P = m;
    red[i].R = c.r;
    red[i].out32 = t_save ? t_save[i] : nullptr;
    red[i].sccd = c.scale;
    red[i].outcd = ws + P.t + i * 64 * es;
    red[i].ldcd = 128;
    red[i].wcd = 64;
    b[i] = c.lora_b;
    ldb[i] = round_up(c.r, 8);
    if (c.r % 8) {
      b[i] = ws + P.bpad[i];
      pads[np++] = PadRows{(const uint16_t*)c.lora_b, (uint16_t*)(ws + P.bpad[i]), c.r, (int)ldb[i]};
    }
  }
  if (np) {
    ProfScope prof(QLORA_K_REDUCE, s);
    const dim3 grid(grid_for(n * std::max(pads[0].ld, pads[np - 1].ld)), np);
    k_pad_rows<<<grid, dim3(kThreads), 0, s>>>(pads[0], pads[np - 1], n);
    if ((rc = check_launch("k_pad_rows"))) return rc;
  }
  // W~ of both, the reductions of T riding on the launch
  if ((rc = dequant_group_into(w, 2, c0.cd, out, red, s))) return rc;
  return gemm16_gated(c0.cd, c0.x, m, n, K, out, ws + P.t, b, ldb, bias, act, h, pre, s);
}

// The tiled backward's workspace.
struct BwdPlan {
  int S;        // slices of dg B and du B
  int64_t per;  // columns of a slice
  int64_t dpre, wdt, dt, at, t0, b[2], dtt[2], t0t[2], rank[2], pa, pb, total;
};
BwdPlan plan_bwd(const GroupCall& gc) {
  BwdPlan P = {};
  const LayerCall& c0 = gc.c[0];
  const int64_t m = c0.m, n = c0.w.rows, K = c0.w.cols, es = cd_bytes(c0.cd), m64 = round_up(m, 64);
  // slices of whole 64 columns, two workgroups to a compute unit
  P.per = 64 * std::max<int64_t>(1, ceil_div(n / 64, std::min<int64_t>(kRedMaxS, std::max<int64_t>(1, ceil_div(512, ceil_div(m, 128))))));
  P.S = (int)ceil_div(n, P.per);
  int64_t o = 0;
  P.dpre = o; o += al(2 * m * n * es);
  P.wdt = o; o += al(2 * K * n * es);
  P.dt = o; o += al(m * 128 * es);
  P.at = o; o += al(K * 128 * es);
  P.t0 = o; o += al(2 * m * 64 * 4);
  int64_t down = 0;
  for (int i = 0; i < 2; ++i) {
    const int32_t r = gc.c[i].r;
    P.b[i] = o; o += al(n * 64 * es);
    P.dtt[i] = o; o += al(r * m64 * es);
    P.t0t[i] = o; o += al(r * m64 * es);
    down = std::max<int64_t>((int64_t)skinny_part_bytes(m, K), P.S * m * 64 * 4);
    P.rank[i] = o; o += al(down);
  }
  P.pa = o; o += al((int64_t)skinny_part_bytes(K, m64));
  P.pb = o; o += al((int64_t)skinny_part_bytes(n, m64));
  P.total = o;
  return P;
}

template <int CD>
int gate_rank(int act, const GateRank& p, int S, hipStream_t s) {
  ProfScope prof(QLORA_K_GATE, s);
  const dim3 grid((unsigned)ceil_div(p.m, 128), (unsigned)S), b(kThreads);
  if (act == QLORA_ACT_SILU) k_gate_rank<CD, QLORA_ACT_SILU><<<grid, b, 0, s>>>(p);
  else if (act == QLORA_ACT_GELU) k_gate_rank<CD, QLORA_ACT_GELU><<<grid, b, 0, s>>>(p);
  else k_gate_rank<CD, QLORA_ACT_GELU_TANH><<<grid, b, 0, s>>>(p);
  return check_launch("k_gate_rank");
}

// dg, du and dT of both; W~^T of both beside each other, the reductions of dT riding on them; dX by one GEMM over
// both projections' rows; the products of dA and dB.
int backward_tiled(const GroupCall& gc, int act, const void* dh, const void* pre, const float* const* t_saved, void* dx,
                   void* const* d_a, void* const* d_b, int gd, char* ws, hipStream_t s) {
  const BwdPlan P = plan_bwd(gc);
  const LayerCall& c0 = gc.c[0];
  const int64_t m = c0.m, n = c0.w.rows, K = c0.w.cols, es = cd_bytes(c0.cd), m64 = round_up(m, 64);
  int rc;
  const float* t0[2];
  if (t_saved) {
    t0[0] = t_saved[0];
    t0[1] = t_saved[1];
  } else {
    SkSpec specs[2];
    float* parts[2];
    int S[2];
    for (int i = 0; i < 2; ++i) {
      specs[i].a = c0.x;
      specs[i].lda = specs[i].ldb = specs[i].Kc = K;
      specs[i].arows = specs[i].P = m;
      specs[i].b = gc.c[i].lora_a;
      specs[i].R = gc.c[i].r;
      parts[i] = (float*)(ws + P.rank[i]);
    }
    if ((rc = skinny_many(c0.cd, specs, parts, S, 2, s, QLORA_K_LORA_DOWN))) return rc;
    SkRed red[2];
    for (int i = 0; i < 2; ++i) {
      red[i].part = parts[i];
      red[i].S = S[i];
      red[i].P = m;
      red[i].R = gc.c[i].r;
      red[i].out32 = (float*)(ws + P.t0) + i * m * 64;
      t0[i] = red[i].out32;
    }
    if ((rc = skinny_reduce_jobs(c0.cd, red[0], &red[1], s))) return rc;
  }
  TransposeSpec ta[2];
  RankFrags rf = {};
  rf.n = n;
  SkRed red[2];
  GateRank gr = {};
  gr.pre = pre;
  gr.dh = dh;
  gr.dpre = ws + P.dpre;
  gr.m = m;
  gr.n = n;
  gr.per = P.per;
  for (int i = 0; i < 2; ++i) {
    const LayerCall& c = gc.c[i];
    rf.b[i] = (const uint16_t*)c.lora_b;
    rf.out[i] = (u32x4_t*)(ws + P.b[i]);
    rf.r[i] = c.r;
    ta[i].src = c.lora_a;
    ta[i].ld_src = K;
    ta[i].rows = c.r;
    ta[i].cols = K;
    ta[i].dst = ws + P.at + i * 64 * es;
    ta[i].ld_dst = 128;
    ta[i].w_dst = 64;
    gr.b[i] = rf.out[i];
    gr.part[i] = (float*)(ws + P.rank[i]);
    red[i].part = gr.part[i];
    red[i].S = P.S;
    red[i].P = m;
    red[i].R = c.r;
    red[i].sccd = c.scale;
    red[i].outcd = ws + P.dt + i * 64 * es;
    red[i].ldcd = 128;
    red[i].wcd = 64;
    red[i].outt = ws + P.dtt[i];
    red[i].ldt = m64;
    red[i].side = t0[i];
    red[i].side_t = ws + P.t0t[i];
  }
  if (dx && (rc = transpose_jobs(c0.cd, ta[0], &ta[1], s))) return rc;
  {
    ProfScope prof(QLORA_K_REDUCE, s);
    k_rank_frags<<<dim3((unsigned)ceil_div(n * 8, kThreads), 2), dim3(kThreads), 0, s>>>(rf);
    if ((rc = check_launch("k_rank_frags"))) return rc;
  }
  if ((rc = c0.cd == CD_BF16 ? gate_rank<CD_BF16>(act, gr, P.S, s) : gate_rank<CD_F16>(act, gr, P.S, s))) return rc;
  if (dx) {
    for (int i = 0; i < 2; ++i)
      if ((rc = dequant_into(gc.c[i].w, c0.cd, ws + P.wdt + i * n * es, true, s, &red[i], 2 * n))) return rc;
    if ((rc = gemm16_plain(c0.cd, gr.dpre, m, K, 2 * n, ws + P.wdt, ws + P.dt, 128, ws + P.at, 128, nullptr, dx,
                           QLORA_K_BWD_DX, s)))
      return rc;
  } else if ((rc = skinny_reduce_jobs(c0.cd, red[0], &red[1], s))) {
    return rc;
  }
  for (int i = 0; i < 2; ++i) {
    const LayerCall& c = gc.c[i];
    SkSpec pa, pb;  // dA: x^T against dT^T;  dB: dpre^T against T0^T
    pa.a = c.x;
    pa.lda = K;
    pa.arows = m;
    pa.b = ws + P.dtt[i];
    pa.ldb = m64;
    pa.P = K;
    pa.R = c.r;
    pa.Kc = m64;
    pb.a = ws + P.dpre + i * n * es;
    pb.lda = 2 * n;
    pb.arows = m;
    pb.b = ws + P.t0t[i];
    pb.ldb = m64;
    pb.P = n;
    pb.R = c.r;
    pb.Kc = m64;
    SkRed ra, rb;
    ra.part = (float*)(ws + P.pa);
    ra.P = K;
    ra.R = c.r;
    rb.part = (float*)(ws + P.pb);
    rb.P = n;
    rb.R = c.r;
    if ((rc = skinny_jobs(c.cd, true, pa, (float*)(ws + P.pa), &ra.S, &pb, (float*)(ws + P.pb), &rb.S, s, QLORA_K_BWD_DA)))
      return rc;
    gradient_jobs(ra, rb, c.scale, d_a[i], d_b[i], gd == CD_F32);
    if ((rc = skinny_reduce_jobs(c.cd, ra, &rb, s))) return rc;
  }
  return QLORA_OK;
}

}  // namespace

// h [m][n] from pre.
int gate(int cd, int act, const void* pre, int64_t m, int64_t n, void* h, hipStream_t s) {
  if (cd == CD_BF16) return gate_cd<CD_BF16>(act, pre, n, m * n, h, s);
  if (cd == CD_F16) return gate_cd<CD_F16>(act, pre, n, m * n, h, s);
  return gate_cd<CD_F32>(act, pre, n, m * n, h, s);
}

size_t gated_workspace_bytes(int op, const GroupCall& gc) {
  if (op == QLORA_OP_FWD) return (size_t)plan_fwd(gc).total;
  if (!tuned_bwd(gc)) return (size_t)planes_workspace(op, gc.c, 2, false);
  return (size_t)plan_bwd(gc).total;
}

int launch_gated_fwd(const GroupCall& gc, int act, const void* bias, void* h, void* pre, float* const* t_save, void* ws,
                     hipStream_t s) {
  const FwdPlan P = plan_fwd(gc);
  const LayerCall& c = gc.c[0];
  if (P.way == DECODE) {
    LayerCall pair[2] = {gc.c[0], gc.c[1]};
    for (int i = 0; i < 2; ++i) {
      pair[i].bias = bias ? (const char*)bias + i * c.w.rows * cd_bytes(c.cd) : nullptr;
      pair[i].ws = ws;
    }
    return gemv_gated(pair, act, h, pre, t_save);
  }
  if (P.way == TILED) return forward_tiled(gc, P, act, bias, h, pre, t_save, (char*)ws, s);
  const PlanesFwd q = {gc.c, 2, nullptr, act, bias, h, pre, t_save};
  return planes_forward(q, ws, nullptr);
}

int launch_gated_bwd(const GroupCall& gc, int act, const void* dh, const void* pre, const float* const* t_saved, void* dx,
                     void* const* d_a, void* const* d_b, int gd, void* ws, hipStream_t s) {
  if (t_saved && !(t_saved[0] && t_saved[1])) t_saved = nullptr;  // both are formed where one is missing
  if (tuned_bwd(gc)) return backward_tiled(gc, act, dh, pre, t_saved, dx, d_a, d_b, gd, (char*)ws, s);
  const PlanesBwd q = {gc.c, 2, nullptr, act, dh, pre, t_saved, dx, d_a, d_b, gd};
  return planes_backward(q, ws, nullptr);
}

}  // namespace qnf4
