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

// dpre [m][2 n] from dh [m][n] and pre.
template <int CD, int ACT, int E>
__global__ __launch_bounds__(kThreads) void k_gate_bwd(const void* __restrict__ pre, const void* __restrict__ dh,
                                                       int64_t n, int64_t total, void* __restrict__ dpre) {
  const int64_t per = n / E;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
    const int64_t row = i / per, at = 2 * n * row + E * (i - row * per);
    float d[E], g[E], u[E];
    load_n<CD, E>(dh, E * i, d);
    load_n<CD, E>(pre, at, g);
    load_n<CD, E>(pre, at + n, u);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float value, slope;
      act_grad<ACT>(g[e], value, slope);
      g[e] = d[e] * u[e] * slope;
      u[e] = d[e] * value;
    }
    store_n<CD, E>(dpre, at, g);
    store_n<CD, E>(dpre, at + n, u);
  }
}

int64_t al(int64_t b) { return round_up(b, 256); }
unsigned grid_for(int64_t n) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>(1 << 16, ceil_div(n, kThreads))); }

template <int CD, int ACT, int E>
int gate_n(const void* pre, const void* dh, int64_t n, int64_t total, void* out, hipStream_t s) {
  ProfScope prof(QLORA_K_GATE, s);
  const dim3 g(grid_for(total / E)), b(kThreads);
  if (dh) k_gate_bwd<CD, ACT, E><<<g, b, 0, s>>>(pre, dh, n, total / E, out);
  else k_gate<CD, ACT, E><<<g, b, 0, s>>>(pre, n, total / E, out);
  return check_launch(dh ? "k_gate_bwd" : "k_gate");
}
template <int CD, int ACT>
int gate_t(const void* pre, const void* dh, int64_t n, int64_t total, void* out, hipStream_t s) {
  if constexpr (CD != CD_F32)
    if (n % 8 == 0) return gate_n<CD, ACT, 8>(pre, dh, n, total, out, s);
  return gate_n<CD, ACT, 1>(pre, dh, n, total, out, s);
}
template <int CD>
int gate_cd(int act, const void* pre, const void* dh, int64_t n, int64_t total, void* out, hipStream_t s) {
  if (act == QLORA_ACT_SILU) return gate_t<CD, QLORA_ACT_SILU>(pre, dh, n, total, out, s);
  if (act == QLORA_ACT_GELU) return gate_t<CD, QLORA_ACT_GELU>(pre, dh, n, total, out, s);
  return gate_t<CD, QLORA_ACT_GELU_TANH>(pre, dh, n, total, out, s);
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
  return c0.cd != CD_F32 && c0.w.rows % 64 == 0 && fast_layout(c0.w) && fast_layout(c1.w) && skinny_ok(c0.cd, c0.r) &&
         skinny_ok(c1.cd, c1.r);
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

}  // namespace

// dh null: out = h [m][n]; else out = dpre [m][2 n].
int gate(int cd, int act, const void* pre, const void* dh, int64_t m, int64_t n, void* out, hipStream_t s) {
  if (cd == CD_BF16) return gate_cd<CD_BF16>(act, pre, dh, n, m * n, out, s);
  if (cd == CD_F16) return gate_cd<CD_F16>(act, pre, dh, n, m * n, out, s);
  return gate_cd<CD_F32>(act, pre, dh, n, m * n, out, s);
}

size_t gated_workspace_bytes(int op, const GroupCall& gc) {
  if (op == QLORA_OP_FWD) return (size_t)plan_fwd(gc).total;
  if (!tuned_bwd(gc)) return (size_t)planes_workspace(op, gc.c, 2, false);
  return (size_t)al(gc.c[0].m * gc.N * cd_bytes(gc.c[0].cd)) + group_workspace_bytes(op, gc);  // [dg | du] first
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
  const LayerCall& c = gc.c[0];
  if (!tuned_bwd(gc)) {
    const PlanesBwd q = {gc.c, 2, nullptr, act, dh, pre, t_saved, dx, d_a, d_b, gd};
    return planes_backward(q, ws, nullptr);
  }
  const int rc = gate(c.cd, act, pre, dh, c.m, c.w.rows, ws, s);
  return rc ? rc : launch_backward_group_as(gc, ws, t_saved, dx, d_a, d_b, gd, true,
                                            (char*)ws + al(c.m * gc.N * cd_bytes(c.cd)), s);
}

}  // namespace qnf4
