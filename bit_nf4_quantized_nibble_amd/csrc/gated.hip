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

#include "mlp.h"

namespace qnf4 {
namespace {

constexpr int kThreads = 256;

// act(z) and its derivative, in fp32.
//   silu       z q,  q = 1 / (1 + exp(-z));          derivative q + z q (1 - q)
//   gelu       z c,  c = erfc(-z / sqrt 2) / 2;      derivative c + z exp(-z^2 / 2) / sqrt(2 pi)
//   gelu_tanh  z q(2 t),  t = sqrt(2 / pi) (z + 0.044715 z^3)  (1/2 (1 + tanh t) = q(2 t))
// 1 - q is formed as q(-z): no cancellation where q is near 1.
__device__ __forceinline__ float sigmoid(float z) { return 1.f / (1.f + __expf(-z)); }
constexpr float kTanhA = 1.5957691216057308f;           // 2 sqrt(2 / pi)
constexpr float kTanhB = kTanhA * 0.044715f;
// The cubic's argument: beyond 30 q is 0 or 1, and z^3 must not leave fp32's range.
__device__ __forceinline__ float limited(float z) { return fminf(fmaxf(z, -30.f), 30.f); }
__device__ __forceinline__ float tanh_arg(float z) {
  const float l = limited(z);
  return l * fmaf(kTanhB * l, l, kTanhA);
}
template <int ACT>
__device__ __forceinline__ float act_of(float z) {
  if constexpr (ACT == QLORA_ACT_SILU) return z * sigmoid(z);
  else if constexpr (ACT == QLORA_ACT_GELU) return z * (0.5f * erfcf(-0.70710678118654752f * z));
  else return z * sigmoid(tanh_arg(z));
}
template <int ACT>
__device__ __forceinline__ void act_grad(float z, float& value, float& slope) {
  if constexpr (ACT == QLORA_ACT_GELU) {
    const float c = 0.5f * erfcf(-0.70710678118654752f * z);
    value = z * c;
    slope = fmaf(z * 0.39894228040143268f, __expf(-0.5f * z * z), c);
  } else if constexpr (ACT == QLORA_ACT_SILU) {
    const float q = sigmoid(z);
    value = z * q;
    slope = fmaf(value, sigmoid(-z), q);
  } else {
    const float t = tanh_arg(z), q = sigmoid(t), zl = limited(z);
    value = z * q;
    slope = fmaf(value * sigmoid(-t), fmaf(3.f * kTanhB * zl, zl, kTanhA), q);
  }
}

// h [m][n] = act(pre[:, :n]) pre[:, n:], one element to a thread.
template <int CD, int ACT>
__global__ __launch_bounds__(kThreads) void k_gate(const void* __restrict__ pre, int64_t n, int64_t total,
                                                   void* __restrict__ h) {
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
    const int64_t row = i / n, at = 2 * n * row + (i - row * n);
    store_cd<CD>(h, i, act_of<ACT>(load_cd<CD>(pre, at)) * load_cd<CD>(pre, at + n));
  }
}

// dpre [m][2 n] from dh [m][n] and pre.
template <int CD, int ACT>
__global__ __launch_bounds__(kThreads) void k_gate_bwd(const void* __restrict__ pre, const void* __restrict__ dh,
                                                       int64_t n, int64_t total, void* __restrict__ dpre) {
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
    const int64_t row = i / n, at = 2 * n * row + (i - row * n);
    const float d = load_cd<CD>(dh, i);
    float value, slope;
    act_grad<ACT>(load_cd<CD>(pre, at), value, slope);
    store_cd<CD>(dpre, at, d * load_cd<CD>(pre, at + n) * slope);
    store_cd<CD>(dpre, at + n, d * value);
  }
}

int64_t al(int64_t b) { return round_up(b, 256); }
unsigned grid_for(int64_t n) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>(1 << 16, ceil_div(n, kThreads))); }

template <int CD, int ACT>
int gate_t(const void* pre, const void* dh, int64_t n, int64_t total, void* out, hipStream_t s) {
  ProfScope prof(QLORA_K_GATE, s);
  if (dh) k_gate_bwd<CD, ACT><<<dim3(grid_for(total)), dim3(kThreads), 0, s>>>(pre, dh, n, total, out);
  else k_gate<CD, ACT><<<dim3(grid_for(total)), dim3(kThreads), 0, s>>>(pre, n, total, out);
  return check_launch(dh ? "k_gate_bwd" : "k_gate");
}
template <int CD>
int gate_cd(int act, const void* pre, const void* dh, int64_t n, int64_t total, void* out, hipStream_t s) {
  if (act == QLORA_ACT_SILU) return gate_t<CD, QLORA_ACT_SILU>(pre, dh, n, total, out, s);
  if (act == QLORA_ACT_GELU) return gate_t<CD, QLORA_ACT_GELU>(pre, dh, n, total, out, s);
  return gate_t<CD, QLORA_ACT_GELU_TANH>(pre, dh, n, total, out, s);
}
// dh null: out = h [m][n]; else out = dpre [m][2 n].
int gate(int cd, int act, const void* pre, const void* dh, int64_t m, int64_t n, void* out, hipStream_t s) {
  if (cd == CD_BF16) return gate_cd<CD_BF16>(act, pre, dh, n, m * n, out, s);
  if (cd == CD_F16) return gate_cd<CD_F16>(act, pre, dh, n, m * n, out, s);
  return gate_cd<CD_F32>(act, pre, dh, n, m * n, out, s);
}

}  // namespace

// [g | u] (or its gradient) and the group call's own workspace.
size_t gated_workspace_bytes(int op, const GroupCall& gc) {
  return (size_t)al(gc.c[0].m * gc.N * cd_bytes(gc.c[0].cd)) + group_workspace_bytes(op, gc);
}

int launch_gated_fwd(const GroupCall& gc, int act, const void* bias, void* h, void* pre, float* const* t_save, void* ws,
                     hipStream_t s) {
  const LayerCall& c = gc.c[0];
  void* z = pre ? pre : ws;
  const int rc = launch_forward_group(gc, bias, z, t_save, (char*)ws + al(c.m * gc.N * cd_bytes(c.cd)), s);
  return rc ? rc : gate(c.cd, act, z, nullptr, c.m, c.w.rows, h, s);
}

int launch_gated_bwd(const GroupCall& gc, int act, const void* dh, const void* pre, const float* const* t_saved, void* dx,
                     void* const* d_a, void* const* d_b, int gd, void* ws, hipStream_t s) {
  const LayerCall& c = gc.c[0];
  const int rc = gate(c.cd, act, pre, dh, c.m, c.w.rows, ws, s);
  return rc ? rc : launch_backward_group_as(gc, ws, t_saved, dx, d_a, d_b, gd,
                                            (char*)ws + al(c.m * gc.N * cd_bytes(c.cd)), s);
}

}  // namespace qnf4
