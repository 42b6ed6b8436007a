// mlp.h -- host entry points of the 8-bit floating-point product (fp8.hip), of the gated block
// (gated.hip) and of the layer with seeded dropout (gemm.hip, dropout.hip).
#pragma once
#include "common.h"
#include "philox.h"

namespace qnf4 {
int launch_fp8_quantize(const void* w, int64_t ldw, int dtype, const qlora_fp8_t* q, hipStream_t s);
size_t fp8_workspace_bytes(const qlora_fp8_t* w, int64_t m, int cd);
int launch_fp8_linear(const qlora_fp8_t* w, const void* x, int64_t m, int64_t ldx, const void* bias, int cd, void* y,
                      void* ws, hipStream_t s);

// The layer with an optional seeded dropout (null: none) and the adapters' gradients in gd (fp32 or
// the call's own type).
int launch_forward_seeded(const LayerCall& c, const Seeded& sd, void* y, float* t_save);
int launch_backward_as(const LayerCall& c, const Seeded* sd, const void* dy, const float* t_saved, void* dx, void* d_a,
                       void* d_b, int gd);
// Where the reductions of dA (ra, its sums [cols][r]) and dB (rb, [rows][r], times scale) write:
// fp32, or rounded into the call's type.
inline void gradient_jobs(SkRed& ra, SkRed& rb, float scale, void* d_a, void* d_b, bool g32) {
  rb.sc32 = rb.sccd = scale;
  if (g32) {
    ra.out32 = (float*)d_a;
    ra.trans = true;
    rb.out32 = (float*)d_b;
  } else {
    ra.outt = d_a;  // the transposed copy: [r][cols]
    ra.ldt = ra.P;
    rb.outcd = d_b;
    rb.ldcd = rb.R;
  }
}
// What such a call needs in its weight's layout (c.flags holds QLORA_FLAG_DROPOUT).
size_t seeded_workspace_bytes(int op, const LayerCall& c);
// out = x M
int apply_seeded(int cd, const void* x, const Seeded& sd, int64_t rows, int64_t cols, void* out, hipStream_t s);
// Whether the offsets of the rank-product kernels, 32 bits, hold all of a 16-bit matrix (past 2^31 bytes a row that is not there
// still lies behind the buffer's end).
inline bool skinny_addresses(int64_t rows, int64_t ld) { return round_up(rows, 128) * ld * 2 < (1LL << 32); }
// Whether they lie below 2^31 bytes, where the masked forms are used.
inline bool skinny_reaches(int64_t rows, int64_t ld) { return round_up(rows, 64) * ld * 2 < (1LL << 31); }
// lora.hip: one rank product (and, TN, a second without a mask) whose Aop, x [rows][cols], counts under the
// drawn mask.  NT: x A^T; TN: bits not null: the mask's bits are left there, rows of ldbits words.
int skinny_drawn(int cd, bool tn, const SkSpec& a, float* part, int* S_out, const SkSpec* b2, float* part2, int* S2,
                 const Seeded& sd, void* bits, int64_t ldbits, hipStream_t s, int kind);
int rank_add_seeded(int cd, void* dx, const Seeded& sd, const void* dt, int64_t ld_dt, const void* a, int32_t r, int64_t M,
                    int64_t K, hipStream_t s);

// gemv.hip: the gated block's forward of up to 64 tokens (c: gate and up).
size_t gemv_workspace_bytes(int64_t m, int64_t rows, int64_t cols, int32_t r, int cd);
bool gemv_gated_ok(const LayerCall* c);
size_t gemv_gated_workspace_bytes(const LayerCall* c);
int gemv_gated(const LayerCall* c, int act, void* h, void* pre, float* const* t_save);
// gemm16.hip
bool gemm16_ok(int cd, int64_t m, int64_t n, int64_t K);
int gemm16_gated(int cd, const void* x, int64_t m, int64_t n, int64_t K, const void* const* w, const void* t,
                 const void* const* b, const int64_t* ldb, const void* bias, int act, void* h, void* pre, hipStream_t s);
int gemm16_plain(int cd, const void* x, int64_t m, int64_t n, int64_t K, const void* w, const void* t, int64_t ldt,
                 const void* l, int64_t ldl, const void* bias, void* y, int kind, hipStream_t s);
int gemm16_masked_dx(int cd, const void* dy, int64_t m, int64_t n, int64_t K, const void* wt, const void* dt, int64_t ldt,
                     const void* at, int64_t lda, const void* bits, int64_t ldbits, void* dx, hipStream_t s);

// planes.hip: the seeded layer (g = 1) and the gated block (g = 2) in every layout and type.
struct PlanesFwd {
  const LayerCall* c;
  int g;
  const Seeded* sd;  // g = 1
  int act;           // g = 2
  const void* bias;  // [g rows] or null
  void* out;         // y, or h
  void* pre;
  float* const* t_save;
};
struct PlanesBwd {
  const LayerCall* c;
  int g;
  const Seeded* sd;  // g = 1
  int act;           // g = 2
  const void* dy;    // dY, or dh
  const void* pre;
  const float* const* t_saved;
  void* dx;
  void* const* d_a;
  void* const* d_b;
  int gd;
};
// need not null: only the workspace's size is wanted (pointers are not read).
int planes_forward(const PlanesFwd& q, void* ws, int64_t* need);
int planes_backward(const PlanesBwd& q, void* ws, int64_t* need);
// The most that such a call needs in its weights' layout, whichever of its outputs are wanted (0: none that fits).
int64_t planes_workspace(int op, const LayerCall* c, int g, bool seeded);
// gated.hip: h [m][n] from pre
int gate(int cd, int act, const void* pre, int64_t m, int64_t n, void* h, hipStream_t s);

size_t gated_workspace_bytes(int op, const GroupCall& gc);
int launch_gated_fwd(const GroupCall& gc, int act, const void* bias, void* h, void* pre, float* const* t_save, void* ws,
                     hipStream_t s);
int launch_gated_bwd(const GroupCall& gc, int act, const void* dh, const void* pre, const float* const* t_saved, void* dx,
                     void* const* d_a, void* const* d_b, int gd, void* ws, hipStream_t s);
}  // namespace qnf4
