// gemm16.hip -- 16-bit GEMMs with a low-rank part (gfx950):
//
//   plain      y = [x | T] [W~ | B]^T (+ bias)
//   gated      h = act(g) u with [g | u] = [x | T] [W~ | B]^T (+ bias) of two projections
//   masked dX  dX = dY W~ + (dT A) M with M as bits
//
// All stand on the contraction of tile.h; the low-rank part is one or more stages behind the last.
//
// Gated: a tile's 2 C columns are C columns of the gate and the same C of the up projection, in runs
// of 32 that alternate, so that a wave's two blocks of columns are g and u of the same 32 columns and
// h is formed in registers.  The low-rank part is two more stages: T_g against B_g with zeros in the
// up rows, then T_u against B_u with zeros in the gate rows.
//
// Masked: the low-rank part is multiplied after the last stage into sums of its own, masked and added.
// The mask comes as bits, which the launch that draws it for dA leaves behind: drawn here, a counter beside
// the products of each stage, it cost 70 us of 500 (4096 tokens, 4096 x 14336) although the vector pipe stands
// idle there, as the products run at the card's power limit.
#include <algorithm>
#include <type_traits>

#include "act.h"
#include "mlp.h"
#include "tile.h"

namespace qnf4 {
namespace {

using namespace tile;

struct G16 {
  const void* x;       // [m][K] cd: x, or dY
  const void *w0, *w1; // [n][K] cd: W~ of the gate and of the up projection, or W~^T and null
  const void* t;       // [m][ldt] cd: T_g in columns 0 .., T_u in columns 64 .., or T or dT
  int64_t ldt;
  const void *l0, *l1; // [n][ld_l] cd: lora_b of the two, or lora_b or A^T and null
  int64_t ldl0, ldl1;  // multiples of 8; columns from there on count as zeros
  const void* bias;    // [2 n] (gated) or [n] (plain) cd or null
  void* out;           // [m][n] cd: h, y or dX
  void* pre;           // [m][2 n] cd or null
  int64_t m, n, K;
  const uint32_t* bits;  // [m][ldbits]: column k of the mask in bit k % 32 of word k / 32
  int64_t ldbits;
};

enum Mode { PLAIN, GATED, MASKED };

struct Place {
  int rows;
  int64_t m0, n0;
};

// Columns of the output that a tile forms.
template <class T, int MODE>
constexpr int cols_of() { return MODE == GATED ? T::TN / 2 : T::TN; }

// Waves that copy: four of the largest tile's eight, else all.
template <class T>
constexpr int copying() { return T::TM == 256 && T::NS == 2 ? 4 : T::NW; }

// The copies of a tile's stages by one wave: instruction i of copying wave w fills LDS rows
// 8 (w + NW i) .. + 7 of the stage; lane l lands in chunk l % 8 of row l / 8 and fetches the
// logical chunk that lies there.  begin() sets up what a stage's copies read.
template <class T, int MODE>
struct Copies16 {
  static constexpr int NW = copying<T>(), PER_A = T::TM / 8 / NW, PER = (T::TM + T::TN) / 8 / NW, WAVES = NW;
  const G16& p;
  Place pl;
  int KM, KT, wave, lane, chunk;
  int64_t ncols;
  rsrc_t ra, rb[2];
  uint32_t oa, ob, sa, sb, so;
  __device__ __forceinline__ Copies16(const G16& p_, const Place& t, int wave_, int lane_)
      : p(p_), pl(t), wave(wave_), lane(lane_) {
    KM = (int)(p.K >> 6);
    KT = KM + (MODE == GATED ? 2 : MODE == PLAIN ? (int)((p.ldt + 63) >> 6) : 0);
    chunk = (lane & 7) ^ swz(8 * wave + (lane >> 3));
    ncols = min((int64_t)cols_of<T, MODE>(), p.n - t.n0);
  }
  // row of the W-side operand (within its tile) of this lane in copy 0, and the operand of copy i
  __device__ __forceinline__ int brow() const { return (MODE == GATED ? 8 * (wave & 3) : 8 * wave) + (lane >> 3); }
  __device__ __forceinline__ int side(int i) const { return MODE != GATED ? 0 : NW == 8 ? wave >> 2 : i & 1; }
  static constexpr int bstep() { return MODE == GATED ? 32 : 8 * NW; }
  static constexpr int bindex(int i) { return MODE == GATED && NW == 4 ? i >> 1 : i; }
  __device__ __forceinline__ void begin(int stage) {
    const int arow = 8 * wave + (lane >> 3);
    if (stage < KM) {
      const uint32_t k2 = (uint32_t)p.K * 2;
      ra = make_rsrc((const char*)p.x + pl.m0 * p.K * 2, (int64_t)pl.rows * k2);
      rb[0] = make_rsrc((const char*)p.w0 + pl.n0 * p.K * 2, ncols * k2);
      if (MODE == GATED) rb[1] = make_rsrc((const char*)p.w1 + pl.n0 * p.K * 2, ncols * k2);
      oa = arow * k2 + 16 * chunk;
      ob = brow() * k2 + 16 * chunk;
      sa = 8 * NW * k2;
      sb = bstep() * k2;
      so = (uint32_t)stage * 128;
    } else {
      // the low-rank part, or (past it) empty buffers: nothing is fetched
      const int u = stage - KM, at = MODE == PLAIN ? 64 * u : 0;  // first column of the W-side operand
      const bool in = u < (MODE == GATED ? 2 : MODE == PLAIN ? KT - KM : 1);
      const int64_t ldl = MODE == GATED && u ? p.ldl1 : p.ldl0;
      ra = make_rsrc((const char*)p.t + (pl.m0 * p.ldt + 64 * u) * 2, in ? (pl.rows * p.ldt - 64 * u) * 2 : 0);
      const void* l = MODE == GATED && u ? p.l1 : p.l0;
      const rsrc_t some = make_rsrc((const char*)l + (pl.n0 * ldl + at) * 2, in ? (ncols * ldl - at) * 2 : 0);
      const rsrc_t none = make_rsrc(p.x, 0);
      rb[0] = MODE == GATED && u ? none : some;
      if (MODE == GATED) rb[1] = u ? some : none;
      // columns that are not there are zeros on both sides: what lies in their place may be no number
      oa = (uint32_t)(arow * (int)p.ldt * 2 + 16 * chunk) | (64 * u + 8 * chunk < p.ldt ? 0u : 1u << 31);
      ob = (uint32_t)(brow() * (int)ldl * 2 + 16 * chunk) | (at + 8 * chunk < ldl ? 0u : 1u << 31);
      sa = (uint32_t)(8 * NW * (int)p.ldt * 2);
      sb = (uint32_t)(bstep() * (int)ldl * 2);
      so = 0;
    }
  }
  __device__ __forceinline__ void one(char* stage_lds, int, int i) const {
    char* dst = stage_lds + (wave + NW * i) * 1024;
    const int b = i - PER_A;
    if (b < 0) copy16(ra, dst, oa + i * sa, so);
    else copy16(MODE == GATED && side(b) ? rb[1] : rb[0], dst, ob + bindex(b) * sb, so);
  }
  __device__ __forceinline__ void all(char* stage_lds, int stage) {
    if (NW < T::NW && wave >= NW) return;
    begin(stage);
#pragma unroll
    for (int i = 0; i < PER; ++i) one(stage_lds, stage, i);
  }
  __device__ __forceinline__ void scales(int, int (&)[T::WMB], int&) const {}
  __device__ __forceinline__ void shift(int, int (&)[2][T::WMB], int (&)[2]) const {}
};

// 16-byte chunks of `rows` rows of RB bytes in W (chunk c of row r at chunk c ^ (r % NC)) to columns
// col0 .. of rows row0 .. of y [..][ld]; every wave issues exactly NC / 2 stores (chunks outside fall
// past the buffer), then element by element what fills no chunk, and waits for that.
template <int RB>
struct Rows16 {
  static constexpr int NC = RB / 16;
  __device__ static __forceinline__ int at(int r, int byte) { return r * RB + (((byte >> 4) ^ (r & (NC - 1))) << 4) + (byte & 15); }
  __device__ static __forceinline__ void store(const char* W, void* y, int64_t ld, int64_t row0, int64_t col0, int left,
                                               int ncols, int lane) {
    const int whole = ld < (1 << 25) ? ncols & ~7 : 0;
    const bool lines = (ld * 2) % 128 == 0 && ((uintptr_t)y & 127) == 0;
    char* base = (char*)y + (row0 * ld + col0) * 2;
    const rsrc_t r = make_rsrc(base, left > 0 && whole > 0 ? ((left - 1) * ld + whole) * 2 : 0);
    const int c = lane & (NC - 1);
    const uint32_t none = c * 8 < whole ? 0u : 1u << 31;
#pragma unroll
    for (int it = 0; it < NC / 2; ++it) {
      const int m = (64 / NC) * it + lane / NC;
      const u32x4_t v = *(const u32x4_t*)(W + m * RB + ((c ^ (m & (NC - 1))) << 4));
      const uint32_t off = (uint32_t)(m * (int)ld * 2 + c * 16);
      const int o = (int)((m < left ? off : 1u << 31) | none);
      if (lines) __builtin_amdgcn_raw_buffer_store_b128(v, r, o, 0, 2);
      else __builtin_amdgcn_raw_buffer_store_b128(v, r, o, 0, 0);
    }
    if (ncols > whole) {
      const int rest = ncols - whole;
      for (int q = lane; q < 32 * rest; q += 64) {
        const int m = q / rest, cc = whole + q % rest;
        if (m < left) ((uint16_t*)base)[m * ld + cc] = *(const uint16_t*)(W + at(m, 2 * cc));
      }
      wait_vmcnt<0>();
    }
  }
};

// h (and pre) of a wave's blocks: lane (r32, h) of block (i, j) holds row 32 i + r32, columns
// 8 q + 4 h + v in elements 4 q + v; an even j is g, the next is u of the same 32 columns.  Its 16 WNB
// columns of h, g and u pass one after the other through W: rows of whole 128-byte lines where WNB = 4.
// coef: the tile's biases, gate then up.
template <int CD, int ACT, class T>
__device__ __forceinline__ void write_gated(const G16& p, const Place& pl, Acc<T>& acc, const float* coef, char* W,
                                            int wave, int lane) {
  constexpr int C = cols_of<T, GATED>(), PAIRS = T::WNB / 2, RB = 64 * PAIRS;
  const int h = lane >> 5, r32 = lane & 31;
  const int wm = (wave / T::NWN) * 32 * T::WMB, wc = (wave % T::NWN) * 32 * PAIRS;
  const int ncols = (int)max((int64_t)0, min((int64_t)(32 * PAIRS), p.n - pl.n0 - wc));
#pragma unroll
  for (int i = 0; i < T::WMB; ++i) {
    const int row0 = wm + 32 * i, left = min(32, pl.rows - row0);
#pragma unroll
    for (int part = 0; part < 3; ++part) {  // h, g, u
      if (part && !p.pre) break;
#pragma unroll
      for (int j = 0; j < PAIRS; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float o[4];
          if (part == 0) {
            const int at = wc + 32 * j + 8 * q + 4 * h;
            const f32x4_t bg = *(const f32x4_t*)(coef + at), bu = *(const f32x4_t*)(coef + C + at);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              acc[i][2 * j][4 * q + v] += bg[v];
              acc[i][2 * j + 1][4 * q + v] += bu[v];
              o[v] = act_of<ACT>(acc[i][2 * j][4 * q + v]) * acc[i][2 * j + 1][4 * q + v];
            }
          } else {
#pragma unroll
            for (int v = 0; v < 4; ++v) o[v] = acc[i][2 * j + part - 1][4 * q + v];
          }
          *(u32x2_t*)(W + Rows16<RB>::at(r32, 64 * j + 16 * q + 8 * h)) = u32x2_t{pack2<CD>(o[0], o[1]), pack2<CD>(o[2], o[3])};
        }
      wait_lgkm0();  // the wave reads back only what it wrote
      asm volatile("" ::: "memory");
      Rows16<RB>::store(W, part ? p.pre : p.out, part ? 2 * p.n : p.n, pl.m0 + row0, pl.n0 + wc + (part == 2 ? p.n : 0), left,
                        ncols, lane);
      wait_lgkm0();  // the reads are done before the next rows overwrite them
      asm volatile("" ::: "memory");
    }
  }
}

// dX of a wave's blocks: the masked low-rank sums (operands in LDS at `st`, as a stage) added.
template <int CD, class T>
__device__ __forceinline__ void add_masked(Acc<T>& acc, const G16& p, const Place& pl, const char* st, int wave, int lane) {
  const int h = lane >> 5, r32 = lane & 31, xr = swz(r32);
  const int wm = (wave / T::NWN) * 32 * T::WMB, wn = (wave % T::NWN) * 32 * T::WNB;
  uint32_t bits[T::WMB][T::WNB];
  const rsrc_t rm = make_rsrc(p.bits + pl.m0 * p.ldbits, pl.rows * p.ldbits * 4);
#pragma unroll
  for (int i = 0; i < T::WMB; ++i)
#pragma unroll
    for (int j = 0; j < T::WNB; ++j)
      bits[i][j] = __builtin_amdgcn_raw_buffer_load_b32(rm, ((wm + 32 * i + r32) * (int)p.ldbits + (int)((pl.n0 + wn) >> 5) + j) * 4,
                                                        0, 0) >> (4 * h);
  const char *a = st + (wm + r32) * 128, *b = st + (T::TM + wn + r32) * 128;
#pragma unroll
  for (int i = 0; i < T::WMB; ++i)
#pragma unroll
    for (int j = 0; j < T::WNB; ++j) {
      f32x16_t low;
#pragma unroll
      for (int v = 0; v < 16; ++v) low[v] = 0.f;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        Half16<CD>::mma(low, Half16<CD>::read(b + j * 32 * 128, ks, h, xr), Half16<CD>::read(a + i * 32 * 128, ks, h, xr), 0, 0);
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          acc[i][j][4 * q + v] += bits[i][j] >> (8 * q + v) & 1u ? low[4 * q + v] : 0.f;
      // one block's operands at a time: the sums leave room for no more
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("" ::: "memory");
    }
}
// coef: with BIAS the tile's biases.
template <int CD, class T, bool BIAS>
__device__ __forceinline__ void write_plain(const G16& p, const Place& pl, const Acc<T>& acc, const float* coef, char* W,
                                            int wave, int lane) {
  constexpr int RB = 64 * T::WNB;
  const int h = lane >> 5, r32 = lane & 31;
  const int wm = (wave / T::NWN) * 32 * T::WMB, wn = (wave % T::NWN) * 32 * T::WNB;
  const int ncols = (int)max((int64_t)0, min((int64_t)(32 * T::WNB), p.n - pl.n0 - wn));
#pragma unroll
  for (int i = 0; i < T::WMB; ++i) {
#pragma unroll
    for (int j = 0; j < T::WNB; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f32x4_t v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        if (BIAS) v += *(const f32x4_t*)(coef + wn + 32 * j + 8 * q + 4 * h);
        *(u32x2_t*)(W + Rows16<RB>::at(r32, 64 * j + 16 * q + 8 * h)) = u32x2_t{pack2<CD>(v[0], v[1]), pack2<CD>(v[2], v[3])};
      }
    wait_lgkm0();
    asm volatile("" ::: "memory");
    Rows16<RB>::store(W, p.out, p.n, pl.m0 + wm + 32 * i, pl.n0 + wn, min(32, pl.rows - wm - 32 * i), ncols, lane);
    wait_lgkm0();
    asm volatile("" ::: "memory");
  }
}

// The tile of half the rows that an incomplete last round takes, two workgroups to a tile.
template <class T>
struct HalfOf {
  using type = T;
};
template <int WMB, int WNB, int NWM, int NWN>
struct HalfOf<Tile<WMB, WNB, NWM, NWN, 2>> {
  using type = Tile<WMB / 2, WNB, NWM, NWN, 2>;
};

// Bound by the matrix pipes at the card's power limit (us, a trace's fastest and median call): gated, 4096 x 14336 x 4096, 749
// and 850 (1.30 and 1.15 PFLOP/s; pipes busy 76% of the cycles at 1.63 GHz); plain, 4096 x 4096 x 28672, 735 and 792 (73%);
// masked, 4096 x 14336 x 4096, 394 and 440 (67%).
// A workgroup goes through its tiles.  After a tile's last stage the copies of the next tile's first
// stage are requested, so that they land while this one's outputs are formed and stored; those pass
// through LDS behind that stage.  A last round of at most half the workgroups runs as tiles of half
// the rows (the largest tiles).
template <int CD, class T, int MODE, int WGS>
__global__ __launch_bounds__(64 * T::NW, WGS) void k_gemm16(G16 p, int act) {
  using H = typename HalfOf<T>::type;
  constexpr bool HALVES = !std::is_same_v<T, H>;
  constexpr int C = cols_of<T, MODE>(), COEF = MODE == GATED ? 2 * C : MODE == PLAIN ? C : 0, STAGING = MODE == GATED ? 1024 * T::WNB : 2048 * T::WNB;
  static_assert(T::LDS - T::STAGE >= T::NW * STAGING, "staging fits");
  __shared__ __attribute__((aligned(1024))) char lds[T::LDS + 2 * COEF * 4];  // one array: see fp8.hip
  float* coefs = (float*)(lds + T::LDS);  // two sets, used in turn
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tiles_n = (int)((p.n + C - 1) / C), tiles_m = (int)((p.m + T::TM - 1) / T::TM), total = tiles_m * tiles_n;
  const int G = gridDim.x, b = blockIdx.x;
  // The workgroup's tile in round r; rows 0: none (any more).
  auto item = [&](int r) {
    Place pl = {0, 0, 0};
    const int64_t base = (int64_t)r * G;
    if (base >= total) return pl;
    const int rem = total - (int)base, n = min(G, rem);
    const bool cut = HALVES && 2 * rem <= G;
    if (b >= (cut ? 2 * rem : n)) return pl;
    const int pos = xcd_run(b, cut ? 2 * rem : n), half = cut ? pos & 1 : 0;
    int tm, tn;
    grouped_tile((int)base + (cut ? pos >> 1 : pos), tiles_m, tiles_n, tm, tn);
    pl.m0 = (int64_t)__builtin_amdgcn_readfirstlane(tm) * T::TM + half * H::TM;
    pl.n0 = (int64_t)__builtin_amdgcn_readfirstlane(tn) * C;
    pl.rows = (int)max((int64_t)0, min((int64_t)(cut ? H::TM : T::TM), p.m - pl.m0));
    return pl;
  };
  auto coef_of = [&](const Place& pl, int i) {
    const int64_t col = pl.n0 + (i >= C ? i - C : i);
    return p.bias && col < p.n ? load_cd<CD>(p.bias, col + (i >= C ? p.n : 0)) : 0.f;
  };
  auto first_stage = [&](const Place& pl) {
    if (HALVES && pl.rows <= H::TM) Copies16<H, MODE>(p, pl, wave, lane).all(lds, 0);
    else Copies16<T, MODE>(p, pl, wave, lane).all(lds, 0);
  };

  Place cur = item(0);
  if (cur.rows == 0) return;
  if (COEF)
    for (int i = tid; i < COEF; i += 64 * T::NW) coefs[i] = coef_of(cur, i);
  first_stage(cur);
  int set = 0;
  for (int r = 1;; ++r) {
    const Place nxt = item(r);
    static_assert(COEF <= 64 * T::NW, "one coefficient to a thread");
    const float c = COEF && nxt.rows && tid < COEF ? coef_of(nxt, tid) : 0.f;
    auto work = [&](auto shape) {
      using U = decltype(shape);
      // the lane counts as unknown here and after the contraction: addresses of either shape and of the
      // outputs, formed ahead of all tiles, would be kept through the contraction and pushed out to memory
      int ln = lane;
      asm volatile("" : "+v"(ln));
      Copies16<U, MODE> cp(p, cur, wave, ln);
      Acc<U> acc;
      zero<U>(acc);
      wait_vmcnt<0>();
      wait_lgkm0();
      barrier_only();  // stage 0 and the coefficients are there, the staging of the tile before is free
#pragma unroll
      for (int s = 1; s < U::NS; ++s) cp.all(lds + s * U::STAGE, s);
      contract<U, Half16<CD>>(acc, lds, cp, wave, ln);
      asm volatile("" : "+v"(ln));
      if constexpr (MODE == MASKED) {
        add_masked<CD, U>(acc, p, cur, lds + cp.KM % U::NS * U::STAGE, wave, ln);
        __syncthreads();  // every wave is past the low-rank operands
      }
      if (nxt.rows) {
        if (COEF && tid < COEF) coefs[(set ^ 1) * COEF + tid] = c;
        first_stage(nxt);
      }
      char* W = lds + T::STAGE + wave * STAGING;
      if constexpr (MODE == GATED) {
        const float* co = coefs + set * COEF;
        if (act == QLORA_ACT_SILU) write_gated<CD, QLORA_ACT_SILU, U>(p, cur, acc, co, W, wave, ln);
        else if (act == QLORA_ACT_GELU) write_gated<CD, QLORA_ACT_GELU, U>(p, cur, acc, co, W, wave, ln);
        else write_gated<CD, QLORA_ACT_GELU_TANH, U>(p, cur, acc, co, W, wave, ln);
      } else {
        write_plain<CD, U, MODE == PLAIN>(p, cur, acc, coefs + set * COEF, W, wave, ln);
      }
    };
    if (HALVES && cur.rows <= H::TM) work(H{});
    else work(T{});
    if (nxt.rows == 0) return;
    cur = nxt;
    set ^= 1;
  }
}

// 256 rows x 256 columns (128 of each projection), eight waves; a gated wave takes 64 rows of 64
// columns of h, whole lines of the outputs
using FullGated = Tile<2, 4, 4, 2, 2>;
using Full = Tile<4, 2, 2, 4, 2>;
using Wide = Tile<2, 2, 2, 4, 3>;  // 128 x 256, eight waves
using Mid = Tile<2, 2, 2, 2, 4>;   // 128 x 128, four waves
using Low = Tile<1, 2, 2, 2, 3>;   // 64 x 128, four waves; two workgroups fit a compute unit

template <int CD, class T, int MODE, int WGS>
int run(const G16& p, int act, int kind, hipStream_t s) {
  const int64_t tiles = ceil_div(p.m, T::TM) * ceil_div(p.n, cols_of<T, MODE>());
  ProfScope prof(kind, s);
  k_gemm16<CD, T, MODE, WGS><<<dim3((unsigned)std::min<int64_t>(tiles, cu_count() * WGS)), dim3(64 * T::NW), 0, s>>>(p, act);
  return check_launch("k_gemm16");
}

// The smallest tiles that fit the compute units in one round, the largest beyond (us by Low, Mid, Wide, the
// largest, of the whole call, bf16: gated 512 x 2048 x 2048 36, 38, 46, 58, 2048 x 4096 x 1024 79, 77, 70, 59; plain
// 512 x 4096 x 4096 44, 51, 65, 85, 1024 x 4096 x 4096 62, 57, 67, 86, 2048 x 4096 x 4096 106, 96, 84, 92; masked
// 1024 x 4096 x 4096 -, 73, 83, 108, 2048 x 4096 x 4096 -, 115, 102, 119).
template <int CD, int MODE>
int run_cd(const G16& p, int act, int kind, hipStream_t s) {
  auto one_round = [&](int64_t tm, int64_t tn) {
    return ceil_div(p.m, tm) * ceil_div(p.n, MODE == GATED ? tn / 2 : tn) <= cu_count();
  };
  if constexpr (MODE != MASKED)
    if (one_round(64, 128)) return run<CD, Low, MODE, 2>(p, act, kind, s);
  if (one_round(128, 128)) return run<CD, Mid, MODE, 1>(p, act, kind, s);
  if (one_round(128, 256)) return run<CD, Wide, MODE, 1>(p, act, kind, s);
  return run<CD, std::conditional_t<MODE == GATED, FullGated, Full>, MODE, 1>(p, act, kind, s);
}

}  // namespace

// Whether the kernels take a call: 16-bit operands, whole stages of K, offsets within a tile below 2^31.
bool gemm16_ok(int cd, int64_t m, int64_t n, int64_t K) {
  return (cd == CD_BF16 || cd == CD_F16) && K % 64 == 0 && K > 0 && K < (1 << 21) && m > 0 && m < (1LL << 31) && n > 0 &&
         n < (1LL << 31) && ceil_div(m, 64) * ceil_div(n, 64) < (1LL << 31);
}

// h (and pre, if not null) of x [m][K], W~ w[i] [n][K], T [m][128] (T_i in columns 64 i ..), lora_b b[i] [n][ldb[i]]
// with ldb a multiple of 8.
int gemm16_gated(int cd, const void* x, int64_t m, int64_t n, int64_t K, const void* const* w, const void* t,
                 const void* const* b, const int64_t* ldb, const void* bias, int act, void* h, void* pre, hipStream_t s) {
  G16 p = {};
  p.x = x;
  p.w0 = w[0];
  p.w1 = w[1];
  p.t = t;
  p.ldt = 128;
  p.l0 = b[0];
  p.l1 = b[1];
  p.ldl0 = ldb[0];
  p.ldl1 = ldb[1];
  p.bias = bias;
  p.out = h;
  p.pre = pre;
  p.m = m;
  p.n = n;
  p.K = K;
  return cd == CD_BF16 ? run_cd<CD_BF16, GATED>(p, act, QLORA_K_FWD_GEMM, s) : run_cd<CD_F16, GATED>(p, act, QLORA_K_FWD_GEMM, s);
}

// dX [m][n] = dY [m][K] W~^T wt [n][K] + (dT [m][ldt] A^T at [n][lda]) M, ldt and lda multiples of 8, at most 64;
// bits [m][ldbits] words of M's bits.
int gemm16_masked_dx(int cd, const void* dy, int64_t m, int64_t n, int64_t K, const void* wt, const void* dt, int64_t ldt,
                     const void* at, int64_t lda, const void* bits, int64_t ldbits, void* dx, hipStream_t s) {
  G16 p = {};
  p.x = dy;
  p.w0 = wt;
  p.t = dt;
  p.ldt = ldt;
  p.l0 = at;
  p.ldl0 = lda;
  p.out = dx;
  p.m = m;
  p.n = n;
  p.K = K;
  p.bits = (const uint32_t*)bits;
  p.ldbits = ldbits;
  return cd == CD_BF16 ? run_cd<CD_BF16, MASKED>(p, 0, QLORA_K_BWD_DX, s) : run_cd<CD_F16, MASKED>(p, 0, QLORA_K_BWD_DX, s);
}

// y [m][n] = [x [m][K] | t [m][ldt]] [w [n][K] | l [n][ldl]]^T (+ bias), ldt and ldl multiples of 8; x and w rows
// of K elements.
int gemm16_plain(int cd, const void* x, int64_t m, int64_t n, int64_t K, const void* w, const void* t, int64_t ldt,
                 const void* l, int64_t ldl, const void* bias, void* y, int kind, hipStream_t s) {
  G16 p = {};
  p.x = x;
  p.w0 = w;
  p.t = t;
  p.ldt = ldt;
  p.l0 = l;
  p.ldl0 = ldl;
  p.bias = bias;
  p.out = y;
  p.m = m;
  p.n = n;
  p.K = K;
  return cd == CD_BF16 ? run_cd<CD_BF16, PLAIN>(p, 0, kind, s) : run_cd<CD_F16, PLAIN>(p, 0, kind, s);
}

}  // namespace qnf4
