// distill.hip -- distillation loss against a teacher's top logits, with its gradient.
//
// Row i of student logits z [V], the teacher's k highest logits u at vocabulary indices
// idx, temperature T, weight w:
//   p = softmax(u / T) over the present slots,  q = softmax(z / T) over the vocabulary,
//   kl = T^2 sum_j p_j (log p_j - log q[idx_j]),  loss = sum_i w_i kl_i,
//   dz = w T (q - p scattered to idx).
// A slot is absent when its index lies outside [0, V) or its value is -inf.  A row with
// weight 0 or without a present slot has kl 0 and a zero gradient, whatever its logits
// hold.
//
// Bound by HBM: each logit read once, each gradient written once.  A workgroup keeps its
// row in registers (as loaded, 16 bytes per chunk) between the maximum, the sum and the
// gradient, and asks for the next row's chunk as soon as it has written the gradient of
// the one in that register, so reads, writes and the exponentials overlap.  Rows too
// long for the registers are read a second time (they then come from the caches).
#include <math.h>

#include <algorithm>

#include "int8_distill.h"

namespace qnf4 {
namespace {

constexpr int kMaxK = QLORA_DISTILL_MAX_K;
constexpr int kFewSlots = 128;  // slots the small form of the LDS arrays holds

struct Distill {
  const void* z;       // [n][ldz] cd
  int64_t ldz;
  void* dz;            // [n][lddz] cd or null
  int64_t lddz;
  const void* u;       // [n][k] teacher values (ud)
  const void* idx;     // [n][k] int32 or int64
  const float* weight; // [n] or null: w_default
  float* kl;           // [n]
  int64_t n, V;
  int32_t k, ud, idx64;
  float t, c;          // T, log2(e) / T
  float w_default;
};

__device__ __forceinline__ float load_any(const void* p, int64_t i, int cd) {
  return cd == CD_F32 ? load_cd<CD_F32>(p, i) : cd == CD_BF16 ? load_cd<CD_BF16>(p, i) : load_cd<CD_F16>(p, i);
}

// Rows start at any element: the memory system takes 16-byte vectors at any address, and a
// buffer's end keeps the lanes past the last whole chunk from reading or writing.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t make_rsrc(const void* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, bytes, 0x00020000);
}

template <int CD>
struct Elem {
  static constexpr int ES = CD == CD_F32 ? 4 : 2, PC = 16 / ES;  // elements per chunk
  __device__ static __forceinline__ float get(const u32x4_t& v, int e) {
    if constexpr (CD == CD_F32) return __uint_as_float(v[e]);
    else if constexpr (CD == CD_BF16) return __uint_as_float((e & 1) ? v[e >> 1] & 0xffff0000u : v[e >> 1] << 16);
    else return from_cd16<CD>((uint16_t)(v[e >> 1] >> (16 * (e & 1))));
  }
  __device__ static __forceinline__ u32x4_t pack(const float (&g)[PC]) {
    u32x4_t o;
    if constexpr (CD == CD_F32) {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = __float_as_uint(g[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = pack2<CD>(g[2 * e], g[2 * e + 1]);
    }
    return o;
  }
};

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// A row's teacher slots in LDS.  Slot j hangs in the list (head / next) of the thread that
// writes the gradient of the chunk its index lies in: that thread, after its chunks, writes
// the entries of its list once more with the teacher's share taken off (stores of one thread
// to one address keep their order).  Two sets, used in turn by the rows that are not left
// out: a wave that is ahead fills the next such row's set while others still read this
// row's, and that row's first barrier holds it until they are done.
template <int TPB, int KC>
struct Slots {
  int32_t head[TPB];    // first slot of the thread's list, -1: none
  int32_t next[KC];
  int32_t idx[KC];   // -1: absent
  float e[KC];       // exp((u - max) / T)
  float share[KC];   // p summed over the slots of the same index, at the first of them; else -1
  float z[KC];       // the student's logit at the index
  float zmax[TPB / 64], umax[TPB / 64], zsum[TPB / 64], usum[TPB / 64], kl[TPB / 64];  // one per wave
  int any[TPB / 64];
};
// The passes read a chunk's register anew: without this the compiler keeps every converted
// element and exponential of one pass alive for the next, which takes many times the
// registers the row itself does.
__device__ __forceinline__ void opaque(u32x4_t& x) { asm volatile("" : "+v"(x)); }

// NV > 0: rows of at most NV * TPB whole chunks, kept in registers.  NV = 0: rows of any
// length, read twice.  Entries past the last whole chunk (fewer than a chunk) go one to a
// thread.
template <int CD, int TPB, int NV, int KC>
__global__ __launch_bounds__(TPB, TPB <= 256 ? 3 : 4) void k_distill(Distill p) {
  using E = Elem<CD>;
  constexpr int PC = E::PC, NW = TPB / 64, SPT = (KC + TPB - 1) / TPB, NR = NV > 0 ? NV : 1;
  __shared__ Slots<TPB, KC> sets[2];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int V = (int)p.V;
  const int full = V / PC, left = V - full * PC;  // whole chunks, entries past them
  const uint32_t toff = tid * 16;
  auto weight_of = [&](int64_t i) { return p.weight ? p.weight[i] : p.w_default; };
  auto zrow_of = [&](int64_t i) { return (const char*)p.z + i * p.ldz * E::ES; };
  auto owner = [&](int ix) { return ix < full * PC ? (ix / PC) % TPB : ix - full * PC; };

  u32x4_t v[NR];
  float vl = -INFINITY;  // the thread's entry past the last whole chunk
  // A row's whole chunks as a buffer: lanes past them read nothing and write nothing; for a
  // row that is left out (weight 0, or none) the buffer is empty.
  auto chunks_of = [&](const void* row, bool there) { return make_rsrc(row, there ? full * 16 : 0); };
  auto fetch = [&](rsrc_t r, int s) {
    v[s] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)toff, s * TPB * 16, 0));
  };
  auto fetch_left = [&](const char* row) {
    if (tid < left) vl = load_cd<CD>(row, (int64_t)full * PC + tid);
  };
  int64_t i = blockIdx.x;
  float w = weight_of(i);
  if (NV > 0 && w != 0.f) {
#pragma unroll
    for (int s = 0; s < NV; ++s) fetch(chunks_of(zrow_of(i), true), s);
    fetch_left(zrow_of(i));
  }
  int turn = 0;
  while (i < p.n) {
    const char* zr = zrow_of(i);
    char* dr = p.dz ? (char*)p.dz + i * p.lddz * E::ES : nullptr;
    const int64_t ni = i + gridDim.x;
    const float nw = ni < p.n ? weight_of(ni) : 0.f;
    const char* nz = zrow_of(ni);  // read only where nw is not 0
    const rsrc_t rn = chunks_of(nz, nw != 0.f);
    bool live = w != 0.f;
    Slots<TPB, KC>& S = sets[turn];
    if (live) turn ^= 1;
    float m = 0.f, sum = 0.f, umax = 0.f, usum = 0.f;
    if (live) {
      // the row's slots, and the largest logit of the thread's entries
      float su[SPT], sz[SPT];
      int32_t si[SPT];
      S.head[tid] = -1;
      float um = -INFINITY;
      bool here = false;
#pragma unroll
      for (int s = 0; s < SPT; ++s) {
        const int j = tid + s * TPB;
        si[s] = -1;
        if (j < p.k) {
          const int64_t at = i * p.k + j;
          const int64_t ix = p.idx64 ? ((const int64_t*)p.idx)[at] : (int64_t)((const int32_t*)p.idx)[at];
          su[s] = load_any(p.u, at, p.ud);
          if (ix >= 0 && ix < V && !(su[s] == -INFINITY)) {
            si[s] = (int32_t)ix;
            sz[s] = load_cd<CD>(zr, ix);
            S.z[j] = sz[s];
            um = fmaxf(um, su[s]);
            here = true;
          }
          S.idx[j] = si[s];
        }
      }
      float zm = -INFINITY, zs = 0.f;
      if constexpr (NV > 0) {
#pragma unroll
        for (int s = 0; s < NV; ++s)
          if (s * TPB + wave * 64 < full) {
            opaque(v[s]);
            float cm = E::get(v[s], 0);
#pragma unroll
            for (int e = 1; e < PC; ++e) cm = fmaxf(cm, E::get(v[s], e));
            zm = fmaxf(zm, s * TPB + tid < full ? cm : -INFINITY);
            __builtin_amdgcn_sched_barrier(0);
          }
        zm = fmaxf(zm, vl);
      } else {
        // running maximum and sum of the thread's entries, four chunks at a time while the next
        // four are on their way
        auto add = [&](float cm, auto share) {
          const float nm = fmaxf(zm, cm);
          // a thread that has met only -inf so far has no share yet, and one that has met NaN as
          // well (fmaxf passes over it) has a NaN, which stays
          zs = (zm == -INFINITY ? zs : zs * __builtin_amdgcn_exp2f((zm - nm) * p.c)) + share(nm);
          zm = nm;
        };
        auto part = [&](float y, float nm) { return y == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((y - nm) * p.c); };
        constexpr int B = 4;
        u32x4_t x[2][B];
        auto ask = [&](u32x4_t (&to)[B], int c0) {  // past the last whole chunk: an empty buffer
          const int here = min(max(full - c0, 0), B * TPB);
          const rsrc_t r = make_rsrc(zr + (int64_t)c0 * 16, here * 16);
#pragma unroll
          for (int s = 0; s < B; ++s)
            to[s] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)toff, s * TPB * 16, 0));
        };
        auto take = [&](const u32x4_t (&of)[B], int c0) {
#pragma unroll
          for (int s = 0; s < B; ++s)
            if (c0 + s * TPB + tid < full) {
              float cm = E::get(of[s], 0);
#pragma unroll
              for (int e = 1; e < PC; ++e) cm = fmaxf(cm, E::get(of[s], e));
              add(cm, [&](float nm) {
                float cs = 0.f;
#pragma unroll
                for (int e = 0; e < PC; ++e) cs += part(E::get(of[s], e), nm);
                return cs;
              });
            }
        };
        ask(x[0], 0);
        for (int c0 = 0; c0 < full; c0 += 2 * B * TPB) {
          ask(x[1], c0 + B * TPB);
          take(x[0], c0);
          ask(x[0], c0 + 2 * B * TPB);
          take(x[1], c0 + B * TPB);
        }
        vl = -INFINITY;
        fetch_left(zr);
        if (tid < left) add(vl, [&](float nm) { return part(vl, nm); });
      }
      const float zm_own = zm;
      zm = wave_max(zm);
      um = wave_max(um);
      const bool wave_here = __any(here);
      if (lane == 0) {
        S.zmax[wave] = zm;
        S.umax[wave] = um;
        S.any[wave] = wave_here;
      }
      __syncthreads();
      m = S.zmax[0];
      umax = S.umax[0];
      int any = S.any[0];
#pragma unroll
      for (int x = 1; x < NW; ++x) {
        m = fmaxf(m, S.zmax[x]);
        umax = fmaxf(umax, S.umax[x]);
        any |= S.any[x];
      }
      live = any != 0;
      if (live) {
        float us = 0.f;
#pragma unroll
        for (int s = 0; s < SPT; ++s)
          if (si[s] >= 0) {
            const int j = tid + s * TPB;
            const float ex = __builtin_amdgcn_exp2f((su[s] - umax) * p.c);
            S.e[j] = ex;
            us += ex;
            S.next[j] = atomicExch(&S.head[owner(si[s])], j);
          }
        if constexpr (NV > 0) {
#pragma unroll
          for (int s = 0; s < NV; ++s) {
            opaque(v[s]);
            if (s * TPB + wave * 64 < full) {
              float cs[2] = {0.f, 0.f};
#pragma unroll
              for (int e = 0; e < PC; ++e) cs[e & 1] += __builtin_amdgcn_exp2f((E::get(v[s], e) - m) * p.c);
              zs += s * TPB + tid < full ? cs[0] + cs[1] : 0.f;
              __builtin_amdgcn_sched_barrier(0);
            }
          }
          if (tid < left) zs += __builtin_amdgcn_exp2f((vl - m) * p.c);
        } else {
          // the thread's share under the row's maximum; all of it -inf: none (a NaN stays)
          zs = zm_own == -INFINITY && zs == 0.f ? 0.f : zs * __builtin_amdgcn_exp2f((zm_own - m) * p.c);
        }
        zs = wave_sum(zs);
        us = wave_sum(us);
        if (lane == 0) {
          S.zsum[wave] = zs;
          S.usum[wave] = us;
        }
        __syncthreads();
        sum = S.zsum[0];
        usum = S.usum[0];
#pragma unroll
        for (int x = 1; x < NW; ++x) {
          sum += S.zsum[x];
          usum += S.usum[x];
        }
        // kl = sum_j T p_j (u_j - z_j + T log(...)), with no 1 / T: fp32 holds a difference against
        // a logit at the type's lowest value, but not its quotient by a T below 1; and the share
        // each index carries
        const float lsum = p.t * (logf(sum) - logf(usum)), uinv = 1.0f / usum;
        float kl = 0.f;
#pragma unroll
        for (int s = 0; s < SPT; ++s)
          if (si[s] >= 0) {
            const int j = tid + s * TPB;
            const float pr = S.e[j] * uinv;
            if (pr != 0.f) kl += pr * p.t * (((su[s] - umax) - (sz[s] - m)) + lsum);
            int first = j, same = 0;
            for (int l = S.head[owner(si[s])]; l >= 0; l = S.next[l])
              if (S.idx[l] == si[s]) {
                first = min(first, l);
                ++same;
              }
            float share = -1.f;
            if (first == j) {
              share = pr;
              if (same > 1) {  // in slot order, so that the sum is the same every time
                share = 0.f;
                for (int l = j; l < p.k; ++l)
                  if (S.idx[l] == si[s]) share += S.e[l] * uinv;
              }
            }
            S.share[j] = share;
          }
        kl = wave_sum(kl);
        if (lane == 0) S.kl[wave] = kl;
        __syncthreads();
        if (tid == 0) {
          float t = S.kl[0];
#pragma unroll
          for (int x = 1; x < NW; ++x) t += S.kl[x];
          p.kl[i] = t;
        }
      }
    }
    if (!live && tid == 0) p.kl[i] = 0.f;
    const float wt = w * p.t, inv = 1.0f / sum, gs = wt * inv;
    // a chunk's gradient before the teacher's shares; zeros for a row that is left out
    auto grad = [&](const u32x4_t& x) {
      u32x4_t o = {0u, 0u, 0u, 0u};
      if (live) {
        float g[PC];
#pragma unroll
        for (int e = 0; e < PC; ++e) g[e] = gs * __builtin_amdgcn_exp2f((E::get(x, e) - m) * p.c);
        o = E::pack(g);
      }
      return o;
    };
    if constexpr (NV > 0) {
      const rsrc_t rd = chunks_of(dr, dr != nullptr);
#pragma unroll
      for (int s = 0; s < NV; ++s) {
        opaque(v[s]);
        if (s * TPB + wave * 64 < full)
          __builtin_amdgcn_raw_buffer_store_b128(grad(v[s]), rd, (int)toff, s * TPB * 16, 0);
        fetch(rn, s);
        __builtin_amdgcn_sched_barrier(0);  // one chunk's exponentials at a time
      }
    } else if (dr) {
      constexpr int B = 4;
      u32x4_t x[2][B];
      auto ask = [&](u32x4_t (&to)[B], int c0) {
        const int here = min(max(full - c0, 0), B * TPB);
        const rsrc_t r = make_rsrc(zr + (int64_t)c0 * 16, live ? here * 16 : 0);
#pragma unroll
        for (int s = 0; s < B; ++s)
          to[s] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)toff, s * TPB * 16, 0));
      };
      auto give = [&](const u32x4_t (&of)[B], int c0) {
        const int here = min(max(full - c0, 0), B * TPB);
        const rsrc_t r = make_rsrc(dr + (int64_t)c0 * 16, here * 16);
#pragma unroll
        for (int s = 0; s < B; ++s)
          if (c0 + s * TPB + wave * 64 < full)
            __builtin_amdgcn_raw_buffer_store_b128(grad(of[s]), r, (int)toff, s * TPB * 16, 0);
      };
      ask(x[0], 0);
      for (int c0 = 0; c0 < full; c0 += 2 * B * TPB) {
        ask(x[1], c0 + B * TPB);
        give(x[0], c0);
        ask(x[0], c0 + 2 * B * TPB);
        give(x[1], c0 + B * TPB);
      }
    }
    if (dr) {
      if (tid < left)
        store_cd<CD>(dr, (int64_t)full * PC + tid, live ? gs * __builtin_amdgcn_exp2f((vl - m) * p.c) : 0.f);
      for (int l = live ? S.head[tid] : -1; l >= 0; l = S.next[l]) {
        const float share = S.share[l];
        if (share < 0.f) continue;  // a later slot of the same index
        const float q = __builtin_amdgcn_exp2f((S.z[l] - m) * p.c) * inv;
        store_cd<CD>(dr, S.idx[l], wt * (q - share));
      }
    }
    if (NV > 0 && nw != 0.f) fetch_left(nz);
    i = ni;
    w = nw;
  }
}

// loss = sum of w_i kl_i in a fixed order, in 64 bits, rounded once.
constexpr int kSumThreads = 1024;
__global__ __launch_bounds__(kSumThreads) void k_distill_sum(const float* __restrict__ kl,
                                                             const float* __restrict__ weight, int64_t n,
                                                             float w_default, float* __restrict__ loss) {
  __shared__ double red[kSumThreads / 64];
  double acc = 0.0;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < n; i += kSumThreads) {
    const float w = weight ? weight[i] : w_default;
    acc += w == 0.f ? 0.0 : (double)w * (double)kl[i];
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) acc += __shfl_xor(acc, off, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = red[0];
#pragma unroll
    for (int x = 1; x < kSumThreads / 64; ++x) t += red[x];
    loss[0] = (float)t;
  }
}

// ------------------------------------------------------------------- a few rows
// With few rows a workgroup to a row leaves most of the chip idle, so a row is cut into parts
// of kPartChunks chunks, a workgroup each, in two launches: k_distill_part leaves each part's
// maximum and sum (and the student's logits at the teacher's entries, before an in-place
// gradient overwrites them), k_distill_join reads the parts' statistics and writes its part
// of the gradient.  The first part's workgroup also forms the row's kl, and the last of
// those workgroups to finish adds the rows up (in row order: the loss does not depend on
// which one that is).
constexpr int kPartThreads = 256;
constexpr int kPartNV = 2;
constexpr int kPartChunks = kPartThreads * kPartNV;

struct Split {
  float2* part;     // [n][parts] maximum, sum of exp((z - maximum) / T)
  float* zslot;     // [n][k] the student's logits at the teacher's entries
  uint32_t* done;   // rows whose kl is there
  float* loss;
  int parts;
};

// What both kernels do with part `part` of a row: its chunks into registers, the entry past
// the last whole chunk (last part only) into vl.
template <int CD>
struct Part {
  using E = Elem<CD>;
  int V, full, left, c0, here;  // here: whole chunks of this part
  __device__ __forceinline__ Part(int64_t V_, int part, int parts) {
    V = (int)V_;
    full = V / E::PC;
    c0 = part * kPartChunks;
    here = min(kPartChunks, full - c0);
    left = part == parts - 1 ? V - full * E::PC : 0;
  }
  __device__ __forceinline__ void load(const char* row, u32x4_t (&v)[kPartNV], float& vl) const {
    const rsrc_t r = make_rsrc(row + (int64_t)c0 * 16, here > 0 ? here * 16 : 0);
#pragma unroll
    for (int s = 0; s < kPartNV; ++s)
      v[s] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                             r, (int)(threadIdx.x * 16), s * kPartThreads * 16, 0));
    vl = (int)threadIdx.x < left ? load_cd<CD>(row, (int64_t)full * E::PC + threadIdx.x) : -INFINITY;
  }
  __device__ __forceinline__ bool has(int s) const { return (int)threadIdx.x + s * kPartThreads < here; }
};

__device__ __forceinline__ float block_max(float v, float* red) {
  v = wave_max(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
}
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

__device__ __forceinline__ int64_t slot_index(const Distill& p, int64_t at) {
  return p.idx64 ? ((const int64_t*)p.idx)[at] : (int64_t)((const int32_t*)p.idx)[at];
}

template <int CD>
__global__ __launch_bounds__(kPartThreads) void k_distill_part(Distill p, Split sp) {
  using E = Elem<CD>;
  __shared__ float red[2][kPartThreads / 64];
  const int64_t i = blockIdx.y;
  const int part = blockIdx.x, tid = threadIdx.x;
  if (i == 0 && part == 0 && tid == 0) *sp.done = 0;  // read by the next launch only
  if ((p.weight ? p.weight[i] : p.w_default) == 0.f) return;
  const char* row = (const char*)p.z + i * p.ldz * E::ES;
  const Part<CD> P(p.V, part, sp.parts);
  u32x4_t v[kPartNV];
  float vl;
  P.load(row, v, vl);
  if (part == 0)
    for (int j = tid; j < p.k; j += kPartThreads) {
      const int64_t ix = slot_index(p, i * p.k + j);
      if (ix >= 0 && ix < p.V) sp.zslot[i * p.k + j] = load_cd<CD>(row, ix);
    }
  float m = vl;
#pragma unroll
  for (int s = 0; s < kPartNV; ++s)
    if (P.has(s))
#pragma unroll
      for (int e = 0; e < E::PC; ++e) m = fmaxf(m, E::get(v[s], e));
  m = block_max(m, red[0]);
  float sum = 0.f;
  // a part of nothing but -inf has no share (a NaN in it still counts)
  auto add = [&](float z) { sum += z == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((z - m) * p.c); };
#pragma unroll
  for (int s = 0; s < kPartNV; ++s)
    if (P.has(s))
#pragma unroll
      for (int e = 0; e < E::PC; ++e) add(E::get(v[s], e));
  add(vl);
  sum = block_sum(sum, red[1]);
  if (tid == 0) sp.part[i * sp.parts + part] = make_float2(m, sum);
}

template <int CD, int KC>
__global__ __launch_bounds__(kPartThreads) void k_distill_join(Distill p, Split sp) {
  using E = Elem<CD>;
  constexpr int TPB = kPartThreads, SPT = (KC + TPB - 1) / TPB;
  __shared__ __attribute__((aligned(16))) int32_t s_idx[KC];  // the row's slots; -1: absent, or past the last
  __shared__ float s_e[KC], red[5][TPB / 64];
  __shared__ int s_last;
  const int64_t i = blockIdx.y;
  const int part = blockIdx.x, tid = threadIdx.x;
  const float w = p.weight ? p.weight[i] : p.w_default;
  const Part<CD> P(p.V, part, sp.parts);
  const char* row = (const char*)p.z + i * p.ldz * E::ES;
  char* dr = p.dz ? (char*)p.dz + i * p.lddz * E::ES : nullptr;
  float kl = 0.f, m = 0.f, inv = 0.f, umax = -INFINITY, usum = 0.f;
  bool live = w != 0.f;
  u32x4_t v[kPartNV];
  float vl = 0.f, su[SPT], sz[SPT];
  int32_t si[SPT];
  if (live) {
    if (dr) P.load(row, v, vl);
    bool here = false;
#pragma unroll
    for (int s = 0; s < SPT; ++s) {
      const int j = tid + s * TPB;
      si[s] = -1;
      if (j < p.k) {
        const int64_t at = i * p.k + j, ix = slot_index(p, at);
        su[s] = load_any(p.u, at, p.ud);
        if (ix >= 0 && ix < p.V && !(su[s] == -INFINITY)) {
          si[s] = (int32_t)ix;
          sz[s] = sp.zslot[at];
          umax = fmaxf(umax, su[s]);
          here = true;
        }
      }
      if (j < KC) s_idx[j] = si[s];
    }
    // the row's maximum and sum from its parts'
    float pm = -INFINITY;
    for (int q = tid; q < sp.parts; q += TPB) pm = fmaxf(pm, sp.part[i * sp.parts + q].x);
    m = block_max(pm, red[0]);
    umax = block_max(umax, red[1]);
    live = __syncthreads_or(here);
    if (live) {
      float ps = 0.f, us = 0.f;
      for (int q = tid; q < sp.parts; q += TPB) {
        const float2 x = sp.part[i * sp.parts + q];
        // a part of nothing but -inf adds nothing, unless the whole row is that (NaN)
        ps += x.x == -INFINITY && x.y == 0.f && m != -INFINITY ? 0.f : x.y * __builtin_amdgcn_exp2f((x.x - m) * p.c);
      }
#pragma unroll
      for (int s = 0; s < SPT; ++s)
        if (si[s] >= 0) {
          const float ex = __builtin_amdgcn_exp2f((su[s] - umax) * p.c);
          s_e[tid + s * TPB] = ex;
          us += ex;
        }
      const float sum = block_sum(ps, red[2]);
      usum = block_sum(us, red[3]);
      inv = 1.0f / sum;
      if (part == 0) {
        const float lsum = p.t * (logf(sum) - logf(usum));
#pragma unroll
        for (int s = 0; s < SPT; ++s)
          if (si[s] >= 0) {
            const float pr = s_e[tid + s * TPB] / usum;
            if (pr != 0.f) kl += pr * p.t * (((su[s] - umax) - (sz[s] - m)) + lsum);
          }
        kl = block_sum(kl, red[4]);
      }
    }
  }
  if (dr) {
    const float wt = w * p.t, gs = wt * inv;
    const rsrc_t rd = make_rsrc(dr + (int64_t)P.c0 * 16, P.here > 0 ? P.here * 16 : 0);
#pragma unroll
    for (int s = 0; s < kPartNV; ++s) {
      u32x4_t o = {0u, 0u, 0u, 0u};
      if (live) {
        float g[E::PC];
#pragma unroll
        for (int e = 0; e < E::PC; ++e) g[e] = gs * __builtin_amdgcn_exp2f((E::get(v[s], e) - m) * p.c);
        o = E::pack(g);
      }
      __builtin_amdgcn_raw_buffer_store_b128(o, rd, (int)(tid * 16), s * TPB * 16, 0);
    }
    if (tid < P.left)
      store_cd<CD>(dr, (int64_t)P.full * E::PC + tid, live ? gs * __builtin_amdgcn_exp2f((vl - m) * p.c) : 0.f);
    if (live) {
      // the part's entries that the teacher names, once more with its share taken off: after
      // every wave's stores above have reached memory
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
      const int first = P.c0 * E::PC, last = P.left ? P.V : (P.c0 + P.here) * E::PC;
#pragma unroll
      for (int s = 0; s < SPT; ++s) {
        const int j = tid + s * TPB;
        if (si[s] < first || si[s] >= last) continue;  // absent slots are below 0
        // does another slot name the same entry?  (16 at a time: one after the other, 217 slots
        // took 15 us)
        int same = 0;
        for (int l = 0; l < p.k; l += 16)
#pragma unroll
          for (int x = 0; x < 16; x += 4) {
            const int4 id = *(const int4*)&s_idx[l + x];
            same += (id.x == si[s]) + (id.y == si[s]) + (id.z == si[s]) + (id.w == si[s]);
          }
        float share = s_e[j] / usum;
        bool mine = true;
        if (same > 1) {  // the first of them writes, with the shares added in slot order
          share = 0.f;
          for (int l = 0; l < p.k; ++l)
            if (s_idx[l] == si[s]) {
              mine &= l >= j;
              share += s_e[l] / usum;
            }
        }
        if (mine) store_cd<CD>(dr, si[s], wt * (__builtin_amdgcn_exp2f((sz[s] - m) * p.c) * inv - share));
      }
    }
  }
  if (part != 0) return;
  if (tid == 0) {
    // The kl is exchanged, and the count raised once that has answered: both act where every
    // compute unit sees them, so who counts the last row sees every kl.  (A release would have
    // the XCD write back all of its L2, gradients included, for each row.)
    float old = __hip_atomic_exchange(&p.kl[i], live ? kl : 0.f, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("" : "+v"(old)::"memory");
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
    s_last = __hip_atomic_fetch_add(sp.done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)p.n - 1;
  }
  __syncthreads();
  if (!s_last || tid >= 64) return;
  double acc = 0.0;
  for (int64_t r = tid; r < p.n; r += 64) {
    const float wr = p.weight ? p.weight[r] : p.w_default;
    const float x = __hip_atomic_load(&p.kl[r], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    acc += wr == 0.f ? 0.0 : (double)wr * (double)x;
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) acc += __shfl_xor(acc, off, 64);
  if (tid == 0) sp.loss[0] = (float)acc;
}

// Rows that are cut into parts: a few long ones, more of them the longer they are (with the
// gradient; whole rows against rows in parts, us):
//            32000 bf16   64000 bf16   128000 bf16   250000 bf16   128000 f32   250000 f32
//   8 rows    9.5   8.9   13.3   9.3   21.7    9.3   39.2   10.7   27.0  10.7   45.7   11.7
//   32       10.2   9.8   14.2  10.6   22.5   12.5   40.7   16.7   29.4  16.1   54.9   24.3
//   64       10.3  11.1   14.8  12.8   24.9   17.5   41.7   25.6   33.0  24.7   64.3   39.3
//   96       10.6  12.4   16.5  14.8   27.0   23.8   49.6   34.8   42.3  33.1   86.3   55.0
//   160                                                            49.1  47.3    114   95.9
//   256                                33.4   48.4                 83.5  78.7    159    149
// The loss alone gains from about the same rows on.  The rule is coarser than the table: it leaves
// 32 rows of 32000 bf16, 64 and 96 of 64000, 96 of 128000, and of f32 160 of 128000 and 256 of 128000
// and 250000 whole, where parts are 4 to 14% faster.
constexpr int64_t kSplitRows = 256;
bool split_rows(int64_t n, int64_t V, int cd) {
  const int64_t bytes = V * cd_bytes(cd);
  return n <= kSplitRows && bytes >= std::max<int64_t>(49152, n * (n <= 64 ? 2048 : 4096));
}
int64_t parts_of(int64_t V, int cd) { return std::max<int64_t>(1, ceil_div(V * cd_bytes(cd) / 16, kPartChunks)); }

size_t al(size_t b) { return (b + 255) & ~(size_t)255; }

template <int CD>
int distill_split(const Distill& p, const Split& sp, hipStream_t s) {
  const dim3 g((unsigned)sp.parts, (unsigned)p.n), b(kPartThreads);
  k_distill_part<CD><<<g, b, 0, s>>>(p, sp);
  const int rc = check_launch("k_distill_part");
  if (rc) return rc;
  const dim3 gj(p.dz ? g.x : 1, g.y);  // the loss alone: what the first part's workgroup does
  if (p.k <= kPartThreads) k_distill_join<CD, kPartThreads><<<gj, b, 0, s>>>(p, sp);
  else k_distill_join<CD, kMaxK><<<gj, b, 0, s>>>(p, sp);
  return check_launch("k_distill_join");
}

// Workgroups of 1024 threads: as many as are resident at once, each going through its rows;
// smaller ones: one to a row, several to a compute unit (4096 x 32000 bf16: 111.8 us, going
// through rows 117.6; 4096 x 30000, loss alone: 50.6 against 56.5), as
// far as a launch of fewer than 2^32 threads has them.
template <int CD, int TPB, int NV, int KC>
void launch_rows(const Distill& p, int per_cu, hipStream_t s) {
  const int64_t most = TPB < 1024 ? (1LL << 31) / TPB : (int64_t)per_cu * cu_count();
  const int64_t g = std::min(p.n, most);
  k_distill<CD, TPB, NV, KC><<<dim3((unsigned)g), dim3(TPB), 0, s>>>(p);
}

// Threads and registers for a row of `chunks` 16-byte chunks.  With a gradient the row is kept
// where registers hold it: a wave for each of very many short rows (8192 x 2678 bf16: 31.0
// against 41.4 us; 1216 x 4000: 12.5 against 11.1), 256 threads (several rows to a compute
// unit), 512 (two: 2000 x 50000 bf16 87.6 us, 106.5 with one of 1024), then 1024; with no
// more rows than compute units 1024 from four chunks each on.  The loss alone reads a row
// once either way and does better with small workgroups that hold nothing (4096 x 128000 bf16:
// 187 against 278 us, 1024 x 32000: 20.7 against 27.6).
template <int CD>
int distill_rows(const Distill& p, hipStream_t s) {
  const int64_t chunks = p.V / Elem<CD>::PC;
  const bool few = p.n <= cu_count(), slots = p.k <= kFewSlots;
  if (chunks <= 64 * 8 && slots && p.n >= 8 * cu_count()) {
    launch_rows<CD, 64, 8, kFewSlots>(p, 1, s);
  } else if (chunks <= 256 * 4) {
    if (slots) launch_rows<CD, 256, 4, kFewSlots>(p, 1, s);
    else launch_rows<CD, 256, 4, kMaxK>(p, 1, s);
  } else if (!p.dz && few) {
    launch_rows<CD, 1024, 0, kMaxK>(p, 1, s);
  } else if (!p.dz) {
    if (slots) launch_rows<CD, 256, 0, kFewSlots>(p, 1, s);
    else launch_rows<CD, 256, 0, kMaxK>(p, 1, s);
  } else if (chunks <= 256 * 16 && !few) {
    if (slots && chunks <= 256 * 8) launch_rows<CD, 256, 8, kFewSlots>(p, 1, s);
    else if (slots) launch_rows<CD, 256, 16, kFewSlots>(p, 1, s);
    else launch_rows<CD, 256, 16, kMaxK>(p, 1, s);
  } else if (chunks <= 512 * 16 && !few) {
    if (slots) launch_rows<CD, 512, 16, kFewSlots>(p, 1, s);
    else launch_rows<CD, 512, 16, kMaxK>(p, 1, s);
  } else if (chunks <= 1024 * 4) launch_rows<CD, 1024, 4, kMaxK>(p, 1, s);
  else if (chunks <= 1024 * 8) launch_rows<CD, 1024, 8, kMaxK>(p, 1, s);
  else if (chunks <= 1024 * 16) launch_rows<CD, 1024, 16, kMaxK>(p, 1, s);
  else if (chunks <= 1024 * 20) launch_rows<CD, 1024, 20, kMaxK>(p, 1, s);
  else launch_rows<CD, 1024, 0, kMaxK>(p, 2, s);
  return check_launch("k_distill");
}

}  // namespace

size_t distill_workspace_bytes(int64_t n, int64_t V, int32_t k, int cd) {
  size_t b = al((size_t)std::max<int64_t>(n, 1) * 4);  // kl
  if (n > 0 && split_rows(n, V, cd))
    b += al((size_t)n * parts_of(V, cd) * sizeof(float2)) + al((size_t)n * k * 4) + al(4);
  return b;
}

int launch_distill(const void* z, int64_t n, int64_t V, int64_t ldz, int cd, const void* u, int ud, const void* idx,
                   int idx64, int32_t k, float temperature, const float* weight, float* loss, float* row_kl, void* dz,
                   int64_t lddz, void* ws, hipStream_t s) {
  char* base = (char*)ws;
  float* kl = row_kl ? row_kl : (float*)base;
  ProfScope prof(QLORA_K_LOSS, s);
  Distill p = {};
  p.z = z;
  p.ldz = ldz;
  p.dz = dz;
  p.lddz = lddz;
  p.u = u;
  p.idx = idx;
  p.weight = weight;
  p.kl = kl;
  p.n = n;
  p.V = V;
  p.k = k;
  p.ud = ud;
  p.idx64 = idx64;
  p.t = temperature;
  p.c = (float)(1.4426950408889634074 / (double)temperature);
  p.w_default = n > 0 ? (float)(1.0 / (double)n) : 0.f;
  if (n > 0 && split_rows(n, V, cd)) {
    Split sp;
    sp.parts = (int)parts_of(V, cd);
    char* at = base + al((size_t)n * 4);
    sp.part = (float2*)at;
    at += al((size_t)n * sp.parts * sizeof(float2));
    sp.zslot = (float*)at;
    at += al((size_t)n * k * 4);
    sp.done = (uint32_t*)at;
    sp.loss = loss;
    if (cd == CD_BF16) return distill_split<CD_BF16>(p, sp, s);
    if (cd == CD_F16) return distill_split<CD_F16>(p, sp, s);
    return distill_split<CD_F32>(p, sp, s);
  }
  if (n > 0) {
    int rc;
    if (cd == CD_BF16) rc = distill_rows<CD_BF16>(p, s);
    else if (cd == CD_F16) rc = distill_rows<CD_F16>(p, s);
    else rc = distill_rows<CD_F32>(p, s);
    if (rc) return rc;
  }
  k_distill_sum<<<dim3(1), dim3(kSumThreads), 0, s>>>(kl, weight, n, p.w_default, loss);
  return check_launch("k_distill_sum");
}

}  // namespace qnf4
