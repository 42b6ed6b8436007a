// distill.hip -- distillation loss against a teacher's top logits, with its gradient.
//
// Row i of student logits z [V], the teacher's k highest logits u at vocabulary indices
// idx, temperature T, weight w:
//   p = softmax(u / T) over the present slots,  q = softmax(z / T) over the vocabulary,
//   kl = T^2 sum_j p_j (log p_j - log q[idx_j]),  loss = sum_i w_i kl_i,
//   dz = w T (q - p scattered to idx).
// A slot is absent when its index lies outside [0, V) or its value is -inf.  A row with
// weight 0 or without a present slot has kl 0 and a zero gradient, whatever its logits
// hold; they are not read.
#include <math.h>

#include <algorithm>

#include "common.h"

namespace qnf4 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxK = QLORA_DISTILL_MAX_K;

struct Distill {
  const void* z;       // [n][ldz] cd
  int64_t ldz;
  void* dz;            // [n][lddz] cd or null
  int64_t lddz;
  const void* u;       // [n][k] teacher values (ud)
  int ud;
  const void* idx;     // [n][k] int32 or int64
  int idx64;
  const float* weight; // [n] or null: 1 / n
  float* kl;           // [n]
  int64_t n, V;
  int k;
  float inv_t, t, w_default;
};

__device__ __forceinline__ float load_any(const void* p, int64_t i, int cd) {
  return cd == CD_F32 ? load_cd<CD_F32>(p, i) : cd == CD_BF16 ? load_cd<CD_BF16>(p, i) : load_cd<CD_F16>(p, i);
}

template <bool MAX>
__device__ __forceinline__ float block_reduce(float v, float* red) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const float o = __shfl_xor(v, off, 64);
    v = MAX ? fmaxf(v, o) : v + o;
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = red[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) s = MAX ? fmaxf(s, red[w]) : s + red[w];
  return s;
}

template <int CD>
__global__ __launch_bounds__(kThreads) void k_distill(Distill p) {
  __shared__ float red[kThreads / 64];
  __shared__ int32_t si[kMaxK];   // index of a present slot, -1 of an absent one
  __shared__ float sp[kMaxK];     // (u - max) / T, then p
  const int64_t i = blockIdx.x;
  const int tid = threadIdx.x;
  const float w = p.weight ? p.weight[i] : p.w_default;
  float umax = -INFINITY;
  int any = 0;
  for (int j = tid; j < p.k; j += kThreads) {
    const int64_t ix = p.idx64 ? ((const int64_t*)p.idx)[i * p.k + j] : (int64_t)((const int32_t*)p.idx)[i * p.k + j];
    const float u = load_any(p.u, i * p.k + j, p.ud);
    const bool here = ix >= 0 && ix < p.V && !(u == -INFINITY);
    si[j] = here ? (int32_t)ix : -1;
    sp[j] = u;
    if (here) umax = fmaxf(umax, u);
    any |= here;
  }
  any = __syncthreads_or(any);
  if (w == 0.f || !any) {
    if (tid == 0) p.kl[i] = 0.f;
    if (p.dz)
      for (int64_t j = tid; j < p.V; j += kThreads) store_cd<CD>(p.dz, i * p.lddz + j, 0.f);
    return;
  }
  umax = block_reduce<true>(umax, red);
  float usum = 0.f;
  for (int j = tid; j < p.k; j += kThreads)
    if (si[j] >= 0) {
      const float v = expf((sp[j] - umax) * p.inv_t);
      usum += v;
    }
  usum = block_reduce<false>(usum, red);
  float m = -INFINITY;
  for (int64_t j = tid; j < p.V; j += kThreads) m = fmaxf(m, load_cd<CD>(p.z, i * p.ldz + j));
  m = block_reduce<true>(m, red);
  float sum = 0.f;
  for (int64_t j = tid; j < p.V; j += kThreads) sum += expf((load_cd<CD>(p.z, i * p.ldz + j) - m) * p.inv_t);
  sum = block_reduce<false>(sum, red);
  const float lsum = logf(sum), lu = logf(usum);
  float kl = 0.f;
  for (int j = tid; j < p.k; j += kThreads)
    if (si[j] >= 0) {
      const float a = sp[j] - umax, b = load_cd<CD>(p.z, i * p.ldz + si[j]) - m;
      const float pr = expf(a * p.inv_t) / usum;
      if (pr != 0.f) kl += pr * ((a - b) * p.inv_t + (lsum - lu));
    }
  kl = block_reduce<false>(kl, red);
  if (tid == 0) p.kl[i] = p.t * p.t * kl;
  if (!p.dz) return;
  const float wt = w * p.t;
  // the slots' gradients are formed before the row is overwritten (dz may be z)
  float g[kMaxK / kThreads];
#pragma unroll
  for (int s = 0; s < kMaxK / kThreads; ++s) {
    const int j = tid + s * kThreads;
    g[s] = 0.f;
    if (j < p.k && si[j] >= 0) {
      float pr = 0.f;  // an index may appear more than once
      for (int l = 0; l < p.k; ++l)
        if (si[l] == si[j]) pr += expf((sp[l] - umax) * p.inv_t) / usum;
      g[s] = wt * (expf((load_cd<CD>(p.z, i * p.ldz + si[j]) - m) * p.inv_t) / sum - pr);
    }
  }
  __syncthreads();
  for (int64_t j = tid; j < p.V; j += kThreads)
    store_cd<CD>(p.dz, i * p.lddz + j, wt * (expf((load_cd<CD>(p.z, i * p.ldz + j) - m) * p.inv_t) / sum));
  __threadfence_block();
  __syncthreads();
#pragma unroll
  for (int s = 0; s < kMaxK / kThreads; ++s) {
    const int j = tid + s * kThreads;
    if (j < p.k && si[j] >= 0) store_cd<CD>(p.dz, i * p.lddz + si[j], g[s]);
  }
}

// loss = sum of w_i kl_i in a fixed order, in 64 bits, rounded once.
__global__ __launch_bounds__(kThreads) void k_distill_sum(const float* __restrict__ kl, const float* __restrict__ weight,
                                                          int64_t n, float w_default, float* __restrict__ loss) {
  __shared__ double red[kThreads / 64];
  double acc = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kThreads) {
    const float w = weight ? weight[i] : w_default;
    acc += w == 0.f ? 0.0 : (double)w * (double)kl[i];
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) acc += __shfl_xor(acc, off, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = acc;
  __syncthreads();
  if (threadIdx.x == 0) loss[0] = (float)((red[0] + red[1]) + (red[2] + red[3]));
}

}  // namespace

int launch_distill(const void* z, int64_t n, int64_t V, int64_t ldz, int cd, const void* u, int ud, const void* idx,
                   int idx64, int32_t k, float temperature, const float* weight, float* loss, float* kl, void* dz,
                   int64_t lddz, hipStream_t s) {
  ProfScope prof(QLORA_K_LOSS, s);
  Distill p = {};
  p.z = z;
  p.ldz = ldz;
  p.dz = dz;
  p.lddz = lddz;
  p.u = u;
  p.ud = ud;
  p.idx = idx;
  p.idx64 = idx64;
  p.weight = weight;
  p.kl = kl;
  p.n = n;
  p.V = V;
  p.k = k;
  p.t = temperature;
  p.inv_t = 1.0f / temperature;
  p.w_default = n > 0 ? (float)(1.0 / (double)n) : 0.f;
  int rc;
  if (n > 0) {
    const dim3 g((unsigned)n), b(kThreads);
    if (cd == CD_BF16) k_distill<CD_BF16><<<g, b, 0, s>>>(p);
    else if (cd == CD_F16) k_distill<CD_F16><<<g, b, 0, s>>>(p);
    else k_distill<CD_F32><<<g, b, 0, s>>>(p);
    if ((rc = check_launch("k_distill"))) return rc;
  }
  k_distill_sum<<<dim3(1), dim3(kThreads), 0, s>>>(kl, weight, n, p.w_default, loss);
  return check_launch("k_distill_sum");
}

}  // namespace qnf4
