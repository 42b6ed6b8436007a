// int8_distill.h -- host entry points of the 8-bit products (int8.hip) and of the
// distillation loss (distill.hip).
#pragma once
#include "common.h"

namespace qnf4 {
int launch_int8_quantize(const void* w, int64_t ldw, int dtype, const qlora_int8_t* q, hipStream_t s);
size_t int8_workspace_bytes(const qlora_int8_t* w, int64_t m, bool grouped);
int launch_int8_linear(const qlora_int8_t* w, const void* x, int64_t m, int64_t ldx, const int32_t* offsets,
                       const void* bias, int cd, void* y, void* ws, hipStream_t s);
int launch_distill(const void* z, int64_t n, int64_t V, int64_t ldz, int cd, const void* u, int ud, const void* idx,
                   int idx64, int32_t k, float temperature, const float* weight, float* loss, float* row_kl, void* dz,
                   int64_t lddz, void* ws, hipStream_t s);
size_t distill_workspace_bytes(int64_t n, int64_t V, int32_t k, int cd);
}  // namespace qnf4
