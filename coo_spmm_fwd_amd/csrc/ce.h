// ce.h -- what the two forms of the linear cross entropy share: ce.hip (tiles
// of many tokens) and ce_few.hip (up to kFewTokens tokens).  Private header.
#pragma once

#include "common.h"
#include "device_util.h"

namespace csp {

constexpr float kLog2e = 1.44269504088896340736f;

__host__ __device__ inline int64_t round_up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// dmean / count, with the count that the forward divided by.
__device__ __forceinline__ float grad_scale(const float *dmean, const float *total)
{
    return dmean[0] / fmaxf(total[1], 1.0f);
}

constexpr int64_t kFewTokens = 64;
size_t ce_few_bytes(int64_t N, int64_t V, int64_t D, int dtype, bool backward);
csp_status ce_few_fwd(const void *X, const void *W, const int64_t *targets, int64_t N, int64_t V, int64_t D, int dtype,
                      float *loss, float *lse, float *total, char *work, hipStream_t s);
csp_status ce_few_bwd(const void *X, const void *W, const int64_t *targets, int64_t N, int64_t V, int64_t D, int dtype,
                      const float *lse, const float *dmean, const float *total, void *dX, void *dW, char *work,
                      hipStream_t s);

}  // namespace csp
