// ce.h -- what the two forms of the linear cross entropy share: ce.hip (tiles
// of many tokens) and ce_few.hip (few tokens).  Private header.
#pragma once

#include "common.h"
#include "device_util.h"

namespace csp {

constexpr float kLog2e = 1.44269504088896340736f;

__host__ __device__ inline int64_t round_up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// exp(x - b) from b log2 e: one operation less, and off by the rounding of b log2 e, which is that of b.
__device__ __forceinline__ float exp_less(float x, float b2) { return __builtin_amdgcn_exp2f(fmaf(x, kLog2e, -b2)); }

// {lse, loss} of a token from its target's logit and the maximum and sum of exp(z - maximum) of all others.
// The target stays out of the sum so that a small loss keeps its digits: with d = the others' log-sum less z,
// loss = max(d, 0) + log(1 + e^-|d|), off by d's rounding times itself, where lse - z is off by that of lse.
// In fp64: it is done once a token, and mx + log s alone would cost half a step of a number of ten and more.
__device__ __forceinline__ float2 loss_of(float mx, float s, float z)
{
    const double rest = (double)mx + log((double)s), d = rest - (double)z, l = log1p(exp(-fabs(d)));
    // (nothing besides the target: rest and d are -infinity, and loss is 0)
    return z == INFINITY ? make_float2(NAN, NAN) : make_float2((float)(fmax(rest, (double)z) + l), (float)(fmax(d, 0.0) + l));
}

// P at a token's target, p - 1, from p and the sum of its others.  p alone is off by half a step of lse, 10^-6
// beside logits of 20, and the gradient of a smaller loss, 1 - p, would be lost.  All of exp(z - lse) are off by
// the same factor, which the quotient takes out.
__device__ __forceinline__ float target_of(float p, float others) { return -others / (others + p); }

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)  // round to nearest even
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}
__device__ __forceinline__ float low_of(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float high_of(uint32_t p) { return __uint_as_float(p & 0xFFFF0000u); }

// Two floats as three pairs of bf16, x = x0 + x1 + x2: each the rest rounded to nearest.  Values past the
// largest bf16 leave the excess to the second plane.  An infinity ends as NaN (infinity less infinity).
__device__ __forceinline__ void split_pair(float a, float b, uint32_t (&p)[3])
{
    constexpr float kMax = 3.38953139e38f;
    p[0] = pack_bf16(__builtin_amdgcn_fmed3f(a, -kMax, kMax), __builtin_amdgcn_fmed3f(b, -kMax, kMax));
    a -= low_of(p[0]);
    b -= high_of(p[0]);
    p[1] = pack_bf16(a, b);
    p[2] = pack_bf16(a - low_of(p[1]), b - high_of(p[1]));
}

// Two floats as two pairs of bf16, 16 bits of each: the rest of the first rounding is rounded again.
__device__ __forceinline__ void split_pair(float a, float b, uint32_t (&p)[2])
{
    p[0] = pack_bf16(a, b);
    p[1] = pack_bf16(a - low_of(p[0]), b - high_of(p[0]));
}

// dmean / count, with the count that the forward divided by; 0 where no token takes part, whatever dmean is.
__device__ __forceinline__ float grad_scale(const float *dmean, const float *total)
{
    return total[1] > 0.0f ? dmean[0] / total[1] : 0.0f;
}

namespace {
// dX[n] = the sum of the splits' rows of its place in the list (acc[split][place][lda], lda a multiple of
// 4), scaled and rounded; zeros if it has none.  Without a list (slot), place n.  One thread for 4 columns.
template <typename E>
__global__ __launch_bounds__(256) void k_ce_out(const float *__restrict__ acc, int64_t lda, int64_t plane, int splits,
                                                const int32_t *__restrict__ slot, int64_t N, int64_t D,
                                                const float *__restrict__ dmean, const float *__restrict__ total,
                                                typename E::T *__restrict__ dX)
{
    typedef float f32x4 __attribute__((ext_vector_type(4)));
    constexpr int kAhead = 8;
    const int64_t groups = (D + 3) / 4, all = N * groups;
    const float scale = grad_scale(dmean, total);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int64_t n = i / groups, c = (i - n * groups) * 4;
        const int64_t m = slot ? slot[n] : n;
        f32x4 s{0.0f, 0.0f, 0.0f, 0.0f};
        if (m >= 0) {
            const float *p = acc + m * lda + c;
            int k = 0;
            for (; k + kAhead <= splits; k += kAhead) {
                f32x4 x[kAhead];
#pragma unroll
                for (int j = 0; j < kAhead; ++j) x[j] = *(const f32x4 *)(p + (k + j) * plane);
#pragma unroll
                for (int j = 0; j < kAhead; ++j) s += x[j];
            }
            for (; k < splits; ++k) s += *(const f32x4 *)(p + k * plane);
            s *= scale;
        }
        if (c + 4 <= D) {
            if constexpr (sizeof(typename E::T) == 4) {
                store16(dX + n * D + c, __builtin_bit_cast(u32x4, s));
            } else {
                struct __attribute__((packed, aligned(2))) Two {
                    uint32_t a, b;
                };
                *(Two *)(dX + n * D + c) = Two{pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3])};
            }
        } else {
            for (int k = 0; c + k < D; ++k) dX[n * D + c + k] = E::from_f(s[k]);
        }
    }
}
inline unsigned out_blocks(int64_t N, int64_t D)
{
    const int64_t b = (N * ((D + 3) / 4) + 255) / 256;
    return (unsigned)(b < 65536 ? b : 65536);
}
}  // namespace

// Up to how many tokens: 64 in bf16, 128 in fp32, where the other form copies W.
constexpr int64_t kFewMost = 128;
inline bool ce_is_few(int64_t N, int dtype) { return N <= (dtype == CSP_F32 ? 128 : 64); }

size_t ce_few_bytes(int64_t N, int64_t V, int64_t D, int dtype, bool backward);
csp_status ce_few_fwd(const void *X, const void *W, const int64_t *targets, int64_t N, int64_t V, int64_t D, int dtype,
                      float *loss, float *lse, float *total, char *work, hipStream_t s);
// dX or dW may be NULL: not asked for.
csp_status ce_few_bwd(const void *X, const void *W, const int64_t *targets, int64_t N, int64_t V, int64_t D, int dtype,
                      const float *lse, const float *dmean, const float *total, void *dX, void *dW, char *work,
                      hipStream_t s);

}  // namespace csp
