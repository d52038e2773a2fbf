// ce.hip -- softmax cross entropy over a large vocabulary, fused with the
// product that makes the logits, and its gradient.
//
//   z[n, v] = sum_c X[n, c] W[v, c]
//   lse[n]  = log sum_v exp z[n, v] = m + log sum_v exp(z[n, v] - m)
//   loss[n] = lse[n] - z[n, t_n]
//   G[n, v] = (exp(z[n, v] - lse[n]) - [v = t_n]) * dmean / count
//   dX = G W,  dW = G^T X
//
// A token whose target is outside [0, V) takes no part: loss, lse and its row
// of dX are 0 and it adds nothing to dW, whatever its row of X holds.  The
// tokens that take part are listed first (k_ce_rows); every product runs over
// that list alone, so masked tokens cost nothing.  The logits are never
// stored: the forward keeps a maximum and a sum for each (vocabulary tile,
// token); the backward recomputes the logits, a piece of the vocabulary at a
// time, from the saved lse.
#include "common.h"
#include "device_util.h"

namespace csp {
namespace {

constexpr int kTile = 64;   // tokens and vocabulary rows (or columns) of a tile
constexpr int kStep = 16;   // depth of a staged slice
constexpr int kCeThreads = 256;

// Tokens that take part, in order: rows[0 .. count).  One workgroup.
__global__ __launch_bounds__(1024) void k_ce_rows(const int64_t *__restrict__ targets, int64_t N, int64_t V,
                                                  int32_t *__restrict__ rows, int32_t *__restrict__ count)
{
    __shared__ uint32_t lds[17];
    uint32_t run = 0;
    for (int64_t base = 0; base < N; base += 1024) {
        const int64_t i = base + threadIdx.x;
        const int64_t t = i < N ? targets[i] : -1;
        const bool part = t >= 0 && t < V;
        uint32_t total;
        const uint32_t at = block_exclusive_scan(part ? 1u : 0u, lds, &total);
        if (part) rows[run + at] = (int32_t)i;
        run += total;
    }
    if (threadIdx.x == 0) count[0] = (int32_t)run;
}

// acc[i][j] = sum over k of A(m, k) B(n, k), thread (ty, tx) of 16 x 16 holding rows m = 4 ty + i and
// columns n = 4 tx + j of a 64 x 64 tile.
template <typename FA, typename FB>
__device__ __forceinline__ void tile_product(FA A, FB B, int64_t K, float (&acc)[4][4])
{
    __shared__ float a[kStep][kTile + 4], b[kStep][kTile + 4];
    const int t = threadIdx.x, tx = t & 15, ty = t >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
    for (int64_t k0 = 0; k0 < K; k0 += kStep) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int e = j * kCeThreads + t, r = e >> 4, k = e & 15;
            a[k][r] = k0 + k < K ? A(r, k0 + k) : 0.0f;
            b[k][r] = k0 + k < K ? B(r, k0 + k) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kStep; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += a[k][4 * ty + i] * b[k][4 * tx + j];
    }
}

// z of a tile: tokens m0.. (of the list), vocabulary rows n0..
template <typename E>
__device__ __forceinline__ void logits_tile(const typename E::T *__restrict__ X, const typename E::T *__restrict__ W,
                                            const int32_t *__restrict__ rows, int64_t cnt, int64_t V, int64_t D,
                                            int64_t m0, int64_t n0, float (&acc)[4][4])
{
    tile_product([&](int r, int64_t k) { return m0 + r < cnt ? E::load(X, (int64_t)rows[m0 + r] * D + k) : 0.0f; },
                 [&](int r, int64_t k) { return n0 + r < V ? E::load(W, (n0 + r) * D + k) : 0.0f; }, D, acc);
}

// Per (vocabulary tile, listed token): maximum and sum of exp(z - maximum); the target's logit.
template <typename E>
__global__ __launch_bounds__(kCeThreads) void k_ce_stats(const typename E::T *__restrict__ X,
                                                         const typename E::T *__restrict__ W,
                                                         const int64_t *__restrict__ targets,
                                                         const int32_t *__restrict__ rows,
                                                         const int32_t *__restrict__ count, int64_t N, int64_t V,
                                                         int64_t D, float2 *__restrict__ part, float *__restrict__ zt)
{
    const int64_t cnt = count[0], m0 = (int64_t)blockIdx.y * kTile, n0 = (int64_t)blockIdx.x * kTile;
    if (m0 >= cnt) return;
    float z[4][4];
    logits_tile<E>(X, W, rows, cnt, V, D, m0, n0, z);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + 4 * ty + i;
        const int64_t t = m < cnt ? targets[rows[m]] : -1;
        float mx = -INFINITY, s = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t v = n0 + 4 * tx + j;
            if (v >= V) continue;
            if (v == t) zt[m] = z[i][j];
            mx = fmaxf(mx, z[i][j]);
        }
#pragma unroll
        for (int off = 8; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor(mx, off, 64));
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n0 + 4 * tx + j < V) s += expf(z[i][j] - mx);
#pragma unroll
        for (int off = 8; off >= 1; off >>= 1) s += __shfl_xor(s, off, 64);
        if (tx == 0 && m < cnt) part[(int64_t)blockIdx.x * N + m] = make_float2(mx, s);
    }
}

__global__ void k_ce_clear(int64_t N, float *__restrict__ loss, float *__restrict__ lse)
{
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i < N) loss[i] = lse[i] = 0.0f;
}

__global__ void k_ce_join(const float2 *__restrict__ part, const float *__restrict__ zt,
                          const int32_t *__restrict__ rows, const int32_t *__restrict__ count, int64_t N, int64_t tiles,
                          float *__restrict__ loss, float *__restrict__ lse)
{
    const int64_t m = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (m >= count[0]) return;
    float mx = -INFINITY, s = 0.0f;
    for (int64_t t = 0; t < tiles; ++t) mx = fmaxf(mx, part[t * N + m].x);
    for (int64_t t = 0; t < tiles; ++t) s += part[t * N + m].y * expf(part[t * N + m].x - mx);
    const float l = mx + logf(s);
    lse[rows[m]] = l;
    loss[rows[m]] = l - zt[m];
}

__global__ __launch_bounds__(1024) void k_ce_total(const float *__restrict__ loss, const int32_t *__restrict__ count,
                                                   int64_t N, float *__restrict__ total)
{
    __shared__ double lds[16];
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < N; i += 1024) s += loss[i];
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off, 64);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x != 0) return;
    double r = 0.0;
    for (int w = 0; w < 16; ++w) r += lds[w];
    const int32_t c = count[0];
    total[0] = (float)r;
    total[1] = (float)c;
    total[2] = (float)(r / (double)(c > 0 ? c : 1));
}

// P[m, v - v0] = exp(z - lse) - [v = t] of the listed tokens, vocabulary rows v0 .. v0 + nv.
template <typename E>
__global__ __launch_bounds__(kCeThreads) void k_ce_probs(const typename E::T *__restrict__ X,
                                                         const typename E::T *__restrict__ W,
                                                         const int64_t *__restrict__ targets,
                                                         const float *__restrict__ lse,
                                                         const int32_t *__restrict__ rows,
                                                         const int32_t *__restrict__ count, int64_t V, int64_t D,
                                                         int64_t v0, int64_t nv, float *__restrict__ P)
{
    const int64_t cnt = count[0], m0 = (int64_t)blockIdx.y * kTile, n0 = (int64_t)blockIdx.x * kTile;
    if (m0 >= cnt) return;
    float z[4][4];
    logits_tile<E>(X, W + v0 * D, rows, cnt, nv, D, m0, n0, z);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + 4 * ty + i;
        if (m >= cnt) continue;
        const int64_t t = targets[rows[m]] - v0;
        const float l = lse[rows[m]];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t v = n0 + 4 * tx + j;
            if (v < nv) P[m * nv + v] = expf(z[i][j] - l) - (v == t ? 1.0f : 0.0f);
        }
    }
}

// dmean / count, with the count that the forward divided by.
__device__ __forceinline__ float grad_scale(const float *dmean, const float *total)
{
    return dmean[0] / fmaxf(total[1], 1.0f);
}

// acc[m, c] += sum over the piece of P[m, v] W[v, c]; the first piece overwrites, the last one scales,
// rounds and puts the rows in their place.
template <typename E>
__global__ __launch_bounds__(kCeThreads) void k_ce_dx(const float *__restrict__ P, const typename E::T *__restrict__ W,
                                                      const int32_t *__restrict__ rows,
                                                      const int32_t *__restrict__ count, int64_t D, int64_t v0,
                                                      int64_t nv, float *__restrict__ acc, bool first, bool last,
                                                      const float *__restrict__ dmean, const float *__restrict__ total,
                                                      typename E::T *__restrict__ dX)
{
    const int64_t cnt = count[0], m0 = (int64_t)blockIdx.y * kTile, c0 = (int64_t)blockIdx.x * kTile;
    if (m0 >= cnt) return;
    float z[4][4];
    tile_product([&](int r, int64_t k) { return m0 + r < cnt ? P[(m0 + r) * nv + k] : 0.0f; },
                 [&](int r, int64_t k) { return c0 + r < D ? E::load(W, (v0 + k) * D + c0 + r) : 0.0f; }, nv, z);
    const float g = grad_scale(dmean, total);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + 4 * ty + i;
        if (m >= cnt) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t c = c0 + 4 * tx + j;
            if (c >= D) continue;
            const float v = z[i][j] + (first ? 0.0f : acc[m * D + c]);
            if (last) dX[(int64_t)rows[m] * D + c] = E::from_f(v * g);
            else acc[m * D + c] = v;
        }
    }
}

// The rows of dX of tokens that take no part.
template <typename E>
__global__ __launch_bounds__(kCeThreads) void k_ce_dx_clear(const int64_t *__restrict__ targets, int64_t V, int64_t D,
                                                            typename E::T *__restrict__ dX)
{
    const int64_t n = blockIdx.x, t = targets[n];
    if (t >= 0 && t < V) return;
    for (int64_t c = threadIdx.x; c < D; c += kCeThreads) dX[n * D + c] = E::from_f(0.0f);
}

template <typename E>
__global__ __launch_bounds__(kCeThreads) void k_ce_dw(const float *__restrict__ P, const typename E::T *__restrict__ X,
                                                      const int32_t *__restrict__ rows,
                                                      const int32_t *__restrict__ count, int64_t D, int64_t v0,
                                                      int64_t nv, const float *__restrict__ dmean,
                                                      const float *__restrict__ total,
                                                      typename E::T *__restrict__ dW)
{
    const int64_t cnt = count[0], n0 = (int64_t)blockIdx.y * kTile, c0 = (int64_t)blockIdx.x * kTile;
    float z[4][4];
    tile_product([&](int r, int64_t k) { return n0 + r < nv ? P[k * nv + n0 + r] : 0.0f; },
                 [&](int r, int64_t k) { return c0 + r < D ? E::load(X, (int64_t)rows[k] * D + c0 + r) : 0.0f; }, cnt, z);
    const float g = grad_scale(dmean, total);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t v = n0 + 4 * ty + i;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t c = c0 + 4 * tx + j;
            if (v < nv && c < D) dW[(v0 + v) * D + c] = E::from_f(z[i][j] * g);
        }
    }
}

// Bytes of one piece's gradient at the logits.
constexpr int64_t kPieceBytes = (int64_t)256 << 20;

struct CePlan {
    int64_t tiles, piece;
    size_t rows, count, part, zt, P, acc, total;
};

CePlan ce_plan(int64_t N, int64_t V, int64_t D, bool backward)
{
    CePlan p{};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t r = at;
        at += (bytes + 255) / 256 * 256;
        return r;
    };
    p.tiles = ceil_div(V, kTile);
    p.count = take(4);
    p.rows = take(4 * (size_t)N);
    if (!backward) {
        p.part = take(8 * (size_t)N * (size_t)p.tiles);
        p.zt = take(4 * (size_t)N);
    } else {
        p.piece = N > 0 ? kPieceBytes / (4 * N) / kTile * kTile : V;
        if (p.piece < kTile) p.piece = kTile;
        if (p.piece > V) p.piece = V;
        p.P = take(4 * (size_t)N * (size_t)p.piece);
        p.acc = take(4 * (size_t)N * (size_t)D);
    }
    p.total = at;
    return p;
}

csp_status ce_args(int64_t N, int64_t V, int64_t D, int dtype)
{
    constexpr int64_t kLimit = 0x7FFFFFFF;
    if (N < 0 || N >= kLimit || V < 1 || V >= kLimit || D < 1 || D >= kLimit)
        return set_error(CSP_ERR_INVALID_ARG, "bad shape: %lld tokens, vocabulary %lld, width %lld", (long long)N,
                         (long long)V, (long long)D);
    if (dtype != CSP_F32 && dtype != CSP_BF16) return set_error(CSP_ERR_DTYPE, "unsupported dtype %d", dtype);
    return CSP_OK;
}

bool aligned(const void *p, size_t a) { return p && (uintptr_t)p % a == 0; }

template <typename E>
csp_status fwd_impl(const void *X, const void *W, const int64_t *targets, int64_t N, int64_t V, int64_t D, float *loss,
                    float *lse, float *total, char *w, hipStream_t s)
{
    using T = typename E::T;
    const CePlan p = ce_plan(N, V, D, false);
    int32_t *rows = (int32_t *)(w + p.rows), *count = (int32_t *)(w + p.count);
    float2 *part = (float2 *)(w + p.part);
    float *zt = (float *)(w + p.zt);
    k_ce_rows<<<1, 1024, 0, s>>>(targets, N, V, rows, count);
    CSP_LAUNCHED("k_ce_rows");
    if (N > 0) {
        k_ce_stats<E><<<dim3((unsigned)p.tiles, (unsigned)ceil_div(N, kTile)), kCeThreads, 0, s>>>(
            (const T *)X, (const T *)W, targets, rows, count, N, V, D, part, zt);
        CSP_LAUNCHED("k_ce_stats");
        k_ce_clear<<<(unsigned)ceil_div(N, 256), 256, 0, s>>>(N, loss, lse);
        CSP_LAUNCHED("k_ce_clear");
        k_ce_join<<<(unsigned)ceil_div(N, 64), 64, 0, s>>>(part, zt, rows, count, N, p.tiles, loss, lse);
        CSP_LAUNCHED("k_ce_join");
    }
    k_ce_total<<<1, 1024, 0, s>>>(loss, count, N, total);
    CSP_LAUNCHED("k_ce_total");
    return CSP_OK;
}

template <typename E>
csp_status bwd_impl(const void *X, const void *W, const int64_t *targets, int64_t N, int64_t V, int64_t D,
                    const float *lse, const float *dmean, const float *total, void *dX, void *dW, char *w,
                    hipStream_t s)
{
    using T = typename E::T;
    const CePlan p = ce_plan(N, V, D, true);
    int32_t *rows = (int32_t *)(w + p.rows), *count = (int32_t *)(w + p.count);
    float *P = (float *)(w + p.P), *acc = (float *)(w + p.acc);
    k_ce_rows<<<1, 1024, 0, s>>>(targets, N, V, rows, count);
    CSP_LAUNCHED("k_ce_rows");
    const unsigned mt = (unsigned)ceil_div(N, kTile), ct = (unsigned)ceil_div(D, kTile);
    if (N > 0) {
        k_ce_dx_clear<E><<<(unsigned)N, kCeThreads, 0, s>>>(targets, V, D, (T *)dX);
        CSP_LAUNCHED("k_ce_dx_clear");
    }
    for (int64_t v0 = 0; v0 < V; v0 += p.piece) {
        const int64_t nv = V - v0 < p.piece ? V - v0 : p.piece;
        const unsigned vt = (unsigned)ceil_div(nv, kTile);
        if (N > 0) {
            k_ce_probs<E><<<dim3(vt, mt), kCeThreads, 0, s>>>((const T *)X, (const T *)W, targets, lse, rows, count, V,
                                                              D, v0, nv, P);
            CSP_LAUNCHED("k_ce_probs");
            k_ce_dx<E><<<dim3(ct, mt), kCeThreads, 0, s>>>(P, (const T *)W, rows, count, D, v0, nv, acc, v0 == 0,
                                                           v0 + nv == V, dmean, total, (T *)dX);
            CSP_LAUNCHED("k_ce_dx");
        }
        k_ce_dw<E><<<dim3(ct, vt), kCeThreads, 0, s>>>(P, (const T *)X, rows, count, D, v0, nv, dmean, total,
                                                            (T *)dW);
        CSP_LAUNCHED("k_ce_dw");
    }
    return CSP_OK;
}

}  // namespace
}  // namespace csp

extern "C" {

int64_t linear_ce_workspace(int64_t N, int64_t V, int64_t D, csp_dtype dtype, int32_t backward)
{
    if (csp::ce_args(N, V, D, dtype) != CSP_OK) return -1;
    return (int64_t)csp::ce_plan(N, V, D, backward != 0).total;
}

csp_status linear_ce_fwd(const void *X, const void *W, const int64_t *targets, int64_t N, int64_t V, int64_t D,
                         csp_dtype dtype, float *loss, float *lse, float *total, void *workspace,
                         int64_t workspace_bytes, void *stream)
{
    using namespace csp;
    csp_status st = ce_args(N, V, D, dtype);
    if (st != CSP_OK) return st;
    const size_t e = dtype == CSP_BF16 ? 2 : 4;
    if (!aligned(W, e) || !aligned(total, 4) ||
        (N > 0 && (!aligned(X, e) || !aligned(targets, 8) || !aligned(loss, 4) || !aligned(lse, 4))))
        return set_error(CSP_ERR_INVALID_ARG, "NULL or misaligned pointer");
    const size_t need = ce_plan(N, V, D, false).total;
    if (!aligned(workspace, 16) || workspace_bytes < (int64_t)need)
        return set_error(CSP_ERR_INVALID_ARG, "workspace of %lld bytes, %zu needed", (long long)workspace_bytes, need);
    if (dtype == CSP_BF16)
        return fwd_impl<BF16>(X, W, targets, N, V, D, loss, lse, total, (char *)workspace, (hipStream_t)stream);
    return fwd_impl<F32>(X, W, targets, N, V, D, loss, lse, total, (char *)workspace, (hipStream_t)stream);
}

csp_status linear_ce_bwd(const void *X, const void *W, const int64_t *targets, int64_t N, int64_t V, int64_t D,
                         csp_dtype dtype, const float *lse, const float *dmean, const float *total, void *dX, void *dW,
                         void *workspace, int64_t workspace_bytes, void *stream)
{
    using namespace csp;
    csp_status st = ce_args(N, V, D, dtype);
    if (st != CSP_OK) return st;
    const size_t e = dtype == CSP_BF16 ? 2 : 4;
    if (!aligned(W, e) || !aligned(dW, e) || !aligned(dmean, 4) || !aligned(total, 4) ||
        (N > 0 && (!aligned(X, e) || !aligned(targets, 8) || !aligned(lse, 4) || !aligned(dX, e))))
        return set_error(CSP_ERR_INVALID_ARG, "NULL or misaligned pointer");
    const size_t need = ce_plan(N, V, D, true).total;
    if (!aligned(workspace, 16) || workspace_bytes < (int64_t)need)
        return set_error(CSP_ERR_INVALID_ARG, "workspace of %lld bytes, %zu needed", (long long)workspace_bytes, need);
    if (dtype == CSP_BF16)
        return bwd_impl<BF16>(X, W, targets, N, V, D, lse, dmean, total, dX, dW, (char *)workspace, (hipStream_t)stream);
    return bwd_impl<F32>(X, W, targets, N, V, D, lse, dmean, total, dX, dW, (char *)workspace, (hipStream_t)stream);
}

}  // extern "C"
