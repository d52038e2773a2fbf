// embed.hip -- embedding lookup with scaling, and its gradient by sorted tokens.
//
//   forward   Y[n, :]  = scale * E[ids[n], :]
//   backward  dE[v, :] = scale * sum over n with ids[n] = v of dY[n, :]
//
// An id outside [0, V) takes no part: a zero row of Y, no term in dE.  Both
// are bound by memory.  The gradient adds the rows of one id in token order
// in fp32 and rounds once, without floating-point atomics.
#include "common.h"
#include "device_util.h"

namespace csp {
namespace {

constexpr int kEmbedThreads = 256;

template <typename E>
__global__ __launch_bounds__(kEmbedThreads) void k_embed_fwd(const typename E::T *__restrict__ table, int64_t V,
                                                             int64_t D, const int64_t *__restrict__ ids, float scale,
                                                             typename E::T *__restrict__ Y)
{
    const int64_t n = blockIdx.x;
    const int64_t id = ids[n];
    const bool part = id >= 0 && id < V;
    for (int64_t c = threadIdx.x; c < D; c += kEmbedThreads)
        Y[n * D + c] = part ? E::from_f(E::load(table, id * D + c) * scale) : E::from_f(0.0f);
}

__global__ void k_embed_keys(const int64_t *__restrict__ ids, int64_t N, int64_t V, uint32_t *__restrict__ key,
                             int32_t *__restrict__ pos)
{
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= N) return;
    const int64_t id = ids[i];
    key[i] = id >= 0 && id < V ? (uint32_t)id : (uint32_t)V;
    pos[i] = (int32_t)i;
}

template <typename E>
__global__ __launch_bounds__(kEmbedThreads) void k_embed_bwd(const typename E::T *__restrict__ dY, int64_t D,
                                                             const int32_t *__restrict__ order,
                                                             const int32_t *__restrict__ ptr, float scale,
                                                             typename E::T *__restrict__ dE)
{
    const int64_t v = blockIdx.x;
    const int32_t a = ptr[v], b = ptr[v + 1];
    for (int64_t c = threadIdx.x; c < D; c += kEmbedThreads) {
        float s = 0.0f;
        for (int32_t k = a; k < b; ++k) s += E::load(dY, (int64_t)order[k] * D + c);
        dE[v * D + c] = E::from_f(s * scale);
    }
}

struct EmbedPlan {
    size_t key[3], pos[3], ptr, hist, total;
};

EmbedPlan embed_plan(int64_t N, int64_t V)
{
    EmbedPlan p;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t r = at;
        at += (bytes + 255) / 256 * 256;
        return r;
    };
    for (int i = 0; i < 3; ++i) p.key[i] = take(4 * (size_t)N), p.pos[i] = take(4 * (size_t)N);
    p.ptr = take(4 * (size_t)(V + 1));
    p.hist = take(4 * sort_hist_words(N));
    p.total = at;
    return p;
}

csp_status embed_args(int64_t N, int64_t V, int64_t D, int dtype)
{
    constexpr int64_t kLimit = 0x7FFFFFFF;
    if (N < 0 || N >= kLimit || V < 1 || V >= kLimit || D < 1 || D >= kLimit)
        return set_error(CSP_ERR_INVALID_ARG, "bad shape: %lld tokens, table %lld x %lld", (long long)N, (long long)V, (long long)D);
    if (dtype != CSP_F32 && dtype != CSP_BF16) return set_error(CSP_ERR_DTYPE, "unsupported dtype %d", dtype);
    return CSP_OK;
}

bool aligned(const void *p, int dtype) { return p && (uintptr_t)p % (dtype == CSP_BF16 ? 2 : 4) == 0; }

template <typename E>
csp_status bwd_impl(const void *dY, const int64_t *ids, int64_t N, int64_t V, int64_t D, float scale, void *dE,
                    char *w, hipStream_t s)
{
    const EmbedPlan p = embed_plan(N, V);
    uint32_t *key = (uint32_t *)(w + p.key[0]);
    int32_t *pos = (int32_t *)(w + p.pos[0]), *ptr = (int32_t *)(w + p.ptr), *order = (int32_t *)(w + p.pos[2]);
    if (N > 0) {
        k_embed_keys<<<(unsigned)ceil_div(N, 256), 256, 0, s>>>(ids, N, V, key, pos);
        CSP_LAUNCHED("k_embed_keys");
    }
    csp_status st = radix_sort_pairs(4, key, pos, w + p.key[2], order, w + p.key[1], (int32_t *)(w + p.pos[1]), N,
                                     bits_for((uint64_t)V), (uint32_t *)(w + p.hist), s);
    if (st != CSP_OK) return st;
    st = segment_offsets((const int32_t *)(w + p.key[2]), N, ptr, V, s);
    if (st != CSP_OK) return st;
    k_embed_bwd<E><<<(unsigned)V, kEmbedThreads, 0, s>>>((const typename E::T *)dY, D, order, ptr, scale,
                                                         (typename E::T *)dE);
    CSP_LAUNCHED("k_embed_bwd");
    return CSP_OK;
}

}  // namespace
}  // namespace csp

extern "C" {

csp_status embed_fwd(const void *E, const int64_t *ids, int64_t N, int64_t V, int64_t D, csp_dtype dtype, float scale,
                     void *Y, void *stream)
{
    using namespace csp;
    csp_status st = embed_args(N, V, D, dtype);
    if (st != CSP_OK) return st;
    if (N == 0) return CSP_OK;
    if (!aligned(E, dtype) || !aligned(Y, dtype) || !ids || (uintptr_t)ids % 8)
        return set_error(CSP_ERR_INVALID_ARG, "NULL or misaligned pointer");
    hipStream_t s = (hipStream_t)stream;
    if (dtype == CSP_BF16)
        k_embed_fwd<BF16><<<(unsigned)N, kEmbedThreads, 0, s>>>((const uint16_t *)E, V, D, ids, scale, (uint16_t *)Y);
    else
        k_embed_fwd<F32><<<(unsigned)N, kEmbedThreads, 0, s>>>((const float *)E, V, D, ids, scale, (float *)Y);
    CSP_LAUNCHED("k_embed_fwd");
    return CSP_OK;
}

int64_t embed_bwd_workspace(int64_t N, int64_t V, int64_t D, csp_dtype dtype)
{
    if (csp::embed_args(N, V, D, dtype) != CSP_OK) return -1;
    return (int64_t)csp::embed_plan(N, V).total;
}

csp_status embed_bwd(const void *dY, const int64_t *ids, int64_t N, int64_t V, int64_t D, csp_dtype dtype, float scale,
                     void *dE, void *workspace, int64_t workspace_bytes, void *stream)
{
    using namespace csp;
    csp_status st = embed_args(N, V, D, dtype);
    if (st != CSP_OK) return st;
    if (!aligned(dE, dtype) || (N > 0 && (!aligned(dY, dtype) || !ids || (uintptr_t)ids % 8)))
        return set_error(CSP_ERR_INVALID_ARG, "NULL or misaligned pointer");
    const size_t need = embed_plan(N, V).total;
    if (!workspace || (uintptr_t)workspace % 16 || workspace_bytes < (int64_t)need)
        return set_error(CSP_ERR_INVALID_ARG, "workspace of %lld bytes, %zu needed", (long long)workspace_bytes, need);
    if (dtype == CSP_BF16) return bwd_impl<BF16>(dY, ids, N, V, D, scale, dE, (char *)workspace, (hipStream_t)stream);
    return bwd_impl<F32>(dY, ids, N, V, D, scale, dE, (char *)workspace, (hipStream_t)stream);
}

}  // extern "C"
