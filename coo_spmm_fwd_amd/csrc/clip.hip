// clip.hip -- the global gradient norm over many tensors, and clipping by it.
//
//   norm = sqrt(sum over all tensors and elements of g^2)
//   out  = g * min(1, max_norm / (norm + 1e-6))
//
// Both passes are bound by memory: the norm reads every element once, the
// clipping reads it again and writes it.  All tensors together are one list of
// 16 KiB chunks; a workgroup takes a contiguous run of chunks, so it looks its
// first tensor up once and then walks.  Squares are summed in fp64 (exact for
// fp32 and bf16 squares up to rounding of the sum; no overflow below 1e154):
// at one fp64 multiply-add per element the vector units are idle most of the
// time of the read.  Sums are joined in a fixed order, so results do not
// depend on scheduling.
#include "common.h"
#include "device_util.h"

namespace csp {
namespace {

constexpr int kClipThreads = 256;
constexpr int kVecPerThread = 4;                                   // 16-byte loads in flight per thread
constexpr int64_t kChunkBytes = kClipThreads * kVecPerThread * 16;  // 16 KiB
constexpr int64_t kClipBlocks = 2048;                               // 8 workgroups a CU
constexpr int kInline = 64;                                         // table entries that fit the kernel arguments

struct Entry {
    const void *g;
    void *o;
    int64_t n;
    int64_t first;  // the tensor's first chunk << 1 | 1 for bf16
};
struct InlineTable {
    Entry e[kInline];
};

__global__ void k_table_put(InlineTable t, int n, Entry *__restrict__ dst)
{
    if ((int)threadIdx.x < n) dst[threadIdx.x] = t.e[threadIdx.x];
}

// Last tensor whose first chunk is at most c (tensors of no chunk are skipped by taking the last).
__device__ __forceinline__ int find_tensor(const Entry *__restrict__ e, int count, int64_t c)
{
    int lo = 0, hi = count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((e[mid].first >> 1) <= c) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ void bf16_pair(uint32_t w, float &a, float &b)
{
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xFFFF0000u);
}

// Block sum of one double per thread, in a fixed order; every thread gets it.
__device__ __forceinline__ double block_sum(double v, double *lds)
{
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.0;
    for (int w = 0; w < (int)(blockDim.x >> 6); ++w) s += lds[w];
    return s;
}

__device__ __forceinline__ double square_chunk(const Entry &t, int64_t chunk)
{
    const bool bf = t.first & 1;
    const int per = bf ? 8 : 4;  // elements a 16-byte load
    const int64_t base = chunk * (kChunkBytes / 16) * per;
    double acc = 0.0;
    u32x4 v[kVecPerThread];
    const char *g = (const char *)t.g;
#pragma unroll
    for (int j = 0; j < kVecPerThread; ++j) {
        const int64_t i = base + (int64_t)(j * kClipThreads + threadIdx.x) * per;
        v[j] = u32x4{0u, 0u, 0u, 0u};
        if (i + per <= t.n) v[j] = load16(g + (bf ? 2 : 4) * i);
        else if (i < t.n) {  // the tensor's end: element by element
            for (int64_t k = i; k < t.n; ++k) {
                const double x = bf ? (double)BF16::load((const uint16_t *)g, k) : (double)((const float *)g)[k];
                acc += x * x;
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kVecPerThread; ++j) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (bf) {
                float a, b;
                bf16_pair(v[j][q], a, b);
                acc += (double)a * (double)a;
                acc += (double)b * (double)b;
            } else {
                const double x = (double)__uint_as_float(v[j][q]);
                acc += x * x;
            }
        }
    }
    return acc;
}

template <bool kInTable>
__global__ __launch_bounds__(kClipThreads) void k_square_sums(InlineTable it, const Entry *__restrict__ table,
                                                              int count, int64_t chunks,
                                                              double *__restrict__ partial)
{
    __shared__ double lds[kClipThreads / 64];
    const Entry *e = kInTable ? table : it.e;
    const int64_t c0 = chunks * blockIdx.x / gridDim.x, c1 = chunks * (blockIdx.x + 1) / gridDim.x;
    double acc = 0.0;
    int t = find_tensor(e, count, c0);
    for (int64_t c = c0; c < c1; ++c) {
        while (t + 1 < count && (e[t + 1].first >> 1) <= c) ++t;
        acc += square_chunk(e[t], c - (e[t].first >> 1));
    }
    const double s = block_sum(acc, lds);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__device__ __forceinline__ float norm_of(const double *__restrict__ partial, int n, double *lds)
{
    double a = 0.0;
    for (int i = threadIdx.x; i < n; i += blockDim.x) a += partial[i];
    return (float)sqrt(block_sum(a, lds));
}

__global__ __launch_bounds__(kClipThreads) void k_norm(const double *__restrict__ partial, int n,
                                                       float *__restrict__ norm)
{
    __shared__ double lds[kClipThreads / 64];
    const float r = norm_of(partial, n, lds);
    if (threadIdx.x == 0) norm[0] = r;
}

__device__ __forceinline__ void scale_chunk(const Entry &t, int64_t chunk, float c)
{
    const bool bf = t.first & 1;
    const int per = bf ? 8 : 4;
    const int64_t base = chunk * (kChunkBytes / 16) * per;
    const char *g = (const char *)t.g;
    char *o = (char *)t.o;
    u32x4 v[kVecPerThread];
#pragma unroll
    for (int j = 0; j < kVecPerThread; ++j) {
        const int64_t i = base + (int64_t)(j * kClipThreads + threadIdx.x) * per;
        v[j] = u32x4{0u, 0u, 0u, 0u};
        if (i + per <= t.n) v[j] = load16(g + (bf ? 2 : 4) * i);
    }
#pragma unroll
    for (int j = 0; j < kVecPerThread; ++j) {
        const int64_t i = base + (int64_t)(j * kClipThreads + threadIdx.x) * per;
        if (i + per <= t.n) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (bf) {
                    float a, b;
                    bf16_pair(v[j][q], a, b);
                    v[j][q] = (uint32_t)BF16::from_f(a * c) | (uint32_t)BF16::from_f(b * c) << 16;
                } else {
                    v[j][q] = __float_as_uint(__uint_as_float(v[j][q]) * c);
                }
            }
            store16(o + (bf ? 2 : 4) * i, v[j]);
        } else if (i < t.n) {
            for (int64_t k = i; k < t.n; ++k) {
                if (bf) ((uint16_t *)o)[k] = BF16::from_f(BF16::load((const uint16_t *)g, k) * c);
                else ((float *)o)[k] = ((const float *)g)[k] * c;
            }
        }
    }
}

template <bool kInTable>
__global__ __launch_bounds__(kClipThreads) void k_clip_scale(InlineTable it, const Entry *__restrict__ table,
                                                             int count, int64_t chunks,
                                                             const double *__restrict__ partial, int npartial,
                                                             float max_norm, float *__restrict__ norm)
{
    __shared__ double lds[kClipThreads / 64];
    const Entry *e = kInTable ? table : it.e;
    const float r = norm_of(partial, npartial, lds);
    if (blockIdx.x == 0 && threadIdx.x == 0) norm[0] = r;
    const float q = max_norm / (r + 1e-6f);
    const float c = q > 1.0f ? 1.0f : q;  // a NaN norm stays NaN
    const int64_t c0 = chunks * blockIdx.x / gridDim.x, c1 = chunks * (blockIdx.x + 1) / gridDim.x;
    int t = find_tensor(e, count, c0);
    for (int64_t k = c0; k < c1; ++k) {
        while (t + 1 < count && (e[t + 1].first >> 1) <= k) ++t;
        if (c == 1.0f && e[t].o == e[t].g) continue;  // in place and nothing to change
        scale_chunk(e[t], k - (e[t].first >> 1), c);
    }
}

struct ClipPlan {
    size_t partial_off, total;
};
ClipPlan clip_plan(int64_t count)
{
    ClipPlan p;
    p.partial_off = (size_t)ceil_div(count * (int64_t)sizeof(Entry), 256) * 256;
    p.total = p.partial_off + sizeof(double) * kClipBlocks;
    return p;
}

csp_status run_clip(const void *const *grads, void *const *outs, const int64_t *numel, const int32_t *dtypes,
                    int64_t count, float max_norm, float *norm, void *work, int64_t work_bytes, bool clip,
                    hipStream_t s)
{
    if (count < 0 || count >= 0x7FFFFFFF) return set_error(CSP_ERR_INVALID_ARG, "bad tensor count %lld", (long long)count);
    if (count > 0 && (!grads || !numel || !dtypes || (clip && !outs)))
        return set_error(CSP_ERR_INVALID_ARG, "NULL tensor list");
    if (!norm || (uintptr_t)norm % 4) return set_error(CSP_ERR_INVALID_ARG, "bad norm pointer");
    if (clip && !(max_norm >= 0.0f)) return set_error(CSP_ERR_INVALID_ARG, "max_norm must not be negative or NaN");
    const ClipPlan p = clip_plan(count);
    if (!work || (uintptr_t)work % 16 || work_bytes < (int64_t)p.total)
        return set_error(CSP_ERR_INVALID_ARG, "workspace of %lld bytes, %zu needed", (long long)work_bytes, p.total);
    int64_t chunks = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (dtypes[i] != CSP_F32 && dtypes[i] != CSP_BF16)
            return set_error(CSP_ERR_DTYPE, "tensor %lld: unsupported dtype %d", (long long)i, dtypes[i]);
        const int64_t esz = dtypes[i] == CSP_BF16 ? 2 : 4;
        if (numel[i] < 0 || numel[i] > (int64_t)1 << 56)
            return set_error(CSP_ERR_INVALID_ARG, "tensor %lld: bad element count", (long long)i);
        if (numel[i] > 0 && (!grads[i] || (uintptr_t)grads[i] % esz || (clip && (!outs[i] || (uintptr_t)outs[i] % esz))))
            return set_error(CSP_ERR_INVALID_ARG, "tensor %lld: NULL or misaligned pointer", (long long)i);
        chunks += ceil_div(numel[i] * esz, kChunkBytes);
    }
    Entry *table = (Entry *)work;
    double *partial = (double *)((char *)work + p.partial_off);
    InlineTable it{};
    int64_t first = 0;
    int used = 0;
    int64_t put = 0;
    const bool in_table = count > kInline;
    for (int64_t i = 0; i < count; ++i) {
        const int64_t esz = dtypes[i] == CSP_BF16 ? 2 : 4;
        it.e[used++] = Entry{grads[i], clip ? outs[i] : nullptr, numel[i], first << 1 | (dtypes[i] == CSP_BF16 ? 1 : 0)};
        first += ceil_div(numel[i] * esz, kChunkBytes);
        if (in_table && (used == kInline || i + 1 == count)) {
            k_table_put<<<1, 64, 0, s>>>(it, used, table + put);
            CSP_LAUNCHED("k_table_put");
            put += used;
            used = 0;
        }
    }
    const unsigned blocks = (unsigned)(chunks < kClipBlocks ? (chunks > 0 ? chunks : 1) : kClipBlocks);
    if (in_table) k_square_sums<true><<<blocks, kClipThreads, 0, s>>>(it, table, (int)count, chunks, partial);
    else k_square_sums<false><<<blocks, kClipThreads, 0, s>>>(it, table, (int)count, chunks, partial);
    CSP_LAUNCHED("k_square_sums");
    if (!clip) {
        k_norm<<<1, kClipThreads, 0, s>>>(partial, (int)blocks, norm);
        CSP_LAUNCHED("k_norm");
        return CSP_OK;
    }
    if (in_table)
        k_clip_scale<true><<<blocks, kClipThreads, 0, s>>>(it, table, (int)count, chunks, partial, (int)blocks, max_norm, norm);
    else
        k_clip_scale<false><<<blocks, kClipThreads, 0, s>>>(it, table, (int)count, chunks, partial, (int)blocks, max_norm, norm);
    CSP_LAUNCHED("k_clip_scale");
    return CSP_OK;
}

}  // namespace
}  // namespace csp

extern "C" {

int64_t grad_clip_workspace(int64_t count)
{
    if (count < 0 || count >= 0x7FFFFFFF) {
        csp::set_error(CSP_ERR_INVALID_ARG, "bad tensor count %lld", (long long)count);
        return -1;
    }
    return (int64_t)csp::clip_plan(count).total;
}

csp_status grad_norm(const void *const *grads, const int64_t *numel, const int32_t *dtypes, int64_t count, float *norm,
                     void *workspace, int64_t workspace_bytes, void *stream)
{
    return csp::run_clip(grads, nullptr, numel, dtypes, count, 0.0f, norm, workspace, workspace_bytes, false,
                         (hipStream_t)stream);
}

csp_status grad_clip(const void *const *grads, void *const *outs, const int64_t *numel, const int32_t *dtypes,
                     int64_t count, float max_norm, float *norm, void *workspace, int64_t workspace_bytes,
                     void *stream)
{
    return csp::run_clip(grads, outs, numel, dtypes, count, max_norm, norm, workspace, workspace_bytes, true,
                         (hipStream_t)stream);
}

}  // extern "C"
