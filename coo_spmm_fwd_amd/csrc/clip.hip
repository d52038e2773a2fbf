// clip.hip -- the global gradient norm over many tensors, and clipping by it.
//
//   norm = sqrt(sum over all tensors and elements of g^2)
//   out  = g * min(1, max_norm / (norm + 1e-6))
//
// Both passes are bound by memory: the norm reads every element once, the
// clipping reads it again and writes it.  All tensors together are one list of
// 8 KiB chunks of whole 16-byte vectors (the elements before a tensor's first
// 16-byte boundary go with its first chunk).  The sums go through the list
// from front to back, 8 chunks a workgroup and turn, so that a workgroup looks
// its tensor up once a turn; the scaling goes from back to front, a few chunks
// a workgroup, and so begins with what the memory-side cache still holds.
// Squares are summed in fp64 (no overflow below 1e154): at one fp64
// multiply-add per element the vector units are idle most of the time of the
// read.  Sums are joined in a fixed order, so results do not depend on
// scheduling.
//
// Measured (a 4 GiB copy on this card moves 4.8 TB/s): norm of 400 million fp32
// 258 us a call (6.2 TB/s), norm and clipping 805 (4.8 GB, 6.0 TB/s; 991 in one
// order with 2048 workgroups of 16 KiB chunks); 400 tensors of both types, 500
// million elements, 822 us (1067).  For 3 tensors of 1.9 MB the call is 18 us
// of host work, for hundreds 0.45 us a tensor in place and 0.8 with outputs apart.
#include <algorithm>
#include <memory>
#include <new>

#include "common.h"
#include "device_util.h"

namespace csp {
namespace {

constexpr int kClipThreads = 256;
constexpr int kVecPerThread = 2;                                   // 16-byte loads in flight per thread
constexpr int64_t kChunkBytes = kClipThreads * kVecPerThread * 16;  // 8 KiB
constexpr int64_t kClipBlocks = 1024;                               // workgroups of the sums, as many partial sums
constexpr int64_t kScaleBlocks = 8192;                              // workgroups of the scaling up to kScaleRun chunks each
constexpr int64_t kScaleRun = 3;                                    // ... and above that as many as it takes
constexpr int64_t kMaxBlocks = (int64_t)1 << 23;                    // a launch has fewer than 2^32 threads
constexpr int64_t kRun = 8;                                         // chunks that a workgroup of the sums takes in a row, once there are so many for each
constexpr int kInline = 64;                                         // tensors that go as kernel arguments
constexpr int kPut = 112;                                           // of more, those that one launch writes to the table

struct Entry {
    const void *g;
    void *o;
    int64_t n;
    int64_t first;  // the tensor's first chunk << 1 | 1 for bf16
};
struct InlineTable {
    Entry e[kInline];
};
struct PutTable {
    Entry e[kPut];
};

__global__ void k_table_put(PutTable t, int n, Entry *__restrict__ dst)
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

// Elements before the first 16-byte boundary: vectors are counted from there, since a tensor that is a
// slice of a bucket begins anywhere.
__host__ __device__ inline int64_t head_of(const void *g, int64_t n, int64_t esz)
{
    const int64_t h = (int64_t)((16 - (uintptr_t)g % 16) % 16) / esz;
    return h < n ? h : n;
}
__host__ __device__ inline int64_t chunks_of(const void *g, int64_t n, int64_t esz)
{
    const int64_t body = ((n - head_of(g, n, esz)) * esz + kChunkBytes - 1) / kChunkBytes;
    return n > 0 && body == 0 ? 1 : body;
}

__device__ __forceinline__ double square_of(const void *g, bool bf, int64_t k)
{
    const double x = bf ? (double)BF16::load((const uint16_t *)g, k) : (double)((const float *)g)[k];
    return x * x;
}

__device__ __forceinline__ double square_chunk(const Entry &t, int64_t chunk)
{
    const bool bf = t.first & 1;
    const int per = bf ? 8 : 4;  // elements a 16-byte load
    const char *g = (const char *)t.g;
    const int64_t head = head_of(g, t.n, bf ? 2 : 4);
    const int64_t base = head + chunk * (kChunkBytes / 16) * per;
    double acc = 0.0;
    if (chunk == 0 && threadIdx.x < head) acc = square_of(g, bf, threadIdx.x);
    u32x4 v[kVecPerThread];
#pragma unroll
    for (int j = 0; j < kVecPerThread; ++j) {
        const int64_t i = base + (int64_t)(j * kClipThreads + threadIdx.x) * per;
        v[j] = u32x4{0u, 0u, 0u, 0u};
        if (i + per <= t.n) v[j] = *(const u32x4 *)(g + (bf ? 2 : 4) * i);
        else  // the tensor's end: element by element
            for (int64_t k = i; k < t.n; ++k) acc += square_of(g, bf, k);
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
                                                              int count, int64_t chunks, int64_t run,
                                                              double *__restrict__ partial)
{
    __shared__ double lds[kClipThreads / 64];
    const Entry *e = kInTable ? table : it.e;
    double acc = 0.0;
    for (int64_t c0 = blockIdx.x * run; c0 < chunks; c0 += gridDim.x * run) {
        const int64_t c1 = c0 + run < chunks ? c0 + run : chunks;
        int t = find_tensor(e, count, c0);
        for (int64_t c = c0; c < c1; ++c) {
            while (t + 1 < count && (e[t + 1].first >> 1) <= c) ++t;
            acc += square_chunk(e[t], c - (e[t].first >> 1));
        }
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

__device__ __forceinline__ void scale_one(const void *g, void *o, bool bf, int64_t k, float c)
{
    if (bf) ((uint16_t *)o)[k] = BF16::from_f(BF16::load((const uint16_t *)g, k) * c);
    else ((float *)o)[k] = ((const float *)g)[k] * c;
}

template <bool kStream>
__device__ __forceinline__ void scale_chunk(const Entry &t, int64_t chunk, float c)
{
    const bool bf = t.first & 1;
    const int per = bf ? 8 : 4;
    const char *g = (const char *)t.g;
    char *o = (char *)t.o;
    const int64_t head = head_of(g, t.n, bf ? 2 : 4);
    const int64_t base = head + chunk * (kChunkBytes / 16) * per;
    if (chunk == 0 && threadIdx.x < head) scale_one(g, o, bf, threadIdx.x, c);
    u32x4 v[kVecPerThread];
#pragma unroll
    for (int j = 0; j < kVecPerThread; ++j) {
        const int64_t i = base + (int64_t)(j * kClipThreads + threadIdx.x) * per;
        v[j] = u32x4{0u, 0u, 0u, 0u};
        if (i + per <= t.n) v[j] = *(const u32x4 *)(g + (bf ? 2 : 4) * i);
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
            if constexpr (kStream) store16_nt(o + (bf ? 2 : 4) * i, v[j]);
            else store16(o + (bf ? 2 : 4) * i, v[j]);
        } else {
            for (int64_t k = i; k < t.n; ++k) scale_one(g, o, bf, k, c);
        }
    }
}

// The chunks of a workgroup in the reverse of the order that k_square_sums read them in: the last ones
// are still in the memory-side cache.
template <bool kInTable, bool kStream>
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
    const int64_t place = gridDim.x - 1 - blockIdx.x;
    const int64_t c0 = chunks * place / gridDim.x, c1 = chunks * (place + 1) / gridDim.x;
    if (c0 == c1) return;
    int t = find_tensor(e, count, c1 - 1);
    for (int64_t k = c1; k-- > c0;) {
        while (t > 0 && (e[t].first >> 1) > k) --t;
        if (c == 1.0f && e[t].o == e[t].g) continue;  // in place and nothing to change
        scale_chunk<kStream>(e[t], k - (e[t].first >> 1), c);
    }
}

// Outputs of tensors past half the memory-side cache (256 MB) bypass L2 and leave it to the gradients.
constexpr int64_t kStreamBytes = (int64_t)128 << 20;

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

// Outputs share no byte with each other, nor with any gradient but their own in place: workgroups read and
// write in no order.  Sorted by address, each has to end before the next begins (400 tensors: 6 us on the host).
struct Span {
    uintptr_t first, last;
    int64_t i;
};
csp_status outputs_apart(const void *const *grads, void *const *outs, const int64_t *numel, const int32_t *dtypes,
                         int64_t count)
{
    std::unique_ptr<Span[]> w(new (std::nothrow) Span[(size_t)count]);
    if (!w) return set_error(CSP_ERR_NO_MEMORY, "no host memory for %lld tensors", (long long)count);
    auto span = [&](const void *p, int64_t i) {
        return Span{(uintptr_t)p, (uintptr_t)p + (uintptr_t)numel[i] * (dtypes[i] == CSP_BF16 ? 2 : 4), i};
    };
    auto overlap = [&](int64_t a, int64_t b) {
        return set_error(CSP_ERR_INVALID_ARG, "tensors %lld and %lld overlap", (long long)a, (long long)b);
    };
    int64_t n = 0;
    for (int64_t i = 0; i < count; ++i)
        if (numel[i] > 0) w[n++] = span(outs[i], i);
    std::sort(w.get(), w.get() + n, [](const Span &a, const Span &b) { return a.first < b.first; });
    for (int64_t k = 1; k < n; ++k)
        if (w[k].first < w[k - 1].last) return overlap(w[k - 1].i, w[k].i);
    for (int64_t i = 0; i < count; ++i) {
        if (numel[i] == 0 || grads[i] == outs[i]) continue;  // in place: compared with the others above
        const Span g = span(grads[i], i);
        const Span *past = std::lower_bound(w.get(), w.get() + n, g.last,
                                            [](const Span &a, uintptr_t end) { return a.first < end; });
        if (past != w.get() && past[-1].last > g.first) return overlap(i, past[-1].i);
    }
    return CSP_OK;
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
    int64_t chunks = 0, bytes = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (dtypes[i] != CSP_F32 && dtypes[i] != CSP_BF16)
            return set_error(CSP_ERR_DTYPE, "tensor %lld: unsupported dtype %d", (long long)i, dtypes[i]);
        const int64_t esz = dtypes[i] == CSP_BF16 ? 2 : 4;
        if (numel[i] < 0 || numel[i] > (int64_t)1 << 56)
            return set_error(CSP_ERR_INVALID_ARG, "tensor %lld: bad element count", (long long)i);
        if (numel[i] > 0 && (!grads[i] || (uintptr_t)grads[i] % esz || (clip && (!outs[i] || (uintptr_t)outs[i] % esz))))
            return set_error(CSP_ERR_INVALID_ARG, "tensor %lld: NULL or misaligned pointer", (long long)i);
        chunks += chunks_of(grads[i], numel[i], esz);
        bytes += numel[i] * esz;
    }
    if (clip) {
        const csp_status st = outputs_apart(grads, outs, numel, dtypes, count);
        if (st != CSP_OK) return st;
    }
    Entry *table = (Entry *)work;
    double *partial = (double *)((char *)work + p.partial_off);
    InlineTable it;
    PutTable put;
    int64_t first = 0;
    int used = 0;
    int64_t done = 0;
    const bool in_table = count > kInline;
    for (int64_t i = 0; i < count; ++i) {
        const int64_t esz = dtypes[i] == CSP_BF16 ? 2 : 4;
        (in_table ? put.e : it.e)[used++] =
            Entry{grads[i], clip ? outs[i] : nullptr, numel[i], first << 1 | (dtypes[i] == CSP_BF16 ? 1 : 0)};
        first += chunks_of(grads[i], numel[i], esz);
        if (in_table && (used == kPut || i + 1 == count)) {
            k_table_put<<<1, 128, 0, s>>>(put, used, table + done);
            CSP_LAUNCHED("k_table_put");
            done += used;
            used = 0;
        }
    }
    const unsigned blocks = (unsigned)(chunks < kClipBlocks ? (chunks > 0 ? chunks : 1) : kClipBlocks);
    const int64_t run = chunks < kRun * blocks ? (chunks > blocks ? chunks / blocks : 1) : kRun;
    auto sums = in_table ? k_square_sums<true> : k_square_sums<false>;
    sums<<<blocks, kClipThreads, 0, s>>>(it, table, (int)count, chunks, run, partial);
    CSP_LAUNCHED("k_square_sums");
    if (!clip) {
        k_norm<<<1, kClipThreads, 0, s>>>(partial, (int)blocks, norm);
        CSP_LAUNCHED("k_norm");
        return CSP_OK;
    }
    const bool stream = bytes > kStreamBytes;
    auto scale = in_table ? (stream ? k_clip_scale<true, true> : k_clip_scale<true, false>)
                          : (stream ? k_clip_scale<false, true> : k_clip_scale<false, false>);
    int64_t most = chunks < kScaleBlocks ? (chunks > 0 ? chunks : 1) : kScaleBlocks;
    if (most * kScaleRun < chunks) most = ceil_div(chunks, kScaleRun);
    if (most > kMaxBlocks) most = kMaxBlocks;
    scale<<<(unsigned)most, kClipThreads, 0, s>>>(it, table, (int)count, chunks, partial, (int)blocks, max_norm, norm);
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
