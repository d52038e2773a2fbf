// embed.hip -- embedding lookup with scaling, and its gradient by sorted tokens.
//
//   forward   Y[n, :]  = scale * E[ids[n], :]
//   backward  dE[v, :] = scale * sum over n with ids[n] = v of dY[n, :]
//
// An id outside [0, V) takes no part: a zero row of Y, no term in dE.  Both
// are bound by memory: the forward by the rows it reads and writes, the
// backward by dE, every row of which is written, and dY.  The gradient adds
// the rows of one id in token order in fp32 and rounds once, without
// floating-point atomics, so the same inputs give the same bits.
//
// Backward in three launches:
//   sort   tokens by id, stably (k_embed_sort, or the radix sort): order[],
//          and ptr[v] = first place of id v.
//   rows   one pass over dE: adds an id's tokens, or writes zeros.  The places
//          are also cut at every kPart-th, and an id with more than kPart
//          tokens (text has a few that make up a tenth of it) is summed a
//          piece at a time by as many waves, into fp32 rows: slot 2k for the
//          piece that comes into cut k from before it, 2k + 1 for one that
//          starts in it and goes on.  The pieces' workgroups are strewn among
//          those of the rows, so that their chains of loads run under the
//          writing.
//   join   adds the pieces of such ids in order.
// A wave owns 64 16-byte vectors of a row (or several narrower rows), so
// widths cost no idle lanes beyond a row's last part.
//
// Measured (a 4 GiB copy on this card moves 4.8 TB/s): lookup of 16384 rows of
// 4096 bf16, 32 us a call; gradient of 32768 such rows into 65536, 197 us a
// call, of which sort 20, rows 144 (805 MB, 5.6 TB/s), join 7; 4093 rows of 768
// fp32 into 50257: sort 7.5, rows 25 (167 MB, 6.7 TB/s), join 4.
#include "common.h"
#include "device_util.h"

namespace csp {
namespace {

constexpr int kEmbedThreads = 256;
constexpr int kRowsPerLane = 8;   // rows of dE a lane group takes one after another
constexpr int64_t kPart = 64;     // tokens a wave adds one after another
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortIds = 256;     // ids a workgroup of k_embed_sort looks for
constexpr int64_t kMaxBlocks = ((int64_t)1 << 24) - 1;  // a launch has fewer than 2^32 threads

template <typename E> struct Vec;
template <> struct Vec<F32> {
    static constexpr int kPer = 4;
    __device__ static void add(u32x4 v, float (&s)[4])
    {
#pragma unroll
        for (int q = 0; q < 4; ++q) s[q] += __uint_as_float(v[q]);
    }
    __device__ static u32x4 pack(const float (&s)[4], float scale)
    {
        u32x4 v;
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = __float_as_uint(s[q] * scale);
        return v;
    }
};
template <> struct Vec<BF16> {
    static constexpr int kPer = 8;
    __device__ static void add(u32x4 v, float (&s)[8])
    {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            s[2 * q] += __uint_as_float(v[q] << 16);
            s[2 * q + 1] += __uint_as_float(v[q] & 0xFFFF0000u);
        }
    }
    __device__ static u32x4 pack(const float (&s)[8], float scale)
    {
        u32x4 v;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            v[q] = (uint32_t)BF16::from_f(s[2 * q] * scale) | (uint32_t)BF16::from_f(s[2 * q + 1] * scale) << 16;
        return v;
    }
};

// How rows of D elements are dealt to lanes: `lanes` lanes (a power of two, 64 at most) take a strip of
// as many vectors.  A row's last vector starts early enough to be whole: lanes that overlap compute and
// write the same values.  Rows narrower than a vector go element by element, one lane a row.
struct Strips {
    int log2_lanes;
    uint32_t strips;
};
Strips strips_of(int64_t D, int per)
{
    const int64_t nvec = ceil_div(D, per);
    Strips s{0, 1};
    while (s.log2_lanes < 6 && ((int64_t)1 << s.log2_lanes) < nvec) ++s.log2_lanes;
    s.strips = (uint32_t)ceil_div(nvec, (int64_t)1 << s.log2_lanes);
    return s;
}
// A lane's group, and its vector and first element of the row; lanes past the row (not `live`) shadow
// its last vector, so that the whole group stays together.
struct Lane {
    uint32_t group;
    int64_t vec, col;
    bool live;
};
__device__ __forceinline__ Lane lane_place(Strips sp, uint32_t block, int64_t D, int per)
{
    uint32_t gl = (block * kEmbedThreads + threadIdx.x) >> sp.log2_lanes;
    if (sp.log2_lanes == 6) gl = __builtin_amdgcn_readfirstlane(gl);
    Lane p;
    p.group = gl / sp.strips;
    p.vec = ((int64_t)(gl - p.group * sp.strips) << sp.log2_lanes) + (threadIdx.x & ((1 << sp.log2_lanes) - 1));
    p.live = p.vec * per < D;
    if (!p.live) p.vec = (D - 1) / per;
    p.col = p.vec * per;
    if (p.col + per > D && D >= per) p.col = D - per;
    return p;
}

template <typename E>
__device__ __forceinline__ void add_row(const typename E::T *__restrict__ p, int64_t D, float (&s)[Vec<E>::kPer])
{
    if (D >= Vec<E>::kPer) Vec<E>::add(load16(p), s);
    else
        for (int64_t c = 0; c < D; ++c) s[c] += E::load(p, c);
}
template <typename E, bool kStream>
__device__ __forceinline__ void put_row(typename E::T *__restrict__ p, int64_t D, const float (&s)[Vec<E>::kPer],
                                        float scale)
{
    if (D >= Vec<E>::kPer) kStream ? store16_nt(p, Vec<E>::pack(s, scale)) : store16(p, Vec<E>::pack(s, scale));
    else
        for (int64_t c = 0; c < D; ++c) p[c] = E::from_f(s[c] * scale);
}

template <typename E, bool kStream>
__global__ __launch_bounds__(kEmbedThreads) void k_embed_fwd(const typename E::T *__restrict__ table, int64_t V,
                                                             int64_t D, const int64_t *__restrict__ ids, int64_t N,
                                                             float scale, Strips sp, typename E::T *__restrict__ Y)
{
    const Lane p = lane_place(sp, blockIdx.x, D, Vec<E>::kPer);
    if (!p.live || p.group >= N) return;
    const int64_t id = ids[p.group];
    float s[Vec<E>::kPer] = {};
    const bool part = id >= 0 && id < V;
    if (part) add_row<E>(table + id * D + p.col, D, s);
    put_row<E, kStream>(Y + p.group * D + p.col, D, s, part ? scale : 0.0f);  // zero whatever the scale is
}

// order[] and ptr[] for one range of kSortIds ids a workgroup.  Each workgroup reads all N ids (from
// L2: 32768 of them are 256 KiB), a contiguous share a wave, twice: once to count, for its own ids by
// wave and for all smaller ids together, and once to place its tokens in order.  No other workgroup's
// result is needed, so this is the whole sort.
__global__ __launch_bounds__(kSortThreads) void k_embed_sort(const int64_t *__restrict__ ids, int64_t N, int64_t V,
                                                             int32_t *__restrict__ order, int32_t *__restrict__ ptr)
{
    __shared__ uint32_t at[kSortWaves][kSortIds];
    __shared__ uint32_t lds[17], below_all;
    constexpr int kAhead = 8;  // loads in flight
    const int l = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t v0 = blockIdx.x * kSortIds, vocab = (uint32_t)V;
    const uint32_t mine = vocab - v0 < kSortIds ? vocab - v0 : kSortIds;
    const int n_all = (int)N, share = (n_all + 64 * kSortWaves - 1) / (64 * kSortWaves) * 64;
    const int n0 = w * share < n_all ? w * share : n_all, n1 = n0 + share < n_all ? n0 + share : n_all;
    for (int i = threadIdx.x; i < kSortWaves * kSortIds; i += kSortThreads) (&at[0][0])[i] = 0;
    if (threadIdx.x == 0) below_all = 0;
    __syncthreads();
    // f(token, id as 32 bits) over the wave's share, 64 tokens at a time; no id for those that take no part
    auto walk = [&](auto &&f) {
        for (int b = n0; b < n1; b += 64 * kAhead) {
            uint64_t id[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int n = b + 64 * j + l;
                id[j] = (uint64_t)ids[n < n1 ? n : n0];
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int n = b + 64 * j + l;
                f(n, id[j] < (uint64_t)vocab && n < n1 ? (uint32_t)id[j] : 0xFFFFFFFFu);
            }
        }
    };
    uint32_t below = 0;
    walk([&](int, uint32_t id) {
        below += (uint32_t)__popcll(__ballot(id < v0));
        const bool in = id - v0 < mine;
        if (__ballot(in) == 0) return;
        if (in) atomicAdd(&at[w][id - v0], 1u);
    });
    if (l == 0) atomicAdd(&below_all, below);
    __syncthreads();
    uint32_t sum = 0, total;
    if (threadIdx.x < kSortIds)
        for (int i = 0; i < kSortWaves; ++i) sum += at[i][threadIdx.x];
    uint32_t first = block_exclusive_scan(sum, lds, &total) + below_all;
    if (threadIdx.x < kSortIds) {
        if (threadIdx.x < mine) ptr[v0 + threadIdx.x] = (int32_t)first;
        for (int i = 0; i < kSortWaves; ++i) {
            const uint32_t c = at[i][threadIdx.x];
            at[i][threadIdx.x] = first;
            first += c;
        }
    }
    if (threadIdx.x == 0 && vocab - v0 <= kSortIds) ptr[V] = (int32_t)(below_all + total);
    __syncthreads();
    if (total == 0) return;
    walk([&](int n, uint32_t id) {
        const bool in = id - v0 < mine;
        uint64_t left = __ballot(in), same = 0;
        if (left == 0) return;
        for (int i = 0; i < 6 && left != 0; ++i) {  // mostly one or two ids; the ballots below cost as much as 8
            const uint32_t first_id = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)left) - 1);
            const uint64_t m = __ballot(id == first_id);
            if (id == first_id) same = m;
            left &= ~m;
        }
        if (left != 0) same = lanes_with_same_byte(id - v0, in);
        uint32_t place = 0;
        if (in && (same & lanes_below()) == 0) place = atomicAdd(&at[w][id - v0], (uint32_t)__popcll(same));
        place = __shfl(place, in ? __ffsll((unsigned long long)same) - 1 : l, 64);
        if (in) order[place + __popcll(same & lanes_below())] = n;
    });
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

// s += row(k) + ... + row(n - 1), in that order, kAhead rows loaded at a time.
template <int kAhead, typename Load, typename Add>
__device__ __forceinline__ void add_rows(int &k, int n, Load &&load, Add &&add)
{
    for (; k + kAhead <= n; k += kAhead) {
        decltype(load(0)) v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) v[j] = load(k + j);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) add(v[j]);
    }
    if constexpr (kAhead > 1) add_rows<kAhead / 2>(k, n, load, add);
}

// s += rows order[a .. b) of dY, in that order.  The lanes of a group load its next tokens together
// and hand them round.
template <typename E>
__device__ __forceinline__ void add_tokens(const typename E::T *__restrict__ dY, int64_t D, int64_t col, Strips sp,
                                           const int32_t *__restrict__ order, int32_t a, int32_t b,
                                           float (&s)[Vec<E>::kPer])
{
    const int lanes = 1 << sp.log2_lanes, l = threadIdx.x & 63, g0 = l & ~(lanes - 1);
    for (int32_t t = a; t < b; t += lanes) {
        const int n = b - t < lanes ? b - t : lanes;
        const int32_t mine = order[t + (l - g0 < n ? l - g0 : 0)];
        int k = 0;
        if (D < Vec<E>::kPer) {
            for (; k < n; ++k) add_row<E>(dY + (int64_t)__shfl(mine, g0 + k, 64) * D, D, s);
        } else if (lanes == 64) {  // one row for the whole wave: its address is a scalar
            add_rows<4>(k, n, [&](int j) { return load16(dY + (int64_t)__builtin_amdgcn_readlane(mine, j) * D + col); },
                        [&](u32x4 v) { Vec<E>::add(v, s); });
        } else {
            add_rows<4>(k, n, [&](int j) { return load16(dY + (int64_t)__shfl(mine, g0 + j, 64) * D + col); },
                        [&](u32x4 v) { Vec<E>::add(v, s); });
        }
    }
}

struct EmbedGrad {
    const int32_t *order, *ptr;
    const int64_t *ids;
    int64_t D, V, N;
    Strips sp;
    float *part;
    int64_t ldp;
    float scale;
};

// The piece of slot sl: its id and places [from, to); false if no id of more than kPart tokens has one there.
__device__ __forceinline__ bool slot_piece(const EmbedGrad &a, int64_t sl, int64_t &id, int32_t &from, int32_t &to)
{
    const int64_t k0 = (sl >> 1) * kPart, have = a.ptr[a.V];
    if (k0 >= have) return false;
    const int64_t end = k0 + kPart < have ? k0 + kPart : have;
    const bool starts = sl & 1;
    id = a.ids[a.order[starts ? end - 1 : k0]];
    const int32_t first = a.ptr[id], last = a.ptr[id + 1];
    from = starts ? first : (int32_t)k0;
    to = last < end ? last : (int32_t)end;
    return last - first > kPart && (first >= k0) == starts;
}

template <typename E, bool kStream>
__global__ __launch_bounds__(kEmbedThreads, 8) void k_embed_rows(EmbedGrad a, const typename E::T *__restrict__ dY,
                                                              uint32_t piece_blocks, uint32_t every,
                                                              typename E::T *__restrict__ dE)
{
    constexpr int kPer = Vec<E>::kPer;
    const uint32_t turn = blockIdx.x / every;  // of every `every` workgroups the first is a piece's
    if (turn < piece_blocks && turn * every == blockIdx.x) {
        const Lane p = lane_place(a.sp, turn, a.D, kPer);
        const int64_t sl = p.group;
        int64_t id;
        int32_t from, to;
        if (sl >= 2 * ceil_div(a.N, kPart) || !slot_piece(a, sl, id, from, to)) return;
        float s[kPer] = {};
        add_tokens<E>(dY, a.D, p.col, a.sp, a.order, from, to, s);
        float *q = a.part + sl * a.ldp + p.vec * kPer;
        if (p.live)
#pragma unroll
            for (int c = 0; c < kPer; c += 4) *(float4 *)(q + c) = make_float4(s[c], s[c + 1], s[c + 2], s[c + 3]);
        return;
    }
    const Lane p = lane_place(a.sp, blockIdx.x - (turn < piece_blocks ? turn + 1 : piece_blocks), a.D, kPer);
    const int64_t first = (int64_t)p.group * kRowsPerLane;
    // the rows' offsets: one load a lane, handed round
    const int lanes = 1 << a.sp.log2_lanes, l = threadIdx.x & 63, g0 = l & ~(lanes - 1);
    const int64_t left = a.V - first;
    if (left <= 0) return;
    const int rows = left < kRowsPerLane ? (int)left : kRowsPerLane;
    int32_t at0 = a.ptr[first];
    int32_t ends = 0;
#pragma unroll 1
    for (int r = 0; r < rows; ++r) {
        if ((r & (lanes - 1)) == 0) ends = a.ptr[first + 1 + (r + l - g0 < rows ? r + l - g0 : r)];
        const int32_t at1 = lanes == 64 ? __builtin_amdgcn_readlane(ends, r) : __shfl(ends, g0 + (r & (lanes - 1)), 64);
        if (at1 - at0 <= kPart) {
            float s[kPer] = {};
            add_tokens<E>(dY, a.D, p.col, a.sp, a.order, at0, at1, s);
            if (p.live) put_row<E, kStream>(dE + (first + r) * a.D + p.col, a.D, s, at1 > at0 ? a.scale : 0.0f);
        }
        at0 = at1;
    }
}

// One lane group for each cut in which an id of more than kPart tokens starts.
template <typename E>
__global__ __launch_bounds__(kEmbedThreads) void k_embed_join(EmbedGrad a, typename E::T *__restrict__ dE)
{
    constexpr int kPer = Vec<E>::kPer;
    struct Row {
        float4 x[kPer / 4];
    };
    const Lane p = lane_place(a.sp, blockIdx.x, a.D, kPer);
    const int64_t cut = p.group;
    int64_t id;
    int32_t from, to;
    if (cut >= ceil_div(a.N, kPart) || !slot_piece(a, 2 * cut + 1, id, from, to)) return;
    const int n = (int)((a.ptr[id + 1] - 1) / kPart - cut) + 1;
    const float *q = a.part + 2 * cut * a.ldp + p.vec * kPer;
    float s[kPer] = {};
    int k = 0;
    add_rows<8>(k, n,
                [&](int j) {
                    Row r;
                    const float *x = q + (j == 0 ? 1 : 2 * (int64_t)j) * a.ldp;
#pragma unroll
                    for (int c = 0; c < kPer / 4; ++c) r.x[c] = *(const float4 *)(x + 4 * c);
                    return r;
                },
                [&](const Row &r) {
#pragma unroll
                    for (int c = 0; c < kPer / 4; ++c) {
                        s[4 * c] += r.x[c].x;
                        s[4 * c + 1] += r.x[c].y;
                        s[4 * c + 2] += r.x[c].z;
                        s[4 * c + 3] += r.x[c].w;
                    }
                });
    if (p.live) put_row<E, false>(dE + id * a.D + p.col, a.D, s, a.scale);
}

// k_embed_sort costs N id reads to each of ceil(V / kSortIds) workgroups, more where few ids share the tokens;
// the radix sort a dozen launches.  The whole gradient at d 64 bf16, range / radix, us: V 65536: 8192 tokens 22 /
// 90, 65536 64 / 113; V 250000: 8192 37 / 98, 32768 71 / 111, 131072 194 / 133; V 3000: 8192 42 / 86, 32768 80 /
// 105, 131072 227 / 166; V 200: 8192 73 / 97, 32768 124 / 116.
constexpr int64_t kSortReads = (int64_t)1 << 25, kSortTokens = (int64_t)1 << 16;
bool sort_by_range(int64_t N, int64_t V)
{
    return V <= (int64_t)1 << 24 && N <= (V < 4096 ? kSortTokens / 2 : kSortTokens) && ceil_div(V, kSortIds) * N <= kSortReads;
}

struct EmbedPlan {
    size_t key[3], pos[3], ptr, hist, part, total;
    int64_t ldp;
};

EmbedPlan embed_plan(int64_t N, int64_t V, int64_t D)
{
    EmbedPlan p{};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t r = at;
        at += (bytes + 255) / 256 * 256;
        return r;
    };
    p.pos[2] = take(4 * (size_t)N);
    p.ptr = take(4 * (size_t)(V + 1));
    if (!sort_by_range(N, V)) {
        for (int i = 0; i < 3; ++i) p.key[i] = take(4 * (size_t)N);
        for (int i = 0; i < 2; ++i) p.pos[i] = take(4 * (size_t)N);
        p.hist = take(4 * sort_hist_words(N));
    }
    p.ldp = ceil_div(D, 8) * 8;
    p.part = take(N > kPart ? 8 * (size_t)ceil_div(N, kPart) * (size_t)p.ldp : 0);
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

// Workgroups of `groups` lane groups (rows, or slots).
int64_t blocks_of(Strips sp, int64_t groups) { return ceil_div(groups * sp.strips, kEmbedThreads >> sp.log2_lanes); }

// Workgroups of the gradient's rows and pieces.  A workgroup of rows is 16 KiB of dE and more where there are many:
// what one launch cannot hold, memory could not.
struct GradBlocks {
    int64_t cuts, rows, pieces;
};
GradBlocks grad_blocks(int64_t N, int64_t V, int64_t D, int dtype)
{
    const Strips sp = strips_of(D, dtype == CSP_BF16 ? Vec<BF16>::kPer : Vec<F32>::kPer);
    const int64_t cuts = N > kPart ? ceil_div(N, kPart) : 0;
    return {cuts, blocks_of(sp, ceil_div(V, kRowsPerLane)), blocks_of(sp, 2 * cuts)};
}
csp_status embed_bwd_args(int64_t N, int64_t V, int64_t D, int dtype)
{
    const csp_status st = embed_args(N, V, D, dtype);
    if (st != CSP_OK) return st;
    const GradBlocks b = grad_blocks(N, V, D, dtype);
    if (b.rows + b.pieces > kMaxBlocks)
        return set_error(CSP_ERR_INVALID_ARG, "gradient of %lld x %lld and %lld tokens is too large for a launch",
                         (long long)V, (long long)D, (long long)N);
    return CSP_OK;
}

// Stores that are not kept in L2, for outputs that pass it anyway: dirty lines of the output then do not
// stand in the way of the rows being read.  Lookup: Y of 32 MB and more (d 4096 bf16, plain / streamed:
// 8192 tokens 19.4 / 18.4 us, 16384 41.0 / 32.8, 32768 103 / 63; none faster below).  Gradient: dE and
// twice dY (it is read in between) past the 256 MB of the memory-side cache (dE 134 MB, dY 67: 56.0 / 45.2 us,
// 537 and 268: 208 / 198; but dE 154 and 206 MB, dY 13 and 17: 36.6 / 43.0 and 42.0 / 49.7).
constexpr int64_t kStreamFwd = (int64_t)32 << 20, kStreamBwd = (int64_t)256 << 20;

template <typename E, bool kStream>
csp_status fwd_impl(const void *table, const int64_t *ids, int64_t N, int64_t V, int64_t D, float scale, void *Y,
                    hipStream_t s)
{
    using T = typename E::T;
    const Strips sp = strips_of(D, Vec<E>::kPer);
    const int64_t most = kMaxBlocks * (kEmbedThreads >> sp.log2_lanes) / sp.strips;  // rows of a launch
    for (int64_t n = 0; n < N; n += most) {
        k_embed_fwd<E, kStream><<<(unsigned)blocks_of(sp, N - n < most ? N - n : most), kEmbedThreads, 0, s>>>(
            (const T *)table, V, D, ids + n, N - n, scale, sp, (T *)Y + n * D);
        CSP_LAUNCHED("k_embed_fwd");
    }
    return CSP_OK;
}

template <typename E, bool kStream>
csp_status bwd_impl(const void *dY, const int64_t *ids, int64_t N, int64_t V, int64_t D, float scale, void *dE,
                    char *w, hipStream_t s)
{
    using T = typename E::T;
    const EmbedPlan p = embed_plan(N, V, D);
    int32_t *ptr = (int32_t *)(w + p.ptr), *order = (int32_t *)(w + p.pos[2]);
    csp_status st = CSP_OK;
    if (sort_by_range(N, V)) {
        k_embed_sort<<<(unsigned)ceil_div(V, kSortIds), kSortThreads, 0, s>>>(ids, N, V, order, ptr);
        CSP_LAUNCHED("k_embed_sort");
    } else {
        uint32_t *key = (uint32_t *)(w + p.key[0]);
        int32_t *pos = (int32_t *)(w + p.pos[0]);
        if (N > 0) {
            k_embed_keys<<<(unsigned)ceil_div(N, 256), 256, 0, s>>>(ids, N, V, key, pos);
            CSP_LAUNCHED("k_embed_keys");
        }
        st = radix_sort_pairs(4, key, pos, w + p.key[2], order, w + p.key[1], (int32_t *)(w + p.pos[1]), N,
                              bits_for((uint64_t)V), (uint32_t *)(w + p.hist), s);
        if (st != CSP_OK) return st;
        st = segment_offsets((const int32_t *)(w + p.key[2]), N, ptr, V, s);
        if (st != CSP_OK) return st;
    }
    const Strips sp = strips_of(D, Vec<E>::kPer);
    const EmbedGrad a{order, ptr, ids, D, V, N, sp, (float *)(w + p.part), p.ldp, scale};
    const GradBlocks b = grad_blocks(N, V, D, sizeof(T) == 2 ? CSP_BF16 : CSP_F32);
    const unsigned first = (unsigned)b.pieces, all = first + (unsigned)b.rows;
    const unsigned every = all >= 5 * first ? 5 : all >= 3 * first ? 3 : 1;  // odd: all XCDs
    k_embed_rows<E, kStream><<<all, kEmbedThreads, 0, s>>>(a, (const T *)dY, first, every, (T *)dE);
    CSP_LAUNCHED("k_embed_rows");
    if (b.cuts == 0) return CSP_OK;
    k_embed_join<E><<<(unsigned)blocks_of(sp, b.cuts), kEmbedThreads, 0, s>>>(a, (T *)dE);
    CSP_LAUNCHED("k_embed_join");
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
    const bool past_cache = N * D >= kStreamFwd / (dtype == CSP_BF16 ? 2 : 4);
    auto run = dtype == CSP_BF16 ? (past_cache ? fwd_impl<BF16, true> : fwd_impl<BF16, false>)
                                 : (past_cache ? fwd_impl<F32, true> : fwd_impl<F32, false>);
    return run(E, ids, N, V, D, scale, Y, (hipStream_t)stream);
}

int64_t embed_bwd_workspace(int64_t N, int64_t V, int64_t D, csp_dtype dtype)
{
    if (csp::embed_bwd_args(N, V, D, dtype) != CSP_OK) return -1;
    return (int64_t)csp::embed_plan(N, V, D).total;
}

csp_status embed_bwd(const void *dY, const int64_t *ids, int64_t N, int64_t V, int64_t D, csp_dtype dtype, float scale,
                     void *dE, void *workspace, int64_t workspace_bytes, void *stream)
{
    using namespace csp;
    csp_status st = embed_bwd_args(N, V, D, dtype);
    if (st != CSP_OK) return st;
    if (!aligned(dE, dtype) || (N > 0 && (!aligned(dY, dtype) || !ids || (uintptr_t)ids % 8)))
        return set_error(CSP_ERR_INVALID_ARG, "NULL or misaligned pointer");
    const size_t need = embed_plan(N, V, D).total;
    if (!workspace || (uintptr_t)workspace % 16 || workspace_bytes < (int64_t)need)
        return set_error(CSP_ERR_INVALID_ARG, "workspace of %lld bytes, %zu needed", (long long)workspace_bytes, need);
    const bool past_cache = (V + 2 * N) * D > kStreamBwd / (dtype == CSP_BF16 ? 2 : 4);
    auto run = dtype == CSP_BF16 ? (past_cache ? bwd_impl<BF16, true> : bwd_impl<BF16, false>)
                                 : (past_cache ? bwd_impl<F32, true> : bwd_impl<F32, false>);
    return run(dY, ids, N, V, D, scale, dE, (char *)workspace, (hipStream_t)stream);
}

}  // extern "C"
