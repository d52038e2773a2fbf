// ce_few.hip -- linear cross entropy of up to 64 tokens, or 128 in fp32 (formulas in ce.hip).
//
// With so few tokens every product is bound by the bytes of W and dW: 2 N
// operations a byte of bf16 W at N = 64 is 64, where the matrix units and the
// memory balance near 400.  So W is read straight from memory into the matrix
// units' operand registers, once in the forward and twice in the backward,
// without a copy or a pass through LDS, whatever its width and alignment; only
// the tokens go through LDS.  fp32 elements are split into three bf16 planes in
// registers on their way.
//
//   forward   k_few_prep, k_few_rows (logits -> maximum and sum of each 128
//             vocabulary rows), k_few_join
//   backward  k_few_prep, k_few_rows (logits -> P -> dW rows, and P for dX),
//             k_few_targets (the targets' elements of P and their rows of dW),
//             k_few_dx, k_ce_out
//
// Measured: one token, W 50257 x 768 fp32 (154 MB): rows 35 us, the call 47 of
// which 12 are the two small kernels and the gaps.  One token, 65536 x 4096 bf16
// (537 MB): 99 us a call, 5.4 TB/s.  64 tokens on that W: forward 118 us a call;
// the training step 550 (2.15 GB, 3.9 TB/s; a 4 GiB copy moves 4.8).  32 tokens
// on the fp32 W: rows 39, backward rows 74 (308 MB), dX 39, the step 188.
//
// A wave holds 32 vocabulary rows.  Its logits come out with a vocabulary row
// a lane (lane % 16) and tokens 4 (lane / 16) + r in the registers, which is
// also how the product for dW wants P (tokens as depth, in that order): P goes
// from one product into the next without leaving the registers.
//
// Fragments: a matrix operand of 16 rows and depth 32 is 64 lanes of 8 bf16,
// row = lane % 16; what depth the lane's 8 elements are is free as long as both
// operands agree.  fp32 rows of W are loaded 4 elements at a time, so there
// lane / 16 = q has depth 4 q .. + 3 and 16 + 4 q .. + 3; bf16 rows have 8 q .. + 7.
#include "ce.h"

namespace csp {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kFewThreads = 256, kFewWaves = 4;
constexpr int kWaveRows = 32;                      // vocabulary rows of a wave
constexpr int kFewRows = kFewWaves * kWaveRows;    // of a workgroup
constexpr int kFewCols = 64;                       // columns of dW a step

template <typename E> struct Form;
template <> struct Form<BF16> {
    // planes of X and W, and of P; depth steps of 32 a chunk; elements of 16 bytes
    static constexpr int kPlanes = 1, kPPlanes = 2, kSteps = 4, kPer = 8;
};
template <> struct Form<F32> {
    static constexpr int kPlanes = 3, kPPlanes = 3, kSteps = 2, kPer = 4;
};
template <typename E> constexpr int kChunk = 32 * Form<E>::kSteps;  // depth of a chunk: 4 16-byte loads a row and lane

// Depth of element j of a lane with lane / 16 = q within a step of 32.
template <typename E> __host__ __device__ constexpr int depth_of(int q, int j)
{
    return Form<E>::kPlanes == 1 ? 8 * q + j : (j & 4) * 4 + 4 * q + (j & 3);
}
// Column of dW of row m (0..15) of fragment f: a lane's results of one (fp32) or two (bf16) fragments are 16
// bytes of a row.
template <typename E> __host__ __device__ constexpr int column_of(int f, int m)
{
    return Form<E>::kPlanes == 1 ? 32 * (f >> 1) + 8 * (m >> 2) + 4 * (f & 1) + (m & 3) : 16 * f + m;
}

template <int kPlanes> struct Planes {
    bf16x8 p[kPlanes];
};
template <typename E> using Frag = Planes<Form<E>::kPlanes>;    // of X or W
template <typename E> using PFrag = Planes<Form<E>::kPPlanes>;  // of P
// The 8 elements of a lane from floats.
template <int kPlanes>
__device__ __forceinline__ Planes<kPlanes> planes_of(const float (&x)[8])
{
    Planes<kPlanes> f;
    uint32_t w[kPlanes][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t p[kPlanes];
        if constexpr (kPlanes == 1) p[0] = pack_bf16(x[2 * i], x[2 * i + 1]);
        else split_pair(x[2 * i], x[2 * i + 1], p);
#pragma unroll
        for (int k = 0; k < kPlanes; ++k) w[k][i] = p[k];
    }
#pragma unroll
    for (int k = 0; k < kPlanes; ++k)
        f.p[k] = __builtin_bit_cast(bf16x8, u32x4{w[k][0], w[k][1], w[k][2], w[k][3]});
    return f;
}

__device__ __forceinline__ f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
// c += A B; of fp32 operands the six plane products above 2^-25 of the whole, small ones first.  P stands
// beside bf16 operands in two planes, 16 bits: rounded to 8 it would add to a gradient of few terms, as those
// of few tokens are, as much error again as the output's own rounding (one token: 0.0027 of the norm for 0.0016;
// 64: 0.0019 for 0.0017), and it costs 7 us of 523 at 64 tokens.  A third plane changed no digit of that error
// (64 tokens: 15 us more).
__device__ __forceinline__ f32x4 product(const Frag<BF16> &a, const Frag<BF16> &b, f32x4 c)
{
    return mma(a.p[0], b.p[0], c);
}
__device__ __forceinline__ f32x4 product(const Frag<BF16> &a, const PFrag<BF16> &b, f32x4 c)
{
    return mma(a.p[0], b.p[0], mma(a.p[0], b.p[1], c));
}
__device__ __forceinline__ f32x4 product(const Frag<F32> &a, const Frag<F32> &b, f32x4 c)
{
    c = mma(a.p[2], b.p[0], c);
    c = mma(a.p[0], b.p[2], c);
    c = mma(a.p[1], b.p[1], c);
    c = mma(a.p[1], b.p[0], c);
    c = mma(a.p[0], b.p[1], c);
    return mma(a.p[0], b.p[0], c);
}

// 16 bytes of a row from element k on, zeros from element D on.
template <typename E>
__device__ __forceinline__ u32x4 load_edge(const typename E::T *row, int64_t k, int64_t D)
{
    if (k + Form<E>::kPer <= D) return load16(row + k);
    u32x4 v{0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < Form<E>::kPer; ++i)
        if (k + i < D) {
            if constexpr (Form<E>::kPer == 8) v[i >> 1] |= (uint32_t)row[k + i] << (16 * (i & 1));
            else v[i] = __float_as_uint(row[k + i]);
        }
    return v;
}

// LDS and barriers without a wait for the global loads in flight, which the next step wants.
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// ---------------------------------------------------------------------------
// The tokens that take part, in order, and their rows of X as fragments:
//   Xf[step][block][plane]   rows: 16 tokens, depth: 32 columns   (logits)
//   Xt[frag][pair][plane]    rows: 16 columns, depth: 32 tokens   (dW; tokens 4 q + j, 16 + 4 q + j)
// Zeros for tokens past the list and columns past D.
// ---------------------------------------------------------------------------
struct FewList {
    int32_t *rows, *tgt, *slot, *count;
};

template <typename E, int NB>
__global__ __launch_bounds__(kFewThreads) void k_few_prep(const typename E::T *__restrict__ X,
                                                          const int64_t *__restrict__ targets, int N, int64_t V,
                                                          int64_t D, FewList list, u32x4 *__restrict__ Xf, int64_t nf,
                                                          u32x4 *__restrict__ Xt, int64_t nt,
                                                          float *__restrict__ loss, float *__restrict__ lse)
{
    constexpr int P = Form<E>::kPlanes, Q = (NB + 1) / 2;
    __shared__ int32_t rows[kFewMost];
    __shared__ int shared_count;
    if (threadIdx.x < 64) {
        int before = 0;
#pragma unroll
        for (int n = threadIdx.x; n < (NB > 4 ? 128 : 64); n += 64) {
            const int64_t t = n < N ? targets[n] : -1;
            const bool part = t >= 0 && t < V;
            const uint64_t mask = __ballot(part);
            const int at = before + __popcll(mask & lanes_below());
            if (part) rows[at] = n;
            if (blockIdx.x == 0) {
                if (part) {
                    list.rows[at] = n;
                    list.tgt[at] = (int32_t)t;
                }
                if (n < N) {
                    list.slot[n] = part ? at : -1;
                    if (!part && loss) loss[n] = lse[n] = 0.0f;
                }
            }
            before += __popcll(mask);
        }
        if (threadIdx.x == 0) {
            shared_count = before;
            if (blockIdx.x == 0) list.count[0] = before;
        }
    }
    __syncthreads();
    const int count = shared_count;
    const int64_t i = (int64_t)blockIdx.x * kFewThreads + threadIdx.x;
    const int l = (int)(i & 63), q = l >> 4;
    float x[8];
    u32x4 *dst;
    if (i < nf) {
        const int64_t sb = i >> 6, k = sb / NB * 32;
        const int n = (int)(sb % NB) * 16 + (l & 15);
        const typename E::T *row = X + (n < count ? rows[n] : 0) * D;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t c = k + depth_of<E>(q, j);
            x[j] = n < count && c < D ? E::load(row, c) : 0.0f;
        }
        dst = Xf + sb * P * 64 + l;
    } else if (i < nf + nt) {
        const int64_t fq = (i - nf) >> 6, c = column_of<E>((int)(fq / Q), l & 15);
        const int n0 = (int)(fq % Q) * 32;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int n = n0 + (j & 4) * 4 + 4 * q + (j & 3);
            x[j] = n < count && c < D ? E::load(X + rows[n] * D, c) : 0.0f;
        }
        dst = Xt + fq * P * 64 + l;
    } else {
        return;
    }
    const Frag<E> f = planes_of<P>(x);
#pragma unroll
    for (int p = 0; p < P; ++p) dst[p * 64] = __builtin_bit_cast(u32x4, f.p[p]);
}

// ---------------------------------------------------------------------------
// 128 vocabulary rows a workgroup.  The rows of a wave arrive 4 loads ahead in
// registers (8 KiB a wave), the tokens' fragments of a chunk through LDS (two
// buffers, one barrier a chunk).  Workgroups begin at different chunks: all rows
// are in work at once, and with a common stride their reads of one chunk meet
// in the same memory channels (one token, 65536 x 4096 bf16: 136 us in step, 99
// us, 5.4 TB/s, apart).
// ---------------------------------------------------------------------------
struct FewArgs {
    const int32_t *rows, *tgt, *count;
    const u32x4 *Xf, *Xt;
    int64_t V, D;
    // forward
    float2 *part;  // [workgroup][16 NB]: maximum and sum of exp(z - maximum)
    float *zt;
    // backward
    const float *lse, *dmean, *total;
    u32x4 *Pf;     // [vocabulary / 32][block][plane]: rows 16 tokens, depth 32 vocabulary rows 8 q + j
    float *others; // [token][workgroup]: sum of P besides the target
    float *pt;     // exp(z - lse) at the target
};

template <typename E, int NB, bool kBackward, bool kStream>
__global__ __launch_bounds__(kFewThreads, NB > 4 ? 1 : 2) void k_few_rows(FewArgs a, const typename E::T *__restrict__ W,
                                                             typename E::T *__restrict__ dW)
{
    using T = typename E::T;
    constexpr int P = Form<E>::kPlanes, S = Form<E>::kSteps, Q = (NB + 1) / 2, kPer = Form<E>::kPer;
    constexpr int kXChunk = S * NB * P * 64;                    // 16-byte vectors of a chunk of Xf
    constexpr int kXLoads = (kXChunk + kFewThreads - 1) / kFewThreads;
    constexpr int kFrags = kFewCols / 16;
    constexpr int kTChunk = kFrags * Q * P * 64, kTLoads = kTChunk / kFewThreads;
    constexpr int PP = Form<E>::kPPlanes, kPWave = NB * PP * 64;  // vectors of a wave's P
    constexpr int kLds = 2 * kXChunk > (kBackward ? (2 * kTChunk > 4 * kPWave ? 2 * kTChunk : 4 * kPWave) : 0)
                             ? 2 * kXChunk : (2 * kTChunk > 4 * kPWave ? 2 * kTChunk : 4 * kPWave);
    __shared__ u32x4 lds[kLds];
    __shared__ float2 join[kFewWaves][16 * NB];
    const int tid = threadIdx.x, l = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), q = l >> 4;
    const int64_t V = a.V, D = a.D, v0 = (int64_t)blockIdx.x * kFewRows + w * kWaveRows;
    const int64_t v[2] = {v0 + (l & 15), v0 + 16 + (l & 15)};  // the lane's vocabulary rows
    const T *row[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) row[b] = W + (v[b] < V ? v[b] : V - 1) * D;

    f32x4 acc[2][NB];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int t = 0; t < NB; ++t) acc[b][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // Up to 32 tokens: a chunk's products start from zero and are added with the lost digits carried along.  The
    // loss of a token or two shows each rounding of its logit; over more of them they average out.
    constexpr bool kExact = NB <= 2;
    f32x4 sum[2][NB], lost[2][NB];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int t = 0; t < NB; ++t) sum[b][t] = lost[b][t] = acc[b][t];
    const int chunks = (int)((D + kChunk<E> - 1) / kChunk<E>);
    const int turn = (int)((blockIdx.x >> 3) % (unsigned)chunks);
    auto chunk_of = [&](int c) { return c + turn < chunks ? c + turn : c + turn - chunks; };
    auto load_x = [&](int c, u32x4 (&x)[kXLoads]) {
#pragma unroll
        for (int i = 0; i < kXLoads; ++i) {
            const int e = i * kFewThreads + tid;
            x[i] = a.Xf[(int64_t)chunk_of(c) * kXChunk + (e < kXChunk ? e : 0)];
        }
    };
    auto put_x = [&](int c, const u32x4 (&x)[kXLoads]) {
#pragma unroll
        for (int i = 0; i < kXLoads; ++i) {
            const int e = i * kFewThreads + tid;
            if (kXChunk % kFewThreads == 0 || e < kXChunk) lds[(c & 1) * kXChunk + e] = x[i];
        }
    };
    auto load_w = [&](int c, u32x4 (&r)[2][4]) {
        const int64_t k0 = (int64_t)chunk_of(c) * kChunk<E>, k = k0 + kPer * q;
        const bool whole = k0 + kChunk<E> <= D;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t e = k + i * (kPer == 8 ? 32 : 16);
                if (!whole) r[b][i] = load_edge<E>(row[b], e, D);
                else if constexpr (kStream) r[b][i] = load16_nt(row[b] + e);
                else r[b][i] = load16(row[b] + e);
            }
    };
    auto multiply = [&](int c, const u32x4 (&r)[2][4]) {
        const u32x4 *x = lds + (c & 1) * kXChunk + l;
        if constexpr (kExact) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int t = 0; t < NB; ++t) acc[b][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            Frag<E> wf[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if constexpr (P == 1) {
                    wf[b].p[0] = __builtin_bit_cast(bf16x8, r[b][s]);
                } else {
                    float f[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(r[b][2 * s + (j >> 2)][j & 3]);
                    wf[b] = planes_of<P>(f);
                }
            }
#pragma unroll
            for (int t = 0; t < NB; ++t) {
                Frag<E> xf;
#pragma unroll
                for (int p = 0; p < P; ++p) xf.p[p] = __builtin_bit_cast(bf16x8, x[((s * NB + t) * P + p) * 64]);
#pragma unroll
                for (int b = 0; b < 2; ++b) acc[b][t] = product(xf, wf[b], acc[b][t]);
            }
        }
        if constexpr (kExact) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int t = 0; t < NB; ++t) {
                    const f32x4 y = acc[b][t] - lost[b][t], n = sum[b][t] + y;
                    const f32x4 off = (n - sum[b][t]) - y;
#pragma unroll
                    for (int r = 0; r < 4; ++r) lost[b][t][r] = fabsf(n[r]) < INFINITY ? off[r] : 0.0f;  // infinities stay
                    sum[b][t] = n;
                }
        }
    };
    {
        u32x4 x[kXLoads], r0[2][4], r1[2][4];
        load_x(0, x);
        load_w(0, r0);
        put_x(0, x);
        lds_barrier();
        for (int c = 0; c < chunks; c += 2) {
            const int c1 = c + 1 < chunks ? c + 1 : c, c2 = c + 2 < chunks ? c + 2 : c;
            load_x(c1, x);
            load_w(c1, r1);
            __builtin_amdgcn_sched_barrier(0);  // the next chunk's loads are under way before this one's products
            multiply(c, r0);
            if (c + 1 >= chunks) break;
            put_x(c1, x);
            lds_barrier();
            load_x(c2, x);
            load_w(c2, r0);
            __builtin_amdgcn_sched_barrier(0);
            multiply(c1, r1);
            put_x(c2, x);
            lds_barrier();
        }
        lds_barrier();  // LDS is free
        if constexpr (kExact) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int t = 0; t < NB; ++t) acc[b][t] = sum[b][t];
        }
    }

    const int count = a.count[0];
    if constexpr (!kBackward) {
#pragma unroll
        for (int t = 0; t < NB; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int n = 16 * t + 4 * q + r;
                const int64_t tgt = n < count ? a.tgt[n] : -1;
                float x[2], mx = -INFINITY, s = 0.0f;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    x[b] = v[b] < V ? acc[b][t][r] : -INFINITY;
                    if (v[b] == tgt) {  // kept apart (loss_of)
                        a.zt[n] = x[b];
                        x[b] = -INFINITY;
                    }
                    mx = fmaxf(mx, x[b]);
                }
#pragma unroll
                for (int off = 1; off < 16; off <<= 1) mx = fmaxf(mx, __shfl_xor(mx, off, 64));
                const float base = mx == -INFINITY ? 0.0f : mx;  // nothing of the vocabulary in this wave
#pragma unroll
                for (int b = 0; b < 2; ++b) s += exp_of(x[b] - base);
#pragma unroll
                for (int off = 1; off < 16; off <<= 1) s += __shfl_xor(s, off, 64);
                if ((l & 15) == 0) join[w][n] = make_float2(mx, s);
            }
        __syncthreads();
        if (tid < 16 * NB) {
            float mx = -INFINITY, s = 0.0f;
            for (int i = 0; i < kFewWaves; ++i) mx = fmaxf(mx, join[i][tid].x);
            const float base = mx == -INFINITY ? 0.0f : mx;
            for (int i = 0; i < kFewWaves; ++i) s += join[i][tid].y * exp_of(join[i][tid].x - base);
            a.part[(int64_t)blockIdx.x * (16 * NB) + tid] = make_float2(mx, s);
        }
    } else {
        // P without the targets' elements (k_few_targets), its sums, and its planes: pf[b][pair] with tokens as depth
        PFrag<E> pf[2][Q];
        float others[4 * NB] = {};
        uint16_t *mine = (uint16_t *)(lds + w * kPWave);
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int u = 0; u < Q; ++u) {
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int t = 2 * u + (j >> 2), n = 16 * t + 4 * q + (j & 3);
                    x[j] = 0.0f;
                    if (t < NB && n < count && v[b] < V) {
                        x[j] = exp_of(acc[b][t < NB ? t : 0][j & 3] - a.lse[a.rows[n]]);
                        if (v[b] == a.tgt[n]) {
                            a.pt[n] = x[j];
                            x[j] = 0.0f;
                        }
                        others[4 * (t < NB ? t : 0) + (j & 3)] += x[j];
                    }
                }
                pf[b][u] = planes_of<PP>(x);
                // the same with vocabulary rows as depth, for dX
#pragma unroll
                for (int p = 0; p < PP; ++p) {
                    const u32x4 y = __builtin_bit_cast(u32x4, pf[b][u].p[p]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int t = 2 * u + (j >> 2);
                        if (t >= NB) continue;
                        const int vl = 16 * b + (l & 15), to = 4 * q + (j & 3) + 16 * (vl >> 3);
                        mine[((t * PP + p) * 64 + to) * 8 + (vl & 7)] = (uint16_t)(y[j >> 1] >> (16 * (j & 1)));
                    }
                }
            }
#pragma unroll
        for (int i = 0; i < 4 * NB; ++i) {
#pragma unroll
            for (int off = 1; off < 16; off <<= 1) others[i] += __shfl_xor(others[i], off, 64);
            if ((l & 15) == 0) join[w][16 * (i >> 2) + 4 * q + (i & 3)].x = others[i];
        }
        lds_barrier();
        if (tid < 16 * NB)
            a.others[(int64_t)tid * gridDim.x + blockIdx.x] = join[0][tid].x + join[1][tid].x + join[2][tid].x + join[3][tid].x;
        u32x4 *out = a.Pf + ((int64_t)blockIdx.x * kFewWaves + w) * kPWave + l;
#pragma unroll
        for (int i = 0; i < NB * PP; ++i) out[i * 64] = lds[w * kPWave + i * 64 + l];
        lds_barrier();

        if (!dW) return;
        // dW[v][c] = scale * sum over tokens of X[n][c] P[n][v], 64 columns at a time
        const float scale = grad_scale(a.dmean, a.total);
        const int steps = (int)((D + kFewCols - 1) / kFewCols);
        u32x4 x[kTLoads];
        auto load_t = [&](int c) {
#pragma unroll
            for (int i = 0; i < kTLoads; ++i) x[i] = a.Xt[(int64_t)c * kTChunk + i * kFewThreads + tid];
        };
        auto put_t = [&](int c) {
#pragma unroll
            for (int i = 0; i < kTLoads; ++i) lds[(c & 1) * kTChunk + i * kFewThreads + tid] = x[i];
        };
        load_t(0);
        put_t(0);
        lds_barrier();
        for (int c = 0; c < steps; ++c) {
            load_t(c + 1 < steps ? c + 1 : c);
            __builtin_amdgcn_sched_barrier(0);
            const u32x4 *xt = lds + (c & 1) * kTChunk + l;
            f32x4 y[2][kFrags];
#pragma unroll
            for (int f = 0; f < kFrags; ++f) {
#pragma unroll
                for (int b = 0; b < 2; ++b) y[b][f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int u = 0; u < Q; ++u) {
                    Frag<E> xf;
#pragma unroll
                    for (int p = 0; p < P; ++p) xf.p[p] = __builtin_bit_cast(bf16x8, xt[((f * Q + u) * P + p) * 64]);
#pragma unroll
                    for (int b = 0; b < 2; ++b) y[b][f] = product(xf, pf[b][u], y[b][f]);
                }
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if (v[b] >= V) continue;
                T *o = dW + v[b] * D;
#pragma unroll
                for (int f = 0; f < kFrags; f += kPer / 4) {
                    const int64_t col = (int64_t)c * kFewCols + column_of<E>(f, 4 * q);
                    u32x4 z;
                    if constexpr (kPer == 8) {
                        z = u32x4{pack_bf16(y[b][f][0] * scale, y[b][f][1] * scale),
                                  pack_bf16(y[b][f][2] * scale, y[b][f][3] * scale),
                                  pack_bf16(y[b][f + 1][0] * scale, y[b][f + 1][1] * scale),
                                  pack_bf16(y[b][f + 1][2] * scale, y[b][f + 1][3] * scale)};
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r) z[r] = __float_as_uint(y[b][f][r] * scale);
                    }
                    if (col + kPer <= D) {
                        store16(o + col, z);
                    } else {
#pragma unroll
                        for (int i = 0; i < kPer; ++i)
                            if (col + i < D) {
                                if constexpr (kPer == 8) o[col + i] = (uint16_t)(z[i >> 1] >> (16 * (i & 1)));
                                else o[col + i] = __uint_as_float(z[i]);
                            }
                    }
                }
            }
            put_t(c + 1);
            lds_barrier();
        }
    }
}

// The targets' elements of P, put into Pf, and the rows of dW that they are in, written anew: a token's
// element takes the sum of all its others (target_of), which a workgroup of k_few_rows does not have.  One workgroup for 256 columns of the row of the first token of each target; it is bound by the
// latency of its loads, tens of KiB of P and X from L2 (32 tokens, width 768 fp32: 6 us; 64, 4096 bf16: 12).
template <typename E, int NB>
__global__ __launch_bounds__(kFewThreads) void k_few_targets(FewArgs a, const typename E::T *__restrict__ X, int64_t tiles,
                                                             typename E::T *__restrict__ dW)
{
    constexpr int PP = Form<E>::kPPlanes, kMost = 16 * NB, kAhead = 16;
    __shared__ float p[kMost];
    __shared__ int32_t from[kMost], tgt[kMost];
    const int cnt = a.count[0], m = blockIdx.x % kMost, tid = threadIdx.x, l = tid & 63, w = tid >> 6;
    const int64_t D = a.D, c0 = (int64_t)(blockIdx.x / kMost) * kFewThreads;
    if (m >= cnt) return;
    if (tid < kMost) {
        from[tid] = a.rows[tid < cnt ? tid : m];
        tgt[tid] = tid < cnt ? a.tgt[tid] : -1;
    }
    __syncthreads();
    const int32_t v = tgt[m];
    if (__syncthreads_or(tid < m && tgt[tid] == v)) return;
    // P[k][v] of Pf: tokens k, plane pl
    uint16_t *column = (uint16_t *)(a.Pf + (int64_t)(v >> 5) * (NB * PP * 64) + 16 * (v >> 3 & 3)) + (v & 7);
    auto place = [&](int k, int pl) { return (((k >> 4) * PP + pl) * 64 + (k & 15)) * 8; };
    if (tid < kMost && tgt[tid] != v) {
        float s = 0.0f;
        if (tid < cnt)
#pragma unroll
            for (int pl = PP - 1; pl >= 0; --pl) s += __uint_as_float((uint32_t)column[place(tid, pl)] << 16);
        p[tid] = s;
    }
    for (int k = m + w; k < cnt; k += kFewWaves) {  // the same sum in each of the row's workgroups
        if (tgt[k] != v) continue;
        float s = 0.0f;
        for (int64_t t = l; t < tiles; t += 64 * kAhead) {
            float x[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) x[j] = t + 64 * j < tiles ? a.others[k * tiles + t + 64 * j] : 0.0f;
#pragma unroll
            for (int j = 0; j < kAhead; ++j) s += x[j];
        }
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) s += __shfl_xor(s, off, 64);
        if (l == 0) p[k] = target_of(a.pt[k], s);
    }
    __syncthreads();
    if (c0 == 0 && tid < kMost && tgt[tid] == v) {
        uint32_t planes[PP];
        split_pair(p[tid], 0.0f, planes);
#pragma unroll
        for (int pl = 0; pl < PP; ++pl) column[place(tid, pl)] = (uint16_t)planes[pl];
    }
    const int64_t c = c0 + tid;
    if (c >= D || !dW) return;
    float s = 0.0f;
    for (int k = 0; k < cnt; k += kAhead) {  // past the list: P 0 beside a row that takes part
        float x[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) x[j] = E::load(X, from[k + j] * D + c);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) s = fmaf(p[k + j], x[j], s);
    }
    dW[v * D + c] = E::from_f(s * grad_scale(a.dmean, a.total));
}

// Joins the workgroups' maxima and sums, and adds the losses up.  One workgroup.
template <int NB>
__global__ __launch_bounds__(1024) void k_few_join(const float2 *__restrict__ part, const float *__restrict__ zt,
                                                   const int32_t *__restrict__ rows,
                                                   const int32_t *__restrict__ count, int64_t tiles,
                                                   float *__restrict__ loss, float *__restrict__ lse,
                                                   float *__restrict__ total)
{
    constexpr int kTokens = 16 * NB, kGroups = 1024 / kTokens;
    __shared__ float2 join[kGroups][kTokens];
    const int n = threadIdx.x % kTokens, g = threadIdx.x / kTokens, cnt = count[0];
    float mx = -INFINITY, s = 0.0f;
    constexpr int kAhead = 4;
    for (int64_t t = g; t < tiles; t += kAhead * kGroups) {
        float2 p[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int64_t u = t + j * kGroups;
            p[j] = part[(u < tiles ? u : t) * kTokens + n];
            if (u >= tiles) p[j] = make_float2(-INFINITY, 0.0f);
        }
        float up = mx;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) up = fmaxf(up, p[j].x);
        const float base = up == -INFINITY ? 0.0f : up;
        s *= exp_of(mx - base);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) s += p[j].y * exp_of(p[j].x - base);
        mx = up;
    }
    join[g][n] = make_float2(mx, s);
    for (int half = kGroups / 2; half >= 1; half /= 2) {
        __syncthreads();
        if (g < half) {
            const float2 a = join[g][n], b = join[g + half][n];
            const float up = fmaxf(a.x, b.x), base = up == -INFINITY ? 0.0f : up;
            join[g][n] = make_float2(up, a.y * exp_of(a.x - base) + b.y * exp_of(b.x - base));
        }
    }
    __syncthreads();
    if (threadIdx.x >= 64) return;
    double l = 0.0;
    for (int m = threadIdx.x; m < kTokens && m < cnt; m += 64) {
        const float2 r = loss_of(join[0][m].x, join[0][m].y, zt[m]);
        lse[rows[m]] = r.x;
        loss[rows[m]] = r.y;
        l += r.y;
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) l += __shfl_xor(l, off, 64);
    if (threadIdx.x == 0) {
        total[0] = (float)l;
        total[1] = (float)cnt;
        total[2] = (float)(l / (double)(cnt > 0 ? cnt : 1));
    }
}

// ---------------------------------------------------------------------------
// dX: acc[split][n][c] = sum over a split's vocabulary rows of P[n, v] W[v, c].
// A lane loads 16 bytes of each of 8 rows: as columns of 8 they are the operand
// (bf16: after a transpose of 8 x 8 in registers), with the columns dealt
// to fragments by their place in the 16 bytes.  The waves of a workgroup take
// a quarter of the split each and add up through LDS.
// ---------------------------------------------------------------------------
template <typename E> constexpr int kDxCols = 16 * Form<E>::kPer;  // columns of a workgroup

struct FewDx {
    const u32x4 *Pf;
    int64_t V, D;
    int splits, per;  // per: vocabulary rows of a wave, a multiple of 32
    float *acc;
    int64_t lda, plane;
};

template <typename E, int NB>
__global__ __launch_bounds__(kFewThreads, NB >= 4 ? 1 : 2) void k_few_dx(FewDx a, const typename E::T *__restrict__ W)
{
    using T = typename E::T;
    constexpr int P = Form<E>::kPlanes, PP = Form<E>::kPPlanes, kPer = Form<E>::kPer, C = kDxCols<E>, kStride = C + 4;
    __shared__ __attribute__((aligned(16))) float sum[kFewWaves][16][kStride];
    const int tid = threadIdx.x, l = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), q = l >> 4;
    // workgroups go round the 8 XCDs and splits are a multiple of 8: all columns of a split meet its P in one L2
    const int split = blockIdx.x % a.splits, cg = blockIdx.x / a.splits;
    const int64_t V = a.V, D = a.D, c0 = (int64_t)cg * C, col = c0 + kPer * (l & 15);
    const bool edge = c0 + C > D;
    const int64_t first = ((int64_t)split * kFewWaves + w) * a.per;
    const int steps = first < V ? (int)(((V - first < a.per ? V - first : a.per) + 31) / 32) : 0;
    const int64_t rowbytes = D * (int64_t)sizeof(T);
    const uint32_t lane_off = (uint32_t)(8 * q) * (uint32_t)rowbytes + 16 * (l & 15);
    f32x4 acc[kPer][NB];
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
        for (int t = 0; t < NB; ++t) acc[i][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto load_p = [&](int64_t v, u32x4 (&p)[NB * PP]) {
        const char *ps = (const char *)(a.Pf + (v >> 5) * (NB * PP * 64));
#pragma unroll
        for (int i = 0; i < NB * PP; ++i) p[i] = *(const u32x4 *)(ps + (uint32_t)(l * 16) + i * 1024);
    };
    // a row's address is a scalar, with one offset a lane for all
    auto load = [&](int s, u32x4 (&r)[8], u32x4 (&p)[NB * PP]) {
        const int64_t v = first + 32 * (int64_t)s;
        load_p(v, p);
        const char *ws = (const char *)(W + v * D + c0);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = load16(ws + j * rowbytes + lane_off);
    };
    auto load_guarded = [&](int s, u32x4 (&r)[8], u32x4 (&p)[NB * PP]) {
        const int64_t v = first + 32 * (int64_t)s;
        load_p(v, p);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t u = v + 8 * q + j;
            r[j] = load_edge<E>(W + (u < V ? u : V - 1) * D, col, D);  // P is 0 past V
        }
    };
    auto multiply = [&](const u32x4 (&r)[8], const u32x4 (&p)[NB * PP]) {
        PFrag<E> pf[NB];
#pragma unroll
        for (int t = 0; t < NB; ++t)
#pragma unroll
            for (int k = 0; k < PP; ++k) pf[t].p[k] = __builtin_bit_cast(bf16x8, p[t * PP + k]);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            Frag<E> wf;
            if constexpr (P == 1) {
                u32x4 x;
#pragma unroll
                for (int h = 0; h < 4; ++h)  // halves i & 1 of word i / 2 of rows 2 h and 2 h + 1
                    x[h] = __builtin_amdgcn_perm(r[2 * h + 1][i >> 1], r[2 * h][i >> 1], i & 1 ? 0x07060302u : 0x05040100u);
                wf.p[0] = __builtin_bit_cast(bf16x8, x);
            } else {
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(r[j][i]);
                wf = planes_of<P>(f);
            }
#pragma unroll
            for (int t = 0; t < NB; ++t) acc[i][t] = product(wf, pf[t], acc[i][t]);
        }
    };
    u32x4 r0[8], r1[8], p0[NB * PP], p1[NB * PP];
    const int whole = edge ? 0 : first + 32 * (int64_t)steps <= V ? steps : steps - 1;  // steps without a guard
    if (whole > 0) {
        load(0, r0, p0);
        for (int s = 0; s < whole; s += 2) {
            load(s + 1 < whole ? s + 1 : s, r1, p1);
            __builtin_amdgcn_sched_barrier(0);
            multiply(r0, p0);
            if (s + 1 >= whole) break;
            load(s + 2 < whole ? s + 2 : s, r0, p0);
            __builtin_amdgcn_sched_barrier(0);
            multiply(r1, p1);
        }
    }
    for (int s = whole < 0 ? 0 : whole; s < steps; ++s) {
        load_guarded(s, r0, p0);
        multiply(r0, p0);
    }
    // token l % 16 of block t, columns kPer (4 q + r) + i
#pragma unroll
    for (int t = 0; t < NB; ++t) {
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int i = 0; i < kPer; i += 4)
                *(f32x4 *)&sum[w][l & 15][kPer * (4 * q + r) + i] =
                    f32x4{acc[i][t][r], acc[i + 1][t][r], acc[i + 2][t][r], acc[i + 3][t][r]};
        __syncthreads();
        for (int e = tid; e < 16 * C / 4; e += kFewThreads) {
            const int n = e / (C / 4), c = e % (C / 4) * 4;
            f32x4 s = *(const f32x4 *)&sum[0][n][c];
#pragma unroll
            for (int i = 1; i < kFewWaves; ++i) s += *(const f32x4 *)&sum[i][n][c];
            *(f32x4 *)(a.acc + split * a.plane + (16 * t + n) * a.lda + c0 + c) = s;
        }
    }
}

struct FewPlan {
    int nb, splits, per;
    int64_t steps, frags, tiles, lda;  // depth steps of 32 of Xf, fragments of Xt, workgroups of 128 rows
    size_t rows, tgt, slot, count, Xf, Xt, part, zt, Pf, others, pt, acc, total;
};

FewPlan few_plan(int64_t N, int64_t V, int64_t D, int dtype, bool backward)
{
    FewPlan p{};
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t r = at;
        at += (size_t)round_up(bytes, 256);
        return r;
    };
    const int planes = dtype == CSP_F32 ? 3 : 1;
    p.nb = N <= 16 ? 1 : N <= 32 ? 2 : N <= 64 ? 4 : 8;
    p.steps = round_up(D, dtype == CSP_F32 ? kChunk<F32> : kChunk<BF16>) / 32;
    p.tiles = ceil_div(V, kFewRows);
    p.rows = take(4 * kFewMost);
    p.tgt = take(4 * kFewMost);
    p.slot = take(4 * kFewMost);
    p.count = take(4);
    p.Xf = take(p.steps * p.nb * planes * 1024);
    if (!backward) {
        p.part = take(p.tiles * 16 * p.nb * 8);
        p.zt = take(4 * kFewMost);
    } else {
        const int64_t cols = dtype == CSP_F32 ? kDxCols<F32> : kDxCols<BF16>, groups = ceil_div(D, cols);
        p.frags = round_up(D, kFewCols) / 16;
        p.Xt = take(p.frags * ((p.nb + 1) / 2) * planes * 1024);
        p.Pf = take(p.tiles * kFewWaves * p.nb * (dtype == CSP_F32 ? 3 : 2) * 1024);
        p.others = take(p.tiles * 16 * p.nb * 4);
        p.pt = take(4 * kFewMost);
        // about two workgroups a CU; a wave has at least one step of 32 rows
        int64_t s = round_up(ceil_div(512, groups), 8);
        if (s > 128) s = 128;
        if (s > round_up(p.tiles, 8)) s = round_up(p.tiles, 8);
        p.splits = (int)s;
        p.per = (int)round_up(ceil_div(V, s * kFewWaves), 32);
        p.lda = groups * cols;
        p.acc = take(s * 16 * p.nb * p.lda * 4);
    }
    p.total = at;
    return p;
}

template <typename E, int NB>
csp_status few_begin(const FewPlan &p, const void *X, const int64_t *targets, int64_t N, int64_t V, int64_t D,
                     bool backward, float *loss, float *lse, char *w, hipStream_t s)
{
    const FewList list{(int32_t *)(w + p.rows), (int32_t *)(w + p.tgt), (int32_t *)(w + p.slot), (int32_t *)(w + p.count)};
    const int64_t nf = p.steps * NB * 64, nt = backward ? p.frags * ((NB + 1) / 2) * 64 : 0;
    k_few_prep<E, NB><<<(unsigned)ceil_div(nf + nt, kFewThreads), kFewThreads, 0, s>>>(
        (const typename E::T *)X, targets, (int)N, V, D, list, (u32x4 *)(w + p.Xf), nf, (u32x4 *)(w + p.Xt), nt, loss, lse);
    CSP_LAUNCHED("k_few_prep");
    return CSP_OK;
}

FewArgs few_args(const FewPlan &p, int64_t V, int64_t D, char *w)
{
    FewArgs a{};
    a.rows = (const int32_t *)(w + p.rows);
    a.tgt = (const int32_t *)(w + p.tgt);
    a.count = (const int32_t *)(w + p.count);
    a.Xf = (const u32x4 *)(w + p.Xf);
    a.Xt = (const u32x4 *)(w + p.Xt);
    a.V = V;
    a.D = D;
    return a;
}

template <typename E, int NB>
csp_status fwd_few(const void *X, const void *W, const int64_t *targets, int64_t N, int64_t V, int64_t D, float *loss,
                   float *lse, float *total, char *w, hipStream_t s)
{
    const FewPlan p = few_plan(N, V, D, Form<E>::kPlanes == 3 ? CSP_F32 : CSP_BF16, false);
    csp_status st = few_begin<E, NB>(p, X, targets, N, V, D, false, loss, lse, w, s);
    if (st != CSP_OK) return st;
    FewArgs a = few_args(p, V, D, w);
    a.part = (float2 *)(w + p.part);
    a.zt = (float *)(w + p.zt);
    if (N > 0) {
        k_few_rows<E, NB, false, false><<<(unsigned)p.tiles, kFewThreads, 0, s>>>(a, (const typename E::T *)W, nullptr);
        CSP_LAUNCHED("k_few_rows");
    }
    k_few_join<NB><<<1, 1024, 0, s>>>(a.part, a.zt, a.rows, a.count, N > 0 ? p.tiles : 0, loss, lse, total);
    CSP_LAUNCHED("k_few_join");
    return CSP_OK;
}

template <typename E, int NB>
csp_status bwd_few(const void *X, const void *W, const int64_t *targets, int64_t N, int64_t V, int64_t D,
                   const float *lse, const float *dmean, const float *total, void *dX, void *dW, char *w, hipStream_t s)
{
    using T = typename E::T;
    const FewPlan p = few_plan(N, V, D, Form<E>::kPlanes == 3 ? CSP_F32 : CSP_BF16, true);
    csp_status st = few_begin<E, NB>(p, X, targets, N, V, D, true, nullptr, nullptr, w, s);
    if (st != CSP_OK) return st;
    FewArgs a = few_args(p, V, D, w);
    a.lse = lse;
    a.dmean = dmean;
    a.total = total;
    a.Pf = (u32x4 *)(w + p.Pf);
    a.others = (float *)(w + p.others);
    a.pt = (float *)(w + p.pt);
    // A bf16 W past the memory-side cache (256 MB) is not there for k_few_dx anyway, and streaming it leaves the
    // cache to dW (64 tokens, width 4096, step plain / streamed, us: 164 MB 251 / 256, 213 MB 282 / 283, 246 MB 308 /
    // 300, 270 MB 433 / 412, 344 MB 456 / 434, 537 MB 581 / 559).  An fp32 W gains nothing (32 tokens, 154 MB 175 /
    // 188, 281 MB 397 / 410, 412 MB 459 / 461; 128 tokens, 322 MB 764 / 765).
    constexpr bool kMayStream = Form<E>::kPlanes == 1;
    if (kMayStream && V * D * (int64_t)sizeof(T) > (int64_t)256 << 20)
        k_few_rows<E, NB, true, kMayStream><<<(unsigned)p.tiles, kFewThreads, 0, s>>>(a, (const T *)W, (T *)dW);
    else
        k_few_rows<E, NB, true, false><<<(unsigned)p.tiles, kFewThreads, 0, s>>>(a, (const T *)W, (T *)dW);
    CSP_LAUNCHED("k_few_rows");
    if (N == 0) return CSP_OK;
    k_few_targets<E, NB><<<(unsigned)(16 * NB * (dW ? ceil_div(D, kFewThreads) : 1)), kFewThreads, 0, s>>>(
        a, (const T *)X, p.tiles, (T *)dW);
    CSP_LAUNCHED("k_few_targets");
    if (!dX) return CSP_OK;
    const FewDx d{a.Pf, V, D, p.splits, p.per, (float *)(w + p.acc), p.lda, 16 * NB * p.lda};
    k_few_dx<E, NB><<<(unsigned)(p.splits * ceil_div(D, kDxCols<E>)), kFewThreads, 0, s>>>(d, (const T *)W);
    CSP_LAUNCHED("k_few_dx");
    k_ce_out<E><<<out_blocks(N, D), 256, 0, s>>>(d.acc, p.lda, d.plane, p.splits, (const int32_t *)(w + p.slot), N, D,
                                                 dmean, total, (T *)dX);
    CSP_LAUNCHED("k_ce_out");
    return CSP_OK;
}

}  // namespace

size_t ce_few_bytes(int64_t N, int64_t V, int64_t D, int dtype, bool backward)
{
    return few_plan(N, V, D, dtype, backward).total;
}

csp_status ce_few_fwd(const void *X, const void *W, const int64_t *targets, int64_t N, int64_t V, int64_t D, int dtype,
                      float *loss, float *lse, float *total, char *work, hipStream_t s)
{
    auto run = dtype == CSP_BF16 ? (N <= 16 ? fwd_few<BF16, 1> : N <= 32 ? fwd_few<BF16, 2> : fwd_few<BF16, 4>)
                                 : (N <= 16 ? fwd_few<F32, 1> : N <= 32 ? fwd_few<F32, 2> : N <= 64 ? fwd_few<F32, 4>
                                                                                                  : fwd_few<F32, 8>);
    return run(X, W, targets, N, V, D, loss, lse, total, work, s);
}

csp_status ce_few_bwd(const void *X, const void *W, const int64_t *targets, int64_t N, int64_t V, int64_t D, int dtype,
                      const float *lse, const float *dmean, const float *total, void *dX, void *dW, char *work,
                      hipStream_t s)
{
    auto run = dtype == CSP_BF16 ? (N <= 16 ? bwd_few<BF16, 1> : N <= 32 ? bwd_few<BF16, 2> : bwd_few<BF16, 4>)
                                 : (N <= 16 ? bwd_few<F32, 1> : N <= 32 ? bwd_few<F32, 2> : N <= 64 ? bwd_few<F32, 4>
                                                                                                  : bwd_few<F32, 8>);
    return run(X, W, targets, N, V, D, lse, dmean, total, dX, dW, work, s);
}

}  // namespace csp
