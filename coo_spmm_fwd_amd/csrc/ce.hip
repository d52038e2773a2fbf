// ce.hip -- softmax cross entropy over a large vocabulary, fused with the
// product that makes the logits, and its gradient.
//
//   z[n, v] = sum_c X[n, c] W[v, c]
//   lse[n]  = log sum_v exp z[n, v] = m + log sum_v exp(z[n, v] - m)
//   loss[n] = lse[n] - z[n, t_n], from the target's logit and the sum of the others (loss_of in ce.h)
//   G[n, v] = (exp(z[n, v] - lse[n]) - [v = t_n]) * dmean / count
//   dX = G W,  dW = G^T X
//
// A token whose target is outside [0, V) takes no part: loss, lse and its row
// of dX are 0 and it adds nothing to dW, whatever its row of X holds.  The
// tokens that take part are listed first (k_ce_rows) and their rows of X
// gathered (k_ce_gather); every product runs over that list alone, so masked
// tokens cost nothing.  The logits are not stored: the forward keeps a
// maximum and a sum for each (vocabulary tile, token); the backward recomputes
// the logits, a piece of the vocabulary at a time, from the saved lse, and
// keeps P = exp(z - lse) - [v = t] of that piece only; P at the target takes the
// sum of the others (target_of in ce.h).  (A small vocabulary
// times few tokens makes too few tiles for 256 CUs: there the width is cut,
// and the parts' logits, a few MiB in the workspace, are read once more.)
//
// All three products run on the tile product of mfma_tile.h, each with the
// dimension that is contiguous in its output as m, so that a lane holds 4
// neighbours of an output row:
//   logits  m = vocabulary, n = token,      k = width       (W and X by rows)
//   dX      m = width,      n = token,      k = vocabulary  (W by depth, P by rows)
//   dW      m = width,      n = vocabulary, k = token       (X and P by depth)
// P enters the gradient products as bf16 planes: beside bf16 operands two, off by
// 2^-16 of each term at most, 1/256 of the rounding of the outputs.  Rounded to bf16
// alone it put the gradients off by 0.0019 of their norm where the outputs' rounding
// is 0.0017, and a step took two thirds of the time (8192 tokens 13.7 for 20.6 ms).
// The scale dmean / count is applied to the fp32 sums.  In fp32, X, W and P are split
// into three bf16 planes (mfma_tile.h).
//
// Measured, 8192 tokens, 65536 x 4096 bf16 (4.4 TFLOP a product): forward
// logits 3.40 ms (1290 TFLOP/s), backward logits 3.70 (1190), dX 7.02 and dW 6.75
// for two products each (1250, 1300); the library's plain product of that shape
// reaches 1485.  The matrix units are busy 68% of the forward's cycles and 61 to 62%
// of the backward's, at 1.8 to 2.0 GHz.  fp32 at 2048 tokens, 30000 x 1024: 2.65 ms a step,
// 190 TFLOP/s of fp32 (1140 of bf16 products).
//
// Up to 64 tokens (128 in fp32) go to ce_few.hip, where the products are bound by
// the bytes of W.  A step here / there, us: 64 tokens bf16, 65536 x 4096 784 / 558 and
// 30000 x 1024 129 / 114; 32 fp32, 50257 x 768 523 / 175; 30000 x 1024 fp32, 65 tokens 474 /
// 284 and 128 tokens 475 / 296.  Past them, 30000 x 1024, 65 bf16 take 136, 129 fp32 502.
#include "ce.h"
#include "mfma_tile.h"

namespace csp {
namespace {

constexpr int kCeThreads = 256;
constexpr int kBM = 256;       // vocabulary rows (or columns of X) of a tile
constexpr int64_t kPad = 256;  // token and vocabulary strides are multiples of it
// fp32 or bf16 elements as bf16 planes.
template <typename E> struct Split;
template <> struct Split<BF16> {
    static constexpr bool kMany = false;
};
template <> struct Split<F32> {
    static constexpr bool kMany = true;
};
// Plane products of the logits, and of the gradients; planes of P.
template <bool kMany> constexpr int kLogitProducts = kMany ? kPlaneProducts : 1;
template <bool kMany> constexpr int kGradProducts = kMany ? kPlaneProducts : 2;
template <bool kMany> constexpr int kPPlanes = kMany ? kPlanes : 2;
// Tokens that take part, in order: rows[0 .. count) and their targets tgt; slot[n] = place in that
// list, or -1.  Clears loss and lse (if given) of the others.  One workgroup.
__global__ __launch_bounds__(1024) void k_ce_rows(const int64_t *__restrict__ targets, int64_t N, int64_t V,
                                                  int32_t *__restrict__ rows, int32_t *__restrict__ tgt,
                                                  int32_t *__restrict__ slot, int32_t *__restrict__ count,
                                                  float *__restrict__ loss, float *__restrict__ lse)
{
    __shared__ uint32_t lds[17];
    uint32_t run = 0;
    for (int64_t base = 0; base < N; base += 1024) {
        const int64_t i = base + threadIdx.x;
        const int64_t t = i < N ? targets[i] : -1;
        const bool part = t >= 0 && t < V;
        uint32_t total;
        const uint32_t at = block_exclusive_scan(part ? 1u : 0u, lds, &total);
        if (part) {
            rows[run + at] = (int32_t)i;
            tgt[run + at] = (int32_t)t;
        }
        if (i < N) {
            slot[i] = part ? (int32_t)(run + at) : -1;
            if (!part && loss) loss[i] = lse[i] = 0.0f;
        }
        run += total;
    }
    if (threadIdx.x == 0) count[0] = (int32_t)run;
}

// dst[plane][r][0 .. ld) = planes of src row (rows ? rows[r] : r), zeros past D; with `rows`, rows
// from count up to the next multiple of 64 are zeros (the depth of dW).  One workgroup a row.
template <typename E>
__global__ __launch_bounds__(kCeThreads) void k_ce_gather(const typename E::T *__restrict__ src, int64_t D,
                                                          const int32_t *__restrict__ rows,
                                                          const int32_t *__restrict__ count,
                                                          uint16_t *__restrict__ dst, int64_t ld, int64_t plane)
{
    const int64_t r = blockIdx.x;
    bool real = true;
    if (rows) {
        const int64_t cnt = count[0];
        if (r >= round_up(cnt, kDepth)) return;
        real = r < cnt;
    }
    const int64_t from = real ? (rows ? rows[r] : r) : 0;
    for (int64_t c = threadIdx.x * 8; c < ld; c += kCeThreads * 8) {  // ld is a multiple of 64
        const typename E::T *p = src + from * D + c;
        u32x4 out[kPlanes];
        if constexpr (Split<E>::kMany) {
            float x[8];
            if (real && c + 8 <= D) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const u32x4 v = load16(p + 4 * h);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[4 * h + i] = __uint_as_float(v[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = real && c + i < D ? p[i] : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t q[kPlanes];
                split_pair(x[2 * i], x[2 * i + 1], q);
#pragma unroll
                for (int k = 0; k < kPlanes; ++k) out[k][i] = q[k];
            }
        } else {
            out[0] = u32x4{0u, 0u, 0u, 0u};
            if (real && c + 8 <= D) {
                out[0] = load16(p);
            } else if (real) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c + i < D) out[0][i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
            }
        }
#pragma unroll
        for (int k = 0; k < (Split<E>::kMany ? kPlanes : 1); ++k) *(u32x4 *)(dst + k * plane + r * ld + c) = out[k];
    }
}

// The place of a workgroup in a grid of mt x nt tiles (and `splits` of the depth).  Workgroups go
// round the 8 XCDs; each XCD takes one contiguous run of tiles, walked in columns 4 tiles wide, so
// that the tiles an XCD holds at a time share operands in its L2.
struct TilePlace {
    int64_t m, n, split;
    bool ok;
};
__device__ __forceinline__ TilePlace tile_place(int64_t mt, int64_t nt, int64_t splits)
{
    const int64_t total = mt * nt * splits, b = blockIdx.x;
    TilePlace t{0, 0, 0, b < total};
    if (!t.ok) return t;
    const int64_t x = b & 7, q = total >> 3, r = total & 7;
    int64_t id = x * q + (x < r ? x : r) + (b >> 3);
    t.split = id / (mt * nt);
    id -= t.split * (mt * nt);
    const int64_t grp = id / (mt * 4), rem = id - grp * mt * 4, width = nt - grp * 4 < 4 ? nt - grp * 4 : 4;
    t.m = rem / width;
    t.n = grp * 4 + rem % width;
    return t;
}

// Waves of a tile of 256 x BN: 2 x 4, or 4 x 2 for 128 tokens.
template <int BN> constexpr int kWavesM = BN == 256 ? 2 : 4;
template <int BN> constexpr int kWavesN = kTileWaves / kWavesM<BN>;

struct Logits {
    const uint16_t *X, *W;  // planes: listed tokens [.][ldx], vocabulary rows of the piece [.][ldw]
    int64_t ldx, ldw, planex, planew;
    const int32_t *tgt, *count;
    int64_t nv, v0, npad;   // vocabulary rows of the piece, its first, token stride
    int64_t depth;
};

// Runs the logits tile of this workgroup; false if it has none.
template <int BN, bool kMany, typename T>
__device__ __forceinline__ bool logits_tile(const Logits &a, T &tile, TilePlace &at, char *smem)
{
    at = tile_place(ceil_div(a.nv, kBM), ceil_div((int64_t)a.count[0], BN), 1);
    if (!at.ok) return false;
    const int64_t m0 = at.m * kBM, n0 = at.n * BN;
    const TileOperand A{a.W + m0 * a.ldw, a.ldw, a.planew, (int32_t)(a.nv - m0 < kBM ? a.nv - m0 : kBM)};
    const TileOperand B{a.X + n0 * a.ldx, a.ldx, a.planex, BN};
    tile.run(A, B, a.depth, kLogitProducts<kMany>, smem);
    return true;
}

// Per (vocabulary tile, listed token): maximum and sum of exp(z - maximum) besides the target; its logit.
template <int BN, bool kMany>
__global__ __launch_bounds__(kTileThreads, 2) void k_ce_stats(Logits a, float2 *__restrict__ part,
                                                                                float *__restrict__ zt)
{
    using T = Tile<false, false, kBM, BN, kWavesM<BN>, kWavesN<BN>>;
    __shared__ __attribute__((aligned(1024))) char smem[T::kLds];
    T tile;
    TilePlace at;
    if (!logits_tile<BN, kMany>(a, tile, at, smem)) return;
    const int l = threadIdx.x & 63, g = l >> 4, wm = T::wave_m(), wn = T::wave_n();
    const int64_t cnt = a.count[0], vw = at.m * kBM + wm * (16 * T::FM);  // the wave's first row of the piece
    float2 *join = (float2 *)smem;                                        // [wave row][BN]
    const int valid = (int)(a.nv - vw < 16 * T::FM ? a.nv - vw : 16 * T::FM) - 4 * g;  // rows from the lane's first on
    const bool edge = a.nv - vw < 16 * T::FM;
#pragma unroll
    for (int j = 0; j < T::FN; ++j) {
        const int nl = (wn * T::FN + j) * 16 + (l & 15);
        const int64_t n = at.n * BN + nl;
        float x[T::FM][4], mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < T::FM; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                x[i][r] = tile.acc[i][j][r];
                if (edge) x[i][r] = 16 * i + r >= valid ? -INFINITY : x[i][r];
            }
        // the target's logit: few waves hold one
        const int64_t t64 = n < cnt ? a.tgt[n] - a.v0 - vw - 4 * g : -1;
        const int t = t64 >= 0 && t64 < 16 * T::FM && (t64 & 12) == 0 ? (int)t64 : -1;
        if (__ballot(t >= 0) != 0) {
            float z = 0.0f;
#pragma unroll
            for (int i = 0; i < T::FM; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (t == 16 * i + r) {  // kept apart (loss_of)
                        z = x[i][r];
                        x[i][r] = -INFINITY;
                    }
            if (t >= 0) zt[n] = z;
        }
#pragma unroll
        for (int i = 0; i < T::FM; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) mx = fmaxf(mx, x[i][r]);
        mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
        mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
        const float base = mx == -INFINITY ? 0.0f : mx;  // nothing of the vocabulary in this wave
        const float base2 = base * kLog2e;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < T::FM; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) s += exp_less(x[i][r], base2);
        s += __shfl_xor(s, 16, 64);
        s += __shfl_xor(s, 32, 64);
        if (g == 0) join[wm * BN + nl] = make_float2(mx, s);
    }
    __syncthreads();
    for (int nl = threadIdx.x; nl < BN; nl += kTileThreads) {
        const int64_t n = at.n * BN + nl;
        if (n >= cnt) continue;
        float mx = join[nl].x, s = 0.0f;
        for (int w = 1; w < kWavesM<BN>; ++w) mx = fmaxf(mx, join[w * BN + nl].x);
        const float base = mx == -INFINITY ? 0.0f : mx;
        for (int w = 0; w < kWavesM<BN>; ++w)
            s += join[w * BN + nl].y * exp_of(join[w * BN + nl].x - base);
        part[(a.v0 / kBM + at.m) * a.npad + n] = make_float2(mx, s);
    }
}

// Joins the tiles' maxima and sums: 16 threads a token, each over every 16th tile.
__global__ __launch_bounds__(1024) void k_ce_join(const float2 *__restrict__ part, const float *__restrict__ zt,
                                                  const int32_t *__restrict__ rows, const int32_t *__restrict__ count,
                                                  int64_t npad, int64_t tiles, float *__restrict__ loss,
                                                  float *__restrict__ lse)
{
    __shared__ float2 join[16][64];
    const int l = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t m = (int64_t)blockIdx.x * 64 + l, cnt = count[0];
    if ((int64_t)blockIdx.x * 64 >= cnt) return;
    float mx = -INFINITY, s = 0.0f;
    if (m < cnt) {
        for (int64_t t = w; t < tiles; t += 16) {
            const float2 p = part[t * npad + m];
            const float up = fmaxf(mx, p.x);
            const float base = up == -INFINITY ? 0.0f : up;
            s = s * exp_of(mx - base) + p.y * exp_of(p.x - base);
            mx = up;
        }
    }
    join[w][l] = make_float2(mx, s);
    __syncthreads();
    if (w != 0 || m >= cnt) return;
    mx = -INFINITY;
    for (int i = 0; i < 16; ++i) mx = fmaxf(mx, join[i][l].x);
    const float base = mx == -INFINITY ? 0.0f : mx;
    s = 0.0f;
    for (int i = 0; i < 16; ++i) s += join[i][l].y * exp_of(join[i][l].x - base);
    const float2 r = loss_of(mx, s, zt[m]);
    lse[rows[m]] = r.x;
    loss[rows[m]] = r.y;
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

// A wave's tile goes out through its own part of LDS, so that stores cover whole row segments: FN *
// 16 output rows (n) of TM elements (m), 16 bytes of padding a row against bank conflicts.
template <int TM, int kRows, typename O>
struct Stage {
    static constexpr int kStride = TM * (int)sizeof(O) + 16;
    static constexpr int kBytes = kRows * kStride;
    static constexpr int kPer = 16 / (int)sizeof(O);          // elements of 16 bytes
    static constexpr int kLanes = TM / kPer;                  // lanes a row
    // Rows [0, rows) and elements [0, cols) of the staged tile to out[row * ld + element].
    __device__ static void store(const char *mine, O *out, int64_t ld, int64_t rows, int64_t cols)
    {
        const int l = threadIdx.x & 63, e = (l % kLanes) * kPer;
#pragma unroll 4
        for (int r = l / kLanes; r < kRows; r += 64 / kLanes) {
            if (r >= rows || e >= cols) continue;
            const u32x4 v = *(const u32x4 *)(mine + r * kStride + (l % kLanes) * 16);
            O *p = out + r * ld + e;
            if (e + kPer <= cols) store16(p, v);
            else
                for (int k = 0; e + k < cols; ++k) p[k] = ((const O *)(mine + r * kStride))[e + k];
        }
    }
};

// ---------------------------------------------------------------------------
// Few tiles of logits (a small vocabulary, or not many tokens): their depth is
// cut and the parts' logits are kept, a few MiB, for one of two passes over
// them: loss, or P.
// ---------------------------------------------------------------------------
struct Parts {
    float *z;            // [split][token][ldz]
    int64_t ldz, plane, splits, per;  // per: depth of a split, a multiple of 64
};
template <int BN, bool kMany>
__global__ __launch_bounds__(kTileThreads, 2) void k_ce_logits(Logits a, Parts z)
{
    using T = Tile<false, false, kBM, BN, kWavesM<BN>, kWavesN<BN>>;
    __shared__ __attribute__((aligned(1024))) char smem[T::kLds];
    const int64_t cnt = a.count[0];
    const TilePlace at = tile_place(ceil_div(a.nv, kBM), ceil_div(cnt, BN), z.splits);
    if (!at.ok) return;
    const int64_t m0 = at.m * kBM, n0 = at.n * BN, k0 = at.split * z.per;
    const int64_t depth = a.depth - k0 < z.per ? (a.depth - k0 > 0 ? a.depth - k0 : 0) : z.per;
    const TileOperand A{a.W + m0 * a.ldw + k0, a.ldw, a.planew, (int32_t)(a.nv - m0 < kBM ? a.nv - m0 : kBM)};
    const TileOperand B{a.X + n0 * a.ldx + k0, a.ldx, a.planex, BN};
    T tile;
    tile.run(A, B, depth, kLogitProducts<kMany>, smem);
    const int l = threadIdx.x & 63, g = l >> 4;
#pragma unroll
    for (int j = 0; j < T::FN; ++j) {
        const int64_t n = n0 + (T::wave_n() * T::FN + j) * 16 + (l & 15);
        if (n >= cnt) continue;
#pragma unroll
        for (int i = 0; i < T::FM; ++i)
            *(f32x4 *)(z.z + at.split * z.plane + n * z.ldz + m0 + (T::wave_m() * T::FM + i) * 16 + 4 * g) = tile.acc[i][j];
    }
}

// 4 logits of a token from v on (of columns past the vocabulary: whatever the tiles wrote there).
__device__ __forceinline__ f32x4 logits_at(const Parts &z, int64_t n, int64_t v)
{
    const float *p = z.z + n * z.ldz + v;
    f32x4 s = *(const f32x4 *)p;
    for (int64_t k = 1; k < z.splits; ++k) s += *(const f32x4 *)(p + k * z.plane);
    return s;
}

// loss and lse of listed token blockIdx.x.
__global__ __launch_bounds__(kCeThreads) void k_ce_loss(Parts z, const int32_t *__restrict__ rows,
                                                        const int32_t *__restrict__ tgt,
                                                        const int32_t *__restrict__ count, int64_t V,
                                                        float *__restrict__ loss, float *__restrict__ lse)
{
    __shared__ float2 join[kCeThreads / 64];
    const int64_t n = blockIdx.x;
    if (n >= count[0]) return;
    const int64_t t = tgt[n];
    float mx = -INFINITY, s = 0.0f;
    for (int64_t v = threadIdx.x * 4; v < V; v += kCeThreads * 4) {
        f32x4 x = logits_at(z, n, v);
        float up = mx;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (v + r >= V || v + r == t) x[r] = -INFINITY;  // the target is kept apart (loss_of)
            up = fmaxf(up, x[r]);
        }
        const float base = up == -INFINITY ? 0.0f : up;
        s *= exp_of(mx - base);
#pragma unroll
        for (int r = 0; r < 4; ++r) s += exp_of(x[r] - base);
        mx = up;
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const float omx = __shfl_xor(mx, off, 64), os = __shfl_xor(s, off, 64), up = fmaxf(mx, omx);
        const float base = up == -INFINITY ? 0.0f : up;
        s = s * exp_of(mx - base) + os * exp_of(omx - base);
        mx = up;
    }
    if ((threadIdx.x & 63) == 0) join[threadIdx.x >> 6] = make_float2(mx, s);
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int w = 1; w < kCeThreads / 64; ++w) {
        const float up = fmaxf(mx, join[w].x), base = up == -INFINITY ? 0.0f : up;
        s = s * exp_of(mx - base) + join[w].y * exp_of(join[w].x - base);
        mx = up;
    }
    const float2 r = loss_of(mx, s, logits_at(z, n, t & ~(int64_t)3)[t & 3]);
    lse[rows[n]] = r.x;
    loss[rows[n]] = r.y;
}

// An element of P into its planes.
template <bool kMany>
__device__ __forceinline__ void put_p(uint16_t *p, int64_t plane, float x)
{
    uint32_t b[kPPlanes<kMany>];
    split_pair(x, 0.0f, b);
#pragma unroll
    for (int pl = 0; pl < kPPlanes<kMany>; ++pl) p[pl * plane] = (uint16_t)b[pl];
}

// P of row blockIdx.x (planes), zeros for columns past the vocabulary and for tokens past the list, up to the
// next multiple of 64 (the depth of dW).
template <bool kMany>
__global__ __launch_bounds__(kCeThreads) void k_ce_p(Parts z, const int32_t *__restrict__ rows,
                                                     const int32_t *__restrict__ tgt, const int32_t *__restrict__ count,
                                                     int64_t V, const float *__restrict__ lse,
                                                     uint16_t *__restrict__ P, int64_t ldp, int64_t planep)
{
    const int64_t n = blockIdx.x, cnt = count[0];
    if (n >= round_up(cnt, kDepth)) return;
    const bool on = n < cnt;
    const float ls = on ? lse[rows[n]] * kLog2e : 0.0f;
    const int64_t t = on ? tgt[n] : -1;
    __shared__ float sum[kCeThreads / 64], pt;
    float others = 0.0f;
    for (int64_t v = threadIdx.x * 4; v < ldp; v += kCeThreads * 4) {
        float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (on && v < V) {
            const f32x4 y = logits_at(z, n, v);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (v + r < V) x[r] = exp_less(y[r], ls);
                if (v + r == t) {
                    pt = x[r];
                    x[r] = 0.0f;
                }
                others += x[r];
            }
        }
        uint32_t b[2][kPPlanes<kMany>];
#pragma unroll
        for (int h = 0; h < 2; ++h) split_pair(x[2 * h], x[2 * h + 1], b[h]);
#pragma unroll
        for (int pl = 0; pl < kPPlanes<kMany>; ++pl)
            *(uint2 *)(P + pl * planep + n * ldp + v) = make_uint2(b[0][pl], b[1][pl]);
    }
    if (!on) return;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) others += __shfl_xor(others, off, 64);
    if ((threadIdx.x & 63) == 0) sum[threadIdx.x >> 6] = others;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int w = 1; w < kCeThreads / 64; ++w) others += sum[w];
    put_p<kMany>(P + n * ldp + t, planep, target_of(pt, others));
}

// P of the piece (planes) without the targets' elements: P[n][v], zeros for tokens past the list and columns
// past the piece, so that it can serve as depth up to the next multiple of 64.  For k_ce_targets: the sum of the
// elements of each wave row of the vocabulary tiles and token, and exp(z - lse) at the target.
template <int BN, bool kMany>
__global__ __launch_bounds__(kTileThreads, 2) void k_ce_probs(Logits a,
                                                                                const float *__restrict__ lse,
                                                                                const int32_t *__restrict__ rows,
                                                                                uint16_t *__restrict__ P, int64_t ldp,
                                                                                int64_t planep,
                                                                                float *__restrict__ others,
                                                                                float *__restrict__ pt)
{
    using T = Tile<false, false, kBM, BN, kWavesM<BN>, kWavesN<BN>>;
    using S = Stage<16 * T::FM, 16, uint16_t>;
    static_assert(kTileWaves * kPlanes * S::kBytes <= T::kLds, "the staged rows fit the tile's LDS");
    __shared__ __attribute__((aligned(1024))) char smem[T::kLds];
    T tile;
    TilePlace at;
    if (!logits_tile<BN, kMany>(a, tile, at, smem)) return;
    const int l = threadIdx.x & 63, g = l >> 4, wm = T::wave_m(), wn = T::wave_n();
    const int64_t cnt = a.count[0], vw = at.m * kBM + wm * (16 * T::FM), nw = at.n * BN + wn * (16 * T::FN);
    const int valid = (int)(a.nv - vw < 16 * T::FM ? a.nv - vw : 16 * T::FM) - 4 * g;  // rows from the lane's first on
    const bool edge = a.nv - vw < 16 * T::FM || nw + 16 * T::FN > cnt;
    constexpr int kOut = kPPlanes<kMany>;
    char *mine = smem + (threadIdx.x >> 6) * (kOut * S::kBytes);
#pragma unroll
    for (int j = 0; j < T::FN; ++j) {  // 16 tokens at a time
        const int64_t n = nw + j * 16 + (l & 15);
        const bool on = n < cnt;
        const int64_t t64 = on ? a.tgt[n] - a.v0 - vw - 4 * g : -1;
        const int t = t64 >= 0 && t64 < 16 * T::FM && (t64 & 12) == 0 ? (int)t64 : -1;
        const bool target = __ballot(t >= 0) != 0;  // few waves hold one
        const float ls = on ? lse[rows[n]] * kLog2e : 0.0f;
        const int end = on ? valid : 0;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            float x[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = exp_less(tile.acc[i][j][r], ls);
            if (target)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (t == 16 * i + r) {
                        pt[n] = x[r];
                        x[r] = 0.0f;
                    }
            if (edge)
#pragma unroll
                for (int r = 0; r < 4; ++r) x[r] = 16 * i + r < end ? x[r] : 0.0f;
            sum += (x[0] + x[1]) + (x[2] + x[3]);
            uint32_t b[2][kOut];
#pragma unroll
            for (int h = 0; h < 2; ++h) split_pair(x[2 * h], x[2 * h + 1], b[h]);
#pragma unroll
            for (int pl = 0; pl < kOut; ++pl)
                *(uint2 *)(mine + pl * S::kBytes + (l & 15) * S::kStride + (16 * i + 4 * g) * 2) =
                    make_uint2(b[0][pl], b[1][pl]);
        }
        wait_lds();
#pragma unroll
        for (int pl = 0; pl < kOut; ++pl)
            S::store(mine + pl * S::kBytes, P + pl * planep + (nw + j * 16) * ldp + vw, ldp, 16, 16 * T::FM);
        sum += __shfl_xor(sum, 16, 64);
        sum += __shfl_xor(sum, 32, 64);
        if (g == 0 && on) others[((a.v0 / kBM + at.m) * kWavesM<BN> + wm) * a.npad + n] = sum;
        wait_lds();
    }
}

// The targets' elements of the piece [v0, v0 + nv), from the sum of each token's others over all `parts` of the
// vocabulary.  16 threads a token, each over every 16th part.
template <bool kMany>
__global__ __launch_bounds__(1024) void k_ce_targets(const float *__restrict__ others, int64_t npad, int64_t parts,
                                                     const float *__restrict__ pt,
                                                     const int32_t *__restrict__ tgt, const int32_t *__restrict__ count,
                                                     int64_t v0, int64_t nv, uint16_t *__restrict__ P, int64_t ldp,
                                                     int64_t planep)
{
    constexpr int kAhead = 8;
    __shared__ float join[16][64];
    const int l = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t m = (int64_t)blockIdx.x * 64 + l, cnt = count[0];
    if ((int64_t)blockIdx.x * 64 >= cnt) return;
    float s = 0.0f;
    if (m < cnt)
        for (int64_t t = w; t < parts; t += 16 * kAhead) {
            float x[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) x[j] = t + 16 * j < parts ? others[(t + 16 * j) * npad + m] : 0.0f;
#pragma unroll
            for (int j = 0; j < kAhead; ++j) s += x[j];
        }
    join[w][l] = s;
    __syncthreads();
    if (w != 0 || m >= cnt) return;
    for (int i = 1; i < 16; ++i) s += join[i][l];
    const int64_t t = tgt[m] - v0;
    if (t >= 0 && t < nv) put_p<kMany>(P + m * ldp + t, planep, target_of(pt[m], s));
}

// acc[split][n][c] (+)= sum over the split's part of the piece of P[n, v] W[v, c].
struct InputGrad {
    const uint16_t *P, *W;
    int64_t ldp, ldw, planep, planew;
    const int32_t *count;
    int64_t nv, D, splits, per;  // per: depth of a split, a multiple of 64
    float *acc;
    int64_t lda, plane;
    int add;
};
template <int BN, bool kMany>
__global__ __launch_bounds__(kTileThreads, 2) void k_ce_dx(InputGrad a)
{
    using T = Tile<true, false, kBM, BN, kWavesM<BN>, kWavesN<BN>>;
    __shared__ __attribute__((aligned(1024))) char smem[T::kLds];
    const int64_t cnt = a.count[0];
    const TilePlace at = tile_place(ceil_div(a.D, kBM), ceil_div(cnt, BN), a.splits);
    if (!at.ok) return;
    const int64_t m0 = at.m * kBM, n0 = at.n * BN, k0 = at.split * a.per;
    const int64_t depth = a.nv - k0 < a.per ? (a.nv - k0 > 0 ? a.nv - k0 : 0) : a.per;
    const TileOperand A{a.W + k0 * a.ldw + m0, a.ldw, a.planew, (int32_t)(a.ldw - m0 < kBM ? a.ldw - m0 : kBM)};
    const TileOperand B{a.P + n0 * a.ldp + k0, a.ldp, a.planep, BN};
    T tile;
    tile.run(A, B, depth, kGradProducts<kMany>, smem);
    const int l = threadIdx.x & 63, g = l >> 4;
#pragma unroll
    for (int j = 0; j < T::FN; ++j) {
        const int64_t n = n0 + (T::wave_n() * T::FN + j) * 16 + (l & 15);
        if (n >= cnt) continue;
#pragma unroll
        for (int i = 0; i < T::FM; ++i) {
            const int64_t c = m0 + (T::wave_m() * T::FM + i) * 16 + 4 * g;
            if (c >= a.lda) continue;
            f32x4 *p = (f32x4 *)(a.acc + at.split * a.plane + n * a.lda + c);
            *p = a.add ? *p + tile.acc[i][j] : tile.acc[i][j];
        }
    }
}

struct WeightGrad {
    const uint16_t *P, *X;
    int64_t ldp, ldx, planep, planex;
    const int32_t *count;
    int64_t nv, D;
    const float *dmean, *total;
    int64_t splits, per;  // per: tokens of a split, a multiple of 64
    float *acc;           // several splits: their sums, [split][vocabulary][lda]
    int64_t lda, plane;
};
template <typename E, bool kSplit>
__global__ __launch_bounds__(kTileThreads, 2) void k_ce_dw(WeightGrad a, typename E::T *__restrict__ dW)
{
    using T = Tile<true, true, kBM, 256, kWavesM<256>, kWavesN<256>>;
    constexpr int kPass = sizeof(typename E::T) == 4 ? 2 : 1;  // fp32 rows leave in two passes
    using S = Stage<16 * T::FM, 16 * T::FN / kPass, typename E::T>;
    constexpr int kLds = T::kLds > kTileWaves * S::kBytes ? T::kLds : kTileWaves * S::kBytes;
    __shared__ __attribute__((aligned(1024))) char smem[kLds];
    const TilePlace at = tile_place(ceil_div(a.D, kBM), ceil_div(a.nv, 256), kSplit ? a.splits : 1);
    if (!at.ok) return;
    const int64_t m0 = at.m * kBM, n0 = at.n * 256, k0 = kSplit ? at.split * a.per : 0;
    int64_t depth = round_up(a.count[0], kDepth) - k0;
    if (kSplit) depth = depth < 0 ? 0 : depth < a.per ? depth : a.per;
    const TileOperand A{a.X + k0 * a.ldx + m0, a.ldx, a.planex, (int32_t)(a.ldx - m0 < kBM ? a.ldx - m0 : kBM)};
    const TileOperand B{a.P + k0 * a.ldp + n0, a.ldp, a.planep, 256};
    T tile;
    tile.run(A, B, depth, kGradProducts<Split<E>::kMany>, smem);
    if constexpr (kSplit) {
        const int l = threadIdx.x & 63, g = l >> 4;
#pragma unroll
        for (int j = 0; j < T::FN; ++j) {
            const int64_t n = n0 + (T::wave_n() * T::FN + j) * 16 + (l & 15);
            if (n >= a.nv) continue;
#pragma unroll
            for (int i = 0; i < T::FM; ++i) {
                const int64_t c = m0 + (T::wave_m() * T::FM + i) * 16 + 4 * g;
                if (c < a.lda) *(f32x4 *)(a.acc + at.split * a.plane + n * a.lda + c) = tile.acc[i][j];
            }
        }
        return;
    }
    const float s = grad_scale(a.dmean, a.total);
    const int l = threadIdx.x & 63, g = l >> 4;
    const int64_t mw = m0 + T::wave_m() * (16 * T::FM), nw = n0 + T::wave_n() * (16 * T::FN);
    char *mine = smem + (threadIdx.x >> 6) * S::kBytes;
#pragma unroll
    for (int pass = 0; pass < kPass; ++pass) {
#pragma unroll
        for (int jj = 0; jj < T::FN / kPass; ++jj) {
            const int j = pass * (T::FN / kPass) + jj;
#pragma unroll
            for (int i = 0; i < T::FM; ++i) {
                char *p = mine + (jj * 16 + (l & 15)) * S::kStride + (16 * i + 4 * g) * (int)sizeof(typename E::T);
                const f32x4 v = tile.acc[i][j];
                if constexpr (kPass == 2) {
                    *(f32x4 *)p = f32x4{v[0] * s, v[1] * s, v[2] * s, v[3] * s};
                } else {
                    *(uint2 *)p = make_uint2(pack_bf16(v[0] * s, v[1] * s), pack_bf16(v[2] * s, v[3] * s));
                }
            }
        }
        wait_lds();
        const int64_t n = nw + pass * (16 * T::FN / kPass);
        S::store(mine, dW + n * a.D + mw, a.D, a.nv - n, a.D - mw);
        wait_lds();
    }
}

// Memory of a call: pieces of the vocabulary are taken so that P stays within kPieceBytes (or 256 vocabulary rows
// of all tokens, if that is more), and the planes (or the padded copy) of W within kCopyBytes.  Sums of parts that
// run side by side take 512 MiB at most for each of the logits, dX and dW (cuts).  Beside these a call has the rows
// of X (planes), dX in fp32, and 8 bytes (the backward 16) a token and 256 vocabulary rows.  The backward of several pieces makes the logits of all of them first, for the sums that the
// targets' elements are made of, and once more: so a piece is large.
constexpr int64_t kPieceBytes = (int64_t)4 << 30;
constexpr int64_t kCopyBytesF32 = (int64_t)1 << 30, kCopyBytesBF16 = (int64_t)256 << 20;

// A launch has fewer than 2^32 threads, 512 a tile.
constexpr int64_t kMaxTiles = ((int64_t)1 << 23) - 1;

// Tiles of logits up to which their depth is cut (step, whole / cut: 51 tiles, 2056 tokens x 707 x 1472, fp32 374 /
// 240 us, bf16 150 / 142; 4 tiles, 209 x 501 x 2241, 432 / 138 and 145 / 106; 48 tiles, 500 x 3000 x 300, 153 / 137 and
// 115 / 115; but 88, 245 x 11095 x 192, 147 / 153 and 91 / 91, and 108, 300 x 9000 x 1024, 395 / 424 and 118 / 123).
constexpr int64_t kFewTiles = 64;

struct CePlan {
    int64_t npad, ldx, piece, tiles, splits, dw_splits, z_splits;
    int bn;
    bool copy;  // W is copied, a piece at a time: planes, or rows that are no multiple of 128 bytes
    size_t rows, tgt, slot, count, X, W, part, zt, P, others, pt, acc, dw_acc, z, total;
};

// Into how many parts the depth of a product of `tiles` tiles is cut, so that its rounds of 256 (one tile a CU)
// are full: the number with the least time, counting 1% for each part's sums, up to `most` parts and 512 MiB of
// sums (bytes each).
int64_t cuts(int64_t tiles, int64_t most, int64_t bytes)
{
    const int64_t room = ((int64_t)512 << 20) / bytes;
    if (most > room) most = room;
    if (most > 64) most = 64;
    int64_t r = 1;
    double best = 1e30;
    for (int64_t k = 1; k <= most; ++k) {
        const double t = (double)ceil_div(tiles * k, 256) / (double)k * (1.0 + 0.01 * (double)k);
        if (t < best) {
            best = t;
            r = k;
        }
    }
    return r;
}

CePlan ce_plan(int64_t N, int64_t V, int64_t D, int dtype, bool backward, bool w_aligned)
{
    CePlan p{};
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t r = at;
        at += (size_t)round_up(bytes, 1024);
        return r;
    };
    const int64_t planes = dtype == CSP_F32 ? kPlanes : 1, p_planes = dtype == CSP_F32 ? kPPlanes<true> : kPPlanes<false>;
    p.npad = round_up(N > 0 ? N : 1, kPad);
    p.ldx = round_up(D, kDepth);
    // Tiles of 128 tokens for few of them, or where tiles of 256 would leave half of the CUs without work (step, tiles
    // of 256 / 128: 256 tokens, 30000 x 1024, fp32 646 / 555 us, bf16 184 / 165; 300, 9000 x 1024, 494 / 393 and 149 /
    // 118; 384, 30000 x 1024, 783 / 825 and 229 / 239; 256, 65536 x 2048, 2093 / 2260 and 545 / 583).
    p.bn = N <= 128 || ceil_div(V, kBM) * ceil_div(N, 256) <= 128 ? 128 : 256;
    p.copy = dtype == CSP_F32 || D % kDepth != 0 || !w_aligned;
    p.tiles = ceil_div(V, kBM);
    p.piece = round_up(V, kPad);
    auto limit = [&](int64_t bytes, int64_t row_bytes) {
        int64_t r = bytes / row_bytes / kPad * kPad;
        if (r < kPad) r = kPad;
        if (r < p.piece) p.piece = r;
    };
    // and each launch within kMaxTiles
    auto tiles_within = [&](int64_t others) { limit(kMaxTiles / others * kBM, 1); };
    tiles_within(ceil_div(N > 0 ? N : 1, p.bn));
    if (backward) tiles_within(ceil_div(D, kBM));
    if (p.copy) limit(dtype == CSP_F32 ? kCopyBytesF32 : kCopyBytesBF16, planes * 2 * p.ldx);
    if (backward) limit(kPieceBytes, p_planes * 2 * p.npad);
    // an fp32 step of depth is six: its parts may be shorter
    const int64_t least = dtype == CSP_F32 ? 2 * kDepth : 8 * kDepth;
    const int64_t tiles = ceil_div(V, kBM) * ceil_div(N, p.bn), vpad = round_up(V, kPad);
    p.z_splits = tiles <= kFewTiles && p.piece >= vpad ? cuts(tiles, ceil_div(p.ldx, least), 4 * p.npad * vpad) : 1;
    if (p.z_splits > 1) p.z = take(4 * p.z_splits * p.npad * vpad);
    p.count = take(4);
    p.rows = take(4 * N);
    p.tgt = take(4 * N);
    p.slot = take(4 * N);
    p.X = take(planes * 2 * p.npad * p.ldx);
    if (p.copy) p.W = take(planes * 2 * p.piece * p.ldx);
    if (!backward) {
        p.part = take(8 * p.npad * p.tiles);
        p.zt = take(4 * p.npad);
    } else {
        p.P = take(p_planes * 2 * p.npad * p.piece);
        p.others = take(4 * p.npad * p.tiles * kWavesM<128>);
        p.pt = take(4 * p.npad);
        p.splits = cuts(ceil_div(D, kBM) * ceil_div(p.npad, p.bn), ceil_div(p.piece, least), 4 * p.npad * p.ldx);
        p.dw_splits = cuts(ceil_div(D, kBM) * ceil_div(p.piece, 256), ceil_div(N, least), 4 * p.piece * p.ldx);
        if (p.dw_splits > 1) p.dw_acc = take(4 * p.dw_splits * p.piece * p.ldx);
        p.acc = take(4 * p.splits * p.npad * p.ldx);
    }
    p.total = at;
    return p;
}

size_t ce_bytes(int64_t N, int64_t V, int64_t D, int dtype, bool backward)
{
    if (ce_is_few(N, dtype)) return ce_few_bytes(N, V, D, dtype, backward);
    const size_t a = ce_plan(N, V, D, dtype, backward, true).total, b = ce_plan(N, V, D, dtype, backward, false).total;
    return a > b ? a : b;
}

csp_status ce_args(int64_t N, int64_t V, int64_t D, int dtype)
{
    // A launch has fewer than 2^32 threads: 256 a token (of a multiple of 64), 2 a vocabulary row, 512 a tile of dX
    // (those of the logits and dW are cut with the vocabulary, ce_plan); 32-bit offsets in a tile.
    if (N < 0 || N > ((int64_t)1 << 24) - kDepth || V < 1 || V > (int64_t)1 << 30 || D < 1 || D >= (int64_t)1 << 22 ||
        ceil_div(N, 256) * ceil_div(D, kBM) > kMaxTiles)
        return set_error(CSP_ERR_INVALID_ARG, "bad shape: %lld tokens, vocabulary %lld, width %lld", (long long)N,
                         (long long)V, (long long)D);
    if (dtype != CSP_F32 && dtype != CSP_BF16) return set_error(CSP_ERR_DTYPE, "unsupported dtype %d", dtype);
    return CSP_OK;
}

bool aligned(const void *p, size_t a) { return p && (uintptr_t)p % a == 0; }

enum Asked { kInput = 1, kWeight = 2 };

// What both directions begin with: the list, the gathered rows of X, and the Logits arguments of a piece.
template <typename E>
csp_status ce_begin(const CePlan &p, const void *X, const int64_t *targets, int64_t N, int64_t V, int64_t D,
                    float *loss, float *lse, char *w, hipStream_t s)
{
    k_ce_rows<<<1, 1024, 0, s>>>(targets, N, V, (int32_t *)(w + p.rows), (int32_t *)(w + p.tgt),
                                 (int32_t *)(w + p.slot), (int32_t *)(w + p.count), loss, lse);
    CSP_LAUNCHED("k_ce_rows");
    if (N == 0) return CSP_OK;
    k_ce_gather<E><<<(unsigned)round_up(N, kDepth), kCeThreads, 0, s>>>(
        (const typename E::T *)X, D, (const int32_t *)(w + p.rows), (const int32_t *)(w + p.count),
        (uint16_t *)(w + p.X), p.ldx, p.npad * p.ldx);
    CSP_LAUNCHED("k_ce_gather");
    return CSP_OK;
}

template <typename E>
csp_status ce_piece(const CePlan &p, const void *W, int64_t V, int64_t D, int64_t v0, char *w, Logits *a, hipStream_t s)
{
    using T = typename E::T;
    const int64_t nv = V - v0 < p.piece ? V - v0 : p.piece;
    *a = Logits{(const uint16_t *)(w + p.X), (const uint16_t *)((const T *)W + v0 * D), p.ldx, D, p.npad * p.ldx, 0,
                (const int32_t *)(w + p.tgt), (const int32_t *)(w + p.count), nv, v0, p.npad, p.ldx};
    if (!p.copy) return CSP_OK;
    a->W = (const uint16_t *)(w + p.W);
    a->ldw = p.ldx;
    a->planew = p.piece * p.ldx;
    k_ce_gather<E><<<(unsigned)nv, kCeThreads, 0, s>>>((const T *)W + v0 * D, D, nullptr, nullptr,
                                                       (uint16_t *)(w + p.W), p.ldx, a->planew);
    CSP_LAUNCHED("k_ce_gather");
    return CSP_OK;
}

template <bool kMany>
csp_status ce_logits(const CePlan &p, const Logits &a, int64_t N, char *w, Parts *z, hipStream_t s)
{
    const int64_t ldz = round_up(a.nv, kPad);
    *z = Parts{(float *)(w + p.z), ldz, p.npad * ldz, p.z_splits, round_up(ceil_div(p.ldx, p.z_splits), kDepth)};
    const unsigned grid = (unsigned)(ceil_div(a.nv, kBM) * ceil_div(N, p.bn) * p.z_splits);
    if (p.bn == 128) k_ce_logits<128, kMany><<<grid, kTileThreads, 0, s>>>(a, *z);
    else k_ce_logits<256, kMany><<<grid, kTileThreads, 0, s>>>(a, *z);
    CSP_LAUNCHED("k_ce_logits");
    return CSP_OK;
}

template <typename E>
csp_status fwd_impl(const void *X, const void *W, const int64_t *targets, int64_t N, int64_t V, int64_t D, float *loss,
                    float *lse, float *total, char *w, hipStream_t s)
{
    constexpr bool kMany = Split<E>::kMany;
    const CePlan p = ce_plan(N, V, D, kMany ? CSP_F32 : CSP_BF16, false, aligned(W, 16));
    int32_t *rows = (int32_t *)(w + p.rows), *count = (int32_t *)(w + p.count);
    float2 *part = (float2 *)(w + p.part);
    float *zt = (float *)(w + p.zt);
    csp_status st = ce_begin<E>(p, X, targets, N, V, D, loss, lse, w, s);
    if (st != CSP_OK) return st;
    for (int64_t v0 = 0; N > 0 && v0 < V; v0 += p.piece) {
        Logits a;
        st = ce_piece<E>(p, W, V, D, v0, w, &a, s);
        if (st != CSP_OK) return st;
        if (p.z_splits > 1) {
            Parts z;
            st = ce_logits<kMany>(p, a, N, w, &z, s);
            if (st != CSP_OK) return st;
            k_ce_loss<<<(unsigned)N, kCeThreads, 0, s>>>(z, rows, a.tgt, count, V, loss, lse);
            CSP_LAUNCHED("k_ce_loss");
            break;
        }
        const unsigned grid = (unsigned)(ceil_div(a.nv, kBM) * ceil_div(N, p.bn));
        if (p.bn == 128) k_ce_stats<128, kMany><<<grid, kTileThreads, 0, s>>>(a, part, zt);
        else k_ce_stats<256, kMany><<<grid, kTileThreads, 0, s>>>(a, part, zt);
        CSP_LAUNCHED("k_ce_stats");
    }
    if (N > 0 && p.z_splits == 1) {
        k_ce_join<<<(unsigned)ceil_div(N, 64), 1024, 0, s>>>(part, zt, rows, count, p.npad, p.tiles, loss, lse);
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
    constexpr bool kMany = Split<E>::kMany;
    const CePlan p = ce_plan(N, V, D, kMany ? CSP_F32 : CSP_BF16, true, aligned(W, 16));
    int32_t *rows = (int32_t *)(w + p.rows), *count = (int32_t *)(w + p.count);
    uint16_t *P = (uint16_t *)(w + p.P);
    const int64_t planep = p.npad * p.piece;
    csp_status st = ce_begin<E>(p, X, targets, N, V, D, nullptr, nullptr, w, s);
    if (st != CSP_OK) return st;
    float *others = (float *)(w + p.others), *pt = (float *)(w + p.pt);
    auto probs = [&](const Logits &a) {
        const unsigned grid = (unsigned)(ceil_div(a.nv, kBM) * ceil_div(N, p.bn));
        if (p.bn == 128) k_ce_probs<128, kMany><<<grid, kTileThreads, 0, s>>>(a, lse, rows, P, p.piece, planep, others, pt);
        else k_ce_probs<256, kMany><<<grid, kTileThreads, 0, s>>>(a, lse, rows, P, p.piece, planep, others, pt);
        CSP_LAUNCHED("k_ce_probs");
        return CSP_OK;
    };
    for (int64_t v0 = 0; N > 0 && V > p.piece && v0 < V; v0 += p.piece) {  // the sums of all pieces
        Logits a;
        st = ce_piece<E>(p, W, V, D, v0, w, &a, s);
        if (st != CSP_OK) return st;
        st = probs(a);
        if (st != CSP_OK) return st;
    }
    const int64_t per = round_up(ceil_div(p.piece, p.splits), kDepth);
    for (int64_t v0 = 0; v0 < V; v0 += p.piece) {
        Logits a;
        st = ce_piece<E>(p, W, V, D, v0, w, &a, s);
        if (st != CSP_OK) return st;
        if (N > 0) {
            if (p.z_splits > 1) {
                Parts z;
                st = ce_logits<kMany>(p, a, N, w, &z, s);
                if (st != CSP_OK) return st;
                k_ce_p<kMany><<<(unsigned)round_up(N, kDepth), kCeThreads, 0, s>>>(z, rows, a.tgt, count, V, lse, P,
                                                                                   p.piece, planep);
                CSP_LAUNCHED("k_ce_p");
            } else {
                st = probs(a);
                if (st != CSP_OK) return st;
                k_ce_targets<kMany><<<(unsigned)ceil_div(N, 64), 1024, 0, s>>>(
                    others, p.npad, p.tiles * (p.bn == 128 ? kWavesM<128> : kWavesM<256>), pt, a.tgt, count, v0, a.nv,
                    P, p.piece, planep);
                CSP_LAUNCHED("k_ce_targets");
            }
        }
        if (N > 0 && dX) {
            const InputGrad d{P, a.W, p.piece, a.ldw, planep, a.planew, count, a.nv, D, p.splits, per,
                              (float *)(w + p.acc), p.ldx, p.npad * p.ldx, v0 > 0};
            const unsigned gx = (unsigned)(ceil_div(D, kBM) * ceil_div(N, p.bn) * p.splits);
            if (p.bn == 128) k_ce_dx<128, kMany><<<gx, kTileThreads, 0, s>>>(d);
            else k_ce_dx<256, kMany><<<gx, kTileThreads, 0, s>>>(d);
            CSP_LAUNCHED("k_ce_dx");
        }
        if (!dW) continue;
        const WeightGrad g{P, a.X, p.piece, p.ldx, planep, a.planex, count, a.nv, D, dmean, total, p.dw_splits,
                           round_up(ceil_div(p.npad, p.dw_splits), kDepth), (float *)(w + p.dw_acc), p.ldx,
                           p.piece * p.ldx};
        const unsigned gw = (unsigned)(ceil_div(D, kBM) * ceil_div(a.nv, 256) * p.dw_splits);
        if (p.dw_splits == 1) {
            k_ce_dw<E, false><<<gw, kTileThreads, 0, s>>>(g, (T *)dW + v0 * D);
            CSP_LAUNCHED("k_ce_dw");
        } else {
            k_ce_dw<E, true><<<gw, kTileThreads, 0, s>>>(g, nullptr);
            CSP_LAUNCHED("k_ce_dw");
            k_ce_out<E><<<out_blocks(a.nv, D), 256, 0, s>>>(g.acc, p.ldx, g.plane, (int)p.dw_splits, nullptr, a.nv, D,
                                                            dmean, total, (T *)dW + v0 * D);
            CSP_LAUNCHED("k_ce_out");
        }
    }
    if (N > 0 && dX) {
        k_ce_out<E><<<out_blocks(N, D), 256, 0, s>>>((const float *)(w + p.acc), p.ldx, p.npad * p.ldx, (int)p.splits,
                                                     (const int32_t *)(w + p.slot), N, D, dmean, total, (T *)dX);
        CSP_LAUNCHED("k_ce_out");
    }
    return CSP_OK;
}

csp_status ce_bwd(const void *X, const void *W, const int64_t *targets, int64_t N, int64_t V, int64_t D, int dtype,
                  const float *lse, const float *dmean, const float *total, void *dX, void *dW, int asked,
                  void *workspace, int64_t workspace_bytes, hipStream_t stream)
{
    csp_status st = ce_args(N, V, D, dtype);
    if (st != CSP_OK) return st;
    const size_t e = dtype == CSP_BF16 ? 2 : 4;
    if (!aligned(W, e) || (asked & kWeight && !aligned(dW, e)) || !aligned(dmean, 4) || !aligned(total, 4) ||
        (N > 0 && (!aligned(X, e) || !aligned(targets, 8) || !aligned(lse, 4) || (asked & kInput && !aligned(dX, e)))))
        return set_error(CSP_ERR_INVALID_ARG, "NULL or misaligned pointer");
    const size_t need = ce_bytes(N, V, D, dtype, true);
    if (!aligned(workspace, 16) || workspace_bytes < (int64_t)need)
        return set_error(CSP_ERR_INVALID_ARG, "workspace of %lld bytes, %zu needed", (long long)workspace_bytes, need);
    auto run = dtype == CSP_BF16 ? bwd_impl<BF16> : bwd_impl<F32>;
    if (ce_is_few(N, dtype))
        return ce_few_bwd(X, W, targets, N, V, D, dtype, lse, dmean, total, dX, dW, (char *)workspace, stream);
    return run(X, W, targets, N, V, D, lse, dmean, total, dX, dW, (char *)workspace, stream);
}

}  // namespace
}  // namespace csp

extern "C" {

int64_t linear_ce_workspace(int64_t N, int64_t V, int64_t D, csp_dtype dtype, int32_t backward)
{
    if (csp::ce_args(N, V, D, dtype) != CSP_OK) return -1;
    return (int64_t)csp::ce_bytes(N, V, D, dtype, backward != 0);
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
    const size_t need = ce_bytes(N, V, D, dtype, false);
    if (!aligned(workspace, 16) || workspace_bytes < (int64_t)need)
        return set_error(CSP_ERR_INVALID_ARG, "workspace of %lld bytes, %zu needed", (long long)workspace_bytes, need);
    if (ce_is_few(N, dtype))
        return ce_few_fwd(X, W, targets, N, V, D, dtype, loss, lse, total, (char *)workspace, (hipStream_t)stream);
    if (dtype == CSP_BF16)
        return fwd_impl<BF16>(X, W, targets, N, V, D, loss, lse, total, (char *)workspace, (hipStream_t)stream);
    return fwd_impl<F32>(X, W, targets, N, V, D, loss, lse, total, (char *)workspace, (hipStream_t)stream);
}

csp_status linear_ce_bwd(const void *X, const void *W, const int64_t *targets, int64_t N, int64_t V, int64_t D,
                         csp_dtype dtype, const float *lse, const float *dmean, const float *total, void *dX, void *dW,
                         void *workspace, int64_t workspace_bytes, void *stream)
{
    return csp::ce_bwd(X, W, targets, N, V, D, dtype, lse, dmean, total, dX, dW, csp::kInput | csp::kWeight, workspace,
                       workspace_bytes, (hipStream_t)stream);
}

csp_status linear_ce_bwd_input(const void *X, const void *W, const int64_t *targets, int64_t N, int64_t V, int64_t D,
                               csp_dtype dtype, const float *lse, const float *dmean, const float *total, void *dX,
                               void *workspace, int64_t workspace_bytes, void *stream)
{
    return csp::ce_bwd(X, W, targets, N, V, D, dtype, lse, dmean, total, dX, nullptr, csp::kInput, workspace,
                       workspace_bytes, (hipStream_t)stream);
}

csp_status linear_ce_bwd_weight(const void *X, const void *W, const int64_t *targets, int64_t N, int64_t V, int64_t D,
                                csp_dtype dtype, const float *lse, const float *dmean, const float *total, void *dW,
                                void *workspace, int64_t workspace_bytes, void *stream)
{
    return csp::ce_bwd(X, W, targets, N, V, D, dtype, lse, dmean, total, nullptr, dW, csp::kWeight, workspace,
                       workspace_bytes, (hipStream_t)stream);
}

}  // extern "C"
