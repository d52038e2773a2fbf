// mfma_tile.h -- the tile product of the dense kernels (linear cross entropy):
//
//   acc[m][n] = sum over k of A(m, k) B(n, k),   bf16 operands, fp32 sums
//
// for a BM x BN tile by 8 waves.  An operand is either stored with k along its
// rows (kDepthMajor = false: element (r, k) at base[r * ld + k]) or with k
// down its columns (kDepthMajor = true: base[k * ld + r]); both kinds reach
// LDS by 16-byte loads that bypass the registers, and the second is turned on
// its way out of LDS by the transposing 64-bit read.
//
// Depth is walked in steps of 64 with two LDS buffers and, inside a step, two
// register sets of 32: while the matrix units work on one half, the next half
// (of the same step, or of the following one) is read from LDS.  One barrier
// a step: it comes between the halves, when every wave has read its second
// half (so the buffer is free for step + 2) and its own loads of step + 1
// have landed.
//
// fp32 operands are held as three bf16 planes, x = x0 + x1 + x2 with each
// plane the rest rounded to nearest, 24 bits in all.  Six of the nine plane
// products are taken; the three left out are below 2^-25 of |x w|, under the
// rounding of the fp32 sum itself.  They are walked as six steps of depth in
// place of one.
#pragma once

#include "common.h"
#include "device_util.h"

namespace csp {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kDepth = 64;        // k of a step
constexpr int kTileWaves = 8;
constexpr int kTileThreads = 64 * kTileWaves;
constexpr int kPlanes = 3;        // planes of an fp32 operand
constexpr int kPlaneProducts = 6;

// One operand of a tile.  rows: valid rows (r) from the tile's first on;
// loads past them repeat the last one.  For kDepthMajor, ld - (first r) bounds
// r instead, in groups of 8, and depth rows past `depth` repeat the last.
struct TileOperand {
    const uint16_t *base;  // the tile's first element
    int64_t ld;            // elements
    int64_t plane;         // elements from one plane to the next
    int32_t rows;          // valid r from the tile's first (kDepthMajor: a multiple of 8)
};

// 16 bytes a lane from base + off into LDS at lds + 16 * lane.  The compiler
// does not see the load: wait_loads() and a barrier come before any read.
__device__ __forceinline__ void load_to_lds(const uint16_t *base, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :
                 : "v"(off), "s"(base), "s"(lds)
                 : "memory");  // m0 is the compiler's only for instructions that none of these kernels has
}
// Waits as builtins: the compiler counts them, and adds none of its own for what they cover.
__device__ __forceinline__ void wait_loads()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
    asm volatile("" ::: "memory");
}
__device__ __forceinline__ void wait_lds()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    asm volatile("" ::: "memory");
}
__device__ __forceinline__ void tile_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <typename T>
__device__ __forceinline__ T *uniform_ptr(T *p)
{
    const uint64_t u = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)u), hi = __builtin_amdgcn_readfirstlane((uint32_t)(u >> 32));
    return (T *)((uint64_t)hi << 32 | lo);
}

typedef __attribute__((address_space(3))) char lds_char;

// One operand's side of the tile: BR rows, of which each wave uses the FR
// blocks of 16 that start at block wb.
template <bool kDepthMajor, int BR, int FR>
struct TileSide {
    static constexpr int kLoads = BR / 64;             // 1 KiB loads a wave and step
    static constexpr int kBytes = BR * kDepth * 2;     // one buffer
    static constexpr int kGroups = BR / 8;             // 16-byte groups of a depth row (kDepthMajor)
    static constexpr int kAddrs = kDepthMajor ? FR : 2;

    uint32_t off[kLoads];
    uint32_t addr[kAddrs];

    // LDS image, rows with k along them: 128 bytes a row, its 16-byte group c
    // at c ^ (row & 7), so that the 8 rows a read touches at once lie in
    // different banks.  Depth rows: 2 BR bytes each, 32-byte pairs of groups
    // at pair ^ f(k), f = 2 low bits of k and bit 3: the rows that one
    // transposing read touches at once.
    __device__ static int fold(int k) { return (k & 3) | ((k >> 3) & 1) << 2; }

    __device__ void setup(const TileOperand &o, int wb, uint32_t lds)
    {
        const int l = threadIdx.x & 63, w = threadIdx.x >> 6;
        if constexpr (!kDepthMajor) {
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int r = (w + kTileWaves * j) * 8 + (l >> 3);
                off[j] = (uint32_t)(min(r, o.rows - 1)) * (uint32_t)(2 * o.ld) + (uint32_t)(((l & 7) ^ (l >> 3)) * 16);
            }
            const int r = wb * 16 + (l & 15);
#pragma unroll
            for (int h = 0; h < 2; ++h) addr[h] = lds + r * 128 + (((l >> 4) + 4 * h) ^ (l & 7)) * 16;
        } else {
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int e = (w + kTileWaves * j) * 64 + l, k = e / kGroups;
                const int q = (e % kGroups) ^ (fold(k) << 1);
                off[j] = (uint32_t)k * (uint32_t)(2 * o.ld) + (uint32_t)min(q, o.rows / 8 - 1) * 16u;
            }
            const int i = l & 15, k = 8 * (l >> 4) + (i >> 2);
#pragma unroll
            for (int b = 0; b < FR; ++b) addr[b] = lds + k * (2 * BR) + ((wb + b) ^ fold(k)) * 32 + 8 * (i & 3);
        }
    }

    // Issues the loads of one step; `left` = depth rows from the step's first to the end (kDepthMajor).
    __device__ void load(const TileOperand &o, int64_t at, int64_t left, uint32_t lds)
    {
        const uint16_t *p = uniform_ptr(o.base + at);
        const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            uint32_t f = off[j];
            if constexpr (kDepthMajor) {
                if (left < kDepth) {  // the last step of a depth that is no multiple of 64
                    const int l = threadIdx.x & 63, e = (w + kTileWaves * j) * 64 + l, k = e / kGroups;
                    const int q = (e % kGroups) ^ (fold(k) << 1);
                    f = (uint32_t)min(k, (int)left - 1) * (uint32_t)(2 * o.ld) + (uint32_t)min(q, o.rows / 8 - 1) * 16u;
                }
            }
            load_to_lds(p, f, lds + (w + kTileWaves * j) * 1024);
        }
    }

    // The FR blocks of half h from the buffer at byte `buf` past the first.
    template <int kHalf, int kBuf>
    __device__ void read(bf16x8 (&frag)[FR])
    {
#pragma unroll
        for (int b = 0; b < FR; ++b) {
            if constexpr (!kDepthMajor) {
                frag[b] = *(const __attribute__((address_space(3))) bf16x8 *)(uintptr_t)(addr[kHalf] + kBuf * kBytes + b * 2048);
            } else {
                const uint32_t a = addr[b] + kBuf * kBytes + kHalf * 32 * (2 * BR);
                const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(uintptr_t)a);
                const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) s16x4 *)(uintptr_t)(a + 4 * (2 * BR)));
                const s16x8 z = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
                frag[b] = __builtin_bit_cast(bf16x8, z);
            }
        }
    }
};

// Wave (wm, wn) of kWM x kWN holds rows m = (wm FM + i) 16 + 4 (lane / 16) + r
// and columns n = (wn FN + j) 16 + lane % 16 in acc[i][j][r].
template <bool kADepth, bool kBDepth, int BM, int BN, int kWM, int kWN>
struct Tile {
    static_assert(kWM * kWN == kTileWaves, "8 waves");
    static constexpr int FM = BM / kWM / 16, FN = BN / kWN / 16;
    using SideA = TileSide<kADepth, BM, FM>;
    using SideB = TileSide<kBDepth, BN, FN>;
    static constexpr int kLds = 2 * (SideA::kBytes + SideB::kBytes);

    f32x4 acc[FM][FN];

    __device__ static int wave_m() { return (threadIdx.x >> 6) / kWN; }
    __device__ static int wave_n() { return (threadIdx.x >> 6) % kWN; }

    __device__ __forceinline__ void multiply(const bf16x8 (&a)[FM], const bf16x8 (&b)[FN])
    {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
    }

    // depth: valid k (operands with k along their rows are readable, and zero on one side, up to a
    // multiple of 64); planes: 1, or kPlanes for fp32 operands.
    __device__ __forceinline__ void run(const TileOperand &A, const TileOperand &B, int64_t depth, bool planes,
                                        char *smem)
    {
        const uint32_t lds = (uint32_t)(uintptr_t)(lds_char *)smem;
        const uint32_t la = lds, lb = lds + 2 * SideA::kBytes;
        SideA sa;
        SideB sb;
        sa.setup(A, wave_m() * FM, la);
        sb.setup(B, wave_n() * FN, lb);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const int steps = (int)((depth + kDepth - 1) / kDepth) * (planes ? kPlaneProducts : 1);
        if (steps == 0) return;
        int64_t k0 = 0;
        int seg = 0;
        auto load = [&](int buf) {  // the next step into buffer buf
            const int pa = planes ? 0x850 >> (2 * seg) & 3 : 0, pb = planes ? 0x244 >> (2 * seg) & 3 : 0;
            sa.load(A, pa * A.plane + (kADepth ? k0 * A.ld : k0), depth - k0, la + buf * SideA::kBytes);
            sb.load(B, pb * B.plane + (kBDepth ? k0 * B.ld : k0), depth - k0, lb + buf * SideB::kBytes);
            if (!planes || ++seg == kPlaneProducts) {
                seg = 0;
                k0 += kDepth;
            }
        };
        bf16x8 a0[FM], b0[FN], a1[FM], b1[FN];
        load(0);
        wait_loads();
        tile_barrier();
        if (steps > 1) load(1);
        sa.template read<0, 0>(a0);
        sb.template read<0, 0>(b0);
        for (int t = 0; t < steps; t += 2) {
            step<0>(sa, sb, a0, b0, a1, b1, t, steps, load);
            if (t + 1 < steps) step<1>(sa, sb, a0, b0, a1, b1, t + 1, steps, load);
        }
        wait_lds();
        tile_barrier();  // LDS is the caller's now
    }

    template <int kBuf, typename Load>
    __device__ __forceinline__ void step(SideA &sa, SideB &sb, bf16x8 (&a0)[FM], bf16x8 (&b0)[FN], bf16x8 (&a1)[FM],
                                         bf16x8 (&b1)[FN], int t, int steps, Load &load)
    {
        sa.template read<1, kBuf>(a1);
        sb.template read<1, kBuf>(b1);
        __builtin_amdgcn_sched_barrier(0);  // reads first: the products below wait for none of them
        multiply(a0, b0);
        __builtin_amdgcn_sched_barrier(0);
        wait_lds();
        wait_loads();
        tile_barrier();
        if (t + 2 < steps) load(kBuf);
        // after the last step: the buffer of the step before, read and not used
        sa.template read<0, 1 - kBuf>(a0);
        sb.template read<0, 1 - kBuf>(b0);
        __builtin_amdgcn_sched_barrier(0);
        multiply(a1, b1);
        __builtin_amdgcn_sched_barrier(0);
    }
};

}  // namespace csp
