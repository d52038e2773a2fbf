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
// Depth is walked in steps of 32 through a ring of 5 LDS slots and two register
// sets: while the matrix units work on step h, step h + 1 is read from LDS into
// the other registers, steps h + 2 to h + 4 are on their way, and the loads of
// step h + 5 go into the slot that step h was read from.  One barrier a step:
// every wave has read step h + 1, and its own loads of step h + 2 have landed.
// A load so has three to four steps, of 1024 cycles of the matrix units each,
// to arrive.
//
// 8 waves, two a SIMD: while one issues reads, loads or its epilogue, the other
// feeds the matrix unit (4 waves of 128 x 128 read less from LDS, but LDS is
// not the bound, and every instruction between their products is a gap).  Reads
// and loads are issued between blocks of products, a few at a time.  The
// products are written as asm with their sums tied in place: left to itself
// the compiler moves sums from register to register in the loop.  What it would
// do for them is done by hand: two wait states before a block (operands may
// come from a move), and 16 after a pair of steps (a loop may end there).
//
// fp32 operands are held as three bf16 planes, x = x0 + x1 + x2 with each
// plane the rest rounded to nearest, 24 bits in all.  Six of the nine plane
// products are taken; the three left out are below 2^-25 of |x w|, under the
// rounding of the fp32 sum itself.  They are walked as six pairs of steps in
// place of one.  An operand B of two planes beside a single A takes the first two.
#pragma once

#include <type_traits>

#include "common.h"
#include "device_util.h"

namespace csp {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kDepth = 64;        // k of a pair of steps
constexpr int kStep = 32;         // k of a step
constexpr int kSlots = 5;
constexpr int kTileWaves = 8;
constexpr int kTileThreads = 64 * kTileWaves;
constexpr int kPlanes = 3;        // planes of an fp32 operand
constexpr int kPlaneProducts = 6; // (A, B) planes (0, 0), (0, 1), (1, 0), (1, 1), (0, 2), (2, 0)

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
template <int kLeft = 0>  // all but the last kLeft loads
__device__ __forceinline__ void wait_loads()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (kLeft & 15) | (kLeft >> 4) << 14);
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
    static constexpr int kLoads = BR * kStep * 2 / 1024 / kTileWaves;  // 1 KiB loads a wave and step
    static constexpr int kBytes = BR * kStep * 2;                      // one slot
    static constexpr int kGroups = BR / 8;                             // 16-byte groups of a depth row (kDepthMajor)
    static constexpr int kAddrs = kDepthMajor ? FR : 1;
    static constexpr int kKinds = kDepthMajor ? 2 : 1;

    uint32_t off[kKinds][kLoads];  // kDepthMajor: of even and odd steps (they differ in a last part)
    uint32_t addr[kAddrs];

    // LDS image, rows with k along them: 64 bytes a row, its 16-byte group c
    // at c ^ (row / 2 & 3), so that the 8 rows a read touches at once lie in
    // different banks.  Depth rows: 2 BR bytes each, 32-byte pairs of groups
    // at pair ^ f(k), f = 2 low bits of k and bit 3: the rows that one
    // transposing read touches at once.
    __device__ static int fold(int k) { return (k & 3) | ((k >> 3) & 1) << 2; }

    // Offset of load j of a depth-major step, depth rows from `left` on repeating the one before.
    __device__ static uint32_t depth_off(const TileOperand &o, int j, int left)
    {
        const int e = ((int)(threadIdx.x >> 6) + kTileWaves * j) * 64 + (int)(threadIdx.x & 63), k = e / kGroups;
        const int q = (e % kGroups) ^ (fold(k) << 1);
        return (uint32_t)min(k, left - 1) * (uint32_t)(2 * o.ld) + (uint32_t)min(q, o.rows / 8 - 1) * 16u;
    }

    __device__ void setup(const TileOperand &o, int wb, uint32_t lds)
    {
        const int l = threadIdx.x & 63, w = threadIdx.x >> 6;
        if constexpr (!kDepthMajor) {
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int r = (w + kTileWaves * j) * 16 + (l >> 2);
                off[0][j] = (uint32_t)(min(r, o.rows - 1)) * (uint32_t)(2 * o.ld) + (uint32_t)(((l & 3) ^ (r >> 1 & 3)) * 16);
            }
            const int r = wb * 16 + (l & 15);
            addr[0] = lds + r * 64 + ((l >> 4) ^ (r >> 1 & 3)) * 16;
        } else {
            clamp<0>(o, kStep);
            clamp<1>(o, kStep);
            const int i = l & 15, k = 8 * (l >> 4) + (i >> 2);
#pragma unroll
            for (int b = 0; b < FR; ++b) addr[b] = lds + k * (2 * BR) + ((wb + b) ^ fold(k)) * 32 + 8 * (i & 3);
        }
    }
    template <int kKind>
    __device__ void clamp(const TileOperand &o, int left)
    {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) off[kKind][j] = depth_off(o, j, left);
    }

    // Load j of an even or odd step, from p (uniform) into the slot at lds.
    template <int kKind>
    __device__ void load(const uint16_t *p, int j, uint32_t lds)
    {
        load_to_lds(p, off[kKinds == 2 ? kKind : 0][j], lds + (uint32_t)j * (kTileWaves * 1024));
    }

    // Moves the reads to another slot.
    __device__ void turn(int bytes)
    {
#pragma unroll
        for (int i = 0; i < kAddrs; ++i) addr[i] += (uint32_t)bytes;
    }

    // Block b from the current slot.
    __device__ bf16x8 read(int b)
    {
        if constexpr (!kDepthMajor) {
            return *(const __attribute__((address_space(3))) bf16x8 *)(uintptr_t)(addr[0] + b * 1024);
        } else {
            const uint32_t a = addr[b];
            const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(uintptr_t)a);
            const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4 *)(uintptr_t)(a + 4 * (2 * BR)));
            const s16x8 z = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
            return __builtin_bit_cast(bf16x8, z);
        }
    }
};

// c[j] += a b[j] of 16 x 16 x 32.
__device__ __forceinline__ void products(f32x4 (&c)[4], bf16x8 a, const bf16x8 (&b)[4])
{
    asm volatile("s_nop 1\n\t"
                 "v_mfma_f32_16x16x32_bf16 %0, %4, %5, %0\n\t"
                 "v_mfma_f32_16x16x32_bf16 %1, %4, %6, %1\n\t"
                 "v_mfma_f32_16x16x32_bf16 %2, %4, %7, %2\n\t"
                 "v_mfma_f32_16x16x32_bf16 %3, %4, %8, %3"
                 : "+a"(c[0]), "+a"(c[1]), "+a"(c[2]), "+a"(c[3])
                 : "v"(a), "v"(b[0]), "v"(b[1]), "v"(b[2]), "v"(b[3]));
}

// Wave (wm, wn) of kWM x kWN holds rows m = (wm FM + i) 16 + 4 (lane / 16) + r
// and columns n = (wn FN + j) 16 + lane % 16 in acc[i][j][r].
template <bool kADepth, bool kBDepth, int BM, int BN, int kWM, int kWN>
struct Tile {
    static_assert(kWM * kWN == kTileWaves, "8 waves");
    static constexpr int FM = BM / kWM / 16, FN = BN / kWN / 16;
    using SideA = TileSide<kADepth, BM, FM>;
    using SideB = TileSide<kBDepth, BN, FN>;
    static constexpr int kLds = kSlots * (SideA::kBytes + SideB::kBytes);

    f32x4 acc[FM][FN];

    __device__ static int wave_m() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / kWN; }
    __device__ static int wave_n() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % kWN; }

    // Products of one step, and between their blocks the reads of the next into (an, bn), early enough to be
    // there at the end, and other(i).
    template <typename Other>
    __device__ __forceinline__ void step(SideA &sa, SideB &sb, const bf16x8 (&a)[FM], const bf16x8 (&b)[FN],
                                         bf16x8 (&an)[FM], bf16x8 (&bn)[FN], Other &&other)
    {
        constexpr int kEach = (FM + FN + FM - 3) / (FM - 2);  // all reads under all blocks but two
#pragma unroll
        for (int i = 0; i < FM; ++i) {
#pragma unroll
            for (int r = i * kEach; r < (i + 1) * kEach && r < FM + FN; ++r) {
                if (r < FN) bn[r] = sb.read(r);
                else an[r - FN] = sa.read(r - FN);
            }
            other(i);
            __builtin_amdgcn_sched_barrier(0);
            products(acc[i], a[i], b);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // depth: valid k (operands with k along their rows are readable, and zero on one side, up to a
    // multiple of 64); segs: how many of the plane products are taken (1, 2 or all).
    __device__ __forceinline__ void run(const TileOperand &A, const TileOperand &B, int64_t depth, int segs,
                                        char *smem)
    {
        const uint32_t lds = (uint32_t)(uintptr_t)(lds_char *)smem;
        const uint32_t la = lds, lb = lds + kSlots * SideA::kBytes;
        SideA sa;
        SideB sb;
        sa.setup(A, wave_m() * FM, la);
        sb.setup(B, wave_n() * FN, lb);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const int steps = (int)((depth + kDepth - 1) / kDepth) * segs * 2;  // even
        if (steps == 0) return;
        const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 1024;
        int64_t k0 = 0;
        int seg = 0, made = 0, slot = 0;
        const uint16_t *pa, *pb;
        // Where the operands of the next step begin, an even or odd one; steps past the end repeat the last
        // two.  No branch: the loops below are single blocks, in which the sums keep their registers.
        auto next = [&](auto odd) {
            constexpr int kOdd = decltype(odd)::value;
            const int qa = segs > 2 ? 0x850 >> (2 * seg) & 3 : 0, qb = segs > 1 ? 0x244 >> (2 * seg) & 3 : 0;
            const int64_t k = k0 + kOdd * kStep, kd = k < depth ? k : depth - 1;
            pa = uniform_ptr(A.base + qa * A.plane + (kADepth ? kd * A.ld : k));
            pb = uniform_ptr(B.base + qb * B.plane + (kBDepth ? kd * B.ld : k));
            if constexpr (kOdd) {
                made += 2;
                const bool wrap = seg + 1 == segs, more = made < steps;
                seg = more ? (wrap ? 0 : seg + 1) : seg;
                k0 += more && wrap ? kDepth : 0;
            }
        };
        // load i of that step into the free slot
        constexpr int kAll = SideA::kLoads + SideB::kLoads;
        static_assert(kAll <= FM, "a load for each block of products");
        auto load = [&](auto odd, int i) {
            constexpr int kOdd = decltype(odd)::value;
            if (i < SideA::kLoads) sa.template load<kOdd>(pa, i, la + wave + slot * SideA::kBytes);
            else if (i < kAll) sb.template load<kOdd>(pb, i - SideA::kLoads, lb + wave + slot * SideB::kBytes);
        };
        // Loads from the last part of a depth that is no multiple of 64: steps from `tail` on.
        const int tail = steps - 2 * segs, left = (int)(depth - (depth - 1) / kDepth * kDepth);
        auto clamp = [&](auto odd) {
            constexpr int kOdd = decltype(odd)::value;
            if (left == kDepth) return;
            const int part = kOdd ? (left > kStep ? left - kStep : 1) : left;
            if constexpr (kADepth) sa.template clamp<kOdd>(A, part);
            if constexpr (kBDepth) sb.template clamp<kOdd>(B, part);
        };
        const std::integral_constant<int, 0> even;
        const std::integral_constant<int, 1> odd;
        auto first = [&](int h, auto kind) {
            if (h == tail || (h == 0 && tail < 0)) clamp(even);
            if (h == tail + 1) clamp(odd);
            next(kind);
#pragma unroll
            for (int i = 0; i < kAll; ++i) load(kind, i);
            slot = slot + 1 == kSlots ? 0 : slot + 1;
        };
        first(0, even);
        first(1, odd);
        first(2, even);
        first(3, odd);
        first(4, even);
        bf16x8 a0[FM], b0[FN], a1[FM], b1[FN];
        wait_loads<3 * kAll>();
        tile_barrier();
#pragma unroll
        for (int i = 0; i < FM; ++i) a0[i] = sa.read(i);
#pragma unroll
        for (int j = 0; j < FN; ++j) b0[j] = sb.read(j);
        wait_lds();
        tile_barrier();
        auto turn = [&]() {  // the reads move to slot + 1, then the loads too
            sa.turn(slot + 1 == kSlots ? -(kSlots - 1) * SideA::kBytes : SideA::kBytes);
            sb.turn(slot + 1 == kSlots ? -(kSlots - 1) * SideB::kBytes : SideB::kBytes);
        };
        auto pair = [&]() {
            turn();
            next(odd);
            step(sa, sb, a0, b0, a1, b1, [&](int i) { load(odd, i); });
            wait_lds();
            wait_loads<3 * kAll>();
            tile_barrier();
            slot = slot + 1 == kSlots ? 0 : slot + 1;
            turn();
            next(even);
            step(sa, sb, a1, b1, a0, b0, [&](int i) { load(even, i); });
            asm volatile("s_nop 15");  // the sums are written before anything that follows a loop moves them
            wait_lds();
            wait_loads<3 * kAll>();
            tile_barrier();
            slot = slot + 1 == kSlots ? 0 : slot + 1;
        };
        int h = 0;
        for (; h + 6 < tail; h += 2) pair();
        if (tail > 4) clamp(even);
        if (h < steps && h + 5 < tail) {
            pair();
                h += 2;
        }
        if (tail + 1 > 4) clamp(odd);
        for (; h < steps; h += 2) pair();
        wait_loads();
        wait_lds();
        tile_barrier();  // LDS is the caller's now (the loads that nothing uses have landed)
    }
};

}  // namespace csp
