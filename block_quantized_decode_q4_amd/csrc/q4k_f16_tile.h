// q4k_f16_tile.h -- a tile of y = x W^T on fp16 mirrors (q4k_f16.hip describes
// the product), for rows grouped by matrix and for products with an epilogue.
// Internal.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace q4k {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t v4u_t __attribute__((ext_vector_type(4)));

constexpr int kGK = 64;                  // k per step

// The grouped products' tile: BM x BN by WM x WN waves, each with a
// (BM / WM) x (BN / WN) part.  A larger side takes less from the L2 and the LDS
// per product, which is what bounds the 128 x 128 tile above (4096 rows in
// eight groups, n 14336, k 4096: 757 us with it, 619 us with 128 x 256 on
// eight waves, 780 TFLOP/s; 256 x 256 617 us, but 20-70 % slower where the
// groups are shorter).  A step takes GK of k (64; 256 where the tiles are few, see
// the rule below).  LDS rows of GK halves without padding, the 16-byte piece c of
// row r at place c ^ r in its low three bits (four from 16 pieces on): neither the
// stores of a row's consecutive bytes nor the reads of a 16 x 32 operand collide.
// One register set: a step has twice the products to hide a load behind.
template <int BM, int BN, int GK, int WM, int WN, typename XRow, typename Put>
__device__ __forceinline__ void
f16_wide_tile(const _Float16* __restrict__ w16, XRow xrow, Put put, int row_w0, int n, int k,
              unsigned char* smem)
{
    constexpr int kThreads = 64 * WM * WN;
    constexpr int kPieces = GK / 8;          // 16-byte pieces of a tile row
    constexpr int kSpread = kPieces < 16 ? 7 : 15;        // the pieces' bits that rows permute
    constexpr int kRows = kThreads / kPieces;             // tile rows per load of all threads
    constexpr int LA = BM / kRows;           // 16-byte loads of the x tile per thread and step
    constexpr int LB = BN / kRows;
    constexpr int FA = BM / WM / 16;         // 16-row MFMA blocks per wave
    constexpr int FB = BN / WN / 16;
    constexpr int kXs = BM * GK * 2;         // LDS bytes of one x tile
    constexpr int kStage = (BM + BN) * GK * 2;
    static_assert(kRows % (kSpread + 1) == 0, "a thread's rows share their permutation");
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = tid >> 6;
    const int wm = wave % WM;
    const int wn = wave / WM;
    const int g = lane >> 4;
    const int j = lane & 15;
    // load role: 16 bytes of a tile row per thread and load
    const _Float16* xsrc[LA];
    const _Float16* wsrc[LB];
    const int lrow = tid / kPieces;
    const int lpiece = tid % kPieces;
    const int loff = lrow * (2 * GK) + ((lpiece ^ (lrow & kSpread)) << 4);
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        xsrc[i] = xrow(lrow + kRows * i) + lpiece * 8;
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
        wsrc[i] = w16 + (int64_t)min(row_w0 + lrow + kRows * i, n - 1) * k + lpiece * 8;
    }
    v4u_t xa[LA], wa[LB];
    auto load = [&](int kb) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < LA; ++i) {
            xa[i] = *reinterpret_cast<const v4u_t*>(xsrc[i] + kb * GK);
        }
#pragma unroll
        for (int i = 0; i < LB; ++i) {
            wa[i] = *reinterpret_cast<const v4u_t*>(wsrc[i] + kb * GK);
        }
    };
    auto stage = [&](int st) __attribute__((always_inline)) {
        unsigned char* base = smem + st * kStage + loff;
#pragma unroll
        for (int i = 0; i < LA; ++i) {
            *reinterpret_cast<v4u_t*>(base + i * (kRows * 2 * GK)) = xa[i];
        }
#pragma unroll
        for (int i = 0; i < LB; ++i) {
            *reinterpret_cast<v4u_t*>(base + kXs + i * (kRows * 2 * GK)) = wa[i];
        }
    };
    f32x4_t acc[FA][FB];
#pragma unroll
    for (int a = 0; a < FA; ++a) {
#pragma unroll
        for (int b = 0; b < FB; ++b) {
            acc[a][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
    }
    const int KB = k / GK;
    load(0);
    stage(0);
    load(min(1, KB - 1));
    __syncthreads();
    for (int kb = 0; kb < KB; ++kb) {
        const unsigned char* xs = smem + (kb & 1) * kStage + ((BM / WM) * wm + j) * (2 * GK);
        const unsigned char* ws = smem + (kb & 1) * kStage + kXs + ((BN / WN) * wn + j) * (2 * GK);
#pragma unroll
        for (int s = 0; s < GK / 32; ++s) {
            const int c = ((4 * s + g) ^ (j & kSpread)) << 4;
            half8_t av[FA], bv[FB];
#pragma unroll
            for (int a = 0; a < FA; ++a) {
                av[a] = *reinterpret_cast<const half8_t*>(xs + a * (32 * GK) + c);
            }
#pragma unroll
            for (int b = 0; b < FB; ++b) {
                bv[b] = *reinterpret_cast<const half8_t*>(ws + b * (32 * GK) + c);
            }
#pragma unroll
            for (int a = 0; a < FA; ++a) {
#pragma unroll
                for (int b = 0; b < FB; ++b) {
                    acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(av[a], bv[b], acc[a][b],
                                                                       0, 0, 0);
                }
            }
        }
        stage((kb + 1) & 1);
        load(min(kb + 2, KB - 1));
        if constexpr (GK == kGK) {
            // the order of a step's instructions (masks: 0x8 matrix, 0x100 LDS
            // read, 0x200 LDS write, 0x20 load): operand reads run ahead of the
            // products that take them, then a store or a load after each product
            // (128 x 256: 639 -> 619 us on the shape below)
            constexpr int kReads = 2 * (FA + FB);
            constexpr int kAhead = FB + 3;
            constexpr int kMfma = 2 * FA * FB;
            __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
            for (int i = 0; i < kReads - kAhead; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x8, 2, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
#pragma unroll
            for (int i = 0; i < LA + LB; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
            }
#pragma unroll
            for (int i = 0; i < LA + LB; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x20, 1, 0);
            }
            __builtin_amdgcn_sched_group_barrier(0x8, kMfma, 0);
        }
        __syncthreads();
    }
    // D[4 g + r][j] of block (a, b)
#pragma unroll
    for (int a = 0; a < FA; ++a) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            put((BM / WM) * wm + 16 * a + 4 * g + r,
                [&](auto out) __attribute__((always_inline)) {
#pragma unroll
                    for (int b = 0; b < FB; ++b) {
                        const int wr = row_w0 + (BN / WN) * wn + 16 * b + j;
                        if (wr < n) {
                            out(wr, acc[a][b][r]);
                        }
                    }
                });
        }
    }
}

}  // namespace q4k
