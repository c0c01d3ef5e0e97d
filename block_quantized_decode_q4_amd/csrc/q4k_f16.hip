// q4k_f16.hip -- the prefill step beside the decode GEMV: a row-major fp16
// mirror of the weights (built by the dequant kernels of q4k_kernels.hip and
// q4k_q6k.hip) times fp16 activations on the matrix cores, f32 accumulation
// (memra-engine 0.83.1, src/f16_ffi.rs: `memra_f16_cvt`, the f32 -> fp16
// activation convert; `memra_f16_pp_gemm` / `try_f16_gemm`,
// y[m, n] = x[m, k] @ (fp16 W)^T, f32 accumulate, for prefill batches), and the
// same product for rows grouped by matrix (the experts of a prompt).
//
// GEMM: a 256-thread workgroup computes a 128 x 128 tile of y (128 vectors x
// 128 weight rows; 64 x 128 or 64 x 64 when that gives too few tiles to
// fill the chip) over k in steps of 64: both operands are k-contiguous
// (x rows and mirror rows), staged through LDS in rows of 64 halves padded
// to 144 bytes (consecutive rows start 16 bytes apart in the banks), two
// LDS stages and two register sets of loaded tiles, so a step's global
// loads have two steps of MFMAs to arrive in.  (Mirror blocks loaded by
// each wave straight into its operand registers, with only x staged,
// measured 1.5-2.3 x slower.)  Wave
// (wm, wn) of the 2 x 2 layout holds a quarter of the tile (64 x 64 for
// 128 x 128) as 16 x 16 blocks of v_mfma_f32_16x16x32_f16 accumulators: lane l = 16 g + j holds
// A[i = j][k = 8 g .. 8 g + 7] (an x row), B[k = 8 g .. 8 g + 7][j] (a
// mirror row) and D[4 g + r][j].  Workgroups that share a block of mirror
// rows run on the same XCD one after another (its L2 serves the repeats):
// the mirror, the large operand, is read from HBM about once.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>
#include <mutex>

#include "q4k_groups.h"
#include "q4k_kernels.h"

namespace q4k {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t v4u_t __attribute__((ext_vector_type(4)));

constexpr int kGK = 64;                  // k per step
constexpr int kGRow = kGK * 2 + 16;      // LDS bytes per staged row (padded)
constexpr int kGXcd = 8;                 // XCDs: workgroups go round-robin over them

// f32 -> fp16, round to nearest even (inf beyond the fp16 range, NaN kept).
__global__ void __launch_bounds__(256)
f16_cvt_kernel(const float* __restrict__ x, _Float16* __restrict__ out, int64_t count)
{
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i + 4 <= count) {
        const float4 v = *reinterpret_cast<const float4*>(x + i);
        typedef _Float16 h4_t __attribute__((ext_vector_type(4)));
        const h4_t h = {(_Float16)v.x, (_Float16)v.y, (_Float16)v.z, (_Float16)v.w};
        *reinterpret_cast<h4_t*>(out + i) = h;
    } else {
        for (int64_t t = i; t < count; ++t) {
            out[t] = (_Float16)x[t];
        }
    }
}

// y[b * n + r] = sum_c w16[r * k + c] x16[b * k + c] (f32 accumulation).
// Tiles of BM x rows by BN mirror rows (64 or 128 each); four waves in a
// 2 x 2 layout, each with (BM / 32) x (BN / 32) MFMA blocks of 16 x 16.
// Grid: kGXcd * ceil(NT / kGXcd) * MT workgroups (MT, NT: tiles of x rows
// and of mirror rows); k % 64 == 0.
template <int BM, int BN>
__global__ void __launch_bounds__(256, 2)
f16_gemm_kernel(const _Float16* __restrict__ w16, const _Float16* __restrict__ x16,
                float* __restrict__ y, int m, int n, int k, int MT, int NT)
{
    static_assert((BM == 64 || BM == 128) && (BN == 64 || BN == 128), "tile");
    constexpr int LA = BM / 32;              // 16-byte loads of the x tile per thread and step
    constexpr int LB = BN / 32;
    constexpr int FA = BM / 32;              // 16-row MFMA blocks per wave
    constexpr int FB = BN / 32;
    constexpr int kXs = BM * kGRow;          // LDS bytes of one x tile
    constexpr int kStage = (BM + BN) * kGRow;
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = tid >> 6;
    // XCD-aware tile order: workgroup b runs on XCD b % 8; within an XCD
    // the x tiles of one mirror tile follow each other
    const int bid = blockIdx.x;
    const int xcd = bid % kGXcd;
    const int local = bid / kGXcd;
    const int tm = local % MT;
    const int tn = (local / MT) * kGXcd + xcd;
    if (tn >= NT) {
        return;
    }
    const int row_x0 = tm * BM;
    const int row_w0 = tn * BN;

    // load role: 16 bytes of a tile row per thread and load (tile row
    // idx / 8, 16-byte chunk idx % 8 of its 128 bytes)
    const _Float16* xsrc[LA];
    const _Float16* wsrc[LB];
    int xoff[LA], woff[LB];
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        const int idx = tid + 256 * i;
        xsrc[i] = x16 + (int64_t)min(row_x0 + (idx >> 3), m - 1) * k + (idx & 7) * 8;
        xoff[i] = (idx >> 3) * kGRow + (idx & 7) * 16;
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
        const int idx = tid + 256 * i;
        wsrc[i] = w16 + (int64_t)min(row_w0 + (idx >> 3), n - 1) * k + (idx & 7) * 8;
        woff[i] = kXs + (idx >> 3) * kGRow + (idx & 7) * 16;
    }
    // kSets register sets of loaded tiles: a set is refilled with the loads
    // of step kb + 1 + kSets right after its tiles of step kb + 1 are staged,
    // so a load has kSets steps of MFMAs to arrive in
    constexpr int kSets = 2;
    static_assert(kSets == 2, "the step loop below alternates two sets");
    v4u_t xa[kSets][LA], wa[kSets][LB];
    auto load = [&](int kb, auto set) __attribute__((always_inline)) {
        constexpr int q = decltype(set)::value;
#pragma unroll
        for (int i = 0; i < LA; ++i) {
            xa[q][i] = *reinterpret_cast<const v4u_t*>(xsrc[i] + kb * kGK);
        }
#pragma unroll
        for (int i = 0; i < LB; ++i) {
            wa[q][i] = *reinterpret_cast<const v4u_t*>(wsrc[i] + kb * kGK);
        }
    };
    auto stage = [&](int st, auto set) __attribute__((always_inline)) {
        constexpr int q = decltype(set)::value;
        unsigned char* base = smem + st * kStage;
#pragma unroll
        for (int i = 0; i < LA; ++i) {
            *reinterpret_cast<v4u_t*>(base + xoff[i]) = xa[q][i];
        }
#pragma unroll
        for (int i = 0; i < LB; ++i) {
            *reinterpret_cast<v4u_t*>(base + woff[i]) = wa[q][i];
        }
    };

    // compute role: wave (wm, wn), lane (g, j)
    const int wm = wave & 1;
    const int wn = wave >> 1;
    const int g = lane >> 4;
    const int j = lane & 15;
    f32x4_t acc[FA][FB];
#pragma unroll
    for (int a = 0; a < FA; ++a) {
#pragma unroll
        for (int b = 0; b < FB; ++b) {
            acc[a][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
    }
    const int KB = k / kGK;
    // set q holds steps q, q + kSets, q + 2 kSets, ...  Prologue: steps
    // 0 .. kSets - 1 into the sets (past the end the last step again: no
    // branch around a load), step 0 staged and its set refilled with step
    // kSets
    load(0, std::integral_constant<int, 0>());
    load(min(1, KB - 1), std::integral_constant<int, 1>());
    stage(0, std::integral_constant<int, 0>());
    load(min(kSets, KB - 1), std::integral_constant<int, 0>());
    __syncthreads();
    // step kb: its tiles are in LDS stage kb & 1; set (kb + 1) % kSets holds
    // step kb + 1, staged after the MFMAs into the other stage and then
    // refilled with step kb + 1 + kSets
    auto step = [&](int kb, auto nset) __attribute__((always_inline)) {
        const int st = kb & 1;
        const unsigned char* xs = smem + st * kStage;
        const unsigned char* ws = xs + kXs;
#pragma unroll
        for (int s = 0; s < kGK / 32; ++s) {
            half8_t av[FA], bv[FB];
#pragma unroll
            for (int a = 0; a < FA; ++a) {
                av[a] = *reinterpret_cast<const half8_t*>(
                    xs + ((BM / 2) * wm + 16 * a + j) * kGRow + (32 * s + 8 * g) * 2);
            }
#pragma unroll
            for (int b = 0; b < FB; ++b) {
                bv[b] = *reinterpret_cast<const half8_t*>(
                    ws + ((BN / 2) * wn + 16 * b + j) * kGRow + (32 * s + 8 * g) * 2);
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
        stage(st ^ 1, nset);
        load(min(kb + 1 + kSets, KB - 1), nset);
        __syncthreads();
    };
    for (int kb = 0; kb < KB; kb += kSets) {
        step(kb, std::integral_constant<int, 1>());
        if (kb + 1 < KB) {
            step(kb + 1, std::integral_constant<int, 0>());
        }
    }
    // D[4 g + r][j] of block (a, b): x row (BM / 2) wm + 16 a + 4 g + r,
    // mirror row (BN / 2) wn + 16 b + j
#pragma unroll
    for (int a = 0; a < FA; ++a) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int xr = row_x0 + (BM / 2) * wm + 16 * a + 4 * g + r;
            if (xr < m) {
#pragma unroll
                for (int b = 0; b < FB; ++b) {
                    const int wr = row_w0 + (BN / 2) * wn + 16 * b + j;
                    if (wr < n) {
                        y[(int64_t)xr * n + wr] = acc[a][b][r];
                    }
                }
            }
        }
    }
}

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

// The same product for rows grouped by matrix: a tile holds up to BM positions
// of one group, its mirror is the group's; NT column blocks of BN.  Positions
// that are left out read x row 0 and are not written.
template <int BM, int BN, int GK, int WM, int WN>
__global__ void __launch_bounds__(64 * WM * WN, WM * WN / 4)
f16_gemm_grouped_kernel(const _Float16* __restrict__ w16, const _Float16* __restrict__ x16,
                        float* __restrict__ y, GroupRows rows, int n, int k, int NT)
{
    extern __shared__ __align__(16) unsigned char smem[];
    const GroupTiles tiles =
        count_tiles<BM>(rows.offsets, rows.groups, rows.rows, (int)gridDim.x / NT);
    const GroupWork work =
        find_work<BM>(tiles, rows.offsets, rows.groups, rows.rows, NT, blockIdx.x);
    const GroupTile t = work.tile;
    if (t.count == 0) {
        return;
    }
    auto x_row = [&](int i) -> int {            // -1: left out
        if (i >= t.count) {
            return -1;
        }
        const int p = t.begin + i;
        const int r = rows.x_rows ? rows.x_rows[p] : p;
        return r < 0 || r / rows.x_div >= rows.x_count ? -1 : r / rows.x_div;
    };
    const auto xrow = [&](int i) { return x16 + (int64_t)max(x_row(i), 0) * k; };
    const auto put = [&](int i, auto each) {
        if (x_row(i) >= 0) {
            const int r = rows.y_rows ? rows.y_rows[t.begin + i] : t.begin + i;
            if (r >= 0 && r < rows.y_count) {
                float* const out = y + (int64_t)r * n;
                each([&](int c, float v) { out[c] = v; });
            }
        }
    };
    const _Float16* const w = w16 + (int64_t)t.group * n * k;
    f16_wide_tile<BM, BN, GK, WM, WN>(w, xrow, put, work.block * BN, n, k, smem);
}

hipError_t launch_f16_cvt(const float* x, void* out, int64_t count, hipStream_t stream)
{
    const int64_t blocks = (count + 1023) / 1024;
    hipLaunchKernelGGL(f16_cvt_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, x,
                       static_cast<_Float16*>(out), count);
    return hipGetLastError();
}

// The tile: 128 x 128 while that gives at least 384 tiles (about 1.5 per
// CU), else 64 x 128 while that gives a tile for every CU (a wave's 32 x 64
// block reads a third less LDS per flop than 32 x 32: m 512, n 4096,
// k 14336 in 100 us against 105 us on 64 x 64), else 64 x 64 (more,
// smaller tiles for short m or n with long k).
void f16_gemm_tile(int64_t m, int64_t n, int* bm, int* bn)
{
    auto tiles = [&](int a, int b) { return ((m + a - 1) / a) * ((n + b - 1) / b); };
    if (tiles(128, 128) >= 384) {
        *bm = 128; *bn = 128;
    } else if (tiles(64, 128) >= 256) {
        *bm = 64; *bn = 128;
    } else {
        *bm = 64; *bn = 64;
    }
}

size_t f16_gemm_lds_bytes(int bm, int bn)
{
    return (size_t)2 * (bm + bn) * kGRow;
}

int64_t f16_gemm_grid(int64_t m, int64_t n)
{
    int bm, bn;
    f16_gemm_tile(m, n, &bm, &bn);
    const int64_t MT = (m + bm - 1) / bm;
    const int64_t NT = (n + bn - 1) / bn;
    return kGXcd * ((NT + kGXcd - 1) / kGXcd) * MT;
}

template <int BM, int BN>
static hipError_t launch_f16_gemm_t(const void* w16, const void* x16, float* y, int m, int n,
                                    int k, hipStream_t stream)
{
    const int MT = (m + BM - 1) / BM;
    const int NT = (n + BN - 1) / BN;
    const int64_t grid = kGXcd * ((int64_t)(NT + kGXcd - 1) / kGXcd) * MT;
    hipLaunchKernelGGL((f16_gemm_kernel<BM, BN>), dim3((unsigned)grid), dim3(256),
                       f16_gemm_lds_bytes(BM, BN), stream, static_cast<const _Float16*>(w16),
                       static_cast<const _Float16*>(x16), y, m, n, k, MT, NT);
    return hipGetLastError();
}

hipError_t launch_f16_gemm(const void* w16, const void* x16, float* y, int m, int n, int k,
                           hipStream_t stream)
{
    int bm, bn;
    f16_gemm_tile(m, n, &bm, &bn);
    if (bm == 128) {
        return launch_f16_gemm_t<128, 128>(w16, x16, y, m, n, k, stream);
    }
    if (bn == 128) {
        return launch_f16_gemm_t<64, 128>(w16, x16, y, m, n, k, stream);
    }
    return launch_f16_gemm_t<64, 64>(w16, x16, y, m, n, k, stream);
}

// The tile.  64 x 128 where the groups are short or the tiles few: a product is
// mostly the mirror's bytes then (128 x 256 against 64 x 128 at 64 positions a
// group and 176 tiles 84 / 75 us, at 256 positions and 46 tiles 23 / 14 us; at 256
// positions and 176 tiles 71 / 88 us).  Else 128 rows by 256 or 192 columns, which
// are as fast per column; one workgroup of the first fits a CU, two of the second.
// 256 while the rounds of the chip times the columns of one say so (a group of any
// length ends half a tile early), up to four rounds; beyond, 192, whose last round
// is shorter.  256 / 192 columns, uneven groups: 19 tiles of n = k = 4096 138 / 114
// us, 25 tiles of n 4096, k 2048 85 / 91 us, 95 tiles of n 1001, k 2048 94 / 102 us, 37
// tiles of n 14336, k 4096 633 / 594 us, 36 tiles 593 / 598 us.
// Where even 64 columns leave CUs without work, a step's latency is what counts:
// 256 of k a step instead of 64, and 32 or 64 rows by 64 columns (68 rows in five
// groups, n 398, k 7168: 64 x 128 / 32 x 64 / 64 x 64 47 / 26 / 33 us; 910 rows in 23,
// n 534, k 8192: 87 / 70 / 54 us; more tiles than CUs, 400 rows in eight groups, n = k
// = 2048: 29 / 35 / 33 us).
constexpr int64_t kCus = 256;
constexpr int kDeepGK = 256;

struct F16GroupedTile {
    int rows, columns, depth;
};

static F16GroupedTile f16_grouped_tile(int64_t rows, int64_t groups, int64_t n, int64_t k)
{
    // twice the tiles to expect: a group of any length ends half a tile early
    const int64_t ends = groups < rows ? groups : rows;
    auto halves = [&](int64_t tile) { return 2 * rows / tile + ends; };
    const int64_t columns64 = (n + 63) / 64;
    if (k % kDeepGK == 0 && halves(32) * columns64 <= 2 * kCus) {
        return {32, 64, kDeepGK};
    }
    if (k % kDeepGK == 0 && halves(64) * columns64 <= 2 * kCus) {
        return {64, 64, kDeepGK};
    }
    if (rows < 96 * groups || most_tiles(rows, groups, 128) * ((n + 255) / 256) < 128) {
        return {64, 128, kGK};
    }
    const int64_t wide = halves(128) * ((n + 255) / 256);
    const int64_t narrow = halves(128) * ((n + 191) / 192);
    auto rounds = [](int64_t half_tiles) { return (half_tiles + 2 * kCus - 1) / (2 * kCus); };
    if (rounds(narrow) > 4 || rounds(narrow) * 192 < rounds(wide) * 256) {
        return {128, 192, kGK};
    }
    return {128, 256, kGK};
}

int64_t f16_grouped_grid(int64_t rows, int64_t groups, int64_t n, int64_t k)
{
    const F16GroupedTile t = f16_grouped_tile(rows, groups, n, k);
    return (most_tiles(rows, groups, t.rows) * ((n + t.columns - 1) / t.columns) + 7) / 8 * 8;
}

template <int BM, int BN, int GK, int WM, int WN>
static hipError_t launch_f16_grouped_t(const void* w16, const void* x16, float* y,
                                       const GroupRows& g, int n, int k, hipStream_t stream)
{
    const int NT = (n + BN - 1) / BN;
    const int64_t grid = f16_grouped_grid(g.rows, g.groups, n, k);
    hipLaunchKernelGGL((f16_gemm_grouped_kernel<BM, BN, GK, WM, WN>), dim3((unsigned)grid),
                       dim3(64 * WM * WN), 2 * (BM + BN) * GK * 2, stream,
                       static_cast<const _Float16*>(w16), static_cast<const _Float16*>(x16), y, g,
                       n, k, NT);
    return hipGetLastError();
}

hipError_t launch_f16_gemm_grouped(const void* w16, const void* x16, float* y, const GroupRows& g,
                                   int n, int k, hipStream_t stream)
{
    const F16GroupedTile t = f16_grouped_tile(g.rows, g.groups, n, k);
    if (t.columns == 256) {
        return launch_f16_grouped_t<128, 256, kGK, 2, 4>(w16, x16, y, g, n, k, stream);
    }
    if (t.columns == 192) {
        return launch_f16_grouped_t<128, 192, kGK, 2, 4>(w16, x16, y, g, n, k, stream);
    }
    if (t.columns == 128) {
        return launch_f16_grouped_t<64, 128, kGK, 2, 4>(w16, x16, y, g, n, k, stream);
    }
    if (t.rows == 64) {
        return launch_f16_grouped_t<64, 64, kDeepGK, 2, 4>(w16, x16, y, g, n, k, stream);
    }
    return launch_f16_grouped_t<32, 64, kDeepGK, 2, 4>(w16, x16, y, g, n, k, stream);
}

// ------------------------------------------------- allocation-free variant
// The fp16 activations of q4k_f16_gemm_f32x_noalloc live in this array, one
// copy per device, kept until the process ends.  In host code `scratch` is
// only a stand-in for the symbol: its device address comes from
// hipGetSymbolAddress, looked up once per device with that device current.
static __device__ __align__(256) _Float16 scratch[kScratchHalves];

namespace {
constexpr int kScratchDevices = 64;
std::atomic<void*> g_scratch[kScratchDevices];
std::mutex g_scratch_lock;
}  // namespace

hipError_t f16_scratch(void** out)
{
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) {
        return e;
    }
    if (dev < 0 || dev >= kScratchDevices) {
        return hipErrorInvalidDevice;
    }
    void* p = g_scratch[dev].load(std::memory_order_acquire);
    if (p == nullptr) {
        std::lock_guard<std::mutex> lk(g_scratch_lock);
        p = g_scratch[dev].load(std::memory_order_relaxed);
        if (p == nullptr) {
            e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
            if (e != hipSuccess) {
                return e;
            }
            g_scratch[dev].store(p, std::memory_order_release);
        }
    }
    *out = p;
    return hipSuccess;
}

}  // namespace q4k
