// q4k_f16_act.hip -- the prompts' products on fp16 mirrors with an epilogue:
//   y = act(x W^T + bias) gate + residual,
// dense or for rows grouped by matrix.  The tile is q4k_f16_dma.h's; here are its
// shapes, the order of the tiles and the choice between them.
//
// Measured (us a call among others; floor: a large matrix product's rate, 1.29
// PFLOP/s, or the bytes):
//   2048 x rows, 14336 x 4096, silu and a binary16 gate, out in binary16  237-243 (187):
//     1.0 PFLOP/s, the matrix pipe busy 51 % of the launch
//   2048 tokens, 2 of 8 experts of 14336 x 4096, the same epilogue  554-589 (373): 0.84
//     PFLOP/s, busy 54 %; the groups' last tiles are part empty
//   509 x rows, 4096 x 14336, bias and residual  97 (46): 256 workgroups of 128 x 64, one
//     per CU, 5.5 MB of operands into each one's LDS; busy 26 %, two thirds of the waves'
//     time waiting to issue
// What bounds them: the operands' way into LDS.  A CU takes in about 31 B a clock at most,
// whatever the stages' size or number, so a tile's time per step is its operands' bytes,
// and a tile as large as the accumulators allow is best; 256 x 256 (256 of them per lane)
// made the compiler spill.  Beside the steps a tile of 128 x 224 takes 13 us for its first
// loads and its epilogue (52 of the 237 us), during which its CU multiplies nothing.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4k_epilogue.h"
#include "q4k_f16_dma.h"
#include "q4k_f16_tile.h"
#include "q4k_groups.h"
#include "q4k_kernels.h"

namespace q4k {

namespace {

constexpr int64_t kCus = 256;
constexpr int64_t kBandTiles = 8;      // tiles of x rows that share a mirror tile's reads

// ------------------------------------------------------------------- kernels
// Workgroup b runs on XCD b % 8: XCD x takes the x-th eighth of the list of tiles,
// which runs over bands of eight tiles of x rows, in them over the mirror's tiles
// and, innermost, the band's: the 32 tiles that an XCD works on share few rows of
// both operands.
template <typename T, bool GATED>
__global__ void __launch_bounds__(T::kThreads, 1)
f16_act_kernel(const _Float16* __restrict__ w16, const _Float16* __restrict__ x16, EpArgs ep,
               int m, int n, int k, int MT, int NT)
{
    extern __shared__ __align__(16) unsigned char smem[];
    const int64_t total = (int64_t)MT * NT;
    const int64_t share = (total + 7) / 8;
    const int64_t at = (int64_t)(blockIdx.x & 7) * share + (blockIdx.x >> 3);
    if ((int64_t)(blockIdx.x >> 3) >= share || at >= total) {
        return;
    }
    const int64_t band = at / (kBandTiles * NT);
    const int64_t in = at % (kBandTiles * NT);
    const int64_t rows = min((int64_t)MT - band * kBandTiles, kBandTiles);
    const int row0 = (int)(band * kBandTiles + in % rows) * T::BM;
    const int col0 = (int)(in / rows) * T::BN;
    const auto xoff = [&](int i) {
        return (uint32_t)min(i, m - 1 - row0) * (uint32_t)(2 * k);
    };
    const auto yrow = [&](int i) { return i < m - row0 ? row0 + i : -1; };
    f16_dma_tile<T, GATED>(w16, x16 + (int64_t)row0 * k, xoff, yrow, ep, ep.bias, col0, n, k, smem);
}

// The x row of a group's position i (-1: left out), and its y row
__device__ __forceinline__ int x_row_of(const GroupRows& rows, const GroupTile& t, int i)
{
    if (i >= t.count) {
        return -1;
    }
    const int r = rows.x_rows ? rows.x_rows[t.begin + i] : t.begin + i;
    return r < 0 || r / rows.x_div >= rows.x_count ? -1 : r / rows.x_div;
}

__device__ __forceinline__ int y_row_of(const GroupRows& rows, const GroupTile& t, int i)
{
    if (x_row_of(rows, t, i) < 0) {
        return -1;
    }
    const int r = rows.y_rows ? rows.y_rows[t.begin + i] : t.begin + i;
    return r < rows.y_count ? r : -1;          // a negative one is left out too
}

// Positions that are left out read x row 0 and are not written.
template <typename T, bool GATED>
__global__ void __launch_bounds__(T::kThreads, 1)
f16_act_grouped_kernel(const _Float16* __restrict__ w16, const _Float16* __restrict__ x16,
                       EpArgs ep, GroupRows rows, int n, int k, int NT)
{
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ int yrows[T::BM];
    const GroupTiles tiles =
        count_tiles<T::BM>(rows.offsets, rows.groups, rows.rows, (int)gridDim.x / NT);
    const GroupWork work =
        find_work<T::BM>(tiles, rows.offsets, rows.groups, rows.rows, NT, blockIdx.x);
    const GroupTile t = work.tile;
    if (t.count == 0) {
        return;
    }
    for (int i = threadIdx.x; i < T::BM; i += T::kThreads) {
        yrows[i] = y_row_of(rows, t, i);       // read after the barriers of the product
    }
    const auto xoff = [&](int i) {
        return (uint32_t)max(x_row_of(rows, t, i), 0) * (uint32_t)(2 * k);
    };
    const auto yrow = [&](int i) { return yrows[i]; };
    const float* const bias = ep.bias != nullptr ? ep.bias + (int64_t)t.group * n : nullptr;
    f16_dma_tile<T, GATED>(w16 + (int64_t)t.group * n * k, x16, xoff, yrow, ep, bias,
                           work.block * T::BN, n, k, smem);
}

// Rows so long, or x so large, that an operand's offsets pass 32 bits: tiles whose
// operands come through registers, by 64-bit addresses.
constexpr int kFarBM = 64, kFarBN = 128;

__global__ void __launch_bounds__(512, 2)
f16_act_far_kernel(const _Float16* __restrict__ w16, const _Float16* __restrict__ x16, EpArgs ep,
                   GroupRows rows, int n, int k, int NT)
{
    extern __shared__ __align__(16) unsigned char smem[];
    GroupWork work;
    if (rows.offsets != nullptr) {
        const GroupTiles tiles =
            count_tiles<kFarBM>(rows.offsets, rows.groups, rows.rows, (int)gridDim.x / NT);
        work = find_work<kFarBM>(tiles, rows.offsets, rows.groups, rows.rows, NT, blockIdx.x);
    } else {                                   // one group of all rows
        const int tile = blockIdx.x / NT;
        work.block = blockIdx.x % NT;
        work.tile = {0, tile * kFarBM, min(kFarBM, rows.rows - tile * kFarBM)};
    }
    const GroupTile t = work.tile;
    if (t.count <= 0) {
        return;
    }
    const auto xrow = [&](int i) { return x16 + (int64_t)max(x_row_of(rows, t, i), 0) * k; };
    const auto put = [&](int i, auto each) {
        const int row = y_row_of(rows, t, i);
        if (row >= 0) {
            each([&](int c, float v) {
                const int64_t at = (int64_t)row * n + c;
                const EpOperands o = ep_fetch(ep, at, (int64_t)t.group * n + c);
                ep_store(ep, at, ep_value(ep, o, v + o.bias));
            });
        }
    };
    f16_wide_tile<kFarBM, kFarBN, kGK, 2, 4>(w16 + (int64_t)t.group * n * k, xrow, put,
                                             work.block * kFarBN, n, k, smem);
}

// --------------------------------------------------------------------- shapes
// us of a round of the chip: per 64 of k, and beside them (one tile per CU, all CUs;
// the operands mostly in the caches), as measured.  The choice takes the least sum over
// the rounds that a call needs; it took the best of all six in each of these (us, silu and a
// binary16 gate, in the order of the table):
//   2048 x 14336 x 4096  252 / 234 / 279 / 400 / 379 / 534 (128 x 224: four full rounds)
//   2048 x 4096 x 14336  212 / 354 / 269 / 379 / 334 / 483 (128 x 256: one full round)
//   1000 x 4096 x 4096    56 /  89 /  38 /  53 /  51 /  61
//   509 x 4096 x 14336   190 / 178 / 133 / 102 /  93 / 128 (256 tiles, the waves along k)
//   200 x 7168 x 4096     47 /  43 /  30 /  23 /  23 /  30
//   64 x 4096 x 4096      46 /  74 /  29 /  20 /  21 /  15
struct ShapeCost {
    int bm, bn;
    bool deep;                         // steps of 128 of k, an even number of them
    double step, fixed;
};

constexpr ShapeCost kShapes[] = {
    {128, 256, false, 0.787, 13.6}, {128, 224, false, 0.708, 13.1}, {128, 128, false, 0.439, 11.2},
    {64, 128, false, 0.30, 9.0},    {128, 64, true, 0.266, 9.9},    {64, 64, true, 0.177, 7.0}};
constexpr int kShapeCount = 6;

template <typename F>
auto with_shape(int shape, F f)
{
    switch (shape) {
    case 0: return f(DmaShape<2, 2, 1, 4, 8, 64, 3>());
    case 1: return f(DmaShape<2, 2, 1, 4, 7, 64, 3>());
    case 2: return f(DmaShape<2, 2, 1, 4, 4, 64, 4>());
    case 3: return f(DmaShape<2, 2, 1, 2, 4, 64, 4>());
    case 4: return f(DmaShape<1, 1, 4, 8, 4, 128, 3>());
    default: return f(DmaShape<1, 1, 4, 4, 4, 128, 4>());
    }
}

// The shape whose rounds take the least time: `tiles` of x rows by their height
template <typename Tiles>
int best_shape(Tiles tiles, int64_t n, int64_t k)
{
    int best = 0;
    double least = 0;
    for (int s = 0; s < kShapeCount; ++s) {
        const ShapeCost& c = kShapes[s];
        if (c.deep && k % 256 != 0) {
            continue;
        }
        const double count = (double)tiles(c.bm) * (double)((n + c.bn - 1) / c.bn);
        const double rounds = (double)(int64_t)((count + kCus - 1) / kCus);
        const double us = rounds * ((double)(k / 64) * c.step + c.fixed);
        if (s == 0 || us < least) {
            best = s;
            least = us;
        }
    }
    return best;
}

int dense_shape(int64_t m, int64_t n, int64_t k)
{
    return best_shape([&](int64_t bm) { return (m + bm - 1) / bm; }, n, k);
}

// Tiles to expect: a group of any length ends half a tile early
int grouped_shape(int64_t rows, int64_t groups, int64_t n, int64_t k)
{
    const int64_t ends = groups < rows ? groups : rows;
    return best_shape([&](int64_t bm) { return (2 * rows / bm + ends + 1) / 2; }, n, k);
}

// Offsets within an operand that pass 32 bits
bool far(int64_t x_rows, int64_t k)
{
    return k > ((int64_t)1 << 22) || x_rows > ((int64_t)1 << 31) / k;
}

bool gated(const EpArgs& ep)
{
    return ep.gate != nullptr && ep.gate_type == kTypeF16 && ep.residual == nullptr;
}

int64_t far_grid(int64_t rows, int64_t groups, int64_t n)
{
    return (most_tiles(rows, groups, kFarBM) * ((n + kFarBN - 1) / kFarBN) + 7) / 8 * 8;
}

hipError_t launch_far(const void* w16, const void* x16, const EpArgs& ep, const GroupRows& g, int n,
                      int k, hipStream_t stream)
{
    const int NT = (n - 1) / kFarBN + 1;
    hipLaunchKernelGGL(f16_act_far_kernel, dim3((unsigned)far_grid(g.rows, g.groups, n)), dim3(512),
                       2 * (kFarBM + kFarBN) * kGK * 2, stream, static_cast<const _Float16*>(w16),
                       static_cast<const _Float16*>(x16), ep, g, n, k, NT);
    return hipGetLastError();
}

}  // namespace

// The workgroups of a launch, 512 threads at most each
int64_t f16_act_grid(int64_t m, int64_t n, int64_t k)
{
    if (far(128, k)) {
        return far_grid(m, 1, n);
    }
    const ShapeCost& c = kShapes[dense_shape(m, n, k)];
    return (((m + c.bm - 1) / c.bm) * ((n + c.bn - 1) / c.bn) + 7) / 8 * 8;
}

hipError_t launch_f16_gemm_act(const void* w16, const void* x16, const EpArgs& ep, int m, int n,
                               int k, hipStream_t stream)
{
    if (far(128, k)) {                         // offsets are within a tile of x
        const GroupRows all = {nullptr, nullptr, nullptr, 1, m, 1, m, m};
        return launch_far(w16, x16, ep, all, n, k, stream);
    }
    return with_shape(dense_shape(m, n, k), [&](auto shape) {
        using T = decltype(shape);
        const int MT = (m - 1) / T::BM + 1, NT = (n - 1) / T::BN + 1;
        const auto kernel = gated(ep) ? f16_act_kernel<T, true> : f16_act_kernel<T, false>;
        hipLaunchKernelGGL(kernel, dim3((unsigned)f16_act_grid(m, n, k)), dim3(T::kThreads),
                           T::kLds, stream, static_cast<const _Float16*>(w16),
                           static_cast<const _Float16*>(x16), ep, m, n, k, MT, NT);
        return hipGetLastError();
    });
}

int64_t f16_grouped_act_grid(int64_t rows, int64_t groups, int64_t x_count, int64_t n, int64_t k)
{
    if (far(x_count, k)) {
        return far_grid(rows, groups, n);
    }
    const ShapeCost& c = kShapes[grouped_shape(rows, groups, n, k)];
    return (most_tiles(rows, groups, c.bm) * ((n + c.bn - 1) / c.bn) + 7) / 8 * 8;
}

hipError_t launch_f16_grouped_act(const void* w16, const void* x16, const EpArgs& ep,
                                  const GroupRows& g, int n, int k, hipStream_t stream)
{
    if (far(g.x_count, k)) {
        return launch_far(w16, x16, ep, g, n, k, stream);
    }
    return with_shape(grouped_shape(g.rows, g.groups, n, k), [&](auto shape) {
        using T = decltype(shape);
        const auto kernel =
            gated(ep) ? f16_act_grouped_kernel<T, true> : f16_act_grouped_kernel<T, false>;
        hipLaunchKernelGGL(kernel,
                           dim3((unsigned)f16_grouped_act_grid(g.rows, g.groups, g.x_count, n, k)),
                           dim3(T::kThreads), T::kLds, stream, static_cast<const _Float16*>(w16),
                           static_cast<const _Float16*>(x16), ep, g, n, k, (n - 1) / T::BN + 1);
        return hipGetLastError();
    });
}

}  // namespace q4k
