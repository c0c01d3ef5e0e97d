// q4k_f16_act.hip -- the prompts' products on fp16 mirrors with an epilogue:
//   y = act(x W^T + bias) gate + residual,
// dense or for rows grouped by matrix.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4k_epilogue.h"
#include "q4k_f16_tile.h"
#include "q4k_groups.h"
#include "q4k_kernels.h"

namespace q4k {

namespace {

constexpr int kXcd = 8;

template <int BM, int BN>
__global__ void __launch_bounds__(512, 2)
f16_act_kernel(const _Float16* __restrict__ w16, const _Float16* __restrict__ x16, EpArgs ep,
               int m, int n, int k, int MT, int NT)
{
    extern __shared__ __align__(16) unsigned char smem[];
    const int xcd = blockIdx.x % kXcd;
    const int local = blockIdx.x / kXcd;
    const int tm = local % MT;
    const int tn = (local / MT) * kXcd + xcd;
    if (tn >= NT) {
        return;
    }
    const int row0 = tm * BM;
    const auto xrow = [&](int i) { return x16 + (int64_t)min(row0 + i, m - 1) * k; };
    const auto put = [&](int i, auto each) {
        if (row0 + i < m) {
            const int64_t at = (int64_t)(row0 + i) * n;
            each([&](int c, float v) {
                const float z = v + (ep.bias != nullptr ? ep.bias[c] : 0.f);
                ep_store(ep, at + c, ep_value(ep, at + c, z));
            });
        }
    };
    f16_wide_tile<BM, BN, kGK, 2, 4>(w16, xrow, put, tn * BN, n, k, smem);
}

template <int BM, int BN>
__global__ void __launch_bounds__(512, 2)
f16_act_grouped_kernel(const _Float16* __restrict__ w16, const _Float16* __restrict__ x16,
                       EpArgs ep, GroupRows rows, int n, int k, int NT)
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
                const int64_t at = (int64_t)r * n;
                each([&](int c, float v) {
                    const float z =
                        v + (ep.bias != nullptr ? ep.bias[(int64_t)t.group * n + c] : 0.f);
                    ep_store(ep, at + c, ep_value(ep, at + c, z));
                });
            }
        }
    };
    f16_wide_tile<BM, BN, kGK, 2, 4>(w16 + (int64_t)t.group * n * k, xrow, put, work.block * BN, n,
                                     k, smem);
}

constexpr int kBM = 64, kBN = 128;

}  // namespace

int64_t f16_act_grid(int64_t m, int64_t n, int64_t)
{
    const int64_t NT = (n + kBN - 1) / kBN;
    return kXcd * ((NT + kXcd - 1) / kXcd) * ((m + kBM - 1) / kBM);
}

hipError_t launch_f16_gemm_act(const void* w16, const void* x16, const EpArgs& ep, int m, int n,
                               int k, hipStream_t stream)
{
    hipLaunchKernelGGL((f16_act_kernel<kBM, kBN>), dim3((unsigned)f16_act_grid(m, n, k)),
                       dim3(512), 2 * (kBM + kBN) * kGK * 2, stream,
                       static_cast<const _Float16*>(w16), static_cast<const _Float16*>(x16), ep, m,
                       n, k, (m + kBM - 1) / kBM, (n + kBN - 1) / kBN);
    return hipGetLastError();
}

int64_t f16_grouped_act_grid(int64_t rows, int64_t groups, int64_t n, int64_t)
{
    return (most_tiles(rows, groups, kBM) * ((n + kBN - 1) / kBN) + 7) / 8 * 8;
}

hipError_t launch_f16_grouped_act(const void* w16, const void* x16, const EpArgs& ep,
                                  const GroupRows& g, int n, int k, hipStream_t stream)
{
    hipLaunchKernelGGL((f16_act_grouped_kernel<kBM, kBN>),
                       dim3((unsigned)f16_grouped_act_grid(g.rows, g.groups, n, k)), dim3(512),
                       2 * (kBM + kBN) * kGK * 2, stream, static_cast<const _Float16*>(w16),
                       static_cast<const _Float16*>(x16), ep, g, n, k, (n + kBN - 1) / kBN);
    return hipGetLastError();
}

}  // namespace q4k
