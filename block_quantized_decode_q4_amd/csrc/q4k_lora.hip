// q4k_lora.hip -- low-rank adapters of many requests beside a shared
// projection: y[row] = base[row] + scale_a B_a (A_a x[row]) for the rows of
// adapter a, A_a (r x k) and B_a (n x r) in binary16, a rank of its own
// (ranks[a] <= r) per adapter.
//
// Two launches, because every output needs all of A x: lora_down_kernel
// writes v = scale A x (f32, rows x r rounded up to 16) to the caller's
// workspace, lora_up_kernel adds B v to the base.  Both take tiles of 16 rows
// of one adapter (q4k_groups.h), so an adapter is read once per 16 of its
// rows.
//
// x in binary16 goes through v_mfma_f32_16x16x32_f16; f32 (and bfloat16)
// x through v_mfma_f32_16x16x4_f32 with A widened to f32, as does B v: no
// operand is rounded, the sums are f32.  A row or column of an adapter at or
// beyond its rank is never read, whatever it holds.
//
// Down: the sixteen waves of a workgroup share k, 64 ranks at a time (x is read
// once for r <= 64), and add up their parts in LDS in wave order.  Up: bound
// by reading the base and writing y; B's rows are the matrix operand's rows,
// so a lane holds four consecutive columns of one y row (16-byte accesses).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4k_groups.h"
#include "q4k_kernels.h"

namespace q4k {

namespace {

typedef _Float16 h4_t __attribute__((ext_vector_type(4)));
typedef _Float16 h8_t __attribute__((ext_vector_type(8)));
typedef uint16_t u16x8_t __attribute__((ext_vector_type(8)));
typedef float f4_t __attribute__((ext_vector_type(4)));

constexpr int kTile = 16;              // rows per tile
constexpr int kRanks = 4;              // rank tiles of 16 per down workgroup
constexpr int kDownWaves = 16;

__device__ __forceinline__ int rank_of(const LoraArgs& a, int adapter)
{
    return a.ranks ? min(max(a.ranks[adapter], 0), a.r) : a.r;
}

// The row of position p, -1 for one that is left out
__device__ __forceinline__ int row_of(const LoraArgs& a, int p)
{
    const int r = a.order ? a.order[p] : p;
    return r >= 0 && r < a.rows ? r : -1;
}

// Eight consecutive x elements, as the matrix operands take them
template <int TYPE>
struct X8 {
    f4_t lo, hi;                               // f32 (bfloat16 widened)
};
template <>
struct X8<kTypeF16> {
    h8_t v;
};

template <int TYPE>
__device__ __forceinline__ X8<TYPE> load_x8(const void* base, int64_t at)
{
    X8<TYPE> r;
    if constexpr (TYPE == kTypeF16) {
        r.v = *reinterpret_cast<const h8_t*>(static_cast<const _Float16*>(base) + at);
    } else if constexpr (TYPE == kTypeF32) {
        const float* p = static_cast<const float*>(base) + at;
        r.lo = *reinterpret_cast<const f4_t*>(p);
        r.hi = *reinterpret_cast<const f4_t*>(p + 4);
    } else {
        const u16x8_t v =
            *reinterpret_cast<const u16x8_t*>(static_cast<const uint16_t*>(base) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r.lo[i] = __builtin_bit_cast(float, (uint32_t)v[i] << 16);
            r.hi[i] = __builtin_bit_cast(float, (uint32_t)v[i + 4] << 16);
        }
    }
    return r;
}

// One wave's part of v for the tile: k steps of 32 from wave * 32 on, every
// kDownWaves-th, U of them in flight.  acc[i]: rank tile i.
template <int TYPE, int NT, int U>
__device__ __forceinline__ void down_part(const LoraArgs& a, int64_t xat, bool there, int group,
                                          int rank0, int rank, f4_t* acc)
{
    const int lane = threadIdx.x & 63;
    const int j = lane & 15;
    const int g = lane >> 4;
    // rank tile i: this lane's row of A, read only below the rank
    const _Float16* arow[NT];
    bool has[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int rr = rank0 + 16 * i + j;
        has[i] = rr < rank;
        arow[i] = static_cast<const _Float16*>(a.a) +
                  ((int64_t)group * a.r + (has[i] ? rr : 0)) * a.k;
        acc[i] = f4_t{0.f, 0.f, 0.f, 0.f};
    }
    for (int k0 = (threadIdx.x >> 6) * 32; k0 < a.k; k0 += 32 * kDownWaves * U) {
        X8<TYPE> x[U];
        h8_t w[U][NT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = k0 + u * 32 * kDownWaves + 8 * g;
            const bool in = at < a.k;          // k % 8 == 0: all eight or none
            x[u] = X8<TYPE>{};
            if (there && in) {
                x[u] = load_x8<TYPE>(a.x, xat + at);
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                w[u][i] = h8_t{0, 0, 0, 0, 0, 0, 0, 0};
                if (has[i] && in) {
                    w[u][i] = *reinterpret_cast<const h8_t*>(arow[i] + at);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                if constexpr (TYPE == kTypeF16) {
                    acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[u].v, w[u][i], acc[i], 0, 0,
                                                                    0);
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                            x[u].lo[c], (float)w[u][i][c], acc[i], 0, 0, 0);
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                            x[u].hi[c], (float)w[u][i][c + 4], acc[i], 0, 0, 0);
                    }
                }
            }
        }
    }
}

// v[p][rank] for the tile's positions and 64 ranks from blockIdx.y * 64 on
template <int TYPE>
__global__ void __launch_bounds__(64 * kDownWaves)
lora_down_kernel(LoraArgs a)
{
    __shared__ f4_t part[kDownWaves][kRanks][64];
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int j = lane & 15;
    const int g = lane >> 4;
    const GroupTile t = find_tile<kTile>(a.offsets, a.adapters, a.rows, blockIdx.x);
    if (t.count == 0) {
        return;
    }
    const int rank = rank_of(a, t.group);
    const int rank0 = blockIdx.y * 16 * kRanks;
    if (rank0 >= rank) {
        return;
    }
    const int row = j < t.count ? row_of(a, t.begin + j) : -1;
    const bool there = row >= 0;
    const int64_t xat = (int64_t)(there ? row : 0) * a.k;
    f4_t acc[kRanks];
    // as many rank tiles as the adapter has; steps in flight by the registers
    // that leaves
    const int left = rank - rank0;
    if (left <= 16) {
        down_part<TYPE, 1, TYPE == kTypeF16 ? 8 : 4>(a, xat, there, t.group, rank0, rank, acc);
    } else if (left <= 32) {
        down_part<TYPE, 2, 4>(a, xat, there, t.group, rank0, rank, acc);
    } else {
        down_part<TYPE, 4, TYPE == kTypeF16 ? 4 : 2>(a, xat, there, t.group, rank0, rank, acc);
    }
    const int tiles = left <= 16 ? 1 : left <= 32 ? 2 : 4;
#pragma unroll
    for (int i = 0; i < kRanks; ++i) {
        if (i < tiles) {
            part[wave][i][lane] = acc[i];
        }
    }
    __syncthreads();
    const int i = wave;
    if (i >= kRanks || 16 * i >= left) {
        return;
    }
    f4_t sum = part[0][i][lane];
#pragma unroll
    for (int w = 1; w < kDownWaves; ++w) {
        sum += part[w][i][lane];
    }
    const float scale = a.scales ? a.scales[t.group] : 1.f;
    // D[4 g + c][j]: position 4 g + c, rank j; zero at ranks that are not there
    const int pitch = (a.r + 15) / 16 * 16;
    const int rr = rank0 + 16 * i + j;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int slot = 4 * g + c;
        if (slot < t.count) {
            a.v[(int64_t)(t.begin + slot) * pitch + rr] = rr < rank ? scale * sum[c] : 0.f;
        }
    }
}

// y of the tile's positions, 64 columns per wave from blockIdx.y * 256 on.
// VB: rows of B are multiples of four halves; VY: rows of y and base
// multiples of four floats.  The base is the accumulators' start.
template <bool VB, bool VY>
__global__ void __launch_bounds__(256)
lora_up_kernel(LoraArgs a)
{
    const int lane = threadIdx.x & 63;
    const int j = lane & 15;
    const int g = lane >> 4;
    const int col0 = (int)blockIdx.y * 256 + (threadIdx.x >> 6) * 64;
    const GroupTile t = find_tile<kTile>(a.offsets, a.adapters, a.rows, blockIdx.x);
    if (t.count == 0 || col0 >= a.n) {
        return;
    }
    const int rank = rank_of(a, t.group);
    const int row = j < t.count ? row_of(a, t.begin + j) : -1;
    const int pitch = (a.r + 15) / 16 * 16;
    const float* v = a.v + (int64_t)(t.begin + min(j, t.count - 1)) * pitch + 4 * g;
    // D[4 g + c][j]: column col0 + 16 i + 4 g + c of position j
    f4_t acc[4];
    const _Float16* b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = col0 + 16 * i + 4 * g;
        const int64_t o = (int64_t)row * a.n + at;
        acc[i] = f4_t{0.f, 0.f, 0.f, 0.f};
        if (a.base != nullptr && row >= 0) {
            if constexpr (VY) {
                if (at < a.n) {                        // n % 4 == 0: all four or none
                    acc[i] = *reinterpret_cast<const f4_t*>(a.base + o);
                }
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    acc[i][c] = at + c < a.n ? a.base[o + c] : 0.f;
                }
            }
        }
        // B row of this lane, as a matrix row
        const int col = min(col0 + 16 * i + j, a.n - 1);
        b[i] = static_cast<const _Float16*>(a.b) + ((int64_t)t.group * a.n + col) * a.r + 4 * g;
    }
    for (int k0 = 0; k0 < rank; k0 += 16) {
        const int left = rank - k0 - 4 * g;            // ranks of this lane's four
        const f4_t vv = *reinterpret_cast<const f4_t*>(v + k0);
        h4_t bv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            bv[i] = h4_t{0, 0, 0, 0};
            if (VB && left >= 4) {
                bv[i] = *reinterpret_cast<const h4_t*>(b[i] + k0);
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    bv[i][c] = c < left ? b[i][k0 + c] : (_Float16)0;
                }
            }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32((float)bv[i][c], vv[c], acc[i], 0, 0,
                                                              0);
            }
        }
    }
    if (row < 0) {
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = col0 + 16 * i + 4 * g;
        const int64_t o = (int64_t)row * a.n + at;
        if constexpr (VY) {
            if (at < a.n) {
                *reinterpret_cast<f4_t*>(a.y + o) = acc[i];
            }
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (at + c < a.n) {
                    a.y[o + c] = acc[i][c];
                }
            }
        }
    }
}

}  // namespace

size_t lora_ws_bytes(int64_t rows, int64_t r)
{
    return (size_t)rows * (size_t)((r + 15) / 16 * 16) * sizeof(float);
}

// The grids: at most 2^32 threads, 65535 workgroups along y
bool lora_fits(int64_t rows, int64_t adapters, int64_t n, int64_t r)
{
    const int64_t tiles = most_tiles(rows, adapters, kTile);
    const int64_t down = (r + 16 * kRanks - 1) / (16 * kRanks);
    const int64_t up = (n + 255) / 256;
    const int64_t most = (int64_t)1 << 32;
    return tiles * down * 64 * kDownWaves < most && up <= 65535 && tiles * up * 256 < most;
}

hipError_t launch_lora(const LoraArgs& a, hipStream_t stream)
{
    const unsigned tiles = (unsigned)most_tiles(a.rows, a.adapters, kTile);
    const dim3 down(tiles, (unsigned)((a.r + 16 * kRanks - 1) / (16 * kRanks)));
    const dim3 threads(64 * kDownWaves);
    if (a.x_type == kTypeF16) {
        hipLaunchKernelGGL(lora_down_kernel<kTypeF16>, down, threads, 0, stream, a);
    } else if (a.x_type == kTypeBF16) {
        hipLaunchKernelGGL(lora_down_kernel<kTypeBF16>, down, threads, 0, stream, a);
    } else {
        hipLaunchKernelGGL(lora_down_kernel<kTypeF32>, down, threads, 0, stream, a);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) {
        return e;
    }
    const dim3 up(tiles, (unsigned)((a.n + 255) / 256));
    const bool vb = a.r % 4 == 0;
    const bool vy = a.n % 4 == 0;
    if (vb && vy) {
        hipLaunchKernelGGL((lora_up_kernel<true, true>), up, dim3(256), 0, stream, a);
    } else if (vb) {
        hipLaunchKernelGGL((lora_up_kernel<true, false>), up, dim3(256), 0, stream, a);
    } else if (vy) {
        hipLaunchKernelGGL((lora_up_kernel<false, true>), up, dim3(256), 0, stream, a);
    } else {
        hipLaunchKernelGGL((lora_up_kernel<false, false>), up, dim3(256), 0, stream, a);
    }
    return hipGetLastError();
}

}  // namespace q4k
