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
// Down: the eight waves of a workgroup share k, 64 ranks at a time (x is read
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
typedef uint16_t u16x4_t __attribute__((ext_vector_type(4)));
typedef float f4_t __attribute__((ext_vector_type(4)));

constexpr int kTile = 16;              // rows per tile
constexpr int kRanks = 4;              // rank tiles of 16 per down workgroup
constexpr int kDownWaves = 8;

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

// Four x elements as f32
template <int TYPE>
__device__ __forceinline__ f4_t load_x4(const void* base, int64_t at)
{
    if constexpr (TYPE == kTypeF32) {
        return *reinterpret_cast<const f4_t*>(static_cast<const float*>(base) + at);
    } else {                                   // bfloat16
        const u16x4_t v =
            *reinterpret_cast<const u16x4_t*>(static_cast<const uint16_t*>(base) + at);
        f4_t r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r[i] = __builtin_bit_cast(float, (uint32_t)v[i] << 16);
        }
        return r;
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
    // rank tile i: this lane's row of A, read only below the rank
    const _Float16* arow[kRanks];
    bool has[kRanks];
#pragma unroll
    for (int i = 0; i < kRanks; ++i) {
        const int rr = rank0 + 16 * i + j;
        has[i] = rr < rank;
        arow[i] = static_cast<const _Float16*>(a.a) +
                  ((int64_t)t.group * a.r + (has[i] ? rr : 0)) * a.k;
    }
    f4_t acc[kRanks];
#pragma unroll
    for (int i = 0; i < kRanks; ++i) {
        acc[i] = f4_t{0.f, 0.f, 0.f, 0.f};
    }
    if constexpr (TYPE == kTypeF16) {
        const _Float16* x = static_cast<const _Float16*>(a.x) + xat;
        for (int kb = wave * 32; kb < a.k; kb += 32 * kDownWaves) {
            const int at = kb + 8 * g;
            const bool in = at < a.k;          // k % 8 == 0: all eight or none
            h8_t xv = {0, 0, 0, 0, 0, 0, 0, 0};
            if (there && in) {
                xv = *reinterpret_cast<const h8_t*>(x + at);
            }
#pragma unroll
            for (int i = 0; i < kRanks; ++i) {
                h8_t av = {0, 0, 0, 0, 0, 0, 0, 0};
                if (has[i] && in) {
                    av = *reinterpret_cast<const h8_t*>(arow[i] + at);
                }
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(xv, av, acc[i], 0, 0, 0);
            }
        }
    } else {
        for (int kb = wave * 16; kb < a.k; kb += 16 * kDownWaves) {
            const int at = kb + 4 * g;
            const bool in = at < a.k;
            f4_t xv = {0.f, 0.f, 0.f, 0.f};
            if (there && in) {
                xv = load_x4<TYPE>(a.x, xat + at);
            }
#pragma unroll
            for (int i = 0; i < kRanks; ++i) {
                h4_t av = {0, 0, 0, 0};
                if (has[i] && in) {
                    av = *reinterpret_cast<const h4_t*>(arow[i] + at);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(xv[c], (float)av[c], acc[i], 0,
                                                                  0, 0);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kRanks; ++i) {
        part[wave][i][lane] = acc[i];
    }
    __syncthreads();
    const int i = wave;
    if (i >= kRanks || rank0 + 16 * i >= rank) {
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

// y of the tile's positions, columns from blockIdx.y * 64 * each on: wave w
// takes 16-column tiles w, w + 4, ...  VB: rows of B are multiples of four
// halves; VY: rows of y and base multiples of four floats.
template <bool VB, bool VY>
__global__ void __launch_bounds__(256)
lora_up_kernel(LoraArgs a, int each)
{
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int j = lane & 15;
    const int g = lane >> 4;
    const GroupTile t = find_tile<kTile>(a.offsets, a.adapters, a.rows, blockIdx.x);
    if (t.count == 0) {
        return;
    }
    const int rank = rank_of(a, t.group);
    const int row = j < t.count ? row_of(a, t.begin + j) : -1;
    const int pitch = (a.r + 15) / 16 * 16;
    const float* v = a.v + (int64_t)(t.begin + min(j, t.count - 1)) * pitch + 4 * g;
    for (int e = 0; e < each; ++e) {
        const int col0 = ((int)blockIdx.y * each + e) * 64 + wave * 16;
        if (col0 >= a.n) {
            return;
        }
        // B row of this lane (as a matrix row), then four columns of y
        const int col = min(col0 + j, a.n - 1);
        const _Float16* b = static_cast<const _Float16*>(a.b) +
                            ((int64_t)t.group * a.n + col) * a.r + 4 * g;
        f4_t acc = {0.f, 0.f, 0.f, 0.f};
        for (int k0 = 0; k0 < rank; k0 += 16) {
            const int left = rank - k0 - 4 * g;        // ranks of this lane's four
            const f4_t vv = *reinterpret_cast<const f4_t*>(v + k0);
            h4_t bv = {0, 0, 0, 0};
            if (VB && left >= 4) {
                bv = *reinterpret_cast<const h4_t*>(b + k0);
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    bv[c] = c < left ? b[k0 + c] : (_Float16)0;
                }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                acc = __builtin_amdgcn_mfma_f32_16x16x4f32((float)bv[c], vv[c], acc, 0, 0, 0);
            }
        }
        // D[4 g + c][j]: column col0 + 4 g + c of position j
        if (row >= 0) {
            const int at = col0 + 4 * g;
            const int64_t o = (int64_t)row * a.n + at;
            if constexpr (VY) {
                if (at < a.n) {                        // n % 4 == 0: all four or none
                    if (a.base != nullptr) {
                        acc += *reinterpret_cast<const f4_t*>(a.base + o);
                    }
                    *reinterpret_cast<f4_t*>(a.y + o) = acc;
                }
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (at + c < a.n) {
                        a.y[o + c] = acc[c] + (a.base != nullptr ? a.base[o + c] : 0.f);
                    }
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
    const int64_t up = (n + 63) / 64;
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
    // several column tiles per wave once there are enough workgroups without
    const int64_t parts = (a.n + 63) / 64;
    const int each = (int64_t)tiles * parts >= 8192 ? 4 : 1;
    const dim3 up(tiles, (unsigned)((parts + each - 1) / each));
    const bool vb = a.r % 4 == 0;
    const bool vy = a.n % 4 == 0;
    if (vb && vy) {
        hipLaunchKernelGGL((lora_up_kernel<true, true>), up, dim3(256), 0, stream, a, each);
    } else if (vb) {
        hipLaunchKernelGGL((lora_up_kernel<true, false>), up, dim3(256), 0, stream, a, each);
    } else if (vy) {
        hipLaunchKernelGGL((lora_up_kernel<false, true>), up, dim3(256), 0, stream, a, each);
    } else {
        hipLaunchKernelGGL((lora_up_kernel<false, false>), up, dim3(256), 0, stream, a, each);
    }
    return hipGetLastError();
}

}  // namespace q4k
