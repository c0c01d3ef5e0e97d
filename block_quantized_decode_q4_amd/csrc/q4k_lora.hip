// q4k_lora.hip -- low-rank adapters of many requests beside a shared
// projection: y[row] = base[row] + scale_a B_a (A_a x[row]) for the rows of
// adapter a, A_a (r x k) and B_a (n x r) in binary16, a rank of its own
// (ranks[a] <= r) per adapter.
//
// Two launches, because every output needs all of A x: lora_down_kernel
// writes v = scale A x (f32, rows x r rounded up to 16) to the caller's
// workspace, lora_up_kernel adds B v to the base.  A workgroup takes a tile of
// rows of one adapter (q4k_groups.h).
//
// x in binary16 goes through v_mfma_f32_16x16x32_f16; f32 (and bfloat16)
// x through v_mfma_f32_16x16x4_f32 with A widened to f32, eight instructions
// for one (2048 rows at rank 64, n = k = 4096, a call: binary16 23.7 us, bfloat16
// 29.5, f32 43.3, of which 3.4 are x's further bytes); no operand of
// A x is rounded.  For B v each row's v, scaled by the power of two that brings its
// largest into [2^14, 2^15), is two binary16 numbers: hi and the rest, lo, which
// leaves at most 2^-22 of the value or 2^-39 of the row's largest, and both go
// through the f16 matrix cores into one f32 sum (an eighth of the f32
// instruction's time, and no widened B in registers).  What an adapter holds at or
// beyond its rank does not matter.
//
// Down: 16 rows times up to 64 ranks; the waves of `parts` workgroups share k
// (few rows: more parts, to fill the chip), a workgroup adds its waves up in
// LDS, and the up kernel adds the parts, always in the same order.  Up: 32
// rows times 256 columns (64 rows read B half as often and leave too few
// workgroups to hide the loads: slower).
//
// Everything passes through LDS: the matrix operands' lane order (a row's
// lanes 16 apart) would take 64 clocks of the vector cache per load where
// neighbouring lanes on neighbouring bytes take about 20, and that bound both
// kernels.  2048 rows at rank 64, n = k = 4096, x binary16 (84 MB): down
// 20 -> 8-10 us, up 27 -> 13-16 us; 24 rows of 16 adapters at rank 16: down 5.4 us,
// up 4-5 us.  An adapter's tiles go to one XCD, whose L2 then reads A and B once
// (over all XCDs: 2048 rows 30.9 us a call instead of 22.8, 8192 rows 98 instead of
// 64).  What bounds them now is the chain of loads that each workgroup waits for
// (offsets, order, operands), about 1 us a link, so whatever can be asked for
// before a wait is: two steps of operands, and up v, B and the base together (base
// behind the products: 3 us more).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "q4k_device.h"
#include "q4k_groups.h"
#include "q4k_kernels.h"

namespace q4k {

namespace {

typedef _Float16 h4_t __attribute__((ext_vector_type(4)));
typedef _Float16 h8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));
typedef float f4_t __attribute__((ext_vector_type(4)));

constexpr int kTile = 16;              // rows per down tile
constexpr int kRanks = 4;              // rank tiles of 16 per down workgroup
constexpr int kDownWaves = 8;
constexpr int kUpTile = 32;            // rows per up tile
constexpr int kUpCols = 256;           // columns per up workgroup

__device__ __forceinline__ int rank_of(const LoraArgs& a, int adapter)
{
    return a.ranks ? min(max(a.ranks[adapter], 0), a.r) : a.r;
}

// order[p]; without an order something else that is there, not to be used
__device__ __forceinline__ int order_at(const LoraArgs& a, int p)
{
    return (a.order ? a.order : a.offsets)[a.order ? p : 0];
}

// This workgroup's tile.  gridDim.x is a multiple of eight, so XCD x takes the x-th
// eighth of the tiles: an adapter's meet in one L2.
template <int ROWS>
__device__ __forceinline__ GroupTile adapter_tile(const LoraArgs& a)
{
    const GroupTiles tiles = count_tiles<ROWS>(a.offsets, a.adapters, a.rows, (int)gridDim.x);
    return find_work<ROWS>(tiles, a.offsets, a.adapters, a.rows, 1, (int)blockIdx.x).tile;
}

// The place of 16-byte piece p of row r in LDS rows of 128 bytes (eight
// pieces) or 64 (four): the 16 rows' reads of a piece do not collide.
__device__ __forceinline__ int at128(int r, int p)
{
    return r * 128 + ((p ^ (r & 7)) << 4);
}

__device__ __forceinline__ int at64(int r, int p)
{
    return r * 64 + ((p ^ ((r >> 3 & 1) * 3)) << 4);
}

// A step of a wave: 128 bytes of each x row (32 f32 or 64 16-bit elements) and
// the same elements of the A rows.
template <int TYPE>
constexpr int kStep = TYPE == kTypeF32 ? 32 : 64;
template <int TYPE, int NT>
constexpr int kDownLds = 16 * 128 + NT * 16 * 2 * kStep<TYPE>;

// One wave's part of v for the tile: every `stride`-th step from `first` on.
// acc[i]: rank tile i.  lds: the wave's own kDownLds bytes.
template <int TYPE, int NT>
__device__ __forceinline__ void down_part(const LoraArgs& a, const GroupTile& t, int rank0,
                                          int rank, int first, int stride, unsigned char* lds,
                                          f4_t* acc)
{
    constexpr int K = kStep<TYPE>;
    constexpr int kSize = TYPE == kTypeF32 ? 4 : 2;
    constexpr int LA = NT * 16 * 2 * K / 1024;   // 1 KB loads of A
    constexpr int kPieces = 2 * K / 16;          // 16-byte pieces of an A row
    const int lane = threadIdx.x & 63;
    const int j = lane & 15;
    const int g = lane >> 4;
    unsigned char* const alds = lds + 16 * 128;
    // load roles: eight rows of 128 bytes of x, 512 / K rows of A at a time.  No
    // load is conditional: positions, ranks and pieces that are not there read
    // ones that are; their sums are not used, and beyond k both become zeros.
    const int xp = (lane & 7) * 16;              // byte of a step
    const int ap = (lane % kPieces) * 16;
    const char* xsrc[2];
    const char* asrc[LA];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int p = t.begin + min(8 * i + (lane >> 3), t.count - 1);
        const int ordered = order_at(a, p);
        const int row = a.order ? ordered : p;
        xsrc[i] = static_cast<const char*>(a.x) +
                  (int64_t)(row >= 0 && row < a.rows ? row : 0) * a.k * kSize;
    }
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        const int rr = min(rank0 + i * (64 / kPieces) + lane / kPieces, rank - 1);
        asrc[i] = static_cast<const char*>(a.a) + ((int64_t)t.group * a.r + rr) * a.k * 2;
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        acc[i] = f4_t{0.f, 0.f, 0.f, 0.f};
    }
    const int steps = (a.k + K - 1) / K;
    u4_t xv[2][2], av[2][LA];
    auto load = [&](int st, auto set) __attribute__((always_inline)) {
        constexpr int I = decltype(set)::value;
        const int64_t at = min(st, steps - 1);
        // (k % 8 == 0: pieces are whole)
        const int64_t xat = min(at * 128 + xp, (int64_t)a.k * kSize - 16);
        const int64_t aat = min(at * (2 * K) + ap, (int64_t)a.k * 2 - 16);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            xv[I][i] = *reinterpret_cast<const u4_t*>(xsrc[i] + xat);
        }
#pragma unroll
        for (int i = 0; i < LA; ++i) {
            av[I][i] = *reinterpret_cast<const u4_t*>(asrc[i] + aat);
        }
    };
    auto step = [&](int st, auto set, auto more) __attribute__((always_inline)) {
        constexpr int I = decltype(set)::value;
        if ((st + 1) * (int64_t)K > a.k) {       // the last step, in part
            const u4_t none = {0u, 0u, 0u, 0u};
            const bool xin = (int64_t)st * 128 + xp < (int64_t)a.k * kSize;
            const bool ain = (int64_t)st * (2 * K) + ap < (int64_t)a.k * 2;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                xv[I][i] = xin ? xv[I][i] : none;
            }
#pragma unroll
            for (int i = 0; i < LA; ++i) {
                av[I][i] = ain ? av[I][i] : none;
            }
        }
        // the wave's own LDS: no barrier
        wave_lds_order();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            *reinterpret_cast<u4_t*>(lds + at128(8 * i + (lane >> 3), lane & 7)) = xv[I][i];
        }
#pragma unroll
        for (int i = 0; i < LA; ++i) {
            const int row = i * (64 / kPieces) + lane / kPieces;
            const int at = kPieces == 8 ? at128(row, lane % kPieces) : at64(row, lane % kPieces);
            *reinterpret_cast<u4_t*>(alds + at) = av[I][i];
        }
        wave_lds_order();
        if constexpr (decltype(more)::value) {
            load(st + 2 * stride, set);          // two steps ahead
        }
        if constexpr (TYPE == kTypeF32) {
            const f4_t lo = *reinterpret_cast<const f4_t*>(lds + at128(j, 2 * g));
            const f4_t hi = *reinterpret_cast<const f4_t*>(lds + at128(j, 2 * g + 1));
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const h8_t w = *reinterpret_cast<const h8_t*>(alds + i * 1024 + at64(j, g));
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(c < 4 ? lo[c & 3] : hi[c & 3],
                                                                  (float)w[c], acc[i], 0, 0, 0);
                }
            }
        } else {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const u4_t xw = *reinterpret_cast<const u4_t*>(lds + at128(j, 4 * s + g));
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const h8_t w =
                        *reinterpret_cast<const h8_t*>(alds + i * 2048 + at128(j, 4 * s + g));
                    if constexpr (TYPE == kTypeF16) {
                        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                            __builtin_bit_cast(h8_t, xw), w, acc[i], 0, 0, 0);
                    } else {
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const uint32_t two = xw[c / 2];
                            const uint32_t one = c % 2 ? two & 0xFFFF0000u : two << 16;
                            acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                                __builtin_bit_cast(float, one), (float)w[c], acc[i], 0, 0, 0);
                        }
                    }
                }
            }
        }
    };
    if (first >= steps) {
        return;
    }
    const std::integral_constant<int, 0> s0;
    const std::integral_constant<int, 1> s1;
    load(first, s0);
    load(first + stride, s1);
    int st = first;
    for (; st + 2 * stride < steps; st += 2 * stride) {
        step(st, s0, std::true_type());
        step(st + stride, s1, std::true_type());
    }
    step(st, s0, std::false_type());
    if (st + stride < steps) {
        step(st + stride, s1, std::false_type());
    }
}

// v[part][p][rank] for the tile's positions, 64 ranks from blockIdx.y * 64 on,
// part blockIdx.z of k
template <int TYPE>
__global__ void __launch_bounds__(64 * kDownWaves)
lora_down_kernel(LoraArgs a)
{
    constexpr int kLds = kDownLds<TYPE, kRanks>;
    static_assert(kLds >= kRanks * 1024, "the waves' sums take the same place");
    __shared__ __align__(16) unsigned char smem[kDownWaves][kLds];
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int j = lane & 15;
    const int g = lane >> 4;
    const GroupTile t = adapter_tile<kTile>(a);
    if (t.count == 0) {
        return;
    }
    const int rank = rank_of(a, t.group);
    const int rank0 = blockIdx.y * 16 * kRanks;
    if (rank0 >= rank) {
        return;
    }
    f4_t acc[kRanks];
    const int left = rank - rank0;
    const int first = blockIdx.z * kDownWaves + wave;
    const int stride = gridDim.z * kDownWaves;
    // as many rank tiles as the adapter has
    if (left <= 16) {
        down_part<TYPE, 1>(a, t, rank0, rank, first, stride, smem[wave], acc);
    } else if (left <= 32) {
        down_part<TYPE, 2>(a, t, rank0, rank, first, stride, smem[wave], acc);
    } else {
        down_part<TYPE, 4>(a, t, rank0, rank, first, stride, smem[wave], acc);
    }
    wave_lds_order();
    f4_t* const mine = reinterpret_cast<f4_t*>(smem[wave]);
#pragma unroll
    for (int i = 0; i < kRanks; ++i) {
        if (16 * i < left) {
            mine[i * 64 + lane] = acc[i];
        }
    }
    __syncthreads();
    const int i = wave;
    if (i >= kRanks || 16 * i >= left) {
        return;
    }
    f4_t sum = reinterpret_cast<const f4_t*>(smem[0])[i * 64 + lane];
#pragma unroll
    for (int w = 1; w < kDownWaves; ++w) {
        sum += reinterpret_cast<const f4_t*>(smem[w])[i * 64 + lane];
    }
    const float scale = a.scales ? a.scales[t.group] : 1.f;
    // D[4 g + c][j]: position 4 g + c, rank j
    const int pitch = (a.r + 15) / 16 * 16;
    const int rr = rank0 + 16 * i + j;
    float* const v = a.v + (int64_t)blockIdx.z * a.rows * pitch;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int slot = 4 * g + c;
        if (slot < t.count) {
            v[(int64_t)(t.begin + slot) * pitch + rr] = scale * sum[c];
        }
    }
}

// y of a tile of 32 positions, 256 columns from blockIdx.y * 256 on, 64 per
// wave; 64 ranks of v and B at a time in LDS.  Rows of any n and r begin on any
// element: the accesses of B, base and y ask for an element's alignment only (rank
// 61, n = 4095, 2048 rows, both products: 66 us element by element, 37 us so).
// WHOLE: r is a multiple of eight, so that no eight ranks pass the end of B.
typedef uint32_t u4u_t __attribute__((ext_vector_type(4), aligned(2)));
typedef float f4u_t __attribute__((ext_vector_type(4), aligned(4)));
constexpr int kBPitch = 72;            // halves per row of v or B (9 pieces of 16 bytes)
constexpr int kYPitch = kUpCols + 4;   // floats per row of the products (65 pieces)

template <int PARTS, bool WHOLE>
__global__ void __launch_bounds__(256, 3)
lora_up_kernel(LoraArgs a)
{
    constexpr int kVBytes = kUpTile * kBPitch * 2;
    constexpr int kLds = 2 * kVBytes + kUpCols * kBPitch * 2;
    static_assert(kUpTile * kYPitch * 4 <= kLds, "operands and products share LDS");
    constexpr int U = kUpTile / 16;
    constexpr int kOwn = kUpTile / 4;          // rows that a wave writes
    __shared__ __align__(16) unsigned char smem[kLds];
    __shared__ int exps[kUpTile], steps[kUpTile];    // the rows' scales, and by how much they rose
    _Float16* const vs = reinterpret_cast<_Float16*>(smem);            // hi, then lo
    _Float16* const bs = reinterpret_cast<_Float16*>(smem + 2 * kVBytes);
    float* const ys = reinterpret_cast<float*>(smem);
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    // wave-uniform, as are all addresses but the lanes' 32-bit offsets below
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & 15;
    const int g = lane >> 4;
    const int col0 = (int)blockIdx.y * kUpCols;
    const GroupTile t = adapter_tile<kUpTile>(a);
    if (t.count == 0) {
        return;
    }
    const int rank = rank_of(a, t.group);
    const int pitch = (a.r + 15) / 16 * 16;
    const _Float16* const bg =
        static_cast<const _Float16*>(a.b) + ((int64_t)t.group * a.n + col0) * a.r;
    const f4_t zero = {0.f, 0.f, 0.f, 0.f};
    f4_t total[U][4];                          // [16 positions][16 columns]
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            total[u][i] = zero;
        }
    }
    // All that comes from memory is asked for here, in the order in which it is
    // waited for: the rows to write, v, B, the base.  None of these loads is
    // conditional (a wait behind a branch would wait for all of them): what is
    // not there reads something that is, and is masked or not written later.
    // The rows that this wave will write: positions wave, wave + 4, ...
    const int mine = t.begin + min(wave + 4 * (lane & (kOwn - 1)), t.count - 1);
    const int ordered = order_at(a, mine);
    // v: positions x 16 quads of ranks, by parts of k
    f4_t vp[U][PARTS];
    const int vq = (tid & 15) * 4;
    auto load_v = [&](int k0) __attribute__((always_inline)) {
        const int quad = min(vq, max(rank - k0 - 1, 0) / 4 * 4);
#pragma unroll
        for (int z = 0; z < PARTS; ++z) {
            const char* const from = reinterpret_cast<const char*>(
                a.v + ((int64_t)z * a.rows + t.begin) * pitch + k0);
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int p = min(16 * i + (tid >> 4), t.count - 1);
                vp[i][z] =
                    *reinterpret_cast<const f4_t*>(from + (uint32_t)(p * pitch + quad) * 4u);
            }
        }
    };
    // B: eight ranks of every 32nd column
    u4_t w[kUpCols / 32];
    const int bq = (tid & 7) * 8;
    auto load_b = [&](int k0) __attribute__((always_inline)) {
        const _Float16* const first = bg + k0;
        const char* const from = reinterpret_cast<const char*>(first);
        const int q = min(bq, max(rank - k0 - 1, 0) / 8 * 8);
        // the last half that eight may begin at, from `first` on
        const int64_t halves = ((int64_t)(a.adapters - t.group) * a.n - col0) * a.r - k0;
        const int end = (int)min(halves, (int64_t)1 << 30) - 8;
#pragma unroll
        for (int i = 0; i < kUpCols / 32; ++i) {
            const int at = min(32 * i + (tid >> 3), a.n - 1 - col0) * a.r + q;
            if constexpr (WHOLE) {
                w[i] = *reinterpret_cast<const u4u_t*>(from + (uint32_t)at * 2u);
            } else {
                if (end >= 0) {
                    w[i] = *reinterpret_cast<const u4u_t*>(from + (uint32_t)min(at, end) * 2u);
                }
                if (at > end) {                    // the last columns: one by one
                    h8_t v;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        v[e] = at + e < end + 8 ? first[at + e] : (_Float16)0;
                    }
                    w[i] = __builtin_bit_cast(u4_t, v);
                }
            }
        }
    };
    load_v(0);
    load_b(0);
    // the base (a row of y is this wave's alone, so base may be y)
    const int lane_row = a.order ? ordered : mine;
    int row[kOwn];
    f4_t base[kOwn];
    const bool four = a.base != nullptr && a.n >= 4;
#pragma unroll
    for (int q = 0; q < kOwn; ++q) {
        row[q] = wave + 4 * q < t.count ? __builtin_amdgcn_readlane(lane_row, q) : -1;
        row[q] = row[q] < a.rows ? row[q] : -1;
        // the last columns read the row's last four (n >= 4), and again below
        const float* const from = four ? a.base + (int64_t)max(row[q], 0) * a.n : a.v;
        const int c = four ? min(col0 + 4 * lane, a.n - 4) : 0;
        base[q] = *reinterpret_cast<const f4u_t*>(reinterpret_cast<const char*>(from) +
                                                  (uint32_t)c * 4u);
    }
    // a row's scale so far: 2^-seen brings the largest |v| into [2^14, 2^15)
    int seen[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        seen[u] = -1000;                       // below any
    }
    for (int k0 = 0; k0 < rank; k0 += 64) {
        if (k0 > 0) {
            __syncthreads();
            load_v(k0);
            load_b(k0);
        }
        const int left = rank - k0;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int p = 16 * i + (tid >> 4);
            const int q = vq;
            f4_t sum = vp[i][0];
#pragma unroll
            for (int z = 1; z < PARTS; ++z) {
                sum += vp[i][z];
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                sum[c] = q + c < left ? sum[c] : 0.f;
            }
            // the 16 lanes of a position
            float top = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                top = fmaxf(top, fabsf(sum[c]));
            }
#pragma unroll
            for (int off = 1; off < 16; off <<= 1) {
                top = fmaxf(top, __shfl_xor(top, off, 64));
            }
            int e = seen[i];
            if (top > 0.f && top < __builtin_inff()) {
                (void)frexpf(top, &e);
                e = max(e - 15, seen[i]);
            }
            const int step = seen[i] - e;
            seen[i] = e;
            h4_t hi, lo;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float x = ldexpf(sum[c], -e);
                hi[c] = (_Float16)x;
                lo[c] = (_Float16)(x - (float)hi[c]);
            }
            *reinterpret_cast<h4_t*>(vs + p * kBPitch + q) = hi;
            *reinterpret_cast<h4_t*>(vs + kUpTile * kBPitch + p * kBPitch + q) = lo;
            if ((tid & 15) == 0) {
                exps[p] = e;
                steps[p] = step;
            }
        }
        u4_t keep;                                     // the halves below the rank
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int have = left - bq - 2 * d;
            keep[d] = have >= 2 ? 0xFFFFFFFFu : have == 1 ? 0xFFFFu : 0u;
        }
#pragma unroll
        for (int i = 0; i < kUpCols / 32; ++i) {
            *reinterpret_cast<u4_t*>(bs + (32 * i + (tid >> 3)) * kBPitch + bq) = w[i] & keep;
        }
        __syncthreads();
        if (k0 > 0) {                              // sums so far, in the new scale
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int step = steps[16 * u + j];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        total[u][i][c] = ldexpf(total[u][i][c], step);
                    }
                }
            }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (32 * s < left) {
                h8_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    w[i] = *reinterpret_cast<const h8_t*>(
                        bs + (wave * 64 + 16 * i + j) * kBPitch + 32 * s + 8 * g);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const _Float16* const vp = vs + (16 * u + j) * kBPitch + 32 * s + 8 * g;
                    const h8_t hi = *reinterpret_cast<const h8_t*>(vp);
                    const h8_t lo = *reinterpret_cast<const h8_t*>(vp + kUpTile * kBPitch);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        total[u][i] =
                            __builtin_amdgcn_mfma_f32_16x16x32_f16(w[i], hi, total[u][i], 0, 0, 0);
                        total[u][i] =
                            __builtin_amdgcn_mfma_f32_16x16x32_f16(w[i], lo, total[u][i], 0, 0, 0);
                    }
                }
            }
        }
    }
    __syncthreads();
    // (rank 0: the sums are zeros, in no scale)
    // D[4 g + c][j] of (u, i): column 16 i + 4 g + c of position 16 u + j
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int e = rank > 0 ? exps[16 * u + j] : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                total[u][i][c] = ldexpf(total[u][i][c], e);
            }
            *reinterpret_cast<f4_t*>(ys + (16 * u + j) * kYPitch + wave * 64 + 16 * i + 4 * g) =
                total[u][i];
        }
    }
    __syncthreads();
    // whole rows of 256 columns
#pragma unroll
    for (int q = 0; q < kOwn; ++q) {
        if (row[q] < 0) {
            continue;
        }
        if (a.base == nullptr) {
            base[q] = zero;
        }
        const float* const yp = ys + (wave + 4 * q) * kYPitch;
        float* const out = a.y + (int64_t)row[q] * a.n;
        const int c = col0 + 4 * lane;
        if (a.n - c >= 4) {
            *reinterpret_cast<f4u_t*>(out + c) =
                base[q] + *reinterpret_cast<const f4_t*>(yp + 4 * lane);
        } else {
            for (int e = 0; e < a.n - c; ++e) {
                const float b = a.base ? a.base[(int64_t)row[q] * a.n + c + e] : 0.f;
                out[c + e] = b + yp[4 * lane + e];
            }
        }
    }
}

template <int PARTS>
void launch_up(const LoraArgs& a, dim3 up, hipStream_t stream)
{
    if (a.r % 8 == 0) {
        hipLaunchKernelGGL((lora_up_kernel<PARTS, true>), up, dim3(256), 0, stream, a);
    } else {
        hipLaunchKernelGGL((lora_up_kernel<PARTS, false>), up, dim3(256), 0, stream, a);
    }
}

// Parts of k: enough workgroups for the chip.  (Sums of v are the caller's
// workspace, so by the rows alone.)  Both products with 1 / 2 / 4 parts, rank 64,
// n = k = 4096: 512 rows 16.5 / 13.7 / 12.2 us, 2048 rows 25.2 / 22.8 / 24.5 us,
// 4096 rows 36.9 / 38.8 / 41.4 us.
constexpr int64_t kRowsOf4 = 512;      // the most rows of four and of two parts
constexpr int64_t kRowsOf2 = 4095;

int down_parts(int64_t rows)
{
    return rows <= kRowsOf4 ? 4 : rows <= kRowsOf2 ? 2 : 1;
}

}  // namespace

size_t lora_ws_bytes(int64_t rows, int64_t r)
{
    return (size_t)down_parts(rows) * (size_t)rows * (size_t)((r + 15) / 16 * 16) * sizeof(float);
}

// The most that `rows` rows or fewer take: 512 rows in four parts are 2048 rows of
// v, and 513 in two are 1026.
size_t lora_ws_most(int64_t rows, int64_t r)
{
    size_t most = lora_ws_bytes(rows, r);
    for (const int64_t step : {kRowsOf4, kRowsOf2}) {
        if (step < rows) {
            most = std::max(most, lora_ws_bytes(step, r));
        }
    }
    return most;
}

// The grids: fewer than 2^32 threads, 65535 workgroups along y
bool lora_fits(int64_t rows, int64_t adapters, int64_t n, int64_t r)
{
    const int64_t down = (most_tiles(rows, adapters, kTile) + 7) *
                         ((r + 16 * kRanks - 1) / (16 * kRanks)) * down_parts(rows);
    const int64_t up = (n + kUpCols - 1) / kUpCols;
    const int64_t most = (int64_t)1 << 32;
    return down * 64 * kDownWaves < most && up <= 65535 &&
           (most_tiles(rows, adapters, kUpTile) + 7) * up * 256 < most;
}

hipError_t launch_lora(const LoraArgs& a, hipStream_t stream)
{
    const int parts = down_parts(a.rows);
    auto eights = [](int64_t tiles) { return (unsigned)((tiles + 7) / 8 * 8); };
    const dim3 down(eights(most_tiles(a.rows, a.adapters, kTile)),
                    (unsigned)((a.r + 16 * kRanks - 1) / (16 * kRanks)), (unsigned)parts);
    const dim3 threads(64 * kDownWaves);
    if (a.x_type == kTypeF16) {
        hipLaunchKernelGGL(lora_down_kernel<kTypeF16>, down, threads, 0, stream, a);
    } else if (a.x_type == kTypeBF16) {
        hipLaunchKernelGGL(lora_down_kernel<kTypeBF16>, down, threads, 0, stream, a);
    } else {
        hipLaunchKernelGGL(lora_down_kernel<kTypeF32>, down, threads, 0, stream, a);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) {
        return e;
    }
    const dim3 up(eights(most_tiles(a.rows, a.adapters, kUpTile)),
                  (unsigned)((a.n + kUpCols - 1) / kUpCols));
    switch (parts) {
    case 1: launch_up<1>(a, up, stream); break;
    case 2: launch_up<2>(a, up, stream); break;
    default: launch_up<4>(a, up, stream); break;
    }
    return hipGetLastError();
}

}  // namespace q4k
