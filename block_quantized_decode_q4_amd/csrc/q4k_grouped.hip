// q4k_grouped.hip -- products of grouped rows with Q4_K matrices: position i
// of group g gives y[row] = W_g x[row], the experts' products of a decode
// batch (a group may be empty, one row or many).
//
// Mathematics.  With w = d sc q - dmin m, a superblock (256 elements, eight
// sub-blocks j) adds
//   d * sum_e (sc_j q_e) x_e  -  dmin * sum_j m_j S_j,   S_j = sum of x over j
// to a row's product.  sc q is an integer up to 945 and so is exact in
// binary16; x is carried as two binary16 numbers: with s the power of two
// that brings the row's largest |x| into [2^14, 2^15),
//   x s = hi + 2^-11 lo + e,   |e| <= max(2^-22 |x s|, 2^-36),
// the second bound for elements below 2^-28 of the row's largest (binary16's
// subnormal step, at 2^-50 of the largest).  The products go through the f16 matrix cores, whose
// products are exact and sums f32: one accumulator for hi, one for lo and one
// for the m_j S_j (S_j as two binary16 numbers too, times m_j and 2^-11 m_j), added up per superblock
// as f32.  Scales folded into the codes leave nothing to do per sub-block.
//
// Two launches: grouped_x_kernel lays each x row out once in the caller's
// workspace (hi, lo and S in the order in which the lanes of the product
// kernel read them); grouped_kernel multiplies.
//
// grouped_kernel: a wave computes 16 weight rows x 16 positions of one group
// (v_mfma_f32_16x16x32_f16, x as the rows, weights as the columns).  Lane
// l = 16 g + j holds weight row j and chunk g of each superblock, so it reads
// two 16-byte pieces of codes and the header, and needs the scales of its own
// two sub-blocks only: 9 instructions for 8 codes (mask, shift, multiply by
// the scale), after which the eight products with hi and the eight with lo
// take the same registers.  The waves of a workgroup share the superblocks of
// its rows among them (few rows) or take rows of their own (many).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4k_device.h"
#include "q4k_groups.h"
#include "q4k_kernels.h"

namespace q4k {

namespace {

typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
typedef _Float16 h4_t __attribute__((ext_vector_type(4)));
typedef _Float16 h8_t __attribute__((ext_vector_type(8)));
typedef float f4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));

// One x row in the workspace: per superblock 512 bytes of hi, 512 of lo (piece
// u of chunk g at 64 u + 16 g) and 32 of S (chunk g at 8 g); the rows' scale
// exponents behind all rows.
constexpr int kXsb = 1056;
constexpr int kTile = 16;              // positions per tile
constexpr int kXcd = 8;

struct XWs {
    char* rows;
    int* exps;
};

__host__ __device__ inline XWs x_ws(void* ws, int S, int64_t x_count)
{
    XWs r;
    r.rows = static_cast<char*>(ws);
    r.exps = reinterpret_cast<int*>(r.rows + x_count * S * kXsb);
    return r;
}

// ------------------------------------------------------------------ x rows
// Elements 4u .. 4u + 3 of sub-blocks 2g (a) and 2g + 1 (b), as f32
template <bool Q8>
__device__ __forceinline__ void load_x(const GroupedArgs& a, int64_t row, int v, float4& lo,
                                       float4& hi)
{
    const int at = (v >> 3) * 64 + (v & 7) * 4;
    if constexpr (Q8) {
        const char4 p = *reinterpret_cast<const char4*>(a.q + row * a.k + at);
        const char4 r = *reinterpret_cast<const char4*>(a.q + row * a.k + at + 32);
        const float* d = a.d + row * (a.k / 32) + at / 32;
        const float dl = d[0], dh = d[1];
        lo = make_float4(dl * p.x, dl * p.y, dl * p.z, dl * p.w);
        hi = make_float4(dh * r.x, dh * r.y, dh * r.z, dh * r.w);
    } else {
        const float* p = a.x + row * a.k + at;
        lo = *reinterpret_cast<const float4*>(p);
        hi = *reinterpret_cast<const float4*>(p + 32);
    }
}

__device__ __forceinline__ void split(float v, _Float16& hi, _Float16& lo)
{
    hi = (_Float16)v;
    lo = (_Float16)((v - (float)hi) * 2048.0f);
}

template <bool Q8>
__global__ void __launch_bounds__(1024)
grouped_x_kernel(GroupedArgs a)
{
    __shared__ float part[16];
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x;
    const int threads = blockDim.x;
    const int S = a.k / kQK;
    const XWs ws = x_ws(a.ws, S, a.g.x_count);
    // the row's largest |x| (a NaN counts as an infinity)
    float top = 0.f;
    for (int v = tid; v < S * 32; v += threads) {
        float4 lo, hi;
        load_x<Q8>(a, row, v, lo, hi);
        const float e[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            top = fmaxf(top, e[i] == e[i] ? fabsf(e[i]) : __builtin_inff());
        }
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        top = fmaxf(top, __shfl_xor(top, off, 64));
    }
    if ((tid & 63) == 0) {
        part[tid >> 6] = top;
    }
    __syncthreads();
    for (int i = 0; i < threads / 64; ++i) {
        top = fmaxf(top, part[i]);
    }
    int e = 15;                            // exponent of a zero or non-finite row: none
    if (top > 0.f && top < __builtin_inff()) {
        (void)frexpf(top, &e);             // top in [2^(e-1), 2^e)
    }
    const int s = 15 - e;
    if (tid == 0) {
        ws.exps[row] = s;
    }
    char* const out = ws.rows + row * S * kXsb;
    for (int v = tid; v < S * 32; v += threads) {
        float4 lo4, hi4;
        load_x<Q8>(a, row, v, lo4, hi4);
        // the codes' order in the matrix operand: bytes 0, 2, 1, 3
        const float e8[8] = {lo4.x, lo4.z, lo4.y, lo4.w, hi4.x, hi4.z, hi4.y, hi4.w};
        float t[8];
        h8_t h, l;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            t[i] = ldexpf(e8[i], s);
            _Float16 a16, b16;
            split(t[i], a16, b16);
            h[i] = a16;
            l[i] = b16;
        }
        const int sb = v >> 5, g = (v >> 3) & 3, u = v & 7;
        char* p = out + (int64_t)sb * kXsb;
        *reinterpret_cast<h8_t*>(p + u * 64 + g * 16) = h;
        *reinterpret_cast<h8_t*>(p + 512 + u * 64 + g * 16) = l;
        // S of the two sub-blocks: the eight lanes of this chunk
        float s0 = (t[0] + t[1]) + (t[2] + t[3]);
        float s1 = (t[4] + t[5]) + (t[6] + t[7]);
#pragma unroll
        for (int off = 1; off < 8; off <<= 1) {
            s0 += __shfl_xor(s0, off, 64);
            s1 += __shfl_xor(s1, off, 64);
        }
        if (u == 0) {
            // 2^-6: at most 32 * 2^15 / 64 = 2^14
            const float q0 = s0 * 0.015625f, q1 = s1 * 0.015625f;
            _Float16 a0, b0, a1, b1;
            split(q0, a0, b0);
            split(q1, a1, b1);
            *reinterpret_cast<h4_t*>(p + 1024 + g * 8) = h4_t{a0, b0, a1, b1};
        }
    }
}

// ---------------------------------------------------------------- products
// One row's piece of a superblock: the header and the lane's 32 code bytes
struct WPiece {
    uint4 h, c0, c1;
};

__device__ __forceinline__ WPiece load_w(const uint8_t* p, int g)
{
    WPiece r;
    r.h = load16(p);
    r.c0 = load16(p + 16 + 32 * g);
    r.c1 = load16(p + 32 + 32 * g);
    return r;
}

// d, dmin, and for the lane's chunk: its scales as pairs sc 2^10 (for codes
// q 2^-24, low nibbles masked in place) and sc 2^6 (q 2^-20, high nibbles),
// so that a product is sc q 2^-14; and the mins as {m0, m0 2^-11, m1, m1 2^-11,
// 0 ...} for S's two numbers.
struct WScales {
    float d, dmin;
    h2_t sl, sh;
    h8_t m;
};

__device__ __forceinline__ WScales scales_of(const uint4& h, uint32_t shift, uint32_t sel)
{
    WScales r;
    const h2_t dd = __builtin_bit_cast(h2_t, h.x);
    r.d = (float)dd.x;
    r.dmin = (float)dd.y;
    const uint32_t y = h.y >> shift;
    const uint32_t z = h.z >> shift;
    const uint32_t wv = h.w >> shift;
    const uint32_t sc_b = (wv & 0x0F0Fu) | ((y >> 2) & 0x3030u);
    const uint32_t m_b = ((wv >> 4) & 0x0F0Fu) | ((z >> 2) & 0x3030u);
    const uint32_t sc = ((y & 0x3F3Fu) & sel) | (sc_b & ~sel);
    const uint32_t mm = ((z & 0x3F3Fu) & sel) | (m_b & ~sel);
    const _Float16 l = (_Float16)((float)(sc & 0xFFu) * 1024.0f);
    const _Float16 u = (_Float16)((float)((sc >> 8) & 0xFFu) * 64.0f);
    const float m0 = (float)(mm & 0xFFu);
    const float m1 = (float)((mm >> 8) & 0xFFu);
    r.sl = h2_t{l, l};
    r.sh = h2_t{u, u};
    constexpr float kLo = 1.0f / 2048.0f;
    const _Float16 o = (_Float16)0;
    r.m = h8_t{(_Float16)m0, (_Float16)(m0 * kLo), (_Float16)m1, (_Float16)(m1 * kLo), o, o, o, o};
    return r;
}

// The matrix operand of one code dword: eight sc q 2^-14, exact
__device__ __forceinline__ h8_t operand(uint32_t D, h2_t sl, h2_t sh)
{
    const uint32_t d8 = D >> 8;
    const h2_t p0 = __builtin_bit_cast(h2_t, D & 0x000F000Fu) * sl;
    const h2_t p1 = __builtin_bit_cast(h2_t, d8 & 0x000F000Fu) * sl;
    const h2_t p2 = __builtin_bit_cast(h2_t, D & 0x00F000F0u) * sh;
    const h2_t p3 = __builtin_bit_cast(h2_t, d8 & 0x00F000F0u) * sh;
    return h8_t{p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
}

// WK waves share the superblocks of a row tile (wave part p takes p, p + WK,
// ...), WN = 8 / WK row tiles per workgroup.
template <int WK>
__global__ void __launch_bounds__(512)
grouped_kernel(GroupedArgs a, int tiles, int row_blocks)
{
    constexpr int WN = 8 / WK;
    __shared__ f4_t part[WK > 1 ? 8 * 64 : 1];
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int j = lane & 15;
    const int g = lane >> 4;
    // a row block's tiles follow each other on one XCD (its L2 keeps the
    // weights that several tiles of one group share)
    const int xcd = blockIdx.x % kXcd;
    const int local = blockIdx.x / kXcd;
    const int block = (local / tiles) * kXcd + xcd;
    if (block >= row_blocks) {
        return;
    }
    const GroupTile t = find_tile<kTile>(a.g.offsets, a.g.groups, a.g.rows, local % tiles);
    if (t.count == 0) {
        return;
    }
    const int S = a.k / kQK;
    const XWs ws = x_ws(a.ws, S, a.g.x_count);
    // the lane's position (as an x row of the matrix operand)
    const int wk = wave % WK;
    int xr = -1, yr = -1;
    if (j < t.count) {
        const int p = t.begin + j;
        xr = a.g.x_rows ? a.g.x_rows[p] : p;
        xr = xr < 0 ? -1 : xr / a.g.x_div;
        yr = a.g.y_rows ? a.g.y_rows[p] : p;
    }
    const bool there = xr >= 0 && xr < a.g.x_count && yr >= 0 && yr < a.g.y_count;
    const uint32_t mask = (uint32_t)(__ballot(there) & 0xFFFFu);
    const int row0 = (block * WN + wave / WK) * 16;
    const int row = row0 + j;
    const int s = there ? ws.exps[xr] : 0;
    const char* xp = ws.rows + (int64_t)(there ? xr : 0) * S * kXsb + g * 16;
    const uint8_t* wp = static_cast<const uint8_t*>(a.w) +
                        ((int64_t)t.group * a.n + min(row, a.n - 1)) * S * kBlockBytes;
    const uint32_t shift = 16 * (g & 1);
    const uint32_t sel = g < 2 ? 0xFFFFFFFFu : 0u;

    f4_t total = {0.f, 0.f, 0.f, 0.f};
    const f4_t zero = {0.f, 0.f, 0.f, 0.f};
    if (row0 < a.n) {
        WPiece w = load_w(wp + (int64_t)min(wk, S - 1) * kBlockBytes, g);
        for (int sb = wk; sb < S; sb += WK) {
            u4_t xh[8], xl[8];
            uint2 xs = {0u, 0u};
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                xh[u] = u4_t{0u, 0u, 0u, 0u};
                xl[u] = u4_t{0u, 0u, 0u, 0u};
            }
            if (there) {
                const char* p = xp + (int64_t)sb * kXsb;
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    xh[u] = *reinterpret_cast<const u4_t*>(p + u * 64);
                    xl[u] = *reinterpret_cast<const u4_t*>(p + 512 + u * 64);
                }
                xs = *reinterpret_cast<const uint2*>(p + 1024 - g * 8);
            }
            const WPiece now = w;
            w = load_w(wp + (int64_t)min(sb + WK, S - 1) * kBlockBytes, g);
            const WScales sc = scales_of(now.h, shift, sel);
            const uint32_t c[8] = {now.c0.x, now.c0.y, now.c0.z, now.c0.w,
                                   now.c1.x, now.c1.y, now.c1.z, now.c1.w};
            f4_t ah = zero, al = zero;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const h8_t b = operand(c[u], sc.sl, sc.sh);
                ah = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8_t, xh[u]), b, ah,
                                                            0, 0, 0);
                al = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8_t, xl[u]), b, al,
                                                            0, 0, 0);
            }
            const u4_t xsv = {xs.x, xs.y, 0u, 0u};
            const f4_t am = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                __builtin_bit_cast(h8_t, xsv), sc.m, zero, 0, 0, 0);
            // 2^14: the operands' 2^-14; lo carries 2^11 more; S is 2^-6
            const float dh = sc.d * 16384.0f;
            const float dm = sc.dmin * 64.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float v = __builtin_fmaf(al[i], 1.0f / 2048.0f, ah[i]);
                total[i] = __builtin_fmaf(dh, v, total[i]);
                total[i] = __builtin_fmaf(-dm, am[i], total[i]);
            }
        }
    }
    if constexpr (WK > 1) {
        part[wave * 64 + lane] = total;
        __syncthreads();
        if (wk != 0) {
            return;
        }
#pragma unroll
        for (int p = 1; p < WK; ++p) {           // in part order
            total += part[(wave + p) * 64 + lane];
        }
    }
    // D[4 g + i][j]: position 4 g + i, weight row j
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int slot = 4 * g + i;
        const int yrow = __shfl(yr, slot, 64);
        const int exp = __shfl(s, slot, 64);
        if (row < a.n && ((mask >> slot) & 1u)) {
            a.y[(int64_t)yrow * a.n + row] = ldexpf(total[i], -exp);
        }
    }
}

template <int WK>
void launch_wk(const GroupedArgs& a, int tiles, hipStream_t stream)
{
    const int row_blocks = (a.n + 16 * (8 / WK) - 1) / (16 * (8 / WK));
    const int64_t grid = (int64_t)((row_blocks + kXcd - 1) / kXcd) * kXcd * tiles;
    hipLaunchKernelGGL(grouped_kernel<WK>, dim3((unsigned)grid), dim3(512), 0, stream, a, tiles,
                       row_blocks);
}

}  // namespace

size_t grouped_ws_bytes(int64_t k, int64_t x_count)
{
    return (size_t)x_count * (size_t)(k / kQK) * kXsb + (size_t)x_count * sizeof(int);
}

// The most workgroups that launch_grouped launches
int64_t grouped_grid(int64_t rows, int64_t groups, int64_t n)
{
    const int64_t blocks = (n + 15) / 16;
    return (blocks + kXcd - 1) / kXcd * kXcd * most_tiles(rows, groups, kTile);
}

hipError_t launch_grouped(const GroupedArgs& a, hipStream_t stream)
{
    const int S = a.k / kQK;
    int threads = (S * 32 + 63) / 64 * 64;
    threads = threads > 1024 ? 1024 : threads;
    if (a.q != nullptr) {
        hipLaunchKernelGGL(grouped_x_kernel<true>, dim3((unsigned)a.g.x_count), dim3(threads), 0,
                           stream, a);
    } else {
        hipLaunchKernelGGL(grouped_x_kernel<false>, dim3((unsigned)a.g.x_count), dim3(threads), 0,
                           stream, a);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) {
        return e;
    }
    const int tiles = (int)most_tiles(a.g.rows, a.g.groups, kTile);
    // waves for every SIMD of 256 CUs, four deep, before a wave takes more
    // superblocks
    const int64_t wave_tiles = (int64_t)tiles * ((a.n + 15) / 16);
    if (S >= 8 && wave_tiles * 8 <= 8192) {
        launch_wk<8>(a, tiles, stream);
    } else if (S >= 4 && wave_tiles * 4 <= 8192) {
        launch_wk<4>(a, tiles, stream);
    } else if (S >= 2 && wave_tiles * 2 <= 8192) {
        launch_wk<2>(a, tiles, stream);
    } else {
        launch_wk<1>(a, tiles, stream);
    }
    return hipGetLastError();
}

}  // namespace q4k
