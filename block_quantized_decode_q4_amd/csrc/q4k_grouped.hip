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
// subnormal step, at 2^-50 of the largest).  The products go through the f16
// matrix cores, whose products are exact and sums f32: one accumulator for hi,
// one for lo and one for the m_j S_j (S_j as two binary16 numbers too, times
// m_j and 2^-11 m_j), added up per superblock as f32.  Scales folded into the
// codes leave nothing to do per sub-block.
//
// Two launches: grouped_x_kernel lays each x row out once in the caller's
// workspace (hi, lo and S in the order in which the lanes of the product
// kernel read them); grouped_kernel multiplies.
//
// grouped_kernel: a wave computes 16 weight rows x 16 positions of one group
// (v_mfma_f32_16x16x32_f16, x as the rows, weights as the columns).  Lane
// l = 16 g + j holds weight row j and two 16-byte pieces of its codes in each
// superblock, and needs the scales of their four sub-blocks only: 9
// instructions for 8 codes (mask, shift, multiply by the scale), and the
// products with hi and with lo take the same registers.  Weights and x both
// pass through LDS: the operands' own lane order would take 64 clocks of the
// vector cache per load instruction where neighbouring lanes on neighbouring
// bytes take about 20 (measured: a skewed batch 151 -> 125 us).
//
// What bounds it: about 150 vector instructions a superblock beside 17 matrix
// ones, on two waves a SIMD for most decode shapes, against the weights' bytes:
// 264 MB (eight experts 4096 x 14336, 16 rows each) in 80 us, 3.3 TB/s.
// Tried and not kept: two superblocks or two row tiles per wave and step, the
// superblocks shared by two waves, 32 positions per tile, x converted by the
// product kernel itself (each within 10 % on one shape and slower on others).

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

// One x row in the workspace: per superblock 512 bytes of hi, 512 of lo (lane
// group g's operand of product u at 64 u + 16 g) and 32 of S (lane group g's at
// 8 g); the rows' scale exponents behind all rows.
constexpr int kXsb = 1056;

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
// Elements 4 p .. 4 p + 3 of the two sub-blocks of a chunk (piece v = 32 sb + 8
// chunk + p of the row), as f32
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

// The larger of top and the eight |x|, a NaN as an infinity
__device__ __forceinline__ float piece_top(const float4& lo, const float4& hi, float top)
{
    const float e[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        top = fmaxf(top, e[i] == e[i] ? fabsf(e[i]) : __builtin_inff());
    }
    return top;
}

// The power of two that brings top into [2^14, 2^15): 15 - e for top in
// [2^(e-1), 2^e), 0 where there is none (a zero, an infinity)
__device__ __forceinline__ int scale_of(float top)
{
    int e = 15;
    if (top > 0.f && top < __builtin_inff()) {
        (void)frexpf(top, &e);
    }
    return 15 - e;
}

// A piece times 2^s as hi and lo, in the codes' order in the matrix operand
// (bytes 0, 2, 1, 3); and, in the lane of piece 0, the two sub-blocks' sums times
// 2^-6 (at most 32 * 2^15 / 64 = 2^14) as two numbers each.  The eight pieces of
// a chunk are in eight neighbouring lanes.
__device__ __forceinline__ void convert(const float4& lo4, const float4& hi4, int s, h8_t& h,
                                        h8_t& l, h4_t& sums)
{
    const float e8[8] = {lo4.x, lo4.z, lo4.y, lo4.w, hi4.x, hi4.z, hi4.y, hi4.w};
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        t[i] = ldexpf(e8[i], s);
        _Float16 a16, b16;
        split(t[i], a16, b16);
        h[i] = a16;
        l[i] = b16;
    }
    float s0 = (t[0] + t[1]) + (t[2] + t[3]);
    float s1 = (t[4] + t[5]) + (t[6] + t[7]);
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) {
        s0 += __shfl_xor(s0, off, 64);
        s1 += __shfl_xor(s1, off, 64);
    }
    _Float16 a0, b0, a1, b1;
    split(s0 * 0.015625f, a0, b0);
    split(s1 * 0.015625f, a1, b1);
    sums = h4_t{a0, b0, a1, b1};
}

// Where piece v of a superblock (chunk v / 8 % 4, half v / 4 % 2, dword v % 4)
// goes: product u, lane group g, and its chunk's sums to lane group sg.
struct PieceAt {
    int u, g, sg;
};

__device__ __forceinline__ PieceAt piece_at(int v)
{
    const int c = (v >> 3) & 3;
    return {(c >> 1) * 4 + (v & 3), (c & 1) * 2 + ((v >> 2) & 1), (c & 1) * 2 + (c >> 1)};
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
    float top = 0.f;
    for (int v = tid; v < S * 32; v += threads) {
        float4 lo, hi;
        load_x<Q8>(a, row, v, lo, hi);
        top = piece_top(lo, hi, top);
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
    const int s = scale_of(top);
    if (tid == 0) {
        ws.exps[row] = s;
    }
    char* const out = ws.rows + row * S * kXsb;
    for (int v = tid; v < S * 32; v += threads) {
        float4 lo4, hi4;
        load_x<Q8>(a, row, v, lo4, hi4);
        h8_t h, l;
        h4_t sums;
        convert(lo4, hi4, s, h, l, sums);
        const PieceAt at = piece_at(v);
        char* p = out + (int64_t)(v >> 5) * kXsb;
        *reinterpret_cast<h8_t*>(p + at.u * 64 + at.g * 16) = h;
        *reinterpret_cast<h8_t*>(p + 512 + at.u * 64 + at.g * 16) = l;
        if ((v & 7) == 0) {
            *reinterpret_cast<h4_t*>(p + 1024 + at.sg * 8) = sums;
        }
    }
}

// ---------------------------------------------------------------- products
// 16 rows of a superblock in flight: lane l holds 16 code bytes each of rows l / 8
// and 8 + l / 8 (piece l % 8), and header dword l % 4 of row l / 4.  Four
// neighbouring lanes then read consecutive bytes, which is what the vector
// caches merge: the matrix operands' own layout (a row's lanes 16 apart) takes
// 64 clocks an instruction instead of about 20.
struct WPiece {
    u4_t c0, c1;
    uint32_t h;
};

// They change lanes through 16 rows of 144 bytes in LDS (the rows as they are
// stored: 36 banks apart, so 16 rows' pieces do not collide).
constexpr int kWStage = 16 * kBlockBytes;

// d, dmin, and for the lane's two chunks: their scales as pairs sc 2^10 (for
// codes q 2^-24, low nibbles masked in place) and sc 2^6 (q 2^-20, high
// nibbles), so that a product is sc q 2^-14; and the mins of chunk g / 2 (g
// even) or 2 + g / 2 (odd) as {m0, m0 2^-11, m1, m1 2^-11, 0 ...} for S's two
// numbers.
struct WScales {
    float d, dmin;
    h2_t sl[2], sh[2];
    h8_t m;
};

// {v, v} as binary16 pairs of the integer v = byte b of x (below 1024), times f
template <int B>
__device__ __forceinline__ h2_t byte_pair(uint32_t x, _Float16 f)
{
    // 0x6400 | v is 1024 + v
    const uint32_t p = __builtin_amdgcn_perm(0x64646464u, x, 0x04000400u | B | (B << 16));
    return (__builtin_bit_cast(h2_t, p) - h2_t{(_Float16)1024, (_Float16)1024}) * h2_t{f, f};
}

// shift = 16 (g / 2): the bytes of sub-blocks 2 (g / 2), + 1 and of 4 above;
// odd: all ones for odd g
__device__ __forceinline__ WScales scales_of(const uint4& h, uint32_t shift, uint32_t odd)
{
    WScales r;
    const h2_t dd = __builtin_bit_cast(h2_t, h.x);
    r.d = (float)dd.x;
    r.dmin = (float)dd.y;
    const uint32_t y = h.y >> shift;
    const uint32_t z = h.z >> shift;
    const uint32_t v = h.w >> shift;
    const uint32_t sc0 = y & 0x3F3Fu;
    const uint32_t sc1 = (v & 0x0F0Fu) | ((y >> 2) & 0x3030u);
    const uint32_t m_hi = ((v >> 4) & 0x0F0Fu) | ((z >> 2) & 0x3030u);
    const uint32_t mm = (m_hi & odd) | (z & 0x3F3Fu & ~odd);
    r.sl[0] = byte_pair<0>(sc0, (_Float16)1024);
    r.sh[0] = byte_pair<1>(sc0, (_Float16)64);
    r.sl[1] = byte_pair<0>(sc1, (_Float16)1024);
    r.sh[1] = byte_pair<1>(sc1, (_Float16)64);
    const h2_t lo = {(_Float16)1, (_Float16)(1.0f / 2048.0f)};
    const h2_t m0 = byte_pair<0>(mm, (_Float16)1) * lo;
    const h2_t m1 = byte_pair<1>(mm, (_Float16)1) * lo;
    const _Float16 o = (_Float16)0;
    r.m = h8_t{m0.x, m0.y, m1.x, m1.y, o, o, o, o};
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

// One superblock of 16 positions' x in LDS: 16-byte pieces c = 32 half + 4 u + g
// at 256 c, position j's 16 bytes in place j ^ g (the reads of a product's
// operand do not collide, the stores of four threads' 64 bytes by twos); then S:
// lane groups 2 h and 2 h + 1 of position j at kXs + 256 h + 16 j.
constexpr int kXs = 16384;
constexpr int kStage = kXs + 512;

// Eight waves of 16 weight rows each; a step is a superblock.  The tile's x is
// staged through two LDS buffers by all waves; the x and the weights of the
// step after the next load while one is computed.
constexpr int kTile = 16;              // positions per tile
constexpr int kWaves = 8;
constexpr int kBlockRows = 16 * kWaves;

__global__ void __launch_bounds__(64 * kWaves, 4)
grouped_kernel(GroupedArgs a, int row_blocks)
{
    __shared__ __align__(16) unsigned char xbuf[2][kStage];
    __shared__ __align__(16) unsigned char wbufs[kWaves][kWStage];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = tid >> 6;
    const int j = lane & 15;
    const int g = lane >> 4;
    const GroupWork work =
        find_work<kTile>(a.g.offsets, a.g.groups, a.g.rows, row_blocks, blockIdx.x);
    const GroupTile t = work.tile;
    if (t.count == 0) {
        return;
    }
    const int S = a.k / kQK;

    // weights: rows beyond the last are the last again, not written
    const int row0 = work.block * kBlockRows + wave * 16;
    const int64_t pitch = (int64_t)S * kBlockBytes;
    const uint8_t* const wrows = static_cast<const uint8_t*>(a.w) + (int64_t)t.group * a.n * pitch;
    const uint8_t* const wp0 =
        wrows + min(row0 + (lane >> 3), a.n - 1) * pitch + 16 + (lane & 7) * 16;
    const uint8_t* const wp1 =
        wrows + min(row0 + 8 + (lane >> 3), a.n - 1) * pitch + 16 + (lane & 7) * 16;
    const uint8_t* const hp = wrows + min(row0 + (lane >> 2), a.n - 1) * pitch + (lane & 3) * 4;
    unsigned char* const wbuf = wbufs[wave];
    WPiece w;
    auto load_w = [&](int sb) __attribute__((always_inline)) {
        const int64_t at = (int64_t)min(sb, S - 1) * kBlockBytes;
        w.c0 = *reinterpret_cast<const u4_t*>(wp0 + at);
        w.c1 = *reinterpret_cast<const u4_t*>(wp1 + at);
        w.h = *reinterpret_cast<const uint32_t*>(hp + at);
    };
    // into the wave's own LDS; its reads of the superblock before are behind it
    // (one wave's LDS accesses are in order)
    auto stage_w = [&]() __attribute__((always_inline)) {
        unsigned char* const c = wbuf + (lane >> 3) * kBlockBytes + 16 + (lane & 7) * 16;
        *reinterpret_cast<u4_t*>(c) = w.c0;
        *reinterpret_cast<u4_t*>(c + 8 * kBlockBytes) = w.c1;
        *reinterpret_cast<uint32_t*>(wbuf + (lane >> 2) * kBlockBytes + (lane & 3) * 4) = w.h;
    };
    load_w(0);

    // x: pieces 4 wave + tid % 4 (and 32 more) of position (tid / 4) % 16, and 16
    // bytes of S of position (tid / 2) % 16.  A position that is left out takes x
    // row 0, nothing is loaded behind the last one; no product of either is
    // written.
    const XWs ws = x_ws(a.ws, S, a.g.x_count);
    auto x_row = [&](int i) -> int {           // -1: left out
        if (i >= t.count) {
            return -1;
        }
        const int p = t.begin + i;
        const int r = a.g.x_rows ? a.g.x_rows[p] : p;
        return r < 0 || r / a.g.x_div >= a.g.x_count ? -1 : r / a.g.x_div;
    };
    const int lj = (tid >> 2) & 15;
    const int sj = (tid >> 1) & 15;
    const bool has_x = lj < t.count;
    const bool has_s = tid < 32 && sj < t.count;
    const char* const xsrc =
        ws.rows + (int64_t)max(x_row(lj), 0) * S * kXsb + wave * 64 + (tid & 3) * 16;
    const char* const ssrc =
        ws.rows + (int64_t)max(x_row(sj), 0) * S * kXsb + 1024 + (tid & 1) * 16;
    const int xdst = wave * 1024 + (tid & 3) * 256 + ((lj ^ (tid & 3)) << 4);
    const int sdst = kXs + (tid & 1) * 256 + sj * 16;
    u4_t xv[2], sv;
    auto load_x = [&](int sb) __attribute__((always_inline)) {
        const int64_t at = (int64_t)min(sb, S - 1) * kXsb;
        if (has_s) {
            sv = *reinterpret_cast<const u4_t*>(ssrc + at);
        }
        if (has_x) {
            xv[0] = *reinterpret_cast<const u4_t*>(xsrc + at);
            xv[1] = *reinterpret_cast<const u4_t*>(xsrc + at + 512);
        }
    };
    auto stage_x = [&](int buf) __attribute__((always_inline)) {
        unsigned char* const base = xbuf[buf];
        if (has_x) {
            *reinterpret_cast<u4_t*>(base + xdst) = xv[0];
            *reinterpret_cast<u4_t*>(base + xdst + 8192) = xv[1];
        }
        if (has_s) {
            *reinterpret_cast<u4_t*>(base + sdst) = sv;
        }
    };
    load_x(0);
    const int xr = x_row(j);
    int yr = -1;
    if (xr >= 0) {
        yr = a.g.y_rows ? a.g.y_rows[t.begin + j] : t.begin + j;
        yr = yr < a.g.y_count ? yr : -1;
    }
    const int exps = xr >= 0 ? ws.exps[xr] : 0;
    const uint32_t shift = 16 * (g >> 1);
    const uint32_t odd = g & 1 ? 0xFFFFFFFFu : 0u;
    const int xlane = g * 256 + ((j ^ g) << 4);
    const f4_t zero = {0.f, 0.f, 0.f, 0.f};
    f4_t total = zero;

    stage_w();
    stage_x(0);
    load_x(1);
    load_w(1);
    __syncthreads();
    for (int sb = 0; sb < S; ++sb) {
        if (row0 < a.n) {
            const unsigned char* const xs = xbuf[sb & 1];
            const unsigned char* const wr = wbuf + j * kBlockBytes;
            const uint4 h = *reinterpret_cast<const uint4*>(wr);
            const uint4 c0 = *reinterpret_cast<const uint4*>(wr + 16 + 16 * g);
            const uint4 c1 = *reinterpret_cast<const uint4*>(wr + 80 + 16 * g);
            const WScales sc = scales_of(h, shift, odd);
            const uint32_t c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
            f4_t ah = zero, al = zero;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const h8_t b = operand(c[u], sc.sl[u / 4], sc.sh[u / 4]);
                const h8_t xh = *reinterpret_cast<const h8_t*>(xs + u * 1024 + xlane);
                const h8_t xl = *reinterpret_cast<const h8_t*>(xs + 8192 + u * 1024 + xlane);
                ah = __builtin_amdgcn_mfma_f32_16x16x32_f16(xh, b, ah, 0, 0, 0);
                al = __builtin_amdgcn_mfma_f32_16x16x32_f16(xl, b, al, 0, 0, 0);
            }
            const uint2 s2 = *reinterpret_cast<const uint2*>(xs + kXs + (g >> 1) * 256 + j * 16 +
                                                             (g & 1) * 8);
            const u4_t sx = {s2.x, s2.y, 0u, 0u};
            const f4_t am = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8_t, sx),
                                                                   sc.m, zero, 0, 0, 0);
            // 2^14: the operands' 2^-14; lo carries 2^11 more; S is 2^-6
            const float dh = sc.d * 16384.0f;
            const float dm = sc.dmin * 64.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float v = __builtin_fmaf(al[e], 1.0f / 2048.0f, ah[e]);
                total[e] = __builtin_fmaf(dh, v, total[e]);
                total[e] = __builtin_fmaf(-dm, am[e], total[e]);
            }
        }
        stage_w();
        stage_x((sb + 1) & 1);
        // x before weights: waiting for x leaves the newest weights in flight
        load_x(sb + 2);
        load_w(sb + 2);
        __syncthreads();
    }
    // D[4 g + e][j]: position 4 g + e, weight row j
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int yrow = __shfl(yr, 4 * g + e, 64);
        const int exp = __shfl(exps, 4 * g + e, 64);
        if (row0 + j < a.n && yrow >= 0) {
            a.y[(int64_t)yrow * a.n + row0 + j] = ldexpf(total[e], -exp);
        }
    }
}

}  // namespace

size_t grouped_ws_bytes(int64_t k, int64_t x_count)
{
    return (size_t)x_count * (size_t)(k / kQK) * kXsb + (size_t)x_count * sizeof(int);
}

// The workgroups of the products
int64_t grouped_grid(int64_t rows, int64_t groups, int64_t n)
{
    const int64_t blocks = (n + kBlockRows - 1) / kBlockRows;
    return (most_tiles(rows, groups, kTile) * blocks + 7) / 8 * 8;
}

hipError_t launch_grouped(const GroupedArgs& a, hipStream_t stream)
{
    // a piece of eight elements per thread and pass
    const int pieces = a.k / 8;
    const dim3 rows((unsigned)a.g.x_count), threads(pieces < 1024 ? (pieces + 63) / 64 * 64 : 1024);
    if (a.q != nullptr) {
        hipLaunchKernelGGL(grouped_x_kernel<true>, rows, threads, 0, stream, a);
    } else {
        hipLaunchKernelGGL(grouped_x_kernel<false>, rows, threads, 0, stream, a);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) {
        return e;
    }
    const int64_t grid = grouped_grid(a.g.rows, a.g.groups, a.n);
    hipLaunchKernelGGL(grouped_kernel, dim3((unsigned)grid), dim3(64 * kWaves), 0, stream, a,
                       (a.n + kBlockRows - 1) / kBlockRows);
    return hipGetLastError();
}

}  // namespace q4k
