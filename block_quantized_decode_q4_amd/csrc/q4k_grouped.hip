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
// Two launches: grouped_x_kernel lays each position's x out once in the
// caller's workspace (hi, lo and S in the order in which the lanes of the
// product kernel read them); grouped_kernel multiplies.  A few rows (the tokens of
// one decode step) take one: the products' waves lay x out themselves.
//
// grouped_kernel: a wave computes 16 weight rows x 16 positions of one group
// (v_mfma_f32_16x16x32_f16, x as the rows, weights as the columns).  Lane
// l = 16 g + j holds weight row j and two 16-byte pieces of its codes in each
// superblock, and needs the scales of their four sub-blocks only: 9
// instructions for 8 codes (mask, shift, multiply by the scale), and the
// products with hi and with lo take the same registers.  The weights change
// lanes through LDS: the operand's own lane order would take 64 clocks of the
// vector cache per load where neighbouring lanes on neighbouring bytes take
// about 20.  x stays in registers over several row tiles; staging it in LDS for
// all waves of a workgroup, superblock by superblock with a barrier each, was
// slower (one token 27 us, 48 tokens on eight wide experts 124 us).
//
// What bounds it: by the counters neither pipe and not the bytes, but latency, with
// too few waves to hide it.  A superblock and row tile takes about 135 vector and 17
// matrix instructions.  48 tokens of uneven experts 4096 x 14336 (ten or eleven tiles
// where six to eight experts are met): 89 us for the products, with 268 MB read (3
// TB/s), the vector pipe busy 46 % of the time and the matrix pipe 21 %; two waves a
// SIMD on average, which wait half of their time to issue an instruction and a sixth
// of it for memory.  One token, two of eight experts 14336 x 4096 (66 MB): 20 us (3.3
// TB/s), the pipes busy 50 and 17 %, 1.5 waves a SIMD, a third of their time waiting
// for memory; the same bytes as 4096 x 14336, 256 workgroups, 26 us.  264 MB (eight
// experts 4096 x 14336, 16 positions each: 256 workgroups, one wave a SIMD) 76-78 us,
// 3.4 TB/s.  Measured without gain at 264 MB: two
// row tiles worked on at once, four row tiles of weights in flight instead of two,
// x of the next superblock asked for ahead (79 us each, and fewer waves a SIMD).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "q4k_device.h"
#include "q4k_groups.h"
#include "q4k_kernels.h"
#include "q4k_out.h"

namespace q4k {

namespace {

typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
typedef _Float16 h4_t __attribute__((ext_vector_type(4)));
typedef _Float16 h8_t __attribute__((ext_vector_type(8)));
typedef float f4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));

// The workspace: x by position, kXsb bytes per position and superblock.  The
// positions begin .. begin + count - 1 of a tile share the bytes of theirs: per
// superblock first the 64 pieces of 16 bytes, c = 32 half + 4 u + g (half 0: hi,
// 1: lo; product u, lane group g), piece c of the tile's position i at
// (c count + i) 16; then S, lane group g of position i at (g count + i) 8.  So an
// operand's load takes consecutive bytes in consecutive lanes, and no byte is
// spent on positions that are not there.  The positions' scale exponents
// follow.
constexpr int kXsb = 1056;
constexpr int kTile = 16;              // positions per tile

struct XWs {
    char* rows;
    int* exps;
};

__host__ __device__ inline XWs x_ws(void* ws, int S, int64_t rows)
{
    XWs r;
    r.rows = static_cast<char*>(ws);
    r.exps = reinterpret_cast<int*>(r.rows + rows * S * kXsb);
    return r;
}

// The x row of position p, -1: left out
__device__ __forceinline__ int x_row_of(const GroupRows& g, int p)
{
    const int r = g.x_rows ? g.x_rows[p] : p;
    return r < 0 || r / g.x_div >= g.x_count ? -1 : r / g.x_div;
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

// v of the lane that DPP control CTRL pairs with this one
template <int CTRL>
__device__ __forceinline__ float paired(float v)
{
    return __builtin_bit_cast(float, dpp_i<CTRL>(__builtin_bit_cast(int, v)));
}

// The largest of a row of 16 lanes (rotations by 8, 4, 2, 1), in all of them
__device__ __forceinline__ float row_top(float v)
{
    v = fmaxf(v, paired<0x128>(v));
    v = fmaxf(v, paired<0x124>(v));
    v = fmaxf(v, paired<0x122>(v));
    return fmaxf(v, paired<0x121>(v));
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
    // pairs and fours within a quad, then the mirrored lane of the eight
    s0 += paired<0xB1>(s0);
    s1 += paired<0xB1>(s1);
    s0 += paired<0x4E>(s0);
    s1 += paired<0x4E>(s1);
    s0 += paired<0x141>(s0);
    s1 += paired<0x141>(s1);
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

// One workgroup per position.  Up to kHeld pieces per thread stay in registers
// between the row's largest and the conversion (k to 16384); the rest of a
// longer row is read again.
constexpr int kHeld = 2;

template <bool Q8>
__global__ void __launch_bounds__(1024)
grouped_x_kernel(GroupedArgs a)
{
    __shared__ float part[16];
    const int p = blockIdx.x;
    const int tid = threadIdx.x;
    const int threads = blockDim.x;
    const int S = a.k / kQK;
    const XWs ws = x_ws(a.ws, S, a.g.rows);
    const int64_t row = x_row_of(a.g, p);
    if (row < 0) {
        return;                                // left out: never read
    }
    float4 held[kHeld][2];
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {          // the row's last piece for those behind it
        load_x<Q8>(a, row, min(h * threads + tid, S * 32 - 1), held[h][0], held[h][1]);
    }
    const GroupTile t = tile_of<kTile>(a.g.offsets, a.g.groups, a.g.rows, p);
    if (t.count == 0) {
        return;                                // in no group
    }
    float top = 0.f;
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
        top = piece_top(held[h][0], held[h][1], top);
    }
    for (int v = kHeld * threads + tid; v < S * 32; v += threads) {
        float4 lo, hi;
        load_x<Q8>(a, row, v, lo, hi);
        top = piece_top(lo, hi, top);
    }
    top = row_top(top);
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    if ((tid & 63) == 0) {
        part[tid >> 6] = top;
    }
    __syncthreads();
    for (int i = 0; i < threads / 64; ++i) {
        top = fmaxf(top, part[i]);
    }
    const int s = scale_of(top);
    if (tid == 0) {
        ws.exps[p] = s;
    }
    const int i = p - t.begin;
    char* const out = ws.rows + (int64_t)t.begin * S * kXsb;
    auto put = [&](int v, const float4& lo4, const float4& hi4) __attribute__((always_inline)) {
        h8_t h, l;
        h4_t sums;
        convert(lo4, hi4, s, h, l, sums);
        const PieceAt at = piece_at(v);
        char* const o = out + (int64_t)(v >> 5) * t.count * kXsb;
        const int c = 4 * at.u + at.g;
        *reinterpret_cast<h8_t*>(o + (c * t.count + i) * 16) = h;
        *reinterpret_cast<h8_t*>(o + ((32 + c) * t.count + i) * 16) = l;
        if ((v & 7) == 0) {
            *reinterpret_cast<h4_t*>(o + t.count * 1024 + (at.sg * t.count + i) * 8) = sums;
        }
    };
    // whole eights of lanes: S * 32 is a multiple of 8
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
        if (h * threads + tid < S * 32) {
            put(h * threads + tid, held[h][0], held[h][1]);
        }
    }
    for (int v = kHeld * threads + tid; v < S * 32; v += threads) {
        float4 lo4, hi4;
        load_x<Q8>(a, row, v, lo4, hi4);
        put(v, lo4, hi4);
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

// Four waves: kw of them share the superblocks (wave part p takes p, p + kw,
// ...), 4 / kw take rows of their own, T tiles of 16 rows each.  A wave keeps the
// x of one superblock in registers, straight from the workspace, and goes
// through its row tiles with it; the sums of all its tiles stay in registers
// too, and the parts are added up once, at the end.  No barrier before that: a
// wave waits for its own loads only.  Up to three waves a SIMD (x alone takes
// 66 registers); few workgroups leave fewer.
constexpr int kWaves = 4;

template <int T>
constexpr int kWaveLds = T * 1024 > kWStage ? T * 1024 : kWStage;   // weights, then sums

// Few positions in all (kFused<T> at most): no launch for x.  A wave lays out the x of
// its superblock itself, in LDS: 32 lanes a position, eight elements a lane, scaled
// by the superblock's largest |x|.  The sums are kept in the scale of the largest
// so far (2^-E of a position; E falls, and the sums with it, when a larger one
// comes), and the parts of k are joined in the smallest E.
enum FusedX { kXLaidOut, kXF32, kXQ8 };
template <int T>
constexpr int kFused = T == 2 ? 16 : 8;            // so that two workgroups fit a CU's LDS
constexpr int kNoScale = 1000;         // nothing but zeros so far
template <int T, int FUSED>
constexpr int kXLds = FUSED == kXLaidOut ? 0 : kFused<T> * kXsb;    // per wave

template <int T, int FUSED>
__device__ __forceinline__ void grouped_tiles(const GroupedOut& a, const GroupTiles& tiles,
                                              int row_blocks, int kw_log2, unsigned char* smem)
{
    constexpr int kLds = kWaveLds<T> + kXLds<T, FUSED>;
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    // wave-uniform, as are all addresses but the lanes' 32-bit offsets below
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & 15;
    const int g = lane >> 4;
    const GroupWork work =
        find_work<kTile>(tiles, a.g.offsets, a.g.groups, a.g.rows, row_blocks, blockIdx.x);
    const GroupTile t = work.tile;
    if (t.count == 0) {
        return;
    }
    const int S = a.k / kQK;
    const int kw = 1 << kw_log2;
    const int wk = wave & (kw - 1);
    const int rows_per_group = 16 * T;
    const int row0 = (work.block * (kWaves >> kw_log2) + (wave >> kw_log2)) * rows_per_group;
    const int slabs = (S + kw - 1) >> kw_log2;

    // weights: a row tile that would pass the last row ends there instead (its
    // rows are then written twice, with the same bits); fewer than 16 rows: the
    // last again, not written
    const int64_t pitch = (int64_t)S * kBlockBytes;
    const uint8_t* const wrows = static_cast<const uint8_t*>(a.w) + (int64_t)t.group * a.n * pitch;
    const int last = max(a.n - 16, 0);
    const uint32_t off0 = (uint32_t)(min(lane >> 3, a.n - 1) * (int)pitch + 16 + (lane & 7) * 16);
    const uint32_t off1 =
        (uint32_t)(min(8 + (lane >> 3), a.n - 1) * (int)pitch + 16 + (lane & 7) * 16);
    const uint32_t offh = (uint32_t)(min(lane >> 2, a.n - 1) * (int)pitch + (lane & 3) * 4);
    unsigned char* const wbuf = smem + wave * kLds;
    WPiece w[2];
    // row tile `tile` (0 .. T - 1) of slab `slab` into set `tile % 2`
    auto load_w = [&](int slab, int tile, auto set) __attribute__((always_inline)) {
        const uint8_t* const at = wrows + min(row0 + 16 * tile, last) * pitch +
                                  (int64_t)min(slab * kw + wk, S - 1) * kBlockBytes;
        WPiece& p = w[decltype(set)::value];
        p.c0 = *reinterpret_cast<const u4_t*>(at + off0);
        p.c1 = *reinterpret_cast<const u4_t*>(at + off1);
        p.h = *reinterpret_cast<const uint32_t*>(at + offh);
    };
    // x: positions behind the last read the last's, whose products are its own
    const XWs ws = x_ws(a.ws, S, a.g.rows);
    const int slot = min(j, t.count - 1);
    const char* const xrows = ws.rows + (int64_t)t.begin * S * kXsb;
    const uint32_t xoff = (uint32_t)((g * t.count + slot) * 16);
    u4_t xh[8], xl[8];
    uint2 xs;
    auto take_x = [&](const char* at) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            xh[u] = *reinterpret_cast<const u4_t*>(at + u * t.count * 64 + xoff);
            xl[u] = *reinterpret_cast<const u4_t*>(at + (8 + u) * t.count * 64 + xoff);
        }
        xs = *reinterpret_cast<const uint2*>(at + t.count * 1024 + xoff / 2);
    };
    // fused: this lane's position is 2 pass + lane / 32; lane p < count also keeps
    // what is known of position p
    unsigned char* const xbuf = wbuf + kWaveLds<T>;
    const int lane_row =
        FUSED ? max(x_row_of(a.g, t.begin + min(lane & (kFused<T> - 1), t.count - 1)), 0) : 0;
    int scale = kNoScale;                      // E
    float4 raw[2];
    auto fetch_x = [&](int slab, int pass) __attribute__((always_inline)) {
        const int64_t row = __shfl(lane_row, min(2 * pass + (lane >> 5), t.count - 1), 64);
        ::q4k::load_x<FUSED == kXQ8>(a, row, min(slab * kw + wk, S - 1) * 32 + (lane & 31), raw[0],
                                     raw[1]);
    };
    float factor[4] = {1.f, 1.f, 1.f, 1.f};    // of positions 4 g + e in this superblock
    const uint32_t shift = 16 * (g >> 1);
    const uint32_t odd = g & 1 ? 0xFFFFFFFFu : 0u;
    const f4_t zero = {0.f, 0.f, 0.f, 0.f};
    f4_t total[T];
#pragma unroll
    for (int i = 0; i < T; ++i) {
        total[i] = zero;
    }
    load_w(0, 0, std::integral_constant<int, 0>());
    load_w(0, 1, std::integral_constant<int, 1>());
    if constexpr (FUSED != kXLaidOut) {
        fetch_x(0, 0);
    }
    for (int slab = 0; slab < slabs; ++slab) {
        const bool in = slab * kw + wk < S;
        if constexpr (FUSED == kXLaidOut) {
            take_x(xrows + (int64_t)min(slab * kw + wk, S - 1) * t.count * kXsb);
        } else if (in) {
            int now = kNoScale;
            wave_lds_order();
            for (int pass = 0; 2 * pass < t.count; ++pass) {
                if (pass > 0) {
                    fetch_x(slab, pass);
                }
                float top = row_top(piece_top(raw[0], raw[1], 0.f));
                top = fmaxf(top, __shfl_xor(top, 16, 64));
                const int p = 2 * pass + (lane >> 5);
                const int sc = scale_of(top);
                h8_t h, l;
                h4_t sums;
                convert(raw[0], raw[1], sc, h, l, sums);
                if (p < t.count) {
                    const PieceAt at = piece_at(lane & 31);
                    const int c = 4 * at.u + at.g;
                    *reinterpret_cast<h8_t*>(xbuf + (c * t.count + p) * 16) = h;
                    *reinterpret_cast<h8_t*>(xbuf + ((32 + c) * t.count + p) * 16) = l;
                    if ((lane & 7) == 0) {
                        *reinterpret_cast<h4_t*>(xbuf + t.count * 1024 +
                                                 (at.sg * t.count + p) * 8) = sums;
                    }
                }
                const int of = __shfl(top > 0.f ? sc : kNoScale, (lane & 1) * 32, 64);
                now = lane >> 1 == pass ? of : now;
            }
            wave_lds_order();
            const int next = min(scale, now);
            if (__any(next < scale)) {                 // the sums so far, in the new scale
                const int down = scale == kNoScale ? 0 : next - scale;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int d = __shfl(down, 4 * g + e, 64);
#pragma unroll
                    for (int i = 0; i < T; ++i) {
                        total[i][e] = ldexpf(total[i][e], d);
                    }
                }
                scale = next;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                factor[e] = ldexpf(1.f, __shfl(scale - now, 4 * g + e, 64));
            }
            take_x(reinterpret_cast<const char*>(xbuf));
            fetch_x(min(slab + 1, slabs - 1), 0);
        }
        auto tile = [&](int i, auto set) __attribute__((always_inline)) {
            // through the wave's own LDS
            wave_lds_order();
            const WPiece& p = w[decltype(set)::value];
            unsigned char* const c = wbuf + (lane >> 3) * kBlockBytes + 16 + (lane & 7) * 16;
            *reinterpret_cast<u4_t*>(c) = p.c0;
            *reinterpret_cast<u4_t*>(c + 8 * kBlockBytes) = p.c1;
            *reinterpret_cast<uint32_t*>(wbuf + (lane >> 2) * kBlockBytes + (lane & 3) * 4) = p.h;
            wave_lds_order();
            // the tile after the next (of the next slab behind the last two)
            load_w(i + 2 < T ? slab : min(slab + 1, slabs - 1), (i + 2) % T, set);
            if (!in) {
                return;
            }
            const unsigned char* const wr = wbuf + j * kBlockBytes;
            const uint4 h = *reinterpret_cast<const uint4*>(wr);
            const uint4 c0 = *reinterpret_cast<const uint4*>(wr + 16 + 16 * g);
            const uint4 c1 = *reinterpret_cast<const uint4*>(wr + 80 + 16 * g);
            const WScales sc = scales_of(h, shift, odd);
            const uint32_t cc[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
            f4_t ah = zero, al = zero;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const h8_t b = operand(cc[u], sc.sl[u / 4], sc.sh[u / 4]);
                ah = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8_t, xh[u]), b, ah,
                                                            0, 0, 0);
                al = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8_t, xl[u]), b, al,
                                                            0, 0, 0);
            }
            const u4_t sx = {xs.x, xs.y, 0u, 0u};
            const f4_t am = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8_t, sx),
                                                                   sc.m, zero, 0, 0, 0);
            // 2^14: the operands' 2^-14; lo carries 2^11 more; S is 2^-6
            const float dh = sc.d * 16384.0f;
            const float dm = sc.dmin * 64.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float v = __builtin_fmaf(al[e], 1.0f / 2048.0f, ah[e]);
                if constexpr (FUSED == kXLaidOut) {
                    total[i][e] = __builtin_fmaf(dh, v, total[i][e]);
                    total[i][e] = __builtin_fmaf(-dm, am[e], total[i][e]);
                } else {
                    const float both = __builtin_fmaf(-dm, am[e], dh * v);
                    total[i][e] = __builtin_fmaf(factor[e], both, total[i][e]);
                }
            }
        };
        static_assert(T % 2 == 0, "two sets in turn");
#pragma unroll
        for (int i = 0; i < T; i += 2) {
            tile(i, std::integral_constant<int, 0>());
            tile(i + 1, std::integral_constant<int, 1>());
        }
    }
    // the parts of k, in their order; every wave joins and writes some tiles
    wave_lds_order();
    f4_t* const part = reinterpret_cast<f4_t*>(wbuf);
#pragma unroll
    for (int i = 0; i < T; ++i) {
        part[i * 64 + lane] = total[i];
    }
    const int p = t.begin + slot;
    int yr = -1;
    if (j < t.count && x_row_of(a.g, p) >= 0) {
        yr = a.g.y_rows ? a.g.y_rows[p] : p;
        yr = yr < a.g.y_count ? yr : -1;
    }
    int exps = 0;
    if constexpr (FUSED == kXLaidOut) {
        exps = ws.exps[p];
    } else if (lane < 16) {
        reinterpret_cast<int*>(xbuf)[lane] = scale;
    }
    __syncthreads();
    for (int q = wave; q < (kWaves >> kw_log2) * T; q += kWaves) {
        const int rg = q / T;
        const int i = q % T;
        const unsigned char* const first = smem + (rg << kw_log2) * kLds;
        const unsigned char* const from = first + (i * 64 + lane) * 16;
        f4_t sum = zero;
        int4 least = make_int4(kNoScale, kNoScale, kNoScale, kNoScale);
        if constexpr (FUSED != kXLaidOut) {
            for (int z = 0; z < kw; ++z) {
                const int4 of =
                    reinterpret_cast<const int4*>(first + z * kLds + kWaveLds<T>)[g];
                least.x = min(least.x, of.x);
                least.y = min(least.y, of.y);
                least.z = min(least.z, of.z);
                least.w = min(least.w, of.w);
            }
        }
        for (int z = 0; z < kw; ++z) {
            f4_t one = *reinterpret_cast<const f4_t*>(from + z * kLds);
            if constexpr (FUSED != kXLaidOut) {
                const int4 of =
                    reinterpret_cast<const int4*>(first + z * kLds + kWaveLds<T>)[g];
                one = f4_t{ldexpf(one[0], least.x - of.x), ldexpf(one[1], least.y - of.y),
                           ldexpf(one[2], least.z - of.z), ldexpf(one[3], least.w - of.w)};
            }
            sum = z == 0 ? one : sum + one;
        }
        const int scales[4] = {least.x, least.y, least.z, least.w};
        const int tile_row = (work.block * (kWaves >> kw_log2) + rg) * rows_per_group + 16 * i;
        const int row = min(tile_row, last) + j;
        // D[4 g + e][j]: position 4 g + e, weight row j
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int yrow = __shfl(yr, 4 * g + e, 64);
            const int exp = FUSED == kXLaidOut ? __shfl(exps, 4 * g + e, 64) : scales[e];
            // with an epilogue once: y may be its residual or gate
            if (row < a.n && yrow >= 0 && (!kEpilogue || row >= tile_row)) {
                put_grouped(a, work.tile.group, yrow, row, ldexpf(sum[e], -exp));
            }
        }
    }
}

constexpr int kCus = 256;

template <int T, int FUSED>
__global__ void __launch_bounds__(64 * kWaves, FUSED == kXLaidOut ? 3 : 2)
grouped_kernel(GroupedOut a, int row_blocks, int kw_log2)
{
    __shared__ __align__(16) unsigned char smem[kWaves * (kWaveLds<T> + kXLds<T, FUSED>)];
    const GroupTiles t =
        count_tiles<kTile>(a.g.offsets, a.g.groups, a.g.rows, (int)gridDim.x / row_blocks);
    grouped_tiles<T, FUSED>(a, t, row_blocks, kw_log2, smem);
}

// T = 8 or, in fine_blocks, T = 4, by the number of tiles, which the host does not
// know: rounds of the chip times the work of one, a tile of the finer cut counting
// 9/8 (x is read twice as often).  So the finer cut is taken where the coarse one
// leaves much of its last round empty: ten tiles of 4096 x 14336, 320 workgroups
// at T = 8, 105 us against 96 us; eight tiles, 256 workgroups, 78 us against 87 us.
__global__ void __launch_bounds__(64 * kWaves, 3)
grouped_either_kernel(GroupedOut a, int row_blocks, int fine_blocks, int kw_log2)
{
    __shared__ __align__(16) unsigned char smem[kWaves * kWaveLds<8>];
    const GroupTiles t =
        count_tiles<kTile>(a.g.offsets, a.g.groups, a.g.rows, (int)gridDim.x / fine_blocks);
    const int coarse = (t.tiles * row_blocks + kCus - 1) / kCus;
    const int fine = (t.tiles * fine_blocks + kCus - 1) / kCus;
    if (coarse * 2 * 8 <= fine * 9) {
        grouped_tiles<8, kXLaidOut>(a, t, row_blocks, kw_log2, smem);
    } else {
        grouped_tiles<4, kXLaidOut>(a, t, fine_blocks, kw_log2, smem);
    }
}

// How the rows are cut: T row tiles per wave and kw waves along k.
//  - T = 2 while T = 4 would give fewer workgroups than CUs (one token, two
//    experts 4096 x 14336: 25.6 us against 35.1);
//  - T = 8 where the groups hold 8 positions or more: x is read once per T
//    tiles (eight experts 4096 x 14336 with 16 positions each 83 us against 93,
//    128 positions each 141 / 157 us), and T = 4 otherwise (one token, eight of
//    64 experts 1536 x 2048: 11.7 us against 15.3).
//  - kw = 4, so that a row's loads are 576 consecutive bytes, but less where more
//    than a fifth of the waves' steps would find no superblock (k = 1536, 64
//    experts of 2048 rows with two positions each: kw 4 / 2 39.5 / 34.9 us); T = 2
//    keeps 4, the shorter way.
//  - x laid out by the products' own waves for a few rows, up to two a group on
//    average (how they are spread is not known here) and k to 8192.  A launch for x
//    against none: one token, eight of 64 experts 1536 x 2048 11.3 / 8.7 us, two of
//    eight 14336 x 4096 21.6 / 20.0 us, 4096 x 14336 25.7 / 25.8 us; 16 rows, two a
//    group, 512 x 2048 9.2 / 6.7 us, eight a group 9.4 / 10.9 us; eight rows of one
//    group 4096 x 4096 15.3 / 21.6 us (every block of rows converts them again).  At
//    T = 4, 16 rows would leave one workgroup a CU.
struct GroupedCut {
    int T, kw_log2;
    bool fused;                        // x laid out by the products' own waves
    int blocks, fine;                  // blocks of rows
    int64_t grid;
};

GroupedCut grouped_cut(int64_t rows, int64_t groups, int64_t n, int64_t k)
{
    const int64_t tiles = most_tiles(rows, groups, kTile);
    const int64_t S = k / kQK;
    GroupedCut c;
    c.T = tiles * ((n + 63) / 64) < 256 ? 2 : rows >= 8 * groups ? 8 : 4;
    c.fused = c.T < 8 && rows <= (c.T == 2 ? kFused<2> : kFused<4>) && rows <= 2 * groups &&
              k <= 8192;
    c.kw_log2 = 2;
    auto steps = [&](int log2) { return (((S - 1) >> log2) + 1) << log2; };  // of all parts
    while (c.T > 2 && c.kw_log2 > 0 && steps(c.kw_log2) * 4 > S * 5) {
        --c.kw_log2;
    }
    const int64_t per = 16 * c.T * (kWaves >> c.kw_log2);
    c.blocks = (int)((n + per - 1) / per);
    // The finer cut's larger grid is only worth its empty workgroups (16 tiles of
    // 4096 x 2048, 23 possible: 26.5 us instead of 24.7) while two rounds of the
    // chip hold the coarse one.
    c.fine = c.T == 8 && tiles * c.blocks <= 2 * kCus ? (int)((2 * n + per - 1) / per) : 0;
    c.grid = (tiles * (c.fine > 0 ? c.fine : c.blocks) + 7) / 8 * 8;
    return c;
}

}  // namespace

#ifndef Q4K_EPILOGUE
size_t grouped_ws_bytes(int64_t k, int64_t rows)
{
    return (size_t)rows * (size_t)(k / kQK) * kXsb + (size_t)rows * sizeof(int);
}

// The workgroups of the products
int64_t grouped_grid(int64_t rows, int64_t groups, int64_t n, int64_t k)
{
    return grouped_cut(rows, groups, n, k).grid;
}
#endif  // Q4K_EPILOGUE

hipError_t launch_grouped(const GroupedOut& a, hipStream_t stream)
{
    const GroupedCut c = grouped_cut(a.g.rows, a.g.groups, a.n, a.k);
    const dim3 grid((unsigned)c.grid), block(64 * kWaves);
    if (c.fused) {                             // T is 2 or 4
        auto launch = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, grid, block, 0, stream, a, c.blocks, c.kw_log2);
        };
        if (c.T == 2) {
            a.q ? launch(grouped_kernel<2, kXQ8>) : launch(grouped_kernel<2, kXF32>);
        } else {
            a.q ? launch(grouped_kernel<4, kXQ8>) : launch(grouped_kernel<4, kXF32>);
        }
        return hipGetLastError();
    }
    // a piece of eight elements per thread and pass
    const int pieces = a.k / 8;
    const dim3 rows((unsigned)a.g.rows), threads(pieces < 1024 ? (pieces + 63) / 64 * 64 : 1024);
    if (a.q != nullptr) {
        hipLaunchKernelGGL(grouped_x_kernel<true>, rows, threads, 0, stream, a);
    } else {
        hipLaunchKernelGGL(grouped_x_kernel<false>, rows, threads, 0, stream, a);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) {
        return e;
    }
    if (c.T == 2) {
        hipLaunchKernelGGL((grouped_kernel<2, kXLaidOut>), grid, block, 0, stream, a, c.blocks,
                           c.kw_log2);
    } else if (c.T == 4) {
        hipLaunchKernelGGL((grouped_kernel<4, kXLaidOut>), grid, block, 0, stream, a, c.blocks,
                           c.kw_log2);
    } else if (c.fine > 0) {
        hipLaunchKernelGGL(grouped_either_kernel, grid, block, 0, stream, a, c.blocks, c.fine,
                           c.kw_log2);
    } else {
        hipLaunchKernelGGL((grouped_kernel<8, kXLaidOut>), grid, block, 0, stream, a, c.blocks,
                           c.kw_log2);
    }
    return hipGetLastError();
}

}  // namespace q4k
