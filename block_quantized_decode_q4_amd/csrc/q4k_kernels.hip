// q4k_kernels.hip -- HIP kernels for the Q4_K fused dequantize-and-multiply
// GEMV on CDNA4 (gfx950, wave64): the fp32 kernels 1 (x-stager) and 2
// (streaming), the dequantizer and the read calibration; launch plans are
// made in q4k_api.hip.
//
// Problem (see include/q4k.h for the page citations): y[b][r] =
// sum_c W[r][c] * x[b][c], W stored as GGUF Q4_K superblocks of 144 bytes /
// 256 weights, w = d*sc_j*q - dmin*m_j.
//
// Design (MI355X-first; the pages' CUDA kernels are prior art only):
//  * Lane map.  Four lanes share a superblock; lane t owns the 64-element
//    chunk c = t % 4 of superblock t / 4, i.e. 32 quant bytes (two 16-byte
//    loads) and the two sub-blocks 2c (low nibbles) and 2c+1 (high
//    nibbles).  One wave pass covers 16 superblocks = 4096 elements (a
//    "span").  Per superblock and row each lane issues three dwordx4 loads:
//    the 16-byte header (d, dmin, scales) and its 32 quant bytes.
//  * Exact weights, exact products.  A 4-bit code placed in the low
//    mantissa bits of an fp16 is the subnormal q*2^-24 (or q*2^-20 for a
//    high nibble masked in place), exactly.  One AND turns a dword of
//    codes into two such fp16 values, and one v_fma_mix_f32 gives the
//    weight fl32(d*sc*q - dmin*m) rounded once, as the format defines it
//    (d*sc*2^24, or 2^20, and dmin*m are exact f32 factors per sub-block).
//    Each weight times its x is exact in f64 and added in f64, so the only
//    error before the final rounding of y to f32 is f64 rounding, for any
//    finite x and weights (no f32 range limit on the products), and inf and
//    NaN propagate as in IEEE arithmetic.
//  * x stager (LDS).  A workgroup stages x (or a K-chunk of it) into LDS in
//    lane order -- [vector][span][v = 0..15][lane] float4 -- so every
//    ds_read_b128 of a wave reads 1 KiB of consecutive LDS (no bank
//    conflicts).  With one span and one vector, x is then held in 64 VGPRs
//    per lane for the whole row loop.
//  * K-chunked path.  When x does not fit the single-stage LDS budget, it is
//    staged spans_per_chunk spans at a time; each lane's partial sums are
//    parked in LDS between chunks, so the accumulation order -- and the
//    result -- is identical to the single-stage path.
//  * Multi-output scheduling.  A workgroup owns rows_per_block consecutive
//    rows; its waves take groups of R rows round-robin and decode R rows per
//    pass against one read of x, and the row loop streams each row once.
//  * Per-row reduction: 64 f64 lane partials -> one value with a butterfly
//    of cross-lane adds, rounded once to f32; y is written once per row
//    (overwrite).
//  * m-batched (m <= 8): each decoded code feeds m accumulators.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4k_device.h"
#include "q4k_kernels.h"
#include "q4k_out.h"

namespace q4k {

// ------------------------------------------------------------ x stager
// Stage spans [span0, span0 + nsp) of every vector into LDS in lane order.
// Slot ((b*nsp + sp)*16 + v)*64 + lane holds, for superblock sb =
// (span0+sp)*16 + lane/4, chunk c = lane%4, u = v/2, h = v%2:
// x[b][sb*256 + 64c + 32h + 4u + {0,2,1,3}].  Superblocks past the row end
// stage zeros.
template <int M>
__device__ __forceinline__ void stage_x(const float* __restrict__ x, int k, int S, int span0,
                                        int nsp, float4* xs, int tid, int nthreads)
{
    const int per_vec = nsp * 1024;
    const int total = M * per_vec;
    // loads in batches of four per thread before the writes (one memory
    // latency per batch rather than per element)
    for (int base = tid; base < total; base += 4 * nthreads) {
        float4 g[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int slot = base + i * nthreads;
            const int b = slot / per_vec;
            const int rem = slot - b * per_vec;
            const int sp = rem >> 10;
            const int v = (rem >> 6) & 15;
            const int ln = rem & 63;
            const int sb = (span0 + sp) * 16 + (ln >> 2);
            g[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (slot < total && sb < S) {
                const int e = sb * 256 + 64 * (ln & 3) + 32 * (v & 1) + 4 * (v >> 1);
                g[i] = *reinterpret_cast<const float4*>(x + (size_t)b * k + e);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int slot = base + i * nthreads;
            if (slot < total) {
                xs[slot] = make_float4(g[i].x, g[i].z, g[i].y, g[i].w);
            }
        }
    }
    __syncthreads();
}

// ---------------------------------------------------------------- GEMV
template <int M, int R, int NW, bool XREG>
__global__ void __launch_bounds__(NW * 64)
gemv_kernel(const uint8_t* __restrict__ w, const float* __restrict__ x, Out y,
            int n, int k, int S, int rows_per_block, int spans_per_chunk)
{
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = tid >> 6;
    const int c = lane & 3;
    const int sbl = lane >> 2;

    const int nspans = (S + 15) >> 4;
    const int chunk_spans = spans_per_chunk < nspans ? spans_per_chunk : nspans;
    const int nchunks = (nspans + chunk_spans - 1) / chunk_spans;
    float4* xs = reinterpret_cast<float4*>(smem);
    double* partial = reinterpret_cast<double*>(xs + M * chunk_spans * 1024);
    const uint32_t shift = (uint32_t)(c & 1) * 16u;
    const uint32_t sel = c < 2 ? 0xFFFFFFFFu : 0u;

    const int row0 = blockIdx.x * rows_per_block;
    const int rows_here = min(rows_per_block, n - row0);
    const int ngroups = (rows_here + R - 1) / R;
    const size_t row_bytes = (size_t)S * 144;

    for (int ch = 0; ch < nchunks; ++ch) {
        const int span0 = ch * chunk_spans;
        const int nsp = min(chunk_spans, nspans - span0);
        if (ch > 0) {
            __syncthreads();            // every wave is done with the previous chunk
        }
        stage_x<M>(x, k, S, span0, nsp, xs, tid, NW * 64);

        float4 xr[XREG ? 16 : 1];
        if constexpr (XREG) {
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                xr[v] = xs[v * 64 + lane];
            }
        }

        for (int g = wave; g < ngroups; g += NW) {
            double acc[R][M];
#pragma unroll
            for (int i = 0; i < R; ++i) {
#pragma unroll
                for (int b = 0; b < M; ++b) {
                    acc[i][b] = ch == 0 ? 0.0 : partial[((g * R + i) * M + b) * 64 + lane];
                }
            }
            for (int sp = 0; sp < nsp; ++sp) {
                const int sb = (span0 + sp) * 16 + sbl;
                const bool sb_ok = sb < S;
                uint4 hd[R], qa[R], qb[R];
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const int rl = g * R + i;
                    if (sb_ok && rl < rows_here) {
                        const uint8_t* p = w + (size_t)(row0 + rl) * row_bytes + (size_t)sb * 144;
                        hd[i] = load16(p);
                        qa[i] = load16(p + 16 + 32 * c);
                        qb[i] = load16(p + 32 + 32 * c);
                    } else {
                        hd[i] = make_uint4(0u, 0u, 0u, 0u);
                        qa[i] = make_uint4(0u, 0u, 0u, 0u);
                        qb[i] = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                ChunkScales cs[R];
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    cs[i] = decode_header(hd[i], shift, sel);
                }
                // low and high sub-block sums apart: two chains per row and vector
                double alo[R][M], ahi[R][M];
#pragma unroll
                for (int i = 0; i < R; ++i) {
#pragma unroll
                    for (int b = 0; b < M; ++b) {
                        alo[i][b] = acc[i][b];
                        ahi[i][b] = 0.0;
                    }
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    float4 xl[M], xh[M];
                    if constexpr (XREG) {
                        xl[0] = xr[2 * u];
                        xh[0] = xr[2 * u + 1];
                    } else {
#pragma unroll
                        for (int b = 0; b < M; ++b) {
                            const float4* xb = xs + (b * nsp + sp) * 1024 + lane;
                            xl[b] = xb[(2 * u) * 64];
                            xh[b] = xb[(2 * u + 1) * 64];
                        }
                    }
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        const uint4& q4 = u < 4 ? qa[i] : qb[i];
                        const int uu = u & 3;
                        const uint32_t D = uu == 0 ? q4.x : uu == 1 ? q4.y : uu == 2 ? q4.z : q4.w;
#pragma unroll
                        for (int b = 0; b < M; ++b) {
                            dot8_exact(D, xl[b], xh[b], cs[i].sl, cs[i].sh, cs[i].ml, cs[i].mh,
                                       alo[i][b], ahi[i][b]);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < R; ++i) {
#pragma unroll
                    for (int b = 0; b < M; ++b) {
                        acc[i][b] = alo[i][b] + ahi[i][b];
                    }
                }
            }
            if (ch == nchunks - 1) {
#pragma unroll
                for (int i = 0; i < R; ++i) {
#pragma unroll
                    for (int b = 0; b < M; ++b) {
                        const double v = wave_sum(acc[i][b]);
                        const int rl = g * R + i;
                        if (lane == 0 && rl < rows_here) {
                            const size_t at = (size_t)b * n + row0 + rl;
                            put_y(y, at, fetch_y(y, true, at, row0 + rl), v);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < R; ++i) {
#pragma unroll
                    for (int b = 0; b < M; ++b) {
                        partial[((g * R + i) * M + b) * 64 + lane] = acc[i][b];
                    }
                }
            }
        }
    }
}

// Stage spans [span0, span0 + nsp) of one vector into LDS in lane order
// (slot (sp*16 + v)*64 + lane; see stage_x).  Loads are issued in batches of
// four per thread before any of them is written, so the stage costs about
// one memory latency rather than one per loop trip.
template <int NT>
__device__ __forceinline__ void stage_x_batched(const float* __restrict__ x, int S, int span0,
                                                int nsp, float4* xs, int tid)
{
    const int total = nsp * 1024;
    for (int base = tid; base < total; base += 4 * NT) {
        float4 g[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int slot = base + i * NT;
            const int sp = slot >> 10;
            const int v = (slot >> 6) & 15;
            const int ln = slot & 63;
            const int sb = (span0 + sp) * 16 + (ln >> 2);
            g[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (slot < total && sb < S) {
                const int e = sb * 256 + 64 * (ln & 3) + 32 * (v & 1) + 4 * (v >> 1);
                g[i] = *reinterpret_cast<const float4*>(x + e);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int slot = base + i * NT;
            if (slot < total) {
                xs[slot] = make_float4(g[i].x, g[i].z, g[i].y, g[i].w);
            }
        }
    }
}

// ------------------------------------------------ streaming GEMV (m = 1)
// One vector, x held in VGPRs, rows streamed with a register prefetch.
//
// Work split.  A workgroup owns rows_per_block consecutive rows.  A task is
// (span s, group of rows_per_task rows): one wave decodes those rows'
// superblocks 16s .. 16s+15 against the 64 x values of its lane (the span's
// x, read once per task from the LDS stage into VGPRs) and produces one
// partial dot per row.  With one span the partial is y; with several, the
// partials go to LDS and are added in span order after a barrier.
//
// Streaming.  Each wave keeps P rows of its task in flight: row t+P is
// requested before row t is decoded, with branch-free (clamped) addresses so
// the compiler's counter waits let the younger loads stay outstanding.  The
// first P rows are requested before the x stage, so their HBM latency
// overlaps it.
//
// x stage.  x is staged per K-chunk (spans_per_chunk spans, bounded LDS)
// in the lane order of gemv_kernel; every wave copies its span into VGPRs
// right after the stage, so a chunk's LDS is free again once the next
// barrier is passed.
//
// Reduction: one DPP butterfly per row (no LDS traffic); lane 63 holds the
// row total.

struct RowData {
    uint4 h, a, b;    // header, quant bytes 32c..32c+15, 32c+16..32c+31
};

__device__ __forceinline__ RowData load_row(const uint8_t* p, int c)
{
    RowData r;
    r.h = load16(p);
    r.a = load16(p + 16 + 32 * c);
    r.b = load16(p + 32 + 32 * c);
    return r;
}

// v of another lane chosen by DPP (CTRL, row mask RM), for an f64 value:
// the two halves move alike; lanes outside the rows get 0.0
template <int CTRL, int RM>
__device__ __forceinline__ double dpp_f64(double v)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const int lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, RM, 0xF, false);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, RM, 0xF, false);
    return __builtin_bit_cast(double, ((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo);
}

// Sum over the 64 lanes with DPP (quad, half-row, row, row broadcasts), in
// f64; the total lands in lane 63.
__device__ __forceinline__ double dpp_sum_to_lane63(double v)
{
    v += dpp_f64<0xB1, 0xF>(v);     // quad_perm 1,0,3,2
    v += dpp_f64<0x4E, 0xF>(v);     // quad_perm 2,3,0,1
    v += dpp_f64<0x141, 0xF>(v);    // row_half_mirror
    v += dpp_f64<0x140, 0xF>(v);    // row_mirror
    v += dpp_f64<0x142, 0xA>(v);    // row_bcast:15
    v += dpp_f64<0x143, 0xC>(v);    // row_bcast:31
    return v;
}

// Lane constants for the header decode of chunk c (see decode_header).
struct LaneDecode {
    uint32_t sh;     // 16 * (c & 1)
    uint32_t sel;    // all ones for c < 2 (j < 4 form), zero otherwise
};

// One row's partial dot for this lane: the 64 weights of chunk c, exact
// weights times x exactly, in f64 (dot8_exact).
__device__ __forceinline__ double row_partial(const RowData& q, const X4D* xr,
                                              const LaneDecode& ld)
{
    const ChunkScales s = decode_header(q.h, ld.sh, ld.sel);
    double alo = 0.0, ahi = 0.0;
    dot8_exact(q.a.x, xr[0], xr[1], s.sl, s.sh, s.ml, s.mh, alo, ahi);
    dot8_exact(q.a.y, xr[2], xr[3], s.sl, s.sh, s.ml, s.mh, alo, ahi);
    dot8_exact(q.a.z, xr[4], xr[5], s.sl, s.sh, s.ml, s.mh, alo, ahi);
    dot8_exact(q.a.w, xr[6], xr[7], s.sl, s.sh, s.ml, s.mh, alo, ahi);
    dot8_exact(q.b.x, xr[8], xr[9], s.sl, s.sh, s.ml, s.mh, alo, ahi);
    dot8_exact(q.b.y, xr[10], xr[11], s.sl, s.sh, s.ml, s.mh, alo, ahi);
    dot8_exact(q.b.z, xr[12], xr[13], s.sl, s.sh, s.ml, s.mh, alo, ahi);
    dot8_exact(q.b.w, xr[14], xr[15], s.sl, s.sh, s.ml, s.mh, alo, ahi);
    return alo + ahi;
}

template <int NW, int P>
__global__ void __launch_bounds__(NW * 64)
gemv_stream_kernel(const uint8_t* __restrict__ w, const float* __restrict__ x,
                   Out y, int n, int k, int S, int rows_per_block,
                   int rows_per_task, int spans_per_chunk)
{
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);   // wave-uniform
    const int c = lane & 3;
    const int sbl = lane >> 2;
    LaneDecode ld;
    ld.sh = (uint32_t)(c & 1) * 16u;
    ld.sel = c < 2 ? 0xFFFFFFFFu : 0u;

    const int nspans = (S + 15) >> 4;
    const int chunk_spans = spans_per_chunk < nspans ? spans_per_chunk : nspans;
    const int nchunks = (nspans + chunk_spans - 1) / chunk_spans;
    const int row0 = blockIdx.x * rows_per_block;
    const int rows_here = min(rows_per_block, n - row0);
    const int ngroups = (rows_here + rows_per_task - 1) / rows_per_task;
    const size_t row_bytes = (size_t)S * 144;

    float4* xs = reinterpret_cast<float4*>(smem);
    double* ypart = reinterpret_cast<double*>(xs + chunk_spans * 1024);
    const auto early = fetch_y(y, tid < rows_here, row0 + tid, row0 + tid);

    for (int ch = 0; ch < nchunks; ++ch) {
        const int span0 = ch * chunk_spans;
        const int nsp = min(chunk_spans, nspans - span0);
        const int ntasks = nsp * ngroups;

        // the first task's prologue goes out before the stage
        int task = wave;
        RowData buf[P];
        if (task < ntasks) {
            const int span = span0 + task % nsp;
            const int rb = (task / nsp) * rows_per_task;
            const int T = min(rows_per_task, rows_here - rb);
            const int sb = min(span * 16 + sbl, S - 1);        // clamped: in bounds
            const uint8_t* base = w + (size_t)(row0 + rb) * row_bytes + (size_t)sb * 144;
#pragma unroll
            for (int j = 0; j < P; ++j) {
                buf[j] = load_row(base + (size_t)min(j, T - 1) * row_bytes, c);
            }
        }
        if (ch > 0) {
            __syncthreads();          // every wave has copied its x of the previous chunk
        }
        stage_x_batched<NW * 64>(x, S, span0, nsp, xs, tid);
        __syncthreads();

        for (; task < ntasks; task += NW) {
            const int sp = task % nsp;
            const int span = span0 + sp;
            const int rb = (task / nsp) * rows_per_task;
            const int T = min(rows_per_task, rows_here - rb);
            const int sb = min(span * 16 + sbl, S - 1);
            const uint8_t* base = w + (size_t)(row0 + rb) * row_bytes + (size_t)sb * 144;
            if (task != wave) {
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    buf[j] = load_row(base + (size_t)min(j, T - 1) * row_bytes, c);
                }
            }
            // the lane's 64 x of the span, in f64 once per task (128 VGPRs)
            X4D xr[16];
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const float4 t4 = xs[(sp * 16 + v) * 64 + lane];
                xr[v] = X4D{(double)t4.x, (double)t4.y, (double)t4.z, (double)t4.w};
            }
            // y (global) or the per-span row sums (LDS): two typed pointers, so
            // that neither store becomes a flat access, which would make the
            // compiler drain the prefetched loads at every row (with an epilogue
            // there is the second one alone: no y to point at)
            float* yout = direct_y(y) + row0 + rb;
            double* pout = ypart + span * rows_per_block + rb;
            const bool direct = !kEpilogue && nspans == 1;
            int t = 0;
            for (; t + P <= T; t += P) {
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const RowData q = buf[j];
                    buf[j] = load_row(base + (size_t)min(t + j + P, T - 1) * row_bytes, c);
                    const double v = dpp_sum_to_lane63(row_partial(q, xr, ld));
                    if (lane == 63) {
                        if (direct) {
                            yout[t + j] = (float)v;
                        } else {
                            pout[t + j] = v;
                        }
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < P; ++j) {
                if (t + j < T) {
                    const double v = dpp_sum_to_lane63(row_partial(buf[j], xr, ld));
                    if (lane == 63) {
                        if (direct) {
                            yout[t + j] = (float)v;
                        } else {
                            pout[t + j] = v;
                        }
                    }
                }
            }
        }
    }
    if (kEpilogue || nspans > 1) {
        __syncthreads();
        for (int r = tid; r < rows_here; r += NW * 64) {
            double acc = 0.0;
            for (int sp = 0; sp < nspans; ++sp) {
                acc += ypart[sp * rows_per_block + r];
            }
            const auto ops = r == tid ? early : fetch_y(y, true, row0 + r, row0 + r);
            put_y(y, row0 + r, ops, acc);
        }
    }
}

#ifndef Q4K_EPILOGUE
// ------------------------------------------------------------- dequant
// One thread per (superblock, chunk c, dword u): decodes 8 weights and
// writes them as two groups of four (f32, or the fp16 mirror: the f32
// weight rounded to nearest even).  w = fma(d*sc, q, -dmin*m); d*sc and
// dmin*m are exact in f32 and so is d*sc*q, so the fma's single rounding is
// the rounding of the exact value.
template <typename T>
__device__ __forceinline__ void store4(T* o, const float4& v);
template <>
__device__ __forceinline__ void store4<float>(float* o, const float4& v)
{
    *reinterpret_cast<float4*>(o) = v;
}
template <>
__device__ __forceinline__ void store4<_Float16>(_Float16* o, const float4& v)
{
    typedef _Float16 h4_t __attribute__((ext_vector_type(4)));
    const h4_t h = {(_Float16)v.x, (_Float16)v.y, (_Float16)v.z, (_Float16)v.w};
    *reinterpret_cast<h4_t*>(o) = h;
}

template <typename T>
__global__ void __launch_bounds__(256)
dequant_kernel(const uint8_t* __restrict__ w, T* __restrict__ out, int64_t nsb)
{
    const int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t sb = t >> 5;
    if (sb >= nsb) {
        return;
    }
    const int part = (int)(t & 31);
    const int c = part >> 3;
    const int u = part & 7;
    const uint8_t* p = w + sb * 144;
    const uint4 h = load16(p);
    const uint32_t D = *reinterpret_cast<const uint32_t*>(p + 16 + 32 * c + 4 * u);
    const half2_t dd = __builtin_bit_cast(half2_t, h.x);
    const float d = (float)dd.x;
    const float dmin = (float)dd.y;
    const uint32_t sh = (uint32_t)(c & 1) * 16u;
    const uint32_t y = h.y >> sh;
    const uint32_t z = h.z >> sh;
    const uint32_t wv = h.w >> sh;
    const uint32_t sc = c < 2 ? (y & 0x3F3Fu) : ((wv & 0x0F0Fu) | ((y >> 2) & 0x3030u));
    const uint32_t mm = c < 2 ? (z & 0x3F3Fu) : (((wv >> 4) & 0x0F0Fu) | ((z >> 2) & 0x3030u));
    const float dsc_lo = d * (float)(sc & 0xFFu);
    const float dsc_hi = d * (float)((sc >> 8) & 0xFFu);
    const float dm_lo = dmin * (float)(mm & 0xFFu);
    const float dm_hi = dmin * (float)((mm >> 8) & 0xFFu);
    float4 lo, hi;
    lo.x = __builtin_fmaf(dsc_lo, (float)(D & 15u), -dm_lo);
    lo.y = __builtin_fmaf(dsc_lo, (float)((D >> 8) & 15u), -dm_lo);
    lo.z = __builtin_fmaf(dsc_lo, (float)((D >> 16) & 15u), -dm_lo);
    lo.w = __builtin_fmaf(dsc_lo, (float)((D >> 24) & 15u), -dm_lo);
    hi.x = __builtin_fmaf(dsc_hi, (float)((D >> 4) & 15u), -dm_hi);
    hi.y = __builtin_fmaf(dsc_hi, (float)((D >> 12) & 15u), -dm_hi);
    hi.z = __builtin_fmaf(dsc_hi, (float)((D >> 20) & 15u), -dm_hi);
    hi.w = __builtin_fmaf(dsc_hi, (float)(D >> 28), -dm_hi);
    T* o = out + sb * 256 + 64 * c + 4 * u;
    store4<T>(o, lo);
    store4<T>(o + 32, hi);
}

// --------------------------------------------------------- calibration
// Streaming read of n16 16-byte words with the same load width the GEMV
// uses; the xor checksum keeps the loads alive.
// The whole grid sweeps the buffer in address order: pass p, thread t of
// workgroup b reads word p * (grid threads) + b * blockDim + t, one
// non-temporal load per thread and pass, so the loads in flight (about
// 32 KiB per CU) always lie in one window of a few MiB that slides through
// the buffer.  Measured on MI355X for the LM head's 73.7 MB in one launch:
// 11.6 us (6.36 TB/s) this way, against 12.4-13.4 us with one contiguous
// slice per workgroup (the slices' loads spread over the whole buffer at
// any moment) and 11.8-12.0 us with two or more loads in flight per thread.
__global__ void __launch_bounds__(kReadThreads)
read_kernel(const u32x4_t* __restrict__ buf, size_t n16, float* __restrict__ out)
{
    uint32_t acc = 0;
    const size_t step = (size_t)gridDim.x * blockDim.x;
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n16; i += step) {
        const u32x4_t a = __builtin_nontemporal_load(buf + i);
        acc ^= a.x ^ a.y ^ a.z ^ a.w;
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        acc ^= (uint32_t)__shfl_xor((int)acc, off, 64);
    }
    __shared__ uint32_t part[kReadThreads / 64];
    if ((threadIdx.x & 63) == 0) {
        part[threadIdx.x >> 6] = acc;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        uint32_t t = 0;
        for (int i = 0; i < (int)(blockDim.x >> 6); ++i) {
            t ^= part[i];
        }
        out[blockIdx.x] = (float)(t & 0xFFFFu);
    }
}

#endif  // Q4K_EPILOGUE

// -------------------------------------------------------------- launch
template <int M, int R, int NW, bool XREG>
static hipError_t launch_one(const GemvPlan& p, const uint8_t* w, const float* x, Out y,
                             hipStream_t stream)
{
    hipLaunchKernelGGL((gemv_kernel<M, R, NW, XREG>), dim3(p.grid), dim3(NW * 64), p.lds_bytes,
                       stream, w, x, y, p.n, p.k, p.S, p.rows_per_block, p.spans_per_chunk);
    return hipGetLastError();
}

template <int M>
static hipError_t launch_m(const GemvPlan& p, const uint8_t* w, const float* x, Out y,
                           hipStream_t stream)
{
    if constexpr (M == 1) {
        if (p.x_in_registers) {
            if (p.waves_per_block == 8) {
                if (p.rows_per_wave == 4) return launch_one<1, 4, 8, true>(p, w, x, y, stream);
                if (p.rows_per_wave == 2) return launch_one<1, 2, 8, true>(p, w, x, y, stream);
                return launch_one<1, 1, 8, true>(p, w, x, y, stream);
            }
            if (p.rows_per_wave == 4) return launch_one<1, 4, 4, true>(p, w, x, y, stream);
            if (p.rows_per_wave == 2) return launch_one<1, 2, 4, true>(p, w, x, y, stream);
            return launch_one<1, 1, 4, true>(p, w, x, y, stream);
        }
        if (p.waves_per_block == 8) {
            if (p.rows_per_wave == 4) return launch_one<1, 4, 8, false>(p, w, x, y, stream);
            if (p.rows_per_wave == 2) return launch_one<1, 2, 8, false>(p, w, x, y, stream);
            return launch_one<1, 1, 8, false>(p, w, x, y, stream);
        }
        if (p.rows_per_wave == 4) return launch_one<1, 4, 4, false>(p, w, x, y, stream);
        if (p.rows_per_wave == 2) return launch_one<1, 2, 4, false>(p, w, x, y, stream);
        return launch_one<1, 1, 4, false>(p, w, x, y, stream);
    } else {
        if (p.waves_per_block == 8) {
            if (p.rows_per_wave == 2) return launch_one<M, 2, 8, false>(p, w, x, y, stream);
            return launch_one<M, 1, 8, false>(p, w, x, y, stream);
        }
        if (p.rows_per_wave == 2) return launch_one<M, 2, 4, false>(p, w, x, y, stream);
        return launch_one<M, 1, 4, false>(p, w, x, y, stream);
    }
}

template <int NW, int P>
static hipError_t launch_stream(const GemvPlan& p, const uint8_t* w, const float* x, Out y,
                                hipStream_t stream)
{
    hipLaunchKernelGGL((gemv_stream_kernel<NW, P>), dim3(p.grid), dim3(NW * 64), p.lds_bytes,
                       stream, w, x, y, p.n, p.k, p.S, p.rows_per_block, p.rows_per_task,
                       p.spans_per_chunk);
    return hipGetLastError();
}

template <int NW>
static hipError_t launch_stream_nw(const GemvPlan& p, const uint8_t* w, const float* x, Out y,
                                   hipStream_t stream)
{
    if (p.ring_depth == 1) return launch_stream<NW, 1>(p, w, x, y, stream);
    if (p.ring_depth == 2) return launch_stream<NW, 2>(p, w, x, y, stream);
    if (p.ring_depth == 3) return launch_stream<NW, 3>(p, w, x, y, stream);
    return launch_stream<NW, 4>(p, w, x, y, stream);
}

hipError_t launch_gemv(const GemvPlan& p, const void* w, const float* x, Out y,
                       hipStream_t stream)
{
    const uint8_t* wb = static_cast<const uint8_t*>(w);
    if (p.kernel == 3) {
        return launch_gemv_dot4(p, w, x, y, stream);
    }
    if (p.kernel >= 4) {
        return launch_gemv_mfma(p, w, x, y, stream);
    }
    if (p.kernel == 2) {
        if (p.waves_per_block == 8) return launch_stream_nw<8>(p, wb, x, y, stream);
        return launch_stream_nw<4>(p, wb, x, y, stream);
    }
    switch (p.m) {
    case 1: return launch_m<1>(p, wb, x, y, stream);
    case 2: return launch_m<2>(p, wb, x, y, stream);
    case 3: return launch_m<3>(p, wb, x, y, stream);
    case 4: return launch_m<4>(p, wb, x, y, stream);
    case 5: return launch_m<5>(p, wb, x, y, stream);
    case 6: return launch_m<6>(p, wb, x, y, stream);
    case 7: return launch_m<7>(p, wb, x, y, stream);
    case 8: return launch_m<8>(p, wb, x, y, stream);
    default: return hipErrorInvalidValue;
    }
}

#ifndef Q4K_EPILOGUE
hipError_t launch_dequant(const void* w, float* out, int64_t nsb, hipStream_t stream)
{
    const int64_t threads = nsb * 32;
    const int64_t blocks = (threads + 255) / 256;
    hipLaunchKernelGGL(dequant_kernel<float>, dim3((unsigned)blocks), dim3(256), 0, stream,
                       static_cast<const uint8_t*>(w), out, nsb);
    return hipGetLastError();
}

hipError_t launch_dequant_f16(const void* w, void* out, int64_t nsb, hipStream_t stream)
{
    const int64_t threads = nsb * 32;
    const int64_t blocks = (threads + 255) / 256;
    hipLaunchKernelGGL(dequant_kernel<_Float16>, dim3((unsigned)blocks), dim3(256), 0, stream,
                       static_cast<const uint8_t*>(w), static_cast<_Float16*>(out), nsb);
    return hipGetLastError();
}

hipError_t launch_read(const void* buf, size_t n16, float* out, hipStream_t stream)
{
    hipLaunchKernelGGL(read_kernel, dim3(kReadBlocks), dim3(kReadThreads), 0, stream,
                       static_cast<const u32x4_t*>(buf), n16, out);
    return hipGetLastError();
}
#endif  // Q4K_EPILOGUE

}  // namespace q4k
