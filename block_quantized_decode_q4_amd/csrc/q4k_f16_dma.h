// q4k_f16_dma.h -- a tile of y = act(x W^T + bias) gate + residual on fp16 mirrors,
// its operands loaded straight into LDS.  Internal.
//
// Four waves, a ring of S stages of GK halves of k for both operands.  The loads go from
// memory to LDS without registers on their way (which leaves them to the sums: 112 or
// 128 of a lane's), S - 1 stages ahead, and are waited for by count; a barrier per stage.
// Between the products of one 32 of k stand the LDS reads of the next, and in a stage's
// last phase the loads that refill its place.  Pieces of 16 bytes are turned by their
// row, so that reads have no conflicts (0.02 of the LDS's active cycles).
// Against the same products with operands through registers (512 threads, two stages):
// 2048 x 14336 x 4096 gated 373 -> 237 us, eight experts of 2048 tokens 849 -> 554,
// 509 x 4096 x 14336 141 -> 97.
// Tried without gain: stages of 32 of k, two workgroups a CU on 128 x 128 tiles, all loads
// of a stage at its start, waves that load one operand each (97.5 us for 94 on the last).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "q4k_device.h"
#include "q4k_epilogue.h"
#include "q4k_f16_tile.h"

namespace q4k {

// a row of any n begins on any element
typedef float f32x4u_t __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x4h_t __attribute__((ext_vector_type(4), aligned(2)));
typedef _Float16 half8u_t __attribute__((ext_vector_type(8), aligned(2)));

// 16 bytes from each lane's base + `from` (bytes) into LDS at `to` (bytes, the same
// for the wave) plus 16 times the lane.  The wave waits for it with dma_wait alone:
// the compiler does not know of it.  (M0 is reserved: the compiler sets it before each
// use of its own and keeps nothing there, and in these kernels has no use.)
// The compiler also does not count the wait states that such instructions need behind a
// vector write: five for the base's scalar registers here (they come from scalar
// additions), two for a product's operands below (they come from LDS reads).
// tests/inline_waits.py looks for each of these in the code as it was built.
__device__ __forceinline__ void dma16(uint32_t to, uint32_t from, const void* base)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(to), "v"(from), "s"(base)
                 : "memory");
}

// All but the last LEFT loads of this wave have landed and its LDS reads are done
template <int LEFT>
__device__ __forceinline__ void dma_wait()
{
    static_assert(LEFT < 64, "the counter's width");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"(LEFT) : "memory");
}

// acc += a b in place.  (Of the builtin, the compiler makes an instruction with other
// registers for the result, and moves 200-600 registers in every step.)  It does not
// know of the instruction: mfma_wait and mfma_done stand between the last of them and
// the first use of a sum.
__device__ __forceinline__ void mfma_onto(f32x4_t& acc, const half8_t& a, const half8_t& b)
{
    asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}

// A result can be read 18 wait states after its instruction at the latest; each sum
// goes through mfma_done after the wait, so that no read of it is moved before
__device__ __forceinline__ void mfma_wait()
{
    asm volatile("s_nop 15\n\ts_nop 15" : : : "memory");
}

__device__ __forceinline__ void mfma_done(f32x4_t& acc)
{
    asm volatile("" : "+a"(acc));
}

template <int I, int N, typename F>
__device__ __forceinline__ void unrolled(F f)
{
    if constexpr (I < N) {
        f(std::integral_constant<int, I>());
        unrolled<I + 1, N>(f);
    }
}

// WM x WN x KW waves (four); each has FA x FB blocks of 16 x rows by 16 columns,
// the KW waves of one place every KW-th 32 of k.  S stages of GK halves of k.
template <int WM_, int WN_, int KW_, int FA_, int FB_, int GK_, int S_>
struct DmaShape {
    static constexpr int WM = WM_, WN = WN_, KW = KW_, FA = FA_, FB = FB_, GK = GK_, S = S_;
    static constexpr int BM = 16 * FA * WM;
    static constexpr int BN = 16 * FB * WN;
    static constexpr int kThreads = 64 * WM * WN * KW;
    static constexpr int kStage = (BM + BN) * GK * 2;
    static constexpr int kPitch = BN / WN * 4 + 16;      // LDS bytes of an epilogue row
    static constexpr int kLds = S * kStage;
    static constexpr int kPart = kLds / 4 / 16 * 16;     // a wave's part of it
    static_assert(WM * WN * KW == 4, "four waves");
    static_assert(kLds <= 160 * 1024, "LDS");
    static_assert(FA / KW * 16 * kPitch <= kPart, "the rows that a wave writes out");
};

// ---------------------------------------------------------------- the epilogue
// A wave's sums, NA x FB blocks (lane 16 g + j of a block: x row j, columns 4 g ..
// 4 g + 3), go out by rows: through its part of the LDS, so that neighbouring lanes hold
// neighbouring columns, eight each.  The gate
// and residual of the next 16 rows are on their way while 16 rows are computed: a row
// that is not written reads another's.  Columns that pass n go out one by one.
struct Eight {
    f32x4_t lo, hi;
};

__device__ __forceinline__ Eight eight_at(const float* p)
{
    return {*reinterpret_cast<const f32x4u_t*>(p), *reinterpret_cast<const f32x4u_t*>(p + 4)};
}

__device__ __forceinline__ Eight eight_of(const half8_t& h)
{
    return {f32x4_t{(float)h[0], (float)h[1], (float)h[2], (float)h[3]},
            f32x4_t{(float)h[4], (float)h[5], (float)h[6], (float)h[7]}};
}

template <int ACT, int N>
__device__ __forceinline__ void activate(Eight (&v)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[i].lo[e] = activated<ACT>(v[i].lo[e]);
            v[i].hi[e] = activated<ACT>(v[i].hi[e]);
        }
    }
}

// GATED: a binary16 gate and no residual (a prompt's gated block), whose loads take
// few registers: kDepth blocks of rows on their way; else whatever the epilogue has.
// (One kernel for each: with both in one the sums did not stay in registers.)  The
// other's rows on their way pass through scratch memory (48 or 112 bytes a lane), used
// or not: 2048 x 14336 x 4096 takes 225 us with a binary16 gate, 265 with a residual, 301
// with an f32 gate, 316 with a binary16 gate and a residual.
template <typename T, int NA, bool GATED, typename YRow>
__device__ __forceinline__ void dma_epilogue(const f32x4_t (&acc)[NA][T::FB], int xrow0, int col0,
                                         YRow yrow, const EpArgs& ep, const float* bias, int n,
                                         unsigned char* part)
{
    constexpr int kLanes = 2 * T::FB;                    // lanes per row
    constexpr int kAt = kLanes <= 8 ? 8 : 4;             // rows at a time
    constexpr int IT = 16 / kAt;
    static_assert(kAt * kLanes <= 64, "a wave's lanes");
    const int lane = threadIdx.x & 63;
    const int g = lane >> 4;
    const int j = lane & 15;
    const int lr = min(lane / kLanes, kAt - 1);          // lanes too many repeat the last row
    const int lc = lane % kLanes * 8;
    const bool mine = lane / kLanes < kAt;
    const bool inside = col0 + 16 * T::FB <= n;          // the same for the wave
    const int col = col0 + lc;
    constexpr int kDepth = GATED ? 3 : 1;
    const bool half = GATED || ep.gate_type == kTypeF16;
    struct Rows {
        Eight gate[IT];                                  // eight binary16 numbers in gate.lo
        Eight res[GATED ? 1 : IT];
    };
    auto fetch = [&](int blk, Rows& r) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int row = yrow(xrow0 + 16 * blk + kAt * i + lr);
            const int64_t at = (int64_t)max(row, 0) * n + col;
            if (GATED || (ep.gate != nullptr && half)) {
                r.gate[i].lo = *reinterpret_cast<const f32x4h_t*>(
                    static_cast<const _Float16*>(ep.gate) + at);
            } else if (ep.gate != nullptr) {
                r.gate[i] = eight_at(static_cast<const float*>(ep.gate) + at);
            }
            if constexpr (!GATED) {
                if (ep.residual != nullptr) {
                    r.res[i] = eight_at(ep.residual + at);
                }
            }
        }
    };
    Eight add = {};
    Rows way[kDepth] = {};
    if (inside) {
        if (bias != nullptr) {
            add = eight_at(bias + col);
        }
#pragma unroll
        for (int q = 0; q < kDepth; ++q) {
            fetch(min(q, NA - 1), way[q]);
        }
    }
#pragma unroll
    for (int a = 0; a < NA; ++a) {
#pragma unroll
        for (int b = 0; b < T::FB; ++b) {
            *reinterpret_cast<f32x4_t*>(part + (a * 16 + j) * T::kPitch + (16 * b + 4 * g) * 4) =
                acc[a][b];
        }
    }
    wave_lds_order();                                    // other lanes read what a lane wrote
#pragma unroll 1
    for (int blk = 0; blk < NA; ++blk) {
        const unsigned char* const rows = part + blk * 16 * T::kPitch;
        if (!inside) {
            // element by element: lane l takes every 64th
            for (int at = lane; at < 16 * 16 * T::FB; at += 64) {
                const int c = at % (16 * T::FB);
                const int row = yrow(xrow0 + 16 * blk + at / (16 * T::FB));
                if (row >= 0 && col0 + c < n) {
                    const float v = *reinterpret_cast<const float*>(
                        rows + at / (16 * T::FB) * T::kPitch + 4 * c);
                    const int64_t to = (int64_t)row * n + col0 + c;
                    const EpOperands o = ep_fetch(ep, to, 0);     // its bias is not used
                    const float z = v + (bias != nullptr ? bias[col0 + c] : 0.f);
                    ep_store(ep, to, ep_value(ep, o, z));
                }
            }
            continue;
        }
        const Rows r = way[0];
#pragma unroll
        for (int q = 0; q + 1 < kDepth; ++q) {
            way[q] = way[q + 1];
        }
        fetch(min(blk + kDepth, NA - 1), way[kDepth - 1]);
        Eight v[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const unsigned char* const from = rows + (kAt * i + lr) * T::kPitch + lc * 4;
            v[i].lo = *reinterpret_cast<const f32x4_t*>(from) + add.lo;
            v[i].hi = *reinterpret_cast<const f32x4_t*>(from + 16) + add.hi;
        }
        switch (ep.act) {                                // the same for the whole launch
        case kActRelu: activate<kActRelu>(v); break;
        case kActSilu: activate<kActSilu>(v); break;
        case kActGelu: activate<kActGelu>(v); break;
        case kActGeluTanh: activate<kActGeluTanh>(v); break;
        case kActSigmoid: activate<kActSigmoid>(v); break;
        default: break;
        }
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            if (GATED || ep.gate != nullptr) {
                const Eight f = half ? eight_of(__builtin_bit_cast(half8_t, r.gate[i].lo))
                                     : r.gate[i];
                v[i].lo *= f.lo;
                v[i].hi *= f.hi;
            }
            if constexpr (!GATED) {
                if (ep.residual != nullptr) {
                    v[i].lo += r.res[i].lo;
                    v[i].hi += r.res[i].hi;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int row = yrow(xrow0 + 16 * blk + kAt * i + lr);
            if (mine && row >= 0) {
                const int64_t at = (int64_t)row * n + col;
                if (ep.y != nullptr) {
                    *reinterpret_cast<f32x4u_t*>(ep.y + at) = v[i].lo;
                    *reinterpret_cast<f32x4u_t*>(ep.y + at + 4) = v[i].hi;
                }
                if (ep.y16 != nullptr) {
                    *reinterpret_cast<half8u_t*>(static_cast<_Float16*>(ep.y16) + at) = half8u_t{
                        (_Float16)v[i].lo[0], (_Float16)v[i].lo[1], (_Float16)v[i].lo[2],
                        (_Float16)v[i].lo[3], (_Float16)v[i].hi[0], (_Float16)v[i].hi[1],
                        (_Float16)v[i].hi[2], (_Float16)v[i].hi[3]};
                }
            }
        }
    }
}

// Piece c (16 bytes) of an operand's row r lies at place c ^ dma_turn(r) of its LDS
// row, so that the reads of 16 rows' pieces do not meet in a bank
template <int GK>
__device__ __forceinline__ int dma_turn(int row)
{
    static_assert(GK == 64 || GK == 128, "the stages' depth");
    return GK == 64 ? row & 7 : row & 15;
}

// xoff(i): where the tile's x row i (i < BM) begins, in bytes behind x; yrow(i): its y row, -1 where
// it is not written; w: the mirror's first row; columns col0 .. of n; bias: of the
// mirror's first row (may be null).
template <typename T, bool GATED, typename XOff, typename YRow>
__device__ __forceinline__ void f16_dma_tile(const _Float16* __restrict__ w,
                                             const _Float16* __restrict__ x, XOff xoff, YRow yrow,
                                             const EpArgs& ep, const float* bias, int col0, int n,
                                             int k, unsigned char* smem)
{
    constexpr int kPieces = T::GK / 8;                   // 16-byte pieces of a row
    constexpr int kRows = T::kThreads / kPieces;         // rows per load of all threads
    constexpr int LA = T::BM / kRows;
    constexpr int LB = T::BN / kRows;
    constexpr int L = LA + LB;
    constexpr int FA = T::FA, FB = T::FB, S = T::S;
    constexpr int kSub = T::GK / 32 / T::KW;             // 32s of k per wave and stage
    static_assert(T::BM % kRows == 0 && T::BN % kRows == 0, "whole loads");
    static_assert(kSub == 1 || kSub == 2, "phases of a stage");
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % T::WM;
    const int wn = wave / T::WM % T::WN;
    const int wk = wave / (T::WM * T::WN);
    const int g = lane >> 4;
    const int j = lane & 15;
    const uint32_t lds0 =
        (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)smem;

    // load role: a row's piece c lies at place c ^ row of its LDS row
    const int lrow = tid / kPieces;
    const int lpiece = (tid % kPieces) ^ dma_turn<T::GK>(lrow);
    uint32_t src[L];
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        src[i] = xoff(lrow + kRows * i) + lpiece * 16;
    }
    const _Float16* const wtile = w + (int64_t)col0 * k;
#pragma unroll
    for (int i = 0; i < LB; ++i) {
        src[LA + i] = (uint32_t)min(lrow + kRows * i, n - 1 - col0) * (uint32_t)(2 * k) +
                      lpiece * 16;
    }
    const uint32_t to0 = lds0 + wave * 1024;
    // load i of stage kb into place st
    auto load = [&](int kb, int st, auto ic) __attribute__((always_inline)) {
        constexpr int i = decltype(ic)::value;
        dma16(to0 + st * T::kStage + i * (T::kThreads * 16), src[i],
              (i < LA ? x : wtile) + (int64_t)kb * T::GK);
    };
    const unsigned char* const xs = smem + ((16 * FA) * wm + j) * (2 * T::GK);
    const unsigned char* const ws =
        smem + T::BM * (2 * T::GK) + ((16 * FB) * wn + j) * (2 * T::GK);

    f32x4_t acc[FA][FB];
#pragma unroll
    for (int a = 0; a < FA; ++a) {
#pragma unroll
        for (int b = 0; b < FB; ++b) {
            acc[a][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
    }
    half8_t av[2][FA], bv[2][FB];
    // operand r of set q from 32s `sub` of stage st
    auto read = [&](int st, int sub, auto qc, auto rc) __attribute__((always_inline)) {
        constexpr int q = decltype(qc)::value;
        constexpr int r = decltype(rc)::value;
        const int c = ((4 * (sub * T::KW + wk) + g) ^ dma_turn<T::GK>(j)) << 4;
        if constexpr (r < FB) {
            bv[q][r] =
                *reinterpret_cast<const half8_t*>(ws + st * T::kStage + r * (32 * T::GK) + c);
        } else {
            av[q][r - FB] = *reinterpret_cast<const half8_t*>(xs + st * T::kStage +
                                                              (r - FB) * (32 * T::GK) + c);
        }
    };
    // the products of set q, and between them the reads of the other set from 32s
    // `sub` of place st and, with FILL, the loads of stage kb into place `to`
    auto phase = [&](auto qc, int st, int sub, auto fill, int kb, int to)
                     __attribute__((always_inline)) {
        constexpr int q = decltype(qc)::value;
        constexpr int R = FA + FB;
        unrolled<0, R>([&](auto rc) __attribute__((always_inline)) {
            constexpr int r = decltype(rc)::value;
            read(st, sub, std::integral_constant<int, 1 - q>(), rc);
            if constexpr (decltype(fill)::value) {
                unrolled<r * L / R, (r + 1) * L / R>(
                    [&](auto ic) __attribute__((always_inline)) { load(kb, to, ic); });
            }
            constexpr int from = r * (FA * FB) / R, upto = (r + 1) * (FA * FB) / R;
            unrolled<from, upto>([&](auto ic) __attribute__((always_inline)) {
                constexpr int a = decltype(ic)::value / FB, b = decltype(ic)::value % FB;
                mfma_onto(acc[a][b], bv[q][b], av[q][a]);
            });
            __builtin_amdgcn_sched_barrier(0);
        });
    };

    const int KB = k / T::GK;
#pragma unroll
    for (int t = 0; t < S; ++t) {
        unrolled<0, L>(
            [&](auto ic) __attribute__((always_inline)) { load(min(t, KB - 1), t, ic); });
    }
    // Every wave's loads but those of LEFT later stages have landed, and it has read
    // the operands that it asked for.
    auto meet = [&](auto left) __attribute__((always_inline)) {
        dma_wait<decltype(left)::value * L>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" : : : "memory");
    };
    using std::integral_constant;
    const integral_constant<int, 0> first;
    const integral_constant<int, 1> other;
    const integral_constant<bool, true> fill;
    const integral_constant<bool, false> rest;
    meet(integral_constant<int, S - 1>());
    unrolled<0, FA + FB>(
        [&](auto rc) __attribute__((always_inline)) { read(0, 0, first, rc); });
    // Stage kb in place st.  Its last phase begins when every wave has read its
    // operands and the next stage has landed: its place is then filled with stage kb +
    // S.  One loop without branches, in which beyond the last stage that one is loaded
    // again and not used: a loop of its own for the end made the compiler move all
    // registers in every step.
    int st = 0;
    auto one = [&](int kb, auto qc) __attribute__((always_inline)) {
        constexpr int q = decltype(qc)::value;
        const int after = st + 1 == S ? 0 : st + 1;
        if constexpr (kSub == 2) {
            phase(qc, st, 1, rest, 0, 0);
        }
        meet(integral_constant<int, S - 2>());
        phase(integral_constant<int, kSub == 2 ? 1 - q : q>(), after, 0, fill,
              min(kb + S, KB - 1), st);
        st = after;
    };
    if constexpr (kSub == 2) {
        for (int kb = 0; kb < KB; ++kb) {
            one(kb, first);
        }
    } else {
        int kb = 0;
        do {                                             // KB is even
            one(kb, first);
            one(kb + 1, other);
            kb += 2;
        } while (kb < KB);
    }
    // every wave is done with the operands, no load is on its way
    mfma_wait();
#pragma unroll
    for (int a = 0; a < FA; ++a) {
#pragma unroll
        for (int b = 0; b < FB; ++b) {
            mfma_done(acc[a][b]);
        }
    }
    dma_wait<0>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" : : : "memory");

    if constexpr (T::KW > 1) {
        // the sums of the waves along k meet: each adds up a share of the rows, in the
        // waves' order
        constexpr int kWaveBytes = FA * FB * 1024;
        constexpr int kShare = FA * FB / T::KW;          // blocks that a wave adds up
        static_assert(T::WM * T::WN == 1 && FA % T::KW == 0, "whole rows of blocks");
        static_assert(T::KW * kWaveBytes <= T::kLds, "the sums fit");
        unsigned char* const mine = smem + wk * kWaveBytes + lane * 16;
#pragma unroll
        for (int a = 0; a < FA; ++a) {
#pragma unroll
            for (int b = 0; b < FB; ++b) {
                *reinterpret_cast<f32x4_t*>(mine + (a * FB + b) * 1024) = acc[a][b];
            }
        }
        __syncthreads();
        f32x4_t sum[FA / T::KW][FB];
#pragma unroll
        for (int i = 0; i < kShare; ++i) {
            const unsigned char* const at = smem + (wk * kShare + i) * 1024 + lane * 16;
            f32x4_t s = *reinterpret_cast<const f32x4_t*>(at);
#pragma unroll
            for (int z = 1; z < T::KW; ++z) {
                s += *reinterpret_cast<const f32x4_t*>(at + z * kWaveBytes);
            }
            sum[i / FB][i % FB] = s;
        }
        __syncthreads();
        dma_epilogue<T, FA / T::KW, GATED>(sum, (FA / T::KW) * wk * 16, col0, yrow, ep, bias, n,
                                    smem + wave * T::kPart);
    } else {
        dma_epilogue<T, FA, GATED>(acc, 16 * FA * wm, col0 + 16 * FB * wn, yrow, ep, bias, n,
                            smem + wave * T::kPart);
    }
}

}  // namespace q4k
