// q4k_norm.hip -- the root-mean-square norm in front of the projections, with
// the residual's addition and, for the int8 products, its output in Q8.
//
//   h = x + residual                    (f32, one rounding; h = x without one)
//   y = h * w / sqrt(sum h^2 / k + eps)
//
// The squares are summed, and y's two products formed, in f64: no square of a
// finite h overflows or vanishes, and y is within a rounding of the exact
// value (the kernel is bound by memory; the f64 work hides behind it).  y
// goes out as f32, as binary16, as Q8 codes with a scale per 32 elements
// (q4k_q8.h, the rule of q4k_quantize_q8 applied to the f32 y), or as any of
// them together.
//
// One workgroup per row.  A thread holds groups of eight consecutive
// elements: a row of up to P * 8 * threads elements is read once and stays in
// registers between the sum and the output.  Longer rows are read again (h
// from sum_out where it is kept, else x and the residual once more).  Four
// neighbouring lanes hold one Q8 block, so its largest |y| takes two lane
// exchanges.
//
// What bounds it: the bytes.  8192 rows of 4096, binary16 in, residual in and out,
// binary16 out (402 MB): 73 us, 5.5 TB/s (a large copy on this card: 4.9).  One
// row of 4096: 3.3 us, the latency of a load, the row's sum and a store.
//
// The norms on both sides of a block, and layer norms, are further down.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4k_device.h"
#include "q4k_kernels.h"
#include "q4k_q8.h"

namespace q4k {

namespace {

// Rows of any length begin on any element: the vector accesses ask for an
// element's alignment only (they cost the same; element by element, eight
// consecutive ones to a lane, a row of 8189 took four times as long).
typedef float f4u_t __attribute__((ext_vector_type(4), aligned(4)));
typedef uint16_t u16x8_t __attribute__((ext_vector_type(8), aligned(2)));
typedef _Float16 h8u_t __attribute__((ext_vector_type(8), aligned(2)));

template <int TYPE>
__device__ __forceinline__ float element(const void* base, int64_t at)
{
    if constexpr (TYPE == kTypeF32) {
        return static_cast<const float*>(base)[at];
    } else {
        const uint16_t b = static_cast<const uint16_t*>(base)[at];
        return TYPE == kTypeF16 ? (float)__builtin_bit_cast(_Float16, b)
                                : __builtin_bit_cast(float, (uint32_t)b << 16);
    }
}

// Eight elements of base from `at` on
template <int TYPE>
__device__ __forceinline__ void load8(const void* base, int64_t at, float* e)
{
    if constexpr (TYPE == kTypeF32) {
        const float* p = static_cast<const float*>(base) + at;
        const f4u_t a = *reinterpret_cast<const f4u_t*>(p);
        const f4u_t b = *reinterpret_cast<const f4u_t*>(p + 4);
        e[0] = a.x; e[1] = a.y; e[2] = a.z; e[3] = a.w;
        e[4] = b.x; e[5] = b.y; e[6] = b.z; e[7] = b.w;
    } else {
        const u16x8_t v =
            *reinterpret_cast<const u16x8_t*>(static_cast<const uint16_t*>(base) + at);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint16_t b = v[i];
            e[i] = TYPE == kTypeF16 ? (float)__builtin_bit_cast(_Float16, b)
                                    : __builtin_bit_cast(float, (uint32_t)b << 16);
        }
    }
}

__device__ __forceinline__ void store8(float* p, const float* e)
{
    *reinterpret_cast<f4u_t*>(p) = f4u_t{e[0], e[1], e[2], e[3]};
    *reinterpret_cast<f4u_t*>(p + 4) = f4u_t{e[4], e[5], e[6], e[7]};
}

// Where the group at column c is read: TAIL (k is no multiple of eight), a last
// group that is not whole reads the row's last eight elements and is then read
// again element by element.
template <bool TAIL>
__device__ __forceinline__ int read_at(const NormArgs& a, int c)
{
    return TAIL ? min(c, a.k - 8) : c;
}

// h of the group at column c: x + residual (rounded once), or x; zeros beyond
// the row
template <int TYPE, bool TAIL>
__device__ __forceinline__ void load_h(const NormArgs& a, int64_t row, int c, float* h)
{
    if (!TAIL || a.k >= 8) {
        load8<TYPE>(a.x, row * a.x_stride + read_at<TAIL>(a, c), h);
        if (a.residual != nullptr) {
            float r[8];
            load8<kTypeF32>(a.residual, row * a.k + read_at<TAIL>(a, c), r);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[i] += r[i];
            }
        }
    }
    if (TAIL && a.k - c < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            h[i] = 0.f;
            if (c + i < a.k) {
                h[i] = element<TYPE>(a.x, row * a.x_stride + c + i);
                h[i] += a.residual != nullptr ? a.residual[row * a.k + c + i] : 0.f;
            }
        }
    }
}

template <bool TAIL>
__device__ __forceinline__ void put_f32(const NormArgs& a, float* base, int64_t row, int c,
                                        const float* e)
{
    float* const p = base + row * a.k + c;
    if (!TAIL || a.k - c >= 8) {
        store8(p, e);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (c + i < a.k) {
                p[i] = e[i];
            }
        }
    }
}

// Eight f32 of base from `from` + c on (c the group's column); zeros beyond the row
template <bool TAIL>
__device__ __forceinline__ void load_f32(const NormArgs& a, const float* base, int64_t from, int c,
                                         float* e)
{
    if (!TAIL || a.k >= 8) {
        load8<kTypeF32>(base, from + read_at<TAIL>(a, c), e);
    }
    if (TAIL && a.k - c < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            e[i] = c + i < a.k ? base[from + c + i] : 0.f;
        }
    }
}

// The outputs of one group from its y
template <bool TAIL>
__device__ __forceinline__ void put_outputs(const NormArgs& a, int64_t row, int c, const float* y)
{
    const int64_t at = row * a.k + c;
    if (a.y != nullptr) {
        put_f32<TAIL>(a, a.y, row, c, y);
    }
    if (a.y16 != nullptr) {
        h8u_t v;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = (_Float16)y[i];
        }
        _Float16* p = static_cast<_Float16*>(a.y16) + at;
        if (!TAIL || a.k - c >= 8) {
            *reinterpret_cast<h8u_t*>(p) = v;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (c + i < a.k) {
                    p[i] = v[i];
                }
            }
        }
    }
    if constexpr (!TAIL) {
        if (a.q != nullptr) {              // k % 32 == 0: four whole groups per block
            float amax = 0.f;
            int nan = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                amax = fmaxf(amax, fabsf(y[i]));
                nan |= y[i] != y[i];
            }
#pragma unroll
            for (int off = 1; off < 4; off <<= 1) {
                amax = fmaxf(amax, __shfl_xor(amax, off, 64));
                nan |= __shfl_xor(nan, off, 64);
            }
            const Q8Scale s = q8_scale(amax, nan != 0);
            uint2 v;
            v.x = q8_pack(q8_code(y[0], s.inv), q8_code(y[1], s.inv), q8_code(y[2], s.inv),
                          q8_code(y[3], s.inv));
            v.y = q8_pack(q8_code(y[4], s.inv), q8_code(y[5], s.inv), q8_code(y[6], s.inv),
                          q8_code(y[7], s.inv));
            *reinterpret_cast<uint2*>(a.q + at) = v;
            if ((c & 31) == 0) {
                a.d[at / 32] = s.d;
            }
        }
    }
}

// The outputs of one group from its h (and the row's factor r)
template <bool TAIL>
__device__ __forceinline__ void put_y(const NormArgs& a, int64_t row, int c, const float* h,
                                      double r)
{
    float w[8], y[8];
    load_f32<TAIL>(a, a.weight, 0, c, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[i] = (float)((double)h[i] * r * (double)w[i]);
    }
    put_outputs<TAIL>(a, row, c, y);
}

// P: groups of eight elements that a thread keeps in registers; the groups
// beyond P * threads are read twice.
template <int TYPE, int P, bool TAIL>
__global__ void __launch_bounds__(1024)
rmsnorm_kernel(NormArgs a)
{
    __shared__ double part[16];
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x;
    const int threads = blockDim.x;
    const int groups = (a.k - 1) / 8 + 1;
    float h[P][8];
    double sum = 0.0;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int gi = p * threads + tid;
        if (gi < groups) {
            load_h<TYPE, TAIL>(a, row, gi * 8, h[p]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[p][i] = 0.f;
            }
        }
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int gi = p * threads + tid;
        if (a.sum != nullptr && gi < groups) {
            put_f32<TAIL>(a, a.sum, row, gi * 8, h[p]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sum = __builtin_fma((double)h[p][i], (double)h[p][i], sum);
        }
    }
    for (int gi = P * threads + tid; gi < groups; gi += threads) {
        float t[8];
        load_h<TYPE, TAIL>(a, row, gi * 8, t);
        if (a.sum != nullptr) {
            put_f32<TAIL>(a, a.sum, row, gi * 8, t);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sum = __builtin_fma((double)t[i], (double)t[i], sum);
        }
    }
    sum = wave_sum(sum);
    const int waves = threads >> 6;
    if (waves > 1) {
        if ((tid & 63) == 0) {
            part[tid >> 6] = sum;
        }
        __syncthreads();
        sum = part[0];
        for (int i = 1; i < waves; ++i) {      // in wave order, the same in every thread
            sum += part[i];
        }
    }
    const double r = 1.0 / __builtin_sqrt(sum / (double)a.k + (double)a.eps);
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int gi = p * threads + tid;
        if (gi < groups) {
            put_y<TAIL>(a, row, gi * 8, h[p], r);
        }
    }
    for (int gi = P * threads + tid; gi < groups; gi += threads) {
        float t[8];
        if (a.sum != nullptr && (!TAIL || a.k - gi * 8 >= 8)) {
            load8<kTypeF32>(a.sum, row * a.k + gi * 8, t);       // this thread's own stores
        } else if (a.sum != nullptr) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                t[i] = gi * 8 + i < a.k ? a.sum[row * a.k + gi * 8 + i] : 0.f;
            }
        } else {
            load_h<TYPE, TAIL>(a, row, gi * 8, t);
        }
        put_y<TAIL>(a, row, gi * 8, t, r);
    }
}

template <int TYPE, int P>
hipError_t launch_p(const NormArgs& a, int threads, hipStream_t stream)
{
    const dim3 grid((unsigned)a.m), block(threads);
    if (a.k % 8 != 0) {
        hipLaunchKernelGGL((rmsnorm_kernel<TYPE, P, true>), grid, block, 0, stream, a);
    } else {
        hipLaunchKernelGGL((rmsnorm_kernel<TYPE, P, false>), grid, block, 0, stream, a);
    }
    return hipGetLastError();
}

template <int TYPE>
hipError_t launch_t(const NormArgs& a, hipStream_t stream)
{
    const int groups = (a.k - 1) / 8 + 1;
    // One group per thread where a workgroup holds the row (8192 rows of 4096,
    // binary16 in and out, with the residual: 73 us, against 78 with two and 87
    // with four groups per thread; 64 rows 6.6 / 6.9 / 6.7 us).  Longer rows, four
    // per thread: the fewest threads that hold the row where the rows fill the
    // chip (1024 rows of 14336: 29 us against 33 with 1024 threads), all 1024
    // where they do not (256 rows 9.3 us against 9.9).
    if (groups <= 1024) {
        return launch_p<TYPE, 1>(a, (groups + 63) / 64 * 64, stream);
    }
    const int threads = a.m < 1024 ? 1024 : ((groups + 3) / 4 + 63) / 64 * 64;
    return launch_p<TYPE, 4>(a, threads < 1024 ? threads : 1024, stream);
}

// ------------------------------------------------ norms on both sides of a block
//   p = N(x; post_weight, post_bias)      (x itself without post_weight)
//   h = residual + scale gate p           (f32, one rounding)
//   y = N(h; weight, bias)
// N divides by sqrt(mean v^2 + eps), the layer norm after taking the mean off
// (its squares are summed in a second step: a row far from zero loses nothing).
// The same split as above: a workgroup per row, groups of eight elements in registers
// from the loads to the outputs.  The sums are f64; the elements are f32, a power of
// two s = about 1 / sqrt(..) taken out first, so that nothing overflows or vanishes:
//   N = ((v s - mean s) r) weight + bias,   r sqrt(..) s = 1, mean s in two f32,
// (v s is exact, its difference from the mean is rounded at its own size).  For a
// constant row, whose root is eps's alone, s is smaller, so that mean s stays in f32.
// An h that is not finite is formed again with its products in f64 (block_h_far).
//
// What bounds it: the bytes.  4096 rows of 8192, binary16 in, residual in and out, binary16
// out (402 MB): 80 us, 5.0 TB/s; a copy on this card runs at 5.1.  One row of 4096: 4.7 us,
// two loads, two sums across waves and a store, one after the other.  1000 rows of 2049,
// layer norms: 14-16 us, four sums across waves in a row.
struct RowNorm {
    float s, high, low, r;
};

__device__ __forceinline__ RowNorm row_factors(double mean, double squares, const BlockNormArgs& a)
{
    const double r = 1.0 / __builtin_sqrt(squares / (double)a.k + (double)a.eps);
    int power = 0;                             // of a zero, an infinity or NaN: any
    (void)frexp(r, &power);
    // A mean more than 2^100 times sqrt(..) is that of a row whose elements are all the
    // same (others deviate by 2^-24 / sqrt(k) of it at least): their difference is 0 at
    // any scale.
    int far = 0;                               // of an infinity or NaN: any
    (void)frexp(mean, &far);
    power = min(max(power, -126), mean == 0.0 ? 127 : min(100 - far, 127));
    RowNorm n;
    n.s = __builtin_bit_cast(float, (uint32_t)max(power + 127, 1) << 23);
    n.r = (float)ldexp(r, -power);
    n.high = (float)(mean * (double)n.s);
    n.low = (float)(mean * (double)n.s - (double)n.high);
    return n;
}

__device__ __forceinline__ float normed(float v, const RowNorm& n)
{
    return (__builtin_fmaf(v, n.s, -n.high) - n.low) * n.r;
}

// The workgroup's sum of v (each thread's); `part` is this sum's own
__device__ __forceinline__ double block_sum(double v, double* part, int waves)
{
    v = wave_sum(v);
    if (waves > 1) {
        if ((threadIdx.x & 63) == 0) {
            part[threadIdx.x >> 6] = v;
        }
        __syncthreads();
        v = part[0];
        for (int i = 1; i < waves; ++i) {      // in wave order, the same in every thread
            v += part[i];
        }
    }
    return v;
}

// The residual of the group at column c, zeros where there is none
template <bool TAIL>
__device__ __forceinline__ void block_residual(const BlockNormArgs& a, int64_t row, int c,
                                               float* r)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        r[i] = 0.f;
    }
    if (a.residual != nullptr) {
        load_f32<TAIL>(a, a.residual, row * a.k, c, r);
    }
}

// h of the elements that are not finite, again, its products in f64: a product of x, the
// weight or the gate may have passed f32 although h does not.  One element at a time
// and from memory: few rows come here, and the others keep their registers.
template <int TYPE>
__device__ __forceinline__ void block_h_far(const BlockNormArgs& a, int64_t row, int c,
                                            const RowNorm& n, float* h)
{
    if (!(n.r < __builtin_inff())) {
        return;                                // x's norm is NaN throughout
    }
    uint32_t lost = 0;                         // never an element behind the row's end
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lost |= fabsf(h[i]) < __builtin_inff() ? 0u : 1u << i;
    }
    for (; lost != 0; lost &= lost - 1) {
        const int i = __builtin_ctz(lost);
        const int at = c + i;
        const float x = element<TYPE>(a.x, row * a.x_stride + at);
        double p = x;
        if (a.post_weight != nullptr) {
            p = (double)normed(x, n) * (double)a.post_weight[at];
            p = a.post_bias != nullptr ? p + (double)a.post_bias[at] : p;
        }
        if (a.gate != nullptr) {
            p *= (double)a.gate[row * a.gate_stride + at];
        }
        const double r = a.residual != nullptr ? (double)a.residual[row * a.k + at] : 0.0;
        const float value = (float)__builtin_fma(p, (double)a.scale, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            h[e] = e == i ? value : h[e];
        }
    }
}

// h of the group at column c from its x and residual
template <int TYPE, bool TAIL>
__device__ __forceinline__ void block_h(const BlockNormArgs& a, int64_t row, int c, const float* x,
                                        const float* r, const RowNorm& n, float* h)
{
    float p[8], t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        p[i] = x[i];
    }
    if (a.post_weight != nullptr) {
        load_f32<TAIL>(a, a.post_weight, 0, c, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            p[i] = normed(p[i], n) * t[i];
        }
        if (a.post_bias != nullptr) {
            load_f32<TAIL>(a, a.post_bias, 0, c, t);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[i] += t[i];
            }
        }
    }
    if (a.gate != nullptr) {
        load_f32<TAIL>(a, a.gate, row * a.gate_stride, c, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            p[i] *= t[i];
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        h[i] = __builtin_fmaf(p[i], a.scale, r[i]);
        if (TAIL && c + i >= a.k) {
            h[i] = 0.f;
        }
    }
    // an infinity or NaN among them: their sum of products with 0 is NaN
    float none = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        none = __builtin_fmaf(h[i], 0.f, none);
    }
    if (__builtin_expect(__any(none != 0.f), 0)) {
        block_h_far<TYPE>(a, row, c, n, h);
    }
}

template <bool TAIL>
__device__ __forceinline__ void block_y(const BlockNormArgs& a, int64_t row, int c, const float* h,
                                        const RowNorm& n)
{
    float w[8], b[8], y[8];
    load_f32<TAIL>(a, a.weight, 0, c, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        b[i] = 0.f;
    }
    if (a.bias != nullptr) {
        load_f32<TAIL>(a, a.bias, 0, c, b);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[i] = __builtin_fmaf(normed(h[i], n), w[i], b[i]);
    }
    put_outputs<TAIL>(a, row, c, y);
}

// The residual is asked for with x.  Registers for eight waves a SIMD where they suffice.
template <int TYPE, int P, bool TAIL>
__global__ void __launch_bounds__(1024, P == 1 || (P == 2 && !TAIL) ? 8 : 4)
block_norm_kernel(BlockNormArgs a)
{
    __shared__ double part[4][16];
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x;
    const int threads = blockDim.x;
    const int waves = threads >> 6;
    const int groups = (a.k - 1) / 8 + 1;
    auto load_x = [&](int c, float* v) {
        if (!TAIL || a.k >= 8) {
            load8<TYPE>(a.x, row * a.x_stride + read_at<TAIL>(a, c), v);
        }
        if (TAIL && a.k - c < 8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = c + i < a.k ? element<TYPE>(a.x, row * a.x_stride + c + i) : 0.f;
            }
        }
    };
    // sum over the row's elements v of f(v); `more` gives those of a group beyond
    // the registers
    auto row_sum = [&](const float (&v)[P][8], auto more, double* place, auto f) {
        double sum = 0.0;
        auto add = [&](const float* e, int c) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sum += !TAIL || c + i < a.k ? f((double)e[i]) : 0.0;
            }
        };
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int gi = p * threads + tid;
            if (gi < groups) {
                add(v[p], gi * 8);
            }
        }
        for (int gi = P * threads + tid; gi < groups; gi += threads) {
            float e[8];
            more(gi * 8, e);
            add(e, gi * 8);
        }
        return block_sum(sum, place, waves);
    };
    auto row_norm = [&](const float (&v)[P][8], auto more, int which) {
        double mean = 0.0;
        if (a.layer) {
            mean = row_sum(v, more, part[2 * which], [](double e) { return e; }) / (double)a.k;
        }
        const double squares = row_sum(v, more, part[2 * which + 1],
                                       [mean](double e) { return (e - mean) * (e - mean); });
        return row_factors(mean, squares, a);
    };

    float v[P][8], res[P][8];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int gi = p * threads + tid;
        if (gi < groups) {
            load_x(gi * 8, v[p]);
            block_residual<TAIL>(a, row, gi * 8, res[p]);
        }
    }
    RowNorm n = {1.f, 0.f, 0.f, 1.f};
    if (a.post_weight != nullptr) {
        n = row_norm(v, load_x, 0);
    }
    const RowNorm post = n;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int gi = p * threads + tid;
        if (gi < groups) {
            block_h<TYPE, TAIL>(a, row, gi * 8, v[p], res[p], post, v[p]);
            if (a.sum != nullptr) {
                put_f32<TAIL>(a, a.sum, row, gi * 8, v[p]);
            }
        }
    }
    // h of a group beyond the registers: from sum where it is kept (this thread's
    // own stores; x and residual may have been there), else once more
    auto load_sum = [&](int c, float* h) {
        if (a.sum != nullptr) {
            load_f32<TAIL>(a, a.sum, row * a.k, c, h);
        } else {
            float x[8], r[8];
            load_x(c, x);
            block_residual<TAIL>(a, row, c, r);
            block_h<TYPE, TAIL>(a, row, c, x, r, post, h);
        }
    };
    if (a.sum != nullptr) {
        for (int gi = P * threads + tid; gi < groups; gi += threads) {
            float x[8], r[8];
            load_x(gi * 8, x);
            block_residual<TAIL>(a, row, gi * 8, r);
            block_h<TYPE, TAIL>(a, row, gi * 8, x, r, post, x);
            put_f32<TAIL>(a, a.sum, row, gi * 8, x);
        }
    }
    if (a.y == nullptr && a.y16 == nullptr && a.q == nullptr) {
        return;
    }
    n = row_norm(v, load_sum, 1);
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int gi = p * threads + tid;
        if (gi < groups) {
            block_y<TAIL>(a, row, gi * 8, v[p], n);
        }
    }
    for (int gi = P * threads + tid; gi < groups; gi += threads) {
        float h[8];
        load_sum(gi * 8, h);
        block_y<TAIL>(a, row, gi * 8, h, n);
    }
}

template <int TYPE, int P>
hipError_t launch_block_p(const BlockNormArgs& a, int threads, hipStream_t stream)
{
    const dim3 grid((unsigned)a.m), block(threads);
    if (a.k % 8 != 0) {
        hipLaunchKernelGGL((block_norm_kernel<TYPE, P, true>), grid, block, 0, stream, a);
    } else {
        hipLaunchKernelGGL((block_norm_kernel<TYPE, P, false>), grid, block, 0, stream, a);
    }
    return hipGetLastError();
}

// Groups of eight per thread, by what was measured (us with one / two / four):
//  - one for few rows (one row of 4096 4.3 / 4.6 / 5.8) and short ones (1000 rows of 2049
//    15.7 / 16.0 / 17.4, 4096 of 2048 25.2 / 26.4 / 26.1);
//  - two for many rows from 4096 elements on, whose workgroups, half as large, are in
//    different phases of theirs (4096 rows of 8192 100 / 87 / 92, 4096 of 4095 65 / 56 /
//    65, 2048 of 5120 34 / 31 / 34, 256 of 8192 9.6 / 9.1 / 10.2);
//  - beyond 8192 elements two, or four for many rows (256 rows of 14336 - / 12.5 / 13.0,
//    1024 rows - / 47 / 44); from 16384 on four.
template <int TYPE>
hipError_t launch_block_t(const BlockNormArgs& a, hipStream_t stream)
{
    const int groups = (a.k - 1) / 8 + 1;
    const auto threads = [&](int each) {
        const int64_t t = ((int64_t)(groups - 1) / each + 1 + 63) / 64 * 64;
        return (int)(t < 1024 ? t : 1024);
    };
    if (groups > 2048 || (groups > 1024 && a.m >= 1024)) {
        return launch_block_p<TYPE, 4>(a, threads(4), stream);
    }
    if (groups > 1024 || (groups >= 512 && a.m >= 256)) {
        return launch_block_p<TYPE, 2>(a, threads(2), stream);
    }
    return launch_block_p<TYPE, 1>(a, threads(1), stream);
}

}  // namespace

hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t stream)
{
    switch (a.x_type) {
    case kTypeF16: return launch_block_t<kTypeF16>(a, stream);
    case kTypeBF16: return launch_block_t<kTypeBF16>(a, stream);
    default: return launch_block_t<kTypeF32>(a, stream);
    }
}

hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t stream)
{
    switch (a.x_type) {
    case kTypeF16: return launch_t<kTypeF16>(a, stream);
    case kTypeBF16: return launch_t<kTypeBF16>(a, stream);
    default: return launch_t<kTypeF32>(a, stream);
    }
}

}  // namespace q4k
