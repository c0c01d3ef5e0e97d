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

// The outputs of one group from its h (and the row's factor r)
template <bool TAIL>
__device__ __forceinline__ void put_y(const NormArgs& a, int64_t row, int c, const float* h,
                                      double r)
{
    float w[8], y[8];
    if (!TAIL || a.k >= 8) {
        load8<kTypeF32>(a.weight, read_at<TAIL>(a, c), w);
    }
    if (TAIL && a.k - c < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[i] = c + i < a.k ? a.weight[c + i] : 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[i] = (float)((double)h[i] * r * (double)w[i]);
    }
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

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t stream)
{
    switch (a.x_type) {
    case kTypeF16: return launch_t<kTypeF16>(a, stream);
    case kTypeBF16: return launch_t<kTypeBF16>(a, stream);
    default: return launch_t<kTypeF32>(a, stream);
    }
}

}  // namespace q4k
