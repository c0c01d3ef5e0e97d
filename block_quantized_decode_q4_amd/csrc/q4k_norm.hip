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

typedef uint16_t u16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 h8_t __attribute__((ext_vector_type(8)));

// Eight elements at p[0..], those at or beyond `left` as zero.  VEC: all
// eight are there and p is 16-byte aligned.
template <int TYPE, bool VEC>
__device__ __forceinline__ void load8(const void* base, int64_t at, int left, float* e)
{
    if constexpr (TYPE == kTypeF32) {
        const float* p = static_cast<const float*>(base) + at;
        if constexpr (VEC) {
            const float4 a = *reinterpret_cast<const float4*>(p);
            const float4 b = *reinterpret_cast<const float4*>(p + 4);
            e[0] = a.x; e[1] = a.y; e[2] = a.z; e[3] = a.w;
            e[4] = b.x; e[5] = b.y; e[6] = b.z; e[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                e[i] = i < left ? p[i] : 0.f;
            }
        }
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(base) + at;
        u16x8_t v;
        if constexpr (VEC) {
            v = *reinterpret_cast<const u16x8_t*>(p);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = i < left ? p[i] : (uint16_t)0;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint16_t b = v[i];
            e[i] = TYPE == kTypeF16 ? (float)__builtin_bit_cast(_Float16, b)
                                    : __builtin_bit_cast(float, (uint32_t)b << 16);
        }
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(float* base, int64_t at, int left, const float* e)
{
    float* p = base + at;
    if constexpr (VEC) {
        *reinterpret_cast<float4*>(p) = make_float4(e[0], e[1], e[2], e[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(e[4], e[5], e[6], e[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i < left) {
                p[i] = e[i];
            }
        }
    }
}

// h of the group at column c: x + residual (rounded once), or x.  XVEC: x's
// rows are 16-byte aligned too.
template <int TYPE, bool VEC, bool XVEC>
__device__ __forceinline__ void load_h(const NormArgs& a, int64_t row, int c, float* h)
{
    const int left = a.k - c;
    load8<TYPE, XVEC>(a.x, row * a.x_stride + c, left, h);
    if (a.residual != nullptr) {
        float r[8];
        load8<kTypeF32, VEC>(a.residual, row * a.k + c, left, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            h[i] += r[i];
        }
    }
}

// The outputs of one group from its h (and the row's factor r)
template <bool VEC>
__device__ __forceinline__ void put_y(const NormArgs& a, int64_t row, int c, const float* h,
                                      double r)
{
    const int left = a.k - c;
    float w[8], y[8];
    load8<kTypeF32, VEC>(a.weight, c, left, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[i] = (float)((double)h[i] * r * (double)w[i]);
    }
    const int64_t at = row * a.k + c;
    if (a.y != nullptr) {
        store8<VEC>(a.y, at, left, y);
    }
    if (a.y16 != nullptr) {
        h8_t v;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = (_Float16)y[i];
        }
        _Float16* p = static_cast<_Float16*>(a.y16) + at;
        if constexpr (VEC) {
            *reinterpret_cast<h8_t*>(p) = v;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (i < left) {
                    p[i] = v[i];
                }
            }
        }
    }
    if constexpr (VEC) {
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
// beyond P * threads are read twice.  VEC: 16-byte accesses (k a multiple of
// eight); XVEC: for x too (and its row stride).
template <int TYPE, int P, bool VEC, bool XVEC>
__global__ void __launch_bounds__(1024)
rmsnorm_kernel(NormArgs a)
{
    __shared__ double part[16];
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x;
    const int threads = blockDim.x;
    const int groups = (a.k + 7) / 8;
    float h[P][8];
    double sum = 0.0;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int gi = p * threads + tid;
        if (gi < groups) {
            load_h<TYPE, VEC, XVEC>(a, row, gi * 8, h[p]);
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
            store8<VEC>(a.sum, row * a.k + gi * 8, a.k - gi * 8, h[p]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sum = __builtin_fma((double)h[p][i], (double)h[p][i], sum);
        }
    }
    for (int gi = P * threads + tid; gi < groups; gi += threads) {
        float t[8];
        load_h<TYPE, VEC, XVEC>(a, row, gi * 8, t);
        if (a.sum != nullptr) {
            store8<VEC>(a.sum, row * a.k + gi * 8, a.k - gi * 8, t);
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
            put_y<VEC>(a, row, gi * 8, h[p], r);
        }
    }
    for (int gi = P * threads + tid; gi < groups; gi += threads) {
        float t[8];
        if (a.sum != nullptr) {                // this thread's own stores
            load8<kTypeF32, VEC>(a.sum, row * a.k + gi * 8, a.k - gi * 8, t);
        } else {
            load_h<TYPE, VEC, XVEC>(a, row, gi * 8, t);
        }
        put_y<VEC>(a, row, gi * 8, t, r);
    }
}

template <int TYPE, int P>
hipError_t launch_p(const NormArgs& a, int threads, hipStream_t stream)
{
    const dim3 grid((unsigned)a.m), block(threads);
    if (a.k % 8 != 0) {
        hipLaunchKernelGGL((rmsnorm_kernel<TYPE, P, false, false>), grid, block, 0, stream, a);
    } else if (a.x_stride % 8 != 0) {
        hipLaunchKernelGGL((rmsnorm_kernel<TYPE, P, true, false>), grid, block, 0, stream, a);
    } else {
        hipLaunchKernelGGL((rmsnorm_kernel<TYPE, P, true, true>), grid, block, 0, stream, a);
    }
    return hipGetLastError();
}

template <int TYPE>
hipError_t launch_t(const NormArgs& a, hipStream_t stream)
{
    const int groups = (a.k + 7) / 8;
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
