// q4k_q8.h -- the Q8 block rule (32 consecutive elements, an f32 scale, int8
// codes), shared by the kernels that quantize activations (q4k_q8.hip,
// q4k_norm.hip).  Internal.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace q4k {

// The scale and reciprocal of a block from its largest |x| (NaN if the
// block holds one): d = amax / 127, inv = 127 / amax (0 where amax is 0 or
// NaN), both correctly rounded f32 quotients.
struct Q8Scale {
    float d, inv;
};

__device__ __forceinline__ Q8Scale q8_scale(float amax, bool has_nan)
{
    Q8Scale s;
    const float a = has_nan ? __builtin_nanf("") : amax;
    s.d = a / 127.0f;
    s.inv = a > 0.0f ? 127.0f / a : 0.0f;
    return s;
}

// The code of one element: nearest-even integer of x * inv, 0 if that
// product is not finite.
__device__ __forceinline__ int q8_code(float x, float inv)
{
    const float v = x * inv;
    return __builtin_isfinite(v) ? (int)__builtin_rintf(v) : 0;
}

// Four codes as the bytes of one dword (element 4t + i in byte i)
__device__ __forceinline__ uint32_t q8_pack(int a, int b, int c, int d)
{
    return ((uint32_t)a & 0xFFu) | (((uint32_t)b & 0xFFu) << 8) | (((uint32_t)c & 0xFFu) << 16) |
           ((uint32_t)d << 24);
}

}  // namespace q4k
