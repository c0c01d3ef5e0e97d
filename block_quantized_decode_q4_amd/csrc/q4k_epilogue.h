// q4k_epilogue.h -- what a product's sum z (its bias added) goes through:
//   y = act(z) gate + residual
// in f32, each step rounded once (the last two may be one fused step), y16 the
// nearest binary16 of that y.  Internal.
//
// The activations, each without cancellation for negative z:
//   silu        z / (1 + e^-z)
//   gelu        z/2 erfc(-z / sqrt 2)
//   gelu, tanh  z/2 (1 + tanh u) = z / (1 + e^-2u), u = sqrt(2/pi) (z + 0.044715 z^3)
//   sigmoid     1 / (1 + e^-z)
// e^x and 1 / x are the hardware's (a rounding or two each; the bound that the header
// gives for act(z) allows for e^x's product, |z| 2^-24), erfc is the library's.
//
// Bound by nothing of its own: the operands are read once and y is written once, on the
// way out of the product.  2048 x 14336 x 4096 with silu and a gate takes 240 us a call,
// 1930 in separate operations in f32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4k_kernels.h"

namespace q4k {

// enum q4k_act of include/q4k.h
constexpr int kActNone = 0;
constexpr int kActRelu = 1;
constexpr int kActSilu = 2;
constexpr int kActGelu = 3;
constexpr int kActGeluTanh = 4;
constexpr int kActSigmoid = 5;

// e^x by the hardware's 2^x: the product's rounding is x 2^-24 of it, the rest a few
// steps; above 2^128 infinity, below 2^-126 0
__device__ __forceinline__ float fast_exp(float x)
{
    return __builtin_amdgcn_exp2f(x * 1.44269504f);
}

template <int ACT>
__device__ __forceinline__ float activated(float z)
{
    if constexpr (ACT == kActRelu) {
        return z < 0.f ? 0.f : z;              // a NaN stays one
    } else if constexpr (ACT == kActSilu) {
        return z * __builtin_amdgcn_rcpf(1.f + fast_exp(-z));
    } else if constexpr (ACT == kActGelu) {
        return 0.5f * z * erfcf(z * -0.707106781f);
    } else if constexpr (ACT == kActGeluTanh) {
        const float u2 = 1.59576912f * (z + 0.044715f * z * z * z);
        return z * __builtin_amdgcn_rcpf(1.f + fast_exp(-u2));
    } else if constexpr (ACT == kActSigmoid) {
        return __builtin_amdgcn_rcpf(1.f + fast_exp(-z));
    } else {
        return z;
    }
}

__device__ __forceinline__ float activated(int act, float z)
{
    switch (act) {                             // the same for the whole launch
    case kActRelu: return activated<kActRelu>(z);
    case kActSilu: return activated<kActSilu>(z);
    case kActGelu: return activated<kActGelu>(z);
    case kActGeluTanh: return activated<kActGeluTanh>(z);
    case kActSigmoid: return activated<kActSigmoid>(z);
    default: return z;
    }
}

// What an element's epilogue reads, asked for together
struct EpOperands {
    float bias, gate, residual;
};

// of element `at` of y and weight row `row` (both within their tensors)
__device__ __forceinline__ EpOperands ep_fetch(const EpArgs& e, int64_t at, int64_t row)
{
    EpOperands o = {0.f, 1.f, 0.f};
    if (e.bias != nullptr) {
        o.bias = e.bias[row];
    }
    if (e.gate != nullptr) {
        o.gate = e.gate_type == kTypeF16 ? (float)static_cast<const _Float16*>(e.gate)[at]
                                         : static_cast<const float*>(e.gate)[at];
    }
    if (e.residual != nullptr) {
        o.residual = e.residual[at];
    }
    return o;
}

// y from its z (the bias added)
__device__ __forceinline__ float ep_value(const EpArgs& e, const EpOperands& o, float z)
{
    float v = activated(e.act, z);
    v = e.gate != nullptr ? v * o.gate : v;
    return e.residual != nullptr ? v + o.residual : v;
}

__device__ __forceinline__ void ep_store(const EpArgs& e, int64_t at, float v)
{
    if (e.y != nullptr) {
        e.y[at] = v;
    }
    if (e.y16 != nullptr) {
        static_cast<_Float16*>(e.y16)[at] = (_Float16)v;
    }
}

}  // namespace q4k
