// q4k_out.h -- where the results of the Q4_K products go: to y itself or, in the
// files that define Q4K_EPILOGUE and include a product's source (q4k_act_*.hip),
// through an epilogue.  Internal.
#pragma once

#include "q4k_epilogue.h"
#include "q4k_kernels.h"

namespace q4k {

#ifdef Q4K_EPILOGUE

typedef EpArgs Out;
typedef GroupedActArgs GroupedOut;
constexpr bool kEpilogue = true;

// Whether a workgroup's sums meet in LDS even where each is whole: the operands
// of the epilogue are then read by all threads at once, beside one another, and
// not by a few lanes of a wave in the middle of its weight stream.
__device__ __forceinline__ bool parked(const EpArgs& e) { return e.parked != 0; }
__device__ __forceinline__ float* direct_y(const EpArgs&) { return nullptr; }

// What the element `at` of y, of weight row `row`, reads beside its sum; with `there`
// false nothing.  Kernels ask for a thread's first one when they start, so that it does
// not wait for it at the end (one token, 4096 x 4096 with bias and residual: 7.24 -> 7.08
// us, 14336 x 4096 gated 10.7 -> 10.5).
__device__ __forceinline__ EpOperands fetch_y(const EpArgs& e, bool there, size_t at, int row)
{
    EpOperands o = {0.f, 1.f, 0.f};
    if (there) {
        o = ep_fetch(e, (int64_t)at, row);
    }
    return o;
}

// The sum v of the element that o was fetched for
__device__ __forceinline__ void put_y(const EpArgs& e, size_t at, const EpOperands& o, double v)
{
    const float z = (float)(v + (double)o.bias);
    ep_store(e, (int64_t)at, ep_value(e, o, z));
}

// z of weight row `row` of matrix g, in y row yrow
__device__ __forceinline__ void put_grouped(const GroupedActArgs& a, int g, int yrow, int row,
                                            float z)
{
    const int64_t at = (int64_t)yrow * a.n + row;
    const EpOperands o = ep_fetch(a.ep, at, (int64_t)g * a.n + row);
    ep_store(a.ep, at, ep_value(a.ep, o, z + o.bias));
}

#else

typedef float* __restrict__ Out;
typedef GroupedArgs GroupedOut;
constexpr bool kEpilogue = false;

__device__ __forceinline__ constexpr bool parked(const float*) { return false; }
__device__ __forceinline__ float* direct_y(float* y) { return y; }
struct NoOperands {
};
__device__ __forceinline__ NoOperands fetch_y(const float*, bool, size_t, int) { return {}; }
__device__ __forceinline__ void put_y(float* y, size_t at, NoOperands, double v)
{
    y[at] = (float)v;
}
__device__ __forceinline__ void put_grouped(const GroupedArgs& a, int, int yrow, int row, float z)
{
    a.y[(int64_t)yrow * a.n + row] = z;
}

#endif

}  // namespace q4k
