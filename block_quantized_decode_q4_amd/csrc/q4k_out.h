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

// The sum v of weight row `row`, y's element `at`
__device__ __forceinline__ void put_y(const EpArgs& e, size_t at, int row, double v)
{
    const float z = (float)(v + (e.bias != nullptr ? (double)e.bias[row] : 0.0));
    ep_store(e, (int64_t)at, ep_value(e, (int64_t)at, z));
}

// z of weight row `row` of matrix g, in y row yrow
__device__ __forceinline__ void put_grouped(const GroupedActArgs& a, int g, int yrow, int row,
                                            float z)
{
    const int64_t at = (int64_t)yrow * a.n + row;
    z += a.ep.bias != nullptr ? a.ep.bias[(int64_t)g * a.n + row] : 0.f;
    ep_store(a.ep, at, ep_value(a.ep, at, z));
}

#else

typedef float* __restrict__ Out;
typedef GroupedArgs GroupedOut;
constexpr bool kEpilogue = false;

__device__ __forceinline__ constexpr bool parked(const float*) { return false; }
__device__ __forceinline__ float* direct_y(float* y) { return y; }
__device__ __forceinline__ void put_y(float* y, size_t at, int, double v) { y[at] = (float)v; }
__device__ __forceinline__ void put_grouped(const GroupedArgs& a, int, int yrow, int row, float z)
{
    a.y[(int64_t)yrow * a.n + row] = z;
}

#endif

}  // namespace q4k
