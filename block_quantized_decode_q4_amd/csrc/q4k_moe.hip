// q4k_moe.hip -- the routing of tokens to experts, and the weighted sum of
// the experts' outputs.
//
// Route: of each token's E logits the topk largest (equal ones: the lowest
// expert first), with weights
//   p_j = exp(l_j - max) / sum exp(l - max),
// the sum over the chosen experts or over all of them, in f32.  A logit that
// is NaN or -inf is masked: never chosen, nothing in the sum.  A token with
// fewer than topk experts left gets id -1 and weight 0 in the rest.
//
// Group: the slots (token t's choice j is slot t * topk + j) in the order of
// their ids, equal ids in slot order, and where each id begins.  A slot
// whose id is no group is in none; the order's tail is -1.
//
// A wave routes a token: lane i holds experts i, i + 64, ...; each of the
// topk steps is a maximum over the wave and a ballot for its lowest expert.
// The grouping is a counting sort.  Few slots: one workgroup, in one launch
// with the routing; a slot's place is the number of slots that sort before
// it, counted by reading all of them from LDS.  More: the routing launch
// counts each chunk's slots per expert, and a second launch places them: each
// workgroup adds up the counts of all chunks (they are few) for itself, so
// no third launch scans them, and each wave places 64 slots at a time by
// matching ids across its lanes.  Integer counts only: the result is the same
// every time.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4k_groups.h"
#include "q4k_kernels.h"

namespace q4k {

namespace {

constexpr int kPlaceThreads = 1024;
constexpr int kPlaceWaves = kPlaceThreads / 64;

// One step of a wave reduction: v of the lane that DPP control CTRL names (its
// own where there is none).
template <int CTRL>
__device__ __forceinline__ float dpp_f(float v)
{
    const int i = __builtin_bit_cast(int, v);
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(i, i, CTRL, 0xF, 0xF, false));
}

// Wave maximum of f32 values that are not NaN: within rows of 16 lanes (row
// shifts by 1, 2, 4, 8), then across them (broadcasts of lanes 15 and 31), so
// lane 63 has it.
__device__ __forceinline__ float wave_max(float v)
{
    v = fmaxf(v, dpp_f<0x111>(v));
    v = fmaxf(v, dpp_f<0x112>(v));
    v = fmaxf(v, dpp_f<0x114>(v));
    v = fmaxf(v, dpp_f<0x118>(v));
    v = fmaxf(v, dpp_f<0x142>(v));
    v = fmaxf(v, dpp_f<0x143>(v));
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

__device__ __forceinline__ float wave_sum_f(float v)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        v += __shfl_xor(v, off, 64);
    }
    return v;
}

// One token's experts, by one wave.  NL: logits per lane (experts lane,
// lane + 64, ...).  Lane j (j < topk) returns the j-th choice and weight.
template <int NL>
__device__ __forceinline__ void route_token(const float* logits, int experts, int topk, int renorm,
                                            int& id, float& weight)
{
    const float kNone = -__builtin_inff();
    const int lane = threadIdx.x & 63;
    float l[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int e = i * 64 + lane;
        const float v = e < experts ? logits[e] : kNone;
        l[i] = v == v ? v : kNone;
    }
    float all = 0.f;
    if (!renorm) {
        float top = kNone;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            top = fmaxf(top, l[i]);
        }
        top = wave_max(top);
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            // equal infinities would leave inf - inf: the largest counts 1
            all += l[i] == kNone ? 0.f : l[i] == top ? 1.f : expf(l[i] - top);
        }
        all = wave_sum_f(all);
    }
    id = -1;
    weight = 0.f;
    float first = 0.f;
    for (int j = 0; j < topk; ++j) {
        float best = l[0];
#pragma unroll
        for (int i = 1; i < NL; ++i) {
            best = fmaxf(best, l[i]);
        }
        best = wave_max(best);
        if (best == kNone) {
            break;                             // nothing left: id -1, weight 0
        }
        if (j == 0) {
            first = best;
        }
        int chosen = -1;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const uint64_t has = __ballot(l[i] == best);
            if (chosen < 0 && has != 0) {
                chosen = i * 64 + __builtin_ctzll(has);
            }
        }
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            if (i * 64 + lane == chosen) {
                l[i] = kNone;
            }
        }
        if (lane == j) {
            id = chosen;
            weight = best == first ? 1.f : expf(best - first);
        }
    }
    if (renorm) {
        all = wave_sum_f(lane < topk ? weight : 0.f);
    }
    weight = id >= 0 ? weight / all : 0.f;
}

// Few slots: routing and grouping in one workgroup.  ROUTE false: the ids are
// given.  slots <= kFewSlots.
template <int NL, bool ROUTE>
__global__ void __launch_bounds__(kPlaceThreads)
group_few_kernel(RouteArgs a)
{
    __shared__ __align__(16) int ids[kFewSlots];
    const int tid = threadIdx.x;
    const int slots = a.slots;
    for (int i = slots + tid; i < kFewSlots; i += kPlaceThreads) {
        ids[i] = 0x7fffffff;                   // sorts behind everything
    }
    if constexpr (ROUTE) {
        const int lane = tid & 63;
        for (int t = tid >> 6; t < a.m; t += kPlaceWaves) {
            int id;
            float weight;
            route_token<NL>(a.logits + t * a.stride, a.groups, a.topk, a.renorm, id, weight);
            if (lane < a.topk) {
                const int s = t * a.topk + lane;
                a.ids[s] = id;
                a.weights[s] = weight;
                ids[s] = id < 0 ? 0x7fffffff : id;
            }
        }
    } else {
        for (int i = tid; i < slots; i += kPlaceThreads) {
            const int id = a.ids[i];
            ids[i] = id < 0 || id >= a.groups ? 0x7fffffff : id;
        }
    }
    if (a.offsets == nullptr) {
        return;
    }
    __syncthreads();
    // place of slot i: the slots with a smaller id, and those with the same
    // id before it.  One thread per slot, then per offset (the slots whose id
    // is below g), four ids per LDS read (the same for all lanes: broadcast).
    const int quads = (slots + 3) / 4;
    for (int i = tid; i < slots + a.groups + 1; i += kPlaceThreads) {
        const bool slot = i < slots;
        const int mine = slot ? ids[i] : i - slots;
        int below = 0, same = 0;
        for (int v = 0; v < quads; ++v) {
            const int4 o = *reinterpret_cast<const int4*>(ids + 4 * v);
            below += (o.x < mine) + (o.y < mine) + (o.z < mine) + (o.w < mine);
            same += (o.x == mine && 4 * v < i) + (o.y == mine && 4 * v + 1 < i) +
                    (o.z == mine && 4 * v + 2 < i) + (o.w == mine && 4 * v + 3 < i);
        }
        if (slot) {
            // a slot in no group still has a place of its own, in the tail
            a.order[below + same] = mine == 0x7fffffff ? -1 : i;
        } else {
            a.offsets[mine] = below;
        }
    }
}

// More slots: chunk c counts its slots per group into counts[c][0..groups).
// With ROUTE it routes the chunk's tokens first.
template <int NL, bool ROUTE>
__global__ void __launch_bounds__(kPlaceThreads)
group_count_kernel(RouteArgs a)
{
    extern __shared__ int hist[];
    const int tid = threadIdx.x;
    for (int g = tid; g < a.groups; g += kPlaceThreads) {
        hist[g] = 0;
    }
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * a.chunk;
    const int64_t hi = min(lo + a.chunk, (int64_t)a.slots);
    if constexpr (ROUTE) {
        const int lane = tid & 63;
        const int64_t last = hi / a.topk;      // a chunk holds whole tokens
        for (int64_t t = lo / a.topk + (tid >> 6); t < last; t += kPlaceWaves) {
            int id;
            float weight;
            route_token<NL>(a.logits + t * a.stride, a.groups, a.topk, a.renorm, id, weight);
            if (lane < a.topk) {
                a.ids[t * a.topk + lane] = id;
                a.weights[t * a.topk + lane] = weight;
                if (id >= 0) {
                    atomicAdd(&hist[id], 1);
                }
            }
        }
    } else {
        for (int64_t i = lo + tid; i < hi; i += kPlaceThreads) {
            const int id = a.ids[i];
            if (id >= 0 && id < a.groups) {
                atomicAdd(&hist[id], 1);
            }
        }
    }
    __syncthreads();
    if (a.counts == nullptr) {
        return;                                // routing alone
    }
    for (int g = tid; g < a.groups; g += kPlaceThreads) {
        a.counts[(int64_t)blockIdx.x * a.groups + g] = hist[g];
    }
}

// Places the slots of chunk c.  LDS: cur[kPlaceWaves][groups], the next place
// of each group in each wave's part of the chunk; begin[groups]; sums.
__global__ void __launch_bounds__(kPlaceThreads)
group_place_kernel(RouteArgs a)
{
    extern __shared__ int smem[];
    int* const cur = smem;                     // kPlaceWaves * groups
    int* const begin = smem + kPlaceWaves * a.groups;        // groups + 1
    int* const part = begin + a.groups + 1;    // 2 * kPlaceThreads
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = tid >> 6;
    const int c = blockIdx.x;
    const int G = a.groups;
    // the chunks' counts per group, all and before this chunk: threads t,
    // t + G, ... share group t % G's chunks between them
    const int shares = max(1, min(kPlaceThreads / G, a.chunks));
    for (int i = tid; i < kPlaceWaves * G; i += kPlaceThreads) {
        cur[i] = 0;
    }
    const int g0 = tid % G;
    const int share = tid / G;
    int all = 0, before = 0;
    if (share < shares) {
#pragma unroll 8
        for (int k = share; k < a.chunks; k += shares) {
            const int v = a.counts[(int64_t)k * G + g0];
            all += v;
            before += k < c ? v : 0;
        }
    }
    part[tid] = all;
    part[kPlaceThreads + tid] = before;
    __syncthreads();
    if (tid < G) {
        for (int k = 1; k < shares; ++k) {
            all += part[k * G + tid];
            before += part[kPlaceThreads + k * G + tid];
        }
    }
    __syncthreads();
    part[tid] = tid < G ? all : 0;
    __syncthreads();
    // where the groups begin: a scan over the totals (wave 0, 64 at a time)
    if (wave == 0) {
        int sum = 0;
        for (int base = 0; base < G; base += 64) {
            const int g = base + lane;
            const int v = g < G ? part[g] : 0;
            const int upto = wave_scan_add(v, lane);
            if (g < G) {
                begin[g] = sum + upto - v;
            }
            sum += __builtin_amdgcn_readlane(upto, 63);
        }
        if (lane == 0) {
            begin[G] = sum;
        }
    }
    // this chunk's slots per wave and group
    const int64_t lo = (int64_t)c * a.chunk;
    const int64_t hi = min(lo + a.chunk, (int64_t)a.slots);
    const int64_t each = ((a.chunk + kPlaceWaves - 1) / kPlaceWaves + 63) / 64 * 64;
    const int64_t wlo = min(lo + wave * each, hi);
    const int64_t whi = min(wlo + each, hi);
    // volatile: lanes of one wave read each other's updates below
    volatile int* const mine = cur + wave * G;
    for (int64_t i = wlo + lane; i < whi; i += 64) {
        const int id = a.ids[i];
        if (id >= 0 && id < G) {
            atomicAdd(&cur[wave * G + id], 1);
        }
    }
    __syncthreads();
    // counts to places: group g's slots of this chunk begin behind those of
    // the chunks and waves before
    if (tid < G) {
        int at = begin[tid] + before;
        for (int w = 0; w < kPlaceWaves; ++w) {
            const int n = cur[w * G + tid];
            cur[w * G + tid] = at;
            at += n;
        }
        if (c == 0) {
            a.offsets[tid] = begin[tid];
        }
    }
    if (c == 0 && tid == 0) {
        a.offsets[G] = begin[G];
    }
    __syncthreads();
    int bits = 0;
    while ((1 << bits) < G) {
        ++bits;
    }
    for (int64_t i0 = wlo; i0 < whi; i0 += 64) {
        const int64_t i = i0 + lane;
        const int id = i < whi ? a.ids[i] : -1;
        const bool in = id >= 0 && id < G;
        // the lanes with the same id
        uint64_t peers = __ballot(in);
        for (int b = 0; b < bits; ++b) {
            const uint64_t set = __ballot((id >> b) & 1);
            peers &= (id >> b) & 1 ? set : ~set;
        }
        if (in) {
            const int rank = __popcll(peers & ((1ull << lane) - 1));
            const int at = mine[id];
            a.order[at + rank] = (int)i;
            // every peer has read `at` (one wave, in lockstep); the last moves it on
            __builtin_amdgcn_wave_barrier();
            if ((peers >> lane) == 1) {
                mine[id] = at + rank + 1;
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
    // the tail: slots in no group
    for (int64_t i = (int64_t)begin[G] + (int64_t)c * kPlaceThreads + tid; i < a.slots;
         i += (int64_t)a.chunks * kPlaceThreads) {
        a.order[i] = -1;
    }
}

// out[t][c] = residual[t][c] + sum_j weights[t][j] y[t * topk + j][c], over
// the choices with an id (f32, in the order of j).  A thread owns V
// consecutive columns of one token.
template <int V>
__global__ void __launch_bounds__(256)
combine_kernel(CombineArgs a)
{
    const int64_t t = blockIdx.x / a.parts;
    const int c = ((int)(blockIdx.x % a.parts) * 256 + (int)threadIdx.x) * V;
    if (c >= a.n) {
        return;
    }
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        acc[i] = 0.f;
    }
    const float* y = a.y + t * a.topk * a.n + c;
#pragma unroll 4
    for (int j = 0; j < a.topk; ++j) {
        const float w = a.weights[t * a.topk + j];
        if (a.ids != nullptr && a.ids[t * a.topk + j] < 0) {
            continue;                          // no expert: its row was not written
        }
        const float* p = y + (int64_t)j * a.n;
        if constexpr (V == 4) {
            const float4 v = *reinterpret_cast<const float4*>(p);
            acc[0] = __builtin_fmaf(w, v.x, acc[0]);
            acc[1] = __builtin_fmaf(w, v.y, acc[1]);
            acc[2] = __builtin_fmaf(w, v.z, acc[2]);
            acc[3] = __builtin_fmaf(w, v.w, acc[3]);
        } else {
            acc[0] = __builtin_fmaf(w, p[0], acc[0]);
        }
    }
    if constexpr (V == 4) {
        if (a.residual != nullptr) {
            const float4 r = *reinterpret_cast<const float4*>(a.residual + t * a.n + c);
            acc[0] += r.x; acc[1] += r.y; acc[2] += r.z; acc[3] += r.w;
        }
        *reinterpret_cast<float4*>(a.out + t * a.n + c) =
            make_float4(acc[0], acc[1], acc[2], acc[3]);
    } else {
        if (a.residual != nullptr) {
            acc[0] += a.residual[t * a.n + c];
        }
        a.out[t * a.n + c] = acc[0];
    }
}

// Slots per chunk: whole tokens, about 256 chunks (each placing workgroup
// adds up all chunks' counts), and at least 64 slots.
int64_t chunk_slots(int64_t slots, int64_t topk)
{
    int64_t c = (slots + 255) / 256;
    c = c < 64 ? 64 : c;
    return (c + topk - 1) / topk * topk;
}

size_t place_lds(int groups)
{
    return sizeof(int) * ((size_t)(kPlaceWaves + 1) * groups + 1 + 2 * kPlaceThreads);
}

template <int NL, bool ROUTE>
hipError_t launch_route_t(RouteArgs a, hipStream_t stream)
{
    if (a.slots <= kFewSlots) {
        hipLaunchKernelGGL((group_few_kernel<NL, ROUTE>), dim3(1), dim3(kPlaceThreads), 0, stream,
                           a);
        return hipGetLastError();
    }
    a.chunk = chunk_slots(a.slots, a.topk);
    a.chunks = (int)((a.slots + a.chunk - 1) / a.chunk);
    if (a.offsets == nullptr) {
        a.counts = nullptr;
    }
    hipLaunchKernelGGL((group_count_kernel<NL, ROUTE>), dim3(a.chunks), dim3(kPlaceThreads),
                       sizeof(int) * a.groups, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.offsets == nullptr) {
        return e;
    }
    hipLaunchKernelGGL(group_place_kernel, dim3(a.chunks), dim3(kPlaceThreads),
                       place_lds(a.groups), stream, a);
    return hipGetLastError();
}

}  // namespace

size_t group_ws_bytes(int64_t slots, int64_t groups, int64_t topk)
{
    if (slots <= kFewSlots) {
        return 0;
    }
    const int64_t chunk = chunk_slots(slots, topk);
    return sizeof(int) * (size_t)((slots + chunk - 1) / chunk) * (size_t)groups;
}

hipError_t launch_route(const RouteArgs& a, hipStream_t stream)
{
    if (a.logits == nullptr) {
        return launch_route_t<1, false>(a, stream);
    }
    if (a.groups <= 64) {
        return launch_route_t<1, true>(a, stream);
    }
    if (a.groups <= 128) {
        return launch_route_t<2, true>(a, stream);
    }
    if (a.groups <= 256) {
        return launch_route_t<4, true>(a, stream);
    }
    if (a.groups <= 512) {
        return launch_route_t<8, true>(a, stream);
    }
    return launch_route_t<16, true>(a, stream);
}

hipError_t launch_combine(CombineArgs a, hipStream_t stream)
{
    const int v = a.n % 4 == 0 ? 4 : 1;
    a.parts = (a.n + 256 * v - 1) / (256 * v);
    const dim3 grid((unsigned)((int64_t)a.m * a.parts));
    if (v == 4) {
        hipLaunchKernelGGL(combine_kernel<4>, grid, dim3(256), 0, stream, a);
    } else {
        hipLaunchKernelGGL(combine_kernel<1>, grid, dim3(256), 0, stream, a);
    }
    return hipGetLastError();
}

}  // namespace q4k
