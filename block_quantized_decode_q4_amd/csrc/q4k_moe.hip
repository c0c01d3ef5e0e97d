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
// A token's logits are spread over 16 lanes (up to 256 experts, four tokens per
// wave) or a wave; each of the topk steps is a maximum over the lanes and a
// minimum of the experts that have it, both by lane moves (DPP).  Four tokens
// per wave instead of one: 8192 tokens of 128 experts, topk 8, 6.3 us instead of
// 11 us for the routing launch.  Bound by those steps, each a chain of lane
// moves; the bytes (5 MB) would take 1 us.
// The grouping is a counting sort.  Few slots: one workgroup, in one launch
// with the routing; a slot's place is the number of slots that sort before
// it, counted by reading all of them from LDS.  More: the routing launch
// counts each chunk's slots per expert, and a second launch places them: each
// workgroup adds up the counts of all chunks (they are few) for itself, so
// no third launch scans them, and each wave places 64 slots at a time by
// matching ids across its lanes (6.4-7 us for those 65536 slots, the latency of its
// three passes over them).  Integer counts only: the result is the same every
// time.  Eight tokens, 64 experts, all in one launch: 5.3 us.
//
// The weighted sum reads every row of y once, four columns a thread: 201 MB
// (4096 tokens, topk 2) in 35 us, 5.7 TB/s, bound by the bytes.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4k_groups.h"
#include "q4k_kernels.h"

namespace q4k {

namespace {

constexpr int kPlaceThreads = 1024;
constexpr int kPlaceWaves = kPlaceThreads / 64;
constexpr int kCountThreads = 512;

// v of the lane that DPP control CTRL names: its own where there is none (OLD
// v), or 0 there and in the rows outside ROWS
template <int CTRL>
__device__ __forceinline__ int dpp(int v)
{
    return __builtin_amdgcn_update_dpp(v, v, CTRL, 0xF, 0xF, false);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_or_0(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                         0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xF, true));
}

__device__ __forceinline__ int as_int(float v) { return __builtin_bit_cast(int, v); }
__device__ __forceinline__ float as_float(int v) { return __builtin_bit_cast(float, v); }

// Reductions over a token's lanes, known to all of them.  16 lanes (a DPP row):
// rotations by 8, 4, 2, 1.  64: shifts within the rows by 1, 2, 4, 8, then the
// broadcasts of lanes 15 and 31 across rows, so that lane 63 has the result.
template <int LANES>
__device__ __forceinline__ float lanes_max(float v)       // no NaN
{
    if constexpr (LANES == 16) {
        v = fmaxf(v, as_float(dpp<0x128>(as_int(v))));
        v = fmaxf(v, as_float(dpp<0x124>(as_int(v))));
        v = fmaxf(v, as_float(dpp<0x122>(as_int(v))));
        v = fmaxf(v, as_float(dpp<0x121>(as_int(v))));
        return v;
    } else {
        v = fmaxf(v, as_float(dpp<0x111>(as_int(v))));
        v = fmaxf(v, as_float(dpp<0x112>(as_int(v))));
        v = fmaxf(v, as_float(dpp<0x114>(as_int(v))));
        v = fmaxf(v, as_float(dpp<0x118>(as_int(v))));
        v = fmaxf(v, as_float(dpp<0x142>(as_int(v))));
        v = fmaxf(v, as_float(dpp<0x143>(as_int(v))));
        return as_float(__builtin_amdgcn_readlane(as_int(v), 63));
    }
}

template <int LANES>
__device__ __forceinline__ int lanes_min(int v)
{
    if constexpr (LANES == 16) {
        v = min(v, dpp<0x128>(v));
        v = min(v, dpp<0x124>(v));
        v = min(v, dpp<0x122>(v));
        v = min(v, dpp<0x121>(v));
        return v;
    } else {
        v = min(v, dpp<0x111>(v));
        v = min(v, dpp<0x112>(v));
        v = min(v, dpp<0x114>(v));
        v = min(v, dpp<0x118>(v));
        v = min(v, dpp<0x142>(v));
        v = min(v, dpp<0x143>(v));
        return __builtin_amdgcn_readlane(v, 63);
    }
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v)
{
    if constexpr (LANES == 16) {
        v += as_float(dpp<0x128>(as_int(v)));
        v += as_float(dpp<0x124>(as_int(v)));
        v += as_float(dpp<0x122>(as_int(v)));
        v += as_float(dpp<0x121>(as_int(v)));
        return v;
    } else {
        v += dpp_or_0<0x111, 0xF>(v);
        v += dpp_or_0<0x112, 0xF>(v);
        v += dpp_or_0<0x114, 0xF>(v);
        v += dpp_or_0<0x118, 0xF>(v);
        v += dpp_or_0<0x142, 0xA>(v);
        v += dpp_or_0<0x143, 0xC>(v);
        return as_float(__builtin_amdgcn_readlane(as_int(v), 63));
    }
}

constexpr float kNone = -__builtin_inff();

// The logits of a wave's 64 / LANES tokens from `token` on, NL per lane: experts
// i, i + LANES, ... in lane i of a token's LANES.  A token at or beyond `last`
// has none.
template <int LANES, int NL>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t token, int64_t last,
                                            float* l)
{
    const int lane = threadIdx.x & 63;
    const int64_t t = token + lane / LANES;
    const float* p = a.logits + t * a.stride;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int e = i * LANES + lane % LANES;
        l[i] = t < last && e < a.groups ? p[e] : kNone;
    }
}

// Their experts.  Lane i of a token gets its choices i, i + LANES, ... (those
// below topk; kMaxTopk / LANES at most).
template <int LANES>
constexpr int kChoices = LANES < kMaxTopk ? kMaxTopk / LANES : 1;

template <int LANES, int NL>
__device__ __forceinline__ void route_tokens(const RouteArgs& a, float* l, int* id, float* weight)
{
    constexpr int C = kChoices<LANES>;
    const int i0 = threadIdx.x & (LANES - 1);
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        l[i] = l[i] == l[i] ? l[i] : kNone;
    }
    float all = 0.f;
    if (!a.renorm) {
        float top = kNone;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            top = fmaxf(top, l[i]);
        }
        top = lanes_max<LANES>(top);
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            // equal infinities would leave inf - inf: the largest counts 1
            all += l[i] == kNone ? 0.f : l[i] == top ? 1.f : expf(l[i] - top);
        }
        all = lanes_sum<LANES>(all);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        id[c] = -1;
        weight[c] = kNone;                     // the chosen logit, so far
    }
    float first = 0.f;
    for (int j = 0; j < a.topk; ++j) {
        float best = l[0];
#pragma unroll
        for (int i = 1; i < NL; ++i) {
            best = fmaxf(best, l[i]);
        }
        best = lanes_max<LANES>(best);
        if (__all(best == kNone)) {
            break;                             // nothing left in any token
        }
        first = j == 0 ? best : first;
        // the lowest expert with it
        int mine = 0x7fffffff;
#pragma unroll
        for (int i = NL - 1; i >= 0; --i) {
            mine = l[i] == best ? i * LANES + i0 : mine;
        }
        const int chosen = lanes_min<LANES>(mine);
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            l[i] = i * LANES + i0 == chosen ? kNone : l[i];
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const bool here = j == c * LANES + i0 && best != kNone;
            id[c] = here ? chosen : id[c];
            weight[c] = here ? best : weight[c];
        }
    }
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        weight[c] = id[c] < 0 ? 0.f : weight[c] == first ? 1.f : expf(weight[c] - first);
        sum += weight[c];
    }
    if (a.renorm) {
        all = lanes_sum<LANES>(sum);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        weight[c] = id[c] < 0 ? 0.f : weight[c] / all;
    }
}

// Few slots: routing and grouping in one workgroup.  NL 0: the ids are given.
// slots <= kFewSlots.
template <int LANES, int NL>
__global__ void __launch_bounds__(kPlaceThreads)
group_few_kernel(RouteArgs a)
{
    __shared__ __align__(16) int ids[kFewSlots];
    const int tid = threadIdx.x;
    const int slots = a.slots;
    for (int i = slots + tid; i < kFewSlots; i += kPlaceThreads) {
        ids[i] = 0x7fffffff;                   // sorts behind everything
    }
    if constexpr (NL > 0) {
        constexpr int kTokens = 64 / LANES;    // per wave
        const int lane = tid & 63;
        for (int t0 = (tid >> 6) * kTokens; t0 < a.m; t0 += kPlaceWaves * kTokens) {
            int id[kChoices<LANES>];
            float weight[kChoices<LANES>], l[NL];
            load_logits<LANES, NL>(a, t0, a.m, l);
            route_tokens<LANES, NL>(a, l, id, weight);
            const int t = t0 + lane / LANES;
#pragma unroll
            for (int c = 0; c < kChoices<LANES>; ++c) {
                const int j = c * LANES + lane % LANES;
                if (t < a.m && j < a.topk) {
                    const int s = t * a.topk + j;
                    a.ids[s] = id[c];
                    a.weights[s] = weight[c];
                    ids[s] = id[c] < 0 ? 0x7fffffff : id[c];
                }
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
// With NL > 0 it routes the chunk's tokens first.
template <int LANES, int NL>
__global__ void __launch_bounds__(kCountThreads)
group_count_kernel(RouteArgs a)
{
    extern __shared__ int hist[];
    const int tid = threadIdx.x;
    for (int g = tid; g < a.groups; g += kCountThreads) {
        hist[g] = 0;
    }
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * a.chunk;
    const int64_t hi = min(lo + a.chunk, (int64_t)a.slots);
    if constexpr (NL > 0) {
        constexpr int kTokens = 64 / LANES;    // per wave
        constexpr int kPass = kCountThreads / LANES;
        const int lane = tid & 63;
        const int64_t last = hi / a.topk;      // a chunk holds whole tokens
        int64_t t0 = lo / a.topk + (tid >> 6) * kTokens;
        float next[NL];
        load_logits<LANES, NL>(a, t0, last, next);
        for (; t0 < last; t0 += kPass) {
            int id[kChoices<LANES>];
            float weight[kChoices<LANES>], l[NL];
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                l[i] = next[i];
            }
            load_logits<LANES, NL>(a, t0 + kPass, last, next);     // on the way
            route_tokens<LANES, NL>(a, l, id, weight);
            const int64_t t = t0 + lane / LANES;
#pragma unroll
            for (int c = 0; c < kChoices<LANES>; ++c) {
                const int j = c * LANES + lane % LANES;
                if (t < last && j < a.topk) {
                    a.ids[t * a.topk + j] = id[c];
                    a.weights[t * a.topk + j] = weight[c];
                    if (id[c] >= 0) {
                        atomicAdd(&hist[id[c]], 1);
                    }
                }
            }
        }
    } else {
        for (int64_t i = lo + tid; i < hi; i += kCountThreads) {
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
    for (int g = tid; g < a.groups; g += kCountThreads) {
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
            const int upto = wave_scan_add(v);
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
            // always, unless another call writes the workspace or the ids meanwhile
            if ((uint32_t)(at + rank) < (uint32_t)a.slots) {
                a.order[at + rank] = (int)i;
            }
            // every peer has read `at` (one wave, in lockstep); the last moves it on
            __builtin_amdgcn_wave_barrier();
            if ((peers >> lane) == 1) {
                mine[id] = at + rank + 1;
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
    // the tail: slots in no group
    for (int64_t i = max(begin[G], 0) + (int64_t)c * kPlaceThreads + tid; i < a.slots;
         i += (int64_t)a.chunks * kPlaceThreads) {
        a.order[i] = -1;
    }
}

// out[t][c] = residual[t][c] + sum_j weights[t][j] y[t * topk + j][c], over
// the choices with an id (f32, in the order of j).  A thread owns V consecutive
// columns of one token; with V = 4 (n >= 4) a row's last ones read the row's last
// four and write what is theirs.  Rows of any n begin on any element: the accesses
// ask for an element's alignment only (4096 tokens, topk 2, n = 4095, residual: one
// column a thread 88 us, four 48 us).
typedef float f4u_t __attribute__((ext_vector_type(4), aligned(4)));

template <int V>
__global__ void __launch_bounds__(256)
combine_kernel(CombineArgs a)
{
    const int64_t t = blockIdx.x / a.parts;
    const int c = ((int)(blockIdx.x % a.parts) * (int)blockDim.x + (int)threadIdx.x) * V;
    if (c >= a.n) {
        return;
    }
    const int from = min(c, a.n - V);
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        acc[i] = 0.f;
    }
    const float* y = a.y + t * a.topk * a.n + from;
#pragma unroll 4
    for (int j = 0; j < a.topk; ++j) {
        const float w = a.weights[t * a.topk + j];
        if (a.ids != nullptr && a.ids[t * a.topk + j] < 0) {
            continue;                          // no expert: its row was not written
        }
        const float* p = y + (int64_t)j * a.n;
        if constexpr (V == 4) {
            const f4u_t v = *reinterpret_cast<const f4u_t*>(p);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                acc[i] = __builtin_fmaf(w, v[i], acc[i]);
            }
        } else {
            acc[0] = __builtin_fmaf(w, p[0], acc[0]);
        }
    }
    float* const out = a.out + t * a.n + from;
    if constexpr (V == 4) {
        f4u_t r = {acc[0], acc[1], acc[2], acc[3]};
        if (a.residual != nullptr) {
            r += *reinterpret_cast<const f4u_t*>(a.residual + t * a.n + from);
        }
        if (from == c) {
            *reinterpret_cast<f4u_t*>(out) = r;
        } else {
            // out may be residual: the elements before c are another thread's
#pragma unroll
            for (int i = 1; i < V; ++i) {
                if (from + i >= c) {
                    out[i] = r[i];
                }
            }
        }
    } else {
        if (a.residual != nullptr) {
            acc[0] += a.residual[t * a.n + c];
        }
        out[0] = acc[0];
    }
}

// Slots per chunk: whole tokens, about 256 chunks (each placing workgroup
// adds up all chunks' counts), and at least 64 slots.  8192 tokens of 128
// experts, topk 8, with 128 / 256 / 512 chunks: 14.4 / 12.4 / 18.2 us.
constexpr int64_t kChunks = 256;
constexpr int64_t kChunkSlots = 64;

int64_t chunk_slots(int64_t slots, int64_t topk)
{
    int64_t c = (slots + kChunks - 1) / kChunks;
    c = c < kChunkSlots ? kChunkSlots : c;
    return (c + topk - 1) / topk * topk;
}

size_t place_lds(int groups)
{
    return sizeof(int) * ((size_t)(kPlaceWaves + 1) * groups + 1 + 2 * kPlaceThreads);
}

template <int LANES, int NL>
hipError_t launch_route_t(RouteArgs a, hipStream_t stream)
{
    if (group_in_one(a.slots, a.groups, a.topk, NL > 0)) {
        hipLaunchKernelGGL((group_few_kernel<LANES, NL>), dim3(1), dim3(kPlaceThreads), 0, stream,
                           a);
        return hipGetLastError();
    }
    a.chunk = chunk_slots(a.slots, a.topk);
    a.chunks = (int)((a.slots + a.chunk - 1) / a.chunk);
    if (a.offsets == nullptr) {
        a.counts = nullptr;
    }
    hipLaunchKernelGGL((group_count_kernel<LANES, NL>), dim3(a.chunks), dim3(kCountThreads),
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

// Whether one workgroup does it all: few enough slots to count each place
// directly (the work is their square), and (routing) the tokens in a pass or two
// of its waves.  One workgroup against two launches over the chip, a call: 64
// slots 5.8 / 8.5 us, 192 slots 7.5 / 8.6 us, 256 slots 9.3 / 8.6 us; routing, topk
// 8: 8 tokens of 64 experts 6.7 / 9.4 us, 24 tokens 9.9 / 9.8 us, 64 tokens 23 /
// 10 us, 8 tokens of 512 experts 7.5 / 10 us, 30 tokens 21 / 11 us.
bool group_in_one(int64_t slots, int64_t groups, int64_t topk, bool route)
{
    const int64_t tokens = groups <= kRowExperts ? 2 * kPlaceThreads / 16 : kPlaceThreads / 64;
    return slots <= kFewSlots && (!route || slots <= tokens * topk);
}

size_t group_ws_bytes(int64_t slots, int64_t groups, int64_t topk, bool route)
{
    if (group_in_one(slots, groups, topk, route)) {
        return 0;
    }
    const int64_t chunk = chunk_slots(slots, topk);
    return sizeof(int) * (size_t)((slots + chunk - 1) / chunk) * (size_t)groups;
}

// The most that `slots` slots or fewer take: the chunks of the rule above, without
// its rounding (16385 slots are 253 chunks of 65, 16384 are 256 of 64).
size_t group_ws_most(int64_t slots, int64_t groups, int64_t topk)
{
    if (group_in_one(slots, groups, topk, true)) {
        return 0;                          // routing takes more than grouping
    }
    const int64_t chunks = (slots + kChunkSlots - 1) / kChunkSlots;
    return sizeof(int) * (size_t)(chunks < kChunks ? chunks : kChunks) * (size_t)groups;
}

hipError_t launch_route(const RouteArgs& a, hipStream_t stream)
{
    if (a.logits == nullptr) {
        return launch_route_t<64, 0>(a, stream);
    }
    if (a.groups <= 32) {
        return launch_route_t<16, 2>(a, stream);
    }
    if (a.groups <= 64) {
        return launch_route_t<16, 4>(a, stream);
    }
    if (a.groups <= 128) {
        return launch_route_t<16, 8>(a, stream);
    }
    if (a.groups <= kRowExperts) {
        return launch_route_t<16, 16>(a, stream);
    }
    if (a.groups <= 512) {
        return launch_route_t<64, 8>(a, stream);
    }
    return launch_route_t<64, 16>(a, stream);
}

hipError_t launch_combine(CombineArgs a, hipStream_t stream)
{
    const int v = a.n >= 4 ? 4 : 1;
    const int pieces = (a.n + v - 1) / v;
    const int threads = pieces < 256 ? (pieces + 63) / 64 * 64 : 256;
    a.parts = (pieces + threads - 1) / threads;
    const dim3 grid((unsigned)((int64_t)a.m * a.parts));
    if (v == 4) {
        hipLaunchKernelGGL(combine_kernel<4>, grid, dim3(threads), 0, stream, a);
    } else {
        hipLaunchKernelGGL(combine_kernel<1>, grid, dim3(threads), 0, stream, a);
    }
    return hipGetLastError();
}

}  // namespace q4k
