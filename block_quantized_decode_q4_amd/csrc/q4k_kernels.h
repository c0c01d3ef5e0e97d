// q4k_kernels.h -- internal interface between the C-ABI layer (q4k_api.hip)
// and the kernels (q4k_kernels.hip, q4k_dpp.hip, q4k_mfma.hip, q4k_q8.hip,
// q4k_q6k.hip, q4k_f16.hip).  Not installed, not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace q4k {

constexpr int kQK = 256;          // weights per superblock
constexpr int kBlockBytes = 144;  // bytes per superblock
constexpr int kSpanSB = 16;       // superblocks per wave pass (4 lanes each)
constexpr int kSpan = kSpanSB * kQK;
constexpr int kMaxM = 8;         // vectors per launch that every kernel takes
constexpr int kMaxMStaged = 16;  // kernels 5 and 7: x of at most four vector quads in LDS
constexpr int kMaxMWide = 32;    // kernel 6 (eight quads, x per wave and column)
constexpr int kReadBlocks = 1024;    // four 512-lane workgroups per CU of a 256-CU part
constexpr int kReadThreads = 512;

// One resolved launch of the GEMV kernel.
struct GemvPlan {
    int n, k, S, m;
    int nspans;            // ceil(S / 16)
    int spans_per_chunk;   // spans of x staged at once (== nspans: single-stage)
    int nchunks;
    int rows_per_block;
    int rows_per_wave;     // R: 1, 2 or 4 (4 only for m = 1)
    int waves_per_block;   // 4 or 8
    int x_in_registers;    // 1: x kept in VGPRs (single span, m = 1)
    int grid;
    size_t lds_bytes;
    int kernel;            // 1: x-stager, 2: streaming, 3: line-streamed int8 dot products
                           // (vector ALU), 4: line-streamed int8 matrix-core,
                           // 5: sub-block int8 matrix-core, 6: the same with x
                           // converted per column by each wave
    int ring_depth;        // kernel 2: rows in flight per wave; 3-6: lines in flight
    int rows_per_task;     // streaming kernel: rows per wave task
    int cols_per_task;     // line-streamed kernels: superblock columns per task
};

hipError_t launch_gemv(const GemvPlan& p, const void* w, const float* x, float* y,
                       hipStream_t stream);
hipError_t launch_gemv_mfma(const GemvPlan& p, const void* w, const float* x, float* y,
                            hipStream_t stream);
size_t lines_lds_bytes(int S, int m, int waves);
size_t sub_lds_bytes(int S, int m);
size_t jit_lds_bytes(int S, int m);
int jit_waves(int m);      // waves per workgroup of kernel 6 for m vectors
size_t win_lds_bytes(int S, int m);
hipError_t launch_gemv_dot4(const GemvPlan& p, const void* w, const float* x, float* y,
                            hipStream_t stream);
size_t dot4_lds_bytes(int S, int waves);
hipError_t launch_dequant(const void* w, float* out, int64_t nsb, hipStream_t stream);
// the integer-dot variant with x quantized to Q8 (q4k_q8.hip)
hipError_t launch_gemv_q8(const GemvPlan& p, const void* w, const float* x, float* y,
                          hipStream_t stream);
hipError_t launch_quantize_q8(const float* x, int8_t* q, float* d, int64_t nblocks,
                              hipStream_t stream);
size_t q8_lds_bytes(int S, int waves);
hipError_t launch_read(const void* buf, size_t n16, float* out, hipStream_t stream);

// The GEMV over Q6_K weights (q4k_q6k.hip), one vector.
struct Q6kPlan {
    int n, k, S;
    int64_t row_stride;    // bytes from one row to the next (a multiple of 16)
    int unit;              // bytes of a row one load instruction reads: 64, or 128
                           // (whole lines; w 128-byte aligned)
    int batch;             // bytes of a row per batch: 256 (no row has a phase within
                           // its line: unit 64, or a row stride that is a multiple
                           // of 128) or 128
    int waves_per_block;   // 8, or 4 when the LDS cannot hold eight rings
    int rows_per_block;    // 16 per tile
    int ncg;               // column groups per tile (the tasks of one tile)
    int grid;
    size_t lds_bytes;
};
hipError_t launch_q6k_gemv(const Q6kPlan& p, const void* w, const float* x, float* y,
                           hipStream_t stream);
hipError_t launch_q6k_dequant(const void* w, float* out, int64_t n, int S, int64_t row_stride,
                              hipStream_t stream);
size_t q6k_lds_bytes(int S, int waves, int rows_per_block, int ncg);

// The fp16 mirror and the prefill GEMM (q4k_f16.hip; mirror builds in
// q4k_kernels.hip and q4k_q6k.hip).
hipError_t launch_dequant_f16(const void* w, void* out, int64_t nsb, hipStream_t stream);
hipError_t launch_q6k_dequant_f16(const void* w, void* out, int64_t n, int S, int64_t row_stride,
                                  hipStream_t stream);
hipError_t launch_f16_cvt(const float* x, void* out, int64_t count, hipStream_t stream);
hipError_t launch_f16_gemm(const void* w16, const void* x16, float* y, int m, int n, int k,
                           hipStream_t stream);
void f16_gemm_tile(int64_t m, int64_t n, int* bm, int* bn);
// the static scratch of q4k_f16_gemm_f32x_noalloc: 4 Mi halves (8 MiB) per
// device; f16_scratch gives its device address on the current device
constexpr int64_t kScratchHalves = (int64_t)4 << 20;
hipError_t f16_scratch(void** out);
size_t f16_gemm_lds_bytes(int bm, int bn);
int64_t f16_gemm_grid(int64_t m, int64_t n);

// The types of the activations that q4k_rmsnorm and q4k_lora take (enum
// q4k_type of include/q4k.h).
constexpr int kTypeF32 = 0;
constexpr int kTypeF16 = 1;
constexpr int kTypeBF16 = 2;

// The norm (q4k_norm.hip): m rows of k elements; any output may be null.
struct NormArgs {
    const void* x;
    const float* residual;
    const float* weight;
    float* sum;
    float* y;
    void* y16;
    int8_t* q;
    float* d;
    int64_t x_stride;
    int x_type, k, m;
    float eps;
};
hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t stream);

// Routing and grouping (q4k_moe.hip).  logits null: the ids are given.
constexpr int kFewSlots = 192;         // slots that one workgroup groups in one launch
constexpr int kMaxGroups = 1024;       // experts (ids) that routing and grouping take
constexpr int kMaxTopk = 32;
struct RouteArgs {
    const float* logits;
    int* ids;
    float* weights;
    int* offsets;                      // null: no grouping
    int* order;
    int* counts;                       // chunks x groups (workspace)
    int64_t stride;                    // floats from one token's logits to the next
    int64_t chunk;                     // slots per chunk (set by the launch)
    int chunks;
    int m, groups, topk, renorm;
    int slots;                         // m * topk
};
hipError_t launch_route(const RouteArgs& a, hipStream_t stream);
constexpr int kRowExperts = 256;       // experts that 16 lanes route
bool group_in_one(int64_t slots, int64_t groups, int64_t topk, bool route);
size_t group_ws_bytes(int64_t slots, int64_t groups, int64_t topk, bool route);
size_t group_ws_most(int64_t slots, int64_t groups, int64_t topk);       // or fewer slots

struct CombineArgs {
    const float* y;
    const float* weights;
    const int* ids;                    // null: every slot counts
    const float* residual;             // may be null
    float* out;
    int n, topk, m;
    int parts;                         // workgroups per token (set by the launch)
};
hipError_t launch_combine(CombineArgs a, hipStream_t stream);

// Rows grouped by a matrix: position i (offsets[g] <= i < offsets[g + 1])
// takes x row (x_rows ? x_rows[i] : i) / x_div and writes y row
// (y_rows ? y_rows[i] : i); a position whose row is outside 0 .. x_count - 1
// or 0 .. y_count - 1 is left out.
struct GroupRows {
    const int* offsets;
    const int* x_rows;
    const int* y_rows;
    int groups, rows;
    int x_div, x_count, y_count;
};

// Q4_K matrices (q4k_grouped.hip): x f32, or (x null) Q8 codes and scales.
struct GroupedArgs {
    const void* w;
    const float* x;
    const int8_t* q;
    const float* d;
    float* y;
    void* ws;
    GroupRows g;
    int n, k;
};
hipError_t launch_grouped(const GroupedArgs& a, hipStream_t stream);
size_t grouped_ws_bytes(int64_t k, int64_t rows);
int64_t grouped_grid(int64_t rows, int64_t groups, int64_t n, int64_t k);
constexpr int64_t kMaxGroupedK = (int64_t)1 << 24;   // 16 rows within 32-bit offsets

// The fp16 mirror (q4k_f16.hip).
hipError_t launch_f16_gemm_grouped(const void* w16, const void* x16, float* y, const GroupRows& g,
                                   int n, int k, hipStream_t stream);
int64_t f16_grouped_grid(int64_t rows, int64_t groups, int64_t n, int64_t k);

// Low-rank adapters (q4k_lora.hip).
struct LoraArgs {
    const void* x;
    const void* a;                     // adapters x r x k halves
    const void* b;                     // adapters x n x r halves
    const float* base;                 // null: y is overwritten with the product alone
    float* y;
    const int* ranks;                  // null: r
    const float* scales;               // null: 1
    const int* offsets;
    const int* order;                  // null: position i is row i
    float* v;                          // parts of k x rows x r up to 16s (workspace)
    int x_type, n, k, r, adapters, rows;
};
hipError_t launch_lora(const LoraArgs& a, hipStream_t stream);
size_t lora_ws_bytes(int64_t rows, int64_t r);
size_t lora_ws_most(int64_t rows, int64_t r);          // or fewer rows
bool lora_fits(int64_t rows, int64_t adapters, int64_t n, int64_t r);    // the launch limits

}  // namespace q4k
