// ops.cuh -- what the C entry points of the operators around the layer hand to
// their kernels: the norm with an 8-bit copy and the widening of 8-bit rows
// (rows.cu), the projection with low-rank adapters (project.cu), sampling
// (sample.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace ds4 {

constexpr int kQ8E4M3 = 0, kQ8Int8 = 1;

struct AddNormArgs {
    const void* x;        // [n][H]
    const void* res;      // [n][H] or nullptr
    const float* w;       // [H]
    void* sum;            // [n][H] of res's type, or nullptr
    void* out;            // [n][H] or nullptr
    uint8_t* q;           // [n][H] or nullptr
    float* scale;         // [n][groups]
    int64_t n;
    int H;
    int group;            // columns per scale (32, 64, 128), 0: the row
    int fmt;              // kQ8E4M3 or kQ8Int8
    int out_bf16;
    float eps, qmax;
    int warps_per_row;    // set by the launcher
    double inv_H;
};
cudaError_t launch_add_rmsnorm(AddNormArgs a, bool x_bf16, int res_kind, bool vec, int n_sm, cudaStream_t st);

cudaError_t launch_widen_rows(const uint8_t* q, int fmt, const float* scale, int group, int n, int H, void* out,
                              bool out_bf16, cudaStream_t st);

constexpr int kSampleMaxVocab = 1 << 18;

struct SampleArgs {
    const void* logits;   // [n] rows of V elements, ld elements apart
    int64_t ld;
    int V;
    const float* temp;    // [n] or nullptr (1)
    const int32_t* top_k; // [n] or nullptr (off)
    const float* top_p;   // [n] or nullptr (off)
    const float* min_p;   // [n] or nullptr (off)
    const float* u;       // [n]
    int32_t* token;       // [n]
    float* prob;          // [n] or nullptr
    float* probs;         // [n][V] or nullptr
    int slice, seg;       // tokens per CTA and per warp, set by the launcher
};
cudaError_t launch_sample(SampleArgs a, bool bf16, int n, int n_sm, cudaStream_t st);

struct ShrinkArgs {
    const __nv_bfloat16* x;     // [n][fin]
    const __nv_bfloat16* A;     // [n_adapters][rank][fin]
    const float* scale;         // [n_adapters]
    const int32_t* ids;         // [n]
    int n, fin, n_adapters, rank;
    int bn, cap, split;         // rows per tile, entries per tile, CTAs per 64 rows (set by the launcher)
    int32_t* counts;            // [tiles] distinct adapters of a tile
    int32_t* entry;             // [tiles][cap] their indices
    __nv_bfloat16* t;           // [tiles][cap][bn][2 * rank rounded to 16]
    float* rows;                // or, for a decode batch, t in binary32 [n][rank] (counts, entry, t: nullptr)
};
struct ProjectArgs {
    __nv_bfloat16* out;         // [n][fout]
    int n, fin, fout, rank;
    const int32_t* counts;      // as above, nullptr without adapters and for a decode batch
    const int32_t* entry;
    const float* rows;          // a decode batch's t
    const __nv_bfloat16* B;     // [n_adapters][fout][rank]
    const int32_t* ids;         // [n]
    int n_adapters;
    int in_time;                // tiles of each CTA (or pair) whose waits have their limit; those behind give up at once
    int bn, row_tiles, cap, kblocks, tiles, split, stages;   // set by the launcher
};
struct ProjectWork {            // layout of the caller's work buffer
    bool rows;                  // a decode batch: the adapters' second product outside the MMAs
    bool pair;                  // CTA pairs of 512 output features per tile; else 128
    int split;                  // CTAs that share a tile
    int bn, row_tiles, cap;     // rows per tile, tiles along the rows, entries per tile
    size_t off_entry, off_t, total;
};
ProjectWork project_work(int n, int fin, int fout, int n_adapters, int rank);
cudaError_t launch_project(ProjectArgs p, ShrinkArgs s, const ProjectWork& wk, const void* W, int n_sm, cudaStream_t st);
cudaError_t read_project_error(uint32_t* code, cudaStream_t st);

}  // namespace ds4
