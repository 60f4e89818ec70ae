// qmm_linear.h -- launch interface of linear attention (qmm_linear.cu,
// qmm_linear_chunk.cu), called by qmm_linear_api.cu.
#pragma once

#include "qmm_internal.h"

namespace qmm {

struct Linear {
    const float *q, *k, *v;      // row r of sequence s at row s * n_new + r
    const float *decay;          // [rows][n_heads], or [n_heads]
    const float *state;          // [n_seqs][n_heads][dk][dv]
    float *state_out, *out;
    const int32_t *lens;         // NULL: every row is a position and no sequence begins here
    int64_t q_stride, k_stride, v_stride, out_stride, decay_stride;  // decay_stride 0: one decay per head
    int64_t n_new;
    int n_seqs, n_heads, n_qk, dk, dv;
    float scale;
    bool vec;                    // rows of q, k and v start on 16-byte boundaries
    void *workspace;
};
// dims that the kernels take: dk 32, 64, 96 or 128, dv a multiple of 32 up to 256
bool linear_supports(int64_t dk, int64_t dv);
size_t linear_workspace_bytes(const Linear &l, const DeviceInfo &dev);
cudaError_t launch_linear(const Linear &l, const DeviceInfo &dev, cudaStream_t s);

namespace linear {

// How a prompt is divided: `segments` runs of `rows` rows, each a CTA's work per
// sequence, head and tile of dv.
struct Split {
    int tiles, tile;     // of dv
    int segments;
    int64_t rows;        // a multiple of kChunk
};
constexpr int kChunk = 32;

// Rows of a call that belong to a sequence: [first, n_new), and whether it
// starts from a state of zeros; idle: it has no position at all.
struct Span {
    int64_t first;
    bool begins, idle;
};
__device__ __forceinline__ Span span_of(const Linear &l, int seq) {
    Span s = {0, false, false};
    if (l.lens) {
        const int64_t n = l.lens[seq];
        s.idle = n <= 0;
        s.begins = n <= l.n_new;
        s.first = s.idle ? l.n_new : n < l.n_new ? l.n_new - n : 0;
    }
    return s;
}
// A decay as the kernels take it: at most 0 (a factor of 1), and at least
// -110, whose factor fp32 holds as 0 (so that sums with -Inf stay numbers). NaN stays.
__device__ __forceinline__ float decay_of(float g) {
    g = g > 0.0f ? 0.0f : g;
    return g < -110.0f ? -110.0f : g;
}

cudaError_t launch_chunks(const Linear &l, const Split &split, const DeviceInfo &dev, cudaStream_t s);
size_t chunks_workspace_bytes(const Linear &l, const Split &split);

}  // namespace linear

}  // namespace qmm
