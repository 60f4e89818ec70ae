// qmm_experts.h -- launch interfaces and kernel parameters of the experts'
// feed-forward network (qmm_experts.cu, qmm_experts_kernel.cuh) and of the
// choice of experts (qmm_route.cu), called by qmm_experts_api.cu.
#pragma once

#include "qmm_internal.h"

namespace qmm {

struct Route {
    const float *logits;
    int64_t logits_stride;
    int32_t *ids;
    float *weights;
    int64_t n_pos;
    int n_experts, top_k;
    int score;       // 0 softmax, 1 logistic
    bool normalize;
    float scale;
};
cudaError_t launch_route(const Route &r, const DeviceInfo &dev, cudaStream_t s);

constexpr int kMaxExperts = 4096, kMaxTopK = 64;
constexpr int64_t kMaxPairs = 65535;

struct ExpertsFfn {
    int act;                 // 1 SwiGLU, 2 GeGLU
    int fmt, fmt_down;
    const uint8_t *gate, *up, *down;
    int64_t row_bytes, down_row_bytes;
    const float *x;          // [n_pos][k]
    const int32_t *ids;      // [n_pos][top_k]
    const float *weights;    // [n_pos][top_k]
    float *y;                // [n_pos][k]
    int64_t n_pos;
    int k, n_ff, n_experts, top_k;
    bool accumulate;
    void *workspace;         // >= experts_ffn_workspace_bytes
};
size_t experts_ffn_workspace_bytes(const ExpertsFfn &f);
cudaError_t launch_experts_ffn(const ExpertsFfn &f, const DeviceInfo &dev, cudaStream_t s);

namespace experts {

// Rows of one expert that a CTA multiplies at a time.
struct Tile {
    int expert;
    int start, count;  // of the pairs in expert order
    int pad;
};

// One of the two products over the tiles.
struct ProductParams {
    const uint8_t *w[2];     // gate and up, or down (twice)
    int64_t slice_bytes, row_bytes;
    int rows;                // of a slice
    int k, blocks;           // contraction length, and its blocks of 32
    const uint8_t *x;        // activations as terms: [row][padded blocks][frag_bytes]; single rows: records (see put_record)
    const float *x_scale, *x_sum; // [row][padded blocks] (see put_terms)
    int64_t x_row_bytes;
    int x_blocks;            // padded blocks of a row
    const Tile *tiles;
    const int *n_tiles;
    const int *order;        // pairs in expert order
    int top_k;
    // first product: act(gate) up times the pair's weight, as terms (records) for the second
    const float *weights;
    uint8_t *h;
    float *h_scale, *h_sum;
    int64_t h_row_bytes;
    int h_blocks;            // padded
    int h_fmt, act;
    // second product
    float *out;              // [pair][rows]; row by row: y
    // row by row (see qmm_experts_rows.cuh)
    int slices;              // set by the launch
    int n_pos;
    const float *x32;        // one position: x
    const int32_t *ids;
    int n_experts, accumulate;
    unsigned int *err;
};

// columns (activation rows) of a tile: 8 or 16
template <int FMT>
cudaError_t launch_product(bool down, int columns, const ProductParams &p, int max_tiles, const DeviceInfo &dev, cudaStream_t s);
// tiles of 48 (see qmm_experts_tile.cuh): x: terms of rows under one power of two each; h: fp32
template <int FMT>
cudaError_t launch_tile(bool down, const ProductParams &p, int max_tiles, const DeviceInfo &dev, cudaStream_t s);
// row by row
template <int FMT>
cudaError_t launch_single(bool down, const ProductParams &p, const DeviceInfo &dev, cudaStream_t s);

}  // namespace experts
}  // namespace qmm
