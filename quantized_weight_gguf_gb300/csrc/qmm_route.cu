// qmm_route.cu -- the choice of a position's experts from the router's logits:
// the top_k largest, ties to the lowest index, and their weights.
//
// One warp per row. Logits become integers of the same order, so that a choice
// is two warp reductions (the largest, then the lowest index that has it); the
// row stays in registers up to 512 experts. Every round looks at all of a lane's keys again: bound by instructions
// where rows are many (8 of 256 experts: 980 of a warp a row; issue slots 60 % used, ALU 66 %), by the launch where
// they are few. Measured: one row 2.3 us, 4099 rows of 256 experts 6.0 us in a stream of such calls.
#include <cmath>

#include "qmm_device.cuh"
#include "qmm_experts.h"

namespace qmm {

namespace {

constexpr int kRouteWarps = 4;

// Larger logits give larger keys; 0 (below all): -Inf and NaN, which are never chosen.
__device__ __forceinline__ uint32_t key_of(float v) {
    if (!(v > -INFINITY)) return 0;
    const uint32_t b = __float_as_uint(v + 0.0f);  // -0 equals 0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// log of the logistic function
__device__ __forceinline__ float log_logistic(float v) { return fminf(v, 0.0f) - log1pf(expf(-fabsf(v))); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// N: experts per lane held in registers; 0: any number, read again in every round.
template <int N>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const __grid_constant__ Route r) {
    pdl_wait_prev();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
    if (row >= r.n_pos) return;
    const float *logits = r.logits + row * r.logits_stride;
    uint32_t keys[N ? N : 1];
    bool nan = false;
    if constexpr (N > 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = 32 * i + lane;
            const float v = e < r.n_experts ? logits[e] : -INFINITY;
            nan |= v != v;
            keys[i] = key_of(v);
        }
    } else {
        for (int e = lane; e < r.n_experts; e += 32) nan |= logits[e] != logits[e];
    }
    nan = __any_sync(~0u, nan);

    uint32_t chosen[2] = {0, 0};   // of slots lane and lane + 32
    int ids[2] = {-1, -1};
    uint32_t last = 0xFFFFFFFFu;   // the round before: its key and index
    int last_id = -1;
    float total = 0.0f;            // softmax over all: sum of exp(logit - largest)
    for (int s = 0; s < r.top_k; ++s) {
        uint32_t best = 0;
        int at = INT32_MAX;
        if constexpr (N > 0) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (keys[i] > best) {
                    best = keys[i];
                    at = 32 * i + lane;
                }
        } else {
            for (int e = lane; e < r.n_experts; e += 32) {
                const uint32_t k = key_of(logits[e]);
                if (k > best && (k < last || (k == last && e > last_id))) {
                    best = k;
                    at = e;
                }
            }
        }
        const uint32_t top = __reduce_max_sync(~0u, best);
        if (top == 0) break;
        const int id = __reduce_min_sync(~0u, best == top ? at : INT32_MAX);
        if (s == 0 && r.score == 0 && !r.normalize) {
            const float m = logit_of(top);
            if constexpr (N > 0) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (keys[i]) total += expf(logit_of(keys[i]) - m);
            } else {
                for (int e = lane; e < r.n_experts; e += 32)
                    if (logits[e] > -INFINITY) total += expf(logits[e] - m);
            }
            total = warp_sum(total);
        }
        if constexpr (N > 0) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (32 * i + lane == id) keys[i] = 0;
        }
        last = top;
        last_id = id;
        if (lane == (s & 31)) {
            chosen[s >> 5] = top;
            ids[s >> 5] = id;
        }
    }

    // the first slot holds the largest
    const float m = logit_of(__shfl_sync(~0u, chosen[0], 0));
    const float base = r.score == 0 ? m : log_logistic(m);
    float w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float v = logit_of(chosen[i]);
        const float l = r.score == 0 ? v : log_logistic(v);
        w[i] = ids[i] < 0 ? 0.0f : expf(r.score == 0 || r.normalize ? l - base : l);
    }
    if (r.normalize) total = warp_sum(w[0] + w[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int s = lane + 32 * i;
        if (s >= r.top_k) break;
        float v = r.score == 0 || r.normalize ? w[i] / total : w[i];
        if (nan) v = NAN;
        r.ids[row * r.top_k + s] = ids[i];
        r.weights[row * r.top_k + s] = ids[i] < 0 ? 0.0f : v * r.scale;
    }
}

template <int N>
cudaError_t launch(const Route &r, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((r.n_pos + kRouteWarps - 1) / kRouteWarps));
    cfg.blockDim = dim3(kRouteWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, route_kernel<N>, r);
}

}  // namespace

cudaError_t launch_route(const Route &r, const DeviceInfo &, cudaStream_t s) {
    if (r.n_experts <= 64) return launch<2>(r, s);
    if (r.n_experts <= 128) return launch<4>(r, s);
    if (r.n_experts <= 256) return launch<8>(r, s);
    if (r.n_experts <= 512) return launch<16>(r, s);
    return launch<0>(r, s);
}

}  // namespace qmm
