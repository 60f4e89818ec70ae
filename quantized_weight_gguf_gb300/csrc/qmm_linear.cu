// qmm_linear.cu -- linear attention with a decay for each head, row by row:
//     S_t = e^(g_t) S_(t-1) + k_t v_t^T,   o_t = scale S_t^T q_t,
// and the choice between this kernel and the one for prompts.
//
// A CTA keeps 32 columns (dims of v) of a head's state in registers: 16 rows
// of the state at a time are one float4 per thread, 128 bytes a row. The state
// is read and written once, 8 bytes per element and call against 4 flops a
// row: bound by memory. 32 columns, so that one sequence of 32 heads makes 128
// CTAs, and 16 CTAs a SM have 256 KB of state on their way. Measured: 64 sequences of 32 heads of 128 / 128
// 46 us, 0.87 of the copy rate; one sequence 2.9 us, a launch and two trips to memory.
#include "qmm_device.cuh"
#include "qmm_linear.h"

namespace qmm {

namespace linear {

namespace {

constexpr int kStepThreads = 128, kStepCols = 32;
constexpr int kStepRows = kStepThreads / (kStepCols / 4);  // rows of the state in one pass

template <int DK>
__global__ void __launch_bounds__(kStepThreads) step_kernel(const __grid_constant__ Linear l) {
    constexpr int N = DK / kStepRows;
    __shared__ float4 part[kStepThreads / 32][kStepCols / 4];
    pdl_wait_prev();
    pdl_launch_dependents();
    const int tiles = l.dv / kStepCols;
    const int tile = blockIdx.x % tiles, head = blockIdx.x / tiles % l.n_heads, seq = blockIdx.x / tiles / l.n_heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int col = tile * kStepCols + 4 * (tid & 7), row = tid >> 3;
    const int64_t at = ((int64_t)seq * l.n_heads + head) * DK * l.dv + col;
    const Span span = span_of(l, seq);

    float4 s[N];
    if (span.begins && !span.idle) {
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = make_float4(0, 0, 0, 0);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            s[i] = *reinterpret_cast<const float4 *>(l.state + at + (int64_t)(row + i * kStepRows) * l.dv);
    }
    const int qk = head / (l.n_heads / l.n_qk) * DK + row;
    for (int64_t r = 0; r < l.n_new; ++r) {
        const int64_t x = seq * l.n_new + r;
        float4 o = make_float4(0, 0, 0, 0);
        if (r >= span.first) {
            const float a = expf(decay_of(l.decay[x * l.decay_stride + head]));
            const float *vp = l.v + x * l.v_stride + head * l.dv + col;
            const float4 v = l.vec ? *reinterpret_cast<const float4 *>(vp) : make_float4(vp[0], vp[1], vp[2], vp[3]);
            const float *kp = l.k + x * l.k_stride + qk, *qp = l.q + x * l.q_stride + qk;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float k = kp[i * kStepRows], q = qp[i * kStepRows];
                s[i].x = fmaf(s[i].x, a, k * v.x);
                s[i].y = fmaf(s[i].y, a, k * v.y);
                s[i].z = fmaf(s[i].z, a, k * v.z);
                s[i].w = fmaf(s[i].w, a, k * v.w);
                o.x = fmaf(q, s[i].x, o.x);
                o.y = fmaf(q, s[i].y, o.y);
                o.z = fmaf(q, s[i].z, o.z);
                o.w = fmaf(q, s[i].w, o.w);
            }
        }
        // the sum over the rows of the state: four of a warp, then the warps
#pragma unroll
        for (int d = 8; d < 32; d <<= 1) {
            o.x += __shfl_xor_sync(~0u, o.x, d);
            o.y += __shfl_xor_sync(~0u, o.y, d);
            o.z += __shfl_xor_sync(~0u, o.z, d);
            o.w += __shfl_xor_sync(~0u, o.w, d);
        }
        if (r) __syncthreads();  // the row before has been taken
        if (lane < kStepCols / 4) part[warp][lane] = o;
        __syncthreads();
        if (tid < kStepCols) {
            const float *p = reinterpret_cast<const float *>(part) + tid;
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kStepThreads / 32; ++w) sum += p[w * kStepCols];
            l.out[x * l.out_stride + head * l.dv + tile * kStepCols + tid] = r >= span.first ? sum * l.scale : 0.0f;
        }
    }
    if (span.idle && l.state_out == l.state) return;
#pragma unroll
    for (int i = 0; i < N; ++i)
        *reinterpret_cast<float4 *>(l.state_out + at + (int64_t)(row + i * kStepRows) * l.dv) = s[i];
}

template <int DK>
cudaError_t launch_step(const Linear &l, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((int64_t)l.n_seqs * l.n_heads * (l.dv / kStepCols)));
    cfg.blockDim = dim3(kStepThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, step_kernel<DK>, l);
}

// Rows per sequence up to which they are taken one by one.
constexpr int64_t kStepMaxRows = 8;

Split split_of(const Linear &l, const DeviceInfo &dev) {
    Split s;
    s.tiles = l.dv > 128 ? 2 : 1;
    s.tile = l.dv / s.tiles;
    // Segments fill one wave of two CTAs a SM where sequences and heads alone
    // leave more than a third of it idle (the segments' own states are a pass of
    // about two fifths of the work more).
    const int64_t ctas = (int64_t)l.n_seqs * l.n_heads * s.tiles, wave = 2 * dev.sm_count;
    int64_t n = 3 * ctas > 2 * wave ? 1 : wave / ctas;
    const int64_t most = l.n_new / (4 * kChunk);
    if (n > most) n = most;
    if (n < 1) n = 1;
    const int64_t chunks = (l.n_new + kChunk - 1) / kChunk, per = (chunks + n - 1) / n;
    s.rows = per * kChunk;
    s.segments = (int)((chunks + per - 1) / per);
    return s;
}

}  // namespace

}  // namespace linear

bool linear_supports(int64_t dk, int64_t dv) {
    return dk >= 32 && dk <= 128 && dk % 32 == 0 && dv >= 32 && dv <= 256 && dv % 32 == 0;
}

size_t linear_workspace_bytes(const Linear &l, const DeviceInfo &dev) {
    if (l.n_new <= linear::kStepMaxRows) return 0;
    return linear::chunks_workspace_bytes(l, linear::split_of(l, dev));
}

cudaError_t launch_linear(const Linear &l, const DeviceInfo &dev, cudaStream_t s) {
    if (l.n_new > linear::kStepMaxRows) return linear::launch_chunks(l, linear::split_of(l, dev), dev, s);
    switch (l.dk) {
    case 32: return linear::launch_step<32>(l, s);
    case 64: return linear::launch_step<64>(l, s);
    case 96: return linear::launch_step<96>(l, s);
    case 128: return linear::launch_step<128>(l, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace qmm
