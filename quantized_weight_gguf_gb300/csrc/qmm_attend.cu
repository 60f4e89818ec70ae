// qmm_attend.cu -- attention of new rows over the paged key-value cache.
//
// o = sum_t softmax_t(scale q . k_t) v_t. One CTA per (row, head): each warp
// takes every fourth position, its lanes four dims each, and keeps a running
// maximum m, total l = sum e^(s - m) and sum of e^(s - m) v in fp32; the four
// warps' results are joined in a fixed order at the end.
#include "qmm_kv.cuh"
#include "qmm_kv_launch.h"

namespace qmm {

namespace {

constexpr int kWarps = 4;

__global__ void __launch_bounds__(kWarps * 32) attend_kernel(const Attend a) {
    pdl_wait_prev();
    __shared__ float sm[kWarps], sl[kWarps], so[kWarps][256];
    const KvView &c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = blockIdx.x / a.n_heads;
    const int head = (int)(blockIdx.x - row * a.n_heads);
    const int h = head / (a.n_heads / c.n_kv);
    const int s = (int)(row / a.n_new);
    const int len = kv_length(c, s);
    const int64_t pos = (int64_t)max(__ldg(c.lens + s), 0) - a.n_new + (row - s * a.n_new);
    const int64_t lo = a.window && pos + 1 > a.window ? pos + 1 - a.window : 0;
    const int64_t hi = pos + 1 < len ? pos + 1 : len;
    float q[8], o[8];
    const float *qr = a.q + row * a.q_stride + (int64_t)head * c.dim;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int d = (i >> 2) * 128 + lane * 4 + (i & 3);
        q[i] = d < c.dim ? qr[d] * a.scale : 0.0f;
        o[i] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    for (int64_t t = lo + warp; t < hi; t += kWarps) {
        const uint8_t *strip = kv_strip(c, s, h, (int)(t / kStrip));
        if (!strip) continue;
        const int tt = (int)(t % kStrip);
        float v[8], x = 0.0f;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int d = g * 128 + lane * 4;
            float4 kk = make_float4(0.f, 0.f, 0.f, 0.f), vv = kk;
            if (d < c.dim) {
                kk = kv_load4(strip, c.fmt_k, c.dim, tt, d);
                vv = kv_load4(strip + c.v_off, c.fmt_v, c.dim, tt, d);
            }
            x += q[4 * g] * kk.x + q[4 * g + 1] * kk.y + q[4 * g + 2] * kk.z + q[4 * g + 3] * kk.w;
            v[4 * g] = vv.x; v[4 * g + 1] = vv.y; v[4 * g + 2] = vv.z; v[4 * g + 3] = vv.w;
        }
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) x += __shfl_xor_sync(~0u, x, i);
        const float mn = fmaxf(m, x);
        const float f = expf(m - mn), p = expf(x - mn);
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = o[i] * f + p * v[i];
        m = mn;
    }
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) so[warp][(i >> 2) * 128 + lane * 4 + (i & 3)] = o[i];
    __syncthreads();
    float mm = -INFINITY, ll = 0.0f;
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm[w]);
    float f[kWarps];
    for (int w = 0; w < kWarps; ++w) {
        f[w] = sm[w] == -INFINITY ? 0.0f : expf(sm[w] - mm);
        ll += f[w] * sl[w];
    }
    float *out = a.out + row * a.out_stride + (int64_t)head * c.dim;
    for (int d = threadIdx.x; d < c.dim; d += kWarps * 32) {
        float r = 0.0f;
        for (int w = 0; w < kWarps; ++w) r += f[w] * so[w][d];
        out[d] = ll > 0.0f ? r / ll : mm != mm || ll != ll ? NAN : 0.0f;
    }
}

}  // namespace

bool attend_supports(int dim) {
    return dim == 64 || dim == 96 || dim == 128 || dim == 192 || dim == 256;
}

size_t attend_workspace_bytes(const Attend &, const DeviceInfo &) { return 0; }

cudaError_t launch_attend(const Attend &a, const DeviceInfo &, cudaStream_t s) {
    const int64_t grid = (int64_t)a.c.n_seqs * a.n_new * a.n_heads;
    if (grid == 0) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attend_kernel, a);
}

}  // namespace qmm
