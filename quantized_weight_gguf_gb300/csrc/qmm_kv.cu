// qmm_kv.cu -- appending to the paged key-value cache (rotary embedding of q
// and k, quantising write of k and v) and reading it back.
//
// Both kernels move each value once and do a few operations on it, so memory
// bounds them. A lane takes four dims, so that fp32 loads and stores are 16
// bytes wide; the 32 dims of a block are eight neighbouring lanes, so that its
// maximum takes three shuffles and its codes are one 32-byte sector.
#include "qmm_kv.cuh"
#include "qmm_kv_launch.h"

namespace qmm {

namespace {

constexpr int kKvThreads = 256;

__device__ __forceinline__ float4 load4(const float *p, bool vec) {
    return vec ? *reinterpret_cast<const float4 *>(p) : make_float4(p[0], p[1], p[2], p[3]);
}
__device__ __forceinline__ void store4(float *p, float4 v, bool vec) {
    if (vec) {
        *reinterpret_cast<float4 *>(p) = v;
    } else {
        p[0] = v.x; p[1] = v.y; p[2] = v.z; p[3] = v.w;
    }
}

// The rotation of dims d0 .. d0 + 3 of a head's row x, by the table row r of
// its position. Products and sums are rounded one by one (no fma), so the
// result does not depend on how a compiler contracts the formula.
__device__ __forceinline__ float4 rotate4(const float *x, float4 v, const float *r, int d0,
                                          int n_rot, int style, bool vec) {
    if (d0 >= n_rot) return v;
    if (style == 1) {  // pairs (2a, 2a + 1): both halves of a pair are in this lane
        const float4 cs = *reinterpret_cast<const float4 *>(r + d0);
        return make_float4(__fsub_rn(__fmul_rn(v.x, cs.x), __fmul_rn(v.y, cs.y)),
                           __fadd_rn(__fmul_rn(v.x, cs.y), __fmul_rn(v.y, cs.x)),
                           __fsub_rn(__fmul_rn(v.z, cs.z), __fmul_rn(v.w, cs.w)),
                           __fadd_rn(__fmul_rn(v.z, cs.w), __fmul_rn(v.w, cs.z)));
    }
    const int half = n_rot >> 1;
    const bool second = d0 >= half;
    const int a = second ? d0 - half : d0;
    const float4 o = load4(x + (second ? a : a + half), vec);
    const float4 c0 = *reinterpret_cast<const float4 *>(r + 2 * a);
    const float4 c1 = *reinterpret_cast<const float4 *>(r + 2 * a + 4);
    if (second)  // x1' = x0 s + x1 c
        return make_float4(__fadd_rn(__fmul_rn(o.x, c0.y), __fmul_rn(v.x, c0.x)),
                           __fadd_rn(__fmul_rn(o.y, c0.w), __fmul_rn(v.y, c0.z)),
                           __fadd_rn(__fmul_rn(o.z, c1.y), __fmul_rn(v.z, c1.x)),
                           __fadd_rn(__fmul_rn(o.w, c1.w), __fmul_rn(v.w, c1.z)));
    return make_float4(__fsub_rn(__fmul_rn(v.x, c0.x), __fmul_rn(o.x, c0.y)),
                       __fsub_rn(__fmul_rn(v.y, c0.z), __fmul_rn(o.y, c0.w)),
                       __fsub_rn(__fmul_rn(v.z, c1.x), __fmul_rn(o.z, c1.y)),
                       __fsub_rn(__fmul_rn(v.w, c1.z), __fmul_rn(o.w, c1.w)));
}

// Codes and scale of block b, held by eight neighbouring lanes, written to
// position t of a strip half; l is the lane's place among the eight. All of
// `lanes` call it together; blocks past the head's dims are not written.
__device__ __forceinline__ void put_block(uint8_t *half, int f, int dim, int t, int b, int l,
                                          float4 v, unsigned lanes) {
    const bool inside = b * 32 < dim;
    if (!kv_quantised(f)) {
        if (!inside) return;
        uint2 w;
        if (f == F_F16) {
            const __half2 a = __floats2half2_rn(v.x, v.y), c = __floats2half2_rn(v.z, v.w);
            w = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                           *reinterpret_cast<const uint32_t *>(&c));
        } else {
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(v.y), "f"(v.x));
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(v.w), "f"(v.z));
        }
        const int d0 = b * 32 + l * 4;
        *reinterpret_cast<uint2 *>(half + (d0 >> 4) * 512 + t * 32 + (d0 & 15) * 2) = w;
        return;
    }
    float hi = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
    float lo = fminf(fminf(v.x, v.y), fminf(v.z, v.w));
    // x - x is 0 for every finite x and NaN otherwise
    float odd = (v.x - v.x) + (v.y - v.y) + (v.z - v.z) + (v.w - v.w);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
        hi = fmaxf(hi, __shfl_xor_sync(lanes, hi, o));
        lo = fminf(lo, __shfl_xor_sync(lanes, lo, o));
        odd += __shfl_xor_sync(lanes, odd, o);
    }
    if (!inside) return;
    const float m = f == F_Q8_0 ? __fdiv_rn(fmaxf(hi, -lo), 127.0f)
                                : (hi >= -lo ? hi : lo) * -0.125f;
    // odd is 0 or NaN; a scale that f16 cannot hold saturates
    const __half dh = __float2half_rn(fminf(fmaxf(m, -65504.0f), 65504.0f));
    const float d = __half2float(dh);
    const float inv = d != 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
    const bool bad = odd != 0.0f;
    const float s = bad ? 0.0f : inv;
    const float top = f == F_Q8_0 ? 127.0f : 7.0f, bot = f == F_Q8_0 ? -127.0f : -8.0f;
    float4 q = make_float4(rintf(__fmul_rn(v.x, s)), rintf(__fmul_rn(v.y, s)),
                           rintf(__fmul_rn(v.z, s)), rintf(__fmul_rn(v.w, s)));
    const int q0 = (int)fminf(fmaxf(q.x, bot), top), q1 = (int)fminf(fmaxf(q.y, bot), top);
    const int q2 = (int)fminf(fmaxf(q.z, bot), top), q3 = (int)fminf(fmaxf(q.w, bot), top);
    if (f == F_Q8_0) {
        *reinterpret_cast<uint32_t *>(half + b * 512 + t * 32 + l * 4) =
            (uint32_t)(q0 & 255) | (uint32_t)(q1 & 255) << 8 | (uint32_t)(q2 & 255) << 16 |
            (uint32_t)(q3 & 255) << 24;
    } else {
        *reinterpret_cast<uint16_t *>(half + b * 256 + t * 16 + l * 2) =
            (uint16_t)((q0 + 8) | (q1 + 8) << 4 | (q2 + 8) << 8 | (q3 + 8) << 12);
    }
    if (l == 0)
        *reinterpret_cast<uint16_t *>(half + kv_code_bytes(f, dim) + (b * kStrip + t) * 2) =
            bad ? (uint16_t)0x7fffu : __half_as_ushort(dh);
}

// LPU lanes take one head of one row (q, k or v), NI times four dims each
// (dims 4 l + 4 LPU i); every load of the head comes before its stores, so
// q_out may be q.
template <int LPU, int NI>
__global__ void __launch_bounds__(kKvThreads) append_kernel(const KvAppend a) {
    pdl_wait_prev();
    const KvView &c = a.c;
    const int per_row = a.n_heads + 2 * c.n_kv;
    const int64_t total = (int64_t)c.n_seqs * a.n_new * per_row;
    const int l = threadIdx.x % LPU;
    const unsigned lanes = LPU == 32 ? ~0u : 0xffffu << (threadIdx.x & 16);
    for (int64_t u = (int64_t)blockIdx.x * (kKvThreads / LPU) + threadIdx.x / LPU; u < total;
         u += (int64_t)gridDim.x * (kKvThreads / LPU)) {
        const int64_t row = u / per_row;
        int h = (int)(u - row * per_row);
        const int s = (int)(row / a.n_new);
        const int len = __ldg(c.lens + s);
        const int64_t pos = (int64_t)(len < 0 ? 0 : len) - a.n_new + (row - (int64_t)s * a.n_new);
        bool live = pos >= 0;
        if (live && (pos >= c.capacity || (a.rope && pos >= a.rope_len))) {
            record_error(c.err, DERR_BAD_PAGE);
            live = false;
        }
        const bool is_q = h < a.n_heads, is_v = !is_q && h - a.n_heads >= c.n_kv;
        if (!is_q) h -= is_v ? a.n_heads + c.n_kv : a.n_heads;
        if (!live && !is_q) continue;
        const float *x = (is_q ? a.q + row * a.q_stride
                               : is_v ? a.v + row * a.v_stride : a.k + row * a.k_stride) +
                         (int64_t)h * c.dim;
        float4 v[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int d0 = 4 * l + 4 * LPU * i;
            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (d0 < c.dim && live) {
                v[i] = load4(x + d0, a.vec);
                if (a.rope && !is_v) v[i] = rotate4(x, v[i], a.rope + pos * a.n_rot, d0, a.n_rot, a.style, a.vec);
            }
        }
        if (is_q) {
            __syncwarp(lanes);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int d0 = 4 * l + 4 * LPU * i;
                if (d0 < c.dim) store4(a.q_out + row * a.q_out_stride + (int64_t)h * c.dim + d0, v[i], a.vec);
            }
            continue;
        }
        uint8_t *half = kv_strip(c, s, h, (int)(pos / kStrip));
        if (!half) continue;
        if (is_v) half += c.v_off;
#pragma unroll
        for (int i = 0; i < NI; ++i)
            put_block(half, is_v ? c.fmt_v : c.fmt_k, c.dim, (int)(pos % kStrip), (l >> 3) + LPU / 8 * i,
                      l & 7, v[i], lanes);
    }
}

__global__ void __launch_bounds__(kKvThreads) read_kernel(const KvRead a) {
    pdl_wait_prev();
    const KvView &c = a.c;
    const int quads = c.dim / 4;
    const int64_t total = (int64_t)c.n_seqs * a.count * c.n_kv * quads;
    for (int64_t u = (int64_t)blockIdx.x * kKvThreads + threadIdx.x; u < total;
         u += (int64_t)gridDim.x * kKvThreads) {
        const int64_t rh = u / quads;
        const int d0 = (int)(u - rh * quads) * 4;
        const int64_t row = rh / c.n_kv;
        const int h = (int)(rh - row * c.n_kv);
        const int s = (int)(row / a.count);
        const int len = kv_length(c, s);
        const int64_t i = row - (int64_t)s * a.count;
        const int64_t pos = a.first < 0 ? (int64_t)__ldg(c.lens + s) - a.count + i : a.first + i;
        const uint8_t *strip =
            pos >= 0 && pos < len ? kv_strip(c, s, h, (int)(pos / kStrip)) : nullptr;
        const int t = (int)(pos & (kStrip - 1));
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
        if (a.k) store4(a.k + rh * c.dim + d0, strip ? kv_load4(strip, c.fmt_k, c.dim, t, d0) : zero, a.vec);
        if (a.v)
            store4(a.v + rh * c.dim + d0,
                   strip ? kv_load4(strip + c.v_off, c.fmt_v, c.dim, t, d0) : zero, a.vec);
    }
}

// Every launch is a programmatic dependent of the kernel before it and waits
// for it before reading anything: stream order holds, the launch is hidden.
template <class P>
cudaError_t launch(void (*kernel)(P), const P &p, int64_t units, int64_t per_cta,
                   const DeviceInfo &dev, cudaStream_t s) {
    if (units == 0) return cudaSuccess;
    const int64_t most = (int64_t)dev.sm_count * 64;
    int64_t grid = (units + per_cta - 1) / per_cta;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(grid < most ? grid : most));
    cfg.blockDim = dim3(kKvThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppend &a, const DeviceInfo &dev, cudaStream_t s) {
    const int64_t units = (int64_t)a.c.n_seqs * a.n_new * (a.n_heads + 2 * a.c.n_kv);
    if (a.c.dim <= 64) return launch(append_kernel<16, 1>, a, units, kKvThreads / 16, dev, s);
    if (a.c.dim <= 128) return launch(append_kernel<32, 1>, a, units, kKvThreads / 32, dev, s);
    if (a.c.dim <= 256) return launch(append_kernel<32, 2>, a, units, kKvThreads / 32, dev, s);
    return launch(append_kernel<32, 4>, a, units, kKvThreads / 32, dev, s);
}

cudaError_t launch_kv_read(const KvRead &a, const DeviceInfo &dev, cudaStream_t s) {
    const int64_t units = (int64_t)a.c.n_seqs * a.count * a.c.n_kv * (a.c.dim / 4);
    return launch(read_kernel, a, units, kKvThreads, dev, s);
}

}  // namespace qmm
