// qmm_kv.cu -- appending to the paged key-value cache (rotary embedding of q
// and k, quantising write of k and v) and reading it back.
//
// Both kernels move each value once and do a few operations on it, so memory
// bounds them: 8000 rows of 48 heads of 128 rotated and appended in F16 take
// 55 us (6.6 TB/s, 96 % of a copy's rate), 16 sequences of up to 8111 positions of
// 8 heads of 128 read back from Q8_0 / Q4_0 182 us (6.6 TB/s). A lane takes four
// dims, so that fp32 loads and stores are 16 bytes wide; the 32 dims of a block
// are eight neighbouring lanes, so that its maximum takes three shuffles and its
// codes are one 32-byte sector.
#include "qmm_kv.cuh"
#include "qmm_kv_launch.h"

namespace qmm {

namespace {

constexpr int kKvThreads = 128;

template <bool VEC>
__device__ __forceinline__ float4 load4(const float *p) {
    if constexpr (VEC) return *reinterpret_cast<const float4 *>(p);
    else return make_float4(p[0], p[1], p[2], p[3]);
}
__device__ __forceinline__ void store4(float *p, float4 v, bool vec) {
    if (vec) {
        *reinterpret_cast<float4 *>(p) = v;
    } else {
        p[0] = v.x; p[1] = v.y; p[2] = v.z; p[3] = v.w;
    }
}

// The rotation of four dims v of a head. PAIRS: both dims of a pair are here,
// cs0 = c s c s of the two. HALF: o holds the dims' partners, n_rot / 2 away
// (`second`: v are the pairs' second dims), c0 and c1 = c s of the four.
// Products and sums are rounded one by one (no fma), so the result does not
// depend on how a compiler contracts the formula.
__device__ __forceinline__ float4 rotate_pairs(float4 v, float4 cs0) {
    return make_float4(__fsub_rn(__fmul_rn(v.x, cs0.x), __fmul_rn(v.y, cs0.y)),
                       __fadd_rn(__fmul_rn(v.x, cs0.y), __fmul_rn(v.y, cs0.x)),
                       __fsub_rn(__fmul_rn(v.z, cs0.z), __fmul_rn(v.w, cs0.w)),
                       __fadd_rn(__fmul_rn(v.z, cs0.w), __fmul_rn(v.w, cs0.z)));
}
__device__ __forceinline__ float4 rotate_half(float4 v, float4 o, float4 c0, float4 c1, bool second) {
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
// position t of a strip half in format F; l is the lane's place among the
// eight. All of `lanes` call it together; blocks past the head's dims are not
// written.
template <int F>
__device__ __forceinline__ void put_block(uint8_t *half, int dim, int t, int b, int l, float4 v,
                                          unsigned lanes) {
    const bool inside = b * 32 < dim;
    if constexpr (!kv_quantised(F)) {
        uint2 w;
        if constexpr (F == F_F16) {
            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(v.y), "f"(v.x));
            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(v.w), "f"(v.z));
        } else {
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(v.y), "f"(v.x));
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(v.w), "f"(v.z));
        }
        const int d0 = b * 32 + l * 4;
        if (inside) *reinterpret_cast<uint2 *>(half + (d0 >> 4) * 512 + t * 32 + (d0 & 15) * 2) = w;
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
    const float m = F == F_Q8_0 ? __fdiv_rn(fmaxf(hi, -lo), 127.0f) : (hi >= -lo ? hi : lo) * -0.125f;
    // odd is 0 or NaN; a scale that f16 cannot hold saturates
    const __half dh = __float2half_rn(fminf(fmaxf(m, -65504.0f), 65504.0f));
    const float d = __half2float(dh);
    const bool bad = odd != 0.0f;
    const float s = d != 0.0f && !bad ? __fdiv_rn(1.0f, d) : 0.0f;
    constexpr float kTop = F == F_Q8_0 ? 127.0f : 7.0f, kBottom = F == F_Q8_0 ? -127.0f : -8.0f;
    const int q0 = (int)fminf(fmaxf(rintf(__fmul_rn(v.x, s)), kBottom), kTop);
    const int q1 = (int)fminf(fmaxf(rintf(__fmul_rn(v.y, s)), kBottom), kTop);
    const int q2 = (int)fminf(fmaxf(rintf(__fmul_rn(v.z, s)), kBottom), kTop);
    const int q3 = (int)fminf(fmaxf(rintf(__fmul_rn(v.w, s)), kBottom), kTop);
    if constexpr (F == F_Q8_0) {
        *reinterpret_cast<uint32_t *>(half + b * 512 + t * 32 + l * 4) =
            (uint32_t)(q0 & 255) | (uint32_t)(q1 & 255) << 8 | (uint32_t)(q2 & 255) << 16 |
            (uint32_t)(q3 & 255) << 24;
    } else {
        *reinterpret_cast<uint16_t *>(half + b * 256 + t * 16 + l * 2) =
            (uint16_t)((q0 + 8) | (q1 + 8) << 4 | (q2 + 8) << 8 | (q3 + 8) << 12);
    }
    if (l == 0)
        *reinterpret_cast<uint16_t *>(half + kv_code_bytes(F, dim) + (b * kStrip + t) * 2) =
            bad ? (uint16_t)0x7fffu : __half_as_ushort(dh);
}

constexpr int kTurnHalf = 0, kTurnPairs = 1, kTurnNone = 2;

// The dims of one head that a lane holds: dims 4 l + 4 LPU i, and (for HALF)
// the other dims of their pairs.
template <int NI>
struct Dims {
    float4 v[NI], o[NI];
};
template <int LPU, int NI, bool VEC, int TURN>
__device__ __forceinline__ void load_dims(Dims<NI> &x, const float *p, int l, int dim, int half_rot) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int d0 = 4 * l + 4 * LPU * i;
        x.v[i] = x.o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (d0 < dim) x.v[i] = load4<VEC>(p + d0);
        if (TURN == kTurnHalf && d0 < 2 * half_rot)
            x.o[i] = load4<VEC>(p + (d0 < half_rot ? d0 + half_rot : d0 - half_rot));
    }
}
// cos and sin for those dims at one position (`r`: its row of the table)
template <int NI>
struct Turn {
    float4 c0[NI], c1[NI];
};
template <int LPU, int NI, int TURN>
__device__ __forceinline__ void load_turn(Turn<NI> &t, const float *r, int l, int n_rot) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int d0 = 4 * l + 4 * LPU * i;
        if (TURN == kTurnNone || d0 >= n_rot) continue;
        if (TURN == kTurnHalf) {
            const int p = d0 < n_rot / 2 ? d0 : d0 - n_rot / 2;
            t.c0[i] = *reinterpret_cast<const float4 *>(r + 2 * p);
            t.c1[i] = *reinterpret_cast<const float4 *>(r + 2 * p + 4);
        } else {
            t.c0[i] = *reinterpret_cast<const float4 *>(r + d0);
        }
    }
}
template <int LPU, int NI, int TURN>
__device__ __forceinline__ void turn_dims(Dims<NI> &x, const Turn<NI> &t, int l, int n_rot) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int d0 = 4 * l + 4 * LPU * i;
        if (TURN == kTurnNone || d0 >= n_rot) continue;
        x.v[i] = TURN == kTurnHalf ? rotate_half(x.v[i], x.o[i], t.c0[i], t.c1[i], d0 >= n_rot / 2)
                                   : rotate_pairs(x.v[i], t.c0[i]);
    }
}

// K and V rows of kv heads first, first + step, ... < n_kv into the cache
template <int FK, int FV, int LPU, int NI, bool VEC, int TURN>
__device__ __forceinline__ void put_heads(const KvAppend &a, int row, int first, int step, uint8_t *strip,
                                          int t, const Turn<NI> &turn, int l, unsigned lanes) {
    const KvView &c = a.c;
    const int v_off = kv_half_bytes(FK, c.dim);
    for (int h = first; h < c.n_kv; h += step) {
        Dims<NI> k, v;
        load_dims<LPU, NI, VEC, TURN>(k, a.k + row * a.k_stride + (int64_t)h * c.dim, l, c.dim, a.n_rot / 2);
        load_dims<LPU, NI, VEC, kTurnNone>(v, a.v + row * a.v_stride + (int64_t)h * c.dim, l, c.dim, 0);
        turn_dims<LPU, NI, TURN>(k, turn, l, a.n_rot);
        uint8_t *half = strip + h * c.head_bytes;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            put_block<FK>(half, c.dim, t, (l >> 3) + LPU / 8 * i, l & 7, k.v[i], lanes);
            put_block<FV>(half + v_off, c.dim, t, (l >> 3) + LPU / 8 * i, l & 7, v.v[i], lanes);
        }
    }
}

// A team of LPU lanes takes every a.teams-th head of a row, NI times four dims
// per lane, U heads of q at a time, and K and V of a kv head together. The row's
// position, page and rotary entries are looked up once, while the first heads
// are loading (lengths, page table and rotary table are loads that wait for
// one another). The loads of a head come before its stores, so q_out may be q.
template <int LPU, int NI, int U, bool VEC, int TURN>
__global__ void __launch_bounds__(kKvThreads) append_kernel(const KvAppend a) {
    pdl_wait_prev();
    const KvView &c = a.c;
    const int l = threadIdx.x % LPU, step = a.teams;
    const unsigned lanes = LPU == 32 ? ~0u : 0xffffu << (threadIdx.x & 16);
    const int64_t id = (int64_t)blockIdx.x * (kKvThreads / LPU) + threadIdx.x / LPU;
    const int row = (int)(id / step), team = (int)(id - (int64_t)row * step);
    if (row >= c.n_seqs * (int)a.n_new) return;
    bool looked = false, live = false;
    int t = 0;
    uint8_t *strip = nullptr;
    Turn<NI> turn;
    auto look = [&]() {
        const int s = a.n_new == 1 ? row : row / (int)a.n_new;
        const int len = __ldg(c.lens + s);
        const int64_t pos = (int64_t)(len < 0 ? 0 : len) - a.n_new + (row - s * a.n_new);
        live = pos >= 0;
        if (live && (pos >= c.capacity || (TURN != kTurnNone && pos >= a.rope_len))) {
            record_error(c.err, DERR_BAD_PAGE);
            live = false;
        }
        t = (int)pos & (kStrip - 1);
        if (live) {
            load_turn<LPU, NI, TURN>(turn, a.rope + pos * a.n_rot, l, a.n_rot);
            strip = kv_strip(c, s, 0, (int)(pos / kStrip));
        }
        looked = true;
    };
    for (int h0 = team; h0 < a.n_heads; h0 += step * U) {
        Dims<NI> x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * step;
            if (h < a.n_heads)
                load_dims<LPU, NI, VEC, TURN>(x[u], a.q + row * a.q_stride + (int64_t)h * c.dim, l, c.dim,
                                              a.n_rot / 2);
        }
        if (!looked) look();
        __syncwarp(lanes);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * step;
            if (h >= a.n_heads) continue;
            if (live) turn_dims<LPU, NI, TURN>(x[u], turn, l, a.n_rot);
            float *to = a.q_out + row * a.q_out_stride + (int64_t)h * c.dim;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int d0 = 4 * l + 4 * LPU * i;
                if (d0 < c.dim) store4(to + d0, live ? x[u].v[i] : make_float4(0.f, 0.f, 0.f, 0.f), VEC);
            }
        }
    }
    if (!looked) look();
    if (!strip) return;
    // the kv heads go to the teams after those that took the last heads of q
    const int first = (team - a.n_heads % step + step) % step;
    if (c.fmt_k == F_F16)
        put_heads<F_F16, F_F16, LPU, NI, VEC, TURN>(a, row, first, step, strip, t, turn, l, lanes);
    else if (c.fmt_k == F_BF16)
        put_heads<F_BF16, F_BF16, LPU, NI, VEC, TURN>(a, row, first, step, strip, t, turn, l, lanes);
    else if (c.fmt_k == F_Q4_0)
        put_heads<F_Q4_0, F_Q4_0, LPU, NI, VEC, TURN>(a, row, first, step, strip, t, turn, l, lanes);
    else if (c.fmt_v == F_Q4_0)
        put_heads<F_Q8_0, F_Q4_0, LPU, NI, VEC, TURN>(a, row, first, step, strip, t, turn, l, lanes);
    else
        put_heads<F_Q8_0, F_Q8_0, LPU, NI, VEC, TURN>(a, row, first, step, strip, t, turn, l, lanes);
}

// LPU lanes read positions t0, t0 + step, ... < kStrip (a warp's lanes and SPLIT
// warps share a strip) of a strip half in format F: K's or V's rows of one head,
// `stride` floats apart in out; rows outside [from, to) are zeros.
template <int F, int LPU, int NI, int SPLIT>
__device__ __forceinline__ void read_half(const uint8_t *half, float *out, int64_t stride, int dim,
                                          int t0, int from, int to, int rows, int l, bool vec) {
    constexpr int step = 32 / LPU * SPLIT, kMine = kStrip / step;
    constexpr int kMost = NI >= 4 ? 2 : NI == 2 ? 4 : 8;  // rows in flight
    constexpr int kDeep = kMine < kMost ? kMine : kMost;
    for (int t = t0; t < kStrip; t += step * kDeep) {
        float4 v[kDeep][NI];
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int d0 = 4 * l + 4 * LPU * i, at = t + k * step;
                v[k][i] = half && d0 < dim && at < kStrip && at >= from && at < to
                              ? kv_load4(half, F, dim, at, d0)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int d0 = 4 * l + 4 * LPU * i, at = t + k * step;
                if (d0 < dim && at < kStrip && at >= from && at < rows) store4(out + at * stride + d0, v[k][i], vec);
            }
    }
}
template <int LPU, int NI, int SPLIT>
__device__ __forceinline__ void read_half(int f, const uint8_t *half, float *out, int64_t stride, int dim,
                                          int t0, int from, int to, int rows, int l, bool vec) {
    switch (f) {
    case F_F16: return read_half<F_F16, LPU, NI, SPLIT>(half, out, stride, dim, t0, from, to, rows, l, vec);
    case F_BF16: return read_half<F_BF16, LPU, NI, SPLIT>(half, out, stride, dim, t0, from, to, rows, l, vec);
    case F_Q8_0: return read_half<F_Q8_0, LPU, NI, SPLIT>(half, out, stride, dim, t0, from, to, rows, l, vec);
    default: return read_half<F_Q4_0, LPU, NI, SPLIT>(half, out, stride, dim, t0, from, to, rows, l, vec);
    }
}

// A warp takes one strip of one head of K (blockIdx.z 0) or V, or every
// SPLIT-th position of it, with up to eight 16-byte stores per lane in
// flight. blockIdx.y: sequence; the strips are those that its rows touch.
template <int LPU, int NI, int SPLIT>
__global__ void __launch_bounds__(kKvThreads) read_kernel(const KvRead a) {
    pdl_wait_prev();
    const KvView &c = a.c;
    const int warp = blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5);
    const int unit = warp / SPLIT, sub = warp % SPLIT;
    const int k = unit / c.n_kv, h = unit - k * c.n_kv;
    const bool is_v = a.k == nullptr || blockIdx.z == 1;
    for (int s = blockIdx.y; s < c.n_seqs; s += gridDim.y) {
        const int64_t first = a.first < 0 ? (int64_t)max(__ldg(c.lens + s), 0) - a.count : a.first;
        // the strip's first position, and which of its positions have rows
        const int64_t begin = ((first >> 4) + k) * kStrip;
        const int64_t from = first - begin, rows = first + a.count - begin;
        if (rows <= 0) continue;
        const int64_t to = kv_length(c, s) - begin;
        const uint8_t *strip = begin >= 0 && to > 0 ? kv_strip(c, s, h, (int)(begin / kStrip)) : nullptr;
        float *out = (is_v ? a.v : a.k) + (((int64_t)s * a.count - from) * c.n_kv + h) * c.dim;
        read_half<LPU, NI, SPLIT>(is_v ? c.fmt_v : c.fmt_k, strip ? strip + (is_v ? c.v_off : 0) : nullptr, out,
                           (int64_t)c.n_kv * c.dim, c.dim, (threadIdx.x & 31) / LPU + 32 / LPU * sub,
                           (int)(from > 0 ? from : 0), (int)(to < kStrip ? to : kStrip),
                           (int)(rows < kStrip ? rows : kStrip), threadIdx.x % LPU, a.vec);
    }
}

// Every launch is a programmatic dependent of the kernel before it and waits
// for it before reading anything: stream order holds, the launch is hidden.
template <class P>
cudaError_t launch(void (*kernel)(P), const P &p, dim3 grid, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kKvThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int LPU, int NI, int U>
cudaError_t launch_append(const KvAppend &a, const DeviceInfo &dev, cudaStream_t s) {
    // Teams per row: one per kv head, at most eight, so that teams have equal
    // work and several heads in flight; more, up to one per head, where there
    // are too few rows to give every SM 64 warps. (Eight teams for 8 heads of q
    // and 2 of k and v kept six of them waiting for two, in blocks of 256
    // threads: 57 us instead of 28 for 5331 rows of 256 dims, Q4_0. Blocks of 128
    // take 25.)
    const int64_t rows = a.c.n_seqs * a.n_new, in_block = kKvThreads / LPU;
    int64_t teams = a.c.n_kv < 8 ? a.c.n_kv : 8;
    const int64_t fill = (dev.sm_count * 16 * in_block + rows - 1) / rows;
    if (teams < fill) teams = fill;
    if (teams > a.n_heads + a.c.n_kv) teams = a.n_heads + a.c.n_kv;
    KvAppend p = a;
    p.teams = (int)teams;
    const dim3 grid((unsigned)((rows * teams + in_block - 1) / in_block));
    if (a.vec) {
        if (!a.rope) return launch(append_kernel<LPU, NI, U, true, kTurnNone>, p, grid, s);
        if (a.style == 0) return launch(append_kernel<LPU, NI, U, true, kTurnHalf>, p, grid, s);
        return launch(append_kernel<LPU, NI, U, true, kTurnPairs>, p, grid, s);
    }
    if (!a.rope) return launch(append_kernel<LPU, NI, U, false, kTurnNone>, p, grid, s);
    if (a.style == 0) return launch(append_kernel<LPU, NI, U, false, kTurnHalf>, p, grid, s);
    return launch(append_kernel<LPU, NI, U, false, kTurnPairs>, p, grid, s);
}

template <int LPU, int NI>
cudaError_t launch_read(const KvRead &a, const DeviceInfo &dev, cudaStream_t s) {
    // strips that `count` positions can touch, from any first one
    const int64_t strips = a.first < 0 ? (a.count + 2 * kStrip - 2) / kStrip
                                       : ((a.first % kStrip) + a.count + kStrip - 1) / kStrip;
    // A strip per warp where that gives every SM 16 warps; four warps share
    // one where there are few (200 positions of 8 heads of 128: 2.9 us, 3.8 with
    // one warp each).
    const int64_t halves = (int64_t)a.c.n_seqs * (a.k && a.v ? 2 : 1);
    const int split = strips * a.c.n_kv * halves >= (int64_t)dev.sm_count * 16 ? 1 : 4;
    const int64_t blocks = (strips * a.c.n_kv * split + kKvThreads / 32 - 1) / (kKvThreads / 32);
    const dim3 grid((unsigned)blocks, (unsigned)(a.c.n_seqs < 65535 ? a.c.n_seqs : 65535), a.k && a.v ? 2 : 1);
    if (split == 1) return launch(read_kernel<LPU, NI, 1>, a, grid, s);
    return launch(read_kernel<LPU, NI, 4>, a, grid, s);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppend &a, const DeviceInfo &dev, cudaStream_t s) {
    if (a.c.dim <= 64) return launch_append<16, 1, 4>(a, dev, s);
    if (a.c.dim <= 128) return launch_append<32, 1, 4>(a, dev, s);
    if (a.c.dim <= 256) return launch_append<32, 2, 2>(a, dev, s);
    return launch_append<32, 4, 1>(a, dev, s);
}

cudaError_t launch_kv_read(const KvRead &a, const DeviceInfo &dev, cudaStream_t s) {
    if (a.c.dim <= 64) return launch_read<16, 1>(a, dev, s);
    if (a.c.dim <= 128) return launch_read<32, 1>(a, dev, s);
    if (a.c.dim <= 256) return launch_read<32, 2>(a, dev, s);
    return launch_read<32, 4>(a, dev, s);
}

}  // namespace qmm
