// qmm_linear_chunk.cu -- linear attention over many rows of a sequence, in
// chunks of C = 32. With G_i the sum of the chunk's decays up to row i and S the
// state before the chunk,
//     o_i = e^(G_i) S^T q_i + sum_(j <= i) e^(G_i - G_j) (q_i . k_j) v_j,
//     S' = e^(G_C) S + sum_j e^(G_C - G_j) k_j v_j^T :
// four products per chunk, on the tensor cores.
//
// A warp owns 16 dims of v for the whole run and keeps S^T (16 x dk) as the
// accumulator fragments of m16n8k16, which are A fragments of S^T Q^T as they
// stand. The 32 x 32 scores are shared: one 16 x 8 tile a warp. fp32 values enter
// as two fp16 terms (22 bits) under powers of two per row of q and k and per
// dim of S and of what a chunk adds to it, three products of terms each; scores times v, the
// smallest of the four, as three bf16 terms and six products, which need no power of two: a row's
// scores are of very different sizes where decays are strong. Accumulators start fresh after at most
// 32 values of depth and the small products come first, since the
// tensor cores cut what they add. Sums of decays are formed in 64 bits and kept as
// two floats, so that differences of long sums stay exact.
//
// A prompt too short of sequences and heads to fill the GPU is cut into segments: their own end states
// first (one product of the four), a scan over the segments, then everything.
//
// Bound by instructions and the latency that 16 warps an SM, whose states take the registers, do not hide: 2540 a warp and
// chunk at dk = dv = 128, of which 246 are products (1080 in the segments' own states); issue slots 48 % used, tensor pipe
// 37 %. Measured: 12001 rows of 16 heads of 128 / 128 325 us (91 the segments' own states, 227 the second pass), six ragged
// sequences to 1777 rows of 12 heads of 64 / 96 141 us, against 58 and 17 us that their bytes take. The decays' sums in
// one warp, terms in vectors and factors read instead of formed took the first from 477 us to 310; three terms of scores
// and v, and powers of two beyond fp32's exponents, cost 15 us of that.
#include "qmm_device.cuh"
#include "qmm_linear.h"

#include <type_traits>

#include <cuda_fp16.h>

namespace qmm {

namespace linear {

namespace {

constexpr int C = kChunk;
constexpr int kMaxWarps = 8;

struct ChunkParams {
    Linear l;
    Split split;
    float *starts;        // [segments][n_seqs][n_heads][dk][dv]: the state before each segment (one segment: not used)
    float *seg_decay;     // [segments][n_seqs][n_heads]: sum of a segment's decays (log2 of the factor)
};

// Shared memory, in bytes from its start: q and k as they come, v of two
// chunks, q and k as two terms each, the scores as three, small arrays.
struct Plan {
    int raw_q, raw_k, raw_v, v_bytes, q16, k16, term, p16, p_term, small, bytes;
};
__host__ __device__ constexpr int pitch_of(int dk) { return (dk + 8) * 2; }  // 8 rows of 16 bytes on different banks
constexpr int kPPitch = (C + 8) * 2;
// Scores, at most 2^37 times q's and k's powers of two, in units of 2^24: no larger than k.
constexpr int kScoreUnit = 24;
// bf16 terms end at 2^-133: where all of a chunk's k have powers of two below this one they are multiplied up to it,
// and dims of v below 2^-64 by 2^64.
constexpr int kTinyK = -40, kTinyUp = 64;
constexpr uint32_t kTinyBits = 0x1F800000;  // 2^-64
// Of the sums G_i of a chunk's decays: high and low parts, e^(G_i), e^(G_C - G_i), and (padded) e^(G_C).
constexpr int kDecayFloats = 4 * C + 4;
__host__ __device__ constexpr Plan plan_of(int dk, int tile) {
    Plan p = {};
    p.raw_q = 0;
    p.raw_k = p.raw_q + C * dk * 4;
    p.raw_v = p.raw_k + C * dk * 4;
    p.v_bytes = C * (tile + 4) * 4;  // rows 4 floats apart beyond their length: fragments' loads meet no bank twice
    p.term = C * pitch_of(dk);
    p.q16 = p.raw_v + 2 * p.v_bytes;
    p.k16 = p.q16 + 2 * p.term;
    p.p_term = C * kPPitch;
    p.p16 = p.k16 + 2 * p.term;
    p.small = p.p16 + 3 * p.p_term;
    p.bytes = p.small + (2 * kDecayFloats + 3 * C) * 4;
    return p;
}

#define QMM_MMA_OF(T) "mma.sync.aligned.m16n8k16.row.col.f32." T "." T ".f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
#define QMM_MMA QMM_MMA_OF("f16")
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(QMM_MMA "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// from zero
__device__ __forceinline__ void mma_new(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(QMM_MMA "{%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
// bf16 operands
__device__ __forceinline__ void mma_bf(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(QMM_MMA_OF("bf16") "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
#undef QMM_MMA
#undef QMM_MMA_OF
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldm4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldm2(uint32_t (&r)[2], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const float *src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const float *src, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(on ? 4 : 0) : "memory");
}

// Two values as fp16 pairs: the rounded ones and what is left of them.
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    const __half2 r = __floats2half2_rn(x - f.x, y - f.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&r);
}
// Two values as bf16 pairs: three terms that are cut, 8 bits each, so that they hold all 24.
__device__ __forceinline__ void cut3(float x, float y, uint32_t (&t)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
        t[i] = prmt(a, b, 0x7632u);
        x -= __uint_as_float(a & 0xFFFF0000u);
        y -= __uint_as_float(b & 0xFFFF0000u);
    }
}
// The exponent that brings values whose largest has this biased exponent to
// [2^14, 2^15) is -e; it stays in what 2^e and 2^-e can be as normal numbers.
__device__ __forceinline__ int exponent_for(uint32_t biased) {
    const int e = (int)biased - 127 - 14;
    return biased == 255 ? 0 : e < -126 ? -126 : e;
}
// 2^n, of the normal numbers
__device__ __forceinline__ float pow2_of(int n) { return __uint_as_float((uint32_t)(n + 127) << 23); }
__device__ __forceinline__ bool is_normal(int n) { return (uint32_t)(n + 126) <= 253u; }
// 2^n, 0 below the normal numbers, 2^127 above
__device__ __forceinline__ float pow2(int n) { return __uint_as_float((uint32_t)(min(max(n, -127), 127) + 127) << 23); }
__device__ __forceinline__ uint32_t exponent_bits(float v) { return (__float_as_uint(v) >> 23) & 255u; }
// 2^n times v, for n to twice what a float's exponent can be
__device__ __forceinline__ float times_pow2(float v, int n) {
    const int m = min(max(n, -126), 127);
    return v * pow2(n - m) * pow2_of(m);
}
// 2^-exponent_for()
__device__ __forceinline__ float up_for(int e) { return __uint_as_float((uint32_t)(127 - e) << 23); }
// max(top, |v|), NaN if v is
__device__ __forceinline__ float top_of(float top, float v) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(top), "f"(fabsf(v)));
    return r;
}
__device__ __forceinline__ bool finite(float top) { return __float_as_uint(top) < 0x7F800000u; }
__device__ __forceinline__ int exponent_of(float top) { return exponent_for(__float_as_uint(top) >> 23); }
// over the four lanes of a dim
__device__ __forceinline__ float top_over_4(float v) {
    v = top_of(v, __shfl_xor_sync(~0u, v, 1));
    return top_of(v, __shfl_xor_sync(~0u, v, 2));
}

// OUT: outputs and, of the last segment, the state; else the end states of all
// segments but the last, from zeros (the first: from the call's state).
template <int DK, bool OUT>
__global__ void __launch_bounds__(kMaxWarps * 32, 2) chunk_kernel(const __grid_constant__ ChunkParams p) {
    constexpr int KS = DK / 16;    // 16-deep steps over dk; pairs of 8-wide tiles
    constexpr int PITCH = pitch_of(DK);
    extern __shared__ __align__(128) uint8_t smem[];
    const Linear &l = p.l;
    const int tile_cols = p.split.tile, nw = tile_cols / 16;
    const Plan plan = plan_of(DK, tile_cols);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = nw * 32;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t base = smem_addr(smem);
    float *const gs = reinterpret_cast<float *>(smem + plan.small);
    int *const q_exp = reinterpret_cast<int *>(gs + 2 * kDecayFloats), *const k_exp = q_exp + C, *const k_bad = k_exp + C;

    pdl_wait_prev();
    pdl_launch_dependents();
    int at = blockIdx.x;
    const int tile = at % p.split.tiles;
    at /= p.split.tiles;
    const int head = at % l.n_heads;
    at /= l.n_heads;
    const int seq = at % l.n_seqs, seg = at / l.n_seqs;
    const Span span = span_of(l, seq);
    const int64_t row0 = seg * p.split.rows, row1 = min(l.n_new, row0 + p.split.rows);
    const bool last = seg == p.split.segments - 1;
    const int64_t which = (int64_t)seq * l.n_heads + head, states = (int64_t)l.n_seqs * l.n_heads;
    const int64_t size = (int64_t)DK * l.dv;
    const int cols = head * l.dv + tile * tile_cols;      // first column of the tile in rows of v and out
    const int mine = tile * tile_cols + warp * 16 + g;    // this lane's dims of the state: mine, mine + 8

    if (OUT) {
        // rows before the sequence's first
        const int64_t n = min(span.first, row1) - row0;
        for (int64_t i = tid; i < n * tile_cols; i += threads)
            l.out[(seq * l.n_new + row0 + i / tile_cols) * l.out_stride + cols + i % tile_cols] = 0.0f;
    }
    if (span.idle) {
        if (OUT && last && l.state_out != l.state)
            for (int i = tid; i < DK * tile_cols; i += threads) {
                const int64_t x = which * size + (int64_t)(i / tile_cols) * l.dv + tile * tile_cols + i % tile_cols;
                l.state_out[x] = l.state[x];
            }
        return;
    }

    // S^T: [8-wide tile of dk][fragment]
    float s[2 * KS][4];
    const float *from = nullptr;
    // several segments: the first pass keeps a copy of the call's state, since the last segment may write over it
    // while the first one has yet to start
    const bool copied = OUT && p.split.segments > 1;
    if (seg == 0 && !span.begins) from = copied ? p.starts + which * size : l.state + which * size;
    if (OUT && seg > 0) from = p.starts + (seg * states + which) * size;
#pragma unroll
    for (int n = 0; n < 2 * KS; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            s[n][i] = from ? from[(int64_t)(8 * n + 2 * t + (i & 1)) * l.dv + mine + 8 * (i >> 1)] : 0.0f;
    auto store = [&](float *to) {
#pragma unroll
        for (int n = 0; n < 2 * KS; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) to[(int64_t)(8 * n + 2 * t + (i & 1)) * l.dv + mine + 8 * (i >> 1)] = s[n][i];
    };
    if (!OUT && from) store(p.starts + which * size);

    const int64_t begin = span.first > row0 ? row0 + (span.first - row0) / C * C : row0;
    const float *const qk_of[2] = {l.q + head / (l.n_heads / l.n_qk) * DK, l.k + head / (l.n_heads / l.n_qk) * DK};
    auto load = [&](int64_t row, int buffer) {
        const int64_t x0 = seq * l.n_new + row;
        const int lo = (int)max((int64_t)0, span.first - row), n = (int)min((int64_t)C, row1 - row) - lo;  // rows that are there
        auto rows = [&](uint32_t dst, int pitch, const float *src, int64_t stride, int width) {
            src += x0 * stride;
            if (l.vec) {
                // a row per warp, 16 bytes a lane
                if (4 * lane < width) {
                    const float *at = src + warp * stride + 4 * lane;
                    dst += (warp * pitch + 4 * lane) * 4;
                    for (int r = warp; r < C; r += nw, at += nw * stride, dst += nw * pitch * 4) {
                        const bool on = (uint32_t)(r - lo) < (uint32_t)n;
                        copy16(dst, on ? at : src + lo * stride, on);
                    }
                }
            } else {
                for (int i = tid; i < C * width; i += threads) {
                    const int r = i / width, c = i % width;
                    const bool on = (uint32_t)(r - lo) < (uint32_t)n;
                    copy4(dst + (r * pitch + c) * 4, on ? src + r * stride + c : src + lo * stride, on);
                }
            }
        };
        if (OUT) rows(base + plan.raw_q, DK, qk_of[0], l.q_stride, DK);
        rows(base + plan.raw_k, DK, qk_of[1], l.k_stride, DK);
        rows(base + plan.raw_v + buffer * plan.v_bytes, tile_cols + 4, l.v + cols, l.v_stride, tile_cols);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto load_decay = [&](int64_t row) {
        const int64_t r = row + lane;
        return r >= span.first && r < row1 ? decay_of(l.decay[(seq * l.n_new + r) * l.decay_stride + head]) : 0.0f;
    };
    // The last warp sums a chunk's decays while the others are at the scores of the chunk before: lane j row
    // j, log2 of the factors, 64 bits.
    const bool sums_decays = warp == nw - 1;
    double seg_total = 0.0;
    auto sum_decays = [&](float decay, int buffer) {
        double total = (double)decay * 1.4426950408889634;
#pragma unroll
        for (int o = 1; o < C; o <<= 1) {
            const double a = __shfl_up_sync(~0u, total, o);
            if (lane >= o) total += a;
        }
        const double chunk_total = __shfl_sync(~0u, total, C - 1);
        const float high = (float)total;
        float *const at = gs + buffer * kDecayFloats;
        at[lane] = high;
        at[C + lane] = (float)(total - (double)high);
        at[2 * C + lane] = exp2f((float)total);
        at[3 * C + lane] = exp2f((float)(chunk_total - total));
        if (lane == 0) at[4 * C] = exp2f((float)chunk_total);
        seg_total += chunk_total;
    };

    float next_decay = 0.0f;
    if (begin < row1) {
        load(begin, 0);
        if (sums_decays) {
            sum_decays(load_decay(begin), 0);
            next_decay = load_decay(begin + C);
        }
    }
    int buffer = 0;
    for (int64_t row = begin; row < row1; row += C, buffer ^= 1) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();  // the rows are there, and the chunk before has been used up
        // q and k as terms, a row per warp
#pragma unroll 2
        for (int i = warp; i < C; i += nw) {
#pragma unroll
            for (int is_k = OUT ? 0 : 1; is_k < 2; ++is_k) {
                constexpr int V = DK / 32;
                const float *raw = reinterpret_cast<const float *>(smem + (is_k ? plan.raw_k : plan.raw_q)) + i * DK + lane * V;
                float x[V];
                if constexpr (V == 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(raw);
                    x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
                } else if constexpr (V == 2) {
                    const float2 f = *reinterpret_cast<const float2 *>(raw);
                    x[0] = f.x, x[1] = f.y;
                } else {
#pragma unroll
                    for (int v = 0; v < V; ++v) x[v] = raw[v];
                }
                float most = 0.0f;
#pragma unroll
                for (int v = 0; v < V; ++v) most = top_of(most, x[v]);
                uint32_t top = __reduce_max_sync(~0u, __float_as_uint(most));
                if (is_k) {
                    const bool bad = top >= 0x7F800000u;
                    if (bad) {
                        // a k that is not finite must not meet the zeros of rows before it: it is taken out here,
                        // and the rows from its own on become NaN
                        most = 0.0f;
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            if (exponent_bits(x[v]) == 255) x[v] = 0.0f;
                            most = top_of(most, x[v]);
                        }
                        top = __reduce_max_sync(~0u, __float_as_uint(most));
                    }
                    if (lane == 0) k_bad[i] = bad;
                }
                const int e = is_k || top ? exponent_for(top >> 23) : 0;
                const float up = up_for(e);
                if (lane == 0) (is_k ? k_exp : q_exp)[i] = e;
                uint8_t *const hi = smem + (is_k ? plan.k16 : plan.q16) + i * PITCH + lane * V * 2, *const lo = hi + plan.term;
                if constexpr (V % 2 == 0) {
                    uint32_t h[V / 2], r[V / 2];
#pragma unroll
                    for (int v = 0; v < V / 2; ++v) split2(x[2 * v] * up, x[2 * v + 1] * up, h[v], r[v]);
                    if constexpr (V == 4) {
                        *reinterpret_cast<uint2 *>(hi) = make_uint2(h[0], h[1]);
                        *reinterpret_cast<uint2 *>(lo) = make_uint2(r[0], r[1]);
                    } else {
                        *reinterpret_cast<uint32_t *>(hi) = h[0];
                        *reinterpret_cast<uint32_t *>(lo) = r[0];
                    }
                } else {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const float y = x[v] * up;
                        const __half h = __float2half_rn(y);
                        reinterpret_cast<__half *>(hi)[v] = h;
                        reinterpret_cast<__half *>(lo)[v] = __float2half_rn(y - __half2float(h));
                    }
                }
            }
        }
        __syncthreads();  // terms are there, raw q and k are free
        if (row + C < row1) {
            load(row + C, buffer ^ 1);
            if (sums_decays) {
                sum_decays(next_decay, buffer ^ 1);
                next_decay = load_decay(row + 2 * C);
            }
        }
        const float *const gh = gs + buffer * kDecayFloats, *const gl = gh + C;
        const float *const from_start = gl + C, *const to_end = from_start + C;
        const int ke = k_exp[lane];
        // the largest k's exponent among the rows as they are decayed at the chunk's end
        const int k_top = __reduce_max_sync(~0u, __float2int_ru((float)ke + (gh[C - 1] - gh[lane])));
        const int k_up = max(0, kTinyK - __reduce_max_sync(~0u, ke));
        // the first row that a k or decay makes NaN
        const uint32_t bad_rows = __ballot_sync(~0u, k_bad[lane] || gh[lane] != gh[lane]);
        const int bad_from = bad_rows ? __ffs(bad_rows) - 1 : C;

        float o[4][4];
        int se[2];
        bool wide = false;  // the outputs' parts have powers of two that are not normal numbers: applied in two factors
        const int c_exp = kScoreUnit - k_up;
        if (OUT) {
            // scores: 16 x 8 tiles (the two right of the diagonal are never read), in units of q's power of two and
            // 2^kScoreUnit. Three bf16 terms hold a score, and one of v, without a power of two that rows share: it
            // would be that of the largest, be it after a row or forgotten before it.
            const float k_scale = pow2(ke + k_up);
            for (int i = warp; i < 6; i += nw) {
                const int mi = i < 2 ? 0 : 1, nj = i < 2 ? i : i - 2;
                float cross[4] = {0, 0, 0, 0}, main[2][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
                const uint32_t qa = base + plan.q16 + (mi * 16 + (lane & 15)) * PITCH + (lane >> 4) * 16;
                const uint32_t kb = base + plan.k16 + (nj * 8 + (lane & 7)) * PITCH + ((lane >> 3) & 1) * 16;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t ah[4], al[4], bh[2], bl[2];
                    ldm4(ah, qa + ks * 32);
                    ldm4(al, qa + ks * 32 + plan.term);
                    ldm2(bh, kb + ks * 32);
                    ldm2(bl, kb + ks * 32 + plan.term);
                    mma(cross, al, bh[0], bh[1]);
                    mma(cross, ah, bl[0], bl[1]);
                    mma(main[ks & 1], ah, bh[0], bh[1]);
                }
                const int c = nj * 8 + 2 * t;
                const float2 ch = *reinterpret_cast<const float2 *>(gh + c), cl = *reinterpret_cast<const float2 *>(gl + c);
                const float k0 = __shfl_sync(~0u, k_scale, c), k1 = __shfl_sync(~0u, k_scale, c + 1);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int r = mi * 16 + 8 * u + g;
                    const float rh = gh[r], rl = gl[r];
                    constexpr float unit = 1.0f / (1 << kScoreUnit);
                    const float dot0 = (main[0][2 * u] + main[1][2 * u] + cross[2 * u]) * unit;
                    const float dot1 = (main[0][2 * u + 1] + main[1][2 * u + 1] + cross[2 * u + 1]) * unit;
                    const float v0 = c <= r ? dot0 * exp2f((rh - ch.x) + (rl - cl.x)) * k0 : 0.0f;
                    const float v1 = c + 1 <= r ? dot1 * exp2f((rh - ch.y) + (rl - cl.y)) * k1 : 0.0f;
                    uint32_t terms[3];
                    cut3(v0, v1, terms);
                    uint8_t *const dst = smem + plan.p16 + r * kPPitch + c * 2;
#pragma unroll
                    for (int x = 0; x < 3; ++x) *reinterpret_cast<uint32_t *>(dst + x * plan.p_term) = terms[x];
                }
            }

            // what the state gives: S^T Q^T
            float top[2] = {0, 0}, up[2];
#pragma unroll
            for (int n = 0; n < 2 * KS; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) top[i >> 1] = fmaxf(top[i >> 1], fabsf(s[n][i]));
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                se[u] = exponent_of(top_over_4(top[u]));
                up[u] = up_for(se[u]);
            }
            const int q_e = q_exp[lane], q_low = __reduce_min_sync(~0u, q_e), q_high = __reduce_max_sync(~0u, q_e);
            wide = __any_sync(~0u, q_low + min(c_exp, min(se[0], se[1])) < -126 || q_high + max(c_exp, max(se[0], se[1])) > 127);
#pragma unroll
            for (int k2 = 0; k2 < KS; k2 += 2) {
                float c[4][4];
                uint32_t ah[2][4], al[2][4];
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const float(&x)[4] = s[2 * (k2 + k) + n];
                            split2(x[2 * u] * up[u], x[2 * u + 1] * up[u], ah[k][2 * n + u], al[k][2 * n + u]);
                        }
                const uint32_t qb = base + plan.q16 + ((lane & 7) + ((lane >> 4) << 3)) * PITCH + ((lane >> 3) & 1) * 16 + k2 * 32;
#pragma unroll
                for (int np = 0; np < 2; ++np) {
                    uint32_t bh[2][4], bl[2][4];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        ldm4(bh[k], qb + np * 16 * PITCH + k * 32);
                        ldm4(bl[k], qb + np * 16 * PITCH + k * 32 + plan.term);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float(&d)[4] = c[2 * np + h];
                        mma_new(d, al[0], bh[0][2 * h], bh[0][2 * h + 1]);
                        mma(d, ah[0], bl[0][2 * h], bl[0][2 * h + 1]);
                        mma(d, al[1], bh[1][2 * h], bh[1][2 * h + 1]);
                        mma(d, ah[1], bl[1][2 * h], bl[1][2 * h + 1]);
                        mma(d, ah[0], bh[0][2 * h], bh[0][2 * h + 1]);
                        mma(d, ah[1], bh[1][2 * h], bh[1][2 * h + 1]);
                    }
                }
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[n][i] = k2 ? o[n][i] + c[n][i] : c[n][i];
            }
            __syncthreads();  // scores are there
        }

        // this warp's dims of v, of which each lane has its own: rows 16 k + 2t, +1, +8, +9, dims g and g + 8
        const int v_pitch = tile_cols + 4;
        float *const vp = reinterpret_cast<float *>(smem + plan.raw_v + buffer * plan.v_bytes) + 2 * t * v_pitch + warp * 16 + g;
        auto v_at = [&](int k, int u, int i) -> float & { return vp[(16 * k + (i & 1) + 8 * (i >> 1)) * v_pitch + 8 * u]; };
        int v_bad[2] = {C, C};  // first row of each dim that is not finite
        int v_up[2] = {0, 0};
        {
            float v_top[2] = {0, 0};
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) v_top[u] = top_of(v_top[u], v_at(k, u, i));
            auto plain = [](float top) { return __float_as_uint(top) - kTinyBits < 0x7F800000u - kTinyBits; };  // neither tiny nor not finite
            if (__any_sync(~0u, !plain(v_top[0]) || !plain(v_top[1]))) {
                // tiny ones are multiplied up; those that are not finite must not meet the zeros of rows before them: they
                // are taken out, and the dim's rows from them on become NaN
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (__float_as_uint(top_over_4(v_top[u])) < kTinyBits) v_up[u] = kTinyUp;
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (exponent_bits(v_at(k, u, i)) == 255) {
                                v_bad[u] = min(v_bad[u], 16 * k + 2 * t + (i & 1) + 8 * (i >> 1));
                                v_at(k, u, i) = 0.0f;
                            }
                    v_bad[u] = min(v_bad[u], __shfl_xor_sync(~0u, v_bad[u], 1));
                    v_bad[u] = min(v_bad[u], __shfl_xor_sync(~0u, v_bad[u], 2));
                }
            }
        }

        if (OUT) {
            // what the chunk's own rows give: V^T P^T, products of terms down to 2^-16 of the first ones'
            float c[4][4] = {};
            uint32_t first[2][4];
            const float v_scale[2] = {pow2_of(v_up[0]), pow2_of(v_up[1])};
            const uint32_t pb = base + plan.p16 + ((lane & 7) + ((lane >> 4) << 3)) * kPPitch + ((lane >> 3) & 1) * 16;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t a[3][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t terms[3];
                    cut3(v_at(k, i & 1, 2 * (i >> 1)) * v_scale[i & 1], v_at(k, i & 1, 2 * (i >> 1) + 1) * v_scale[i & 1], terms);
#pragma unroll
                    for (int x = 0; x < 3; ++x) a[x][i] = terms[x];
                    first[k][i] = terms[0];
                }
#pragma unroll
                for (int np = k; np < 2; ++np) {
                    uint32_t b[3][4];
#pragma unroll
                    for (int x = 0; x < 3; ++x) ldm4(b[x], pb + np * 16 * kPPitch + k * 32 + x * plan.p_term);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float(&d)[4] = c[2 * np + h];
                        mma_bf(d, a[2], b[0][2 * h], b[0][2 * h + 1]);
                        mma_bf(d, a[1], b[1][2 * h], b[1][2 * h + 1]);
                        mma_bf(d, a[0], b[2][2 * h], b[2][2 * h + 1]);
                        mma_bf(d, a[1], b[0][2 * h], b[0][2 * h + 1]);
                        mma_bf(d, a[0], b[1][2 * h], b[1][2 * h + 1]);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int np = k; np < 2; ++np) {
                    uint32_t b[4];
                    ldm4(b, pb + np * 16 * kPPitch + k * 32);
#pragma unroll
                    for (int h = 0; h < 2; ++h) mma_bf(c[2 * np + h], first[k], b[2 * h], b[2 * h + 1]);
                }
            const bool in_two = wide || __any_sync(~0u, v_up[0] + v_up[1]);
            auto join = [&](auto two) {
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float2 a = *reinterpret_cast<const float2 *>(from_start + 8 * n + 2 * t);
                    const int2 e = *reinterpret_cast<const int2 *>(q_exp + 8 * n + 2 * t);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int of_state = (i & 1 ? e.y : e.x) + se[i >> 1], of_chunk = (i & 1 ? e.y : e.x) + c_exp;
                        const float x = o[n][i] * (i & 1 ? a.y : a.x);
                        if constexpr (two) o[n][i] = times_pow2(x, of_state) + times_pow2(c[n][i], of_chunk - v_up[i >> 1]);
                        else o[n][i] = fmaf(c[n][i], pow2_of(of_chunk), x * pow2_of(of_state));
                        o[n][i] *= l.scale;
                    }
                }
            };
            if (in_two) join(std::true_type{});
            else join(std::false_type{});
            if (__any_sync(~0u, min(bad_from, min(v_bad[0], v_bad[1])) < C)) {
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (8 * n + 2 * t + (i & 1) >= min(bad_from, v_bad[i >> 1])) o[n][i] = NAN;
            }
            const int lo = (int)max((int64_t)0, span.first - row), rows = (int)min((int64_t)C, row1 - row) - lo;
            float *const out = l.out + (seq * l.n_new + row + 2 * t) * l.out_stride + head * l.dv + mine;
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int w = 0; w < 2; ++w)
                    if ((uint32_t)(8 * n + 2 * t + w - lo) < (uint32_t)rows) {
                        float *const dst = out + (8 * n + w) * l.out_stride;
                        dst[0] = o[n][w];
                        dst[8] = o[n][2 + w];
                    }
        }

        // the state: S^T e^(G_C) + (V f)^T K, f_j = e^(G_C - G_j) and k_j's power of two
        {
            const float f = to_end[lane] * pow2(ke - k_top);
            uint32_t ah[2][4], al[2][4];
            // the products' own largest sets their power of two: an old row's v may be large and forgotten
            float v[2][2][4];  // [step][dim][row]
            float most[2] = {0, 0};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float fr[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) fr[i] = __shfl_sync(~0u, f, 16 * k + 2 * t + (i & 1) + 8 * (i >> 1));
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[k][u][i] = v_at(k, u, i) * fr[i];
                        most[u] = fmaxf(most[u], fabsf(v[k][u][i]));
                    }
            }
            int be[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                be[u] = exponent_of(top_over_4(most[u]));
                const float up = up_for(be[u]);
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[k][u][i] *= up;
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) split2(v[k][i & 1][2 * (i >> 1)], v[k][i & 1][2 * (i >> 1) + 1], ah[k][i], al[k][i]);
            const float keep = bad_from < C ? NAN : gh[4 * C];
            float gain[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) gain[u] = v_bad[u] < C ? NAN : pow2_of(min(max(k_top + be[u], -126), 127));
            // (as above; a loop of its own for this costs more registers than the branches in this one)
            const bool wide = __any_sync(~0u, !is_normal(k_top + be[0]) || !is_normal(k_top + be[1]));
            const uint32_t kb = base + plan.k16 + ((lane & 7) + (((lane >> 3) & 1) << 3)) * PITCH + (lane >> 4) * 16;
#pragma unroll
            for (int n2 = 0; n2 < KS; ++n2) {
                float c[2][4];
                uint32_t bh[2][4], bl[2][4];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    ldm4_trans(bh[k], kb + k * 16 * PITCH + n2 * 32);
                    ldm4_trans(bl[k], kb + k * 16 * PITCH + n2 * 32 + plan.term);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    mma_new(c[h], al[0], bh[0][2 * h], bh[0][2 * h + 1]);
                    mma(c[h], ah[0], bl[0][2 * h], bl[0][2 * h + 1]);
                    mma(c[h], al[1], bh[1][2 * h], bh[1][2 * h + 1]);
                    mma(c[h], ah[1], bl[1][2 * h], bl[1][2 * h + 1]);
                    mma(c[h], ah[0], bh[0][2 * h], bh[0][2 * h + 1]);
                    mma(c[h], ah[1], bh[1][2 * h], bh[1][2 * h + 1]);
                }
                if (wide) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int e = k_top + be[i >> 1];
                            c[h][i] *= pow2(e - min(max(e, -126), 127));
                        }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[2 * n2 + h][i] = fmaf(c[h][i], gain[i >> 1], s[2 * n2 + h][i] * keep);
            }
        }
    }

    if (OUT) {
        if (last) store(l.state_out + which * size);
    } else {
        store(p.starts + ((seg + 1) * states + which) * size);
        if (sums_decays && lane == 0 && tile == 0) p.seg_decay[(seg + 1) * states + which] = (float)seg_total;
    }
}

constexpr int kScanThreads = 256, kScanAhead = 8;

// From the end states E_i that the segments come to from zeros (in the place of
// segment i + 1; the first one's from the call's state) to the states before
// them: S_1 = E_0, S_(i+1) = e^(G_i) S_i + E_i. A float4 per thread.
__global__ void __launch_bounds__(kScanThreads) scan_kernel(const __grid_constant__ ChunkParams p) {
    pdl_wait_prev();
    pdl_launch_dependents();
    const int64_t states = (int64_t)p.l.n_seqs * p.l.n_heads, size = (int64_t)p.l.dk * p.l.dv;
    const int64_t i = ((int64_t)blockIdx.x * kScanThreads + threadIdx.x) * 4;
    if (i >= states * size) return;
    const int64_t which = i / size;
    if (span_of(p.l, (int)(which / p.l.n_heads)).idle) return;
    float4 s = *reinterpret_cast<const float4 *>(p.starts + states * size + i);
    // the loads of eight segments at once (one after the other: 14 us for 19 segments of 1 MB)
    for (int first = 2; first < p.split.segments; first += kScanAhead) {
        float4 e[kScanAhead];
        float a[kScanAhead];
#pragma unroll
        for (int j = 0; j < kScanAhead; ++j) {
            const int seg = min(first + j, p.split.segments - 1);
            e[j] = *reinterpret_cast<const float4 *>(p.starts + seg * states * size + i);
            a[j] = exp2f(p.seg_decay[seg * states + which]);
        }
#pragma unroll
        for (int j = 0; j < kScanAhead; ++j) {
            if (first + j >= p.split.segments) break;
            s.x = fmaf(s.x, a[j], e[j].x);
            s.y = fmaf(s.y, a[j], e[j].y);
            s.z = fmaf(s.z, a[j], e[j].z);
            s.w = fmaf(s.w, a[j], e[j].w);
            *reinterpret_cast<float4 *>(p.starts + (first + j) * states * size + i) = s;
        }
    }
}

cudaError_t launch(void (*kernel)(ChunkParams), const ChunkParams &p, int64_t grid, int threads, int smem, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int DK>
cudaError_t launch_dk(const ChunkParams &p, cudaStream_t s) {
    constexpr int most = plan_of(DK, 16 * kMaxWarps).bytes;
    static OncePerDevice once[2];
    cudaError_t e = allow_smem(once[0], chunk_kernel<DK, true>, most);
    if (e == cudaSuccess) e = allow_smem(once[1], chunk_kernel<DK, false>, most);
    if (e != cudaSuccess) return e;
    const int threads = p.split.tile / 16 * 32, smem = plan_of(DK, p.split.tile).bytes;
    const int64_t ctas = (int64_t)p.l.n_seqs * p.l.n_heads * p.split.tiles;
    if (p.split.segments > 1) {
        e = launch(chunk_kernel<DK, false>, p, ctas * (p.split.segments - 1), threads, smem, s);
        if (e != cudaSuccess) return e;
        const int64_t quads = (int64_t)p.l.n_seqs * p.l.n_heads * p.l.dk * p.l.dv / 4;
        e = launch(scan_kernel, p, (quads + kScanThreads - 1) / kScanThreads, kScanThreads, 0, s);
        if (e != cudaSuccess) return e;
    }
    return launch(chunk_kernel<DK, true>, p, ctas * p.split.segments, threads, smem, s);
}

size_t starts_bytes(const Linear &l, const Split &split) {
    return (size_t)split.segments * (size_t)l.n_seqs * (size_t)l.n_heads * (size_t)l.dk * (size_t)l.dv * 4;
}

}  // namespace

size_t chunks_workspace_bytes(const Linear &l, const Split &split) {
    if (split.segments < 2) return 0;
    return starts_bytes(l, split) + (size_t)split.segments * (size_t)l.n_seqs * (size_t)l.n_heads * 4;
}

cudaError_t launch_chunks(const Linear &l, const Split &split, const DeviceInfo &, cudaStream_t s) {
    ChunkParams p;
    p.l = l;
    p.split = split;
    p.starts = static_cast<float *>(l.workspace);
    p.seg_decay = split.segments > 1 ? reinterpret_cast<float *>(static_cast<uint8_t *>(l.workspace) + starts_bytes(l, split))
                                     : nullptr;
    switch (l.dk) {
    case 32: return launch_dk<32>(p, s);
    case 64: return launch_dk<64>(p, s);
    case 96: return launch_dk<96>(p, s);
    case 128: return launch_dk<128>(p, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace linear

}  // namespace qmm
