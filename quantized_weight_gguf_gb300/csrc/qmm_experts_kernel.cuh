// qmm_experts_kernel.cuh -- the two products of the experts' feed-forward
// network over pairs sorted by expert: h = act(x Wg) (x Wu) w, then h Wd.
//
// A unit of work is a tile (up to 8 NT pairs of one expert) times a block of
// rows of its matrix. Every warp takes 32 rows as two m16 tiles: of the first
// product the same 16 rows of the gate and of the up matrix, so that act(g) u
// happens in registers; of the second 32 rows of the down matrix. The k loop
// runs over chunks (chunk_k weights): each warp copies its own rows' bytes and
// the CTA's warps share the activations' terms, both by cp.async into the stage
// after the one being multiplied, also across units.
#pragma once

#include "qmm_experts.h"
#include "qmm_experts_frag.cuh"

namespace qmm {
namespace experts {

// Warps per CTA: four where a tile has 8 columns (more, smaller units: a few
// tokens' work has to reach every SM), eight above (the activations' stage is
// shared by more rows).
__host__ __device__ constexpr int warps_of(int nt) { return nt == 1 ? 4 : 8; }
constexpr int kWarpRows = 32;

// Shared memory of a CTA: stages of {W rows, activations, scales}, then the
// first product's results on their way to becoming terms.
struct Layout {
    int w_bytes, x_bytes, s_bytes, stage, stages, h_bytes, smem, ctas;
};
__host__ __device__ constexpr Layout layout_of(int fmt, int nt, bool down) {
    Layout l = {};
    const int blocks = chunk_k(fmt) / 32;
    l.w_bytes = warps_of(nt) * kWarpRows * row_pitch(fmt);
    l.x_bytes = nt * 8 * blocks * frag_bytes(fmt);
    l.s_bytes = nt * 8 * blocks * 8;
    l.stage = l.w_bytes + l.x_bytes + l.s_bytes;
    // 16 columns of 16 values a warp, padded so that a fragment's stores meet no bank twice
    l.h_bytes = down ? 0 : nt * 8 * (warps_of(nt) * 16 + 4) * 4;
    // as many CTAs per SM as make 16 warps, if two stages of each fit (228 KB, 1 KB a CTA the system's)
    l.ctas = 16 / warps_of(nt);
    while (l.ctas > 1 && 2 * l.stage + l.h_bytes > 228 * 1024 / l.ctas - 1024) --l.ctas;
    l.stages = (228 * 1024 / l.ctas - 1024 - l.h_bytes) / l.stage;
    if (l.stages > 4) l.stages = 4;
    l.smem = l.stages * l.stage + l.h_bytes;
    return l;
}

// 8-byte asynchronous copy
__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// What the copies need of a unit.
template <int XR>
struct Source {
    const uint8_t *row[2][2];  // this lane's rows of W: [m16 tile][upper 8]
    int64_t x_row[XR];         // activation rows that this warp copies; -1: none
};

template <int FMT, int NT, bool DOWN>
__global__ void __launch_bounds__(warps_of(NT) * 32, layout_of(FMT, NT, DOWN).ctas)
    product_kernel(const __grid_constant__ ProductParams p) {
    constexpr Layout L = layout_of(FMT, NT, DOWN);
    constexpr int W = warps_of(NT), TN = NT * 8, NS = L.stages;
    constexpr int KB = chunk_k(FMT) / 32;               // blocks per chunk
    constexpr int FB = frag_bytes(FMT), TERMS = terms_of(FMT);
    constexpr int PITCH = row_pitch(FMT), NP = chunk_pieces(FMT);
    constexpr int CTA_ROWS = W * (DOWN ? 32 : 16);
    constexpr int XR = TN / W;
    constexpr int HP = W * 16 + 4;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t smem0 = smem_addr(smem);

    pdl_wait_prev();
    pdl_launch_dependents();

    const int row_blocks = (p.rows + CTA_ROWS - 1) / CTA_ROWS;
    const int units = *p.n_tiles * row_blocks;
    const int chunks = (p.blocks + KB - 1) / KB;
    const int mine = (int)blockIdx.x < units ? (units - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x : 0;
    const int64_t steps = (int64_t)mine * chunks;

    // ---- copies: the unit and chunk that are loaded next ----
    Source<XR> src;
    int load_unit = blockIdx.x, load_chunk = 0;
    // first row of this warp's m16 tile m in a block of rows
    auto first_row = [&](int block, int m) {
        return block * CTA_ROWS + (DOWN ? warp * 32 + m * 16 : warp * 16);
    };
    auto open_unit = [&](int unit) {
        const Tile tile = p.tiles[unit / row_blocks];
        const int block = unit % row_blocks;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const uint8_t *base = p.w[m] + tile.expert * p.slice_bytes;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                // rows past the end are copies of the last one; their results are dropped
                const int r = min(first_row(block, m) + 8 * u + g, p.rows - 1);
                src.row[m][u] = base + r * p.row_bytes;
            }
        }
#pragma unroll
        for (int i = 0; i < XR; ++i) {
            const int c = warp + W * i;
            src.x_row[i] = c >= tile.count ? -1 : DOWN ? tile.start + c : p.order[tile.start + c] / p.top_k;
        }
    };
    auto load = [&](int slot) {
        const uint32_t at = smem0 + slot * L.stage;
        // W: four lanes a row, 16 bytes each in turn
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint32_t dst = at + (warp * kWarpRows + m * 16 + u * 8 + g) * PITCH;
                if constexpr (FMT == F_Q4_K) {
                    // header, then half of the codes
                    const uint8_t *b = src.row[m][u] + (load_chunk >> 1) * 144;
                    const uint8_t *codes = b + 16 + 64 * (load_chunk & 1);
                    if (t == 0) cp_async16(dst, b, 16);
                    cp_async16(dst + 16 + 16 * t, codes + 16 * t, 16);
                } else {
                    const uint8_t *b = src.row[m][u] + (int64_t)load_chunk * chunk_bytes(FMT);
                    const int64_t left = p.row_bytes - (int64_t)load_chunk * chunk_bytes(FMT);
                    const int off = (int)(reinterpret_cast<uintptr_t>(b) & 15u);
                    // bytes from the first piece's start to the chunk's end; what follows is zeros
                    const int end = off + (left < chunk_bytes(FMT) ? (int)left : chunk_bytes(FMT));
                    const uint8_t *b0 = b - off;
#pragma unroll
                    for (int i = 0; i < (NP + 3) / 4; ++i) {
                        const int piece = 4 * i + t, n = end - 16 * piece;
                        if (piece < NP) cp_async16(dst + 16 * piece, b0 + (n > 0 ? 16 * piece : 0), n <= 0 ? 0 : n < 16 ? n : 16);
                    }
                }
            }
        // activations: a row's blocks of the chunk lie one after the other
#pragma unroll
        for (int i = 0; i < XR; ++i) {
            if (src.x_row[i] < 0) continue;
            const int c = warp + W * i, cg = c & 7;
            const uint32_t xs = at + L.w_bytes + (c >> 3) * (KB * 8 * FB);
            const uint8_t *from = p.x + src.x_row[i] * p.x_row_bytes + (int64_t)load_chunk * (KB * FB);
#pragma unroll
            for (int j = 0; j < (KB * FB / 16 + 31) / 32; ++j) {
                const int piece = 32 * j + lane;
                if (piece >= KB * FB / 16) break;
                const int b = piece / (FB / 16);
                int q = piece % (FB / 16);
                // odd columns hold their two terms in the other order (no bank is met twice); three
                // terms' 192 bytes fall well by themselves
                if (TERMS == 2) q ^= (cg & 1) << 2;
                cp_async16(xs + (b * 8 + cg) * FB + 16 * q, from + 16 * piece, 16);
            }
            if (lane < KB)
                cp_async8(at + L.w_bytes + L.x_bytes + ((c >> 3) * KB + lane) * 64 + cg * 8,
                          p.x_scale + src.x_row[i] * p.x_blocks + (int64_t)load_chunk * KB + lane);
        }
    };
    auto load_next = [&](int64_t step, int slot) {
        if (step < steps) {
            if (load_chunk == 0) open_unit(load_unit);
            load(slot);
            if (++load_chunk == chunks) {
                load_chunk = 0;
                load_unit += gridDim.x;
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < NS - 1; ++i) load_next(i, i);

    // ---- products ----
    float acc[2][NT][4];
    int unit = blockIdx.x, chunk = 0, slot = 0, block = 0;
    Tile tile = {};
    uint32_t start[2][2] = {};  // low bits of this lane's rows' addresses
    for (int64_t step = 0; step < steps; ++step) {
        cp_async_wait<NS - 2>();
        __syncthreads();  // the stage is there for all, and the one before it is free
        load_next(step + NS - 1, slot == 0 ? NS - 1 : slot - 1);
        if (chunk == 0) {
            tile = p.tiles[unit / row_blocks];
            block = unit % row_blocks;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    start[m][u] = (uint32_t)(reinterpret_cast<uintptr_t>(p.w[m]) + tile.expert * p.slice_bytes +
                                             min(first_row(block, m) + 8 * u + g, p.rows - 1) * p.row_bytes);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
            }
        }
        if (first_row(block, 0) < p.rows) {
            const uint8_t *stage = smem + slot * L.stage;
            const uint8_t *xs = stage + L.w_bytes, *ss = xs + L.x_bytes;
            const uint8_t *rows[2][2];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t off = FMT == F_Q4_K ? 0 : (start[m][u] + (uint32_t)(chunk * chunk_bytes(FMT))) & 15u;
                    rows[m][u] = stage + (warp * kWarpRows + m * 16 + u * 8 + g) * PITCH + off;
                }
            const int here = min(KB, p.blocks - chunk * KB);
            constexpr int G = Row<FMT>::kGroup;
#pragma unroll
            for (int grp = 0; grp < KB / G; ++grp) {
                if (grp * G >= here) break;
                Row<FMT> lo[2], hi[2];
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    lo[m].load(rows[m][0], grp, chunk & 1, t);
                    hi[m].load(rows[m][1], grp, chunk & 1, t);
                }
#pragma unroll
                for (int sub = 0; sub < G; ++sub) {
                    const int b = grp * G + sub;  // blocks of a group are all there or none (k % 64, 128 or 256 = 0)
                    uint32_t a[2][8];
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        uint32_t r[4], s[4];
                        lo[m].pairs(sub, r);
                        hi[m].pairs(sub, s);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            a[m][2 * i] = r[i];
                            a[m][2 * i + 1] = s[i];
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint8_t *rec = xs + ((n * KB + b) * 8 + g) * FB + 16 * t;
                        uint4 x[TERMS];
#pragma unroll
                        for (int i = 0; i < TERMS; ++i)
                            x[i] = *reinterpret_cast<const uint4 *>(rec + 64 * (TERMS == 2 ? i ^ (g & 1) : i));
                        // columns 2t and 2t + 1: scale, sum, scale, sum
                        const float4 sc = *reinterpret_cast<const float4 *>(ss + (n * KB + b) * 64 + 16 * t);
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            float(&o)[4] = acc[m][n];
                            if constexpr (FMT == F_BF16) {
                                float c[4] = {0, 0, 0, 0};
#pragma unroll
                                for (int i = 0; i < TERMS; ++i) {
                                    mma_bf16(c, a[m], x[i].x, x[i].y);
                                    mma_bf16(c, a[m] + 4, x[i].z, x[i].w);
                                }
#pragma unroll
                                for (int i = 0; i < 4; ++i) o[i] += c[i];
                            } else if constexpr (Row<FMT>::kScales == 2) {
#pragma unroll
                                for (int u = 0; u < 2; ++u) {
                                    float c[4] = {0, 0, 0, 0};
#pragma unroll
                                    for (int i = 0; i < TERMS; ++i)
                                        mma_f16(c, a[m] + 4 * u, u ? x[i].z : x[i].x, u ? x[i].w : x[i].y);
                                    const float dl = lo[m].scale(sub, u), dh = hi[m].scale(sub, u);
                                    o[0] = fmaf(c[0], dl * sc.x, o[0]);
                                    o[1] = fmaf(c[1], dl * sc.z, o[1]);
                                    o[2] = fmaf(c[2], dh * sc.x, o[2]);
                                    o[3] = fmaf(c[3], dh * sc.z, o[3]);
                                }
                            } else {
                                float c[4] = {0, 0, 0, 0};
#pragma unroll
                                for (int i = 0; i < TERMS; ++i) {
                                    mma_f16(c, a[m], x[i].x, x[i].y);
                                    mma_f16(c, a[m] + 4, x[i].z, x[i].w);
                                }
                                const float dl = lo[m].scale(sub, 0), dh = hi[m].scale(sub, 0);
                                o[0] = fmaf(c[0], dl * sc.x, o[0]);
                                o[1] = fmaf(c[1], dl * sc.z, o[1]);
                                o[2] = fmaf(c[2], dh * sc.x, o[2]);
                                o[3] = fmaf(c[3], dh * sc.z, o[3]);
                                if (Row<FMT>::kMin) {
                                    const float ml = lo[m].min(sub), mh = hi[m].min(sub);
                                    o[0] = fmaf(ml, sc.y, o[0]);
                                    o[1] = fmaf(ml, sc.w, o[1]);
                                    o[2] = fmaf(mh, sc.y, o[2]);
                                    o[3] = fmaf(mh, sc.w, o[3]);
                                }
                            }
                        }
                    }
                }
            }
        }
        if (++slot == NS) slot = 0;
        if (++chunk < chunks) continue;

        // ---- the unit's results ----
        if constexpr (DOWN) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int c = n * 8 + 2 * t + u;
                    if (c >= tile.count) continue;
                    float *out = p.out + (int64_t)p.order[tile.start + c] * p.rows;
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const int r = first_row(block, m) + g;
                        if (r < p.rows) out[r] = acc[m][n][u];
                        if (r + 8 < p.rows) out[r + 8] = acc[m][n][2 + u];
                    }
                }
        } else {
            float *hs = reinterpret_cast<float *>(smem + NS * L.stage);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int c = n * 8 + 2 * t + u;
                    if (c >= tile.count) continue;
                    const float w = p.weights[p.order[tile.start + c]];
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const int r = warp * 16 + 8 * v + g;
                        const float gate = acc[0][n][2 * v + u], up = acc[1][n][2 * v + u];
                        const float h = glu_gate(gate, glu_arg(p.act, gate)) * up * w;
                        hs[c * HP + r] = block * CTA_ROWS + r < p.rows ? h : 0.0f;
                    }
                }
            __syncthreads();
            // blocks of 32 rows of every column
            constexpr int HB = CTA_ROWS / 32;
            for (int i = warp; i < tile.count * HB; i += W) {
                const int c = i / HB, b = i % HB, at = block * HB + b;
                if (at >= p.h_blocks) continue;
                const int64_t row = tile.start + c;
                const float v = hs[c * HP + 32 * b + lane];
                uint8_t *rec = p.h + row * p.h_row_bytes + (int64_t)at * 64 * (p.h_bf16 ? 3 : 2);
                const float2 s = put_block(v, lane, p.h_bf16, rec);
                if (lane == 0) p.h_scale[row * p.h_blocks + at] = s;
            }
            // the next unit's results come after the next barrier at the earliest
        }
        chunk = 0;
        unit += gridDim.x;
    }
    cp_async_wait<0>();
}

template <int FMT, int NT, bool DOWN>
cudaError_t launch_one(const ProductParams &p, int max_tiles, const DeviceInfo &dev, cudaStream_t s) {
    constexpr Layout L = layout_of(FMT, NT, DOWN);
    static_assert(L.stages >= 2, "two stages");
    constexpr int CTA_ROWS = warps_of(NT) * (DOWN ? 32 : 16);
    static OncePerDevice once;
    cudaError_t e = allow_smem(once, product_kernel<FMT, NT, DOWN>, L.smem);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)max_tiles * ((p.rows + CTA_ROWS - 1) / CTA_ROWS);
    const int64_t wave = (int64_t)dev.sm_count * L.ctas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units < wave ? units : wave));
    cfg.blockDim = dim3(warps_of(NT) * 32);
    cfg.dynamicSmemBytes = L.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, product_kernel<FMT, NT, DOWN>, p);
}

template <int FMT>
cudaError_t launch_product(bool down, int columns, const ProductParams &p, int max_tiles, const DeviceInfo &dev,
                           cudaStream_t s) {
    if (down) {
        if (columns == 8) return launch_one<FMT, 1, true>(p, max_tiles, dev, s);
        if (columns == 16) return launch_one<FMT, 2, true>(p, max_tiles, dev, s);
        return launch_one<FMT, 4, true>(p, max_tiles, dev, s);
    }
    if (columns == 8) return launch_one<FMT, 1, false>(p, max_tiles, dev, s);
    if (columns == 16) return launch_one<FMT, 2, false>(p, max_tiles, dev, s);
    return launch_one<FMT, 4, false>(p, max_tiles, dev, s);
}

}  // namespace experts
}  // namespace qmm
