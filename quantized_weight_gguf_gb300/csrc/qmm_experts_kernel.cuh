// qmm_experts_kernel.cuh -- the two products of the experts' feed-forward
// network over pairs sorted by expert: h = act(x Wg) (x Wu) w, then h Wd.
//
// A unit of work is a tile (pairs of one expert) times a block of rows of its
// matrix. The k loop runs over chunks (chunk_k weights): each warp copies its own rows' bytes
// and the CTA's warps share the activations' terms, both by cp.async into a
// later stage than the one being multiplied, also across units.
//
// Bound by unpacking and scales, about 130 instructions per 16 x 16 x 32 of Q4_K, of which 8 are products (issue slots 58
// to 68 % used, tensor pipe 17 to 29 %); BF16 weights by their three terms and DRAM. Measured: 24 positions of 1536 x 640, six of 40,
// BF16 56 us (0.61 of the copy rate); Q4_K 2048 x 768, eight of 64, 8 rows an expert 147 us, 16 rows 186 us.
#pragma once

#include "qmm_experts.h"
#include "qmm_experts_frag.cuh"

namespace qmm {
namespace experts {

// How a tile of 8 or 16 activation rows is worked on: by 8 warps of
// `m_tiles` tiles of 16 rows each. With 8 columns, where the work is decoding, one tile a warp, so
// that few registers let many warps hide one another's latencies; of the first product, half of the
// warps take gate's rows and half the same rows of up. Above, where activations' terms are read
// most, two tiles a warp share them, gate's and up's of the same rows. (Single rows:
// qmm_experts_rows.cuh.)
struct Shape {
    int warps, m_tiles, n_tiles, ctas;
};
__host__ __device__ constexpr Shape shape_of(int columns) {
    return columns == 8 ? Shape{8, 1, 1, 3} : Shape{8, 2, columns / 8, 2};
}
// Rows of a CTA's block.
__host__ __device__ constexpr int cta_rows(int columns, bool down) {
    return shape_of(columns).warps * shape_of(columns).m_tiles * 16 / (down ? 1 : 2);
}

// Shared memory of a CTA: stages of {W rows, activations, scales}, then the
// first product's results on their way to becoming terms.
struct Layout {
    int w_bytes, x_bytes, s_bytes, stage, stages, h_bytes, smem, ctas;
};
__host__ __device__ constexpr Layout layout_of(int fmt, int columns, bool down, bool even) {
    Layout l = {};
    const Shape s = shape_of(columns);
    const int blocks = chunk_k(fmt) / 32;
    l.w_bytes = s.warps * s.m_tiles * 16 * row_pitch(fmt, even);
    l.x_bytes = columns * blocks * frag_bytes(fmt);
    l.s_bytes = columns * blocks * 8;
    l.stage = l.w_bytes + l.x_bytes + l.s_bytes;
    // gate's sums and the products of a column's rows, padded so that a fragment's stores meet no bank twice
    l.h_bytes = down ? 0 : columns * (cta_rows(columns, false) + 4) * 4;
    // as many CTAs per SM as planned, if two stages of each fit (228 KB, 1 KB a CTA the system's)
    l.ctas = s.ctas;
    while (l.ctas > 1 && 2 * l.stage + l.h_bytes > 228 * 1024 / l.ctas - 1024) --l.ctas;
    l.stages = (228 * 1024 / l.ctas - 1024 - l.h_bytes) / l.stage;
    if (l.stages > 4) l.stages = 4;
    l.smem = l.stages * l.stage + l.h_bytes;
    return l;
}

// 4-byte asynchronous copy
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A group of blocks of 32 (see Row) of MT m16 tiles times NT tiles of 8 columns, added to
// acc[tile][columns][row g, row g + 8][column 2t, 2t + 1] of lane (g, t). xs: terms of the columns in the order
// [tile of columns][block][column][term], this lane's column and place; ss: their powers of two
// [tile of columns][block][column], the lane's columns, and after them the sums. Blocks of a group
// are all there or none.
template <int FMT, int MT, int NT, bool EVEN>
__device__ __forceinline__ void multiply_group(const RowAt<EVEN> (&rows)[MT][2], int grp, int half, int g, int t,
                                               const uint8_t *xs, const uint8_t *ss, float (&acc)[MT][NT][4]) {
    constexpr int G = Row<FMT>::kGroup, FB = frag_bytes(FMT), TERMS = terms_of(FMT), KB = chunk_k(FMT) / 32;
    Row<FMT> lo[MT], hi[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        lo[m].load(rows[m][0], grp, half, t);
        hi[m].load(rows[m][1], grp, half, t);
    }
#pragma unroll
    for (int sub = 0; sub < G; ++sub) {
        const int b = grp * G + sub;
        uint32_t a[MT][8];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
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
            const uint8_t *rec = xs + (n * KB + b) * 8 * FB;
            uint4 x[TERMS];
#pragma unroll
            for (int i = 0; i < TERMS; ++i)
                x[i] = *reinterpret_cast<const uint4 *>(rec + 64 * (TERMS == 2 ? i ^ (g & 1) : i));
            // columns 2t and 2t + 1
            float2 scales = {}, sums = {};
            if (FMT != F_BF16) {
                const uint8_t *q = ss + (n * KB + b) * 32;
                scales = *reinterpret_cast<const float2 *>(q);
                if (Row<FMT>::kMin) sums = *reinterpret_cast<const float2 *>(q + NT * KB * 32);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                float(&o)[4] = acc[m][n];
                // sums that different powers of two multiply are kept apart
                constexpr int STEPS = Row<FMT>::kScales == 2 ? 2 : 1;
#pragma unroll
                for (int u = 0; u < STEPS; ++u) {
                    // the low terms' products come first: the tensor cores cut what they add
                    float c[4];
                    constexpr int LAST = TERMS - 1;
                    if constexpr (FMT == F_BF16) {
                        mma_bf16_new(c, a[m], x[LAST].x, x[LAST].y);
                        mma_bf16(c, a[m] + 4, x[LAST].z, x[LAST].w);
#pragma unroll
                        for (int i = LAST - 1; i >= 0; --i) {
                            mma_bf16(c, a[m], x[i].x, x[i].y);
                            mma_bf16(c, a[m] + 4, x[i].z, x[i].w);
                        }
                    } else if constexpr (STEPS == 2) {
                        mma_f16_new(c, a[m] + 4 * u, u ? x[1].z : x[1].x, u ? x[1].w : x[1].y);
                        mma_f16(c, a[m] + 4 * u, u ? x[0].z : x[0].x, u ? x[0].w : x[0].y);
                    } else {
                        mma_f16_new(c, a[m], x[1].x, x[1].y);
                        mma_f16(c, a[m] + 4, x[1].z, x[1].w);
                        mma_f16(c, a[m], x[0].x, x[0].y);
                        mma_f16(c, a[m] + 4, x[0].z, x[0].w);
                    }
                    if constexpr (FMT == F_BF16) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[i] += c[i];
                    } else {
                        const float dl = FMT == F_F16 ? 1.0f : lo[m].scale(sub, u), dh = FMT == F_F16 ? 1.0f : hi[m].scale(sub, u);
                        o[0] = fmaf(c[0], dl * scales.x, o[0]);
                        o[1] = fmaf(c[1], dl * scales.y, o[1]);
                        o[2] = fmaf(c[2], dh * scales.x, o[2]);
                        o[3] = fmaf(c[3], dh * scales.y, o[3]);
                    }
                }
                if (Row<FMT>::kMin) {
                    const float ml = lo[m].min(sub), mh = hi[m].min(sub);
                    o[0] = fmaf(ml, sums.x, o[0]);
                    o[1] = fmaf(ml, sums.y, o[1]);
                    o[2] = fmaf(mh, sums.x, o[2]);
                    o[3] = fmaf(mh, sums.y, o[3]);
                }
            }
        }
    }
}

template <int FMT, int TN, bool DOWN, bool EVEN>
__global__ void __launch_bounds__(shape_of(TN).warps * 32, layout_of(FMT, TN, DOWN, EVEN).ctas)
    product_kernel(const __grid_constant__ ProductParams p) {
    constexpr Layout L = layout_of(FMT, TN, DOWN, EVEN);
    constexpr Shape S = shape_of(TN);
    constexpr int NT = S.n_tiles, MT = S.m_tiles, NS = L.stages;
    constexpr int TG = 8;                               // columns of a tile
    constexpr int KB = chunk_k(FMT) / 32;               // blocks per chunk
    constexpr int CB = chunk_bytes(FMT);
    constexpr int FB = frag_bytes(FMT), TERMS = terms_of(FMT);
    constexpr int PITCH = row_pitch(FMT, EVEN), NP = chunk_pieces(FMT, EVEN);
    constexpr int CTA_ROWS = cta_rows(TN, DOWN);
    constexpr bool APART = !DOWN && MT == 1;            // gate and up are different warps'
    constexpr int XR = TN / S.warps;
    constexpr int HP = CTA_ROWS + 4;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t smem0 = smem_addr(smem);
    const int x_at = L.w_bytes, s_at = x_at + L.x_bytes;

    pdl_wait_prev();

    const int row_blocks = (p.rows + CTA_ROWS - 1) / CTA_ROWS;
    const int units = *p.n_tiles * row_blocks;
    const int chunks = (p.blocks + KB - 1) / KB;
    const int mine = (int)blockIdx.x < units ? (units - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x : 0;
    const int steps = mine * chunks;

    // ---- copies: the unit and chunk that are loaded next ----
    int load_unit = blockIdx.x, load_chunk = 0;
    const uint8_t *load_base[MT] = {};  // this warp's first row of each tile
    int load_rows[MT] = {};             // the tile's rows that exist, less one (at least 0)
    int x_row[XR];                      // activation rows that this warp copies; -1: none
    // matrix and first row of this warp's m16 tile m in a block of rows
    const int matrix = APART ? warp & 1 : 0;
    const int in_block = APART ? warp / 2 * 16 : DOWN ? warp * MT * 16 : warp * 16;
    auto first_row = [&](int block, int m) { return block * CTA_ROWS + in_block + (DOWN ? m * 16 : 0); };
    auto base_of = [&](int m) { return p.w[APART ? matrix : DOWN ? 0 : m]; };
    auto open_unit = [&](int unit) {
        const Tile tile = p.tiles[unit / row_blocks];
        const int block = unit % row_blocks;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            // rows past the end are copies of the last one; their results are dropped
            const int first = min(first_row(block, m), p.rows - 1);
            load_base[m] = base_of(m) + tile.expert * p.slice_bytes + first * p.row_bytes;
            load_rows[m] = min(15, p.rows - 1 - first);
        }
#pragma unroll
        for (int i = 0; i < XR; ++i) {
            const int c = warp + S.warps * i;
            x_row[i] = c >= tile.count ? -1 : DOWN ? tile.start + c : p.order[tile.start + c] / p.top_k;
        }
    };
    // 16 bytes a lane, row after row: neighbouring lanes' copies share the sectors of L2 and the wavefronts of
    // the shared memory (with four lanes a row a copy of 512 bytes took 15 of these)
    constexpr int COPIES = (16 * NP + 31) / 32;
    int piece_at[COPIES];  // of a tile's first row
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
        const int piece = 32 * i + lane, row = piece / NP;
        piece_at[i] = row * (int)p.row_bytes + 16 * (piece - row * NP);
    }
    auto load = [&](int slot) {
        const uint32_t at = smem0 + slot * L.stage;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const uint32_t dst = at + (warp * MT + m) * 16 * PITCH;
            const int begin = FMT == F_Q4_K ? (load_chunk >> 1) * 144 : load_chunk * CB, from = begin & ~15;
            if (load_rows[m] == 15 && (FMT == F_Q4_K || (!EVEN && from + 16 * NP <= (int)p.row_bytes))) {
                const uint8_t *b = load_base[m] + from;
                const int half = 64 * (load_chunk & 1);  // (Q4_K: the header, then half of the codes)
#pragma unroll
                for (int i = 0; i < COPIES; ++i) {
                    const int piece = 32 * i + lane;
                    if ((16 * NP) % 32 && i + 1 == COPIES && piece >= 16 * NP) break;
                    const uint32_t to = PITCH == 16 * NP ? 16 * piece : piece / NP * PITCH + 16 * (piece % NP);
                    cp_async16(dst + to, b + piece_at[i] + (FMT == F_Q4_K && piece % NP ? half : 0), 16);
                }
            } else {
#pragma unroll 1
                for (int piece = lane; piece < 16 * NP; piece += 32) {
                    const int row = piece / NP, t = piece - row * NP;
                    const uint8_t *r = load_base[m] + min(row, load_rows[m]) * p.row_bytes;
                    const uint32_t to = dst + row * PITCH + 16 * t;
                    if (FMT == F_Q4_K) {
                        cp_async16(to, r + begin + 16 * t + (t ? 64 * (load_chunk & 1) : 0), 16);
                        continue;
                    }
                    const uint8_t *b = r + begin;
                    const int off = (int)(reinterpret_cast<uintptr_t>(b) & 15u);
                    // bytes past the chunk's end are zeros
                    const int n = off + min(CB, (int)p.row_bytes - begin) - 16 * t;
                    cp_async16(to, n > 0 ? b - off + 16 * t : b - off, n <= 0 ? 0 : n < 16 ? n : 16);
                }
            }
        }
        // activations: a row's blocks of the chunk lie one after the other
#pragma unroll
        for (int i = 0; i < XR; ++i) {
            const int c = warp + S.warps * i, cg = c & 7;
            if (x_row[i] < 0) continue;
            const uint32_t xs = at + x_at + (c >> 3) * (KB * TG * FB) + cg * FB;
            const uint8_t *from = p.x + (int64_t)x_row[i] * p.x_row_bytes + load_chunk * (KB * FB);
#pragma unroll
            for (int j = 0; j < (KB * FB / 16 + 31) / 32; ++j) {
                const int piece = 32 * j + lane;
                if (piece >= KB * FB / 16) break;
                const int b = piece / (FB / 16);
                int q = piece % (FB / 16);
                // odd columns hold their two terms in the other order (no bank is met twice); three
                // terms' 192 bytes fall well by themselves
                if (TERMS == 2) q ^= (cg & 1) << 2;
                cp_async16(xs + b * TG * FB + 16 * q, from + 16 * piece, 16);
            }
            if (FMT != F_BF16 && lane < KB) {
                const int64_t from_s = (int64_t)x_row[i] * p.x_blocks + load_chunk * KB + lane;
                const uint32_t to = at + s_at + (((c >> 3) * KB + lane) * TG + cg) * 4;
                cp_async4(to, p.x_scale + from_s);
                if (Row<FMT>::kMin) cp_async4(to + TN * KB * 4, p.x_sum + from_s);
            }
        }
    };
    auto load_next = [&](int step, int slot) {
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
    float acc[MT][NT][4];  // [m16 tile][columns][row g, g + 8][column 2t, 2t + 1]
    int unit = blockIdx.x, chunk = 0, slot = 0, block = 0;
    Tile tile = {};
    uint32_t start[MT][2] = {};  // low bits of this lane's rows' addresses
    for (int step = 0; step < steps; ++step) {
        cp_async_wait<NS - 2>();
        __syncthreads();  // the stage is there for all, and the one before it is free
        load_next(step + NS - 1, slot == 0 ? NS - 1 : slot - 1);
        if (chunk == 0) {
            tile = p.tiles[unit / row_blocks];
            block = unit % row_blocks;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    start[m][u] = (uint32_t)(reinterpret_cast<uintptr_t>(base_of(m)) + tile.expert * p.slice_bytes +
                                             min(first_row(block, m) + 8 * u + g, p.rows - 1) * p.row_bytes);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
            }
        }
        const int here = min(KB, p.blocks - chunk * KB);
        if (first_row(block, 0) < p.rows) {
            const uint8_t *stage = smem + slot * L.stage;
            const uint8_t *xs = stage + x_at + g * FB + 16 * t;
            const uint8_t *ss = stage + s_at + 8 * t;
            RowAt<EVEN> rows[MT][2];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t off = FMT == F_Q4_K ? 0 : ((EVEN ? start[m][u] : 0) + (uint32_t)(chunk * CB)) & 15u;
                    rows[m][u].set(stage + (warp * MT * 16 + m * 16 + u * 8 + g) * PITCH + off, off & 2u);
                }
            constexpr int G = Row<FMT>::kGroup;
            auto multiply = [&](int grp) {
                multiply_group<FMT, MT, NT, EVEN>(rows, grp, chunk & 1, g, t, xs, ss, acc);
            };
            // a whole chunk in one piece, so that its blocks' latencies overlap
            if (here == KB) {
#pragma unroll
                for (int grp = 0; grp < KB / G; ++grp) multiply(grp);
            } else {
#pragma unroll 1
                for (int grp = 0; grp * G < here; ++grp) multiply(grp);
            }
        }
        if (++slot == NS) slot = 0;
        if (++chunk < chunks) continue;

        // ---- the unit's results ----
        // values of this thread: [m16 tile][columns][row g + 8 v][column 2t + u]
        float2 v[MT][NT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) v[m][n][i] = make_float2(acc[m][n][2 * i], acc[m][n][2 * i + 1]);
        uint8_t *const extra = smem + NS * L.stage;
        if constexpr (DOWN) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int c = n * 8 + 2 * t + u;
                    if (c >= tile.count) continue;
                    float *out = p.out + (int64_t)p.order[tile.start + c] * p.rows;
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int r = first_row(block, m) + 8 * i + g;
                            if (r < p.rows) out[r] = u ? v[m][n][i].y : v[m][n][i].x;
                        }
                }
        } else {
            float *const hs = reinterpret_cast<float *>(extra);
            if constexpr (APART) {
                // gate's sums go through shared memory to the warps that have up's
                if (matrix == 0) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                hs[(n * 8 + 2 * t + u) * HP + in_block + 8 * i + g] = u ? v[0][n][i].y : v[0][n][i].x;
                }
                __syncthreads();
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int c = n * 8 + 2 * t + u;
                    if (c >= tile.count || (APART && matrix == 0)) continue;
                    const float w = p.weights[p.order[tile.start + c]];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = in_block + 8 * i + g;
                        float &at = hs[c * HP + r];
                        const float up = u ? v[MT - 1][n][i].y : v[MT - 1][n][i].x;
                        const float gate = APART ? at : u ? v[0][n][i].y : v[0][n][i].x;
                        const float h = glu_gate(gate, glu_arg(p.act, gate)) * up * w;
                        at = block * CTA_ROWS + r < p.rows ? h : 0.0f;
                    }
                }
            __syncthreads();
            // blocks of 32 rows of every column
            constexpr int HB = CTA_ROWS / 32;
            for (int i = warp; i < tile.count * HB; i += S.warps) {
                const int c = i / HB, b = i % HB, at = block * HB + b;
                if (at >= p.h_blocks) continue;
                const int64_t row = tile.start + c;
                const float x = hs[c * HP + 32 * b + lane];
                uint8_t *rec = p.h + row * p.h_row_bytes + (int64_t)at * frag_bytes(p.h_fmt);
                const float2 s = put_terms(x, lane, p.h_fmt, rec);
                if (lane == 0) {
                    p.h_scale[row * p.h_blocks + at] = s.x;
                    p.h_sum[row * p.h_blocks + at] = s.y;
                }
            }
        }
        // (what the next unit writes to `extra` comes after the next barrier)
        chunk = 0;
        unit += gridDim.x;
    }
    cp_async_wait<0>();
    // The next kernel's CTAs are let in only now: earlier ones would take the
    // places that this grid leaves free, several on one SM, and stay there.
    pdl_launch_dependents();
}

template <int FMT, int TN, bool DOWN, bool EVEN>
cudaError_t launch_one(const ProductParams &p, int max_tiles, const DeviceInfo &dev, cudaStream_t s) {
    constexpr Layout L = layout_of(FMT, TN, DOWN, EVEN);
    static_assert(L.stages >= 2, "two stages");
    constexpr int CTA_ROWS = cta_rows(TN, DOWN);
    static OncePerDevice once;
    cudaError_t e = allow_smem(once, product_kernel<FMT, TN, DOWN, EVEN>, L.smem);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)max_tiles * ((p.rows + CTA_ROWS - 1) / CTA_ROWS);
    const int64_t wave = (int64_t)dev.sm_count * L.ctas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units < wave ? units : wave));
    cfg.blockDim = dim3(shape_of(TN).warps * 32);
    cfg.dynamicSmemBytes = L.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, product_kernel<FMT, TN, DOWN, EVEN>, p);
}

// Rows that do not start on 16-byte boundaries take the EVEN kernels (Q4_K's
// always do, Q6_K's hardly ever).
template <int FMT, int TN, bool DOWN>
cudaError_t launch_aligned(const ProductParams &p, int max_tiles, const DeviceInfo &dev, cudaStream_t s) {
    if constexpr (FMT == F_Q4_K) {
        return launch_one<FMT, TN, DOWN, false>(p, max_tiles, dev, s);
    } else if constexpr (FMT == F_Q6_K) {
        return launch_one<FMT, TN, DOWN, true>(p, max_tiles, dev, s);
    } else {
        return p.row_bytes % 16 ? launch_one<FMT, TN, DOWN, true>(p, max_tiles, dev, s)
                                : launch_one<FMT, TN, DOWN, false>(p, max_tiles, dev, s);
    }
}

template <int FMT, bool DOWN>
cudaError_t launch_columns(int columns, const ProductParams &p, int max_tiles, const DeviceInfo &dev, cudaStream_t s) {
    switch (columns) {
    case 8: return launch_aligned<FMT, 8, DOWN>(p, max_tiles, dev, s);
    default: return launch_aligned<FMT, 16, DOWN>(p, max_tiles, dev, s);
    }
}

template <int FMT>
cudaError_t launch_product(bool down, int columns, const ProductParams &p, int max_tiles, const DeviceInfo &dev, cudaStream_t s) {
    return down ? launch_columns<FMT, true>(columns, p, max_tiles, dev, s)
                : launch_columns<FMT, false>(columns, p, max_tiles, dev, s);
}

}  // namespace experts
}  // namespace qmm
