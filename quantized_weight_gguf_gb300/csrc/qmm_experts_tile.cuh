// qmm_experts_tile.cuh -- the experts' two products for many rows per expert, over quantised weights, on tcgen05.
//
// A unit of work is a tile of up to 48 pairs of one expert times 128 rows of W (of the first product 64 of the gate and
// the same 64 of the up matrix). The tensor cores see the integer codes of a block of 32 weights as fp16, exact, against
// the activations as two fp16 terms under one power of two per row; each block's sums start fresh, and are
// multiplied by the block's scale in fp32 as they leave the tensor memory, so nothing of W is rounded and no sum in the
// tensor cores, which cut what they add, is longer than 32 values. With a row of W per lane, as tensor memory has
// them, a scale is decoded once and multiplies up to 48 sums, two per packed instruction.
//
// Warps 0 .. 3: a lane takes a row of W; unpacks a block's codes to tensor memory (two stages of A and D), then takes
// the sums of the block before. Each copies its own rows into a ring of its own. Warp 4 copies the pairs' terms, 6 KB
// a block, into the 128-byte swizzle that the products read, and one lane of it issues them: four per block (two
// 16-deep steps, the low term's first).
//
// Bound by the warps that unpack and take, whose time hardly depends on the columns: about 1450 instructions a block and
// CTA of Q4_K against four products (98.2 M of warps in the first product below), at 20 warps an SM, held there by registers
// and tensor memory; issue slots 51 to 58 % used, the tensor pipe 11 %.
// Four CTAs an SM (286 us with three, 259 with four, before the last change of the codes). Measured: 256 positions, Q4_K
// 2048 x 1024, eight of 64 experts 274 us, of which the first product 178, the second 79 (mma.sync: 395); 128 rows an
// expert at 2048 x 768 560 us (903). Blocks in pairs per handshake took 300 us instead of 268 (one stage of D, so that a
// product waits for the sums before it), tiles of 32 columns 272 instead of 251.
#pragma once

#include "qmm_experts_kernel.cuh"
#include "qmm_experts_rows.cuh"

namespace qmm {
namespace experts {

constexpr int kTileColumns = 48, kTileRows = 128, kTileWarps = 4;
constexpr int kTileThreads = 32 * (kTileWarps + 1);
constexpr int kTermBytes = 128;                        // of a block of a row: 32 high terms, 32 low ones
constexpr int kXSlots = 3;                             // blocks of terms in shared memory
constexpr int kXBytes = kTileColumns * kTermBytes;
// Sums of a block that leave separately (Q6_K has a scale per 16 weights), and columns of a stage of tensor memory.
__host__ __device__ constexpr int tile_sums(int fmt) { return fmt == F_Q6_K ? 2 : 1; }
__host__ __device__ constexpr int tile_stage_cols(int fmt) { return 16 + kTileColumns * tile_sums(fmt); }
__host__ __device__ constexpr int tile_tmem_cols(int fmt) { return fmt == F_Q6_K ? 256 : 128; }

struct TileLayout {
    int pieces, w_stage, stages, x_at, sums_at, h_at, bars_at, smem, ctas;
};
__host__ __device__ constexpr TileLayout tile_layout(int fmt, bool down) {
    TileLayout l = {};
    l.pieces = chunk_pieces(fmt, true);  // rows may start at any even address
    l.w_stage = 32 * 16 * l.pieces;
    const int x = kXSlots * (kXBytes + kTileColumns * 4), h = down ? 0 : kTileColumns * 64 * 4, bars = 256;
    // as many CTAs per SM as tensor memory has room for, if two stages of W fit beside them
    for (l.ctas = 512 / tile_tmem_cols(fmt); l.ctas > 1; --l.ctas) {
        // (1 KB is the system's, 1 KB for alignment)
        l.stages = (228 * 1024 / l.ctas - 1024 - 1024 - x - h - bars) / (kTileWarps * l.w_stage);
        if (l.stages >= 2) break;
    }
    if (l.stages > 4) l.stages = 4;
    l.x_at = 0;
    l.sums_at = l.x_at + kXSlots * kXBytes;
    l.h_at = l.sums_at + kXSlots * kTileColumns * 4;
    l.bars_at = l.h_at + h;
    l.smem = 1024 + l.bars_at + bars + l.stages * kTileWarps * l.w_stage;
    return l;
}

// Tests the phase, and waits for it as long as the hardware does by itself.
__device__ __forceinline__ bool try_now(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// Waits for the phase, up to the limit; then, or when another warp has given up, goes on all the same: the
// results are wrong and reported, and every later wait is short.
__device__ __forceinline__ void wait_for(uint32_t bar, uint32_t parity, volatile int *stop, unsigned int *err,
                                         unsigned int code) {
    if (try_now(bar, parity)) return;
    uint64_t t0 = 0;
    for (uint32_t i = 1; !try_now(bar, parity); ++i) {
        if (i & 63u) continue;
        if (*stop) return;
        const uint64_t t = global_ns();
        if (t0 == 0) t0 = t;
        if (t - t0 > kWaitLimitNs) {
            record_error(err, code);
            *stop = 1;
        }
    }
}
// An arrival by the warp's first lane, for all of it.
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
    __syncwarp();
    asm volatile("{\n .reg .pred p;\n setp.eq.s32 p, %1, 0;\n @p mbarrier.arrive.shared::cta.b64 _, [%0];\n}\n" ::"r"(bar),
                 "r"(lane)
                 : "memory");
}

// 16 columns of this warp's lanes, in pairs.
__device__ __forceinline__ void tmem_take16(uint32_t taddr, uint64_t (&v)[8]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("mov.b64 %0, {%1, %2};" : "=l"(v[i]) : "r"(r[2 * i]), "r"(r[2 * i + 1]));
}
__device__ __forceinline__ void add_times(uint64_t &sum, uint64_t v, uint64_t by) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(sum) : "l"(v), "l"(by));
}
__device__ __forceinline__ float half_of(uint64_t v, int second) {
    return __uint_as_float(second ? (uint32_t)(v >> 32) : (uint32_t)v);
}

// Place of element e of a block in a term's 32: what masks leave of a word's bytes, 0 and 2, then 1 and 3.
__device__ __forceinline__ int tile_place(int e) { return (e & ~3) | ((e & 1) << 1) | ((e & 2) >> 1); }

// The codes of a lane's row: block b of a chunk as 16 registers of fp16 pairs, its scales and what the
// sum of its activations is multiplied by.
template <int FMT>
struct TileRow {
    static constexpr bool kMin = false;
    __device__ __forceinline__ void open(const uint8_t *, int) {}
    __device__ __forceinline__ void block(const uint8_t *chunk, int b, uint32_t (&r)[16], float (&scale)[2], float &) const {
        const uint8_t *p = chunk + block_bytes(FMT) * b;
        scale[0] = f16_bits_to_f32(ld16(p));
        if constexpr (FMT == F_Q4_0) {
            uint32_t w[4];
            words_at<4>(p + 2, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                low_nibbles<8>(w[i], r[2 * i], r[2 * i + 1]);
                high_nibbles<8>(w[i], r[8 + 2 * i], r[9 + 2 * i]);
            }
        } else if constexpr (FMT == F_Q5_0) {
            uint32_t w[5];
            words_at<5>(p + 2, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                bytes<16>((w[1 + i] & 0x0F0F0F0Fu) | Row<F_Q5_0>::spread(w[0] >> (4 * i)), r[2 * i], r[2 * i + 1]);
                bytes<16>(((w[1 + i] >> 4) & 0x0F0F0F0Fu) | Row<F_Q5_0>::spread(w[0] >> (16 + 4 * i)), r[8 + 2 * i],
                          r[9 + 2 * i]);
            }
        } else {
            static_assert(FMT == F_Q8_0, "formats of codes");
            uint32_t w[8];
            words_at<8>(p + 2, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) signed_bytes(w[i], r[2 * i], r[2 * i + 1]);
        }
    }
};
template <>
struct TileRow<F_Q4_K> {
    static constexpr bool kMin = true;
    uint32_t sc, m;
    float d, dmin;
    // half: of the super-block
    __device__ __forceinline__ void open(const uint8_t *chunk, int half) {
        const uint4 h = *reinterpret_cast<const uint4 *>(chunk);
        d = f16_bits_to_f32(h.x & 0xFFFFu);
        dmin = f16_bits_to_f32(h.x >> 16);
        sc = half ? (h.w & 0x0F0F0F0Fu) | ((h.y >> 2) & 0x30303030u) : h.y & 0x3F3F3F3Fu;
        m = half ? ((h.w >> 4) & 0x0F0F0F0Fu) | ((h.z >> 2) & 0x30303030u) : h.z & 0x3F3F3F3Fu;
    }
    __device__ __forceinline__ void block(const uint8_t *chunk, int b, uint32_t (&r)[16], float (&scale)[2], float &min) const {
        // (the nibbles as they lie, subnormal fp16 numbers, would do without a conversion, but the tensor cores cut their
        // products ten bits too high: 3e-6 off instead of 5e-7)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 v = *reinterpret_cast<const uint4 *>(chunk + 16 + 32 * (b >> 1) + 16 * i);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (b & 1) high_nibbles<0>(w[j], r[8 * i + 2 * j], r[8 * i + 2 * j + 1]);
                else low_nibbles<0>(w[j], r[8 * i + 2 * j], r[8 * i + 2 * j + 1]);
            }
        }
        scale[0] = d * (float)((sc >> (8 * b)) & 255u);
        min = -dmin * (float)((m >> (8 * b)) & 255u);
    }
};
template <>
struct TileRow<F_Q6_K> {
    static constexpr bool kMin = false;
    float d;
    __device__ __forceinline__ void open(const uint8_t *chunk, int) { d = f16_bits_to_f32(ld16(chunk + 208)); }
    __device__ __forceinline__ void block(const uint8_t *chunk, int b, uint32_t (&r)[16], float (&scale)[2], float &) const {
        // half b / 4, quarter b % 4: nibbles of ql bytes 32 (b & 1) .., two bits of the qh bytes
        const uint32_t q = b & 3, low = 4 * (q >> 1), high = 2 * q;
        uint32_t w[8], u[8];
        words_at<8>(chunk + 64 * (b >> 2) + 32 * (q & 1), w);
        words_at<8>(chunk + 128 + 32 * (b >> 2), u);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            bytes<32>(((w[i] >> low) & 0x0F0F0F0Fu) | (((u[i] >> high) & 0x03030303u) << 4), r[2 * i], r[2 * i + 1]);
        const uint32_t sc = ld16(chunk + 192 + 2 * b);
        scale[0] = d * (float)(int)(int8_t)(sc & 255u);
        scale[1] = d * (float)(int)(int8_t)(sc >> 8);
    }
};

template <int FMT, bool DOWN>
__global__ void __launch_bounds__(kTileThreads, tile_layout(FMT, DOWN).ctas)
    tile_kernel(const __grid_constant__ ProductParams p) {
    constexpr TileLayout L = tile_layout(FMT, DOWN);
    constexpr int KB = chunk_k(FMT) / 32, CB = chunk_bytes(FMT), NP = L.pieces, PITCH = 16 * NP, NS = L.stages;
    constexpr int SUMS = tile_sums(FMT), SC = tile_stage_cols(FMT);
    constexpr bool MIN = TileRow<FMT>::kMin;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *const smem = smem_raw + (-smem_addr(smem_raw) & 1023u);  // the swizzle's atoms are 1 KB
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t base = smem_addr(smem);
    const uint32_t bars = base + L.bars_at;
    auto a_full = [&](int s) { return bars + 8u * s; };
    auto d_full = [&](int s) { return bars + 8u * (2 + s); };
    auto x_empty = [&](int s) { return bars + 8u * (5 + s); };
    const uint32_t crossed = bars + 8u * 4;
    volatile uint32_t *const slot = reinterpret_cast<volatile uint32_t *>(smem + L.bars_at + 8 * (5 + kXSlots));
    volatile int *const stop = reinterpret_cast<volatile int *>(slot + 1);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(a_full(i), kTileWarps);
            mbar_init(d_full(i), 1 + MIN);
        }
        for (int i = 0; i < kXSlots; ++i) {
            mbar_init(x_empty(i), 1 + (MIN ? kTileWarps : 0));
        }
        mbar_init(crossed, kTileWarps);
        *stop = 0;
        fence_barrier_init();
    }
    if (warp == kTileWarps) {
        tmem_alloc(bars + 8 * (5 + kXSlots), tile_tmem_cols(FMT));
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *slot;

    pdl_wait_prev();

    constexpr int UNIT = DOWN ? kTileRows : kTileRows / 2;  // rows of a matrix
    const int row_blocks = (p.rows + UNIT - 1) / UNIT;
    const int units = *p.n_tiles * row_blocks;
    const int chunks = (p.blocks + KB - 1) / KB;

    if (warp == kTileWarps) {
        // ---- the pairs' terms, and the products ----
        const int mine = (int)blockIdx.x < units ? (units - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
        const int64_t blocks = (int64_t)mine * p.blocks;
        int load_unit = blockIdx.x, load_block = 0, load_x = 0, x = 0, s = 0;
        uint32_t load_px = 1, px = 0, ps = 0;  // (a fresh barrier: the phase before has completed)
        const uint8_t *from[kTileColumns / 4] = {};
        int load_groups = 0, unit = blockIdx.x, block = 0;
        uint32_t idesc = 0;
        const float *sums = nullptr, *sums2 = nullptr;
        // piece 32 i + lane of a block: 16 bytes of column 4 i + lane / 8
        const uint32_t to = base + L.x_at + (lane >> 3) * kTermBytes + (((lane & 7) ^ (lane >> 3)) << 4);
        auto load = [&]() {
            if (load_block == 0) {
                // columns past the tile's, up to 16 of them, repeat its last one; their sums are dropped
                const Tile tile = p.tiles[load_unit / row_blocks];
                auto row_of = [&](int c) {
                    const int at = tile.start + min(c, tile.count - 1);
                    return DOWN ? at : p.order[at] / p.top_k;
                };
#pragma unroll
                for (int i = 0; i < kTileColumns / 4; ++i)
                    from[i] = p.x + row_of(4 * i + (lane >> 3)) * p.x_row_bytes + 16 * (lane & 7);
                if (MIN) {
                    sums = p.x_sum + (int64_t)row_of(lane) * p.x_blocks;
                    sums2 = p.x_sum + (int64_t)row_of(32 + (lane & 15)) * p.x_blocks;
                }
                load_groups = (tile.count + 15) / 16;
            }
            wait_for(x_empty(load_x), load_px, stop, p.err, DERR_MMA_EMPTY);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kTileColumns / 4; ++i) {
                if (i / 4 >= load_groups) break;
                cp_async16((to + load_x * kXBytes + 512 * i) ^ (64 * (i & 1)), from[i], 16);
                from[i] += kTermBytes;
            }
            if (MIN) {
                cp_async4(base + L.sums_at + (load_x * kTileColumns + lane) * 4, sums + load_block);
                if (lane < 16) cp_async4(base + L.sums_at + (load_x * kTileColumns + 32 + lane) * 4, sums2 + load_block);
            }
            if (++load_x == kXSlots) load_x = 0, load_px ^= 1;
            if (++load_block == p.blocks) {
                load_block = 0;
                load_unit += gridDim.x;
            }
        };
        // all copies but the last block's have landed, and the products may read them
        auto landed = [&]() {
            cp_async_commit();
            cp_async_wait<1>();
            fence_proxy_async_smem();
            __syncwarp();
        };
        for (int i = 0; i < 2; ++i) {
            if (i < blocks) load();
            landed();
        }
        for (int64_t n = 0; n < blocks; ++n) {
            if (block == 0) idesc = idesc_f16_f32(kTileRows, (p.tiles[unit / row_blocks].count + 15) & ~15);
            if (++block == p.blocks) {
                block = 0;
                unit += gridDim.x;
            }
            if (lane == 0) {
                wait_for(a_full(s), ps, stop, p.err, DERR_MMA_A);
                tc_fence_after();
                const uint64_t terms = sdesc_sw128(base + L.x_at + x * kXBytes);
                const uint32_t a = tmem + s * SC, d = a + 16;
                // 16 values are 8 columns of A and 32 bytes of terms, the low ones 64 bytes on
                tc_mma_f16_ts(d, a, terms + 4, idesc, 0);
                tc_mma_f16_ts(d + kTileColumns * (SUMS - 1), a + 8, terms + 6, idesc, SUMS == 1);
                tc_mma_f16_ts(d, a, terms, idesc, 1);
                tc_mma_f16_ts(d + kTileColumns * (SUMS - 1), a + 8, terms + 2, idesc, 1);
                tc_commit(d_full(s));
                if (MIN) mbar_arrive(d_full(s));  // (passes on that the activations' sums are there)
                tc_commit(x_empty(x));
                // no arrival is under way to a CTA that has gone
                if (n + 1 == blocks) wait_for(x_empty(x), px, stop, p.err, DERR_TEARDOWN);
            }
            __syncwarp();
            if (n + 2 < blocks) load();
            landed();
            if (++x == kXSlots) x = 0, px ^= 1;
            s ^= 1;
            ps ^= s == 0;
        }
        cp_async_wait<0>();
    } else {
        // ---- codes and sums ----
        uint8_t *const ring = smem + L.bars_at + 256 + warp * NS * L.w_stage;
        const int matrix = DOWN ? 0 : warp >> 1;
        const int in_unit = DOWN ? 32 * warp : 32 * (warp & 1);
        const uint32_t mine = tmem + ((uint32_t)(32 * warp) << 16);

        int load_unit = blockIdx.x, load_chunk = 0, load_first = 0;
        const uint8_t *load_slice = nullptr;
        int row_at[NP];  // of piece 32 i + lane: its row's bytes from the first
#pragma unroll
        for (int i = 0; i < NP; ++i) row_at[i] = (32 * i + lane) / NP * (int)p.row_bytes;
        auto load_next = [&](int stage) {
            if (load_unit < units) {
                if (load_chunk == 0) {
                    load_slice = p.w[matrix] + p.tiles[load_unit / row_blocks].expert * p.slice_bytes;
                    load_first = load_unit % row_blocks * UNIT + in_unit;
                }
                const uint32_t to = smem_addr(ring) + stage * L.w_stage + 16 * lane;
                const int at = FMT == F_Q4_K ? (load_chunk >> 1) * 144 : load_chunk * CB;
                const int half = FMT == F_Q4_K ? 64 * (load_chunk & 1) : 0;
                if (load_first + 32 <= p.rows &&
                    (FMT == F_Q4_K || (int64_t)(load_first + 31) * p.row_bytes + at + 16 * NP <= p.slice_bytes)) {
                    // the whole pieces that a row's chunk lies in
                    const uint8_t *b = load_slice + load_first * p.row_bytes + at;
#pragma unroll
                    for (int i = 0; i < NP; ++i) {
                        const int t = (32 * i + lane) % NP;
                        const uint8_t *r = b + row_at[i];
                        if (FMT != F_Q4_K) r -= reinterpret_cast<uintptr_t>(r) & 15u;
                        cp_async16(to + 512 * i, r + 16 * t + (FMT == F_Q4_K && t ? half : 0), 16);
                    }
                } else {
                    const int left = (int)p.row_bytes - at;
#pragma unroll 1
                    for (int i = 0; i < NP; ++i) {
                        const int piece = 32 * i + lane, row = piece / NP, t = piece - row * NP;
                        // rows past the end are copies of the last one; their results are dropped
                        const uint8_t *r = load_slice + min(load_first + row, p.rows - 1) * p.row_bytes + at;
                        if (FMT == F_Q4_K) {
                            cp_async16(to + 512 * i, r + 16 * t + (t ? half : 0), 16);
                            continue;
                        }
                        const int off = (int)(reinterpret_cast<uintptr_t>(r) & 15u);
                        const int n = off + min(CB, left) - 16 * t;
                        cp_async16(to + 512 * i, n > 0 ? r - off + 16 * t : r - off, n <= 0 ? 0 : n < 16 ? n : 16);
                    }
                }
                if (++load_chunk == chunks) {
                    load_chunk = 0;
                    load_unit += gridDim.x;
                }
            }
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < NS - 1; ++i) load_next(i);

        TileRow<FMT> row;
        uint64_t sum[kTileColumns / 2];  // of columns 2 i and 2 i + 1
        int groups = 0;                  // of 16 columns that the tile has
        int stage = 0, s = 0, x = 0;
        uint32_t phase = 0, cross_phase = 0;  // of what is taken next
        float scale[2] = {}, min_of = 0.0f, was[2] = {}, min_was = 0.0f;
        // the sums of the block before this one, from stage `at`
        auto take = [&](int at) {
            wait_for(d_full(at), phase, stop, p.err, DERR_MMA_ACC);
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < SUMS; ++i) {
                const uint64_t by = pack_f2(was[i], was[i]);
#pragma unroll
                for (int q = 0; q < kTileColumns / 16; ++q) {
                    if (q >= groups) break;
                    uint64_t v[8];
                    tmem_take16(mine + at * SC + 16 + kTileColumns * i + 16 * q, v);
#pragma unroll
                    for (int c = 0; c < 8; ++c) add_times(sum[8 * q + c], v[c], by);
                }
            }
            if (MIN) {
                const ulonglong2 *const xs = reinterpret_cast<const ulonglong2 *>(smem + L.sums_at + x * kTileColumns * 4);
                const uint64_t by = pack_f2(min_was, min_was);
#pragma unroll
                for (int q = 0; q < kTileColumns / 16; ++q) {
                    if (q >= groups) break;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const ulonglong2 v = xs[4 * q + c];
                        add_times(sum[8 * q + 2 * c], v.x, by);
                        add_times(sum[8 * q + 2 * c + 1], v.y, by);
                    }
                }
                warp_arrive(x_empty(x), lane);
                if (++x == kXSlots) x = 0;
            }
            if (at == 1) phase ^= 1;
        };
        // all four warps have come here
        auto cross = [&]() {
            warp_arrive(crossed, lane);
            wait_for(crossed, cross_phase, stop, p.err, DERR_MMA_ACC);
            __syncwarp();
            cross_phase ^= 1;
        };
        for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
            const Tile tile = p.tiles[unit / row_blocks];
            const int first = unit % row_blocks * UNIT + in_unit, r = first + lane;
            const uint32_t start = (uint32_t)(reinterpret_cast<uintptr_t>(p.w[matrix]) + tile.expert * p.slice_bytes +
                                              min(r, p.rows - 1) * p.row_bytes);
#pragma unroll
            for (int c = 0; c < kTileColumns / 2; ++c) sum[c] = 0;
            groups = (tile.count + 15) / 16;
            for (int chunk = 0; chunk < chunks; ++chunk) {
                cp_async_wait<NS - 2>();
                __syncwarp();  // the stage is there for every lane, and the one before it is free
                load_next(stage == 0 ? NS - 1 : stage - 1);
                const uint32_t off = FMT == F_Q4_K ? 0 : (start + (uint32_t)(chunk * CB)) & 15u;
                const uint8_t *const at = ring + stage * L.w_stage + lane * PITCH + off;
                const int here = min(KB, p.blocks - chunk * KB);
                row.open(at, chunk & 1);
#pragma unroll
                for (int b = 0; b < KB; ++b) {
                    if (b >= here) break;
                    uint32_t a[16];
                    row.block(at, b, a, scale, min_of);
                    tmem_st16(mine + s * SC, a);
                    tmem_st_wait();
                    tc_fence_before();
                    warp_arrive(a_full(s), lane);
                    if (chunk || b) take(s ^ 1);
                    s ^= 1;
#pragma unroll
                    for (int i = 0; i < 2; ++i) was[i] = scale[i];
                    min_was = min_of;
                }
                if (++stage == NS) stage = 0;
            }
            take(s ^ 1);

            // ---- the unit's results ----
            int pair[2];  // of columns `lane` and 32 + lane
            float x_scale[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int c = min(32 * i + lane, tile.count - 1);
                pair[i] = p.order[tile.start + c];
                x_scale[i] = p.x_scale[DOWN ? tile.start + c : pair[i] / p.top_k];
            }
            if constexpr (DOWN) {
#pragma unroll
                for (int c = 0; c < kTileColumns; ++c) {
                    if (c % 16 == 0 && c / 16 >= groups) break;
                    const float v = half_of(sum[c / 2], c & 1) * __shfl_sync(~0u, x_scale[c / 32], c & 31);
                    const int to = __shfl_sync(~0u, pair[c / 32], c & 31);
                    if (c < tile.count && r < p.rows) p.out[(int64_t)to * p.rows + r] = v;
                }
            } else {
                // the gate's warps finish the even columns, the up matrix's the odd ones: what the other needs goes over
                float *const across = reinterpret_cast<float *>(smem + L.h_at) + in_unit + lane;
#pragma unroll
                for (int c = 0; c < kTileColumns / 2; ++c) {
                    if (c % 8 == 0 && c / 8 >= groups) break;
                    across[(2 * c + (matrix ^ 1)) * 64] = half_of(sum[c], matrix ^ 1);
                }
                cross();
                const float weight[2] = {p.weights[pair[0]], p.weights[pair[1]]};
                float *const h = reinterpret_cast<float *>(p.h) + (int64_t)tile.start * p.rows + r;
#pragma unroll
                for (int c = 0; c < kTileColumns / 2; ++c) {
                    if (c % 8 == 0 && c / 8 >= groups) break;
                    const int at = 2 * c + matrix;
                    const float scale_of = __shfl_sync(~0u, x_scale[c / 16], at & 31);
                    const float w = __shfl_sync(~0u, weight[c / 16], at & 31);
                    const float other = across[at * 64] * scale_of, own = half_of(sum[c], matrix) * scale_of;
                    const float gate = matrix == 0 ? own : other, up = matrix == 0 ? other : own;
                    if (at < tile.count && r < p.rows) h[(int64_t)at * p.rows] = glu_gate(gate, glu_arg(p.act, gate)) * up * w;
                }
                cross();  // what went over has been taken
            }
        }
        cp_async_wait<0>();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kTileWarps) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, tile_tmem_cols(FMT));
    }
    pdl_launch_dependents();
}

template <int FMT, bool DOWN>
cudaError_t launch_tile_of(const ProductParams &p, int max_tiles, const DeviceInfo &dev, cudaStream_t s) {
    constexpr TileLayout L = tile_layout(FMT, DOWN);
    static_assert(L.stages >= 2, "two stages");
    static_assert(tile_tmem_cols(FMT) >= 2 * tile_stage_cols(FMT) && tile_tmem_cols(FMT) * L.ctas <= 512, "tensor memory");
    static OncePerDevice once;
    cudaError_t e = allow_smem(once, tile_kernel<FMT, DOWN>, L.smem);
    if (e != cudaSuccess) return e;
    constexpr int UNIT = DOWN ? kTileRows : kTileRows / 2;
    const int64_t units = (int64_t)max_tiles * ((p.rows + UNIT - 1) / UNIT), wave = (int64_t)dev.sm_count * L.ctas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units < wave ? units : wave));
    cfg.blockDim = dim3(kTileThreads);
    cfg.dynamicSmemBytes = L.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tile_kernel<FMT, DOWN>, p);
}

template <int FMT>
cudaError_t launch_tile(bool down, const ProductParams &p, int max_tiles, const DeviceInfo &dev, cudaStream_t s) {
    return down ? launch_tile_of<FMT, true>(p, max_tiles, dev, s) : launch_tile_of<FMT, false>(p, max_tiles, dev, s);
}

}  // namespace experts
}  // namespace qmm
