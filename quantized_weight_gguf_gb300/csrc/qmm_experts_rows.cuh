// qmm_experts_rows.cuh -- the experts' two products for single activation rows:
// one position, or several that hardly share an expert.
//
// A lane takes a block of 32 weights of a row; 8 lanes take 8 neighbouring blocks (a run) and
// hold the activations that these meet in registers over many rows of W. Quantised weights are multiplied in
// integers: an activation is split into three signed digits of 8 bits under a power of two per block (24 bits,
// to 2^-23 of the block's largest), codes are unpacked to bytes, and four products are one dp4a. A block's integer sums
// are exact; they become floats without a conversion, since they start from the bit pattern of 1.5 * 2^23,
// less the codes' zero point times the digits' sum. 24 dp4a of 95 to 106 instructions a warp for 32 blocks (Q4_0, Q8_0; copies
// and sums among them); tiles for the tensor cores take 74 instead of 66 us at one row per expert of Q8_0. 16-bit weights:
// fp32 multiply-adds.
//
// A unit of work of the first product is 32 rows of a pair's gate matrix and the same 32 of its up matrix (one block of
// the second product's activations); of the second 16 rows of y, over the blocks of the position's slots as one long
// sum, so that y needs no further pass. `slices` warps take a unit, each every slices-th run. A warp copies what
// it multiplies into a ring of its own and waits for nobody until the unit's end, where the slices' sums are added up
// in order. Pairs are taken as they stand: sorted by expert, which took a launch's time, they came from L2 no more often.
//
// One position: the first product turns x into digits itself while its first weights are on their way.
//
// Bound by the latency that 12 to 16 warps an SM do not hide (111 to 128 registers; issue slots 47 to 58 % used and DRAM
// half where all SMs are busy), and by fixed steps where the work is small. Measured: 4096 x 14336, two of 8 experts, Q4_0
// 59.8 us (0.49 of the copy rate); eight positions, Q8_0 64 us (0.48); 2048 x 768, eight of 64, Q4_K / Q6_K 17.5 us,
// BF16 17.2 us; five positions of 1376 x 352, Q5_0 / Q8_0 20.5 us.
#pragma once

#include "qmm_experts_kernel.cuh"

namespace qmm {
namespace experts {

constexpr int kRowWarps = 8;
constexpr int kOneBlocks = 160;  // of x that one position's first product holds (k up to 5120)
// Rows of W in a unit.
__host__ __device__ constexpr int unit_rows(bool down) { return down ? 16 : 64; }

// A record of a block of 32 activations, 144 bytes (eight lanes' 16-byte loads from records that lie one after the
// other meet no bank twice). Quantised weights: digits [3][32] (element e is sum_i 256^i digit_i[e] times the
// scale), scale, sum, and per digit the sums of elements 0-15 and 16-31 as 16-bit halves of a word; 16-bit weights:
// the values.
constexpr int kRecord = 144;
__host__ __device__ constexpr bool is_16bit(int fmt) { return fmt == F_BF16 || fmt == F_F16; }

// -------------------------------------------------------- activations ----

constexpr int kMagic = 0x4B400000;  // 1.5 * 2^23: plus an integer below 2^22 in size, a float that is that much larger
__device__ __forceinline__ float from_magic(int v) { return __int_as_float(v) - 12582912.0f; }

// Writes the record of a block (lane e holds element e).
__device__ __forceinline__ void put_record(float v, int e, int fmt, uint8_t *rec) {
    if (is_16bit(fmt)) {
        reinterpret_cast<float *>(rec)[e] = v;
        return;
    }
    float sum = v;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    const uint32_t top = __reduce_max_sync(~0u, __float_as_uint(v) & 0x7FFFFFFFu);
    // the largest times 2^(22 - its exponent), or half of that, is at most 127 * (65536 + 256 + 1)
    const uint32_t b = max(top >> 23, 24u) + ((top & 0x7FFFFFu) > 0x7EFEFCu);
    const bool plain = top < 0x7F800000u;
    const float up = __uint_as_float((276u - b) << 23);    // 2^(22 + 127 - b)
    const float down = __uint_as_float((b - 22u) << 23);   // 1 / up
    const int x = plain ? __float2int_rn(v * up) : 0;
    int digit[3];
    digit[0] = (int)(int8_t)x;
    const int x1 = (x - digit[0]) >> 8;
    digit[1] = (int)(int8_t)x1;
    digit[2] = (x1 - digit[1]) >> 8;
    uint32_t sums[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int first = __reduce_add_sync(~0u, e < 16 ? digit[i] : 0);
        const int all = __reduce_add_sync(~0u, digit[i]);
        sums[i] = ((uint32_t)first & 0xFFFFu) | ((uint32_t)(all - first) << 16);
        rec[32 * i + e] = (uint8_t)digit[i];
    }
    if (e == 0) {
        *reinterpret_cast<float2 *>(rec + 96) = make_float2(plain ? down : NAN, sum);
        *reinterpret_cast<uint2 *>(rec + 104) = make_uint2(sums[0], sums[1]);
        *reinterpret_cast<uint32_t *>(rec + 112) = sums[2];
    }
}

// A block's activations in a lane's registers.
template <int FMT>
struct Digits {
    int d[3][8];
    float scale, sum;
    int init[2][3];  // [first half, second half (Q6_K; else the first holds the block)][digit]
    __device__ __forceinline__ void load(const uint8_t *rec, int) {
        constexpr int Z = FMT == F_Q4_0 ? 8 : FMT == F_Q5_0 ? 16 : FMT == F_Q6_K ? 32 : 0;
#pragma unroll
        for (int i = 0; i < 6; ++i) {
            const int4 v = *reinterpret_cast<const int4 *>(rec + 16 * i);
            int(&r)[8] = d[i / 2];
            r[i % 2 * 4] = v.x;
            r[i % 2 * 4 + 1] = v.y;
            r[i % 2 * 4 + 2] = v.z;
            r[i % 2 * 4 + 3] = v.w;
        }
        const float2 f = *reinterpret_cast<const float2 *>(rec + 96);
        scale = f.x;
        sum = f.y;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int s = *reinterpret_cast<const int *>(rec + 104 + 4 * i);
            const int first = (int)(int16_t)s, second = s >> 16;
            init[0][i] = kMagic - Z * (FMT == F_Q6_K ? first : first + second);
            init[1][i] = kMagic - Z * second;
        }
    }
};
template <>
struct Digits<F_F16> {
    float4 v[8];
    // for 16-byte pieces of W in the order p, p + 1, p + 2, p + 3 (mod 4), so that lanes meet no bank twice
    __device__ __forceinline__ void load(const uint8_t *rec, int p) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const float4 *>(rec + (((p + i / 2) & 3) * 2 + i % 2) * 16);
    }
};
template <>
struct Digits<F_BF16> : Digits<F_F16> {};

// --------------------------------------------------------------- blocks ----

// N words from p, which is even.
template <int N>
__device__ __forceinline__ void words_at(const uint8_t *p, uint32_t (&w)[N]) {
    const uint32_t odd = (uint32_t)reinterpret_cast<uintptr_t>(p) & 2u;
    const uint8_t *a = p - odd;
    const uint32_t sel = odd ? 0x5432u : 0x3210u;
    uint32_t r[N + 1];
#pragma unroll
    for (int i = 0; i <= N; ++i) r[i] = ld32(a + 4 * i);
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = prmt(r[i], r[i + 1], sel);
}

// Codes 4 j .. 4 j + 3 as bytes times the digits.
template <int FMT>
__device__ __forceinline__ void dots(const Digits<FMT> &x, int j, uint32_t codes, int (&acc)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) acc[i] = __dp4a(x.d[i][j], (int)codes, acc[i]);
}
__device__ __forceinline__ float joined(const int (&acc)[3]) {
    return fmaf(from_magic(acc[2]), 65536.0f, fmaf(from_magic(acc[1]), 256.0f, from_magic(acc[0])));
}

// A block times its activations. p: the block, or (K-quants) its super-block, of which it is the l-th block.
template <int FMT>
__device__ __forceinline__ float block_times(const uint8_t *p, int l, const Digits<FMT> &x) {
    int acc[3] = {x.init[0][0], x.init[0][1], x.init[0][2]};
    if constexpr (FMT == F_Q4_0) {
        uint32_t w[4];
        words_at<4>(p + 2, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            dots<FMT>(x, j, w[j] & 0x0F0F0F0Fu, acc);
            dots<FMT>(x, 4 + j, (w[j] >> 4) & 0x0F0F0F0Fu, acc);
        }
        return joined(acc) * (f16_bits_to_f32(ld16(p)) * x.scale);
    } else if constexpr (FMT == F_Q5_0) {
        uint32_t w[5];
        words_at<5>(p + 2, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            dots<FMT>(x, j, (w[1 + j] & 0x0F0F0F0Fu) | Row<F_Q5_0>::spread(w[0] >> (4 * j)), acc);
            dots<FMT>(x, 4 + j, ((w[1 + j] >> 4) & 0x0F0F0F0Fu) | Row<F_Q5_0>::spread(w[0] >> (16 + 4 * j)), acc);
        }
        return joined(acc) * (f16_bits_to_f32(ld16(p)) * x.scale);
    } else if constexpr (FMT == F_Q8_0) {
        uint32_t w[8];
        words_at<8>(p + 2, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) dots<FMT>(x, j, w[j], acc);
        return joined(acc) * (f16_bits_to_f32(ld16(p)) * x.scale);
    } else if constexpr (FMT == F_Q4_K) {
        // block l: nibbles l & 1 of code bytes 32 (l / 2) ..; scales l of the header
        const uint4 h = *reinterpret_cast<const uint4 *>(p);
        const uint32_t pick = 0x4440u | (l & 3);
        const uint32_t a = prmt(h.y, 0u, pick), c = prmt(h.z, 0u, pick), e = prmt(h.w, 0u, pick);
        const uint32_t sc = l < 4 ? a & 63u : (e & 15u) | ((a >> 6) << 4);
        const uint32_t m = l < 4 ? c & 63u : (e >> 4) | ((c >> 6) << 4);
        const uint32_t shift = 4 * (l & 1);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p + 16 + 32 * (l >> 1) + 16 * i);
            dots<FMT>(x, 4 * i, (v.x >> shift) & 0x0F0F0F0Fu, acc);
            dots<FMT>(x, 4 * i + 1, (v.y >> shift) & 0x0F0F0F0Fu, acc);
            dots<FMT>(x, 4 * i + 2, (v.z >> shift) & 0x0F0F0F0Fu, acc);
            dots<FMT>(x, 4 * i + 3, (v.w >> shift) & 0x0F0F0F0Fu, acc);
        }
        const float d = f16_bits_to_f32(h.x & 0xFFFFu) * (byte_magic23<0>(sc) - 8388608.0f);
        const float dm = f16_bits_to_f32(h.x >> 16) * (8388608.0f - byte_magic23<0>(m));
        return fmaf(dm, x.sum, joined(acc) * (d * x.scale));
    } else {
        static_assert(FMT == F_Q6_K, "formats of codes");
        // block l: half l / 4, quarter r = l % 4: nibbles r / 2 of ql bytes 32 (r & 1) .., bits 2r of the qh bytes
        const uint32_t r = l & 3, low = 4 * (r >> 1), high = 2 * r;
        uint32_t w[8], u[8];
        words_at<8>(p + 64 * (l >> 2) + 32 * (r & 1), w);
        words_at<8>(p + 128 + 32 * (l >> 2), u);
        int acc2[3] = {x.init[1][0], x.init[1][1], x.init[1][2]};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t code = ((w[j] >> low) & 0x0F0F0F0Fu) | (((u[j] >> high) & 0x03030303u) << 4);
            if (j < 4) dots<FMT>(x, j, code, acc);
            else dots<FMT>(x, j, code, acc2);
        }
        const uint32_t sc = ld16(p + 192 + 2 * l);
        const float d = f16_bits_to_f32(ld16(p + 208)) * x.scale;
        return fmaf(joined(acc), d * (float)(int)(int8_t)(sc & 0xFFu), joined(acc2) * (d * (float)(int)(int8_t)(sc >> 8)));
    }
}
// 16-bit weights: the block's pieces in the order that the activations have. WIDE: p is 16-byte aligned (else 4).
template <int FMT, bool WIDE>
__device__ __forceinline__ float block_times16(const uint8_t *p, int first, const Digits<FMT> &x) {
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint8_t *q = p + 16 * ((first + i) & 3);
        uint4 v;
        if (WIDE) v = *reinterpret_cast<const uint4 *>(q);
        else v = make_uint4(ld32(q), ld32(q + 4), ld32(q + 8), ld32(q + 12));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        const float *f = reinterpret_cast<const float *>(&x.v[2 * i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float a = FMT == F_BF16 ? __uint_as_float(w[j] << 16) : f16_bits_to_f32(w[j] & 0xFFFFu);
            const float b = FMT == F_BF16 ? __uint_as_float(w[j] & 0xFFFF0000u) : f16_bits_to_f32(w[j] >> 16);
            s[0] = fmaf(a, f[2 * j], s[0]);
            s[1] = fmaf(b, f[2 * j + 1], s[1]);
        }
    }
    return s[0] + s[1];
}

// Sums over the 8 lanes of v[0 .. 7]; lane l gets v[l]'s.
__device__ __forceinline__ float sum_over_8(float *v, int l) {
#pragma unroll
    for (int n = 4; n; n >>= 1) {
        const bool up = l & n;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor_sync(~0u, give, n);
        }
    }
    return v[0];
}

// --------------------------------------------------------------- kernel ----

// Rows of a stage, bytes of a run of a row, and the 16-byte pieces that cover them (an odd number, so that 4 rows'
// words fall on different banks; 16-bit formats' lanes see to that themselves).
__host__ __device__ constexpr int stage_rows(int fmt, int unit, bool even) {
    const int r = is_16bit(fmt) ? 8 : (fmt == F_Q4_0 && !even) || fmt == F_Q4_K ? 32 : 16;
    return r < unit ? r : unit;
}
__host__ __device__ constexpr int run_bytes(int fmt) {
    return block_elems(fmt) == 256 ? block_bytes(fmt) : 256 / block_elems(fmt) * block_bytes(fmt);
}
__host__ __device__ constexpr int run_pieces(int fmt, bool even) {
    const int n = (run_bytes(fmt) + (even ? 14 : 0) + 15) / 16;
    return is_16bit(fmt) ? n : n | 1;
}
struct RowLayout {
    int w_bytes, stage, stages, ring, part_bytes, one_bytes, smem;
};
__host__ __device__ constexpr RowLayout row_layout(int fmt, bool held, bool down, bool even) {
    RowLayout l = {};
    const int unit = unit_rows(down);
    l.w_bytes = stage_rows(fmt, unit, even) * run_pieces(fmt, even) * 16;
    l.stage = l.w_bytes + (held ? 0 : 8 * kRecord);
    l.part_bytes = kRowWarps * unit * 4;
    l.one_bytes = held ? kOneBlocks * kRecord : 0;
    l.stages = (228 * 1024 / 2 - 1024 - 512 - l.part_bytes - l.one_bytes) / kRowWarps / l.stage;
    if (l.stages > 4) l.stages = 4;
    l.ring = l.stages * l.stage;
    l.smem = kRowWarps * l.ring + l.part_bytes + l.one_bytes;
    return l;
}

// HELD: the first product of one position.
template <int FMT, bool HELD, bool DOWN, bool EVEN>
__global__ void __launch_bounds__(kRowWarps * 32, 2) rows_kernel(const __grid_constant__ ProductParams p) {
    static_assert(!(HELD && DOWN), "the first product");
    constexpr RowLayout L = row_layout(FMT, HELD, DOWN, EVEN);
    constexpr int UNIT = unit_rows(DOWN), W = kRowWarps, NS = L.stages;
    constexpr int SR = stage_rows(FMT, UNIT, EVEN), PARTS = UNIT / SR;
    constexpr int CB = run_bytes(FMT), NP = run_pieces(FMT, EVEN), PITCH = 16 * NP;
    constexpr int PER = block_elems(FMT) == 256 ? 8 : 1;       // blocks that block_times' pointer covers
    constexpr int BB = is_16bit(FMT) ? 64 : block_bytes(FMT);  // its bytes
    constexpr int ROWS = DOWN ? UNIT : 32;                     // of a matrix, per unit
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int l = lane & 7, q = lane >> 3;
    uint8_t *const ring = smem + warp * L.ring;
    float *const part = reinterpret_cast<float *>(smem + W * L.ring);
    uint8_t *const one = smem + W * L.ring + L.part_bytes;

    pdl_wait_prev();

    const int slices = p.slices, groups = W / slices;
    const int group = warp / slices, slice = warp % slices;
    const int row_blocks = (p.rows + ROWS - 1) / ROWS;
    const int runs = (p.blocks + 7) / 8;
    const int units = (DOWN ? p.n_pos : p.n_pos * p.top_k) * row_blocks;
    const int items = DOWN ? p.top_k * runs : runs;  // of a unit: runs, of the slots one after the other
    const int first_unit = blockIdx.x * groups + group, unit_step = gridDim.x * groups;
    if (HELD && blockIdx.x == 0 && warp == 0)  // (several positions: the launch before has looked)
        for (int i = lane; i < p.top_k; i += 32)
            if (p.ids[i] < -1 || p.ids[i] >= p.n_experts) record_error(p.err, DERR_BAD_ID);

    // the experts of a unit's slots (in lanes, 32 at a time), -1: none
    struct Unit {
        int pair, row;  // its first
        int experts[DOWN ? 2 : 1];
        __device__ __forceinline__ int expert(int slot) const {
            return DOWN ? __shfl_sync(~0u, experts[DOWN && slot >= 32], slot & 31) : experts[0];
        }
    };
    auto unit_of = [&](int unit) {
        Unit u;
        const int at = unit / row_blocks;
        u.pair = DOWN ? at * p.top_k : at;
        u.row = (unit - at * row_blocks) * ROWS;
#pragma unroll
        for (int i = 0; i < (DOWN ? 2 : 1); ++i) {
            const int slot = DOWN ? 32 * i + lane : 0;
            const int e = slot < p.top_k ? p.ids[u.pair + slot] : -1;
            u.experts[i] = e >= 0 && e < p.n_experts ? e : -1;
        }
        return u;
    };
    // row of the matrix for a unit's row (the last one in place of those past the end, whose results are dropped)
    auto row_of = [&](int row, int u) { return min(row + (DOWN ? u : u & 31), p.rows - 1); };

    // ---- copies: the unit, run and part that are loaded next ----
    int load_unit = first_unit, load_item = slice, load_run = slice, load_slot = 0, load_part = 0;
    bool opened = false, turned = false;
    int load_expert = -1;
    Unit from = {};
    const uint8_t *records = nullptr, *slice_at[2] = {};
    constexpr int COPIES = (SR * NP + 31) / 32;
    int piece_at[COPIES];  // of a stage's first row (EVEN: its row)
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
        const int piece = 32 * i + lane, row = piece / NP;
        piece_at[i] = row * (int)p.row_bytes + (EVEN ? 0 : 16 * (piece - row * NP));
    }
    auto load = [&](int slot) {
        const uint32_t at = smem_addr(ring) + slot * L.stage;
        const int at_run = load_run * CB, left = (int)p.row_bytes - at_run;
        // 16 bytes a lane, row after row: neighbouring lanes' copies share the sectors of L2 and the
        // wavefronts of the shared memory (four lanes a row took 2.5 times as many of these)
        const int u0 = load_part * SR;
        if (!EVEN && left >= CB && from.row + ROWS <= p.rows) {
            const uint8_t *b = (DOWN || u0 < 32 ? slice_at[0] : slice_at[1]) +
                               (int64_t)(from.row + (DOWN ? u0 : u0 & 31)) * p.row_bytes + at_run;
#pragma unroll
            for (int i = 0; i < COPIES; ++i)
                if ((SR * NP) % 32 == 0 || i + 1 < COPIES || 32 * i + lane < SR * NP)
                    cp_async16(at + 512 * i + 16 * lane, b + piece_at[i], 16);
        } else if (EVEN && (left >= CB || !is_16bit(FMT)) && from.row + ROWS <= p.rows &&
                   (int64_t)(from.row + ROWS - 1) * p.row_bytes + at_run + 16 * NP <= p.slice_bytes) {
            // the whole pieces that a run lies in: what they hold beside it stays unused (a 16-bit block may end
            // inside the run's last one, and takes the zeros below)
            const uint8_t *b = (DOWN || u0 < 32 ? slice_at[0] : slice_at[1]) +
                               (int64_t)(from.row + (DOWN ? u0 : u0 & 31)) * p.row_bytes + at_run;
#pragma unroll
            for (int i = 0; i < COPIES; ++i)
                if ((SR * NP) % 32 == 0 || i + 1 < COPIES || 32 * i + lane < SR * NP) {
                    const int piece = 32 * i + lane;
                    const uint8_t *r = b + piece_at[i];
                    r -= reinterpret_cast<uintptr_t>(r) & 15u;
                    cp_async16(at + 512 * i + 16 * lane, r + 16 * (piece % NP), 16);
                }
        } else {
#pragma unroll 1
            for (int piece = lane; piece < SR * NP; piece += 32) {
                const int row = piece / NP, t = piece - row * NP, u = u0 + row;
                const uint8_t *b = (DOWN || u < 32 ? slice_at[0] : slice_at[1]) + row_of(from.row, u) * p.row_bytes + at_run;
                const int off = EVEN ? (int)(reinterpret_cast<uintptr_t>(b) & 15u) : 0;
                // bytes past the run's end are zeros
                const int n = off + min(CB, left) - 16 * t;
                cp_async16(at + 16 * piece, n > 0 ? b - off + 16 * t : b - off, n <= 0 ? 0 : n < 16 ? n : 16);
            }
        }
        if (!HELD && load_part == 0) {
            const uint8_t *r = records + load_run * (8 * kRecord) + 16 * lane;
#pragma unroll
            for (int j = 0; j < 8 * kRecord; j += 512)
                if (j + 512 <= 8 * kRecord || j + 16 * lane < 8 * kRecord) cp_async16(at + L.w_bytes + j + 16 * lane, r + j, 16);
        }
    };
    auto load_next = [&](int slot) {
        // on to this warp's next item that has an expert
        while (load_unit < units) {
            if (!opened) {
                from = unit_of(load_unit);
                load_item = load_run = slice;
                load_slot = 0;
                opened = turned = true;
            }
            if (load_item >= items) {
                load_unit += unit_step;
                opened = false;
                continue;
            }
            if (DOWN)
                while (load_run >= runs) {
                    load_run -= runs;
                    ++load_slot;
                    turned = true;
                }
            if (turned) {
                turned = false;
                load_expert = from.expert(load_slot);
                const int64_t base = load_expert * p.slice_bytes;
                slice_at[0] = p.w[0] + base;
                slice_at[1] = p.w[1] + base;
                records = p.x + (DOWN ? from.pair + load_slot : from.pair / p.top_k) * p.x_row_bytes;
            }
            if (load_expert >= 0) break;
            load_item += slices;
            load_run += slices;
        }
        if (load_unit < units) {
            load(slot);
            if (++load_part == PARTS) {
                load_part = 0;
                load_item += slices;
                load_run += slices;
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < NS - 1; ++i) load_next(i);

    if constexpr (HELD) {
        // x's records, while the first weights are on their way
        for (int b = warp; b < runs * 8; b += W) {
            const int e = 32 * b + lane;
            put_record(e < p.k ? p.x32[e] : 0.0f, lane, FMT, one + b * kRecord);
        }
        __syncthreads();
    }

    // ---- products ----
    int slot = 0;
    float *const sums = part + group * slices * UNIT;
    for (int unit = first_unit; unit < units; unit += unit_step) {
        const Unit here = unit_of(unit);
        if (!DOWN && here.expert(0) < 0) continue;
        float sum[UNIT / 4];  // rows 4 j + q
#pragma unroll
        for (int j = 0; j < UNIT / 4; ++j) sum[j] = 0.0f;
        int run = slice, j0 = 0, expert = -1;
        bool turn = true;
        for (int item = slice; item < items; item += slices) {
            if (DOWN)
                while (run >= runs) {
                    run -= runs;
                    ++j0;
                    turn = true;
                }
            if (turn) expert = here.expert(j0);
            turn = false;
            if (expert < 0) {  // nothing has been loaded for it
                run += slices;
                continue;
            }
            Digits<FMT> x;
            const bool on = run * 8 + l < p.blocks;
#pragma unroll
            for (int a = 0; a < PARTS; ++a) {
                cp_async_wait<NS - 2>();
                __syncwarp();  // the stage is there for every lane, and the one before it is free
                load_next(slot == 0 ? NS - 1 : slot - 1);
                const uint8_t *stage = ring + slot * L.stage;
                if (a == 0) x.load((HELD ? one + run * (8 * kRecord) : stage + L.w_bytes) + l * kRecord, l >> 1);
                const uint8_t *r = stage + q * PITCH + (PER == 8 ? 0 : l * BB);
                uint32_t low = 0;
                if (EVEN)
                    low = (uint32_t)(reinterpret_cast<uintptr_t>(p.w[DOWN ? 0 : a * SR >> 5]) + expert * p.slice_bytes) + run * CB;
#pragma unroll
                for (int i = 0; i < SR / 4; ++i) {
                    const uint8_t *b = r + 4 * i * PITCH;
                    if (EVEN) b += (low + (uint32_t)row_of(here.row, a * SR + 4 * i + q) * (uint32_t)p.row_bytes) & 15u;
                    float v;
                    if constexpr (is_16bit(FMT)) v = block_times16<FMT, !EVEN>(b, l >> 1, x);
                    else v = block_times<FMT>(b, l, x);
                    // (a block past the row's end has been copied as zeros, but meets no record)
                    if (on) sum[a * (SR / 4) + i] += v;
                }
                if (++slot == NS) slot = 0;
            }
            run += slices;
        }

        // ---- the unit's results: the slices' sums, in order ----
        // 64 rows: lane (q, l) gets rows 4 l + q and 4 l + q + 32; 16 rows: lanes l = 0 .. 3 get row 4 l + q
        float s[UNIT / 32 ? UNIT / 32 : 1];
        if constexpr (UNIT == 64) {
            s[0] = sum_over_8(sum, l);
            s[1] = sum_over_8(sum + 8, l);
        } else {
            static_assert(UNIT == 16 && PARTS == UNIT / SR, "16 or 64 rows");
            float v[8] = {sum[0], sum[1], sum[2], sum[3], 0, 0, 0, 0};
            s[0] = sum_over_8(v, l);
        }
        const int r = 4 * l + q;
        const bool mine = UNIT == 64 || l < 4;
        if (slices > 1) {
            float *const to = sums + slice * UNIT;
            if (mine) {
                to[r] = s[0];
                if (UNIT == 64) to[r + 32] = s[UNIT / 64];
            }
            named_barrier(1 + group, slices * 32);
            if (slice == 0 && mine) {
                for (int i = 1; i < slices; ++i) {
                    s[0] += sums[i * UNIT + r];
                    if (UNIT == 64) s[UNIT / 64] += sums[i * UNIT + r + 32];
                }
            }
        }
        if (slice == 0) {
            if constexpr (DOWN) {
                float *const out = p.out + (int64_t)(unit / row_blocks) * p.rows + here.row + r;
                if (mine && here.row + r < p.rows) *out = p.accumulate ? *out + s[0] : s[0];
            } else {
                const float w = p.weights[here.pair];
                const float h = here.row + r < p.rows ? glu_gate(s[0], glu_arg(p.act, s[0])) * s[1] * w : 0.0f;
                put_record(h, r, p.h_fmt, p.h + here.pair * p.h_row_bytes + (int64_t)(here.row / 32) * kRecord);
            }
        }
        if (slices > 1) named_barrier(1 + group, slices * 32);  // the sums have been taken
    }
    cp_async_wait<0>();
    pdl_launch_dependents();
}

template <int FMT, bool HELD, bool DOWN, bool EVEN>
cudaError_t launch_rows(const ProductParams &p, const DeviceInfo &dev, cudaStream_t s) {
    constexpr RowLayout L = row_layout(FMT, HELD, DOWN, EVEN);
    static_assert(L.stages >= 2, "two stages");
    static OncePerDevice once;
    cudaError_t e = allow_smem(once, rows_kernel<FMT, HELD, DOWN, EVEN>, L.smem);
    if (e != cudaSuccess) return e;
    constexpr int ROWS = DOWN ? unit_rows(DOWN) : 32;
    const int64_t units = (int64_t)p.n_pos * (DOWN ? 1 : p.top_k) * ((p.rows + ROWS - 1) / ROWS);
    const int64_t wave = (int64_t)dev.sm_count * 2;
    // as few slices as give every warp a unit's share, or two (with fewer, a
    // warp that has two units keeps all others waiting), and no more than there are runs
    const int runs = (p.blocks + 7) / 8 * (DOWN ? p.top_k : 1);
    ProductParams r = p;
    r.slices = 1;
    while (r.slices < kRowWarps && 2 * r.slices <= runs && units * r.slices < 2 * wave * kRowWarps) r.slices *= 2;
    const int64_t ctas = (units * r.slices + kRowWarps - 1) / kRowWarps;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(ctas < wave ? ctas : wave));
    cfg.blockDim = dim3(kRowWarps * 32);
    cfg.dynamicSmemBytes = L.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rows_kernel<FMT, HELD, DOWN, EVEN>, r);
}

// EVEN: rows that are not made of whole 16 bytes
template <int FMT, bool HELD, bool DOWN>
cudaError_t launch_rows(const ProductParams &p, const DeviceInfo &dev, cudaStream_t s) {
    if constexpr (FMT == F_Q4_K) {
        return launch_rows<FMT, HELD, DOWN, false>(p, dev, s);
    } else if constexpr (FMT == F_Q6_K) {
        return launch_rows<FMT, HELD, DOWN, true>(p, dev, s);
    } else {
        return p.row_bytes % 16 ? launch_rows<FMT, HELD, DOWN, true>(p, dev, s) : launch_rows<FMT, HELD, DOWN, false>(p, dev, s);
    }
}

template <int FMT>
cudaError_t launch_single(bool down, const ProductParams &p, const DeviceInfo &dev, cudaStream_t s) {
    if (down) return launch_rows<FMT, false, true>(p, dev, s);
    return p.x32 ? launch_rows<FMT, true, false>(p, dev, s) : launch_rows<FMT, false, false>(p, dev, s);
}

}  // namespace experts
}  // namespace qmm
