// qmm_attend_kernel.cuh -- attention of new rows over the paged key-value
// cache, o = sum_t softmax_t(scale q . k_t) v_t, read in its packed form.
//
// Work. An item is one query row (one new position of one sequence), one kv
// head and up to eight of the query heads that share it, so that every cached
// byte fetched serves all of them, and all query rows of an item see the same
// positions. An item's positions are cut into strips of 16 (one contiguous
// piece of a page). The strips of all items, laid end to end, are divided
// evenly among the CTAs of one resident wave, whatever the lengths are; an
// item whose strips fall to several CTAs is joined by attend_join_kernel from
// partial results (maximum, total, weighted sum).
//
// A CTA is kWarps warps that take an item's strips in turn. Each warp streams
// its strips through a ring of its own in shared memory with bulk copies (one
// or two per strip, issued by one lane, no barrier between warps) and keeps a running
// maximum m, total l and weighted sums in registers, fp32.
//
// Scores and sums are tensor-core products (mma.m16n8k16) on fragments that
// are unpacked from the strip in registers:
//  - S = Q K^T: eight query rows are the 16 rows of A as two fp16 terms each
//    (rows g and g + 8 of a fragment are the high part and the remainder, 22
//    significant bits, after a power-of-two scale per row), the strip's 16
//    positions are two n-tiles. Integer codes enter as exact fp16 integers; a
//    block's scale multiplies its fp32 partial sum.
//  - O^T = V^T P^T: 16 dims are the rows of A, the eight query rows the columns
//    of B. The weights p enter as two fp16 terms as well (two products into
//    one accumulator). For quantised V a block's scale d is folded into the
//    weight first: w = p d. A common power of two keeps the largest w near
//    2^14, where both terms are normal numbers: p's exponent carries it, as
//    part of the maximum that is subtracted, and it follows the largest |d|
//    seen, like the maximum itself.
//  - BF16 K and V are bf16 operands; q and p then have three bf16 terms.
// The scores of a strip come out of the first product in the lanes that need
// them for the second, so p stays in registers.
#pragma once

#include "qmm_attend.h"

namespace qmm {

namespace attend {

// ---------------------------------------------------------- small pieces ----

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
template <int F>
__device__ __forceinline__ void mma16(float (&c)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
    if constexpr (F == F_BF16) mma_bf16(c, a, b0, b1);
    else mma_f16(c, a, b0, b1);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}
__device__ __forceinline__ float2 unpack_bf16(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
// A pair of fp32 values as 16-bit terms whose sum they are: two of fp16 (22
// bits), three of bf16 (24 bits).
template <bool BF>
__device__ __forceinline__ void split(float x, float y, uint32_t (&t)[3]) {
    if constexpr (BF) {
        t[0] = pack_bf16(x, y);
        const float2 a = unpack_bf16(t[0]);
        const float rx = x - a.x, ry = y - a.y;
        t[1] = pack_bf16(rx, ry);
        const float2 b = unpack_bf16(t[1]);
        t[2] = pack_bf16(rx - b.x, ry - b.y);
    } else {
        t[0] = pack_f16(x, y);
        const float2 a = unpack_f16(t[0]);
        t[1] = pack_f16(x - a.x, y - a.y);
        t[2] = 0;
    }
}

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Bytes (two's complement, bit 7 already flipped) I0 and I1 of w as an exact
// fp16 pair: the byte under the exponent of 1024, less 1024 + 128.
template <int SEL>
__device__ __forceinline__ uint32_t bytes_f16(uint32_t w) {
    return hsub2(prmt(w, 0x64646464u, SEL), 0x64806480u);
}
// The two nibbles that sit at bits SH and SH + 16 of w (SH 0 or 4), less 8, as
// an exact fp16 pair: 1024 + n - 1032, or (1024 + 16 n) / 16 - 72.
template <int SH>
__device__ __forceinline__ uint32_t nibbles_f16(uint32_t w) {
    if constexpr (SH == 0) return hsub2((w & 0x000f000fu) | 0x64006400u, 0x64086408u);
    else return hfma2((w & 0x00f000f0u) | 0x64006400u, 0x2c002c00u, 0xd480d480u);
}

// ------------------------------------------------------------- fragments ----
// Lane 4 g + j of a warp. Position n of n-tile x is position
// 8 x + (n ^ (n >> 2)) of the strip: with this order both the eight positions
// g of a K fragment and the positions 2 j + e of a V fragment (e fixed) fall
// on distinct banks of a plane.

// B fragments of K: per 16 dims ("step") two registers for one n-tile.
// dims of lane j, step k: 16-bit: 16 k + 4 j + {0, 1 | 2, 3}; Q8_0: plane k/2,
// 8 j + 4 (k % 2) + {0, 1 | 2, 3}; Q4_0: plane k/2, 8 j + 2 (k % 2) +
// {0, 4 | 1, 5}.
// For a plane p of K at `base`, `row` = the lane's position times the row
// bytes plus its byte offset: fills the steps of that plane.
template <int F>
__device__ __forceinline__ void k_frag(uint32_t base, int p, uint32_t row, uint32_t (&b)[4]) {
    if constexpr (!kv_quantised(F)) {
        const uint2 w = lds64(base + p * 512 + row);
        b[0] = w.x;
        b[1] = w.y;
    } else if constexpr (F == F_Q8_0) {
        uint2 w = lds64(base + p * 512 + row);
        w.x ^= 0x80808080u;
        w.y ^= 0x80808080u;
        b[0] = bytes_f16<0x4140>(w.x);
        b[1] = bytes_f16<0x4342>(w.x);
        b[2] = bytes_f16<0x4140>(w.y);
        b[3] = bytes_f16<0x4342>(w.y);
    } else {
        const uint32_t w = lds32(base + p * 256 + row), v = w >> 8;
        b[0] = nibbles_f16<0>(w);
        b[1] = nibbles_f16<4>(w);
        b[2] = nibbles_f16<0>(v);
        b[3] = nibbles_f16<4>(v);
    }
}

// A fragments of V^T from plane p: rows are dims, columns positions. 16-bit:
// one tile, rows g and g + 8 are dims 16 p + 2 g and + 1. Quantised: two
// tiles, rows g and g + 8 of tile u are dims 32 p + 4 g + 2 u and + 1.
// row[x][e]: byte offset of the lane's position e of n-tile x and its dims.
template <int F>
__device__ __forceinline__ void v_frag(uint32_t base, int p, const uint32_t (&row)[2][2],
                                       uint4 (&a)[2]) {
    if constexpr (!kv_quantised(F)) {
        const uint32_t w00 = lds32(base + p * 512 + row[0][0]), w01 = lds32(base + p * 512 + row[0][1]);
        const uint32_t w10 = lds32(base + p * 512 + row[1][0]), w11 = lds32(base + p * 512 + row[1][1]);
        a[0] = make_uint4(prmt(w00, w01, 0x5410), prmt(w00, w01, 0x7632), prmt(w10, w11, 0x5410),
                          prmt(w10, w11, 0x7632));
    } else if constexpr (F == F_Q8_0) {
        uint32_t lo[2], hi[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint32_t w0 = lds32(base + p * 512 + row[x][0]) ^ 0x80808080u;
            const uint32_t w1 = lds32(base + p * 512 + row[x][1]) ^ 0x80808080u;
            lo[x] = prmt(w0, w1, 0x5140);
            hi[x] = prmt(w0, w1, 0x7362);
        }
        a[0] = make_uint4(bytes_f16<0x4140>(lo[0]), bytes_f16<0x4342>(lo[0]), bytes_f16<0x4140>(lo[1]),
                          bytes_f16<0x4342>(lo[1]));
        a[1] = make_uint4(bytes_f16<0x4140>(hi[0]), bytes_f16<0x4342>(hi[0]), bytes_f16<0x4140>(hi[1]),
                          bytes_f16<0x4342>(hi[1]));
    } else {
        uint32_t w[2], v[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            w[x] = prmt(lds16(base + p * 256 + row[x][0]), lds16(base + p * 256 + row[x][1]), 0x5410);
            v[x] = w[x] >> 8;
        }
        a[0] = make_uint4(nibbles_f16<0>(w[0]), nibbles_f16<4>(w[0]), nibbles_f16<0>(w[1]),
                          nibbles_f16<4>(w[1]));
        a[1] = make_uint4(nibbles_f16<0>(v[0]), nibbles_f16<4>(v[0]), nibbles_f16<0>(v[1]),
                          nibbles_f16<4>(v[1]));
    }
}

// ----------------------------------------------------------------- config ----

template <int FK, int FV, int D>
struct Cfg {
    static constexpr Shape kShape = shape_of(FK, FV, D);
    static constexpr int kUnits = kShape.units, kSlots = kShape.slots, kSlotBytes = kShape.slot_bytes;
    static constexpr int kBytesK = kv_half_bytes(FK, D), kBytesV = kv_half_bytes(FV, D);
    static constexpr int kSteps = D / 16;
    static constexpr int kQBytes = kShape.q_bytes;
    static constexpr int kRingBytes = kShape.ring_bytes;
    static constexpr int kMergeRow = D + 4;  // floats; + 4 spreads the rows j over the banks
    static constexpr int kSmem = kShape.smem;
    static_assert(kSlots >= 2, "a ring needs two slots");
    static_assert(kShape.ctas * (kSmem + 1024) <= 228 * 1024, "shared memory of an SM");
    static_assert(kSlotBytes % 16 == 0 && kBytesK % 16 == 0 && kRingBytes % 16 == 0 && kQBytes % 16 == 0,
                  "alignment");
};

// ---------------------------------------------------------------- kernel ----

template <int FK, int FV, int D>
__global__ void __launch_bounds__(kThreads, Cfg<FK, FV, D>::kShape.ctas)
    attend_kernel(const AttendParams a) {
    using C = Cfg<FK, FV, D>;
    constexpr bool kBfK = FK == F_BF16, kBfV = FV == F_BF16;
    constexpr int kPlanesK = D / kv_plane_dims(FK), kPlanesV = D / kv_plane_dims(FV);
    constexpr int kStepsPerPlane = kv_plane_dims(FK) / 16;  // 2 for quantised K
    constexpr int kTilesPerPlane = kv_plane_dims(FV) / 16;  // 2 for quantised V
    extern __shared__ __align__(128) uint8_t smem[];
    // fixed part: barriers, flags, row scales, softmax states, work search
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem);                      // [kWarps][kMaxSlots]
    uint32_t *skip = reinterpret_cast<uint32_t *>(smem + kWarps * 64);        // [kWarps][kMaxSlots]
    float *row_scale = reinterpret_cast<float *>(smem + kWarps * 96);         // [kRows]
    float *state_m = row_scale + kRows;                                       // [kWarps][kRows]
    float *state_l = state_m + kWarps * kRows;                                // [kWarps][kRows]
    WorkSearch *search = reinterpret_cast<WorkSearch *>(state_l + kWarps * kRows);
    uint8_t *q_frag = smem + kFixedBytes;
    const KvView &c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, j = lane & 3;
    const uint32_t bar0 = smem_addr(bars + warp * kMaxSlots);
    uint8_t *ring_ptr = q_frag + C::kQBytes + warp * C::kRingBytes;
    const uint32_t ring = smem_addr(ring_ptr), qf = smem_addr(q_frag);
    if (lane == 0) {
        for (int i = 0; i < C::kSlots; ++i) mbar_init(bar0 + 8 * i, 1);
        fence_barrier_init();
    }
    pdl_wait_prev();
    pdl_launch_dependents();

    Work w;
    if (!find_work(a, (int)blockIdx.x, search, w)) {
        if (threadIdx.x == 0) a.joins[blockIdx.x].parts = 0;
        return;
    }
    Join next_join;
    next_join.parts = 0;

    // positions of this lane's fragments in a strip
    const uint32_t k_pos = g ^ (g >> 2);
    const uint32_t k_row = k_pos * kv_row_bytes(FK) + j * (FK == F_Q4_0 ? 4 : 8);
    uint32_t v_row[2][2];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e)
            v_row[x][e] = (8 * x + ((2 * j + e) ^ (j >> 1))) * kv_row_bytes(FV) + g * (FV == F_Q4_0 ? 2 : 4);
    const uint32_t swap = (j >> 1) ? 0x1032u : 0x3210u;  // order of a pair of scales

    int issued = 0, taken = 0;  // strips of this warp over the whole launch: ring phases
    bool dead = false;
    Item it;
    while (next_item(a, w, it)) {
        // ---- copies of the first strips ----
        const int mine =
            !dead && it.end > it.begin + warp ? (it.end - it.begin - warp + kWarps - 1) / kWarps : 0;
        // copies ("units") are numbered over the whole launch; strip n of this
        // warp and item is it.begin + warp + kWarps n
        const int base = issued, goal = issued + mine * C::kUnits;
        const uint8_t *src = nullptr;
        auto issue = [&]() {
            const int n = (issued - base) / C::kUnits;
            const bool is_v = C::kUnits == 2 && ((issued - base) & 1);
            if ((n & 31) == 0 && !is_v) {  // the addresses of the next 32 strips, one per lane
                const int strip = it.begin + warp + kWarps * (n + lane);
                src = strip < it.end && it.live ? kv_strip(c, it.seq, it.head, it.first + strip) : nullptr;
            }
            const int slot = issued % C::kSlots;
            if (lane == (n & 31)) {
                skip[warp * kMaxSlots + slot] = src == nullptr;
                if (src) {
                    const uint32_t bytes = C::kUnits == 1 ? C::kBytesK + C::kBytesV
                                           : is_v         ? C::kBytesV
                                                          : C::kBytesK;
                    mbar_arrive_expect_tx(bar0 + 8 * slot, bytes);
                    bulk_g2s(ring + slot * C::kSlotBytes, is_v ? src + C::kBytesK : src, bytes, bar0 + 8 * slot);
                } else {
                    mbar_arrive(bar0 + 8 * slot);
                }
            }
            ++issued;
        };
        // unit `taken` has landed; its slot
        auto await = [&]() {
            const int slot = taken % C::kSlots;
            if (!mbar_wait(bar0 + 8 * slot, (uint32_t)(taken / C::kSlots) & 1u)) {
                if (lane == 0) record_error(c.err, DERR_ATTEND);
                dead = true;
            }
            return slot;
        };
        // unit `taken` has been read by the whole warp: its slot is refilled
        auto release = [&]() {
            ++taken;
            fence_proxy_async_smem();
            __syncwarp();
            if (issued < goal) issue();
        };
        while (issued < goal && issued < taken + C::kSlots) issue();

        // ---- query rows as A fragments ----
        {
            const int row = threadIdx.x >> 4, part = threadIdx.x & 15;
            const bool there = row < it.heads;
            const float *q = a.q + it.row * a.q_stride + (int64_t)(it.head0 + row) * D;
            float x[(D + 127) / 128][8];
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < (D + 127) / 128; ++i) {
                const int d = 8 * (part + 16 * i);
#pragma unroll
                for (int k = 0; k < 8; ++k) x[i][k] = 0.0f;
                if (there && d < D) {
                    if (a.vec) {
                        const float4 u = *reinterpret_cast<const float4 *>(q + d);
                        const float4 v = *reinterpret_cast<const float4 *>(q + d + 4);
                        x[i][0] = u.x; x[i][1] = u.y; x[i][2] = u.z; x[i][3] = u.w;
                        x[i][4] = v.x; x[i][5] = v.y; x[i][6] = v.z; x[i][7] = v.w;
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k) x[i][k] = q[d + k];
                    }
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(x[i][k]));
            }
            float up = 1.0f, down = 1.0f;
            if constexpr (!kBfK) {  // largest |q| of the row into [2^13, 2^14)
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
                const int e = (int)(__float_as_uint(top) >> 23) - 127;
                const int k = top == 0.0f ? 0 : max(-114, min(126, 13 - e));
                up = __uint_as_float((uint32_t)(127 + k) << 23);
                // 2^-126 for k = 126 is the smallest normal number
                down = __uint_as_float((uint32_t)(127 - k) << 23);
            }
            if (part == 0) row_scale[row] = a.scale_log2 * down;
#pragma unroll
            for (int i = 0; i < (D + 127) / 128; ++i) {
                const int d = 8 * (part + 16 * i);
                if (d < D) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        // four dims: step and lane they belong to (see k_frag)
                        int step, jj;
                        float v0, v1, v2, v3;
                        if constexpr (FK == F_Q4_0) {
                            step = d / 32 * 2 + h;
                            jj = d % 32 / 8;
                            v0 = x[i][2 * h]; v1 = x[i][2 * h + 4];
                            v2 = x[i][2 * h + 1]; v3 = x[i][2 * h + 5];
                        } else {
                            step = FK == F_Q8_0 ? d / 32 * 2 + h : d / 16;
                            jj = FK == F_Q8_0 ? d % 32 / 8 : d % 16 / 4 + h;
                            v0 = x[i][4 * h]; v1 = x[i][4 * h + 1];
                            v2 = x[i][4 * h + 2]; v3 = x[i][4 * h + 3];
                        }
                        uint32_t s[3], t[3];
                        split<kBfK>(v0 * up, v1 * up, s);
                        split<kBfK>(v2 * up, v3 * up, t);
                        const int at = step * 32 + row * 4 + jj;
                        sts128(qf + at * 16, s[0], s[1], t[0], t[1]);
                        if constexpr (kBfK) {
                            uint32_t *p = reinterpret_cast<uint32_t *>(q_frag + C::kSteps * 512) + 2 * at;
                            p[0] = s[2];
                            p[1] = t[2];
                        }
                    }
                }
            }
        }
        __syncthreads();

        // ---- the strips ----
        const float rs = row_scale[g];
        float o[D / 16][4];
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[i][k] = 0.0f;
        // m: running maximum of the scores (log2 domain); ref: what is
        // subtracted, m less the exponent `up` that the weights carry
        float m = -INFINITY, ref = -INFINITY, l = 0.0f;
        float up = kBfV ? 0.0f : kv_quantised(FV) ? 38.0f : 14.0f;
        while (taken < goal && !dead) {
            int slot = await();
            if (dead) break;
            const uint32_t sk = ring + slot * C::kSlotBytes;
            const int first = (it.first + it.begin + warp + kWarps * ((taken - base) / C::kUnits)) * kStrip;
            const bool edge = first < it.lo || first + kStrip > it.hi;
            const bool absent = skip[warp * kMaxSlots + slot];
            float s[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
            if (!absent) {
                // scores
                float acc[2][4];
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[x][k] = 0.0f;
#pragma unroll
                for (int p = 0; p < kPlanesK; ++p) {
                    uint32_t b[2][4];
                    k_frag<FK>(sk, p, k_row, b[0]);
                    k_frag<FK>(sk, p, k_row + 8 * kv_row_bytes(FK), b[1]);
#pragma unroll
                    for (int k = 0; k < kStepsPerPlane; ++k) {
                        const int step = p * kStepsPerPlane + k;
                        const uint4 q = lds128(qf + (step * 32 + lane) * 16);
                        mma16<FK>(acc[0], q, b[0][2 * k], b[0][2 * k + 1]);
                        mma16<FK>(acc[1], q, b[1][2 * k], b[1][2 * k + 1]);
                        if constexpr (kBfK) {
                            const uint2 r = lds64(qf + C::kSteps * 512 + (step * 32 + lane) * 8);
                            const uint4 q3 = make_uint4(r.x, 0, r.y, 0);
                            mma16<FK>(acc[0], q3, b[0][0], b[0][1]);
                            mma16<FK>(acc[1], q3, b[1][0], b[1][1]);
                        }
                    }
                    if constexpr (kv_quantised(FK)) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint32_t dd =
                                lds32(sk + kv_code_bytes(FK, D) + (p * kStrip + 8 * x + 2 * j) * 2);
                            const float2 d = unpack_f16(prmt(dd, dd, swap));
                            s[x][0] = fmaf(d.x, acc[x][0] + acc[x][2], s[x][0]);
                            s[x][1] = fmaf(d.y, acc[x][1] + acc[x][3], s[x][1]);
#pragma unroll
                            for (int k = 0; k < 4; ++k) acc[x][k] = 0.0f;
                        }
                    }
                }
                if constexpr (!kv_quantised(FK)) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        s[x][0] = acc[x][0] + acc[x][2];
                        s[x][1] = acc[x][1] + acc[x][3];
                    }
                }
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        s[x][e] *= rs;
                        if (edge) {
                            const int t = first + 8 * x + ((2 * j + e) ^ (j >> 1));
                            if (t < it.lo || t >= it.hi) s[x][e] = -INFINITY;
                        }
                    }

            }
            if constexpr (C::kUnits == 2) {
                release();
                slot = await();
                if (dead) break;
            }
            const uint32_t sv = ring + slot * C::kSlotBytes + (C::kUnits == 1 ? C::kBytesK : 0);
            if (!absent) {
                if (edge) {
                    // positions that the row does not see: weights of 0 must
                    // not meet an Inf or NaN, so their V (or its scales) is cleared
                    uint8_t *v = ring_ptr + (sv - ring);
                    if constexpr (kv_quantised(FV)) {
                        uint16_t *d = reinterpret_cast<uint16_t *>(v + kv_code_bytes(FV, D));
                        for (int i = lane; i < D / 2; i += 32) {
                            const int t = first + (i & 15);
                            if (t < it.lo || t >= it.hi) d[i] = 0;
                        }
                    } else {
                        for (int i = lane; i < 2 * D; i += 32) {
                            const int t = first + ((i >> 1) & 15);
                            if (t < it.lo || t >= it.hi)
                                *reinterpret_cast<uint4 *>(v + i * 16) = make_uint4(0, 0, 0, 0);
                        }
                    }
                    __syncwarp();
                }

                // V's scales, and the exponent that they leave to the weights
                uint32_t dv[kv_quantised(FV) ? kPlanesV : 1][2];
                if constexpr (kv_quantised(FV)) {
                    uint32_t big = 0;
#pragma unroll
                    for (int p = 0; p < kPlanesV; ++p)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            dv[p][x] = lds32(sv + kv_code_bytes(FV, D) + (p * kStrip + 8 * x + 2 * j) * 2);
                            big = hmax2(big, dv[p][x] & 0x7fff7fffu);
                        }
                    big = hmax2(big, big >> 16 | big << 16);
                    big = hmax2(big, __shfl_xor_sync(~0u, big, 1));
                    big = hmax2(big, __shfl_xor_sync(~0u, big, 2));
                    // exponent of the largest scale (0 for none): weights below 2^15
                    const float top = unpack_f16(big).x;
                    const int e = (int)(__float_as_uint(top) >> 23) - 127;
                    up = fminf(up, (float)(14 - max(-24, min(15, e))));
                }

                // running maximum
                float mx = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2));
                m = fmaxf(m, mx);
                const float ref_new = m - up;  // -inf while nothing has been seen
                const float sub = ref_new == -INFINITY ? 0.0f : ref_new;
                if (__any_sync(~0u, ref_new != ref)) {
                    const float f = exp2_fast(ref - sub);
                    l *= f;
                    const float f0 = __shfl_sync(~0u, f, 8 * j), f1 = __shfl_sync(~0u, f, 8 * j + 4);
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        o[i][0] *= f0;
                        o[i][1] *= f1;
                        o[i][2] *= f0;
                        o[i][3] *= f1;
                    }
                    ref = ref_new;
                }
                float pr[2][2];
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int e = 0; e < 2; ++e) pr[x][e] = exp2_fast(s[x][e] - sub);
                l += (pr[0][0] + pr[0][1]) + (pr[1][0] + pr[1][1]);

                // weighted sum of V
                uint32_t b0[3], b1[3];
                if constexpr (!kv_quantised(FV)) {
                    split<kBfV>(pr[0][0], pr[0][1], b0);
                    split<kBfV>(pr[1][0], pr[1][1], b1);
                }
#pragma unroll
                for (int p = 0; p < kPlanesV; ++p) {
                    if constexpr (kv_quantised(FV)) {
                        const float2 d0 = unpack_f16(prmt(dv[p][0], dv[p][0], swap));
                        const float2 d1 = unpack_f16(prmt(dv[p][1], dv[p][1], swap));
                        split<false>(pr[0][0] * d0.x, pr[0][1] * d0.y, b0);
                        split<false>(pr[1][0] * d1.x, pr[1][1] * d1.y, b1);
                    }
                    uint4 v[2];
                    v_frag<FV>(sv, p, v_row, v);
#pragma unroll
                    for (int u = 0; u < kTilesPerPlane; ++u) {
                        mma16<FV>(o[p * kTilesPerPlane + u], v[u], b0[0], b1[0]);
                        mma16<FV>(o[p * kTilesPerPlane + u], v[u], b0[1], b1[1]);
                        if constexpr (kBfV) mma16<FV>(o[p * kTilesPerPlane + u], v[u], b0[2], b1[2]);
                    }
                }
            }
            release();
        }
        if (dead) {
            // nothing more is issued; copies in flight land before the block ends
            for (; taken < issued; ++taken)
                if (!mbar_wait(bar0 + 8 * (taken % C::kSlots), (uint32_t)(taken / C::kSlots) & 1u))
                    if (lane == 0) record_error(c.err, DERR_TEARDOWN);
            issued = taken;
        }

        // ---- the warps' results joined ----
        l += __shfl_xor_sync(~0u, l, 1);
        l += __shfl_xor_sync(~0u, l, 2);
        if (j == 0) {
            state_m[warp * kRows + g] = ref;
            state_l[warp * kRows + g] = l;
        }
        float *merge = reinterpret_cast<float *>(ring_ptr);  // this warp's ring, all of it taken
        if (mine > 0) {
#pragma unroll
            for (int p = 0; p < kPlanesV; ++p)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float *to = merge + (2 * j + r) * C::kMergeRow;
                    if constexpr (kv_quantised(FV))
                        *reinterpret_cast<float4 *>(to + 32 * p + 4 * g) =
                            make_float4(o[2 * p][r], o[2 * p][2 + r], o[2 * p + 1][r], o[2 * p + 1][2 + r]);
                    else
                        *reinterpret_cast<float2 *>(to + 16 * p + 2 * g) = make_float2(o[p][r], o[p][2 + r]);
                }
        }
        __syncthreads();
        const bool whole = it.begin == 0 && it.end == it.strips;
        float *part = nullptr;
        if (!whole) part = a.parts + (int64_t)(2 * (int)blockIdx.x + (it.begin == 0)) * part_floats(D);
        for (int i = threadIdx.x; i < kRows * D / 4; i += kThreads) {
            const int row = i / (D / 4), d = (i - row * (D / 4)) * 4;
            float top = -INFINITY;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) top = fmaxf(top, state_m[k * kRows + row]);
            float total = 0.0f;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float mk = state_m[k * kRows + row];
                if (mk == -INFINITY) continue;  // saw nothing
                const float f = exp2_fast(mk - top);
                const float4 v = *reinterpret_cast<const float4 *>(
                    q_frag + C::kQBytes + k * C::kRingBytes + (row * C::kMergeRow + d) * 4);
                total = fmaf(f, state_l[k * kRows + row], total);
                sum.x = fmaf(f, v.x, sum.x);
                sum.y = fmaf(f, v.y, sum.y);
                sum.z = fmaf(f, v.z, sum.z);
                sum.w = fmaf(f, v.w, sum.w);
            }
            if (whole) {
                if (row < it.heads) put_out(a, it.row, it.head0 + row, d, D, sum, total);
            } else {
                if (d == 0) {
                    part[row] = top;
                    part[kRows + row] = total;
                }
                *reinterpret_cast<float4 *>(part + 2 * kRows + row * D + d) = sum;
            }
        }
        if (it.end < it.strips) next_join = make_join(a, w, it);
        fence_proxy_async_smem();  // the merge buffers' accesses, before copies land there again
        __syncthreads();
    }
    if (threadIdx.x == 0) a.joins[blockIdx.x] = next_join;
}

template <int FK, int FV, int D>
cudaError_t launch_one(const AttendParams &a, int grid, cudaStream_t s) {
    using C = Cfg<FK, FV, D>;
    static const cudaError_t ready = cudaFuncSetAttribute(
        attend_kernel<FK, FV, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (ready != cudaSuccess) return ready;
    return launch_programmatic(attend_kernel<FK, FV, D>, a, grid, kThreads, C::kSmem, s);
}

template <int FK, int FV>
cudaError_t launch_format(const AttendParams &a, int grid, cudaStream_t s) {
    switch (a.c.dim) {
    case 64: return launch_one<FK, FV, 64>(a, grid, s);
    case 96: return launch_one<FK, FV, 96>(a, grid, s);
    case 128: return launch_one<FK, FV, 128>(a, grid, s);
    case 192: return launch_one<FK, FV, 192>(a, grid, s);
    case 256: return launch_one<FK, FV, 256>(a, grid, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace attend

}  // namespace qmm
