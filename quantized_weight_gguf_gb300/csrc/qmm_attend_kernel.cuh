// qmm_attend_kernel.cuh -- attention of new rows over the paged key-value
// cache, o = sum_t softmax_t(scale q . k_t) v_t, read in its packed form.
//
// Work. The query rows that read one kv head of one sequence (its group of
// query heads, at each of the n_new new positions) are taken eight at a time:
// an item, for which every cached byte is fetched and unpacked once. The
// positions that one of its rows sees are cut into strips of 16 (one
// contiguous piece of a page); rows of several new positions differ at the
// range's ends only, where scores are dropped row by row. The strips of all
// items, laid end to end, are divided evenly among the CTAs of one resident
// wave, whatever the lengths are; an item whose strips fall to several CTAs is
// joined by attend_join_kernel from partial results (maximum, total, weighted
// sum). Short items are dealt out whole (see whole_strips).
//
// A CTA is kWarps warps that take an item's strips in turn, up to four at a
// time where the ring has room. Each warp streams its strips through a ring of its
// own in shared memory with bulk copies (one or two per strip, issued by one
// lane, no barrier between warps) and keeps totals and weighted sums in
// registers, fp32.
//
// Scores and sums are tensor-core products (mma.m16n8k16) on fragments that
// are unpacked from the strip in registers:
//  - S = Q K^T: eight query rows are the 16 rows of A as two fp16 terms each
//    (rows g and g + 8 of a fragment are the high part and the remainder, 22
//    significant bits, after a power-of-two scale per row), a strip's 16
//    positions are two n-tiles. A block's scale multiplies its fp32 sum.
//  - O^T = V^T P^T: 16 dims are the rows of A, the eight query rows the columns
//    of B. The weights p enter as two fp16 terms as well (two products). For
//    quantised V a block's scale d is folded into the weight's terms first,
//    w = p d = h + r: h = fl(p_h d), and with one fma each
//    r = fl(p_r d + (p_h d - h)), where the bracket is exact unless it falls
//    below 2^-24, fp16's last place (see the spans below). The product over
//    the strips taken together starts from zero and is added to the running
//    sums in fp32, so their rounding is to nearest.
//  - Integer codes enter as exact fp16 integers: the code with its offset
//    under the exponent of 1024 (a byte permute or a mask), less 1024 and the
//    offset. (Leaving the offset in, to be subtracted from the sums, or taking
//    the code as a subnormal, saves that subtraction, but the tensor cores cut
//    each product at the largest one's last bits: the sum over 15 Q4_0
//    positions then missed the tests' bound.)
//  - BF16 K and V are bf16 operands; q and p then have three bf16 terms.
// The scores of a strip come out of the first product in the lanes that need
// them for the second, so p stays in registers.
//
// The softmax subtracts a reference R per row that is not the exact running
// maximum: a weight p = 2^(s - R) may grow to 2^15 (2^12 over Q4_0 V, whose
// scales are larger; 2^-12 over BF16 V, whose values may be as large as fp32's,
// so that thousands of them can be summed before the division by the total).
// Only when a score passes that limit is R moved, to 4 below
// the limit for the largest score seen, and the sums rescaled; so a strip
// normally takes no shuffles.
//
// The terms of w = p d reach from 2^15 down to 2^-24. For scales d between 2^-11
// and 1 (2^-8 and 8 for Q4_0) they hold the largest weight's product to 22 bits
// and more. A run of strips with a scale outside goes through the second product
// lifted: d times a power of two (exact) that brings the run's largest scale to
// the top of that range, and the product's sums brought down again in fp32. Where
// its scales spread over more than 2^11 that is done once per span of 2^11, with
// that span's scales alone. Without lifts 4000 positions of V of size 1e-5 in Q8_0
// were off by 1.2e-3. Looking for such scales costs 1 us of 45 with 64 dims in
// Q4_0 and nothing that shows elsewhere; lifted, 16 sequences of 8000 positions
// over 16 kv heads of 64 in Q4_0 take 61 us (49 without) and with two spans in
// every run 93.
//
// What bounds it (fractions are of a copy's 6.8 TB/s; device times in a graph).
// 16-bit caches and 8-bit ones: DRAM, and for short work the way to the first
// strip (about 4 us: lengths, page table and strip wait for one another) and
// the join (3 to 4 us). 64 ragged F16 sequences of up to 8190 positions (1.18 GB)
// take 182 us, 6.5 TB/s, 96 %, with the arithmetic left out 177; one Q8_0
// sequence of 131071 (285 MB) 52 us, 81 %, 49 without the arithmetic, 45
// without the copies. 4-bit caches: the unpacking's integer and fp16
// instructions, about 300 warp instructions for a strip of 64 dims (1152
// bytes): 16 sequences with 16 kv heads (129 MB) take 46 us, 41 % (when it was
// 45.4: 41 without the copies, 28 without the arithmetic); the schedulers
// issue in 59 % of their cycles, the tensor pipe is busy in 31 %. Several new
// positions: the same instructions, shared by up to eight query rows: 8
// positions of 16 heads over 4-bit caches take 19 us, where one position at a
// time took 78.
#pragma once

#include <cfloat>

#include "qmm_attend.h"

namespace qmm {

namespace attend {

// ---------------------------------------------------------- small pieces ----

// d = a b + c on one m16n8k16 fragment, operands in fp16 or bf16
template <bool BF>
__device__ __forceinline__ float4 mma(const uint4 &a, uint32_t b0, uint32_t b1, const float4 &c) {
    float4 d;
    if constexpr (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%10, %11, %12, %13};"
            : "=f"(d.x), "=f"(d.y), "=f"(d.z), "=f"(d.w)
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(c.x), "f"(c.y), "f"(c.z),
              "f"(c.w));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%10, %11, %12, %13};"
            : "=f"(d.x), "=f"(d.y), "=f"(d.z), "=f"(d.w)
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(c.x), "f"(c.y), "f"(c.z),
              "f"(c.w));
    return d;
}

// pairs of fp32 in one 64-bit register
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
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
// (x, y) less the fp16 pair t
__device__ __forceinline__ float2 less_f16(float x, float y, uint32_t t) {
    float2 r;
    asm("{\n .reg .b16 l, h, m;\n mov.b32 {l, h}, %2;\n mov.b16 m, 0xbc00;\n"
        " fma.rn.f32.f16 %0, l, m, %3;\n fma.rn.f32.f16 %1, h, m, %4;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "r"(t), "f"(x), "f"(y));
    return r;
}
// A pair of fp32 values as 16-bit terms whose sum they are: two of fp16 (22
// bits), three of bf16 (24 bits).
template <bool BF>
__device__ __forceinline__ void split(float x, float y, uint32_t (&t)[3]) {
    if constexpr (BF) {
        t[0] = pack_bf16(x, y);
        const float rx = x - __uint_as_float(t[0] << 16), ry = y - __uint_as_float(t[0] & 0xffff0000u);
        t[1] = pack_bf16(rx, ry);
        t[2] = pack_bf16(rx - __uint_as_float(t[1] << 16), ry - __uint_as_float(t[1] & 0xffff0000u));
    } else {
        t[0] = pack_f16(x, y);
        const float2 r = less_f16(x, y, t[0]);
        t[1] = pack_f16(r.x, r.y);
        t[2] = 0;
    }
}

// Whether the phase with this parity has completed (no waiting).
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
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
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// a b - c
__device__ __forceinline__ uint32_t hfms2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("{\n .reg .b32 n;\n neg.f16x2 n, %3;\n fma.rn.f16x2 %0, %1, %2, n;\n}"
        : "=r"(r)
        : "r"(a), "r"(b), "r"(c));
    return r;
}
// A value that the compiler takes for a variable: constants that every
// fragment needs stay in registers instead of being moved there each time
// (with one immediate per instruction, permutes and masks need them there).
__device__ __forceinline__ uint32_t held(uint32_t v) {
    uint32_t r;
    asm volatile("mov.b32 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// Two bytes of w (two's complement, bit 7 already flipped) as an exact fp16
// pair: 1024 + 128 + code, less 1152. k0: 0x64646464.
template <int SEL>
__device__ __forceinline__ uint32_t bytes_f16(uint32_t w, uint32_t k0) {
    return hsub2(prmt(w, k0, SEL), 0x64806480u);
}
// The two nibbles that sit at bits SH and SH + 16 of w (SH 0 or 4), less 8, as
// an exact fp16 pair: 1024 + n - 1032, or (1024 + 16 n) / 16 - 72. k0:
// 0x64006400, k1: 1/16 twice.
template <int SH>
__device__ __forceinline__ uint32_t nibbles_f16(uint32_t w, uint32_t k0, uint32_t k1) {
    uint32_t r;  // (w & mask) | k0
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(w), "n"(SH == 0 ? 0x000f000f : 0x00f000f0), "r"(k0));
    if constexpr (SH == 0) return hsub2(r, 0x64086408u);
    else return hfma2(r, k1, 0xd480d480u);
}

__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
// four 8 x 8 tiles of 16-bit values, transposed; each lane gives a row's address
__device__ __forceinline__ uint4 ldsm_trans(uint32_t a) {
    uint4 v;
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a));
    return v;
}

template <bool V>
struct Flag {
    static constexpr bool value = V;
};
// Which of the positions at and at + 1 are seen, as a mask of 16-bit halves.
__device__ __forceinline__ uint32_t seen_pair(const Range &r, int at) {
    return (at >= r.lo && at < r.hi ? 0xffffu : 0u) |
           (at + 1 >= r.lo && at + 1 < r.hi ? 0xffff0000u : 0u);
}
// Whether one of eight 16-bit values is Inf or NaN.
template <bool BF>
__device__ __forceinline__ bool not_finite(const uint4 &v) {
    constexpr uint32_t e = BF ? 0x7f807f80u : 0x7c007c00u;
    return (__vcmpeq2(v.x & e, e) | __vcmpeq2(v.y & e, e) | __vcmpeq2(v.z & e, e) |
            __vcmpeq2(v.w & e, e)) != 0;
}

// ------------------------------------------------------------- fragments ----
// Lane 4 g + j of a warp.

// B fragments of K from plane p of a strip: one or two steps of 16 dims, two
// registers each. `row`: the lane's position (g, or 8 + g) times the row bytes
// plus its bytes in the row. The dims of lane j: 16-bit: 4 j + {0, 1 | 2, 3};
// Q8_0, step k: 8 j + 4 k + {0, 1 | 2, 3}; Q4_0, step k: 8 j + 2 k + {0, 4 | 1, 5}.
template <int F>
__device__ __forceinline__ void k_frag(uint32_t base, int p, uint32_t row, uint32_t k0, uint32_t k1,
                                       uint32_t (&b)[4]) {
    if constexpr (!kv_quantised(F)) {
        const uint2 w = lds64(base + p * 512 + row);
        b[0] = w.x;
        b[1] = w.y;
    } else if constexpr (F == F_Q8_0) {
        uint2 w = lds64(base + p * 512 + row);
        w.x ^= 0x80808080u;
        w.y ^= 0x80808080u;
        b[0] = bytes_f16<0x4140>(w.x, k0);
        b[1] = bytes_f16<0x4342>(w.x, k0);
        b[2] = bytes_f16<0x4140>(w.y, k0);
        b[3] = bytes_f16<0x4342>(w.y, k0);
    } else {
        const uint32_t w = lds32(base + p * 256 + row), v = w >> 8;
        b[0] = nibbles_f16<0>(w, k0, k1);
        b[1] = nibbles_f16<4>(w, k0, k1);
        b[2] = nibbles_f16<0>(v, k0, k1);
        b[3] = nibbles_f16<4>(v, k0, k1);
    }
}

// A fragments of V^T from plane p: rows are dims, columns positions. 16-bit:
// one tile, rows g and g + 8 are dims 16 p + g and 16 p + 8 + g (`row` is the
// lane's ldmatrix row). Quantised: two tiles, rows g and g + 8 of tile u are
// dims 32 p + 4 g + 2 u and + 1; `row` is the byte offset of position 2 j and
// dims 4 g.
template <int F>
__device__ __forceinline__ void v_frag(uint32_t base, int p, uint32_t row, uint32_t k0, uint32_t k1,
                                       uint4 (&a)[2]) {
    if constexpr (!kv_quantised(F)) {
        a[0] = ldsm_trans(base + p * 512 + row);
    } else if constexpr (F == F_Q8_0) {
        uint32_t lo[2], hi[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint32_t w0 = lds32(base + p * 512 + row + x * 256) ^ 0x80808080u;
            const uint32_t w1 = lds32(base + p * 512 + row + x * 256 + 32) ^ 0x80808080u;
            lo[x] = prmt(w0, w1, 0x5140);
            hi[x] = prmt(w0, w1, 0x7362);
        }
        a[0] = make_uint4(bytes_f16<0x4140>(lo[0], k0), bytes_f16<0x4342>(lo[0], k0),
                          bytes_f16<0x4140>(lo[1], k0), bytes_f16<0x4342>(lo[1], k0));
        a[1] = make_uint4(bytes_f16<0x4140>(hi[0], k0), bytes_f16<0x4342>(hi[0], k0),
                          bytes_f16<0x4140>(hi[1], k0), bytes_f16<0x4342>(hi[1], k0));
    } else {
        uint32_t w[2], v[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            w[x] = prmt(lds16(base + p * 256 + row + x * 128), lds16(base + p * 256 + row + x * 128 + 16),
                        0x5410);
            v[x] = w[x] >> 8;
        }
        a[0] = make_uint4(nibbles_f16<0>(w[0], k0, k1), nibbles_f16<4>(w[0], k0, k1),
                          nibbles_f16<0>(w[1], k0, k1), nibbles_f16<4>(w[1], k0, k1));
        a[1] = make_uint4(nibbles_f16<0>(v[0], k0, k1), nibbles_f16<4>(v[0], k0, k1),
                          nibbles_f16<0>(v[1], k0, k1), nibbles_f16<4>(v[1], k0, k1));
    }
}

// ------------------------------------------------------- spans of V scales ----
// f16 scales up to the binade `top` (a biased exponent, 1 to 30) fall into spans
// of 11 binades: span 0 is top and the ten below it (and Inf and NaN), span 1 the
// next eleven, span 2 the rest.

// The spans of a pair of scales, as bits; a scale of 0 is in none.
__device__ __forceinline__ uint32_t spans_of(uint32_t d, int top) {
    uint32_t spans = 0;
#pragma unroll
    for (int e = 0; e < 32; e += 16) {
        const uint32_t one = d >> e & 0x7fffu;
        if (one) spans |= 1u << max(0, top - (int)(one >> 10)) / 11;
    }
    return spans;
}
// A pair of scales: 0 for one that is not in `span`.
__device__ __forceinline__ uint32_t in_span(uint32_t d, int top, int span) {
    const uint32_t from = max(1, (top - 11 * span - 10) << 10), to = span ? ((top - 11 * span + 1) << 10) - 1 : 0x7fff;
    const uint32_t size = d & 0x7fff7fffu;
    return d & __vcmpgeu2(size, from * 0x10001u) & __vcmpleu2(size, to * 0x10001u);
}
// 2^e (-16 <= e <= 15) as an fp16 pair
__device__ __forceinline__ uint32_t power_f16(int e) {
    return (e < -14 ? 1u << (e + 24) : (uint32_t)(e + 15) << 10) * 0x10001u;
}

// ----------------------------------------------------------------- config ----

template <int FK, int FV, int D>
struct Cfg {
    static constexpr Shape kShape = shape_of(FK, FV, D);
    static constexpr int kUnits = kShape.units, kSlots = kShape.slots, kSlotBytes = kShape.slot_bytes;
    static constexpr int kBytesK = kv_half_bytes(FK, D), kBytesV = kv_half_bytes(FV, D);
    static constexpr int kSteps = D / 16;
    static constexpr int kStep = kShape.step, kGroups = kSlots / kStep;
    static constexpr int kQBytes = kShape.q_bytes;
    static constexpr int kRingBytes = kShape.ring_bytes;
    static constexpr int kMergeRow = D + 4;  // floats; + 4 spreads the rows j over the banks
    static constexpr int kSmem = kShape.smem;
    static_assert(kSlots % kStep == 0 && kGroups >= 2 && kSlots <= kMaxSlots, "a ring holds two runs");
    static_assert(kWarps * kMaxSlots * 12 + kRows * 12 + kWarps * kRows * 8 + sizeof(WorkSearch) <= kFixedBytes,
                  "fixed part of shared memory");
    static_assert(kShape.ctas * (kSmem + 1024) <= 228 * 1024, "shared memory of an SM");
    static_assert(kSlotBytes % 16 == 0 && kBytesK % 16 == 0 && kRingBytes % 16 == 0 && kQBytes % 16 == 0,
                  "alignment");
};

// ---------------------------------------------------------------- kernel ----

template <int FK, int FV, int D, bool MANY>
__global__ void __launch_bounds__(kThreads, Cfg<FK, FV, D>::kShape.ctas)
    attend_kernel(const AttendParams a) {
    using C = Cfg<FK, FV, D>;
    constexpr bool kBfK = FK == F_BF16, kBfV = FV == F_BF16;
    constexpr int kPlanesK = D / kv_plane_dims(FK), kPlanesV = D / kv_plane_dims(FV);
    // planes of 16-bit K that are summed by the tensor cores, which cut rather
    // than round, before they are added to a score in fp32: with 4 (64 dims)
    // outputs of 128 F16 dims are off by 5.0e-7 of their norm and of 256 BF16 dims
    // by 5.7e-7, with all planes 7.9e-7 and 15e-7; the shorter chains also take
    // 44.4 instead of 47.6 us for 3 positions over 8 BF16 sequences of 16000
    constexpr int kSumPlanes = 4;
    constexpr int kStepsPerPlane = kv_plane_dims(FK) / 16;  // 2 for quantised K
    constexpr int kTilesPerPlane = kv_plane_dims(FV) / 16;  // 2 for quantised V
    // the weights' limit, and the f16 patterns of the smallest and the largest of
    // V's scales that do without a lift (see the top of the file)
    constexpr float kLim = kBfV ? -12.0f : FV == F_Q4_0 ? 12.0f : 15.0f;
    constexpr uint32_t kLeast = FV == F_Q4_0 ? 7 << 10 : 4 << 10, kMost = kLeast + (11 << 10) - 1;
    constexpr int S = C::kStep;                             // strips taken at a time
    extern __shared__ __align__(128) uint8_t smem[];
    // fixed part: barriers, flags, row scales, softmax states, work search
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem);                      // [kWarps][kMaxSlots]
    uint32_t *landed = reinterpret_cast<uint32_t *>(smem + kWarps * 64);      // [kWarps][kMaxSlots]
    float *row_scale = reinterpret_cast<float *>(smem + kWarps * 96);         // [kRows]
    float *state_m = row_scale + kRows;                                       // [kWarps][kRows]
    float *state_l = state_m + kWarps * kRows;                                // [kWarps][kRows]
    Range *seen = reinterpret_cast<Range *>(state_l + kWarps * kRows);        // [kRows]
    WorkSearch *search = reinterpret_cast<WorkSearch *>(seen + kRows);
    uint8_t *q_frag = smem + kFixedBytes;
    const KvView &c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, j = lane & 3;
    const uint32_t bar0 = smem_addr(bars + warp * kMaxSlots);
    uint8_t *ring_ptr = q_frag + C::kQBytes + warp * C::kRingBytes;
    const uint32_t ring = smem_addr(ring_ptr), qf = smem_addr(q_frag);
    if (lane == 0) {
        for (int i = 0; i < C::kGroups; ++i) mbar_init(bar0 + 8 * i, 1);
        fence_barrier_init();
    }
    pdl_wait_prev();

    Work w;
    if (!find_work<MANY>(a, (int)blockIdx.x, search, w)) {
        if (threadIdx.x == 0 && !a.whole) a.joins[blockIdx.x].parts = 0;
        return;
    }
    Join next_join;
    next_join.parts = 0;

    const uint32_t k_row = g * kv_row_bytes(FK) + j * (FK == F_Q4_0 ? 4 : 8);
    const uint32_t v_row = kv_quantised(FV) ? 2 * j * kv_row_bytes(FV) + g * (FV == F_Q4_0 ? 2 : 4)
                                            : ((lane & 7) + (lane >> 4) * 8) * 32 + ((lane >> 3) & 1) * 16;

    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    const uint32_t kk0 = FK == F_Q8_0 ? held(0x64646464u) : FK == F_Q4_0 ? held(0x64006400u) : 0;
    const uint32_t vk0 = FV == FK ? kk0 : FV == F_Q4_0 ? held(0x64006400u) : 0;
    const uint32_t vk1 = FV == F_Q4_0 ? held(0x2c002c00u) : 0, kk1 = FK == F_Q4_0 ? vk1 : 0;

    // Ring of this warp, over the whole launch: groups of S slots (the strips
    // of a run, or their K or V halves) with one barrier each; the next group
    // to be filled and to be taken, and the phase of the latter.
    int fill = 0, take = 0, flying = 0;
    uint32_t phase = 0;
    bool dead = false;
    Item it;
    while (next_item<MANY>(a, w, it)) {
        if (!it.live) {
            for (int i = threadIdx.x; i < kRows * D / 4; i += kThreads) {
                const int row = i / (D / 4);
                put_out<MANY>(a, it, row, (i - row * (D / 4)) * 4, D, zero, 0.0f);
            }
            continue;
        }
        // ---- query rows on their way (before the page table's entries are waited for) ----
        const int q_row = threadIdx.x >> 4, q_part = threadIdx.x & 15;
        float x[(D + 127) / 128][8];
        {
            int64_t q_at;
            const bool there = row_offset<MANY>(a, it, q_row, D, a.q_stride, q_at);
            const float *q = a.q + q_at;
#pragma unroll
            for (int i = 0; i < (D + 127) / 128; ++i) {
                const int d = 8 * (q_part + 16 * i);
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
            }
        }

        // ---- copies of the first strips ----
        // The warps take runs of S strips in turn.
        const int runs = (it.end - it.begin + S - 1) / S;
        const int mine = !dead && runs > warp ? (runs - warp + kWarps - 1) / kWarps : 0;
        int left = mine * C::kUnits, strip = 0;  // groups to be issued; the next one's first strip
        bool half_v = false;
        const uint8_t *src = nullptr;            // of lane l: strip l of the current 32 of this warp
        uint32_t have = 0;                       // which of them exist
        int length = 1;                          // strips that this lane copies at once
        auto issue = [&]() {
            if ((strip & 31) == 0 && !half_v) {
                const int at = it.begin + S * warp + (strip + lane) / S * S * kWarps + lane % S;
                src = at < it.end ? kv_strip(c, it.seq, it.head, it.first + at) : nullptr;
                have = __ballot_sync(~0u, src != nullptr);
                if constexpr (C::kUnits == 1) {
                    // strips of a run that lie one after the other are one copy,
                    // made by the first one's lane
                    const uint64_t before = __shfl_up_sync(~0u, (uint64_t)src, 1);
                    const uint32_t joined = __ballot_sync(
                        ~0u, lane % S != 0 && src && (uint64_t)src == before + C::kSlotBytes);
                    const uint32_t after = joined >> lane >> 1;  // the strips that follow this one
                    length = joined >> lane & 1 ? 0 : __ffs(~after);
                }
            }
            const uint32_t bytes = C::kUnits == 1 ? C::kBytesK + C::kBytesV : half_v ? C::kBytesV : C::kBytesK;
            const uint32_t bar = bar0 + 8 * fill, t = lane - (strip & 31);
            const uint32_t these = (have >> (strip & 31)) & ((1u << S) - 1);
            if (t == 0) {
                landed[warp * kMaxSlots + fill] = these;
                mbar_arrive_expect_tx(bar, __popc(these) * bytes);
            }
            __syncwarp();
            if (t < S && src && length > 0)
                bulk_g2s(ring + (fill * S + t) * C::kSlotBytes, half_v ? src + C::kBytesK : src, length * bytes,
                         bar);
            if (C::kUnits == 1 || half_v) strip += S;
            if (C::kUnits == 2) half_v = !half_v;
            if (++fill == C::kGroups) fill = 0;
            ++flying;
            --left;
        };
        // waits for the next group; its index
        auto await = [&]() {
            const int group = take;
            if (!__all_sync(~0u, mbar_test(bar0 + 8 * group, phase)))
                if (__any_sync(~0u, !mbar_wait(bar0 + 8 * group, phase))) {
                    if (lane == 0) record_error(c.err, DERR_ATTEND);
                    dead = true;
                }
            if (++take == C::kGroups) {
                take = 0;
                phase ^= 1;
            }
            --flying;
            return group;
        };
        // the group last taken has been read by the whole warp: it is refilled
        auto refill = [&]() {
            fence_proxy_async_smem();
            __syncwarp();
            if (left > 0) issue();
        };
        while (left > 0 && flying < C::kGroups) issue();

        // ---- query rows as A fragments ----
        {
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < (D + 127) / 128; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(x[i][k]));
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
            if (q_part == 0) {
                row_scale[q_row] = a.scale_log2 * down;
                if (MANY) seen[q_row] = seen_from(a, it.pos0 + new_of<MANY>(a, it.tile * kRows + q_row));
            }
#pragma unroll
            for (int i = 0; i < (D + 127) / 128; ++i) {
                const int d = 8 * (q_part + 16 * i);
                if (d < D) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        // four dims: the step and lane that they belong to (see k_frag)
                        int step, jj;
                        float v0, v1, v2, v3;
                        if constexpr (FK == F_Q4_0) {
                            step = d / 32 * 2 + h;
                            jj = d % 32 / 8;
                            v0 = x[i][2 * h] * up; v1 = x[i][2 * h + 4] * up;
                            v2 = x[i][2 * h + 1] * up; v3 = x[i][2 * h + 5] * up;
                        } else {
                            step = FK == F_Q8_0 ? d / 32 * 2 + h : d / 16;
                            jj = FK == F_Q8_0 ? d % 32 / 8 : d % 16 / 4 + h;
                            v0 = x[i][4 * h] * up; v1 = x[i][4 * h + 1] * up;
                            v2 = x[i][4 * h + 2] * up; v3 = x[i][4 * h + 3] * up;
                        }
                        uint32_t s[3], t[3];
                        split<kBfK>(v0, v1, s);
                        split<kBfK>(v2, v3, t);
                        const int at = step * 32 + q_row * 4 + jj;
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
        // positions that all rows see (both ends of a row's range grow with the row)
        const int all_lo = MANY ? seen[kRows - 1].lo : it.lo, all_hi = MANY ? seen[0].hi : it.hi;
        uint64_t o[D / 16][2];  // [tile]: rows g and g + 8 (dims), columns 2 j and 2 j + 1 (query rows)
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = 0;
        // the reference of the row's weights and their total (of positions
        // 2 j and 2 j + 1 of the n-tiles)
        float ref = -FLT_MAX;
        uint64_t l = 0;
        for (int n = 0; n < mine; ++n) {
            const int first = (it.first + it.begin + S * (warp + kWarps * n)) * kStrip;
            int group = await();
            if (dead) break;
            const uint32_t sk = ring + group * S * C::kSlotBytes;
            const uint32_t here = landed[warp * kMaxSlots + group];
            const bool edge = first < all_lo || first + S * kStrip > all_hi || here != (1u << S) - 1;
            float s[S][2][2];  // [strip][n-tile][position 8 x + 2 j + e]
            // scores
            {
                float4 acc[S][2];
                uint64_t sum[S][2];
#pragma unroll
                for (int t = 0; t < S; ++t) sum[t][0] = sum[t][1] = 0;
#pragma unroll
                for (int p = 0; p < kPlanesK; ++p) {
                    uint32_t b[S][2][4];
#pragma unroll
                    for (int t = 0; t < S; ++t) {
                        k_frag<FK>(sk + t * C::kSlotBytes, p, k_row, kk0, kk1, b[t][0]);
                        k_frag<FK>(sk + t * C::kSlotBytes, p, k_row + 8 * kv_row_bytes(FK), kk0,
                                   kk1, b[t][1]);
                    }
                    if (kv_quantised(FK) || p % kSumPlanes == 0) {
#pragma unroll
                        for (int t = 0; t < S; ++t)
#pragma unroll
                            for (int x = 0; x < 2; ++x) acc[t][x] = zero;
                    }
#pragma unroll
                    for (int k = 0; k < kStepsPerPlane; ++k) {
                        const int step = p * kStepsPerPlane + k;
                        const uint4 q = lds128(qf + (step * 32 + lane) * 16);
#pragma unroll
                        for (int t = 0; t < S; ++t)
#pragma unroll
                            for (int x = 0; x < 2; ++x)
                                acc[t][x] = mma<kBfK>(q, b[t][x][2 * k], b[t][x][2 * k + 1], acc[t][x]);
                        if constexpr (kBfK) {
                            const uint2 r = lds64(qf + C::kSteps * 512 + (step * 32 + lane) * 8);
                            const uint4 q3 = make_uint4(r.x, 0, r.y, 0);
#pragma unroll
                            for (int t = 0; t < S; ++t)
#pragma unroll
                                for (int x = 0; x < 2; ++x)
                                    acc[t][x] = mma<kBfK>(q3, b[t][x][0], b[t][x][1], acc[t][x]);
                        }
                    }
                    if (kv_quantised(FK) || p % kSumPlanes == kSumPlanes - 1 || p == kPlanesK - 1) {
#pragma unroll
                        for (int t = 0; t < S; ++t)
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const uint64_t both = add2(pack_f2(acc[t][x].x, acc[t][x].y),
                                                           pack_f2(acc[t][x].z, acc[t][x].w));
                                if constexpr (kv_quantised(FK)) {
                                    const float2 d = unpack_f16(lds32(
                                        sk + t * C::kSlotBytes + kv_code_bytes(FK, D) + (p * kStrip + 8 * x + 2 * j) * 2));
                                    sum[t][x] = fma2(pack_f2(d.x, d.y), both, sum[t][x]);
                                } else {
                                    sum[t][x] = add2(sum[t][x], both);
                                }
                            }
                    }
                }
#pragma unroll
                for (int t = 0; t < S; ++t)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        // 0 times a sum that is not finite is NaN: a K value of Inf
                        // makes the row NaN whatever its sign, not by the signs of
                        // the query's terms
                        const uint64_t f = fma2(sum[t][x], pack_f2(0.0f, 0.0f), pack_f2(rs, rs));
                        const float2 v = unpack2(mul2(sum[t][x], f));
                        s[t][x][0] = v.x;
                        s[t][x][1] = v.y;
                    }
            }
            if constexpr (C::kUnits == 2) {
                refill();
                group = await();
                if (dead) break;
            }
            const uint32_t sv = ring + group * S * C::kSlotBytes + (C::kUnits == 1 ? C::kBytesK : 0);
            // Positions that a row does not see: its scores are dropped, and since
            // weights of 0 must not meet an Inf or NaN, what no row sees of V (of
            // its scales) is cleared. Where a value (a scale) that only some rows
            // see is not finite, the others' products are kept apart.
            bool apart = false;
            if (edge) {
                const int any_lo = MANY ? seen[0].lo : it.lo, any_hi = MANY ? seen[kRows - 1].hi : it.hi;
                const Range sees = MANY ? seen[g] : Range{it.lo, it.hi};
#pragma unroll
                for (int t = 0; t < S; ++t) {
                    const int from = first + t * kStrip;
                    const bool there = here >> t & 1;
                    const int lo = sees.lo - from, hi = there ? sees.hi - from : 0;
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int at = 8 * x + 2 * j + e;
                            if (at < lo || at >= hi) s[t][x][e] = -INFINITY;
                        }
                    uint8_t *v = ring_ptr + (sv - ring) + t * C::kSlotBytes;
                    auto nobody = [&](int at) { return !there || at < any_lo || at >= any_hi; };
                    auto somebody = [&](int at) { return at < all_lo || at >= all_hi; };
                    if constexpr (kv_quantised(FV)) {
                        uint16_t *d = reinterpret_cast<uint16_t *>(v + kv_code_bytes(FV, D));
                        for (int i = lane; i < D / 2; i += 32) {
                            const int at = from + (i & 15);
                            if (nobody(at)) d[i] = 0x3800u;  // 1/2; its weight is 0
                            else if (MANY && somebody(at) && (d[i] & 0x7c00u) == 0x7c00u) apart = true;
                        }
                    } else {
                        for (int i = lane; i < 2 * D; i += 32) {
                            const int at = from + ((i >> 1) & 15);
                            uint4 *to = reinterpret_cast<uint4 *>(v + i * 16);
                            if (nobody(at)) *to = make_uint4(0, 0, 0, 0);
                            else if (MANY && somebody(at) && not_finite<kBfV>(*to)) apart = true;
                        }
                    }
                }
                if (MANY) apart = __any_sync(~0u, apart);
                __syncwarp();
            }

            // limits of the weights
            float mx = s[0][0][0];
#pragma unroll
            for (int i = 1; i < 4 * S; ++i) mx = fmaxf(mx, s[i >> 2][(i >> 1) & 1][i & 1]);
            bool over = mx - ref > kLim, far = false;
            uint32_t dv[S][kv_quantised(FV) ? kPlanesV : 1][2];  // V's scales
            auto scales = [&](int t, int p, int x) {  // of positions 8 x + 2 j and + 1
                return lds32(sv + t * C::kSlotBytes + kv_code_bytes(FV, D) + (p * kStrip + 8 * x + 2 * j) * 2);
            };
            // for the limits each lane looks at a few of them, two at a time
            constexpr int kWords = kPlanesV * 8, kLook = (S * kWords + 31) / 32;
            auto look = [&](int i) {
                const int at = min(lane + 32 * i, S * kWords - 1), t = at / kWords;
                return lds32(sv + t * C::kSlotBytes + kv_code_bytes(FV, D) + (at - t * kWords) * 4);
            };
            if constexpr (kv_quantised(FV)) {
                uint32_t big = 0, small = ~0u;
#pragma unroll
                for (int i = 0; i < kLook; ++i) {
                    // Q8_0's scales have no sign
                    const uint32_t d = look(i) & (FV == F_Q8_0 ? ~0u : 0x7fff7fffu);
                    big = __vmaxu2(big, d);
                    small = __vminu2(small, d);
                }
                far = max(big & 0xffffu, big >> 16) > kMost || min(small & 0xffffu, small >> 16) < kLeast;
#pragma unroll
                for (int t = 0; t < S; ++t)
#pragma unroll
                    for (int p = 0; p < kPlanesV; ++p)
#pragma unroll
                        for (int x = 0; x < 2; ++x) dv[t][p][x] = scales(t, p, x);
            }
            uint32_t spans = 0;  // that V's scales fall into, where they need lifts; from bit 8 on: top
            if (__any_sync(~0u, over || far)) {
                if constexpr (kv_quantised(FV)) {
                    if (__any_sync(~0u, far)) {
                        uint32_t all = 0;
#pragma unroll
                        for (int i = 0; i < kLook; ++i) all = __vmaxu2(all, look(i) & 0x7fff7fffu);
                        int top = (int)__reduce_max_sync(~0u, max(all & 0xffffu, all >> 16)) >> 10;
                        top = max(1, min(30, top));
#pragma unroll
                        for (int i = 0; i < kLook; ++i) spans |= spans_of(look(i), top);
                        spans = __reduce_or_sync(~0u, spans);
                        if (spans) spans |= (uint32_t)top << 8;
                    }
                }
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2));
                const float r = mx - ref > kLim ? mx - (kLim - 4.0f) : ref;
                const float f = exp2_fast(ref - r);
                ref = r;
                l = mul2(l, pack_f2(f, f));
                const uint64_t ff = pack_f2(__shfl_sync(~0u, f, 8 * j), __shfl_sync(~0u, f, 8 * j + 4));
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    o[i][0] = mul2(o[i][0], ff);
                    o[i][1] = mul2(o[i][1], ff);
                }
            }

            // weights, as the terms of n-tiles 0 and 1
            uint32_t w0[S][3], w1[S][3];
            const uint64_t less = pack_f2(-ref, -ref);
#pragma unroll
            for (int t = 0; t < S; ++t) {
                float2 x0 = unpack2(add2(pack_f2(s[t][0][0], s[t][0][1]), less));
                float2 x1 = unpack2(add2(pack_f2(s[t][1][0], s[t][1][1]), less));
                x0 = make_float2(exp2_fast(x0.x), exp2_fast(x0.y));
                x1 = make_float2(exp2_fast(x1.x), exp2_fast(x1.y));
                l = add2(l, add2(pack_f2(x0.x, x0.y), pack_f2(x1.x, x1.y)));
                split<kBfV>(x0.x, x0.y, w0[t]);
                split<kBfV>(x1.x, x1.y, w1[t]);
            }
            // weighted sum of V, `down`: without the scales' lift
            uint64_t down = pack_f2(1.0f, 1.0f);
            auto weigh = [&](auto by_row) {
#pragma unroll
                for (int p = 0; p < kPlanesV; ++p) {
                    // products with the weights' low terms have sums of their own
                    // where unpacking is what takes time (shorter chains: 48
                    // ragged Q4_0 sequences 62.7 us, 64.2 in one sum)
                    float4 acc[2] = {zero, zero}, low[2] = {zero, zero};
#pragma unroll
                    for (int t = 0; t < S; ++t) {
                        uint32_t b0[3], b1[3];
                        if constexpr (kv_quantised(FV)) {
                            const uint32_t d0 = dv[t][p][0], d1 = dv[t][p][1];
                            b0[0] = hmul2(w0[t][0], d0);
                            b1[0] = hmul2(w1[t][0], d1);
                            b0[1] = hfma2(w0[t][1], d0, hfms2(w0[t][0], d0, b0[0]));
                            b1[1] = hfma2(w1[t][1], d1, hfms2(w1[t][0], d1, b1[0]));
                        } else {
#pragma unroll
                            for (int k = 0; k < 3; ++k) {
                                b0[k] = w0[t][k];
                                b1[k] = w1[t][k];
                            }
                        }
                        uint4 v[2];
                        v_frag<FV>(sv + t * C::kSlotBytes, p, v_row, vk0, vk1, v);
                        auto product = [&](const uint4 &of, float4 &to, float4 &lo) {
                            if constexpr (kBfV) lo = mma<kBfV>(of, b0[2], b1[2], lo);
                            lo = mma<kBfV>(of, b0[1], b1[1], lo);
                            to = mma<kBfV>(of, b0[0], b1[0], to);
                        };
                        if constexpr (by_row.value && !kv_quantised(FV)) {
                            // columns 2 j and 2 j + 1 of the sum are rows: each
                            // is kept from the product with the V that it sees
#pragma unroll 1
                            for (int r = 0; r < kRows; ++r) {
                                const int at = first + t * kStrip + 2 * j;
                                const uint32_t m0 = seen_pair(seen[r], at), m1 = seen_pair(seen[r], at + 8);
                                float4 x = acc[0];
                                product(make_uint4(v[0].x & m0, v[0].y & m0, v[0].z & m1, v[0].w & m1), x, x);
                                if (r == 2 * j) acc[0].x = x.x, acc[0].z = x.z;
                                if (r == 2 * j + 1) acc[0].y = x.y, acc[0].w = x.w;
                            }
                        } else {
#pragma unroll
                            for (int u = 0; u < kTilesPerPlane; ++u)
                                product(v[u], acc[u], kv_quantised(FV) ? low[u] : acc[u]);
                        }
                    }
#pragma unroll
                    for (int u = 0; u < kTilesPerPlane; ++u) {
                        uint64_t(&to)[2] = o[p * kTilesPerPlane + u];
                        if constexpr (kv_quantised(FV) && !by_row.value) {
                            to[0] = add2(to[0], pack_f2(acc[u].x, acc[u].y));
                            to[1] = add2(to[1], pack_f2(acc[u].z, acc[u].w));
                            to[0] = add2(to[0], pack_f2(low[u].x, low[u].y));
                            to[1] = add2(to[1], pack_f2(low[u].z, low[u].w));
                        } else if constexpr (kv_quantised(FV)) {
                            to[0] = fma2(pack_f2(acc[u].x, acc[u].y), down, to[0]);
                            to[1] = fma2(pack_f2(acc[u].z, acc[u].w), down, to[1]);
                            to[0] = fma2(pack_f2(low[u].x, low[u].y), down, to[0]);
                            to[1] = fma2(pack_f2(low[u].z, low[u].w), down, to[1]);
                        } else {
                            to[0] = add2(to[0], pack_f2(acc[u].x, acc[u].y));
                            to[1] = add2(to[1], pack_f2(acc[u].z, acc[u].w));
                        }
                    }
                }
            };
            if constexpr (MANY && !kv_quantised(FV)) {
                if (apart) weigh(Flag<true>());
                else weigh(Flag<false>());
            } else if constexpr (kv_quantised(FV)) {
                if (__builtin_expect(!spans, 1)) {
                    weigh(Flag<false>());
                } else {
                    const bool some = (MANY && apart) || (spans & (spans - 1) & 7u) != 0;
                    const int top = (int)(spans >> 8);
                    spans &= 7u;
                    do {  // the next span's scales, lifted
                        const int span = __ffs(spans) - 1, lift = min(15, (int)(kMost >> 10) - top + 11 * span);
                        const uint32_t up = power_f16(lift);
                        const float d = __uint_as_float((uint32_t)(127 - lift) << 23);
                        down = pack_f2(d, d);
                        spans &= spans - 1;
#pragma unroll
                        for (int t = 0; t < S; ++t)
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const uint32_t m =
                                    MANY && apart ? seen_pair(seen[g], first + t * kStrip + 8 * x + 2 * j) : ~0u;
#pragma unroll
                                for (int p = 0; p < kPlanesV; ++p) {
                                    dv[t][p][x] = scales(t, p, x);
                                    if (some) dv[t][p][x] = m & in_span(dv[t][p][x], top, span);
                                    dv[t][p][x] = hmul2(dv[t][p][x], up);
                                }
                            }
                        weigh(Flag<true>());
                    } while (spans);
                }
            } else {
                weigh(Flag<false>());
            }
            refill();
        }
        // after an expired wait nothing more is issued; copies in flight land
        // (or their waits expire too) before the block ends
        while (dead && flying > 0) await();

        // ---- the warps' results joined ----
        const float2 l2 = unpack2(l);
        float total_l = l2.x + l2.y;
        total_l += __shfl_xor_sync(~0u, total_l, 1);
        total_l += __shfl_xor_sync(~0u, total_l, 2);
        if (j == 0) {
            // -Inf: saw nothing (a NaN score moves no reference, but makes the total NaN)
            state_m[warp * kRows + g] = ref == -FLT_MAX && total_l == 0.0f ? -INFINITY : ref;
            state_l[warp * kRows + g] = total_l;
        }
        float *merge = reinterpret_cast<float *>(ring_ptr);  // this warp's ring, all of it taken
        if (mine > 0) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const float2 even = unpack2(o[i][0]), odd = unpack2(o[i][1]);
                float *r0 = merge + 2 * j * C::kMergeRow, *r1 = r0 + C::kMergeRow;
                if constexpr (kv_quantised(FV)) {
                    const int d = 32 * (i / 2) + 4 * g + 2 * (i & 1);
                    *reinterpret_cast<float2 *>(r0 + d) = make_float2(even.x, odd.x);
                    *reinterpret_cast<float2 *>(r1 + d) = make_float2(even.y, odd.y);
                } else {
                    r0[16 * i + g] = even.x;
                    r1[16 * i + g] = even.y;
                    r0[16 * i + 8 + g] = odd.x;
                    r1[16 * i + 8 + g] = odd.y;
                }
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
                if (mk == -INFINITY) continue;
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
                put_out<MANY>(a, it, row, d, D, sum, total);
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
    if (threadIdx.x == 0 && !a.whole) a.joins[blockIdx.x] = next_join;
    pdl_launch_dependents();
}

template <int FK, int FV, int D, bool MANY>
cudaError_t launch_one(const AttendParams &a, int grid, cudaStream_t s) {
    using C = Cfg<FK, FV, D>;
    static OncePerDevice once;
    const cudaError_t ready = allow_smem(once, attend_kernel<FK, FV, D, MANY>, C::kSmem);
    if (ready != cudaSuccess) return ready;
    return launch_programmatic(attend_kernel<FK, FV, D, MANY>, a, grid, kThreads, C::kSmem, s);
}

// One new position per sequence (decoding) has a kernel without the rows'
// separate ranges: 48 ragged Q8_0 sequences take 62.8 us with it and 64.8
// without, 16 Q4_0 ones with 16 kv heads of 64 dims (two strips at a time) 50.0
// and 51.5.
template <int FK, int FV, int D>
cudaError_t launch_dim(const AttendParams &a, int grid, cudaStream_t s) {
    return a.n_new == 1 ? launch_one<FK, FV, D, false>(a, grid, s) : launch_one<FK, FV, D, true>(a, grid, s);
}

template <int FK, int FV>
cudaError_t launch_format(const AttendParams &a, int grid, cudaStream_t s) {
    switch (a.c.dim) {
    case 64: return launch_dim<FK, FV, 64>(a, grid, s);
    case 96: return launch_dim<FK, FV, 96>(a, grid, s);
    case 128: return launch_dim<FK, FV, 128>(a, grid, s);
    case 192: return launch_dim<FK, FV, 192>(a, grid, s);
    case 256: return launch_dim<FK, FV, 256>(a, grid, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace attend

}  // namespace qmm
