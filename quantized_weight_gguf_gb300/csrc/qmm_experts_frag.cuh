// qmm_experts_frag.cuh -- packed weights as operands of mma.sync m16n8k16, for
// the experts' feed-forward kernels.
//
// A warp multiplies 16 rows of W (the A operand) by 8 activation rows (B). The
// tensor cores see the integer codes, which 16 bits hold exactly; block scales
// multiply the sums of a block in fp32. An fp32 activation enters as two fp16
// terms under a power of two per 32 values (22 bits of it; three bf16 terms,
// all 24 bits, against BF16 weights), so every product is exact and the result
// is as good as an fp32 dot.
//
// The order of the 32 values of a block inside the two 16-deep steps is free
// as long as both operands share it (order_of): it is chosen so that lane (g, t) of
// the fragment (g = lane / 4, t = lane % 4) finds its eight values of row g in few words and
// few operations leave them in pairs.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qmm_device.cuh"

namespace qmm {
namespace experts {

// 16-bit terms of an activation; bytes of a block of 32 of them (see put_terms).
__host__ __device__ constexpr int terms_of(int fmt) { return fmt == F_BF16 ? 3 : 2; }
__host__ __device__ constexpr int frag_bytes(int fmt) { return 64 * terms_of(fmt); }

// Which elements of a block lane t takes, in the order of its operand registers
// (two pairs for the first step, two for the second):
//   kCodes:  4t, 4t+2 | 4t+1, 4t+3 | 16+4t, 16+4t+2 | 16+4t+1, 16+4t+3 -- what masks of a
//            word of nibbles (low ones first) or of bytes leave
//   kHalves: 4t, 4t+1 | 4t+2, 4t+3 | 16+4t, 16+4t+1 | 16+4t+2, 16+4t+3 -- 16-bit values as they are
// Either way the first step holds elements 0 .. 15.
enum Order : int { kCodes, kHalves };
__host__ __device__ constexpr Order order_of(int fmt) {
    return fmt == F_BF16 || fmt == F_F16 ? kHalves : kCodes;
}
// Place (0..31, in units of one value) of element e of a block in a term's 64
// bytes: lane t's values lie at 8t .. 8t+7.
__host__ __device__ constexpr int place_of(int order, int e) {
    return (e & 15) / 4 * 8 + (e & 16) / 4 + (order == kHalves ? e & 3 : ((e & 1) << 1) + ((e & 2) >> 1));
}

// Weights of a row that are copied to shared memory at a time, and the bytes
// of such a chunk in the row. (K-quants: a super-block's header and one half of
// its codes for Q4_K, a whole super-block for Q6_K.)
__host__ __device__ constexpr int chunk_k(int fmt) {
    return fmt == F_Q6_K ? 256 : fmt == F_BF16 || fmt == F_F16 ? 64 : 128;
}
__host__ __device__ constexpr int chunk_bytes(int fmt) {
    return fmt == F_Q4_K ? 80 : chunk_k(fmt) / block_elems(fmt) * block_bytes(fmt);
}
// 16-byte pieces that cover a chunk (rows start at even addresses, or at
// multiples of 16 and chunks at multiples of 8), and the distance of rows in shared memory: an odd
// multiple of 16 bytes, so that the 8 rows of a fragment's word loads fall on different
// banks (of 32 bytes for the 16-bit formats' 8-byte loads).
__host__ __device__ constexpr int chunk_pieces(int fmt, bool even) {
    return fmt == F_BF16 || fmt == F_F16 ? (even ? 9 : 8) : fmt == F_Q4_K ? 5 : (chunk_bytes(fmt) + (even ? 14 : 8) + 15) / 16 | 1;
}
__host__ __device__ constexpr int row_pitch(int fmt, bool even) {
    return fmt == F_BF16 || fmt == F_F16 ? 160 : 16 * chunk_pieces(fmt, even);
}

// A fresh sum (c is written only), and one that goes on.
__device__ __forceinline__ void mma_f16_new(float (&c)[4], const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_bf16_new(float (&c)[4], const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ------------------------------------------------------------- loads ----

__device__ __forceinline__ uint32_t ld16(const uint8_t *p) {
    return *reinterpret_cast<const unsigned short *>(p);
}
__device__ __forceinline__ uint32_t ld32(const uint8_t *p) {
    return *reinterpret_cast<const uint32_t *>(p);
}
// A row's chunk in shared memory. EVEN: it starts at an even address, and words
// at offsets whose value mod 4 is known come from two aligned words and a
// permute whose selector is formed once per chunk; else it starts at a multiple of 8
// bytes, and words at offsets 0 mod 4 are read as they are.
template <bool EVEN>
struct RowAt {
    const uint8_t *p;       // the chunk
    const uint8_t *a0, *a2; // EVEN: aligned addresses for offsets that are 0 and 2 mod 4
    uint32_t sel0;          // EVEN: selector for offsets 0 mod 4; 2 mod 4 takes the other one
    __device__ __forceinline__ void set(const uint8_t *chunk, uint32_t odd) {  // odd: 0 or 2
        p = chunk;
        if (EVEN) {
            a0 = chunk - odd;
            a2 = chunk + odd - 2;
            sel0 = odd ? 0x5432u : 0x3210u;
        }
    }
    // the word at offset `at` + `lane`, `at` even and known when compiled, `lane` a multiple of 4
    __device__ __forceinline__ uint32_t word(int at, int lane) const {
        if (!EVEN && (at & 2) == 0) return ld32(p + at + lane);
        const uint8_t *q = (EVEN ? (at & 2) ? a2 : a0 : p - 2) + at + lane;
        return prmt(ld32(q), ld32(q + 4), !EVEN ? 0x5432u : (at & 2) ? sel0 ^ 0x6622u : sel0);
    }
    __device__ __forceinline__ float f16(int at) const { return f16_bits_to_f32(ld16(p + at)); }
};

// ------------------------------------------------------------ decode ----

__device__ __forceinline__ uint32_t sub2(uint32_t x, uint32_t y) {
    const __half2 r = __hsub2(*reinterpret_cast<__half2 *>(&x), *reinterpret_cast<__half2 *>(&y));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t fma2(uint32_t x, uint32_t y, uint32_t z) {
    const __half2 r = __hfma2(*reinterpret_cast<__half2 *>(&x), *reinterpret_cast<__half2 *>(&y),
                              *reinterpret_cast<__half2 *>(&z));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__host__ __device__ constexpr uint32_t twice(uint32_t h) { return h | (h << 16); }
// fp16 patterns: 1024 + z, and the constants that take 1024 + 16 q to q - z
__host__ __device__ constexpr uint32_t h1024(uint32_t z) { return 0x6400u + z; }
__host__ __device__ constexpr uint32_t neg64(uint32_t z) { return 0xD400u + 16 * z; }  // -(64 + z), z < 64

// Low (high) nibbles of a word's bytes 0, 2 and 1, 3, less Z, as fp16 pairs: a
// nibble under the exponent of 1024 is 1024 + q (1024 + 16 q), exact.
template <int Z>
__device__ __forceinline__ void low_nibbles(uint32_t w, uint32_t &r0, uint32_t &r1) {
    r0 = sub2((w & 0x000F000Fu) | 0x64006400u, twice(h1024(Z)));
    r1 = sub2(((w >> 8) & 0x000F000Fu) | 0x64006400u, twice(h1024(Z)));
}
template <int Z>
__device__ __forceinline__ void high_nibbles(uint32_t w, uint32_t &r0, uint32_t &r1) {
    r0 = fma2((w & 0x00F000F0u) | 0x64006400u, twice(0x2C00u), twice(neg64(Z)));
    r1 = fma2(((w >> 8) & 0x00F000F0u) | 0x64006400u, twice(0x2C00u), twice(neg64(Z)));
}
// bytes 0, 2 and 1, 3 of a word, less Z (at most 255 - Z in size)
template <int Z>
__device__ __forceinline__ void bytes(uint32_t w, uint32_t &r0, uint32_t &r1) {
    r0 = sub2(prmt(w, 0x64646464u, 0x4240u), twice(h1024(Z)));
    r1 = sub2(prmt(w, 0x64646464u, 0x4341u), twice(h1024(Z)));
}

// signed bytes 0, 2 and 1, 3: the sign bit turned over makes them 128 + q
__device__ __forceinline__ void signed_bytes(uint32_t w, uint32_t &r0, uint32_t &r1) {
    r0 = sub2((w & 0x00FF00FFu) ^ 0x64806480u, twice(h1024(128)));
    r1 = sub2(((w >> 8) & 0x00FF00FFu) ^ 0x64806480u, twice(h1024(128)));
}

// A row's share of a group of blocks of 32: load() takes the codes from the
// row's chunk in shared memory, pairs(sub) gives block `sub` of the group as
// four operand registers of lane t, and the scales follow. kGroup: blocks that
// share loads. kScales: scales per block (2: one for each 16-deep step);
// kMin: a term that multiplies the sum of the activations is added.
template <int FMT>
struct Row;

template <>
struct Row<F_Q4_0> {
    static constexpr int kGroup = 1, kScales = 1;
    static constexpr bool kMin = false;
    uint32_t w;
    float d;
    template <bool EVEN>
    __device__ __forceinline__ void load(const RowAt<EVEN> &row, int group, int, int t) {
        d = row.f16(18 * group);
        w = row.word(18 * group + 2, 4 * t);
    }
    __device__ __forceinline__ void pairs(int, uint32_t (&r)[4]) const {
        low_nibbles<8>(w, r[0], r[1]);
        high_nibbles<8>(w, r[2], r[3]);
    }
    __device__ __forceinline__ float scale(int, int) const { return d; }
    __device__ __forceinline__ float min(int) const { return 0.0f; }
};

template <>
struct Row<F_Q5_0> {
    static constexpr int kGroup = 1, kScales = 1;
    static constexpr bool kMin = false;
    uint32_t w, high;  // nibbles; the fifth bits of elements 4t .. 4t+3 (0..3) and 16+4t .. (16..19)
    float d;
    template <bool EVEN>
    __device__ __forceinline__ void load(const RowAt<EVEN> &row, int group, int, int t) {
        d = row.f16(22 * group);
        high = row.word(22 * group + 2, 0) >> (4 * t);
        w = row.word(22 * group + 6, 4 * t);
    }
    // bits 0..3 to bit 4 of bytes 0..3
    static __device__ __forceinline__ uint32_t spread(uint32_t b) {
        return (((b & 15u) * 0x00204081u) & 0x01010101u) << 4;
    }
    __device__ __forceinline__ void pairs(int, uint32_t (&r)[4]) const {
        bytes<16>((w & 0x0F0F0F0Fu) | spread(high), r[0], r[1]);
        bytes<16>(((w >> 4) & 0x0F0F0F0Fu) | spread(high >> 16), r[2], r[3]);
    }
    __device__ __forceinline__ float scale(int, int) const { return d; }
    __device__ __forceinline__ float min(int) const { return 0.0f; }
};

template <>
struct Row<F_Q8_0> {
    static constexpr int kGroup = 1, kScales = 1;
    static constexpr bool kMin = false;
    uint32_t w[2];
    float d;
    template <bool EVEN>
    __device__ __forceinline__ void load(const RowAt<EVEN> &row, int group, int, int t) {
        d = row.f16(34 * group);
        w[0] = row.word(34 * group + 2, 4 * t);
        w[1] = row.word(34 * group + 18, 4 * t);
    }
    __device__ __forceinline__ void pairs(int, uint32_t (&r)[4]) const {
        signed_bytes(w[0], r[0], r[1]);
        signed_bytes(w[1], r[2], r[3]);
    }
    __device__ __forceinline__ float scale(int, int) const { return d; }
    __device__ __forceinline__ float min(int) const { return 0.0f; }
};

// A chunk is the 16-byte header and half `half` of a super-block's codes.
template <>
struct Row<F_Q4_K> {
    static constexpr int kGroup = 2, kScales = 1;
    static constexpr bool kMin = true;
    uint32_t w0, w1;   // 32 code bytes: low nibbles the first block, high ones the second
    uint32_t sc, m;    // the group's two scales and mins, bytes 0 and 1
    float d, dmin;
    template <bool EVEN>
    __device__ __forceinline__ void load(const RowAt<EVEN> &row, int group, int half, int t) {
        const uint8_t *const chunk = row.p;
        const uint4 h = *reinterpret_cast<const uint4 *>(chunk);
        d = f16_bits_to_f32(h.x & 0xFFFFu);
        dmin = f16_bits_to_f32(h.x >> 16);
        sc = half ? (h.w & 0x0F0F0F0Fu) | ((h.y >> 2) & 0x30303030u) : h.y & 0x3F3F3F3Fu;
        m = half ? ((h.w >> 4) & 0x0F0F0F0Fu) | ((h.z >> 2) & 0x30303030u) : h.z & 0x3F3F3F3Fu;
        if (group) {
            sc >>= 16;
            m >>= 16;
        }
        w0 = ld32(chunk + 16 + 32 * group + 4 * t);
        w1 = ld32(chunk + 32 + 32 * group + 4 * t);
    }
    __device__ __forceinline__ void pairs(int sub, uint32_t (&r)[4]) const {
        if (sub == 0) {
            low_nibbles<0>(w0, r[0], r[1]);
            low_nibbles<0>(w1, r[2], r[3]);
        } else {
            high_nibbles<0>(w0, r[0], r[1]);
            high_nibbles<0>(w1, r[2], r[3]);
        }
    }
    // bytes as floats 2^23 + v; v and the products with d are exact
    __device__ __forceinline__ float scale(int sub, int) const {
        const float v = sub ? byte_magic23<1>(sc) : byte_magic23<0>(sc);
        return d * (v - 8388608.0f);
    }
    __device__ __forceinline__ float min(int sub) const {
        const float v = sub ? byte_magic23<1>(m) : byte_magic23<0>(m);
        return dmin * (8388608.0f - v);
    }
};

// A chunk is a super-block; a group is half of it (128 weights).
template <>
struct Row<F_Q6_K> {
    static constexpr int kGroup = 4, kScales = 2;
    static constexpr bool kMin = false;
    uint32_t ql[4], qh[2];  // [32 bytes (2)][16-deep step], [step]
    uint32_t sc[2];         // the group's eight int8 scales
    float d;
    template <bool EVEN>
    __device__ __forceinline__ void load(const RowAt<EVEN> &row, int group, int, int t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) ql[i] = row.word(16 * i, 64 * group + 4 * t);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            qh[i] = row.word(128 + 16 * i, 32 * group + 4 * t);
            sc[i] = row.word(192, 8 * group + 4 * i);
        }
        d = row.f16(208);
    }
    __device__ __forceinline__ void pairs(int sub, uint32_t (&r)[4]) const {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint32_t low = ql[2 * (sub & 1) + u] >> (sub & 2 ? 4 : 0);
            const uint32_t high = sub < 2 ? qh[u] << (4 - 2 * sub) : qh[u] >> (2 * sub - 4);
            bytes<32>((low & 0x0F0F0F0Fu) | (high & 0x30303030u), r[2 * u], r[2 * u + 1]);
        }
    }
    __device__ __forceinline__ float scale(int sub, int step) const {
        const int i = 2 * sub + step;
        return d * (float)(int)(int8_t)(sc[i >> 2] >> (8 * (i & 3)));
    }
    __device__ __forceinline__ float min(int) const { return 0.0f; }
};

template <>
struct Row<F_F16> {
    static constexpr int kGroup = 1, kScales = 0;
    static constexpr bool kMin = false;
    uint32_t w[4];
    // EVEN: rows start at multiples of 4 bytes (k is even)
    template <bool EVEN>
    __device__ __forceinline__ void load(const RowAt<EVEN> &row, int group, int, int t) {
        const uint8_t *p = row.p + 64 * group + 8 * t;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (EVEN) {
                w[2 * i] = ld32(p + 32 * i);
                w[2 * i + 1] = ld32(p + 32 * i + 4);
            } else {
                const uint2 v = *reinterpret_cast<const uint2 *>(p + 32 * i);
                w[2 * i] = v.x;
                w[2 * i + 1] = v.y;
            }
        }
    }
    __device__ __forceinline__ void pairs(int, uint32_t (&r)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = w[i];
    }
    __device__ __forceinline__ float scale(int, int) const { return 1.0f; }
    __device__ __forceinline__ float min(int) const { return 0.0f; }
};
template <>
struct Row<F_BF16> : Row<F_F16> {};

// ------------------------------------------------------- activations ----

// Writes a block of 32 activations (lane e holds element e) as the B operand's terms for weights of
// format `fmt`: `rec` holds the terms one after the other, 64 bytes each, element e at
// place_of(e). Returns, in every lane, {scale, sum}: the power of two that the
// terms' sum is multiplied by to give the value, and the block's sum.
// fp16: the largest of the values is brought to [2^14, 2^15), so that the low
// term of a value 2^-17 of it is still a normal number. Values among which there is an
// Inf or NaN are taken as they are.
__device__ __forceinline__ float2 put_terms(float v, int e, int fmt, uint8_t *rec) {
    float sum = v;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    const uint32_t top = __reduce_max_sync(~0u, (__float_as_uint(v) >> 23) & 255u);
    const int at = place_of(order_of(fmt), e);
    if (fmt == F_BF16) {
        float rest = v;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const __nv_bfloat16 h = __float2bfloat16_rz(rest);  // cut: three times 8 bits are all 24
            reinterpret_cast<__nv_bfloat16 *>(rec + 64 * i)[at] = h;
            const float f = __bfloat162float(h);
            rest = isfinite(f) ? rest - f : 0.0f;
        }
        return make_float2(1.0f, sum);
    }
    const uint32_t b = top < 15 ? 15 : top;
    const bool plain = top == 255;
    const float up = plain ? 1.0f : __uint_as_float((268u - b) << 23);   // 2^(14 + 127 - b)
    const float down = plain ? 1.0f : __uint_as_float((b - 14u) << 23);  // 1 / up
    const float x = v * up;
    const __half hi = __float2half_rn(x);
    const float f = __half2float(hi);
    reinterpret_cast<__half *>(rec)[at] = hi;
    reinterpret_cast<__half *>(rec + 64)[at] = __float2half_rn(isfinite(f) ? x - f : 0.0f);
    return make_float2(down, sum);
}

}  // namespace experts
}  // namespace qmm
