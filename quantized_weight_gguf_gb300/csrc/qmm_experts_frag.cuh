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
// as long as both operands share it. Lane (g, t) of the fragment (g = lane / 4,
// t = lane % 4) takes, of row g and in this order,
//     4t, 4t+2 | 4t+1, 4t+3 (first step)   16+4t, 16+4t+2 | 16+4t+1, 16+4t+3 (second):
// one 4-byte word of codes gives what a lane needs of a step, and masks of a
// 4-bit word leave its values in just these pairs.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qmm_device.cuh"

namespace qmm {
namespace experts {

// 16-bit terms of an activation; bytes of a block of 32 of them (see put_block).
__host__ __device__ constexpr int terms_of(int fmt) { return fmt == F_BF16 ? 3 : 2; }
__host__ __device__ constexpr int frag_bytes(int fmt) { return 64 * terms_of(fmt); }

// Place (0..31, in units of one value) of element e of a block in a term's 64 bytes.
__host__ __device__ constexpr int place_of(int e) {
    return (e & 15) / 4 * 8 + (e & 16) / 4 + ((e & 1) << 1) + ((e & 2) >> 1);
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
// 16-byte pieces that cover a chunk wherever it starts (rows start at even
// addresses), and the distance of rows in shared memory: an odd multiple of 16
// bytes, so that the 8 rows of a fragment's word loads fall on different banks
// (of 32 bytes for the 16-bit formats' 8-byte loads).
__host__ __device__ constexpr int chunk_pieces(int fmt) {
    return fmt == F_Q4_K ? 5 : (chunk_bytes(fmt) + 14 + 15) / 16;
}
__host__ __device__ constexpr int row_pitch(int fmt) {
    return fmt == F_BF16 || fmt == F_F16 ? 160 : 16 * (chunk_pieces(fmt) | 1);
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
// the 4 bytes at p, which is even
__device__ __forceinline__ uint32_t ld32_even(const uint8_t *p) {
    const uint32_t odd = (uint32_t)reinterpret_cast<uintptr_t>(p) & 2u;
    const uint32_t w0 = ld32(p - odd), w1 = ld32(p - odd + 4);
    return prmt(w0, w1, odd ? 0x5432u : 0x3210u);
}
__device__ __forceinline__ float f16_at(const uint8_t *p) { return f16_bits_to_f32(ld16(p)); }

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
    __device__ __forceinline__ void load(const uint8_t *chunk, int group, int, int t) {
        const uint8_t *p = chunk + 18 * group;
        d = f16_at(p);
        w = ld32_even(p + 2 + 4 * t);
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
    __device__ __forceinline__ void load(const uint8_t *chunk, int group, int, int t) {
        const uint8_t *p = chunk + 22 * group;
        d = f16_at(p);
        high = ld32_even(p + 2) >> (4 * t);
        w = ld32_even(p + 6 + 4 * t);
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
    uint32_t w0, w1;
    float d;
    __device__ __forceinline__ void load(const uint8_t *chunk, int group, int, int t) {
        const uint8_t *p = chunk + 34 * group;
        d = f16_at(p);
        w0 = ld32_even(p + 2 + 4 * t);
        w1 = ld32_even(p + 18 + 4 * t);
    }
    __device__ __forceinline__ void pairs(int, uint32_t (&r)[4]) const {
        bytes<128>(w0 ^ 0x80808080u, r[0], r[1]);
        bytes<128>(w1 ^ 0x80808080u, r[2], r[3]);
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
    __device__ __forceinline__ void load(const uint8_t *chunk, int group, int half, int t) {
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
    __device__ __forceinline__ void load(const uint8_t *chunk, int group, int, int t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) ql[i] = ld32_even(chunk + 64 * group + 16 * i + 4 * t);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            qh[i] = ld32_even(chunk + 128 + 32 * group + 16 * i + 4 * t);
            sc[i] = ld32_even(chunk + 192 + 8 * group + 4 * i);
        }
        d = f16_at(chunk + 208);
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
    // rows start at multiples of 4 bytes (k is even)
    __device__ __forceinline__ void load(const uint8_t *chunk, int group, int, int t) {
        const uint8_t *p = chunk + 64 * group + 8 * t;
        w[0] = ld32(p);
        w[1] = ld32(p + 4);
        w[2] = ld32(p + 32);
        w[3] = ld32(p + 36);
    }
    __device__ __forceinline__ void pairs(int, uint32_t (&r)[4]) const {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            r[2 * u] = prmt(w[2 * u], w[2 * u + 1], 0x5410u);
            r[2 * u + 1] = prmt(w[2 * u], w[2 * u + 1], 0x7632u);
        }
    }
    __device__ __forceinline__ float scale(int, int) const { return 1.0f; }
    __device__ __forceinline__ float min(int) const { return 0.0f; }
};
template <>
struct Row<F_BF16> : Row<F_F16> {};

// ------------------------------------------------------- activations ----

// Writes a block of 32 activations (lane e holds element e) as the B operand's
// terms: `rec` holds the terms one after the other, 64 bytes each, element e at
// place_of(e). Returns, in every lane, {scale, sum}: the power of two that the
// terms' sum is multiplied by to give the value, and the block's sum.
// fp16: the block's largest value is brought to [2^14, 2^15), so that the low
// term of a value 2^-17 of it is still a normal number. A block that holds an
// Inf or NaN is taken as it is.
__device__ __forceinline__ float2 put_block(float v, int lane, bool bf16, uint8_t *rec) {
    float sum = v;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    const int at = place_of(lane);
    if (bf16) {
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
    const uint32_t top = __reduce_max_sync(~0u, __float_as_uint(v) & 0x7F800000u) >> 23;
    const uint32_t e = top < 15 ? 15 : top;
    const bool plain = top == 255;
    const float up = plain ? 1.0f : __uint_as_float((268u - e) << 23);   // 2^(14 + 127 - e)
    const float down = plain ? 1.0f : __uint_as_float((e - 14u) << 23);  // 1 / up
    const float x = v * up;
    const __half hi = __float2half_rn(x);
    const float f = __half2float(hi);
    reinterpret_cast<__half *>(rec)[at] = hi;
    reinterpret_cast<__half *>(rec + 64)[at] = __float2half_rn(isfinite(f) ? x - f : 0.0f);
    return make_float2(down, sum);
}

}  // namespace experts
}  // namespace qmm
