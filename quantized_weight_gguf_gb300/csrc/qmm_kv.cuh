// qmm_kv.cuh -- layout of the paged key-value cache (include/qmm.h), shared by
// the kernels that append to it, read it back and attend to it.
//
// A page holds, per kv head, strips of 16 positions; a strip is contiguous:
// K codes, K scales, V codes, V scales. Codes are grouped in planes of one
// row of 32 bytes (16-bit formats: 16 dims; Q8_0: 32 dims) or 16 bytes (Q4_0:
// 32 dims) per position. One strip is one bulk copy, and in shared memory the
// 8 positions x 4 lanes of a tensor-core fragment read 256 consecutive bytes
// of a plane, without bank conflicts and without a swizzle.
#pragma once

#include <stdint.h>

#include "qmm_device.cuh"

namespace qmm {

constexpr int kStrip = 16;  // positions per strip

__host__ __device__ constexpr bool kv_quantised(int f) { return f == F_Q8_0 || f == F_Q4_0; }
__host__ __device__ constexpr int kv_row_bytes(int f) { return f == F_Q4_0 ? 16 : 32; }
__host__ __device__ constexpr int kv_plane_dims(int f) { return kv_quantised(f) ? 32 : 16; }
// bytes of a strip's K (or V) codes and scales
__host__ __device__ constexpr int kv_code_bytes(int f, int dim) {
    return dim / kv_plane_dims(f) * kStrip * kv_row_bytes(f);
}
__host__ __device__ constexpr int kv_scale_bytes(int f, int dim) {
    return kv_quantised(f) ? dim / 32 * kStrip * 2 : 0;
}
__host__ __device__ constexpr int kv_half_bytes(int f, int dim) {
    return kv_code_bytes(f, dim) + kv_scale_bytes(f, dim);
}
__host__ __device__ constexpr int kv_strip_bytes(int fk, int fv, int dim) {
    return kv_half_bytes(fk, dim) + kv_half_bytes(fv, dim);
}

// The cache as the kernels see it.
struct KvView {
    uint8_t *pages;
    const int32_t *table;
    const int32_t *lens;
    int64_t head_bytes;    // bytes of one kv head in a page
    int64_t table_stride;
    int64_t n_pages;
    int64_t capacity;      // positions that a table row can hold
    int fmt_k, fmt_v;
    int n_kv, dim, page_size;
    int strip_bytes, v_off;
    int n_seqs;
    unsigned int *err;
};

// Strip `strip` (of 16 positions, counted from the sequence's start) of head
// h of sequence s, or nullptr (with the error recorded) when the table names
// no page of the pool. strip * 16 < capacity.
__device__ __forceinline__ uint8_t *kv_strip(const KvView &c, int s, int h, int strip) {
    const int per = c.page_size / kStrip;
    const int entry = strip / per;
    const int page = __ldg(c.table + (int64_t)s * c.table_stride + entry);
    if ((unsigned)page >= (unsigned long long)c.n_pages) {
        record_error(c.err, DERR_BAD_PAGE);
        return nullptr;
    }
    return c.pages + ((int64_t)page * c.n_kv + h) * c.head_bytes +
           (int64_t)(strip - entry * per) * c.strip_bytes;
}

// A sequence's length within its table; a longer one is reported and cut.
__device__ __forceinline__ int kv_length(const KvView &c, int s) {
    const int n = __ldg(c.lens + s);
    if (n > c.capacity) {
        record_error(c.err, DERR_BAD_PAGE);
        return (int)c.capacity;
    }
    return n < 0 ? 0 : n;
}

// Dims d0 .. d0 + 3 (d0 % 4 == 0) of position t of a strip half (K or V) in
// format f, as fp32 (exact).
__device__ __forceinline__ float4 kv_load4(const uint8_t *half, int f, int dim, int t, int d0) {
    if (!kv_quantised(f)) {
        const uint2 w = *reinterpret_cast<const uint2 *>(half + (d0 >> 4) * 512 + t * 32 +
                                                         (d0 & 15) * 2);
        if (f == F_BF16)
            return make_float4(bf16_bits_to_f32(w.x & 0xffffu), bf16_bits_to_f32(w.x >> 16),
                               bf16_bits_to_f32(w.y & 0xffffu), bf16_bits_to_f32(w.y >> 16));
        return make_float4(f16_bits_to_f32(w.x & 0xffffu), f16_bits_to_f32(w.x >> 16),
                           f16_bits_to_f32(w.y & 0xffffu), f16_bits_to_f32(w.y >> 16));
    }
    const int b = d0 >> 5;
    const float d = f16_bits_to_f32(
        *reinterpret_cast<const uint16_t *>(half + kv_code_bytes(f, dim) + (b * kStrip + t) * 2));
    if (f == F_Q8_0) {
        const char4 q = *reinterpret_cast<const char4 *>(half + b * 512 + t * 32 + (d0 & 31));
        return make_float4(d * q.x, d * q.y, d * q.z, d * q.w);
    }
    const unsigned w = *reinterpret_cast<const uint16_t *>(half + b * 256 + t * 16 + ((d0 & 31) >> 1));
    return make_float4(d * ((int)(w & 15u) - 8), d * ((int)((w >> 4) & 15u) - 8),
                       d * ((int)((w >> 8) & 15u) - 8), d * ((int)(w >> 12) - 8));
}

}  // namespace qmm
