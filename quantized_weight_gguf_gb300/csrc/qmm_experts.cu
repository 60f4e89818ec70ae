// qmm_experts.cu -- the experts' feed-forward network over packed weights:
//     y[p] (+)= sum_s w[p][s] Wd_e (act(Wg_e x[p]) * (Wu_e x[p])),  e = ids[p][s].
// Few rows go row by row: x becomes digits (one launch; one position: the next one does it), the gate and up products
// with the activation, and the down product over each position's slots. More take four launches: the pairs (position,
// slot) are sorted by expert while x becomes 16-bit terms; the gate and up products; the down product, a row per pair;
// the sum of each position's rows. Many take a fifth, which makes the gate and up products' results terms once whole
// rows of them are there. Each is a programmatic dependent of the one before. This file holds all but the
// products, and the host side.
#include <algorithm>

#include "qmm_experts.h"
#include "qmm_experts_tile.cuh"

namespace qmm {

namespace experts {

// one translation unit per group of formats
#define QMM_EXPERTS_FORMAT(FMT) \
    extern template cudaError_t launch_product<FMT>(bool, int, const ProductParams &, int, const DeviceInfo &, cudaStream_t); \
    extern template cudaError_t launch_single<FMT>(bool, const ProductParams &, const DeviceInfo &, cudaStream_t);
#define QMM_EXPERTS_CODES(FMT) \
    QMM_EXPERTS_FORMAT(FMT) \
    extern template cudaError_t launch_tile<FMT>(bool, const ProductParams &, int, const DeviceInfo &, cudaStream_t);
QMM_EXPERTS_FORMAT(F_BF16)
QMM_EXPERTS_FORMAT(F_F16)
QMM_EXPERTS_CODES(F_Q4_0)
QMM_EXPERTS_CODES(F_Q4_K)
QMM_EXPERTS_CODES(F_Q6_K)
QMM_EXPERTS_CODES(F_Q8_0)
QMM_EXPERTS_CODES(F_Q5_0)
#undef QMM_EXPERTS_CODES
#undef QMM_EXPERTS_FORMAT

namespace {

constexpr int kPrepareThreads = 256, kPrepareWarps = kPrepareThreads / 32;

struct PrepareParams {
    const int32_t *ids;
    int pairs, n_experts, columns;
    Tile *tiles;
    int *n_tiles, *order;
    const float *x;
    int n_pos, k, x_blocks, fmt;
    uint8_t *terms;
    float *scales, *sums;
    int64_t x_row_bytes;
    unsigned int *err;
};

// Exclusive prefix sum of `v` over the block's threads; *total: the sum of all.
__device__ __forceinline__ int block_scan(int v, int *warp_sums, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(~0u, inc, o);
        if (lane >= o) inc += a;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < kPrepareWarps; ++w) {
        before += w < warp ? warp_sums[w] : 0;
        all += warp_sums[w];
    }
    __syncthreads();
    *total = all;
    return before + inc - v;
}

// The pairs in the order of their experts, and the tiles of up to `columns` of
// them. Which place a pair takes among its expert's is up to the atomics; no
// result depends on it (a pair's sums are its column's alone).
__device__ void sort_pairs(const PrepareParams &p) {
    __shared__ int count[kMaxExperts];
    __shared__ int warp_sums[kPrepareWarps];
    const int tid = threadIdx.x;
    for (int e = tid; e < p.n_experts; e += kPrepareThreads) count[e] = 0;
    __syncthreads();
    for (int i = tid; i < p.pairs; i += kPrepareThreads) {
        const int e = p.ids[i];
        if (e >= 0 && e < p.n_experts) atomicAdd(&count[e], 1);
        else if (e != -1) record_error(p.err, DERR_BAD_ID);
    }
    __syncthreads();
    const int per = (p.n_experts + kPrepareThreads - 1) / kPrepareThreads;
    const int e0 = min(tid * per, p.n_experts), e1 = min(e0 + per, p.n_experts);
    int rows = 0, tiles = 0;
    for (int e = e0; e < e1; ++e) {
        rows += count[e];
        tiles += (count[e] + p.columns - 1) / p.columns;
    }
    int all_rows, all_tiles;
    int row = block_scan(rows, warp_sums, &all_rows);
    int tile = block_scan(tiles, warp_sums, &all_tiles);
    for (int e = e0; e < e1; ++e) {
        const int n = count[e];
        count[e] = row;  // becomes the place of the expert's next pair
        for (int at = 0; at < n; at += p.columns) {
            Tile x;
            x.expert = e;
            x.start = row + at;
            x.count = min(p.columns, n - at);
            x.pad = 0;
            p.tiles[tile++] = x;
        }
        row += n;
    }
    if (tid == 0) *p.n_tiles = all_tiles;
    __syncthreads();
    for (int i = tid; i < p.pairs; i += kPrepareThreads) {
        const int e = p.ids[i];
        if (e >= 0 && e < p.n_experts) p.order[atomicAdd(&count[e], 1)] = i;
    }
}

// Block 0 sorts the pairs (row by row: looks at their ids), the others turn x into terms (records), a block of 32
// values per warp.
__global__ void __launch_bounds__(kPrepareThreads) prepare_kernel(const __grid_constant__ PrepareParams p) {
    pdl_wait_prev();
    if (blockIdx.x == 0) {
        if (p.columns > 1) {
            sort_pairs(p);
        } else {
            for (int i = threadIdx.x; i < p.pairs; i += kPrepareThreads)
                if (p.ids[i] < -1 || p.ids[i] >= p.n_experts) record_error(p.err, DERR_BAD_ID);
        }
        return;
    }
    const int lane = threadIdx.x & 31;
    const int64_t all = (int64_t)p.n_pos * p.x_blocks, step = (int64_t)(gridDim.x - 1) * kPrepareWarps;
    for (int64_t i = (int64_t)(blockIdx.x - 1) * kPrepareWarps + (threadIdx.x >> 5); i < all; i += step) {
        const int64_t row = i / p.x_blocks;
        const int b = (int)(i % p.x_blocks), e = 32 * b + lane;
        const float v = e < p.k ? p.x[row * p.k + e] : 0.0f;
        if (p.columns == 1) {
            put_record(v, lane, p.fmt, p.terms + row * p.x_row_bytes + (int64_t)b * kRecord);
            continue;
        }
        const float2 s = put_terms(v, lane, p.fmt, p.terms + row * p.x_row_bytes + (int64_t)b * frag_bytes(p.fmt));
        if (lane == 0) {
            p.scales[i] = s.x;
            p.sums[i] = s.y;
        }
    }
}

// Rows of activations as the tile kernels' terms, a row per CTA at a time: each term 32 fp16 of a block,
// under the power of two that brings the row's largest to [2^14, 2^15) (the scale is its inverse), and the sums
// of the scaled blocks. With ids, block 0 sorts the pairs. Rows with an Inf or NaN are taken as they are.
__global__ void __launch_bounds__(kPrepareThreads) tile_terms_kernel(const __grid_constant__ PrepareParams p) {
    __shared__ uint32_t tops[kPrepareWarps];
    pdl_wait_prev();
    const int sorts = p.ids != nullptr;
    if (sorts && blockIdx.x == 0) {
        sort_pairs(p);
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t row = (int64_t)blockIdx.x - sorts; row < p.n_pos; row += gridDim.x - sorts) {
        const float *const x = p.x + row * p.k;
        uint32_t top = 0;
        for (int i = threadIdx.x; i < p.k; i += kPrepareThreads) top = max(top, (__float_as_uint(x[i]) >> 23) & 255u);
        top = __reduce_max_sync(~0u, top);
        if (lane == 0) tops[warp] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPrepareWarps; ++i) top = max(top, tops[i]);
        __syncthreads();
        const uint32_t b = top < 15 ? 15 : top;
        const bool plain = top == 255;
        const float up = plain ? 1.0f : __uint_as_float((268u - b) << 23);  // 2^(14 + 127 - b)
        if (threadIdx.x == 0) p.scales[row] = plain ? 1.0f : __uint_as_float((b - 14u) << 23);
        for (int i = warp; i < p.k / 32; i += kPrepareWarps) {
            const float v = x[32 * i + lane] * up;
            const __half hi = __float2half_rn(v);
            const float f = __half2float(hi);
            uint8_t *const block = p.terms + row * p.x_row_bytes + (int64_t)i * kTermBytes;
            __half *const to = reinterpret_cast<__half *>(block) + tile_place(lane);
            to[0] = hi;
            to[32] = __float2half_rn(isfinite(f) ? v - f : 0.0f);
            if (p.fmt == F_Q4_K) {
                float sum = v;
#pragma unroll
                for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
                if (lane == 0) p.sums[row * p.x_blocks + i] = sum;
            }
        }
    }
}

struct SumParams {
    const float *rows;       // [pairs][k]
    const int32_t *ids;
    float *y;
    int64_t values;          // n_pos * k
    int k, top_k, n_experts;
    int accumulate;
};
constexpr int kSumThreads = 256;

// y[p] (+)= the sum of the position's rows, slots in order; slots without an
// expert have no row. V values per thread.
template <int V>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(const __grid_constant__ SumParams p) {
    pdl_wait_prev();
    const int64_t at = ((int64_t)blockIdx.x * kSumThreads + threadIdx.x) * V;
    if (at >= p.values) return;
    const int64_t pos = at / p.k;
    const int j = (int)(at % p.k);
    float s[V];
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = 0.0f;
    for (int t = 0; t < p.top_k; ++t) {
        const int e = p.ids[pos * p.top_k + t];
        if (e < 0 || e >= p.n_experts) continue;
        const float *r = p.rows + (pos * p.top_k + t) * p.k + j;
        if constexpr (V == 4) {
            const float4 v = *reinterpret_cast<const float4 *>(r);
            s[0] += v.x;
            s[1] += v.y;
            s[2] += v.z;
            s[3] += v.w;
        } else {
            s[0] += *r;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (p.accumulate) s[i] += p.y[at + i];
        p.y[at + i] = s[i];
    }
}

template <class P>
cudaError_t launch_next(void (*kernel)(P), const P &p, int64_t grid, int threads, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

// Blocks of 32 of a row of terms, padded to the largest chunk.
int padded_blocks(int k) { return (k + 255) / 256 * 8; }

// One position whose x fits the shared memory: two launches.
bool is_one(const ExpertsFfn &f) { return f.n_pos == 1 && (f.k + 31) / 32 <= kOneBlocks; }

// How the products are taken, by the rows that an expert gets when all are chosen equally often. Measured at 64 experts,
// top 8, 2048 x 768, in us: row by row (1), tiles of 8 and 16 columns on mma.sync, and of 48 on tcgen05 (T):
//   rows           1/4           1           3/2             8             16            24            32            64
//   Q4_K    1:20 8:41   1:56 8:73   1:77  8:91  8:147 16:142  16:186 T:197  16:276 T:210  16:308 T:219  16:551 T:362
//   Q8_0    1:23 8:40   1:66 8:74   1:89  8:89  8:139 16:137  16:181 T:244  16:255 T:257  16:287 T:264  16:505 T:478
//   Q6_K    1:31 8:48   1:99 8:97  1:141 8:117  8:190 16:182  16:237 T:300  16:341 T:314  16:407 T:324  16:689 T:582
//   BF16    1:33 8:45   1:93 8:94  1:129 8:106  8:146 16:154
// One set of borders for all formats: at the sizes above it gives away up to 15 % (Q4_K at 3/2 rows), and 2 to 4 % at 8.
// Tiles on tcgen05 are for codes, whose blocks' sums a scale multiplies on their way out.
bool is_tile(const ExpertsFfn &f) {
    const bool codes = f.fmt != F_BF16 && f.fmt != F_F16 && f.fmt_down != F_BF16 && f.fmt_down != F_F16;
    return codes && !is_one(f) && f.n_pos * f.top_k > 20 * (int64_t)f.n_experts;
}
int columns_of(const ExpertsFfn &f) {
    const int64_t pairs = f.n_pos * f.top_k, n = f.n_experts;
    return is_tile(f) ? kTileColumns : pairs <= n || is_one(f) ? 1 : pairs <= 8 * n ? 8 : 16;
}

// The most tiles that the ids can make: each expert that is chosen leaves at
// most one tile that is not full.
int64_t max_tiles(const ExpertsFfn &f, int columns) {
    const int64_t pairs = f.n_pos * f.top_k;
    return std::min<int64_t>(pairs, pairs / columns + std::min<int64_t>(f.n_experts, pairs));
}

// The parts of the workspace.
struct Scratch {
    size_t tiles, n_tiles, order, x, x_scale, x_sum, h, h_scale, h_sum, out, bytes;
    size_t h32;  // tiles: the first product's results
    bool tile;
    int columns;
    int64_t x_row_bytes, h_row_bytes;
    int x_blocks, h_blocks;
};
Scratch scratch_of(const ExpertsFfn &f) {
    Scratch s = {};
    const size_t pairs = (size_t)(f.n_pos * f.top_k);
    s.tile = is_tile(f);
    s.columns = columns_of(f);
    s.x_blocks = padded_blocks(f.k);
    s.h_blocks = padded_blocks(f.n_ff);
    s.x_row_bytes = (int64_t)s.x_blocks * (s.columns == 1 ? kRecord : s.tile ? kTermBytes : frag_bytes(f.fmt));
    s.h_row_bytes = (int64_t)s.h_blocks * (s.columns == 1 ? kRecord : s.tile ? kTermBytes : frag_bytes(f.fmt_down));
    size_t at = 0;
    auto part = [&](size_t bytes) {
        const size_t here = at;
        at += round256(bytes);
        return here;
    };
    s.h = part((size_t)s.h_row_bytes * pairs);
    if (is_one(f)) {  // h alone
        s.bytes = at;
        return s;
    }
    s.x = part((size_t)s.x_row_bytes * (size_t)f.n_pos);
    if (s.columns == 1) {
        s.bytes = at;
        return s;
    }
    s.h_scale = part(sizeof(float) * (size_t)s.h_blocks * pairs);
    s.h_sum = part(sizeof(float) * (size_t)s.h_blocks * pairs);
    s.n_tiles = part(sizeof(int));
    s.tiles = part(sizeof(Tile) * (size_t)max_tiles(f, s.columns));
    s.order = part(sizeof(int) * pairs);
    s.x_scale = part(sizeof(float) * (size_t)s.x_blocks * (size_t)f.n_pos);
    s.x_sum = part(sizeof(float) * (size_t)s.x_blocks * (size_t)f.n_pos);
    s.out = part(sizeof(float) * (size_t)f.k * pairs);
    if (s.tile) s.h32 = part(sizeof(float) * (size_t)f.n_ff * pairs);
    s.bytes = at;
    return s;
}

template <int FMT>
cudaError_t product_of(bool down, bool tile, int columns, const ProductParams &p, int tiles, const DeviceInfo &dev,
                       cudaStream_t s) {
    if constexpr (FMT != F_BF16 && FMT != F_F16)
        if (tile) return launch_tile<FMT>(down, p, tiles, dev, s);
    return columns == 1 ? launch_single<FMT>(down, p, dev, s)
                        : launch_product<FMT>(down, columns, p, tiles, dev, s);
}
cudaError_t product(int fmt, bool down, bool tile, int columns, const ProductParams &p, int tiles, const DeviceInfo &dev,
                    cudaStream_t s) {
    switch (fmt) {
    case F_BF16: return product_of<F_BF16>(down, tile, columns, p, tiles, dev, s);
    case F_F16: return product_of<F_F16>(down, tile, columns, p, tiles, dev, s);
    case F_Q4_0: return product_of<F_Q4_0>(down, tile, columns, p, tiles, dev, s);
    case F_Q4_K: return product_of<F_Q4_K>(down, tile, columns, p, tiles, dev, s);
    case F_Q6_K: return product_of<F_Q6_K>(down, tile, columns, p, tiles, dev, s);
    case F_Q8_0: return product_of<F_Q8_0>(down, tile, columns, p, tiles, dev, s);
    default: return product_of<F_Q5_0>(down, tile, columns, p, tiles, dev, s);
    }
}

}  // namespace

}  // namespace experts

size_t experts_ffn_workspace_bytes(const ExpertsFfn &f) { return experts::scratch_of(f).bytes; }

cudaError_t launch_experts_ffn(const ExpertsFfn &f, const DeviceInfo &dev, cudaStream_t s) {
    using namespace experts;
    const Scratch l = scratch_of(f);
    uint8_t *const ws = static_cast<uint8_t *>(f.workspace);
    const int pairs = (int)(f.n_pos * f.top_k);
    const int tiles = (int)max_tiles(f, l.columns);

    PrepareParams a = {};
    a.ids = f.ids;
    a.pairs = pairs;
    a.n_experts = f.n_experts;
    a.columns = l.columns;
    a.tiles = reinterpret_cast<Tile *>(ws + l.tiles);
    a.n_tiles = reinterpret_cast<int *>(ws + l.n_tiles);
    a.order = reinterpret_cast<int *>(ws + l.order);
    a.x = f.x;
    a.n_pos = (int)f.n_pos;
    a.k = f.k;
    a.x_blocks = l.x_blocks;
    a.fmt = f.fmt;
    a.terms = ws + l.x;
    a.scales = reinterpret_cast<float *>(ws + l.x_scale);
    a.sums = reinterpret_cast<float *>(ws + l.x_sum);
    a.x_row_bytes = l.x_row_bytes;
    a.err = dev.err;
    cudaError_t e = cudaSuccess;
    const int64_t warps = f.n_pos * l.x_blocks;
    const int64_t blocks = std::min<int64_t>((warps + kPrepareWarps - 1) / kPrepareWarps, (int64_t)dev.sm_count * 8);
    const bool one = is_one(f);
    const int64_t rows_at_once = (int64_t)dev.sm_count * 8;
    if (l.tile) e = launch_next(tile_terms_kernel, a, 1 + std::min(f.n_pos, rows_at_once), kPrepareThreads, s);
    else if (!one) e = launch_next(prepare_kernel, a, 1 + blocks, kPrepareThreads, s);
    if (e != cudaSuccess) return e;

    ProductParams p = {};
    p.w[0] = f.gate;
    p.w[1] = f.up;
    p.row_bytes = f.row_bytes;
    p.slice_bytes = f.row_bytes * f.n_ff;
    p.rows = f.n_ff;
    p.k = f.k;
    p.blocks = (f.k + 31) / 32;
    p.x = a.terms;
    p.x_scale = a.scales;
    p.x_sum = a.sums;
    p.x_row_bytes = l.x_row_bytes;
    p.x_blocks = l.x_blocks;
    p.tiles = a.tiles;
    p.n_tiles = a.n_tiles;
    p.order = a.order;
    p.top_k = f.top_k;
    p.n_experts = f.n_experts;
    p.weights = f.weights;
    p.h = ws + (l.tile ? l.h32 : l.h);
    p.h_scale = reinterpret_cast<float *>(ws + l.h_scale);
    p.h_sum = reinterpret_cast<float *>(ws + l.h_sum);
    p.h_row_bytes = l.h_row_bytes;
    p.h_blocks = l.h_blocks;
    p.h_fmt = f.fmt_down;
    p.act = f.act;
    p.n_pos = (int)f.n_pos;
    p.x32 = one ? f.x : nullptr;
    p.ids = f.ids;
    p.accumulate = f.accumulate;
    p.err = dev.err;
    e = product(f.fmt, false, l.tile, l.columns, p, tiles, dev, s);
    if (e != cudaSuccess) return e;

    if (l.tile) {
        a.ids = nullptr;
        a.x = reinterpret_cast<const float *>(ws + l.h32);
        a.n_pos = pairs;
        a.k = f.n_ff;
        a.x_blocks = l.h_blocks;
        a.fmt = f.fmt_down;
        a.terms = ws + l.h;
        a.scales = p.h_scale;
        a.sums = p.h_sum;
        a.x_row_bytes = l.h_row_bytes;
        e = launch_next(tile_terms_kernel, a, std::min<int64_t>(pairs, rows_at_once), kPrepareThreads, s);
        if (e != cudaSuccess) return e;
        p.h = ws + l.h;
    }
    p.w[0] = p.w[1] = f.down;
    p.row_bytes = f.down_row_bytes;
    p.slice_bytes = f.down_row_bytes * f.k;
    p.rows = f.k;
    p.k = f.n_ff;
    p.blocks = (f.n_ff + 31) / 32;
    p.x = p.h;
    p.x_scale = p.h_scale;
    p.x_sum = p.h_sum;
    p.x_row_bytes = l.h_row_bytes;
    p.x_blocks = l.h_blocks;
    p.out = l.columns == 1 ? f.y : reinterpret_cast<float *>(ws + l.out);
    e = product(f.fmt_down, true, l.tile, l.columns, p, tiles, dev, s);
    if (e != cudaSuccess || l.columns == 1) return e;

    SumParams q = {};
    q.rows = p.out;
    q.ids = f.ids;
    q.y = f.y;
    q.values = f.n_pos * f.k;
    q.k = f.k;
    q.top_k = f.top_k;
    q.n_experts = f.n_experts;
    q.accumulate = f.accumulate;
    if (f.k % 4 == 0)
        return launch_next(sum_kernel<4>, q, (q.values / 4 + kSumThreads - 1) / kSumThreads, kSumThreads, s);
    return launch_next(sum_kernel<1>, q, (q.values + kSumThreads - 1) / kSumThreads, kSumThreads, s);
}

}  // namespace qmm
