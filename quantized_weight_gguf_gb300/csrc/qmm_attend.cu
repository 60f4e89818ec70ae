// qmm_attend.cu -- host side of the attention over the paged key-value cache
// (the kernel is in qmm_attend_kernel.cuh), and the join of items whose
// positions were split over several CTAs.
#include "qmm_attend.h"

namespace qmm {

namespace attend {

// Joins split items: out = sum_k 2^(m_k - M) s_k / sum_k 2^(m_k - M) l_k over
// an item's parts k. Block c serves the boundary between the shares of CTAs
// c and c + 1, if an item straddles it; the blocks of one item's boundaries
// divide its 8 x dim values evenly, so an item of many parts has as many
// blocks. Threads take the parts in a fixed order: the sum is the same on
// every call. Its time is that of its launch and of two loads that wait for one
// another (3 to 4 us of a call; 456 blocks that joined inside the attention
// kernel, the last to finish an item's part, made one sequence of 131071
// positions 65 us instead of 56).
constexpr int kBatch = 4;  // parts that a thread loads at once
__global__ void __launch_bounds__(kThreads) attend_join_kernel(const AttendParams a) {
    pdl_wait_prev();
    pdl_launch_dependents();
    const Join x = a.joins[blockIdx.x];
    if (x.parts < 2) return;
    // values f0 .. f1 - 1 are this block's; all numbers here are far below 2^32
    const unsigned dim = a.c.dim, quads = kRows * dim / 4, blocks = x.parts - 1, me = blockIdx.x - x.first;
    const int f0 = (int)(me * quads / blocks), f1 = (int)((me + 1) * quads / blocks);
    if (f0 >= f1) return;
    // `wide` neighbouring lanes share a value and take its parts in turn
    int log_wide = 0;
    while (log_wide < 5 && (f1 - f0) << (log_wide + 1) <= kThreads) ++log_wide;
    const int wide = 1 << log_wide, l = threadIdx.x & (wide - 1), f_of = f0 + (int)(threadIdx.x >> log_wide);
    for (int f = f_of; f - f_of + f0 < f1; f += kThreads >> log_wide) {
        const int row = (unsigned)f / (dim / 4), d = (f - row * ((int)dim / 4)) * 4;
        float m = -INFINITY, total = 0.0f;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = l; k0 < x.parts; k0 += kBatch * wide) {
            float mk[kBatch], lk[kBatch];
            float4 v[kBatch];
            float top = m;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int k = k0 + i * wide;
                mk[i] = -INFINITY;
                lk[i] = 0.0f;
                v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (f < f1 && k < x.parts) {
                    // the first part is its CTA's last item, the others their CTAs' first
                    const float *p = a.parts + (int64_t)(2 * (x.first + k) + (k == 0)) * part_floats(dim);
                    mk[i] = p[row];
                    lk[i] = p[kRows + row];
                    v[i] = *reinterpret_cast<const float4 *>(p + 2 * kRows + row * dim + d);
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) top = fmaxf(top, mk[i]);
            const float base = top == -INFINITY ? 0.0f : top;
            const float fo = exp2f(m - base);
            total *= fo;
            s = make_float4(s.x * fo, s.y * fo, s.z * fo, s.w * fo);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const float fn = exp2f(mk[i] - base);
                total = fmaf(fn, lk[i], total);
                s.x = fmaf(fn, v[i].x, s.x);
                s.y = fmaf(fn, v[i].y, s.y);
                s.z = fmaf(fn, v[i].z, s.z);
                s.w = fmaf(fn, v[i].w, s.w);
            }
            m = top;
        }
        float top = m;
        for (int o = 1; o < wide; o <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        const float fo = m == -INFINITY ? 0.0f : exp2f(m - top);
        total *= fo;
        s = make_float4(s.x * fo, s.y * fo, s.z * fo, s.w * fo);
        for (int o = 1; o < wide; o <<= 1) {
            total += __shfl_xor_sync(~0u, total, o);
            s.x += __shfl_xor_sync(~0u, s.x, o);
            s.y += __shfl_xor_sync(~0u, s.y, o);
            s.z += __shfl_xor_sync(~0u, s.z, o);
            s.w += __shfl_xor_sync(~0u, s.w, o);
        }
        if (f < f1 && l == 0) put_out<true>(a, x, row, d, dim, s, total);
    }
}

namespace {

int cost_of(const Attend &a) {
    return item_cost_of(a.c.fmt_k, a.c.fmt_v, a.c.dim, shape_of(a.c.fmt_k, a.c.fmt_v, a.c.dim).ctas);
}

// Tiles of a sequence and kv head; n_new * group is below 2^31.
int tiles_of(const Attend &a) { return (int)((a.n_new * (a.n_heads / a.c.n_kv) + kRows - 1) / kRows); }

// Strips of the longest rows that the tables can hold.
int64_t most_strips(const Attend &a) {
    int64_t most = a.c.capacity;
    if (a.window && a.window < most) most = a.window + kRows + kStrip - 1;  // of a tile's rows
    return (most + kStrip - 1) / kStrip;
}

int64_t items_of(const Attend &a) { return (int64_t)a.c.n_seqs * tiles_of(a) * a.c.n_kv; }

int wave_of(const Attend &a, const DeviceInfo &dev) {
    return dev.sm_count * shape_of(a.c.fmt_k, a.c.fmt_v, a.c.dim).ctas;
}

bool is_whole(const Attend &a, const DeviceInfo &dev) {
    return most_strips(a) <= whole_strips(items_of(a), wave_of(a, dev), cost_of(a));
}

// CTAs of a launch: one resident wave, or fewer when even the longest rows
// make less work than that.
int grid_of(const Attend &a, const DeviceInfo &dev) {
    const int wave = wave_of(a, dev);
    const int64_t items = items_of(a);
    if (items >= wave) return wave;  // also keeps the product in range
    if (is_whole(a, dev)) return (int)items;
    const int64_t shares = (items * (most_strips(a) + 1 + cost_of(a)) + kMinShare - 1) / kMinShare;
    return shares < wave ? (int)shares : wave;
}

size_t parts_bytes(int dim, int grid) {
    return ((size_t)2 * grid * part_floats(dim) * 4 + 255) & ~(size_t)255;
}

}  // namespace

}  // namespace attend

bool attend_supports(int dim) {
    return dim == 64 || dim == 96 || dim == 128 || dim == 192 || dim == 256;
}

size_t attend_workspace_bytes(const Attend &a, const DeviceInfo &dev) {
    if (attend::is_whole(a, dev)) return 0;
    const int grid = attend::grid_of(a, dev);
    return attend::parts_bytes(a.c.dim, grid) + sizeof(attend::Join) * grid;
}

cudaError_t launch_attend(const Attend &a, const DeviceInfo &dev, cudaStream_t s) {
    const int grid = attend::grid_of(a, dev);
    attend::AttendParams p;
    p.c = a.c;
    p.q = a.q;
    p.out = a.out;
    p.whole = attend::is_whole(a, dev);
    p.parts = static_cast<float *>(a.workspace);
    p.joins = p.whole ? nullptr
                      : reinterpret_cast<attend::Join *>(static_cast<uint8_t *>(a.workspace) +
                                                         attend::parts_bytes(a.c.dim, grid));
    p.q_stride = a.q_stride;
    p.out_stride = a.out_stride;
    p.window = a.window;
    p.n_new = (int)a.n_new;
    p.group = a.n_heads / a.c.n_kv;
    p.tiles = attend::tiles_of(a);
    p.all_tiles = a.c.n_seqs * p.tiles;
    p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
    p.vec = a.vec;
    p.item_cost = attend::cost_of(a);
    cudaError_t e;
    if (a.c.fmt_k == F_F16) e = attend::launch_f16(p, grid, s);
    else if (a.c.fmt_k == F_BF16) e = attend::launch_bf16(p, grid, s);
    else if (a.c.fmt_k == F_Q4_0) e = attend::launch_q4(p, grid, s);
    else if (a.c.fmt_v == F_Q4_0) e = attend::launch_q8q4(p, grid, s);
    else e = attend::launch_q8(p, grid, s);
    if (e != cudaSuccess || p.whole || grid < 2) return e;
    return attend::launch_programmatic(attend::attend_join_kernel, p, grid - 1, attend::kThreads, 0, s);
}

}  // namespace qmm
