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
// every call.
__global__ void __launch_bounds__(kThreads) attend_join_kernel(const AttendParams a) {
    pdl_wait_prev();
    pdl_launch_dependents();
    const Join x = a.joins[blockIdx.x];
    if (x.parts < 2) return;
    const int dim = a.c.dim, quads = kRows * dim / 4, blocks = x.parts - 1;
    const int me = (int)blockIdx.x - x.first;
    const int f0 = (int)((int64_t)me * quads / blocks), f1 = (int)((int64_t)(me + 1) * quads / blocks);
    if (f0 >= f1) return;
    // `wide` neighbouring lanes share a value and take its parts in turn
    int wide = 1;
    while (wide < 32 && 2 * wide * (f1 - f0) <= kThreads) wide *= 2;
    const int l = threadIdx.x % wide;
    for (int f = f0 + threadIdx.x / wide; f - (int)threadIdx.x / wide < f1; f += kThreads / wide) {
        const int row = f / (dim / 4), d = (f - row * (dim / 4)) * 4;
        float m = -INFINITY, total = 0.0f;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (f < f1) {
#pragma unroll 4
            for (int k = l; k < x.parts; k += wide) {
                // the first part is its CTA's last item, the others their CTAs' first
                const float *p = a.parts + (int64_t)(2 * (x.first + k) + (k == 0)) * part_floats(dim);
                const float mk = p[row], lk = p[kRows + row];
                const float4 v = *reinterpret_cast<const float4 *>(p + 2 * kRows + row * dim + d);
                if (mk == -INFINITY) continue;
                const float top = fmaxf(m, mk);
                const float fo = exp2f(m - top), fn = exp2f(mk - top);
                total = total * fo + lk * fn;
                s.x = s.x * fo + v.x * fn;
                s.y = s.y * fo + v.y * fn;
                s.z = s.z * fo + v.z * fn;
                s.w = s.w * fo + v.w * fn;
                m = top;
            }
        }
        for (int o = 1; o < wide; o <<= 1) {
            const float mo = __shfl_xor_sync(~0u, m, o), to = __shfl_xor_sync(~0u, total, o);
            const float4 so = make_float4(__shfl_xor_sync(~0u, s.x, o), __shfl_xor_sync(~0u, s.y, o),
                                          __shfl_xor_sync(~0u, s.z, o), __shfl_xor_sync(~0u, s.w, o));
            const float top = fmaxf(m, mo);
            const float fa = m == -INFINITY ? 0.0f : exp2f(m - top);
            const float fb = mo == -INFINITY ? 0.0f : exp2f(mo - top);
            total = total * fa + to * fb;
            s.x = s.x * fa + so.x * fb;
            s.y = s.y * fa + so.y * fb;
            s.z = s.z * fa + so.z * fb;
            s.w = s.w * fa + so.w * fb;
            m = top;
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

// CTAs of a launch: one resident wave, or fewer when even the longest rows
// that the tables can hold make less work than that.
int grid_of(const Attend &a, const DeviceInfo &dev) {
    const int wave = dev.sm_count * shape_of(a.c.fmt_k, a.c.fmt_v, a.c.dim).ctas;
    int64_t most = a.c.capacity;
    if (a.window && a.window < most) most = a.window + kRows + kStrip - 1;  // of a tile's rows
    const int64_t strips = (most + kStrip - 1) / kStrip + 1;
    const int64_t items = (int64_t)a.c.n_seqs * tiles_of(a) * a.c.n_kv;
    if (items >= wave) return wave;  // also keeps the product in range
    const int64_t shares = (items * (strips + cost_of(a)) + kMinShare - 1) / kMinShare;
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
    const int grid = attend::grid_of(a, dev);
    return attend::parts_bytes(a.c.dim, grid) + sizeof(attend::Join) * grid;
}

cudaError_t launch_attend(const Attend &a, const DeviceInfo &dev, cudaStream_t s) {
    const int grid = attend::grid_of(a, dev);
    attend::AttendParams p;
    p.c = a.c;
    p.q = a.q;
    p.out = a.out;
    p.parts = static_cast<float *>(a.workspace);
    p.joins = reinterpret_cast<attend::Join *>(static_cast<uint8_t *>(a.workspace) +
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
    if (e != cudaSuccess || grid < 2) return e;
    return attend::launch_programmatic(attend::attend_join_kernel, p, grid - 1, attend::kThreads, 0, s);
}

}  // namespace qmm
