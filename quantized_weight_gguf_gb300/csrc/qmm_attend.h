// qmm_attend.h -- parameters, work division and partial results of the
// attention kernels (qmm_attend_kernel.cuh: the strips; qmm_attend.cu: the join of
// split items and the host side).
#pragma once

#include "qmm_kv.cuh"
#include "qmm_kv_launch.h"

namespace qmm {

namespace attend {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 8;            // query rows of an item
constexpr int kFixedBytes = 1024;   // barriers, flags, states (see attend_kernel)

// How the shared memory of an SM (228 KB, of which the system takes 1 KB per
// CTA) is divided for a pair of formats and a head_dim: resident CTAs, and
// each warp's ring. A strip is one copy, or two (K, then V) where whole strips
// would leave a ring of this size fewer than four slots (two pairs). Strips
// are taken up to four at a time, which share the waits, the softmax's checks
// and the additions to the running sums: 16 sequences with 16 kv heads of 64
// dims in Q4_0 take 45.9 us, 50.0 with two at a time; one at a time instead of
// two costs 1 to 4 % more.
struct Shape {
    int q_bytes;     // query fragments: 16 bytes per lane and 16 dims, 24 for bf16's third term
    int units;       // copies per strip
    int slot_bytes, slots;
    int step;        // strips taken at a time: half the ring's slots (copies stay ahead), as far as 1, 2 or 4
    int ring_bytes;  // of one warp; also holds its [kRows][dim + 4] results at an item's end
    int smem, ctas;
};
constexpr int kMaxSlots = 8;
__host__ __device__ constexpr Shape shape_for(int fk, int fv, int dim, int ctas) {
    Shape s = {};
    s.ctas = ctas;
    s.q_bytes = dim / 16 * 32 * (fk == F_BF16 ? 24 : 16);
    const int budget = (228 * 1024 / ctas - 1024 - s.q_bytes - kFixedBytes) / kWarps / 16 * 16;
    const int k = kv_half_bytes(fk, dim), v = kv_half_bytes(fv, dim);
    s.units = budget / (k + v) >= 4 ? 1 : 2;
    s.slot_bytes = s.units == 1 ? k + v : k > v ? k : v;
    s.slots = budget / s.slot_bytes < kMaxSlots ? budget / s.slot_bytes : kMaxSlots;
    s.step = s.slots >= 8 ? 4 : s.slots >= 4 ? 2 : 1;
    s.slots -= s.slots % s.step;
    const int merge = (kRows * (dim + 4) * 4 + 127) / 128 * 128;
    s.ring_bytes = s.slots * s.slot_bytes > merge ? s.slots * s.slot_bytes : merge;
    s.smem = kFixedBytes + s.q_bytes + kWarps * s.ring_bytes;
    return s;
}
// CTAs of 128 threads per SM: four up to 64 dims (128 registers a thread),
// three above (168; with four at 96 and 128 dims 64 F16 sequences took 186 us
// instead of 183, 48 Q8_0 ones 67 instead of 65); fewer where their rings would
// have less than two slots.
__host__ __device__ constexpr Shape shape_of(int fk, int fv, int dim) {
    int ctas = dim <= 64 ? 4 : 3;
    while (ctas > 1 && shape_for(fk, fv, dim, ctas).slots < 2) --ctas;
    return shape_for(fk, fv, dim, ctas);
}

// What an item costs a CTA beside its strips, in strips: first copies on their
// way, query rows converted, the warps' results joined; about 5 us, where a
// strip takes the CTA its share of an SM's 45 GB/s (at least 0.25 us: the
// arithmetic on a strip of Q4_0). With 4 strips for every format, CTAs with
// several items finished 6 us (of 63) after the others on 48 ragged sequences;
// with 3 us instead of 5 they take 1 us longer, with 4 or 6.5 the same.
__host__ __device__ constexpr int item_cost_of(int fk, int fv, int dim, int ctas) {
    const int ns = kv_strip_bytes(fk, fv, dim) * ctas / 45;
    return 5000 / (ns > 250 ? ns : 250);
}

// Strips (and item costs) below which a CTA's share is not cut further: two
// strips per warp.
constexpr int kMinShare = 8;

// Where no row can see more strips than a few item costs (by the tables' size
// and the window), items are not split: CTA c takes items c, c + grid, ... as
// they are, and no join is launched. 16 sequences of up to 400 positions over 8
// kv heads of 128 in Q8_0 take 7.4 us so, 11.8 split, 96 of them 22.4 and 27.4.
// The limit is 2 costs (one sequence of 400 positions over 8 kv heads of 256 in
// Q8_0: 13.8 us whole, 11.5 split), 4 where items are an eighth of the CTAs or
// more (96 sequences of it: 37 whole, 45 split; 800 positions are about equal).
__host__ __device__ constexpr int whole_strips(int64_t items, int wave, int item_cost) {
    return (8 * items >= wave ? 4 : 2) * item_cost;
}

// A split item, written by each CTA whose share ends inside one: the CTAs
// first .. first + parts - 1 hold its partial results.
struct Join {
    int parts;   // 0: none
    int first;
    int seq, head, tile;
};

struct AttendParams {
    KvView c;
    const float *q;
    float *out;
    float *parts;      // [2 grid][part_floats]: results of a share's first (0) and last (1) item
    Join *joins;       // [grid]
    int64_t q_stride, out_stride, window;
    int n_new, group;        // new positions per sequence, query heads per kv head
    int tiles, all_tiles;    // kRows of the n_new x group query rows of a sequence and kv head; of all sequences
    int item_cost;           // see item_cost_of
    float scale_log2;  // scale * log2(e)
    bool vec;
    bool whole;        // items are not split (see whole_strips); then parts and joins are not used
};

// a partial result: [kRows] maxima, [kRows] totals, [kRows][dim] sums
__host__ __device__ constexpr int part_floats(int dim) { return kRows * (dim + 2); }

// The positions [lo, hi) that the row of position pos sees. Both ends grow with
// pos, also where nothing is seen (before the sequence's start lo = hi = 0, with
// the window past the tables' end lo = hi = capacity), so that a tile's ends are
// its first row's lo and its last row's hi.
struct Range {
    int lo, hi;
};
__device__ __forceinline__ int within(int64_t pos, int64_t capacity) {
    return (int)(pos < 0 ? 0 : pos < capacity ? pos : capacity);
}
__device__ __forceinline__ Range seen_from(const AttendParams &a, int64_t pos) {
    Range x;
    x.lo = a.window ? within(pos + 1 - a.window, a.c.capacity) : 0;
    x.hi = within(pos + 1, a.c.capacity);
    return x;
}

// Query row x of a sequence and kv head is new position x / group and head
// x % group of the kv head's; x past the last counts as the last. MANY: there
// are several new positions (see launch_one).
template <bool MANY>
__device__ __forceinline__ int new_of(const AttendParams &a, int x) {
    return MANY ? min(x / a.group, a.n_new - 1) : 0;
}

// Tile r of all sequences' tiles: its sequence, the positions that one of its
// rows sees, and their strips. pos0: the sequence's first new position.
struct TileRange {
    int seq, tile, lo, hi, first, strips;
    int64_t pos0;
};
template <bool MANY>
__device__ __forceinline__ TileRange tile_range(const AttendParams &a, int r) {
    TileRange x;
    x.seq = a.tiles == 1 ? r : r / a.tiles;
    x.tile = r - x.seq * a.tiles;
    const int held = __ldg(a.c.lens + x.seq);
    x.pos0 = (int64_t)(held < 0 ? 0 : held) - a.n_new;
    const int64_t last = x.pos0 + new_of<MANY>(a, x.tile * kRows + kRows - 1);
    if (last + 1 > a.c.capacity) record_error(a.c.err, DERR_BAD_PAGE);
    const Range l = seen_from(a, last);
    x.lo = MANY ? seen_from(a, x.pos0 + new_of<MANY>(a, x.tile * kRows)).lo : l.lo;
    x.hi = l.hi;
    x.first = x.lo / kStrip;
    x.strips = x.hi > x.lo ? (x.hi + kStrip - 1) / kStrip - x.first : 0;
    return x;
}
// An item of no strips counts as one that holds nothing, so that its output
// is written like any other.
__device__ __forceinline__ int item_strips(const TileRange &x) { return x.strips > 0 ? x.strips : 1; }
__device__ __forceinline__ int item_weight(const AttendParams &a, const TileRange &x) {
    return x.strips > 0 ? x.strips + a.item_cost : 1 + a.item_cost / 4;
}

// Where a CTA's share begins.
struct WorkSearch {
    long long sum[kWarps];
    long long base;
    int tile;
};
struct Work {
    int64_t at, end;     // the share, in strips and item costs of all items end to end; of whole items:
                         // the next item and the number of all
    int64_t total;
    int shares;          // CTAs that have one
    int tile;            // the tile of all sequences' that `at` is in
    int64_t base;        // and where that begins
};

// a / b of non-negative numbers; a 64-bit division takes an order of magnitude
// longer than a 32-bit one, and nearly all numbers here fit
__device__ __forceinline__ int64_t quotient(int64_t a, int b) {
    return a >> 32 ? a / b : (int64_t)((unsigned)a / (unsigned)b);
}

// The share of CTA `cta`; false when it has none. Every thread of the block
// calls it. The tiles' weights are summed by the block's threads, a run of
// tiles each: a few loads for a decoding batch.
template <bool MANY>
__device__ __forceinline__ bool find_work(const AttendParams &a, int cta, WorkSearch *sh, Work &w) {
    if (a.whole) {
        w.at = cta;
        w.end = (int64_t)a.all_tiles * a.c.n_kv;
        return w.at < w.end;
    }
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.all_tiles + kThreads - 1) / kThreads;
    const int r0 = min(tid * per, a.all_tiles), r1 = min(r0 + per, a.all_tiles);
    int64_t mine = 0;
    for (int r = r0; r < r1; ++r) mine += item_weight(a, tile_range<MANY>(a, r));
    mine *= a.c.n_kv;
    int64_t upto = mine;  // inclusive sums over the warp, then over the warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(~0u, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) sh->sum[warp] = upto;
    __syncthreads();
    int64_t before = 0, total = 0;
    for (int k = 0; k < kWarps; ++k) {
        if (k < warp) before += sh->sum[k];
        total += sh->sum[k];
    }
    w.total = total;
    const int64_t most = (total + kMinShare - 1) / kMinShare;
    w.shares = most < (int64_t)gridDim.x ? (int)most : (int)gridDim.x;
    if (cta >= w.shares) return false;
    w.at = quotient((int64_t)cta * total, w.shares);
    w.end = quotient((int64_t)(cta + 1) * total, w.shares);
    int64_t base = before + upto - mine;
    if (w.at >= base && w.at < base + mine) {
        for (int r = r0; r < r1; ++r) {
            const int64_t n = (int64_t)item_weight(a, tile_range<MANY>(a, r)) * a.c.n_kv;
            if (w.at < base + n) {
                sh->tile = r;
                sh->base = base;
                break;
            }
            base += n;
        }
    }
    __syncthreads();
    w.tile = sh->tile;
    w.base = sh->base;
    return true;
}

// The CTA whose share holds position v of the strips laid end to end.
__device__ __forceinline__ int share_of(const Work &w, int64_t v) {
    // the last c with c total < (v + 1) shares, from an estimate that is off by
    // one at most (shares < 2^11)
    const int64_t limit = (v + 1) * w.shares;
    int c = (int)((float)limit / (float)w.total);
    while (c * w.total >= limit) --c;
    while ((c + 1) * w.total < limit) ++c;
    return c;
}

// The next item of a share: which query rows, which positions, and the part
// [begin, end) of its strips that the share holds.
struct Item {
    int64_t base;        // where its strips begin
    int64_t pos0;        // the sequence's first new position
    int seq, head, tile; // sequence, kv head, tile of its query rows
    int lo, hi, first;   // positions that one of the rows sees, first strip
    int strips, begin, end;
    bool live;           // has strips at all
};
template <bool MANY>
__device__ __forceinline__ bool next_item(const AttendParams &a, Work &w, Item &it) {
    while (w.at < w.end) {
        if (a.whole) w.tile = (int)(w.at / a.c.n_kv);
        const TileRange x = tile_range<MANY>(a, w.tile);
        const int n = item_strips(x);
        if (a.whole) {
            it.head = (int)(w.at - (int64_t)w.tile * a.c.n_kv);
            it.begin = 0;
            it.end = n;
            w.at += gridDim.x;
        } else {
            const int cost = item_weight(a, x);
            const int64_t all = (int64_t)cost * a.c.n_kv;
            if (w.at >= w.base + all) {
                w.base += all;
                ++w.tile;
                continue;
            }
            it.head = (int)quotient(w.at - w.base, cost);
            it.base = w.base + (int64_t)it.head * cost;
            const int64_t stop = it.base + cost < w.end ? it.base + cost : w.end;
            it.begin = (int)(w.at - it.base);
            it.end = stop - it.base < n ? (int)(stop - it.base) : n;
            w.at = stop;
            if (it.begin >= it.end) continue;  // only of the item's cost
        }
        it.pos0 = x.pos0;
        it.seq = x.seq;
        it.tile = x.tile;
        it.lo = x.lo;
        it.hi = x.hi;
        it.first = x.first;
        it.strips = n;
        it.live = x.strips > 0;
        return true;
    }
    return false;
}

__device__ __forceinline__ Join make_join(const AttendParams &, const Work &w, const Item &it) {
    Join x;
    x.first = share_of(w, it.base);
    x.parts = share_of(w, it.base + it.strips - 1) - x.first + 1;
    x.seq = it.seq;
    x.head = it.head;
    x.tile = it.tile;
    return x;
}

// Row `row` of a tile (it: an item or a join): whether there is one, and its
// offset among q's (or out's) rows of `stride` floats.
template <bool MANY, class T>
__device__ __forceinline__ bool row_offset(const AttendParams &a, const T &it, int row, int dim,
                                           int64_t stride, int64_t &at) {
    const int x = it.tile * kRows + row, i = new_of<MANY>(a, x);
    at = ((int64_t)it.seq * a.n_new + i) * stride + ((int64_t)it.head * a.group + x - i * a.group) * dim;
    return x < a.n_new * a.group;
}

// out = sum / total: 0 where nothing was seen.
template <bool MANY, class T>
__device__ __forceinline__ void put_out(const AttendParams &a, const T &it, int row, int d, int dim,
                                        float4 sum, float total) {
    int64_t at;
    if (!row_offset<MANY>(a, it, row, dim, a.out_stride, at)) return;
    float *o = a.out + at + d;
    const float f = total == 0.0f ? 0.0f : __fdiv_rn(1.0f, total);
    const float4 v = make_float4(sum.x * f, sum.y * f, sum.z * f, sum.w * f);
    if (a.vec) {
        *reinterpret_cast<float4 *>(o) = v;
    } else {
        o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w;
    }
}

// Launches `kernel` as a programmatic dependent of the kernel before it in
// the stream (which it waits for before it reads or writes anything).
template <class P>
cudaError_t launch_programmatic(void (*kernel)(P), const P &p, int grid, int threads, size_t smem,
                                cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// one translation unit per pair of formats
cudaError_t launch_f16(const AttendParams &a, int grid, cudaStream_t s);
cudaError_t launch_bf16(const AttendParams &a, int grid, cudaStream_t s);
cudaError_t launch_q8(const AttendParams &a, int grid, cudaStream_t s);
cudaError_t launch_q4(const AttendParams &a, int grid, cudaStream_t s);
cudaError_t launch_q8q4(const AttendParams &a, int grid, cudaStream_t s);

}  // namespace attend

}  // namespace qmm
