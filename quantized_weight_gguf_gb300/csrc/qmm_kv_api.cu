// qmm_kv_api.cu -- C entry points of the paged key-value cache: checks of the
// arguments on the host, scratch, launches. Nothing here synchronises.
#include <cmath>

#include "qmm.h"
#include "qmm_kv_launch.h"

namespace {

using qmm::set_error;

bool aligned(const void *p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

bool format_ok(int f) { return f == QMM_F16 || f == QMM_BF16 || f == QMM_Q8_0 || f == QMM_Q4_0; }

constexpr int64_t kMaxPage = 65536, kMaxHeads = 65536, kMaxDim = 512;
constexpr int64_t kMaxRows = (int64_t)1 << 30;

// Formats, page size, head count and head_dim of a cache.
int check_geometry(int fk, int fv, int64_t page, int64_t heads, int64_t dim) {
    if (!format_ok(fk) || !format_ok(fv))
        return set_error(QMM_ERR_FORMAT, "cache formats are F16, BF16, Q8_0 and Q4_0 (got %d, %d)", fk, fv);
    if (fk != fv && !(fk == QMM_Q8_0 && fv == QMM_Q4_0))
        return set_error(QMM_ERR_FORMAT,
                         "K and V have one format, or K Q8_0 and V Q4_0 (got %d, %d)", fk, fv);
    if (page < 16 || page > kMaxPage || page % 16)
        return set_error(QMM_ERR_SHAPE, "page_size %lld must be a multiple of 16 up to %lld",
                         (long long)page, (long long)kMaxPage);
    if (heads < 1 || heads > kMaxHeads)
        return set_error(QMM_ERR_SHAPE, "n_kv_heads %lld must be 1 to %lld", (long long)heads,
                         (long long)kMaxHeads);
    if (dim < 32 || dim > kMaxDim || dim % 32)
        return set_error(QMM_ERR_SHAPE, "head_dim %lld must be a multiple of 32 up to %lld",
                         (long long)dim, (long long)kMaxDim);
    return QMM_OK;
}

size_t page_bytes(int fk, int fv, int64_t page, int64_t heads, int64_t dim) {
    return (size_t)heads * (size_t)(page / 16) * (size_t)qmm::kv_strip_bytes(fk, fv, (int)dim);
}

// The cache of a call with `rows` rows per sequence: its geometry, and its
// pointers unless only sizes are asked for; fills the kernels' view but for
// the error word.
int check_cache(const qmm_kv_cache &c, int64_t rows, qmm::KvView *v, bool pointers = true) {
    int st = check_geometry(c.fmt_k, c.fmt_v, c.page_size, c.n_kv_heads, c.head_dim);
    if (st != QMM_OK) return st;
    if (c.n_pages < 0 || c.n_pages > INT32_MAX)
        return set_error(QMM_ERR_SHAPE, "n_pages %lld must be 0 to 2^31 - 1", (long long)c.n_pages);
    if (c.n_seqs < 0 || rows < 0 || (c.n_seqs > 0 && rows > kMaxRows / c.n_seqs))
        return set_error(QMM_ERR_SHAPE, "n_seqs %lld with %lld rows each: at most 2^30 rows",
                         (long long)c.n_seqs, (long long)rows);
    if (c.max_pages < 0 || c.max_pages > INT32_MAX || c.table_stride < c.max_pages)
        return set_error(QMM_ERR_SHAPE, "max_pages %lld must be 0 to 2^31 - 1 and table_stride %lld no less",
                         (long long)c.max_pages, (long long)c.table_stride);
    const size_t pb = page_bytes(c.fmt_k, c.fmt_v, c.page_size, c.n_kv_heads, c.head_dim);
    size_t all = 0;
    if (__builtin_mul_overflow(pb, (size_t)c.n_pages, &all) || all > (size_t)INT64_MAX)
        return set_error(QMM_ERR_SHAPE, "n_pages %lld of %zu bytes overflow", (long long)c.n_pages, pb);
    if (c.pages_len != 0 && c.pages_len != all)
        return set_error(QMM_ERR_SIZE, "cache bytes %zu != n_pages * page bytes = %zu", c.pages_len, all);
    if (pointers && c.n_seqs > 0 && rows > 0) {
        if (!c.lens || (c.max_pages > 0 && !c.page_table) || (c.n_pages > 0 && !c.pages))
            return set_error(QMM_ERR_NULL, "pages, page_table or lens is NULL");
        if (!aligned(c.pages, 16)) return set_error(QMM_ERR_ALIGN, "pages must be 16-byte aligned");
        if (!aligned(c.page_table, 4) || !aligned(c.lens, 4))
            return set_error(QMM_ERR_ALIGN, "page_table and lens must be 4-byte aligned");
    }
    v->pages = static_cast<uint8_t *>(c.pages);
    v->table = c.page_table;
    v->lens = c.lens;
    v->head_bytes = (int64_t)(pb / (size_t)c.n_kv_heads);
    v->table_stride = c.table_stride;
    v->n_pages = c.n_pages;
    const int64_t cap = c.max_pages * c.page_size;
    v->capacity = cap < INT32_MAX - 16 ? cap : (INT32_MAX - 16) / 16 * 16;
    v->fmt_k = c.fmt_k;
    v->fmt_v = c.fmt_v;
    v->n_kv = (int)c.n_kv_heads;
    v->dim = (int)c.head_dim;
    v->page_size = (int)c.page_size;
    v->strip_bytes = qmm::kv_strip_bytes(c.fmt_k, c.fmt_v, v->dim);
    v->v_off = qmm::kv_half_bytes(c.fmt_k, v->dim);
    v->n_seqs = (int)c.n_seqs;
    v->err = nullptr;
    return QMM_OK;
}

int check_rows(const char *name, const float *p, int64_t stride, int64_t width) {
    if (!p) return set_error(QMM_ERR_NULL, "%s is NULL", name);
    if (!aligned(p, 4)) return set_error(QMM_ERR_ALIGN, "%s must be 4-byte aligned", name);
    if (stride < width || stride > ((int64_t)1 << 32))
        return set_error(QMM_ERR_SHAPE, "%s: row stride %lld must be %lld (its heads' floats) to 2^32", name,
                         (long long)stride, (long long)width);
    return QMM_OK;
}

bool vec_rows(const float *p, int64_t stride) { return aligned(p, 16) && stride % 4 == 0; }

// Everything about an attention call but its scratch; *empty: nothing to do.
int check_attend(const qmm_attend_args *a, qmm::Attend *l, bool *empty, bool pointers) {
    if (!a) return set_error(QMM_ERR_NULL, "args is NULL");
    if (a->n_new < 1) return set_error(QMM_ERR_SHAPE, "n_new %lld < 1", (long long)a->n_new);
    int st = check_cache(a->cache, a->n_new, &l->c, pointers);
    if (st != QMM_OK) return st;
    if (!qmm::attend_supports(l->c.dim))
        return set_error(QMM_ERR_UNSUPPORTED, "attention takes head_dim 64, 96, 128, 192 or 256 (got %d)",
                         l->c.dim);
    if (a->n_heads < 1 || a->n_heads % a->cache.n_kv_heads || a->n_heads > kMaxHeads)
        return set_error(QMM_ERR_SHAPE, "n_heads %lld must be a multiple of n_kv_heads %lld up to %lld",
                         (long long)a->n_heads, (long long)a->cache.n_kv_heads, (long long)kMaxHeads);
    if (a->cache.n_seqs * a->n_new > INT32_MAX / a->n_heads)
        return set_error(QMM_ERR_SHAPE, "n_seqs * n_new * n_heads must be below 2^31");
    if (!std::isfinite(a->scale)) return set_error(QMM_ERR_SHAPE, "scale is not finite");
    if (a->window < 0) return set_error(QMM_ERR_SHAPE, "window %lld < 0", (long long)a->window);
    if (a->flags) return set_error(QMM_ERR_SHAPE, "unknown flags 0x%x", a->flags);
    *empty = a->cache.n_seqs == 0;
    if (pointers && !*empty) {
        const int64_t width = a->n_heads * l->c.dim;
        st = check_rows("q", a->q, a->q_stride, width);
        if (st == QMM_OK) st = check_rows("out", a->out, a->out_stride, width);
        if (st != QMM_OK) return st;
    }
    l->q = a->q;
    l->out = a->out;
    l->q_stride = a->q_stride;
    l->out_stride = a->out_stride;
    l->n_new = a->n_new;
    l->window = a->window;
    l->n_heads = (int)a->n_heads;
    l->scale = a->scale;
    l->vec = vec_rows(a->q, a->q_stride) && vec_rows(a->out, a->out_stride);
    l->workspace = nullptr;
    return QMM_OK;
}

int cuda_fail(cudaError_t e, const char *what) {
    return set_error(QMM_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

}  // namespace

extern "C" {

size_t qmm_kv_page_bytes(int fmt_k, int fmt_v, int64_t page_size, int64_t n_kv_heads, int64_t head_dim) {
    if (check_geometry(fmt_k, fmt_v, page_size, n_kv_heads, head_dim) != QMM_OK) return 0;
    return page_bytes(fmt_k, fmt_v, page_size, n_kv_heads, head_dim);
}

int qmm_kv_append(const qmm_kv_append_args *a) {
    set_error(QMM_OK, "%s", "");
    if (!a) return set_error(QMM_ERR_NULL, "args is NULL");
    if (a->n_new < 1) return set_error(QMM_ERR_SHAPE, "n_new %lld < 1", (long long)a->n_new);
    qmm::KvAppend l;
    int st = check_cache(a->cache, a->n_new, &l.c);
    if (st != QMM_OK) return st;
    const int64_t width = (int64_t)l.c.n_kv * l.c.dim;
    if (a->q && (a->n_heads < 1 || a->n_heads > kMaxHeads))
        return set_error(QMM_ERR_SHAPE, "n_heads %lld must be 1 to %lld", (long long)a->n_heads,
                         (long long)kMaxHeads);
    if (a->rope) {
        if (a->n_rot < 8 || a->n_rot % 8 || a->n_rot > l.c.dim)
            return set_error(QMM_ERR_SHAPE, "n_rot %lld must be a multiple of 8 up to head_dim %d",
                             (long long)a->n_rot, l.c.dim);
        if (a->rope_len < 0) return set_error(QMM_ERR_SHAPE, "rope_len %lld < 0", (long long)a->rope_len);
        if (a->rope_style != QMM_ROPE_HALF && a->rope_style != QMM_ROPE_PAIRS)
            return set_error(QMM_ERR_FORMAT, "unknown rope_style %d", a->rope_style);
        if (!aligned(a->rope, 16)) return set_error(QMM_ERR_ALIGN, "rope must be 16-byte aligned");
    }
    if (a->flags) return set_error(QMM_ERR_SHAPE, "unknown flags 0x%x", a->flags);
    if (a->cache.n_seqs == 0) return QMM_OK;
    st = check_rows("k", a->k, a->k_stride, width);
    if (st == QMM_OK) st = check_rows("v", a->v, a->v_stride, width);
    if (st == QMM_OK && a->q) st = check_rows("q", a->q, a->q_stride, a->n_heads * l.c.dim);
    if (st == QMM_OK && a->q) st = check_rows("q_out", a->q_out, a->q_out_stride, a->n_heads * l.c.dim);
    if (st != QMM_OK) return st;
    if (a->q && a->q_out == a->q && a->q_stride != a->q_out_stride)
        return set_error(QMM_ERR_SHAPE, "q_out is q: their row strides must be the same");
    qmm::DeviceInfo *dev = nullptr;
    st = qmm::current_device(&dev);
    if (st != QMM_OK) return st;
    l.c.err = dev->err;
    l.k = a->k;
    l.v = a->v;
    l.q = a->q;
    l.q_out = a->q_out;
    l.rope = a->rope;
    l.k_stride = a->k_stride;
    l.v_stride = a->v_stride;
    l.q_stride = a->q ? a->q_stride : 0;
    l.q_out_stride = a->q ? a->q_out_stride : 0;
    l.n_new = a->n_new;
    l.rope_len = a->rope_len;
    l.n_heads = a->q ? (int)a->n_heads : 0;
    l.n_rot = (int)a->n_rot;
    l.style = a->rope_style;
    l.vec = vec_rows(a->k, a->k_stride) && vec_rows(a->v, a->v_stride) &&
            (!a->q || (vec_rows(a->q, a->q_stride) && vec_rows(a->q_out, a->q_out_stride)));
    cudaError_t e = qmm::launch_kv_append(l, *dev, static_cast<cudaStream_t>(a->stream));
    return e == cudaSuccess ? QMM_OK : cuda_fail(e, "cache append launch");
}

int qmm_kv_read(const qmm_kv_read_args *a) {
    set_error(QMM_OK, "%s", "");
    if (!a) return set_error(QMM_ERR_NULL, "args is NULL");
    if (a->first < -1 || a->first > INT32_MAX)
        return set_error(QMM_ERR_RANGE, "first %lld must be -1 to 2^31 - 1", (long long)a->first);
    if (a->flags) return set_error(QMM_ERR_SHAPE, "unknown flags 0x%x", a->flags);
    qmm::KvRead l;
    int st = check_cache(a->cache, a->count, &l.c);
    if (st != QMM_OK) return st;
    if (a->cache.n_seqs == 0 || a->count == 0 || (!a->k && !a->v)) return QMM_OK;
    if (!aligned(a->k, 4) || !aligned(a->v, 4))
        return set_error(QMM_ERR_ALIGN, "k and v must be 4-byte aligned");
    qmm::DeviceInfo *dev = nullptr;
    st = qmm::current_device(&dev);
    if (st != QMM_OK) return st;
    l.c.err = dev->err;
    l.k = a->k;
    l.v = a->v;
    l.first = a->first;
    l.count = a->count;
    l.vec = aligned(a->k, 16) && aligned(a->v, 16);
    cudaError_t e = qmm::launch_kv_read(l, *dev, static_cast<cudaStream_t>(a->stream));
    return e == cudaSuccess ? QMM_OK : cuda_fail(e, "cache read launch");
}

size_t qmm_attend_workspace_bytes(const qmm_attend_args *a) {
    qmm::Attend l;
    bool empty = false;
    if (check_attend(a, &l, &empty, false) != QMM_OK || empty) return 0;
    qmm::DeviceInfo *dev = nullptr;
    if (qmm::current_device(&dev) != QMM_OK) return 0;
    return qmm::attend_workspace_bytes(l, *dev);
}

int qmm_attend(const qmm_attend_args *a) {
    set_error(QMM_OK, "%s", "");
    qmm::Attend l;
    bool empty = false;
    int st = check_attend(a, &l, &empty, true);
    if (st != QMM_OK || empty) return st;
    qmm::DeviceInfo *dev = nullptr;
    st = qmm::current_device(&dev);
    if (st != QMM_OK) return st;
    l.c.err = dev->err;
    const size_t need = qmm::attend_workspace_bytes(l, *dev);
    l.workspace = a->workspace;
    if (a->workspace) {
        if (a->workspace_bytes < need)
            return set_error(QMM_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", a->workspace_bytes, need);
        if (!aligned(a->workspace, 256))
            return set_error(QMM_ERR_ALIGN, "workspace must be 256-byte aligned");
    } else if (need) {
        st = qmm::scratch_of_library(need, &l.workspace);
        if (st != QMM_OK) return st;
    }
    cudaError_t e = qmm::launch_attend(l, *dev, static_cast<cudaStream_t>(a->stream));
    return e == cudaSuccess ? QMM_OK : cuda_fail(e, "attention launch");
}

}  // extern "C"
