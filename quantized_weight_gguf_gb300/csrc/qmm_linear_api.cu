// qmm_linear_api.cu -- C entry points of linear attention: checks of the
// arguments on the host, scratch, launches. Nothing here synchronises.
#include <cmath>

#include "qmm.h"
#include "qmm_linear.h"

namespace {

using qmm::set_error;

bool aligned(const void *p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

int check_rows(const char *name, const float *p, int64_t stride, int64_t width) {
    if (!p) return set_error(QMM_ERR_NULL, "%s is NULL", name);
    if (!aligned(p, 4)) return set_error(QMM_ERR_ALIGN, "%s must be 4-byte aligned", name);
    if (stride < width || stride > ((int64_t)1 << 32))
        return set_error(QMM_ERR_SHAPE, "%s: row stride %lld must be %lld (its heads' floats) to 2^32", name,
                         (long long)stride, (long long)width);
    return QMM_OK;
}

// Everything but the scratch; *empty: nothing to do.
int check_linear(const qmm_linear_args *a, qmm::Linear *l, bool *empty, bool pointers) {
    if (!a) return set_error(QMM_ERR_NULL, "args is NULL");
    if (a->n_new < 1) return set_error(QMM_ERR_SHAPE, "n_new %lld < 1", (long long)a->n_new);
    if (!qmm::linear_supports(a->dk, a->dv))
        return set_error(QMM_ERR_SHAPE, "dk %lld must be 32, 64, 96 or 128, and dv %lld a multiple of 32 up to 256",
                         (long long)a->dk, (long long)a->dv);
    if (a->n_heads < 1 || a->n_heads > 65536 || a->n_qk_heads < 1 || a->n_heads % a->n_qk_heads)
        return set_error(QMM_ERR_SHAPE, "n_heads %lld must be a multiple of n_qk_heads %lld up to 65536",
                         (long long)a->n_heads, (long long)a->n_qk_heads);
    if (a->n_seqs < 0 || a->n_seqs > ((int64_t)1 << 24) / a->n_heads)
        return set_error(QMM_ERR_SHAPE, "n_seqs * n_heads (%lld x %lld) must be at most 2^24", (long long)a->n_seqs,
                         (long long)a->n_heads);
    if (a->n_seqs && a->n_new > ((int64_t)1 << 30) / a->n_seqs)
        return set_error(QMM_ERR_SHAPE, "n_seqs %lld with %lld rows each: at most 2^30 rows", (long long)a->n_seqs,
                         (long long)a->n_new);
    if (a->decay_stride != 0 && (a->decay_stride < a->n_heads || a->decay_stride > ((int64_t)1 << 32)))
        return set_error(QMM_ERR_SHAPE, "decay: row stride %lld must be 0 (one per head) or %lld to 2^32",
                         (long long)a->decay_stride, (long long)a->n_heads);
    if (!std::isfinite(a->scale)) return set_error(QMM_ERR_SHAPE, "scale is not finite");
    if (a->flags) return set_error(QMM_ERR_SHAPE, "unknown flags 0x%x", a->flags);
    *empty = a->n_seqs == 0;
    if (pointers && !*empty) {
        int st = check_rows("q", a->q, a->q_stride, a->n_qk_heads * a->dk);
        if (st == QMM_OK) st = check_rows("k", a->k, a->k_stride, a->n_qk_heads * a->dk);
        if (st == QMM_OK) st = check_rows("v", a->v, a->v_stride, a->n_heads * a->dv);
        if (st == QMM_OK) st = check_rows("out", a->out, a->out_stride, a->n_heads * a->dv);
        if (st != QMM_OK) return st;
        if (!a->decay || !a->state || !a->state_out) return set_error(QMM_ERR_NULL, "decay, state or state_out is NULL");
        if (!aligned(a->decay, 4) || !aligned(a->lens, 4))
            return set_error(QMM_ERR_ALIGN, "decay and lens must be 4-byte aligned");
        if (!aligned(a->state, 16) || !aligned(a->state_out, 16))
            return set_error(QMM_ERR_ALIGN, "state and state_out must be 16-byte aligned");
    }
    l->q = a->q;
    l->k = a->k;
    l->v = a->v;
    l->decay = a->decay;
    l->state = a->state;
    l->state_out = a->state_out;
    l->out = a->out;
    l->lens = a->lens;
    l->q_stride = a->q_stride;
    l->k_stride = a->k_stride;
    l->v_stride = a->v_stride;
    l->out_stride = a->out_stride;
    l->decay_stride = a->decay_stride;
    l->n_new = a->n_new;
    l->n_seqs = (int)a->n_seqs;
    l->n_heads = (int)a->n_heads;
    l->n_qk = (int)a->n_qk_heads;
    l->dk = (int)a->dk;
    l->dv = (int)a->dv;
    l->scale = a->scale;
    l->vec = aligned(a->q, 16) && aligned(a->k, 16) && aligned(a->v, 16) && a->q_stride % 4 == 0 &&
             a->k_stride % 4 == 0 && a->v_stride % 4 == 0;
    l->workspace = nullptr;
    return QMM_OK;
}

}  // namespace

extern "C" {

size_t qmm_linear_attend_workspace_bytes(const qmm_linear_args *a) {
    qmm::Linear l;
    bool empty = false;
    if (check_linear(a, &l, &empty, false) != QMM_OK || empty) return 0;
    qmm::DeviceInfo *dev = nullptr;
    if (qmm::current_device(&dev) != QMM_OK) return 0;
    return qmm::linear_workspace_bytes(l, *dev);
}

int qmm_linear_attend(const qmm_linear_args *a) {
    set_error(QMM_OK, "%s", "");
    qmm::Linear l;
    bool empty = false;
    int st = check_linear(a, &l, &empty, true);
    if (st != QMM_OK || empty) return st;
    qmm::DeviceInfo *dev = nullptr;
    st = qmm::current_device(&dev);
    if (st != QMM_OK) return st;
    const size_t need = qmm::linear_workspace_bytes(l, *dev);
    l.workspace = a->workspace;
    if (a->workspace) {
        if (a->workspace_bytes < need)
            return set_error(QMM_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", a->workspace_bytes, need);
        if (!aligned(a->workspace, 256)) return set_error(QMM_ERR_ALIGN, "workspace must be 256-byte aligned");
    } else if (need) {
        st = qmm::scratch_of_library(need, &l.workspace);
        if (st != QMM_OK) return st;
    }
    const cudaError_t e = qmm::launch_linear(l, *dev, static_cast<cudaStream_t>(a->stream));
    return e == cudaSuccess ? QMM_OK : set_error(QMM_ERR_CUDA, "linear attention launch: %s", cudaGetErrorString(e));
}

}  // extern "C"
