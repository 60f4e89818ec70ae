// qmm_experts_api.cu -- C entry points of the choice of experts and of their
// feed-forward network: checks of the arguments on the host, scratch, launches.
// Nothing here synchronises.
#include <cmath>

#include "qmm.h"
#include "qmm_experts.h"

namespace {

using qmm::set_error;

bool aligned(const void *p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

constexpr int64_t kMaxWidth = (int64_t)1 << 20;  // of a matrix side

int check_width(const char *name, int64_t n, int fmt) {
    if (n < 1 || n > kMaxWidth)
        return set_error(QMM_ERR_SHAPE, "%s %lld must be 1 to %lld", name, (long long)n, (long long)kMaxWidth);
    if (qmm_weight_bytes(fmt, n, 1) == 0)
        return set_error(QMM_ERR_SHAPE, "%s %lld is not a whole number of blocks of format %d", name, (long long)n, fmt);
    return QMM_OK;
}

// Everything but the scratch; *empty: nothing to do.
int check_ffn(const qmm_experts_ffn_args *a, qmm::ExpertsFfn *l, bool *empty, bool pointers) {
    if (!a) return set_error(QMM_ERR_NULL, "args is NULL");
    if (a->act != QMM_ACT_SWIGLU && a->act != QMM_ACT_GEGLU)
        return set_error(QMM_ERR_FORMAT, "unknown activation %d", a->act);
    for (int f : {a->fmt, a->fmt_down})
        if (f < QMM_BF16 || f > QMM_Q5_0)
            return set_error(QMM_ERR_FORMAT, "the experts' formats are the GGUF ones (got %d, %d)", a->fmt, a->fmt_down);
    int st = check_width("k", a->k, a->fmt);
    if (st == QMM_OK) st = check_width("n_ff", a->n_ff, a->fmt_down);
    if (st != QMM_OK) return st;
    if (a->n_experts < 1 || a->n_experts > qmm::kMaxExperts)
        return set_error(QMM_ERR_SHAPE, "n_experts %lld must be 1 to %d", (long long)a->n_experts, qmm::kMaxExperts);
    if (a->top_k < 1 || a->top_k > qmm::kMaxTopK)
        return set_error(QMM_ERR_SHAPE, "top_k %lld must be 1 to %d", (long long)a->top_k, qmm::kMaxTopK);
    if (a->n_pos < 0 || a->n_pos > qmm::kMaxPairs / a->top_k)
        return set_error(QMM_ERR_SHAPE, "n_pos * top_k (%lld x %lld) must be at most %lld", (long long)a->n_pos,
                         (long long)a->top_k, (long long)qmm::kMaxPairs);
    if (a->flags) return set_error(QMM_ERR_SHAPE, "unknown flags 0x%x", a->flags);
    const size_t row = qmm_weight_bytes(a->fmt, a->k, 1), down_row = qmm_weight_bytes(a->fmt_down, a->n_ff, 1);
    const size_t len = row * (size_t)a->n_ff * (size_t)a->n_experts;
    const size_t down_len = down_row * (size_t)a->k * (size_t)a->n_experts;
    if (a->w_len && a->w_len != len)
        return set_error(QMM_ERR_SIZE, "gate and up bytes %zu != %zu", a->w_len, len);
    if (a->w_down_len && a->w_down_len != down_len)
        return set_error(QMM_ERR_SIZE, "down bytes %zu != %zu", a->w_down_len, down_len);
    *empty = a->n_pos == 0;
    if (pointers && !*empty) {
        if (!a->w_gate || !a->w_up || !a->w_down || !a->x || !a->ids || !a->weights || !a->y)
            return set_error(QMM_ERR_NULL, "a weight, x, ids, weights or y pointer is NULL");
        if (!aligned(a->w_gate, 16) || !aligned(a->w_up, 16) || !aligned(a->w_down, 16))
            return set_error(QMM_ERR_ALIGN, "w_gate, w_up and w_down must be 16-byte aligned");
        if (!aligned(a->x, 4) || !aligned(a->ids, 4) || !aligned(a->weights, 4) || !aligned(a->y, 4))
            return set_error(QMM_ERR_ALIGN, "x, ids, weights and y must be 4-byte aligned");
    }
    l->act = a->act;
    l->fmt = a->fmt;
    l->fmt_down = a->fmt_down;
    l->gate = static_cast<const uint8_t *>(a->w_gate);
    l->up = static_cast<const uint8_t *>(a->w_up);
    l->down = static_cast<const uint8_t *>(a->w_down);
    l->row_bytes = (int64_t)row;
    l->down_row_bytes = (int64_t)down_row;
    l->x = a->x;
    l->ids = a->ids;
    l->weights = a->weights;
    l->y = a->y;
    l->n_pos = a->n_pos;
    l->k = (int)a->k;
    l->n_ff = (int)a->n_ff;
    l->n_experts = (int)a->n_experts;
    l->top_k = (int)a->top_k;
    l->accumulate = a->accumulate != 0;
    l->workspace = nullptr;
    return QMM_OK;
}

}  // namespace

extern "C" {

int qmm_route_experts(const qmm_route_args *a) {
    set_error(QMM_OK, "%s", "");
    if (!a) return set_error(QMM_ERR_NULL, "args is NULL");
    if (a->n_experts < 1 || a->n_experts > qmm::kMaxExperts)
        return set_error(QMM_ERR_SHAPE, "n_experts %lld must be 1 to %d", (long long)a->n_experts, qmm::kMaxExperts);
    if (a->top_k < 1 || a->top_k > a->n_experts || a->top_k > qmm::kMaxTopK)
        return set_error(QMM_ERR_SHAPE, "top_k %lld must be 1 to %d and at most n_experts %lld", (long long)a->top_k,
                         qmm::kMaxTopK, (long long)a->n_experts);
    if (a->n_pos < 0 || a->n_pos > ((int64_t)1 << 30))
        return set_error(QMM_ERR_SHAPE, "n_pos %lld must be 0 to 2^30", (long long)a->n_pos);
    if (a->logits_stride < a->n_experts || a->logits_stride > ((int64_t)1 << 32))
        return set_error(QMM_ERR_SHAPE, "logits: row stride %lld must be n_experts %lld to 2^32",
                         (long long)a->logits_stride, (long long)a->n_experts);
    if (a->score != QMM_SCORE_SOFTMAX && a->score != QMM_SCORE_SIGMOID)
        return set_error(QMM_ERR_FORMAT, "unknown score %d", a->score);
    if (!std::isfinite(a->scale)) return set_error(QMM_ERR_SHAPE, "scale is not finite");
    if (a->flags) return set_error(QMM_ERR_SHAPE, "unknown flags 0x%x", a->flags);
    if (a->n_pos == 0) return QMM_OK;
    if (!a->logits || !a->ids || !a->weights) return set_error(QMM_ERR_NULL, "logits, ids or weights is NULL");
    if (!aligned(a->logits, 4) || !aligned(a->ids, 4) || !aligned(a->weights, 4))
        return set_error(QMM_ERR_ALIGN, "logits, ids and weights must be 4-byte aligned");
    qmm::DeviceInfo *dev = nullptr;
    const int st = qmm::current_device(&dev);
    if (st != QMM_OK) return st;
    qmm::Route r;
    r.logits = a->logits;
    r.logits_stride = a->logits_stride;
    r.ids = a->ids;
    r.weights = a->weights;
    r.n_pos = a->n_pos;
    r.n_experts = (int)a->n_experts;
    r.top_k = (int)a->top_k;
    r.score = a->score;
    r.normalize = a->normalize != 0;
    r.scale = a->scale;
    const cudaError_t e = qmm::launch_route(r, *dev, static_cast<cudaStream_t>(a->stream));
    return e == cudaSuccess ? QMM_OK : set_error(QMM_ERR_CUDA, "expert choice launch: %s", cudaGetErrorString(e));
}

size_t qmm_experts_ffn_workspace_bytes(const qmm_experts_ffn_args *a) {
    qmm::ExpertsFfn l;
    bool empty = false;
    if (check_ffn(a, &l, &empty, false) != QMM_OK || empty) return 0;
    return qmm::experts_ffn_workspace_bytes(l);
}

int qmm_experts_ffn(const qmm_experts_ffn_args *a) {
    set_error(QMM_OK, "%s", "");
    qmm::ExpertsFfn l;
    bool empty = false;
    int st = check_ffn(a, &l, &empty, true);
    if (st != QMM_OK || empty) return st;
    qmm::DeviceInfo *dev = nullptr;
    st = qmm::current_device(&dev);
    if (st != QMM_OK) return st;
    const size_t need = qmm::experts_ffn_workspace_bytes(l);
    l.workspace = a->workspace;
    if (a->workspace) {
        if (a->workspace_bytes < need)
            return set_error(QMM_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", a->workspace_bytes, need);
        if (!aligned(a->workspace, 256)) return set_error(QMM_ERR_ALIGN, "workspace must be 256-byte aligned");
    } else if (need) {
        st = qmm::scratch_of_library(need, &l.workspace);
        if (st != QMM_OK) return st;
    }
    const cudaError_t e = qmm::launch_experts_ffn(l, *dev, static_cast<cudaStream_t>(a->stream));
    return e == cudaSuccess ? QMM_OK : set_error(QMM_ERR_CUDA, "experts launch: %s", cudaGetErrorString(e));
}

}  // extern "C"
