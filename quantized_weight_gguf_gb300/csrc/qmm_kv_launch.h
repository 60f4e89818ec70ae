// qmm_kv_launch.h -- launch interfaces of the paged key-value cache kernels
// (qmm_kv.cu, qmm_attend.cu), called by the entry points in qmm_kv_api.cu.
#pragma once

#include "qmm_internal.h"
#include "qmm_kv.cuh"

namespace qmm {

struct KvAppend {
    KvView c;
    const float *k, *v, *q;
    float *q_out;
    const float *rope;
    int64_t k_stride, v_stride, q_stride, q_out_stride;
    int64_t n_new, rope_len;
    int n_heads, n_rot, style;  // n_heads 0: no q
    int teams;                  // of lanes per row; set by launch_kv_append
    bool vec;                   // every row starts on a 16-byte boundary
};
cudaError_t launch_kv_append(const KvAppend &a, const DeviceInfo &dev, cudaStream_t s);

struct KvRead {
    KvView c;
    float *k, *v;
    int64_t first, count;
    bool vec;
};
cudaError_t launch_kv_read(const KvRead &a, const DeviceInfo &dev, cudaStream_t s);

struct Attend {
    KvView c;
    const float *q;
    float *out;
    int64_t q_stride, out_stride;
    int64_t n_new, window;  // window 0: none
    int n_heads;
    float scale;
    bool vec;               // rows of q and out start on 16-byte boundaries
    void *workspace;
};
bool attend_supports(int dim);
size_t attend_workspace_bytes(const Attend &a, const DeviceInfo &dev);
cudaError_t launch_attend(const Attend &a, const DeviceInfo &dev, cudaStream_t s);

}  // namespace qmm
