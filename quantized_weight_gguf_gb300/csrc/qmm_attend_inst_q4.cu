// qmm_attend_inst_q4.cu -- attention kernels over Q4_0 caches.
#include "qmm_attend_kernel.cuh"

namespace qmm {
namespace attend {
cudaError_t launch_q4(const AttendParams &a, int grid, cudaStream_t s) {
    return launch_format<F_Q4_0, F_Q4_0>(a, grid, s);
}
}  // namespace attend
}  // namespace qmm
