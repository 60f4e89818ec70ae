// qmm_attend_inst_q8q4.cu -- attention kernels over caches of Q8_0 keys and Q4_0 values.
#include "qmm_attend_kernel.cuh"

namespace qmm {
namespace attend {
cudaError_t launch_q8q4(const AttendParams &a, int grid, cudaStream_t s) {
    return launch_format<F_Q8_0, F_Q4_0>(a, grid, s);
}
}  // namespace attend
}  // namespace qmm
