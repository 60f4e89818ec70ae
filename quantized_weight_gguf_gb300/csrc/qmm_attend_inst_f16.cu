// qmm_attend_inst_f16.cu -- attention kernels over F16 caches.
#include "qmm_attend_kernel.cuh"

namespace qmm {
namespace attend {
cudaError_t launch_f16(const AttendParams &a, int grid, cudaStream_t s) {
    return launch_format<F_F16, F_F16>(a, grid, s);
}
}  // namespace attend
}  // namespace qmm
