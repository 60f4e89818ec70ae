// qmm_attend_inst_bf16.cu -- attention kernels over BF16 caches.
#include "qmm_attend_kernel.cuh"

namespace qmm {
namespace attend {
cudaError_t launch_bf16(const AttendParams &a, int grid, cudaStream_t s) {
    return launch_format<F_BF16, F_BF16>(a, grid, s);
}
}  // namespace attend
}  // namespace qmm
