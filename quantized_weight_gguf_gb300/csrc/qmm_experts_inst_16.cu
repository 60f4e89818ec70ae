// qmm_experts_inst_16.cu -- the experts' products over weights of these formats.
#include "qmm_experts_rows.cuh"

namespace qmm {
namespace experts {
template cudaError_t launch_product<F_BF16>(bool, int, const ProductParams &, int, const DeviceInfo &, cudaStream_t);
template cudaError_t launch_single<F_BF16>(bool, const ProductParams &, const DeviceInfo &, cudaStream_t);
template cudaError_t launch_product<F_F16>(bool, int, const ProductParams &, int, const DeviceInfo &, cudaStream_t);
template cudaError_t launch_single<F_F16>(bool, const ProductParams &, const DeviceInfo &, cudaStream_t);
}  // namespace experts
}  // namespace qmm
