// qmm_experts_inst_q4.cu -- the experts' products over weights of these formats.
#include "qmm_experts_tile.cuh"

namespace qmm {
namespace experts {
template cudaError_t launch_product<F_Q4_0>(bool, int, const ProductParams &, int, const DeviceInfo &, cudaStream_t);
template cudaError_t launch_single<F_Q4_0>(bool, const ProductParams &, const DeviceInfo &, cudaStream_t);
template cudaError_t launch_tile<F_Q4_0>(bool, const ProductParams &, int, const DeviceInfo &, cudaStream_t);
template cudaError_t launch_product<F_Q5_0>(bool, int, const ProductParams &, int, const DeviceInfo &, cudaStream_t);
template cudaError_t launch_single<F_Q5_0>(bool, const ProductParams &, const DeviceInfo &, cudaStream_t);
template cudaError_t launch_tile<F_Q5_0>(bool, const ProductParams &, int, const DeviceInfo &, cudaStream_t);
}  // namespace experts
}  // namespace qmm
