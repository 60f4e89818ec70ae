// qmm_experts_inst_k6.cu -- the experts' products over weights of these formats.
#include "qmm_experts_tile.cuh"

namespace qmm {
namespace experts {
template cudaError_t launch_product<F_Q6_K>(bool, int, const ProductParams &, int, const DeviceInfo &, cudaStream_t);
template cudaError_t launch_single<F_Q6_K>(bool, const ProductParams &, const DeviceInfo &, cudaStream_t);
template cudaError_t launch_tile<F_Q6_K>(bool, const ProductParams &, int, const DeviceInfo &, cudaStream_t);
}  // namespace experts
}  // namespace qmm
