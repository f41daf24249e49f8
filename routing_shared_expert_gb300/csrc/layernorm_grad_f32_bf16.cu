// Gradients of the normalisation of fp32 rows for bf16 dy.
#include "layernorm_grad.cuh"

namespace moe {
template cudaError_t launch_layernorm_grad<float, __nv_bfloat16>(const NormArgs&, int32_t, cudaStream_t);
}  // namespace moe
