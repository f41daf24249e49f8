// Gradients of the normalisation of bf16 rows for fp32 dy.
#include "layernorm_grad.cuh"

namespace moe {
template cudaError_t launch_layernorm_grad<__nv_bfloat16, float>(const NormArgs&, int32_t, cudaStream_t);
}  // namespace moe
