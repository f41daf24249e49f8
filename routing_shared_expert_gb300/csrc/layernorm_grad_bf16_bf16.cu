// Gradients of the normalisation of bf16 rows for bf16 dy.
#include "layernorm_grad.cuh"

namespace moe {
template cudaError_t launch_layernorm_grad<__nv_bfloat16, __nv_bfloat16>(const NormArgs&, int32_t, cudaStream_t);
}  // namespace moe
