// The norms around the end of a drafter block for bf16 tensors (norm.cuh).
#include "norm.cuh"

namespace dspark {

cudaError_t launch_norm_bf16(const NormArgs& a, bool grad) {
  switch (vector_bytes(a)) {
    case 16: return launch_of<__nv_bfloat16, 8>(a, grad);
    case 8: return launch_of<__nv_bfloat16, 4>(a, grad);
    case 4: return launch_of<__nv_bfloat16, 2>(a, grad);
    default: return launch_of<__nv_bfloat16, 1>(a, grad);
  }
}

}  // namespace dspark
