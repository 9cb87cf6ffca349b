// The norms around the end of a drafter block for fp32 tensors (norm.cuh), and what does not
// depend on the type.
#include "norm.cuh"

namespace dspark {

int norm_max_ctas(int H) { return 160 * std::max(1, 2048 / row_threads(H)); }

int norm_span_parts(int T, int span) { return (std::min(span, T) + norm_unit(T) - 1) / norm_unit(T); }

cudaError_t launch_norm_f32(const NormArgs& a, bool grad) {
  switch (vector_bytes(a)) {
    case 16: return launch_of<float, 4>(a, grad);
    case 8: return launch_of<float, 2>(a, grad);
    default: return launch_of<float, 1>(a, grad);
  }
}

}  // namespace dspark
