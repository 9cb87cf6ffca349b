// The norm around the end of a drafter block and the clipping of gradients: the calls'
// arguments as the kernels take them, and the host launchers.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/dspark.h"

namespace dspark {

struct NormArgs {
  int T, H, dtype, span;       // span: gate_span, at most T
  float eps, scale, offset;
  const void *x, *y, *gate, *w_post, *w_pre, *d_h, *d_x_out;
  void *x_out, *h;
  void *d_x, *d_y, *d_gate, *d_w_post, *d_w_pre;
  float* w_part;       // [2][norm_max_ctas][H] column sums of each CTA: w_pre, w_post
  float* gate_part;    // [gate rows][norm_span_parts][H] gate gradients of parts of a span,
                       // when there is more than one
  cudaStream_t stream;
};

constexpr int kNormMaxH = 8192;      // 16 elements for each of 512 threads

int norm_max_ctas(int H);              // CTAs of the gradient kernel, at most
int norm_span_parts(int T, int span);  // parts of the rows that share a gate row
cudaError_t launch_norm_f32(const NormArgs& a, bool grad);    // grad: the backward pass
cudaError_t launch_norm_bf16(const NormArgs& a, bool grad);

constexpr int kClipMaxCtas = 1216;   // CTAs of one pass over the gradients, at most
constexpr int kClipList = 96;        // gradients of one launch

size_t clip_partials(int count);     // fp32 values of workspace
cudaError_t launch_clip_grads(int count, const dspark_grad* grads, float max_norm, float* norm,
                              float* partial, cudaStream_t stream);

}  // namespace dspark
