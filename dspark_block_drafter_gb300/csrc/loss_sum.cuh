// Sums shared by the kernels of the head's losses.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "loss.h"

namespace dspark {

namespace {

// An fp32 sum that carries its rounding errors along (Knuth's two-sum).
struct Sum2 {
  float s = 0.f, c = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float t = s + x, b = t - s;
    c += (s - (t - b)) + (x - b);
    s = t;
  }
  __device__ __forceinline__ void add(const Sum2& o) {
    add(o.s);
    c += o.c;
  }
  __device__ __forceinline__ float value() const { return s + c; }
};

__device__ __forceinline__ Sum2 warp_sum(Sum2 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Sum2 u;
    u.s = __shfl_xor_sync(0xFFFFFFFFu, v.s, o);
    u.c = __shfl_xor_sync(0xFFFFFFFFu, v.c, o);
    v.add(u);
  }
  return v;
}

// Sum over a CTA, in a fixed order; lane 0 of warp 0 gets it.
__device__ __forceinline__ Sum2 block_sum(Sum2 v, float2* s_warp) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
  v = warp_sum(v);
  if (lane == 0) s_warp[warp] = make_float2(v.s, v.c);
  __syncthreads();
  Sum2 u;
  if (warp == 0) {
    if (lane < warps) {
      u.s = s_warp[lane].x;
      u.c = s_warp[lane].y;
    }
    u = warp_sum(u);
  }
  return u;
}

// The sum of the rows' losses by their weights w[i], in a fixed order; thread 0 gets it.
template <int THREADS>
__device__ __forceinline__ Sum2 loss_total(const LossPlan& p, const float* w_of, int n_tok,
                                           float2* s_w) {
  const int tid = threadIdx.x;
  Sum2 a;
  constexpr int kAt = 8;                    // (rows of a thread at once)
  for (int j0 = tid; j0 < n_tok; j0 += kAt * THREADS) {
    float w[kAt], x[kAt];
#pragma unroll
    for (int q = 0; q < kAt; ++q) {
      const int j = j0 + q * THREADS;
      w[q] = j < n_tok ? w_of[j] : 0.f;
      x[q] = j < n_tok ? __ldcg(p.loss + p.tok[j]) : 0.f;
    }
#pragma unroll
    for (int q = 0; q < kAt; ++q) {
      // the product's rounding error goes into the sum too
      const float y = w[q] * x[q];
      a.add(y);
      a.c += fmaf(w[q], x[q], -y);
    }
  }
  return block_sum(a, s_w);
}

// The row of a d2t head whose token is t, or -1.
__device__ __forceinline__ int loss_d2t_row(const int32_t* d2t, int n_rows, int t) {
  // first entry >= t: seven probes at a time, since each is a trip to memory
  int lo = 0, hi = n_rows;
  while (hi > lo) {
    const int n = hi - lo;
    int above = 0;                              // probes whose entry is below t
#pragma unroll
    for (int q = 1; q < 8; ++q) above += d2t[lo + (int)((long long)n * q / 8)] < t;
    // entries lo + n q / 8 (q <= above) are below t, the next one is not
    const int l = lo, h = hi;
    if (above > 0) lo = l + (int)((long long)n * above / 8) + 1;
    if (above < 7) hi = l + (int)((long long)n * (above + 1) / 8);
    else hi = h;
  }
  return lo < n_rows && d2t[lo] == t ? lo : -1;
}

}  // namespace

}  // namespace dspark
