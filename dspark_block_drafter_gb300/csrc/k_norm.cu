// The norms around the end of a drafter block, and their gradient.
//
//   ry = 1 / sqrt(mean(y^2) + eps)   u = y ry (o + w_post)     (u = y without w_post)
//   x' = x + s g u                   rx = 1 / sqrt(mean(x'^2) + eps)
//   h  = x' rx (o + w_pre)
//
// With a = dh (o + w_pre) and xn = x' rx, yn = y ry:
//   dx' = d_x_out + rx (a - xn mean(a xn))      dx = dx'     dw_pre = sum_t dh xn
//   dg = s dx' u                                du = s g dx'  dw_post = sum_t du yn
//   b = du (o + w_post)                         dy = ry (b - yn mean(b yn))
//
// Bound by memory: each input is read once and each output written once, a row stays in
// registers (eight elements a thread) between its reductions, and everything is fp32.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "train.h"

namespace dspark {

namespace {

constexpr int kPer = 8;               // elements of a row per thread
constexpr int kNormUnit = 16;         // rows of one gate row that a CTA takes at a time

int row_threads(int H) { return (H + kPer * 32 - 1) / (kPer * 32) * 32; }

// Column of element e of thread `tid`: vectors of VEC consecutive elements, the threads'
// vectors side by side.
template <int VEC>
__device__ __forceinline__ int column(int e) {
  return ((e / VEC) * (int)blockDim.x + (int)threadIdx.x) * VEC + e % VEC;
}

template <typename E, int VEC>
__device__ __forceinline__ void load_row(float (&r)[kPer], const E* p, int H) {
  struct alignas(sizeof(E) * VEC) Vec { E e[VEC]; };
#pragma unroll
  for (int q = 0; q < kPer; q += VEC) {
    const int c = column<VEC>(q);
    if (c < H) {
      const Vec v = *reinterpret_cast<const Vec*>(p + c);
#pragma unroll
      for (int j = 0; j < VEC; ++j) r[q + j] = to_f32(v.e[j]);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) r[q + j] = 0.f;
    }
  }
}

template <typename E, int VEC>
__device__ __forceinline__ void store_row(E* p, const float (&r)[kPer], int H) {
  struct alignas(sizeof(E) * VEC) Vec { E e[VEC]; };
#pragma unroll
  for (int q = 0; q < kPer; q += VEC) {
    const int c = column<VEC>(q);
    if (c >= H) continue;
    Vec v;
#pragma unroll
    for (int j = 0; j < VEC; ++j) v.e[j] = (E)r[q + j];
    *reinterpret_cast<Vec*>(p + c) = v;
  }
}

// Sums of two values over the CTA, in a fixed order.  `s` holds two buffers, taken in
// turn, so that one barrier a sum is enough.
struct RowSum {
  float2 (*s)[32];
  int turn;
  __device__ float2 operator()(float a, float b) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
      b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
    const int warps = blockDim.x / 32;
    if (warps == 1) return make_float2(a, b);
    if (threadIdx.x % 32 == 0) s[turn][threadIdx.x / 32] = make_float2(a, b);
    __syncthreads();
    const int lane = threadIdx.x % 32;
    const float2 v = lane < warps ? s[turn][lane] : make_float2(0.f, 0.f);
    turn ^= 1;
    a = v.x;
    b = v.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
      b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
    return make_float2(a, b);
  }
};

template <typename E, int VEC>
__global__ void __launch_bounds__(1024) block_norm(const NormArgs a) {
  __shared__ float2 s_sum[2][32];
  RowSum sum{s_sum, 0};
  const int t = blockIdx.x, H = a.H;
  const float inv_h = 1.f / (float)H;
  float x[kPer];
  load_row<E, VEC>(x, (const E*)a.x + (size_t)t * H, H);
  if (a.y) {
    float u[kPer];
    load_row<E, VEC>(u, (const E*)a.y + (size_t)t * H, H);
    float g[kPer];
    if (a.gate) load_row<E, VEC>(g, (const E*)a.gate + (size_t)(t / a.span) * H, H);
    if (a.w_post) {
      float w[kPer];
      load_row<E, VEC>(w, (const E*)a.w_post, H);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < kPer; ++e) ss += u[e] * u[e];
      const float ry = rsqrtf(sum(ss, 0.f).x * inv_h + a.eps);
#pragma unroll
      for (int e = 0; e < kPer; ++e) u[e] = u[e] * ry * (a.offset + w[e]);
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) x[e] += a.scale * (a.gate ? g[e] * u[e] : u[e]);
  }
  if (a.x_out) store_row<E, VEC>((E*)a.x_out + (size_t)t * H, x, H);
  float w[kPer];
  load_row<E, VEC>(w, (const E*)a.w_pre, H);
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < kPer; ++e) ss += x[e] * x[e];   // (0 past the row)
  const float rx = rsqrtf(sum(ss, 0.f).x * inv_h + a.eps);
#pragma unroll
  for (int e = 0; e < kPer; ++e) x[e] = x[e] * rx * (a.offset + w[e]);
  store_row<E, VEC>((E*)a.h + (size_t)t * H, x, H);
}

// A unit is up to kNormUnit consecutive rows of one gate row (one row without a gate);
// CTAs take units in turn and keep their column sums in registers.
template <typename E, int VEC>
__global__ void __launch_bounds__(1024) block_norm_backward(const NormArgs a, int units,
                                                            int per_span) {
  __shared__ float2 s_sum[2][32];
  RowSum sum{s_sum, 0};
  const int H = a.H;
  const float inv_h = 1.f / (float)H;
  float dw_pre[kPer] = {}, dw_post[kPer] = {};
  for (int un = blockIdx.x; un < units; un += gridDim.x) {
    const int row_g = a.gate ? un / per_span : un;
    const int t0 = a.gate ? row_g * a.span + un % per_span * kNormUnit : un;
    const int t1 = a.gate ? min(min(a.T, (row_g + 1) * a.span), t0 + kNormUnit) : un + 1;
    float g[kPer], dg[kPer] = {};
    if (a.gate) load_row<E, VEC>(g, (const E*)a.gate + (size_t)row_g * H, H);
    for (int t = t0; t < t1; ++t) {
      const size_t at = (size_t)t * H;
      float x[kPer], y[kPer], d[kPer], dh[kPer], w[kPer];
      load_row<E, VEC>(x, (const E*)a.x + at, H);
      load_row<E, VEC>(dh, (const E*)a.d_h + at, H);
      if (a.d_x_out) load_row<E, VEC>(d, (const E*)a.d_x_out + at, H);
      float ry = 1.f;
      if (a.y) {
        load_row<E, VEC>(y, (const E*)a.y + at, H);
        if (a.w_post) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < kPer; ++e) ss += y[e] * y[e];
          ry = rsqrtf(sum(ss, 0.f).x * inv_h + a.eps);
          load_row<E, VEC>(w, (const E*)a.w_post, H);
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          y[e] *= ry;                                   // yn
          const float u = a.w_post ? y[e] * (a.offset + w[e]) : y[e];
          x[e] += a.scale * (a.gate ? g[e] * u : u);    // x'
        }
      }
      float wp[kPer];
      load_row<E, VEC>(wp, (const E*)a.w_pre, H);
      float ss = 0.f, ax = 0.f;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        ss += x[e] * x[e];
        ax += dh[e] * (a.offset + wp[e]) * x[e];
      }
      const float2 r = sum(ss, ax);
      const float rx = rsqrtf(r.x * inv_h + a.eps);
      const float mean = r.y * inv_h * rx;              // mean(a xn)
      float by = 0.f;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const float xn = x[e] * rx;
        dw_pre[e] += dh[e] * xn;
        const float v = rx * (dh[e] * (a.offset + wp[e]) - xn * mean);
        x[e] = a.d_x_out ? d[e] + v : v;                // dx'
      }
      store_row<E, VEC>((E*)a.d_x + at, x, H);
      if (!a.y) continue;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const float ow = a.w_post ? a.offset + w[e] : 1.f;
        if (a.gate) dg[e] += a.scale * x[e] * (y[e] * ow);
        const float du = a.scale * (a.gate ? g[e] * x[e] : x[e]);
        dw_post[e] += du * y[e];
        x[e] = du * ow;                                 // b
        by += x[e] * y[e];
      }
      if (a.w_post) {
        const float mb = sum(by, 0.f).x * inv_h;
#pragma unroll
        for (int e = 0; e < kPer; ++e) x[e] = ry * (x[e] - y[e] * mb);
      }
      store_row<E, VEC>((E*)a.d_y + at, x, H);
    }
    if (a.gate) {
      if (per_span == 1)
        store_row<E, VEC>((E*)a.d_gate + (size_t)row_g * H, dg, H);
      else
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          if (column<VEC>(e) < H) a.gate_part[(size_t)un * H + column<VEC>(e)] = dg[e];
    }
  }
  float* part = a.w_part + (size_t)blockIdx.x * H;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int c = column<VEC>(e);
    if (c >= H) continue;
    part[c] = dw_pre[e];
    if (a.w_post) part[(size_t)gridDim.x * H + c] = dw_post[e];
  }
}

// Column sums of part[rows][H] in row order: 32 columns and 8 interleaved row lanes a CTA.
template <typename E>
__global__ void __launch_bounds__(256) column_sums(const float* part, int rows, int H, E* out0,
                                                   E* out1) {
  __shared__ float s[8][33];
  const int c = blockIdx.x * 32 + threadIdx.x % 32, lane = threadIdx.x / 32;
  const float* p = part + (size_t)blockIdx.y * rows * H;
  float a = 0.f;
  if (c < H)
    for (int r = lane; r < rows; r += 8) a += p[(size_t)r * H + c];
  s[lane][threadIdx.x % 32] = a;
  __syncthreads();
  if (lane != 0 || c >= H) return;
  for (int j = 1; j < 8; ++j) a += s[j][threadIdx.x];
  (blockIdx.y == 0 ? out0 : out1)[c] = (E)a;
}

// d_gate rows of long spans, from their parts in order.
template <typename E>
__global__ void __launch_bounds__(256) gate_sums(const float* part, int per_span, int H, E* out) {
  for (int c = threadIdx.x; c < H; c += blockDim.x) {
    float a = 0.f;
    for (int j = 0; j < per_span; ++j) a += part[((size_t)blockIdx.x * per_span + j) * H + c];
    out[(size_t)blockIdx.x * H + c] = (E)a;
  }
}

bool vector_rows(const NormArgs& a) {
  const int es = a.dtype == DSPARK_F32 ? 4 : 2;
  uintptr_t all = (uintptr_t)a.H * es;
  for (const void* p : {a.x, a.y, a.gate, a.w_post, a.w_pre, a.d_h, a.d_x_out,
                        (const void*)a.x_out, (const void*)a.h, (const void*)a.d_x,
                        (const void*)a.d_y, (const void*)a.d_gate})
    all |= (uintptr_t)p;
  return all % 16 == 0;
}

template <typename E, int VEC>
cudaError_t backward(const NormArgs& a) {
  const int threads = row_threads(a.H);
  const int per_span = a.gate ? norm_span_parts(a.T, a.span) : 1;
  const int units = a.gate ? (a.T + a.span - 1) / a.span * per_span : a.T;
  int sms = 0, per_sm = 0;
  cudaError_t e = device_sms(&sms);
  if (e == cudaSuccess)
    e = blocks_per_sm((const void*)block_norm_backward<E, VEC>, threads, 0, &per_sm);
  if (e != cudaSuccess) return e;
  const int grid = std::min({units, std::max(1, per_sm) * sms, norm_max_ctas(a.H)});
  block_norm_backward<E, VEC><<<grid, threads, 0, a.stream>>>(a, units, per_span);
  column_sums<E><<<dim3((a.H + 31) / 32, a.w_post ? 2 : 1), 256, 0, a.stream>>>(
      a.w_part, grid, a.H, (E*)a.d_w_pre, (E*)a.d_w_post);
  if (per_span > 1)
    gate_sums<E><<<units / per_span, 256, 0, a.stream>>>(a.gate_part, per_span, a.H,
                                                         (E*)a.d_gate);
  return cudaGetLastError();
}

}  // namespace

int norm_max_ctas(int H) { return 160 * std::max(1, 2048 / row_threads(H)); }

int norm_span_parts(int T, int span) { return (std::min(span, T) + kNormUnit - 1) / kNormUnit; }

cudaError_t launch_block_norm(const NormArgs& a) {
  const int threads = row_threads(a.H);
  const bool v = vector_rows(a);
  if (a.dtype == DSPARK_F32) {
    if (v) block_norm<float, 4><<<a.T, threads, 0, a.stream>>>(a);
    else block_norm<float, 1><<<a.T, threads, 0, a.stream>>>(a);
  } else {
    if (v) block_norm<__nv_bfloat16, 8><<<a.T, threads, 0, a.stream>>>(a);
    else block_norm<__nv_bfloat16, 1><<<a.T, threads, 0, a.stream>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_block_norm_backward(const NormArgs& a) {
  const bool v = vector_rows(a);
  if (a.dtype == DSPARK_F32) return v ? backward<float, 4>(a) : backward<float, 1>(a);
  return v ? backward<__nv_bfloat16, 8>(a) : backward<__nv_bfloat16, 1>(a);
}

}  // namespace dspark
