// The global norm of a list of gradients, and the clipped list.
//
//   norm = sqrt(sum in^2),   out = in * min(1, max_norm / (norm + 1e-6))
//
// Squares are summed in fp32: within a thread with the rounding errors carried along, then over
// the CTA and over the CTAs pairwise (fp64 runs at a few additions per clock and SM here).
//
// Bound by memory.  Two passes: the first sums squares, CTA by CTA in a fixed assignment of
// chunks; the second first joins the CTAs' sums (every CTA for itself, the same way), then
// scales, from the last chunk to the first, because the last ones read are still in L2.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "launch.h"
#include "train.h"

namespace dspark {

namespace {

constexpr int kThreads = 512;
constexpr int kVec = 16;                         // bytes of a vector access
constexpr int kChunkVecs = 4 * kThreads;         // vectors of a chunk: four a thread
constexpr int kChunkBytes = kChunkVecs * kVec;   // 32 KB

struct ClipList {
  const void* in[kClipList];
  void* out[kClipList];
  long long n[kClipList];
  int first[kClipList + 1];                      // first chunk of each gradient
  int8_t bf16[kClipList], vec[kClipList];
  int count;
};
static_assert(sizeof(ClipList) <= 4000, "kernel parameters");

__device__ __forceinline__ int clip_find(const ClipList& l, int chunk) {
  int lo = 0, hi = l.count - 1;                  // last gradient with first <= chunk
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (l.first[mid] <= chunk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

template <typename E>
__device__ __forceinline__ float square_sum(const uint4& v) {
  const E* e = reinterpret_cast<const E*>(&v);
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < kVec / (int)sizeof(E); ++j) {
    const float x = to_f32(e[j]);
    s = fmaf(x, x, s);
  }
  return s;
}

template <typename E>
__device__ __forceinline__ float chunk_squares(const E* p, long long n, long long c, bool vec) {
  constexpr int kPerVec = kVec / (int)sizeof(E);
  const long long e0 = c * (kChunkBytes / (int)sizeof(E));
  const int len = (int)min(n - e0, (long long)(kChunkBytes / (int)sizeof(E)));
  float s = 0.f;
  if (vec && len == kChunkBytes / (int)sizeof(E)) {
    const uint4* q = reinterpret_cast<const uint4*>(p + e0);
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = q[threadIdx.x + j * kThreads];
#pragma unroll
    for (int j = 0; j < 4; ++j) s += square_sum<E>(v[j]);
  } else if (vec) {
    const uint4* q = reinterpret_cast<const uint4*>(p + e0);
    for (int j = threadIdx.x; j < len / kPerVec; j += kThreads) s += square_sum<E>(q[j]);
    for (int j = len / kPerVec * kPerVec + threadIdx.x; j < len; j += kThreads) {
      const float x = to_f32(p[e0 + j]);
      s = fmaf(x, x, s);
    }
  } else {
    for (int j = threadIdx.x; j < len; j += kThreads) {
      const float x = to_f32(p[e0 + j]);
      s = fmaf(x, x, s);
    }
  }
  return s;
}

// Sum over the CTA in a fixed order; every thread gets it.
__device__ __forceinline__ float clip_block_sum(float v) {
  __shared__ float s[kThreads / 32];
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (lane == 0) s[threadIdx.x / 32] = v;
  __syncthreads();
  v = lane < kThreads / 32 ? s[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

__global__ void __launch_bounds__(kThreads) clip_squares(const __grid_constant__ ClipList l,
                                                         float* partial) {
  pdl_wait();
  pdl_signal();
  float acc = 0.f, low = 0.f;
  for (int c = blockIdx.x; c < l.first[l.count]; c += gridDim.x) {
    const int g = clip_find(l, c);
    const long long lc = c - l.first[g];
    const float x = l.bf16[g]
                        ? chunk_squares((const __nv_bfloat16*)l.in[g], l.n[g], lc, l.vec[g])
                        : chunk_squares((const float*)l.in[g], l.n[g], lc, l.vec[g]);
    const float t = acc + x;                     // (both are >= 0: the larger one's error)
    low += acc >= x ? (acc - t) + x : (x - t) + acc;
    acc = t;
  }
  // (an infinite sum has no rounding error to carry)
  const float s = clip_block_sum(acc < INFINITY ? acc + low : acc);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

template <typename E>
__device__ __forceinline__ uint4 scaled(const uint4& v, float k) {
  uint4 o;
  const E* e = reinterpret_cast<const E*>(&v);
  E* r = reinterpret_cast<E*>(&o);
#pragma unroll
  for (int j = 0; j < kVec / (int)sizeof(E); ++j) r[j] = (E)(to_f32(e[j]) * k);
  return o;
}

template <typename E>
__device__ __forceinline__ void chunk_scale(const E* p, E* out, long long n, long long c,
                                            bool vec, float k) {
  constexpr int kPerVec = kVec / (int)sizeof(E);
  const long long e0 = c * (kChunkBytes / (int)sizeof(E));
  const int len = (int)min(n - e0, (long long)(kChunkBytes / (int)sizeof(E)));
  const int vecs = vec ? len / kPerVec : 0;
  const uint4* q = reinterpret_cast<const uint4*>(p + e0);
  uint4* o = reinterpret_cast<uint4*>(out + e0);
  if (vecs == kChunkVecs) {
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = q[threadIdx.x + j * kThreads];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[threadIdx.x + j * kThreads] = scaled<E>(v[j], k);
    return;
  }
  for (int j = threadIdx.x; j < vecs; j += kThreads) o[j] = scaled<E>(q[j], k);
  for (int j = vecs * kPerVec + threadIdx.x; j < len; j += kThreads)
    out[e0 + j] = (E)(to_f32(p[e0 + j]) * k);
}

__global__ void __launch_bounds__(kThreads) clip_scale(const __grid_constant__ ClipList l,
                                                       const float* partial, int partials,
                                                       float max_norm, float* norm_out) {
  pdl_wait();
  pdl_signal();
  float a = 0.f;
  for (int j = threadIdx.x; j < partials; j += kThreads) a += partial[j];
  const float norm = sqrtf(clip_block_sum(a));
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
  // (a norm that is not finite: everything is left as it is)
  const float k = norm < INFINITY ? fminf(1.f, max_norm / (norm + 1e-6f)) : 1.f;
  for (int c = l.first[l.count] - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
    const int g = clip_find(l, c);
    if (k == 1.f && l.in[g] == l.out[g]) continue;
    const long long lc = c - l.first[g];
    if (l.bf16[g])
      chunk_scale((const __nv_bfloat16*)l.in[g], (__nv_bfloat16*)l.out[g], l.n[g], lc, l.vec[g],
                  k);
    else
      chunk_scale((const float*)l.in[g], (float*)l.out[g], l.n[g], lc, l.vec[g], k);
  }
}

// The gradients [a, a + count) of one launch.
ClipList make_list(const dspark_grad* grads, int count) {
  ClipList l{};
  l.count = count;
  for (int g = 0; g < count; ++g) {
    const int es = grads[g].dtype == DSPARK_BF16 ? 2 : 4;
    l.in[g] = grads[g].in;
    l.out[g] = grads[g].out;
    l.n[g] = grads[g].n;
    l.bf16[g] = grads[g].dtype == DSPARK_BF16;
    l.vec[g] = (((uintptr_t)grads[g].in | (uintptr_t)grads[g].out) & 15) == 0;
    l.first[g + 1] = l.first[g] + (int)((grads[g].n * es + kChunkBytes - 1) / kChunkBytes);
  }
  return l;
}

}  // namespace

size_t clip_partials(int count) {
  return (size_t)((count + kClipList - 1) / kClipList) * kClipMaxCtas;
}

cudaError_t launch_clip_grads(int count, const dspark_grad* grads, float max_norm, float* norm,
                              float* partial, cudaStream_t stream) {
  int sms = 0;
  cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  const int most = std::min(kClipMaxCtas, sms * (2048 / kThreads));
  int partials = 0;
  for (int a = 0; a < count; a += kClipList) {
    const ClipList l = make_list(grads + a, std::min(kClipList, count - a));
    const int grid = std::min(most, std::max(1, l.first[l.count]));
    e = launch_after(clip_squares, grid, kThreads, 0, stream, l, partial + partials);
    if (e != cudaSuccess) return e;
    partials += grid;
  }
  for (int a = (count - 1) / kClipList * kClipList; a >= 0; a -= kClipList) {
    const ClipList l = make_list(grads + a, std::min(kClipList, count - a));
    const int grid = std::min(most, std::max(1, l.first[l.count]));
    e = launch_after(clip_scale, grid, kThreads, 0, stream, l, partial, partials, max_norm,
                     a == 0 ? norm : nullptr);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

}  // namespace dspark
