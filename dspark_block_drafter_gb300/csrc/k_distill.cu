// Distillation from a teacher's listed tokens.  With q_k the teacher's probability of the k-th
// listed token of a row, Q their sum, and p the head's softmax over its whole vocabulary:
//
//   loss  = sum_k q_k (log q_k - log p_k),     d loss / d z_v = Q p_v - sum_k [v = id_k] q_k
//
// The gradient of the logits is the head loss's, times Q, but for the listed entries.  So the
// head loss runs as it is (the row's most probable listed token as its label, Q times its weight), and
// the kernels here take the listed tokens' logits by dot products of their own, 64 of 151936
// columns, in fp32 from the rows of the head (next to the three products of the whole head, 2%
// of the time at 2048 rows), and write the listed entries of the gradient anew.
//
// A listed entry q (Q e^-x - 1), x = log q - log p, loses no digits where head and teacher
// nearly agree: it is q (Q expm1(-x) + (Q - 1)).  x itself is small where they are sure of one
// token: as the label its -log p is the log1p of the other logits' weights, and its -log q the
// log1p of the other listed tokens' (as differences of logits and log-sum-exps near 25, each is off
// by 1e-6, more than such an entry).  In bf16 an entry is rounded to 8 bits like every other; with
// few rows the rounding is carried along (loss_low), otherwise that of the label is
// (LossPlan::qres).
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>

#include "common.cuh"
#include "distill.h"
#include "kernels.h"
#include "launch.h"
#include "loss_sum.cuh"

namespace dspark {

namespace {

constexpr int kPerLane = kMaxTargets / 32;

// One warp a row: which of its listed tokens count, their head rows and log q.
__global__ void __launch_bounds__(128) distill_targets(const DistillPlan d) {
  pdl_wait();
  pdl_signal();
  __shared__ int s_id[4][kMaxTargets];
  const LossPlan& p = d.p;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, t = blockIdx.x * 4 + warp;
  if (t >= p.T) return;
  const size_t at = (size_t)t * d.k;
  float x[kPerLane], top = -INFINITY;
  int row[kPerLane], first = kMaxTargets;
  bool bad = false, none = true;
#pragma unroll
  for (int q = 0; q < kPerLane; ++q) {
    const int k = lane + 32 * q;
    row[q] = -1;
    x[q] = -INFINITY;
    if (k >= d.k) continue;
    const int id = d.ids[at + k];
    float s = d.logits[at + k];
    // (a token of no probability is not listed, whatever its id; one that is not a number is, and
    // tells)
    const bool listed = id >= 0 && !(s == -INFINITY), in = listed && id < p.V;
    bad |= listed && !in;
    s_id[warp][k] = in ? id : -1;
    if (!in) continue;
    int j = p.d2t ? loss_d2t_row(p.d2t, p.Vh, id) : id;
    if (j >= 0 && p.bias && !(p.bias[j] > kEmitMaskLevel)) j = -1;
    row[q] = j;
    if (j < 0) continue;
    none = false;
    // (a mask of the type's lowest value stays a number under a factor above 1)
    x[q] = isfinite(s) ? fminf(fmaxf(d.scale * s, -FLT_MAX), FLT_MAX) : d.scale * s;
    top = x[q] == x[q] ? fmaxf(top, x[q]) : top;
    first = min(first, k);
  }
  __syncwarp();
  // the same token twice: which probability it has is not said
#pragma unroll
  for (int q = 0; q < kPerLane; ++q) {
    const int k = lane + 32 * q;
    if (k >= d.k || s_id[warp][k] < 0) continue;
    for (int o = 0; o < k; ++o) bad |= s_id[warp][o] == s_id[warp][k];
  }
  bad = __any_sync(0xFFFFFFFFu, bad);
  none = __all_sync(0xFFFFFFFFu, none);
  first = __reduce_min_sync(0xFFFFFFFFu, first);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  if (bad || none) {
    if (lane == 0) d.label[t] = bad ? p.V : -1;
    return;
  }
  // the label: the most probable one, the first of equals (where none is a number, the first)
  int label = kMaxTargets;
#pragma unroll
  for (int q = kPerLane - 1; q >= 0; --q)
    if (row[q] >= 0 && x[q] == top) label = lane + 32 * q;
  label = __reduce_min_sync(0xFFFFFFFFu, label);
  if (label == kMaxTargets) label = first;
  float lse = 0.f;
  if (d.t_lse) {
    lse = d.t_lse[t];
  } else {
    // log q from the label's logit, the log-sum-exp of the others beside it
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < kPerLane; ++q)
      if (row[q] >= 0 && lane + 32 * q != label) s += expf(x[q] - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    s = log1pf(s);
#pragma unroll
    for (int q = 0; q < kPerLane; ++q) x[q] = (x[q] - top) - s;
  }
  float mass = 0.f;
#pragma unroll
  for (int q = 0; q < kPerLane; ++q) {
    const int k = lane + 32 * q;
    if (k >= d.k) continue;
    x[q] -= lse;
    d.row[at + k] = row[q];
    d.log_q[at + k] = x[q];
    if (row[q] >= 0) mass += expf(x[q]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mass += __shfl_xor_sync(0xFFFFFFFFu, mass, o);
  if (lane == 0) {
    d.label[t] = s_id[warp][label];
    d.mass[t] = d.t_lse ? mass : (mass == mass ? 1.f : mass);
  }
}

// CTA (compact row i, part y): the logits of its listed tokens, one warp each.  X's row stays in
// L1 while the head's rows pass by.
constexpr int kDotThreads = 256;
template <typename E>
__global__ void __launch_bounds__(kDotThreads) distill_logits(const DistillPlan d) {
  pdl_wait();
  pdl_signal();
  const LossPlan& p = d.p;
  const int i = blockIdx.x, tid = threadIdx.x, lane = tid % 32;
  if (i >= (int)p.ctrl[kLossTok]) return;
  const int t = p.tok[i];
  const E* x = (const E*)p.x + (size_t)i * p.Kx;
  if (tid == 0 && blockIdx.y == 0) {
    const float w = p.wrow[i];
    d.w[i] = w;
    p.wrow[i] = w * d.mass[t];
  }
  constexpr int VE = 16 / sizeof(E);
  const bool wide = p.H % VE == 0 && (uintptr_t)p.lm_head % 16 == 0;
  const int step = gridDim.y * (kDotThreads / 32);
  for (int k = blockIdx.y * (kDotThreads / 32) + tid / 32; k < d.k; k += step) {
    const int j = d.row[(size_t)t * d.k + k];
    if (j < 0) continue;
    const E* wr = (const E*)p.lm_head + (size_t)j * p.H;
    float a[4] = {};
    if (wide) {
      struct alignas(16) Eight { E e[VE]; };
      const Eight* wv = reinterpret_cast<const Eight*>(wr);
      const Eight* xv = reinterpret_cast<const Eight*>(x);
#pragma unroll 4
      for (int c = lane; c < p.H / VE; c += 32) {
        const Eight u = wv[c], y = xv[c];
#pragma unroll
        for (int g = 0; g < VE; ++g) a[g % 4] = fmaf(to_f32(u.e[g]), to_f32(y.e[g]), a[g % 4]);
      }
    } else {
#pragma unroll 4
      for (int c = lane; c < p.H; c += 32) a[0] = fmaf(to_f32(wr[c]), to_f32(x[c]), a[0]);
    }
    const E* w2 = (const E*)p.w2 + j;
#pragma unroll 8
    for (int c = lane; c < p.r; c += 32)
      a[1] = fmaf(to_f32(w2[(size_t)c * p.Vh]), to_f32(x[p.Hp + c]), a[1]);
    float z = (a[0] + a[1]) + (a[2] + a[3]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
    if (lane == 0) {
      d.z[(size_t)i * d.k + k] = p.bias ? z + p.bias[j] : z;
      if (p.vinv) d.row[(size_t)t * d.k + k] = p.vinv[j];
    }
  }
}

// -log p of the k-th listed token of compact row i, column j: that of the label comes from the
// head loss, which keeps the digits of a small one.
__device__ __forceinline__ float minus_log_p(const DistillPlan& d, int i, int k, int j, float lse,
                                             float label_loss) {
  return j == d.p.lab[i] ? label_loss : lse - d.z[(size_t)i * d.k + k];
}

// The entry of the logits' gradient at listed token k of compact row i, column j, where v0 <= j:
// q columns start at v0.
template <typename E>
__device__ __forceinline__ void put_entry(const LossPlan& p, int i, int j, int v0, float w, float mass,
                                          float lq, float minus_lp, bool low) {
  E* q = (E*)p.q + (size_t)i * p.ldq + (j - v0);
  // (far below, which log q of -infinity is too: as the difference, where expm1 could overflow)
  const float x = lq + minus_lp;
  const float g = w * (x > -1.f ? expf(lq) * (mass * expm1f(-x) + (mass - 1.f))
                                : mass * expf(-minus_lp) - expf(lq));
  if constexpr (sizeof(E) == 4) {
    *q = g;
  } else if (j == p.lab[i]) {
    loss_put_label(p, i, low, q, g);
  } else {
    const __nv_bfloat16 b = __float2bfloat16(g);
    *q = b;
    if (low) q[kLossLow * p.ldq] = __float2bfloat16(g - __bfloat162float(b));
  }
}

// One warp a compact row: its loss, and with ENTRIES (the vocabulary in one piece) its listed
// entries; the last CTA takes the total.  `d.z` then holds -log p.
constexpr int kLossThreads = 256;
template <typename E, bool ENTRIES>
__global__ void __launch_bounds__(kLossThreads) distill_loss(const DistillPlan d) {
  pdl_wait();
  pdl_signal();
  __shared__ float2 s_w[32];
  __shared__ bool s_last;
  const LossPlan& p = d.p;
  const int n_tok = (int)p.ctrl[kLossTok], lane = threadIdx.x % 32;
  const int i = blockIdx.x * (kLossThreads / 32) + threadIdx.x / 32;
  if (i < n_tok) {
    const int t = p.tok[i];
    const float lse = p.lse[i], nll = p.loss[t], w = d.w[i], mass = d.mass[t];
    const bool low = ENTRIES && sizeof(E) == 2 && loss_low(p, n_tok);
    Sum2 s;
    for (int k = lane; k < d.k; k += 32) {
      const int j = d.row[(size_t)t * d.k + k];
      if (j < 0) continue;
      const float lq = d.log_q[(size_t)t * d.k + k];
      const float minus_lp = minus_log_p(d, i, k, j, lse, nll);
      if (ENTRIES) put_entry<E>(p, i, j, 0, w, mass, lq, minus_lp, low);
      else d.z[(size_t)i * d.k + k] = minus_lp;
      const float q = expf(lq), x = lq + minus_lp;
      // (0 log 0 is 0)
      s.add(q > 0.f || q != q ? q * x : 0.f);
    }
    s = warp_sum(s);
    __syncwarp();
    if (lane == 0) p.loss[t] = s.value();
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(p.ctrl + kDistillDone, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (s_last) {
    __threadfence();
    const Sum2 a = loss_total<kLossThreads>(p, d.w, n_tok, s_w);
    if (threadIdx.x == 0)
      *p.total = n_tok > 0 ? __uint_as_float(p.ctrl[kLossScale]) * a.value() : 0.f;
  }
}

// One warp a compact row: the entries of the listed tokens among columns [v0, v1).
template <typename E>
__global__ void __launch_bounds__(256) distill_entries(const DistillPlan d, int v0, int v1) {
  pdl_wait();
  pdl_signal();
  const LossPlan& p = d.p;
  const int n_tok = (int)p.ctrl[kLossTok], lane = threadIdx.x % 32;
  const int i = blockIdx.x * 8 + threadIdx.x / 32;
  if (i >= n_tok) return;
  const int t = p.tok[i];
  const float w = d.w[i], mass = d.mass[t];
  const bool low = loss_low(p, n_tok);
  for (int k = lane; k < d.k; k += 32) {
    const int j = d.row[(size_t)t * d.k + k];
    if (j >= v0 && j < v1)
      put_entry<E>(p, i, j, v0, w, mass, d.log_q[(size_t)t * d.k + k], d.z[(size_t)i * d.k + k], low);
  }
}

}  // namespace

cudaError_t launch_distill_targets(const DistillPlan& d) {
  return launch_after(distill_targets, (unsigned)(d.p.T + 3) / 4, 128, 0, d.p.stream, d);
}

cudaError_t launch_distill_logits(const DistillPlan& d) {
  const auto kernel = d.p.dtype == 0 ? distill_logits<float> : distill_logits<__nv_bfloat16>;
  // several CTAs a row where rows alone do not fill the GPU
  const unsigned y = (unsigned)std::max(1, std::min((d.k + 7) / 8, 1216 / d.p.T));
  return launch_after(kernel, dim3((unsigned)d.p.T, y), kDotThreads, 0, d.p.stream, d);
}

cudaError_t launch_distill_loss(const DistillPlan& d, bool entries) {
  const bool f32 = d.p.dtype == 0;
  return launch_after(!entries ? distill_loss<float, false>
                      : f32    ? distill_loss<float, true>
                               : distill_loss<__nv_bfloat16, true>,
                      (unsigned)(d.p.T + 7) / 8, kLossThreads, 0, d.p.stream, d);
}

cudaError_t launch_distill_entries(const DistillPlan& d, int v0, int v1) {
  return launch_after(d.p.dtype == 0 ? distill_entries<float> : distill_entries<__nv_bfloat16>,
                      (unsigned)(d.p.T + 7) / 8, 256, 0, d.p.stream, d, v0, v1);
}

}  // namespace dspark
