// The training loss of the head, all but its products: which rows carry a loss, the
// operand rows X, the softmax statistics joined over the vocabulary, the losses and their
// total, and the gradients that are sums over rows of X's gradient.
//
// Every kernel here is bound by its traffic or its latency; sums over rows are taken in a
// fixed order, in fp64 where they join many values.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "loss.h"

namespace dspark {

namespace {

constexpr int kPlanThreads = 1024;

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16(x);
}

// Sum over a CTA of up to 1024 threads, in a fixed order; every thread gets it.
template <typename S>
__device__ __forceinline__ S block_sum(S v, S* s_warp) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = (blockDim.x + 31) / 32;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  __syncthreads();
  if (lane == 0) s_warp[warp] = v;
  __syncthreads();
  S t = 0;
  for (int w = 0; w < warps; ++w) t += s_warp[w];
  return t;
}

// Bias form: the compact vocabulary's size, inverse map and biases.  vinv is -1 before.
__global__ void __launch_bounds__(256) loss_vocab(const LossPlan p, int chunks) {
  __shared__ int s_n;
  if (threadIdx.x == 0) {
    int n = 0;
    for (int c = 0; c < chunks; ++c) n += p.vchunk[c];
    s_n = n;
    if (blockIdx.x == 0) p.ctrl[kLossVoc] = (uint32_t)n;
  }
  __syncthreads();
  const int n = s_n;
  for (int j = blockIdx.x * blockDim.x + threadIdx.x; j < n; j += gridDim.x * blockDim.x) {
    const int v = p.vlist[j];
    p.vinv[v] = j;
    p.biasc[j] = p.bias[v];
  }
}

// The compact head row of token `t`, or -1.
__device__ __forceinline__ int loss_label_row(const LossPlan& p, int t) {
  int row = t;
  if (p.d2t) {
    int lo = 0, hi = p.Vh;                    // first entry >= t
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (p.d2t[mid] < t) lo = mid + 1; else hi = mid;
    }
    if (lo >= p.Vh || p.d2t[lo] != t) return -1;
    row = lo;
  }
  return p.vinv ? p.vinv[row] : row;
}

// One CTA: compacts the rows that carry a loss, in order, and sums their weights.
__global__ void __launch_bounds__(kPlanThreads) loss_tokens(const LossPlan p) {
  __shared__ int s_cnt[32];
  __shared__ double s_w[32];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  if (tid < 64 && tid != kLossVoc) p.ctrl[tid] = 0;
  if (tid == 64 && !p.vlist) p.ctrl[kLossVoc] = (uint32_t)p.Vh;
  __syncthreads();
  int base = 0;
  double wsum = 0.0;
  for (int t0 = 0; t0 < p.T; t0 += kPlanThreads) {
    const int t = t0 + tid;
    int j = -1, pv = 0;
    if (t < p.T) {
      const int label = p.labels[t];
      if (label >= p.V)
        flag_error(p.ctrl, kErrBadToken);
      else if (label >= 0)
        j = loss_label_row(p, label);
      if (j >= 0 && p.r > 0) {
        pv = p.prev[t];
        if (pv < 0 || pv >= p.V) {
          flag_error(p.ctrl, kErrBadToken);
          j = -1;
        }
      }
    }
    const unsigned m = __ballot_sync(0xFFFFFFFFu, j >= 0);
    __syncthreads();
    if (lane == 0) s_cnt[warp] = __popc(m);
    __syncthreads();
    int before = base, all = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) before += s_cnt[w];
      all += s_cnt[w];
    }
    if (t < p.T) {
      const int i = before + __popc(m & ((1u << lane) - 1));
      p.pos[t] = j >= 0 ? i : -1;
      if (j >= 0) {
        const float w = p.weights ? p.weights[t] : 1.f;
        p.tok[i] = t;
        p.lab[i] = j;
        p.prevc[i] = pv;
        p.wrow[i] = w;
        wsum += (double)w;
      }
    }
    base += all;
  }
  const double w = block_sum(wsum, s_w);
  if (tid == 0) {
    p.ctrl[kLossTok] = (uint32_t)base;
    float k = p.loss_scale;
    if (p.reduction == 1) k = w > 0.0 ? (float)((double)p.loss_scale / w) : 0.f;
    p.ctrl[kLossScale] = __float_as_uint(k);
    if (p.n_rows) *p.n_rows = base;
  }
}

// CTA t: row t's part of X (or its zero outputs, when it carries no loss), and X's padding
// row t.
template <typename E>
__global__ void __launch_bounds__(256) loss_gather(const LossPlan p) {
  const int t = blockIdx.x, tid = threadIdx.x;
  E* x = (E*)p.x;
  const E zero = from_f32<E>(0.f);
  if (t >= (int)p.ctrl[kLossTok])
    for (int k = tid; k < p.Kx; k += blockDim.x) x[(size_t)t * p.Kx + k] = zero;
  if (t >= p.T) return;
  const int i = p.pos[t];
  if (i < 0) {
    if (tid == 0) p.loss[t] = 0.f;
    if (p.d_hidden)
      for (int k = tid; k < p.H; k += blockDim.x) ((E*)p.d_hidden)[(size_t)t * p.H + k] = zero;
    return;
  }
  const E* h = (const E*)p.hidden + (size_t)t * p.H;
  for (int k = tid; k < p.Hp; k += blockDim.x)
    x[(size_t)i * p.Kx + k] = k < p.H ? h[k] : zero;
  if (p.rp) {
    const E* w = (const E*)p.w1 + (size_t)p.prevc[i] * p.r;
    for (int k = tid; k < p.rp; k += blockDim.x)
      x[(size_t)i * p.Kx + p.Hp + k] = k < p.r ? w[k] : zero;
  }
}

// CTA i: joins row i's statistics over the vocabulary tiles into its log-sum-exp and its
// loss; the last CTA to finish sums the losses.
__global__ void __launch_bounds__(128) loss_rows(const LossPlan p) {
  __shared__ float s_f[32];
  __shared__ double s_d[32];
  __shared__ bool s_last;
  const int n_tok = (int)p.ctrl[kLossTok], n_voc = (int)p.ctrl[kLossVoc];
  const int i = blockIdx.x, tid = threadIdx.x;
  if (i < n_tok) {
    const int n = (n_voc + p.stat_cols - 1) / p.stat_cols;
    const float2* st = p.stat + (size_t)i * p.n_stat;
    // running maximum and sum; a tile whose logits are all -inf has sum 0
    float m = -INFINITY, s = 0.f;
    for (int j = tid; j < n; j += blockDim.x) {
      const float2 a = st[j];
      const float mm = fmaxf(m, a.x);
      if (mm > -INFINITY) s = s * __expf(m - mm) + a.y * __expf(a.x - mm);
      else s += a.y;
      m = mm;
    }
    float mx = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
    if (tid % 32 == 0) s_f[tid / 32] = mx;
    __syncthreads();
    mx = s_f[0];
    for (int w = 1; w < (int)blockDim.x / 32; ++w) mx = fmaxf(mx, s_f[w]);
    if (mx > -INFINITY) s *= expf(m - mx);
    const double sum = block_sum((double)s, s_d);
    if (tid == 0) {
      const float lse = (float)((double)mx + log(sum));
      p.lse[i] = lse;
      p.loss[p.tok[i]] = (float)((double)mx + log(sum) - (double)p.zlab[i]);
    }
  }
  if (tid == 0) {
    __threadfence();
    s_last = atomicAdd(p.ctrl + kLossDone, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  double a = 0.0;
  for (int j = tid; j < n_tok; j += blockDim.x)
    a += (double)p.wrow[j] * (double)__ldcg(p.loss + p.tok[j]);
  const double t = block_sum(a, s_d);
  if (tid == 0) {
    const double k = (double)__uint_as_float(p.ctrl[kLossScale]);
    *p.total = n_tok > 0 ? (float)(k * t) : 0.f;
  }
}

// q = w (softmax - onehot) in place, columns [v0, v1): fp32 from stored logits.
__global__ void __launch_bounds__(256) loss_dz_f32(const LossPlan p, int v0, int v1) {
  const int n_tok = (int)p.ctrl[kLossTok], i = blockIdx.x;
  if (i >= n_tok) return;
  const int end = min(v1, (int)p.ctrl[kLossVoc]);
  float* q = (float*)p.q + (size_t)i * p.ldq;
  const float lse = p.lse[i], w = p.wrow[i];
  const int lab = p.lab[i];
  for (int v = v0 + blockIdx.y * blockDim.x + threadIdx.x; v < end; v += gridDim.y * blockDim.x)
    q[v - v0] = w * (__expf(q[v - v0] - lse) - (v == lab ? 1.f : 0.f));
}

// The same in bf16 from the stored distances (one piece: v0 = 0), over whole 256-column
// tiles: columns past the vocabulary become 0.  Eight columns a thread.
__global__ void __launch_bounds__(256) loss_dz_bf16(const LossPlan p) {
  const int n_tok = (int)p.ctrl[kLossTok], n_voc = (int)p.ctrl[kLossVoc], i = blockIdx.x;
  if (i >= n_tok) return;
  uint4* q = (uint4*)((uint16_t*)p.q + (size_t)i * p.ldq);
  const float lse = p.lse[i], w = p.wrow[i];
  const int lab = p.lab[i], end = (n_voc + 255) / 256 * 32, tiles = (n_voc + 127) / 128;
  for (int c = blockIdx.y * blockDim.x + threadIdx.x; c < end; c += gridDim.y * blockDim.x) {
    const uint4 x = q[c];
    const int tile = min(c / 16, tiles - 1);          // (a tile past the last is all far)
    const float s = (p.stat[(size_t)i * p.n_stat + tile].x - lse) * 1.44269504f;
    const uint32_t g[4] = {x.x, x.y, x.z, x.w};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int v = 8 * c + 2 * j;
      float e0 = w * loss_gap_exp(g[j] & 0xFFFFu, s), e1 = w * loss_gap_exp(g[j] >> 16, s);
      if (v == lab) e0 = loss_label_grad(p, i, e0 - w);
      if (v + 1 == lab) e1 = loss_label_grad(p, i, e1 - w);
      const __nv_bfloat162 b = __floats2bfloat162_rn(e0, e1);
      o[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    q[c] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// The compact head of a bias-form bf16 head: its rows and its columns of markov_w2, then
// zeros up to a multiple of 256.
__global__ void __launch_bounds__(256) loss_gather_head(const LossPlan p) {
  const int n = (int)p.ctrl[kLossVoc];
  const int end = min(p.Vh, (n + 255) / 256 * 256), per = p.H / 8;
  const uint4* w = (const uint4*)p.lm_head;
  uint4* wc = (uint4*)p.wc;
  for (int j = blockIdx.x; j < end; j += gridDim.x) {
    const size_t from = j < n ? (size_t)p.vlist[j] * per : 0;
    for (int k = threadIdx.x; k < per; k += blockDim.x)
      wc[(size_t)j * per + k] = j < n ? w[from + k] : make_uint4(0, 0, 0, 0);
  }
  const __nv_bfloat16* w2 = (const __nv_bfloat16*)p.w2;
  __nv_bfloat16* w2c = (__nv_bfloat16*)p.w2c;
  for (int j = blockIdx.x * blockDim.x + threadIdx.x; j < end; j += gridDim.x * blockDim.x) {
    const int v = j < n ? p.vlist[j] : -1;
    for (int k = 0; k < p.r; ++k)
      w2c[(size_t)k * p.Vh + j] = v >= 0 ? w2[(size_t)k * p.Vh + v] : __float2bfloat16(0.f);
  }
}

// CTA i: row i of the gradient of X, summed over the splits of the vocabulary (and, in
// bf16, with what q lost at the label), times the scale: d_hidden's row, and the gradient of
// markov_w1's row prev (left in split 0).
template <typename E>
__global__ void __launch_bounds__(256) loss_dx_rows(const LossPlan p) {
  const int i = blockIdx.x;
  if (i >= (int)p.ctrl[kLossTok]) return;
  const float k = __uint_as_float(p.ctrl[kLossScale]);
  const size_t step = (size_t)p.Tp * p.Kx;
  float* x = p.dxp + (size_t)i * p.Kx;
  const float lost = p.qres ? p.qres[i] : 0.f;
  const size_t row = (size_t)loss_head_row(p, p.lab[i]);
  for (int c = threadIdx.x; c < p.Kx; c += blockDim.x) {
    const bool head = c < p.Hp;
    if (head ? !p.d_hidden || c >= p.H : !p.d_w1 || c - p.Hp >= p.r) continue;
    float a = x[c];
    for (int s = 1; s < p.splits; ++s) a += x[s * step + c];
    if (p.qres)
      a += lost * to_f32(head ? ((const E*)p.lm_head)[row * p.H + c]
                              : ((const E*)p.w2)[(size_t)(c - p.Hp) * p.Vh + row]);
    a *= k;
    if (head)
      ((E*)p.d_hidden)[(size_t)p.tok[i] * p.H + c] = from_f32<E>(a);
    else
      x[c] = a;
  }
}

// CTA i, when row i is the first with its prev: sums the gradients of the rows with that
// prev in row order, each warp over its share of the rows, the warps in order.
template <typename E>
__global__ void __launch_bounds__(256) loss_w1_rows(const LossPlan p) {
  __shared__ bool s_seen;
  extern __shared__ float s_acc[];             // [warps][rp]
  const int n_tok = (int)p.ctrl[kLossTok], i = blockIdx.x, tid = threadIdx.x;
  const int lane = tid % 32, warp = tid / 32, warps = blockDim.x / 32;
  if (i >= n_tok) return;
  const int pv = p.prevc[i];
  if (tid == 0) s_seen = false;
  __syncthreads();
  bool seen = false;
  for (int j = tid; j < i; j += blockDim.x) seen |= p.prevc[j] == pv;
  if (seen) s_seen = true;
  __syncthreads();
  if (s_seen) return;
  float* acc = s_acc + (size_t)warp * p.rp;
  for (int c = lane; c < p.rp; c += 32) acc[c] = 0.f;
  const int share = (n_tok - i + warps * 32 - 1) / (warps * 32) * 32;
  const int j0 = i + warp * share, j1 = min(n_tok, j0 + share);
  for (int jb = j0; jb < j1; jb += 32) {
    unsigned m = __ballot_sync(0xFFFFFFFFu, jb + lane < j1 && p.prevc[jb + lane] == pv);
    while (m) {
      const int j = jb + __ffs(m) - 1;
      m &= m - 1;
      const float* g = p.dxp + (size_t)j * p.Kx + p.Hp;
      for (int c = lane; c < p.rp; c += 32) acc[c] += g[c];
    }
  }
  __syncthreads();
  for (int c = tid; c < p.r; c += blockDim.x) {
    float a = 0.f;
    for (int w = 0; w < warps; ++w) a += s_acc[(size_t)w * p.rp + c];
    ((E*)p.d_w1)[(size_t)pv * p.r + c] = from_f32<E>(a);
  }
}

}  // namespace

cudaError_t launch_loss_plan(const LossPlan& p) {
  cudaError_t e = cudaSuccess;
  if (p.vlist) {
    int chunks = 0;
    e = launch_emit_rows(p.bias, p.Vh, p.vchunk, p.vlist, &chunks, p.stream);
    if (e != cudaSuccess) return e;
    e = cudaMemsetAsync(p.vinv, 0xFF, sizeof(int32_t) * (size_t)p.Vh, p.stream);
    if (e != cudaSuccess) return e;
    loss_vocab<<<std::min(256, (p.Vh + 255) / 256), 256, 0, p.stream>>>(p, chunks);
    if (p.wc) loss_gather_head<<<1216, 256, 0, p.stream>>>(p);
  }
  loss_tokens<<<1, kPlanThreads, 0, p.stream>>>(p);
  const size_t es = p.dtype == 0 ? 4 : 2;
  if (p.d_w1) {
    e = cudaMemsetAsync(p.d_w1, 0, es * (size_t)p.V * p.r, p.stream);
    if (e != cudaSuccess) return e;
  }
  if (p.vlist && p.d_lm_head) {
    e = cudaMemsetAsync(p.d_lm_head, 0, es * (size_t)p.Vh * p.H, p.stream);
    if (e != cudaSuccess) return e;
  }
  if (p.vlist && p.d_w2) {
    e = cudaMemsetAsync(p.d_w2, 0, es * (size_t)p.Vh * p.r, p.stream);
    if (e != cudaSuccess) return e;
  }
  if (p.dtype == 0)
    loss_gather<float><<<p.Tp, 256, 0, p.stream>>>(p);
  else
    loss_gather<__nv_bfloat16><<<p.Tp, 256, 0, p.stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_loss_rows(const LossPlan& p) {
  loss_rows<<<p.T, 128, 0, p.stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_loss_dz(const LossPlan& p, int v0, int v1) {
  if (p.dtype == 0) {
    const unsigned blocks = (unsigned)std::min(64, (v1 - v0 + 255) / 256);
    loss_dz_f32<<<dim3((unsigned)p.T, blocks), 256, 0, p.stream>>>(p, v0, v1);
  } else {
    const unsigned blocks = (unsigned)std::min(16, (p.Vh + 2047) / 2048);
    loss_dz_bf16<<<dim3((unsigned)p.T, blocks), 256, 0, p.stream>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_loss_dx(const LossPlan& p) {
  const bool f32 = p.dtype == 0;
  if (f32)
    loss_dx_rows<float><<<p.T, 256, 0, p.stream>>>(p);
  else
    loss_dx_rows<__nv_bfloat16><<<p.T, 256, 0, p.stream>>>(p);
  if (p.d_w1) {
    const size_t smem = sizeof(float) * 8 * (size_t)p.rp;
    if (f32)
      loss_w1_rows<float><<<p.T, 256, smem, p.stream>>>(p);
    else
      loss_w1_rows<__nv_bfloat16><<<p.T, 256, smem, p.stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace dspark
