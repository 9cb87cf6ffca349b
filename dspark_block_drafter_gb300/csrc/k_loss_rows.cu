// The training loss of the head, all but its products: which rows carry a loss, the
// operand rows X, the softmax statistics joined over the vocabulary, the losses and their
// total, and the gradients that are sums over rows of X's gradient.
//
// Every kernel here is bound by its traffic or its latency; sums over rows are taken in a
// fixed order.  Sums of many values carry their rounding errors along in a second fp32 value:
// fp64 additions run at a few per clock and SM here (with them the compaction alone took
// 16 us for a handful of rows).
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "launch.h"
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

// Copies n elements, sixteen bytes at a time where both sides allow it.
template <typename E>
__device__ __forceinline__ void copy_row(E* dst, const E* src, int n) {
  constexpr int kVec = 16 / sizeof(E);
  int at = 0;
  if ((((uintptr_t)dst | (uintptr_t)src) & 15) == 0) {
    at = n / kVec * kVec;
    for (int k = threadIdx.x; k < n / kVec; k += blockDim.x)
      reinterpret_cast<uint4*>(dst)[k] = reinterpret_cast<const uint4*>(src)[k];
  }
  for (int k = at + threadIdx.x; k < n; k += blockDim.x) dst[k] = src[k];
}

template <typename E>
__device__ __forceinline__ void zero_row(E* dst, int n) {
  constexpr int kVec = 16 / sizeof(E);
  int at = 0;
  if (((uintptr_t)dst & 15) == 0) {
    at = n / kVec * kVec;
    for (int k = threadIdx.x; k < n / kVec; k += blockDim.x)
      reinterpret_cast<uint4*>(dst)[k] = make_uint4(0, 0, 0, 0);
  }
  for (int k = at + threadIdx.x; k < n; k += blockDim.x) dst[k] = from_f32<E>(0.f);
}

// Bias form: the compact vocabulary's size, inverse map and biases.  vinv is -1 before.
__global__ void __launch_bounds__(256) loss_vocab(const LossPlan p, int chunks) {
  pdl_wait();
  pdl_signal();
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
    // first entry >= t: seven probes at a time, since each is a trip to memory
    int lo = 0, hi = p.Vh;
    while (hi > lo) {
      const int n = hi - lo;
      int above = 0;                              // probes whose entry is below t
#pragma unroll
      for (int q = 1; q < 8; ++q) above += p.d2t[lo + (int)((long long)n * q / 8)] < t;
      // entries lo + n q / 8 (q <= above) are below t, the next one is not
      const int l = lo, h = hi;
      if (above > 0) lo = l + (int)((long long)n * above / 8) + 1;
      if (above < 7) hi = l + (int)((long long)n * (above + 1) / 8);
      else hi = h;
    }
    if (lo >= p.Vh || p.d2t[lo] != t) return -1;
    row = lo;
  }
  return p.vinv ? p.vinv[row] : row;
}

// Splits of the vocabulary in dX's sum over it, chosen by one warp once the rows are counted.
// bf16: a unit (a tile of dX over one split) costs its K-blocks of 64, about 12 K-blocks'
// time for filling the pipeline and writing its partial result, and that result's traffic
// (256 KB written and read: 0.23 K-blocks' time of the whole GPU); CTAs (pairs above 128
// rows) take the units in waves, and pairs the tiles of dW after them, which even out an
// incomplete wave.  The count with the least total is taken.  Measured for dX and its sum
// alone, 512 rows of the 151936 x 4096 head: 2 splits 409 us (chosen), 1 698 us, 3 530 us,
// 5 501 us, 13 442 us.
__device__ __forceinline__ int loss_pick_splits(const LossPlan& p, int n_tok, int n_voc, int lane) {
  if (p.dtype == 0) return p.splits;
  const bool pairs = p.T > 128;
  const int cols = min(p.piece_cols, n_voc), head = (p.Hp + 255) / 256, markov = (p.rp + 255) / 256;
  const int tiles = max(1, (n_tok + 255) / 256) * ((p.d_hidden ? head : 0) + (p.d_w1 ? markov : 0));
  const int ctas = pairs ? 76 : 152, nkb = (cols + 63) / 64;
  const int n_dw = pairs ? (cols + 255) / 256 * ((p.d_lm_head ? head : 0) + (p.d_w2 ? markov : 0)) : 0;
  const float dw = (float)n_dw * fmaxf((float)((n_tok + 63) / 64) + 2.f, 11.f);
  const int most = (int)min((size_t)p.splits, p.dx_rows / loss_split_rows(n_tok));
  float cost = INFINITY;
  int best = 1;
  for (int s = 1 + lane; s <= most && (s == 1 || s * 8 <= nkb); s += 32) {
    const float unit = (float)nkb / (float)s + 12.f;
    const float waves = (float)((tiles * s + ctas - 1) / ctas) * unit;
    const float even = ((float)(tiles * s) * unit + dw) / (float)ctas;
    const float c = fmaxf(waves, even) + 0.23f * (float)(tiles * s);
    if (c < cost) {
      cost = c;
      best = s;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float c = __shfl_xor_sync(0xFFFFFFFFu, cost, o);
    const int b = __shfl_xor_sync(0xFFFFFFFFu, best, o);
    if (c < cost || (c == cost && b < best)) {
      cost = c;
      best = b;
    }
  }
  return best;
}

// One CTA: compacts the rows that carry a loss, in order, and sums their weights.  Each
// thread takes kPlanRows rows of a sweep, so that their loads overlap.
constexpr int kPlanRows = 4;
__global__ void __launch_bounds__(kPlanThreads) loss_tokens(const LossPlan p) {
  pdl_wait();
  pdl_signal();
  __shared__ int s_cnt[32];
  __shared__ float2 s_w[32];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, warps = blockDim.x / 32;
  for (int c = tid; c < 64; c += blockDim.x)
    if (c != kLossVoc) p.ctrl[c] = 0;
  if (tid == 0 && !p.vlist) p.ctrl[kLossVoc] = (uint32_t)p.Vh;
  __syncthreads();
  int base = 0;
  Sum2 wsum;
  for (int t0 = 0; t0 < p.T; t0 += kPlanRows * blockDim.x) {
    int j[kPlanRows], pv[kPlanRows];
    float w[kPlanRows];
#pragma unroll
    for (int q = 0; q < kPlanRows; ++q) {
      const int t = t0 + q * blockDim.x + tid;
      j[q] = t < p.T ? p.labels[t] : -1;
      pv[q] = t < p.T && p.r > 0 ? p.prev[t] : 0;
      w[q] = t < p.T && p.weights ? p.weights[t] : 1.f;
    }
#pragma unroll
    for (int q = 0; q < kPlanRows; ++q) {
      if (j[q] >= p.V) {
        flag_error(p.ctrl, kErrBadToken);
        j[q] = -1;
      }
      if (j[q] >= 0) j[q] = loss_label_row(p, j[q]);
      if (j[q] >= 0 && p.r > 0 && (pv[q] < 0 || pv[q] >= p.V)) {
        flag_error(p.ctrl, kErrBadToken);
        j[q] = -1;
      }
    }
#pragma unroll
    for (int q = 0; q < kPlanRows; ++q) {
      const int t = t0 + q * blockDim.x + tid;
      const unsigned m = __ballot_sync(0xFFFFFFFFu, j[q] >= 0);
      __syncthreads();
      if (lane == 0) s_cnt[warp] = __popc(m);
      __syncthreads();
      int n = lane < warps ? s_cnt[lane] : 0;     // inclusive scan over the warps
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, n, o);
        if (lane >= o) n += y;
      }
      const int all = __shfl_sync(0xFFFFFFFFu, n, 31);
      const int before = warp > 0 ? __shfl_sync(0xFFFFFFFFu, n, warp - 1) : 0;
      if (t < p.T) {
        const int i = base + before + __popc(m & ((1u << lane) - 1));
        p.pos[t] = j[q] >= 0 ? i : -1;
        if (j[q] >= 0) {
          p.tok[i] = t;
          p.lab[i] = j[q];
          p.prevc[i] = pv[q];
          p.wrow[i] = w[q];
          wsum.add(w[q]);
        }
      }
      base += all;
    }
  }
  if (warp == 0 && p.dxp) {
    const int best = loss_pick_splits(p, base, (int)p.ctrl[kLossVoc], lane);
    if (lane == 0) p.ctrl[kLossSplits] = (uint32_t)best;
  }
  const float w = block_sum(wsum, s_w).value();
  if (tid == 0) {
    p.ctrl[kLossTok] = (uint32_t)base;
    float k = p.loss_scale;
    if (p.reduction == 1) k = w > 0.f ? p.loss_scale / w : 0.f;
    p.ctrl[kLossScale] = __float_as_uint(k);
    if (p.n_rows) *p.n_rows = base;
  }
}

// fp32: the plan's zeros, by all CTAs of the launch (bf16 writes them beside its products).
template <typename E>
__device__ __forceinline__ void zero_outputs(const LossPlan& p) {
  if (sizeof(E) != 4) return;
  for (int z = 0; z < p.n_zero; ++z) {
    float* f = (float*)p.zero[z].p;
    const size_t n = p.zero[z].bytes / 4;
    for (size_t k = (size_t)blockIdx.x * blockDim.x + threadIdx.x; k < n;
         k += (size_t)gridDim.x * blockDim.x)
      f[k] = 0.f;
  }
}

// Row t's part of X as compact row i (and with `low` once more), or its zero outputs when it
// carries no loss (i < 0).
template <typename E>
__device__ __forceinline__ void gather_row(const LossPlan& p, int t, int i, int prev, bool low) {
  if (i < 0) {
    if (threadIdx.x == 0) p.loss[t] = 0.f;
    if (p.d_hidden) zero_row((E*)p.d_hidden + (size_t)t * p.H, p.H);
    return;
  }
  for (int row = i; row <= i + (low ? kLossLow : 0); row += kLossLow) {
    E* xi = (E*)p.x + (size_t)row * p.Kx;
    copy_row(xi, (const E*)p.hidden + (size_t)t * p.H, p.H);
    if (p.H < p.Hp) zero_row(xi + p.H, p.Hp - p.H);
    if (p.rp == 0) continue;
    copy_row(xi + p.Hp, (const E*)p.w1 + (size_t)prev * p.r, p.r);
    if (p.r < p.rp) zero_row(xi + p.Hp + p.r, p.rp - p.r);
  }
}

// Row t of X after the compact rows: zeros, unless a low row's copy goes there.
template <typename E>
__device__ __forceinline__ void pad_row(const LossPlan& p, int t, int n_tok) {
  if (t < n_tok || (loss_low(p, n_tok) && t >= kLossLow && t < kLossLow + n_tok)) return;
  zero_row((E*)p.x + (size_t)t * p.Kx, p.Kx);
}

// CTA t: row t's part of X, and X's padding row t.
template <typename E>
__global__ void __launch_bounds__(256) loss_gather(const LossPlan p) {
  pdl_wait();
  pdl_signal();
  zero_outputs<E>(p);
  const int t = blockIdx.x, n_tok = (int)p.ctrl[kLossTok];
  pad_row<E>(p, t, n_tok);
  if (t >= p.T) return;
  const int i = p.pos[t];
  gather_row<E>(p, t, i, i >= 0 ? p.prevc[i] : 0, loss_low(p, n_tok));
}

// loss_tokens and loss_gather in one launch, for few rows: every CTA looks at every row for
// its own place among them, and CTA 0 writes down what loss_tokens does.  (Rows times rows of
// work: taken up to kPlanFew rows, and not with a d2t map, whose searches would be repeated.)
constexpr int kPlanFew = 512;
template <typename E>
__global__ void __launch_bounds__(256) loss_plan_few(const LossPlan p) {
  pdl_wait();
  pdl_signal();
  __shared__ int s_before[8], s_all[8];
  __shared__ float2 s_w[32];
  const int me = blockIdx.x, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const bool lead = me == 0;
  if (lead) {
    if (tid < 64 && tid != kLossVoc) p.ctrl[tid] = 0;
    if (tid == 64 && !p.vlist) p.ctrl[kLossVoc] = (uint32_t)p.Vh;
    __syncthreads();
  }
  int before = 0, all = 0;                        // rows with a loss: before `me`, in all
  int mine = -1, prev = 0;                        // this CTA's own row
  Sum2 wsum;
  for (int t = tid; t < p.T; t += 256) {
    int j = p.labels[t];
    const int pv = p.r > 0 ? p.prev[t] : 0;
    if (j >= p.V) {
      if (lead) flag_error(p.ctrl, kErrBadToken);
      j = -1;
    }
    if (j >= 0) j = loss_label_row(p, j);
    if (j >= 0 && p.r > 0 && (pv < 0 || pv >= p.V)) {
      if (lead) flag_error(p.ctrl, kErrBadToken);
      j = -1;
    }
    all += j >= 0;
    before += j >= 0 && t < me;
    if (t == me) {
      mine = j;
      prev = pv;
    }
    if (lead && j >= 0) wsum.add(p.weights ? p.weights[t] : 1.f);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
    all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
  }
  if (lane == 0) {
    s_before[warp] = before;
    s_all[warp] = all;
  }
  __shared__ int s_mine, s_prev;
  if (tid == 0) s_mine = -1;
  __syncthreads();
  if (me < p.T && tid == me % 256) {              // (the thread that looked at row `me`)
    s_mine = mine;
    s_prev = prev;
  }
  __syncthreads();
  before = all = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    before += s_before[w];
    all += s_all[w];
  }
  const int label = s_mine;
  zero_outputs<E>(p);
  if (lead) {
    if (warp == 0 && p.dxp) {
      const int best = loss_pick_splits(p, all, (int)p.ctrl[kLossVoc], lane);
      if (lane == 0) p.ctrl[kLossSplits] = (uint32_t)best;
    }
    const float w = block_sum(wsum, s_w).value();
    if (tid == 0) {
      p.ctrl[kLossTok] = (uint32_t)all;
      float k = p.loss_scale;
      if (p.reduction == 1) k = w > 0.f ? p.loss_scale / w : 0.f;
      p.ctrl[kLossScale] = __float_as_uint(k);
      if (p.n_rows) *p.n_rows = all;
    }
  }
  pad_row<E>(p, me, all);
  if (me >= p.T) return;
  if (label >= 0 && tid == 0) {
    p.tok[before] = me;
    p.lab[before] = label;
    p.prevc[before] = s_prev;
    p.wrow[before] = p.weights ? p.weights[me] : 1.f;
  }
  gather_row<E>(p, me, label >= 0 ? before : -1, label >= 0 ? s_prev : 0, loss_low(p, all));
}

// Row i's log-sum-exp and loss, from its label's logit and the statistics of the others over
// the vocabulary tiles (thread 0 has them; the CTA takes part).  Where the label's logit z is
// the largest, the loss is log1p(sum of the others' e^(z_j - z)): a small loss keeps its digits
// (as the difference of log-sum-exp and z, one of 1e-5 was off by 0.6%, and so was the label's
// entry of the gradient).
constexpr int kRowsThreads = 256;
__device__ __forceinline__ float2 join_row(const LossPlan& p, int i, int n_voc, float2* s_w) {
  const int tid = threadIdx.x, n = (n_voc + p.stat_cols - 1) / p.stat_cols;
  const float zl = p.zlab[i];
  const float2* st = p.stat + (size_t)i * p.n_stat;
  // running maximum and sum over sweeps of eight tiles a thread (a maximum of -inf: all its
  // logits are, and its sum is 0)
  float m = -INFINITY, s = 0.f;
  for (int j0 = tid; j0 < n; j0 += 8 * kRowsThreads) {
    float2 a[8];
    float mm = m;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int j = j0 + q * kRowsThreads;
      a[q] = j < n ? st[j] : make_float2(-INFINITY, 0.f);
      mm = fmaxf(mm, a[q].x);
    }
    const float ref = mm > -INFINITY ? mm : 0.f;
    s *= __expf(m - ref);
#pragma unroll
    for (int q = 0; q < 8; ++q) s += a[q].y * __expf(a[q].x - ref);
    m = mm;
  }
  // joined over the CTA: the maxima, then the sums at the common maximum
  float mx = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  if (tid % 32 == 0) s_w[tid / 32].x = mx;
  __syncthreads();
  mx = s_w[0].x;
#pragma unroll
  for (int w = 1; w < kRowsThreads / 32; ++w) mx = fmaxf(mx, s_w[w].x);
  const float ref = mx > -INFINITY ? mx : 0.f;
  Sum2 v;
  v.s = s * __expf(m - ref);
  __syncthreads();
  const float sum = block_sum(v, s_w).value();
  if (zl >= mx) {
    // (z - z: an infinite z is no loss of 0)
    const float l = log1pf(mx > -INFINITY ? sum * expf(mx - zl) : 0.f) + (zl - zl);
    return make_float2(zl + l, l);
  }
  const float l = logf(sum + expf(zl - ref));
  return make_float2(mx + l, (mx - zl) + l);
}

// q = w (softmax - onehot) of row i in place, fp32 from stored logits: columns [v0, v1), every
// `parts`-th run of 256 of them from run `part` on.
__device__ __forceinline__ void row_dz_f32(const LossPlan& p, int i, int v0, int v1, float lse,
                                           float loss, int part, int parts) {
  float* q = (float*)p.q + (size_t)i * p.ldq;
  const float w = p.wrow[i];
  const int lab = p.lab[i];
  for (int v = v0 + part * blockDim.x + threadIdx.x; v < v1; v += parts * blockDim.x)
    q[v - v0] = v == lab ? loss_label_entry(w, loss) : w * __expf(q[v - v0] - lse);
}

// The same in bf16 from the stored distances (one piece: v0 = 0), over whole 256-column
// tiles: columns past the vocabulary become 0.  Two vectors of eight columns a thread and
// sweep; the thread that has the label's column writes it again.
__device__ __forceinline__ void row_dz_bf16(const LossPlan& p, int i, int n_voc, bool low,
                                            float lse, float loss, int part, int parts) {
  uint4* q = (uint4*)((uint16_t*)p.q + (size_t)i * p.ldq);
  const float2* st = p.stat + (size_t)i * p.n_stat;
  const float w = p.wrow[i], log2_w = log2f(w);              // (w = 0: -inf, e = 0)
  const float far = lse - lse;     // 0; NaN in every column when a logit of the row is NaN or +inf
  const int lab = p.lab[i], end = (n_voc + 255) / 256 * 32, tiles = (n_voc + 127) / 128;
  const int step = parts * blockDim.x;
  for (int c0 = part * blockDim.x + threadIdx.x; c0 < end; c0 += 2 * step) {
    uint4 x[2];
    float s[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = c0 + h * step;
      if (c >= end) break;
      x[h] = q[c];
      // (a tile past the last is all far)
      s[h] = fmaf(st[min(c / 16, tiles - 1)].x - lse, 1.44269504f, log2_w);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = c0 + h * step;
      if (c >= end) break;
      const uint32_t g[4] = {x[h].x, x[h].y, x[h].z, x[h].w};
      uint32_t o[4], r[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e0 = loss_gap_exp(g[j] & 0xFFFFu, s[h], far);
        const float e1 = loss_gap_exp(g[j] >> 16, s[h], far);
        const __nv_bfloat162 b = __floats2bfloat162_rn(e0, e1);
        o[j] = *reinterpret_cast<const uint32_t*>(&b);
        if (low) {
          const __nv_bfloat162 l =
              __floats2bfloat162_rn(e0 - __low2float(b), e1 - __high2float(b));
          r[j] = *reinterpret_cast<const uint32_t*>(&l);
        }
      }
      q[c] = make_uint4(o[0], o[1], o[2], o[3]);
      if (low) q[kLossLow * p.ldq / 8 + c] = make_uint4(r[0], r[1], r[2], r[3]);
      if (lab / 8 == c)
        loss_put_label(p, i, low, reinterpret_cast<__nv_bfloat16*>(q) + lab,
                       loss_label_entry(w, loss));
    }
  }
}

// CTAs (i, 0 .. ): each joins row i's statistics, the first writes them down, and with DZ each
// makes its part of the row's q (1: bf16, 2: fp32; one piece).  The last CTA to finish a row
// sums the losses.
template <int DZ>
__global__ void __launch_bounds__(kRowsThreads) loss_rows(const LossPlan p) {
  pdl_wait();
  pdl_signal();
  __shared__ float2 s_w[32];
  __shared__ float2 s_row;
  __shared__ bool s_last;
  const int n_tok = (int)p.ctrl[kLossTok], n_voc = (int)p.ctrl[kLossVoc];
  const int i = blockIdx.x, tid = threadIdx.x;
  const bool first = blockIdx.y == 0;
  if (i < n_tok) {
    const float2 joined = join_row(p, i, n_voc, s_w);
    if (tid == 0) {
      s_row = joined;
      if (first) {
        p.lse[i] = joined.x;
        p.loss[p.tok[i]] = joined.y;
      }
    }
    __syncthreads();
    const float2 r = s_row;
    if (DZ == 1) row_dz_bf16(p, i, n_voc, loss_low(p, n_tok), r.x, r.y, blockIdx.y, gridDim.y);
    if (DZ == 2) row_dz_f32(p, i, 0, n_voc, r.x, r.y, blockIdx.y, gridDim.y);
  }
  if (!first) return;
  if (tid == 0) {
    __threadfence();
    s_last = atomicAdd(p.ctrl + kLossDone, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (s_last) {
    __threadfence();
    Sum2 a;
    constexpr int kAt = 8;                    // (rows of a thread at once)
    for (int j0 = tid; j0 < n_tok; j0 += kAt * kRowsThreads) {
      float w[kAt], x[kAt];
#pragma unroll
      for (int q = 0; q < kAt; ++q) {
        const int j = j0 + q * kRowsThreads;
        w[q] = j < n_tok ? p.wrow[j] : 0.f;
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
    const Sum2 t = block_sum(a, s_w);
    if (tid == 0) *p.total = n_tok > 0 ? __uint_as_float(p.ctrl[kLossScale]) * t.value() : 0.f;
  }
}

// q of columns [v0, v1) from stored logits, once the rows' log-sum-exps are known (pieces).
__global__ void __launch_bounds__(256) loss_dz_f32(const LossPlan p, int v0, int v1) {
  pdl_wait();
  pdl_signal();
  const int i = blockIdx.x;
  if (i >= (int)p.ctrl[kLossTok]) return;
  row_dz_f32(p, i, v0, min(v1, (int)p.ctrl[kLossVoc]), p.lse[i], p.loss[p.tok[i]], blockIdx.y,
             gridDim.y);
}

// The compact head of a bias-form bf16 head, with zeros up to a multiple of 256: its rows, a
// warp each, and behind the first `row_ctas` CTAs its columns of markov_w2, 256 columns x 8
// rows a CTA.
__global__ void __launch_bounds__(256) loss_gather_head(const LossPlan p, int row_ctas) {
  pdl_wait();
  pdl_signal();
  const int n = (int)p.ctrl[kLossVoc], end = min(p.Vh, (n + 255) / 256 * 256);
  if ((int)blockIdx.x >= row_ctas) {
    const int b = blockIdx.x - row_ctas, groups = (p.r + 7) / 8;
    const int j = b / groups * 256 + threadIdx.x, k0 = b % groups * 8;
    if (j >= end) return;
    const __nv_bfloat16* w2 = (const __nv_bfloat16*)p.w2;
    __nv_bfloat16* w2c = (__nv_bfloat16*)p.w2c;
    const int v = j < n ? p.vlist[j] : -1;
    __nv_bfloat16 x[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
      x[q] = v >= 0 && k0 + q < p.r ? w2[(size_t)(k0 + q) * p.Vh + v] : __float2bfloat16(0.f);
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (k0 + q < p.r) w2c[(size_t)(k0 + q) * p.Vh + j] = x[q];
    return;
  }
  const int per = p.H / 8, lane = threadIdx.x % 32;
  const uint4* w = (const uint4*)p.lm_head;
  uint4* wc = (uint4*)p.wc;
  for (int j = blockIdx.x * 8 + threadIdx.x / 32; j < end; j += row_ctas * 8) {
    const bool in = j < n;
    const size_t from = in ? (size_t)p.vlist[j] * per : 0;
    for (int k0 = lane; k0 < per; k0 += 8 * 32) {
      uint4 x[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int k = k0 + 32 * q;
        x[q] = in && k < per ? __ldcs(w + from + k) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (k0 + 32 * q < per) wc[(size_t)j * per + k0 + 32 * q] = x[q];
    }
  }
}

// CTAs (i, 0 .. ): row i of the gradient of X, summed over the splits of the vocabulary (and, in
// bf16, with what q lost at the label), times the scale: d_hidden's row, and the gradient of
// markov_w1's row prev (left in split 0).
template <typename E>
__global__ void __launch_bounds__(256) loss_dx_rows(const LossPlan p) {
  pdl_wait();
  pdl_signal();
  const int i = blockIdx.x;
  if (i >= (int)p.ctrl[kLossTok]) return;
  const float k = __uint_as_float(p.ctrl[kLossScale]);
  const size_t step = (size_t)loss_split_rows((int)p.ctrl[kLossTok]) * p.Kx / 4;
  const int splits = (int)p.ctrl[kLossSplits];
  float4* x = (float4*)(p.dxp + (size_t)i * p.Kx);
  const float lost = p.qres ? p.qres[i] : 0.f;
  const bool low = loss_low(p, (int)p.ctrl[kLossTok]);
  const size_t row = (size_t)loss_head_row(p, p.lab[i]);
  E* dh = p.d_hidden ? (E*)p.d_hidden + (size_t)p.tok[i] * p.H : nullptr;
  // four columns a thread (Hp and Kx are multiples of 64)
  const int from = p.d_hidden ? 0 : p.Hp / 4, to = p.d_w1 ? p.Kx / 4 : p.Hp / 4;
  for (int c4 = from + blockIdx.y * blockDim.x + threadIdx.x; c4 < to;
       c4 += gridDim.y * blockDim.x) {
    float a[4] = {};
    const int parts = low ? 2 * splits : splits;       // (the splits, then the low row's)
    const size_t low0 = (size_t)kLossLow * p.Kx / 4;
    for (int s0 = 0; s0 < parts; s0 += 8) {
      float4 y[8];
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        const int s = s0 + b;
        y[b] = s < parts ? __ldcs(x + (s < splits ? s * step : low0 + (s - splits) * step) + c4)
                         : make_float4(0, 0, 0, 0);
      }
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        a[0] += y[b].x; a[1] += y[b].y; a[2] += y[b].z; a[3] += y[b].w;
      }
    }
    const int c = 4 * c4;
    const bool head = c < p.Hp;
    if (p.qres) {                             // (bf16: H is a multiple of 8)
      if (head) {
        if (c < p.H) {
          struct alignas(4 * sizeof(E)) Four { E e[4]; };
          const Four w = *reinterpret_cast<const Four*>((const E*)p.lm_head + row * p.H + c);
#pragma unroll
          for (int j = 0; j < 4; ++j) a[j] += lost * to_f32(w.e[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (c + j - p.Hp < p.r)
            a[j] += lost * to_f32(((const E*)p.w2)[(size_t)(c + j - p.Hp) * p.Vh + row]);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] *= k;
    if (head) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + j < p.H) dh[c + j] = from_f32<E>(a[j]);
    } else {
      x[c4] = make_float4(a[0], a[1], a[2], a[3]);
    }
  }
}

// CTA i, when row i is the first with its prev: sums the gradients of the rows with that
// prev in row order, each warp over its share of the rows, the warps in order.  A warp looks
// at 128 rows at a time and adds two of them at a time, in registers: common tokens precede many
// rows.  (4096 rows, rank 256: 18 us, with seven different prev 40; one row at a time into shared
// memory 49 and 129.)  Sums of more than kW1Chain rows are sums of such parts: one chain of 131072
// fp32 additions a warp was off by 4e-6.
constexpr int kW1Chain = 4096;
template <typename E>
__global__ void __launch_bounds__(256) loss_w1_rows(const LossPlan p) {
  pdl_wait();
  pdl_signal();
  __shared__ bool s_seen;
  __shared__ int s_list[8][128];
  extern __shared__ float s_acc[];             // [warps][rp]
  const int n_tok = (int)p.ctrl[kLossTok], i = blockIdx.x, tid = threadIdx.x;
  const int lane = tid % 32, warp = tid / 32, warps = blockDim.x / 32;
  if (i >= n_tok) return;
  const int pv = p.prevc[i];
  if (tid == 0) s_seen = false;
  __syncthreads();
  bool seen = false;
#pragma unroll 8
  for (int j = tid; j < i; j += 256) seen |= p.prevc[j] == pv;
  if (seen) s_seen = true;
  __syncthreads();
  if (s_seen) return;
  const int share = (n_tok - i + warps * 32 - 1) / (warps * 32) * 32;
  const int j0 = i + warp * share, j1 = min(n_tok, j0 + share);
  int* list = s_list[warp];
  for (int c0 = lane; c0 < p.rp; c0 += 256) {          // (256 columns at a time)
    float acc[8] = {}, sum[8] = {};
    for (int jb = j0; jb < j1; jb += 128) {
      if (jb > j0 && (jb - j0) % kW1Chain == 0) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          sum[q] += acc[q];
          acc[q] = 0.f;
        }
      }
      bool hit[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int j = jb + 32 * q + lane;
        hit[q] = j < j1 && p.prevc[j] == pv;
      }
      int n = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const unsigned m = __ballot_sync(0xFFFFFFFFu, hit[q]);
        if (hit[q]) list[n + __popc(m & ((1u << lane) - 1u))] = jb + 32 * q + lane;
        n += __popc(m);
      }
      __syncwarp();
      for (int k = 0; k < n; k += 2) {
        float g[2][8];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const float* row = p.dxp + (size_t)list[min(k + b, n - 1)] * p.Kx + p.Hp + c0;
#pragma unroll
          for (int q = 0; q < 8; ++q)
            g[b][q] = k + b < n && c0 + 32 * q < p.rp ? row[32 * q] : 0.f;
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[q] = (acc[q] + g[0][q]) + g[1][q];
      }
      __syncwarp();
    }
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (c0 + 32 * q < p.rp) s_acc[(size_t)warp * p.rp + c0 + 32 * q] = sum[q] + acc[q];
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
  const bool f32 = p.dtype == 0;
  cudaError_t e = cudaSuccess;
  if (p.vlist) {
    int chunks = 0;
    e = cudaMemsetAsync(p.vinv, 0xFF, sizeof(int32_t) * (size_t)p.Vh, p.stream);
    if (e == cudaSuccess) e = launch_emit_rows(p.bias, p.Vh, p.vchunk, p.vlist, &chunks, p.stream);
    if (e == cudaSuccess)
      e = launch_after(loss_vocab, std::min(256, (p.Vh + 255) / 256), 256, 0, p.stream, p, chunks);
    if (e == cudaSuccess && p.wc) {
      const int rows = std::min(1216, (p.Vh + 7) / 8);
      const int cols = (p.Vh + 255) / 256 * ((p.r + 7) / 8);
      e = launch_after(loss_gather_head, rows + cols, 256, 0, p.stream, p, rows);
    }
  }
  if (e != cudaSuccess) return e;
  if (p.T <= kPlanFew && !p.d2t)
    return launch_after(f32 ? loss_plan_few<float> : loss_plan_few<__nv_bfloat16>, p.Tp, 256, 0,
                        p.stream, p);
  e = launch_after(loss_tokens, 1, std::min(kPlanThreads, (p.T + 31) / 32 * 32), 0, p.stream, p);
  if (e == cudaSuccess)
    e = launch_after(f32 ? loss_gather<float> : loss_gather<__nv_bfloat16>, p.Tp, 256, 0, p.stream,
                     p);
  return e;
}

cudaError_t launch_loss_rows(const LossPlan& p, bool dz) {
  if (!dz) return launch_after(loss_rows<0>, p.T, kRowsThreads, 0, p.stream, p);
  // CTAs of a row: enough to fill the GPU, each with some sweeps to do
  const int most = p.dtype == 0 ? (p.Vh + 255) / 256 : (p.Vh + 4095) / 4096;
  const unsigned parts = (unsigned)std::max(1, std::min({16, most, (2 * 1216 + p.T - 1) / p.T}));
  return launch_after(p.dtype == 0 ? loss_rows<2> : loss_rows<1>, dim3((unsigned)p.T, parts),
                      kRowsThreads, 0, p.stream, p);
}

cudaError_t launch_loss_dz_f32(const LossPlan& p, int v0, int v1) {
  const unsigned blocks = (unsigned)std::min(64, (v1 - v0 + 255) / 256);
  return launch_after(loss_dz_f32, dim3((unsigned)p.T, blocks), 256, 0, p.stream, p, v0, v1);
}

cudaError_t launch_loss_dx(const LossPlan& p) {
  const bool f32 = p.dtype == 0;
  // several CTAs a row where rows alone do not fill the GPU: 37 rows of 2304 columns take 14 us
  // with one CTA each, 7 with three
  const unsigned y = (unsigned)std::max(1, std::min((p.Kx / 4 + 255) / 256, 1216 / p.T));
  cudaError_t e = launch_after(f32 ? loss_dx_rows<float> : loss_dx_rows<__nv_bfloat16>,
                               dim3((unsigned)p.T, y), 256, 0, p.stream, p);
  if (e == cudaSuccess && p.d_w1)
    e = launch_after(f32 ? loss_w1_rows<float> : loss_w1_rows<__nv_bfloat16>, p.T, 256,
                     sizeof(float) * 8 * (size_t)p.rp, p.stream, p);
  return e;
}

}  // namespace dspark
