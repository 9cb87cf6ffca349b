// The training loss of the head: its three products on the CUDA cores, in fp32.
//
//   logits  z[i][j]  = X[i] . [lm_head[j] | markov_w2[:, j]] + bias[j]
//   dX      dx[i][c] = sum_j q[i][j] [lm_head | markov_w2^T][j][c]
//   dW      [d_lm_head | d_markov_w2^T][j][c] = scale * sum_i q[i][j] X[i][c]
//
// i: compact rows, j: compact head rows, c: columns of X.  One tile of 64 (16, where that
// holds all rows) x 64 per CTA, 32 (64) deep, four (one) by four results per thread; operands
// pass through shared memory with the index that is contiguous in memory spread over a warp's
// lanes, the next ones waiting in registers while these are multiplied: a small head is bound
// by the trips to memory.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "launch.h"
#include "loss.h"

namespace dspark {

namespace {

constexpr int kTile = 64, kShare = 64;   // (a split of K is a multiple of kShare)

// base[at] where `ok`, else 0.  The load itself is unconditional (base[0] stands in), so that
// a thread's loads are issued together: behind branches they took turns, at a trip to memory
// each.
__device__ __forceinline__ float read_if(bool ok, const float* base, size_t at) {
  const float x = base[ok ? at : 0];
  return ok ? x : 0.f;
}

// acc[a][b] += sum_k a_at(R ty + a, k) b_at(4 tx + b, k) over `depth`, for a tile of 16 R
// rows.  a_along, b_along(k0): whether k is the index contiguous in memory (from depth k0 on;
// b_at gets the latter too).
template <int R, typename FA, typename FB, typename AB>
__device__ __forceinline__ void tile_product(float (&acc)[R][4], int depth, bool a_along,
                                             FA a_at, AB b_along, FB b_at) {
  constexpr int kDepth = R == 1 ? 64 : 32;
  constexpr int kRows = 16 * R, kLoadsA = kRows * kDepth / 256, kLoadsB = kTile * kDepth / 256;
  __shared__ __align__(16) float sa[kDepth][kRows + 4], sb[kDepth][kTile + 4];
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float ra[kLoadsA], rb[kLoadsB];
  auto place = [](bool along, int rows, int q, int& m, int& k) {
    const int e = threadIdx.x + 256 * q;
    k = along ? e % kDepth : e / rows;
    m = along ? e / kDepth : e % rows;
  };
  auto load = [&](int k0) {
    const bool bl = b_along(k0);
    int m, k;
#pragma unroll
    for (int q = 0; q < kLoadsA; ++q) {
      place(a_along, kRows, q, m, k);
      ra[q] = a_at(m, k0 + k);
    }
#pragma unroll
    for (int q = 0; q < kLoadsB; ++q) {
      place(bl, kTile, q, m, k);
      rb[q] = b_at(m, k0 + k, bl);
    }
  };
  load(0);
  for (int k0 = 0; k0 < depth; k0 += kDepth) {
    const bool bl = b_along(k0);
    int m, n;
#pragma unroll
    for (int q = 0; q < kLoadsA; ++q) {
      place(a_along, kRows, q, m, n);
      sa[n][m] = ra[q];
    }
#pragma unroll
    for (int q = 0; q < kLoadsB; ++q) {
      place(bl, kTile, q, m, n);
      sb[n][m] = rb[q];
    }
    __syncthreads();
    if (k0 + kDepth < depth) load(k0 + kDepth);
#pragma unroll 8
    for (int k = 0; k < kDepth; ++k) {
      const float4 b4 = *reinterpret_cast<const float4*>(&sb[k][4 * tx]);
      const float b[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float a = sa[k][R * ty + i];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a, b[j], acc[i][j]);
      }
    }
    __syncthreads();
  }
}

// Columns [v0, v1) of the logits: their statistics per 64-column tile and the labels'
// logits (`stats`), and the logits themselves (`store`).
template <int R>
__global__ void __launch_bounds__(256)
loss_logits(const LossPlan p, int v0, int v1, bool stats, bool store) {
  pdl_wait();
  pdl_signal();
  const int n_tok = (int)p.ctrl[kLossTok], n_voc = min(v1, (int)p.ctrl[kLossVoc]);
  const int m0 = blockIdx.y * 16 * R, j0 = v0 + blockIdx.x * kTile;
  if (m0 >= n_tok || j0 >= n_voc) return;
  const float* x = (const float*)p.x;
  const float* w = (const float*)p.lm_head;
  const float* w2 = (const float*)p.w2;
  __shared__ int s_row[kTile];
  if (threadIdx.x < kTile)
    s_row[threadIdx.x] = j0 + (int)threadIdx.x < n_voc ? loss_head_row(p, j0 + threadIdx.x) : -1;
  __syncthreads();
  float acc[R][4] = {};
  tile_product<R>(
      acc, p.Kx, true, [&](int m, int k) { return x[(size_t)(m0 + m) * p.Kx + k]; },
      [&](int k0) { return k0 < p.Hp; },
      [&](int n, int k, bool head) {
        const int row = s_row[n], c = k - p.Hp;
        return read_if(row >= 0 && (head ? k < p.H : c < p.r), head ? w : w2,
                       head ? (size_t)row * p.H + k : (size_t)c * p.Vh + row);
      });
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll
  for (int a = 0; a < R; ++a) {
    const int i = m0 + R * ty + a;
    float m = -INFINITY;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int j = j0 + 4 * tx + b;
      float z = acc[a][b];
      if (j < n_voc && p.vlist) z += p.biasc[j];
      acc[a][b] = z;
      if (j < n_voc) {
        // (a NaN logit stays NaN in the maximum)
        m = z != z || m != m ? m + z : fmaxf(m, z);
        if (store && i < n_tok) ((float*)p.q)[(size_t)i * p.ldq + (j - v0)] = z;
        if (stats && i < n_tok && j == p.lab[i]) p.zlab[i] = z;
      }
    }
    if (!stats) continue;
    // the row's 16 threads are 16 lanes of one warp
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      const float y = __shfl_xor_sync(0xFFFFFFFFu, m, o);
      m = y != y || m != m ? m + y : fmaxf(m, y);
    }
    float s = 0.f;
#pragma unroll
    for (int b = 0; b < 4; ++b)
      if (j0 + 4 * tx + b < n_voc && m > -INFINITY) s += expf(acc[a][b] - m);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (m != m) s = m;                        // (NaN for the whole row)
    if (tx == 0 && i < n_tok) p.stat[(size_t)i * p.n_stat + j0 / kTile] = make_float2(m, s);
  }
}

// dX of vocabulary columns [v0, v1): tile (bx, by), split bz of their range.
template <int R>
__device__ __forceinline__ void dx_tile(const LossPlan& p, int v0, int v1, bool first, int bx,
                                        int by, int bz) {
  const int n_tok = (int)p.ctrl[kLossTok], n_voc = min(v1, (int)p.ctrl[kLossVoc]);
  const int m0 = by * 16 * R, c0 = bx * kTile;
  if (m0 >= n_tok) return;
  const int share = ((v1 - v0 + p.splits - 1) / p.splits + kShare - 1) / kShare * kShare;
  const int ja = v0 + bz * share, jb = min(n_voc, ja + share);
  const float* q = (const float*)p.q;
  const float* w = (const float*)p.lm_head;
  const float* w2 = (const float*)p.w2;
  float acc[R][4] = {};
  const bool head = c0 < p.Hp;
  if (jb > ja)
    tile_product<R>(
        acc, jb - ja, true,
        [&](int m, int k) {
          const int j = ja + k;
          return read_if(m0 + m < n_tok && j < jb, q, (size_t)(m0 + m) * p.ldq + (j - v0));
        },
        [&](int) { return !head; },
        [&](int n, int k, bool) {
          const int j = min(ja + k, jb - 1), row = loss_head_row(p, j);
          const int c = c0 + n - (head ? 0 : p.Hp);
          return read_if(ja + k < jb && c < (head ? p.H : p.r), head ? w : w2,
                         head ? (size_t)row * p.H + c : (size_t)c * p.Vh + row);
        });
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float* dx = p.dxp + (size_t)bz * p.Tp * p.Kx;
#pragma unroll
  for (int a = 0; a < R; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int i = m0 + R * ty + a, c = c0 + 4 * tx + b;
      if (i >= n_tok) continue;
      float* d = dx + (size_t)i * p.Kx + c;
      *d = first ? acc[a][b] : *d + acc[a][b];
    }
}

// dW of vocabulary columns [v0, v1): tile (bx, by).
__device__ __forceinline__ void dw_tile(const LossPlan& p, int v0, int v1, int bx, int by) {
  const int n_tok = (int)p.ctrl[kLossTok], n_voc = min(v1, (int)p.ctrl[kLossVoc]);
  const int j0 = v0 + by * kTile, c0 = bx * kTile;
  const bool head = c0 < p.Hp;
  if (j0 >= n_voc || (head ? !p.d_lm_head : !p.d_w2)) return;
  const float* q = (const float*)p.q;
  const float* x = (const float*)p.x;
  float acc[4][4] = {};
  tile_product<4>(
      acc, n_tok, false,
      [&](int m, int k) {
        const int j = j0 + m;
        return read_if(j < n_voc && k < n_tok, q, (size_t)k * p.ldq + (j - v0));
      },
      [](int) { return false; },
      [&](int n, int k, bool) { return read_if(k < n_tok, x, (size_t)k * p.Kx + c0 + n); });
  const float scale = __uint_as_float(p.ctrl[kLossScale]);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int j = j0 + 4 * ty + a, c = c0 + 4 * tx + b;
      if (j >= n_voc) continue;
      const int row = loss_head_row(p, j);
      const float g = acc[a][b] * scale;
      if (head) {
        if (c < p.H) ((float*)p.d_lm_head)[(size_t)row * p.H + c] = g;
      } else if (c - p.Hp < p.r) {
        ((float*)p.d_w2)[(size_t)(c - p.Hp) * p.Vh + row] = g;
      }
    }
}

// Both: the first `n_dx` CTAs make dX, the others dW.
template <int R>
__global__ void __launch_bounds__(256)
loss_grads(const LossPlan p, int v0, int v1, bool first, int n_dx) {
  pdl_wait();
  pdl_signal();
  const int across = p.Kx / kTile;
  int b = blockIdx.x;
  if (b < n_dx) {
    const int rows = (p.T + 16 * R - 1) / (16 * R);
    dx_tile<R>(p, v0, v1, first, b % across, b / across % rows, b / across / rows);
  } else {
    b -= n_dx;
    dw_tile(p, v0, v1, b % across, b / across);
  }
}

}  // namespace

// Splits of the vocabulary for dX: enough CTAs to fill the GPU when rows are few.
int loss_simt_splits(int T, int Kx, int cols) {
  const int tiles = ((T + kTile - 1) / kTile) * (Kx / kTile);
  return std::max(1, std::min({(304 + tiles - 1) / tiles, (cols + 255) / 256, 64}));
}

// (rows of a tile: 16 where that holds them all, else 64)
cudaError_t launch_loss_logits_simt(const LossPlan& p, int v0, int v1, bool stats, bool store) {
  const bool few = p.T <= 16;
  const dim3 grid((v1 - v0 + kTile - 1) / kTile, few ? 1 : (p.T + kTile - 1) / kTile);
  return launch_after(few ? loss_logits<1> : loss_logits<4>, grid, 256, 0, p.stream, p, v0, v1,
                      stats, store);
}

cudaError_t launch_loss_grads_simt(const LossPlan& p, int v0, int v1, bool first) {
  const bool few = p.T <= 16;
  const int across = p.Kx / kTile, rows = few ? 1 : (p.T + kTile - 1) / kTile;
  const long long n_dx = p.dxp ? (long long)across * rows * p.splits : 0;
  const long long n_dw =
      p.d_lm_head || p.d_w2 ? (long long)across * ((v1 - v0 + kTile - 1) / kTile) : 0;
  if (n_dx + n_dw > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  return launch_after(few ? loss_grads<1> : loss_grads<4>, (unsigned)(n_dx + n_dw), 256, 0,
                      p.stream, p, v0, v1, first, (int)n_dx);
}

}  // namespace dspark
