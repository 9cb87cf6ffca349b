// The training loss of the head: its three products on the CUDA cores, in fp32.
//
//   logits  z[i][j]  = X[i] . [lm_head[j] | markov_w2[:, j]] + bias[j]
//   dX      dx[i][c] = sum_j q[i][j] [lm_head | markov_w2^T][j][c]
//   dW      [d_lm_head | d_markov_w2^T][j][c] = scale * sum_i q[i][j] X[i][c]
//
// i: compact rows, j: compact head rows, c: columns of X.  One tile of 64 x 64 per CTA, 32
// deep, four by four results per thread; operands pass through shared memory with the index
// that is contiguous in memory spread over a warp's lanes, the next ones waiting in registers
// while these are multiplied.
//
// Up to 16 rows take other kernels.  There every product reads the head once and does little
// with it, and what bounds a small one are its trips to memory: a thread asks for many values
// of the head at once and meets them with all rows.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "launch.h"
#include "loss.h"

namespace dspark {

namespace {

constexpr int kTile = 64, kShare = 64;   // (a split of K is a multiple of kShare)
constexpr int R = 4;                     // a tile's results of a thread: R x 4
constexpr int kFewRows = 16;             // rows of the kernels for few
// Terms of one chain of additions in dX and dW; longer sums add such parts up in their output (one
// chain over 2^20 rows was off by 1.3e-4, over 70000 by 1.6e-5; in parts 1e-6).
constexpr int kChain = 4096;

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
template <typename FA, typename FB, typename AB>
__device__ __forceinline__ void tile_product(float (&acc)[R][4], int depth, bool a_along,
                                             FA a_at, AB b_along, FB b_at) {
  constexpr int kDepth = 32;
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

// Row i's logits of columns j0 + 4 tx + (0 .. 3), from their products `acc`: the statistics of
// the 64-column tile and the label's logit (`stats`), and the logits themselves (`store`).  A
// row's 16 threads are 16 lanes of one warp.
__device__ __forceinline__ void finish_logits(const LossPlan& p, int i, int n_tok, int v0, int j0,
                                              int n_voc, int tx, float (&acc)[4], bool stats,
                                              bool store) {
  float m = -INFINITY;
  const int lab = stats && i < n_tok ? p.lab[i] : -1;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int j = j0 + 4 * tx + b;
    float z = acc[b];
    if (j < n_voc && p.vlist) z += p.biasc[j];
    if (j < n_voc && store && i < n_tok) ((float*)p.q)[(size_t)i * p.ldq + (j - v0)] = z;
    if (j == lab) {                           // (kept out of the statistics)
      p.zlab[i] = z;
      z = -INFINITY;
    }
    if (j >= n_voc) z = -INFINITY;
    acc[b] = z;
    // (a NaN logit stays NaN in the maximum)
    m = z != z || m != m ? m + z : fmaxf(m, z);
  }
  if (!stats) return;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const float y = __shfl_xor_sync(0xFFFFFFFFu, m, o);
    m = y != y || m != m ? m + y : fmaxf(m, y);
  }
  float s = 0.f;
#pragma unroll
  for (int b = 0; b < 4; ++b)
    if (m > -INFINITY) s += expf(acc[b] - m);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if (m != m) s = m;                          // (NaN for the whole row)
  if (tx == 0 && i < n_tok) p.stat[(size_t)i * p.n_stat + j0 / kTile] = make_float2(m, s);
}

// Columns [v0, v1) of the logits.
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
  tile_product(
      acc, p.Kx, true, [&](int m, int k) { return x[(size_t)(m0 + m) * p.Kx + k]; },
      [&](int k0) { return k0 < p.Hp; },
      [&](int n, int k, bool head) {
        const int row = s_row[n], c = k - p.Hp;
        return read_if(row >= 0 && (head ? k < p.H : c < p.r), head ? w : w2,
                       head ? (size_t)row * p.H + k : (size_t)c * p.Vh + row);
      });
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll
  for (int a = 0; a < R; ++a)
    finish_logits(p, m0 + R * ty + a, n_tok, v0, j0, n_voc, tx, acc[a], stats, store);
}

// The same for up to NT rows: a warp takes 64 / NT head rows, its lanes the columns of X, and
// keeps the partial sums of all 64 logits; the lanes' sums are added at the end.  (8 rows,
// 256 x 4096 head: 10 us, 2048 x 32000 head: 78 us; through the tile's shared memory 17 and
// 241.  At 216 registers, the next values loaded ahead but one CTA on an SM: 14 and 193.)
template <int NT>
__global__ void __launch_bounds__(32 * NT, 16 / NT)
loss_logits_few(const LossPlan p, int v0, int v1, bool stats, bool store) {
  constexpr int kA = 64 / NT, kDeep = 32 / kA;   // 32 values of the head at once
  pdl_wait();
  pdl_signal();
  const int n_tok = (int)p.ctrl[kLossTok], n_voc = min(v1, (int)p.ctrl[kLossVoc]);
  const int j0 = v0 + blockIdx.x * kTile;
  if (n_tok == 0 || j0 >= n_voc) return;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  __shared__ float s_z[NT][kTile];
  size_t row[kA];
#pragma unroll
  for (int a = 0; a < kA; ++a)                // (past the last: logits that nobody reads)
    row[a] = (size_t)loss_head_row(p, min(j0 + kA * warp + a, n_voc - 1));
  float sum[NT * kA] = {};                    // [row of X][head row]
  // adds the products of columns [0, n) of x with at(row, column)
  auto add = [&](const float* x, int n, auto at) {
    for (int k0 = 0; k0 < n; k0 += 32 * kDeep) {
      float w[kDeep][kA];
#pragma unroll
      for (int q = 0; q < kDeep; ++q) {
        const int k = k0 + 32 * q + lane;
#pragma unroll
        for (int a = 0; a < kA; ++a) w[q][a] = *at(row[a], min(k, n - 1));
#pragma unroll
        for (int a = 0; a < kA; ++a) w[q][a] = k < n ? w[q][a] : 0.f;
      }
#pragma unroll
      for (int q = 0; q < kDeep; ++q) {
        const int k = min(k0 + 32 * q + lane, n - 1);
#pragma unroll
        for (int m = 0; m < NT; ++m) {
          const float xm = x[(size_t)m * p.Kx + k];
#pragma unroll
          for (int a = 0; a < kA; ++a) sum[m * kA + a] = fmaf(xm, w[q][a], sum[m * kA + a]);
        }
      }
    }
  };
  const float* x = (const float*)p.x;
  const float* w = (const float*)p.lm_head;
  const float* w2 = (const float*)p.w2;
  add(x, p.H, [&](size_t r, int k) { return w + r * p.H + k; });
  if (p.r > 0) add(x + p.Hp, p.r, [&](size_t r, int k) { return w2 + (size_t)k * p.Vh + r; });
  // each step halves the sums that a lane keeps
#pragma unroll
  for (int o = 16, n = 32; o > 0; o >>= 1, n >>= 1) {
    const bool upper = lane & o;
#pragma unroll
    for (int e = 0; e < n; ++e) {
      const float mine = upper ? sum[n + e] : sum[e], other = upper ? sum[e] : sum[n + e];
      sum[e] = mine + __shfl_xor_sync(0xFFFFFFFFu, other, o);
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int at = 2 * lane + e;
    s_z[at / kA][kA * warp + at % kA] = sum[e];
  }
  __syncthreads();
  const int tx = threadIdx.x % 16, i = threadIdx.x / 16;
  if (i >= NT) return;                        // (whole warps)
  float acc[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) acc[b] = s_z[i][4 * tx + b];
  finish_logits(p, i, n_tok, v0, j0, n_voc, tx, acc, stats, store);
}

// dX of vocabulary columns [v0, v1): tile (bx, by), split bz of their range.
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
  const bool head = c0 < p.Hp;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float* dx = p.dxp + (size_t)bz * loss_split_rows(n_tok) * p.Kx;
  int j0 = ja;
  do {                                        // (an empty range writes zeros)
    const int j1 = min(jb, j0 + kChain);
    float acc[R][4] = {};
    if (j1 > j0)
      tile_product(
          acc, j1 - j0, true,
          [&](int m, int k) {
            const int j = j0 + k;
            return read_if(m0 + m < n_tok && j < j1, q, (size_t)(m0 + m) * p.ldq + (j - v0));
          },
          [&](int) { return !head; },
          [&](int n, int k, bool) {
            const int j = min(j0 + k, j1 - 1), row = loss_head_row(p, j);
            const int c = c0 + n - (head ? 0 : p.Hp);
            return read_if(j0 + k < j1 && c < (head ? p.H : p.r), head ? w : w2,
                           head ? (size_t)row * p.H + c : (size_t)c * p.Vh + row);
          });
    const bool add = !first || j0 > ja;
#pragma unroll
    for (int a = 0; a < R; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int i = m0 + R * ty + a, c = c0 + 4 * tx + b;
        if (i >= n_tok) continue;
        float* d = dx + (size_t)i * p.Kx + c;
        *d = add ? *d + acc[a][b] : acc[a][b];
      }
    j0 += kChain;
  } while (j0 < jb);
}

// dW of vocabulary columns [v0, v1): tile (bx, by).
__device__ __forceinline__ void dw_tile(const LossPlan& p, int v0, int v1, int bx, int by) {
  const int n_tok = (int)p.ctrl[kLossTok], n_voc = min(v1, (int)p.ctrl[kLossVoc]);
  const int j0 = v0 + by * kTile, c0 = bx * kTile;
  const bool head = c0 < p.Hp;
  if (j0 >= n_voc || (head ? !p.d_lm_head : !p.d_w2)) return;
  const float* q = (const float*)p.q;
  const float* x = (const float*)p.x;
  const float scale = __uint_as_float(p.ctrl[kLossScale]);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  int i0 = 0;
  do {                                        // (no rows: zeros)
    const int i1 = min(n_tok, i0 + kChain);
    float acc[R][4] = {};
    tile_product(
        acc, i1 - i0, false,
        [&](int m, int k) {
          const int j = j0 + m;
          return read_if(j < n_voc && i0 + k < i1, q, (size_t)(i0 + k) * p.ldq + (j - v0));
        },
        [](int) { return false; },
        [&](int n, int k, bool) {
          return read_if(i0 + k < i1, x, (size_t)(i0 + k) * p.Kx + c0 + n);
        });
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int j = j0 + 4 * ty + a, c = c0 + 4 * tx + b;
        if (j >= n_voc || (head ? c >= p.H : c - p.Hp >= p.r)) continue;
        const int row = loss_head_row(p, j);
        float* d = head ? (float*)p.d_lm_head + (size_t)row * p.H + c
                        : (float*)p.d_w2 + (size_t)(c - p.Hp) * p.Vh + row;
        const float g = acc[a][b] * scale;
        *d = i0 > 0 ? *d + g : g;
      }
    i0 += kChain;
  } while (i0 < n_tok);
}

// Both: the first `n_dx` CTAs make dX, the others dW.
__global__ void __launch_bounds__(256)
loss_grads(const LossPlan p, int v0, int v1, bool first, int n_dx) {
  pdl_wait();
  pdl_signal();
  const int across = p.Kx / kTile;
  int b = blockIdx.x;
  if (b < n_dx) {
    const int rows = (p.T + 16 * R - 1) / (16 * R);
    dx_tile(p, v0, v1, first, b % across, b / across % rows, b / across / rows);
  } else {
    b -= n_dx;
    dw_tile(p, v0, v1, b % across, b / across);
  }
}

// The same for up to NT rows.  dX: a thread has two columns of X and all rows, and an eighth of
// the split's head rows; the eighths are added at the end.  dW: a thread has one column of X
// (of markov_w2: one head row), so that a warp's stores lie side by side, and 16 of the other.
// (The same heads: 10 and 138 us, as tiles 18 and 423; the second one writes 262 MB of dW.)
template <int NT>
__global__ void __launch_bounds__(256)
loss_grads_few(const LossPlan p, int v0, int v1, bool first, int n_dx) {
  constexpr int kChunk = 256;                 // head rows of dX at a time
  __shared__ __align__(16) float smem[8 * NT * kTile];
  __shared__ __align__(16) int s_row[kChunk];
  float(*s_q)[NT] = reinterpret_cast<float(*)[NT]>(smem);
  static_assert(kChunk * NT <= 8 * NT * kTile, "");
  pdl_wait();
  pdl_signal();
  const int n_tok = (int)p.ctrl[kLossTok], n_voc = min(v1, (int)p.ctrl[kLossVoc]);
  const int across = p.Kx / kTile, tid = threadIdx.x, lane = tid % kTile, group = tid / kTile;
  const float* q = (const float*)p.q;
  int b = blockIdx.x;
  const bool dx = b < n_dx;
  if (!dx) b -= n_dx;
  const int c0 = b % across * kTile, part = b / across;
  const bool head = c0 < p.Hp;
  if (dx) {
    if (n_tok == 0) return;                   // (no row of dX; dW is zero and is written)
    const float* w = (const float*)(head ? p.lm_head : p.w2);
    const int share = ((v1 - v0 + p.splits - 1) / p.splits + kShare - 1) / kShare * kShare;
    const int ja = v0 + part * share, jb = min(n_voc, ja + share);
    const int l = tid % 32, warp = tid / 32;
    bool in[2];
    size_t at[2], row_step = head ? p.H : 1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {             // (a column that does not exist reads the first)
      const int c = c0 + l + 32 * h - (head ? 0 : p.Hp);
      in[h] = c < (head ? p.H : p.r);
      at[h] = in[h] ? (head ? (size_t)c : (size_t)c * p.Vh) : 0;
    }
    float(*s_sum)[8][kTile] = reinterpret_cast<float(*)[8][kTile]>(smem);   // [NT]
    float* out = p.dxp + (size_t)part * loss_split_rows(n_tok) * p.Kx;
    int j0 = ja;
    do {                                      // (an empty range writes zeros)
      const int end = min(jb, j0 + 8 * kChain);
      float sum[2][NT] = {};
      for (int j1 = j0; j1 < end; j1 += kChunk) {
        const int n = min(kChunk, end - j1);
        __syncthreads();
        // (past the range: a row that exists, times zero)
        const int j = min(tid, n - 1);
        s_row[tid] = loss_head_row(p, j1 + j);
#pragma unroll
        for (int m = 0; m < NT; ++m)
          s_q[tid][m] = read_if(tid < n && m < n_tok, q, (size_t)m * p.ldq + (j1 - v0 + j));
        __syncthreads();
        for (int k0 = warp * 16; k0 < n; k0 += 8 * 16) {
          float y[2][16];
#pragma unroll
          for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) y[h][k] = w[at[h] + s_row[k0 + k] * row_step];
#pragma unroll
          for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int m = 0; m < NT; ++m) {
              const float g = s_q[k0 + k][m];
#pragma unroll
              for (int h = 0; h < 2; ++h) sum[h][m] = fmaf(g, y[h][k], sum[h][m]);
            }
        }
      }
      __syncthreads();
#pragma unroll
      for (int m = 0; m < NT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) s_sum[m][warp][l + 32 * h] = in[h] ? sum[h][m] : 0.f;
      __syncthreads();
      for (int m = group; m < n_tok; m += 4) {
        float g = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) g += s_sum[m][e][lane];
        float* d = out + (size_t)m * p.Kx + c0 + lane;
        *d = first && j0 == ja ? g : *d + g;
      }
      j0 += 8 * kChain;
    } while (j0 < jb);
    return;
  }
  const int j0 = v0 + part * kTile;
  if (j0 >= n_voc || (head ? !p.d_lm_head : !p.d_w2)) return;
  const float scale = __uint_as_float(p.ctrl[kLossScale]);
  const float* x = (const float*)p.x;
  float(*s_x)[kTile] = reinterpret_cast<float(*)[kTile]>(smem + kTile * NT);
  if (tid < kTile) s_row[tid] = j0 + tid < n_voc ? loss_head_row(p, j0 + tid) : -1;
#pragma unroll
  for (int m0 = 0; m0 < NT; m0 += 4) {
    const int m = m0 + group;
    s_x[m][lane] = read_if(m < n_tok, x, (size_t)m * p.Kx + c0 + lane);
    s_q[lane][m] = scale * read_if(m < n_tok && j0 + lane < n_voc, q,
                                   (size_t)m * p.ldq + (j0 - v0 + lane));
  }
  __syncthreads();
  float mine[NT];
  if (head) {
    if (c0 + lane >= p.H) return;
#pragma unroll
    for (int m = 0; m < NT; ++m) mine[m] = s_x[m][lane];
#pragma unroll 4
    for (int j = group; j < kTile; j += 4) {
      float g = 0.f;
#pragma unroll
      for (int m = 0; m < NT; ++m) g = fmaf(s_q[j][m], mine[m], g);
      if (s_row[j] >= 0) ((float*)p.d_lm_head)[(size_t)s_row[j] * p.H + c0 + lane] = g;
    }
  } else {
    const int row = s_row[lane], end = min(kTile, p.r - (c0 - p.Hp));
    if (row < 0) return;
#pragma unroll
    for (int m = 0; m < NT; ++m) mine[m] = s_q[lane][m];
#pragma unroll 4
    for (int c = group; c < end; c += 4) {
      float g = 0.f;
#pragma unroll
      for (int m = 0; m < NT; ++m) g = fmaf(mine[m], s_x[m][c], g);
      ((float*)p.d_w2)[(size_t)(c0 - p.Hp + c) * p.Vh + row] = g;
    }
  }
}

}  // namespace

// Splits of the vocabulary for dX: enough CTAs to fill the GPU when rows are few.
int loss_simt_splits(int T, int Kx, int cols) {
  const int tiles = ((T + kTile - 1) / kTile) * (Kx / kTile);
  return std::max(1, std::min({(304 + tiles - 1) / tiles, (cols + 255) / 256, 64}));
}

// The form that holds the rows with the fewest to spare.
using LogitsKernel = void (*)(const LossPlan, int, int, bool, bool);
using GradsKernel = void (*)(const LossPlan, int, int, bool, int);

cudaError_t launch_loss_logits_simt(const LossPlan& p, int v0, int v1, bool stats, bool store) {
  const bool few = p.T <= kFewRows;
  const LogitsKernel k = p.T <= 8 ? loss_logits_few<8> : few ? loss_logits_few<16> : loss_logits;
  const dim3 grid((v1 - v0 + kTile - 1) / kTile, few ? 1 : (p.T + kTile - 1) / kTile);
  return launch_after(k, grid, p.T > 8 && few ? 512 : 256, 0, p.stream, p, v0, v1, stats, store);
}

cudaError_t launch_loss_grads_simt(const LossPlan& p, int v0, int v1, bool first) {
  const bool few = p.T <= kFewRows;
  const GradsKernel k = p.T <= 8 ? loss_grads_few<8> : few ? loss_grads_few<16> : loss_grads;
  const int across = p.Kx / kTile, rows = few ? 1 : (p.T + kTile - 1) / kTile;
  const long long n_dx = p.dxp ? (long long)across * rows * p.splits : 0;
  const long long n_dw =
      p.d_lm_head || p.d_w2 ? (long long)across * ((v1 - v0 + kTile - 1) / kTile) : 0;
  if (n_dx + n_dw > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  return launch_after(k, (unsigned)(n_dx + n_dw), 256, 0, p.stream, p, v0, v1, first, (int)n_dx);
}

}  // namespace dspark
