// The training loss of the head: the call's plan (sizes, inputs, outputs, workspace
// regions) and the kernels' host launchers.
//
// A call first compacts its rows (those with a label the head can emit) and, for a head in
// the bias form, its vocabulary (the rows that are not masked).  Everything after works on
// the compact rows i < n_tok and compact head rows j < n_voc; both counts stay on the
// device.  The operand rows of the logits are X[i] = [hidden | markov_w1[prev]], each part
// padded with zeros to a multiple of 64, so that the Markov term is part of the one
// product z = X . [lm_head | markov_w2^T]^T and its gradients are columns of the others'.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dspark {

// Words of the control block at the head of the workspace (word 0: the error word).
enum : int {
  kLossTok = 1,      // compact rows
  kLossVoc = 2,      // compact head rows
  kLossScale = 3,    // float: loss_scale / D, the factor of every gradient
  kLossDone = 4,     // row CTAs whose loss is written
  kLossSplits = 5,   // splits of the vocabulary in dX's sum, at most LossPlan::splits
};

// Gradient memory that no product writes: `bytes` from `p` on, or, with `keep`, the rows of
// `row_bytes` whose keep entry is negative.  `early`: dW writes there too, so the zeros come
// before it.
struct LossZero {
  char* p;
  size_t bytes;
  const int32_t* keep;
  int row_bytes;
  bool early;
};

struct LossPlan {
  int T, H, V, Vh, r, dtype, reduction;
  float loss_scale;
  int Hp, rp, Kx, Tp;          // padded sizes: multiples of 64, Kx = Hp + rp, Tp of 256
  // inputs
  const void *hidden, *lm_head, *w1, *w2;
  const float *bias, *weights;
  const int32_t *d2t, *prev, *labels;
  // outputs (NULL where not asked for)
  float *loss, *total;
  int32_t* n_rows;
  void *d_hidden, *d_lm_head, *d_w1, *d_w2;
  // workspace
  uint32_t* ctrl;
  int32_t *tok, *lab, *prevc, *pos;   // [Tp] compact rows: row, label's compact head row,
                                      // prev; [T] row -> compact row or -1
  float* wrow;                        // [Tp] w_t of the compact rows
  int32_t *vlist, *vinv;              // bias form: compact head row -> head row [Vh], and
                                      // the inverse or -1
  int* vchunk;                        // counts per chunk of the bias
  float* biasc;                       // [Vh] bias of the compact head rows
  void *wc, *w2c;                     // bf16 bias form: the compact head [Vh][H], [r][Vh]
                                      // (zeros up to a multiple of 256 rows past n_voc)
  void* x;                            // [Tp][Kx]
  float2* stat;                       // [Tp][n_stat] per vocabulary tile, the label aside: the
                                      // maximum of z, and the sum of exp(z - maximum)
  int n_stat, stat_cols;
  float *zlab, *lse;                  // [Tp]
  void* q;                            // [Tp][ldq]; fp32: logits, then their gradient; bf16:
                                      // the logits' distances from their tile's maximum
                                      // (16 bits, loss_gap), then the gradient
  size_t ldq;
  int pieces, piece_cols;             // pieces of the vocabulary, columns of each
  float* qres;                        // [Tp] bf16: what rounding the label's entry of q lost
  float* dxp;                         // [splits][loss_split_rows][Kx] partial gradients of X
  int splits;                         // the most; fp32: what is used
  size_t dx_rows;                     // rows that dxp has room for, over all splits
  bool grads;                         // any gradient asked for
  LossZero zero[3];
  int n_zero;
  cudaStream_t stream;
};

constexpr int kLossLow = 64;        // see loss_low

// The label's entry of a row of q: w (p - 1) = w expm1(-loss), which loses no digits where p is
// nearly 1.
__device__ __forceinline__ float loss_label_entry(float w, float loss) {
  return w * expm1f(-loss);
}
// That of row i rounded to bf16 at q; what the rounding lost goes to the low row, or is kept for
// the gradient of X (this entry makes up most of it).
__device__ __forceinline__ void loss_put_label(const LossPlan& p, int i, bool low, __nv_bfloat16* q,
                                               float x) {
  const __nv_bfloat16 b = __float2bfloat16(x);
  const float lost = x - __bfloat162float(b);
  *q = b;
  if (low) q[kLossLow * p.ldq] = __float2bfloat16(lost);
  p.qres[i] = low ? 0.f : lost;
}

// bf16, up to kLossLow compact rows: row kLossLow + i of q holds what rounding row i of it lost
// (and row kLossLow + i of X is row i again), so that the gradient products see q with 16 bits:
// its label's entry and, with several pieces, all of it; with one piece the other entries come
// from the kept distances and are good to 11 bits.  Few rows do not average their roundings out,
// and within one 128-row tile this costs nothing.
__device__ __forceinline__ bool loss_low(const LossPlan& p, int n_tok) {
  return p.dtype == 1 && p.T <= 2 * kLossLow && n_tok <= kLossLow;
}

// Rows of one split's part of dxp.
__device__ __forceinline__ int loss_split_rows(int n_tok) { return max(256, (n_tok + 255) / 256 * 256); }

// compact -> head row, for kernels that read the head's own arrays
__device__ __forceinline__ int loss_head_row(const LossPlan& p, int j) {
  return p.vlist ? p.vlist[j] : j;
}

// A logit's distance d >= 0 below its tile's maximum in 16 bits: steps of 1 / 896, so that a
// probability is off by at most 0.06% (a bf16 rounding: 0.39%) down to e^-73 of the tile's
// largest, below every fp32 gradient that sums to anything; kLossFar from there on (and for
// anything that is not a number: the row's log-sum-exp is none either, and says so).
constexpr float kLossSteps = 896.f;
constexpr uint32_t kLossFar = 0xFFFFu;
__device__ __forceinline__ uint32_t loss_gap(float d) {
  // adding 2^23 rounds to an integer and leaves it in the low bits
  const float t = fminf(fmaf(d, kLossSteps, 8388608.f), 8388608.f + 65535.f);
  return __float_as_uint(t) & 0xFFFFu;
}
// 2^x and e^x of the hardware, results below 2^-126 taken as 0 (to keep those takes three more
// instructions, for probabilities that no bf16 gradient shows)
__device__ __forceinline__ float loss_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float loss_exp(float x) { return loss_exp2(x * 1.44269504f); }
// scale * exp(-distance), given log2(scale); `far` for kLossFar
__device__ __forceinline__ float loss_gap_exp(uint32_t gap, float log2_scale, float far) {
  const float d = __uint_as_float(0x4B000000u | gap) - 8388608.f;
  const float e = loss_exp2(fmaf(d, -1.44269504f / kLossSteps, log2_scale));
  return gap == kLossFar ? far : e;
}

// k_loss_rows.cu: everything but the products
cudaError_t launch_loss_plan(const LossPlan& p);         // compaction, X, zeroed outputs
cudaError_t launch_loss_rows(const LossPlan& p, bool dz);   // lse, losses, total, and with `dz`
                                                          // q of the one piece
cudaError_t launch_loss_dz_f32(const LossPlan& p, int v0, int v1);   // q from stored logits
cudaError_t launch_loss_dx(const LossPlan& p);           // d_hidden and d_w1 from dxp

// the products of columns [v0, v1) of the compact vocabulary.  Logits: with `stats` their
// statistics, and with `store` what q is made from; without `stats` q's input again
// (fp32) or q itself (bf16).  dX: `first` overwrites dxp, otherwise it is added to.
// k_loss_simt.cu (fp32, on the CUDA cores)
int loss_simt_splits(int T, int Kx, int cols);
cudaError_t launch_loss_logits_simt(const LossPlan& p, int v0, int v1, bool stats, bool store);
cudaError_t launch_loss_grads_simt(const LossPlan& p, int v0, int v1, bool first);   // dX, dW
// k_loss_tc.cu (bf16, on the tensor cores).  The logits with statistics and the first dX also
// write the plan's zeros, each a share (all in the logits when there is no dX, or early).
int loss_tc_splits(int T, int Hp, int rp);   // the most that may be chosen
cudaError_t launch_loss_logits_tc(const LossPlan& p, int v0, int v1, bool stats, bool store);
cudaError_t launch_loss_grads_tc(const LossPlan& p, int v0, int v1, bool first);   // dX, dW

}  // namespace dspark
