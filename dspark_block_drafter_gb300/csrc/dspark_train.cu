// The C ABI of the head's training operators: argument validation, workspace carve-up and
// kernel dispatch.
#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <string>

#include "../../include/dspark.h"
#include "common.cuh"
#include "kernels.h"
#include "loss.h"
#include "status.h"
#include "train.h"

namespace dspark {

static constexpr size_t kAlign = 256;
static constexpr int kMaxLossRows = 1 << 20;
// bf16: room for the partial gradients of X, where one for every row takes less.  With 4352 columns
// of X, up to 5120 rows with a loss choose among all splits; more rows fill the GPU with fewer (by
// the choice's own estimate at most 4% of dX is lost, and the room no longer grows sixfold with T).
static constexpr size_t kDxBytes = (size_t)1 << 29;

static bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Arrays of elements of `size` bytes, NULL where they are absent.
static dspark_status check_elements(std::initializer_list<const void*> arrays, size_t size) {
  for (const void* p : arrays)
    if (!aligned(p, size))
      return fail(DSPARK_ERR_INVALID_ARG, "an array of " + std::to_string(size) +
                                              "-byte elements is not aligned to them");
  return DSPARK_OK;
}

static dspark_status check_workspace(const void* ws, size_t have, size_t need) {
  if (!ws || !aligned(ws, kAlign))
    return fail(DSPARK_ERR_WORKSPACE, "workspace must be non-NULL and 256-byte aligned");
  if (have < need)
    return fail(DSPARK_ERR_WORKSPACE,
                "workspace too small: need " + std::to_string(need) + " bytes");
  return DSPARK_OK;
}

// ------------------------------------------------------------------ head loss
static dspark_status validate_loss(const dspark_loss_config* c, const dspark_head* h,
                                   const dspark_loss_outputs* o) {
  if (!c) return fail(DSPARK_ERR_INVALID_ARG, "config is NULL");
  if (!h) return fail(DSPARK_ERR_INVALID_ARG, "head is NULL");
  if (!o) return fail(DSPARK_ERR_INVALID_ARG, "outputs is NULL");
  if (c->T < 1 || c->H < 1 || c->V < 1 || c->r < 0)
    return fail(DSPARK_ERR_INVALID_ARG, "T, H and V must be >= 1, r >= 0");
  if (c->dtype != DSPARK_F32 && c->dtype != DSPARK_BF16)
    return fail(DSPARK_ERR_INVALID_ARG, "dtype must be DSPARK_F32 or DSPARK_BF16");
  if (c->reduction != DSPARK_LOSS_SUM && c->reduction != DSPARK_LOSS_MEAN)
    return fail(DSPARK_ERR_INVALID_ARG, "reduction must be DSPARK_LOSS_SUM or DSPARK_LOSS_MEAN");
  if (c->vocab_pieces < 0) return fail(DSPARK_ERR_INVALID_ARG, "vocab_pieces must be >= 0");
  if (!std::isfinite(c->loss_scale))
    return fail(DSPARK_ERR_INVALID_ARG, "loss_scale must be finite");
  if (!h->lm_head) return fail(DSPARK_ERR_INVALID_ARG, "lm_head is required");
  if (c->r > 0 && (!h->markov_w1 || !h->markov_w2))
    return fail(DSPARK_ERR_INVALID_ARG, "markov_w1 and markov_w2 are required when r > 0");
  if (c->r == 0 && (o->d_markov_w1 || o->d_markov_w2))
    return fail(DSPARK_ERR_INVALID_ARG, "r = 0: there are no Markov weights to differentiate");
  if (h->V_head < 1 || h->V_head > c->V)
    return fail(DSPARK_ERR_INVALID_ARG, "V_head must be in [1, V]");
  if (!h->d2t && h->V_head != c->V)
    return fail(DSPARK_ERR_INVALID_ARG, "without d2t, V_head must equal V");
  if (c->r > 512) return fail(DSPARK_ERR_UNSUPPORTED, "Markov rank above 512");
  if (c->T > kMaxLossRows) return fail(DSPARK_ERR_UNSUPPORTED, "more than 2^20 rows");
  if (c->H > (1 << 16) || c->V > (1 << 24))
    return fail(DSPARK_ERR_UNSUPPORTED, "H above 2^16 or V above 2^24");
  if (c->dtype == DSPARK_BF16) {
    if (c->H % 8 != 0)
      return fail(DSPARK_ERR_UNSUPPORTED, "bf16 path needs H % 8 == 0 (16-byte rows)");
    if (h->V_head % 8 != 0)
      return fail(DSPARK_ERR_UNSUPPORTED, "bf16 path needs V_head % 8 == 0 (16-byte rows)");
    if (!aligned(h->lm_head, 16) || (c->r > 0 && !aligned(h->markov_w2, 16)))
      return fail(DSPARK_ERR_INVALID_ARG, "bf16 weights must be 16-byte aligned");
    if (!aligned(o->d_lm_head, 16) || !aligned(o->d_markov_w1, 16) || !aligned(o->d_markov_w2, 16))
      return fail(DSPARK_ERR_INVALID_ARG, "bf16 weight gradients must be 16-byte aligned");
  }
  const dspark_status st =
      check_elements({h->lm_head, h->markov_w1, h->markov_w2, o->d_hidden, o->d_lm_head,
                      o->d_markov_w1, o->d_markov_w2}, c->dtype == DSPARK_F32 ? 4 : 2);
  if (st != DSPARK_OK) return st;
  return check_elements({h->lm_bias, h->d2t, o->loss, o->total, o->n_rows}, 4);
}

// Sizes and workspace regions (offsets from `ws`, which is NULL when only the size is
// wanted); returns the bytes used.
static size_t plan_loss(const dspark_loss_config* c, const dspark_head* h,
                        const dspark_loss_outputs* o, char* ws, LossPlan* p) {
  *p = LossPlan{};
  p->T = c->T; p->H = c->H; p->V = c->V; p->Vh = h->V_head; p->r = c->r;
  p->dtype = c->dtype; p->reduction = c->reduction; p->loss_scale = c->loss_scale;
  p->Hp = (int)align_up((size_t)c->H, 64);
  p->rp = (int)align_up((size_t)c->r, 64);
  p->Kx = p->Hp + p->rp;
  p->Tp = (int)align_up((size_t)c->T, 256);
  p->lm_head = h->lm_head; p->w1 = h->markov_w1; p->w2 = h->markov_w2;
  p->bias = h->lm_bias; p->d2t = h->d2t;
  p->loss = o->loss; p->total = o->total; p->n_rows = o->n_rows;
  p->d_hidden = o->d_hidden; p->d_lm_head = o->d_lm_head;
  p->d_w1 = o->d_markov_w1; p->d_w2 = o->d_markov_w2;
  p->grads = o->d_hidden || o->d_lm_head || o->d_markov_w1 || o->d_markov_w2;

  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* at = ws + off;
    off = align_up(off + bytes, kAlign);
    return (void*)at;
  };
  const size_t Tp = (size_t)p->Tp, Vh = (size_t)p->Vh, es = c->dtype == DSPARK_F32 ? 4 : 2;
  const bool tc = c->dtype == DSPARK_BF16;
  p->ctrl = (uint32_t*)take(256);
  p->tok = (int32_t*)take(4 * Tp);
  p->lab = (int32_t*)take(4 * Tp);
  p->prevc = (int32_t*)take(4 * Tp);
  p->pos = (int32_t*)take(4 * Tp);
  p->wrow = (float*)take(4 * Tp);
  p->zlab = (float*)take(4 * Tp);
  p->lse = (float*)take(4 * Tp);
  if (h->lm_bias) {
    p->vlist = (int32_t*)take(4 * Vh);
    p->vinv = (int32_t*)take(4 * Vh);
    p->biasc = (float*)take(4 * Vh);
    p->vchunk = (int*)take(4 * (size_t)emit_chunks(p->Vh));
    if (tc) {
      p->wc = take(es * Vh * p->H);
      p->w2c = take(es * Vh * p->r);
    }
  }
  p->x = take(es * Tp * p->Kx);
  p->stat_cols = tc ? 128 : 64;
  p->n_stat = (p->Vh + p->stat_cols - 1) / p->stat_cols;
  p->stat = (float2*)take(sizeof(float2) * Tp * p->n_stat);
  if (p->grads) {
    const int most = (p->Vh + 255) / 256;
    int pieces = c->vocab_pieces;
    if (pieces == 0) {
      // keep the whole vocabulary's numerators while they take no more than 8 GiB (a
      // second computation of the logits costs a third more products)
      const size_t all = Tp * align_up(Vh, 256) * es, limit = (size_t)8 << 30;
      pieces = (int)std::min<size_t>((all + limit - 1) / limit, (size_t)most);
    }
    pieces = std::min(pieces, most);
    p->piece_cols = (most + pieces - 1) / pieces * 256;
    p->pieces = (p->Vh + p->piece_cols - 1) / p->piece_cols;
    p->ldq = (size_t)p->piece_cols;
    p->q = take(es * Tp * p->ldq);
    if (tc) p->qres = (float*)take(4 * Tp);
    if (p->d_hidden || p->d_w1) {
      p->splits = tc ? loss_tc_splits(p->T, p->d_hidden ? p->Hp : 0, p->d_w1 ? p->rp : 0)
                     : loss_simt_splits(p->T, p->Kx, p->piece_cols);
      p->dx_rows = Tp * p->splits;
      if (tc) {
        const size_t room = kDxBytes / (sizeof(float) * p->Kx) / 256 * 256;
        p->dx_rows = std::min(p->dx_rows, std::max(Tp, room));
      }
      p->dxp = (float*)take(sizeof(float) * p->dx_rows * p->Kx);
    }
  }
  auto zero = [&](void* g, size_t bytes, const int32_t* keep, size_t row_bytes, bool early) {
    if (g) p->zero[p->n_zero++] = {(char*)g, bytes, keep, (int)row_bytes, early};
  };
  zero(p->d_w1, es * c->V * c->r, nullptr, 0, false);
  if (h->lm_bias) {
    // (fp32: all of it)
    zero(p->d_lm_head, es * Vh * c->H, tc ? p->vinv : nullptr, es * c->H, false);
    zero(p->d_w2, es * Vh * c->r, nullptr, 0, true);
  }
  return off;
}

static cudaError_t run_loss(const LossPlan& p) {
  const bool tc = p.dtype == DSPARK_BF16;
  const auto logits = tc ? launch_loss_logits_tc : launch_loss_logits_simt;
  const auto grads = tc ? launch_loss_grads_tc : launch_loss_grads_simt;
  cudaError_t e = launch_loss_plan(p);
  if (e != cudaSuccess) return e;
  const bool keep = p.grads && p.pieces == 1;
  e = logits(p, 0, p.Vh, true, keep);
  if (e == cudaSuccess) e = launch_loss_rows(p, keep);
  if (e != cudaSuccess || !p.grads) return e;
  for (int c = 0; c < p.pieces; ++c) {
    const int v0 = c * p.piece_cols, v1 = std::min(p.Vh, v0 + p.piece_cols);
    if (!keep) e = logits(p, v0, v1, false, true);
    if (e == cudaSuccess && !keep && !tc) e = launch_loss_dz_f32(p, v0, v1);
    if (e == cudaSuccess) e = grads(p, v0, v1, c == 0);
    if (e != cudaSuccess) return e;
  }
  return p.dxp ? launch_loss_dx(p) : cudaSuccess;
}

// ------------------------------------------------------------------ block norm
static dspark_status validate_norm(const dspark_norm_config* c) {
  if (!c) return fail(DSPARK_ERR_INVALID_ARG, "config is NULL");
  if (c->T < 1 || c->H < 1 || c->gate_span < 1)
    return fail(DSPARK_ERR_INVALID_ARG, "T, H and gate_span must be >= 1");
  if (c->dtype != DSPARK_F32 && c->dtype != DSPARK_BF16)
    return fail(DSPARK_ERR_INVALID_ARG, "dtype must be DSPARK_F32 or DSPARK_BF16");
  if (!(c->eps > 0.f) || !std::isfinite(c->eps) || !std::isfinite(c->residual_scale) ||
      !std::isfinite(c->weight_offset))
    return fail(DSPARK_ERR_INVALID_ARG,
                "eps must be positive, residual_scale and weight_offset finite");
  if (c->H > kNormMaxH) return fail(DSPARK_ERR_UNSUPPORTED, "H above 8192");
  if (c->T > (1 << 30)) return fail(DSPARK_ERR_UNSUPPORTED, "more than 2^30 rows");
  return DSPARK_OK;
}

static dspark_status check_norm_inputs(const void* x, const void* y, const void* gate,
                                       const void* w_post, const void* w_pre) {
  if (!x || !w_pre) return fail(DSPARK_ERR_INVALID_ARG, "x and w_pre are required");
  if (!y && (gate || w_post))
    return fail(DSPARK_ERR_INVALID_ARG, "gate and w_post act on y: they need it");
  return DSPARK_OK;
}

static size_t plan_norm(const dspark_norm_config* c, char* ws, NormArgs* a) {
  size_t off = 0;
  auto take = [&](size_t floats) {
    char* at = ws + off;
    off = align_up(off + 4 * floats, kAlign);
    return (float*)at;
  };
  // (as many CTAs as there are units: rows, or parts of the rows that share a gate row)
  const size_t parts = (size_t)norm_span_parts(c->T, c->gate_span);
  const size_t rows = ((size_t)c->T + c->gate_span - 1) / c->gate_span;
  const size_t units = std::max((size_t)c->T, rows * parts);
  a->w_part = take(2 * std::min(units, (size_t)norm_max_ctas(c->H)) * c->H);
  a->gate_part = parts > 1 ? take(rows * parts * c->H) : nullptr;
  return off;
}

static bool norm_f32(const dspark_norm_config* c) { return c->dtype == DSPARK_F32; }

static void fill_norm(const dspark_norm_config* c, NormArgs* a) {
  a->T = c->T; a->H = c->H; a->dtype = c->dtype;
  a->span = std::min(c->gate_span, c->T);     // (the same grouping; T + span stays an int)
  a->eps = c->eps; a->scale = c->residual_scale; a->offset = c->weight_offset;
}

// ------------------------------------------------------------------ clipping
static dspark_status validate_clip(int32_t count, const dspark_grad* g) {
  if (count < 1 || !g) return fail(DSPARK_ERR_INVALID_ARG, "at least one gradient is needed");
  if (count > (1 << 20)) return fail(DSPARK_ERR_UNSUPPORTED, "more than 2^20 gradients");
  for (int i = 0; i < count; ++i) {
    if (g[i].n < 0 || (g[i].n > 0 && (!g[i].in || !g[i].out)))
      return fail(DSPARK_ERR_INVALID_ARG,
                  "gradient " + std::to_string(i) + ": n must be >= 0, in and out non-NULL");
    if (g[i].dtype != DSPARK_F32 && g[i].dtype != DSPARK_BF16)
      return fail(DSPARK_ERR_INVALID_ARG, "gradient " + std::to_string(i) +
                                              ": dtype must be DSPARK_F32 or DSPARK_BF16");
    const size_t es = g[i].dtype == DSPARK_F32 ? 4 : 2;
    if (!aligned(g[i].in, es) || !aligned(g[i].out, es))
      return fail(DSPARK_ERR_INVALID_ARG,
                  "gradient " + std::to_string(i) + ": in and out must be element aligned");
    if (g[i].n > (1ll << 38)) return fail(DSPARK_ERR_UNSUPPORTED, "a gradient above 2^38 elements");
  }
  return DSPARK_OK;
}

}  // namespace dspark

using namespace dspark;

static_assert(sizeof(dspark_loss_config) == 32, "dspark_loss_config layout");
static_assert(sizeof(dspark_loss_outputs) == 56, "dspark_loss_outputs layout");
static_assert(sizeof(dspark_norm_config) == 28, "dspark_norm_config layout");
static_assert(sizeof(dspark_grad) == 32, "dspark_grad layout");

extern "C" {

size_t dspark_head_loss_workspace_size(const dspark_loss_config* cfg, const dspark_head* head,
                                       const dspark_loss_outputs* out) {
  if (validate_loss(cfg, head, out) != DSPARK_OK) return 0;
  LossPlan p;
  return plan_loss(cfg, head, out, nullptr, &p);
}

dspark_status dspark_head_loss(const dspark_loss_config* cfg, const dspark_head* head,
                               const void* hidden, const int32_t* prev, const int32_t* labels,
                               const float* weights, const dspark_loss_outputs* out,
                               void* workspace, size_t workspace_bytes, void* stream) {
  dspark_status st = validate_loss(cfg, head, out);
  if (st != DSPARK_OK) return st;
  if (!hidden || !labels || (cfg->r > 0 && !prev))
    return fail(DSPARK_ERR_INVALID_ARG, "hidden, labels and (for r > 0) prev are required");
  if (!out->loss || !out->total)
    return fail(DSPARK_ERR_INVALID_ARG, "outputs loss and total are required");
  st = check_elements({hidden}, cfg->dtype == DSPARK_F32 ? 4 : 2);
  if (st == DSPARK_OK) st = check_elements({cfg->r > 0 ? prev : nullptr, labels, weights}, 4);
  if (st != DSPARK_OK) return st;
  LossPlan p;
  const size_t need = plan_loss(cfg, head, out, (char*)workspace, &p);
  st = check_workspace(workspace, workspace_bytes, need);
  if (st != DSPARK_OK) return st;
  p.hidden = hidden;
  p.prev = prev;
  p.labels = labels;
  p.weights = weights;
  p.stream = (cudaStream_t)stream;
  const cudaError_t e = run_loss(p);
  if (e != cudaSuccess) return cuda_fail(e, "head loss");
  return DSPARK_OK;
}

dspark_status dspark_block_norm(const dspark_norm_config* cfg, const void* x, const void* y,
                                const void* gate, const void* w_post, const void* w_pre,
                                void* x_out, void* h, void* stream) {
  dspark_status st = validate_norm(cfg);
  if (st == DSPARK_OK) st = check_norm_inputs(x, y, gate, w_post, w_pre);
  if (st != DSPARK_OK) return st;
  if (!h) return fail(DSPARK_ERR_INVALID_ARG, "h is required");
  st = check_elements({x, y, gate, w_post, w_pre, x_out, h}, norm_f32(cfg) ? 4 : 2);
  if (st != DSPARK_OK) return st;
  NormArgs a{};
  fill_norm(cfg, &a);
  a.x = x; a.y = y; a.gate = gate; a.w_post = w_post; a.w_pre = w_pre;
  a.x_out = x_out;
  a.h = h;
  a.stream = (cudaStream_t)stream;
  const cudaError_t e = norm_f32(cfg) ? launch_norm_f32(a, false) : launch_norm_bf16(a, false);
  if (e != cudaSuccess) return cuda_fail(e, "block norm kernel");
  return DSPARK_OK;
}

size_t dspark_block_norm_workspace_size(const dspark_norm_config* cfg) {
  if (validate_norm(cfg) != DSPARK_OK) return 0;
  NormArgs a{};
  return plan_norm(cfg, nullptr, &a);
}

dspark_status dspark_block_norm_backward(const dspark_norm_config* cfg, const void* x,
                                         const void* y, const void* gate, const void* w_post,
                                         const void* w_pre, const void* d_h,
                                         const void* d_x_out, void* d_x, void* d_y,
                                         void* d_gate, void* d_w_post, void* d_w_pre,
                                         void* workspace, size_t workspace_bytes,
                                         void* stream) {
  dspark_status st = validate_norm(cfg);
  if (st == DSPARK_OK) st = check_norm_inputs(x, y, gate, w_post, w_pre);
  if (st != DSPARK_OK) return st;
  if (!d_h || !d_x || !d_w_pre)
    return fail(DSPARK_ERR_INVALID_ARG, "d_h, d_x and d_w_pre are required");
  if (!y != !d_y || !gate != !d_gate || !w_post != !d_w_post)
    return fail(DSPARK_ERR_INVALID_ARG,
                "d_y, d_gate and d_w_post go with y, gate and w_post: both or neither");
  st = check_elements({x, y, gate, w_post, w_pre, d_h, d_x_out, d_x, d_y, d_gate, d_w_post, d_w_pre},
                      norm_f32(cfg) ? 4 : 2);
  if (st != DSPARK_OK) return st;
  NormArgs a{};
  fill_norm(cfg, &a);
  const size_t need = plan_norm(cfg, (char*)workspace, &a);
  st = check_workspace(workspace, workspace_bytes, need);
  if (st != DSPARK_OK) return st;
  a.x = x; a.y = y; a.gate = gate; a.w_post = w_post; a.w_pre = w_pre;
  a.d_h = d_h; a.d_x_out = d_x_out; a.d_x = d_x; a.d_y = d_y; a.d_gate = d_gate;
  a.d_w_post = d_w_post; a.d_w_pre = d_w_pre;
  a.stream = (cudaStream_t)stream;
  const cudaError_t e = norm_f32(cfg) ? launch_norm_f32(a, true) : launch_norm_bf16(a, true);
  if (e != cudaSuccess) return cuda_fail(e, "block norm gradient kernels");
  return DSPARK_OK;
}

size_t dspark_clip_grads_workspace_size(int32_t count, const dspark_grad* grads) {
  if (validate_clip(count, grads) != DSPARK_OK) return 0;
  return align_up(sizeof(float) * clip_partials(count), kAlign);
}

dspark_status dspark_clip_grads(int32_t count, const dspark_grad* grads, float max_norm,
                                float* norm, void* workspace, size_t workspace_bytes,
                                void* stream) {
  dspark_status st = validate_clip(count, grads);
  if (st != DSPARK_OK) return st;
  if (!(max_norm >= 0.f)) return fail(DSPARK_ERR_INVALID_ARG, "max_norm must be >= 0");
  if (!norm) return fail(DSPARK_ERR_INVALID_ARG, "norm is required");
  st = check_elements({norm}, 4);
  if (st != DSPARK_OK) return st;
  st = check_workspace(workspace, workspace_bytes,
                       align_up(sizeof(float) * clip_partials(count), kAlign));
  if (st != DSPARK_OK) return st;
  const cudaError_t e = launch_clip_grads(count, grads, max_norm, norm, (float*)workspace,
                                          (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "gradient clipping kernels");
  return DSPARK_OK;
}

}  // extern "C"
