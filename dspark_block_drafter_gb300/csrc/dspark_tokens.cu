// The C ABI of the operators on tokens and rows of logits: argument validation, workspace
// carve-up and kernel dispatch.
#include <cmath>
#include <initializer_list>
#include <string>

#include "../../include/dspark.h"
#include "common.cuh"
#include "status.h"
#include "tokens.h"

namespace dspark {

static constexpr size_t kAlign = 256;
static constexpr int kMaxRows = 1 << 20, kMaxVocab = 1 << 24, kMaxH = 1 << 16;

static bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

static dspark_status check_elements(std::initializer_list<const void*> arrays, size_t size) {
  for (const void* p : arrays)
    if (!aligned(p, size))
      return fail(DSPARK_ERR_INVALID_ARG, "an array of " + std::to_string(size) +
                                              "-byte elements is not aligned to them");
  return DSPARK_OK;
}

static size_t element(int32_t dtype) { return dtype == DSPARK_F32 ? 4 : 2; }

static dspark_status validate_rows(int32_t T, int32_t V, int64_t ld, int32_t dtype) {
  if (T < 1 || V < 1) return fail(DSPARK_ERR_INVALID_ARG, "T and V must be >= 1");
  if (dtype != DSPARK_F32 && dtype != DSPARK_BF16)
    return fail(DSPARK_ERR_INVALID_ARG, "dtype must be DSPARK_F32 or DSPARK_BF16");
  if (ld < V) return fail(DSPARK_ERR_INVALID_ARG, "ld must be at least V");
  if (T > kMaxRows || V > kMaxVocab)
    return fail(DSPARK_ERR_UNSUPPORTED, "more than 2^20 rows or V above 2^24");
  if (ld > (1ll << 32)) return fail(DSPARK_ERR_UNSUPPORTED, "ld above 2^32");
  return DSPARK_OK;
}

static dspark_status validate_embed(const dspark_embed_config* c) {
  if (!c) return fail(DSPARK_ERR_INVALID_ARG, "config is NULL");
  if (c->T < 1 || c->V < 1 || c->H < 1)
    return fail(DSPARK_ERR_INVALID_ARG, "T, V and H must be >= 1");
  if (c->dtype != DSPARK_F32 && c->dtype != DSPARK_BF16)
    return fail(DSPARK_ERR_INVALID_ARG, "dtype must be DSPARK_F32 or DSPARK_BF16");
  if (!std::isfinite(c->scale)) return fail(DSPARK_ERR_INVALID_ARG, "scale must be finite");
  if (c->T > kMaxRows || c->V > kMaxVocab || c->H > kMaxH)
    return fail(DSPARK_ERR_UNSUPPORTED, "more than 2^20 rows, V above 2^24 or H above 2^16");
  return DSPARK_OK;
}

// Whether two arrays share memory.
static bool overlap(const void* p, size_t n, const void* q, size_t m) {
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  return p && q && a < b + m && b < a + n;
}

struct Span {
  const void* p;
  size_t n;
};

// Refuses outputs that share memory with an input or with one another: rows of one launch are read
// and written in no order.
static dspark_status check_apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span& o : outs) {
    for (const Span& i : ins)
      if (overlap(o.p, o.n, i.p, i.n)) return fail(DSPARK_ERR_INVALID_ARG, "an output overlaps an input");
    for (const Span& i : outs)
      if (&i != &o && overlap(o.p, o.n, i.p, i.n))
        return fail(DSPARK_ERR_INVALID_ARG, "two outputs overlap");
  }
  return DSPARK_OK;
}
static size_t rows_bytes(int32_t T, int32_t V, int64_t ld, int32_t dtype) {
  return ((size_t)(T - 1) * (size_t)ld + (size_t)V) * element(dtype);
}

static EmbedArgs embed_args(const dspark_embed_config* c) {
  EmbedArgs a{};
  a.T = c->T; a.V = c->V; a.H = c->H; a.dtype = c->dtype;
  a.scale = c->scale;
  return a;
}

static size_t plan_embed_workspace(char* ws, EmbedArgs* a) {
  plan_embed(a);
  size_t off = 0;
  auto take = [&](size_t words) {
    char* at = ws + off;
    off = align_up(off + 4 * words, kAlign);
    return (uint32_t*)at;
  };
  const size_t T = (size_t)a->T, parts = (size_t)a->chunks * 2;
  a->ctrl = take(64);
  a->there = (uint8_t*)take(((size_t)a->V + 3) / 4);
  for (int i = 0; i < 2; ++i) {
    a->key[i] = take(T);
    a->pos[i] = take(T);
  }
  a->hist = take(embed_hist_words(*a));
  a->part_tok = (int32_t*)take(parts);
  a->part = (float*)take(parts * a->H);
  return off;
}

}  // namespace dspark

using namespace dspark;

static_assert(sizeof(dspark_sample_config) == 40, "dspark_sample_config layout");
static_assert(sizeof(dspark_sample_rows) == 32, "dspark_sample_rows layout");
static_assert(sizeof(dspark_embed_config) == 20, "dspark_embed_config layout");

extern "C" {

dspark_status dspark_sample(const dspark_sample_config* cfg, const dspark_sample_rows* rows,
                            const void* logits, const float* uniform, int32_t* tokens,
                            float* logp, void* stream) {
  if (!cfg) return fail(DSPARK_ERR_INVALID_ARG, "config is NULL");
  dspark_status st = validate_rows(cfg->T, cfg->V, cfg->ld, cfg->dtype);
  if (st != DSPARK_OK) return st;
  if (std::isnan(cfg->temperature) || std::isnan(cfg->top_p) || std::isnan(cfg->min_p))
    return fail(DSPARK_ERR_INVALID_ARG, "temperature, top_p and min_p must be numbers");
  if (!logits || !uniform || !tokens)
    return fail(DSPARK_ERR_INVALID_ARG, "logits, uniform and tokens are required");
  st = check_elements({logits}, element(cfg->dtype));
  if (st == DSPARK_OK) st = check_elements({uniform, tokens, logp}, 4);
  if (st == DSPARK_OK && rows)
    st = check_elements({rows->top_k, rows->temperature, rows->top_p, rows->min_p}, 4);
  if (st != DSPARK_OK) return st;
  const size_t each = 4 * (size_t)cfg->T;
  const dspark_sample_rows own = rows ? *rows : dspark_sample_rows{};
  st = check_apart({{tokens, each}, {logp, each}},
                   {{logits, rows_bytes(cfg->T, cfg->V, cfg->ld, cfg->dtype)}, {uniform, each},
                    {own.top_k, each}, {own.temperature, each}, {own.top_p, each}, {own.min_p, each}});
  if (st != DSPARK_OK) return st;
  RowArgs a{};
  a.T = cfg->T; a.V = cfg->V; a.ld = cfg->ld; a.dtype = cfg->dtype;
  a.logits = logits;
  a.temperature = cfg->temperature; a.top_p = cfg->top_p; a.min_p = cfg->min_p;
  a.top_k = cfg->top_k;
  if (rows) {
    a.row_temperature = rows->temperature; a.row_top_p = rows->top_p;
    a.row_min_p = rows->min_p; a.row_top_k = rows->top_k;
  }
  a.uniform = uniform; a.tokens = tokens; a.logp = logp;
  a.stream = (cudaStream_t)stream;
  const cudaError_t e = launch_rows(a);
  if (e != cudaSuccess) return cuda_fail(e, "sampling kernel");
  return DSPARK_OK;
}

dspark_status dspark_top_logits(int32_t T, int32_t V, int64_t ld, int32_t dtype, int32_t k,
                                const void* logits, int32_t* ids, float* values, float* lse,
                                void* stream) {
  dspark_status st = validate_rows(T, V, ld, dtype);
  if (st != DSPARK_OK) return st;
  if (k < 1 || k > V) return fail(DSPARK_ERR_INVALID_ARG, "k must be in [1, V]");
  if (k > kMaxTop)
    return fail(DSPARK_ERR_UNSUPPORTED, "k above " + std::to_string(kMaxTop));
  if (!logits || !ids || !values)
    return fail(DSPARK_ERR_INVALID_ARG, "logits, ids and values are required");
  st = check_elements({logits}, element(dtype));
  if (st == DSPARK_OK) st = check_elements({ids, values, lse}, 4);
  if (st != DSPARK_OK) return st;
  const size_t each = 4 * (size_t)T;
  st = check_apart({{ids, each * k}, {values, each * k}, {lse, each}},
                   {{logits, rows_bytes(T, V, ld, dtype)}});
  if (st != DSPARK_OK) return st;
  RowArgs a{};
  a.T = T; a.V = V; a.ld = ld; a.dtype = dtype;
  a.logits = logits;
  a.k = k; a.ids = ids; a.values = values; a.lse = lse;
  a.stream = (cudaStream_t)stream;
  const cudaError_t e = launch_rows(a);
  if (e != cudaSuccess) return cuda_fail(e, "top logits kernel");
  return DSPARK_OK;
}

dspark_status dspark_embed(const dspark_embed_config* cfg, const void* table,
                           const int32_t* ids, void* out, void* stream) {
  dspark_status st = validate_embed(cfg);
  if (st != DSPARK_OK) return st;
  if (!table || !ids || !out)
    return fail(DSPARK_ERR_INVALID_ARG, "table, ids and out are required");
  st = check_elements({table, out}, element(cfg->dtype));
  if (st == DSPARK_OK) st = check_elements({ids}, 4);
  if (st != DSPARK_OK) return st;
  const size_t row = (size_t)cfg->H * element(cfg->dtype);
  st = check_apart({{out, cfg->T * row}}, {{table, cfg->V * row}, {ids, 4 * (size_t)cfg->T}});
  if (st != DSPARK_OK) return st;
  EmbedArgs a = embed_args(cfg);
  a.table = table; a.ids = ids; a.out = out;
  a.stream = (cudaStream_t)stream;
  const cudaError_t e = launch_embed(a);
  if (e != cudaSuccess) return cuda_fail(e, "embedding kernel");
  return DSPARK_OK;
}

size_t dspark_embed_workspace_size(const dspark_embed_config* cfg) {
  if (validate_embed(cfg) != DSPARK_OK) return 0;
  EmbedArgs a = embed_args(cfg);
  return plan_embed_workspace(nullptr, &a);
}

dspark_status dspark_embed_backward(const dspark_embed_config* cfg, const int32_t* ids,
                                    const void* d_out, const void* add, void* d_table,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  dspark_status st = validate_embed(cfg);
  if (st != DSPARK_OK) return st;
  if (!ids || !d_out || !d_table)
    return fail(DSPARK_ERR_INVALID_ARG, "ids, d_out and d_table are required");
  st = check_elements({d_out, add, d_table}, element(cfg->dtype));
  if (st == DSPARK_OK) st = check_elements({ids}, 4);
  if (st != DSPARK_OK) return st;
  const size_t row = (size_t)cfg->H * element(cfg->dtype);
  st = check_apart({{d_table, cfg->V * row}},
                   {{d_out, cfg->T * row}, {ids, 4 * (size_t)cfg->T},
                    {add == d_table ? nullptr : add, cfg->V * row}});
  if (st != DSPARK_OK) return st;
  EmbedArgs a = embed_args(cfg);
  const size_t need = plan_embed_workspace((char*)workspace, &a);
  if (!workspace || !aligned(workspace, kAlign))
    return fail(DSPARK_ERR_WORKSPACE, "workspace must be non-NULL and 256-byte aligned");
  if (workspace_bytes < need)
    return fail(DSPARK_ERR_WORKSPACE, "workspace too small: need " + std::to_string(need) + " bytes");
  a.ids = ids; a.d_out = d_out; a.add = add; a.d_table = d_table;
  a.stream = (cudaStream_t)stream;
  const cudaError_t e = launch_embed_backward(a);
  if (e != cudaSuccess) return cuda_fail(e, "embedding gradient kernels");
  return DSPARK_OK;
}

}  // extern "C"
