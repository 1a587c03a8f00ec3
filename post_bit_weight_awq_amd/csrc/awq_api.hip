// C ABI of the AWQ search library: argument validation, workspace planning and
// kernel launches.  All checks run on the host before anything is enqueued.
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include "../../include/awq_mi355x.h"
#include "awq_internal.h"
#include "kv4_internal.h"

namespace {

thread_local char g_err[512] = "";

int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof g_err, fmt, ap);
  va_end(ap);
  return code;
}

int ok() {
  g_err[0] = '\0';
  return AWQ_OK;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// Largest dimensions accepted: they keep every index inside int64 and the
// launch grids inside their limits.
constexpr int64_t kMaxTokens = (int64_t)1 << 24;  // exact 64-bit saliency sums
constexpr int64_t kMaxFeatures = (int64_t)1 << 20;
constexpr int64_t kMaxWeights = (int64_t)1 << 34;  // one work-item per 8 weights < 2^32

int check_config(const awq_config* cfg) {
  if (!cfg) return fail(AWQ_ERR_INVALID_ARG, "cfg is NULL");
  if (cfg->w_bit != 4 && cfg->w_bit != 3)
    return fail(AWQ_ERR_UNSUPPORTED, "w_bit=%d: 3 and 4 are implemented", cfg->w_bit);
  if (cfg->group_size != 128 && cfg->group_size != 64 && cfg->group_size != 32)
    return fail(AWQ_ERR_UNSUPPORTED, "group_size=%d: 32, 64 and 128 are implemented",
                cfg->group_size);
  if (cfg->zero_point != 1 && cfg->zero_point != 0)
    return fail(AWQ_ERR_UNSUPPORTED, "zero_point=%d: 1 (asymmetric) or 0 (symmetric)",
                cfg->zero_point);
  if (cfg->n_grid < 1 || cfg->n_grid > 64)
    return fail(AWQ_ERR_INVALID_ARG, "n_grid=%d outside 1..64", cfg->n_grid);
  if (!(cfg->sal_floor > 0.0f) || !(cfg->sal_floor < 3.4e38f))
    return fail(AWQ_ERR_INVALID_ARG, "sal_floor must be finite and > 0");
  return AWQ_OK;
}

int check_dims(int64_t n_tokens, int64_t in_features, int64_t out_features, bool need_tokens,
               bool need_out, int64_t in_multiple) {
  if (need_tokens && (n_tokens < 1 || n_tokens > kMaxTokens))
    return fail(AWQ_ERR_INVALID_ARG, "n_tokens=%lld outside 1..%lld", (long long)n_tokens,
                (long long)kMaxTokens);
  if (in_features < in_multiple || in_features > kMaxFeatures || in_features % in_multiple)
    return fail(AWQ_ERR_INVALID_ARG, "in_features=%lld must be a positive multiple of %lld (max %lld)",
                (long long)in_features, (long long)in_multiple, (long long)kMaxFeatures);
  if (need_out && (out_features < 1 || out_features > kMaxFeatures))
    return fail(AWQ_ERR_INVALID_ARG, "out_features=%lld outside 1..%lld", (long long)out_features,
                (long long)kMaxFeatures);
  if (need_out && out_features * in_features > kMaxWeights)
    return fail(AWQ_ERR_INVALID_ARG, "out_features*in_features=%lld above %lld",
                (long long)(out_features * in_features), (long long)kMaxWeights);
  return AWQ_OK;
}

int check_ptr(const void* p, const char* name) {
  if (!p) return fail(AWQ_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned16(p)) return fail(AWQ_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  return AWQ_OK;
}

awq::QuantSpec quant_spec(const awq_config* cfg) {
  awq::QuantSpec q;
  q.group = cfg->group_size;
  q.w_bit = cfg->w_bit;
  q.zero_point = cfg->zero_point != 0;
  return q;
}

int hip_result(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(AWQ_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

// Sizes and types of a packed-weight operator; `rows` counts the packed
// matrix's rows.
int check_w4(int64_t n_tokens, int64_t in_features, int64_t rows, int group_size, int dtype) {
  int rc;
  if ((rc = check_dims(1, in_features, rows, false, true, 128))) return rc;
  if (n_tokens < 1 || n_tokens > awq::kMaxW4OpTokens)
    return fail(AWQ_ERR_INVALID_ARG, "n_tokens=%lld outside 1..%lld", (long long)n_tokens,
                (long long)awq::kMaxW4OpTokens);
  if (group_size != 128 && group_size != 64 && group_size != 32)
    return fail(AWQ_ERR_UNSUPPORTED, "group_size=%d: 32, 64 and 128 are implemented", group_size);
  if (dtype != AWQ_F16 && dtype != AWQ_BF16)
    return fail(AWQ_ERR_UNSUPPORTED, "dtype=%d: AWQ_F16 and AWQ_BF16 are implemented", dtype);
  return AWQ_OK;
}

// The gated forms take half the packed matrix's rows.
int check_w4_gated(int64_t n_tokens, int64_t in_features, int64_t half, int group_size, int dtype,
                   int act) {
  if (half < 1 || half > kMaxFeatures / 2)
    return fail(AWQ_ERR_INVALID_ARG, "half_features=%lld outside 1..%lld", (long long)half,
                (long long)(kMaxFeatures / 2));
  if (act != AWQ_ACT_SILU && act != AWQ_ACT_GELU_TANH)
    return fail(AWQ_ERR_UNSUPPORTED, "act=%d: AWQ_ACT_SILU and AWQ_ACT_GELU_TANH are implemented",
                act);
  return check_w4(n_tokens, in_features, 2 * half, group_size, dtype);
}

awq::W4Args w4_args(int64_t n_tokens, int64_t in_features, int64_t rows, int group_size, int dtype,
                    int act, const int32_t* qweight, const void* step16, const void* zero16) {
  awq::W4Args a{};
  a.N = n_tokens;
  a.K = in_features;
  a.O = rows;
  a.group = group_size;
  a.type = a.y_type = dtype;
  a.act = act;
  a.qweight = qweight;
  a.step16 = step16;
  a.zero16 = zero16;
  return a;
}

int check_layer(const int32_t* qweight, const void* step16, const void* zero16) {
  int rc;
  if ((rc = check_ptr(qweight, "qweight")) || (rc = check_ptr(step16, "step16"))) return rc;
  return check_ptr(zero16, "zero16");
}

// Bytes of the activation arguments, in the order of W4Args.
struct W4Bytes {
  int64_t in0, in1, out0, out1;
};

// A stretch of memory of an argument; NULL ones have none.
struct Span {
  const void* p;
  int64_t n;
};
// What a call writes (the first `written`) shares no byte with anything else.
int check_spans(const Span* r, int written, int count) {
  for (int i = 0; i < written; ++i)
    for (int j = i + 1; j < count; ++j) {
      const uintptr_t x = (uintptr_t)r[i].p, y = (uintptr_t)r[j].p;
      if (x && y && r[i].n && r[j].n && x < y + r[j].n && y < x + r[i].n)
        return fail(AWQ_ERR_INVALID_ARG, "an output or the workspace overlaps another argument");
    }
  return AWQ_OK;
}

int run_w4(awq::W4Op op, awq::W4Args& a, const W4Bytes& b, void* workspace, size_t workspace_bytes,
           void* stream, const char* what) {
  const size_t need = awq::w4_workspace(op, a);
  if (need) {
    int rc;
    if ((rc = check_ptr(workspace, "workspace"))) return rc;
    if (workspace_bytes < need)
      return fail(AWQ_ERR_WORKSPACE, "workspace %zu bytes < %zu required", workspace_bytes, need);
  }
  a.ws = workspace;
  // what is written (the first three) shares no byte with anything else
  const int64_t groups = 2 * a.O * (a.K / a.group);
  const Span r[8] = {{a.out0, b.out0},   {a.out1, b.out1},       {a.ws, (int64_t)need},
                     {a.in0, b.in0},     {a.in1, b.in1},         {a.qweight, a.O * a.K / 2},
                     {a.step16, groups}, {a.zero16, groups}};
  int rc;
  if ((rc = check_spans(r, 3, 8))) return rc;
  return hip_result(awq::launch_w4(op, a, (hipStream_t)stream), what);
}

int check_16bit(int dtype) {
  if (dtype != AWQ_F16 && dtype != AWQ_BF16)
    return fail(AWQ_ERR_UNSUPPORTED, "dtype=%d: AWQ_F16 and AWQ_BF16 are implemented", dtype);
  return AWQ_OK;
}

int check_count(int64_t n, int64_t most, const char* name) {
  if (n < 1 || n > most)
    return fail(AWQ_ERR_INVALID_ARG, "%s=%lld outside 1..%lld", name, (long long)n, (long long)most);
  return AWQ_OK;
}

// Sizes of a 4-bit cache, without its pointers.
int check_kv4(const awq_kv4_cache* c, awq::Kv4* out) {
  int rc;
  if (!c) return fail(AWQ_ERR_INVALID_ARG, "cache is NULL");
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return fail(AWQ_ERR_UNSUPPORTED, "page_size=%d: 16, 32, 64 and 128 are implemented", c->page_size);
  if (c->head_dim != 64 && c->head_dim != 128)
    return fail(AWQ_ERR_UNSUPPORTED, "head_dim=%d: 64 and 128 are implemented", c->head_dim);
  if ((c->group_size != 32 && c->group_size != 64 && c->group_size != 128) ||
      c->group_size > c->head_dim)
    return fail(AWQ_ERR_UNSUPPORTED, "group_size=%d: 32, 64 and 128, at most head_dim=%d",
                c->group_size, c->head_dim);
  if ((rc = check_count(c->n_heads, 1024, "cache n_heads")) ||
      (rc = check_count(c->n_pages, 0x7fffffff / c->page_size, "n_pages")))
    return rc;
  out->k_codes = (uint32_t*)c->k_codes;
  out->v_codes = (uint32_t*)c->v_codes;
  out->k_params = (uint32_t*)c->k_params;
  out->v_params = (uint32_t*)c->v_params;
  out->pages = c->n_pages;
  out->heads = c->n_heads;
  out->shift = __builtin_ctz((unsigned)c->page_size);
  out->dim = c->head_dim;
  out->group = c->group_size;
  return AWQ_OK;
}
int check_kv4_arrays(const awq::Kv4& c) {
  int rc;
  if ((rc = check_ptr(c.k_codes, "k_codes")) || (rc = check_ptr(c.v_codes, "v_codes")) ||
      (rc = check_ptr(c.k_params, "k_params")) || (rc = check_ptr(c.v_params, "v_params")))
    return rc;
  return AWQ_OK;
}
int64_t kv4_code_bytes(const awq::Kv4& c) { return (c.pages << c.shift) * c.heads * (c.dim / 2); }
int64_t kv4_param_bytes(const awq::Kv4& c) {
  return (c.pages << c.shift) * c.heads * (c.dim / c.group) * 4;
}

int check_stride(int64_t s, const char* name) {
  if (s < 0 || s % 8 || s > ((int64_t)1 << 40))
    return fail(AWQ_ERR_INVALID_ARG, "%s=%lld: a multiple of 8 from 0 to 2^40", name, (long long)s);
  return AWQ_OK;
}
int64_t rows_bytes(int64_t tokens, int64_t heads, int64_t dim, int64_t ts, int64_t hs) {
  return 2 * ((tokens - 1) * ts + (heads - 1) * hs + dim);
}
int check_index(const void* p, const char* name) {
  if (!p) return fail(AWQ_ERR_INVALID_ARG, "%s is NULL", name);
  if ((uintptr_t)p & 3u) return fail(AWQ_ERR_INVALID_ARG, "%s is not 4-byte aligned", name);
  return AWQ_OK;
}

int kv4_attention_args(const awq_kv4_cache* cache, int64_t n_tokens, int64_t n_heads, int64_t n_seqs,
                       int64_t max_pages, bool ragged, awq::Kv4Attention* a) {
  int rc;
  if ((rc = check_kv4(cache, &a->cache)) ||
      (rc = check_count(n_tokens, awq::kMaxW4OpTokens, "n_tokens")) ||
      (rc = check_count(n_seqs, awq::kMaxW4OpTokens, "n_seqs")) ||
      (rc = check_count(max_pages, ((int64_t)1 << 30) >> a->cache.shift, "max_pages")))
    return rc;
  if (n_heads < 1 || n_heads % a->cache.heads || n_heads / a->cache.heads > 1024 ||
      n_tokens * n_heads > 0x7fffffff)
    return fail(AWQ_ERR_INVALID_ARG,
                "n_heads=%lld must be a multiple of the cache's %d, up to 1024 times, and n_tokens * "
                "n_heads below 2^31",
                (long long)n_heads, a->cache.heads);
  if (!ragged && n_tokens != n_seqs)
    return fail(AWQ_ERR_INVALID_ARG, "n_tokens=%lld and n_seqs=%lld differ and starts is NULL",
                (long long)n_tokens, (long long)n_seqs);
  a->heads = (int)n_heads;
  a->tokens = n_tokens;
  a->seqs = n_seqs;
  a->per_seq = max_pages;
  static const int32_t here = 0;
  a->starts = ragged ? &here : nullptr;
  return AWQ_OK;
}

int check_adapters(int64_t n_adapters, int rank, int64_t in_features, int64_t out_features) {
  int rc;
  if (rank < 8 || rank > 128 || rank % 8)
    return fail(AWQ_ERR_UNSUPPORTED, "rank=%d: multiples of 8 from 8 to 128 are implemented", rank);
  if ((rc = check_count(n_adapters, awq::kMaxAdapters, "n_adapters"))) return rc;
  if (n_adapters * rank * in_features > kMaxWeights || n_adapters * rank * out_features > kMaxWeights)
    return fail(AWQ_ERR_INVALID_ARG, "n_adapters=%lld of rank %d are more than %lld values",
                (long long)n_adapters, rank, (long long)kMaxWeights);
  return AWQ_OK;
}
int check_y_type(int dtype, int y_dtype) {
  if (y_dtype != dtype && y_dtype != AWQ_F32)
    return fail(AWQ_ERR_UNSUPPORTED, "y_dtype=%d: dtype (%d) or AWQ_F32", y_dtype, dtype);
  return AWQ_OK;
}

int run_adapted(awq::W4Args& a, const awq::W4Adapt& d, bool backward, void* workspace,
                size_t workspace_bytes, void* stream, const char* what) {
  int rc;
  if ((rc = check_ptr(d.A, "A")) || (rc = check_ptr(d.B, "B")) || (rc = check_index(d.scale, "scale")) ||
      (rc = check_index(d.ids, "adapter")))
    return rc;
  const size_t need = awq::w4_adapt_workspace(a, d, backward);
  if (need) {
    if ((rc = check_ptr(workspace, "workspace"))) return rc;
    if (workspace_bytes < need)
      return fail(AWQ_ERR_WORKSPACE, "workspace %zu bytes < %zu required", workspace_bytes, need);
  }
  a.ws = workspace;
  const int64_t x = 2 * a.N * a.K, y = (a.y_type == AWQ_F32 ? 4 : 2) * a.N * a.O;
  const int64_t params = 2 * a.O * (a.K / a.group), na = d.count * (int64_t)d.rank * a.K,
                nb = d.count * (int64_t)d.rank * a.O, low = 4 * a.N * d.rank;
  const Span layer[7] = {{a.qweight, a.O * a.K / 2}, {a.step16, params}, {a.zero16, params},
                         {d.A, 2 * na},              {d.B, 2 * nb},      {d.scale, 4 * (int64_t)d.count},
                         {d.ids, 4 * a.N}};
  Span r[14] = {{a.ws, (int64_t)need}};
  int n = 1, written;
  if (backward) {
    r[n++] = {a.out0, x};
    r[n++] = {d.dA, 4 * na};
    r[n++] = {d.dB, 4 * nb};
    written = n;
    r[n++] = {a.in0, y};
    r[n++] = {a.in1, x};
    r[n++] = {d.low, low};
  } else {
    r[n++] = {a.out0, y};
    r[n++] = {d.low, low};
    written = n;
    r[n++] = {a.in0, x};
  }
  for (const Span& s : layer) r[n++] = s;
  if ((rc = check_spans(r, written, n))) return rc;
  return hip_result(awq::launch_w4_adapt(a, d, backward, (hipStream_t)stream), what);
}

awq::W4Adapt adapt_args(const void* A, const void* B, const float* scale, int64_t n_adapters,
                        int rank, const int32_t* adapter) {
  awq::W4Adapt d{};
  d.A = A;
  d.B = B;
  d.scale = scale;
  d.ids = adapter;
  d.count = (int)n_adapters;
  d.rank = rank;
  return d;
}

}  // namespace

extern "C" {

void awq_default_config(awq_config* cfg) {
  if (!cfg) return;
  cfg->w_bit = 4;
  cfg->group_size = 128;
  cfg->n_grid = 20;
  cfg->sal_floor = 1e-4f;
  cfg->zero_point = 1;
}

const char* awq_last_error(void) { return g_err; }

const char* awq_version(void) { return "awq_mi355x 0.1 gfx950"; }

size_t awq_act_stats_workspace_size(int64_t n_tokens, int64_t in_features) {
  if (check_dims(n_tokens, in_features, 1, true, false, 8) != AWQ_OK) return 0;
  return awq::stats_plan(n_tokens, in_features).workspace_bytes;
}

int awq_act_stats(const void* X, int64_t n_tokens, int64_t in_features, float* sal_out,
                  void* workspace, size_t workspace_bytes, void* stream) {
  int rc;
  if ((rc = check_dims(n_tokens, in_features, 1, true, false, 8))) return rc;
  if ((rc = check_ptr(X, "X")) || (rc = check_ptr(sal_out, "sal_out")) ||
      (rc = check_ptr(workspace, "workspace")))
    return rc;
  const size_t need = awq::stats_plan(n_tokens, in_features).workspace_bytes;
  if (workspace_bytes < need)
    return fail(AWQ_ERR_WORKSPACE, "workspace %zu bytes < %zu required", workspace_bytes, need);
  return hip_result(awq::launch_act_stats(X, n_tokens, in_features, sal_out, workspace,
                                          (hipStream_t)stream),
                    "awq_act_stats launch");
}

int awq_act_stats_noalloc(const void* X, int64_t n_tokens, int64_t in_features, float* sal_out,
                          void* stream) {
  int rc;
  if ((rc = check_dims(n_tokens, in_features, 1, true, false, 8))) return rc;
  if ((rc = check_ptr(X, "X")) || (rc = check_ptr(sal_out, "sal_out"))) return rc;
  const size_t need = awq::stats_scratch_need(n_tokens, in_features);
  if (need > awq::kStatsScratchBytes)
    return fail(AWQ_ERR_WORKSPACE,
                "n_tokens=%lld x in_features=%lld needs %zu bytes of partial sums, above the "
                "%zu-byte scratch of awq_act_stats_noalloc (awq_act_stats takes a workspace)",
                (long long)n_tokens, (long long)in_features, need, awq::kStatsScratchBytes);
  void* ws = nullptr;
  if ((rc = hip_result(awq::scratch_address(&ws), "awq_act_stats_noalloc scratch address")))
    return rc;
  return hip_result(awq::launch_act_stats(X, n_tokens, in_features, sal_out, ws,
                                          (hipStream_t)stream),
                    "awq_act_stats_noalloc launch");
}

int awq_search_plan_query(int64_t n_tokens, int64_t in_features, int64_t out_features,
                          const awq_config* cfg, awq_search_plan* plan) {
  int rc;
  if ((rc = check_config(cfg))) return rc;
  if ((rc = check_dims(n_tokens, in_features, out_features, true, true, 128))) return rc;
  if (!plan) return fail(AWQ_ERR_INVALID_ARG, "plan is NULL");
  const awq::SearchPlan p = awq::search_plan(n_tokens, in_features, out_features, cfg->n_grid,
                                                 quant_spec(cfg));
  if (p.grid_blocks > awq::kMaxGridBlocks)
    return fail(AWQ_ERR_INVALID_ARG, "layer too large for one search launch (%lld tiles)",
                (long long)(p.n_t_tiles * p.n_o_tiles));
  plan->tile_tokens = p.tile_m;
  plan->tile_out = p.tile_n;
  plan->n_token_tiles = p.n_t_tiles;
  plan->n_out_tiles = p.n_o_tiles;
  plan->partials_offset = p.off_partials;
  plan->scales_offset = p.off_s;
  plan->workspace_bytes = p.bytes;
  return ok();
}

size_t awq_search_workspace_size(int64_t n_tokens, int64_t in_features, int64_t out_features,
                                 const awq_config* cfg) {
  awq_search_plan plan;
  if (awq_search_plan_query(n_tokens, in_features, out_features, cfg, &plan) != AWQ_OK) return 0;
  return plan.workspace_bytes;
}

int awq_search_layer(const void* X, const void* W, const float* sal, int64_t n_tokens,
                     int64_t in_features, int64_t out_features, const awq_config* cfg,
                     double* losses_out, int32_t* best_idx_out, float* s_best_out,
                     void* workspace, size_t workspace_bytes, void* stream) {
  return awq_search_layer_stages(AWQ_STAGE_ALL, X, W, sal, n_tokens, in_features, out_features,
                                 cfg, losses_out, best_idx_out, s_best_out, workspace,
                                 workspace_bytes, stream);
}

int awq_search_layer_stages(int stage_mask, const void* X, const void* W, const float* sal,
                            int64_t n_tokens, int64_t in_features, int64_t out_features,
                            const awq_config* cfg, double* losses_out, int32_t* best_idx_out,
                            float* s_best_out, void* workspace, size_t workspace_bytes,
                            void* stream) {
  int rc;
  if (stage_mask < 1 || stage_mask > AWQ_STAGE_ALL)
    return fail(AWQ_ERR_INVALID_ARG, "stage_mask=%d: must be a non-empty OR of AWQ_STAGE_*",
                stage_mask);
  if ((rc = check_config(cfg))) return rc;
  if ((rc = check_dims(n_tokens, in_features, out_features, true, true, 128))) return rc;
  if ((rc = check_ptr(X, "X")) || (rc = check_ptr(W, "W")) || (rc = check_ptr(sal, "sal")) ||
      (rc = check_ptr(losses_out, "losses_out")) ||
      (rc = check_ptr(s_best_out, "s_best_out")) || (rc = check_ptr(workspace, "workspace")))
    return rc;
  if (!best_idx_out) return fail(AWQ_ERR_INVALID_ARG, "best_idx_out is NULL");
  const awq::SearchPlan p = awq::search_plan(n_tokens, in_features, out_features, cfg->n_grid,
                                                 quant_spec(cfg));
  if (p.grid_blocks > awq::kMaxGridBlocks)
    return fail(AWQ_ERR_INVALID_ARG, "layer too large for one search launch (%lld tiles)",
                (long long)(p.n_t_tiles * p.n_o_tiles));
  if (workspace_bytes < p.bytes)
    return fail(AWQ_ERR_WORKSPACE, "workspace %zu bytes < %zu required", workspace_bytes, p.bytes);
  return hip_result(awq::launch_search(X, W, sal, n_tokens, in_features, out_features,
                                       cfg->n_grid, cfg->sal_floor, losses_out, best_idx_out,
                                       s_best_out, workspace, p, stage_mask, (hipStream_t)stream),
                    "awq_search_layer launch");
}

int awq_pack(const void* W, const float* s, int64_t in_features, int64_t out_features,
             const awq_config* cfg, int32_t* qweight_out, void* step_out, void* zero_out,
             void* stream) {
  int rc;
  if ((rc = check_config(cfg))) return rc;
  if ((rc = check_dims(1, in_features, out_features, false, true, 128))) return rc;
  if ((rc = check_ptr(W, "W")) || (rc = check_ptr(s, "s")) ||
      (rc = check_ptr(qweight_out, "qweight_out")))
    return rc;
  if (!step_out || !zero_out) return fail(AWQ_ERR_INVALID_ARG, "step_out/zero_out is NULL");
  if (((uintptr_t)step_out & 1u) || ((uintptr_t)zero_out & 1u))
    return fail(AWQ_ERR_INVALID_ARG, "step_out/zero_out must be 2-byte aligned");
  return hip_result(awq::launch_pack(W, s, in_features, out_features, quant_spec(cfg), qweight_out,
                                     step_out, zero_out, (hipStream_t)stream),
                    "awq_pack launch");
}

int awq_w4a16_matmul(const void* X, int64_t n_tokens, int64_t in_features, int64_t out_features,
                     const int32_t* qweight, const void* step16, const void* zero16, float* Y,
                     void* stream) {
  int rc;
  if ((rc = check_dims(1, in_features, out_features, false, true, 128))) return rc;
  if (n_tokens < 1 || n_tokens > awq::kMaxW4Tokens)
    return fail(AWQ_ERR_INVALID_ARG, "n_tokens=%lld outside 1..%lld", (long long)n_tokens,
                (long long)awq::kMaxW4Tokens);
  if ((rc = check_ptr(X, "X")) || (rc = check_ptr(qweight, "qweight"))) return rc;
  if (!step16 || !zero16 || !Y) return fail(AWQ_ERR_INVALID_ARG, "step16/zero16/Y is NULL");
  if (((uintptr_t)step16 & 1u) || ((uintptr_t)zero16 & 1u) || ((uintptr_t)Y & 3u))
    return fail(AWQ_ERR_INVALID_ARG, "step16/zero16 must be 2-byte and Y 4-byte aligned");
  return hip_result(awq::launch_w4a16(X, n_tokens, in_features, out_features, qweight, step16,
                                      zero16, Y, (hipStream_t)stream),
                    "awq_w4a16_matmul launch");
}

size_t awq_w4a16_linear_workspace_size(int64_t n_tokens, int64_t in_features, int64_t out_features,
                                       int group_size, int dtype) {
  if (check_w4(n_tokens, in_features, out_features, group_size, dtype)) return (size_t)-1;
  ok();
  return awq::w4_workspace(awq::kOpLinear, w4_args(n_tokens, in_features, out_features, group_size,
                                                   dtype, 0, nullptr, nullptr, nullptr));
}

int awq_w4a16_linear(const void* X, int dtype, int64_t n_tokens, int64_t in_features,
                     int64_t out_features, int group_size, const int32_t* qweight,
                     const void* step16, const void* zero16, void* Y, int y_dtype, void* workspace,
                     size_t workspace_bytes, void* stream) {
  int rc;
  if ((rc = check_w4(n_tokens, in_features, out_features, group_size, dtype))) return rc;
  if ((rc = check_y_type(dtype, y_dtype))) return rc;
  if ((rc = check_ptr(X, "X")) || (rc = check_layer(qweight, step16, zero16)) ||
      (rc = check_ptr(Y, "Y")))
    return rc;
  awq::W4Args a = w4_args(n_tokens, in_features, out_features, group_size, dtype, 0, qweight,
                          step16, zero16);
  a.y_type = y_dtype;
  a.in0 = X;
  a.out0 = Y;
  const W4Bytes b{2 * a.N * a.K, 0, (y_dtype == AWQ_F32 ? 4 : 2) * a.N * a.O, 0};
  return run_w4(awq::kOpLinear, a, b, workspace, workspace_bytes, stream, "awq_w4a16_linear launch");
}

size_t awq_w4a16_gated_workspace_size(int64_t n_tokens, int64_t in_features, int64_t half_features,
                                      int group_size, int dtype) {
  if (check_w4_gated(n_tokens, in_features, half_features, group_size, dtype, 0)) return (size_t)-1;
  ok();
  return awq::w4_workspace(awq::kOpGated, w4_args(n_tokens, in_features, 2 * half_features,
                                                  group_size, dtype, 0, nullptr, nullptr, nullptr));
}

int awq_w4a16_gated(const void* X, int dtype, int64_t n_tokens, int64_t in_features,
                    int64_t half_features, int group_size, int act, const int32_t* qweight,
                    const void* step16, const void* zero16, void* H, void* pre, void* workspace,
                    size_t workspace_bytes, void* stream) {
  int rc;
  if ((rc = check_w4_gated(n_tokens, in_features, half_features, group_size, dtype, act))) return rc;
  if ((rc = check_ptr(X, "X")) || (rc = check_layer(qweight, step16, zero16)) ||
      (rc = check_ptr(H, "H")) || (pre && (rc = check_ptr(pre, "pre"))))
    return rc;
  awq::W4Args a = w4_args(n_tokens, in_features, 2 * half_features, group_size, dtype, act, qweight,
                          step16, zero16);
  a.in0 = X;
  a.out0 = H;
  a.out1 = pre;
  const W4Bytes b{2 * a.N * a.K, 0, a.N * a.O, 2 * a.N * a.O};
  return run_w4(awq::kOpGated, a, b, workspace, workspace_bytes, stream, "awq_w4a16_gated launch");
}

size_t awq_w4a16_input_grad_workspace_size(int64_t n_tokens, int64_t in_features,
                                           int64_t out_features, int group_size, int dtype) {
  if (check_w4(n_tokens, in_features, out_features, group_size, dtype)) return (size_t)-1;
  ok();
  return awq::w4_workspace(awq::kOpInputGrad, w4_args(n_tokens, in_features, out_features,
                                                      group_size, dtype, 0, nullptr, nullptr,
                                                      nullptr));
}

int awq_w4a16_input_grad(const void* dY, int dtype, int64_t n_tokens, int64_t in_features,
                         int64_t out_features, int group_size, const int32_t* qweight,
                         const void* step16, const void* zero16, void* dX, void* workspace,
                         size_t workspace_bytes, void* stream) {
  int rc;
  if ((rc = check_w4(n_tokens, in_features, out_features, group_size, dtype))) return rc;
  if ((rc = check_ptr(dY, "dY")) || (rc = check_layer(qweight, step16, zero16)) ||
      (rc = check_ptr(dX, "dX")))
    return rc;
  awq::W4Args a = w4_args(n_tokens, in_features, out_features, group_size, dtype, 0, qweight,
                          step16, zero16);
  a.in0 = dY;
  a.out0 = dX;
  const W4Bytes b{2 * a.N * a.O, 0, 2 * a.N * a.K, 0};
  return run_w4(awq::kOpInputGrad, a, b, workspace, workspace_bytes, stream,
                "awq_w4a16_input_grad launch");
}

size_t awq_w4a16_gated_backward_workspace_size(int64_t n_tokens, int64_t in_features,
                                               int64_t half_features, int group_size, int dtype) {
  if (check_w4_gated(n_tokens, in_features, half_features, group_size, dtype, 0)) return (size_t)-1;
  ok();
  return awq::w4_workspace(awq::kOpGatedBackward,
                           w4_args(n_tokens, in_features, 2 * half_features, group_size, dtype, 0,
                                   nullptr, nullptr, nullptr));
}

int awq_w4a16_gated_backward(const void* dH, const void* pre, int dtype, int64_t n_tokens,
                             int64_t in_features, int64_t half_features, int group_size, int act,
                             const int32_t* qweight, const void* step16, const void* zero16,
                             void* dpre, void* dX, void* workspace, size_t workspace_bytes,
                             void* stream) {
  int rc;
  if ((rc = check_w4_gated(n_tokens, in_features, half_features, group_size, dtype, act))) return rc;
  if ((rc = check_ptr(dH, "dH")) || (rc = check_ptr(pre, "pre")) ||
      (rc = check_layer(qweight, step16, zero16)) || (rc = check_ptr(dpre, "dpre")) ||
      (rc = check_ptr(dX, "dX")))
    return rc;
  awq::W4Args a = w4_args(n_tokens, in_features, 2 * half_features, group_size, dtype, act, qweight,
                          step16, zero16);
  a.in0 = dH;
  a.in1 = pre;
  a.out0 = dX;
  a.out1 = dpre;
  const W4Bytes b{a.N * a.O, 2 * a.N * a.O, 2 * a.N * a.K, 2 * a.N * a.O};
  return run_w4(awq::kOpGatedBackward, a, b, workspace, workspace_bytes, stream,
                "awq_w4a16_gated_backward launch");
}

size_t awq_w4a16_param_grad_workspace_size(int64_t n_tokens, int64_t in_features,
                                           int64_t out_features, int group_size, int dtype) {
  if (check_w4(n_tokens, in_features, out_features, group_size, dtype)) return (size_t)-1;
  ok();
  return awq::w4_workspace(awq::kOpParamGrad, w4_args(n_tokens, in_features, out_features,
                                                      group_size, dtype, 0, nullptr, nullptr,
                                                      nullptr));
}

int awq_w4a16_param_grad(const void* dY, const void* X, int dtype, int64_t n_tokens,
                         int64_t in_features, int64_t out_features, int group_size,
                         const int32_t* qweight, const void* step16, const void* zero16,
                         float* dstep, float* dzero, void* workspace, size_t workspace_bytes,
                         void* stream) {
  int rc;
  if ((rc = check_w4(n_tokens, in_features, out_features, group_size, dtype))) return rc;
  if ((rc = check_ptr(dY, "dY")) || (rc = check_ptr(X, "X")) ||
      (rc = check_layer(qweight, step16, zero16)) || (rc = check_ptr(dstep, "dstep")) ||
      (rc = check_ptr(dzero, "dzero")))
    return rc;
  awq::W4Args a = w4_args(n_tokens, in_features, out_features, group_size, dtype, 0, qweight,
                          step16, zero16);
  a.in0 = dY;
  a.in1 = X;
  a.out0 = dstep;
  a.out1 = dzero;
  const int64_t params = 4 * a.O * (a.K / a.group);
  const W4Bytes b{2 * a.N * a.O, 2 * a.N * a.K, params, params};
  return run_w4(awq::kOpParamGrad, a, b, workspace, workspace_bytes, stream,
                "awq_w4a16_param_grad launch");
}

size_t awq_w4a16_adapted_workspace_size(int64_t n_tokens, int64_t in_features, int64_t out_features,
                                        int group_size, int dtype, int y_dtype, int64_t n_adapters,
                                        int rank, int /* keep_low */) {
  if (check_w4(n_tokens, in_features, out_features, group_size, dtype) ||
      check_y_type(dtype, y_dtype) || check_adapters(n_adapters, rank, in_features, out_features))
    return (size_t)-1;
  ok();
  awq::W4Args a = w4_args(n_tokens, in_features, out_features, group_size, dtype, 0, nullptr, nullptr,
                          nullptr);
  a.y_type = y_dtype;
  return awq::w4_adapt_workspace(a, adapt_args(nullptr, nullptr, nullptr, n_adapters, rank, nullptr), false);
}

int awq_w4a16_adapted(const void* X, int dtype, int64_t n_tokens, int64_t in_features,
                      int64_t out_features, int group_size, const int32_t* qweight,
                      const void* step16, const void* zero16, const void* A, const void* B,
                      const float* scale, int64_t n_adapters, int rank, const int32_t* adapter,
                      void* Y, int y_dtype, float* low, void* workspace, size_t workspace_bytes,
                      void* stream) {
  int rc;
  if ((rc = check_w4(n_tokens, in_features, out_features, group_size, dtype)) ||
      (rc = check_y_type(dtype, y_dtype)) ||
      (rc = check_adapters(n_adapters, rank, in_features, out_features)) || (rc = check_ptr(X, "X")) ||
      (rc = check_layer(qweight, step16, zero16)) || (rc = check_ptr(Y, "Y")) ||
      (low && (rc = check_ptr(low, "low"))))
    return rc;
  awq::W4Args a = w4_args(n_tokens, in_features, out_features, group_size, dtype, 0, qweight, step16,
                          zero16);
  a.y_type = y_dtype;
  a.in0 = X;
  a.out0 = Y;
  awq::W4Adapt d = adapt_args(A, B, scale, n_adapters, rank, adapter);
  d.low = low;
  return run_adapted(a, d, false, workspace, workspace_bytes, stream, "awq_w4a16_adapted launch");
}

size_t awq_w4a16_adapted_backward_workspace_size(int64_t n_tokens, int64_t in_features,
                                                 int64_t out_features, int group_size, int dtype,
                                                 int64_t n_adapters, int rank) {
  if (check_w4(n_tokens, in_features, out_features, group_size, dtype) ||
      check_adapters(n_adapters, rank, in_features, out_features))
    return (size_t)-1;
  ok();
  return awq::w4_adapt_workspace(
      w4_args(n_tokens, in_features, out_features, group_size, dtype, 0, nullptr, nullptr, nullptr),
      adapt_args(nullptr, nullptr, nullptr, n_adapters, rank, nullptr), true);
}

int awq_w4a16_adapted_backward(const void* dY, const void* X, const float* low, int dtype,
                               int64_t n_tokens, int64_t in_features, int64_t out_features,
                               int group_size, const int32_t* qweight, const void* step16,
                               const void* zero16, const void* A, const void* B, const float* scale,
                               int64_t n_adapters, int rank, const int32_t* adapter, void* dX,
                               float* dA, float* dB, void* workspace, size_t workspace_bytes,
                               void* stream) {
  int rc;
  if ((rc = check_w4(n_tokens, in_features, out_features, group_size, dtype)) ||
      (rc = check_adapters(n_adapters, rank, in_features, out_features)) ||
      (rc = check_ptr(dY, "dY")) || (rc = check_ptr(X, "X")) || (rc = check_ptr(low, "low")) ||
      (rc = check_layer(qweight, step16, zero16)) || (rc = check_ptr(dX, "dX")) ||
      (rc = check_ptr(dA, "dA")) || (rc = check_ptr(dB, "dB")))
    return rc;
  awq::W4Args a = w4_args(n_tokens, in_features, out_features, group_size, dtype, 0, qweight, step16,
                          zero16);
  a.in0 = dY;
  a.in1 = X;
  a.out0 = dX;
  awq::W4Adapt d = adapt_args(A, B, scale, n_adapters, rank, adapter);
  d.low = const_cast<float*>(low);
  d.dA = dA;
  d.dB = dB;
  return run_adapted(a, d, true, workspace, workspace_bytes, stream,
                     "awq_w4a16_adapted_backward launch");
}

int awq_kv4_append(const awq_kv4_cache* cache, const void* k, const void* v, int dtype,
                   int64_t n_tokens, int64_t k_token_stride, int64_t k_head_stride,
                   int64_t v_token_stride, int64_t v_head_stride, const int32_t* slots,
                   void* stream) {
  int rc;
  awq::Kv4 c;
  if ((rc = check_kv4(cache, &c)) || (rc = check_16bit(dtype)) ||
      (rc = check_count(n_tokens, awq::kMaxW4OpTokens, "n_tokens")) || (rc = check_kv4_arrays(c)) ||
      (rc = check_ptr(k, "k")) || (rc = check_ptr(v, "v")) || (rc = check_index(slots, "slots")) ||
      (rc = check_stride(k_token_stride, "k_token_stride")) ||
      (rc = check_stride(k_head_stride, "k_head_stride")) ||
      (rc = check_stride(v_token_stride, "v_token_stride")) ||
      (rc = check_stride(v_head_stride, "v_head_stride")))
    return rc;
  const Span r[7] = {{c.k_codes, kv4_code_bytes(c)},
                     {c.v_codes, kv4_code_bytes(c)},
                     {c.k_params, kv4_param_bytes(c)},
                     {c.v_params, kv4_param_bytes(c)},
                     {k, rows_bytes(n_tokens, c.heads, c.dim, k_token_stride, k_head_stride)},
                     {v, rows_bytes(n_tokens, c.heads, c.dim, v_token_stride, v_head_stride)},
                     {slots, 4 * n_tokens}};
  if ((rc = check_spans(r, 4, 7))) return rc;
  const awq::Kv4Rows rows{k, v, k_token_stride, k_head_stride, v_token_stride, v_head_stride};
  return hip_result(awq::launch_kv4_append(c, rows, dtype, n_tokens, slots, (hipStream_t)stream),
                    "awq_kv4_append launch");
}

int awq_kv4_gather(const awq_kv4_cache* cache, const int32_t* slots, int64_t n_tokens, void* k,
                   void* v, int dtype, void* stream) {
  int rc;
  awq::Kv4 c;
  if ((rc = check_kv4(cache, &c)) || (rc = check_16bit(dtype)) ||
      (rc = check_count(n_tokens, awq::kMaxW4OpTokens, "n_tokens")) || (rc = check_kv4_arrays(c)) ||
      (rc = check_index(slots, "slots")) || (rc = check_ptr(k, "k")) || (rc = check_ptr(v, "v")))
    return rc;
  const int64_t bytes = 2 * n_tokens * c.heads * c.dim;
  const Span r[7] = {{k, bytes},
                     {v, bytes},
                     {slots, 4 * n_tokens},
                     {c.k_codes, kv4_code_bytes(c)},
                     {c.v_codes, kv4_code_bytes(c)},
                     {c.k_params, kv4_param_bytes(c)},
                     {c.v_params, kv4_param_bytes(c)}};
  if ((rc = check_spans(r, 2, 7))) return rc;
  return hip_result(awq::launch_kv4_gather(c, n_tokens, slots, k, v, dtype, (hipStream_t)stream),
                    "awq_kv4_gather launch");
}

size_t awq_kv4_attention_workspace_size(const awq_kv4_cache* cache, int64_t n_tokens,
                                        int64_t n_heads, int64_t n_seqs, int64_t max_pages,
                                        int has_starts) {
  awq::Kv4Attention a{};
  if (kv4_attention_args(cache, n_tokens, n_heads, n_seqs, max_pages, has_starts != 0, &a))
    return (size_t)-1;
  ok();
  return awq::kv4_attention_workspace(a);
}

int awq_kv4_attention(const awq_kv4_cache* cache, const void* q, int dtype, int64_t n_tokens,
                      int64_t n_heads, int64_t q_token_stride, int64_t q_head_stride,
                      int64_t n_seqs, const int32_t* starts, const int32_t* table,
                      int64_t max_pages, const int32_t* lens, float scale, void* out,
                      void* workspace, size_t workspace_bytes, void* stream) {
  int rc;
  awq::Kv4Attention a{};
  if ((rc = kv4_attention_args(cache, n_tokens, n_heads, n_seqs, max_pages, starts != nullptr, &a)) ||
      (rc = check_16bit(dtype)) || (rc = check_kv4_arrays(a.cache)) || (rc = check_ptr(q, "q")) ||
      (rc = check_ptr(out, "out")) || (rc = check_index(table, "table")) ||
      (rc = check_index(lens, "lens")) || (starts && (rc = check_index(starts, "starts"))) ||
      (rc = check_stride(q_token_stride, "q_token_stride")) ||
      (rc = check_stride(q_head_stride, "q_head_stride")))
    return rc;
  // up to it what the kernels cut of bf16 queries (below 2^-94) costs less than 2^-34 of a weight
  if (!(scale >= -0x1p32f && scale <= 0x1p32f))
    return fail(AWQ_ERR_INVALID_ARG, "scale=%g outside -2^32..2^32", (double)scale);
  const size_t need = awq::kv4_attention_workspace(a);
  if (need) {
    if ((rc = check_ptr(workspace, "workspace"))) return rc;
    if (workspace_bytes < need)
      return fail(AWQ_ERR_WORKSPACE, "workspace %zu bytes < %zu required", workspace_bytes, need);
  }
  a.q = q;
  a.out = out;
  a.type = dtype;
  a.q_token = q_token_stride;
  a.q_head = q_head_stride;
  a.starts = starts;
  a.table = table;
  a.lens = lens;
  a.scale = scale;
  a.ws = workspace;
  const awq::Kv4& c = a.cache;
  const Span r[10] = {{out, 2 * n_tokens * n_heads * c.dim},
                      {workspace, (int64_t)need},
                      {q, rows_bytes(n_tokens, n_heads, c.dim, q_token_stride, q_head_stride)},
                      {starts, 4 * (n_seqs + 1)},
                      {table, 4 * n_seqs * max_pages},
                      {lens, 4 * n_seqs},
                      {c.k_codes, kv4_code_bytes(c)},
                      {c.v_codes, kv4_code_bytes(c)},
                      {c.k_params, kv4_param_bytes(c)},
                      {c.v_params, kv4_param_bytes(c)}};
  if ((rc = check_spans(r, 2, 10))) return rc;
  return hip_result(awq::launch_kv4_attention(a, (hipStream_t)stream), "awq_kv4_attention launch");
}

int awq_fold_inverse_scale(const void* src, const float* s, int64_t rows, int64_t cols, void* dst,
                           void* stream) {
  if (!src || !s || !dst) return fail(AWQ_ERR_INVALID_ARG, "src/s/dst is NULL");
  if (rows < 1 || rows > kMaxFeatures || cols < 1 || cols > kMaxFeatures || rows * cols > kMaxWeights)
    return fail(AWQ_ERR_INVALID_ARG, "rows=%lld cols=%lld out of range", (long long)rows,
                (long long)cols);
  if (((uintptr_t)src & 1u) || ((uintptr_t)dst & 1u) || ((uintptr_t)s & 3u))
    return fail(AWQ_ERR_INVALID_ARG, "src/dst must be 2-byte and s 4-byte aligned");
  const char* a = (const char*)src;
  const char* b = (const char*)dst;
  const int64_t bytes = rows * cols * 2;
  if (a != b && a < b + bytes && b < a + bytes)
    return fail(AWQ_ERR_INVALID_ARG, "src and dst overlap without being the same array");
  return hip_result(awq::launch_fold(src, s, rows, cols, dst, (hipStream_t)stream),
                    "awq_fold_inverse_scale launch");
}

int awq_select_top_channels(const float* sal, int64_t n, int64_t n_keep, float* sal_out,
                            void* stream) {
  if (!sal || !sal_out) return fail(AWQ_ERR_INVALID_ARG, "sal/sal_out is NULL");
  if (n < 1 || n > kMaxFeatures)
    return fail(AWQ_ERR_INVALID_ARG, "n=%lld outside 1..%lld", (long long)n, (long long)kMaxFeatures);
  if (n_keep < 0 || n_keep > n)
    return fail(AWQ_ERR_INVALID_ARG, "n_keep=%lld outside 0..n", (long long)n_keep);
  if (((uintptr_t)sal & 3u) || ((uintptr_t)sal_out & 3u))
    return fail(AWQ_ERR_INVALID_ARG, "sal/sal_out must be 4-byte aligned");
  if (sal != sal_out && sal < sal_out + n && sal_out < sal + n)
    return fail(AWQ_ERR_INVALID_ARG, "sal and sal_out overlap without being the same array");
  return hip_result(awq::launch_select_top(sal, n, n_keep, sal_out, (hipStream_t)stream),
                    "awq_select_top_channels launch");
}

}  // extern "C"
