// Exported C ABI of the token operators (include/seacells_token.h): host-side
// validation and dispatch onto the caller's stream. Argument checks run
// before any HIP call, so they also work on a machine without a GPU.
#include <cmath>

#include "seacells_debug.h"
#include "seacells_token.h"
#include "token.hpp"

using namespace seacells;

namespace {

constexpr uint32_t kTooLarge = 0x80000000u;
constexpr uint32_t kMaxWidth = SEACELLS_MAX_WIDTH;

bool aligned(const void *p, uint32_t dtype) {
  return (reinterpret_cast<uintptr_t>(p) & (dtype_size(dtype) - 1u)) == 0;
}

// Rows of d elements: sizes in range, the stride at least the row's length.
int check_rows(uint32_t n, uint32_t d, uint64_t ld) {
  if (d == 0 || ld < d) return SEACELLS_E_SHAPE;
  if (n >= kTooLarge || d > kMaxWidth || ld >= (1ull << 40)) return SEACELLS_E_TOO_LARGE;
  return SEACELLS_OK;
}

// Whether rows written in place of an operand's would lie on other rows of it.
bool in_place_apart(uint32_t n, const void *out, uint64_t out_ld, const void *in, uint64_t in_ld) {
  return n > 1 && out != nullptr && out == in && out_ld != in_ld;
}

int check_workspace(const void *ws, size_t bytes, size_t need) {
  if (need == 0) return SEACELLS_OK;
  if (ws == nullptr || bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
    return SEACELLS_E_WORKSPACE;
  return SEACELLS_OK;
}

hipStream_t hip_stream(seacells_stream_t s) { return reinterpret_cast<hipStream_t>(s); }

int done(hipError_t e, const char *what) {
  return e == hipSuccess ? SEACELLS_OK : hip_fail(e, what);
}

}  // namespace

extern "C" {

int seacells_embed(const void *table, uint32_t dtype, uint32_t v, uint32_t d, uint64_t table_ld,
                   const int32_t *tokens, uint32_t n, float scale, void *out, uint64_t out_ld,
                   uint32_t *status, seacells_stream_t stream) {
  if (table == nullptr || status == nullptr) return SEACELLS_E_NULL;
  if (n > 0 && (tokens == nullptr || out == nullptr)) return SEACELLS_E_NULL;
  if (!dtype_known(dtype) || !aligned(table, dtype) || !aligned(out, dtype) || !aligned(tokens, 0))
    return SEACELLS_E_TYPE;
  if (v == 0) return SEACELLS_E_SHAPE;
  int rc;
  if ((rc = check_rows(v, d, table_ld)) != SEACELLS_OK) return rc;
  if ((rc = check_rows(n, d, out_ld)) != SEACELLS_OK) return rc;
  return done(launch_embed(table, dtype, v, d, table_ld, tokens, n, scale, out, out_ld, status,
                           hip_stream(stream)),
              "embed launch");
}

size_t seacells_embed_grad_workspace(uint32_t n, uint32_t v, uint32_t d) {
  if (v == 0 || d == 0 || n >= kTooLarge || v >= kTooLarge || d > kMaxWidth) return 0;
  return plan_embed_grad(n, v, d).ws_bytes;
}

int seacells_embed_grad(const int32_t *tokens, uint32_t n, const void *d_out, uint32_t d_out_type,
                        uint64_t d_out_ld, uint32_t v, uint32_t d, float scale,
                        const void *add_to, void *d_table, uint32_t d_table_type,
                        uint64_t d_table_ld, void *workspace, size_t workspace_bytes,
                        uint32_t *status, seacells_stream_t stream) {
  if (d_table == nullptr || status == nullptr) return SEACELLS_E_NULL;
  if (n > 0 && (tokens == nullptr || d_out == nullptr)) return SEACELLS_E_NULL;
  if (!dtype_known(d_out_type) || !dtype_known(d_table_type) ||
      (d_table_type != d_out_type && d_table_type != SEACELLS_F32))
    return SEACELLS_E_TYPE;
  if (!aligned(d_out, d_out_type) || !aligned(d_table, d_table_type) ||
      !aligned(add_to, d_table_type) || !aligned(tokens, 0))
    return SEACELLS_E_TYPE;
  if (v == 0) return SEACELLS_E_SHAPE;
  int rc;
  if ((rc = check_rows(n, d, d_out_ld)) != SEACELLS_OK) return rc;
  if ((rc = check_rows(v, d, d_table_ld)) != SEACELLS_OK) return rc;
  const EmbedGradPlan plan = plan_embed_grad(n, v, d);
  if ((rc = check_workspace(workspace, workspace_bytes, plan.ws_bytes)) != SEACELLS_OK) return rc;
  return done(launch_embed_grad(plan, tokens, n, d_out, d_out_type, d_out_ld, v, d, scale, add_to,
                                d_table, d_table_type, d_table_ld, workspace, status,
                                hip_stream(stream)),
              "embed_grad launch");
}

int seacells_layer_norm(const void *x, uint32_t dtype, uint32_t n, uint32_t d, uint64_t x_ld,
                        const void *weight, const void *bias, uint32_t weight_type, float eps,
                        void *out, uint64_t out_ld, float *mean, float *rstd,
                        seacells_stream_t stream) {
  if (n > 0 && (x == nullptr || out == nullptr)) return SEACELLS_E_NULL;
  if (!dtype_known(dtype) || !dtype_known(weight_type) ||
      (weight_type != dtype && weight_type != SEACELLS_F32))
    return SEACELLS_E_TYPE;
  if (!aligned(x, dtype) || !aligned(out, dtype) || !aligned(weight, weight_type) ||
      !aligned(bias, weight_type) || !aligned(mean, 0) || !aligned(rstd, 0))
    return SEACELLS_E_TYPE;
  if (!(eps >= 0.0f && std::isfinite(eps))) return SEACELLS_E_SHAPE;
  if (in_place_apart(n, out, out_ld, x, x_ld)) return SEACELLS_E_SHAPE;
  int rc;
  if ((rc = check_rows(n, d, x_ld)) != SEACELLS_OK) return rc;
  if ((rc = check_rows(n, d, out_ld)) != SEACELLS_OK) return rc;
  return done(launch_layer_norm(x, dtype, n, d, x_ld, weight, bias, weight_type, eps, out, out_ld,
                                mean, rstd, hip_stream(stream)),
              "layer_norm launch");
}

size_t seacells_layer_norm_grad_workspace(uint32_t n, uint32_t d) {
  if (d == 0 || n >= kTooLarge || d > kMaxWidth) return 0;
  return plan_layer_norm_grad(n, d).ws_bytes;
}

int seacells_layer_norm_grad(const void *d_out, uint64_t d_out_ld, const void *x, uint32_t dtype,
                             uint32_t n, uint32_t d, uint64_t x_ld, const float *mean,
                             const float *rstd, const void *weight, uint32_t weight_type,
                             void *d_x, uint64_t d_x_ld, void *d_weight, void *d_bias,
                             void *workspace, size_t workspace_bytes, seacells_stream_t stream) {
  if (n > 0 && (d_out == nullptr || x == nullptr || mean == nullptr || rstd == nullptr))
    return SEACELLS_E_NULL;
  if (!dtype_known(dtype) || !dtype_known(weight_type) ||
      (weight_type != dtype && weight_type != SEACELLS_F32))
    return SEACELLS_E_TYPE;
  if (!aligned(d_out, dtype) || !aligned(x, dtype) || !aligned(d_x, dtype) ||
      !aligned(weight, weight_type) || !aligned(d_weight, weight_type) ||
      !aligned(d_bias, weight_type) || !aligned(mean, 0) || !aligned(rstd, 0))
    return SEACELLS_E_TYPE;
  if (in_place_apart(n, d_x, d_x_ld, x, x_ld) || in_place_apart(n, d_x, d_x_ld, d_out, d_out_ld))
    return SEACELLS_E_SHAPE;
  int rc;
  if ((rc = check_rows(n, d, d_out_ld)) != SEACELLS_OK) return rc;
  if ((rc = check_rows(n, d, x_ld)) != SEACELLS_OK) return rc;
  if (d_x != nullptr && (rc = check_rows(n, d, d_x_ld)) != SEACELLS_OK) return rc;
  const NormGradPlan plan = plan_layer_norm_grad(n, d);
  if ((rc = check_workspace(workspace, workspace_bytes, plan.ws_bytes)) != SEACELLS_OK) return rc;
  return done(launch_layer_norm_grad(plan, d_out, d_out_ld, x, dtype, n, d, x_ld, mean, rstd,
                                     weight, weight_type, d_x, d_x_ld, d_weight, d_bias, workspace,
                                     hip_stream(stream)),
              "layer_norm_grad launch");
}

size_t seacells_logprobs_workspace(uint32_t n, uint32_t v, uint32_t top_k) {
  if (v == 0 || n >= kTooLarge || v > kMaxWidth || top_k > SEACELLS_TOP_MAX) return 0;
  // one size covers every element type
  const size_t wide = plan_logprobs(SEACELLS_F32, n, v, top_k).ws_bytes;
  const size_t half = plan_logprobs(SEACELLS_BF16, n, v, top_k).ws_bytes;
  return wide > half ? wide : half;
}

int seacells_logprobs(const void *logits, uint32_t dtype, uint32_t n, uint32_t v, uint64_t ld,
                      const int32_t *targets, uint32_t top_k, float *logp, float *entropy,
                      float *stats, int32_t *top_idx, float *top_logp, void *workspace,
                      size_t workspace_bytes, uint32_t *status, seacells_stream_t stream) {
  if (status == nullptr || (logp != nullptr && targets == nullptr && n > 0)) return SEACELLS_E_NULL;
  if (n > 0 && (logits == nullptr || (top_k > 0 && (top_idx == nullptr || top_logp == nullptr))))
    return SEACELLS_E_NULL;
  if (!dtype_known(dtype) || !aligned(logits, dtype) || !aligned(targets, 0) || !aligned(logp, 0) ||
      !aligned(entropy, 0) || !aligned(stats, 0) || !aligned(top_idx, 0) || !aligned(top_logp, 0))
    return SEACELLS_E_TYPE;
  if (top_k > SEACELLS_TOP_MAX) return SEACELLS_E_SHAPE;
  int rc;
  if ((rc = check_rows(n, v, ld)) != SEACELLS_OK) return rc;
  const LogprobsPlan plan = plan_logprobs(dtype, n, v, top_k);
  if ((rc = check_workspace(workspace, workspace_bytes,
                            seacells_logprobs_workspace(n, v, top_k))) != SEACELLS_OK)
    return rc;
  return done(launch_logprobs(plan, logits, dtype, n, v, ld, targets, top_k, logp, entropy, stats,
                              top_idx, top_logp, workspace, status, hip_stream(stream)),
              "logprobs launch");
}

int seacells_logprobs_grad(const void *logits, uint32_t dtype, uint32_t n, uint32_t v,
                           uint64_t ld, const int32_t *targets, const float *stats,
                           const float *entropy, const float *d_logp, const float *d_entropy,
                           void *d_logits, uint64_t d_logits_ld, uint32_t *status,
                           seacells_stream_t stream) {
  if (status == nullptr) return SEACELLS_E_NULL;
  if (n > 0 && (logits == nullptr || stats == nullptr || d_logits == nullptr ||
                (d_entropy != nullptr && entropy == nullptr)))
    return SEACELLS_E_NULL;
  if (!dtype_known(dtype) || !aligned(logits, dtype) || !aligned(d_logits, dtype) ||
      !aligned(targets, 0) || !aligned(stats, 0) || !aligned(entropy, 0) || !aligned(d_logp, 0) ||
      !aligned(d_entropy, 0))
    return SEACELLS_E_TYPE;
  int rc;
  if ((rc = check_rows(n, v, ld)) != SEACELLS_OK) return rc;
  if ((rc = check_rows(n, v, d_logits_ld)) != SEACELLS_OK) return rc;
  if (d_logits == logits && d_logits_ld != ld) return SEACELLS_E_SHAPE;
  return done(launch_logprobs_grad(logits, dtype, n, v, ld, targets, stats, entropy, d_logp,
                                   d_entropy, d_logits, d_logits_ld, status, hip_stream(stream)),
              "logprobs_grad launch");
}

int seacells_debug_embed_plan(uint32_t n, uint32_t v, uint32_t d, seacells_embed_plan *out) {
  if (out == nullptr) return SEACELLS_E_NULL;
  if (v == 0 || d == 0) return SEACELLS_E_SHAPE;
  if (n >= kTooLarge || v >= kTooLarge || d > kMaxWidth) return SEACELLS_E_TOO_LARGE;
  const EmbedGradPlan p = plan_embed_grad(n, v, d);
  out->shift = p.shift;
  out->buckets = p.buckets;
  out->counters = p.counters;
  out->chunks = p.chunks;
  out->chunk_len = p.chunk_len;
  out->frequent = p.own ? 1u : 0u;
  out->cuts_offset = p.off_cuts;
  return SEACELLS_OK;
}

}  // extern "C"
