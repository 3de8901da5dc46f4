// route_api.hip -- the extern "C" entry points of the router: argument checks on the host, then kernel launches on the
// caller's stream.  Nothing here allocates, synchronizes or keeps state.
#include <math.h>

#include "route_internal.hpp"

using namespace moe;

namespace {

bool aligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

int check_shape(const moe_route_shape_t *s) {
  if (!s) return MOE_ERR_ARG;
  if (s->num_tokens < 0 || s->num_ids <= 0 || s->topk <= 0 || s->num_groups <= 0 || s->topk_groups <= 0 ||
      s->topk_groups > s->num_groups || s->num_ids % s->num_groups != 0)
    return MOE_ERR_SHAPE;
  if (s->topk > (int64_t)s->topk_groups * (s->num_ids / s->num_groups)) return MOE_ERR_SHAPE;
  if (s->num_tokens >= 1 << 24 || s->num_ids > 2048 || s->topk > 16 || s->num_groups > 64) return MOE_ERR_UNSUPPORTED;
  if ((s->score != MOE_SCORE_SOFTMAX && s->score != MOE_SCORE_SIGMOID) ||
      (s->group_score != MOE_GROUP_MAX && s->group_score != MOE_GROUP_TOP2) ||
      (s->renormalize != 0 && s->renormalize != 1) || !isfinite(s->scale))
    return MOE_ERR_ARG;
  return MOE_OK;
}

int check_balance(const moe_route_shape_t *s, const moe_balance_t *b) {
  if (!b) return MOE_ERR_ARG;
  if (b->segments <= 0 || s->num_tokens % b->segments != 0) return MOE_ERR_SHAPE;
  return b->segments <= 4096 ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

int done(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// rows: those of grad_weights where there is a dst_row
int route_grad(const moe_route_shape_t *shape, int32_t logits_fp32, const void *logits, const int32_t *topk_idx,
               const float *grad_weights, int32_t rows, const int32_t *dst_row, const uint8_t *x_active_mask,
               const moe_balance_t *balance, const int32_t *counts, const int32_t *segment_tokens,
               const float *grad_losses, void *grad_logits, void *stream) {
  int st = check_shape(shape);
  if (st == MOE_OK && balance) st = check_balance(shape, balance);
  if (st != MOE_OK) return st;
  if (logits_fp32 != 0 && logits_fp32 != 1) return MOE_ERR_ARG;
  if (!balance && (counts || segment_tokens || grad_losses)) return MOE_ERR_ARG;
  if (shape->num_tokens == 0) return MOE_OK;
  if ((!balance || dst_row) && !grad_weights) return MOE_ERR_ARG;
  if (!logits || !grad_logits || !aligned(logits, 16) || !aligned(grad_logits, 16)) return MOE_ERR_ARG;
  if (grad_weights && (!topk_idx || !aligned(topk_idx, 4) || !aligned(grad_weights, 4) || !aligned(dst_row, 4)))
    return MOE_ERR_ARG;
  if (balance && (!counts || !segment_tokens || !aligned(counts, 4) || !aligned(segment_tokens, 4) || !aligned(grad_losses, 4)))
    return MOE_ERR_ARG;
  RouteGradArgs a;
  a.logits = logits;
  a.idx = topk_idx;
  a.gw = grad_weights;
  a.dst = dst_row;
  a.mask = x_active_mask;
  a.counts = counts;
  a.tokens = segment_tokens;
  a.gl = grad_losses;
  a.out = grad_logits;
  a.T = shape->num_tokens;
  a.E = shape->num_ids;
  a.K = shape->topk;
  a.S = balance ? balance->segments : 1;
  a.renorm = shape->renormalize;
  a.rows = rows;
  a.scale = shape->scale;
  a.balance_coef = balance ? balance->balance_coef : 0.0f;
  a.z_coef = balance ? balance->z_coef : 0.0f;
  return done(launch_route_grad(a, shape->score, logits_fp32 != 0, (hipStream_t)stream));
}

}  // namespace

extern "C" {

int moe_route_check_shape(const moe_route_shape_t *shape) { return check_shape(shape); }

int moe_route(const moe_route_shape_t *shape, int32_t logits_fp32, const void *logits, const float *bias,
              const uint8_t *x_active_mask, int32_t *topk_idx, float *topk_weights, void *stream) {
  const int st = check_shape(shape);
  if (st != MOE_OK) return st;
  if (logits_fp32 != 0 && logits_fp32 != 1) return MOE_ERR_ARG;
  if (shape->num_tokens == 0) return MOE_OK;
  if (!logits || !topk_idx || !topk_weights || !aligned(logits, 16) || !aligned(bias, 4) || !aligned(topk_idx, 4) ||
      !aligned(topk_weights, 4))
    return MOE_ERR_ARG;
  RouteArgs a;
  a.logits = logits;
  a.bias = bias;
  a.mask = x_active_mask;
  a.idx = topk_idx;
  a.w = topk_weights;
  a.T = shape->num_tokens;
  a.E = shape->num_ids;
  a.K = shape->topk;
  a.G = shape->num_groups;
  a.keep = shape->topk_groups;
  a.two = shape->group_score == MOE_GROUP_TOP2;
  a.renorm = shape->renormalize;
  a.scale = shape->scale;
  return done(launch_route(a, shape->score, logits_fp32 != 0, (hipStream_t)stream));
}

size_t moe_balance_workspace_size(const moe_route_shape_t *shape, const moe_balance_t *balance) {
  if (check_shape(shape) != MOE_OK || check_balance(shape, balance) != MOE_OK) return 0;
  return balance_workspace(shape->num_tokens, shape->num_ids, balance->segments);
}

int moe_balance_loss(const moe_route_shape_t *shape, const moe_balance_t *balance, int32_t logits_fp32,
                     const void *logits, const int32_t *topk_idx, const uint8_t *x_active_mask, float *losses,
                     int32_t *counts, float *prob_sums, int32_t *segment_tokens, void *workspace,
                     size_t workspace_bytes, void *stream) {
  int st = check_shape(shape);
  if (st == MOE_OK) st = check_balance(shape, balance);
  if (st != MOE_OK) return st;
  if (logits_fp32 != 0 && logits_fp32 != 1) return MOE_ERR_ARG;
  if (!losses || !counts || !prob_sums || !segment_tokens || !workspace || !aligned(losses, 4) || !aligned(counts, 4) ||
      !aligned(prob_sums, 4) || !aligned(segment_tokens, 4) || !aligned(workspace, 16))
    return MOE_ERR_ARG;
  if (workspace_bytes < balance_workspace(shape->num_tokens, shape->num_ids, balance->segments)) return MOE_ERR_ARG;
  if (shape->num_tokens > 0 && (!logits || !topk_idx || !aligned(logits, 16) || !aligned(topk_idx, 4))) return MOE_ERR_ARG;
  BalanceArgs a;
  a.logits = logits;
  a.idx = topk_idx;
  a.mask = x_active_mask;
  a.losses = losses;
  a.counts = counts;
  a.sums = prob_sums;
  a.tokens = segment_tokens;
  a.ws = (char *)workspace;
  a.T = shape->num_tokens;
  a.E = shape->num_ids;
  a.K = shape->topk;
  a.S = balance->segments;
  a.balance_coef = balance->balance_coef;
  a.z_coef = balance->z_coef;
  return done(launch_balance(a, shape->score, logits_fp32 != 0, (hipStream_t)stream));
}

int moe_route_grad(const moe_route_shape_t *shape, int32_t logits_fp32, const void *logits, const int32_t *topk_idx,
                   const float *grad_topk_weights, const int32_t *dst_row, const uint8_t *x_active_mask,
                   const moe_balance_t *balance, const int32_t *counts, const int32_t *segment_tokens,
                   const float *grad_losses, void *grad_logits, void *stream) {
  return route_grad(shape, logits_fp32, logits, topk_idx, grad_topk_weights, INT32_MAX, dst_row, x_active_mask, balance, counts,
                    segment_tokens, grad_losses, grad_logits, stream);
}

int moe_route_grad_rows(const moe_route_shape_t *shape, int32_t logits_fp32, const void *logits, const int32_t *topk_idx,
                        const float *grad_row_weights, int64_t rows, const int32_t *dst_row, const uint8_t *x_active_mask,
                        const moe_balance_t *balance, const int32_t *counts, const int32_t *segment_tokens,
                        const float *grad_losses, void *grad_logits, void *stream) {
  const int st = check_shape(shape);
  if (st != MOE_OK) return st;
  if (rows < 0) return MOE_ERR_SHAPE;
  if (rows > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  if (shape->num_tokens > 0 && (!dst_row || (rows > 0 && !grad_row_weights))) return MOE_ERR_ARG;
  // without rows there is nothing to read, and the slots' gradients are zeros
  const float *g = rows > 0 ? grad_row_weights : (const float *)dst_row;
  return route_grad(shape, logits_fp32, logits, topk_idx, g, (int32_t)rows, dst_row, x_active_mask, balance, counts,
                    segment_tokens, grad_losses, grad_logits, stream);
}

}  // extern "C"
