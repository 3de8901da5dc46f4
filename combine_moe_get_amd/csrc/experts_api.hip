// experts_api.hip -- the extern "C" entry points of the expert stage: argument checks on the host, then
// kernel launches on the caller's stream.  Nothing here allocates, synchronizes or keeps state.
#include <string.h>

#include "experts_internal.hpp"

using namespace moe;

namespace {

bool aligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

int step_of(int row_type) { return row_type == MOE_ROWS_BF16 ? 8 : row_type == MOE_ROWS_INT8 ? 16 : 32; }

// rows, windows and experts (not the feature counts)
int check_groups(const moe_experts_shape_t *s) {
  if (!s) return MOE_ERR_ARG;
  if (s->rows < 0 || s->rank_stride < 0) return MOE_ERR_SHAPE;
  if (s->num_ranks <= 0 || s->num_experts <= 0 || s->num_experts > 2048 || s->num_experts % s->num_ranks != 0)
    return MOE_ERR_SHAPE;
  if (s->rows >= (int64_t)1 << 27) return MOE_ERR_UNSUPPORTED;
  if (s->rank_stride > s->rows / s->num_ranks) return MOE_ERR_CAPACITY;
  return MOE_OK;
}

int check_shape(const moe_experts_shape_t *s, int row_type) {
  const int st = check_groups(s);
  if (st != MOE_OK) return st;
  if (row_type < MOE_ROWS_BF16 || row_type > MOE_ROWS_MXFP4) return MOE_ERR_ARG;
  if (s->in_features <= 0 || s->out_features <= 0) return MOE_ERR_SHAPE;
  if (s->in_features > 65536 || s->out_features > 65536 || s->in_features % step_of(row_type) != 0 ||
      s->out_features % 8 != 0)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

RowGroups groups(const moe_experts_shape_t *s, const int32_t *off) {
  RowGroups g;
  g.off = off;
  g.rows = s->rows;
  g.stride = s->rank_stride;
  g.E = s->num_experts;
  g.L = s->num_experts / s->num_ranks;
  return g;
}

// the sizes of a product's operands
ExpertsArgs sizes(const moe_experts_shape_t *s, int op, const int32_t *off) {
  ExpertsArgs a;
  memset(&a, 0, sizeof a);
  a.g = groups(s, off);
  a.K = op == OP_FORWARD ? s->in_features : op == OP_DGRAD ? s->out_features : 0;
  a.M = op == OP_WGRAD ? s->out_features : 0;
  a.N = op == OP_FORWARD ? s->out_features : s->in_features;
  return a;
}

// the sizes, rows and weights that the gate and its gradient have in common
int swiglu_args(int64_t rows, int32_t features, const float *row_weights, const moe_experts_shape_t *shape,
                const int32_t *expert_offsets, SwigluArgs &a) {
  if (rows < 0 || features <= 0) return MOE_ERR_SHAPE;
  if (features > 65536 || features % 8 != 0 || rows >= ((int64_t)1 << 42) / features) return MOE_ERR_UNSUPPORTED;
  memset(&a, 0, sizeof a);
  if (shape || expert_offsets) {
    const int st = check_groups(shape);
    if (st != MOE_OK) return st;
    if (shape->rows != rows || shape->in_features != features) return MOE_ERR_SHAPE;
    if (!expert_offsets || !aligned(expert_offsets, 4)) return MOE_ERR_ARG;
    a.g = groups(shape, expert_offsets);
  }
  if (!aligned(row_weights, 4)) return MOE_ERR_ARG;
  a.w = row_weights;
  a.rows = rows;
  a.I = features;
  return MOE_OK;
}

int done(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

}  // namespace

extern "C" {

int moe_experts_check_shape(const moe_experts_shape_t *shape, int32_t row_type) { return check_shape(shape, row_type); }

int moe_experts_tile(const moe_experts_shape_t *shape, int32_t op, int32_t row_type, int32_t act, int32_t tile[3]) {
  const int st = check_shape(shape, row_type);
  if (st != MOE_OK) return st;
  if (!tile || op < MOE_EXPERTS_FORWARD || op > MOE_EXPERTS_WGRAD || (act != MOE_ACT_NONE && act != MOE_ACT_SWIGLU))
    return MOE_ERR_ARG;
  if (op != MOE_EXPERTS_FORWARD && (row_type != MOE_ROWS_BF16 || act != MOE_ACT_NONE)) return MOE_ERR_ARG;
  const bool wide = row_type != MOE_ROWS_MXFP4 || mx_scales_wide(shape->in_features, nullptr, nullptr);
  const ExpertsTile t = experts_tile(sizes(shape, op, nullptr), op, row_type, act == MOE_ACT_SWIGLU, wide);
  tile[0] = t.rows;
  tile[1] = t.columns;
  tile[2] = t.stages;
  return MOE_OK;
}

int moe_experts_matmul(const moe_experts_shape_t *shape, int32_t row_type, int32_t act, const void *x,
                       const void *row_scales, const void *w, const void *w_scales, const int32_t *expert_offsets,
                       uint16_t *out, void *stream) {
  const int st = check_shape(shape, row_type);
  if (st != MOE_OK) return st;
  if (act != MOE_ACT_NONE && act != MOE_ACT_SWIGLU) return MOE_ERR_ARG;
  if (row_type == MOE_ROWS_BF16 && (row_scales || w_scales)) return MOE_ERR_ARG;
  if (row_type == MOE_ROWS_INT8 && (!aligned(row_scales, 4) || !aligned(w_scales, 4))) return MOE_ERR_ARG;
  if (shape->rows == 0) return MOE_OK;
  if (!x || !w || !expert_offsets || !out || !aligned(x, 16) || !aligned(w, 16) || !aligned(out, 16) ||
      !aligned(expert_offsets, 4))
    return MOE_ERR_ARG;
  if (row_type == MOE_ROWS_MXFP4 && (!row_scales || !w_scales)) return MOE_ERR_ARG;
  ExpertsArgs a = sizes(shape, OP_FORWARD, expert_offsets);
  a.m = x;
  a.n = w;
  a.ms = row_scales;
  a.ns = w_scales;
  a.out = out;
  return done(launch_experts(a, OP_FORWARD, row_type, act, false, (hipStream_t)stream));
}

int moe_experts_matmul_dgrad(const moe_experts_shape_t *shape, const uint16_t *grad_out, const uint16_t *w,
                             const int32_t *expert_offsets, uint16_t *grad_x, void *stream) {
  const int st = check_shape(shape, MOE_ROWS_BF16);
  if (st != MOE_OK) return st;
  if (shape->rows == 0) return MOE_OK;
  if (!grad_out || !w || !expert_offsets || !grad_x || !aligned(grad_out, 16) || !aligned(w, 16) ||
      !aligned(grad_x, 16) || !aligned(expert_offsets, 4))
    return MOE_ERR_ARG;
  ExpertsArgs a = sizes(shape, OP_DGRAD, expert_offsets);
  a.m = grad_out;
  a.n = w;
  a.out = grad_x;
  return done(launch_experts(a, OP_DGRAD, MOE_ROWS_BF16, MOE_ACT_NONE, false, (hipStream_t)stream));
}

int moe_experts_matmul_wgrad(const moe_experts_shape_t *shape, int32_t grad_w_fp32, const uint16_t *grad_out,
                             const uint16_t *x, const int32_t *expert_offsets, void *grad_w, void *stream) {
  const int st = check_shape(shape, MOE_ROWS_BF16);
  if (st != MOE_OK) return st;
  if (grad_w_fp32 != 0 && grad_w_fp32 != 1) return MOE_ERR_ARG;
  if (!expert_offsets || !grad_w || !aligned(grad_w, 16) || !aligned(expert_offsets, 4)) return MOE_ERR_ARG;
  if (shape->rows > 0 && (!grad_out || !x || !aligned(grad_out, 16) || !aligned(x, 16))) return MOE_ERR_ARG;
  ExpertsArgs a = sizes(shape, OP_WGRAD, expert_offsets);
  a.m = grad_out;
  a.n = x;
  a.out = grad_w;
  return done(launch_experts(a, OP_WGRAD, MOE_ROWS_BF16, MOE_ACT_NONE, grad_w_fp32 != 0, (hipStream_t)stream));
}

int moe_quantize_rows(int32_t row_type, int64_t rows, int32_t features, const uint16_t *x, void *codes,
                      void *scales, const moe_experts_shape_t *shape, const int32_t *expert_offsets, void *stream) {
  if (row_type != MOE_ROWS_INT8 && row_type != MOE_ROWS_MXFP4) return MOE_ERR_ARG;
  if (rows < 0 || features <= 0) return MOE_ERR_SHAPE;
  if (features > 65536 || features % step_of(row_type) != 0 || rows > ((int64_t)1 << 43) / features)
    return MOE_ERR_UNSUPPORTED;
  RowsQuantArgs a;
  memset(&a, 0, sizeof a);
  if (shape || expert_offsets) {
    const int st = check_groups(shape);
    if (st != MOE_OK) return st;
    if (shape->rows != rows || shape->in_features != features) return MOE_ERR_SHAPE;
    if (!expert_offsets || !aligned(expert_offsets, 4)) return MOE_ERR_ARG;
    a.g = groups(shape, expert_offsets);
  }
  if (rows == 0) return MOE_OK;
  if (!x || !codes || !scales || !aligned(x, 16) || !aligned(codes, 16)) return MOE_ERR_ARG;
  if (row_type == MOE_ROWS_INT8 && !aligned(scales, 4)) return MOE_ERR_ARG;
  a.x = x;
  a.codes = codes;
  a.scales = scales;
  a.rows = rows;
  a.H = features;
  return done(launch_rows_quant(a, row_type, (hipStream_t)stream));
}

int moe_swiglu(int64_t rows, int32_t features, const uint16_t *h0, const float *row_weights,
               const moe_experts_shape_t *shape, const int32_t *expert_offsets, uint16_t *out, int8_t *codes,
               float *scales, void *stream) {
  SwigluArgs a;
  const int st = swiglu_args(rows, features, row_weights, shape, expert_offsets, a);
  if (st != MOE_OK) return st;
  if (rows == 0) return MOE_OK;
  if (!h0 || !out || !aligned(h0, 16) || !aligned(out, 16) || !codes != !scales || !aligned(codes, 16) ||
      !aligned(scales, 4))
    return MOE_ERR_ARG;
  a.h0 = h0;
  a.out = out;
  a.codes = codes;
  a.scales = scales;
  return done(launch_swiglu(a, (hipStream_t)stream));
}

int moe_swiglu_grad(int64_t rows, int32_t features, const uint16_t *grad_out, const uint16_t *h0, const int8_t *codes,
                    const float *scales, const float *row_weights, const moe_experts_shape_t *shape,
                    const int32_t *expert_offsets, uint16_t *grad_h0, uint16_t *out, float *grad_row_weights,
                    void *stream) {
  SwigluArgs a;
  const int st = swiglu_args(rows, features, row_weights, shape, expert_offsets, a);
  if (st != MOE_OK) return st;
  if (rows == 0) return MOE_OK;
  if (!grad_out || !aligned(grad_out, 16) || !codes != !scales || !h0 == !codes || !aligned(h0, 16) ||
      !aligned(codes, 16) || !aligned(scales, 4))
    return MOE_ERR_ARG;
  if ((!grad_h0 && !out && !grad_row_weights) || !aligned(grad_h0, 16) || !aligned(out, 16) || !aligned(grad_row_weights, 4))
    return MOE_ERR_ARG;
  a.go = grad_out;
  a.h0 = h0;
  a.codes = const_cast<int8_t *>(codes);
  a.scales = const_cast<float *>(scales);
  a.gh0 = grad_h0;
  a.out = out;
  a.gw = grad_row_weights;
  return done(launch_swiglu_grad(a, (hipStream_t)stream));
}

int moe_combine_grad(const moe_get_shape_t *shape, const uint16_t *grad_out, const uint16_t *expert_out,
                     const int32_t *topk_idx, const float *topk_weights, const uint8_t *x_active_mask,
                     const int32_t *dst_row, const uint16_t *ori_x, const uint16_t *const_alpha1,
                     const uint16_t *const_alpha2, const uint16_t *const_v, uint16_t *grad_expert_out,
                     float *grad_topk_weights, uint16_t *grad_ori_x, float *grad_alpha1, float *grad_alpha2,
                     float *grad_v, void *stream) {
  const int st = moe_get_check_shape(shape);
  if (st != MOE_OK) return st;
  const int T = shape->num_tokens, C = shape->copy_expert_num, Kc = shape->const_expert_num;
  if (!grad_expert_out && !grad_topk_weights && !grad_ori_x && !grad_alpha1 && !grad_alpha2 && !grad_v)
    return MOE_ERR_ARG;
  if (Kc == 0 && (grad_alpha1 || grad_alpha2 || grad_v)) return MOE_ERR_ARG;
  if (!aligned(grad_alpha1, 4) || !aligned(grad_alpha2, 4) || !aligned(grad_v, 4) || !aligned(grad_topk_weights, 4))
    return MOE_ERR_ARG;
  if (T > 0) {
    if (!grad_out || !topk_idx || !topk_weights || !dst_row || !aligned(grad_out, 16)) return MOE_ERR_ARG;
    if (grad_topk_weights && (!expert_out || !aligned(expert_out, 16))) return MOE_ERR_ARG;
    if (!aligned(grad_expert_out, 16) || !aligned(grad_ori_x, 16)) return MOE_ERR_ARG;
    if (C + Kc > 0 && (!ori_x || !aligned(ori_x, 16))) return MOE_ERR_ARG;
  }
  if (Kc > 0 && (!const_alpha1 || !const_alpha2 || !const_v || !aligned(const_alpha1, 16) ||
                 !aligned(const_alpha2, 16) || !aligned(const_v, 16)))
    return MOE_ERR_ARG;
  CombineGradArgs a;
  memset(&a, 0, sizeof a);
  a.c.y = expert_out;
  a.c.topk_idx = topk_idx;
  a.c.w = topk_weights;
  a.c.mask = x_active_mask;
  a.c.dst_row = dst_row;
  a.c.ori_x = C + Kc > 0 ? ori_x : nullptr;
  a.c.a1 = const_alpha1;
  a.c.a2 = const_alpha2;
  a.c.cv = const_v;
  a.c.T = T;
  a.c.H = shape->hidden;
  a.c.K = shape->topk;
  a.c.E = shape->num_experts;
  a.c.Z = shape->zero_expert_num;
  a.c.C = C;
  a.c.Kc = Kc;
  a.go = grad_out;
  a.gy = grad_expert_out;
  a.gw = grad_topk_weights;
  a.gx = grad_ori_x;
  a.ga1 = grad_alpha1;
  a.ga2 = grad_alpha2;
  a.gv = grad_v;
  return done(launch_combine_grad(a, (hipStream_t)stream));
}

}  // extern "C"
