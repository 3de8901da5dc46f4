// experts_internal.hpp -- argument blocks and launchers of the expert stage (experts.hip,
// rows_quant.hip, combine_grad.hip) shared with its entry points (experts_api.hip).
#pragma once

#include "moe_internal.hpp"

namespace moe {

// Where the rows of each expert lie (see "the expert stage" in moe_get.h).
struct RowGroups {
  const int32_t *off;    // [E + 1]
  int64_t rows, stride;  // rows of the buffers; window length (0: compact)
  int32_t E, L;          // experts, experts per rank
};

// rows [lo, lo + n) of expert e, cut to its window and to the buffer whatever the offsets hold
__device__ __forceinline__ void expert_rows(const RowGroups &g, int e, int64_t &lo, int &n) {
  const int64_t a = g.off[e], b = g.off[e + 1];
  int64_t first = 0, end = g.rows, at = a;
  if (g.stride > 0) {
    const int r = e / g.L;
    first = (int64_t)r * g.stride;
    if (first + g.stride < end) end = first + g.stride;
    at = first + a - g.off[r * g.L];
  }
  at = at < first ? first : at > end ? end : at;
  int64_t c = b - a;
  c = c < 0 ? 0 : c > end - at ? end - at : c;
  lo = at;
  n = (int)c;
}

enum ExpertsOp : int {
  OP_FORWARD = MOE_EXPERTS_FORWARD,
  OP_DGRAD = MOE_EXPERTS_DGRAD,
  OP_WGRAD = MOE_EXPERTS_WGRAD
};

struct ExpertsArgs {
  RowGroups g;
  const void *m;         // operand whose index runs over the result's rows: x, grad_out (dgrad, wgrad)
  const void *n;         // operand whose index runs over its columns: w, w (dgrad), x (wgrad)
  const void *ms, *ns;   // scales of their rows (forward) or null
  void *out;
  int32_t K;             // contraction: in_features (forward), out_features (dgrad), none (wgrad)
  int32_t M;             // wgrad: rows of a result (out_features)
  int32_t N;             // columns of the result
};

// The tile that a product runs on; wide: MXFP4 scales of a row begin at multiples of four bytes (else true).
struct ExpertsTile {
  int32_t rows, columns, stages;
};
ExpertsTile experts_tile(const ExpertsArgs &a, int op, int row_type, bool gated, bool wide);

// MXFP4: whether every row of scales begins at a multiple of four bytes
inline bool mx_scales_wide(int K, const void *ms, const void *ns) {
  return K % 128 == 0 && (((uintptr_t)ms | (uintptr_t)ns) & 3) == 0;
}

hipError_t launch_experts(const ExpertsArgs &a, int op, int row_type, int act, bool out_fp32, hipStream_t stream);

struct RowsQuantArgs {
  RowGroups g;           // off null: every row
  const uint16_t *x;
  void *codes, *scales;
  int64_t rows;
  int32_t H;
};
hipError_t launch_rows_quant(const RowsQuantArgs &a, int row_type, hipStream_t stream);

struct CombineGradArgs {
  CombineArgs c;         // the combine's inputs (out unused)
  const uint16_t *go;
  uint16_t *gy;
  float *gw;
  uint16_t *gx;
  float *ga1, *ga2, *gv;
  int32_t vectors;       // workgroups for those three (set by the launcher)
};
hipError_t launch_combine_grad(const CombineGradArgs &a, hipStream_t stream);

}  // namespace moe
