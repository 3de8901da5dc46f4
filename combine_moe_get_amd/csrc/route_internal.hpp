// route_internal.hpp -- argument blocks and launchers of the router (route.hip, balance.hip) shared with its entry
// points (route_api.hip), and the device code that both have in common: how a token's logits lie on the lanes of a wave.
#pragma once

#include <float.h>

#include "moe_internal.hpp"

namespace moe {

struct RouteArgs {
  const void *logits;
  const float *bias;
  const uint8_t *mask;
  int32_t *idx;
  float *w;
  int32_t T, E, K, G, keep;
  int32_t two, renorm;
  float scale;
  // set by the launcher: div_magic of the ids of a group; lanes that hold four each of them, if these are a power of two and
  // no more than a token has (else 0), and its logarithm
  uint32_t div_per;
  int32_t span, span_log;
};
hipError_t launch_route(const RouteArgs &a, int score, bool fp32, hipStream_t stream);

struct BalanceArgs {
  const void *logits;
  const int32_t *idx;
  const uint8_t *mask;
  float *losses;
  int32_t *counts;
  float *sums;
  int32_t *tokens;
  char *ws;
  int32_t T, E, K, S;
  float balance_coef, z_coef;
};
size_t balance_workspace(int T, int E, int S);
hipError_t launch_balance(const BalanceArgs &a, int score, bool fp32, hipStream_t stream);

struct RouteGradArgs {
  const void *logits;
  const int32_t *idx;
  const float *gw;
  const int32_t *dst;              // null: gw is [T, K]; else it is of `rows` receive rows, and this their map
  const uint8_t *mask;
  const int32_t *counts, *tokens;  // null: no losses
  const float *gl;
  void *out;
  int32_t T, E, K, S;
  int32_t renorm, rows;
  float scale, balance_coef, z_coef;
};
hipError_t launch_route_grad(const RouteGradArgs &a, int score, bool fp32, hipStream_t stream);

#define MOE_NEG_INF (-__builtin_inff())

// ---- a token on L lanes of a wave (16, 32 or 64), 64 / L tokens a wave --------------------------------
//
// A lane holds NV of its token's logits, four neighbouring ids at a time: value i is of id (i / 4 * L + lane) * 4 + i % 4.
// Sixteen lanes are a DPP row, whose folds need no LDS; what a wave does once it does for all its tokens, but few tokens
// leave the chip empty, and many values a lane take its registers.
template <int L, int NV>
struct Token {
  static constexpr int LANES = L, VALUES = NV;
};

// f(Token) for T tokens of E ids.  By lanes a token, us in graph replays (2.9 of them the launch):
//   the choice of 8 of 256,  4096 tokens   16: 5.0   32: 4.2   64: 4.9       65536 tokens   16: 25.8   32: 22.2   64: 35.3
//   the choice of 8 of 128,  4096 tokens   16: 4.3   32: 3.8                 16384 tokens   16: 5.0    32: 5.9
//   the choice of 8 of 512,  4096 tokens             32: 4.8   64: 5.3       65536 tokens              32: 46.7   64: 44.7
//   the gradient of 512,     4096 tokens             32: 11.2  64: 10.2
template <class F>
inline void with_token(int T, int E, F &&f) {
  if (E <= 64) f(Token<16, 4>{});
  else if (E <= 128 && T < 8192) f(Token<32, 4>{});
  else if (E <= 128) f(Token<16, 8>{});
  else if (E <= 256) f(Token<32, 8>{});
  else if (E <= 512) f(Token<64, 8>{});
  else if (E <= 1024) f(Token<64, 16>{});
  else f(Token<64, 32>{});
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false));
}
template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xf, 0xf, false);
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  return __hiloint2double(__builtin_amdgcn_update_dpp(0, __double2hiint(v), CTRL, 0xf, 0xf, false),
                          __builtin_amdgcn_update_dpp(0, __double2loint(v), CTRL, 0xf, 0xf, false));
}

// op over the L lanes of a token, to each of them, in a fixed order.  Every lane of the wave must call it.
template <int L, class V, class Op>
__device__ __forceinline__ V fold(V v, Op op) {
  v = op(v, dpp<0xb1>(v));   // quad_perm 1 0 3 2
  v = op(v, dpp<0x4e>(v));   // quad_perm 2 3 0 1
  v = op(v, dpp<0x141>(v));  // row_half_mirror
  v = op(v, dpp<0x140>(v));  // row_mirror
  if constexpr (L > 16) v = op(v, __shfl_xor(v, 16));
  if constexpr (L > 32) v = op(v, __shfl_xor(v, 32));
  return v;
}
template <int L>
__device__ __forceinline__ float max_of(float v) {
  return fold<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int L>
__device__ __forceinline__ double max_of(double v) {
  return fold<L>(v, [](double a, double b) { return fmax(a, b); });
}
template <int L, class V>
__device__ __forceinline__ V sum_of(V v) {
  return fold<L>(v, [](V a, V b) { return a + b; });
}

// bits of a token's lanes in a ballot
template <int L>
__device__ __forceinline__ uint64_t token_bits(uint64_t m) {
  return L == 64 ? m : (m >> (threadIdx.x & 63 & ~(L - 1))) & ((1ull << (L & 63)) - 1);
}

// LDS accesses of a wave are in order; this keeps the compiler to it
__device__ __forceinline__ void lds_order() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// a logit that counts: +inf as the largest finite value, NaN as -inf
__device__ __forceinline__ float usable(float l) { return l > MOE_NEG_INF ? fminf(l, FLT_MAX) : MOE_NEG_INF; }

__device__ __forceinline__ float logit_at(const void *logits, bool fp32, int64_t i) {
  return usable(fp32 ? ((const float *)logits)[i] : __uint_as_float((uint32_t)((const uint16_t *)logits)[i] << 16));
}

// the id of a lane's value i
template <int L>
__device__ __forceinline__ int id_of(int lane, int i) {
  return ((i >> 2) * L + lane) * 4 + (i & 3);
}

// The rows of the wave's tokens, t0 on, in a [T, E] array of elements of `size` bytes, as a buffer resource: what lies behind
// the last row is read as 0 and not written.  The check is of the vector offset with the instruction's, not of a scalar one,
// which stays 0.
template <int L>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t wave_rows(const void *p, int64_t t0, int T, int E, int size) {
  const int64_t left = T - t0;
  const int rows = left < 0 ? 0 : left < 64 / L ? (int)left : 64 / L;
  return __builtin_amdgcn_make_buffer_rsrc((char *)const_cast<void *>(p) + t0 * E * size, (short)0, rows * E * size, 0x00020000);
}
constexpr int kNowhere = 0x7ffffff0;  // an offset behind every such resource

// A lane's logits of its token; -inf where there is none (`on`: whether the token counts).  t0: the wave's first token, the
// same for all lanes.  Rows of a multiple of four ids are read four at a time, others one at a time: no branches either way.
template <int L, int NV, bool F32>
__device__ __forceinline__ void load_logits(const void *logits, int64_t t0, int T, int E, int lane, bool on, float *l) {
  constexpr int SIZE = F32 ? 4 : 2;
  const __amdgpu_buffer_rsrc_t rows = wave_rows<L>(logits, t0, T, E, SIZE);
  const int off = ((int)(threadIdx.x & 63) / L * E + lane * 4) * SIZE;
  if ((E & 3) == 0) {
#pragma unroll
    for (int c = 0; c < NV / 4; ++c) {
      if constexpr (F32) {
        const u32x4 x = __builtin_amdgcn_raw_buffer_load_b128(rows, off + c * L * 4 * SIZE, 0, 0);
#pragma unroll
        for (int k = 0; k < 4; ++k) l[c * 4 + k] = __uint_as_float(x[k]);
      } else {
        const u32x2 x = __builtin_amdgcn_raw_buffer_load_b64(rows, off + c * L * 4 * SIZE, 0, 0);
#pragma unroll
        for (int k = 0; k < 4; ++k) l[c * 4 + k] = k & 1 ? bf16_hi(x[k >> 1]) : bf16_lo(x[k >> 1]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = off + ((i >> 2) * L * 4 + (i & 3)) * SIZE;
      if constexpr (F32) l[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rows, at, 0, 0));
      else l[i] = __uint_as_float((uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rows, at, 0, 0) << 16);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) l[i] = usable(on && id_of<L>(lane, i) < E ? l[i] : MOE_NEG_INF);
}

template <int L, int NV>
__device__ __forceinline__ float row_max(const float *l) {
  float m = l[0];
#pragma unroll
  for (int i = 1; i < NV; ++i) m = fmaxf(m, l[i]);
  return max_of<L>(m);
}

// exp(x) for x <= 0 (below -200, -inf and NaN: 0), good to some two steps of fp32: 2^t of t = x log2(e) rounded, and the rest
// of the product as a factor
__device__ __forceinline__ float exp_neg(float x) {
  const float c = fmaxf(x, -200.0f);
  const float t = c * 1.44269502e+00f;
  const float r = __builtin_fmaf(c, 1.92596299e-8f, __builtin_fmaf(c, 1.44269502e+00f, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e * 0.693147182f, r, e);
}

// 1 / (1 + exp(-l)) and 1 minus it, for l that is not -inf or where neither is used
__device__ __forceinline__ float sigmoid(float l, float &rest) {
  const float e = exp_neg(-fabsf(l)), r = __builtin_amdgcn_rcpf(1.0f + e), er = e * r;
  rest = l > 0.0f ? er : r;
  return l > 0.0f ? r : er;
}

// The scores of some of a token's logits up to a common factor, s, and for sigmoids 1 - sigmoid, rest.  m: the largest of them.
// Softmax: exp(l - m).  Sigmoid: where no logit is above -60 divided by exp(m), so that they do not vanish.  s is 0 where
// there is no logit (also where there is none at all).
template <int NV, int SCORE>
__device__ __forceinline__ void scores(const float *l, float m, float *s, float *rest) {
  if constexpr (SCORE == MOE_SCORE_SOFTMAX) {
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] = exp_neg(l[i] - m);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] = sigmoid(l[i], rest[i]);
    if (ballot(m < -60.0f)) {
#pragma unroll
      for (int i = 0; i < NV; ++i) s[i] = m < -60.0f ? exp_neg(l[i] - m) : s[i];
    }
  }
}

}  // namespace moe
