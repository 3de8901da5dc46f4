// route_internal.hpp -- argument blocks and launchers of the router (route.hip, balance.hip) shared with its entry
// points (route_api.hip), and the device code that both have in common: a wave of 64 lanes holds one token's logits.
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
  const int32_t *dst;              // null: gw is [T, K]; else it is of receive rows, and this their map
  const uint8_t *mask;
  const int32_t *counts, *tokens;  // null: no losses
  const float *gl;
  void *out;
  int32_t T, E, K, S;
  int32_t renorm;
  float scale, balance_coef, z_coef;
};
hipError_t launch_route_grad(const RouteGradArgs &a, int score, bool fp32, hipStream_t stream);

#define MOE_NEG_INF (-__builtin_inff())

// a DPP move of a value of 4 or 8 bytes; lanes without a source take `old`
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float dpp(float old, float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(v), CTRL, ROW_MASK, 0xf, false));
}
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ double dpp(double old, double v) {
  const int lo = __builtin_amdgcn_update_dpp(__double2loint(old), __double2loint(v), CTRL, ROW_MASK, 0xf, false);
  const int hi = __builtin_amdgcn_update_dpp(__double2hiint(old), __double2hiint(v), CTRL, ROW_MASK, 0xf, false);
  return __hiloint2double(hi, lo);
}
__device__ __forceinline__ float lane_value(float v, int lane) { return readlane_f(v, lane); }
__device__ __forceinline__ double lane_value(double v, int lane) {
  return __hiloint2double(readlane(__double2hiint(v), lane), readlane(__double2loint(v), lane));
}

// max and sum over the 64 lanes, to every lane (see wave_max, wave_inclusive_sum); in a fixed order
__device__ __forceinline__ double wave_max(double v) {
  v = fmax(v, dpp<0x111, 0xf>(v, v));
  v = fmax(v, dpp<0x112, 0xf>(v, v));
  v = fmax(v, dpp<0x114, 0xf>(v, v));
  v = fmax(v, dpp<0x118, 0xf>(v, v));
  v = fmax(v, dpp<0x142, 0xa>(v, v));
  v = fmax(v, dpp<0x143, 0xc>(v, v));
  return lane_value(v, 63);
}
template <class F>
__device__ __forceinline__ F wave_sum(F v) {
  v += dpp<0x111, 0xf>(F(0), v);
  v += dpp<0x112, 0xf>(F(0), v);
  v += dpp<0x114, 0xf>(F(0), v);
  v += dpp<0x118, 0xf>(F(0), v);
  v += dpp<0x142, 0xa>(F(0), v);
  v += dpp<0x143, 0xc>(F(0), v);
  return lane_value(v, 63);
}

// a logit that counts: +inf as the largest finite value, NaN as -inf
__device__ __forceinline__ float usable(float l) { return l > MOE_NEG_INF ? fminf(l, FLT_MAX) : MOE_NEG_INF; }

__device__ __forceinline__ float logit_at(const void *logits, bool fp32, int64_t i) {
  return usable(fp32 ? ((const float *)logits)[i] : __uint_as_float((uint32_t)((const uint16_t *)logits)[i] << 16));
}

// a lane's NV consecutive logits lane * NV, .. of the token's E; -inf behind the last.  Wide loads where rows begin at
// multiples of NV.
template <int NV, bool F32>
__device__ __forceinline__ void load_logits(const void *logits, int64_t t, int E, int lane, float *l) {
  const int e0 = lane * NV;
  if (E % NV == 0) {
    if (e0 < E) {
      if constexpr (F32) {
        constexpr int B = NV < 4 ? NV : 4;
        typedef float vec __attribute__((ext_vector_type(B)));
        const float *p = (const float *)logits + t * E + e0;
#pragma unroll
        for (int i = 0; i < NV; i += B) {
          if constexpr (B == 1) l[i] = p[i];
          else {
            const vec v = *(const vec *)(p + i);
#pragma unroll
            for (int k = 0; k < B; ++k) l[i + k] = v[k];
          }
        }
      } else {
        constexpr int B = NV < 8 ? NV : 8;
        typedef uint16_t vec __attribute__((ext_vector_type(B)));
        const uint16_t *p = (const uint16_t *)logits + t * E + e0;
#pragma unroll
        for (int i = 0; i < NV; i += B) {
          if constexpr (B == 1) l[i] = __uint_as_float((uint32_t)p[i] << 16);
          else {
            const vec v = *(const vec *)(p + i);
#pragma unroll
            for (int k = 0; k < B; ++k) l[i + k] = __uint_as_float((uint32_t)v[k] << 16);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) l[i] = usable(l[i]);
      return;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] = MOE_NEG_INF;
    return;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) l[i] = e0 + i < E ? logit_at(logits, F32, t * E + e0 + i) : MOE_NEG_INF;
}

// the largest of a token's logits, to every lane
template <int NV>
__device__ __forceinline__ float row_max(const float *l) {
  float m = l[0];
#pragma unroll
  for (int i = 1; i < NV; ++i) m = fmaxf(m, l[i]);
  return wave_max(m);
}

// p = scores of the logits divided by their sum, for a token with a logit; m: the largest logit.  Softmax: exp(l - m).
// Sigmoid: exp(min(l, 0)) / (1 + exp(-|l|)); where all of them are small, both divided by exp(m), so that none vanishes.
template <int NV, int SCORE>
__device__ __forceinline__ void probabilities(const float *l, float m, float *p) {
  float sum = 0.0f;
  const float shift = SCORE == MOE_SCORE_SOFTMAX ? m : fminf(m, 0.0f);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if constexpr (SCORE == MOE_SCORE_SOFTMAX) p[i] = expf(l[i] - shift);
    else p[i] = expf(fminf(l[i], 0.0f) - shift) / (1.0f + expf(-fabsf(l[i])));
    if (!(l[i] > MOE_NEG_INF)) p[i] = 0.0f;
    sum += p[i];
  }
  const float r = 1.0f / wave_sum(sum);
#pragma unroll
  for (int i = 0; i < NV; ++i) p[i] *= r;
}

// the logarithm of a sigmoid
__device__ __forceinline__ float log_sigmoid(float l) { return fminf(l, 0.0f) - log1pf(expf(-fabsf(l))); }

// kernels are built for rows of up to 64 NV logits: f(NV) for the least NV that holds E
template <class F>
inline void with_values(int E, F &&f) {
  if (E <= 64) f(std::integral_constant<int, 1>{});
  else if (E <= 128) f(std::integral_constant<int, 2>{});
  else if (E <= 256) f(std::integral_constant<int, 4>{});
  else if (E <= 512) f(std::integral_constant<int, 8>{});
  else if (E <= 1024) f(std::integral_constant<int, 16>{});
  else f(std::integral_constant<int, 32>{});
}

}  // namespace moe
