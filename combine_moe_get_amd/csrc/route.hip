// route.hip -- the router's choice: the K best ids of each token and their weights.
#include "route_internal.hpp"

namespace moe {

// A key to compare by: in 64 bits, its last 11 replaced by the id, so that no two of a token's are the same and the lower id
// is the larger of two that were.  An fp32 logit keeps all its bits; a score keeps 42.
constexpr uint32_t kTag = 2047;
__device__ __forceinline__ double tagged(double key, int id) {
  const int hi = __double2hiint(key);
  const uint32_t tag = (uint32_t)id ^ (hi < 0 ? 0u : kTag);
  return __hiloint2double(hi, (int)(((uint32_t)__double2loint(key) & ~kTag) | tag));
}
__device__ __forceinline__ int id_in(double key) {
  return (int)(((uint32_t)__double2loint(key) & kTag) ^ (__double2hiint(key) < 0 ? 0u : kTag));
}
__device__ __forceinline__ double untagged(double key) {
  return __hiloint2double(__double2hiint(key), (int)((uint32_t)__double2loint(key) & ~kTag));
}

// the two best of (a, b) and (c, d), each pair in order
__device__ __forceinline__ void best_two(double &a, double &b, double c, double d) {
  const double low = fmin(a, c);
  a = fmax(a, c);
  b = fmax(low, fmax(b, d));
}

template <int L, int NV, int SCORE, bool F32, bool WIDE>
__device__ __forceinline__ void route_token(const RouteArgs &a, double *groups) {
  constexpr int PER = 64 / L;
  const int lane = threadIdx.x & (L - 1), sub = (threadIdx.x & 63) / L;  // of the token; the token of the wave
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = ((int64_t)blockIdx.x * 4 + wave) * PER + sub;
  const int E = a.E, K = a.K;
  const bool on = t < a.T && (!a.mask || a.mask[t]);
  const double none = (double)MOE_NEG_INF;
  float l[NV];
  load_logits<L, NV, F32>(a.logits, t, E, lane, on, l);
  float m = 0.0f;  // the largest logit
  if (WIDE || (SCORE == MOE_SCORE_SOFTMAX && !a.renorm)) m = row_max<L, NV>(l);

  double key[NV];
  if constexpr (WIDE) {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (SCORE == MOE_SCORE_SOFTMAX) {
        key[i] = l[i] > MOE_NEG_INF ? exp((double)l[i] - (double)m) : 0.0;
        sum += key[i];
      } else {
        key[i] = 1.0 / (1.0 + exp(-(double)l[i]));
      }
    }
    if (SCORE == MOE_SCORE_SOFTMAX) {
      sum = sum_of<L>(sum);
#pragma unroll
      for (int i = 0; i < NV; ++i) key[i] /= sum;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = id_of<L>(lane, i);
      bool ok = l[i] > MOE_NEG_INF;
      if (a.bias && e < E) {
        const float b = a.bias[e];
        ok = ok && b > MOE_NEG_INF;
        key[i] = fmin(key[i] + (double)b, DBL_MAX);
      }
      key[i] = ok ? tagged(key[i], e) : none;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      key[i] = l[i] > MOE_NEG_INF ? tagged((double)(l[i] + 0.0f), id_of<L>(lane, i)) : none;  // one zero
  }

  if (a.keep < a.G) {
    const int per = E / a.G;
    double *gs = groups + (wave * PER + sub) * 64;
    for (int g = 0; g < a.G; ++g) {
      double one = none, two = none;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const double k = (uint32_t)(id_of<L>(lane, i) - g * per) < (uint32_t)per ? key[i] : none;
        best_two(one, two, k, none);
      }
      if (a.two) {
        const double first = max_of<L>(one);
        const double second = max_of<L>(one == first ? two : one);
        one = first;
        if (second > none) one = tagged(fmin(untagged(first) + untagged(second), DBL_MAX), g);
      } else {
        one = max_of<L>(one);
      }
      if (lane == g % L) gs[g] = one;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    uint64_t kept = 0;
    for (int g0 = 0; g0 < a.G; g0 += L) {
      const int g = g0 + lane;
      const double mine = g < a.G ? gs[g] : none;
      int better = 0;
      for (int o = 0; o < a.G; ++o) better += gs[o] > mine;
      const uint64_t hit = ballot(mine > none && better < a.keep);
      kept |= (L == 64 ? hit : (hit >> (sub * L)) & ((1ull << (L & 63)) - 1)) << g0;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = id_of<L>(lane, i);
      if (!(kept >> (fast_div(e, a.div_per) & 63) & 1)) key[i] = none;
    }
  }

  // The lane's three best, in order; a round takes the best of all lanes.  A lane that gave all three looks for the next
  // ones below the last (of 16 lanes a few in a hundred do, for 8 of 256).
  double b0, b1, b2;
  auto look = [&](double below) {
    b0 = b1 = b2 = none;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      double k = key[i] < below ? key[i] : none;
      const double k1 = fmin(b0, k);
      b0 = fmax(b0, k);
      const double k2 = fmin(b1, k1);
      b1 = fmax(b1, k1);
      b2 = fmax(b2, k2);
    }
  };
  look((double)__builtin_inf());
  double mine = none;  // of slot `lane`
  int taken = 0;
  for (int j = 0; j < K; ++j) {
    const double top = max_of<L>(b0);
    if (lane == j) mine = top;
    const bool hit = b0 == top && top > none;
    if (hit) {
      b0 = b1;
      b1 = b2;
      b2 = none;
      ++taken;
    }
    if (ballot(hit && taken == 3)) {
      const bool empty = hit && taken == 3;
      const double o0 = b0, o1 = b1, o2 = b2;
      look(top);
      if (empty) {
        taken = 0;
      } else {
        b0 = o0;
        b1 = o1;
        b2 = o2;
      }
    }
  }
  const bool some = mine > none;
  const int id = some ? id_in(mine) : -1;
  float lj = WIDE ? (some ? logit_at(a.logits, F32, t * E + id) : 0.0f) : some ? (float)mine : 0.0f;  // the tag is far below its last bit
  float w;
  if (a.renorm) {
    const float q = !some ? MOE_NEG_INF : SCORE == MOE_SCORE_SOFTMAX ? lj : log_sigmoid(lj);
    const float mq = max_of<L>(q);
    w = some ? exp_neg(q - mq) : 0.0f;
    const float sum = sum_of<L>(w);
    w = some ? w / sum * a.scale : 0.0f;
  } else if constexpr (SCORE == MOE_SCORE_SOFTMAX) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) sum += l[i] > MOE_NEG_INF ? exp_neg(l[i] - m) : 0.0f;
    sum = sum_of<L>(sum);
    w = some ? exp_neg(lj - m) / sum * a.scale : 0.0f;
  } else {
    w = some ? 1.0f / (1.0f + expf(-lj)) * a.scale : 0.0f;
  }
  if (t < a.T && lane < K) {
    a.idx[t * K + lane] = id;
    a.w[t * K + lane] = w;
  }
}

template <int L, int NV, int SCORE, bool F32, bool WIDE>
__global__ void __launch_bounds__(256) route_kernel(RouteArgs a) {
  __shared__ double groups[4 * (64 / L) * 64];
  route_token<L, NV, SCORE, F32, WIDE>(a, groups);
}

template <int L, int NV>
static void launch_sized(const RouteArgs &a, int score, bool fp32, bool wide, hipStream_t st) {
  constexpr int TOKENS = 4 * (64 / L);  // a workgroup
  const dim3 grid((unsigned)((a.T + TOKENS - 1) / TOKENS)), block(256);
  auto go = [&](auto sc, auto f32, auto wd) {
    hipLaunchKernelGGL((route_kernel<L, NV, decltype(sc)::value, decltype(f32)::value, decltype(wd)::value>), grid, block, 0,
                       st, a);
  };
  auto types = [&](auto sc) {
    if (fp32 && wide) go(sc, std::true_type{}, std::true_type{});
    else if (fp32) go(sc, std::true_type{}, std::false_type{});
    else if (wide) go(sc, std::false_type{}, std::true_type{});
    else go(sc, std::false_type{}, std::false_type{});
  };
  if (score == MOE_SCORE_SOFTMAX) types(std::integral_constant<int, MOE_SCORE_SOFTMAX>{});
  else types(std::integral_constant<int, MOE_SCORE_SIGMOID>{});
}

hipError_t launch_route(const RouteArgs &a_, int score, bool fp32, hipStream_t st) {
  RouteArgs a = a_;
  if (a.T == 0) return hipSuccess;
  a.div_per = div_magic(a.E / a.G);
  const bool wide = a.bias || (a.two && a.keep < a.G);
  with_token(a.E, [&](auto tok) { launch_sized<decltype(tok)::LANES, decltype(tok)::VALUES>(a, score, fp32, wide, st); });
  return hipGetLastError();
}

}  // namespace moe
