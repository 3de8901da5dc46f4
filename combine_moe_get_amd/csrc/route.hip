// route.hip -- the router's choice: the K best ids of each token and their weights.
#include "route_internal.hpp"

namespace moe {

// One wave a token, a lane NV consecutive ids.
template <int NV, int SCORE, bool F32, bool WIDE>
__global__ void __launch_bounds__(256) route_kernel(RouteArgs a) {
  using Key = typename std::conditional<WIDE, double, float>::type;
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= a.T) return;
  const int E = a.E, K = a.K;
  int id = -1;  // of slot `lane`
  float w = 0.0f;
  float l[NV];
  if (a.mask && !a.mask[t]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] = MOE_NEG_INF;
  } else {
    load_logits<NV, F32>(a.logits, t, E, lane, l);
  }
  const float m = row_max<NV>(l);
  if (m > MOE_NEG_INF) {
    Key key[NV];
    if constexpr (WIDE) {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        key[i] = SCORE == MOE_SCORE_SOFTMAX ? exp((double)l[i] - (double)m) : 1.0 / (1.0 + exp(-(double)l[i]));
        sum += key[i];
      }
      if (SCORE == MOE_SCORE_SOFTMAX) sum = wave_sum(sum);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = lane * NV + i;
        if (SCORE == MOE_SCORE_SOFTMAX) key[i] /= sum;
        bool ok = l[i] > MOE_NEG_INF;
        if (a.bias && e < E) {
          const float b = a.bias[e];
          ok = ok && b > MOE_NEG_INF;
          key[i] += (double)b;
        }
        if (!ok) key[i] = (double)MOE_NEG_INF;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) key[i] = l[i];
    }
    const Key none = (Key)MOE_NEG_INF;
    if (a.keep < a.G) {
      const int per = E / a.G;
      Key score = none;  // of group `lane`
      for (int g = 0; g < a.G; ++g) {
        Key one = none, two = none;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int e = lane * NV + i;
          const Key k = e >= g * per && e < (g + 1) * per ? key[i] : none;
          two = k > one ? one : k > two ? k : two;
          one = k > one ? k : one;
        }
        const Key first = wave_max(one);
        Key s = first;
        if (WIDE && a.two) {
          const uint64_t has = ballot(one == first);
          const Key second = wave_max((int)__builtin_ctzll(has) == lane ? two : one);
          if (second > none) s += second;
        }
        if (lane == g) score = s;
      }
      uint64_t kept = 0;
      for (int n = 0; n < a.keep; ++n) {
        const Key best = wave_max(score);
        if (!(best > none)) break;
        const int g = __builtin_ctzll(ballot(score == best));
        kept |= 1ull << g;
        if (lane == g) score = none;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = lane * NV + i;
        if (e >= E || !(kept >> (e / per) & 1)) key[i] = none;
      }
    }
    Key best;
    int at;
    auto look = [&]() {
      best = key[0];
      at = 0;
#pragma unroll
      for (int i = 1; i < NV; ++i)
        if (key[i] > best) {
          best = key[i];
          at = i;
        }
    };
    look();
    for (int j = 0; j < K; ++j) {
      const Key top = wave_max(best);
      if (!(top > none)) break;
      const int from = __builtin_ctzll(ballot(best == top));
      const int e = readlane(lane * NV + at, from);
      if (lane == j) id = e;
      if (lane == from) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (i == at) key[i] = none;
        look();
      }
    }
    const float lj = id >= 0 ? logit_at(a.logits, F32, t * E + id) : MOE_NEG_INF;
    if (a.renorm) {
      const float q = id < 0 ? MOE_NEG_INF : SCORE == MOE_SCORE_SOFTMAX ? lj : log_sigmoid(lj);
      const float mq = wave_max(q);
      w = id < 0 ? 0.0f : expf(q - mq);
      const float sum = wave_sum(w);
      w = id < 0 ? 0.0f : w / sum * a.scale;
    } else if constexpr (SCORE == MOE_SCORE_SOFTMAX) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) sum += expf(l[i] - m);
      sum = wave_sum(sum);
      w = id < 0 ? 0.0f : expf(lj - m) / sum * a.scale;
    } else {
      w = id < 0 ? 0.0f : 1.0f / (1.0f + expf(-lj)) * a.scale;
    }
  }
  if (lane < K) {
    a.idx[t * K + lane] = id;
    a.w[t * K + lane] = w;
  }
}

hipError_t launch_route(const RouteArgs &a, int score, bool fp32, hipStream_t st) {
  if (a.T == 0) return hipSuccess;
  const dim3 grid((unsigned)((a.T + 3) / 4)), block(256);
  const bool wide = a.bias || (a.two && a.keep < a.G);
  with_values(a.E, [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    auto go = [&](auto sc, auto f32, auto wd) {
      hipLaunchKernelGGL((route_kernel<NV, decltype(sc)::value, decltype(f32)::value, decltype(wd)::value>), grid, block, 0,
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
  });
  return hipGetLastError();
}

}  // namespace moe
