// route.hip -- the router's choice: the K best ids of each token and their weights.
//
// s = softmax(l) or 1 / (1 + exp(-l)); key = s + bias, or l, which has the order of s; the topk_groups best groups by their best
// key or two; of their ids the K best keys, ties to the lowest; w_j = scale s_j, or s_j / sum s.
// A score in 32 bits does not tell all keys of a batch apart, and its rounding would choose; 64 bits for all ids take 9.0 us for
// 7.0 (4096 tokens of 256, sigmoids with a bias, four of eight groups) and 68 for 49 (65536).  So keys in 32 bits, known to
// within some 2^-21, pick candidates: the K-th largest of the lanes' largest is a bound that at least K ids reach, and only some
// 9 of 256 do (K = 8).  Each of those is computed in 64 bits by a lane of its own and compared with the others, at once and not
// in rounds of one best after the other.  Groups whose 32-bit scores are too near at the border, and rows of so many equal values
// that the candidates do not fit, go a longer way in 64 bits.
// Many tokens are bound by instructions (with a bias and the groups' two best 937 a wave of two tokens: vector instructions in 80% of
// the cycles at 16384 tokens, in all at 65536; with groups alone 538, 71%), up to some 4000 by the launch and by the chain of folds,
// LDS and 64-bit steps of the one wave that a SIMD has (44% with the bias at 4096): 16384 tokens of 256 fp32 logits 7.4 us (17 MB;
// at a copy's rate 3.3, and 2.9 for the launch), with four of eight groups 9.5, sigmoids with a bias and the groups' two best 18;
// 128 tokens 3.8, 4.7, 6.2.  By rounds, in 64 bits: 16384 tokens with groups 30 us on a wave a token, 13 on 16 lanes.
// How many go the longer way depends on the logits, since the error of a key in 32 bits is known as 2^-21 + 2^-23 of it: scores
// below some 1e-6 look alike unless a bias sets them apart.  16384 tokens of 256, us, for softmax logits of deviation 1 / 5 / 10 / 15
// and sigmoids around 0 / -8 / -12 / -16:
//   groups by two, no bias      12 / 13 / 17 / 19     11 / 14 / 19 / 20
//   a bias of zeros             16 / 24 / 37 / 45     12 / 12 / 12 / 43
//   both                        22 / 38 / 64 / 69     15 / 18 / 24 / 69
//   a bias of deviation 0.1     18 / 18 / 18 / 18     17 / 15 / 15 / 15
#include "route_internal.hpp"

namespace moe {

// A logit to compare by, its id in the last 11 bits of a double: no two of a token's are the same, and the lower id is the
// larger of two that were.  An fp32 value leaves 29 bits free.
constexpr uint32_t kTag = 2047;
__device__ __forceinline__ double tagged(float logit, int id) {
  const double key = (double)(logit + 0.0f);  // one zero
  const int hi = __double2hiint(key);
  return __hiloint2double(hi, __double2loint(key) | (int)((uint32_t)id ^ (hi < 0 ? 0u : kTag)));
}
__device__ __forceinline__ int id_in(double key) {
  return (int)(((uint32_t)__double2loint(key) & kTag) ^ (__double2hiint(key) < 0 ? 0u : kTag));
}

// the two best of (a, b) and (c, d), each pair in order
template <class V>
__device__ __forceinline__ void best_two(V &a, V &b, V c, V d) {
  const V low = a > c ? c : a;
  a = a > c ? a : c;
  const V next = b > d ? b : d;
  b = low > next ? low : next;
}

// For each of a token's groups put(its best value, its second best, the group), on one lane; value(i): of the lane's i-th id,
// none where it is not available.  Without a.two the second is not looked for.
template <int L, int NV, class V, class Value, class Put>
__device__ __forceinline__ void group_best(const RouteArgs &a, int lane, V none, Value value, Put put) {
  if (a.span) {  // a group is `span` neighbouring lanes' four values: all groups of a round at once
#pragma unroll
    for (int c = 0; c < NV / 4; ++c) {
      V one = none, two = none;
#pragma unroll
      for (int k = 0; k < 4; ++k) best_two(one, two, value(c * 4 + k), none);
      auto step = [&](auto move) {
        const V other = move(one);
        if (a.two) best_two(one, two, other, move(two));
        else one = one > other ? one : other;
      };
      if (a.span > 1) step([](V x) { return dpp<0xb1>(x); });
      if (a.span > 2) step([](V x) { return dpp<0x4e>(x); });
      if (a.span > 4) step([](V x) { return dpp<0x141>(x); });
      if (a.span > 8) step([](V x) { return dpp<0x140>(x); });
      if (L > 16 && a.span > 16) step([](V x) { return __shfl_xor(x, 16); });
      if (L > 32 && a.span > 32) step([](V x) { return __shfl_xor(x, 32); });
      const int at = c * L + lane, g = at >> a.span_log;
      if ((at & (a.span - 1)) == 0 && g < a.G) put(one, two, g);
    }
  } else {
    const int per = a.E / a.G;
    for (int g = 0; g < a.G; ++g) {
      V one = none, two = none;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        best_two(one, two, (uint32_t)(id_of<L>(lane, i) - g * per) < (uint32_t)per ? value(i) : none, none);
      const V first = max_of<L>(one);
      // of the lanes that have the best one, one gives it up
      const int has = __builtin_ctzll(ballot(one == first) >> (threadIdx.x & 63 & ~(L - 1)));
      const V second = a.two ? max_of<L>(lane == has ? two : one) : none;
      if (lane == g % L) put(first, second, g);
    }
  }
}

// LDS of a token: up to 4 L candidates (before them the groups' scores), its K results
template <int L>
struct RouteLds {
  static constexpr int CANDIDATES = 4 * L;
  __align__(16) double cand[CANDIDATES + 4];
  __align__(16) int ids[CANDIDATES + 4];
  double best[16];
};

// The groups that a token's ids may come from (bit g), by scores in 64 bits: value(i) as in group_best.
template <int L, int NV, class Value>
__device__ __forceinline__ uint64_t groups_wide(const RouteArgs &a, int lane, double *gs, Value value) {
  const double none = (double)MOE_NEG_INF;
  group_best<L, NV>(a, lane, none, value, [&](double one, double two, int g) {
    gs[g] = a.two && two > none ? fmin(one + two, DBL_MAX) : one;
  });
  lds_order();
  uint64_t kept = 0;
  for (int g0 = 0; g0 < a.G; g0 += L) {
    const int g = g0 + lane;
    const double mine = g < a.G ? gs[g] : none;
    int better = 0;
    for (int o = 0; o < a.G; ++o) better += gs[o] > mine || (gs[o] == mine && o < g);
    kept |= token_bits<L>(ballot(mine > none && better < a.keep)) << g0;
  }
  lds_order();
  return kept;
}

// The best K by rounds, each the best of what comes behind the last round's: the id of slot j on lane j, or -1.  key(i): in 64
// bits, of the lane's i-th id.
template <int L, int NV, class Key>
__device__ __forceinline__ int choose_by_rounds(int K, int lane, Key key) {
  const double none = (double)MOE_NEG_INF;
  double last = (double)__builtin_inf();
  int last_id = -1, mine = -1;
  for (int j = 0; j < K; ++j) {
    double best = none;
    int id = 1 << 30;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const double k = key(i);
      const int e = id_of<L>(lane, i);
      if ((k < last || (k == last && e > last_id)) && (k > best || (k == best && e < id))) {
        best = k;
        id = e;
      }
    }
    last = max_of<L>(best);
    last_id = fold<L>(best == last ? id : 1 << 30, [](int x, int y) { return x < y ? x : y; });
    if (lane == j && last > none) mine = last_id;
  }
  return mine;
}

// L lanes a token, NV logits a lane.
template <int L, int NV, int SCORE, bool F32, bool BIAS>
__global__ void __launch_bounds__(256) route_kernel(RouteArgs a) {
  constexpr int PER = 64 / L;
  __shared__ RouteLds<L> lds[4 * PER];
  const int lane = threadIdx.x & (L - 1);
  RouteLds<L> &my = lds[threadIdx.x / L];
  const int64_t t0 = (int64_t)blockIdx.x * (4 * PER) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * PER;  // the wave's first
  const int64_t t = t0 + (threadIdx.x & 63) / L;
  const int E = a.E, K = a.K;
  const bool on = t < a.T && (!a.mask || a.mask[t]), grouped = a.keep < a.G;
  const double none = (double)MOE_NEG_INF;
  const float nonef = MOE_NEG_INF;
  float l[NV];
  load_logits<L, NV, F32>(a.logits, t0, a.T, E, lane, on, l);

  // What the formulas of softmax need of the whole row: its largest logit, the sum of exponentials.
  float m = 0.0f, sum = 1.0f;
  double whole = 1.0;
  if (SCORE == MOE_SCORE_SOFTMAX && (BIAS || (grouped && a.two) || !a.renorm)) m = row_max<L, NV>(l);
  if (SCORE == MOE_SCORE_SOFTMAX && !a.renorm) {
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) sum += exp_neg(l[i] - m);
    sum = sum_of<L>(sum);
  }
  if (SCORE == MOE_SCORE_SOFTMAX && BIAS) {
    whole = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) whole += l[i] > nonef ? exp((double)l[i] - (double)m) : 0.0;
    whole = 1.0 / sum_of<L>(whole);
  }

  // Scores and keys (a logit; with a bias a score and it) in 64 bits.
  auto score = [&](float v) -> double {
    return SCORE == MOE_SCORE_SOFTMAX ? exp((double)v - (double)m) * whole : 1.0 / (1.0 + exp(-(double)v));
  };
  auto key_of = [&](float v, int id) -> double {
    if (!(v > nonef)) return none;
    if (!BIAS) return tagged(v, id);
    const float b = a.bias[id];
    return b > nonef ? fmin(score(v) + (double)b, DBL_MAX) : none;
  };

  // Keys in 32 bits: logits as they are; scores, at most 1, are good to 2^-22, and with a bias the sum to 2^-24 of itself.
  auto err = [](float v) { return __builtin_fmaf(fabsf(v), 0x1p-23f, 0x1p-21f); };
  float k[NV];
  if constexpr (BIAS) {
    float rest[NV];
    if (SCORE == MOE_SCORE_SOFTMAX) scores<NV, SCORE>(l, m, k, rest);
    else
#pragma unroll
      for (int i = 0; i < NV; ++i) k[i] = sigmoid(l[i], rest[i]);
    const float f = (float)whole;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int id = id_of<L>(lane, i);
      const float b = id < E ? a.bias[id] : nonef;
      k[i] = l[i] > nonef && b > nonef ? fminf(__builtin_fmaf(k[i], f, b), FLT_MAX) : nonef;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) k[i] = l[i];
  }
  if (grouped) {
    float *gs = (float *)my.cand;  // what a group's score is at least; 64 on, at most
    const bool exact = !BIAS && !a.two;
    auto bounds = [&](float one, float two, int g) {
      const bool both = a.two && two > nonef;
      const float s = both ? fminf(one + two, FLT_MAX) : one;
      const float e = exact ? 0.0f : both ? err(one) + err(two) + fabsf(s) * 0x1p-23f : err(one);
      gs[g] = one > nonef ? s - e : nonef;
      gs[64 + g] = one > nonef ? s + e : nonef;
    };
    if (!BIAS && a.two) {
      float s[NV], rest[NV];
      if (SCORE == MOE_SCORE_SOFTMAX) scores<NV, SCORE>(l, m, s, rest);
      else
#pragma unroll
        for (int i = 0; i < NV; ++i) s[i] = sigmoid(l[i], rest[i]);
      group_best<L, NV>(a, lane, nonef, [&](int i) { return l[i] > nonef ? s[i] : nonef; }, bounds);
    } else {
      group_best<L, NV>(a, lane, nonef, [&](int i) { return k[i]; }, bounds);
    }
    lds_order();
    uint64_t kept = 0;
    bool open = false;
    for (int g0 = 0; g0 < a.G; g0 += L) {
      const int g = g0 + lane;
      const float least = g < a.G ? gs[g] : nonef, most = g < a.G ? gs[64 + g] : nonef;
      const bool some = most > nonef;
      int above = 0, near = -1;
      bool in;
      if (exact) {
#pragma unroll 4
        for (int o = 0; o < a.G; ++o) above += (int)(gs[o] > most) | ((int)(gs[o] == most) & (int)(o < g));
        in = some && above < a.keep;
      } else {
#pragma unroll 4
        for (int o = 0; o < a.G; ++o) {
          above += gs[o] > most;
          near += gs[64 + o] >= least;
        }
        in = some && near < a.keep;
        open = open || (some && !in && above < a.keep);
      }
      kept |= token_bits<L>(ballot(in)) << g0;
    }
    lds_order();
    if (ballot(open))  // two groups too near one another at the border: few tokens while scores are far above 2^-21
      kept = groups_wide<L, NV>(a, lane, my.cand, [&](int i) {
        const int id = id_of<L>(lane, i);
        return BIAS ? key_of(l[i], id) : l[i] > nonef ? score(l[i]) : none;
      });
    if (a.span) {
#pragma unroll
      for (int c = 0; c < NV / 4; ++c) {
        const bool in = kept >> ((c * L + lane) >> a.span_log & 63) & 1;
#pragma unroll
        for (int i = c * 4; i < c * 4 + 4; ++i) {
          l[i] = in ? l[i] : nonef;
          k[i] = in ? k[i] : nonef;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (!(kept >> (fast_div(id_of<L>(lane, i), a.div_per) & 63) & 1)) l[i] = k[i] = nonef;
    }
  }

  // The K-th largest of the lanes' largest is a bound that at least K keys reach; the few that reach it are compared with one
  // another, each by a lane of its own.
  float top = nonef;
#pragma unroll
  for (int i = 0; i < NV; ++i) top = fmaxf(top, k[i]);
  if (BIAS) top -= err(top);
  float *tops = (float *)my.cand;
  tops[lane] = top;
  if (lane < 16) my.best[lane] = none;
  lds_order();
  int rank = 0;
#pragma unroll
  for (int o = 0; o < L; o += 4) {
    const f32x4 v = *(const f32x4 *)(tops + o);
    rank += (v[0] > top) + (v[1] > top) + (v[2] > top) + (v[3] > top);
  }
  lds_order();
  float bound = fold<L>(rank < K ? top : __builtin_inff(), [](float x, float y) { return fminf(x, y); });
  if (BIAS) bound -= 2.0f * err(bound);  // of a key that reaches it, and of the subtraction
  bound = fmaxf(bound, -FLT_MAX);
  int n = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) n += k[i] >= bound;
  const int upto = wave_inclusive_sum(n);  // over the wave
  const int first = threadIdx.x & 63 & ~(L - 1), last = __shfl(upto, (first - 1) & 63);
  const int before = first ? last : 0;  // in the wave's other tokens
  int at = upto - n - before;
  n = __shfl(upto, L - 1, L) - before;
  int id = -1;  // of slot `lane`
  float lj = 0.0f;
  if (ballot(n > RouteLds<L>::CANDIDATES)) {  // rows of one value, or nearly
    id = choose_by_rounds<L, NV>(K, lane, [&](int i) { return key_of(l[i], id_of<L>(lane, i)); });
    if (id >= 0) lj = logit_at(a.logits, F32, t * E + id);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (k[i] >= bound) my.cand[at++] = __hiloint2double(__float_as_int(l[i]), id_of<L>(lane, i));
    lds_order();
    for (int c = lane; ballot(c < n); c += L)
      if (c < n) {
        const int e = __double2loint(my.cand[c]);
        my.cand[c] = key_of(__int_as_float(__double2hiint(my.cand[c])), e);
        if (BIAS) my.ids[c] = e;
      }
    if (lane < 4) my.cand[n + lane] = none;
    lds_order();
    for (int c = lane; ballot(c < n); c += L) {
      const double key = c < n ? my.cand[c] : none;
      const int e = BIAS && c < n ? my.ids[c] : 0;  // without a bias no two keys are the same, and no id is below 0
      int r = 0;
      for (int o = 0; o < n; o += 4) {  // four at once, without branches
        typedef double f64x2 __attribute__((ext_vector_type(2)));
        typedef int i32x4 __attribute__((ext_vector_type(4)));
        const f64x2 x = *(const f64x2 *)(my.cand + o), y = *(const f64x2 *)(my.cand + o + 2);
        i32x4 id4 = {0, 0, 0, 0};
        if (BIAS) id4 = *(const i32x4 *)(my.ids + o);
        r += (int)(x[0] > key) | ((int)(x[0] == key) & (int)(id4[0] < e));
        r += (int)(x[1] > key) | ((int)(x[1] == key) & (int)(id4[1] < e));
        r += (int)(y[0] > key) | ((int)(y[0] == key) & (int)(id4[2] < e));
        r += (int)(y[1] > key) | ((int)(y[1] == key) & (int)(id4[3] < e));
      }
      if (key > none && r < K) my.best[r] = BIAS ? (double)e : key;
    }
    lds_order();
    const double best = lane < K ? my.best[lane] : none;
    if (best > none) {
      id = BIAS ? (int)best : id_in(best);
      lj = BIAS ? logit_at(a.logits, F32, t * E + id) : (float)best;  // the tag is far below the last bit of 32
    }
  }
  const bool some = id >= 0;

  float w, rest;
  if (a.renorm) {
    const float lw = some ? lj : nonef;
    scores<1, SCORE>(&lw, max_of<L>(lw), &w, &rest);
    w = some ? w : 0.0f;
    const float all = sum_of<L>(w);
    w = some ? w / all : 0.0f;
  } else {
    w = SCORE == MOE_SCORE_SOFTMAX ? exp_neg(lj - m) / sum : sigmoid(lj, rest);
    w = some ? w : 0.0f;
  }
  w *= a.scale;
  if (t < a.T && lane < K) {
    a.idx[t * K + lane] = id;
    a.w[t * K + lane] = w;
  }
}

template <int L, int NV>
static void launch_sized(const RouteArgs &a_, int score, bool fp32, hipStream_t st) {
  constexpr int TOKENS = 4 * (64 / L);  // a workgroup
  RouteArgs a = a_;
  const int per = a.E / a.G, quads = per / 4;
  a.span = per % 4 == 0 && (quads & (quads - 1)) == 0 && quads <= L ? quads : 0;
  a.span_log = a.span ? __builtin_ctz(a.span) : 0;
  const dim3 grid((unsigned)((a.T + TOKENS - 1) / TOKENS)), block(256);
  auto go = [&](auto sc, auto f32, auto bias) {
    hipLaunchKernelGGL((route_kernel<L, NV, decltype(sc)::value, decltype(f32)::value, decltype(bias)::value>), grid, block, 0,
                       st, a);
  };
  auto types = [&](auto sc) {
    if (fp32 && a.bias) go(sc, std::true_type{}, std::true_type{});
    else if (fp32) go(sc, std::true_type{}, std::false_type{});
    else if (a.bias) go(sc, std::false_type{}, std::true_type{});
    else go(sc, std::false_type{}, std::false_type{});
  };
  if (score == MOE_SCORE_SOFTMAX) types(std::integral_constant<int, MOE_SCORE_SOFTMAX>{});
  else types(std::integral_constant<int, MOE_SCORE_SIGMOID>{});
}

hipError_t launch_route(const RouteArgs &a_, int score, bool fp32, hipStream_t st) {
  RouteArgs a = a_;
  if (a.T == 0) return hipSuccess;
  a.div_per = div_magic(a.E / a.G);
  with_token(a.T, a.E, [&](auto tok) { launch_sized<decltype(tok)::LANES, decltype(tok)::VALUES>(a, score, fp32, st); });
  return hipGetLastError();
}

}  // namespace moe
