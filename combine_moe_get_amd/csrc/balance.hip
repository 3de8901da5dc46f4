// balance.hip -- the router's balance losses, and the gradient of its logits.
//
// p = s / sum s; per segment c_e = slots that hold e, P_e = sum_t p_te, T_g live tokens:
//   balance = coef / S sum_g E / (K T_g^2) sum_e c_e P_e,   z = z_coef / T sum_t lse_t^2,
// and back: dbalance / dp_te = A_e = coef E c_e / (S K T_g^2), so of log s it is p_e (A_e - sum_f A_f p_f); through the weights
// a_j (see moe_route_grad); of l: the same for softmax, times 1 - s_e for sigmoids; z adds 2 z_coef lse / T softmax(l).
// Both read the logits once.  The gradient is bound by instructions (two exponentials or an exponential and a reciprocal an id:
// vector instructions in 79% of the cycles at 16384 tokens of 256, 97 at 65536), the sums by how few tokens are under way (44%, 75%)
// and, below some 4000 tokens, both by launches: 16384 tokens of 256 in 64 segments, sigmoids: sums 10.3 us (17 MB), losses 5.0,
// gradient 13.5 (34 MB; 6.7 at a copy's rate); 4096 of 64 in bf16: 4.7, 5.3, 4.7.
// Where a reciprocal is the instruction's (of a sum of scores, of a segment's tokens, in the sigmoid) it is good to one step of fp32,
// 2^-23: sigmoids to 2.1 steps, their p to 3.1 of 2048 ids, those of softmax to 3 and half a step for each 1 that the logit is below
// the largest (measured).  The weights' sum is divided by, as in the choice: there a remnant of 1 - w would stand for 0.
#include "route_internal.hpp"

namespace moe {

// ---- the losses ----------------------------------------------------------------------------------

constexpr int kSumGroups = 1024;  // workgroups for the sums, at most: half as many are as fast (17.9 us for 18.4 on 16384 x 256)

// As with_token: here all four tokens of a wave pay at any number (4096 of 256 ids: 12.2 us on 16 lanes, 13.6 on 32).
template <class F>
static void with_sums_token(int E, F &&f) {
  if (E <= 64) f(Token<16, 4>{});
  else if (E <= 128) f(Token<16, 8>{});
  else if (E <= 256) f(Token<16, 16>{});
  else if (E <= 512) f(Token<32, 16>{});
  else if (E <= 1024) f(Token<64, 16>{});
  else f(Token<64, 32>{});
}

// Workgroups that share a segment's tokens: twice as many tokens each as it takes at a time, up to kSumGroups in all; more
// where a lane would add more than 64 tokens in fp32.
static int slices(int T, int E, int S) {
  int tokens = 0;
  with_sums_token(E, [&](auto tok) { tokens = 4 * (64 / decltype(tok)::LANES); });
  const int n = T / S, most = (n + 2 * tokens - 1) / (2 * tokens), want = (kSumGroups + S - 1) / S;
  const int least = (n + 64 * tokens - 1) / (64 * tokens), some = most < want ? most : want;
  const int L = some > least ? some : least;
  return L < 1 ? 1 : L;
}

// workspace: a counter (16 bytes); per slice the sum of squares of log sum exp (double), then live tokens (int32), then of
// each column the sum of p (float) and the slots (int32); per workgroup of the second kernel a part of the loss (double)
struct BalanceSpace {
  uint32_t *counter;
  double *z, *part;
  int32_t *live, *cnt;
  float *sum;
  size_t bytes;
};
static __host__ __device__ BalanceSpace balance_space(char *ws, int L, int E, int S) {
  BalanceSpace b;
  const size_t n = (size_t)S * L, parts = (size_t)S * ((E + 63) / 64);
  size_t at = 16;
  b.counter = (uint32_t *)ws;
  b.z = (double *)(ws + at);
  at += n * 8;
  b.part = (double *)(ws + at);
  at += parts * 8;
  b.live = (int32_t *)(ws + at);
  at += n * 4;
  b.cnt = (int32_t *)(ws + at);
  at += n * E * 4;
  b.sum = (float *)(ws + at);
  at += n * E * 4;
  b.bytes = at;
  return b;
}

size_t balance_workspace(int T, int E, int S) { return balance_space(nullptr, slices(T, E, S), E, S).bytes; }

// balance_coef E / (segments K T_g^2)
__device__ __forceinline__ double segment_factor(const BalanceArgs &a, int live) {
  return live > 0 ? (double)a.balance_coef * a.E / ((double)a.S * a.K * live * live) : 0.0;
}

// First kernel: a workgroup sums over a slice of a segment's tokens; ALONE: the only workgroup over all tokens of each segment
// in turn, and writes the results itself.
template <int L, int NV, int SCORE, bool F32, bool ALONE>
__global__ void __launch_bounds__(256) balance_sums_kernel(BalanceArgs a, int slices) {
  constexpr int TOKENS = 4 * (64 / L);  // at a time
  __shared__ __align__(16) float red[TOKENS][L * NV];
  __shared__ int cnt[L * NV];
  __shared__ double zs[TOKENS];
  __shared__ int lives[TOKENS];
  const int lane = threadIdx.x & (L - 1), sub = threadIdx.x / L;
  const int wave0 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * (64 / L);  // the wave's first token
  const int E = a.E, K = a.K, n = a.T / a.S, s = ALONE ? 0 : blockIdx.x % slices;
  double loss = 0.0, all_z = 0.0;  // ALONE: of this thread's columns; of all tokens
  int all_live = 0;
  for (int g = ALONE ? 0 : blockIdx.x / slices; g < (ALONE ? a.S : blockIdx.x / slices + 1); ++g) {
    for (int e = threadIdx.x; e < E; e += 256) cnt[e] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)g * n + (int64_t)n * s / slices, t1 = (int64_t)g * n + (int64_t)n * (s + 1) / slices;
    float acc[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) acc[i] = 0.0f;
    double z = 0.0;
    int live = 0;
    float next[NV];
    int next_id = -1;
    auto fetch = [&](int64_t tb) {
      const int64_t t = tb + sub;
      const bool on = t < t1 && (!a.mask || a.mask[t]);
      load_logits<L, NV, F32>(a.logits, tb + wave0, a.T, E, lane, on, next);
      next_id = on && lane < K ? a.idx[t * K + lane] : -1;
    };
    if (t0 < t1) fetch(t0);
    for (int64_t tb = t0; tb < t1; tb += TOKENS) {  // the same for all lanes of the wave
      float l[NV], p[NV], rest[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) l[i] = next[i];
      const int id = next_id;
      if (tb + TOKENS < t1) fetch(tb + TOKENS);  // under way meanwhile
      const float m = row_max<L, NV>(l);
      const bool counts = m > MOE_NEG_INF;
      scores<NV, SCORE>(l, m, p, rest);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) sum += p[i];
      sum = sum_of<L>(sum);
      const float r = counts ? __builtin_amdgcn_rcpf(sum) : 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) acc[i] = __builtin_fmaf(p[i], r, acc[i]);
      if (a.z_coef != 0.0f) {
        if constexpr (SCORE == MOE_SCORE_SIGMOID) {
          sum = 0.0f;
#pragma unroll
          for (int i = 0; i < NV; ++i) sum += exp_neg(l[i] - m);
          sum = sum_of<L>(sum);
        }
        const double lse = counts ? m + logf(sum) : 0.0f;
        z += lse * lse;
      }
      live += counts;
      if (counts && id >= 0 && id < E) atomicAdd(&cnt[id], 1);  // integers: in any order
    }
#pragma unroll
    for (int c = 0; c < NV / 4; ++c)
      *(f32x4 *)&red[sub][id_of<L>(lane, c * 4)] = f32x4{acc[c * 4], acc[c * 4 + 1], acc[c * 4 + 2], acc[c * 4 + 3]};
    if (lane == 0) {
      zs[sub] = z;
      lives[sub] = live;
    }
    __syncthreads();
    z = zs[0];
    live = lives[0];
#pragma unroll
    for (int k = 1; k < TOKENS; ++k) {
      z += zs[k];
      live += lives[k];
    }
    const double f = ALONE ? segment_factor(a, live) : 0.0;
    BalanceSpace ws;
    if (!ALONE) ws = balance_space(a.ws, slices, E, a.S);
    for (int e = threadIdx.x; e < E; e += 256) {
      double v = (double)red[0][e];  // of at most 64 tokens each
#pragma unroll
      for (int k = 1; k < TOKENS; ++k) v += (double)red[k][e];
      if constexpr (ALONE) {
        a.sums[(int64_t)g * E + e] = (float)v;
        a.counts[(int64_t)g * E + e] = cnt[e];
        loss += f * cnt[e] * v;
      } else {
        ws.sum[(int64_t)blockIdx.x * E + e] = (float)v;
        ws.cnt[(int64_t)blockIdx.x * E + e] = cnt[e];
      }
    }
    if constexpr (ALONE) {
      if (threadIdx.x == 0) a.tokens[g] = live;
      all_z += z;
      all_live += live;
      __syncthreads();
    } else if (threadIdx.x == 0) {
      ws.z[blockIdx.x] = z;
      ws.live[blockIdx.x] = live;
      if (blockIdx.x == 0) *ws.counter = 0;
    }
  }
  if constexpr (ALONE) {
    loss = sum_of<64>(loss);
    if ((threadIdx.x & 63) == 0) zs[threadIdx.x >> 6] = loss;
    __syncthreads();
    if (threadIdx.x == 0) {
      a.losses[0] = (float)((zs[0] + zs[1]) + (zs[2] + zs[3]));
      a.losses[1] = all_live > 0 ? (float)((double)a.z_coef * all_z / all_live) : 0.0f;
    }
  }
}

// Whether a single workgroup does it all: rounds of its tokens, in values a lane.  Against two launches, us in graph replays
// (and the second launch costs the host 3 more): 16 tokens of 64 ids 3.2 / 6.9, 128 8.2 / 8.3, 256 13.8 / 8.5; 16 of 256
// 4.9 / 8.2, 64 10.5 / 10.2.
constexpr int kAloneValues = 32;

// Second kernel: a workgroup C columns of a segment, 1024 / C parts of its slices; the last one to finish adds the parts of
// the losses, in order.
template <int C>
__global__ void __launch_bounds__(1024) balance_losses_kernel(BalanceArgs a, int slices) {
  constexpr int PARTS = 1024 / C;
  __shared__ double red[PARTS][C];
  __shared__ int redc[PARTS][C];
  __shared__ double reds[16];
  __shared__ int last;
  const int tid = threadIdx.x, col = tid & (C - 1), part = tid / C;
  const int E = a.E, nb = (E + C - 1) / C, g = blockIdx.x / nb, e = (blockIdx.x - g * nb) * C + col;
  const BalanceSpace ws = balance_space(a.ws, slices, E, a.S);
  double sum = 0.0;
  int cnt = 0, n = 0;
  if (e < E) {
#pragma unroll 4
    for (int s = part; s < slices; s += PARTS) {
      sum += (double)ws.sum[((int64_t)g * slices + s) * E + e];
      cnt += ws.cnt[((int64_t)g * slices + s) * E + e];
    }
  }
  red[part][col] = sum;
  redc[part][col] = cnt;
  if (part == 0)  // by each of its waves
    for (int s = tid & 63; s < slices; s += 64) n += ws.live[(int64_t)g * slices + s];
  __syncthreads();
  if (part == 0) {
    n = sum_of<64>(n);
#pragma unroll
    for (int v = 1; v < PARTS; ++v) {
      sum += red[v][col];
      cnt += redc[v][col];
    }
    if (e < E) {
      a.counts[(int64_t)g * E + e] = cnt;
      a.sums[(int64_t)g * E + e] = (float)sum;
    }
    if (e == 0) a.tokens[g] = n;
    const double mine = sum_of<64>(segment_factor(a, n) * cnt * sum);
    if ((tid & 63) == 0) reds[tid >> 6] = mine;
  }
  __syncthreads();
  if (tid == 0) {
    double mine = reds[0];
    for (int v = 1; v < C / 64; ++v) mine += reds[v];
    // the part is in memory, past this XCD's caches, before the count says so
    __hip_atomic_store(&ws.part[blockIdx.x], mine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    last = __hip_atomic_fetch_add(ws.counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  double loss = 0.0, z = 0.0;
  n = 0;
  for (int i = tid; i < (int)gridDim.x; i += 1024)
    loss += __hip_atomic_load(&ws.part[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (int i = tid; i < a.S * slices; i += 1024) {
    z += ws.z[i];
    n += ws.live[i];
  }
  loss = sum_of<64>(loss);
  z = sum_of<64>(z);
  n = sum_of<64>(n);
  double *lr = &red[0][0], *zr = lr + 16;
  int *nr = &redc[0][0];
  if ((tid & 63) == 0) {
    lr[tid >> 6] = loss;
    zr[tid >> 6] = z;
    nr[tid >> 6] = n;
  }
  __syncthreads();
  if (tid == 0) {
    for (int v = 1; v < 16; ++v) {
      loss += lr[v];
      z += zr[v];
      n += nr[v];
    }
    a.losses[0] = (float)loss;
    a.losses[1] = n > 0 ? (float)((double)a.z_coef * z / n) : 0.0f;
  }
}

// f(score, whether fp32) with both as constants
template <class F>
static void with_types(int score, bool fp32, F &&f) {
  using Soft = std::integral_constant<int, MOE_SCORE_SOFTMAX>;
  using Sig = std::integral_constant<int, MOE_SCORE_SIGMOID>;
  if (score == MOE_SCORE_SOFTMAX && fp32) f(Soft{}, std::true_type{});
  else if (score == MOE_SCORE_SOFTMAX) f(Soft{}, std::false_type{});
  else if (fp32) f(Sig{}, std::true_type{});
  else f(Sig{}, std::false_type{});
}

hipError_t launch_balance(const BalanceArgs &a, int score, bool fp32, hipStream_t st) {
  const int n = slices(a.T, a.E, a.S);
  bool alone = false;
  with_sums_token(a.E, [&](auto tok) {
    constexpr int L = decltype(tok)::LANES, NV = decltype(tok)::VALUES, TOKENS = 4 * (64 / L);
    alone = NV <= 16 && (int64_t)a.S * ((a.T / a.S + TOKENS - 1) / TOKENS) * NV <= kAloneValues;
    with_types(score, fp32, [&](auto sc, auto f32) {
      constexpr int SC = decltype(sc)::value;
      constexpr bool F32 = decltype(f32)::value;
      if constexpr (NV <= 16) {
        if (alone) {
          hipLaunchKernelGGL((balance_sums_kernel<L, NV, SC, F32, true>), dim3(1), dim3(256), 0, st, a, 1);
          return;
        }
      }
      hipLaunchKernelGGL((balance_sums_kernel<L, NV, SC, F32, false>), dim3((unsigned)(a.S * n)), dim3(256), 0, st, a, n);
    });
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || alone) return e;
  if (n >= 16) hipLaunchKernelGGL((balance_losses_kernel<64>), dim3((unsigned)(a.S * ((a.E + 63) / 64))), dim3(1024), 0, st, a, n);
  else hipLaunchKernelGGL((balance_losses_kernel<256>), dim3((unsigned)(a.S * ((a.E + 255) / 256))), dim3(1024), 0, st, a, n);
  return hipGetLastError();
}

// ---- the gradient --------------------------------------------------------------------------------

template <int L, int NV, bool F32>
__device__ __forceinline__ void store_grad(void *out, int64_t t0, int T, int E, int lane, const float *d) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  constexpr int SIZE = F32 ? 4 : 2;
  const __amdgpu_buffer_rsrc_t rows = wave_rows<L>(out, t0, T, E, SIZE);
  const int off = ((int)(threadIdx.x & 63) / L * E + lane * 4) * SIZE;
#pragma unroll
  for (int c = 0; c < NV / 4; ++c) {
    const float *v = d + c * 4;
    const int e = id_of<L>(lane, c * 4), at = off + c * L * 4 * SIZE;
    const bf16x2 h[2] = {{(__bf16)v[0], (__bf16)v[1]}, {(__bf16)v[2], (__bf16)v[3]}};  // to nearest even
    const u32x2 b = {__builtin_bit_cast(uint32_t, h[0]), __builtin_bit_cast(uint32_t, h[1])};
    if ((E & 3) == 0) {
      const int to = e < E ? at : kNowhere;
      if constexpr (F32)
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])}, rows, to, 0, 0);
      else __builtin_amdgcn_raw_buffer_store_b64(b, rows, to, 0, 0);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int to = e + k < E ? at + k * SIZE : kNowhere;
        if constexpr (F32) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[k]), rows, to, 0, 0);
        else __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(b[k >> 1] >> (16 * (k & 1))), rows, to, 0, 0);
      }
    }
  }
}

template <int L, int NV, int SCORE, bool F32>
__global__ void __launch_bounds__(256) route_grad_kernel(RouteGradArgs a) {
  constexpr int TOKENS = 4 * (64 / L);
  __shared__ __align__(16) float rows[TOKENS][L * NV];  // what goes to a token's chosen ids
  __shared__ int parts[4];
  const int lane = threadIdx.x & (L - 1), sub = threadIdx.x / L;
  const int wave0 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * (64 / L);  // the wave's first token
  const int E = a.E, K = a.K;
  const bool losses = a.counts != nullptr, zloss = losses && a.z_coef != 0.0f;
  const float per_balance = losses ? (float)((double)(a.gl ? a.gl[0] : 1.0f) * a.balance_coef * E / ((double)a.S * K)) : 0.0f;
  const float mean_count = (float)K / (float)E;
  float per_z = 0.0f;  // of a token
  if (zloss) {
    int n = 0;
    for (int i = threadIdx.x; i < a.S; i += 256) n += a.tokens[i];
    n = sum_of<64>(n);
    if ((threadIdx.x & 63) == 0) parts[threadIdx.x >> 6] = n;
    __syncthreads();
    n = parts[0] + parts[1] + parts[2] + parts[3];
    per_z = n > 0 ? (float)(2.0 * a.z_coef * (a.gl ? a.gl[1] : 1.0f) / n) : 0.0f;
  }
  const uint32_t n = losses ? (uint32_t)(a.T / a.S) : 1;
  for (int64_t tb = (int64_t)blockIdx.x * TOKENS; tb < a.T; tb += (int64_t)gridDim.x * TOKENS) {
    const int64_t t = tb + sub;
    const bool on = t < a.T && (!a.mask || a.mask[t]);
    float l[NV], p[NV], rest[NV], d[NV];
    load_logits<L, NV, F32>(a.logits, tb + wave0, a.T, E, lane, on, l);
    int id = on && a.gw && lane < K ? a.idx[t * K + lane] : -1;
    if (id < 0 || id >= E) id = -1;
    float lj = MOE_NEG_INF, gw = 0.0f;
    if (id >= 0) {
      lj = logit_at(a.logits, F32, t * E + id);
      const int64_t at = t * K + lane;
      if (!a.dst) {
        gw = a.gw[at];
      } else {
        const int r = a.dst[at];
        if (r >= 0 && r < a.rows) gw = a.gw[r];
      }
    }
    const bool some = lj > MOE_NEG_INF;
    if (!some) gw = 0.0f;
    const float m = row_max<L, NV>(l);
    const bool counts = m > MOE_NEG_INF;
    scores<NV, SCORE>(l, m, p, rest);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) sum += p[i];
    sum = sum_of<L>(sum);
    const float r = counts ? __builtin_amdgcn_rcpf(sum) : 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      p[i] *= r;
      d[i] = 0.0f;
    }
    if (a.gw) {
      // of the logarithms of the scores of the token's ids: slot j on lane j
      float aj, sum_a = 0.0f, s, s_rest;
      if (a.renorm) {
        // divided, as in the choice, and about the gradient of a slot with the largest score: one that carries the sum loses no
        // digits of the others', and where one slot alone has a score the result is 0 exactly
        const float top = max_of<L>(lj);
        scores<1, SCORE>(&lj, top, &s, &s_rest);
        const float all = sum_of<L>(some ? s : 0.0f);
        const float w = some ? s / all : 0.0f;
        const uint64_t best = token_bits<L>(ballot(some && lj == top));
        const float g0 = __shfl(gw, best ? __builtin_ctzll(best) : 0, L);
        const float diff = some ? gw - g0 : 0.0f;
        const float mean = sum_of<L>(w * diff);
        aj = some ? a.scale * w * (diff - mean) : 0.0f;
      } else {
        s = SCORE == MOE_SCORE_SOFTMAX ? exp_neg(lj - m) * r : sigmoid(lj, s_rest);
        aj = some ? a.scale * s * gw : 0.0f;
        if (SCORE == MOE_SCORE_SOFTMAX) sum_a = sum_of<L>(aj);
      }
      // to the lanes that hold the ids, through LDS; slots of the same id all carry their sum
      float whole = aj;
      if (id >= 0) rows[sub][id] = __int_as_float(lane);
      lds_order();
      if (ballot(id >= 0 && __float_as_int(rows[sub][id >= 0 ? id : 0]) != lane)) {
        whole = 0.0f;
        for (int j = 0; j < K; ++j) {
          const int o = __shfl(id, j, L);
          const float v = __shfl(aj, j, L);
          whole += o == id ? v : 0.0f;
        }
      }
      lds_order();
#pragma unroll
      for (int c = 0; c < NV / 4; ++c) *(f32x4 *)&rows[sub][id_of<L>(lane, c * 4)] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      lds_order();
      if (id >= 0) rows[sub][id] = whole;
      lds_order();
#pragma unroll
      for (int c = 0; c < NV / 4; ++c) {
        const f32x4 v = *(const f32x4 *)&rows[sub][id_of<L>(lane, c * 4)];
#pragma unroll
        for (int k = 0; k < 4; ++k) d[c * 4 + k] = __builtin_fmaf(-sum_a, p[c * 4 + k], v[k]);
      }
      lds_order();
    }
    if (losses) {
      const uint32_t g = on ? (uint32_t)t / n : 0;
      const int live = a.tokens[g];
      const float over = live > 0 ? __builtin_amdgcn_rcpf((float)live) : 0.0f, f = counts ? per_balance * over * over : 0.0f;
      const float c0 = mean_count * (float)live;  // sum p = 1: any constant may be taken off; the mean loses least
      float A[NV], s = 0.0f;
      const int32_t *ct = a.counts + (int64_t)g * E;
      int c[NV];
#pragma unroll
      for (int q = 0; q < NV / 4; ++q) {
        const int e = id_of<L>(lane, q * 4);
        typedef int i32x4 __attribute__((ext_vector_type(4), aligned(4)));
        i32x4 v = {0, 0, 0, 0};
        if (e + 3 < E) v = *(const i32x4 *)(ct + e);
        else
#pragma unroll
          for (int k = 0; k < 3; ++k) v[k] = e + k < E ? ct[e + k] : 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) c[q * 4 + k] = v[k];
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {  // behind the last id p is 0
        A[i] = (float)c[i] - c0;
        s = __builtin_fmaf(A[i], p[i], s);
      }
      s = sum_of<L>(s);
#pragma unroll
      for (int i = 0; i < NV; ++i) d[i] = __builtin_fmaf(p[i] * f, A[i] - s, d[i]);
    }
    if constexpr (SCORE == MOE_SCORE_SIGMOID) {
#pragma unroll
      for (int i = 0; i < NV; ++i) d[i] *= rest[i];
    }
    if (zloss) {
      float e[NV];
      if constexpr (SCORE == MOE_SCORE_SIGMOID) {
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          e[i] = exp_neg(l[i] - m);
          sum += e[i];
        }
        sum = sum_of<L>(sum);
      }
      const float lse = counts ? m + logf(sum) : 0.0f;
      const float f = counts ? per_z * lse : 0.0f;
      if constexpr (SCORE == MOE_SCORE_SIGMOID) {
        const float fr = counts ? f * __builtin_amdgcn_rcpf(sum) : 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) d[i] = __builtin_fmaf(fr, e[i], d[i]);
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) d[i] = __builtin_fmaf(f, p[i], d[i]);
      }
    }
    store_grad<L, NV, F32>(a.out, tb + wave0, a.T, E, lane, d);
  }
}

hipError_t launch_route_grad(const RouteGradArgs &a, int score, bool fp32, hipStream_t st) {
  if (a.T == 0) return hipSuccess;
  with_token(a.T, a.E, [&](auto tok) {
    constexpr int L = decltype(tok)::LANES, NV = decltype(tok)::VALUES, TOKENS = 4 * (64 / L);
    const int wg = (a.T + TOKENS - 1) / TOKENS;
    with_types(score, fp32, [&](auto sc, auto f32) {
      hipLaunchKernelGGL((route_grad_kernel<L, NV, decltype(sc)::value, decltype(f32)::value>),
                         dim3((unsigned)(wg < 4096 ? wg : 4096)), dim3(256), 0, st, a);
    });
  });
  return hipGetLastError();
}

}  // namespace moe
