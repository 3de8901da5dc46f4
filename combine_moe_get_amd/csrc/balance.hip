// balance.hip -- the router's balance losses, and the gradient of its logits.
#include "route_internal.hpp"

namespace moe {

// ---- the losses ----------------------------------------------------------------------------------

// Workgroups that share a segment's tokens.
static int slices(int T, int S) {
  const int n = T / S, most = (n + 15) / 16, want = (1024 + S - 1) / S;
  const int L = most < want ? most : want;
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

size_t balance_workspace(int T, int E, int S) { return balance_space(nullptr, slices(T, S), E, S).bytes; }

// First kernel: a workgroup sums over a slice of a segment's tokens, a wave one token at a time.
template <int NV, int SCORE, bool F32>
__global__ void __launch_bounds__(256) balance_sums_kernel(BalanceArgs a, int L) {
  __shared__ float red[4][64 * NV];
  __shared__ int cnt[64 * NV];
  __shared__ double zs[4];
  __shared__ int lives[4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int E = a.E, K = a.K, n = a.T / a.S, g = blockIdx.x / L, s = blockIdx.x - g * L;
  const BalanceSpace ws = balance_space(a.ws, L, E, a.S);
  if (blockIdx.x == 0 && threadIdx.x == 0) *ws.counter = 0;
  for (int e = threadIdx.x; e < E; e += 256) cnt[e] = 0;
  __syncthreads();
  const int64_t t0 = (int64_t)g * n + (int64_t)n * s / L, t1 = (int64_t)g * n + (int64_t)n * (s + 1) / L;
  float acc[NV], p[NV], l[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) acc[i] = 0.0f;
  double z = 0.0;
  int live = 0;
  for (int64_t t = t0 + wave; t < t1; t += 4) {
    if (a.mask && !a.mask[t]) continue;
    load_logits<NV, F32>(a.logits, t, E, lane, l);
    const float m = row_max<NV>(l);
    if (!(m > MOE_NEG_INF)) continue;
    ++live;
    probabilities<NV, SCORE>(l, m, p);
#pragma unroll
    for (int i = 0; i < NV; ++i) acc[i] += p[i];
    if (a.z_coef != 0.0f) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) sum += expf(l[i] - m);
      const double lse = (double)m + log((double)wave_sum(sum));
      z += lse * lse;
    }
    const int id = lane < K ? a.idx[t * K + lane] : -1;
    if (id >= 0 && id < E) atomicAdd(&cnt[id], 1);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) red[wave][lane * NV + i] = acc[i];
  if (lane == 0) {
    zs[wave] = z;
    lives[wave] = live;
  }
  __syncthreads();
  const int64_t slot = (int64_t)blockIdx.x;
  for (int e = threadIdx.x; e < E; e += 256) {
    ws.sum[slot * E + e] = (red[0][e] + red[1][e]) + (red[2][e] + red[3][e]);
    ws.cnt[slot * E + e] = cnt[e];
  }
  if (threadIdx.x == 0) {
    ws.z[slot] = (zs[0] + zs[1]) + (zs[2] + zs[3]);
    ws.live[slot] = lives[0] + lives[1] + lives[2] + lives[3];
  }
}

// Second kernel: a workgroup 64 columns of a segment; the last one to finish adds the parts of the losses, in order.
__global__ void __launch_bounds__(256) balance_losses_kernel(BalanceArgs a, int L) {
  __shared__ double red[4][64];
  __shared__ int redc[4][64];
  __shared__ int last;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int E = a.E, nb = (E + 63) / 64, g = blockIdx.x / nb, e = (blockIdx.x - g * nb) * 64 + lane;
  const BalanceSpace ws = balance_space(a.ws, L, E, a.S);
  double sum = 0.0;
  int cnt = 0;
  if (e < E) {
    for (int s = wave; s < L; s += 4) {
      sum += (double)ws.sum[((int64_t)g * L + s) * E + e];
      cnt += ws.cnt[((int64_t)g * L + s) * E + e];
    }
  }
  red[wave][lane] = sum;
  redc[wave][lane] = cnt;
  __syncthreads();
  if (wave == 0) {
    int n = 0;
    for (int s = lane; s < L; s += 64) n += ws.live[(int64_t)g * L + s];
    n = readlane(wave_inclusive_sum(n), 63);
    sum = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
    cnt = redc[0][lane] + redc[1][lane] + redc[2][lane] + redc[3][lane];
    if (e < E) {
      a.counts[(int64_t)g * E + e] = cnt;
      a.sums[(int64_t)g * E + e] = (float)sum;
    }
    if (lane == 0 && e == 0) a.tokens[g] = n;
    const double f = n > 0 ? (double)a.balance_coef * E / ((double)a.S * a.K * n * n) : 0.0;
    const double part = wave_sum(f * cnt * sum);
    if (lane == 0) {
      __hip_atomic_store(&ws.part[blockIdx.x], part, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      last = __hip_atomic_fetch_add(ws.counter, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  double loss = 0.0, z = 0.0;
  int n = 0;
  for (int i = threadIdx.x; i < (int)gridDim.x; i += 256)
    loss += __hip_atomic_load(&ws.part[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (int i = threadIdx.x; i < a.S * L; i += 256) {
    z += ws.z[i];
    n += ws.live[i];
  }
  loss = wave_sum(loss);
  z = wave_sum(z);
  n = readlane(wave_inclusive_sum(n), 63);
  if (lane == 0) {
    red[wave][0] = loss;
    red[wave][1] = z;
    redc[wave][0] = n;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int v = 1; v < 4; ++v) {
      loss += red[v][0];
      z += red[v][1];
      n += redc[v][0];
    }
    a.losses[0] = (float)loss;
    a.losses[1] = n > 0 ? (float)((double)a.z_coef * z / n) : 0.0f;
  }
}

hipError_t launch_balance(const BalanceArgs &a, int score, bool fp32, hipStream_t st) {
  const int L = slices(a.T, a.S);
  with_values(a.E, [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    auto go = [&](auto sc, auto f32) {
      hipLaunchKernelGGL((balance_sums_kernel<NV, decltype(sc)::value, decltype(f32)::value>), dim3((unsigned)(a.S * L)),
                         dim3(256), 0, st, a, L);
    };
    if (score == MOE_SCORE_SOFTMAX) {
      if (fp32) go(std::integral_constant<int, MOE_SCORE_SOFTMAX>{}, std::true_type{});
      else go(std::integral_constant<int, MOE_SCORE_SOFTMAX>{}, std::false_type{});
    } else {
      if (fp32) go(std::integral_constant<int, MOE_SCORE_SIGMOID>{}, std::true_type{});
      else go(std::integral_constant<int, MOE_SCORE_SIGMOID>{}, std::false_type{});
    }
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(balance_losses_kernel, dim3((unsigned)(a.S * ((a.E + 63) / 64))), dim3(256), 0, st, a, L);
  return hipGetLastError();
}

// ---- the gradient --------------------------------------------------------------------------------

template <int NV, bool F32>
__device__ __forceinline__ void store_grad(void *out, int64_t t, int E, int lane, const float *d) {
  typedef __bf16 b16;
  const int e0 = lane * NV;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (e0 + i < E) {
      if constexpr (F32) ((float *)out)[t * E + e0 + i] = d[i];
      else ((b16 *)out)[t * E + e0 + i] = (b16)d[i];  // to nearest even
    }
  }
}

template <int NV, int SCORE, bool F32>
__global__ void __launch_bounds__(256) route_grad_kernel(RouteGradArgs a) {
  __shared__ int parts[4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int E = a.E, K = a.K;
  const bool losses = a.counts != nullptr, zloss = losses && a.z_coef != 0.0f;
  double per_token = 0.0;  // of the z loss
  if (zloss) {
    int n = 0;
    for (int i = threadIdx.x; i < a.S; i += 256) n += a.tokens[i];
    n = wave_inclusive_sum(n);
    if (lane == 63) parts[wave] = n;
    __syncthreads();
    n = parts[0] + parts[1] + parts[2] + parts[3];
    per_token = n > 0 ? 2.0 * a.z_coef * (a.gl ? a.gl[1] : 1.0f) / n : 0.0;
  }
  const int n = losses ? a.T / a.S : 1;
  for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < a.T; t += (int64_t)gridDim.x * 4) {
    float l[NV], p[NV], d[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) d[i] = 0.0f;
    float m = MOE_NEG_INF;
    if (!a.mask || a.mask[t]) {
      load_logits<NV, F32>(a.logits, t, E, lane, l);
      m = row_max<NV>(l);
    }
    if (m > MOE_NEG_INF) {
      probabilities<NV, SCORE>(l, m, p);
      float sum_a = 0.0f, aj = 0.0f;
      int id = -1;
      if (a.gw) {
        if (lane < K) id = a.idx[t * K + lane];
        if (id >= E) id = -1;
        const float lj = id >= 0 ? logit_at(a.logits, F32, t * E + id) : MOE_NEG_INF;
        const bool some = lj > MOE_NEG_INF;
        float gw = 0.0f;
        if (some) {
          if (!a.dst) {
            gw = a.gw[t * K + lane];
          } else {
            const int r = a.dst[t * K + lane];
            if (r >= 0) gw = a.gw[r];
          }
        }
        if (a.renorm) {
          const float q = !some ? MOE_NEG_INF : SCORE == MOE_SCORE_SOFTMAX ? lj : log_sigmoid(lj);
          const float mq = wave_max(q);
          const float e = some ? expf(q - mq) : 0.0f;
          const float sum = wave_sum(e);  // by every lane, as all such sums
          const float w = some ? e / sum : 0.0f;
          const float mean = wave_sum(w * gw);
          aj = some ? a.scale * w * (gw - mean) : 0.0f;
        } else {
          float s;
          if constexpr (SCORE == MOE_SCORE_SOFTMAX) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) sum += expf(l[i] - m);
            sum = wave_sum(sum);
            s = expf(lj - m) / sum;
          } else {
            s = 1.0f / (1.0f + expf(-lj));
          }
          aj = some ? a.scale * s * gw : 0.0f;
          if (SCORE == MOE_SCORE_SOFTMAX) sum_a = wave_sum(aj);
        }
        for (int j = 0; j < K; ++j) {
          const int e = readlane(id, j) - lane * NV;
          const float v = readlane_f(aj, j);
#pragma unroll
          for (int i = 0; i < NV; ++i) d[i] += e == i ? v : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) d[i] -= sum_a * p[i];
      }
      if (losses) {
        const int64_t g = t / n;
        const int live = a.tokens[g];
        const float f = live > 0 ? (float)((double)(a.gl ? a.gl[0] : 1.0f) * a.balance_coef * E / ((double)a.S * K * live * live)) : 0.0f;
        const float c0 = (float)((double)K * live / E);  // sum p = 1: any constant may be taken off; the mean loses least
        float A[NV], s = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int e = lane * NV + i;
          A[i] = e < E ? f * ((float)a.counts[g * E + e] - c0) : 0.0f;
          s += A[i] * p[i];
        }
        s = wave_sum(s);
#pragma unroll
        for (int i = 0; i < NV; ++i) d[i] += p[i] * (A[i] - s);
      }
      if constexpr (SCORE == MOE_SCORE_SIGMOID) {
#pragma unroll
        for (int i = 0; i < NV; ++i) d[i] *= 1.0f / (1.0f + expf(l[i]));
      }
      if (zloss) {
        float e[NV], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          e[i] = expf(l[i] - m);
          sum += e[i];
        }
        sum = wave_sum(sum);
        const float f = (float)(per_token * ((double)m + log((double)sum)) / sum);
#pragma unroll
        for (int i = 0; i < NV; ++i) d[i] += f * e[i];
      }
    }
    store_grad<NV, F32>(a.out, t, E, lane, d);
  }
}

hipError_t launch_route_grad(const RouteGradArgs &a, int score, bool fp32, hipStream_t st) {
  if (a.T == 0) return hipSuccess;
  const int wg = (a.T + 3) / 4;
  const dim3 grid((unsigned)(wg < 2048 ? wg : 2048)), block(256);
  with_values(a.E, [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    auto go = [&](auto sc, auto f32) {
      hipLaunchKernelGGL((route_grad_kernel<NV, decltype(sc)::value, decltype(f32)::value>), grid, block, 0, st, a);
    };
    if (score == MOE_SCORE_SOFTMAX) {
      if (fp32) go(std::integral_constant<int, MOE_SCORE_SOFTMAX>{}, std::true_type{});
      else go(std::integral_constant<int, MOE_SCORE_SOFTMAX>{}, std::false_type{});
    } else {
      if (fp32) go(std::integral_constant<int, MOE_SCORE_SIGMOID>{}, std::true_type{});
      else go(std::integral_constant<int, MOE_SCORE_SIGMOID>{}, std::false_type{});
    }
  });
  return hipGetLastError();
}

}  // namespace moe
