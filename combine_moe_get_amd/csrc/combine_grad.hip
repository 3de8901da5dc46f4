// combine_grad.hip -- the gradient of the weighted combine.
//
// out[t] = sum_j w[t,j] Moe_j(t) (combine.hip), so with g the gradient of out[t]:
//   routed slot     grad of its row: w g;   of w: <g, row>
//   copy slot       grad of x: += w g;      of w: <g, x>
//   constant slot   grad of x: += w alpha1 g; of w: <g, alpha1 x + alpha2 v>;
//                   alpha1 += w g x, alpha2 += w g v, v += w g alpha2 (all element-wise, over all tokens)
//   zero, dropped or masked slot: nothing; w: 0
// One workgroup a token: g is read once, every expert row once and every gradient row is written once, so memory
// bounds it: 4096 tokens of 4096 with 8 of 64 experts (576 MB) 95 us, 6.1 TB/s; 128 tokens of 7168 (31 MB, mostly
// from the caches) 11 us.
// The gradients of the constant experts' vectors are sums over tokens: the launch's first workgroups, one for each 64
// columns of each of these experts, whose waves take equal parts of the tokens in order and are added in order, so
// that the result depends on the shape alone.  They wait for one load after the other and not for the memory's rate,
// and run beside the tokens': 4096 x 8 slots on 128 experts, 2 copy and 2 constant ones, rows of 4096 (570 MB): 104 us, 5.5
// TB/s (in a kernel of their own, behind it: 22 us more; the next slots not under way meanwhile).  Each of them looks at
// all ids, so the work grows with the number of these experts: made for few (4096 tokens of 8192, top 8 of 128 and 2, 16
// or 64 constant ones: 233, 320, 555 us).
#include "experts_internal.hpp"

namespace moe {

__device__ __forceinline__ uint32_t pack2g(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ void unpack8g(const u32x4 &v, float *f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(v[i]);
    f[2 * i + 1] = bf16_hi(v[i]);
  }
}

enum : int { G_NONE = 0, G_ROUTED = 1, G_COPY = 2, G_CONST = 3 };

// The constant experts' vectors: a workgroup 64 columns of one expert.  Wave v of the nw adds the slots of the v-th part
// of the tokens, in order.  It looks at 512 slots at a time (the next 512 under way meanwhile), lists in LDS the ones
// it is looking for and takes eight of them at a time.
constexpr int kScan = 512, kTake = 8;
__device__ __forceinline__ void const_grad(const CombineGradArgs &a, int b, char *lds) {
  const CombineArgs &c = a.c;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nw = blockDim.x >> 6;
  int *slot = (int *)lds + wave * kScan;  // the wave's own: its LDS accesses are in order
  float *sg = (float *)((int *)lds + nw * kScan), *sq = sg + nw * 64;
  const int ncol = (c.H + 63) / 64, k = b / ncol, h = (b - k * ncol) * 64 + lane;
  const int id = c.E + c.Z + c.C + k;
  const int per = (c.T + nw - 1) / nw, lo = wave * per < c.T ? wave * per : c.T, hi = lo + per < c.T ? lo + per : c.T;
  const int s1 = hi * c.K;  // T K <= 2^24
  float g = 0.0f, q = 0.0f;
  int ids[kScan / 64], on[kScan / 64];
  auto look = [&](int s0) {
#pragma unroll
    for (int i = 0; i < kScan / 64; ++i) {
      const int s = s0 + i * 64 + lane;
      ids[i] = s < s1 ? c.topk_idx[s] : -1;
      on[i] = c.mask && s < s1 ? c.mask[s / c.K] : 1;
    }
  };
  look(lo * c.K);
  for (int s0 = lo * c.K; s0 < s1; s0 += kScan) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kScan / 64; ++i) {
      const bool hit = ids[i] == id && on[i] != 0;
      const uint64_t hits = ballot(hit);
      if (hit) slot[n + popc_below(hits)] = s0 + i * 64 + lane;
      n += __builtin_popcountll(hits);
    }
    look(s0 + kScan);
    for (int i = 0; i < n; i += kTake) {
      float w[kTake], gv[kTake], xv[kTake];
#pragma unroll
      for (int u = 0; u < kTake; ++u) {
        w[u] = gv[u] = xv[u] = 0.0f;
        if (i + u < n) {
          const int s = __builtin_amdgcn_readfirstlane(slot[i + u]);
          w[u] = c.w[s];
          if (h < c.H) {
            const size_t at = (size_t)(s / c.K) * c.H + h;
            gv[u] = __uint_as_float((uint32_t)a.go[at] << 16);
            if (a.ga1) xv[u] = __uint_as_float((uint32_t)c.ori_x[at] << 16);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kTake; ++u) {
        if (i + u < n) {
          const float wg = w[u] * gv[u];
          g += wg;
          q = __builtin_fmaf(wg, xv[u], q);
        }
      }
    }
  }
  sg[wave * 64 + lane] = g;
  sq[wave * 64 + lane] = q;
  __syncthreads();
  if (wave == 0 && h < c.H) {
    for (int v = 1; v < nw; ++v) {
      g += sg[v * 64 + lane];
      q += sq[v * 64 + lane];
    }
    const size_t at = (size_t)k * c.H + h;
    if (a.ga1) a.ga1[at] = q;
    if (a.ga2) a.ga2[at] = __uint_as_float((uint32_t)c.cv[at] << 16) * g;
    if (a.gv) a.gv[at] = __uint_as_float((uint32_t)c.a2[at] << 16) * g;
  }
}

// One workgroup a token, a thread one chunk of 8 elements (two a thread, in turn: 99 us for the 95 above, 8.4 for 6.7
// on 16 tokens of 7168); threads past the row's end only take part in the sums.  The slots' kinds, rows and weights are
// wave-uniform; every row is requested before the first is used.  KMAX: the least of 1, 2, 4, 8, 16 that holds the
// slots (K = 8 with 16: 12.5 us for 128 tokens of 7168, 10.7 with 8).  SPECIAL: copy and constant experts can occur;
// without them there is no x to read; with them every token reads its x, also one that has no such slot (two of 132
// experts each, top 8: four of five; some 5% of the bytes).
template <int KMAX, bool SPECIAL>
__global__ void __launch_bounds__(1024) combine_grad_kernel(CombineGradArgs a) {
  const CombineArgs &c = a.c;
  extern __shared__ __align__(16) char lds[];
  __shared__ float part[16][KMAX];
  if (SPECIAL && (int)blockIdx.x < a.vectors) {
    const_grad(a, blockIdx.x, lds);
    return;
  }
  const int t = blockIdx.x - (SPECIAL ? a.vectors : 0), tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int H = c.H, K = c.K, nch = H >> 3;
  const bool live = !c.mask || c.mask[t];

  int id = -1, r = -1;
  float wt = 0.0f;
  if (lane < K) {
    id = c.topk_idx[(size_t)t * K + lane];
    wt = c.w[(size_t)t * K + lane];
    r = c.dst_row[(size_t)t * K + lane];
  }
  const bool in = tid < nch;
  u32x4 gv = {0u, 0u, 0u, 0u}, xv = {0u, 0u, 0u, 0u};
  if (in) {
    gv = ((const u32x4 *)(a.go + (size_t)t * H))[tid];
    if (SPECIAL) xv = ((const u32x4 *)(c.ori_x + (size_t)t * H))[tid];
  }
  int k = G_NONE;
  if (live && lane < K) {
    const int zc = c.E + c.Z;
    if (id >= 0 && id < c.E) {
      k = r >= 0 ? G_ROUTED : G_NONE;
    } else if (SPECIAL && id >= zc && id < zc + c.C) {
      k = G_COPY;
    } else if (SPECIAL && id >= zc + c.C && id < zc + c.C + c.Kc) {
      k = G_CONST;
      r = id - zc - c.C;
    }
  }
  int kind[KMAX], row[KMAX];  // row: of expert_out, or of the constant experts' vectors
  float w[KMAX], dot[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    kind[j] = readlane(k, j);
    row[j] = readlane(r, j);
    w[j] = readlane_f(wt, j);
    dot[j] = 0.0f;
  }
  u32x4 yv[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    yv[j] = u32x4{0u, 0u, 0u, 0u};
    if (kind[j] == G_ROUTED && a.gw && in) yv[j] = __builtin_nontemporal_load((const u32x4 *)c.y + (size_t)row[j] * nch + tid);
  }
  float g[8], x[8], gx[8];
  unpack8g(gv, g);
  unpack8g(xv, x);
#pragma unroll
  for (int e = 0; e < 8; ++e) gx[e] = 0.0f;
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    if (kind[j] == G_NONE) continue;
    float y[8];
    if (!SPECIAL || kind[j] == G_ROUTED) {
      unpack8g(yv[j], y);
      if (a.gy && in) {
        u32x4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = pack2g(w[j] * g[2 * e], w[j] * g[2 * e + 1]);
        __builtin_nontemporal_store(o, (u32x4 *)a.gy + (size_t)row[j] * nch + tid);
      }
    } else if (kind[j] == G_COPY) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] = x[e];
        gx[e] = __builtin_fmaf(w[j], g[e], gx[e]);
      }
    } else {
      float a1[8], a2[8], v[8];
      const size_t at = (size_t)row[j] * nch + (in ? tid : 0);  // threads past the end: g = 0
      unpack8g(((const u32x4 *)c.a1)[at], a1);
      unpack8g(((const u32x4 *)c.a2)[at], a2);
      unpack8g(((const u32x4 *)c.cv)[at], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] = __builtin_fmaf(a1[e], x[e], a2[e] * v[e]);
        gx[e] = __builtin_fmaf(w[j] * a1[e], g[e], gx[e]);
      }
    }
    if (a.gw && in) {
#pragma unroll
      for (int e = 0; e < 8; ++e) dot[j] = __builtin_fmaf(g[e], y[e], dot[j]);
    }
  }
  if (SPECIAL && a.gx && in) {
    u32x4 o;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = pack2g(gx[2 * e], gx[2 * e + 1]);
    __builtin_nontemporal_store(o, (u32x4 *)(a.gx + (size_t)t * H) + tid);
  }
  if (!SPECIAL && a.gx) {  // no copy and no constant experts: zeros
    if (in) ((u32x4 *)(a.gx + (size_t)t * H))[tid] = u32x4{0u, 0u, 0u, 0u};
  }
  if (a.gw) {
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
#pragma unroll
      for (int s = 32; s > 0; s >>= 1) dot[j] += __shfl_xor(dot[j], s);
      if (lane == 0) part[wave][j] = dot[j];
    }
    __syncthreads();
    if (tid < K) {
      float s = 0.0f;
      for (int v = 0; v < (int)(blockDim.x >> 6); ++v) s += part[v][tid];
      a.gw[(size_t)t * K + tid] = s;
    }
  }
}

template <int KMAX>
static void launch_k(const CombineGradArgs &a, hipStream_t st) {
  const int nch = a.c.H >> 3;  // <= 1024
  // at least 8 waves where they search the slots for constant experts
  const unsigned threads = (unsigned)(a.vectors && nch < 512 ? 512 : (nch + 63) / 64 * 64);
  const dim3 grid((unsigned)(a.vectors + (a.gy || a.gw || a.gx ? a.c.T : 0))), block(threads);
  if (grid.x == 0) return;
  const size_t lds = a.vectors ? threads / 64 * (kScan + 2 * 64) * 4 : 0;
  if (a.c.C + a.c.Kc > 0) hipLaunchKernelGGL((combine_grad_kernel<KMAX, true>), grid, block, lds, st, a);
  else hipLaunchKernelGGL((combine_grad_kernel<KMAX, false>), grid, block, 0, st, a);
}

hipError_t launch_combine_grad(const CombineGradArgs &a_, hipStream_t st) {
  CombineGradArgs a = a_;
  a.vectors = a.ga1 || a.ga2 || a.gv ? (a.c.H + 63) / 64 * a.c.Kc : 0;  // T = 0: they are zeros
  if (a.c.K <= 1) launch_k<1>(a, st);
  else if (a.c.K <= 2) launch_k<2>(a, st);
  else if (a.c.K <= 4) launch_k<4>(a, st);
  else if (a.c.K <= 8) launch_k<8>(a, st);
  else launch_k<16>(a, st);
  return hipGetLastError();
}

}  // namespace moe
