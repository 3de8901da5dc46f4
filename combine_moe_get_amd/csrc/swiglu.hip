// swiglu.hip -- the gate between the two products of a layer that trains, silu(g) u with routing weights, and its
// gradient; between the two the gate's input may be kept in 8 bits.
#include <float.h>

#include "dispatch_dev.hpp"
#include "experts_internal.hpp"

namespace moe {

// The logistic function of g and 1 - it, which is never taken as a difference.  With n = exp(-|g|) and R = 1 / (1 + n) it is R for
// g >= 0 and n R below.
struct Logistic {
  float s, rest;
  __device__ __forceinline__ Logistic(float g) {
    constexpr float kLog2e = 1.44269504088896341f;
    const float n = __builtin_amdgcn_exp2f(fabsf(g) * -kLog2e), R = __builtin_amdgcn_rcpf(1.0f + n), nR = n * R;
    s = g >= 0.0f ? R : nR;
    rest = g >= 0.0f ? nR : R;
  }
};
// Below kFar n may be too small for fp32 but not what it multiplies: there it (1 - s is 1) and its products are in 64 bits, n from
// its eighth root, which fp32 holds down to g = -698 (below -366 no bf16 result is left, with weight, gradient and u the largest).
// Element by element of a lane, by its own value: what else the wave has only says whether anything is to be done (far_out).
// 32768 rows of 2 x 2048 with none such / 2%: forward 58 / 64 us, gradient from bf16 135 / 146.
constexpr float kFar = -80.0f;
__device__ __forceinline__ double logistic_far(float g) {
  constexpr float kLog2e = 1.44269504088896341f;
  const double q = __builtin_amdgcn_exp2f(g * (0.125f * kLog2e)), h = q * q, f = h * h;
  return f * f;
}
typedef float f32x8 __attribute__((ext_vector_type(8)));
// whether a lane of the wave has a g so far out
__device__ __forceinline__ bool far_out(const float *g) {
  float least = g[0];
#pragma unroll
  for (int e = 1; e < 8; ++e) least = fminf(least, g[e]);
  return ballot(least < kFar) != 0;
}

__device__ __forceinline__ uint32_t pack2s(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 v = {(__bf16)a, (__bf16)b};  // round to nearest even, NaN stays NaN
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ u32x4 pack8(const float *f) {
  return u32x4{pack2s(f[0], f[1]), pack2s(f[2], f[3]), pack2s(f[4], f[5]), pack2s(f[6], f[7])};
}

// the largest over a row of 16 lanes, to each of them
__device__ __forceinline__ float max16(float v) {
  auto fold = [&](auto ctrl) {
    const int b = __float_as_int(v);
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(b, b, decltype(ctrl)::value, 0xf, 0xf, false)));
  };
  fold(std::integral_constant<int, 0xb1>{});   // quad_perm 1 0 3 2
  fold(std::integral_constant<int, 0x4e>{});   // quad_perm 2 3 0 1
  fold(std::integral_constant<int, 0x141>{});  // row_half_mirror
  fold(std::integral_constant<int, 0x140>{});  // row_mirror
  return v;
}

// 1 / x for x between 2^-100 and 2^100 whose mantissa is a bf16's, or 127 times the reciprocal of one: one Newton step from the
// instruction's value, exact but for its last rounding, which leaves less than 2^-44; none of the 256 mantissas has its
// reciprocal that near to the middle between two fp32 values.
__device__ __forceinline__ float reciprocal(float x) {
  const float r = __builtin_amdgcn_rcpf(x);
  return __builtin_fmaf(__builtin_fmaf(-x, r, 1.0f), r, r);
}

// Four codes: x dyn rounded to a whole number, ties to even, by adding 1.5 2^23, whose last bits are then the code; NaN leaves 0
// there.  No product passes 127 by half a code while dyn is finite.
__device__ __forceinline__ uint32_t codes4(const float *x, float dyn) {
  uint32_t b[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) b[e] = __float_as_uint(x[e] * dyn + 12582912.0f);
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u), __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), 0x05040100u);
}
__device__ __forceinline__ uint32_t codes4_any(const float *x, float dyn) {
  return pack_i8x4(sat_code(x[0] * dyn), sat_code(x[1] * dyn), sat_code(x[2] * dyn), sat_code(x[3] * dyn));
}

constexpr uint64_t kMostGroups = 1 << 20;  // of a launch; they walk what is left

// ---- forward: 16 lanes a block of 128 columns of a row, 8 of each half a lane -----------------------
//
// One pass, bound by memory: 32768 rows of 2 x 2048 with codes 90 us (541 MB, 6.0 TB/s; a large copy reaches 5.1), without 68
// (403 MB, 5.9 TB/s).  A thread's 16 values take 285 vector instructions, in 80% of those cycles; with codes clamped and packed
// one by one, divisions for the reciprocals and 64 bits of address a thread it was these, 467, that bound it (108 us).  Stores
// go past the caches: 116 and 85 us where they do not, the gradient 159 for 155 (all before the instructions were fewer).  Two
// blocks a thread took 107 for 105 us, and 4.8 for 3.8 on 400 rows of 2 x 512.
template <bool KEEP>
__global__ void __launch_bounds__(256) swiglu_kernel(SwigluArgs a) {
  const int sub = threadIdx.x & 15;
  const uint32_t I = a.I, nb = (I + 127) / 128;
  for (uint64_t first = (uint64_t)blockIdx.x * 16; first < (uint64_t)a.rows * nb; first += (uint64_t)gridDim.x * 16) {
    // the workgroup's 16 blocks, in the order of rows: from this row on (floor(first / nb): half a block from the next whole number)
    const int64_t at = (int64_t)(((double)first + 0.5) * a.over_nb);
    const int64_t row0 = (int64_t)__builtin_amdgcn_readfirstlane((int)(at >> 32)) << 32 | (uint32_t)__builtin_amdgcn_readfirstlane((int)at);
    const uint32_t i = (uint32_t)(first - (uint64_t)row0 * nb) + (threadIdx.x >> 4), q = fast_div((int)i, a.div_nb), b = i - q * nb;
    const uint32_t col = b * 128 + sub * 8;
    const bool in = row0 + q < a.rows && col < I && row_used(a.g, row0 + q);
    // within the workgroup's rows 32 bits of offset do: at most 16 rows of one block, or two and some of more
    const uint32_t two = q * 2 * I + col, one = q * I + col;
    u32x4 gv = {0u, 0u, 0u, 0u}, uv = gv;
    float w = 1.0f;
    if (in) {
      const uint16_t *p = a.h0 + row0 * 2 * I;
      gv = *(const u32x4 *)(p + two);
      uv = *(const u32x4 *)(p + two + I);
      if (a.w) w = a.w[row0 + q];
    }
    float g[8], u[8], h[8];
    unpack8(gv, g);
    unpack8(uv, u);
    auto gate = [&](auto far) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[e] = Logistic(g[e]).s * g[e] * u[e] * w;
        if (decltype(far)::value && g[e] < kFar) h[e] = (float)(logistic_far(g[e]) * g[e] * u[e] * w);
      }
    };
    if (__builtin_expect(far_out(g), 0)) gate(std::true_type{});
    else gate(std::false_type{});
    if (in) __builtin_nontemporal_store(pack8(h), (u32x4 *)(a.out + row0 * I + one));
    if constexpr (KEEP) {
      auto largest = [&](const float *x) {
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]));
        return max16(m);
      };
      const float mg = largest(g), mu = largest(u);
      float dg, du, sg, su;
      u32x2 cg, cu;
      if (__builtin_expect(ballot(!(fminf(mg, mu) > 0x1p-100f && fmaxf(mg, mu) < 0x1p100f)) == 0, 1)) {
        dg = 127.0f * reciprocal(mg);
        du = 127.0f * reciprocal(mu);
        sg = reciprocal(dg);
        su = reciprocal(du);
        cg = u32x2{codes4(g, dg), codes4(g + 4, dg)};
        cu = u32x2{codes4(u, du), codes4(u + 4, du)};
      } else {  // a block of zeros, or of values so small or large that reciprocals leave the normal numbers
        dg = mg > 0.0f ? 127.0f * (1.0f / mg) : 0.0f;
        du = mu > 0.0f ? 127.0f * (1.0f / mu) : 0.0f;
        sg = mg > 0.0f ? 1.0f / dg : 0.0f;
        su = mu > 0.0f ? 1.0f / du : 0.0f;
        cg = u32x2{codes4_any(g, dg), codes4_any(g + 4, dg)};
        cu = u32x2{codes4_any(u, du), codes4_any(u + 4, du)};
      }
      if (in) {
        int8_t *c = a.codes + row0 * 2 * I;
        __builtin_nontemporal_store(cg, (u32x2 *)(c + two));
        __builtin_nontemporal_store(cu, (u32x2 *)(c + two + I));
        float *s = a.scales + row0 * 2 * nb;
        if (sub == 0) {
          s[q * 2 * nb + b] = sg;
          s[q * 2 * nb + nb + b] = su;
        }
      }
    }
  }
}

// ---- backward: L threads a row, U chunks of 8 columns a thread at a time -------------------------------
//
// One pass as well: the row's sum for its weight's gradient is folded over the L threads.  32768 rows of 2048 from codes 110 us
// (675 MB, 6.1 TB/s), 8192 of 4096 from bf16 70 us (403 MB, 5.8 TB/s).
__device__ __forceinline__ void unpack_codes(u32x2 v, float scale, float *f) {
  if (__builtin_expect(scale > 0x1p119f, 0)) {  // 128 times it may be infinite
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = (float)((int)(v[e >> 2] << (24 - 8 * (e & 3))) >> 24) * scale;
    return;
  }
  // (code + 128) scale - 128 scale: rounded once, as code scale
  const float off = -128.0f * scale;
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = __builtin_fmaf((float)((v[e >> 2] ^ 0x80808080u) >> (8 * (e & 3)) & 0xffu), scale, off);
}

template <int L, int U, bool KEPT>
__global__ void __launch_bounds__(256) swiglu_grad_kernel(SwigluArgs a) {
  constexpr int R = 256 / L, W = L > 64 ? L / 64 : 1;  // rows of a workgroup, waves of a row
  __shared__ float red[2][4];
  int par = 0;
  const int lane = threadIdx.x % L, I = a.I, nch = I >> 3;
  const uint32_t nb = (uint32_t)(I + 127) / 128;
  for (int64_t r0 = (int64_t)blockIdx.x * R; r0 < a.rows; r0 += (int64_t)gridDim.x * R) {
    const int64_t r = r0 + threadIdx.x / L;
    const bool used = r < a.rows && row_used(a.g, r);
    float dot = 0.0f;
    if (used) {
      const float w = a.w ? a.w[r] : 1.0f;
      for (int c0 = lane; c0 < nch; c0 += L * U) {
        u32x4 dv[U], gv[U], uv[U];
        u32x2 gc[U], uc[U];
        float gs[U], us[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int c = c0 + k * L < nch ? c0 + k * L : c0;
          dv[k] = ((const u32x4 *)(a.go + r * I))[c];
          if constexpr (KEPT) {
            const int8_t *p = a.codes + r * 2 * I + c * 8;
            const float *s = a.scales + r * 2 * nb + (c >> 4);
            gc[k] = *(const u32x2 *)p;
            uc[k] = *(const u32x2 *)(p + I);
            gs[k] = s[0];
            us[k] = s[nb];
          } else {
            const uint16_t *p = a.h0 + r * 2 * I + c * 8;
            gv[k] = *(const u32x4 *)p;
            uv[k] = *(const u32x4 *)(p + I);
          }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int c = c0 + k * L;
          if (c >= nch) continue;
          float g[8], u[8], d[8], dg[8], du[8], h[8];
          unpack8(dv[k], d);
          if constexpr (KEPT) {
            unpack_codes(gc[k], gs[k], g);
            unpack_codes(uc[k], us[k], u);
          } else {
            unpack8(gv[k], g);
            unpack8(uv[k], u);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const Logistic s(g[e]);
            const float wd = w * d[e], act = s.s * g[e], hu = act * u[e];
            du[e] = act * wd;
            dg[e] = s.s * u[e] * wd * __builtin_fmaf(g[e], s.rest, 1.0f);
            h[e] = hu * w;
            const float sum = __builtin_fmaf(d[e], hu, dot);
            dot = g[e] < kFar ? dot : sum;
          }
          if (__builtin_expect(far_out(g), 0)) {  // one element after the other: unrolled it takes 126 registers for 84
            f32x8 gx, ux, dx, dgx, dux, hx;
#pragma unroll
            for (int e = 0; e < 8; ++e) gx[e] = g[e], ux[e] = u[e], dx[e] = d[e], dgx[e] = dg[e], dux[e] = du[e], hx[e] = h[e];
#pragma unroll 1
            for (int e = 0; e < 8; ++e) {
              if (gx[e] < kFar) {
                const double s = logistic_far(gx[e]), act = s * gx[e], wd = (double)w * dx[e];
                dux[e] = (float)(act * wd);
                dgx[e] = (float)(s * ux[e] * wd * (1.0 + gx[e]));
                hx[e] = (float)(act * ux[e] * w);
                dot += (float)(act * ux[e] * dx[e]);
              }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) dg[e] = dgx[e], du[e] = dux[e], h[e] = hx[e];
          }
          if (a.gh0) {
            u32x4 *p = (u32x4 *)(a.gh0 + r * 2 * I + c * 8);
            __builtin_nontemporal_store(pack8(dg), p);
            __builtin_nontemporal_store(pack8(du), p + nch);
          }
          if (a.out) __builtin_nontemporal_store(pack8(h), (u32x4 *)(a.out + r * I) + c);
        }
      }
    }
    if (a.gw) {
#pragma unroll
      for (int s = (L < 64 ? L : 64) / 2; s > 0; s >>= 1) dot += __shfl_xor(dot, s);
      if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) red[par][threadIdx.x >> 6] = dot;
        __syncthreads();
        dot = red[par][threadIdx.x / L * W];
#pragma unroll
        for (int v = 1; v < W; ++v) dot += red[par][threadIdx.x / L * W + v];
        par ^= 1;
      }
      if (used && lane == 0) a.gw[r] = dot;
    }
  }
}

hipError_t launch_swiglu(const SwigluArgs &a_, hipStream_t st) {
  SwigluArgs a = a_;
  if (a.rows == 0) return hipSuccess;
  const int nb = (a.I + 127) / 128;
  a.over_nb = 1.0 / nb;
  a.div_nb = div_magic(nb);  // of numbers below nb + 16
  const uint64_t wg = ((uint64_t)a.rows * nb + 15) / 16;
  const dim3 grid((unsigned)(wg < kMostGroups ? wg : kMostGroups)), block(256);
  if (a.codes) hipLaunchKernelGGL((swiglu_kernel<true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((swiglu_kernel<false>), grid, block, 0, st, a);
  return hipGetLastError();
}

template <int L>
static void launch_grad(const SwigluArgs &a, hipStream_t st) {
  const uint64_t wg = ((uint64_t)a.rows + 256 / L - 1) / (256 / L);
  const dim3 grid((unsigned)(wg < kMostGroups ? wg : kMostGroups)), block(256);
  if (a.codes) hipLaunchKernelGGL((swiglu_grad_kernel<L, 2, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((swiglu_grad_kernel<L, 1, false>), grid, block, 0, st, a);
}

// Threads a row: as many as keep each busy, with two chunks from codes (which are half as wide: a wave has too little under
// way with one), with one from bf16.  us, from codes / from bf16, by threads a row:
//                          16           32           64          128          256
//   65536 rows of  256   34 / 37      43 / 37      70 / 48     104 / 74     177 / 126
//   32768 rows of  512   34 / 41      34 / 38      41 / 37      61 / 44      98 / 71
//   30000 rows of 1024   61 / 72      56 / 67      55 / 64      72 / 63     108 / 78
//   32768 rows of 2048  145 / 189    130 / 158    117 / 145    111 / 140    147 / 132
//    6168 rows of 2056   52 / 62      42 / 51      32 / 39      29 / 34      34 / 32
//    8192 rows of 4096   79 / 95      67 / 83      65 / 76      62 / 74      58 / 72
//     100 rows of 8192   42 / 53      25 / 28      14 / 15     8.9 / 9.6    6.2 / 6.7
hipError_t launch_swiglu_grad(const SwigluArgs &a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  const int chunks = a.I / (a.codes ? 16 : 8);
  if (chunks >= 256) launch_grad<256>(a, st);
  else if (chunks >= 128) launch_grad<128>(a, st);
  else if (chunks >= 64) launch_grad<64>(a, st);
  else if (chunks >= 32) launch_grad<32>(a, st);
  else launch_grad<16>(a, st);
  return hipGetLastError();
}

}  // namespace moe
