// rows_quant.hip -- rows of bf16 to int8 codes with a scale a row, or to microscaled 4-bit floats
// (e2m1 codes, an e8m0 scale per 32 elements).
//
// int8: dyn = fl(127 / amax), code = sat(rne(fl(x dyn))), scale fl(1 / dyn): the dynamic mode of the
// CANN "low_latency_dispatch" page's Formula without smooth scales, as dispatch.hip has it.
// MXFP4: with amax the largest magnitude of 32 elements, s = max(floor(log2 amax) - 2, -127) puts amax
// into [4, 8) 2^s; the e2m1 values are 0, 0.5, 1, 1.5, 2, 3, 4, 6, so x / 2^s (exact: a power of two) is
// rounded to steps of 0.5 below 2, 1 below 4 and 2 above, to nearest with ties to the even code, at most 6.
// One read of x, one write of the codes: bound by memory.
#include "dispatch_dev.hpp"
#include "experts_internal.hpp"

namespace moe {

// whether row r (of all rows the buffers hold) belongs to an expert
__device__ __forceinline__ bool row_used(const RowGroups &g, int64_t r) {
  if (!g.off) return true;
  if (g.stride <= 0) return r >= g.off[0] && r < g.off[g.E];
  const int64_t w = r / g.stride;
  if (w * g.L >= g.E) return false;  // behind the last window
  return r - w * g.stride < (int64_t)g.off[(w + 1) * g.L] - g.off[w * g.L];
}

// the e2m1 code of v (|v| finite)
__device__ __forceinline__ uint32_t e2m1(float v) {
  const float a = fabsf(v);
  const uint32_t sign = (__float_as_uint(v) >> 28) & 8u;
  const float k = a < 2.0f ? 2.0f : a < 4.0f ? 1.0f : 0.5f;
  const float base = a < 2.0f ? 0.0f : a < 4.0f ? 2.0f : 4.0f;
  const float c = fminf(__builtin_rintf(a * k) + base, 7.0f);  // steps of 1 / k: code = a k + base
  return sign | (uint32_t)c;
}

// one workgroup of 256 threads a row
__global__ void __launch_bounds__(256) quant_int8_kernel(RowsQuantArgs a) {
  __shared__ float red[2][16];
  int par = 0;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    if (!row_used(a.g, r)) continue;  // the same for the whole workgroup
    const u32x4 *x = (const u32x4 *)(a.x + r * a.H);
    const int nch = a.H >> 3;
    float m = 0.0f;
    for (int c = threadIdx.x; c < nch; c += 256) {
      float f[8];
      unpack8(x[c], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
    }
    const float amax = block_amax(m, red, par);
    const float dyn = amax > 0.0f ? 127.0f / amax : 0.0f;
    if (threadIdx.x == 0) ((float *)a.scales)[r] = amax > 0.0f ? 1.0f / dyn : 0.0f;
    u32x2 *q = (u32x2 *)((int8_t *)a.codes + r * a.H);
    for (int c = threadIdx.x; c < nch; c += 256) {
      float f[8];
      unpack8(x[c], f);
      int cd[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) cd[e] = sat_code(f[e] * dyn);
      q[c] = u32x2{pack_i8x4(cd[0], cd[1], cd[2], cd[3]), pack_i8x4(cd[4], cd[5], cd[6], cd[7])};
    }
  }
}

// one thread per block of 32 elements
__global__ void __launch_bounds__(256) quant_mxfp4_kernel(RowsQuantArgs a) {
  const int nb = a.H >> 5;
  const int64_t blocks = a.rows * nb;
  for (int64_t b = (int64_t)blockIdx.x * 256 + threadIdx.x; b < blocks; b += (int64_t)gridDim.x * 256) {
    if (!row_used(a.g, b / nb)) continue;
    const u32x4 *x = (const u32x4 *)(a.x + b * 32);
    uint32_t top = 0;  // the largest magnitude's bits: bf16 magnitudes order as integers
    u32x4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = x[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = v[i][j] & 0x7fffu, hi = (v[i][j] >> 16) & 0x7fffu;
        top = top > lo ? top : lo;
        top = top > hi ? top : hi;
      }
    }
    u32x4 out = u32x4{0u, 0u, 0u, 0u};
    uint32_t s;
    if (top >= 0x7f80u) {  // an infinity or a NaN
      s = 255u;
    } else {
      // the exponent field of amax is floor(log2) + 127 (0 for subnormals, whose scale is the smallest anyway)
      s = (top >> 7) > 2u ? (top >> 7) - 2u : 0u;
      const float inv = __uint_as_float((254u - s) << 23);  // 2^(127 - s), s <= 252: a normal number
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float f[8];
        unpack8(v[i], f);
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) w |= e2m1(f[e] * inv) << (4 * e);
        out[i] = w;
      }
    }
    ((u32x4 *)a.codes)[b] = out;
    ((uint8_t *)a.scales)[b] = (uint8_t)s;
  }
}

hipError_t launch_rows_quant(const RowsQuantArgs &a, int row_type, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  if (row_type == MOE_ROWS_INT8) {
    const unsigned grid = (unsigned)(a.rows < (1 << 20) ? a.rows : (1 << 20));
    hipLaunchKernelGGL(quant_int8_kernel, dim3(grid), dim3(256), 0, st, a);
  } else {
    const int64_t wg = (a.rows * (a.H >> 5) + 255) / 256;
    hipLaunchKernelGGL(quant_mxfp4_kernel, dim3((unsigned)(wg < (1 << 20) ? wg : (1 << 20))), dim3(256), 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace moe
