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

// the e2m1 code of v (|v| finite)
__device__ __forceinline__ uint32_t e2m1(float v) {
  const float a = fabsf(v);
  const uint32_t sign = (__float_as_uint(v) >> 28) & 8u;
  const float k = a < 2.0f ? 2.0f : a < 4.0f ? 1.0f : 0.5f;
  const float base = a < 2.0f ? 0.0f : a < 4.0f ? 2.0f : 4.0f;
  const float c = fminf(__builtin_rintf(a * k) + base, 7.0f);  // steps of 1 / k: code = a k + base
  return sign | (uint32_t)c;
}

// int8.  A row is held in registers between the search for its amax and the rounding: 64 W threads a row, NC
// chunks of 8 elements a thread; four rows (W = 1) or one (W = 4) a workgroup.  NC = 0: the row is read twice.
// 6168 rows of 2064 in 10 us (3.8 TB/s), 8192 of 7168 in 33 us (5.3).
template <int W, int NC>
__global__ void __launch_bounds__(256) quant_int8_kernel(RowsQuantArgs a) {
  __shared__ float red[2][16];
  int par = 0;
  const int t = threadIdx.x % (64 * W), nch = a.H >> 3;
  constexpr int R = 4 / W;
  for (int64_t r = (int64_t)blockIdx.x * R + threadIdx.x / (64 * W); r < a.rows; r += (int64_t)gridDim.x * R) {
    if (!row_used(a.g, r)) continue;  // the same for all threads of the row
    const u32x4 *x = (const u32x4 *)(a.x + r * a.H);
    u32x2 *q = (u32x2 *)((int8_t *)a.codes + r * a.H);
    u32x4 v[NC ? NC : 1];
    float m = 0.0f;
    auto top = [&](const u32x4 &c) {
      float f[8];
      unpack8(c, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
    };
    auto put = [&](int c, const u32x4 &w, float dyn) {
      float f[8];
      unpack8(w, f);
      int cd[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) cd[e] = sat_code(f[e] * dyn);
      q[c] = u32x2{pack_i8x4(cd[0], cd[1], cd[2], cd[3]), pack_i8x4(cd[4], cd[5], cd[6], cd[7])};
    };
    if constexpr (NC > 0) {
#pragma unroll
      for (int i = 0; i < NC; ++i) v[i] = t + i * 64 * W < nch ? x[t + i * 64 * W] : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < NC; ++i) top(v[i]);
    } else {
      for (int c = t; c < nch; c += 64 * W) top(x[c]);
    }
    const float amax = W == 1 ? wave_max(m) : block_amax(m, red, par);
    const float dyn = amax > 0.0f ? 127.0f / amax : 0.0f;
    if (t == 0) ((float *)a.scales)[r] = amax > 0.0f ? 1.0f / dyn : 0.0f;
    if constexpr (NC > 0) {
#pragma unroll
      for (int i = 0; i < NC; ++i)
        if (t + i * 64 * W < nch) put(t + i * 64 * W, v[i], dyn);
    } else {
      for (int c = t; c < nch; c += 64 * W) put(c, x[c], dyn);
    }
  }
}

// a thread's 8 of 32 elements: the codes; s: the scale byte of the 32.  Four neighbouring lanes hold a block.
__device__ __forceinline__ uint32_t mx_codes(const u32x4 &v, uint32_t &s) {
  int top = 0;  // the largest magnitude's bits: bf16 magnitudes order as integers
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int lo = v[j] & 0x7fff, hi = (v[j] >> 16) & 0x7fff;
    top = max(top, max(lo, hi));
  }
  top = max(top, __builtin_amdgcn_update_dpp(0, top, 0xb1, 0xf, 0xf, false));  // quad_perm 1 0 3 2
  top = max(top, __builtin_amdgcn_update_dpp(0, top, 0x4e, 0xf, 0xf, false));  // quad_perm 2 3 0 1
  // the exponent field of amax is floor(log2) + 127 (0 for subnormals, whose scale is the smallest anyway)
  s = (top >> 7) > 2 ? (top >> 7) - 2 : 0;
  const float inv = __uint_as_float((254u - s) << 23);  // 2^(127 - s), s <= 253: a normal number
  float f[8];
  unpack8(v, f);
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) w |= e2m1(f[e] * inv) << (4 * e);
  if (top >= 0x7f80) {  // an infinity or a NaN
    s = 255;
    w = 0;
  }
  return w;
}

// MXFP4: a thread takes 16 bytes, 8 elements, so that a wave reads 1 KB and writes 256 bytes at once; four loads
// under way a thread.  32768 rows of 4096 in 68 to 72 us (4.7 to 5.0 TB/s; a large copy reaches 4.9).
constexpr int kMxLoads = 4;
__global__ void __launch_bounds__(256) quant_mxfp4_kernel(RowsQuantArgs a) {
  const int64_t n = a.rows * (a.H >> 3), step = (int64_t)gridDim.x * 256 * kMxLoads;
  for (int64_t first = (int64_t)blockIdx.x * 256 * kMxLoads + threadIdx.x; first - threadIdx.x < n; first += step) {
    u32x4 v[kMxLoads];
#pragma unroll
    for (int i = 0; i < kMxLoads; ++i) {
      const int64_t c = first + i * 256;
      v[i] = c < n ? ((const u32x4 *)a.x)[c] : u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int i = 0; i < kMxLoads; ++i) {
      const int64_t c = first + i * 256;
      uint32_t s;
      const uint32_t w = mx_codes(v[i], s);
      if (c < n) {
        ((uint32_t *)a.codes)[c] = w;
        if ((threadIdx.x & 3) == 0) ((uint8_t *)a.scales)[c >> 2] = (uint8_t)s;
      }
    }
  }
}

// the same for the rows of experts, of which some are not to be touched: a workgroup a row (taken for all rows: 76 us)
__global__ void __launch_bounds__(256) quant_mxfp4_rows_kernel(RowsQuantArgs a) {
  const int nch = a.H >> 3;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    if (!row_used(a.g, r)) continue;
    for (int c = threadIdx.x; c < nch; c += 256) {  // nch is a multiple of 4: a block's lanes go together
      uint32_t s;
      const uint32_t w = mx_codes(((const u32x4 *)(a.x + r * a.H))[c], s);
      ((uint32_t *)a.codes)[r * nch + c] = w;
      if ((c & 3) == 0) ((uint8_t *)a.scales)[(r * nch + c) >> 2] = (uint8_t)s;
    }
  }
}

template <int W, int NC>
static void launch_int8(const RowsQuantArgs &a, hipStream_t st) {
  const int64_t wg = (a.rows + 4 / W - 1) / (4 / W);
  hipLaunchKernelGGL((quant_int8_kernel<W, NC>), dim3((unsigned)(wg < (1 << 20) ? wg : (1 << 20))), dim3(256), 0, st, a);
}

hipError_t launch_rows_quant(const RowsQuantArgs &a, int row_type, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  if (row_type == MOE_ROWS_INT8) {
    // 8192 rows, us, by <W, NC>: of 1024 6.8 <1, 2>, 8.0 <1, 8>, 12.3 <4, 4>; of 4096 18.0 <1, 8>, 18.2 <4, 4>,
    // 20.2 <4, 0>; of 7168 33.4 <4, 4>, 39.7 <4, 0>; of 16384 103 <4, 0>, 125 <1, 0>
    if (a.H <= 1024) launch_int8<1, 2>(a, st);
    else if (a.H <= 4096) launch_int8<1, 8>(a, st);
    else if (a.H <= 8192) launch_int8<4, 4>(a, st);
    else launch_int8<4, 0>(a, st);
  } else if (a.g.off) {
    hipLaunchKernelGGL(quant_mxfp4_rows_kernel, dim3((unsigned)(a.rows < (1 << 20) ? a.rows : (1 << 20))), dim3(256), 0, st, a);
  } else {
    const int64_t wg = (a.rows * (a.H >> 3) + 256 * kMxLoads - 1) / (256 * kMxLoads);
    hipLaunchKernelGGL(quant_mxfp4_kernel, dim3((unsigned)(wg < (1 << 20) ? wg : (1 << 20))), dim3(256), 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace moe
