// experts.hip -- matrix products grouped by expert over ragged rows, on the matrix cores.
//
//   forward  out[r, n] = act( sum_k x[r, k] w[e][n, k] )            m = x rows,        n = w rows
//   dgrad    gx[r, k]  = sum_n go[r, n] w[e][n, k]                  m = go rows,       n = w columns
//   wgrad    gw[e][n, k] = sum_{r of e} go[r, n] x[r, k]            m = go columns,    n = x columns
//
// All three are D[m, n] = sum_k A[m, k] B[n, k] on tiles.  An operand whose k runs along memory
// ("row" operand: 128 bytes of k per stage, 64 bf16, 128 int8 or 256 e2m1) is read from LDS in 16-byte
// pieces; one whose k runs across memory ("column" operand: 64 rows of k per stage, bf16 only) is read
// with the transposing LDS load.  The matrix instructions of all types take 64 bytes of k per row and
// 16 bytes per lane, so one kernel serves them.
#include "experts_internal.hpp"

namespace moe {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) char lds_char;

constexpr uint32_t kOut = 0x80000000u;  // a byte offset past every buffer resource here: reads zero
constexpr int kKB = 128;                // bytes of k per stage of a row operand
constexpr int kKR = 64;                 // rows of k per stage of a column operand

__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const void *p, int64_t bytes) {
  const int n = bytes < 0 ? 0 : bytes > 0x7fffffff ? 0x7fffffff : (int)bytes;
  return __builtin_amdgcn_make_buffer_rsrc((void *)p, (short)0, n, 0x00020000);
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const bf16x2 v = {(__bf16)a, (__bf16)b};  // round to nearest even, NaN stays NaN
  return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + __expf(-g)); }

// chunk permutation of the 16-byte chunks of a stage's rows, so that the lanes of one LDS read fall
// on different banks: row operands are read 16 rows at a time, one chunk of each; column operands
// four rows at a time, on the m side 32 bytes of each, on the n side four pieces of 8 bytes, 32 bytes apart
__device__ __forceinline__ int swz_row(int row) { return row & 7; }
template <bool NSIDE>
__device__ __forceinline__ int swz_col(int k) {
  return NSIDE ? (k & 1) | ((k & 2) << 2) : (k & 3) << 1;
}

template <int TY, int OP, bool GATED, bool F32, int BM, int BN, int WM, int WN>
struct Tile {
  static constexpr int T = 64 * WM * WN;                         // threads
  static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;     // 16 x 16 results of a wave
  static constexpr int CO = GATED ? BN / 2 : BN;                 // result columns
  static constexpr bool MCOL = OP == OP_WGRAD, NCOL = OP != OP_FORWARD;
  static constexpr int ABYTES = BM * kKB, BBYTES = BN * kKB;
  static constexpr int AI = ABYTES / 1024 / (T / 64), BI = BBYTES / 1024 / (T / 64);  // loads of a wave per stage
  static constexpr int E16 = TY == MOE_ROWS_BF16 ? 8 : TY == MOE_ROWS_INT8 ? 16 : 32;  // elements in 16 bytes
  using Acc = typename std::conditional<TY == MOE_ROWS_INT8, i32x4, f32x4>::type;
  static_assert(AI * 1024 * (T / 64) == ABYTES && BI * 1024 * (T / 64) == BBYTES, "whole loads");
};

// the n index (within the tile; for the gate: row of w relative to its half, and the half) of LDS row p
// of the n side.  A wave's FN results of 16 columns are interleaved so that a lane, which holds four
// consecutive columns of each, holds 4 FN consecutive ones in all.
template <class C, bool GATED>
__device__ __forceinline__ int n_of(int p, int &half) {
  constexpr int F = GATED ? C::FN / 2 : C::FN;
  const int b = p / (16 * C::FN), q = p % (16 * C::FN), f = q / 16, r = q % 16;
  half = GATED ? f / F : 0;
  return b * 16 * F + (r / 4) * 4 * F + (f % F) * 4 + (r % 4);
}

template <int TY, int OP, bool GATED, bool F32, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__(64 * WM *WN) experts_kernel(ExpertsArgs a) {
  using C = Tile<TY, OP, GATED, F32, BM, BN, WM, WN>;
  extern __shared__ __align__(1024) char lds[];
  char *la = lds, *lb = lds + C::ABYTES;
  int *first = (int *)(lds + C::ABYTES + C::BBYTES);  // [E + 1] tiles along m before each expert
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / WN, wn = wave % WN;
  const int E = a.g.E;
  const int ntn = (a.N + C::CO - 1) / C::CO;

  if (tid < 64) {  // tiles before each expert, 64 experts at a time
    int base = 0;
    const int most = (int)(a.g.rows / BM) + E;  // what ascending offsets give at most: keeps others in range
    for (int e0 = 0; e0 < E; e0 += 64) {
      int mine = 0;
      if (e0 + lane < E) {
        if (OP == OP_WGRAD) {
          mine = (a.M + BM - 1) / BM;
        } else {
          int64_t lo;
          int n;
          expert_rows(a.g, e0 + lane, lo, n);
          mine = (n + BM - 1) / BM;
        }
      }
      const int incl = wave_inclusive_sum(mine);
      const int before = base + incl - mine;
      if (e0 + lane < E) first[e0 + lane] = OP != OP_WGRAD && before > most ? most : before;
      base += readlane(incl, 63);
      if (OP != OP_WGRAD && base > most) base = most;
    }
    if (lane == 0) first[E] = base;
  }
  __syncthreads();
  const int64_t tiles = (int64_t)first[E] * ntn;

  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int mg = (int)(tile / ntn);
    int e = 0;  // the last expert whose tiles begin at or before mg and that has some
    for (int step = 1024; step > 0; step >>= 1)
      if (e + step < E && first[e + step] <= mg) e += step;
    const int me = first[e + 1] - first[e];
    const int rem = (int)(tile - (int64_t)first[e] * ntn);
    const int nt = rem / me, mt = rem % me;
    int64_t lo;
    int cnt;
    expert_rows(a.g, e, lo, cnt);

    const int m0 = mt * BM, n0 = nt * C::CO;
    const int mlim = OP == OP_WGRAD ? a.M : cnt;  // rows of the result
    const int64_t klen = OP == OP_WGRAD ? cnt : a.K;
    // byte strides of the operands' rows
    const int64_t mrow = (int64_t)(OP == OP_WGRAD ? a.M : a.K) * 16 / C::E16;
    const int64_t nrow = (int64_t)(OP == OP_FORWARD ? a.K : a.N) * 16 / C::E16;
    const int nw = GATED ? 2 * a.N : a.N;  // forward: rows of an expert's weights
    const char *mbase = (const char *)a.m + (OP == OP_WGRAD ? lo * mrow + (int64_t)m0 * 2 : (lo + m0) * mrow);
    const char *nbase = (const char *)a.n + (OP == OP_FORWARD ? ((int64_t)e * nw + n0) * nrow
                                             : OP == OP_DGRAD ? (int64_t)e * a.K * nrow + (int64_t)n0 * 2
                                                              : lo * nrow + (int64_t)n0 * 2);

    typename C::Acc acc[C::FM][C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int j = 0; j < C::FN; ++j) acc[i][j] = typename C::Acc{0, 0, 0, 0};

    const int stages = (int)(C::MCOL || C::NCOL ? (klen + kKR - 1) / kKR : (klen * 16 / C::E16 + kKB - 1) / kKB);
    for (int s = 0; s < stages; ++s) {
      // ---- the stage's operands to LDS, 1 KB a load: lane l's 16 bytes land at l * 16
      const char *mp = mbase + (C::MCOL ? (int64_t)s * kKR * mrow : (int64_t)s * kKB);
      const char *np = nbase + (C::NCOL ? (int64_t)s * kKR * nrow : (int64_t)s * kKB);
      const __amdgpu_buffer_rsrc_t mr = resource(mp, 0x7fffffff);
#pragma unroll
      for (int i = 0; i < C::AI; ++i) {
        const int p = (wave * C::AI + i) * 64 + lane;
        uint32_t off;
        if (C::MCOL) {
          const int k = p / (BM / 8), c = (p % (BM / 8)) ^ swz_col<false>(k);
          off = (int64_t)s * kKR + k < klen && m0 + c * 8 < a.M ? (uint32_t)(k * mrow + c * 16) : kOut;
        } else {
          const int r = p / 8, c = (p % 8) ^ swz_row(r);
          off = m0 + r < cnt && (int64_t)s * kKB + c * 16 < mrow ? (uint32_t)(r * mrow + c * 16) : kOut;
        }
        __builtin_amdgcn_raw_ptr_buffer_load_lds(mr, (lds_char *)(la + (wave * C::AI + i) * 1024), 16, off, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < C::BI; ++i) {
        const int p = (wave * C::BI + i) * 64 + lane;
        uint32_t off;
        if (C::NCOL) {
          const int k = p / (BN / 8), c = (p % (BN / 8)) ^ swz_col<true>(k);
          off = (int64_t)s * kKR + k < klen && n0 + c * 8 < a.N ? (uint32_t)(k * nrow + c * 16) : kOut;
        } else {
          const int r = p / 8, c = (p % 8) ^ swz_row(r);
          int half;
          const int n = n_of<C, GATED>(r, half);
          off = n0 + n < a.N && (int64_t)s * kKB + c * 16 < nrow ? (uint32_t)(n * nrow + c * 16) : kOut;
        }
        // the eight rows of one load are of one half
        const bool up = GATED && ((wave * C::BI + i) * 8 % (16 * C::FN)) / 16 >= C::FN / 2;
        const __amdgpu_buffer_rsrc_t nr = resource(np + (up ? (int64_t)a.N * nrow : 0), 0x7fffffff);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(nr, (lds_char *)(lb + (wave * C::BI + i) * 1024), 16, off, 0, 0, 0);
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();

#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {  // 64 bytes of k: one matrix instruction deep
        i32x4 fa[C::FM], fb[C::FN];
        const int g = lane >> 4, r16 = lane & 15;
#pragma unroll
        for (int i = 0; i < C::FM; ++i) {
          if (C::MCOL) {
            const int m = wm * (BM / WM) + i * 16 + (lane & 3) * 4;
            s16x4 h[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int k = ks * 32 + g * 8 + u * 4 + (r16 >> 2);
              h[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                  (__attribute__((address_space(3))) s16x4 *)(la + k * BM * 2 + (((m >> 3) ^ swz_col<false>(k)) << 4) + (m & 7) * 2));
            }
            fa[i] = __builtin_bit_cast(i32x4, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
          } else {
            const int r = wm * (BM / WM) + i * 16 + r16;
            fa[i] = *(const i32x4 *)(la + r * kKB + (((ks * 4 + g) ^ swz_row(r)) << 4));
          }
        }
#pragma unroll
        for (int j = 0; j < C::FN; ++j) {
          if (C::NCOL) {
            const int n = wn * (BN / WN) + (lane & 3) * 4 * C::FN + j * 4;
            s16x4 h[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int k = ks * 32 + g * 8 + u * 4 + (r16 >> 2);
              h[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                  (__attribute__((address_space(3))) s16x4 *)(lb + k * BN * 2 + (((n >> 3) ^ swz_col<true>(k)) << 4) + (n & 7) * 2));
            }
            fb[j] = __builtin_bit_cast(i32x4, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
          } else {
            const int r = wn * (BN / WN) + j * 16 + r16;
            fb[j] = *(const i32x4 *)(lb + r * kKB + (((ks * 4 + g) ^ swz_row(r)) << 4));
          }
        }
        int sa[C::FM], sb[C::FN];
        if constexpr (TY == MOE_ROWS_MXFP4) {  // the lane's block of 32: one scale byte a row
          const int sw = a.K / 32, blk = s * 8 + ks * 4 + g;
#pragma unroll
          for (int i = 0; i < C::FM; ++i) {
            const int m = m0 + wm * (BM / WM) + i * 16 + r16;
            sa[i] = m < cnt && blk < sw ? ((const uint8_t *)a.ms)[(lo + m) * sw + blk] : 0;
          }
#pragma unroll
          for (int j = 0; j < C::FN; ++j) {
            int half;
            const int n = n0 + n_of<C, GATED>(wn * (BN / WN) + j * 16 + r16, half);
            sb[j] = n < a.N && blk < sw
                        ? ((const uint8_t *)a.ns)[((int64_t)e * nw + n + (GATED && half ? a.N : 0)) * sw + blk]
                        : 0;
          }
        }
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
          for (int j = 0; j < C::FN; ++j) {
            if constexpr (TY == MOE_ROWS_BF16) {
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fb[j]),
                                                                  __builtin_bit_cast(bf16x8, fa[i]), acc[i][j], 0, 0, 0);
            } else if constexpr (TY == MOE_ROWS_INT8) {
              acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
            } else {
              const i32x8 vb = {fb[j][0], fb[j][1], fb[j][2], fb[j][3], 0, 0, 0, 0};
              const i32x8 va = {fa[i][0], fa[i][1], fa[i][2], fa[i][3], 0, 0, 0, 0};
              acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(vb, va, acc[i][j], 4, 4, 0, sb[j], 0, sa[i]);
            }
          }
      }
      __syncthreads();
    }

    // ---- epilogue: lane (g, r16) holds, of result row i * 16 + r16, 4 FN consecutive columns
    constexpr int F = GATED ? C::FN / 2 : C::FN;
    const int g = lane >> 4, r16 = lane & 15;
    const int nl = n0 + wn * 16 * F + g * 4 * F;
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
      const int m = m0 + wm * (BM / WM) + i * 16 + r16;
      if (m >= mlim) continue;
      const float rs = TY == MOE_ROWS_INT8 && a.ms ? ((const float *)a.ms)[lo + m] : 1.0f;
      float v[4 * C::FN];
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float y = (float)acc[i][j][q];
          if constexpr (TY == MOE_ROWS_INT8) {
            const int n = nl + (j % F) * 4 + q;
            if (a.ns && n < a.N) y *= ((const float *)a.ns)[(int64_t)e * nw + n + (j >= F ? a.N : 0)];
            y *= rs;
          }
          v[j * 4 + q] = y;
        }
      if constexpr (GATED) {
#pragma unroll
        for (int q = 0; q < 4 * F; ++q) v[q] = silu(v[q]) * v[4 * F + q];
      }
      const int64_t row = (OP == OP_WGRAD ? (int64_t)e * a.M : lo) + m;
#pragma unroll
      for (int q = 0; q < 4 * F; q += 8) {
        if (nl + q >= a.N) continue;  // N is a multiple of 8
        if constexpr (F32) {
          f32x4 *o = (f32x4 *)((float *)a.out + row * a.N + nl + q);
          o[0] = f32x4{v[q], v[q + 1], v[q + 2], v[q + 3]};
          o[1] = f32x4{v[q + 4], v[q + 5], v[q + 6], v[q + 7]};
        } else {
          *(u32x4 *)((uint16_t *)a.out + row * a.N + nl + q) =
              u32x4{pack2(v[q], v[q + 1]), pack2(v[q + 2], v[q + 3]), pack2(v[q + 4], v[q + 5]), pack2(v[q + 6], v[q + 7])};
        }
      }
    }
  }
}

template <int TY, int OP, bool GATED, bool F32>
static hipError_t launch_tile(const ExpertsArgs &a, hipStream_t st) {
  constexpr int BM = 128, BN = 128, WM = 2, WN = 2;
  using C = Tile<TY, OP, GATED, F32, BM, BN, WM, WN>;
  const int64_t mt = OP == OP_WGRAD ? (int64_t)a.g.E * ((a.M + BM - 1) / BM) : a.g.rows / BM + a.g.E;
  const int64_t tiles = mt * ((a.N + C::CO - 1) / C::CO);
  const size_t lds = C::ABYTES + C::BBYTES + (size_t)(a.g.E + 1) * 4;
  const unsigned grid = (unsigned)(tiles < 1024 ? tiles : 1024);
  hipLaunchKernelGGL((experts_kernel<TY, OP, GATED, F32, BM, BN, WM, WN>), dim3(grid), dim3(C::T), lds, st, a);
  return hipGetLastError();
}

hipError_t launch_experts(const ExpertsArgs &a, int op, int row_type, int act, bool out_fp32, hipStream_t st) {
  if (op != OP_WGRAD && a.g.rows == 0) return hipSuccess;
  if (op == OP_DGRAD) return launch_tile<MOE_ROWS_BF16, OP_DGRAD, false, false>(a, st);
  if (op == OP_WGRAD)
    return out_fp32 ? launch_tile<MOE_ROWS_BF16, OP_WGRAD, false, true>(a, st)
                    : launch_tile<MOE_ROWS_BF16, OP_WGRAD, false, false>(a, st);
  if (act == MOE_ACT_SWIGLU)
    return row_type == MOE_ROWS_BF16   ? launch_tile<MOE_ROWS_BF16, OP_FORWARD, true, false>(a, st)
           : row_type == MOE_ROWS_INT8 ? launch_tile<MOE_ROWS_INT8, OP_FORWARD, true, false>(a, st)
                                       : launch_tile<MOE_ROWS_MXFP4, OP_FORWARD, true, false>(a, st);
  return row_type == MOE_ROWS_BF16   ? launch_tile<MOE_ROWS_BF16, OP_FORWARD, false, false>(a, st)
         : row_type == MOE_ROWS_INT8 ? launch_tile<MOE_ROWS_INT8, OP_FORWARD, false, false>(a, st)
                                     : launch_tile<MOE_ROWS_MXFP4, OP_FORWARD, false, false>(a, st);
}

}  // namespace moe
