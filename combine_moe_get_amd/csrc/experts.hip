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
//
// A workgroup is persistent: it keeps a ring of stages in LDS filled by loads that go past the registers, and multiplies
// one stage's operands while the next one's come from LDS, on to the next tile without a pause where the ring allows it.
// Bounds: few rows an expert, the weights from memory (8 rows of 8 of 64 experts, 4096 -> 2 x 1024 bf16, 134 MB: 24.9 us,
// 5.4 TB/s; 128 rows over 64, 7168 -> 2 x 2048 in 4 bits, 883 MB with the scales: 156 us, 5.7 TB/s).  Many rows: a stage
// of a 256 x 256 tile is 2048 cycles of matrix instructions on each SIMD and 2048 of LDS (64 KB in, 192 KB out, 128 bytes
// a cycle), which do not overlap wholly: 1.72 us, at the 1.95 GHz of such a load 3350.  16 x 2048 rows of 4096 -> 4096
// 840 to 870 us, 1.26 to 1.31 PFLOP/s (torch's plain product of 8192: 1.37, of 16384: 1.61); int8 465 us, 2.4 POP/s,
// 4 bits 307 us, 3.6 PFLOP/s; the gradients 830 and 901.
#include "experts_internal.hpp"

namespace moe {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) char lds_char;

constexpr int kKB = 128;                // bytes of k per stage of a row operand
constexpr int kKR = 64;                 // rows of k per stage of a column operand
constexpr uint32_t kOut = 0x80000000u;  // a byte offset past every buffer resource here: reads zero

// a raw buffer resource of `bytes` bytes (at most 2^31 - 1) at a wave-uniform address; the address has 48 bits
__device__ __forceinline__ i32x4 resource(const void *p, int64_t bytes) {
  const uint64_t u = (uint64_t)(uintptr_t)p;
  const int n = bytes < 0 ? 0 : bytes > 0x7fffffff ? 0x7fffffff : (int)bytes;
  return i32x4{__builtin_amdgcn_readfirstlane((int)(uint32_t)u), __builtin_amdgcn_readfirstlane((int)(u >> 32) & 0xffff),
               __builtin_amdgcn_readfirstlane(n), 0x00020000};
}

// 64 lanes x 16 bytes from `off` + `soff` past the resource's base (behind its end: zeros) to LDS at `at` + `more` +
// lane * 16; all but `off` wave-uniform.  Asm, because for its own loads into LDS the compiler waits before every
// LDS read that it cannot prove disjoint, which here is each: stage_wait() waits instead.  No vector register is written; M0 is,
// which the unused result tells the compiler.
// The wait states that a memory instruction needs are the statement's own, as the compiler does not see one in it: five
// after a vector instruction's write of a scalar register that it reads (the readfirstlanes of resource(), or of an
// operand here), the addition and four idle ones; M0 is good for it after one.
__device__ __forceinline__ void load_to_lds(i32x4 d, uint32_t off, uint32_t soff, uint32_t at, uint32_t more) {
  [[maybe_unused]] int m0;
  asm volatile("s_add_u32 m0, %4, %5\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               : "={m0}"(m0)
               : "v"(off), "s"(d), "s"(soff), "s"(at), "i"(more)
               : "memory", "scc");
}

// until at most N of the wave's loads are under way and its LDS reads are done, then until every wave is there
template <int N>
__device__ __forceinline__ void stage_wait() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// f(0), .., f(N - 1) with the index as a constant
template <int I, int N, class F>
__device__ __forceinline__ void static_for_from(F &&f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for_from<I + 1, N>(f);
  }
}
template <int N, class F>
__device__ __forceinline__ void static_for(F &&f) {
  static_for_from<0, N>(f);
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const bf16x2 v = {(__bf16)a, (__bf16)b};  // round to nearest even, NaN stays NaN
  return __builtin_bit_cast(uint32_t, v);
}

// silu(g) u = g u / (1 + exp(-g)) = (g h) u h / (1 + h h), h = exp(g / 2).  What is too small for fp32 in exp(g), from
// about -87 on, is never alone, so that the product keeps its digits as long as it is itself in range; h is the square of
// exp(g / 4), which the instruction, that gives no subnormals, has down to -349.  Above 17 the divisor is h h to fp32:
// h stays there.  The exponential of a rounded argument, its two squares and the reciprocal are good to about |g| + 8
// steps of fp32, far below the bf16 rounding that follows.  (Four instructions more than with 1 / (1 + exp(-g)), which
// gives 0 below -87: 2 to 3% of the time of 32768 rows, 4096 -> 2 x 2048 in 4 bits.  Choosing by the wave's least g spills.)
constexpr float kLog2e = 1.44269504088896341f;
__device__ __forceinline__ float silu_times(float g, float u) {
  const float q = __builtin_amdgcn_exp2f(fminf(g * (0.25f * kLog2e), 17.0f * 0.25f * kLog2e)), h = q * q;
  return g * h * __builtin_amdgcn_rcpf(__builtin_fmaf(h, h, 1.0f)) * u * h;
}

// Permutation (an XOR of the index) of the 16-byte chunks of a stage's LDS rows, so that the lanes that one
// cycle serves (128 bytes) fall on different banks.
// Row operands: one chunk of each of 8 rows of 128 bytes.
__device__ __forceinline__ int swz_row(int row) { return row & 7; }
// Column operands: four rows of k (k & 3), 32 bytes of each, or on the n side with G = 2 (see n_of) four pieces of
// 8 bytes, a chunk apart.
template <int G>
__device__ __forceinline__ int swz_col(int k) {
  return (k & 3) << G;
}

// TY: row type; BM x BN: the tile (with the gate: BN / 2 columns of the result); WM x WN: its waves;
// NST: stages in LDS; WIDE: MXFP4 scales of a row begin at multiples of four bytes
template <int TY, int OP, bool GATED, bool F32, int BM, int BN, int WM, int WN, int NST, bool WIDE>
struct Tile {
  static constexpr int W = WM * WN, T = 64 * W;               // waves, threads
  static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;  // 16 x 16 results of a wave
  static constexpr int CO = GATED ? BN / 2 : BN;              // result columns
  // 16-column results of a wave per half; and how many of them are interleaved, so that a lane, which holds four
  // consecutive columns of each, stores 16 bytes and four lanes 64 in a row (see n_of)
  static constexpr int F = GATED ? FN / 2 : FN, G = F32 || F < 2 ? 1 : 2;
  static constexpr bool MCOL = OP == OP_WGRAD, NCOL = OP != OP_FORWARD, MX = TY == MOE_ROWS_MXFP4;
  static constexpr int ABYTES = BM * kKB, BBYTES = BN * kKB, STAGE = ABYTES + BBYTES;
  static constexpr int AI = ABYTES / 1024 / W, BI = BBYTES / 1024 / W;  // loads of a wave per stage
  // MXFP4 scales: 16 bytes a row at once, for two stages (PAIR) or for one of them, in as many buffers; a wave's loads
  static constexpr bool PAIR = MX && WIDE && NST == 2;
  static constexpr int SI = MX ? ((BM + BN) / 64 + W - 1) / W : 0, SBYTES = SI * W * 1024;
  static constexpr int LDS = NST * (STAGE + SBYTES);
  static constexpr int E16 = TY == MOE_ROWS_BF16 ? 8 : TY == MOE_ROWS_INT8 ? 16 : 32;  // elements in 16 bytes
  using Acc = typename std::conditional<TY == MOE_ROWS_INT8, i32x4, f32x4>::type;
  static_assert(AI * 1024 * W == ABYTES && BI * 1024 * W == BBYTES, "whole loads");
  // with the gate: halves of w that the rows of a wave's loads are of
  static constexpr int HALVES = GATED && BI > FN ? 2 : 1;
  static_assert(!GATED || FN % BI == 0 || BI == 2 * FN, "a load is of one half");
  static_assert((!MCOL || BM >= 64) && (!NCOL || BN >= 128), "swz_col stays within a row");
  static_assert(F % G == 0 && (!GATED || FN % 2 == 0), "whole groups of results");
  static_assert(!MX || BM % 64 == 0, "a load of scales is of one side");
};

// the n index (within the tile; for the gate: row of w relative to its half, and the half) of LDS row p of the n side:
// of row r of result f of a wave, results interleaved by G
template <class C>
__device__ __forceinline__ int n_of(int p, int &half) {
  const int b = p / (16 * C::FN), q = p % (16 * C::FN), f = q / 16 % C::F, r = q % 16;
  half = q / 16 / C::F;
  return b * 16 * C::F + f / C::G * 16 * C::G + r / 4 * 4 * C::G + f % C::G * 4 + r % 4;
}

#define LAMBDA __attribute__((always_inline))

template <int TY, int OP, bool GATED, bool F32, int BM, int BN, int WM, int WN, int NST, bool RING, bool WIDE>
__global__ void __launch_bounds__(64 * WM *WN, 2) experts_kernel(ExpertsArgs a) {
  using C = Tile<TY, OP, GATED, F32, BM, BN, WM, WN, NST, WIDE>;
  constexpr bool MX = C::MX;
  // Tiles along m that are walked together, by an XCD's 32 workgroups: 8 with 4 along n; in wgrad, where an XCD has a
  // piece of an expert's tiles, 4 with as many along n (64 x 1000 rows, 1024 -> 7168: 943 us, with 8 951).
  constexpr int kGroup = OP == OP_WGRAD ? 4 : 8;
  extern __shared__ __align__(1024) char lds[];
  int *first = (int *)(lds + C::LDS);  // [E + 1] tiles along m before each expert
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int E = a.g.E;
  const int ntn = (a.N + C::CO - 1) / C::CO;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_char *)lds;

  const int lane = tid & 63;
  const int wmt = (a.M + BM - 1) / BM;  // wgrad: tiles along m of every expert
  if (OP != OP_WGRAD) {
    if (tid < 64) {  // tiles before each expert, 64 experts at a time
      int base = 0;
      const int most = (int)(a.g.rows / BM) + E;  // what ascending offsets give at most: keeps others in range
      for (int e0 = 0; e0 < E; e0 += 64) {
        int mine = 0;
        if (e0 + lane < E) {
          int64_t lo;
          int n;
          expert_rows(a.g, e0 + lane, lo, n);
          mine = (n + BM - 1) / BM;
        }
        const int incl = wave_inclusive_sum(mine);
        const int before = base + incl - mine;
        if (e0 + lane < E) first[e0 + lane] = before > most ? most : before;
        base += readlane(incl, 63);
        if (base > most) base = most;
      }
      if (lane == 0) first[E] = base;
    }
    __syncthreads();
  }

  // Workgroups go round the 8 XCDs, each with an L2 of its own: an XCD's workgroups take neighbouring tiles, so that
  // those that run together share operands in that L2.  Forward and dgrad: XCD x takes the x-th eighth of all tiles.
  // wgrad, where a tile costs what its expert has rows: an eighth of each expert's, of expert e the (x + e)-th, so that
  // every eight experts give an XCD as many tiles as one expert has.
  const uint32_t xcd = blockIdx.x & 7, per = (gridDim.x + 7 - xcd) >> 3;  // its workgroups
  const uint32_t each = (uint32_t)wmt * (uint32_t)ntn;                    // wgrad: tiles of an expert
  auto eighth = [&](uint32_t i) LAMBDA { return each * (i & 7) / 8; };    // the first tile of an eighth; each < 2^21
  uint32_t round = 0, last;                                               // fits: see launch_cfg
  if (OP == OP_WGRAD) {
    last = (uint32_t)E / 8 * each;
    for (uint32_t i = xcd; i < xcd + E % 8; ++i) last += ((i & 7) == 7 ? each : eighth(i + 1)) - eighth(i);
  } else {
    const uint64_t tiles = (uint64_t)(uint32_t)first[E] * (uint32_t)ntn;
    round = (uint32_t)(tiles * xcd / 8);
    last = (uint32_t)(tiles * (xcd + 1) / 8);
  }
  // In each round the workgroups' places are turned, so that an expert's last, short tile along m meets others.
  constexpr uint32_t kTurn = 13;
  uint32_t place = blockIdx.x >> 3, tile = round + place;
  if (tile >= last) return;

  // byte strides of the operands' rows
  const int64_t mrow = (int64_t)(OP == OP_WGRAD ? a.M : a.K) * 16 / C::E16;
  const int64_t nrow = (int64_t)(OP == OP_FORWARD ? a.K : a.N) * 16 / C::E16;
  const int nw = GATED ? 2 * a.N : a.N;  // forward: rows of an expert's weights
  const int sw = a.K / 32;               // MXFP4: scales of a row

  const int c16 = ((lane & 7) ^ swz_row(lane >> 3)) * 16;  // row operands: the lane's 16 of a load's 8 x 128 bytes

  // ---- the tile whose stages are being loaded
  int e, cnt, m0, n0, stages;
  int64_t lo, klen;
  const char *mbase, *nbase;
  // A load of 1 KB takes 8 LDS rows of a row operand, or 512 / R rows of k of a column operand with rows of R
  // columns.  Byte offsets of the lane's 16 bytes, the same in all stages:
  uint32_t ao[C::AI], bo[C::BI], so[MX ? C::SI : 1];
  const char *sbase[MX ? C::SI : 1];  // MXFP4 scales: of the operand of the wave's load, and their bytes
  int sbytes[MX ? C::SI : 1], mshift = 0, nshift = 0;
  i32x4 mres, nres[C::HALVES];  // row operands: over the tile's rows
  auto enter = [&]() LAMBDA {
    int me;
    uint32_t rem;  // the expert's tiles along m, and which of its tiles this is
    if (OP == OP_WGRAD) {
      me = wmt;
      e = (int)(tile / each) * 8;
      rem = tile - tile / each * each;  // among the eight experts' eighths: fewer than `each` tiles in all
      for (uint32_t i = xcd;; ++i, ++e) {
        const uint32_t from = eighth(i), n = ((i & 7) == 7 ? each : eighth(i + 1)) - from;
        if (rem < n) {
          rem += from;
          break;
        }
        rem -= n;
      }
    } else {
      // the last expert whose tiles begin at or before mg (it has some): 64 experts compared at once
      const uint32_t mg = tile / (uint32_t)ntn;
      const int step = (E + 63) / 64;
      const int blk = __builtin_popcountll(ballot(lane * step < E && first[lane * step] <= (int)mg)) - 1;
      const int x = blk * step + lane;
      e = blk * step + __builtin_popcountll(ballot(lane < step && x < E && first[x] <= (int)mg)) - 1;
      const int before = __builtin_amdgcn_readfirstlane(first[e]);
      me = __builtin_amdgcn_readfirstlane(first[e + 1]) - before;
      rem = tile - (uint32_t)before * ntn;
    }
    // the expert's tiles in groups of up to kGroup along m, in each along m first
    const uint32_t grp = rem / (uint32_t)(kGroup * ntn), in = rem - grp * kGroup * ntn;
    const uint32_t gm = me - grp * kGroup < kGroup ? me - grp * kGroup : kGroup, nt = in / gm;
    expert_rows(a.g, e, lo, cnt);
    m0 = (int)(grp * kGroup + in - nt * gm) * BM;
    n0 = (int)nt * C::CO;
    klen = OP == OP_WGRAD ? cnt : a.K;
    mbase = (const char *)a.m + (OP == OP_WGRAD ? lo * mrow + (int64_t)m0 * 2 : (lo + m0) * mrow);
    nbase = (const char *)a.n + (OP == OP_FORWARD ? ((int64_t)e * nw + n0) * nrow
                                 : OP == OP_DGRAD ? (int64_t)e * a.K * nrow + (int64_t)n0 * 2
                                                  : lo * nrow + (int64_t)n0 * 2);
    stages = (int)(C::MCOL || C::NCOL ? (klen + kKR - 1) / kKR : (klen * 16 / C::E16 + kKB - 1) / kKB);
#pragma unroll
    for (int i = 0; i < C::AI; ++i) {
      const int p = (wave * C::AI + i) * 64 + lane;
      if (C::MCOL) {
        const int k = p / (BM / 8), c = (p % (BM / 8)) ^ swz_col<1>(k);
        ao[i] = m0 + c * 8 < a.M ? (uint32_t)(k * (int)mrow + c * 16) : kOut;
      } else {
        ao[i] = m0 + p / 8 < cnt ? (uint32_t)(p / 8 * (int)mrow + c16) : kOut;
      }
    }
#pragma unroll
    for (int i = 0; i < C::BI; ++i) {
      const int p = (wave * C::BI + i) * 64 + lane;
      if (C::NCOL) {
        const int k = p / (BN / 8), c = (p % (BN / 8)) ^ swz_col<C::G>(k);
        bo[i] = n0 + c * 8 < a.N ? (uint32_t)(k * (int)nrow + c * 16) : kOut;
      } else {
        int half;
        const int n = n_of<C>(p / 8, half);
        bo[i] = n0 + n < a.N ? (uint32_t)(n * (int)nrow + c16) : kOut;
      }
    }
    if (!C::MCOL) mres = resource(mbase, 0x7fffffff);
    if (!C::NCOL) {
      const bool up = GATED && wave * C::BI * 8 % (16 * C::FN) >= 8 * C::FN;  // HALVES 1: the wave's half
#pragma unroll
      for (int h = 0; h < C::HALVES; ++h) nres[h] = resource(nbase + (up || h ? (int64_t)a.N * nrow : 0), 0x7fffffff);
    }
    if constexpr (MX) {
#pragma unroll
      for (int i = 0; i < C::SI; ++i) {  // LDS rows of scales: the m side's, then the n side's
        const int p = (wave * C::SI + i) * 64 + lane;
        const bool mside = (wave * C::SI + i) * 64 < BM;
        const char *from = mside ? (const char *)a.ms + (lo + m0) * sw : (const char *)a.ns + ((int64_t)e * nw + n0) * sw;
        // whole words: up to three bytes before the first row's and behind the last's are read with theirs
        const int off = WIDE ? 0 : (int)((uintptr_t)from & 3);
        sbase[i] = from - off;
        const int64_t bytes = ((int64_t)(mside ? cnt - m0 : nw - n0) * sw + off + 3) & ~(int64_t)3;
        sbytes[i] = (int)(bytes < 0x7ffffff0 ? bytes : 0x7ffffff0);
        if (p < BM) {
          so[i] = m0 + p < cnt ? (uint32_t)(p * sw + off) & ~3u : kOut;
        } else if (p < BM + BN) {
          int half;
          const int n = n_of<C>(p - BM, half);
          so[i] = n0 + n < a.N ? (uint32_t)((n + (GATED && half ? a.N : 0)) * sw + off) & ~3u : kOut;
        } else {
          so[i] = kOut;
        }
      }
      if constexpr (!WIDE) {  // where in its 16 bytes the lane's row begins: the rows of a lane differ by multiples of four
        const int r = lane & 15;
        mshift = (int)((uintptr_t)a.ms + (lo + m0) * sw + r * sw) & 3;
        nshift = (int)((uintptr_t)a.ns + ((int64_t)e * nw + n0) * sw + r * sw) & 3;
      }
    }
  };
  // load l (of AI + BI) of stage s into buffer b; past the last stage zeros, so that every stage counts the same
  // loads
  constexpr int LOADS = C::AI + C::BI;
  const uint32_t mlds = lds0 + wave * C::AI * 1024, nlds = lds0 + NST * C::ABYTES + wave * C::BI * 1024;
  auto issue = [&](int s, auto b_, auto l_) LAMBDA {
    constexpr int b = decltype(b_)::value, l = decltype(l_)::value;
    constexpr bool mside = l < C::AI;
    constexpr int i = mside ? l : l - C::AI;
    constexpr uint32_t more = (mside ? b * C::ABYTES : b * C::BBYTES) + i * 1024;
    const int64_t row = mside ? mrow : nrow;
    uint32_t o;
    if constexpr (mside) o = ao[i];
    else o = bo[i];
    if constexpr (mside ? C::MCOL : C::NCOL) {  // rows of k past the last are outside of the resource
      const int64_t k = (int64_t)s * kKR, bytes = (klen - k) * row - (int64_t)(mside ? m0 : n0) * 2;
      load_to_lds(resource((mside ? mbase : nbase) + k * row, bytes), o, 0, mside ? mlds : nlds, more);
    } else {  // a piece that begins behind its row's end is not read
      load_to_lds(mside ? mres : nres[C::HALVES == 2 ? i / C::FN : 0], c16 < (int)row - s * kKB ? o : kOut, s * kKB,
                  mside ? mlds : nlds, more);
    }
  };
  // MXFP4 scales, 16 bytes a row at once.  PAIR: of stages 2 u and 2 u + 1, into the other of the two buffers.
  // Otherwise of stage u into buffer b, 8 bytes and what lies around them: rows of scales that begin at any byte
  // (not WIDE) are read from the multiple of four before.  Either way pieces may run on into the next row's
  // scales: see scale_pair.
  int sbuf = 1;
  auto issue_scales = [&](int u, int b) LAMBDA {
#pragma unroll
    for (int i = 0; i < C::SI; ++i) {
      const int from = u * (C::PAIR ? 16 : 8), to = C::PAIR ? sbuf ^ 1 : b;
      load_to_lds(resource(sbase[i] + from, from < sw ? sbytes[i] - from : 0), so[i], 0,
                  lds0 + NST * C::STAGE + to * C::SBYTES + (wave * C::SI + i) * 1024, 0);
    }
  };

  // ---- the lane's part of 16 rows and 64 bytes of k (one matrix instruction deep) of a stage in buffer b:
  // lane group g has the 16-byte piece 2 g + ks of the stage's 8
  const int g = lane >> 4, r16 = lane & 15;
  // LDS holds the m side's NST buffers, then the n side's (so that within one an offset fits the instruction), then
  // the scales.  Addresses in buffer 0; the rest of a piece's address is constant (an XOR with a constant for columns).
  // The empty asm statement keeps them in registers as they are.
  const int mfirst = wm * (BM / WM), nfirst = wn * (BN / WN), kt = g * 16 + (r16 >> 2);
  uint32_t ma[2], na[2];
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    // rows: of piece ks; swz_row is the same in every sixteenth row
    const uint32_t piece = r16 * kKB + (((g * 2 + ks) ^ swz_row(r16)) << 4);
    ma[ks] = lds0 + mfirst * kKB + piece;
    na[ks] = lds0 + NST * C::ABYTES + nfirst * kKB + piece;
  }
  // columns: swz_col looks only at bits of k that ks and u leave alone
  if (C::MCOL) ma[0] = lds0 + kt * BM * 2 + ((((mfirst + (lane & 3) * 4) >> 3) ^ swz_col<1>(kt)) << 4) + (lane & 1) * 8;
  if (C::NCOL) na[0] = lds0 + NST * C::ABYTES + kt * BN * 2 + (((nfirst + (lane & 3) * 4 * C::G) >> 3 ^ swz_col<C::G>(kt)) << 4) + (C::G == 1 ? (lane & 1) * 8 : 0);
  uint32_t sm = lds0 + NST * C::STAGE + (mfirst + r16) * 16 + g * 2, sn = sm + (BM + nfirst - mfirst) * 16;  // scales
  asm volatile("" : "+v"(ma[0]), "+v"(ma[1]), "+v"(na[0]), "+v"(na[1]), "+v"(sm), "+v"(sn));
  auto column = [&](uint32_t at, int R) LAMBDA {  // 8 rows of k, four columns of each
    s16x4 h[2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
      h[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(uintptr_t)(at + u * 4 * R * 2));
    return __builtin_bit_cast(i32x4, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto read_m = [&](int b, int i, int ks) LAMBDA -> i32x4 {
    if (C::MCOL) return column((ma[0] ^ (i << 5)) + b * C::ABYTES + ks * 8 * BM * 2, BM);
    return *(__attribute__((address_space(3))) const i32x4 *)(uintptr_t)(ma[ks] + b * C::ABYTES + i * 16 * kKB);
  };
  auto read_n = [&](int b, int j, int ks) LAMBDA -> i32x4 {
    if (C::NCOL)
      return column((na[0] ^ ((j / C::G) << (4 + C::G))) + j % C::G * 8 + b * C::BBYTES + ks * 8 * BN * 2, BN);
    return *(__attribute__((address_space(3))) const i32x4 *)(uintptr_t)(na[ks] + b * C::BBYTES + j * 16 * kKB);
  };
  // MXFP4: the scale bytes of the lane's two pieces of stage s (even: b = 0), of two rows in one register
  constexpr int SM = MX ? (C::FM + 1) / 2 : 1, SN = MX ? (C::FN + 1) / 2 : 1;
  uint32_t sa[SM], sb[SN];
  auto scale_pair = [&](uint32_t p, int s, int b, int i, int n, int shift) LAMBDA -> uint32_t {
    typedef uint16_t __attribute__((aligned(1))) u16_any;
    auto two = [](uint32_t x) LAMBDA -> uint32_t {
      if constexpr (WIDE) return *(__attribute__((address_space(3))) const uint16_t *)(uintptr_t)x;
      else return *(__attribute__((address_space(3))) const u16_any *)(uintptr_t)x;
    };
    const uint32_t at = p + (C::PAIR ? sbuf * C::SBYTES + b * 8 : b * C::SBYTES + shift) + i * 512;
    uint32_t v = two(at);
    if (2 * i + 1 < n) v |= two(at + 256) << 16;
    // blocks behind the rows' end: not the next rows' scales, which may be NaN (WIDE: sw is a multiple of 4)
    const int left = sw - s * 8 - g * 2;
    return left >= 2 ? v : !WIDE && left == 1 ? v & 0xff00ffu : 0;
  };

  typename C::Acc acc[C::FM][C::FN];
  i32x4 fa[2][C::FM], fb[2][C::FN];  // pieces of this step of 64 bytes of k, and of the next
  auto multiply = [&](auto ks_, auto i_) LAMBDA {  // row i of the wave's results
    constexpr int ks = decltype(ks_)::value, i = decltype(i_)::value;
    static_for<C::FN>([&](auto j_) LAMBDA {
      constexpr int j = decltype(j_)::value;
      if constexpr (TY == MOE_ROWS_BF16) {
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fb[ks][j]),
                                                            __builtin_bit_cast(bf16x8, fa[ks][i]), acc[i][j], 0, 0, 0);
      } else if constexpr (TY == MOE_ROWS_INT8) {
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[ks][j], fa[ks][i], acc[i][j], 0, 0, 0);
      } else {
        const i32x4 n4 = fb[ks][j], m4 = fa[ks][i];
        const i32x8 vb = {n4[0], n4[1], n4[2], n4[3], 0, 0, 0, 0};
        const i32x8 va = {m4[0], m4[1], m4[2], m4[3], 0, 0, 0, 0};
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(vb, va, acc[i][j], 4, 4, (j & 1) * 2 + ks, sb[j / 2],
                                                                     (i & 1) * 2 + ks, sa[i / 2]);
      }
    });
  };

  // ---- a stage, in buffer b of the ring.  The products of one step of 64 bytes of k run while the next step's
  // operands come from LDS.  Before those are the next stage's, every wave has read this stage, so its buffer
  // takes the loads of stage `ahead`, and the next stage's loads have to be there.  after: the next stage (its scales'
  // shifts: msh, nsh).  A wave
  // without rows (IDLE) only loads and waits.
  auto stage = [&](auto b_, auto idle_, int after, int ahead, int msh, int nsh) LAMBDA {
    constexpr int b = decltype(b_)::value, bn = (b + 1) % NST;
    constexpr bool IDLE = decltype(idle_)::value;
    static_for<2>([&](auto ks_) LAMBDA {
      constexpr int ks = decltype(ks_)::value;
      if constexpr (ks == 1) {
        stage_wait<(NST - 2) * (LOADS + (C::PAIR ? 0 : C::SI))>();
        if constexpr (MX) {
          if constexpr (!C::PAIR) {
            issue_scales(ahead, b);
          } else {
            if (b == 1) sbuf ^= 1;
            if (b == 0) issue_scales(ahead / 2, 0);
          }
        }
      }
      static_for<C::FM>([&](auto i_) LAMBDA {
        constexpr int i = decltype(i_)::value;
        if constexpr (!IDLE) multiply(ks_, i_);
        if constexpr (ks == 1) {
          constexpr int l0 = 2 * i * LOADS / C::FM, l1 = 2 * (i + 1) * LOADS / C::FM;  // all in the first half
          static_for_from<(l0 < LOADS ? l0 : LOADS), (l1 < LOADS ? l1 : LOADS)>([&](auto l_) LAMBDA { issue(ahead, b_, l_); });
        }
        if constexpr (IDLE) return;
#pragma unroll
        for (int j = i * C::FN / C::FM; j < (i + 1) * C::FN / C::FM; ++j) fb[ks ^ 1][j] = read_n(ks == 1 ? bn : b, j, ks ^ 1);
        fa[ks ^ 1][i] = read_m(ks == 1 ? bn : b, i, ks ^ 1);
        if constexpr (MX && ks == 1) {  // the next stage's scales, where this one's are done with
          if constexpr (i % 2 == 1 || i == C::FM - 1) sa[i / 2] = scale_pair(sm, after, bn, i / 2, C::FM, msh);
          if constexpr (i == C::FM - 1) {
#pragma unroll
            for (int j = 0; j < SN; ++j) sb[j] = scale_pair(sn, after, bn, j, C::FN, nsh);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      });
    });
  };

  auto fill = [&]() LAMBDA {
    sbuf = 1;
    if constexpr (C::PAIR) issue_scales(0, 0);
    sbuf = 0;
    static_for<NST>([&](auto b_) LAMBDA {
      if constexpr (MX && !C::PAIR) issue_scales(decltype(b_)::value, decltype(b_)::value);
      static_for<LOADS>([&](auto l_) LAMBDA { issue(decltype(b_)::value, b_, l_); });
    });
  };
  auto begin = [&]() LAMBDA {
    stage_wait<(NST - 1) * (LOADS + (C::PAIR ? 0 : C::SI))>();
    if constexpr (MX) {
#pragma unroll
      for (int i = 0; i < SM; ++i) sa[i] = scale_pair(sm, 0, 0, i, C::FM, mshift);
#pragma unroll
      for (int j = 0; j < SN; ++j) sb[j] = scale_pair(sn, 0, 0, j, C::FN, nshift);
    }
#pragma unroll
    for (int j = 0; j < C::FN; ++j) fb[0][j] = read_n(0, j, 0);
#pragma unroll
    for (int i = 0; i < C::FM; ++i) fa[0][i] = read_m(0, i, 0);
  };

  enter();
  fill();
  if constexpr (RING) begin();
  for (;;) {
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int j = 0; j < C::FN; ++j) acc[i][j] = typename C::Acc{0, 0, 0, 0};
    if constexpr (!RING) begin();
    // whole turns of the buffers, so that each tile begins at the first: up to NST - 1 stages of zeros more
    const int turns = stages > NST ? (stages + NST - 1) / NST : 1, full = RING ? turns - 1 : turns;
    auto run = [&](auto idle_) LAMBDA {
      for (int s0 = 0; s0 < full * NST; s0 += NST)
        static_for<NST>([&](auto b_) LAMBDA {
          stage(b_, idle_, s0 + decltype(b_)::value + 1, s0 + decltype(b_)::value + NST, mshift, nshift);
        });
    };
    // a tile that ends before the wave's rows (in RING's last turn the products of such a wave are of no use)
    if (WM > 1 && m0 + mfirst >= (OP == OP_WGRAD ? a.M : cnt)) run(std::true_type{});
    else run(std::false_type{});
    const int m1 = m0, n1 = n0, e1 = e, mlim = OP == OP_WGRAD ? a.M : cnt;  // mlim: rows of the result
    const int64_t lo1 = lo;
    [[maybe_unused]] const int ms1 = mshift, ns1 = nshift;
    round += per;
    place += kTurn % per;
    if (place >= per) place -= per;
    tile = round + place;
    if constexpr (RING) {  // the last turn loads the next tile's first stages
      if (tile < last) enter();  // else this one's again, for nothing
      static_for<NST>([&](auto b_) LAMBDA {
        constexpr int b = decltype(b_)::value;
        constexpr bool same = b + 1 < NST;  // the next stage is this tile's
        stage(b_, std::false_type{}, same ? (turns - 1) * NST + b + 1 : 0, b, same ? ms1 : mshift, same ? ns1 : nshift);
      });
    } else {  // the next tile's first loads go out before this one's results
      stage_wait<0>();
      if (tile < last) {
        enter();
        fill();
      }
    }
    // the products are finished here, not moved behind the branches below
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int j = 0; j < C::FN; ++j) asm volatile("" : "+v"(acc[i][j]));

    // ---- results: lane (g, r16) holds, of row i * 16 + r16, 4 G consecutive columns for each G results
    constexpr int F = C::F, G = C::G;
    const int nl = n1 + wn * 16 * F + g * 4 * G;
    float cs[TY == MOE_ROWS_INT8 ? 4 * C::FN : 1];  // the columns' scales
    if constexpr (TY == MOE_ROWS_INT8) {
#pragma unroll
      for (int q = 0; q < 4 * C::FN; ++q) {
        const int f = q / 4 % F, n = nl + f / G * 16 * G + f % G * 4 + q % 4;
        cs[q] = a.ns && n < a.N ? ((const float *)a.ns)[(int64_t)e1 * nw + n + (q >= 4 * F ? a.N : 0)] : 1.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
      const int m = m1 + mfirst + i * 16 + r16;
      if (m >= mlim) continue;
      const float rs = TY == MOE_ROWS_INT8 && a.ms ? ((const float *)a.ms)[lo1 + m] : 1.0f;
      float v[4 * C::FN];
#pragma unroll
      for (int q = 0; q < 4 * C::FN; ++q) {
        v[q] = (float)acc[i][q / 4][q % 4];
        if constexpr (TY == MOE_ROWS_INT8) v[q] = v[q] * cs[q] * rs;
      }
      if constexpr (GATED) {
#pragma unroll
        for (int q = 0; q < 4 * F; ++q) v[q] = silu_times(v[q], v[4 * F + q]);
      }
      const int64_t at = ((OP == OP_WGRAD ? (int64_t)e1 * a.M : lo1) + m) * a.N + nl;
#pragma unroll
      for (int f = 0; f < F; f += G) {
        const int n = f * 16;
        if (nl + n >= a.N) continue;  // N is a multiple of 8
        const float *y = v + f * 4;
        if constexpr (F32) *(f32x4 *)((float *)a.out + at + n) = f32x4{y[0], y[1], y[2], y[3]};
        else if constexpr (G == 1) *(u32x2 *)((uint16_t *)a.out + at + n) = u32x2{pack2(y[0], y[1]), pack2(y[2], y[3])};
        else *(u32x4 *)((uint16_t *)a.out + at + n) = u32x4{pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7])};
      }
    }
    if (tile >= last) break;
  }
  stage_wait<0>();  // nothing is under way into LDS when the workgroup gives it back
}
#undef LAMBDA

template <int TY, int OP, bool GATED, bool F32, int BM, int BN, int WM, int WN, int NST, bool RING, bool WIDE>
static hipError_t launch_cfg(const ExpertsArgs &a, hipStream_t st) {
  using C = Tile<TY, OP, GATED, F32, BM, BN, WM, WN, NST, WIDE>;
  // Tiles fit 32 bits: 16 rows high only for at most 16 * 2^11 rows, 64 for at most 64 * 2^11, else 128 and more, so at
  // most (2^27 / 128 + 2^11) * 2^10; wgrad: 2^11 experts of at most 2^9 * 2^9
  const int64_t mt = OP == OP_WGRAD ? (int64_t)a.g.E * ((a.M + BM - 1) / BM) : a.g.rows / BM + a.g.E;
  const int64_t tiles = mt * ((a.N + C::CO - 1) / C::CO);
  const size_t lds = C::LDS + (size_t)(a.g.E + 1) * 4;
  const int64_t resident = 256 * (160 * 1024 / lds > 8 / C::W ? 8 / C::W : 160 * 1024 / lds);
  const unsigned grid = (unsigned)(tiles < resident ? (tiles + 7) / 8 * 8 : resident);
  auto k = experts_kernel<TY, OP, GATED, F32, BM, BN, WM, WN, NST, RING, WIDE>;
  hipLaunchKernelGGL(k, dim3(grid), dim3(C::T), lds, st, a);
  return hipGetLastError();
}
// The tile, for `rows` rows spread evenly over the experts (the counts are on the device): 16 x 64 for forward with at most
// 16 an expert (weights streamed once, three workgroups a CU: 8 rows of 8 of 64 experts, 4096 -> 2 x 1024 bf16 in 24.9
// us; 64 x 128: 28.9, 128 x 128: 32.9), 64 x 128 for at most 64; else what comes
// out fastest by rounds of tiles over the CUs x (stages x time of a stage + time between tiles), measured in us
// on one MI355X where the tiles fill the chip:
//                                               stage  between   16 x 2048 rows, 4096 -> 4096 bf16
//   256 x 256, 8 waves, two stages, one a CU     1.72     4      870 us (the four in turn, as below)
//   256 x 128, 8 waves, three stages, one a CU   0.93     2.5    976   (an expert's few rows in one tile, its waves
//                                                                      without rows idle)
//   128 x 128, 4 waves, two stages, two a CU     1.15     1.5    1091
//   128 x 128, 4 waves, four stages, one a CU    0.60     2      1199  (deep: for hardly more tiles than CUs)
// The order that it gives is that of the measured times within 15 % on 1024 to 32768 rows of 4 to 64 experts (128 rows
// of each of 4, 4096 -> 2 x 2048 bf16, in the table's order: 84, 52, 63, 48 us; 200 of 32, 2048 -> 1024: 57, 41, 46,
// 46).  In wgrad a tile costs what its expert has rows: the largest is taken to have three times the mean.
//   MXFP4 has the first and the third.  A stage's scales are a load more where they are read stage by stage, which three
// and four stages would need: the fourth took 36 us against 32 for the third on 128 rows of 4 experts, 4128 -> 2 x 2048.
// The first, with scales at odd addresses (not WIDE), runs out of registers.  64 x 128 with two stages: 16 rows of 32
// experts, 4096 -> 2 x 4096 in 98 us (four: 110); with four for at most 256 tiles: 8 of 8, 4096 -> 2 x 1024 in 11.8 us
// (13.5).  Scales at odd addresses cost 106 us where these cost 98.
ExpertsTile experts_tile(const ExpertsArgs &a, int op, int row_type, bool gated, bool wide) {
  const bool mx = row_type == MOE_ROWS_MXFP4;
  const int e16 = row_type == MOE_ROWS_BF16 ? 8 : row_type == MOE_ROWS_INT8 ? 16 : 32;
  const int64_t E = a.g.E, mean = (a.g.rows + E - 1) / E, m = op == OP_WGRAD ? a.M : mean;
  auto tiles = [&](int bm, int bn) {
    const int64_t co = gated ? bn / 2 : bn;
    // ragged rows leave half a tile an expert empty
    const int64_t mt = op == OP_WGRAD ? E * ((m + bm - 1) / bm) : (a.g.rows + E * bm / 2) / bm;
    return mt * ((a.N + co - 1) / co);
  };
  if (op == OP_FORWARD && !mx && mean <= 16) return {16, 64, 4};
  if (m <= 64) return {64, 128, mx && tiles(64, 128) > 256 ? 2 : 4};
  const double stages = op == OP_FORWARD ? (a.K / e16 + 7) / 8 : op == OP_DGRAD ? (a.K + 63) / 64 : (mean + 63) / 64;
  auto time = [&](int bm, int bn, int slots, double stage, double between) {
    const double rounds = (double)((tiles(bm, bn) + slots - 1) / slots), one = stages * stage + between;
    const double largest = op == OP_WGRAD ? (E < 3 ? E : 3) * stages * stage : 0.0;
    return rounds * one > largest ? rounds * one : largest;
  };
  const double big = time(256, 256, 256, 1.72, 4.0), two = time(128, 128, 512, 1.15, 1.5);
  if (mx) return wide && big <= two ? ExpertsTile{256, 256, 2} : ExpertsTile{128, 128, 2};
  const double flat = time(256, 128, 256, 0.93, 2.5), deep = time(128, 128, 256, 0.60, 2.0);
  if (big <= two && big <= flat && big <= deep) return {256, 256, 2};
  if (flat <= two && flat <= deep) return {256, 128, 3};
  return {128, 128, deep <= two ? 4 : 2};
}

// the kernel of the tile; one is built only where experts_tile can name it
template <int TY, int OP, bool GATED, bool F32, bool WIDE>
static hipError_t launch_tile(const ExpertsArgs &a, hipStream_t st) {
  constexpr bool MX = TY == MOE_ROWS_MXFP4;
  const ExpertsTile t = experts_tile(a, OP, TY, GATED, WIDE);
  if constexpr (OP == OP_FORWARD && !MX) {
    if (t.rows == 16) return launch_cfg<TY, OP, GATED, F32, 16, 64, 1, 2, 4, true, true>(a, st);
  }
  if (t.rows == 64) {
    if constexpr (MX) {
      if (t.stages == 2) return launch_cfg<TY, OP, GATED, F32, 64, 128, 2, 2, 2, true, WIDE>(a, st);
    }
    return launch_cfg<TY, OP, GATED, F32, 64, 128, 2, 2, 4, true, WIDE>(a, st);
  }
  if constexpr (WIDE) {
    if (t.columns == 256) return launch_cfg<TY, OP, GATED, F32, 256, 256, 2, 4, 2, false, WIDE>(a, st);
  }
  if constexpr (!MX) {
    if (t.rows == 256) return launch_cfg<TY, OP, GATED, F32, 256, 128, 4, 2, 3, true, WIDE>(a, st);
    if (t.stages == 4) return launch_cfg<TY, OP, GATED, F32, 128, 128, 2, 2, 4, true, WIDE>(a, st);
  }
  return launch_cfg<TY, OP, GATED, F32, 128, 128, 2, 2, 2, true, WIDE>(a, st);
}

template <int TY, int OP, bool GATED, bool F32>
static hipError_t launch_type(const ExpertsArgs &a, hipStream_t st) {
  if constexpr (TY == MOE_ROWS_MXFP4) {
    if (!mx_scales_wide(a.K, a.ms, a.ns)) return launch_tile<TY, OP, GATED, F32, false>(a, st);
  }
  return launch_tile<TY, OP, GATED, F32, true>(a, st);
}

hipError_t launch_experts(const ExpertsArgs &a, int op, int row_type, int act, bool out_fp32, hipStream_t st) {
  if (op != OP_WGRAD && a.g.rows == 0) return hipSuccess;
  if (op == OP_DGRAD) return launch_type<MOE_ROWS_BF16, OP_DGRAD, false, false>(a, st);
  if (op == OP_WGRAD)
    return out_fp32 ? launch_type<MOE_ROWS_BF16, OP_WGRAD, false, true>(a, st)
                    : launch_type<MOE_ROWS_BF16, OP_WGRAD, false, false>(a, st);
  if (act == MOE_ACT_SWIGLU)
    return row_type == MOE_ROWS_BF16   ? launch_type<MOE_ROWS_BF16, OP_FORWARD, true, false>(a, st)
           : row_type == MOE_ROWS_INT8 ? launch_type<MOE_ROWS_INT8, OP_FORWARD, true, false>(a, st)
                                       : launch_type<MOE_ROWS_MXFP4, OP_FORWARD, true, false>(a, st);
  return row_type == MOE_ROWS_BF16   ? launch_type<MOE_ROWS_BF16, OP_FORWARD, false, false>(a, st)
         : row_type == MOE_ROWS_INT8 ? launch_type<MOE_ROWS_INT8, OP_FORWARD, false, false>(a, st)
                                     : launch_type<MOE_ROWS_MXFP4, OP_FORWARD, false, false>(a, st);
}

}  // namespace moe
