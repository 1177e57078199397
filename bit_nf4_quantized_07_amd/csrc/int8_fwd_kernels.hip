// Forward of the linear layer on a base of 8-bit rows, from activations in
// 8-bit rows:
//
//   Y[m][n] = sx[m] sw[n] sum_k Cx[m][k] Cw[n][k] + s sum_j T[m][j] B[n][j]
//                       (llm-compass "QLoRA", 方法与公式, the equation, with
//                        8-bit rows for W and x)
//
// The first sum is whole numbers, exact in 32 bits for K up to 2^17 (127^2 K <
// 2^31), so it does not depend on how the contraction is cut.  T comes from the
// rank-r kernel as two bf16 terms of s T.
//
// A workgroup of WM x WN waves computes 32 NI WM tokens x 32 NJ WN outputs, each
// wave 32 NI x 32 NJ: NI NJ accumulators of v_mfma_i32_32x32x32_i8, each a 32
// (outputs) x 32 (tokens) block of Y^T.
//  * The contraction advances 128 columns a step (four MFMA steps) through S LDS
//    stages that buffer loads fill directly, S steps ahead: rows of 128 bytes, whole
//    cache lines, whose eight 16-byte pieces are XOR-swizzled by (row >> 1) & 7, so
//    that operand reads are free of bank conflicts.  Rows of 64 bytes asked L2 more than
//    twice as often (4096 x 4096 x 11008 without an adapter: 31 million requests and
//    269 us of a 256 x 256 form, here 13 million and 179).
//  * One barrier a step, in front of its last MFMA step: what that one reads is the
//    next step's, and the loads of S steps on go into the stage that is done.
//    Eight waves: with two on a SIMD one multiplies while the other reads (four
//    waves of 128 x 64 took 1.2 times as long).
//  * The whole sums become fp32, times sx sw, in the accumulators' own
//    registers, and s T B^T is added by bf16 MFMAs.
//  * The bf16 tile goes out through the stages, so that every store
//    instruction writes whole row segments.
// Where the tiles do not fill the device the contraction is split; a split's
// fp32 values go to the workspace and are added in a fixed order.
//
// What bounds it: the large tiles the clock that power leaves (8192^3 450 us, 2.45
// POP/s, level with the library's product on the same codes, 62 % of the cycles in
// MFMAs at 1.8 GHz; 4096 x 4096 x 11008, r = 64, 205); at 2048 x 4096 x 4096 (37 us;
// the library 42) one round of 256 workgroups, a quarter of which is its start and
// epilogue; at 16 tokens the weight (28672 x 8192: 5.2 TB/s of it); at one token the
// latency of what is loaded before the weight.
#include <type_traits>

#include "device_common.h"
#include "int8_loads.h"
#include "kernels.h"
#include "terms.h"

namespace qlk {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

constexpr int kI8Step = 128;    // columns of the contraction per step
static_assert(kPast == kOOB, "the tiles' resources leave this offset out");

struct Int8FwdArgs {
  const int8_t* X;      // [M, K]
  const float* sx;      // [M]
  const int8_t* W;      // [N, K]
  const float* sw;      // [N]
  int M, N, K;
  const uint16_t* T2;   // operands of s T's hi and mid terms (launch_int8_T)
  const uint16_t* B;    // [N, r]
  int r;                // 0: no adapter
  uint16_t* Y;          // [M, N]
  int tiles_m, tiles_n, group_m;
  float* part;          // split contraction: fp32 [splits][M, N]
  int kz_len;           // steps per split; 0: one pass
};

template <int NI, int NJ, int WM, int WN, int S>
__device__ __forceinline__ void int8_tile(const Int8FwdArgs& g) {
  constexpr int TM = 32 * NI * WM, TN = 32 * NJ * WN;             // the tile
  constexpr int XL = 4 * NI / WN, WL = 4 * NJ / WM, L = XL + WL;  // a wave's loads of a stage
  constexpr int XB = TM * kI8Step, WB = TN * kI8Step;             // bytes of a stage
  static_assert(S == 2 || S == 3, "stages");
  static_assert(XL * WN == 4 * NI && WL * WM == 4 * NJ, "whole loads");
  __shared__ __attribute__((aligned(16))) uint8_t x0[XB];
  __shared__ __attribute__((aligned(16))) uint8_t w0[WB];
  __shared__ __attribute__((aligned(16))) uint8_t x1[XB];
  __shared__ __attribute__((aligned(16))) uint8_t w1[WB];
  __shared__ __attribute__((aligned(16))) uint8_t x2[S == 3 ? XB : 16];
  __shared__ __attribute__((aligned(16))) uint8_t w2[S == 3 ? WB : 16];
  uint8_t* const xb[3] = {x0, x1, x2};
  uint8_t* const wb[3] = {w0, w1, w2};
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 31, h = lane >> 5;
  const int fg = wave % WN, tq = wave / WN;   // the wave's outputs and tokens

  const int ntiles = g.tiles_m * g.tiles_n;
  const int z = (int)blockIdx.x / ntiles;
  int tm, tn;
  tile_coords((int)blockIdx.x % ntiles, g.tiles_m, g.tiles_n, g.group_m, tm, tn);
  const int m0 = tm * TM, n0 = tn * TN;
  const int nsteps = (g.K + kI8Step - 1) / kI8Step;
  const int kz0 = g.kz_len ? z * g.kz_len : 0;
  const int kz1 = g.kz_len ? min(nsteps, kz0 + g.kz_len) : nsteps;

  // Load i of wave w fills rows 8 (XL w + i) .. +7 of a stage (1 KB); lane l lands
  // at row l / 8 of them, physical piece l % 8.  Where K ends inside a step, the
  // pieces past it are zero.
  const __amdgpu_buffer_rsrc_t rx = rsrc_whole(g.X, (uint32_t)((int64_t)g.M * g.K));
  const __amdgpu_buffer_rsrc_t rw = rsrc_whole(g.W, (uint32_t)((int64_t)g.N * g.K));
  auto swz = [](int row) { return (row >> 1) & 7; };
  LinePiece xp[XL], wp[WL];
#pragma unroll
  for (int i = 0; i < XL; ++i) xp[i] = line_piece(8 * (XL * wave + i) + (lane >> 3), lane, m0, g.M, g.K);
#pragma unroll
  for (int j = 0; j < WL; ++j) wp[j] = line_piece(8 * (WL * wave + j) + (lane >> 3), lane, n0, g.N, g.K);
  const int kcut = g.K % kI8Step ? nsteps - 1 : -1;   // the step that K ends in
  auto load_l = [&](int l, int buf, int kb) {
    const int k = __builtin_amdgcn_readfirstlane(kb);
    const uint32_t soff = (uint32_t)k * kI8Step;
    if (l < XL)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rx, (__attribute__((address_space(3))) void*)(xb[buf] + 1024 * (XL * wave + l)), 16,
          line_at(xp[l], k == kcut), soff, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rw, (__attribute__((address_space(3))) void*)(wb[buf] + 1024 * (WL * wave + l - XL)), 16,
          line_at(wp[l - XL], k == kcut), soff, 0, 0);
  };
  // Operand of a 32-row block, MFMA step t: row c, logical piece 2 t + h.
  int rd[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) rd[t] = c * kI8Step + (((2 * t + h) ^ swz(c)) * 16);
  auto xfrag = [&](int buf, int i, int t) -> i32x4_t {
    return *reinterpret_cast<const i32x4_t*>(xb[buf] + 32 * (NI * tq + i) * kI8Step + rd[t]);
  };
  auto wfrag = [&](int buf, int j, int t) -> i32x4_t {
    return *reinterpret_cast<const i32x4_t*>(wb[buf] + 32 * (NJ * fg + j) * kI8Step + rd[t]);
  };

  i32x16_t acc[NJ][NI];
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[j][i][v] = 0;

  i32x4_t a[2][NJ], b[2][NI];   // [MFMA step parity][block]
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int l = 0; l < L; ++l) load_l(l, s, min(kz0 + s, kz1 - 1));
  __builtin_amdgcn_s_waitcnt(wait_for((S - 1) * L, 0));   // the first step has landed
  __builtin_amdgcn_s_barrier();
#pragma unroll
  for (int j = 0; j < NJ; ++j) a[0][j] = wfrag(0, j, 0);
#pragma unroll
  for (int i = 0; i < NI; ++i) b[0][i] = xfrag(0, i, 0);

  // One step: four MFMA steps of NI NJ slots.  Each reads the next one's operands
  // in its first slots; the last one reads the next step's, which every wave has
  // waited for before the barrier in front of it (vmcnt).  Before the same barrier
  // every wave's reads of this step's stage, the last of them for MFMA step 3, have
  // ended (lgkmcnt): the loads of step kb + S go into it.
  auto step = [&](auto Pc, int kb) {
    constexpr int P = decltype(Pc)::value;
    constexpr int nxt = (P + 1) % S;
    constexpr int Q = NI * NJ, F = NI + NJ;
    constexpr int R = Q >= F ? F : Q;   // slots that read
    const int kload = min(kb + S, kz1 - 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t == 3) {
        __builtin_amdgcn_s_waitcnt(wait_for((S - 2) * L, 0));
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int j = q / NI, i = q % NI;
        acc[j][i] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[t & 1][j], b[t & 1][i], acc[j][i], 0, 0, 0);
        if (q < R) {
#pragma unroll
          for (int l = q * F / R; l < (q + 1) * F / R; ++l) {
            if (l < NI) b[(t + 1) & 1][l] = xfrag(t == 3 ? nxt : P, l, (t + 1) & 3);
            else a[(t + 1) & 1][l - NI] = wfrag(t == 3 ? nxt : P, l - NI, (t + 1) & 3);
          }
        }
        if (t == 3) {
#pragma unroll
          for (int l = q * L / Q; l < (q + 1) * L / Q; ++l) load_l(l, P, kload);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  // Whole groups of S steps without a branch between them: where paths meet the
  // compiler waits for loads that are not due.
  int kb = kz0;
  for (; kb + S <= kz1; kb += S) {
    step(std::integral_constant<int, 0>(), kb);
    step(std::integral_constant<int, 1>(), kb + 1);
    if constexpr (S == 3) step(std::integral_constant<int, 2>(), kb + 2);
  }
  if (kb < kz1) {
    step(std::integral_constant<int, 0>(), kb);
    if (S == 3 && kb + 1 < kz1) step(std::integral_constant<int, 1>(), kb + 1);
  }
  __builtin_amdgcn_s_waitcnt(0);   // no load into LDS outlives the loop
  __syncthreads();                 // every wave's operand reads are done

  // Accumulator [j][i]: lane holds token mw + 32 i + c and outputs
  // nw + 32 j + 8 (v / 4) + 4 h + (v % 4).  Block column by block column: fp32
  // values, the adapter's term, then bf16 rows of 2 TN bytes in LDS: two blocks of
  // 32 token rows lie in each of w0 and w1, the others in x0 and x1, the 16-byte
  // pieces of a row XOR-swizzled by its number.  N and r are multiples of 8, so
  // that a piece is wholly inside or wholly outside.
  constexpr int PR = TN / 8;       // pieces of a row
  constexpr int BB = 32 * 16 * PR; // bytes of a block
  static_assert(NI * WM <= 4 || (NI * WM == 8 && XB >= 2 * BB), "blocks in the stages");
  auto ob = [&](int k) -> uint8_t* {
    return (k < 2 ? w0 : k < 4 ? w1 : k < 6 ? x0 : x1) + (k & 1) * BB;
  };
  const int nw = n0 + 32 * NJ * fg, mw = m0 + 32 * NI * tq;
  const __amdgpu_buffer_rsrc_t rsx = rsrc_whole(g.sx, (uint32_t)g.M * 4);
  const __amdgpu_buffer_rsrc_t rsw = rsrc_whole(g.sw, (uint32_t)g.N * 4);
  const __amdgpu_buffer_rsrc_t rb = rsrc_whole(g.B, (uint32_t)(g.N * g.r * 2));
  const int r = z == 0 ? g.r : 0, nt = (r + 15) / 16;
  float* const part = g.kz_len ? g.part + (int64_t)z * g.M * g.N : nullptr;
  float sx[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int m = mw + 32 * i + c;
    sx[i] = __uint_as_float(bload32(rsx, m < g.M ? (uint32_t)m * 4 : kOOB));
  }
  f32x16_t out[NJ][NI];
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int n = nw + 32 * j + 8 * q + 4 * h;
      const uint4 sv = bload128(rsw, n < g.N ? (uint32_t)n * 4 : kOOB);
      const float s4[4] = {__uint_as_float(sv.x), __uint_as_float(sv.y), __uint_as_float(sv.z),
                           __uint_as_float(sv.w)};
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          out[j][i][4 * q + e] = (float)acc[j][i][4 * q + e] * sx[i] * s4[e];
    }
  // A token block's operands are 1 KB in a row; a block past the last token has none.
  const __amdgpu_buffer_rsrc_t rt =
      rsrc_whole(g.T2, (uint32_t)((g.M + 31) / 32 * nt) * 2048u);   // up to 2^31
  for (int t = 0; t < nt; ++t) {
    bf16x8_t top[NI][2], bop[NJ];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int blk = mw / 32 + i;
        top[i][e] = __builtin_bit_cast(
            bf16x8_t, bload128(rt, mw + 32 * i < g.M ? (uint32_t)(((blk * nt + t) * 2 + e) * 1024 + 16 * lane)
                                                     : kOOB));
      }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int nb = nw + 32 * j + c, rr = 16 * t + 8 * h;
      bop[j] = __builtin_bit_cast(
          bf16x8_t, bload128(rb, rr < r && nb < g.N ? (uint32_t)((nb * g.r + rr) * 2) : kOOB));
    }
#pragma unroll
    for (int e = 1; e >= 0; --e)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < NI; ++i) out[j][i] = mfma_32x32x16(bop[j], top[i][e], out[j][i]);
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int m = mw + 32 * i + c;
      uint8_t* const row = ob(NI * tq + i) + c * (16 * PR);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x16_t& v = out[j][i];
        if (part) {
          const int n = nw + 32 * j + 8 * q + 4 * h;
          if (m < g.M && n < g.N)
            *reinterpret_cast<float4*>(part + (int64_t)m * g.N + n) =
                make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        } else {
          const int piece = (4 * NJ * fg + 4 * j + q) ^ (c & (PR - 1));
          *reinterpret_cast<uint2*>(row + 16 * piece + 8 * h) =
              make_uint2(pack_bf16x2(v[4 * q], v[4 * q + 1]), pack_bf16x2(v[4 * q + 2], v[4 * q + 3]));
        }
      }
    }
  if (part) return;
  __syncthreads();
  constexpr int RW = 64 * WM * WN / PR;            // rows that a pass of the workgroup stores
  const int prow = tid / PR, pp = tid % PR;
  const __amdgpu_buffer_rsrc_t ry = rsrc_whole(g.Y, (uint32_t)((int64_t)g.M * g.N * 2));
#pragma unroll
  for (int e = 0; e < TM / RW; ++e) {
    const int row = RW * e + prow, rl = row & 31;  // RW divides 32
    const uint4 v = *reinterpret_cast<const uint4*>(ob(RW * e / 32) + rl * (16 * PR) +
                                                    16 * (pp ^ (rl & (PR - 1))));
    const int m = m0 + row, n = n0 + 8 * pp;
    bstore128(ry, v, m < g.M && n < g.N ? (uint32_t)(((int64_t)m * g.N + n) * 2) : kOOB);
  }
}

// The host pass does not keep a kernel template whose body calls these loads
// from a lambda: one plain kernel per form.
__global__ void __launch_bounds__(512) k_int8_fwd_256x256(Int8FwdArgs g) { int8_tile<4, 2, 2, 4, 2>(g); }
__global__ void __launch_bounds__(512) k_int8_fwd_128x256(Int8FwdArgs g) { int8_tile<2, 2, 2, 4, 3>(g); }
__global__ void __launch_bounds__(512) k_int8_fwd_64x256(Int8FwdArgs g) { int8_tile<2, 1, 1, 8, 3>(g); }
__global__ void __launch_bounds__(256) k_int8_fwd_64x64(Int8FwdArgs g) { int8_tile<1, 1, 2, 2, 3>(g); }
__global__ void __launch_bounds__(256) k_int8_fwd_64x128(Int8FwdArgs g) { int8_tile<1, 2, 2, 2, 3>(g); }

// ---------------------------------------------------------------------------
// Up to 16 tokens: the weight is streamed once.  A workgroup takes up to 8 blocks
// of 16 outputs, so that one on every CU covers them; its waves take every
// kGvWaves-th run of 256 columns of a block's rows (four loads of 16 rows x 64
// bytes, four runs in flight) with v_mfma_i32_16x16x64_i8, and add their whole sums
// in LDS (integers: in any order the same).
//  * The tokens' columns lie in LDS, up to kGvCols of them at a time, loaded once
//    per workgroup by whole lines (rows of 128 bytes, pieces XOR-swizzled by
//    (token >> 1) & 7).  Read from memory beside the weight, a row per lane, they
//    took half the address unit's time (16 tokens, 28672 x 8192: 69 us, 3.4 TB/s).
//    Columns past K are zero there, so that it does not matter which the weight's
//    loads then bring.
//  * T = X A^T arrives as kTSplits partial sums, added in a fixed order by every
//    workgroup (the first one writes T), or is computed here.  The partial sums, the
//    first output's scales and its B are waited for before X and the weight are asked
//    for; s T B^T is summed in fp32 while the first weights are on their way.
// Measured: 16 tokens, 28672 x 8192 45 us (5.2 TB/s of weight; a copy reads and
// writes 5.1), one token, 4096 x 4096 7.0 us: 17 MB of weight behind a launch's start and
// the loads above.
constexpr int kGvWaves = 8;
constexpr int kGvThreads = 64 * kGvWaves;
constexpr int kGvBlocks = 8;    // blocks of 16 outputs per workgroup
constexpr int kGvDepth = 4;     // runs in flight per wave

// RT = 0: T's partial sums come from a launch of their own.  RT = 1, 2: every
// workgroup computes T for up to 16 RT ranks from A [r, K], K <= COLS / RT, and its
// tokens in LDS; wave w takes the slices w, w + 8, .. of 64 columns with
// v_mfma_f32_16x16x32_bf16, and the waves' sums are added in order.
template <int COLS, int RT>
__global__ void __launch_bounds__(kGvThreads)
k_int8_gemv(Int8FwdArgs g, const float* __restrict__ Tpart, const uint16_t* __restrict__ A, float s,
            float* __restrict__ T_out, int nb) {
  constexpr int TU = RT ? COLS / 64 / kGvWaves / RT : 1;   // a wave's slices
  __shared__ __attribute__((aligned(16))) uint8_t xs[16 * COLS];
  __shared__ int red[kGvBlocks * 256];             // [block][lane][4]
  __shared__ float yl[kGvBlocks * 256];            // s T B^T of output o
  __shared__ float tl[16 * (RT ? 16 * RT : 256)];  // s T
  __shared__ f32x4_t tw[RT ? kGvWaves * RT : 1][64];   // a wave's sums for T
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i = lane & 15, gq = lane >> 4;
  const int n0 = (int)blockIdx.x * 16 * nb;
  const int outs = 16 * nb * g.M;                  // token o / (16 nb), row o % (16 nb)
  const __amdgpu_buffer_rsrc_t rx = rsrc_whole(g.X, (uint32_t)((int64_t)g.M * g.K));

  // T's partial sums and what the first output needs, before anything else
  float t0 = 0.0f, sxt = 0.0f, sx0 = 0.0f, sw0 = 0.0f;
  uint4 b0 = make_uint4(0, 0, 0, 0), b1 = make_uint4(0, 0, 0, 0);
  uint4 aw[TU][RT ? 2 * RT : 1];
  if constexpr (RT > 0) {
    const __amdgpu_buffer_rsrc_t ra = rsrc_whole(A, (uint32_t)(g.r * g.K * 2));
#pragma unroll
    for (int u = 0; u < TU; ++u)
#pragma unroll
      for (int e = 0; e < 2 * RT; ++e) {
        const int j = 16 * (e >> 1) + i, sl = wave + kGvWaves * u;
        aw[u][e] = bload128(ra, j < g.r && 64 * sl < g.K
                                    ? (uint32_t)((j * g.K + 64 * sl + 16 * gq + 8 * (e & 1)) * 2) : kOOB);
      }
    if (tid < g.M * g.r) sxt = g.sx[tid / g.r];
  }
  if (RT == 0 && tid < g.M * g.r) {
    float p[kTSplits];
#pragma unroll
    for (int z = 0; z < kTSplits; ++z) p[z] = Tpart[z * g.M * g.r + tid];
    sxt = g.sx[tid / g.r];
#pragma unroll
    for (int z = 0; z < kTSplits; ++z) t0 += p[z];
  }
  const int nfirst = n0 + tid % (16 * nb);
  if (tid < outs && nfirst < g.N) {
    sx0 = g.sx[tid / (16 * nb)];
    sw0 = g.sw[nfirst];
  }
  if (g.r && tid < outs && nfirst < g.N) {
    const uint4* const p = reinterpret_cast<const uint4*>(g.B + (int64_t)nfirst * g.r);
    b0 = p[0];
    if (g.r > 8) b1 = p[1];
  }
  for (int e = tid; e < nb * 256; e += kGvThreads) red[e] = 0;

  for (int kc = 0; kc < g.K; kc += COLS) {
    const int cols = min(COLS, g.K - kc), nruns = (cols + 255) / 256;
    if (kc) __syncthreads();                       // every wave is done with the last columns
    // X: load u fills tokens 8 (u % 2) .. +7 of columns 128 (u / 2) .. +127
    for (int u = wave; u < 4 * nruns; u += kGvWaves) {
      const int m = 8 * (u & 1) + (lane >> 3), col = 128 * (u >> 1) + 16 * ((lane & 7) ^ ((m >> 1) & 7));
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rx, (__attribute__((address_space(3))) void*)(xs + 1024 * u), 16,
          m < g.M && col < cols ? (uint32_t)(m * g.K + kc + col) : kOOB, 0, 0, 0);
    }
    // Runs wave, wave + kGvWaves, .. of block after block.
    const int per = (nruns + kGvWaves - 1) / kGvWaves, tasks = per * nb;
    struct Run { uint4 w[4]; };
    int lb = 0, lr = 0;                            // the next task to load
    auto load = [&](Run& R) {
      const int run = lr * kGvWaves + wave, n = n0 + 16 * lb + i;
      const bool ok = lb < nb && run < nruns;
      const __amdgpu_buffer_rsrc_t r = rsrc_whole(g.W, ok ? (uint32_t)((int64_t)g.N * g.K) : 0);
      const uint32_t off = n < g.N ? (uint32_t)((int64_t)n * g.K) + 16 * gq : kOOB;
#pragma unroll
      for (int q = 0; q < 4; ++q) R.w[q] = bload128s(r, off, ok ? run_at(q, run, cols, kc) : 0);
      if (++lr == per) lr = 0, ++lb;
    };
    Run R[kGvDepth];
#pragma unroll
    for (int d = 0; d < kGvDepth; ++d) load(R[d]);
    if (RT == 0 && kc == 0) {
      if (tid < g.M * g.r) {
        const float t = t0 * sxt;
        if (T_out && blockIdx.x == 0) T_out[tid] = t;
        tl[tid] = s * t;
      }
      for (int e = tid + kGvThreads; e < g.M * g.r; e += kGvThreads) {
        float t = 0.0f;
        for (int z = 0; z < kTSplits; ++z) t += Tpart[z * g.M * g.r + e];
        t *= g.sx[e / g.r];
        if (T_out && blockIdx.x == 0) T_out[e] = t;
        tl[e] = s * t;
      }
    }
    // X has landed: its loads are in front of the weight's 4 kGvDepth
    __builtin_amdgcn_s_waitcnt(wait_for(4 * kGvDepth, 0));
    __syncthreads();
    if constexpr (RT > 0) {
      f32x4_t ta[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) ta[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int u = 0; u < TU; ++u) {
        const int sl = wave + kGvWaves * u;
        if (64 * sl >= g.K) break;
        uint4 xv[2];
        codes_to_bf16(*reinterpret_cast<const uint4*>(
                          xs + 2048 * (sl >> 1) + 128 * i + 16 * ((4 * (sl & 1) + gq) ^ ((i >> 1) & 7))), xv);
#pragma unroll
        for (int e = 0; e < 2 * RT; ++e)
          ta[e >> 1] = mfma_16x16x32(__builtin_bit_cast(bf16x8_t, xv[e & 1]),
                                     __builtin_bit_cast(bf16x8_t, aw[u][e]), ta[e >> 1]);
      }
#pragma unroll
      for (int t = 0; t < RT; ++t) tw[wave * RT + t][lane] = ta[t];
      __syncthreads();
      if (tid < g.M * g.r) {                       // 16 RT ranks of 16 tokens at most
        const int m = tid / g.r, j = tid % g.r;
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < kGvWaves; ++w) t += tw[w * RT + (j >> 4)][16 * (m >> 2) + (j & 15)][m & 3];
        t *= sxt;
        if (T_out && blockIdx.x == 0) T_out[tid] = t;
        tl[tid] = s * t;
      }
      __syncthreads();
    }
    if (kc == 0) {
      for (int o = tid; o < outs; o += kGvThreads) {
        const int m = o / (16 * nb), n = n0 + o % (16 * nb);
        float y = 0.0f;
        auto add = [&](const uint4& bv, int j) {
          const uint32_t bw[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y = __builtin_fmaf(tl[m * g.r + j + 2 * e], bf16_to_f32(bw[e] & 0xffffu), y);
            y = __builtin_fmaf(tl[m * g.r + j + 2 * e + 1], bf16_to_f32(bw[e] >> 16), y);
          }
        };
        if (n < g.N) {
          int j = 0;
          if (o == tid && g.r) {
            add(b0, 0);
            if (g.r > 8) add(b1, 8);
            j = 16;
          }
          for (; j < g.r; j += 8) add(*reinterpret_cast<const uint4*>(g.B + (int64_t)n * g.r + j), j);
        }
        yl[o] = y;
      }
    }
    i32x4_t acc = i32x4_t{0, 0, 0, 0};
    int ub = 0, ur = 0;                            // the task in use
    auto use = [&](const Run& R) {
      const int run = ur * kGvWaves + wave;
      const uint8_t* const x = xs + 4096 * min(run, nruns - 1);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4 xv = *reinterpret_cast<const uint4*>(
            x + 2048 * (q >> 1) + 128 * i + 16 * ((4 * (q & 1) + gq) ^ ((i >> 1) & 7)));
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, R.w[q]),
                                                    __builtin_bit_cast(i32x4_t, xv), acc, 0, 0, 0);
      }
      if (++ur == per) {
#pragma unroll
        for (int v = 0; v < 4; ++v) atomicAdd(&red[ub * 256 + 64 * v + lane], acc[v]);
        acc = i32x4_t{0, 0, 0, 0};
        ur = 0;
        ++ub;
      }
    };
    for (int t = 0; t < tasks; t += kGvDepth) {
#pragma unroll
      for (int d = 0; d < kGvDepth; ++d)
        if (t + d < tasks) {
          use(R[d]);
          load(R[d]);
        }
    }
  }
  __syncthreads();
  // The lane that holds row 16 b + 4 q + v of token m is 16 q + m, element v.
  for (int o = tid; o < outs; o += kGvThreads) {
    const int m = o / (16 * nb), row = o % (16 * nb), n = n0 + row;
    if (n >= g.N) continue;
    const int sum = red[(row >> 4) * 256 + 64 * (row & 3) + 16 * ((row & 15) >> 2) + m];
    const float fx = o == tid ? sx0 : g.sx[m], fw = o == tid ? sw0 : g.sw[n];
    g.Y[(int64_t)m * g.N + n] = f32_to_bf16((float)sum * fx * fw + yl[o]);
  }
}

// ------------------------------- launchers ---------------------------------

// Tile and split of the contraction, by the time each would take.  A step of a
// tile takes `alone` us where few workgroups run, and `full` for a workgroup on
// every CU: for the large tiles the power limit's MFMA rate, for the small ones L2
// (18 TB/s of operands); `per_cu` workgroups share a CU's LDS.  A split contraction
// pays a second launch and its partial sums' trip.  Fitted to all forms at one to
// eight splits; the choice against the fastest at twelve sizes of 64 to 4000 tokens
// and 192 to 11072 columns: equal or within 2 us, but for 647 x 9152 x 3288 (42 us,
// with a third split 38).
struct Int8Form {
  void (*kernel)(Int8FwdArgs);
  int tm, tn, threads, per_cu;
  double alone, full;          // rows of whole 128-byte lines
  double alone_cut, full_cut;  // 128 does not divide K: a row's load touches two lines
};
static const Int8Form kForms[] = {{k_int8_fwd_256x256, 256, 256, 512, 1, 0.95, 1.54, 1.12, 1.80},
                                  {k_int8_fwd_128x256, 128, 256, 512, 1, 0.50, 0.85, 0.68, 1.03},
                                  {k_int8_fwd_64x256, 64, 256, 512, 1, 0.33, 0.50, 0.57, 0.66},
                                  {k_int8_fwd_64x128, 64, 128, 256, 2, 0.18, 0.35, 0.31, 0.37},
                                  {k_int8_fwd_64x64, 64, 64, 256, 3, 0.10, 0.22, 0.20, 0.23}};
constexpr int kNumForms = sizeof(kForms) / sizeof(kForms[0]);

// Sixteens of ranks that the single-token forward multiplies itself; 0: none.  It
// saves a launch, and every workgroup reads A: 1024 x 1024 at r = 16 8.4 -> 5.2 us
// (replayed in a graph 5.9 -> 5.3), 4096 x 4096 at r = 16 7.8 -> 9.7 in a graph.
static int int8_gemv_ranks(int64_t K, int r) {
  const int rt = (r + 15) / 16;
  return rt <= 2 && K * rt <= 2048 && K * r <= 16384 ? rt : 0;
}

Int8FwdPlan plan_int8_fwd(int64_t M, int64_t K, int64_t N, int r) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  Int8FwdPlan p{};
  if (M <= kGemvMaxM) {
    p.gemv = true;
    p.bytes = r && !int8_gemv_ranks(K, r) ? up((size_t)kTSplits * M * r * 4) : 0;
    return p;
  }
  const int64_t steps = (K + kI8Step - 1) / kI8Step;
  double best = 0.0;
  for (int f = 0; f < kNumForms; ++f) {
    const Int8Form& F = kForms[f];
    const int64_t tiles = ((M + F.tm - 1) / F.tm) * ((N + F.tn - 1) / F.tn);
    for (int splits = 1; splits <= 8; ++splits) {
      if (splits > 1 && (tiles * splits > F.per_cu * kCUs || steps / splits < 8)) break;
      const int64_t len = (steps + splits - 1) / splits;
      const int64_t wgs = tiles * splits, round = (int64_t)F.per_cu * kCUs, rest = wgs % round;
      const double alone = K % kI8Step ? F.alone_cut : F.alone, full = K % kI8Step ? F.full_cut : F.full;
      double step = (double)(wgs / round) * F.per_cu * full;
      if (rest > kCUs) step += full * ((rest + kCUs - 1) / kCUs);
      else if (rest) step += rest * full / kCUs > alone ? rest * full / kCUs : alone;
      double us = len * step;
      if (splits > 1) us += 2.5 + (double)M * N * splits * 8.0 / 5e6;
      if (best == 0.0 || us < best) {
        best = us;
        p.form = f;
        p.kz_len = splits > 1 ? (int)len : 0;
      }
    }
  }
  p.off_T = 0;
  p.off_down = up(int8_two_bytes(M, r));
  p.off_part = p.off_down + up(int8_T_bytes(M, K, r));
  p.bytes = p.off_part;
  if (p.kz_len) p.bytes += up((size_t)((steps + p.kz_len - 1) / p.kz_len) * M * N * 4);
  return p;
}

hipError_t launch_int8_fwd(const Int8Rows& X, int64_t M, const Int8Rows& W, int64_t N, int64_t K,
                           const uint16_t* A, const uint16_t* B, int r, float s, uint16_t* Y,
                           float* T_out, void* ws, const Int8FwdPlan& p, hipStream_t st) {
  Int8FwdArgs g{};
  g.X = X.codes; g.sx = X.scale; g.W = W.codes; g.sw = W.scale;
  g.M = (int)M; g.N = (int)N; g.K = (int)K;
  g.B = B; g.r = r; g.Y = Y;
  char* const base = reinterpret_cast<char*>(ws);
  if (p.gemv) {
    float* const part = reinterpret_cast<float*>(base + p.off_T);
    const int rt = r ? int8_gemv_ranks(K, r) : 0;
    if (r && !rt) {
      const hipError_t e = launch_int8_T_partial(X.codes, M, K, A, r, part, st);
      if (e != hipSuccess) return e;
    }
    const int blocks = (int)((N + 15) / 16);
    const int nb = min((blocks + kCUs - 1) / kCUs, kGvBlocks);
    const dim3 grid((unsigned)((blocks + nb - 1) / nb)), block(kGvThreads);
    auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, block, 0, st, g, part, A, s, T_out, nb);
    };
    if (rt == 1) launch(k_int8_gemv<2048, 1>);
    else if (rt == 2) launch(k_int8_gemv<2048, 2>);
    else if (K <= 4096) launch(k_int8_gemv<4096, 0>);
    else launch(k_int8_gemv<8192, 0>);
    return hipGetLastError();
  }
  if (r) {
    uint16_t* const T2 = reinterpret_cast<uint16_t*>(base + p.off_T);
    const hipError_t e = launch_int8_T(X, M, K, A, r, s, T_out, T2,
                                       reinterpret_cast<float*>(base + p.off_down), st);
    if (e != hipSuccess) return e;
    g.T2 = T2;
  }
  const Int8Form& F = kForms[p.form];
  g.tiles_m = (int)((M + F.tm - 1) / F.tm);
  g.tiles_n = (int)((N + F.tn - 1) / F.tn);
  g.group_m = group_for(g.tiles_m, g.tiles_n, (double)F.tm * K, (double)F.tn * K);
  g.kz_len = p.kz_len;
  const int steps = (int)((K + kI8Step - 1) / kI8Step);
  const int splits = p.kz_len ? (steps + p.kz_len - 1) / p.kz_len : 1;
  if (p.kz_len) g.part = reinterpret_cast<float*>(base + p.off_part);
  const dim3 grid((unsigned)((int64_t)g.tiles_m * g.tiles_n * splits));
  hipLaunchKernelGGL(F.kernel, grid, dim3(F.threads), 0, st, g);
  if (p.kz_len) return launch_split_reduce(g.part, splits, M * N, Y, false, st);
  return hipGetLastError();
}

}  // namespace qlk
