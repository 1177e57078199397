// Input gradient of the linear layer for any number of outputs (8 | N), on a base in
// 8-bit rows or NF4 as it is stored or on a bf16 one:
//
//   dX[m][k] = sum_n dY[m][n] w_hat[n][k] + sum_j U[m][j] A[j][k],   U = s dY B
//                       (llm-compass "QLoRA", 方法与公式, the equation,
//                        differentiated with respect to x)
//
// Rounded to bf16 on the way, once each: a weight that is not bf16 as it is stored (a
// second term would double the MFMAs), and U, which holds s already so that A goes in
// as it is.  From 64 bits dX is 2.33e-3 at s = 1.7 where the adapter's term is most of
// it (8-bit base; 1.66e-3 of that its own rounding), with s A rounded as well 2.64e-3.
//
// A workgroup computes 32 NI WM tokens x 64 WN features with WM x WN waves, each
// 32 NI tokens x 64 features: 2 NI accumulators of v_mfma_f32_32x32x16_bf16, each a
// 32 (features) x 32 (tokens) block of dX^T.  The contraction advances 64 outputs n
// a step through S LDS stages that buffer loads fill directly, S steps ahead.
//  * dY: rows of 128 bytes, pieces of row m XOR-swizzled by (m >> 1) & 7.
//  * bf16 weight: rows n of 128 WN bytes, pieces XOR-swizzled by 4 (n & 3); an
//    operand is two transposing reads of four rows.
//  * 8-bit weight: rows n of 64 WN bytes, pieces XOR-swizzled by 2 (n & 7); an
//    operand is one transposing read of eight rows' codes, which become bf16(code
//    scale[n]), the value a bf16 copy of the base would hold.  For few tokens that
//    copy is most of the work: without it the backward of 16 tokens x 4096 x 4096
//    takes 18 us, with it 35.  Above 512 tokens decoding once for all of them costs
//    less (kCodesMaxM).
//  * NF4 weight: rows n of 32 WN bytes, pieces XOR-swizzled by n & 6; one transposing
//    read gives eight rows of 32 bytes' columns, whose high nibbles are the operand of
//    the even features and whose low ones that of the odd (so a lane's sums are eight
//    features in a row).  A weight is bf16(level[nibble] constant), the value of the
//    base's own backward; levels from LDS (16 of them, in different banks), the block
//    constants [K / 64, N] decoded in the launch before.  That lookup, a read per
//    weight, is what the step waits for (1.2 us, codes 0.8).
// Where N ends inside a step, both operands past it are zero.  A split contraction's
// fp32 sums go to the workspace and are added in a fixed order.
//
// What bounds it: few tokens, the start of a workgroup and the steps' latency (16 x
// 4096 x 4096 in 16 splits 10 us; its 17 MB of weight are 3.4 at a copy's rate);
// many, the matrix units at the clock that power leaves (4000 x 4096 x 4104 bf16 126
// us, 1.07 PFLOP/s).  The tile engine that takes such N in linear_bwd: 52 us for 300
// tokens (here 22 and 5 for the split's reduction), 84 for 1200.  Where 256 divides N
// a bf16 base stays with launch_dx, whose largest tile keeps its operands in registers
// longer (4001 x 4096 x 11008: 282 us; here, at 11000 outputs, 319).
#include <type_traits>

#include "device_common.h"
#include "int8_grads.h"
#include "kernels.h"

namespace qlk {

constexpr int kDxStep = 64;     // outputs per step

struct Dx8Args {
  const uint16_t* dY;   // [M, N]
  int M, N, K;
  const void* W;        // [N, K] bf16, codes or packed nibbles
  const float* sw;      // codes' row scales, or the nibbles' block constants [K / 64, N]
  float lv[16];         // the nibbles' levels
  const uint16_t* U;    // [M, r] bf16, of s U
  const uint16_t* A;    // [r, K]
  int r;
  uint16_t* dX;         // [M, K]
  int accumulate;
  int tiles_m, tiles_k, group_m;
  float* part;          // split contraction: fp32 [splits][M, K]
  int kz_len;           // steps per split; 0: one pass
  int blocks;           // workgroups of dX; the rest are the gradients'
};

typedef int i32x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i32x2_t* lds_i32x2_ptr;

// Eight codes of consecutive rows times the rows' scales.
__device__ __forceinline__ bf16x8_t scaled_codes(i32x2_t v, const float (&s)[8]) {
  uint32_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int w = v[e >> 1], b = 16 * (e & 1);
    o[e] = pack_bf16x2((float)(int8_t)(w >> b) * s[2 * e], (float)(int8_t)(w >> (b + 8)) * s[2 * e + 1]);
  }
  return __builtin_bit_cast(bf16x8_t, make_uint4(o[0], o[1], o[2], o[3]));
}

constexpr int dx8_row(int base, int features) {   // bytes of a weight row's features
  return base == kDxBf16 ? 2 * features : base == kDxCodes ? features : features / 2;
}
// The stages are arrays of their own (of one array the compiler would wait for every
// load before each read).
template <int BASE, int NI, int WM, int WN, int S>
struct Dx8Lds {
  static constexpr int Y = 32 * NI * WM * 128, W = 64 * dx8_row(BASE, 64 * WN);
  static constexpr int C = BASE == kDxNF4 ? 64 * WN : BASE == kDxCodes ? 64 : 4;
  static constexpr int Y2 = S == 3 ? Y : 16, W2 = S == 3 ? W : 16;
};

template <int BASE, int NI, int WM, int WN, int S>
__device__ __forceinline__ void dx8_tile(const Dx8Args& g, uint8_t* y0, uint8_t* w0, float* s0, uint8_t* y1,
                                         uint8_t* w1, float* s1, uint8_t* y2, uint8_t* w2, float* s2, float* lv) {
  constexpr int NJ = 2, TM = 32 * NI * WM, TF = 64 * WN, NW = WM * WN;
  constexpr bool W8 = BASE == kDxCodes, W4 = BASE == kDxNF4;
  constexpr int RB = dx8_row(BASE, TF), RP = RB / 16;      // bytes and pieces of a weight row
  constexpr int YL = TM / 8 / NW, WL = RB / 16 / NW;       // a wave's loads of a step (1 KB each)
  constexpr int L = YL + WL + (W8 || W4 ? 1 : 0);          // and 64 scales
  constexpr int YB = TM * 128, WB = 64 * RB;
  static_assert(YL * NW * 8 == TM && WL * NW * 16 == RB, "whole loads");
  static_assert(S == 2 || S == 3, "stages");
  // (+: values, not a choice of variables, which would keep them in memory)
  auto yb = [&](int b) { return b == 0 ? +y0 : b == 1 ? +y1 : +y2; };
  auto wb = [&](int b) { return b == 0 ? +w0 : b == 1 ? +w1 : +w2; };
  auto sb = [&](int b) { return b == 0 ? +s0 : b == 1 ? +s1 : +s2; };
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 31, h = lane >> 5, grp = lane >> 4, gi = lane & 15;
  const int fg = wave % WN, tq = wave / WN;                // the wave's features and tokens

  const int ntiles = g.tiles_m * g.tiles_k;
  const int z = (int)blockIdx.x / ntiles;
  int tm, tk;
  tile_coords((int)blockIdx.x % ntiles, g.tiles_m, g.tiles_k, g.group_m, tm, tk);
  const int m0 = tm * TM, k0 = tk * TF;
  const int nsteps = (g.N + kDxStep - 1) / kDxStep;
  const int kz0 = g.kz_len ? z * g.kz_len : 0;
  const int kz1 = g.kz_len ? min(nsteps, kz0 + g.kz_len) : nsteps;
  const int cut = g.N % kDxStep ? nsteps - 1 : -1;         // the step that N ends in
  const int left = g.N - kDxStep * (nsteps - 1);

  // dY: load i of wave w fills rows 8 (YL w + i) .. +7, lane l row l / 8 of them,
  // physical piece l % 8.  Weight: load i of wave w fills the rows of pieces
  // 64 (WL w + i) .. +63.
  const __amdgpu_buffer_rsrc_t ry = rsrc_whole(g.dY, (uint32_t)((int64_t)g.M * g.N * 2));
  const __amdgpu_buffer_rsrc_t rw = rsrc_whole(g.W, (uint32_t)((int64_t)g.N * dx8_row(BASE, g.K)));
  const __amdgpu_buffer_rsrc_t rsw = rsrc_whole(g.sw, W8 ? (uint32_t)g.N * 4 : W4 ? (uint32_t)g.N * (g.K / 64) * 4 : 0);
  auto yswz = [](int row) { return (row >> 1) & 7; };
  auto wswz = [](int row) { return W4 ? row & 6 : W8 ? 2 * (row & 7) : 4 * (row & 3); };
  uint32_t yoff[YL], ycut[YL], woff[WL], wcut[WL];
#pragma unroll
  for (int i = 0; i < YL; ++i) {
    const int row = 8 * (YL * wave + i) + (lane >> 3);
    const int piece = (lane & 7) ^ yswz(row);
    yoff[i] = m0 + row < g.M ? (uint32_t)(((int64_t)(m0 + row) * g.N + piece * 8) * 2) : kOOB;
    ycut[i] = piece * 8 < left ? yoff[i] : kOOB;
  }
#pragma unroll
  for (int i = 0; i < WL; ++i) {
    const int p = 64 * (WL * wave + i) + lane, row = p / RP;
    const int col = k0 + ((p % RP) ^ wswz(row)) * (W4 ? 32 : W8 ? 16 : 8);
    woff[i] = col < g.K ? (uint32_t)((int64_t)row * dx8_row(BASE, g.K) + dx8_row(BASE, col)) : kOOB;
    wcut[i] = row < left ? woff[i] : kOOB;
  }
  const int kblk = k0 / 64 + wave;                         // W4: the wave's blocks
  const uint32_t soff = !W4 ? 4 * lane : kblk < g.K / 64 ? (uint32_t)(kblk * g.N + lane) * 4 : kOOB;
  const uint32_t scut = lane < left ? soff : kOOB;
  const uint32_t wstep = (uint32_t)kDxStep * dx8_row(BASE, g.K);
  typedef __attribute__((address_space(3))) void* lds_ptr;
  auto load_l = [&](int l, int buf, int kb) {
    const uint32_t k = (uint32_t)__builtin_amdgcn_readfirstlane(kb);
    const bool end = (int)k == cut;
    if (l < YL)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ry, (lds_ptr)(yb(buf) + 1024 * (YL * wave + l)), 16,
                                               end ? ycut[l] : yoff[l], k * 128, 0, 0);
    else if (l < YL + WL)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_ptr)(wb(buf) + 1024 * (WL * wave + l - YL)), 16,
                                               end ? wcut[l - YL] : woff[l - YL], k * wstep, 0, 0);
    else   // codes: every wave the same 64
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsw, (lds_ptr)(sb(buf) + (W4 ? 64 * wave : 0)), 4,
                                               end ? scut : soff, k * 256, 0, 0);
  };
  int yrd[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) yrd[t] = c * 128 + (((2 * t + h) ^ yswz(c)) * 16);
  auto yfrag = [&](int buf, int i, int t) -> bf16x8_t {
    return *reinterpret_cast<const bf16x8_t*>(yb(buf) + 32 * (NI * tq + i) * 128 + yrd[t]);
  };
  // Features 64 fg + 32 j + c, rows 16 t + 8 h + 0..7.  j sets a bit of the piece that
  // the swizzle XORs: its place is that of j = 0 XOR 32 features.
  int wrd[2];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int n = W8 || W4 ? 8 * (grp >> 1) + (gi >> 1) : 8 * (grp >> 1) + 4 * half + (gi >> 2);
    const int p = W4 ? 2 * fg + (grp & 1) : W8 ? 4 * fg + (grp & 1) : 8 * fg + 2 * (grp & 1) + ((gi & 3) >> 1);
    wrd[half] = n * RB + ((p ^ wswz(n)) * 16) + 8 * (gi & 1);
  }
  auto wraw = [&](int buf, int j, int t) -> i32x2_t {
    return __builtin_amdgcn_ds_read_tr8_b64_v2i32(
        (lds_i32x2_ptr)(wb(buf) + 16 * RB * t + (W4 ? wrd[0] : wrd[0] ^ (32 * j))));
  };
  auto wfrag = [&](int buf, int j, int t) -> bf16x8_t {
    const uint16_t* const base = reinterpret_cast<const uint16_t*>(wb(buf) + 16 * RB * t);
    const v4s_t lo = lds_read_tr16(base + ((wrd[0] ^ (64 * j)) >> 1));
    const v4s_t hi = lds_read_tr16(base + ((wrd[1] ^ (64 * j)) >> 1));
    typedef short v8s_t __attribute__((ext_vector_type(8)));
    const v8s_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    return __builtin_bit_cast(bf16x8_t, v);
  };

  f32x16_t acc[NJ][NI];
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[j][i][v] = 0.0f;

  bf16x8_t a[2][NJ], b[2][NI];   // [MFMA step parity][block]
  i32x2_t q[4][NJ];              // codes or nibbles, by MFMA step
  float sv[8], lw[W4 ? 16 : 1];  // the next MFMA step's scales, and levels
  // Operands of MFMA step t of the step in stage `buf`.  The nibbles of a whole step
  // come with its first, so that their levels can be looked up in front of the MFMAs
  // (16 x 4096 x 4096 11.8 -> 10.2 us; codes, which need no lookup, lose 4 % by it).
  auto read = [&](int buf, int t) {
#pragma unroll
    for (int i = 0; i < NI; ++i) b[t & 1][i] = yfrag(buf, i, t);
    if constexpr (BASE == kDxBf16)
#pragma unroll
      for (int j = 0; j < NJ; ++j) a[t & 1][j] = wfrag(buf, j, t);
    if constexpr (W8 || W4) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (W4 ? t == 0 : u == t)
#pragma unroll
          for (int j = 0; j < (W4 ? 1 : NJ); ++j) q[u][j] = wraw(buf, j, u);
      const float* const s = sb(buf) + (W4 ? 64 * fg : 0) + 16 * t + 8 * h;
      const float4 lo = *reinterpret_cast<const float4*>(s);
      const float4 hi = *reinterpret_cast<const float4*>(s + 4);
      sv[0] = lo.x; sv[1] = lo.y; sv[2] = lo.z; sv[3] = lo.w;
      sv[4] = hi.x; sv[5] = hi.y; sv[6] = hi.z; sv[7] = hi.w;
    }
  };
  auto look = [&](int t) {       // levels of rows e, even features and odd
    if constexpr (W4)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t w = (uint32_t)q[t][0][e >> 2] >> (8 * (e & 3));
        lw[2 * e] = lv[w >> 4 & 15];
        lw[2 * e + 1] = lv[w & 15];
      }
  };
  auto convert = [&](int t) {
    if constexpr (W8)
#pragma unroll
      for (int j = 0; j < NJ; ++j) a[t & 1][j] = scaled_codes(q[t][j], sv);
    if constexpr (W4)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = pack_bf16x2(lw[4 * e + j] * sv[2 * e], lw[4 * e + 2 + j] * sv[2 * e + 1]);
        a[t & 1][j] = __builtin_bit_cast(bf16x8_t, make_uint4(o[0], o[1], o[2], o[3]));
      }
  };
  if constexpr (W4) {
    if (tid < 16) {
      float v = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; ++e) v = tid == e ? g.lv[e] : v;   // no dynamic index
      lv[tid] = v;
    }
    __syncthreads();
  }
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int l = 0; l < L; ++l) load_l(l, s, min(kz0 + s, kz1 - 1));
  __builtin_amdgcn_s_waitcnt(wait_for((S - 1) * L, 0));   // the first step has landed
  __builtin_amdgcn_s_barrier();
  read(0, 0);
  look(0);
  convert(0);

  // One step: four MFMA steps; each reads the next one's operands first and converts
  // them last.  The last one reads the next step's, which every wave has waited for
  // before the barrier in front of it (vmcnt).  Before the same barrier every wave's
  // reads of this step's stage, scales and nibbles too, have ended (lgkmcnt): the loads
  // of step kb + S go into it.
  auto step = [&](auto Pc, int kb) {
    constexpr int P = decltype(Pc)::value, nxt = (P + 1) % S;
    constexpr int Q = NI * NJ;
    const int kload = min(kb + S, kz1 - 1);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      __builtin_amdgcn_sched_barrier(0);
      if (t == 3) {
        __builtin_amdgcn_s_waitcnt(wait_for((S - 2) * L, 0));
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
      }
      read(t == 3 ? nxt : P, (t + 1) & 3);
      if (t < 3) look(t + 1);
      if (t == 3)
#pragma unroll
        for (int l = 0; l < L; ++l) load_l(l, P, kload);
#pragma unroll
      for (int u = 0; u < Q; ++u)
        acc[u / NI][u % NI] = mfma_32x32x16(a[t & 1][u / NI], b[t & 1][u % NI], acc[u / NI][u % NI]);
      if (t == 3) look(0);
      convert((t + 1) & 3);
    }
  };
  // whole groups of S steps without a branch between them
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

  // Adapter term: A^T U^T over r in steps of 16 into the accumulators.
  const int kw = k0 + 64 * fg;               // first feature of this wave
  const int mw = m0 + 32 * NI * tq;          // first token
  const __amdgpu_buffer_rsrc_t ru = rsrc_whole(g.U, (uint32_t)(g.M * g.r * 2));
  const __amdgpu_buffer_rsrc_t ra = rsrc_whole(g.A, (uint32_t)(g.r * g.K * 2));
  if (z == 0)
    for (int r0 = 0; r0 < g.r; r0 += 16) {
      const int rr = r0 + 8 * h;
      bf16x8_t uop[NI];
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int m = mw + 32 * i + c;
        uop[i] = __builtin_bit_cast(
            bf16x8_t, bload128(ru, m < g.M && rr < g.r ? (uint32_t)((m * g.r + rr) * 2) : kOOB));
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int kf = W4 ? kw + 2 * c + j : kw + 32 * j + c;
        uint32_t av[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          av[e] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(
              ra, kf < g.K && rr < g.r ? ((rr + e) * g.K + kf) * 2 : (int)kOOB, 0, 0);
        const bf16x8_t afr = __builtin_bit_cast(
            bf16x8_t, make_uint4(av[0] | av[1] << 16, av[2] | av[3] << 16, av[4] | av[5] << 16,
                                 av[6] | av[7] << 16));
#pragma unroll
        for (int i = 0; i < NI; ++i) acc[j][i] = mfma_32x32x16(afr, uop[i], acc[j][i]);
      }
    }

  // Accumulator [j][i]: lane holds token mw + 32 i + c and features
  // kw + 32 j + 8 (v / 4) + 4 h + (v % 4).
  // (W4: blocks j = 0, 1 are the even and the odd features: 16 (v / 4) + 8 h + 2 (v % 4) + j.)
  if constexpr (W4) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int m = mw + 32 * i + c;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int k = kw + 16 * v + 8 * h;
        if (m >= g.M || k >= g.K) continue;
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = acc[e & 1][i][4 * v + (e >> 1)];
        const int64_t at = (int64_t)m * g.K + k;
        if (g.kz_len) {
          float4* const part = reinterpret_cast<float4*>(g.part + (int64_t)z * g.M * g.K + at);
          part[0] = make_float4(x[0], x[1], x[2], x[3]);
          part[1] = make_float4(x[4], x[5], x[6], x[7]);
          continue;
        }
        uint4* const out = reinterpret_cast<uint4*>(g.dX + at);
        if (g.accumulate) {
          const uint4 old = *out;
          const uint32_t ow[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[2 * e] += bf16_to_f32(ow[e] & 0xffffu);
            x[2 * e + 1] += bf16_to_f32(ow[e] >> 16);
          }
        }
        *out = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                          pack_bf16x2(x[6], x[7]));
      }
    }
  } else {
    if (g.kz_len) {
      float* const part = g.part + (int64_t)z * g.M * g.K;
  #pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int m = mw + 32 * i + c;
  #pragma unroll
        for (int j = 0; j < NJ; ++j)
  #pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int k = kw + 32 * j + 8 * v + 4 * h;
            if (m < g.M && k < g.K)
              *reinterpret_cast<float4*>(part + (int64_t)m * g.K + k) =
                  make_float4(acc[j][i][4 * v], acc[j][i][4 * v + 1], acc[j][i][4 * v + 2],
                              acc[j][i][4 * v + 3]);
          }
      }
      return;
    }
    // Old values are added here, then the tile goes out as bf16 rows of 2 TF bytes
    // through the stages, 32 tokens (a block) at a time in place of whole stages, the
    // 16-byte pieces of a row XOR-swizzled by its number.
    constexpr int BB = 32 * 2 * TF, PR = TF / 8;             // bytes of a block, pieces of a row
    constexpr int WBL = WB / BB, BLOCKS = NI * WM;           // blocks in a weight stage
    static_assert(WBL >= 1 && BLOCKS <= S * (WBL + YB / BB), "blocks");
    auto ob = [&](int k) -> uint8_t* {
      const int n = k / WBL;
      if (n < S) return wb(n) + (k % WBL) * BB;
      const int y = k - S * WBL, per = YB / BB > 0 ? YB / BB : 1;
      return yb(y / per) + (y % per) * BB;
    };
  #pragma unroll
    for (int i = 0; i < NI; ++i) {
      uint8_t* const row = ob(NI * tq + i) + c * (2 * TF);
      const int m = mw + 32 * i + c;
  #pragma unroll
      for (int j = 0; j < NJ; ++j)
  #pragma unroll
        for (int v = 0; v < 4; ++v) {
          float x[4];
  #pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = acc[j][i][4 * v + e];
          const int k = kw + 32 * j + 8 * v + 4 * h;
          if (g.accumulate && m < g.M && k < g.K) {
            const uint2 old = *reinterpret_cast<const uint2*>(g.dX + (int64_t)m * g.K + k);
            x[0] += bf16_to_f32(old.x & 0xffffu);
            x[1] += bf16_to_f32(old.x >> 16);
            x[2] += bf16_to_f32(old.y & 0xffffu);
            x[3] += bf16_to_f32(old.y >> 16);
          }
          const int piece = (8 * fg + 4 * j + v) ^ (c & (PR - 1));
          *reinterpret_cast<uint2*>(row + 16 * piece + 8 * h) =
              make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
        }
    }
    __syncthreads();
    constexpr int RW = 64 * NW / PR;                         // rows that a pass stores
    const int prow = tid / PR, pp = tid % PR;
  #pragma unroll
    for (int e = 0; e < TM / RW; ++e) {
      const int row = RW * e + prow, rl = row & 31;          // RW divides 32
      const uint4 v = *reinterpret_cast<const uint4*>(ob(RW * e / 32) + rl * (2 * TF) +
                                                      16 * (pp ^ (rl & (PR - 1))));
      const int m = m0 + row, k = k0 + 8 * pp;
      if (m < g.M && k < g.K) *reinterpret_cast<uint4*>(g.dX + (int64_t)m * g.K + k) = v;
    }
  }
}

// The host pass does not keep a kernel template whose body calls these loads from a
// lambda: one plain kernel per form.  Where the workgroups are of four waves, those of
// the gradients follow in the same grid, on LDS of a weight stage: a launch less, and
// the gradients' loads run beside the tiles (the whole backward, 16 x 256 x 256: 13.8
// -> 11.0 us; 16 x 4096 x 4096: 24 -> 18).
#define QLK_DX8_LDS(...)                                                                 \
  typedef Dx8Lds<__VA_ARGS__> L;                                                         \
  __shared__ __attribute__((aligned(16))) uint8_t y0[L::Y], w0[L::W], y1[L::Y], w1[L::W]; \
  __shared__ __attribute__((aligned(16))) uint8_t y2[L::Y2], w2[L::W2];                  \
  __shared__ __attribute__((aligned(16))) float s0[L::C], s1[L::C], s2[L::C], lv[16]
#define QLK_DX8_KERNEL(name, threads, ...)                                               \
  __global__ void __launch_bounds__(threads) name(Dx8Args g) {                           \
    QLK_DX8_LDS(__VA_ARGS__);                                                            \
    dx8_tile<__VA_ARGS__>(g, y0, w0, s0, y1, w1, s1, y2, w2, s2, lv);                        \
  }
#define QLK_DX8_GRADS_KERNEL(name, RT, ...)                                              \
  __global__ void __launch_bounds__(256) name(Dx8Args g, Grad8Args ga) {                 \
    QLK_DX8_LDS(__VA_ARGS__);                                                            \
    __shared__ __attribute__((aligned(16))) uint8_t gl[grads8_lds<RT>() <= L::W ? 16 : grads8_lds<RT>()]; \
    static_assert(kGradWaves8 == 4, "waves");                 \
    if ((int)blockIdx.x < g.blocks) dx8_tile<__VA_ARGS__>(g, y0, w0, s0, y1, w1, s1, y2, w2, s2, lv); \
    else grads8_block<RT>(ga, (int)blockIdx.x - g.blocks, grads8_lds<RT>() <= L::W ? w0 : gl);                           \
  }
QLK_DX8_GRADS_KERNEL(k_dx8_codes_32_r16, 1, kDxCodes, 1, 1, 4, 3)
QLK_DX8_GRADS_KERNEL(k_dx8_codes_32_r32, 2, kDxCodes, 1, 1, 4, 3)
QLK_DX8_GRADS_KERNEL(k_dx8_codes_64_r16, 1, kDxCodes, 2, 1, 4, 3)
QLK_DX8_GRADS_KERNEL(k_dx8_codes_64_r32, 2, kDxCodes, 2, 1, 4, 3)
QLK_DX8_GRADS_KERNEL(k_dx8_codes_128_r16, 1, kDxCodes, 4, 1, 4, 3)
QLK_DX8_GRADS_KERNEL(k_dx8_codes_128_r32, 2, kDxCodes, 4, 1, 4, 3)
QLK_DX8_GRADS_KERNEL(k_dx8_bf16_64_r16, 1, kDxBf16, 2, 1, 4, 3)
QLK_DX8_GRADS_KERNEL(k_dx8_bf16_64_r32, 2, kDxBf16, 2, 1, 4, 3)
QLK_DX8_GRADS_KERNEL(k_dx8_nf4_32_r16, 1, kDxNF4, 1, 1, 4, 3)
QLK_DX8_GRADS_KERNEL(k_dx8_nf4_32_r32, 2, kDxNF4, 1, 1, 4, 3)
QLK_DX8_GRADS_KERNEL(k_dx8_nf4_64_r16, 1, kDxNF4, 2, 1, 4, 3)
QLK_DX8_GRADS_KERNEL(k_dx8_nf4_64_r32, 2, kDxNF4, 2, 1, 4, 3)
QLK_DX8_KERNEL(k_dx8_bf16_128, 512, kDxBf16, 2, 2, 4, 3)
QLK_DX8_KERNEL(k_dx8_bf16_256, 512, kDxBf16, 4, 2, 4, 2)

struct Dx8Form {
  void (*kernel)(Dx8Args);                      // or, with the gradients,
  void (*r16)(Dx8Args, Grad8Args);              // of up to 16 ranks,
  void (*r32)(Dx8Args, Grad8Args);              // of 32 at a time
  int base;
  int tm, threads, per_cu;
  double alone, full;      // us of a step: in one workgroup; with one on every CU
};
// Fitted to 16 to 4000 tokens x 4096 x 4104, one to sixteen splits (all forms; the
// fit is within 3 us of what was measured); 32 splits for a few tokens of a long
// contraction (4 x 128 x 22744: 19 us with 16, 11 with 32).  Fewer tokens a tile: the weight is
// decoded or staged again for each tile row (512 tokens on codes unsplit: 48, 49 and
// 66 us at 32, 64 and 128); more: too few workgroups (16 tokens: 40, 43, 61).
static const Dx8Form kDx8Forms[] = {{nullptr, k_dx8_codes_32_r16, k_dx8_codes_32_r32, kDxCodes, 32, 256, 2, 0.53, 0.58},
                                    {nullptr, k_dx8_codes_64_r16, k_dx8_codes_64_r32, kDxCodes, 64, 256, 2, 0.58, 0.83},
                                    {nullptr, k_dx8_codes_128_r16, k_dx8_codes_128_r32, kDxCodes, 128, 256, 1, 0.86, 1.45},
                                    {nullptr, k_dx8_bf16_64_r16, k_dx8_bf16_64_r32, kDxBf16, 64, 256, 1, 0.45, 0.63},
                                    {nullptr, k_dx8_nf4_32_r16, k_dx8_nf4_32_r32, kDxNF4, 32, 256, 2, 0.90, 1.30},
                                    {nullptr, k_dx8_nf4_64_r16, k_dx8_nf4_64_r32, kDxNF4, 64, 256, 2, 0.90, 1.30},
                                    {k_dx8_bf16_128, nullptr, nullptr, kDxBf16, 128, 512, 1, 0.55, 0.93},
                                    {k_dx8_bf16_256, nullptr, nullptr, kDxBf16, 256, 512, 1, 1.08, 1.72}};
constexpr int kDx8MaxSplits = 32;

// The form and split of the contraction with the least expected time: whole rounds of
// workgroups and a last one whose steps take longer the more CUs it fills, and for a
// split the partial sums' way out and back and the reduction's launch.
Dx8Plan plan_dx8(int64_t M, int64_t K, int64_t N, int base) {
  Dx8Plan p{};
  p.form = -1;
  const int64_t steps = (N + kDxStep - 1) / kDxStep;
  double best = 0.0;
  for (int f = 0; f < (int)(sizeof(kDx8Forms) / sizeof(kDx8Forms[0])); ++f) {
    const Dx8Form& F = kDx8Forms[f];
    if (F.base != base) continue;
    const int64_t tiles = ((M + F.tm - 1) / F.tm) * ((K + 255) / 256);
    for (int splits = 1; splits <= kDx8MaxSplits; ++splits) {
      if (splits > 1 && (tiles * splits > F.per_cu * kCUs || steps / splits < 3)) break;
      const int64_t len = (steps + splits - 1) / splits;
      const int64_t wgs = tiles * splits, whole = wgs / kCUs, rest = wgs % kCUs;
      double us = 6.0 + len * (whole * F.full +
                               (rest ? F.alone + (F.full - F.alone) * rest / kCUs : 0.0));
      if (splits > 1) us += 3.5 + 0.1 * splits + (double)M * K * splits * 8.0 / 8e6;
      if (p.form < 0 || us < best) {
        best = us;
        p.form = f;
        p.kz_len = splits > 1 ? (int)len : 0;
      }
    }
  }
  p.splits = p.kz_len ? (int)((steps + p.kz_len - 1) / p.kz_len) : 1;
  p.grads = !kDx8Forms[p.form].kernel;
  p.bytes = p.kz_len ? (size_t)p.splits * M * K * 4 : 0;
  return p;
}

hipError_t launch_dx8(const uint16_t* dY, int64_t M, int64_t K, int64_t N, const Dx8Base& W,
                      const uint16_t* U, const uint16_t* A, int r, uint16_t* dX, bool accumulate, float* part, const Dx8Plan& p, Grad8Args& ga,
                      hipStream_t st) {
  const Dx8Form& F = kDx8Forms[p.form];
  Dx8Args g{};
  g.dY = dY; g.M = (int)M; g.N = (int)N; g.K = (int)K;
  g.W = W.weight;
  g.sw = W.scale;
  if (F.base == kDxNF4)
    for (int i = 0; i < 16; ++i) g.lv[i] = W.levels[i];
  g.U = U; g.A = A; g.r = r; g.dX = dX;
  g.accumulate = accumulate ? 1 : 0;
  g.tiles_m = (int)((M + F.tm - 1) / F.tm);
  g.tiles_k = (int)((K + 255) / 256);
  g.group_m = group_for(g.tiles_m, g.tiles_k, F.tm * N * 2.0, (double)N * dx8_row(F.base, 256));
  g.part = part;
  g.kz_len = p.kz_len;
  g.blocks = (int)((int64_t)g.tiles_m * g.tiles_k * p.splits);
  const dim3 block(F.threads);
  if (F.kernel)
    hipLaunchKernelGGL(F.kernel, dim3(g.blocks), block, 0, st, g);
  else if (r <= 16)
    hipLaunchKernelGGL(F.r16, dim3(g.blocks + grads8_blocks<1>(ga)), block, 0, st, g, ga);
  else
    hipLaunchKernelGGL(F.r32, dim3(g.blocks + grads8_blocks<2>(ga)), block, 0, st, g, ga);
  if (p.kz_len) return launch_split_reduce(part, p.splits, M * K, dX, accumulate, st);
  return hipGetLastError();
}

}  // namespace qlk
