// The adapter's products where the layer's input is kept in 8-bit rows
// (X = sx Cx), all sums in fp32:
//
//   T = X A^T = sx (Cx A^T)                              [M, r]
//   U = dY B                                             [M, r]
//   dA = s U^T X = s (sx U)^T Cx,   dB = s dY^T T        [r, K], [N, r]
//                       (llm-compass "QLoRA", 方法与公式, the equation and its
//                        derivatives)
//
// Codes are whole numbers up to 127 and exact in bf16, so Cx goes into bf16
// MFMAs without rounding and its scale stays outside the sum.  Where T or U
// feed an MFMA they go in as bf16 terms of their own sign: two where the result
// is rounded to bf16, three (all 24 bits) where it is kept in fp32.
#include <type_traits>

#include "dequant_block.h"
#include "device_common.h"
#include "int8_grads.h"
#include "kernels.h"
#include "terms.h"

namespace qlk {

__device__ __forceinline__ uint4 zero_unless(bool ok, uint4 v) {
  return make_uint4(ok ? v.x : 0u, ok ? v.y : 0u, ok ? v.z : 0u, ok ? v.w : 0u);
}

// What a rank-r product leaves (any may be null), as MFMA operands where bf16
// terms are asked for, 1 KB that a wave loads lane after lane:
//   two     the forward's [block of 32 tokens][rank tile][term][lane][8]: lane
//           (c, h) holds ranks 16 t + 8 h .. +7 of token c; hi and mid terms of
//           s sum; tokens and ranks past the end are zero
//   packed  the gradients' [chunk][term][rank tile][lane][8]: lane (i, g) holds
//           rank 16 t + i of tokens 8 g .. +7 of the chunk; three terms of
//           pscale[m] sum; tokens past the end are zero
struct RankOut {
  float* sum;              // [M, r]
  uint16_t* bf16;          // [M, r], of s sum
  uint16_t* two;
  float s;
  uint16_t* packed;
  const float* pscale;     // [M], or null: 1
};

__device__ __forceinline__ uint32_t pair(uint16_t lo, uint16_t hi) { return lo | (uint32_t)hi << 16; }
__device__ __forceinline__ uint4 eight(const uint16_t (&v)[8]) {
  return make_uint4(pair(v[0], v[1]), pair(v[2], v[3]), pair(v[4], v[5]), pair(v[6], v[7]));
}
// Terms of eight tokens m8 .. m8 + 7 (8 | m8) of rank 16 t + i.
__device__ __forceinline__ void pack_terms(uint16_t* packed, int ntiles, int64_t m8, int t, int i,
                                           const float (&x)[8]) {
  uint16_t w[3][8];
#pragma unroll
  for (int v = 0; v < 8; ++v) {
    const Terms e = split(x[v]);
    w[0][v] = e.hi; w[1][v] = e.mid3; w[2][v] = e.lo;
  }
  uint4* const p = reinterpret_cast<uint4*>(packed);
  const int lane = 16 * (int)((m8 % kChunk) / 8) + i;
#pragma unroll
  for (int z = 0; z < 3; ++z) p[((m8 / kChunk * 3 + z) * ntiles + t) * 64 + lane] = eight(w[z]);
}

// out[m][j] = sum_c S[m][c] W(j, c), W(j, c) = A[j][c] or (WT) B[c][j]; S bf16 or,
// S8, codes whose row scale multiplies the finished sum.  A workgroup owns `rows`
// rows (16, or 8 where that would leave CUs idle; the MFMA's others are zero) and
// all r columns; its NW waves take every NW-th 64-wide slice of the contraction
// (v_mfma_f32_16x16x32_bf16), the next slice in flight.
//  * A load takes whole lines: eight lanes cover 128 bytes of a row (four 64 of
//    codes), and a slice of B is one block of memory.  Loaded as the MFMA wants
//    them, a row per lane, 64 lanes took 60 cycles a load where they take 16 so
//    (T, 4096 columns: 3 loads a slice, 7.0 us at rank 16; 9, 20 us at rank 64,
//    from one workgroup to 128).  The pieces go through a slab of LDS per wave,
//    XOR-swizzled by row so that neither side has bank conflicts.
//  * Loads cost no address arithmetic: a lane's offsets are fixed, a slice moves
//    the scalar offset; a slice past the end reads a resource of no bytes, the
//    last one (where 64 does not divide C) uses offsets of its own.
//  * The waves' sums are added through LDS in a fixed order, a thread per (row,
//    column), then leave as terms, a thread per eight of them.
struct RankJob {
  const void* S;           // [M, C], bf16 or codes
  const float* sx;         // the codes' row scales
  int M, C;
  const uint16_t* W;       // A [r, C] or B [C, r]
  int r, rows;             // rows of a workgroup
  RankOut o;
};
template <bool S8, int RT>
constexpr int rank_slab() { return 1024 * (S8 ? 1 : 2) + 2048 * RT; }   // bytes of a wave's

template <bool S8, bool WT, int RT, int NW>
__device__ __forceinline__ void rank_block(const RankJob& g, int blk, uint8_t* lds) {
  constexpr int RK = 16 * RT;
  constexpr int XN = S8 ? 1 : 2;                   // 1 KB loads of S a slice
  constexpr int SLAB = rank_slab<S8, RT>();
  static_assert(16 * RK * 4 + 128 <= SLAB, "a wave's sums, and the scales, take its slab's place");
  const void* const S = g.S;
  const float* const sx = g.sx;
  const uint16_t* const W = g.W;
  const RankOut& o = g.o;
  const int M = g.M, C = g.C, r = g.r, rows = g.rows;
  float* const rowscale = reinterpret_cast<float*>(lds + 16 * RK * 4);   // in wave 0's slab
  float* const packscale = rowscale + 16;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int row = lane & 15, grp = lane >> 4;
  const int m0 = blk * rows;
  const int nsteps = (C + 63) / 64;
  const int cut = C % 64 ? nsteps - 1 : -1;        // the slice that C ends in
  const int left = C - 64 * (nsteps - 1);          // columns of the last slice
  const uint32_t sbytes = (uint32_t)((int64_t)M * C * (S8 ? 1 : 2));
  const uint32_t wbytes = (uint32_t)((int64_t)C * r * 2);
  uint8_t* const xs = lds + wave * SLAB;
  uint8_t* const ws = xs + 1024 * XN;
  // S: rows of 64 codes in 4 pieces of 16 bytes, or of 64 bf16 in 8
  constexpr int XP = S8 ? 4 : 8;
  auto xswz = [](int i) { return S8 ? (i >> 2) & 3 : (i >> 1) & 7; };
  auto wswz = [](int i) { return (i >> 1) & 7; };
  uint32_t xoff[XN], xcut[XN], xput[XN];
#pragma unroll
  for (int n = 0; n < XN; ++n) {
    const int i = (64 / XP) * n + lane / XP, p = lane % XP;
    xoff[n] = i < rows && m0 + i < M
                  ? (uint32_t)((int64_t)(m0 + i) * C * (S8 ? 1 : 2) + 16 * p) : kOOB;
    xcut[n] = p * (S8 ? 16 : 8) < left ? xoff[n] : kOOB;
    xput[n] = (uint32_t)((i * XP + (p ^ xswz(i))) * 16);
  }
  // A: rank 16 t + 8 n + lane / 8 of load (t, n), 8 pieces of 8 values.  B: piece
  // 64 n + lane of the slice's 64 rows of r8 pieces; the loads past r8 put zeros in
  // the columns past r.  LDS: [t][64 c][16 ranks] as it is read transposed, rows
  // XOR-swizzled by 2 t, so that the tiles' pieces of a row fall on different banks,
  // and in every other 16 by 4, so that the lanes that read two of them do.
  auto bswz = [](int c, int t) { return c ^ (2 * t) ^ ((c >> 2) & 4); };
  const int r8 = r / 8;
  uint32_t woff[2 * RT], wcut[2 * RT], wput[2 * RT];
#pragma unroll
  for (int n = 0; n < 2 * RT; ++n) {
    if constexpr (WT) {
      const int p = 64 * n + lane;
      const int c = n < r8 ? p / r8 : lane, oct = n < r8 ? p % r8 : n;
      woff[n] = n < r8 ? (uint32_t)((c * r + 8 * oct) * 2) : kOOB;
      wcut[n] = c < left ? woff[n] : kOOB;
      wput[n] = (uint32_t)((oct >> 1) * 2048 + bswz(c, oct >> 1) * 32 + 16 * (oct & 1));
    } else {
      const int i = 8 * (n & 1) + lane / 8, p = lane % 8, j = 16 * (n >> 1) + i;
      woff[n] = j < r ? (uint32_t)(((int64_t)j * C + 8 * p) * 2) : kOOB;
      wcut[n] = 8 * p < left ? woff[n] : kOOB;
      wput[n] = (uint32_t)(((j * 8) + (p ^ wswz(i))) * 16);
    }
  }
  const uint32_t wstep = WT ? (uint32_t)(64 * r * 2) : 128u;
  float rs = 0.0f, ps = 1.0f;                      // of row tid
  if (tid < rows && m0 + tid < M) {
    if (S8) rs = sx[m0 + tid];
    if (o.pscale) ps = o.pscale[m0 + tid];
  }

  f32x4_t acc[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) acc[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  struct Batch { uint4 x[XN]; uint4 w[2 * RT]; };
  auto load = [&](Batch& L, int ks) {
    const bool sv = ks < nsteps, end = ks == cut;
    const __amdgpu_buffer_rsrc_t rsr = rsrc_whole(S, sv ? sbytes : 0);
    const __amdgpu_buffer_rsrc_t rw = rsrc_whole(W, sv ? wbytes : 0);
#pragma unroll
    for (int n = 0; n < XN; ++n)
      L.x[n] = bload128s(rsr, end ? xcut[n] : xoff[n], (uint32_t)ks * (S8 ? 64 : 128));
#pragma unroll
    for (int n = 0; n < 2 * RT; ++n)
      L.w[n] = bload128s(rw, end ? wcut[n] : woff[n], (uint32_t)ks * wstep);
  };
  typedef short v8s_t __attribute__((ext_vector_type(8)));
  auto use = [&](const Batch& L) {
    // A wave's LDS operations run in issue order: the stores land after the last
    // slice's reads and before this one's.
#pragma unroll
    for (int n = 0; n < XN; ++n) *reinterpret_cast<uint4*>(xs + xput[n]) = L.x[n];
#pragma unroll
    for (int n = 0; n < 2 * RT; ++n) *reinterpret_cast<uint4*>(ws + wput[n]) = L.w[n];
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
    uint4 xv[2];                          // columns 16 grp + 8 h of the slice
    if constexpr (S8) {
      codes_to_bf16(*reinterpret_cast<const uint4*>(xs + (row * 4 + (grp ^ xswz(row))) * 16), xv);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        xv[h] = *reinterpret_cast<const uint4*>(xs + (row * 8 + ((2 * grp + h) ^ xswz(row))) * 16);
    }
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        bf16x8_t bop;
        if constexpr (WT) {
          const int c = 16 * grp + 8 * h + (row >> 2);
          const uint16_t* const p = reinterpret_cast<const uint16_t*>(ws + 2048 * t) + 4 * (row & 3);
          const v4s_t lo = lds_read_tr16(p + bswz(c, t) * 16);
          const v4s_t hi = lds_read_tr16(p + bswz(c + 4, t) * 16);
          const v8s_t bv = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
          bop = __builtin_bit_cast(bf16x8_t, bv);
        } else {
          bop = *reinterpret_cast<const bf16x8_t*>(
              ws + ((16 * t + row) * 8 + ((2 * grp + h) ^ wswz(row))) * 16);
        }
        acc[t] = mfma_16x16x32(__builtin_bit_cast(bf16x8_t, xv[h]), bop, acc[t]);
      }
  };
  Batch la, lb;
  load(la, wave);
  for (int ks = wave; ks < nsteps; ks += 2 * NW) {
    load(lb, ks + NW);
    __builtin_amdgcn_sched_barrier(0);   // a slice's loads before the other's MFMAs
    use(la);
    load(la, ks + 2 * NW);
    __builtin_amdgcn_sched_barrier(0);
    use(lb);
  }
  if (tid < rows) {
    rowscale[tid] = rs;
    packscale[tid] = ps;
  }
  auto sums = [&](int q, int i, int j) -> float& {
    return reinterpret_cast<float*>(lds + q * SLAB)[i * RK + j];
  };

  // acc[t][v]: row 4 grp + v, column 16 t + row of the tile
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int v = 0; v < 4; ++v) sums(wave, 4 * grp + v, 16 * t + row) = acc[t][v];
  __syncthreads();
  for (int e = tid; e < rows * RK; e += NW * 64) {
    const int i = e / RK, j = e % RK, mm = m0 + i;
    float sum = 0.0f;
    if (mm < M && j < r) {
#pragma unroll
      for (int q = 0; q < NW; ++q) sum += sums(q, i, j);
      if (S8) sum *= rowscale[i];
      if (o.sum) o.sum[(int64_t)mm * r + j] = sum;
      if (o.bf16) o.bf16[(int64_t)mm * r + j] = f32_to_bf16(o.s * sum);
    }
    sums(0, i, j) = sum;                 // this thread's own
  }
  if (!o.two && !o.packed) return;
  __syncthreads();
  const int ntiles = (r + 15) / 16;
  if (o.two)
    for (int e = tid; e < rows * 2 * ntiles; e += NW * 64) {
      const int i = e / (2 * ntiles), oct = e % (2 * ntiles), mm = m0 + i;
      uint16_t hi[8], mid[8];
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        const Terms x = split(o.s * sums(0, i, 8 * oct + v));
        hi[v] = x.hi; mid[v] = x.mid2;
      }
      uint4* const p = reinterpret_cast<uint4*>(o.two) +
                       ((int64_t)(mm / 32) * ntiles + oct / 2) * 128 + (mm % 32) + 32 * (oct & 1);
      p[0] = eight(hi);
      p[64] = eight(mid);
    }
  if (o.packed)
    for (int e = tid; e < rows / 8 * 16 * ntiles; e += NW * 64) {
      const int j = e % (16 * ntiles), i8 = 8 * (e / (16 * ntiles));
      float x[8];
#pragma unroll
      for (int v = 0; v < 8; ++v) x[v] = sums(0, i8 + v, j) * packscale[i8 + v];
      pack_terms(o.packed, ntiles, m0 + i8, j / 16, j % 16, x);
    }
}

// Up to 32 ranks: a workgroup's own sums, no second launch.  Where a row of `bytes`
// is long its one workgroup takes longer than slices of it and a launch that adds
// them (4 to 700 tokens): U at 16 ranks 8192 columns 8 to 11 us against 9 to 12 and a
// launch, 28672 columns 19 to 22 against 14 to 19; at 32 ranks 4096 columns level,
// 8192 11 to 13 against 9 to 11.
constexpr int kRankOnce = 32;
static bool rank_once(int64_t bytes, int r) { return r <= kRankOnce && bytes * ((r + 15) / 16) < 32768; }
template <class F>
static void rank_form(int r, F f) {
  using std::integral_constant;
  if (r <= 16) f(integral_constant<int, 1>());
  else f(integral_constant<int, 2>());
}
constexpr int kRankWaves = 16;
// rows of a workgroup, and workgroups; operands are whole blocks of tokens
static int rank_blocks(RankJob& g) {
  g.rows = (g.M + 15) / 16 < kCUs ? 8 : 16;
  const int64_t m = g.o.packed || g.o.two ? ((int64_t)g.M + kChunk - 1) / kChunk * kChunk : g.M;
  return (int)((m + g.rows - 1) / g.rows);
}

template <int RT>
__global__ void __launch_bounds__(kRankWaves * 64) k_int8_T(RankJob g) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kRankWaves * rank_slab<true, RT>()];
  rank_block<true, false, RT, kRankWaves>(g, blockIdx.x, lds);
}

// ---------------------------------------------------------------------------
// The same products above 32 ranks, where a workgroup that reads all of W for 16
// rows reads it too often (U, 4001 tokens x 4096, rank 64: 25 us), and for long rows
// at fewer (rank_once).  A workgroup
// takes 64 rows, 64 ranks and one of `zs` slices of the contraction; its four waves
// take 32 rows x 32 ranks each (v_mfma_f32_32x32x16_bf16).  The contraction
// advances 64 columns a step through four LDS stages that buffer loads fill three
// steps ahead.  The slices' sums [zs][M][r] go to the workspace; k_int8_finish adds
// them in their order.  Slices are the fast grid index, so that an XCD keeps to its
// part of W.
struct DownJob {
  const void* S;           // [M, C], bf16 or codes
  int M, C;
  const uint16_t* W;       // A [r, C] or B [C, r]
  int r, groups;           // of 64 ranks
  int zs, zlen;            // slices, steps in one
  float* part;
};
constexpr int kDownStage = 16 * 1024;
// Most slices of the contraction: at 4001 tokens 8 took 1 us off the slices' launch and
// put 2 on the sums'; where few tiles leave CUs idle they take 6 us off 25 (2 tokens,
// 28576 columns, r = 64; 16 slices another 3, and 2 more on the sums').
constexpr int kDownSlices = 4, kDownSlicesFew = 8, kDownFewTiles = 16;

// s0 .. s3: the stages, arrays of their own (of one array the compiler would wait
// for every load before each read).
template <bool S8, bool WT>
__device__ __forceinline__ void down_block(const DownJob& g, int blk, uint8_t* s0, uint8_t* s1,
                                           uint8_t* s2, uint8_t* s3) {
  constexpr int XL = S8 ? 1 : 2, WL = 2, L = XL + WL;      // a wave's loads of a step
  constexpr int XB = 64 * (S8 ? 64 : 128);                 // bytes of S in a stage
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 31, h = lane >> 5;
  const int z = blk % g.zs, gr = blk / g.zs % g.groups;
  const int m0 = blk / g.zs / g.groups * 64, j0 = 64 * gr;
  const int M = g.M, C = g.C, r = g.r;
  const int nsteps = (C + 63) / 64;
  const int kz0 = z * g.zlen, kz1 = min(nsteps, kz0 + g.zlen);
  const int cut = C % 64 ? nsteps - 1 : -1;                // the step that C ends in
  const int left = C - 64 * (nsteps - 1);
  // S: load i of wave w fills 1 KB of rows of 64 codes (4 pieces of 16 bytes) or of
  // 64 bf16 (8 pieces); A: rows of 64 values (8 pieces); B: rows of 64 ranks.
  constexpr int XP = S8 ? 4 : 8, XR = 64 / XP;
  auto xswz = [](int i) { return S8 ? (i >> 2) & 3 : (i >> 1) & 7; };
  auto wswz = [](int i) { return WT ? ((i >> 1) & 1) << 2 : (i >> 1) & 7; };
  uint32_t xoff[XL], xcut[XL], woff[WL], wcut[WL];
#pragma unroll
  for (int n = 0; n < XL; ++n) {
    const int i = XR * (XL * wave + n) + lane / XP, p = (lane % XP) ^ xswz(i);
    xoff[n] = m0 + i < M ? (uint32_t)((int64_t)(m0 + i) * C * (S8 ? 1 : 2) + 16 * p) : kOOB;
    xcut[n] = p * (S8 ? 16 : 8) < left ? xoff[n] : kOOB;
  }
#pragma unroll
  for (int n = 0; n < WL; ++n) {
    const int i = 8 * (WL * wave + n) + lane / 8, p = (lane % 8) ^ wswz(i);
    if constexpr (WT) {
      woff[n] = j0 + 8 * p < r ? (uint32_t)((i * r + j0 + 8 * p) * 2) : kOOB;
      wcut[n] = i < left ? woff[n] : kOOB;
    } else {
      woff[n] = j0 + i < r ? (uint32_t)(((int64_t)(j0 + i) * C + 8 * p) * 2) : kOOB;
      wcut[n] = 8 * p < left ? woff[n] : kOOB;
    }
  }
  const uint32_t wstep = WT ? (uint32_t)(64 * r * 2) : 128u;
  const __amdgpu_buffer_rsrc_t rs = rsrc_whole(g.S, (uint32_t)((int64_t)M * C * (S8 ? 1 : 2)));
  const __amdgpu_buffer_rsrc_t rw = rsrc_whole(g.W, (uint32_t)((int64_t)C * r * 2));
  typedef __attribute__((address_space(3))) void* lds_ptr;
  uint8_t* const stage[4] = {s0, s1, s2, s3};
  auto load = [&](int buf, int kb) {
    const int k = __builtin_amdgcn_readfirstlane(min(kb, kz1 - 1));
    uint8_t* const st = stage[buf];
    const bool end = k == cut;
#pragma unroll
    for (int n = 0; n < XL; ++n)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr)(st + 1024 * (XL * wave + n)), 16,
                                               end ? xcut[n] : xoff[n], (uint32_t)k * (S8 ? 64 : 128), 0, 0);
#pragma unroll
    for (int n = 0; n < WL; ++n)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_ptr)(st + XB + 1024 * (WL * wave + n)), 16,
                                               end ? wcut[n] : woff[n], (uint32_t)k * wstep, 0, 0);
  };
  const int xrow = 32 * (wave >> 1) + c, wblk = 32 * (wave & 1);
  const int grp = lane >> 4, gi = lane & 15;
  f32x16_t acc;
#pragma unroll
  for (int v = 0; v < 16; ++v) acc[v] = 0.0f;
#pragma unroll
  for (int s = 0; s < 3; ++s) load(s, kz0 + s);
  auto step = [&](auto Pc, int kb) {
    constexpr int P = decltype(Pc)::value;
    // vmcnt(2 L), lgkmcnt(0): this step has landed, and the operand reads of the step
    // before have ended, in every wave that is past the barrier: the loads below go
    // into that step's stage.
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(wait_for(2 * L, 0));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    load((P + 3) % 4, kb + 3);
    const uint8_t* const xs = stage[P];
    const uint8_t* const ws = xs + XB;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      bf16x8_t xop, wop;
      if constexpr (S8) {
        const uint2 v = *reinterpret_cast<const uint2*>(xs + (xrow * 4 + (t ^ xswz(xrow))) * 16 + 8 * h);
        xop = __builtin_bit_cast(bf16x8_t, make_uint4(codes_bf16x2(v.x, 0), codes_bf16x2(v.x, 2),
                                                      codes_bf16x2(v.y, 0), codes_bf16x2(v.y, 2)));
      } else {
        xop = *reinterpret_cast<const bf16x8_t*>(xs + (xrow * 8 + ((2 * t + h) ^ xswz(xrow))) * 16);
      }
      if constexpr (WT) {
        typedef short v8s_t __attribute__((ext_vector_type(8)));
        const int k = 16 * t + 8 * (grp >> 1) + (gi >> 2), col = wblk + 16 * (grp & 1) + 4 * (gi & 3);
        auto at = [&](int row) {
          return reinterpret_cast<const uint16_t*>(ws + row * 128 + ((col >> 3) ^ wswz(row)) * 16) + (col & 7);
        };
        const v4s_t lo = lds_read_tr16(at(k)), hi = lds_read_tr16(at(k + 4));
        const v8s_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        wop = __builtin_bit_cast(bf16x8_t, v);
      } else {
        const int row = wblk + c;
        wop = *reinterpret_cast<const bf16x8_t*>(ws + (row * 8 + ((2 * t + h) ^ wswz(row))) * 16);
      }
      acc = mfma_32x32x16(wop, xop, acc);
    }
  };
  int kb = kz0;   // whole groups of four without a branch between them
  for (; kb + 4 <= kz1; kb += 4) {
    step(std::integral_constant<int, 0>(), kb);
    step(std::integral_constant<int, 1>(), kb + 1);
    step(std::integral_constant<int, 2>(), kb + 2);
    step(std::integral_constant<int, 3>(), kb + 3);
  }
  if (kb < kz1) {
    step(std::integral_constant<int, 0>(), kb);
    if (kb + 1 < kz1) step(std::integral_constant<int, 1>(), kb + 1);
    if (kb + 2 < kz1) step(std::integral_constant<int, 2>(), kb + 2);
  }
  __builtin_amdgcn_s_waitcnt(0);   // no load into LDS outlives the workgroup
  // lane: row xrow, ranks j0 + wblk + 8 (v / 4) + 4 h + (v % 4)
  const int m = m0 + xrow;
  float* const out = g.part + ((int64_t)z * M + m) * r;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int j = j0 + wblk + 8 * q + 4 * h;
    if (m < M && j < r)
      *reinterpret_cast<f32x4_t*>(out + j) = f32x4_t{acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
  }
}
// Slices so that two workgroups a CU are in reach, four steps in one at least.
static int down_blocks(DownJob& g) {
  g.groups = (g.r + 63) / 64;
  const int tiles = (g.M + 63) / 64 * g.groups, steps = (g.C + 63) / 64;
  g.zs = max(1, min(min(2 * kCUs / tiles, steps / 4),
                    tiles <= kDownFewTiles ? kDownSlicesFew : kDownSlices));
  g.zlen = (steps + g.zs - 1) / g.zs;
  g.zs = (steps + g.zlen - 1) / g.zlen;
  return tiles * g.zs;
}
static size_t down_bytes(int64_t M, int64_t C, int r) {
  DownJob g{nullptr, (int)M, (int)C, nullptr, r, 0, 0, 0, nullptr};
  down_blocks(g);
  return (size_t)g.zs * M * r * 4;
}

__global__ void __launch_bounds__(256) k_int8_T_down(DownJob g) {
  __shared__ __attribute__((aligned(16))) uint8_t s0[kDownStage];
  __shared__ __attribute__((aligned(16))) uint8_t s1[kDownStage];
  __shared__ __attribute__((aligned(16))) uint8_t s2[kDownStage];
  __shared__ __attribute__((aligned(16))) uint8_t s3[kDownStage];
  down_block<true, false>(g, blockIdx.x, s0, s1, s2, s3);
}

// A job's slices added, 32 tokens x 64 ranks a workgroup.
struct FinishJob {
  const float* part;
  int zs, M, r;
  const float* sx;         // row scales of codes, or null
  RankOut o;
};
__device__ __forceinline__ void finish_block(const FinishJob& g, int blk, float (*val)[33]) {
  const int groups = (g.r + 63) / 64, ntiles = (g.r + 15) / 16;
  const int m0 = blk / groups * 32, j0 = blk % groups * 64;
  const int i = threadIdx.x >> 3, oct = threadIdx.x & 7, m = m0 + i, j = j0 + 8 * oct;
  const RankOut& o = g.o;
  float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  float ps = 1.0f;
  if (m < g.M && j < g.r) {
    const float s = g.sx ? g.sx[m] : 1.0f;
    if (o.pscale) ps = o.pscale[m];
    // four slices' loads, or all eight's, before the first sum
    auto add = [&](auto nc) {
      constexpr int NZ = decltype(nc)::value;
      float4 a[NZ], b[NZ];
#pragma unroll
      for (int z = 0; z < NZ; ++z) {
        const float4* const p =
            reinterpret_cast<const float4*>(g.part + ((int64_t)min(z, g.zs - 1) * g.M + m) * g.r + j);
        a[z] = p[0];
        b[z] = p[1];
      }
#pragma unroll
      for (int z = 0; z < NZ; ++z) {
        if (z >= g.zs) break;
        x[0] += a[z].x; x[1] += a[z].y; x[2] += a[z].z; x[3] += a[z].w;
        x[4] += b[z].x; x[5] += b[z].y; x[6] += b[z].z; x[7] += b[z].w;
      }
    };
    if (g.zs <= kDownSlices) add(std::integral_constant<int, kDownSlices>());
    else add(std::integral_constant<int, kDownSlicesFew>());
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= s;
    const int64_t at = (int64_t)m * g.r + j;
    if (o.sum) {
      reinterpret_cast<float4*>(o.sum + at)[0] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4*>(o.sum + at)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
    if (o.bf16)
      *reinterpret_cast<uint4*>(o.bf16 + at) =
          make_uint4(pack_bf16x2(o.s * x[0], o.s * x[1]), pack_bf16x2(o.s * x[2], o.s * x[3]),
                     pack_bf16x2(o.s * x[4], o.s * x[5]), pack_bf16x2(o.s * x[6], o.s * x[7]));
  }
  if (o.two && j < 16 * ntiles) {
    uint16_t hi[8], mid[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const Terms t = split(o.s * x[e]);
      hi[e] = t.hi; mid[e] = t.mid2;
    }
    uint4* const p = reinterpret_cast<uint4*>(o.two) + ((int64_t)(m / 32) * ntiles + j / 16) * 128 + (m % 32) +
                     32 * (oct & 1);
    p[0] = eight(hi);
    p[64] = eight(mid);
  }
  if (!o.packed) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) val[8 * oct + e][i] = x[e] * ps;
  __syncthreads();
  const int jj = threadIdx.x & 63, i8 = 8 * (threadIdx.x >> 6);
  if (j0 + jj >= 16 * ntiles) return;
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = val[jj][i8 + e];
  pack_terms(o.packed, ntiles, m0 + i8, (j0 + jj) / 16, jj % 16, v);
}
static int finish_blocks(int64_t M, int r) { return (int)((M + 31) / 32 * ((r + 63) / 64)); }
__global__ void __launch_bounds__(256) k_int8_finish(FinishJob a, int na, FinishJob b) {
  __shared__ float val[64][33];
  if ((int)blockIdx.x < na) finish_block(a, blockIdx.x, val);
  else finish_block(b, (int)blockIdx.x - na, val);
}

size_t int8_two_bytes(int64_t M, int r) {
  return (size_t)((M + kChunk - 1) / kChunk) * ((r + 15) / 16) * 2048;
}

hipError_t launch_int8_T(const Int8Rows& X, int64_t M, int64_t K, const uint16_t* A, int r, float s,
                         float* T, uint16_t* T2, float* part, hipStream_t st) {
  RankOut o{};
  o.sum = T; o.two = T2; o.s = s;
  if (rank_once(K, r)) {
    RankJob g{X.codes, X.scale, (int)M, (int)K, A, r, 0, o};
    const int blocks = rank_blocks(g);
    rank_form(r, [&](auto rt) {
      constexpr int RT = decltype(rt)::value;
      hipLaunchKernelGGL(k_int8_T<RT>, dim3(blocks), dim3(kRankWaves * 64), 0, st, g);
    });
    return hipGetLastError();
  }
  DownJob g{X.codes, (int)M, (int)K, A, r, 0, 0, 0, part};
  const int blocks = down_blocks(g);
  hipLaunchKernelGGL(k_int8_T_down, dim3(blocks), dim3(256), 0, st, g);
  const FinishJob f{part, g.zs, (int)M, r, X.scale, o};
  const int nf = finish_blocks(M, r);
  hipLaunchKernelGGL(k_int8_finish, dim3(nf), dim3(256), 0, st, f, nf, f);
  return hipGetLastError();
}
// Bytes of fp32 sums that launch_int8_T needs room for.
size_t int8_T_bytes(int64_t M, int64_t K, int r) { return rank_once(K, r) ? 0 : down_bytes(M, K, r); }

// T = sum over kTSplits slices of the contraction, without the row scale, for up
// to 16 tokens: a workgroup per (16 ranks, slice), its waves' sums through LDS.
constexpr int kTpWaves = 4;
__global__ void __launch_bounds__(64 * kTpWaves)
k_int8_T_partial(const int8_t* __restrict__ X, int M, int64_t K, const uint16_t* __restrict__ A, int r,
                 float* __restrict__ part) {
  __shared__ f32x4_t red[kTpWaves][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int i = lane & 15, g = lane >> 4;
  const int j = blockIdx.x * 16 + i, z = blockIdx.y;
  const int64_t ns = K / 64, s0 = z * ns / kTSplits, s1 = (z + 1) * ns / kTSplits;
  const int8_t* const x = X + (int64_t)(i < M ? i : 0) * K + 16 * g;
  const uint16_t* const a = A + (int64_t)(j < r ? j : 0) * K + 16 * g;
  f32x4_t acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t k = s0 + wave; k < s1; k += kTpWaves) {
    const uint4 c = zero_unless(i < M, *reinterpret_cast<const uint4*>(x + 64 * k));
    const uint4 w0 = zero_unless(j < r, *reinterpret_cast<const uint4*>(a + 64 * k));
    const uint4 w1 = zero_unless(j < r, *reinterpret_cast<const uint4*>(a + 64 * k + 8));
    uint4 xs[2];
    codes_to_bf16(c, xs);
    acc = mfma_16x16x32(__builtin_bit_cast(bf16x8_t, xs[0]), __builtin_bit_cast(bf16x8_t, w0), acc);
    acc = mfma_16x16x32(__builtin_bit_cast(bf16x8_t, xs[1]), __builtin_bit_cast(bf16x8_t, w1), acc);
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int m = 4 * g + v;
    float sum = acc[v];
#pragma unroll
    for (int w = 1; w < kTpWaves; ++w) sum += red[w][lane][v];
    if (m < M && j < r) part[((int64_t)z * M + m) * r + j] = sum;
  }
}
hipError_t launch_int8_T_partial(const int8_t* X, int64_t M, int64_t K, const uint16_t* A, int r,
                                 float* part, hipStream_t st) {
  hipLaunchKernelGGL(k_int8_T_partial, dim3((unsigned)((r + 15) / 16), kTSplits), dim3(64 * kTpWaves),
                     0, st, X, (int)M, K, A, r, part);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// What the backward's products need first, in one launch whose workgroups do one
// thing each: U = dY B (s U, the dX product's operand, and sx U's terms), T's terms
// (from T, or T computed again), and the bf16 copy of the base for dX, or an NF4
// base's block constants.  U alone waits for memory most of its time and the copy is
// bound by it: side by side they take little more than the longer one.
struct PrepArgs {
  RankJob u;
  int nu;                    // workgroups of U
  RankJob t;                 // T computed again (S null: T is given)
  const float* T;            // [M, r] fp32 (three terms), or
  const uint16_t* T_bf16;    // bf16 (its own only term; the others are 2^-40 of it,
                             // which leaves the sum as it is)
  int nt;                    // workgroups of T
  const int8_t* wcodes;      // an 8-bit base, or null
  const float* wscale;
  NF4Weight w;               // else an NF4 base, if packed is not null
  int64_t words;             // of 16 codes, or of 8 weights, or block constants
  uint32_t k16;              // words of 16 codes in a row
  uint16_t* copy;            // of the base, or
  float* consts;             // an NF4 base's block constants [K / 64, N]
  Codebook4 cb;
};

// Block constants decoded, a thread per (block of a row, row), rows fastest.
constexpr int kConstRounds = 4;
__device__ __forceinline__ void prep_consts(const PrepArgs& g, int64_t blk) {
  const float mean = g.w.mean[0];
  const int64_t N = g.w.N, blocks = g.w.K / kBlock, i0 = blk * (blockDim.x * kConstRounds) + threadIdx.x;
#pragma unroll
  for (int q = 0; q < kConstRounds; ++q) {
    const int64_t i = i0 + q * blockDim.x;
    if (i >= g.words) break;
    const int64_t b = (i % N) * blocks + i / N;
    g.consts[i] = absmax_decode(g.w.codes[b], g.w.scales[b / kDQBlock], mean);
  }
}

// T's terms, a thread per (rank, eight tokens).
__device__ __forceinline__ void pack_T(const PrepArgs& g, int64_t e) {
  const int M = g.t.M, r = g.t.r, ntiles = (r + 15) / 16, width = 16 * ntiles;
  const int64_t m8 = 8 * (e / width);
  const int j = (int)(e % width);
  if (m8 >= (int64_t)(M + kChunk - 1) / kChunk * kChunk) return;
  float x[8];
#pragma unroll
  for (int v = 0; v < 8; ++v) {
    const int64_t m = m8 + v;
    x[v] = 0.0f;
    if (m < M && j < r) x[v] = g.T ? g.T[m * r + j] : bf16_to_f32(g.T_bf16[m * r + j]);
  }
  pack_terms(g.t.o.packed, ntiles, m8, j / 16, j % 16, x);
}

// The base's values rounded to bf16, as dX's own tile rounds them: the forward takes
// codes and scales as they are, dX weights up to half a step of bf16 from them, since
// its products would cost twice as much on two terms.
constexpr int kCopyRounds = 4;   // words of 16 codes per thread
__device__ __forceinline__ void copy_int8(const PrepArgs& g, int64_t blk) {
  const int64_t w0 = (blk * blockDim.x + (threadIdx.x & ~63)) * kCopyRounds + (threadIdx.x & 63);
  uint4 c[kCopyRounds];
  float s[kCopyRounds];
#pragma unroll
  for (int q = 0; q < kCopyRounds; ++q) {
    const int64_t i = min(w0 + 64 * q, g.words - 1);
    c[q] = reinterpret_cast<const uint4*>(g.wcodes)[i];
    s[q] = g.wscale[(uint32_t)i / g.k16];
  }
#pragma unroll
  for (int q = 0; q < kCopyRounds; ++q) {
    const int64_t i = w0 + 64 * q;
    if (i >= g.words) continue;
    const uint32_t w[4] = {c[q].x, c[q].y, c[q].z, c[q].w};
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      o[e] = pack_bf16x2((float)(int8_t)(w[e / 2] >> (16 * (e & 1))) * s[q],
                         (float)(int8_t)(w[e / 2] >> (16 * (e & 1) + 8)) * s[q]);
    reinterpret_cast<uint4*>(g.copy)[2 * i] = make_uint4(o[0], o[1], o[2], o[3]);
    reinterpret_cast<uint4*>(g.copy)[2 * i + 1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

__device__ __forceinline__ void prep_copy(const PrepArgs& g, int64_t blk, uint8_t* lds) {
  if (g.consts) prep_consts(g, blk);
  else if (g.wcodes) copy_int8(g, blk);
  else nf4_dequant_block(g.w.packed, g.w.codes, g.w.scales, g.w.mean, g.words, g.cb, g.copy, blk,
                         reinterpret_cast<float*>(lds));
}
template <int RT>
__global__ void __launch_bounds__(kRankWaves * 64) k_int8_prep(PrepArgs g) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kRankWaves * rank_slab<false, RT>()];   // T's are smaller
  const int b = blockIdx.x;
  if (b < g.nu) rank_block<false, true, RT, kRankWaves>(g.u, b, lds);
  else if (b >= g.nu + g.nt) prep_copy(g, b - g.nu - g.nt, lds);
  else if (g.t.S) rank_block<true, false, RT, kRankWaves>(g.t, b - g.nu, lds);
  else pack_T(g, (int64_t)(b - g.nu) * blockDim.x + threadIdx.x);
}
// Above 32 ranks: sums of slices, which k_int8_finish adds.
__global__ void __launch_bounds__(256) k_int8_prep_down(PrepArgs g, DownJob u, DownJob t) {
  __shared__ __attribute__((aligned(16))) uint8_t s0[kDownStage];
  __shared__ __attribute__((aligned(16))) uint8_t s1[kDownStage];
  __shared__ __attribute__((aligned(16))) uint8_t s2[kDownStage];
  __shared__ __attribute__((aligned(16))) uint8_t s3[kDownStage];
  const int b = blockIdx.x;
  if (b < g.nu) down_block<false, true>(u, b, s0, s1, s2, s3);
  else if (b >= g.nu + g.nt) prep_copy(g, b - g.nu - g.nt, s0);
  else if (t.S) down_block<true, false>(t, b - g.nu, s0, s1, s2, s3);
  else pack_T(g, (int64_t)(b - g.nu) * blockDim.x + threadIdx.x);
}

// ---------------------------------------------------------------------------
template <int RT>
__global__ void __launch_bounds__(64 * kGradWaves8) k_int8_grads(Grad8Args g) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[grads8_lds<RT>()];
  grads8_block<RT>(g, blockIdx.x, lds);
}

// Token count up to which dX reads an 8-bit base as it is stored.  The whole backward
// at 4096 x 4096, r = 16, read as stored and on a copy: 16 tokens 18 and 35 us, 300
// tokens 36 and 46, 512 tokens 44 and 51; 700 tokens on a copy 58.
constexpr int64_t kCodesMaxM = 512;
// And up to which launch_dx decodes an NF4 base on the way, a tile of 256 tokens: 200
// tokens x 4096 x 4096 40 us and 41 on a copy, 4096 x 11008 63 and 71; 300 tokens 50
// and 45, 90 and 80; 1000 tokens 95 and 65, 228 and 150.
constexpr int64_t kNF4MaxM = 256;
// And up to which launch_dx8 does (its tile against launch_dx's, 4096 x 4096: 16
// tokens 20 and 32 us, 64 tokens 28 and 35, 200 tokens 39 and 39; against a copy, 4096
// x 4104: 21 and 32, 29 and 31, 40 and 36).
constexpr int64_t kNibblesMaxM = 128;
Int8BwdPlan plan_int8_bwd(int64_t M, int64_t K, int64_t N, int r, int base, bool dx) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  Int8BwdPlan p{};
  const size_t pack = (size_t)((M + kChunk - 1) / kChunk) * 3 * ((r + 15) / 16) * 1024;
  p.off_U = 0;
  p.off_up = up((size_t)M * r * 2);
  p.off_tp = p.off_up + up(pack);
  p.off_ds = p.off_tp + up(pack);
  p.once = rank_once(2 * N, r);
  p.off_dt = p.off_ds + (p.once ? 0 : up(down_bytes(M, N, r)));
  p.bytes = p.off_dt + (p.once ? 0 : up(down_bytes(M, K, r)));
  // An 8-bit base is read as it is stored up to kCodesMaxM tokens, and above on a
  // bf16 copy made once per call.  An NF4 base is decoded by launch_dx8's tile up to
  // kNibblesMaxM tokens, by launch_dx's up to kNF4MaxM where that has one (256
  // divides N), and else read on a copy.
  const bool whole = dx_nf4_supported(N);
  const bool room = N * K * 2 < ((int64_t)1 << 31);
  if (dx && base == kBaseInt8) p.copy = M > kCodesMaxM;
  if (dx && base == kBaseNF4) {
    p.consts = M <= kNibblesMaxM;
    p.copy = !p.consts && room && (!whole || M > kNF4MaxM);
  }
  p.off_w = p.bytes;
  if (p.copy) p.bytes += up((size_t)N * K * 2);
  if (p.consts) p.bytes += up((size_t)N * (K / kBlock) * 4);
  p.off_part = p.bytes;
  p.any = dx && (base == kBaseInt8 ? !p.copy || !whole
                                   : p.consts || (!whole && (p.copy || base == kBaseBF16)));
  if (p.any) {
    p.dx8 = plan_dx8(M, K, N, p.consts ? kDxNF4 : base == kBaseInt8 && !p.copy ? kDxCodes : kDxBf16);
    p.bytes += up(p.dx8.bytes);
  } else if (dx && whole) {
    p.kz_len = dx_split_len(M, K, N);
    if (p.kz_len) p.bytes += up((size_t)((N / 64 + p.kz_len - 1) / p.kz_len) * M * K * 4);
  }
  return p;
}

hipError_t launch_int8_bwd(const uint16_t* dY, const Int8Rows& X, int64_t M, int64_t K, int64_t N,
                           const Int8Rows* W8, const NF4Weight& w, const uint16_t* A,
                           const uint16_t* B, int r, float s, const float* T,
                           const uint16_t* T_bf16, uint16_t* dX, float* dA, float* dB,
                           bool accumulate, void* ws, const Int8BwdPlan& p, hipStream_t st) {
  char* const base = reinterpret_cast<char*>(ws);
  uint16_t* const U = reinterpret_cast<uint16_t*>(base + p.off_U);
  uint16_t* const up = reinterpret_cast<uint16_t*>(base + p.off_up);
  uint16_t* const tp = reinterpret_cast<uint16_t*>(base + p.off_tp);
  PrepArgs g{};
  g.u = RankJob{dY, nullptr, (int)M, (int)N, B, r, 0, RankOut{}};
  g.u.o.bf16 = dX ? U : nullptr;   // s U rounded once; A is bf16 as it is
  g.u.o.s = s;
  g.u.o.packed = up;
  g.u.o.pscale = X.scale;
  g.t = RankJob{T || T_bf16 ? nullptr : X.codes, X.scale, (int)M, (int)K, A, r, 0, RankOut{}};
  g.t.o.packed = tp;
  g.T = T;
  g.T_bf16 = T_bf16;
  NF4Weight wx = w;
  const bool once = p.once;
  const int threads = once ? kRankWaves * 64 : 256;
  DownJob du{dY, (int)M, (int)N, B, r, 0, 0, 0, reinterpret_cast<float*>(base + p.off_ds)};
  DownJob dt{g.t.S, (int)M, (int)K, A, r, 0, 0, 0, reinterpret_cast<float*>(base + p.off_dt)};
  g.nu = once ? rank_blocks(g.u) : down_blocks(du);
  g.nt = once ? rank_blocks(g.t) : down_blocks(dt);
  if (!g.t.S)
    g.nt = (int)(((M + kChunk - 1) / kChunk * (kChunk / 8) * 16 * ((r + 15) / 16) + threads - 1) / threads);
  int64_t nc = 0;
  if (p.copy) {
    wx.bf16 = g.copy = reinterpret_cast<uint16_t*>(base + p.off_w);
    int64_t each;
    if (W8) {
      g.wcodes = W8->codes; g.wscale = W8->scale;
      g.words = N * K / 16; g.k16 = (uint32_t)(K / 16);
      each = threads * kCopyRounds;
    } else {
      g.w = w; g.cb = nf4_codebook4();
      g.words = N * K / 8;
      each = threads / 64 * kDqWaveWords;
    }
    nc = (g.words + each - 1) / each;
  }
  if (p.consts) {
    g.w = w;
    g.consts = reinterpret_cast<float*>(base + p.off_w);
    g.words = N * (K / kBlock);
    nc = (g.words + threads * kConstRounds - 1) / (threads * kConstRounds);
  }
  const dim3 grid((unsigned)(g.nu + g.nt + nc));
  if (once) {
    rank_form(r, [&](auto rt) {
      constexpr int RT = decltype(rt)::value;
      hipLaunchKernelGGL(k_int8_prep<RT>, grid, dim3(threads), 0, st, g);
    });
  } else {
    hipLaunchKernelGGL(k_int8_prep_down, grid, dim3(threads), 0, st, g, du, dt);
    const FinishJob fu{du.part, du.zs, (int)M, r, nullptr, g.u.o};
    const FinishJob ft{dt.part, dt.zs, (int)M, r, X.scale, g.t.o};
    const int nf = finish_blocks(M, r);
    hipLaunchKernelGGL(k_int8_finish, dim3(g.t.S ? 2 * nf : nf), dim3(256), 0, st, fu, nf, ft);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  Grad8Args ga{};
  ga.ja = Grad8Job{X.codes, K, up, dA, 0};
  ga.jb = Grad8Job{dY, N, tp, dB, 0};
  ga.M = (int)M; ga.r = r; ga.s = s;
  if (dX) {
    float* const part = reinterpret_cast<float*>(base + p.off_part);
    const Codebook4 cb = nf4_codebook4();
    const Dx8Base b8 = p.consts ? Dx8Base{w.packed, g.consts, cb.lv}
                       : W8 && !p.copy ? Dx8Base{W8->codes, W8->scale, nullptr}
                                       : Dx8Base{wx.bf16, nullptr, nullptr};
    e = p.any ? launch_dx8(dY, M, K, N, b8, U, A, r, dX, accumulate, part, p.dx8, ga, st)
              : launch_dx(dY, M, wx, U, A, r, 1.0f, dX, accumulate, st, nullptr, 1.0f,
                          p.kz_len ? part : nullptr, p.kz_len, nullptr);
    if (e != hipSuccess || (p.any && p.dx8.grads)) return e;
  }
  auto grads = [&](auto rt) {
    constexpr int RT = decltype(rt)::value;
    hipLaunchKernelGGL(k_int8_grads<RT>, dim3(grads8_blocks<RT>(ga)), dim3(64 * kGradWaves8), 0, st, ga);
  };
  if (r <= kRankOnce) rank_form(r, grads);
  else grads(std::integral_constant<int, 4>());
  return hipGetLastError();
}

}  // namespace qlk
