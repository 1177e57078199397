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

#include "device_common.h"
#include "kernels.h"
#include "terms.h"

namespace qlk {

constexpr int kChunk = 32;       // tokens of an MFMA step of the gradients

// Sixteen codes as two operands' worth of bf16.
__device__ __forceinline__ uint32_t codes_bf16x2(uint32_t w, int i) {   // codes i, i + 1
  return pack_bf16x2((float)(int8_t)(w >> (8 * i)), (float)(int8_t)(w >> (8 * i + 8)));
}
__device__ __forceinline__ void codes_to_bf16(const uint4& v, uint4 (&o)[2]) {
  o[0] = make_uint4(codes_bf16x2(v.x, 0), codes_bf16x2(v.x, 2), codes_bf16x2(v.y, 0), codes_bf16x2(v.y, 2));
  o[1] = make_uint4(codes_bf16x2(v.z, 0), codes_bf16x2(v.z, 2), codes_bf16x2(v.w, 0), codes_bf16x2(v.w, 2));
}
__device__ __forceinline__ uint4 zero_unless(bool ok, uint4 v) {
  return make_uint4(ok ? v.x : 0u, ok ? v.y : 0u, ok ? v.z : 0u, ok ? v.w : 0u);
}

// What a rank-r product leaves (any may be null).  packed: MFMA operands of the
// gradients, [chunk][term][rank tile][lane][8]: lane (i, g) holds rank 16 t + i
// of tokens 8 g .. +7 of the chunk.
struct RankOut {
  float* sum;              // [M, r]
  uint16_t* bf16;          // [M, r]
  uint16_t* two;           // [M][2][r]: hi and mid terms of s sum
  float s;
  uint16_t* packed;        // terms of pscale[m] sum
  const float* pscale;     // [M], or null: 1
};

__device__ __forceinline__ void pack_terms(uint16_t* packed, int ntiles, int m4, int t, int i,
                                           const float (&x)[4]) {
  // ranks 16 t + i of tokens m4 .. m4 + 3 (4 | m4)
  const int64_t chunk = m4 / kChunk;
  const int lane = 16 * ((m4 % kChunk) / 8) + i;
  Terms e[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) e[v] = split(x[v]);
  const uint32_t w[3][2] = {{e[0].hi | (uint32_t)e[1].hi << 16, e[2].hi | (uint32_t)e[3].hi << 16},
                            {e[0].mid3 | (uint32_t)e[1].mid3 << 16, e[2].mid3 | (uint32_t)e[3].mid3 << 16},
                            {e[0].lo | (uint32_t)e[1].lo << 16, e[2].lo | (uint32_t)e[3].lo << 16}};
#pragma unroll
  for (int z = 0; z < 3; ++z)
    *reinterpret_cast<uint2*>(packed + (((chunk * 3 + z) * ntiles + t) * 64 + lane) * 8 + (m4 % 8)) =
        make_uint2(w[z][0], w[z][1]);
}

// out[m][j] = sum_c S[m][c] W(j, c), W(j, c) = A[j][c] or (WT) B[c][j]; S bf16 or,
// S8, codes whose row scale multiplies the finished sum.  A workgroup owns 16
// rows and all r columns; its NW waves take every NW-th 64-wide slice of the
// contraction (v_mfma_f32_16x16x32_bf16) with the loads of kB slices together,
// and the waves' sums are added through LDS in a fixed order.
// Rows are counted up to a whole chunk, so that packed terms past M are zero.
template <bool S8, bool WT, int RT, int NW, int kB>
__global__ void __launch_bounds__(NW * 64)
k_int8_rank(const void* __restrict__ Sv, const float* __restrict__ sx, int M, int64_t C,
            const uint16_t* __restrict__ W, int r, RankOut o) {
  __shared__ float red[NW - 1][16][RT * 16];
  __shared__ __attribute__((aligned(16))) uint16_t slab[WT ? NW : 1][64 * 16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row = lane & 15, grp = lane >> 4;
  const int m0 = (int)blockIdx.x * 16, m = m0 + row;
  const bool mvalid = m < M;
  const int64_t nsteps = (C + 63) / 64;
  const int64_t srow = (int64_t)(mvalid ? m : 0) * C;
  const uint16_t* const S = reinterpret_cast<const uint16_t*>(Sv) + srow;
  const int8_t* const Q = reinterpret_cast<const int8_t*>(Sv) + srow;
  const int wrow = lane >> 1, wcol = 8 * (lane & 1);
  uint16_t* const my = slab[WT ? wave : 0];
  const int rd = (16 * grp + (row >> 2)) * 16 + 4 * (row & 3);

  f32x4_t acc[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) acc[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  for (int64_t base = wave; base < nsteps; base += (int64_t)NW * kB) {
    uint4 xv[kB][2], wv[kB][RT][2];
#pragma unroll
    for (int b = 0; b < kB; ++b) {
      const int64_t ks = base + (int64_t)NW * b;
      const bool sv = ks < nsteps;
      if constexpr (S8) {   // 64 | C: a slice's 16 codes of a lane are whole
        const uint4 v = *reinterpret_cast<const uint4*>(Q + (sv ? ks * 64 + 16 * grp : 0));
        xv[b][0] = zero_unless(mvalid && sv, v);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t k = ks * 64 + 16 * grp + 8 * h;
        const bool kvalid = sv && k < C;
        if constexpr (!S8) {
          const uint4 v = *reinterpret_cast<const uint4*>(S + (kvalid ? k : 0));
          xv[b][h] = zero_unless(mvalid && kvalid, v);
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          if (!WT) {
            const int j = 16 * t + row;
            const bool ok = kvalid && j < r;
            const uint4 w = *reinterpret_cast<const uint4*>(W + (ok ? (int64_t)j * C + k : 0));
            wv[b][t][h] = zero_unless(ok, w);
          } else {
            const int64_t c = ks * 64 + 32 * h + wrow;
            const int j = 16 * t + wcol;
            const bool ok = sv && c < C && j < r;
            const uint4 w = *reinterpret_cast<const uint4*>(W + (ok ? c * r + j : 0));
            wv[b][t][h] = zero_unless(ok, w);
          }
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);   // every load of the batch before the first MFMA
#pragma unroll
    for (int b = 0; b < kB; ++b) {
      uint4 xs[2] = {xv[b][0], xv[b][1]};
      if constexpr (S8) codes_to_bf16(xv[b][0], xs);
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        bf16x8_t bop[2];
        if (!WT) {
          bop[0] = __builtin_bit_cast(bf16x8_t, wv[b][t][0]);
          bop[1] = __builtin_bit_cast(bf16x8_t, wv[b][t][1]);
        } else {
          // A wave's LDS operations run in issue order: the stores are
          // complete before the reads, which complete before the next stores.
          *reinterpret_cast<uint4*>(my + wrow * 16 + wcol) = wv[b][t][0];
          *reinterpret_cast<uint4*>(my + (32 + wrow) * 16 + wcol) = wv[b][t][1];
          __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const v4s_t lo = lds_read_tr16(my + rd + 8 * h * 16);
            const v4s_t hi = lds_read_tr16(my + rd + (8 * h + 4) * 16);
            typedef short v8s_t __attribute__((ext_vector_type(8)));
            const v8s_t bv = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            bop[h] = __builtin_bit_cast(bf16x8_t, bv);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
          acc[t] = mfma_16x16x32(__builtin_bit_cast(bf16x8_t, xs[h]), bop[h], acc[t]);
      }
    }
  }

  // acc[t][v]: row 4 grp + v, column 16 t + row of the tile.
  if (wave > 0) {
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v) red[wave - 1][4 * grp + v][16 * t + row] = acc[t][v];
  }
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int j = 16 * t + row;
    float p[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int mm = m0 + 4 * grp + v;
      float sum = acc[t][v];
#pragma unroll
      for (int q = 0; q < NW - 1; ++q) sum += red[q][4 * grp + v][j];
      const bool in = mm < M && j < r;
      if (S8 && in) sum *= sx[mm];
      p[v] = !in ? 0.0f : o.pscale ? sum * o.pscale[mm] : sum;
      if (!in) continue;
      if (o.sum) o.sum[(int64_t)mm * r + j] = sum;
      if (o.bf16) o.bf16[(int64_t)mm * r + j] = f32_to_bf16(sum);
      if (o.two) {
        const Terms e = split(o.s * sum);
        o.two[(int64_t)mm * 2 * r + j] = e.hi;
        o.two[((int64_t)mm * 2 + 1) * r + j] = e.mid2;
      }
    }
    if (o.packed && 16 * t < r) pack_terms(o.packed, (r + 15) / 16, m0 + 4 * grp, t, row, p);
  }
}

template <bool S8, bool WT>
static hipError_t int8_rank(const void* S, const float* sx, int64_t M, int64_t C, const uint16_t* W,
                            int r, const RankOut& o, hipStream_t st) {
  int64_t rows = (M + 15) / 16;
  if (o.packed) rows = (M + kChunk - 1) / kChunk * (kChunk / 16);
  const dim3 grid((unsigned)rows);
  const int tiles = (r + 15) / 16;
  if (tiles <= 1) hipLaunchKernelGGL((k_int8_rank<S8, WT, 1, 16, 4>), grid, dim3(1024), 0, st, S, sx, (int)M, C, W, r, o);
  else if (tiles <= 2) hipLaunchKernelGGL((k_int8_rank<S8, WT, 2, 16, 2>), grid, dim3(1024), 0, st, S, sx, (int)M, C, W, r, o);
  else if (tiles <= 4) hipLaunchKernelGGL((k_int8_rank<S8, WT, 4, 8, 1>), grid, dim3(512), 0, st, S, sx, (int)M, C, W, r, o);
  else if (tiles <= 8) hipLaunchKernelGGL((k_int8_rank<S8, WT, 8, 4, 1>), grid, dim3(256), 0, st, S, sx, (int)M, C, W, r, o);
  else hipLaunchKernelGGL((k_int8_rank<S8, WT, 16, 4, 1>), grid, dim3(256), 0, st, S, sx, (int)M, C, W, r, o);
  return hipGetLastError();
}

hipError_t launch_int8_T(const Int8Rows& X, int64_t M, int64_t K, const uint16_t* A, int r, float s,
                         float* T, uint16_t* T2, hipStream_t st) {
  RankOut o{};
  o.sum = T; o.two = T2; o.s = s;
  return int8_rank<true, false>(X.codes, X.scale, M, K, A, r, o, st);
}

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

// T given in fp32 (three terms) or bf16 (its own only term; the others are 2^-40
// of it, which leaves the sum as it is) as the gradients' operands: a thread per
// (rank, four tokens).
template <class E>
__global__ void __launch_bounds__(256)
k_int8_pack_T(const E* __restrict__ T, int M, int r, uint16_t* __restrict__ packed) {
  const int ntiles = (r + 15) / 16, width = 16 * ntiles;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t m4 = 4 * (e / width);
  const int j = (int)(e % width);
  if (m4 >= (int64_t)(M + kChunk - 1) / kChunk * kChunk) return;
  float x[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int64_t m = m4 + v;
    x[v] = 0.0f;
    if (m < M && j < r) {
      if constexpr (sizeof(E) == 4) x[v] = T[m * r + j];
      else x[v] = bf16_to_f32(T[m * r + j]);
    }
  }
  pack_terms(packed, ntiles, (int)m4, j / 16, j % 16, x);
}

// ---------------------------------------------------------------------------
// O[c][j] = s sum_m P[m][c] Q[m][j] for (P, Q) = (Cx, terms of sx U): dA^T, and
// (dY, terms of T): dB, in one launch that reads P once.  A workgroup owns 32
// columns of P and up to 64 ranks and contracts over all tokens itself; its four
// waves take every fourth 32-token chunk.  P goes through a slab of LDS per wave
// (codes as bf16) and comes back transposed as the MFMA operand (v_mfma_f32_16x16x32_bf16);
// Q is loaded as the operands that it is stored as, 1 KB in a row each.  Each
// term takes an MFMA on the same P operand, the small terms first.  The waves'
// sums are added through LDS in a fixed order.
constexpr int kGradCols8 = 32;
constexpr int kGradWaves8 = 4;

struct Grad8Job {
  const void* P;         // [M, ld] codes or bf16
  int64_t ld;            // its columns (a multiple of 8; of 16 for codes)
  const uint16_t* Q;     // packed terms
  float* out;            // trans: [r, ld], else [ld, r]
  int slices;            // workgroups: ceil(ld / 32)
};

template <bool S8, int RT>
__device__ __forceinline__ void grads8(const Grad8Job& g, int lb, int M, int r, int t0, float s,
                                       uint16_t (*slab)[kChunk * kGradCols8],
                                       f32x4_t (*red)[2 * RT][64]) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i = lane & 15, q4 = lane >> 4;
  const int full = (g.slices / kXCDs) * kXCDs;
  const int sl = lb < full ? (lb % kXCDs) * (full / kXCDs) + lb / kXCDs : lb;
  const int64_t c0 = (int64_t)sl * kGradCols8;
  const int ntiles = (r + 15) / 16;
  const __amdgpu_buffer_rsrc_t rp = rsrc_whole(g.P, (uint32_t)((int64_t)M * g.ld * (S8 ? 1 : 2)));
  uint16_t* const my = slab[wave];
  const int nchunks = (M + kChunk - 1) / kChunk;

  f32x4_t acc[2][RT];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[h][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  struct Chunk { uint4 p[S8 ? 1 : 2]; uint4 q[3][RT]; };
  auto load = [&](Chunk& L, int ch) {
    const bool cv = ch < nchunks;
    if constexpr (S8) {
      const int m = ch * kChunk + (lane >> 1);
      const int64_t col = c0 + 16 * (lane & 1);
      L.p[0] = bload128(rp, cv && m < M && col < g.ld ? (uint32_t)(m * g.ld + col) : kOOB);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int m = ch * kChunk + 16 * h + (lane >> 2);
        const int64_t col = c0 + 8 * (lane & 3);
        L.p[h] = bload128(rp, cv && m < M && col < g.ld ? (uint32_t)((m * g.ld + col) * 2) : kOOB);
      }
    }
#pragma unroll
    for (int z = 0; z < 3; ++z)
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        L.q[z][t] = make_uint4(0, 0, 0, 0);
        if (cv && t0 + t < ntiles)
          L.q[z][t] = *reinterpret_cast<const uint4*>(
              g.Q + ((((int64_t)ch * 3 + z) * ntiles + t0 + t) * 64 + lane) * 8);
      }
  };
  auto use = [&](const Chunk& L) {
    // A wave's LDS operations run in issue order: these stores land after the
    // previous chunk's reads and before this one's.
    if constexpr (S8) {
      uint4 o[2];
      codes_to_bf16(L.p[0], o);
      uint4* const d = reinterpret_cast<uint4*>(my + (lane >> 1) * kGradCols8 + 16 * (lane & 1));
      d[0] = o[0];
      d[1] = o[1];
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<uint4*>(my + (16 * h + (lane >> 2)) * kGradCols8 + 8 * (lane & 3)) = L.p[h];
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
    typedef short v8s_t __attribute__((ext_vector_type(8)));
    // source lane 4 s + u of a 16-lane group points at row 8 q4 + 4 e + s, column
    // 4 u of a 16-column band: lane i receives column i of the band's four rows
    const int rr = 8 * q4 + (i >> 2), cc = 4 * (i & 3);
    bf16x8_t aop[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const v4s_t lo = lds_read_tr16(my + rr * kGradCols8 + 16 * h + cc);
      const v4s_t hi = lds_read_tr16(my + (rr + 4) * kGradCols8 + 16 * h + cc);
      const v8s_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      aop[h] = __builtin_bit_cast(bf16x8_t, v);
    }
#pragma unroll
    for (int z = 2; z >= 0; --z)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < RT; ++t)
          acc[h][t] = mfma_16x16x32(aop[h], __builtin_bit_cast(bf16x8_t, L.q[z][t]), acc[h][t]);
  };
  Chunk a, b;
  load(a, wave);
  for (int ch = wave; ch < nchunks; ch += 2 * kGradWaves8) {
    load(b, ch + kGradWaves8);
    use(a);
    load(a, ch + 2 * kGradWaves8);
    use(b);
  }
  // acc[h][t][v] = O[c0 + 16 h + 4 q4 + v][16 (t0 + t) + i]
  if (wave > 0)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < RT; ++t) red[wave - 1][h * RT + t][lane] = acc[h][t];
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      f32x4_t v = acc[h][t];
#pragma unroll
      for (int w = 0; w < kGradWaves8 - 1; ++w) v += red[w][h * RT + t][lane];
      v *= s;
      const int64_t c = c0 + 16 * h + 4 * q4;
      const int j = 16 * (t0 + t) + i;
      if (c >= g.ld || j >= r) continue;
      if (S8) {
        *reinterpret_cast<f32x4_t*>(g.out + (int64_t)j * g.ld + c) = v;   // dA [r, K]
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) g.out[(c + e) * r + j] = v[e];        // dB [N, r]
      }
    }
}

template <int RT>
__global__ void __launch_bounds__(64 * kGradWaves8)
k_int8_grads(Grad8Job ja, Grad8Job jb, int M, int r, float s) {
  __shared__ __attribute__((aligned(16))) uint16_t slab[kGradWaves8][kChunk * kGradCols8];
  __shared__ f32x4_t red[kGradWaves8 - 1][2 * RT][64];
  const int t0 = (int)blockIdx.y * RT;
  if ((int)blockIdx.x < ja.slices) grads8<true, RT>(ja, blockIdx.x, M, r, t0, s, slab, red);
  else grads8<false, RT>(jb, (int)blockIdx.x - ja.slices, M, r, t0, s, slab, red);
}

Int8BwdPlan plan_int8_bwd(int64_t M, int64_t K, int64_t N, int r, int base, bool dx) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  Int8BwdPlan p{};
  const size_t pack = (size_t)((M + kChunk - 1) / kChunk) * 3 * ((r + 15) / 16) * 1024;
  p.off_U = 0;
  p.off_up = up((size_t)M * r * 2);
  p.off_tp = p.off_up + up(pack);
  p.bytes = p.off_tp + up(pack);
  // dX on a bf16 copy of the base, made once per call: always of an 8-bit base,
  // of an NF4 base from the token count where its own backward makes one
  p.copy = dx && (base == kBaseInt8 || (base == kBaseNF4 && M >= kDequantDxMinM &&
                                        dx_nf4_supported(N) && N * K * 2 < ((int64_t)1 << 31)));
  p.off_w = p.bytes;
  if (p.copy) p.bytes += up((size_t)N * K * 2);
  p.kz_len = dx && dx_nf4_supported(N) ? dx_split_len(M, K, N) : 0;
  p.off_part = p.bytes;
  if (p.kz_len) p.bytes += up((size_t)((N / 64 + p.kz_len - 1) / p.kz_len) * M * K * 4);
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
  hipError_t e = hipSuccess;
  // T's terms
  if (!T && !T_bf16) {
    RankOut o{};
    o.packed = tp;
    e = int8_rank<true, false>(X.codes, X.scale, M, K, A, r, o, st);
  } else {
    const int64_t n = (M + kChunk - 1) / kChunk * (kChunk / 4) * 16 * ((r + 15) / 16);
    const dim3 grid((unsigned)((n + 255) / 256));
    if (T) hipLaunchKernelGGL(k_int8_pack_T<float>, grid, dim3(256), 0, st, T, (int)M, r, tp);
    else hipLaunchKernelGGL(k_int8_pack_T<uint16_t>, grid, dim3(256), 0, st, T_bf16, (int)M, r, tp);
    e = hipGetLastError();
  }
  if (e != hipSuccess) return e;
  // U as the dX product's operand and as sx U's terms
  RankOut o{};
  o.bf16 = dX ? U : nullptr;
  o.packed = up;
  o.pscale = X.scale;
  e = int8_rank<false, true>(dY, nullptr, M, N, B, r, o, st);
  if (e != hipSuccess) return e;
  if (dX) {
    NF4Weight wx = w;
    if (p.copy) {
      uint16_t* const wb = reinterpret_cast<uint16_t*>(base + p.off_w);
      e = W8 ? launch_int8_dequant(W8->codes, W8->scale, N, K, false, wb, st)
             : launch_nf4_dequant(w.packed, w.codes, w.scales, w.mean, N * K, nf4_codebook4(), wb, st);
      if (e != hipSuccess) return e;
      wx.bf16 = wb;
    }
    e = launch_dx(dY, M, wx, U, A, r, s, dX, accumulate, st, nullptr, 1.0f,
                  p.kz_len ? reinterpret_cast<float*>(base + p.off_part) : nullptr, p.kz_len, nullptr);
    if (e != hipSuccess) return e;
  }
  const Grad8Job ja{X.codes, K, up, dA, (int)((K + kGradCols8 - 1) / kGradCols8)};
  const Grad8Job jb{dY, N, tp, dB, (int)((N + kGradCols8 - 1) / kGradCols8)};
  const int tiles = (r + 15) / 16;
  const unsigned nx = (unsigned)(ja.slices + jb.slices);
  const dim3 block(64 * kGradWaves8);
  if (tiles <= 1) hipLaunchKernelGGL(k_int8_grads<1>, dim3(nx), block, 0, st, ja, jb, (int)M, r, s);
  else if (tiles <= 2) hipLaunchKernelGGL(k_int8_grads<2>, dim3(nx), block, 0, st, ja, jb, (int)M, r, s);
  else hipLaunchKernelGGL(k_int8_grads<4>, dim3(nx, (unsigned)((tiles + 3) / 4)), block, 0, st, ja, jb, (int)M, r, s);
  return hipGetLastError();
}

}  // namespace qlk
