// Adapters of many requests beside one shared projection: S slots, each with
// A [r, K], B [N, r] and a scale c, and M tokens, each with the slot a(m) the
// token plan gives it (or none):
//
//   forward   T = drop(X) A_a^T            out = Y + c_a T B_a^T
//   backward  U = dY B_a                   dX  = dX0 + drop(c_a U A_a)
//             dA_a = c_a U^T drop(X)       dB_a = c_a dY^T T   (sums over a's tokens)
//                       (llm-compass "QLoRA", 方法与公式, the adapter's term
//                        of the equation and its derivatives, token by token)
//
// drop() is the LoRA dropout of the adapter input with its mask regenerated
// from (seed, element) wherever an element is used: a dropped element is
// cleared as it is loaded (or its sum as it leaves), and 1 / (1 - p) is one
// factor of the finished fp32 sum, so no rounded copy of the input exists.
//
// Sums and the small matrices T and U are fp32.  Where T or U feeds an MFMA
// it goes in as a sum of bf16 terms, x = hi + mid (+ lo): two terms (within
// 2^-17 of x) where the result is rounded to bf16, three (2^-25) where it is
// kept in fp32.
#include <type_traits>

#include "device_common.h"
#include "kernels.h"
#include "philox.h"

namespace qlk {

typedef short v8s_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ uint4 keep_or_zero(bool ok, uint4 v) {
  return make_uint4(ok ? v.x : 0u, ok ? v.y : 0u, ok ? v.z : 0u, ok ? v.w : 0u);
}

// x = hi + mid + lo, bf16 terms; an infinity or NaN is hi alone.
__device__ __forceinline__ void split3(float x, uint16_t& hi, uint16_t& mid, uint16_t& lo) {
  hi = f32_to_bf16(x);
  const float rest = __builtin_isfinite(x) ? x - bf16_to_f32(hi) : 0.0f;
  mid = f32_to_bf16(rest);
  lo = f32_to_bf16(rest - bf16_to_f32(mid));
}

// One row of the plan's tiles, its positions checked against M tokens and S
// slots: a plan that does not fit the batch names no tile.
struct TileRow {
  int slot, first, count;
};
__device__ __forceinline__ TileRow tile_row(const int* tiles, int i, int M, int S) {
  TileRow t{tiles[3 * i], tiles[3 * i + 1], tiles[3 * i + 2]};
  if (t.slot < 0 || t.slot >= S) t.slot = -1;
  if (t.first < 0 || t.count < 0 || t.count > kPlanTile || t.first > M - t.count) t.count = 0;
  return t;
}

// ---------------------------------------------------------------------------
// T = X A_a^T and U = dY B_a, fp32 [M, r].  One workgroup takes `rows` (8 or
// 16) tokens of one slot, gathered through the plan's order; its NW waves take
// every NW-th 64-wide piece of the contraction and add their sums through LDS
// in a fixed order.  Bound: HBM, one pass over X (dY); each workgroup reads
// its slot's A (B) once, from L2 where workgroups share the slot.
constexpr int kDownRows = 16;

struct DownArgs {
  const uint16_t* S;     // [M, C] bf16
  int M;
  int64_t C;
  const uint16_t* W;     // [slots, r, C] or, WT, [slots, C, r]
  int r, slots;
  const int* order;
  const int* tiles;
  int rows;              // tokens per workgroup
  float* out;            // fp32 [M, r]
  uint16_t* planes;      // bf16 terms of out, [3][M, r], or null
  DropKey drop;
  float keep_scale;
};

template <bool WT, bool DROP, int RT, int NW, int kB>
__global__ void __launch_bounds__(NW * 64) k_batch_down(DownArgs g) {
  __shared__ float red[NW - 1][kDownRows][RT * 16];
  // WT: one 64 (c) x 16 (j) slice of B per wave, row-major.
  __shared__ __attribute__((aligned(16))) uint16_t slab[WT ? NW : 1][64 * 16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row = lane & 15, grp = lane >> 4;
  const int subs = kPlanTile / g.rows;
  const TileRow t = tile_row(g.tiles, (int)blockIdx.x / subs, g.M, g.slots);
  const int off = ((int)blockIdx.x % subs) * g.rows;
  const int n = min(g.rows, t.count - off);
  if (n <= 0) return;
  const int r = g.r;
  const int* const ord = g.order + t.first + off;
  if (t.slot < 0) {   // no adapter: zeros
    for (int e = tid; e < n * r; e += NW * 64) {
      const int m = ord[e / r];
      if ((unsigned)m >= (unsigned)g.M) continue;
      g.out[(int64_t)m * r + e % r] = 0.0f;
    }
    return;
  }
  // Rows past the tile read the tile's last row (its lines are loaded anyway).
  int m = ord[min(row, n - 1)];
  const bool mvalid = row < n && (unsigned)m < (unsigned)g.M;
  if ((unsigned)m >= (unsigned)g.M) m = 0;
  const int64_t C = g.C;
  const int64_t nsteps = (C + 63) / 64;
  const uint16_t* const srow = g.S + (int64_t)m * C;
  const uint16_t* const W = g.W + (int64_t)t.slot * C * r;
  const int wrow = lane >> 1, wcol = 8 * (lane & 1);
  uint16_t* const my = slab[WT ? wave : 0];
  const int rd = (16 * grp + (row >> 2)) * 16 + 4 * (row & 3);

  f32x4_t acc[RT];
#pragma unroll
  for (int q = 0; q < RT; ++q) acc[q] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  for (int64_t b0 = wave; b0 < nsteps; b0 += (int64_t)NW * kB) {
    uint4 xv[kB][2], wv[kB][RT][2];
#pragma unroll
    for (int b = 0; b < kB; ++b) {
      const int64_t ks = b0 + (int64_t)NW * b;
      const bool sv = ks < nsteps;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t k = ks * 64 + 16 * grp + 8 * h;   // 8 contraction indices
        const bool kvalid = sv && k < C;
        xv[b][h] = keep_or_zero(mvalid && kvalid,
                                *reinterpret_cast<const uint4*>(srow + (kvalid ? k : 0)));
#pragma unroll
        for (int q = 0; q < RT; ++q) {
          if (!WT) {
            const int j = 16 * q + row;
            const bool ok = kvalid && j < r;
            wv[b][q][h] = keep_or_zero(
                ok, *reinterpret_cast<const uint4*>(W + (ok ? (int64_t)j * C + k : 0)));
          } else {
            const int64_t c = ks * 64 + 32 * h + wrow;
            const int j = 16 * q + wcol;
            const bool ok = sv && c < C && j < r;
            wv[b][q][h] =
                keep_or_zero(ok, *reinterpret_cast<const uint4*>(W + (ok ? c * r + j : 0)));
          }
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);   // every load of the batch before the first MFMA
#pragma unroll
    for (int b = 0; b < kB; ++b) {
      if constexpr (DROP) {
        const int64_t ks = b0 + (int64_t)NW * b;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          xv[b][h] = philox_drop8(
              xv[b][h], (uint64_t)((int64_t)m * C + ks * 64 + 16 * grp + 8 * h), g.drop);
      }
#pragma unroll
      for (int q = 0; q < RT; ++q) {
        bf16x8_t bop[2];
        if (!WT) {
          bop[0] = __builtin_bit_cast(bf16x8_t, wv[b][q][0]);
          bop[1] = __builtin_bit_cast(bf16x8_t, wv[b][q][1]);
        } else {
          // A wave's LDS operations run in issue order: the stores are
          // complete before the reads, which complete before the next stores.
          *reinterpret_cast<uint4*>(my + wrow * 16 + wcol) = wv[b][q][0];
          *reinterpret_cast<uint4*>(my + (32 + wrow) * 16 + wcol) = wv[b][q][1];
          __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const v4s_t lo = lds_read_tr16(my + rd + 8 * h * 16);
            const v4s_t hi = lds_read_tr16(my + rd + (8 * h + 4) * 16);
            const v8s_t bv = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            bop[h] = __builtin_bit_cast(bf16x8_t, bv);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
          acc[q] = mfma_16x16x32(__builtin_bit_cast(bf16x8_t, xv[b][h]), bop[h], acc[q]);
      }
    }
  }

  // acc[q][v]: row 4 grp + v, column 16 q + row of the tile.
  if (wave > 0) {
#pragma unroll
    for (int q = 0; q < RT; ++q)
#pragma unroll
      for (int v = 0; v < 4; ++v) red[wave - 1][4 * grp + v][16 * q + row] = acc[q][v];
  }
  __syncthreads();
  if (wave != 0) return;
  int mo[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) mo[v] = 4 * grp + v < n ? ord[4 * grp + v] : -1;
#pragma unroll
  for (int q = 0; q < RT; ++q) {
    const int j = 16 * q + row;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      float sum = acc[q][v];
#pragma unroll
      for (int w = 0; w < NW - 1; ++w) sum += red[w][4 * grp + v][j];
      if (DROP) sum *= g.keep_scale;
      if ((unsigned)mo[v] >= (unsigned)g.M || j >= r) continue;
      const int64_t o = (int64_t)mo[v] * r + j;
      g.out[o] = sum;
      if (g.planes) {
        const int64_t plane = (int64_t)g.M * r;
        split3(sum, g.planes[o], g.planes[plane + o], g.planes[2 * plane + o]);
      }
    }
  }
}

// The bf16 terms of an fp32 [M, r], for the gradients' kernel.
__global__ void __launch_bounds__(256)
k_batch_split(const float* __restrict__ x, int64_t n, uint16_t* __restrict__ planes) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) split3(x[i], planes[i], planes[n + i], planes[2 * n + i]);
}

// ---------------------------------------------------------------------------
// out = base + c_a t W_a^T with t = T, W = B ([cols, r] per slot), or, WT,
// t = U, W = A ([r, cols] per slot) and the dropout of the product.  One
// workgroup takes a tile of the plan (up to 64 tokens of one slot) and 256
// columns, a wave 64 columns of all its tokens.
//
//  * v_mfma_f32_16x16x32_bf16 with W rows as the row operand and tokens as
//    columns.  Its 32 contraction indices hold 16 ranks twice: the hi terms of
//    c_a t against W, then the mid terms against the same W.
//  * MFMA row rho of pair jj stands for column 8 (rho / 4) + 4 jj + rho % 4 of
//    a 32-column unit, so that a lane's two accumulators of a token are 8
//    consecutive columns: base and out move as 16-byte pieces, a wave four
//    pieces (64 bytes) of 16 tokens per instruction.
//  * A lane reads and writes the same places of base and out, which may
//    therefore be one tensor.
// Bound: HBM, base read and out written once; W comes from L2 once per tile.
constexpr int kUpCols = 256;    // columns per workgroup
constexpr int kUpWaveCols = 64;
constexpr int kUpRanks = 128;   // ranks whose terms are in LDS at a time
// LDS row of a token (elements): 16 hi and 16 mid terms per 16 ranks, padded.
__host__ __device__ constexpr int up_lds_row(int r) {
  return ((r < kUpRanks ? r : kUpRanks) + 15) / 16 * 32 + 8;
}

struct UpArgs {
  const uint16_t* base;  // [M, cols] bf16 or null (zeros)
  uint16_t* out;         // [M, cols] bf16
  int M;
  int64_t cols;
  const float* t;        // fp32 [M, r]
  const uint16_t* W;
  const float* scale;    // [slots]
  int r, slots;
  const int* order;
  const int* tiles;
  DropKey drop;
  float keep_scale;
};

template <bool WT, bool DROP>
__global__ void __launch_bounds__(256) k_batch_up(UpArgs g) {
  extern __shared__ __attribute__((aligned(16))) uint16_t lds[];
  __shared__ __attribute__((aligned(16))) uint16_t slab[WT ? 4 : 1][WT ? 16 * 80 : 8];
  __shared__ int rows[kPlanTile];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i = lane & 15, q4 = lane >> 4;
  const TileRow t = tile_row(g.tiles, blockIdx.x, g.M, g.slots);
  if (t.count <= 0) return;
  const int64_t cols = g.cols;
  const int64_t n0 = (int64_t)blockIdx.y * kUpCols;
  if (tid < kPlanTile) {
    const int m = tid < t.count ? g.order[t.first + tid] : -1;
    rows[tid] = (unsigned)m < (unsigned)g.M ? m : -1;
  }
  __syncthreads();
  if (t.slot < 0) {   // no adapter: the base alone
    if (g.out == g.base) return;
    for (int e = tid; e < t.count * (kUpCols / 8); e += 256) {
      const int m = rows[e / (kUpCols / 8)];
      const int64_t c = n0 + 8 * (e % (kUpCols / 8));
      if (m < 0 || c >= cols) continue;
      const int64_t o = (int64_t)m * cols + c;
      *reinterpret_cast<uint4*>(g.out + o) =
          g.base ? *reinterpret_cast<const uint4*>(g.base + o) : make_uint4(0, 0, 0, 0);
    }
    return;
  }
  const int r = g.r;
  const int ld = up_lds_row(r);
  const float c_a = g.scale[t.slot];
  const uint16_t* const W = g.W + (int64_t)t.slot * cols * r;
  const int64_t nw = n0 + kUpWaveCols * wave;
  f32x4_t acc[4][2][2];   // [token group][unit][pair half]
#pragma unroll
  for (int tg = 0; tg < 4; ++tg)
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int jj = 0; jj < 2; ++jj) acc[tg][u][jj] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  for (int r0 = 0; r0 < r; r0 += kUpRanks) {
    const int rn = min(kUpRanks, r - r0), chunks = (rn + 15) / 16;
    if (r0) __syncthreads();   // the last block's reads
    for (int e = tid; e < kPlanTile * chunks * 16; e += 256) {
      const int tok = e / (chunks * 16), j = e % (chunks * 16);
      const int m = rows[tok];
      uint16_t hi, mid, lo;
      split3(m >= 0 && j < rn ? c_a * g.t[(int64_t)m * r + r0 + j] : 0.0f, hi, mid, lo);
      uint16_t* const d = lds + tok * ld + (j >> 4) * 32 + (j & 15);
      d[0] = hi;
      d[16] = mid;
    }
    __syncthreads();
    for (int ch = 0; ch < chunks; ++ch) {
      bf16x8_t wop[2][2];
      if constexpr (!WT) {
        const int j = r0 + 16 * ch + 8 * (q4 & 1);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int jj = 0; jj < 2; ++jj) {
            const int64_t c = nw + 32 * u + 8 * (i >> 2) + 4 * jj + (i & 3);
            const bool ok = c < cols && j < r;
            wop[u][jj] = __builtin_bit_cast(
                bf16x8_t,
                keep_or_zero(ok, *reinterpret_cast<const uint4*>(W + (ok ? c * r + j : 0))));
          }
      } else {
        // 16 ranks x 64 columns of A through LDS (rows of 80), read back
        // transposed: lane i of a 16-lane group gets column 8 (i / 4) + 4 jj +
        // i % 4 of ranks 8 (q4 & 1) .. +7.
        uint16_t* const my = slab[wave];
        const int jr = r0 + 16 * ch + (lane >> 2);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t c = nw + 16 * (lane & 3) + 8 * h;
          const bool ok = c < cols && jr < r;
          *reinterpret_cast<uint4*>(my + (lane >> 2) * 80 + 16 * (lane & 3) + 8 * h) = keep_or_zero(
              ok, *reinterpret_cast<const uint4*>(W + (ok ? (int64_t)jr * cols + c : 0)));
        }
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): one wave's LDS operations are in order
        const int rr = 8 * (q4 & 1) + (i >> 2);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int jj = 0; jj < 2; ++jj) {
            const int cc = 32 * u + 8 * (i & 3) + 4 * jj;
            const v4s_t lo = lds_read_tr16(my + rr * 80 + cc);
            const v4s_t hi = lds_read_tr16(my + (rr + 4) * 80 + cc);
            const v8s_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            wop[u][jj] = __builtin_bit_cast(bf16x8_t, v);
          }
      }
#pragma unroll
      for (int tg = 0; tg < 4; ++tg) {
        if (16 * tg >= t.count) continue;
        const bf16x8_t top =
            *reinterpret_cast<const bf16x8_t*>(lds + (16 * tg + i) * ld + 32 * ch + 8 * q4);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int jj = 0; jj < 2; ++jj)
            acc[tg][u][jj] = mfma_16x16x32(wop[u][jj], top, acc[tg][u][jj]);
      }
    }
  }
  // acc[tg][u][jj][v]: token 16 tg + i, column nw + 32 u + 8 q4 + 4 jj + v.
#pragma unroll
  for (int tg = 0; tg < 4; ++tg) {
    if (16 * tg >= t.count) continue;
    const int m = rows[16 * tg + i];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t c = nw + 32 * u + 8 * q4;
      if (m < 0 || c >= cols) continue;
      const int64_t o = (int64_t)m * cols + c;
      uint4 b = make_uint4(0, 0, 0, 0);
      if (g.base) b = *reinterpret_cast<const uint4*>(g.base + o);
      const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
      float v[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = acc[tg][u][0][e];
        v[4 + e] = acc[tg][u][1][e];
      }
      if constexpr (DROP) {
        const uint32_t keep = philox_keep8((uint64_t)o, g.drop);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (keep >> e) & 1u ? v[e] * g.keep_scale : 0.0f;
      }
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = pack_bf16x2(bf16_to_f32(bw[e] & 0xffffu) + v[2 * e],
                           bf16_to_f32(bw[e] >> 16) + v[2 * e + 1]);
      *reinterpret_cast<uint4*>(g.out + o) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// ---------------------------------------------------------------------------
// dA_a = c_a U^T drop(X) and dB_a = c_a dY^T T over the tokens of each slot,
// fp32, every slot written (zeros without tokens).  Both contract over tokens:
// O[c][j] = sum P[m][c] Q[m][j], (P, Q) = (X, U) with O = dA^T or (dY, T) with
// O = dB.  A workgroup owns a slot, a slice of 16 H columns of P and up to 64
// ranks, and contracts over all of the slot's tokens, gathered through the
// plan's order: no partial sums in memory, no atomics.  Its four waves take
// every fourth 32-token chunk; the chunk's pieces of P and of the three bf16
// planes of Q pass through a slab of LDS per wave and come back as MFMA
// operands with the transposing read, tokens along the contraction.  The
// waves' sums are added in the order 0, 1, 2, 3.
// Bound: HBM, X and dY read once and all slots' dA and dB written.
constexpr int kGradRanks = 64;

struct BatchGradJob {
  const uint16_t* P;   // [M, cols] bf16
  int64_t cols;
  const uint16_t* Q;   // [3][M, r] bf16 planes
  float* out;          // trans: [slots, r, cols] (dA); else [slots, cols, r] (dB)
  int trans, slices;
  int drop;
};

template <int RT, int H, int KB, bool DROP>
__global__ void __launch_bounds__(256)
k_batch_grads(BatchGradJob ja, BatchGradJob jb, int M, int r, int slots, const float* scale,
              const int* order, const int* start, DropKey drop, float keep_scale) {
  constexpr int C = 16 * H;                        // columns of P per workgroup
  constexpr int PPR = C / 8;                       // 16-byte pieces per row of P
  constexpr int QW = 16 * RT;
  constexpr int CE = 32 * C + 3 * 32 * QW;         // elements of a chunk in the slab
  constexpr int SLAB = 4 * KB * CE * 2, RED = 3 * H * RT * 64 * 16;
  __shared__ __attribute__((aligned(16))) char smem[SLAB > RED ? SLAB : RED];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i = lane & 15, g = lane >> 4;
  const bool first = (int)blockIdx.x < ja.slices;
  const BatchGradJob& jb_ = first ? ja : jb;
  const uint16_t* const P = jb_.P;
  const uint16_t* const Q = jb_.Q;
  const int64_t cols = jb_.cols;
  const int trans = jb_.trans;
  const bool dropped = DROP && jb_.drop;
  const int sl = first ? (int)blockIdx.x : (int)blockIdx.x - ja.slices;
  const int64_t c0 = (int64_t)sl * C;
  const int slot = blockIdx.y;
  const int j0 = (int)blockIdx.z * kGradRanks;
  // The slot's range of the order, cut to M tokens whatever the plan holds.
  const int s0 = min(max(start[slot], 0), M), s1 = min(max(start[slot + 1], s0), M);
  const int nt = s1 - s0;

  const __amdgpu_buffer_rsrc_t rp = rsrc_whole(P, (uint32_t)((int64_t)M * cols * 2));
  const __amdgpu_buffer_rsrc_t rq = rsrc_whole(Q, (uint32_t)((int64_t)M * r * 6));
  const int prow = lane / PPR, pcol = 8 * (lane % PPR);
  const bool pcol_ok = c0 + pcol < cols;
  uint16_t* const my = reinterpret_cast<uint16_t*>(smem) + wave * KB * CE;
  const int nchunks = (nt + 31) / 32;
  const int per_wave = (nchunks + 3) / 4;
  const int nb = (per_wave + KB - 1) / KB;   // batches, the same for every wave

  f32x4_t acc[H][RT];
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[h][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  auto consume = [&](const uint4 (&pv)[KB][H], const uint4 (&qv)[KB][3][RT]) {
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      uint16_t* const c = my + b * CE;
#pragma unroll
      for (int h = 0; h < H; ++h)
        *reinterpret_cast<uint4*>(c + (h * (64 / PPR) + prow) * C + pcol) = pv[b][h];
#pragma unroll
      for (int z = 0; z < 3; ++z)
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          const int p = 64 * t + lane;
          *reinterpret_cast<uint4*>(c + 32 * C + z * 32 * QW + (p / (2 * RT)) * QW +
                                    8 * (p % (2 * RT))) = qv[b][z][t];
        }
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): one wave's LDS operations are in order
    const int rr = 8 * g + (i >> 2), cc = 4 * (i & 3);
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      const uint16_t* const c = my + b * CE;
      bf16x8_t aop[H];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const v4s_t lo = lds_read_tr16(c + rr * C + 16 * h + cc);
        const v4s_t hi = lds_read_tr16(c + (rr + 4) * C + 16 * h + cc);
        const v8s_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        aop[h] = __builtin_bit_cast(bf16x8_t, v);
      }
#pragma unroll
      for (int z = 2; z >= 0; --z)          // the small terms first
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          const uint16_t* const qs = c + 32 * C + z * 32 * QW + 16 * t + cc;
          const v4s_t lo = lds_read_tr16(qs + rr * QW);
          const v4s_t hi = lds_read_tr16(qs + (rr + 4) * QW);
          const v8s_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
          const bf16x8_t bop = __builtin_bit_cast(bf16x8_t, v);
#pragma unroll
          for (int h = 0; h < H; ++h) acc[h][t] = mfma_16x16x32(aop[h], bop, acc[h][t]);
        }
    }
  };

  for (int b = 0; b < nb; ++b) {
    uint4 pv[KB][H], qv[KB][3][RT];
#pragma unroll
    for (int q = 0; q < KB; ++q) {
      const int t0 = ((b * KB + q) * 4 + wave) * 32;   // first position of the chunk
      const int pos = t0 + (lane & 31);
      int tok = pos < nt ? order[s0 + pos] : -1;
      if ((unsigned)tok >= (unsigned)M) tok = -1;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int m = __shfl(tok, h * (64 / PPR) + prow);
        const bool ok = m >= 0 && pcol_ok;
        pv[q][h] = bload128s(rp, ok ? (uint32_t)(((int64_t)m * cols + c0 + pcol) * 2) : kOOB, 0);
      }
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const int p = 64 * t + lane;            // piece p: row p / (2 RT), ranks 8 (p % (2 RT))
        const int m = __shfl(tok, p / (2 * RT));
        const int j = j0 + 8 * (p % (2 * RT));
        const bool ok = m >= 0 && j < r;
#pragma unroll
        for (int z = 0; z < 3; ++z)
          qv[q][z][t] = bload128s(
              rq, ok ? (uint32_t)((((int64_t)z * M + m) * r + j) * 2) : kOOB, 0);
      }
      if (DROP && dropped) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const int m = __shfl(tok, h * (64 / PPR) + prow);
          pv[q][h] = philox_drop8(
              pv[q][h], (uint64_t)((int64_t)max(m, 0) * cols + c0 + pcol), drop);
        }
      }
    }
    consume(pv, qv);
  }

  // acc[h][t][v] = O[c0 + 16 h + 4 g + v][j0 + 16 t + i]
  __syncthreads();   // the slabs are free
  f32x4_t* const red = reinterpret_cast<f32x4_t*>(smem);
  if (wave > 0) {
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int t = 0; t < RT; ++t) red[((wave - 1) * H * RT + h * RT + t) * 64 + lane] = acc[h][t];
  }
  __syncthreads();
  if (wave != 0) return;
  const float s = dropped ? scale[slot] * keep_scale : scale[slot];
  float* const out = jb_.out + (int64_t)slot * cols * r;
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      f32x4_t v = acc[h][t];
#pragma unroll
      for (int w = 0; w < 3; ++w) {
        const f32x4_t o = red[(w * H * RT + h * RT + t) * 64 + lane];
        v[0] += o[0]; v[1] += o[1]; v[2] += o[2]; v[3] += o[3];
      }
      const int64_t c = c0 + 16 * h + 4 * g;     // c .. c + 3 (cols is a multiple of 8)
      const int j = j0 + 16 * t + i;
      if (c >= cols || j >= r) continue;
      // A slot without tokens has no products: plain zeros, whatever its scale.
      const f32x4_t res = nt > 0 ? f32x4_t{s * v[0], s * v[1], s * v[2], s * v[3]}
                                 : f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      if (trans) {
        *reinterpret_cast<f32x4_t*>(out + (int64_t)j * cols + c) = res;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) out[(c + e) * r + j] = res[e];
      }
    }
}

// ------------------------------- launchers ---------------------------------

static inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

BatchWorkspace batch_workspace(int64_t M, int r, bool backward) {
  BatchWorkspace w{};
  const size_t f32 = align256((size_t)M * r * 4), planes = align256((size_t)M * r * 6);
  size_t off = 0;
  w.off_T = off; off += f32;
  if (backward) {
    w.off_U = off; off += f32;
    w.off_Up = off; off += planes;
    w.off_Tp = off; off += planes;
  }
  w.bytes = off;
  return w;
}

template <bool WT, bool DROP>
static hipError_t down(DownArgs g, int ntiles, hipStream_t st) {
  // 8 tokens per workgroup while 16 would leave CUs without one.
  g.rows = (g.M + kDownRows - 1) / kDownRows < kCUs ? 8 : kDownRows;
  const dim3 grid((unsigned)(ntiles * (kPlanTile / g.rows)));
  const int rt = (g.r + 15) / 16;
  if (rt <= 1) hipLaunchKernelGGL((k_batch_down<WT, DROP, 1, 16, 4>), grid, dim3(1024), 0, st, g);
  else if (rt <= 2) hipLaunchKernelGGL((k_batch_down<WT, DROP, 2, 16, 2>), grid, dim3(1024), 0, st, g);
  else if (rt <= 4) hipLaunchKernelGGL((k_batch_down<WT, DROP, 4, 8, 1>), grid, dim3(512), 0, st, g);
  else if (rt <= 8) hipLaunchKernelGGL((k_batch_down<WT, DROP, 8, 4, 1>), grid, dim3(256), 0, st, g);
  else hipLaunchKernelGGL((k_batch_down<WT, DROP, 16, 4, 1>), grid, dim3(256), 0, st, g);
  return hipGetLastError();
}

template <bool WT, bool DROP>
static hipError_t up(const UpArgs& g, int ntiles, hipStream_t st) {
  const dim3 grid((unsigned)ntiles, (unsigned)((g.cols + kUpCols - 1) / kUpCols));
  const size_t lds = (size_t)kPlanTile * up_lds_row(g.r) * 2;
  hipLaunchKernelGGL((k_batch_up<WT, DROP>), grid, dim3(256), lds, st, g);
  return hipGetLastError();
}

#define QLK_TRY(x) do { hipError_t e_ = (x); if (e_ != hipSuccess) return e_; } while (0)

static hipError_t batch_T(const uint16_t* X, const BatchAdapters& a, int64_t M, int64_t K,
                          const BatchDropout& d, float* T, hipStream_t st) {
  DownArgs g{};
  g.S = X; g.M = (int)M; g.C = K; g.W = a.A; g.r = a.r; g.slots = a.slots;
  g.order = a.order; g.tiles = a.tiles; g.out = T; g.planes = nullptr;
  g.drop = DropKey{d.threshold, d.k0, d.k1}; g.keep_scale = d.scale;
  const int nt = (int)adapter_plan_tiles(M, a.slots);
  return d.on ? down<false, true>(g, nt, st) : down<false, false>(g, nt, st);
}

hipError_t launch_batch_fwd(const uint16_t* X, int64_t M, int64_t K, int64_t N,
                            const BatchAdapters& a, const uint16_t* Y, const BatchDropout& d,
                            uint16_t* out, float* T_out, void* ws, hipStream_t st) {
  const BatchWorkspace w = batch_workspace(M, a.r, false);
  float* const T = T_out ? T_out : reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + w.off_T);
  QLK_TRY(batch_T(X, a, M, K, d, T, st));
  UpArgs u{};
  u.base = Y; u.out = out; u.M = (int)M; u.cols = N; u.t = T; u.W = a.B; u.scale = a.scale;
  u.r = a.r; u.slots = a.slots; u.order = a.order; u.tiles = a.tiles;
  return up<false, false>(u, (int)adapter_plan_tiles(M, a.slots), st);
}

hipError_t launch_batch_bwd(const uint16_t* dY, const uint16_t* X, int64_t M, int64_t K, int64_t N,
                            const BatchAdapters& a, const float* T, const uint16_t* dX0,
                            const BatchDropout& d, uint16_t* dX, float* dA, float* dB, void* ws,
                            hipStream_t st) {
  const BatchWorkspace w = batch_workspace(M, a.r, true);
  char* const base = reinterpret_cast<char*>(ws);
  float* const U = reinterpret_cast<float*>(base + w.off_U);
  uint16_t* const Up = reinterpret_cast<uint16_t*>(base + w.off_Up);
  uint16_t* const Tp = reinterpret_cast<uint16_t*>(base + w.off_Tp);
  const int nt = (int)adapter_plan_tiles(M, a.slots);
  if (!T) {
    float* const Tw = reinterpret_cast<float*>(base + w.off_T);
    QLK_TRY(batch_T(X, a, M, K, d, Tw, st));
    T = Tw;
  }
  DownArgs g{};
  g.S = dY; g.M = (int)M; g.C = N; g.W = a.B; g.r = a.r; g.slots = a.slots;
  g.order = a.order; g.tiles = a.tiles; g.out = U; g.planes = Up;
  QLK_TRY((down<true, false>(g, nt, st)));
  const DropKey key{d.threshold, d.k0, d.k1};
  if (dX) {
    UpArgs u{};
    u.base = dX0; u.out = dX; u.M = (int)M; u.cols = K; u.t = U; u.W = a.A; u.scale = a.scale;
    u.r = a.r; u.slots = a.slots; u.order = a.order; u.tiles = a.tiles;
    u.drop = key; u.keep_scale = d.scale;
    QLK_TRY((d.on ? up<true, true>(u, nt, st) : up<true, false>(u, nt, st)));
  }
  const int64_t n = M * a.r;
  hipLaunchKernelGGL(k_batch_split, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, T, n, Tp);
  QLK_TRY(hipGetLastError());
  auto go = [&](auto rt, auto h, auto kb) {
    constexpr int RT = decltype(rt)::value, H = decltype(h)::value, KB = decltype(kb)::value;
    const int C = 16 * H;
    BatchGradJob ja{X, K, Up, dA, 1, (int)((K + C - 1) / C), 1};
    BatchGradJob jb{dY, N, Tp, dB, 0, (int)((N + C - 1) / C), 0};
    const dim3 grid((unsigned)(ja.slices + jb.slices), (unsigned)a.slots,
                    (unsigned)((a.r + kGradRanks - 1) / kGradRanks));
    if (d.on)
      hipLaunchKernelGGL((k_batch_grads<RT, H, KB, true>), grid, dim3(256), 0, st, ja, jb, (int)M,
                         a.r, a.slots, a.scale, a.order, a.start, key, d.scale);
    else
      hipLaunchKernelGGL((k_batch_grads<RT, H, KB, false>), grid, dim3(256), 0, st, ja, jb, (int)M,
                         a.r, a.slots, a.scale, a.order, a.start, key, d.scale);
  };
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  using I4 = std::integral_constant<int, 4>;
  if (a.r <= 16) go(I1(), I2(), I2());
  else if (a.r <= 32) go(I2(), I2(), I1());
  else go(I4(), I2(), I1());
  return hipGetLastError();
}

}  // namespace qlk
