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
// 2^-16 of x) where the result is rounded to bf16, three (2^-39) where it is
// kept in fp32.
#include <type_traits>

#include "device_common.h"
#include "kernels.h"
#include "philox.h"

namespace qlk {

typedef short v8s_t __attribute__((ext_vector_type(8)));
typedef unsigned v4u_t __attribute__((ext_vector_type(4)));

// Store through a buffer resource; a lane at kOOB stores nothing.  The whole
// offset goes in the lane's: with a scalar offset register the compiler takes
// a 16-byte store's data registers as free in the next cycle, and a vector
// instruction that wrote them there has replaced the first word of the last
// lanes' data (seen as column indices in out).
__device__ __forceinline__ void bstore128(__amdgpu_buffer_rsrc_t r, uint4 v, uint32_t off) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u_t, v), r, (int)off, 0, 0);
}

// LDS operations done, then the workgroup's barrier; loads from memory into
// registers stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// x as two bf16 terms, hi + mid2, and as three, hi + mid3 + lo.  A product with
// an infinity has to be what x's own would be, so every term has x's sign and is
// zero only where x is:
//  * hi and mid3 are cut toward zero, which also keeps them finite where x lies
//    above bf16's largest value.  Cut, three terms hold all 24 bits of x; of two
//    the last is rounded (within 2^-16 of x; a first term rounded either way
//    would save one bit more but leave a rest of either sign).
//  * a term that would be zero is 2^-40 of hi, far below the others' rounding (a
//    normal number for |x| down to 2^-86).
//  * all terms of an infinity or NaN are x.
__device__ __forceinline__ uint16_t cut_to_bf16(float x) { return (uint16_t)(__float_as_uint(x) >> 16); }
struct Terms {
  uint16_t hi, mid2, mid3, lo;
};
__device__ __forceinline__ Terms split(float x) {
  if (!__builtin_isfinite(x)) {
    const uint16_t v = f32_to_bf16(x);   // a NaN stays one
    return {v, v, v, v};
  }
  Terms t;
  t.hi = cut_to_bf16(x);
  const float hi = bf16_to_f32(t.hi), rest = x - hi;
  t.mid2 = f32_to_bf16(rest);
  t.mid3 = cut_to_bf16(rest);
  t.lo = f32_to_bf16(rest - bf16_to_f32(t.mid3));   // exact
  const uint16_t tiny = f32_to_bf16(hi * 0x1p-40f);
  if ((t.mid2 & 0x7fffu) == 0) t.mid2 = tiny;
  if ((t.mid3 & 0x7fffu) == 0) t.mid3 = tiny;
  if ((t.lo & 0x7fffu) == 0) t.lo = tiny;
  return t;
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
// T = X A_a^T and U = dY B_a as fp32 sums over slices of the contraction,
// part[z] [M, r].  One workgroup takes a tile of the plan (up to 64 tokens of
// one slot, gathered through the order), one slice and up to 64 ranks; its
// four waves take every fourth 64-wide step, each for all 64 tokens, with the
// loads of the next step in flight, and add their sums through LDS in a fixed
// order.  The readers of T and U add the slices in their order.
//
// Bound: HBM, one pass over X (dY), where there are many tokens; the slot's A
// (B) where there are few.  64 tokens per workgroup make the tile's own bytes
// at least the adapter's (which come from L2) up to rank 64, and slices fill
// the device where there are few tiles.  A slice is the fast grid index, so
// that an XCD keeps to its part of the adapters.
// Measured: T, 2048 tokens x 4096, rank 16: 6.5 us (2.6 TB/s of X); 4096 tokens
// x 4096, rank 64: 13 us.  A single token: 3.2 us, the launch and two trips to
// memory.  With dropout the 2048 tokens take 13.4 us, bound by Philox's 32-bit
// products (10 rounds per four elements) and by the tail: 8 slices of 33 to 36
// tiles are 264 to 288 equal workgroups, so some of the 256 CUs hold two, which
// take twice as long side by side.
// U, 4096 tokens, 4096 x 11008, rank 64: 35 us, 186 MB from L2 at 5.2 TB/s and
// 109 MB of HBM at 3.1: neither, but the wait at every step's barrier with one
// step of loads in flight.
constexpr int kDownWaves = 4;

struct DownArgs {
  const uint16_t* S;     // [M, C] bf16
  int M;
  int64_t C;
  const uint16_t* W;     // [slots, r, C] or, WT, [slots, C, r]
  int r, slots;
  const int* order;
  const int* tiles;
  int zlen;              // steps per slice
  float* part;           // fp32 [slices][M, r]
  DropKey drop;
  float keep_scale;
};

// B at 64 ranks: the sums and operands of 64 tokens leave no room for a second
// wave per SIMD (U, 4096 tokens, 4096 x 11008: 62 us), and 32 tokens per
// workgroup read B twice (39 us).  So two waves share a step, each with 32 of
// the 64 tokens: both write half of B's step to one slab, a barrier per step,
// two slabs in turn (35 us).
template <bool WT, int RT>
constexpr bool down_pairs() { return WT && RT == 4; }

// T at 64 ranks: the sums and two steps of X and A take 296 registers, one wave
// per SIMD.
template <bool WT, bool DROP, int RT>
__global__ void __launch_bounds__(64 * kDownWaves, !WT && RT == 4 ? 1 : 2) k_batch_down(DownArgs g) {
  constexpr bool PAIRS = down_pairs<WT, RT>();
  constexpr int TG = PAIRS ? 2 : 4;   // token groups of 16 of a wave
  constexpr int SW = 16 * RT + 8;   // WT: row of a wave's 64 (c) x 16 RT (j) slab, padded
  constexpr int SLAB = WT ? kDownWaves * 64 * SW * 2 : 16, RED = TG * 3 * RT * 64 * 16;
  __shared__ __attribute__((aligned(16))) char smem[SLAB > RED ? SLAB : RED];
  __shared__ int rows[kPlanTile];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int row = lane & 15, grp = lane >> 4;
  const TileRow t = tile_row(g.tiles, blockIdx.y, g.M, g.slots);
  if (t.count <= 0 || t.slot < 0) return;
  if (tid < kPlanTile) {
    const int m = tid < t.count ? g.order[t.first + tid] : -1;
    rows[tid] = (unsigned)m < (unsigned)g.M ? m : -1;
  }
  const int z = blockIdx.x, j0 = (int)blockIdx.z * 64;
  const int r = g.r, ntg = (t.count + 15) / 16;
  const int half = wave & 1, way = wave >> 1;       // of a pair
  const int tg0 = PAIRS && ntg > 1 ? 2 * half : 0;  // this wave's first token group
  const int C = (int)g.C;
  const int nsteps = (C + 63) / 64;
  const int s0 = z * g.zlen, s1 = min(nsteps, s0 + g.zlen);
  __syncthreads();

  // Byte offsets of a lane's pieces at step 0; a step adds 128 bytes (WT: 64
  // rows of B) through the scalar offset.  Lane (row, grp) holds the 16
  // contiguous indices 16 grp .. +15 of the step, MFMA h takes 16 grp + 8 h ..
  // +7, the same permutation for both operands.  WT: piece 64 q + lane of the
  // step's 64 x 16 RT part of B, row by row.
  const __amdgpu_buffer_rsrc_t rs = rsrc_whole(g.S, (uint32_t)((int64_t)g.M * C * 2));
  const __amdgpu_buffer_rsrc_t rw =
      rsrc_whole(g.W + (int64_t)t.slot * C * r, (uint32_t)((int64_t)C * r * 2));
  constexpr int PR = 2 * RT;              // WT: pieces per row
  uint32_t xoff[TG];
#pragma unroll
  for (int tg = 0; tg < TG; ++tg) {
    const int m = rows[16 * (tg0 + tg) + row];
    xoff[tg] = m >= 0 ? (uint32_t)(((int64_t)m * C + 16 * grp) * 2) : kOOB;
  }
  const uint32_t woff = WT ? (uint32_t)((lane / PR) * r + j0 + 8 * (lane % PR)) * 2
                           : (uint32_t)(((int64_t)(j0 + row) * C + 16 * grp) * 2);
  const bool wok = j0 + 8 * (lane % PR) < r;   // WT: the lane's ranks are
  f32x4_t acc[TG][RT];
#pragma unroll
  for (int tg = 0; tg < TG; ++tg)
#pragma unroll
    for (int q = 0; q < RT; ++q) acc[tg][q] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  uint16_t* const my = reinterpret_cast<uint16_t*>(smem) + (WT ? wave * 64 * SW : 0);
  // The wave's steps for NTG token groups (1, or TG with those past the tile at
  // kOOB).  Loads are issued whether or not there is a step, so that the count
  // of those in flight is the same on every path: a wait for one step's leaves
  // the next step's alone.
  auto steps = [&](auto ntgs) {
    constexpr int NTG = decltype(ntgs)::value;
    auto load_w = [&](int st, uint4 (&wv)[2 * RT]) {
      const int sc = __builtin_amdgcn_readfirstlane(st < s1 ? st : s0);
      const uint32_t ss = (uint32_t)sc;
      const int left = st < s1 ? C - 64 * sc : 0;   // indices of this step inside the operand
#pragma unroll
      for (int q = 0; q < 2 * RT; ++q) {
        if constexpr (WT) {
          const int at = q * (64 / PR) + lane / PR;
          // rows past the operand: keep the scalar offset inside it
          const uint32_t so = q * (64 / PR) < left ? (ss * 64 + q * (64 / PR)) * 2 * (uint32_t)r : 0u;
          wv[q] = bload128s(rw, wok && at < left ? woff : kOOB, so);
        } else {
          const int j = j0 + 16 * (q >> 1);
          const uint32_t so = j < r ? ss * 128u + (uint32_t)(32 * (q >> 1)) * (uint32_t)C : 0u;
          wv[q] = bload128s(
              rw, j + row < r && 16 * grp + 8 * (q & 1) < left ? woff + 16 * (q & 1) : kOOB, so);
        }
      }
    };
    auto load_x = [&](int st, uint4 (&xv)[NTG][2]) {
      const int sc = __builtin_amdgcn_readfirstlane(st < s1 ? st : s0);
      const int left = st < s1 ? C - 64 * sc : 0;
#pragma unroll
      for (int tg = 0; tg < NTG; ++tg)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          xv[tg][h] = bload128s(
              rs, xoff[tg] != kOOB && 16 * grp + 8 * h < left ? xoff[tg] + 16 * h : kOOB,
              (uint32_t)sc * 128u);
    };
    // The products of step st; W's registers take the next step's loads as soon
    // as they are free, X's are two sets.
    auto mul = [&](int st, uint4 (&xv)[NTG][2], uint4 (&xn)[NTG][2], uint4 (&wv)[2 * RT]) {
      if constexpr (DROP) {
#pragma unroll
        for (int tg = 0; tg < NTG; ++tg) {
          if (NTG > 1 && tg >= ntg) break;
          const uint32_t m = (uint32_t)max(rows[16 * tg + row], 0);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            xv[tg][h] = philox_drop8(
                xv[tg][h], (uint64_t)m * (uint32_t)C + (uint32_t)(64 * st + 16 * grp + 8 * h), g.drop);
        }
      }
      if constexpr (WT) {
        // A wave's LDS operations run in issue order: the stores are complete
        // before the reads, which complete before the next stores.
#pragma unroll
        for (int q = 0; q < 2 * RT; ++q)
          *reinterpret_cast<uint4*>(my + (q * (64 / PR) + lane / PR) * SW + 8 * (lane % PR)) = wv[q];
        load_w(st + kDownWaves, wv);
        load_x(st + kDownWaves, xn);
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
      }
#pragma unroll
      for (int q = 0; q < RT; ++q) {
        bf16x8_t wop[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (!WT) {
            wop[h] = __builtin_bit_cast(bf16x8_t, wv[2 * q + h]);
          } else {
            const uint16_t* p = my + (16 * grp + 8 * h + (row >> 2)) * SW + 16 * q + 4 * (row & 3);
            const v4s_t lo = lds_read_tr16(p);
            const v4s_t hi = lds_read_tr16(p + 4 * SW);
            const v8s_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            wop[h] = __builtin_bit_cast(bf16x8_t, v);
          }
        }
#pragma unroll
        for (int tg = 0; tg < NTG; ++tg) {
          if (NTG > 1 && tg >= ntg) break;
#pragma unroll
          for (int h = 0; h < 2; ++h)
            acc[tg][q] = mfma_16x16x32(__builtin_bit_cast(bf16x8_t, xv[tg][h]), wop[h], acc[tg][q]);
        }
      }
    };
    uint4 xa[NTG][2], xb[NTG][2], wa[2 * RT];
    [[maybe_unused]] uint4 wb[2 * RT];
    int st = s0 + wave;
    load_w(st, wa);
    load_x(st, xa);
    while (st < s1) {
      if constexpr (!WT) {
        load_w(st + kDownWaves, wb);
        load_x(st + kDownWaves, xb);
      }
      mul(st, xa, xb, wa);
      st += kDownWaves;
      if (st >= s1) break;
      if constexpr (!WT) {
        load_w(st + kDownWaves, wa);
        load_x(st + kDownWaves, xa);
        mul(st, xb, xa, wb);
      } else {
        mul(st, xb, xa, wa);
      }
      st += kDownWaves;
    }
  };
  // The steps of a pair of waves.
  auto pair_steps = [&]() {
    constexpr int HQ = RT;   // a wave's share of the step's 2 RT pieces of B
    uint16_t* const slabs = reinterpret_cast<uint16_t*>(smem) + way * 2 * 64 * SW;
    uint4 wv[HQ], xv[2][TG][2];
    auto load = [&](int st, uint4 (&xn)[TG][2]) {
      const int sc = __builtin_amdgcn_readfirstlane(st < s1 ? st : s0);
      const int left = st < s1 ? C - 64 * sc : 0;
#pragma unroll
      for (int q = 0; q < HQ; ++q) {
        const int from = (half * HQ + q) * (64 / PR), at = from + lane / PR;
        const uint32_t so = from < left ? (uint32_t)(64 * sc + from) * 2 * (uint32_t)r : 0u;
        wv[q] = bload128s(rw, wok && at < left ? woff : kOOB, so);
      }
#pragma unroll
      for (int tg = 0; tg < TG; ++tg)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          xn[tg][h] = bload128s(
              rs, xoff[tg] != kOOB && 16 * grp + 8 * h < left ? xoff[tg] + 16 * h : kOOB,
              (uint32_t)sc * 128u);
    };
    auto mul = [&](int st, uint4 (&xc)[TG][2], uint4 (&xn)[TG][2], uint16_t* slab) {
#pragma unroll
      for (int q = 0; q < HQ; ++q)
        *reinterpret_cast<uint4*>(slab + ((half * HQ + q) * (64 / PR) + lane / PR) * SW +
                                  8 * (lane % PR)) = wv[q];
      load(st + kDownWaves / 2, xn);
      lds_barrier();   // the other slab's reads, of the last step, were before it
#pragma unroll
      for (int q = 0; q < RT; ++q) {
        bf16x8_t wop[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint16_t* p = slab + (16 * grp + 8 * h + (row >> 2)) * SW + 16 * q + 4 * (row & 3);
          const v4s_t lo = lds_read_tr16(p);
          const v4s_t hi = lds_read_tr16(p + 4 * SW);
          const v8s_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
          wop[h] = __builtin_bit_cast(bf16x8_t, v);
        }
#pragma unroll
        for (int tg = 0; tg < TG; ++tg)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            acc[tg][q] = mfma_16x16x32(__builtin_bit_cast(bf16x8_t, xc[tg][h]), wop[h], acc[tg][q]);
      }
    };
    load(s0 + way, xv[0]);
    for (int st = s0; st < s1; st += kDownWaves) {   // every wave meets every barrier
      mul(st + way, xv[0], xv[1], slabs);
      mul(st + way + kDownWaves / 2, xv[1], xv[0], slabs + 64 * SW);
    }
    // acc[tg][q][v]: token 16 (tg0 + tg) + 4 grp + v, rank j0 + 16 q + row.  Of
    // a pair's two, way w adds token group tg0 + w.
    f32x4_t* const red = reinterpret_cast<f32x4_t*>(smem) + half * RT * 2 * 64 + lane;
    __syncthreads();   // the slabs are free
#pragma unroll
    for (int q = 0; q < RT; ++q) red[((1 - way) * RT + q) * 64] = way ? acc[0][q] : acc[1][q];
    __syncthreads();
    float* const out = g.part + (int64_t)z * g.M * r;
    int mo[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) mo[v] = rows[16 * (tg0 + way) + 4 * grp + v];
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      const f32x4_t sum = (way ? acc[1][q] : acc[0][q]) + red[(way * RT + q) * 64];
      const int j = j0 + 16 * q + row;
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (mo[v] >= 0 && j < r) out[(int64_t)mo[v] * r + j] = sum[v];
    }
  };
  if (ntg == 1) {
    steps(std::integral_constant<int, 1>());
  } else if constexpr (PAIRS) {
    pair_steps();
    return;
  } else {
    steps(std::integral_constant<int, TG>());
  }

  // acc[tg][q][v]: token 16 tg + 4 grp + v, rank j0 + 16 q + row.  Wave w adds
  // the four waves' sums of token group w in the order 0, 1, 2, 3.
  f32x4_t* const red = reinterpret_cast<f32x4_t*>(smem);
  if (WT) __syncthreads();   // the slabs are free
#pragma unroll
  for (int tg = 0; tg < TG; ++tg) {
    if (tg >= ntg || tg == wave) continue;
#pragma unroll
    for (int q = 0; q < RT; ++q)
      red[((tg * 3 + (wave < tg ? wave : wave - 1)) * RT + q) * 64 + lane] = acc[tg][q];
  }
  __syncthreads();
  float* const out = g.part + (int64_t)z * g.M * r;
#pragma unroll
  for (int tg = 0; tg < TG; ++tg) {
    if (tg >= ntg || tg != wave) continue;
    int mo[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) mo[v] = rows[16 * tg + 4 * grp + v];
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      f32x4_t sum = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < kDownWaves; ++w) {
        const f32x4_t a =
            w == tg ? acc[tg][q] : red[((tg * 3 + (w < tg ? w : w - 1)) * RT + q) * 64 + lane];
        sum[0] += a[0]; sum[1] += a[1]; sum[2] += a[2]; sum[3] += a[3];
      }
      const int j = j0 + 16 * q + row;
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (mo[v] >= 0 && j < r) out[(int64_t)mo[v] * r + j] = DROP ? sum[v] * g.keep_scale : sum[v];
    }
  }
}

// ---------------------------------------------------------------------------
// U and T as MFMA operands of the gradients' kernel: the slices of part are
// added, split into bf16 terms and written so that a wave loads each operand as 1 KB in a row, lane after lane, with nothing to gather or
// transpose:
//   cols  [chunk][term][rank tile][lane][8]: rank 16 t + i of tokens 8 g ..
//         8 g + 7 of the chunk, lane = 16 g + i (tokens along the contraction),
//         three terms
//   rows  [chunk][token group][rank tile][lane][8]: token 16 tg + i, ranks
//         16 t + 8 (g & 1) .. +7 of term g / 2 (ranks along the contraction),
//         two terms
// A chunk is 32 positions of the order of one slot; slot s begins at chunk
// start[s] / 32 + s.  Ranks past r and tokens past the slot's last are zeros.
// One workgroup per chunk (half a tile of the plan), U or T, and 64 ranks.
// Bound: latency, one round of loads of the slices and one of stores (4096
// tokens at rank 64: 7.5 us, with a whole tile per workgroup 9.5; 2048 tokens
// at rank 16: 4.2).
struct PackJob {
  const float* part;
  int slices;
  uint16_t* cols;
  uint16_t* rows;     // null: not wanted
};
struct PackArgs {
  PackJob u, t;
  int M, r, slots;
  const int* order;
  const int* start;
  const int* tiles;
  int64_t chunks;     // chunks of one block of 64 ranks
};
__host__ __device__ constexpr int64_t pack_chunks(int64_t M, int S) { return M / 32 + S + 1; }

template <int RT>
__global__ void __launch_bounds__(256) k_batch_pack(PackArgs g) {
  constexpr int QW = 16 * RT, LW = QW + 8;
  __shared__ __attribute__((aligned(16))) uint16_t pl[4][32][LW];   // hi, mid3, lo, mid2
  __shared__ int rows[32];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const PackJob& job = blockIdx.y ? g.t : g.u;
  TileRow t = tile_row(g.tiles, (int)blockIdx.x / 2, g.M, g.slots);
  t.first += (int)blockIdx.x % 2 * 32;
  t.count = min(t.count - (int)blockIdx.x % 2 * 32, 32);
  if (t.count <= 0 || t.slot < 0) return;
  const int in_slot = t.first - g.start[t.slot];   // a multiple of 32
  const int64_t chunk = g.start[t.slot] / 32 + t.slot + in_slot / 32;
  if (in_slot < 0 || chunk < 0 || chunk >= g.chunks) return;   // no such plan
  if (tid < 32) {
    const int m = tid < t.count ? g.order[t.first + tid] : -1;
    rows[tid] = (unsigned)m < (unsigned)g.M ? m : -1;
  }
  __syncthreads();
  const int r = g.r, j0 = (int)blockIdx.z * 64;
  for (int e = tid; e < 32 * QW / 4; e += 256) {
    const int tok = e / (QW / 4), j = 4 * (e % (QW / 4));
    const int m = rows[tok];
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (m >= 0 && j0 + j < r) {
      const int64_t at = (int64_t)m * r + j0 + j, plane = (int64_t)g.M * r;
      for (int z = 0; z < job.slices; z += 8) {   // eight loads at a time
        float4 p[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          p[k] = *reinterpret_cast<const float4*>(job.part + min(z + k, job.slices - 1) * plane + at);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (z + k < job.slices) { v.x += p[k].x; v.y += p[k].y; v.z += p[k].z; v.w += p[k].w; }
      }
    }
    const float f[4] = {v.x, v.y, v.z, v.w};
    uint16_t x[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const Terms q = split(f[k]);
      x[0][k] = q.hi; x[1][k] = q.mid3; x[2][k] = q.lo; x[3][k] = q.mid2;
    }
#pragma unroll
    for (int z = 0; z < 4; ++z)
      *reinterpret_cast<uint2*>(&pl[z][tok][j]) =
          make_uint2(x[z][0] | (uint32_t)x[z][1] << 16, x[z][2] | (uint32_t)x[z][3] << 16);
  }
  __syncthreads();
  const int i = lane & 15, q4 = lane >> 4;
  const int64_t block = (int64_t)blockIdx.z * g.chunks + chunk;
  for (int u = wave; u < 3 * RT; u += 4) {
    const int z = u / RT, k = u % RT;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = pl[z][8 * q4 + 2 * e][16 * k + i] |
             (uint32_t)pl[z][8 * q4 + 2 * e + 1][16 * k + i] << 16;
    *reinterpret_cast<uint4*>(job.cols + ((block * 3 + z) * RT + k) * 512 + 8 * lane) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (job.rows == nullptr) return;
  for (int u = wave; u < 2 * RT; u += 4) {
    const int tg = u / RT, k = u % RT;
    *reinterpret_cast<uint4*>(job.rows + ((block * 2 + tg) * RT + k) * 512 + 8 * lane) =
        *reinterpret_cast<const uint4*>(&pl[q4 >> 1 ? 3 : 0][16 * tg + i][16 * k + 8 * (q4 & 1)]);
  }
}

// ---------------------------------------------------------------------------
// out = base + c_a t W_a^T with t = T, W = B ([cols, r] per slot), or, WT,
// t = U, W = A ([r, cols] per slot) and the dropout of the product (the
// backward's dX beyond the ranks that its fused kernel takes).  One workgroup
// takes a tile of the plan (up to 64 tokens of one slot) and blocks of 128
// columns; each of its four waves takes 32 of the tokens and 64 of the columns.
//
//  * v_mfma_f32_16x16x32_bf16 with W rows as the row operand and tokens as
//    columns.  Up to 16 ranks (RK = 16) its 32 contraction indices hold the hi
//    terms of c_a t against W and then the mid terms against the same W; above,
//    32 ranks, and the hi and mid terms take one MFMA each on one W operand.
//  * Every global access is by whole 128-byte lines of consecutive lanes: a
//    wave instruction whose neighbouring lanes lie in different lines takes
//    the address unit four times as long, which bounded the form of this
//    kernel that loaded operands and base in the MFMA's own layout (4096 x
//    11008 at rank 64: 67 us).  W passes through LDS, and the fp32 products
//    through a per-wave slab from which the lanes take 16-byte pieces of rows.
//  * A lane reads and writes the same places of base and out, which may
//    therefore be one tensor.
//  * base and W of the next block are on their way while a block is computed,
//    the first block's while t is gathered from its slices.
// Bound: HBM, base read and out written once; W comes from L2 once per tile.
// The column block is the fast grid index: an XCD keeps to its part of W.
// Measured: 2048 tokens x 4096, rank 16: 9.9 us (33.6 MB, 3.4 TB/s); 4096 x
// 11008, rank 64: 45 us (180 MB, 4.0 TB/s); 256 single tokens of 64 adapters x
// 11008, rank 16: 10.2 us.
constexpr int kUpCols = 128;    // columns per block
constexpr int kUpWaves = kPlanTile / 16;
constexpr int kUpSlab = 64 + 4; // row of a wave's 16 x 64 fp32 slab

struct UpArgs {
  const uint16_t* base;  // [M, cols] bf16 or null (zeros)
  uint16_t* out;         // [M, cols] bf16
  int M;
  int64_t cols;
  const float* part;     // t: fp32 [slices][M, r], to be added
  int slices;
  float* t_out;          // t itself, fp32 [M, r], or null
  const uint16_t* W;
  const float* scale;    // [slots]
  int r, slots;
  const int* order;
  const int* tiles;
  DropKey drop;
  float keep_scale;
};

// RK ranks of W in LDS at a time, in NS stages (NS = 1: all of them).
template <bool WT, bool DROP, int RK, int NS>
__global__ void __launch_bounds__(64 * kUpWaves) k_batch_up(UpArgs g) {
  constexpr int LD = NS * RK * 2 + 8;            // LDS row of a token: RK hi, RK mid terms per stage
  constexpr int LW = WT ? kUpCols + 8 : RK + 8;  // LDS row of W: a rank's columns or a column's ranks
  constexpr int WP = RK / 16;                    // 16-byte pieces of W per lane and stage
  __shared__ __attribute__((aligned(16))) uint16_t tl[kPlanTile * LD];
  __shared__ __attribute__((aligned(16))) uint16_t wl[WT ? RK * LW : kUpCols * LW];
  __shared__ __attribute__((aligned(16))) float slab[kUpWaves][16 * kUpSlab];
  __shared__ int rows[kPlanTile];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i = lane & 15, q4 = lane >> 4;
  const TileRow t = tile_row(g.tiles, blockIdx.y, g.M, g.slots);
  if (t.count <= 0) return;
  const int cols = (int)g.cols;
  const int blocks = (cols + kUpCols - 1) / kUpCols;
  const int r = g.r;
  if (tid < kPlanTile) {
    const int m = tid < t.count ? g.order[t.first + tid] : -1;
    rows[tid] = (unsigned)m < (unsigned)g.M ? m : -1;
  }
  __syncthreads();
  const int th = wave & 1, wc = 64 * (wave >> 1);   // token half, first column of the wave
  float* const my = slab[wave];
  // Byte offsets of this lane's pieces in block 0; a block adds its columns
  // through the scalar offset, and columns past the last are left out.
  const uint32_t brow = (uint32_t)cols * 2;
  const __amdgpu_buffer_rsrc_t rb = rsrc_whole(g.base, g.base ? (uint32_t)g.M * brow : 0u);
  const __amdgpu_buffer_rsrc_t ro = rsrc_whole(g.out, (uint32_t)g.M * brow);
  // Piece (tg, h): token 32 th + 16 tg + 8 h + lane / 8, columns pc .. of a block.
  const int pc = wc + 8 * (lane & 7);
  const int pt = 32 * th + (lane >> 3);
  uint32_t boff[2][2];
#pragma unroll
  for (int tg = 0; tg < 2; ++tg)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int m = rows[pt + 16 * tg + 8 * h];
      boff[tg][h] = m >= 0 ? (uint32_t)m * brow + (uint32_t)pc * 2 : kOOB;
    }
  // A block past the last has no columns: every lane is at kOOB, and the scalar
  // offset stays inside the operand.
  auto block_at = [&](int cb, uint32_t bytes) { return cb < blocks ? (uint32_t)cb * bytes : 0u; };
  auto load_b = [&](int cb, uint4 (&bv)[2][2]) {
    const bool ok = pc < cols - cb * kUpCols;
    const uint32_t at = block_at(cb, kUpCols * 2);
#pragma unroll
    for (int tg = 0; tg < 2; ++tg)
#pragma unroll
      for (int h = 0; h < 2; ++h) bv[tg][h] = bload128s(rb, ok ? boff[tg][h] : kOOB, at);
  };
  const int step = gridDim.x;
  uint4 ba[2][2], bb[2][2];
  int cb = blockIdx.x;
  if (t.slot < 0) {   // no adapter: t = 0, the base alone
    if (cb < blocks) load_b(cb, ba);
    if (g.t_out && blockIdx.x == 0)
      for (int e = tid; e < t.count * r; e += 64 * kUpWaves)
        if (rows[e / r] >= 0) g.t_out[(int64_t)rows[e / r] * r + e % r] = 0.0f;
    if (g.out == g.base) return;
    auto copy = [&](int cb, const uint4 (&cur)[2][2], uint4 (&next)[2][2]) {
      const bool ok = pc < cols - cb * kUpCols;
      const uint32_t at = (uint32_t)cb * (kUpCols * 2);
      load_b(cb + step, next);
#pragma unroll
      for (int tg = 0; tg < 2; ++tg)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          bstore128(ro, cur[tg][h], ok && boff[tg][h] != kOOB ? boff[tg][h] + at : kOOB);
    };
    while (cb < blocks) {
      copy(cb, ba, bb);
      cb += step;
      if (cb >= blocks) break;
      copy(cb, bb, ba);
      cb += step;
    }
    return;
  }
  const int stages = NS == 1 ? 1 : (r + RK - 1) / RK;
  const float c_a = g.scale[t.slot];
  const uint16_t* const W = g.W + (int64_t)t.slot * cols * r;
  const __amdgpu_buffer_rsrc_t rw = rsrc_whole(W, brow * (uint32_t)r);
  auto load_w = [&](int cb, int j0, uint4 (&wv)[WP]) {
    const int left = cols - cb * kUpCols;
    const uint32_t at = block_at(cb, WT ? kUpCols * 2 : kUpCols * 2 * (uint32_t)r);
#pragma unroll
    for (int q = 0; q < WP; ++q) {
      const int p = 256 * q + tid;
      if constexpr (!WT) {
        const int c = p / (RK / 8), j = j0 + 8 * (p % (RK / 8));
        wv[q] = bload128s(rw, c < left && j < r ? (uint32_t)(c * r + j) * 2 : kOOB, at);
      } else {
        const int j = j0 + p / (kUpCols / 8), c = 8 * (p % (kUpCols / 8));
        wv[q] = bload128s(rw, c < left && j < r ? (uint32_t)j * brow + 2 * c : kOOB, at);
      }
    }
  };
  auto store_w = [&](const uint4 (&wv)[WP]) {
#pragma unroll
    for (int q = 0; q < WP; ++q) {
      const int p = 256 * q + tid;
      constexpr int PPR = WT ? kUpCols / 8 : RK / 8;
      *reinterpret_cast<uint4*>(wl + (p / PPR) * LW + 8 * (p % PPR)) = wv[q];
    }
  };
  // Operands of t: RK ranks of token 32 th + 16 tg + i, as hi and mid terms.
  constexpr int NT = RK == 16 ? 1 : RK / 16;
  bf16x8_t top[2][NT];
  auto load_t = [&](int stage) {
#pragma unroll
    for (int tg = 0; tg < 2; ++tg)
#pragma unroll
      for (int k = 0; k < NT; ++k)
        top[tg][k] = *reinterpret_cast<const bf16x8_t*>(
            tl + (32 * th + 16 * tg + i) * LD + stage * 2 * RK + 32 * k + 8 * q4);
  };
  f32x4_t acc[2][4];   // [token group][columns wc + 16 k + 4 q4 + v]
  auto multiply = [&](int tgs) {
#pragma unroll
    for (int ch = 0; ch < (RK + 31) / 32; ++ch) {
      const int jw = RK == 16 ? 8 * (q4 & 1) : 32 * ch + 8 * q4;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        bf16x8_t wop;
        if constexpr (!WT) {
          wop = *reinterpret_cast<const bf16x8_t*>(wl + (wc + 16 * k + i) * LW + jw);
        } else {
          const uint16_t* const p = wl + (jw + (i >> 2)) * LW + wc + 16 * k + 4 * (i & 3);
          const v4s_t lo = lds_read_tr16(p);
          const v4s_t hi = lds_read_tr16(p + 4 * LW);
          const v8s_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
          wop = __builtin_bit_cast(bf16x8_t, v);
        }
#pragma unroll
        for (int tg = 0; tg < 2; ++tg) {
          if (tg >= tgs) break;
          if (RK > 16) acc[tg][k] = mfma_16x16x32(wop, top[tg][RK / 32 + ch], acc[tg][k]);   // mid first
          acc[tg][k] = mfma_16x16x32(wop, top[tg][ch], acc[tg][k]);
        }
      }
    }
  };
  auto finish = [&](int cb, int tgs, const uint4 (&bv)[2][2]) {
    const bool ok = pc < cols - cb * kUpCols;
    const uint32_t at = (uint32_t)cb * (kUpCols * 2);
#pragma unroll
    for (int tg = 0; tg < 2; ++tg) {
      if (tg >= tgs) break;
      // A wave's LDS operations run in issue order: these stores land after
      // the last group's reads.
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<f32x4_t*>(my + i * kUpSlab + 16 * k + 4 * q4) = acc[tg][k];
      __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float* const e = my + (8 * h + (lane >> 3)) * kUpSlab + 8 * (lane & 7);
        const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(e);
        const f32x4_t hi = *reinterpret_cast<const f32x4_t*>(e + 4);
        float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        if constexpr (DROP) {
          const uint64_t o = (uint64_t)max(rows[pt + 16 * tg + 8 * h], 0) * (uint64_t)cols +
                             (uint64_t)(cb * kUpCols + pc);
          const uint32_t keep = philox_keep8(o, g.drop);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = (keep >> k) & 1u ? v[k] * g.keep_scale : 0.0f;
        }
        const uint4 b = bv[tg][h];
        uint4 w;
        w.x = pack_bf16x2(bf16_to_f32(b.x & 0xffffu) + v[0], bf16_to_f32(b.x >> 16) + v[1]);
        w.y = pack_bf16x2(bf16_to_f32(b.y & 0xffffu) + v[2], bf16_to_f32(b.y >> 16) + v[3]);
        w.z = pack_bf16x2(bf16_to_f32(b.z & 0xffffu) + v[4], bf16_to_f32(b.z >> 16) + v[5]);
        w.w = pack_bf16x2(bf16_to_f32(b.w & 0xffffu) + v[6], bf16_to_f32(b.w >> 16) + v[7]);
        bstore128(ro, w, ok && boff[tg][h] != kOOB ? boff[tg][h] + at : kOOB);
      }
    }
  };

  uint4 wv[WP];
  // A narrow tile's pieces: base of token i, W rows of the wave's 64 columns.
  constexpr bool NARROW = !WT && NS == 1;
  constexpr int NQ = (RK + 31) / 32;
  const bool narrow = NARROW && t.count <= 16;
  uint4 na[2], nb[2], wa[2][NQ][2], wb[2][NQ][2];
  const int mi = rows[i];
  const uint32_t noff = mi >= 0 ? (uint32_t)mi * brow + (uint32_t)(64 * wave + 8 * q4) * 2 : kOOB;
  auto load_n = [&](int cb, uint4 (&bv)[2], uint4 (&w)[2][NQ][2]) {
    const int left = cols - cb * kUpCols;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int c = 64 * wave + 32 * u;
#pragma unroll
      for (int ch = 0; ch < NQ; ++ch)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int n = c + 8 * (i >> 2) + 4 * k + (i & 3);
          const int j = RK == 16 ? 8 * (q4 & 1) : 32 * ch + 8 * q4;
          w[u][ch][k] = bload128s(rw, n < left && j < r ? (uint32_t)(n * r + j) * 2 : kOOB,
                                  block_at(cb, kUpCols * 2 * (uint32_t)r));
        }
      bv[u] = bload128s(rb, noff != kOOB && c + 8 * q4 < left ? noff + 64 * u : kOOB,
                        block_at(cb, kUpCols * 2));
    }
  };
  if (NARROW && narrow) {
    cb = 2 * blockIdx.x;
    load_n(cb, na, wa);
  } else if (cb < blocks) {
    load_b(cb, ba);
    load_w(cb, 0, wv);
  }
  // t of the tile: its slices added in order, eight loads at a time.
  for (int e = tid; e < kPlanTile * NS * RK / 4; e += 64 * kUpWaves) {
    const int tok = e / (NS * RK / 4), j = 4 * (e % (NS * RK / 4));
    const int m = rows[tok];
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (m >= 0 && j < r) {
      const int64_t at = (int64_t)m * r + j, plane = (int64_t)g.M * r;
      for (int z = 0; z < g.slices; z += 8) {
        float4 p[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          p[k] = *reinterpret_cast<const float4*>(g.part + min(z + k, g.slices - 1) * plane + at);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (z + k < g.slices) { v.x += p[k].x; v.y += p[k].y; v.z += p[k].z; v.w += p[k].w; }
      }
      if (g.t_out && blockIdx.x == 0) *reinterpret_cast<float4*>(g.t_out + at) = v;
      v.x *= c_a; v.y *= c_a; v.z *= c_a; v.w *= c_a;
    }
    const float f[4] = {v.x, v.y, v.z, v.w};
    uint16_t hi[4], mid[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const Terms q = split(f[k]);
      hi[k] = q.hi; mid[k] = q.mid2;
    }
    uint16_t* const d = tl + tok * LD + (j / RK) * 2 * RK + j % RK;
    *reinterpret_cast<uint2*>(d) =
        make_uint2(hi[0] | (uint32_t)hi[1] << 16, hi[2] | (uint32_t)hi[3] << 16);
    *reinterpret_cast<uint2*>(d + RK) =
        make_uint2(mid[0] | (uint32_t)mid[1] << 16, mid[2] | (uint32_t)mid[3] << 16);
  }
  __syncthreads();
  if constexpr (NARROW) {
    if (narrow) {
      // Up to 16 tokens (a step of single tokens): W is what is read, once per
      // tile, and goes straight into the MFMA's operand registers, two blocks
      // at a time, a wave 64 columns; no barrier.  Row rho of half k stands for
      // column 8 (rho / 4) + 4 k + rho % 4 of 32, so that a lane's two products
      // of a token are 8 consecutive columns.
      bf16x8_t tn[NT];
#pragma unroll
      for (int k = 0; k < NT; ++k)
        tn[k] = *reinterpret_cast<const bf16x8_t*>(tl + i * LD + 32 * k + 8 * q4);
      auto done = [&](int cb, const uint4 (&bv)[2], const uint4 (&w)[2][NQ][2]) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int c = cb * kUpCols + 64 * wave + 32 * u + 8 * q4;
          f32x4_t d[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            d[k] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int ch = 0; ch < NQ; ++ch) {
              const bf16x8_t wop = __builtin_bit_cast(bf16x8_t, w[u][ch][k]);
              if (RK > 16) d[k] = mfma_16x16x32(wop, tn[RK / 32 + ch], d[k]);   // mid first
              d[k] = mfma_16x16x32(wop, tn[ch], d[k]);
            }
          }
          uint4 o;
          o.x = pack_bf16x2(bf16_to_f32(bv[u].x & 0xffffu) + d[0][0], bf16_to_f32(bv[u].x >> 16) + d[0][1]);
          o.y = pack_bf16x2(bf16_to_f32(bv[u].y & 0xffffu) + d[0][2], bf16_to_f32(bv[u].y >> 16) + d[0][3]);
          o.z = pack_bf16x2(bf16_to_f32(bv[u].z & 0xffffu) + d[1][0], bf16_to_f32(bv[u].z >> 16) + d[1][1]);
          o.w = pack_bf16x2(bf16_to_f32(bv[u].w & 0xffffu) + d[1][2], bf16_to_f32(bv[u].w >> 16) + d[1][3]);
          bstore128(ro, o, noff != kOOB && c < cols ? noff + 64 * u + (uint32_t)cb * (kUpCols * 2) : kOOB);
        }
      };
      const int nstep = 2 * step;
      while (cb < blocks) {
        load_n(cb + nstep, nb, wb);
        done(cb, na, wa);
        cb += nstep;
        if (cb >= blocks) break;
        load_n(cb + nstep, na, wa);
        done(cb, nb, wb);
        cb += nstep;
      }
      return;
    }
  }
  if (NS == 1) load_t(0);
  // One block: W from registers to LDS (every wave is done with the last
  // block's), the next block's loads, the products, the epilogue.  FULL: all
  // token groups hold tokens.  Loads are issued whether or not there is a next
  // block (at kOOB past the last), so that the count of those in flight is the
  // same on every path and a wait for W leaves the younger ones alone.
  auto run = [&](auto full) {
    constexpr bool FULL = decltype(full)::value;
    const int tgs = FULL ? 2 : max(0, min(2, (t.count - 32 * th + 15) / 16));
    auto block = [&](int cb, uint4 (&cur)[2][2], uint4 (&next)[2][2]) {
#pragma unroll
      for (int tg = 0; tg < 2; ++tg)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[tg][k] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      if constexpr (NS == 1) {
        lds_barrier();
        store_w(wv);
        load_w(cb + step, 0, wv);
        if (FULL || tgs > 0) load_b(cb + step, next);
        lds_barrier();
        if (FULL || tgs > 0) multiply(tgs);
      } else {
        for (int stage = 0; stage < stages; ++stage) {
          lds_barrier();
          store_w(wv);
          const bool last = stage + 1 == stages;
          load_w(last ? cb + step : cb, last ? 0 : (stage + 1) * RK, wv);
          lds_barrier();
          load_t(stage);
          multiply(tgs);
        }
        load_b(cb + step, next);
      }
      if (FULL || tgs > 0) finish(cb, tgs, cur);
    };
    while (cb < blocks) {
      block(cb, ba, bb);
      cb += step;
      if (cb >= blocks) break;
      block(cb, bb, ba);
      cb += step;
    }
  };
  if (t.count > kPlanTile - 16) run(std::true_type());
  else run(std::false_type());
}

// ---------------------------------------------------------------------------
// The backward's sums over tokens, dA_a = c_a U^T drop(X) and dB_a = c_a dY^T T
// in fp32 (every slot written, zeros without tokens), and, on the way over X's
// columns, dX = dX0 + drop(c_a U A_a).  Both gradients are O[c][j] = sum P[m][c]
// Q[m][j], (P, Q) = (X, U) with O = dA^T or (dY, T) with O = dB.
//
// A workgroup owns a slot, 64 columns of P (128 for dB at 64 ranks) and up to
// 64 ranks, and contracts over all of the slot's tokens, gathered through the
// plan's order: no partial sums in memory, no atomics.  Its NW waves take every
// NW-th 32-token chunk.  The slot with the most tokens comes first, so that the
// longest sums do not start last (78 -> 70 us below).
//  * Lane L holds columns 8 (L % 8) of tokens 8 h + L / 8, h = 0..3: eight whole
//    128-byte lines per instruction, for P, dX0 and dX alike, so that the
//    dropout's words of X and of dX are drawn once.
//  * P passes through a slab of LDS per wave and comes back as MFMA operands
//    with the transposing read, tokens along the contraction; its registers
//    take the next chunk's loads as soon as they are in the slab.  Q's operands
//    (cols, and for dX rows) come packed from memory: passed through the slab
//    as well, the three terms of 64 ranks bounded the kernel by LDS (4096
//    tokens, 4096 x 11008: 84 us, packed 78).
//  * dX's row operand, the slot's A over these columns, stays in LDS; the
//    products leave through P's slab (16-byte pieces of row i XOR-swizzled by i).
//  * The waves' sums are added in the order 0, 1, ..., NW - 1.
// Bound: up to 32 ranks HBM, X, dY and dX0 read once, dX and all slots' dA and
// dB written (2048 tokens, 4096 x 4096, rank 16: 14.8 us, 67 MB in and out, 4.5
// TB/s; with dropout 23, Philox); at 64 ranks L2 and HBM together, since every
// slice reads Q (4096 tokens, 4096 x 11008: 56.6 us, with dropout 62 to 65: 497
// MB from L2 at 8 TB/s, about 260 MB of HBM at 4.2).
// The tokens of a slot are not split, so the slots in use times (K + N) / 64
// workgroups are all there is: one adapter of 4096 x 4096 takes 20.1 us for the
// same 2048 tokens, of 1024 x 1024 18.7.
constexpr int kGradRanks = 64;
constexpr int kGradSlice = 64;

struct BatchGradJob {
  const uint16_t* P;     // [M, cols] bf16
  int64_t cols;
  const uint16_t* Q;     // packed cols of U or T
  float* out;            // trans: [slots, r, cols] (dA); else [slots, cols, r] (dB)
  int trans, slices;
};
struct BatchGradArgs {
  BatchGradJob a, b;     // dA (with dX), dB
  const uint16_t* Urows; // packed rows of U, for dX
  int64_t chunks;        // chunks of one block of 64 ranks
  int M, r, slots;
  const float* scale;
  const int* order;
  const int* start;
  const uint16_t* A;     // [slots, r, K], for dX
  const uint16_t* dX0;
  uint16_t* dX;
  DropKey drop;
  float keep_scale;
};

// 16 x 32 operand of P's slab of 32 rows of 64: lane (i, q4) gets column 16 band
// + i of rows 8 q4 .. 8 q4 + 7.
__device__ __forceinline__ bf16x8_t slab_operand(const uint16_t* slab, int band, int lane) {
  const int i = lane & 15;
  const uint16_t* const p =
      slab + (8 * (lane >> 4) + (i >> 2)) * kGradSlice + 16 * band + 4 * (i & 3);
  const v4s_t lo = lds_read_tr16(p);
  const v4s_t hi = lds_read_tr16(p + 4 * kGradSlice);
  const v8s_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  return __builtin_bit_cast(bf16x8_t, v);
}

// 64-column blocks of a slice: two for dB at 64 ranks, where Q's bytes, read by
// every slice, are the larger part.
template <int RT>
constexpr int grad_blocks_b() { return RT == 4 ? 2 : 1; }

template <int RT, int NW>
struct GradShape {
  static constexpr int PE = 32 * kGradSlice;        // elements of a chunk of P
  static constexpr int AW = 16 * RT + 8;            // LDS row of a column of A
  static constexpr int SLAB = NW * grad_blocks_b<RT>() * PE * 2, RED = NW * 4 * RT * 64 * 16;
  static constexpr int SMEM = SLAB > RED ? SLAB : RED;
};

// One workgroup's share of dA (and, DX, of dX) or of dB: `sl` is its slice.
// Which of the two is fixed at compile time, so that the count of loads and
// stores in flight is the same on every path of the loop.
template <int RT, bool DROP, bool DX, int NW, int CB>
__device__ __forceinline__ void grads_block(const BatchGradArgs& g, const BatchGradJob& job, int sl,
                                            int slot, char* smem, uint16_t* as) {
  using Sh = GradShape<RT, NW>;
  constexpr int AW = Sh::AW;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i = lane & 15, q4 = lane >> 4;
  const int cols = (int)job.cols;
  const int c0 = sl * CB * kGradSlice;
  const int M = g.M, r = g.r;
  const int j0 = (int)blockIdx.z * kGradRanks;
  // The slot's range of the order, cut to M tokens whatever the plan holds.
  const int s0 = min(max(g.start[slot], 0), M), s1 = min(max(g.start[slot + 1], s0), M);
  const int nt = s1 - s0;
  const int prow = lane >> 3, c = c0 + 8 * (lane & 7);   // this lane's columns
  const uint32_t prowb = (uint32_t)cols * 2;
  const __amdgpu_buffer_rsrc_t rx0 =
      rsrc_whole(g.dX0, DX && g.dX0 ? (uint32_t)M * prowb : 0u);
  const __amdgpu_buffer_rsrc_t rdx = rsrc_whole(g.dX, DX ? (uint32_t)M * prowb : 0u);
  const int nchunks = (nt + 31) / 32;
  // Tokens of chunk ci (lane L: token L % 32), -1 past the slot's last.
  auto tokens = [&](int ci) {
    const int pos = ci * 32 + (lane & 31);
    const int m = pos < nt ? g.order[s0 + pos] : -1;
    return (unsigned)m < (unsigned)M ? m : -1;
  };
  // Byte offsets of this lane's four pieces of P (dX0, dX).
  auto places = [&](int tok, uint32_t (&off)[4]) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int m = __shfl(tok, 8 * h + prow);
      off[h] = m >= 0 && c < cols ? (uint32_t)m * prowb + (uint32_t)c * 2 : kOOB;
    }
  };
  if (DX && slot == g.slots) {   // tokens without an adapter: dX = dX0
    if (g.dX == g.dX0) return;
    int tok = tokens(wave);
    for (int ci = wave; ci < nchunks; ci += NW) {
      uint32_t off[4];
      uint4 v[4];
      places(tok, off);
      tok = tokens(ci + NW);
#pragma unroll
      for (int h = 0; h < 4; ++h) v[h] = bload128s(rx0, off[h], 0);
#pragma unroll
      for (int h = 0; h < 4; ++h) bstore128(rdx, v[h], off[h]);
    }
    return;
  }
  float* const out = job.out + (int64_t)slot * cols * r;
  if (nt == 0) {   // a slot without tokens: zeros, whatever its scale
    constexpr int W = CB * kGradSlice;
    for (int e = tid; e < W * 16 * RT; e += 64 * NW) {
      const int j = job.trans ? e / W : e % (16 * RT);
      const int cc = c0 + (job.trans ? e % W : e / (16 * RT));
      if (cc < cols && j0 + j < r)
        out[job.trans ? (int64_t)(j0 + j) * cols + cc : (int64_t)cc * r + j0 + j] = 0.0f;
    }
    return;
  }
  const __amdgpu_buffer_rsrc_t rp = rsrc_whole(job.P, (uint32_t)M * prowb);
  const float c_a = g.scale[slot];
  // The slot's chunks in the packed operands (a plan that does not fit the
  // batch must not lead past them).
  int64_t first = s0 / 32 + slot;
  if (first + nchunks > g.chunks) first = g.chunks - nchunks;
  first += (int64_t)blockIdx.z * g.chunks;
  const uint4* const qcols = reinterpret_cast<const uint4*>(job.Q) + first * (3 * RT * 64) + lane;
  const uint4* const qrows = reinterpret_cast<const uint4*>(g.Urows) + first * (2 * RT * 64) + lane;

  uint4 pv[CB][4], qv[3][RT], uv[2][RT], xv[4];
  uint32_t off[4], next[4];
  auto load_p = [&](int tok) {
    places(tok, next);
#pragma unroll
    for (int b = 0; b < CB; ++b)
#pragma unroll
      for (int h = 0; h < 4; ++h)
        pv[b][h] = bload128s(rp, b == 0 || (next[h] != kOOB && c + b * kGradSlice < cols)
                                     ? next[h] + b * (kGradSlice * 2) : kOOB, 0);
  };
  // Past the wave's last chunk these load the slot's last again.
  auto load_q = [&](int ci, int z) {
    const uint4* const q = qcols + (int64_t)min(ci, nchunks - 1) * (3 * RT * 64) + z * RT * 64;
#pragma unroll
    for (int t = 0; t < RT; ++t) qv[z][t] = q[64 * t];
  };
  auto load_u = [&](int ci) {
    const uint4* const q = qrows + (int64_t)min(ci, nchunks - 1) * (2 * RT * 64);
#pragma unroll
    for (int tg = 0; tg < 2; ++tg)
#pragma unroll
      for (int t = 0; t < RT; ++t) uv[tg][t] = q[(tg * RT + t) * 64];
  };
  auto load_x = [&]() {
#pragma unroll
    for (int h = 0; h < 4; ++h) xv[h] = bload128s(rx0, next[h], 0);
  };
  int tok = tokens(wave);
#pragma unroll
  for (int z = 2; z >= 0; --z) load_q(wave, z);
  if constexpr (DX) load_u(wave);
  load_p(tok);
  if constexpr (DX) load_x();
  tok = tokens(wave + NW);
  if (DX) {   // as[column][rank] = A, transposed
    const uint16_t* const A = g.A + (int64_t)slot * r * cols;
    for (int e = tid; e < 16 * RT * (kGradSlice / 8); e += 64 * NW) {
      const int j = e / (kGradSlice / 8), k0 = 8 * (e % (kGradSlice / 8));
      uint4 v = make_uint4(0, 0, 0, 0);
      if (j < r && c0 + k0 < cols) v = *reinterpret_cast<const uint4*>(A + (int64_t)j * cols + c0 + k0);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) as[(k0 + k) * AW + j] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
    }
    lds_barrier();
  }

  uint16_t* const my = reinterpret_cast<uint16_t*>(smem) + wave * CB * Sh::PE;
  f32x4_t acc[CB][4][RT];
#pragma unroll
  for (int b = 0; b < CB; ++b)
#pragma unroll
    for (int h = 0; h < 4; ++h)
#pragma unroll
      for (int t = 0; t < RT; ++t) acc[b][h][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const float s = DROP ? c_a * g.keep_scale : c_a;

  for (int ci = wave; ci < nchunks; ci += NW) {
    uint32_t keep = 0;   // 8 bits per piece
#pragma unroll
    for (int h = 0; h < 4; ++h) off[h] = next[h];
    if constexpr (DROP) {
#pragma unroll
      for (int h = 0; h < 4; ++h)
        if (off[h] != kOOB) keep |= philox_keep8(off[h] >> 1, g.drop) << (8 * h);
    }
    // A wave's LDS operations run in issue order: these stores land after the
    // last chunk's reads.
#pragma unroll
    for (int bh = 0; bh < 4 * CB; ++bh) {
      const int h = bh & 3;
      uint4 v = pv[bh >> 2][h];
      if constexpr (DROP) {
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] &= ((keep >> (8 * h + 2 * e)) & 1u ? 0xffffu : 0u) |
                  ((keep >> (8 * h + 2 * e + 1)) & 1u ? 0xffff0000u : 0u);
        v = make_uint4(w[0], w[1], w[2], w[3]);
      }
      *reinterpret_cast<uint4*>(my + 8 * (64 * bh + lane)) = v;
    }
    load_p(tok);
    tok = tokens(ci + 2 * NW);
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
#pragma unroll
    for (int b = 0; b < CB; ++b) {
      bf16x8_t aop[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) aop[h] = slab_operand(my + b * Sh::PE, h, lane);
#pragma unroll
      for (int z = 2; z >= 0; --z) {      // the small terms first
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int h = 0; h < 4; ++h)
            acc[b][h][t] =
                mfma_16x16x32(aop[h], __builtin_bit_cast(bf16x8_t, qv[z][t]), acc[b][h][t]);
        if (b == CB - 1) load_q(ci + NW, z);
      }
    }
    if constexpr (DX) {
      // dX[m][c]: row operand A's column 16 k + i, ranks 16 ch + 8 (q4 & 1) ..;
      // column operand U's token 16 tg + i, the hi terms (q4 < 2) and the mid
      // terms of the same ranks.
      f32x4_t d[2][4];
#pragma unroll
      for (int tg = 0; tg < 2; ++tg)
#pragma unroll
        for (int k = 0; k < 4; ++k) d[tg][k] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int ch = 0; ch < RT; ++ch) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bf16x8_t wop =
              *reinterpret_cast<const bf16x8_t*>(as + (16 * k + i) * AW + 16 * ch + 8 * (q4 & 1));
#pragma unroll
          for (int tg = 0; tg < 2; ++tg)
            d[tg][k] = mfma_16x16x32(wop, __builtin_bit_cast(bf16x8_t, uv[tg][ch]), d[tg][k]);
        }
      }
      load_u(ci + NW);
      float* const e = reinterpret_cast<float*>(my);   // 16 rows of 64 floats
#pragma unroll
      for (int tg = 0; tg < 2; ++tg) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<f32x4_t*>(e + 64 * i + 4 * ((4 * k + q4) ^ i)) = d[tg][k];
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int h = 2 * tg + hh, row = 8 * hh + prow, pp = 2 * (lane & 7);
          const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(e + 64 * row + 4 * (pp ^ row));
          const f32x4_t hi = *reinterpret_cast<const f32x4_t*>(e + 64 * row + 4 * ((pp + 1) ^ row));
          float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            v[k] *= s;
            if (DROP) v[k] = (keep >> (8 * h + k)) & 1u ? v[k] : 0.0f;
          }
          const uint4 b = xv[h];
          uint4 w;
          w.x = pack_bf16x2(bf16_to_f32(b.x & 0xffffu) + v[0], bf16_to_f32(b.x >> 16) + v[1]);
          w.y = pack_bf16x2(bf16_to_f32(b.y & 0xffffu) + v[2], bf16_to_f32(b.y >> 16) + v[3]);
          w.z = pack_bf16x2(bf16_to_f32(b.z & 0xffffu) + v[4], bf16_to_f32(b.z >> 16) + v[5]);
          w.w = pack_bf16x2(bf16_to_f32(b.w & 0xffffu) + v[6], bf16_to_f32(b.w >> 16) + v[7]);
          bstore128(rdx, w, off[h]);
        }
      }
      load_x();
    }
  }

  // acc[b][h][t][v] = O[c0 + 64 b + 16 h + 4 q4 + v][j0 + 16 t + i]; the unit
  // (h, t) is added by wave (h RT + t) mod NW.
  f32x4_t* const red = reinterpret_cast<f32x4_t*>(smem) + lane;
#pragma unroll
  for (int b = 0; b < CB; ++b) {
    lds_barrier();   // the slabs, or the last block's sums, are free
#pragma unroll
    for (int h = 0; h < 4; ++h)
#pragma unroll
      for (int t = 0; t < RT; ++t) red[(wave * 4 * RT + h * RT + t) * 64] = acc[b][h][t];
    lds_barrier();
    for (int unit = wave; unit < 4 * RT; unit += NW) {
      f32x4_t v = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const f32x4_t o = red[(w * 4 * RT + unit) * 64];
        v[0] += o[0]; v[1] += o[1]; v[2] += o[2]; v[3] += o[3];
      }
      // cc .. cc + 3 (cols is a multiple of 8)
      const int cc = c0 + b * kGradSlice + 16 * (unit / RT) + 4 * q4;
      const int j = j0 + 16 * (unit % RT) + i;
      if (cc >= cols || j >= r) continue;
      if (job.trans) {
        *reinterpret_cast<f32x4_t*>(out + (int64_t)j * cols + cc) =
            f32x4_t{s * v[0], s * v[1], s * v[2], s * v[3]};
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) out[(int64_t)(cc + e) * r + j] = s * v[e];
      }
    }
  }
}

// The slot with the n-th most tokens, so that the longest sums start first (up
// to 64 slots; beyond, slot n).
__device__ __forceinline__ int slot_by_size(const int* start, int slots, int n) {
  if (slots > 64) return n;
  const int lane = threadIdx.x & 63;
  const int mine = lane < slots ? start[lane + 1] - start[lane] : -1;
  int before = 0;
  for (int l = 0; l < slots; ++l) {
    const int other = __builtin_amdgcn_readlane(mine, l);
    before += other > mine || (other == mine && l < lane) ? 1 : 0;
  }
  return __builtin_ctzll(__ballot(lane < slots && before == n));
}

template <int RT, bool DROP, bool DX, int NW>
__global__ void __launch_bounds__(64 * NW, RT == 1 ? 3 : 2) k_batch_grads(BatchGradArgs g) {
  using Sh = GradShape<RT, NW>;
  __shared__ __attribute__((aligned(16))) char smem[Sh::SMEM];
  __shared__ __attribute__((aligned(16))) uint16_t as[DX ? kGradSlice * Sh::AW : 8];
  const int slot = (int)blockIdx.y < g.slots ? slot_by_size(g.start, g.slots, blockIdx.y) : g.slots;
  if ((int)blockIdx.x < g.a.slices)
    grads_block<RT, DROP, DX, NW, 1>(g, g.a, blockIdx.x, slot, smem, as);
  else if (slot < g.slots)   // the last row is dX's alone
    grads_block<RT, false, false, NW, grad_blocks_b<RT>()>(g, g.b, (int)blockIdx.x - g.a.slices,
                                                           slot, smem, as);
}

// ------------------------------- launchers ---------------------------------

static inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Tiles that a batch may be expected to have (the host does not know the slots
// in use): its tokens' own, and one more per slot it may hold.  A batch of few
// tokens may be one of single tokens and hold as many adapters; one of many
// holds prompts, and fewer of them.
static int64_t expected_tiles(int64_t M, int S) {
  int64_t more = 32 + M / 32;
  if (more > M) more = M;
  if (more > S) more = S;
  return M / kPlanTile + more;
}

// Steps per slice of the down projections' contraction: slices that give about
// two workgroups per CU, at most kMaxSlices (their sums are read back), and a
// power of two: the slice is the fast grid index, so that an XCD then always
// meets the same slices and reads only their part of the adapters (T, 4096
// tokens, 4096 columns, rank 64: seven slices 33 us, four 12.9).  Four workgroups
// per CU for U of more than 32 ranks, whose waves wait for each other at every
// step (11008 columns, rank 64: 39.9 against 35.1 us; T, whose waves do not:
// 12.9 against 16.4).
constexpr int kMaxSlices = 16;
static int down_zlen(int64_t M, int S, int64_t C, bool pairs) {
  const int64_t steps = (C + 63) / 64;
  const int64_t want = (pairs ? 4 : 2) * kCUs / expected_tiles(M, S);
  int64_t z = 1;
  while (2 * z <= want && 2 * z <= kMaxSlices && 2 * z * kDownWaves <= steps) z *= 2;
  return (int)((steps + z - 1) / z);
}
static int down_slices(int64_t M, int S, int64_t C, bool pairs) {
  const int64_t steps = (C + 63) / 64;
  const int zl = down_zlen(M, S, C, pairs);
  return (int)((steps + zl - 1) / zl);
}
static int slices_T(int64_t M, int S, int64_t K) { return down_slices(M, S, K, false); }
static int slices_U(int64_t M, int S, int64_t N, int r) { return down_slices(M, S, N, r > 32); }

// Rank tiles of 16 in a workgroup of the gradients' kernel and its packing.
static int grad_tiles(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : 4; }

BatchWorkspace batch_workspace(int64_t M, int64_t K, int64_t N, int r, int S, bool backward) {
  BatchWorkspace w{};
  size_t off = 0;
  w.off_T = off; off += align256((size_t)slices_T(M, S, K) * M * r * 4);
  if (backward) {
    // packed operands: 1 KB per chunk, term (or token group) and rank tile
    const size_t chunks = (size_t)pack_chunks(M, S) * ((r + kGradRanks - 1) / kGradRanks);
    const size_t cols = chunks * 3 * grad_tiles(r) * 1024, rows = chunks * 2 * grad_tiles(r) * 1024;
    w.off_U = off; off += align256((size_t)slices_U(M, S, N, r) * M * r * 4);
    w.off_Uc = off; off += cols;
    w.off_Tc = off; off += cols;
    w.off_Ur = off; off += rows;
  }
  w.bytes = off;
  return w;
}

template <bool WT, bool DROP>
static hipError_t down(DownArgs g, hipStream_t st) {
  const bool pairs = WT && g.r > 32;
  g.zlen = down_zlen(g.M, g.slots, g.C, pairs);
  const dim3 grid((unsigned)down_slices(g.M, g.slots, g.C, pairs),
                  (unsigned)adapter_plan_tiles(g.M, g.slots), (unsigned)((g.r + 63) / 64));
  const dim3 block(64 * kDownWaves);
  if (g.r <= 16) hipLaunchKernelGGL((k_batch_down<WT, DROP, 1>), grid, block, 0, st, g);
  else if (g.r <= 32) hipLaunchKernelGGL((k_batch_down<WT, DROP, 2>), grid, block, 0, st, g);
  else hipLaunchKernelGGL((k_batch_down<WT, DROP, 4>), grid, block, 0, st, g);
  return hipGetLastError();
}

template <bool WT, bool DROP>
static hipError_t up(const UpArgs& g, hipStream_t st) {
  // Workgroups per tile: about four per CU in all, two where most tiles are
  // narrow (a narrow tile takes two blocks at a time; 16 single tokens, 28672
  // columns: 7.8 against 11.0 us; 2048 tokens, 4096 columns: 11.0 against 10.2),
  // cut to a whole multiple of the XCDs where there are that many, so that an XCD
  // meets the same part of W in every tile (calls, with and without the cut: 4096
  // tokens, 11008 columns, rank 64: 57 and 65 us).  It undoes equal shares: 15
  // blocks go to eight workgroups, two to seven of them and one to the last,
  // which costs at rank 16, where W is small (2048 tokens: 1664 columns 14.2 and
  // 13.5, 1920 14.0 and 13.8, 11008 25.5 and 24.2, multiples of 1024 level; 256
  // single tokens, 11008 columns: 15.0 and 14.0).  Narrow tiles' rounds of two
  // blocks may differ by one between workgroups too (28672 columns, 16 tiles:
  // three or four).
  const int64_t blocks = (g.cols + kUpCols - 1) / kUpCols;
  const int64_t tiles = expected_tiles(g.M, g.slots);
  int64_t gx = (g.M <= 16 * tiles ? 2 : 4) * kCUs / tiles;
  if (gx < 1) gx = 1;
  if (gx > blocks) gx = blocks;
  const int64_t per = (blocks + gx - 1) / gx;   // no workgroup without its share of blocks
  gx = (blocks + per - 1) / per;
  if (gx >= kXCDs) gx -= gx % kXCDs;
  const dim3 grid((unsigned)gx, (unsigned)adapter_plan_tiles(g.M, g.slots));
  const dim3 block(64 * kUpWaves);
  if constexpr (WT) {
    hipLaunchKernelGGL((k_batch_up<WT, DROP, 64, 4>), grid, block, 0, st, g);
  } else {
    if (g.r <= 16) hipLaunchKernelGGL((k_batch_up<WT, DROP, 16, 1>), grid, block, 0, st, g);
    else if (g.r <= 32) hipLaunchKernelGGL((k_batch_up<WT, DROP, 32, 1>), grid, block, 0, st, g);
    else if (g.r <= 64) hipLaunchKernelGGL((k_batch_up<WT, DROP, 64, 1>), grid, block, 0, st, g);
    else hipLaunchKernelGGL((k_batch_up<WT, DROP, 64, 4>), grid, block, 0, st, g);
  }
  return hipGetLastError();
}

#define QLK_TRY(x) do { hipError_t e_ = (x); if (e_ != hipSuccess) return e_; } while (0)

// The slices of T = drop(X) A^T.
static hipError_t batch_T(const uint16_t* X, const BatchAdapters& a, int64_t M, int64_t K,
                          const BatchDropout& d, float* part, hipStream_t st) {
  DownArgs g{};
  g.S = X; g.M = (int)M; g.C = K; g.W = a.A; g.r = a.r; g.slots = a.slots;
  g.order = a.order; g.tiles = a.tiles; g.part = part;
  g.drop = DropKey{d.threshold, d.k0, d.k1}; g.keep_scale = d.scale;
  return d.on ? down<false, true>(g, st) : down<false, false>(g, st);
}

hipError_t launch_batch_fwd(const uint16_t* X, int64_t M, int64_t K, int64_t N,
                            const BatchAdapters& a, const uint16_t* Y, const BatchDropout& d,
                            uint16_t* out, float* T_out, void* ws, hipStream_t st) {
  const BatchWorkspace w = batch_workspace(M, K, N, a.r, a.slots, false);
  float* const part = reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + w.off_T);
  QLK_TRY(batch_T(X, a, M, K, d, part, st));
  UpArgs u{};
  u.base = Y; u.out = out; u.M = (int)M; u.cols = N; u.part = part;
  u.slices = slices_T(M, a.slots, K); u.t_out = T_out; u.W = a.B; u.scale = a.scale;
  u.r = a.r; u.slots = a.slots; u.order = a.order; u.tiles = a.tiles;
  return up<false, false>(u, st);
}

template <int RT, bool DROP, bool DX>
static void grads(const BatchGradArgs& g, hipStream_t st) {
  const dim3 grid((unsigned)(g.a.slices + g.b.slices), (unsigned)(g.slots + (DX ? 1 : 0)),
                  (unsigned)((g.r + kGradRanks - 1) / kGradRanks));
  // Eight waves per workgroup; four where the sums of 64 ranks, added through
  // the LDS, would fill it.
  constexpr int NW = RT == 4 ? 4 : 8;
  hipLaunchKernelGGL((k_batch_grads<RT, DROP, DX, NW>), grid, dim3(64 * NW), 0, st, g);
}
template <bool DROP, bool DX>
static void grads_rt(const BatchGradArgs& g, hipStream_t st) {
  if (g.r <= 16) grads<1, DROP, DX>(g, st);
  else if (g.r <= 32) grads<2, DROP, DX>(g, st);
  else grads<4, DROP, DX>(g, st);
}

hipError_t launch_batch_bwd(const uint16_t* dY, const uint16_t* X, int64_t M, int64_t K, int64_t N,
                            const BatchAdapters& a, const float* T, const uint16_t* dX0,
                            const BatchDropout& d, uint16_t* dX, float* dA, float* dB, void* ws,
                            hipStream_t st) {
  const BatchWorkspace w = batch_workspace(M, K, N, a.r, a.slots, true);
  char* const base = reinterpret_cast<char*>(ws);
  float* const U = reinterpret_cast<float*>(base + w.off_U);
  uint16_t* const Uc = reinterpret_cast<uint16_t*>(base + w.off_Uc);
  uint16_t* const Tc = reinterpret_cast<uint16_t*>(base + w.off_Tc);
  uint16_t* const Ur = reinterpret_cast<uint16_t*>(base + w.off_Ur);
  // Beyond 64 ranks a workgroup of the gradients' kernel sees only a part of
  // them: dX has its own launch there.
  const bool fused = dX != nullptr && a.r <= kGradRanks;
  PackArgs pk{};
  pk.u = PackJob{U, slices_U(M, a.slots, N, a.r), Uc, fused ? Ur : nullptr};
  pk.t = PackJob{T, 1, Tc, nullptr};
  pk.M = (int)M; pk.r = a.r; pk.slots = a.slots; pk.order = a.order; pk.start = a.start;
  pk.tiles = a.tiles; pk.chunks = pack_chunks(M, a.slots);
  if (!T) {
    float* const part = reinterpret_cast<float*>(base + w.off_T);
    QLK_TRY(batch_T(X, a, M, K, d, part, st));
    pk.t.part = part;
    pk.t.slices = slices_T(M, a.slots, K);
  }
  DownArgs g{};
  g.S = dY; g.M = (int)M; g.C = N; g.W = a.B; g.r = a.r; g.slots = a.slots;
  g.order = a.order; g.tiles = a.tiles; g.part = U;
  QLK_TRY((down<true, false>(g, st)));
  const dim3 pgrid(2 * (unsigned)adapter_plan_tiles(M, a.slots), 2,
                   (unsigned)((a.r + kGradRanks - 1) / kGradRanks));
  switch (grad_tiles(a.r)) {
    case 1: hipLaunchKernelGGL(k_batch_pack<1>, pgrid, dim3(256), 0, st, pk); break;
    case 2: hipLaunchKernelGGL(k_batch_pack<2>, pgrid, dim3(256), 0, st, pk); break;
    default: hipLaunchKernelGGL(k_batch_pack<4>, pgrid, dim3(256), 0, st, pk); break;
  }
  QLK_TRY(hipGetLastError());
  const DropKey key{d.threshold, d.k0, d.k1};
  if (dX && !fused) {
    UpArgs u{};
    u.base = dX0; u.out = dX; u.M = (int)M; u.cols = K; u.part = U; u.slices = pk.u.slices;
    u.t_out = nullptr; u.W = a.A; u.scale = a.scale;
    u.r = a.r; u.slots = a.slots; u.order = a.order; u.tiles = a.tiles;
    u.drop = key; u.keep_scale = d.scale;
    QLK_TRY((d.on ? up<true, true>(u, st) : up<true, false>(u, st)));
  }
  auto slices = [](int64_t cols, int64_t wide) { return (int)((cols + wide - 1) / wide); };
  const int blocks_b = a.r > 32 ? grad_blocks_b<4>() : grad_blocks_b<1>();
  BatchGradArgs ga{};
  ga.a = BatchGradJob{X, K, Uc, dA, 1, slices(K, kGradSlice)};
  ga.b = BatchGradJob{dY, N, Tc, dB, 0, slices(N, kGradSlice * blocks_b)};
  ga.Urows = Ur; ga.chunks = pk.chunks;
  ga.M = (int)M; ga.r = a.r; ga.slots = a.slots; ga.scale = a.scale; ga.order = a.order;
  ga.start = a.start; ga.A = a.A; ga.dX0 = dX0; ga.dX = dX; ga.drop = key; ga.keep_scale = d.scale;
  if (d.on) {
    if (fused) grads_rt<true, true>(ga, st);
    else grads_rt<true, false>(ga, st);
  } else {
    if (fused) grads_rt<false, true>(ga, st);
    else grads_rt<false, false>(ga, st);
  }
  return hipGetLastError();
}

}  // namespace qlk
