// dA and dB from 8-bit rows: the workgroup that k_int8_grads and the tiles of dX for
// few tokens share.
#pragma once

#include "device_common.h"

namespace qlk {

constexpr int kChunk = 32;       // tokens of an MFMA step of the gradients

// O[c][j] = s sum_m P[m][c] Q[m][j] for (P, Q) = (Cx, terms of sx U): dA^T, and
// (dY, terms of T): dB, in one launch that reads P once.  A workgroup owns 32
// or 64 columns of P and up to 64 ranks and contracts over all tokens itself; its four
// waves take every fourth 32-token chunk.  P goes through a slab of LDS per wave
// (codes as bf16) and comes back transposed as the MFMA operand (v_mfma_f32_16x16x32_bf16);
// Q is loaded as the operands that it is stored as, 1 KB in a row each.  Each
// term takes an MFMA on the same P operand, the small terms first.  The waves'
// sums are added through LDS in a fixed order.
constexpr int kGradWaves8 = 4;

struct Grad8Job {
  const void* P;         // [M, ld] codes or bf16
  int64_t ld;            // its columns (a multiple of 8; of 16 for codes)
  const uint16_t* Q;     // packed terms
  float* out;            // trans: [r, ld], else [ld, r]
  int slices;            // workgroups: ceil(ld / columns of one)
};

// CB: bands of 32 columns.  With 64 ranks a workgroup reads 12 KB of Q a chunk, six
// times a band's P: two bands halve that (4001 tokens, 11008 and 4096 columns: 58 us
// with one).
template <int RT>
constexpr int grad_bands() { return RT == 4 ? 2 : 1; }

template <bool S8, int RT>
__device__ __forceinline__ void grads8(const Grad8Job& g, int lb, int M, int r, int t0, float s,
                                       uint8_t* lds) {
  constexpr int CB = grad_bands<RT>(), CW = 32 * CB;      // columns
  constexpr int PL = (S8 ? 1 : 2) * CB;                   // 1 KB loads of P a chunk
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i = lane & 15, q4 = lane >> 4;
  const int full = (g.slices / kXCDs) * kXCDs;
  const int sl = lb < full ? (lb % kXCDs) * (full / kXCDs) + lb / kXCDs : lb;
  const int64_t c0 = (int64_t)sl * CW;
  const int ntiles = (r + 15) / 16;
  const uint32_t pbytes = (uint32_t)((int64_t)M * g.ld * (S8 ? 1 : 2));
  uint16_t* const my = reinterpret_cast<uint16_t*>(lds) + wave * kChunk * CW;
  const int nchunks = (M + kChunk - 1) / kChunk;
  const int cut = M % kChunk ? nchunks - 1 : -1;          // the chunk that M ends in
  // load n: piece 64 n + lane of the chunk's rows of PP pieces of 16 bytes
  constexpr int PP = CW * (S8 ? 1 : 2) / 16;
  uint32_t poff[PL], pcut[PL];
#pragma unroll
  for (int n = 0; n < PL; ++n) {
    const int m = (64 * n + lane) / PP;
    const int64_t col = c0 + (64 * n + lane) % PP * (S8 ? 16 : 8);
    poff[n] = col < g.ld ? (uint32_t)((m * g.ld + col) * (S8 ? 1 : 2)) : kOOB;
    pcut[n] = (nchunks - 1) * kChunk + m < M ? poff[n] : kOOB;
  }

  f32x4_t acc[2 * CB][RT];
#pragma unroll
  for (int h = 0; h < 2 * CB; ++h)
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[h][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  struct Chunk { uint4 p[PL]; uint4 q[3][RT]; };
  auto load = [&](Chunk& L, int ch) {
    const bool cv = ch < nchunks, end = ch == cut;
    const __amdgpu_buffer_rsrc_t rp = rsrc_whole(g.P, cv ? pbytes : 0);
    // a chunk's terms: the resource's base moves, 64 bits wide
    const int64_t qchunk = (int64_t)ntiles * 3 * 1024;
    const __amdgpu_buffer_rsrc_t rq =
        rsrc_whole(reinterpret_cast<const char*>(g.Q) + (cv ? ch * qchunk : 0), cv ? (uint32_t)qchunk : 0);
    const uint32_t soff = (uint32_t)ch * (uint32_t)(kChunk * g.ld * (S8 ? 1 : 2));
#pragma unroll
    for (int n = 0; n < PL; ++n) L.p[n] = bload128s(rp, end ? pcut[n] : poff[n], cv ? soff : 0);
#pragma unroll
    for (int z = 0; z < 3; ++z)
#pragma unroll
      for (int t = 0; t < RT; ++t)   // a rank tile past the last one repeats it (and is not stored)
        L.q[z][t] = bload128s(rq, 16 * lane, (uint32_t)(((z * ntiles) + min(t0 + t, ntiles - 1)) * 1024));
  };
  auto use = [&](const Chunk& L) {
    // A wave's LDS operations run in issue order: these stores land after the
    // previous chunk's reads and before this one's.
#pragma unroll
    for (int n = 0; n < PL; ++n) {
      const int m = (64 * n + lane) / PP, p = (64 * n + lane) % PP;
      uint4* const d = reinterpret_cast<uint4*>(my + m * CW + p * (S8 ? 16 : 8));
      if constexpr (S8) {
        uint4 o[2];
        codes_to_bf16(L.p[n], o);
        d[0] = o[0];
        d[1] = o[1];
      } else {
        d[0] = L.p[n];
      }
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
    typedef short v8s_t __attribute__((ext_vector_type(8)));
    // source lane 4 s + u of a 16-lane group points at row 8 q4 + 4 e + s, column
    // 4 u of a 16-column band: lane i receives column i of the band's four rows
    const int rr = 8 * q4 + (i >> 2), cc = 4 * (i & 3);
    bf16x8_t aop[2 * CB];
#pragma unroll
    for (int h = 0; h < 2 * CB; ++h) {
      const v4s_t lo = lds_read_tr16(my + rr * CW + 16 * h + cc);
      const v4s_t hi = lds_read_tr16(my + (rr + 4) * CW + 16 * h + cc);
      const v8s_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      aop[h] = __builtin_bit_cast(bf16x8_t, v);
    }
#pragma unroll
    for (int z = 2; z >= 0; --z)
#pragma unroll
      for (int h = 0; h < 2 * CB; ++h)
#pragma unroll
        for (int t = 0; t < RT; ++t)
          acc[h][t] = mfma_16x16x32(aop[h], __builtin_bit_cast(bf16x8_t, L.q[z][t]), acc[h][t]);
  };
  Chunk a, b;
  load(a, wave);
  for (int ch = wave; ch < nchunks; ch += 2 * kGradWaves8) {
    load(b, ch + kGradWaves8);
    __builtin_amdgcn_sched_barrier(0);
    use(a);
    load(a, ch + 2 * kGradWaves8);
    __builtin_amdgcn_sched_barrier(0);
    use(b);
  }
  // acc[h][t][v] = O[c0 + 16 h + 4 q4 + v][16 (t0 + t) + i]; the sums take the
  // slabs' place once every wave is done with them
  f32x4_t* const red = reinterpret_cast<f32x4_t*>(lds);
  __syncthreads();
  if (wave > 0)
#pragma unroll
    for (int h = 0; h < 2 * CB; ++h)
#pragma unroll
      for (int t = 0; t < RT; ++t) red[((wave - 1) * 2 * CB * RT + h * RT + t) * 64 + lane] = acc[h][t];
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int h = 0; h < 2 * CB; ++h)
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      f32x4_t v = acc[h][t];
#pragma unroll
      for (int w = 0; w < kGradWaves8 - 1; ++w) v += red[(w * 2 * CB * RT + h * RT + t) * 64 + lane];
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

struct Grad8Args {
  Grad8Job ja, jb;       // dA, dB
  int M, r;
  float s;
};
// Workgroups, their LDS bytes, and one of them: slices of dA, then of dB, for every
// 16 RT ranks.
template <int RT>
inline unsigned grads8_blocks(Grad8Args& g) {
  constexpr int CW = 32 * grad_bands<RT>();
  g.ja.slices = (int)((g.ja.ld + CW - 1) / CW);
  g.jb.slices = (int)((g.jb.ld + CW - 1) / CW);
  return (unsigned)(g.ja.slices + g.jb.slices) * (unsigned)((g.r + 16 * RT - 1) / (16 * RT));
}
template <int RT>
constexpr int grads8_lds() {
  constexpr int CB = grad_bands<RT>();
  constexpr int SLABS = kGradWaves8 * kChunk * 32 * CB * 2, RED = (kGradWaves8 - 1) * 2 * CB * RT * 1024;
  return SLABS > RED ? SLABS : RED;
}
template <int RT>
__device__ __forceinline__ void grads8_block(const Grad8Args& g, int blk, uint8_t* lds) {
  const int all = g.ja.slices + g.jb.slices, t0 = blk / all * RT;
  blk %= all;
  if (blk < g.ja.slices) grads8<true, RT>(g.ja, blk, g.M, g.r, t0, g.s, lds);
  else grads8<false, RT>(g.jb, blk - g.ja.slices, g.M, g.r, t0, g.s, lds);
}

}  // namespace qlk
