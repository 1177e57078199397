// The token plan of a batch whose requests use different adapters (slots)
// beside one shared projection.  From the requests' lengths and slots it
// builds, in one launch:
//
//   token_slot [M]     the slot of every token, -1 without an adapter
//   order [M]          the tokens ordered by slot, within a slot in their own
//                      order; tokens without an adapter last (class S)
//   start [S + 2]      where each class starts in `order`; the last is M
//   tiles [tiles][3]   (slot, first, count): runs of up to 64 positions of
//                      `order` of one class, class after class; unused rows
//                      (-1, 0, 0)
//
// It is a stable counting sort of the REQUESTS (a request's tokens are
// consecutive and share its slot), after which the tokens are written by
// position.  Every workgroup does the whole request-level part -- it is short
// and a second launch or a grid barrier would cost more -- and writes its
// share of the tokens and tiles, so nothing passes between workgroups and no
// result depends on their order.  Bound by latency: a few LDS round trips per
// 1024 requests.
#include "device_common.h"
#include "kernels.h"
#include "plan_sum.h"

namespace qlk {

constexpr int kPlanClasses = kMaxSlots + 1;

__device__ __forceinline__ int wave_incl_scan(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

struct PlanArgs {
  const int* lengths;   // null: every request has one token
  const int* slots;
  int Q, M, S, tiles;
  int* token_slot;
  int* order;
  int* start;
  int* tile;
};

// NT threads take NT requests at a time (a chunk).
template <int NT>
__global__ void __launch_bounds__(NT) k_adapter_plan(PlanArgs g) {
  constexpr int NW = NT / 64;
  __shared__ int tot[kPlanClasses], base[kPlanClasses], tbase[kPlanClasses], carry[kPlanClasses];
  __shared__ int wcnt[NW][kPlanClasses];
  __shared__ int c_start[NT], c_dest[NT], c_slot[NT];
  __shared__ int part[NW], part2[2][NW];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int C = g.S + 1;
  const int bits = 32 - __builtin_clz(g.S);   // of a class, 0 .. S

  // One chunk's requests: this thread's class, its first token and number of
  // tokens; returns the chunk's end.  Lengths are clamped to what the M rows
  // hold: a request's tokens are [min(M, sum before), min(M, sum before +
  // length)).  Every sum is cut at M before it is formed (plan_sum.h): two
  // requests can hold 2^31 tokens.
  int len = 0, cls = 0, beg = 0;
  auto scan_chunk = [&](int q0, int done) {
    int n = 0;
    cls = g.S;
    if (q0 + tid < g.Q) {
      n = g.lengths ? min(max(g.lengths[q0 + tid], 0), g.M) : 1;
      const int s = g.slots[q0 + tid];
      if (s >= 0 && s < g.S) cls = s;
    }
    int v = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(v, d);
      if (lane >= d) v = cut_sum(v, o, g.M);
    }
    if (lane == 63) part[wave] = v;
    __syncthreads();
    int before = done, all = done;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (w == wave) before = all;
      all = cut_sum(all, part[w], g.M);
    }
    const int prev = __shfl_up(v, 1);
    beg = lane ? cut_sum(before, prev, g.M) : before;
    len = cut_sum(before, v, g.M) - beg;
    __syncthreads();   // part is free again
    return all;
  };

  for (int c = tid; c < C; c += NT) tot[c] = 0, carry[c] = 0;
  for (int c = lane; c < C; c += 64) wcnt[wave][c] = 0;
  // 1. Tokens of each class (integer sums: any order gives the same).
  int done = 0;
  for (int q0 = 0; q0 < g.Q; q0 += NT) {
    done = scan_chunk(q0, done);             // its barrier also covers tot
    if (len > 0) atomicAdd(&tot[cls], len);
  }
  const int tokens = done;   // rows behind the last request have no adapter
  __syncthreads();
  // 2. Starts of the classes and of their tiles; a thread takes `per`
  // neighbouring slots, the class without an adapter comes last.
  {
    const int per = (g.S + NT - 1) / NT, c0 = tid * per, c1 = min(g.S, c0 + per);
    int n = 0, t = 0;
    for (int c = c0; c < c1; ++c) n += tot[c], t += (tot[c] + kPlanTile - 1) / kPlanTile;
    const int in = wave_incl_scan(n, lane), it = wave_incl_scan(t, lane);
    if (lane == 63) part2[0][wave] = in, part2[1][wave] = it;
    __syncthreads();
    int bn = in - n, bt = it - t, an = 0, at = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (w < wave) bn += part2[0][w], bt += part2[1][w];
      an += part2[0][w], at += part2[1][w];
    }
    for (int c = c0; c < c1; ++c) {
      base[c] = bn, tbase[c] = bt;
      if (blockIdx.x == 0) g.start[c] = bn;
      bn += tot[c], bt += (tot[c] + kPlanTile - 1) / kPlanTile;
    }
    if (tid == 0) {
      base[g.S] = an, tbase[g.S] = at;
      tot[g.S] += g.M - tokens;
      if (blockIdx.x == 0) g.start[g.S] = an, g.start[C] = g.M;
    }
  }
  __syncthreads();
  for (int i = blockIdx.x * NT + tid; i < g.tiles; i += gridDim.x * NT) {
    int lo = 0, hi = g.S;                // the last class with tbase <= i
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tbase[mid] <= i) lo = mid;
      else hi = mid - 1;
    }
    const int off = (i - tbase[lo]) * kPlanTile;
    const bool real = off < tot[lo];
    g.tile[3 * i] = real && lo < g.S ? lo : -1;
    g.tile[3 * i + 1] = real ? base[lo] + off : 0;
    g.tile[3 * i + 2] = real ? min(kPlanTile, tot[lo] - off) : 0;
  }
  // 3. Place the requests, chunk by chunk, and write this workgroup's tokens.
  const int share = (g.M + gridDim.x - 1) / gridDim.x;
  const int t0 = min(g.M, (int)blockIdx.x * share), t1 = min(g.M, t0 + share);
  done = 0;
  for (int q0 = 0; q0 < g.Q; q0 += NT) {
    int end = tokens;
    if (g.Q > NT) {   // one chunk is still in the registers
      if (q0)
        for (int c = lane; c < C; c += 64) wcnt[wave][c] = 0;
      end = scan_chunk(q0, done);
    }
    // The wave's requests of this class, from a ballot per bit of the class;
    // then the class's tokens in earlier lanes, and the class's sum by its
    // first lane.
    uint64_t same = __ballot(len > 0);
    if (len <= 0) same = 0;
    for (int b = 0; b < bits; ++b) {
      const uint64_t ones = __ballot((cls >> b) & 1);
      same &= (cls >> b) & 1 ? ones : ~ones;
    }
    int before = 0, sum = 0;
    if (__ballot(len > 1) == 0) {
      before = __builtin_popcountll(same & ((1ull << lane) - 1));
      sum = __builtin_popcountll(same);
    } else {
#pragma unroll
      for (int j = 0; j < 64; ++j) {
        const int n = __builtin_amdgcn_readlane(len, j);
        const int mine = (int)(same >> j) & 1 ? n : 0;
        if (j < lane) before += mine;
        sum += mine;
      }
    }
    if (len > 0 && (same & ((1ull << lane) - 1)) == 0) wcnt[wave][cls] = sum;
    __syncthreads();
    for (int c = tid; c < C; c += NT) {
      int run = carry[c];
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const int n = wcnt[w][c];
        wcnt[w][c] = run;
        run += n;
      }
      carry[c] = run;
    }
    __syncthreads();
    c_start[tid] = beg;
    c_dest[tid] = len > 0 ? base[cls] + wcnt[wave][cls] + before : 0;
    c_slot[tid] = cls < g.S ? cls : -1;
    __syncthreads();
    for (int t = max(t0, done) + tid; t < min(t1, end); t += NT) {
      int lo = 0, hi = min(NT, g.Q - q0) - 1;   // the last request with start <= t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (c_start[mid] <= t) lo = mid;
        else hi = mid - 1;
      }
      g.token_slot[t] = c_slot[lo];
      g.order[c_dest[lo] + t - c_start[lo]] = t;
    }
    __syncthreads();
    done = end;
  }
  const int none = base[g.S] + carry[g.S];
  for (int t = max(t0, tokens) + tid; t < t1; t += NT) {
    g.token_slot[t] = -1;
    g.order[none + t - tokens] = t;
  }
}

int64_t adapter_plan_tiles(int64_t M, int S) {
  return M / kPlanTile + (M < S + 1 ? M : S + 1);
}

hipError_t launch_adapter_plan(const int* lengths, const int* slots, int64_t Q, int64_t M, int S,
                               int* token_slot, int* order, int* start, int* tiles, hipStream_t st) {
  PlanArgs g{lengths, slots, (int)Q, (int)M, S, (int)adapter_plan_tiles(M, S),
             token_slot, order, start, tiles};
  // One workgroup per 1024 tokens: each repeats the request-level part (53
  // requests, 16384 tokens: 7.6 us; per 4096 tokens 12.7).
  int64_t blocks = (M + 1023) / 1024;
  if (blocks > kCUs) blocks = kCUs;
  const dim3 grid((unsigned)blocks);
  if (Q <= 256) hipLaunchKernelGGL((k_adapter_plan<256>), grid, dim3(256), 0, st, g);
  else hipLaunchKernelGGL((k_adapter_plan<1024>), grid, dim3(1024), 0, st, g);
  return hipGetLastError();
}

}  // namespace qlk
