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

namespace qlk {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kPlanClasses = kMaxSlots + 1;

__device__ __forceinline__ int wave_incl_scan(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Exclusive scan over the workgroup's threads; *total gets the sum.  `part`
// holds one value per wave; the caller's next use of it is behind a barrier.
__device__ __forceinline__ int block_excl_scan(int v, int tid, int* part, int* total) {
  const int lane = tid & 63, wave = tid >> 6;
  const int inc = wave_incl_scan(v, lane);
  if (lane == 63) part[wave] = inc;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kPlanWaves; ++w) {
    const int x = part[w];
    if (w < wave) before += x;
    all += x;
  }
  __syncthreads();
  *total = all;
  return before + inc - v;
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

__global__ void __launch_bounds__(kPlanThreads) k_adapter_plan(PlanArgs g) {
  __shared__ int tot[kPlanClasses + 1], base[kPlanClasses + 1], tbase[kPlanClasses + 1];
  __shared__ int carry[kPlanClasses];
  __shared__ int wcnt[kPlanWaves][kPlanClasses];
  __shared__ int c_start[kPlanThreads], c_dest[kPlanThreads], c_slot[kPlanThreads];
  __shared__ int part[kPlanWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int C = g.S + 1;
  // Lengths are clamped to what the M rows hold: a request's tokens are
  // [min(M, sum before), min(M, sum before + length)).  Sums saturate at M
  // (saturating addition of non-negative numbers is associative), so no sum
  // leaves 32 bits.
  auto request = [&](int q, int& len, int& cls) {
    len = 0;
    cls = g.S;
    if (q < g.Q) {
      len = g.lengths ? min(max(g.lengths[q], 0), g.M) : 1;
      const int s = g.slots[q];
      if (s >= 0 && s < g.S) cls = s;
    }
  };
  // Inclusive saturating scan of the chunk's lengths behind `done`.
  auto ends = [&](int len, int done) {
    int v = len;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(v, d);
      if (lane >= d) v = min(g.M, v + o);
    }
    if (lane == 63) part[wave] = v;
    __syncthreads();
    int before = done;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w)
      if (w < wave) before = min(g.M, before + part[w]);
    __syncthreads();
    return min(g.M, before + v);
  };

  for (int c = tid; c < C; c += kPlanThreads) tot[c] = 0, carry[c] = 0;
  __syncthreads();
  // 1. Tokens of each class (integer sums: any order gives the same).
  int done = 0;
  for (int q0 = 0; q0 < g.Q; q0 += kPlanThreads) {
    int len, cls;
    request(q0 + tid, len, cls);
    const int end = ends(len, done);
    const int prev = __shfl_up(end, 1);
    if (lane == 63) part[wave] = end;
    __syncthreads();
    const int beg = lane ? prev : (wave ? part[wave - 1] : done);
    if (end > beg) atomicAdd(&tot[cls], end - beg);
    const int last = part[kPlanWaves - 1];
    __syncthreads();
    done = last;
  }
  const int tokens = done;   // rows behind the last request have no adapter
  if (tid == 0) tot[g.S] += g.M - tokens;
  __syncthreads();
  // 2. Starts of the classes and of their tiles.
  {
    int all, tall;
    const int n = tid < g.S ? tot[tid] : 0;
    const int b = block_excl_scan(n, tid, part, &all);
    const int tb = block_excl_scan((n + kPlanTile - 1) / kPlanTile, tid, part, &tall);
    if (tid < g.S) base[tid] = b, tbase[tid] = tb;
    if (tid == 0) base[g.S] = all, tbase[g.S] = tall;
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int c = tid; c < C; c += kPlanThreads) g.start[c] = base[c];
    if (tid == 0) g.start[C] = g.M;
  }
  for (int i = blockIdx.x * kPlanThreads + tid; i < g.tiles; i += gridDim.x * kPlanThreads) {
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
  for (int q0 = 0; q0 < g.Q; q0 += kPlanThreads) {
    int len, cls;
    request(q0 + tid, len, cls);
    const int end = ends(len, done);
    const int prev = __shfl_up(end, 1);
    if (lane == 63) part[wave] = end;
    for (int c = lane; c < C; c += 64) wcnt[wave][c] = 0;
    __syncthreads();
    const int beg = lane ? prev : (wave ? part[wave - 1] : done);
    const int chunk_end = part[kPlanWaves - 1];
    len = end - beg;
    // Tokens of this class in earlier lanes of the wave, class by class.
    int before = 0;
    uint64_t left = __ballot(len > 0);
    const bool single = __ballot(len > 1) == 0;
    while (left) {
      const int c = __builtin_amdgcn_readlane(cls, __builtin_ctzll(left));
      const bool mine = cls == c && len > 0;
      const uint64_t m = __ballot(mine);
      if (single) {
        if (mine) before = __builtin_popcountll(m & ((1ull << lane) - 1));
        if (lane == 0) wcnt[wave][c] = __builtin_popcountll(m);
      } else {
        const int inc = wave_incl_scan(mine ? len : 0, lane);
        if (mine) before = inc - len;
        if (lane == 63) wcnt[wave][c] = inc;
      }
      left &= ~m;
    }
    __syncthreads();
    for (int c = tid; c < C; c += kPlanThreads) {
      int run = carry[c];
#pragma unroll
      for (int w = 0; w < kPlanWaves; ++w) {
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
    for (int t = max(t0, done) + tid; t < min(t1, chunk_end); t += kPlanThreads) {
      int lo = 0, hi = min(kPlanThreads, g.Q - q0) - 1;   // the last request with start <= t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (c_start[mid] <= t) lo = mid;
        else hi = mid - 1;
      }
      g.token_slot[t] = c_slot[lo];
      g.order[c_dest[lo] + t - c_start[lo]] = t;
    }
    __syncthreads();
    done = chunk_end;
  }
  const int none = base[g.S] + carry[g.S];
  for (int t = max(t0, tokens) + tid; t < t1; t += kPlanThreads) {
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
  // One workgroup per 4096 tokens: each repeats the request-level part.
  int64_t blocks = (M + 4095) / 4096;
  if (blocks > kCUs) blocks = kCUs;
  hipLaunchKernelGGL(k_adapter_plan, dim3((unsigned)blocks), dim3(kPlanThreads), 0, st, g);
  return hipGetLastError();
}

}  // namespace qlk
