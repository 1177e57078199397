// Storage in 8 bits: rows of a matrix, or runs of 64 columns of a row, as codes
// and one fp32 scale each.
//
//   a = max |x|,   scale = fp32(a / 127),   code = rne(127 x / a)
//
// A row (run) of zeros has scale 0 and codes 0; one that holds an infinity or a
// NaN has scale NaN and codes 0, so that every value it stands for is NaN.
//
// The quotient: R = 127 / a held as two fp32 words, R_hi near it and R_lo the rest
// (within 2^-44 of R together), n = fma(x, R_hi, x R_lo) is 127 x / a rounded once.
// For bf16 x this gives the exact code: a tie 127 x / a = k + 1/2 is a
// representable number and therefore hit, and what is no tie is at least 2^-9
// of |n| / 254 away from one, since 254 x and (2 k + 1) a are whole multiples
// of x's last place.  Adding 1.5 2^23 rounds n to the nearest integer, ties to
// the even one, and leaves the code in the sum's low byte.  Where a lies outside
// [2^-100, 2^100], x and a are scaled by a power of two first.
//
// The gated activation H = silu(G) U in rows of 8 bits, with G and U kept in
// runs of 64 for the backward, and that backward, read and write these formats
// in one pass.
//
// Bound: HBM.  A row is read once and held in registers (up to 8 pieces of 8
// values per lane) between its maximum and its codes.  Measured (launches in a kernel
// trace): codes of bf16 rows, 2048 x 4096 6.4 us and 4001 x 11008 25.6 (5.2 TB/s), of
// fp32 rows 8.2 and 39 (5.6), values 6.0 and 20.6 (6.4: the codes partly from the
// last-level cache); 4096 x 11008 of the gating 77 us (4.2; three rows a CU, whose
// sigmoids run beside the loads), its backward 64 (5.7).  A copy of 1 GiB: 5.07 TB/s.
#include <type_traits>

#include "device_common.h"
#include "kernels.h"

namespace qlk {

constexpr int kRowPieces = 8;    // pieces of 8 values a lane holds

// 127 x / a for many x of one row or run.  g: 1, or the power of two that scales x
// first; 0 where all codes are 0 (a is zero, infinite or NaN).
struct Inverse {
  float g, hi, lo, scale;
};
// a: the largest magnitude (bits of a non-negative fp32; NaN and infinity from
// 0x7f800000 on).
__device__ __forceinline__ Inverse inverse_of(uint32_t abits) {
#pragma clang fp contract(off)
  Inverse v;
  const float a = __uint_as_float(abits);
  float as = a;
  v.g = 1.0f;
  // fp32(a / 127): the product with fl(1/127) and one correction (the rounded
  // quotient for all 2^23 mantissas, tested against division)
  const float q = a * (1.0f / 127.0f);
  v.scale = __builtin_fmaf(__builtin_fmaf(-q, 127.0f, a), 1.0f / 127.0f, q);
  if (abits - 0x0d800000u > 0x71800000u - 0x0d800000u) {   // outside [2^-100, 2^100]
    const int e = min(max((int)(abits >> 23) - 127, -120), 120);
    const bool none = abits == 0 || abits >= 0x7f800000u;
    v.g = none ? 0.0f : __uint_as_float((uint32_t)(127 - e) << 23);
    as = none ? 1.0f : a * v.g;                            // exact
    v.scale = abits >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : a / 127.0f;
  }
  const float r = __builtin_amdgcn_rcpf(as);
  v.hi = 127.0f * r;
  v.lo = __builtin_fmaf(-v.hi, as, 127.0f) * r;
  return v;
}
// fp32 whose low byte is the code of x.
__device__ __forceinline__ uint32_t code_of(float x, const Inverse& v) {
#pragma clang fp contract(off)
  const float t = x * v.lo;
  const float n = __builtin_fmaf(x, v.hi, t);
  const float s = n + 12582912.0f;
  return __float_as_uint(s);
}
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t ab = __builtin_amdgcn_perm(b, a, 0x0c0c0400u);
  const uint32_t cd = __builtin_amdgcn_perm(d, c, 0x04000c0cu);
  return ab | cd;
}
__device__ __forceinline__ uint2 codes8(const float (&x)[8], const Inverse& v) {
  uint32_t c[8];
  if (__builtin_expect(v.g == 1.0f, 1)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = code_of(x[i], v);
  } else {
    if (v.g == 0.0f) return make_uint2(0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = code_of(x[i] * v.g, v);
  }
  return make_uint2(pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7]));
}

// Eight values as they are stored: bf16 in four words, fp32 in eight.
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    x[2 * q] = __uint_as_float(w[q] << 16);
    x[2 * q + 1] = __uint_as_float(w[q] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}
// Largest magnitude of eight values as fp32 bits (whole-number maximum: a NaN
// counts as the largest).
__device__ __forceinline__ uint32_t amax8(const float (&x)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
  return m;
}
typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t amax8(const uint4& v) {
  auto mag = [](uint32_t w) { return __builtin_bit_cast(u16x2_t, w & 0x7fff7fffu); };
  const u16x2_t m = __builtin_elementwise_max(__builtin_elementwise_max(mag(v.x), mag(v.y)),
                                              __builtin_elementwise_max(mag(v.z), mag(v.w)));
  return (uint32_t)max(m.x, m.y) << 16;
}
template <class T>
struct Piece;
template <>
struct Piece<uint16_t> {
  uint4 v;
  __device__ __forceinline__ void load(const uint16_t* row, int64_t p) { v = reinterpret_cast<const uint4*>(row)[p]; }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ uint32_t amax() const { return amax8(v); }
  __device__ __forceinline__ void values(float (&x)[8]) const { unpack8(v, x); }
};
template <>
struct Piece<float> {
  float x8[8];
  __device__ __forceinline__ void load(const float* row, int64_t p) {
    const float4 lo = reinterpret_cast<const float4*>(row)[2 * p];
    const float4 hi = reinterpret_cast<const float4*>(row)[2 * p + 1];
    x8[0] = lo.x; x8[1] = lo.y; x8[2] = lo.z; x8[3] = lo.w;
    x8[4] = hi.x; x8[5] = hi.y; x8[6] = hi.z; x8[7] = hi.w;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int e = 0; e < 8; ++e) x8[e] = 0.0f;
  }
  __device__ __forceinline__ uint32_t amax() const { return amax8(x8); }
  __device__ __forceinline__ void values(float (&x)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = x8[e];
  }
};
__device__ __forceinline__ uint32_t max_over_wave(uint32_t m) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
  return m;
}
// Over the W waves that share a row (W == 1: a wave's own).
template <int W>
__device__ __forceinline__ uint32_t max_over_row(uint32_t m, uint32_t* red) {
  m = max_over_wave(m);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) m = max(m, red[w]);
  }
  return m;
}

// Rows of X [M, K] (8 | K).  W waves share a row; a lane holds P pieces of it.
// P == 0: rows longer than the registers hold are read a second time.
template <class T, int W, int P>
__global__ void __launch_bounds__(W == 1 ? 256 : 64 * W)
k_int8_quantize(const T* __restrict__ X, int64_t M, int64_t K, int8_t* __restrict__ codes,
                float* __restrict__ scale) {
  __shared__ uint32_t red[W];
  constexpr int R = W == 1 ? 4 : 1;                     // rows of a workgroup
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t m = (int64_t)blockIdx.x * R + (W == 1 ? wave : 0);
  if (W == 1 && m >= M) return;                         // no barrier follows
  const T* const row = X + m * K;
  uint2* const out = reinterpret_cast<uint2*>(codes + m * K);
  const int64_t np = K / 8;
  const int p0 = W == 1 ? lane : (int)threadIdx.x;
  constexpr int stride = 64 * W;
  uint32_t a = 0;
  float x[8];
  if constexpr (P > 0) {
    Piece<T> v[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int p = p0 + i * stride;
      if (p < np) v[i].load(row, p);
      else v[i].zero();
    }
#pragma unroll
    for (int i = 0; i < P; ++i) a = max(a, v[i].amax());
    const Inverse inv = inverse_of(max_over_row<W>(a, red));
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int p = p0 + i * stride;
      v[i].values(x);
      if (p < np) out[p] = codes8(x, inv);
    }
    if (p0 == 0) scale[m] = inv.scale;
  } else {
    Piece<T> v;
    for (int64_t p = p0; p < np; p += stride) {
      v.load(row, p);
      a = max(a, v.amax());
    }
    const Inverse inv = inverse_of(max_over_row<W>(a, red));
    for (int64_t p = p0; p < np; p += stride) {
      v.load(row, p);
      v.values(x);
      out[p] = codes8(x, inv);
    }
    if (p0 == 0) scale[m] = inv.scale;
  }
}

// Waves per row and pieces per lane for np pieces: a wave holds a short row alone
// and needs no barrier; long rows spread over a workgroup, up to kRowPieces pieces a
// lane, and what that does not hold is read twice.
template <class F>
static void for_row(int64_t np, F f) {
  using std::integral_constant;
  auto pieces = [&](auto w) {
    constexpr int W = decltype(w)::value;
    const int64_t need = (np + 64 * W - 1) / (64 * W);
    if (need <= 1) f(w, integral_constant<int, 1>());
    else if (W == 1 || need <= 2) f(w, integral_constant<int, 2>());
    else if constexpr (W > 1) {
      if (need <= 4) f(w, integral_constant<int, 4>());
      else if (need <= 6) f(w, integral_constant<int, 6>());
      else f(w, integral_constant<int, kRowPieces>());
    }
  };
  if (np <= 64 * 2) pieces(integral_constant<int, 1>());
  else if (np <= 256 * kRowPieces) pieces(integral_constant<int, 4>());
  else if (np <= 1024 * 4) f(integral_constant<int, 16>(), integral_constant<int, 4>());
  else if (np <= 1024 * kRowPieces) f(integral_constant<int, 16>(), integral_constant<int, kRowPieces>());
  else f(integral_constant<int, 16>(), integral_constant<int, 0>());
}

template <class T>
static hipError_t int8_quantize_rows(const T* X, int64_t M, int64_t K, int8_t* codes, float* scale,
                                     hipStream_t st) {
  for_row(K / 8, [&](auto w, auto p) {
    constexpr int W = decltype(w)::value, P = decltype(p)::value;
    const int64_t grid = W == 1 ? (M + 3) / 4 : M;
    hipLaunchKernelGGL((k_int8_quantize<T, W, P>), dim3((unsigned)grid), dim3(W == 1 ? 256 : 64 * W),
                       0, st, X, M, K, codes, scale);
  });
  return hipGetLastError();
}
hipError_t launch_int8_quantize(const uint16_t* X, int64_t M, int64_t K, int8_t* codes,
                                float* scale, hipStream_t st) {
  return int8_quantize_rows(X, M, K, codes, scale, st);
}
hipError_t launch_int8_quantize(const float* X, int64_t M, int64_t K, int8_t* codes, float* scale,
                                hipStream_t st) {
  return int8_quantize_rows(X, M, K, codes, scale, st);
}

__device__ __forceinline__ float code_value(uint32_t w, int i) {
  return (float)(int8_t)(w >> (8 * i));
}

// out = bf16(code scale), whole lines of 8 codes a lane (pairs of 16-byte stores a lane
// apart took 22.5 us for 4001 x 11008, here 20).  BLOCK: scales per 64 columns
// (64 | K), else one per row.
constexpr int kDqPieces = 2;
template <bool BLOCK>
__global__ void __launch_bounds__(256)
k_int8_dequant(const int8_t* __restrict__ codes, const float* __restrict__ scale, int64_t n8,
               uint32_t k8, uint16_t* __restrict__ out) {
  // piece e of a thread: 8 codes, 256 pieces on from the last
  const int64_t i0 = (int64_t)blockIdx.x * (256 * kDqPieces) + threadIdx.x;
  uint2 c[kDqPieces];
  float s[kDqPieces];
#pragma unroll
  for (int e = 0; e < kDqPieces; ++e) {
    const int64_t i = min(i0 + 256 * e, n8 - 1);
    c[e] = reinterpret_cast<const uint2*>(codes)[i];
    if constexpr (BLOCK) s[e] = scale[i >> 3];
    else s[e] = scale[(uint32_t)i / k8];   // M K < 2^34: i < 2^31
  }
#pragma unroll
  for (int e = 0; e < kDqPieces; ++e) {
    const int64_t i = i0 + 256 * e;
    float x[8];
#pragma unroll
    for (int v = 0; v < 8; ++v) x[v] = code_value(v < 4 ? c[e].x : c[e].y, v % 4) * s[e];
    if (i < n8) reinterpret_cast<uint4*>(out)[i] = pack8(x);
  }
}

hipError_t launch_int8_dequant(const int8_t* codes, const float* scale, int64_t M, int64_t K,
                               bool block, uint16_t* out, hipStream_t st) {
  const int64_t n8 = M * K / 8;
  const dim3 grid((unsigned)((n8 + 256 * kDqPieces - 1) / (256 * kDqPieces)));
  if (block)
    hipLaunchKernelGGL(k_int8_dequant<true>, grid, dim3(256), 0, st, codes, scale, n8,
                       (uint32_t)(K / 8), out);
  else
    hipLaunchKernelGGL(k_int8_dequant<false>, grid, dim3(256), 0, st, codes, scale, n8,
                       (uint32_t)(K / 8), out);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// H = silu(G) U.  The value that is quantised is the fp32 product; where the
// bf16 H is wanted too, it has the elementwise gating's bits.  The eight lanes of a run of 64 columns hold it whole.
__device__ __forceinline__ uint32_t max_over_8(uint32_t m) {
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
  return m;
}

struct GateOut {
  uint16_t* H;        // bf16 [M, I], or null
  int8_t* H8;         // rows
  float* Hs;
  int8_t* G8;         // runs of 64, or null (then U8 is null too)
  float* Gs;
  int8_t* U8;
  float* Us;
};

// One piece of G or U kept in 8 bits; every lane of the run calls it.
__device__ __forceinline__ void keep8(const uint4& v, const float (&x)[8], int8_t* codes, float* scale,
                                      int64_t row8, int64_t p, bool in) {
  const Inverse inv = inverse_of(max_over_8(amax8(v)));
  if (!in) return;
  reinterpret_cast<uint2*>(codes)[row8 + p] = codes8(x, inv);
  if ((p & 7) == 0) scale[(row8 + p) >> 3] = inv.scale;
}
// silu(g) u for eight values.  The reciprocal is the instruction's, within an ulp, and
// would be 0 where it is subnormal (1 + exp(-g) above 2^126, g below -87.3): it is
// taken of a quarter of that sum, against a quarter of g.
__device__ __forceinline__ void silu_mul8(const float (&g)[8], const float (&u)[8], float (&h)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    h[e] = 0.25f * g[e] * __builtin_amdgcn_rcpf(__builtin_fmaf(0.25f, __expf(-g[e]), 0.25f)) * u[e];
}

struct GateIn {
  uint4 g, u;
};
__device__ __forceinline__ void gate_load(GateIn& v, const uint16_t* grow, const uint16_t* urow, int64_t p,
                                          int64_t np) {
  v.g = v.u = make_uint4(0, 0, 0, 0);
  if (p < np) {
    v.g = reinterpret_cast<const uint4*>(grow)[p];
    v.u = reinterpret_cast<const uint4*>(urow)[p];
  }
}
// H of a piece; `first`: G and U (and the bf16 H) leave as well.
__device__ __forceinline__ void gate_piece(const GateOut& o, const GateIn& v, int64_t row8, int64_t p,
                                           int64_t np, bool first, float (&h)[8]) {
  float g[8], u[8];
  unpack8(v.g, g);
  unpack8(v.u, u);
  silu_mul8(g, u, h);
  if (!first) return;
  const bool in = p < np;
  if (o.H && in) {
    float b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = silu_mul_f32(g[e], u[e]);
    reinterpret_cast<uint4*>(o.H)[row8 + p] = pack8(b);
  }
  if (o.G8) {
    keep8(v.g, g, o.G8, o.Gs, row8, p, in);
    keep8(v.u, u, o.U8, o.Us, row8, p, in);
  }
}

// A row per workgroup of W waves.  LDS: its H stays there in fp32 between the
// maximum and the codes, the next piece's loads in flight; otherwise (a row longer
// than LDS) G and U are read a second time.  (In registers H, G and U took 24 for
// each piece of a lane, and two waves a SIMD did not cover the loads: 4096 x 11008,
// 92 us.)
template <int W, bool LDS>
__global__ void __launch_bounds__(64 * W)
k_silu_mul_fwd_int8(const uint16_t* __restrict__ G, const uint16_t* __restrict__ U, int64_t I, GateOut o) {
  __shared__ uint32_t red[W];
  extern __shared__ float4 hl[];
  const int64_t m = blockIdx.x;
  const int64_t np = I / 8, row8 = m * np;
  constexpr int stride = 64 * W;
  const int tid = threadIdx.x;
  const uint16_t* const grow = G + m * I;
  const uint16_t* const urow = U + m * I;
  uint2* const out = reinterpret_cast<uint2*>(o.H8) + row8;
  uint32_t a = 0;
  float h[8];
  GateIn v, next;
  gate_load(v, grow, urow, tid, np);
  for (int64_t q = 0; q < np; q += stride) {       // whole waves: a run's lanes work together
    const int64_t p = q + tid;
    gate_load(next, grow, urow, p + stride, np);
    gate_piece(o, v, row8, p, np, true, h);
    a = max(a, amax8(h));
    if (LDS && p < np) {
      hl[p] = make_float4(h[0], h[1], h[2], h[3]);
      hl[np + p] = make_float4(h[4], h[5], h[6], h[7]);
    }
    v = next;
  }
  const Inverse inv = inverse_of(max_over_row<W>(a, red));
  for (int64_t p = tid; p < np; p += stride) {
    if constexpr (LDS) {                           // this thread's own
      const float4 x = hl[p], y = hl[np + p];
      const float hv[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
      out[p] = codes8(hv, inv);
    } else {
      gate_load(v, grow, urow, p, np);
      gate_piece(o, v, row8, p, np, false, h);
      out[p] = codes8(h, inv);
    }
  }
  if (tid == 0) o.Hs[m] = inv.scale;
}

hipError_t launch_silu_mul_fwd_int8(const uint16_t* G, const uint16_t* U, int64_t M, int64_t I,
                                    uint16_t* H, int8_t* H8, float* Hs, int8_t* G8, float* Gs,
                                    int8_t* U8, float* Us, hipStream_t st) {
  const GateOut o{H, H8, Hs, G8, Gs, U8, Us};
  const dim3 grid((unsigned)M);
  const size_t lds = (size_t)I * 4;
  if (I <= 512) hipLaunchKernelGGL((k_silu_mul_fwd_int8<1, true>), grid, dim3(64), lds, st, G, U, I, o);
  else if (I <= 8192) hipLaunchKernelGGL((k_silu_mul_fwd_int8<4, true>), grid, dim3(256), lds, st, G, U, I, o);
  else if (I <= 14336) hipLaunchKernelGGL((k_silu_mul_fwd_int8<8, true>), grid, dim3(512), lds, st, G, U, I, o);
  else if (I <= 40000) hipLaunchKernelGGL((k_silu_mul_fwd_int8<16, true>), grid, dim3(1024), lds, st, G, U, I, o);
  else hipLaunchKernelGGL((k_silu_mul_fwd_int8<16, false>), grid, dim3(1024), 0, st, G, U, I, o);
  return hipGetLastError();
}

// dG = dH U sig(G) (1 + G (1 - sig(G))), dU = dH silu(G), from the kept runs.
__global__ void __launch_bounds__(256)
k_silu_mul_bwd_int8(const uint16_t* __restrict__ dH, const int8_t* __restrict__ G8,
                    const float* __restrict__ Gs, const int8_t* __restrict__ U8,
                    const float* __restrict__ Us, int64_t n8, uint16_t* __restrict__ dG,
                    uint16_t* __restrict__ dU) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n8) return;
  float d[8], g[8], u[8];
  unpack8(reinterpret_cast<const uint4*>(dH)[i], d);
  const uint2 gc = reinterpret_cast<const uint2*>(G8)[i], uc = reinterpret_cast<const uint2*>(U8)[i];
  const float gs = Gs[i >> 3], us = Us[i >> 3];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float gv = code_value(e < 4 ? gc.x : gc.y, e % 4) * gs;
    const float uv = code_value(e < 4 ? uc.x : uc.y, e % 4) * us;
    const float sg = sigmoidf_(gv);
    g[e] = d[e] * uv * sg * (1.0f + gv * (1.0f - sg));
    u[e] = d[e] * gv * sg;
  }
  reinterpret_cast<uint4*>(dG)[i] = pack8(g);
  reinterpret_cast<uint4*>(dU)[i] = pack8(u);
}

hipError_t launch_silu_mul_bwd_int8(const uint16_t* dH, const int8_t* G8, const float* Gs,
                                    const int8_t* U8, const float* Us, int64_t M, int64_t I,
                                    uint16_t* dG, uint16_t* dU, hipStream_t st) {
  const int64_t n8 = M * I / 8;
  hipLaunchKernelGGL(k_silu_mul_bwd_int8, dim3((unsigned)((n8 + 255) / 256)), dim3(256), 0, st, dH,
                     G8, Gs, U8, Us, n8, dG, dU);
  return hipGetLastError();
}

}  // namespace qlk
