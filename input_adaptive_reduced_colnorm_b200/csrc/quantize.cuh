// bf16 -> e4m3 with one fp32 scale per block:
//   a = max |x| of the block,  s = fl(a / 448) (1 where that is 0),
//   q = e4m3(fl(x / s)), both divisions IEEE fp32, e4m3 to nearest even.
// Activations: blocks of 1 row x 128 columns (quantize_rows_kernel); weights:
// blocks of 128 x 128 (quantize_blocks_kernel).
//
// Bound by memory (2 bytes read, 1 written per element): 8192 x 14336 takes 55-64 us,
// 0.84-0.98 of the copy bandwidth, eight 4096 x 14336 weights 208-237 us, 0.91-1.0.  It
// takes about 10 instructions per element to stay there (packed arithmetic, 8 lanes a
// block, 32-bit columns, no edge checks where d is a multiple of 16): with 14 the same
// call took 63 us where it took 55 with 10, with IEEE divisions and 16 lanes a block 94,
// bound by issue slots.  Each
// element is read once and stays in registers between the maximum and the division.
//
// The division, on packed pairs: q0 = x r, q = q0 + (x - q0 s) r with r ~ 1 / s
// (Markstein 1990) has a relative error below 2^-44 before its last rounding.
// That gives the codes of the IEEE division: with x and a 8-bit numbers times
// powers of two, 448 x / a either lies at least 2^-14 (relative) off a rounding
// boundary t of e4m3 (an odd 5-bit number), far more than all errors here, or is
// t.  Then s = (a / 448)(1 + e) with e = j / 7 of its last place, j = -3 .. 3, and
// x / s = t (1 - e) to 2^-46; whether that rounds to t or to a neighbour of t in
// fp32 turns on (2 j / 7) t / s (mantissas) against 1, and as they differ (equality
// needs 7 | t, but then a / 448 is exact and e = 0) they do by more than 2^-11.
// The scale itself is a q0-step on 1 / 448: a / 7 is never nearer to an fp32
// midpoint than 1 / 14 of the last place.  The residuals need their products above
// the subnormal range: blocks whose maximum is below 2^-90, infinite or NaN take
// the division itself.  (All 5.3e8 pairs of a finite block maximum and a value up to it
// were compared with the divisions once: the same codes and scales.)
#pragma once
#include <cuda_bf16.h>
#include "ptx.cuh"

namespace rmm {

struct QuantParams {
  const uint16_t* x;
  int64_t ldx;
  uint8_t* q;
  int64_t ldq;
  float* s;
  int64_t lds;        // rows: scale of (row, block) at s[block * lds + row]
  int64_t n, d;       // rows, columns
  int64_t xstride, qstride;  // blocks kernel: elements between matrices
  int dblocks, mblocks;      // blocks kernel: row and column blocks of one matrix
};

// The larger size of each half, NaN if either is; the sign bits mean nothing.
__device__ __forceinline__ uint32_t absmax_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t absmax_words(const uint4& v, uint32_t m) {
  return absmax_bf16x2(absmax_bf16x2(v.x, v.y), absmax_bf16x2(absmax_bf16x2(v.z, v.w), m));
}
// of a packed maximum: the larger half
__device__ __forceinline__ float absmax_value(uint32_t m) {
  return bf16hi(absmax_bf16x2(m, m << 16) & 0x7FFFFFFFu);
}

__device__ __forceinline__ uint64_t pair_f32(float lo, float hi) {
  return static_cast<uint64_t>(__float_as_uint(lo)) | (static_cast<uint64_t>(__float_as_uint(hi)) << 32);
}

// two values to packed e4m3 (first in the low byte)
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t v;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
  return v;
}

struct QuantDiv {
  float s, r;
  bool fast;
  __device__ __forceinline__ explicit QuantDiv(float amax) {
    // (zeros, padding as a rule, divide by 1 on the short path; false for NaN)
    fast = (amax >= 0x1p-90f && amax <= 3.4e38f) || amax == 0.f;
    if (fast) {
      constexpr float k = 1.f / 448.f;
      const float q0 = amax * k;
      s = amax == 0.f ? 1.f : fmaf(fmaf(-q0, 448.f, amax), k, q0);
      asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(s));
    } else {
      s = __fdiv_rn(amax, 448.f);
      if (s == 0.f) s = 1.f;
      r = 0.f;
    }
  }
  // two bf16 -> two e4m3
  __device__ __forceinline__ uint32_t pair_fast(uint32_t w) const {
    const uint64_t x = pair_f32(bf16lo(w), bf16hi(w));
    const uint64_t r2 = pair_f32(r, r), ns2 = pair_f32(-s, -s);
    uint64_t q0, q;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q0) : "l"(x), "l"(r2));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q) : "l"(q0), "l"(ns2), "l"(x));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q) : "l"(q), "l"(r2), "l"(q0));
    return e4m3x2(__uint_as_float(static_cast<uint32_t>(q)), __uint_as_float(static_cast<uint32_t>(q >> 32)));
  }
  __device__ __forceinline__ uint32_t pair_div(uint32_t w) const {
    return e4m3x2(__fdiv_rn(bf16lo(w), s), __fdiv_rn(bf16hi(w), s));
  }
  // 16 bf16 -> 16 e4m3
  __device__ __forceinline__ uint4 sixteen(const uint4& a, const uint4& b) const {
    if (fast)
      return make_uint4(pair_fast(a.x) | (pair_fast(a.y) << 16), pair_fast(a.z) | (pair_fast(a.w) << 16),
                        pair_fast(b.x) | (pair_fast(b.y) << 16), pair_fast(b.z) | (pair_fast(b.w) << 16));
    return make_uint4(pair_div(a.x) | (pair_div(a.y) << 16), pair_div(a.z) | (pair_div(a.w) << 16),
                      pair_div(b.x) | (pair_div(b.y) << 16), pair_div(b.z) | (pair_div(b.w) << 16));
  }
};

// 8 bf16 at x, of which `left` exist (others read as zero); WHOLE: all or none
template <bool WHOLE>
__device__ __forceinline__ uint4 quant_load8(const uint16_t* x, int left) {
  if (WHOLE ? left > 0 : left >= 8) return ld_v4_once(x);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  if (!WHOLE) {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < left) w[e >> 1] |= static_cast<uint32_t>(x[e]) << ((e & 1) * 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// the first `left` of 16 e4m3
template <bool WHOLE>
__device__ __forceinline__ void quant_store16(uint8_t* q, const uint4& v, int left) {
  if (WHOLE ? left > 0 : left >= 16) {
    *reinterpret_cast<uint4*>(q) = v;
  } else if (!WHOLE && left > 0) {
    uint32_t lo = v.x, hi = v.y;
    if (left >= 8) {
      *reinterpret_cast<uint2*>(q) = make_uint2(v.x, v.y);
      q += 8;
      left -= 8;
      lo = v.z;
      hi = v.w;
    }
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < left) q[e] = static_cast<uint8_t>((e < 4 ? lo : hi) >> ((e & 3) * 8));
  }
}

// A team of 8 lanes takes a block of one row, 16 columns per lane; a warp four
// neighbouring blocks (1 KB of the row), U times.  R = 8: the warps of a CTA take
// 8 consecutive rows, whose scales are neighbours in memory; R = 1 (few rows): they
// take consecutive blocks of one row.  WHOLE: d is a multiple of 16, so that a lane
// has 16 columns or none.
template <int R, int U, bool WHOLE>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const QuantParams p) {
  constexpr int WB = 8 / R;               // warps side by side along the blocks
  constexpr int CHUNK = WB * 4 * U;       // blocks of one row in a CTA
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tl = lane & 7;
  const int d = static_cast<int>(p.d);
  const unsigned chunks = (static_cast<unsigned>(d) + CHUNK * 128 - 1) / (CHUNK * 128);
  const int64_t row = static_cast<int64_t>(blockIdx.x / chunks) * R + warp / WB;
  if (row >= p.n) return;
  const int b0 = static_cast<int>(blockIdx.x % chunks) * CHUNK + (warp % WB) * 4 * U + (lane >> 3);
  const int left = d - (b0 * 128 + tl * 16);  // columns from this lane's first on
  const uint16_t* x = p.x + row * p.ldx + b0 * 128 + tl * 16;
  uint8_t* q = p.q + row * p.ldq + b0 * 128 + tl * 16;
  float* s = p.s + b0 * p.lds + row;
  wait_prior_kernels();
  uint4 v[U][2];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    v[u][0] = quant_load8<WHOLE>(x + u * 512, left - u * 512);
    v[u][1] = quant_load8<WHOLE>(x + u * 512 + 8, left - u * 512 - 8);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t m = absmax_words(v[u][1], absmax_words(v[u][0], 0u));
#pragma unroll
    for (int k = 4; k >= 1; k /= 2) m = absmax_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, k));
    const QuantDiv dv(absmax_value(m));
    quant_store16<WHOLE>(q + u * 512, dv.sixteen(v[u][0], v[u][1]), left - u * 512);
    if (tl == 0 && left > u * 512) s[u * 4 * p.lds] = dv.s;
  }
}

// One 128 x 128 block per CTA: 32 rows per pass, 8 lanes x 16 columns per row.
template <bool WHOLE>
__global__ void __launch_bounds__(256) quantize_blocks_kernel(const QuantParams p) {
  __shared__ uint32_t warp_max[8];
  const unsigned blk = blockIdx.x;
  const unsigned mb = blk % static_cast<unsigned>(p.mblocks), rest = blk / static_cast<unsigned>(p.mblocks);
  const unsigned db = rest % static_cast<unsigned>(p.dblocks), mat = rest / static_cast<unsigned>(p.dblocks);
  const int row0 = static_cast<int>(db) * 128 + (threadIdx.x >> 3);
  const int col = static_cast<int>(mb) * 128 + (threadIdx.x & 7) * 16;
  const int rows = static_cast<int>(p.n), left = static_cast<int>(p.d) - col;
  const uint16_t* x = p.x + mat * p.xstride + row0 * p.ldx + col;
  uint8_t* q = p.q + mat * p.qstride + row0 * p.ldq + col;
  wait_prior_kernels();
  uint4 v[4][2];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int here = row0 + u * 32 < rows ? left : 0;
    v[u][0] = quant_load8<WHOLE>(x + u * 32 * p.ldx, here);
    v[u][1] = quant_load8<WHOLE>(x + u * 32 * p.ldx + 8, here - 8);
  }
  uint32_t m = 0u;
#pragma unroll
  for (int u = 0; u < 4; ++u) m = absmax_words(v[u][1], absmax_words(v[u][0], m));
#pragma unroll
  for (int k = 16; k >= 1; k /= 2) m = absmax_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, k));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
  __syncthreads();
  m = warp_max[0];
#pragma unroll
  for (int w = 1; w < 8; ++w) m = absmax_bf16x2(m, warp_max[w]);
  const QuantDiv dv(absmax_value(m));
#pragma unroll
  for (int u = 0; u < 4; ++u)
    quant_store16<WHOLE>(q + u * 32 * p.ldq, dv.sixteen(v[u][0], v[u][1]), row0 + u * 32 < rows ? left : 0);
  if (threadIdx.x == 0) p.s[blk] = dv.s;
}

}  // namespace rmm
