// bf16 -> e4m3 with one fp32 scale per block:
//   a = max |x| of the block,  s = fl(a / 448) (1 where that is 0),
//   q = e4m3(fl(x / s)), both divisions IEEE fp32, e4m3 to nearest even.
// Activations: blocks of 1 row x 128 columns (quantize_rows_kernel); weights:
// blocks of 128 x 128 (quantize_blocks_kernel).
//
// Bound by memory (2 bytes read, 1 written per element); each element is read
// once and stays in registers between the maximum and the division.
//
// The division: with r = fl(1 / s), q0 = fl(x r), the step q = fl(q0 + fl(x - q0 s) r)
// (Markstein 1990) rounds a number within 2^-47 relative of x / s.  It could
// only change the e4m3 result where that straddles an fp32 midpoint next to a
// 5-bit rounding boundary t of e4m3; there x - t s would have to equal half an
// ulp of t times s up to 2^-47, and as x - t s is a multiple of 2^-4 ulp(s), s
// would be a short multiple of a power of two and x / s the midpoint itself,
// which no quotient of fp32 numbers is.  So the codes are those of the IEEE
// division.  The residual needs x - q0 s above the subnormal range: blocks
// whose maximum is below 2^-90, zero, infinite or NaN take the division itself.
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

// |a| and |b| packed, the larger of each half; NaN wins.
__device__ __forceinline__ uint32_t absmax_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a & 0x7FFF7FFFu), "r"(b & 0x7FFF7FFFu));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ uint32_t absmax_words(const uint4& v, uint32_t m) {
  m = absmax_bf16x2(v.x, m);
  m = absmax_bf16x2(v.y, m);
  m = absmax_bf16x2(v.z, m);
  return absmax_bf16x2(v.w, m);
}

__device__ __forceinline__ float quant_scale(float amax) {
  const float s = __fdiv_rn(amax, 448.f);
  return s == 0.f ? 1.f : s;
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
  __device__ __forceinline__ QuantDiv(float amax) : s(quant_scale(amax)) {
    fast = amax >= 0x1p-90f && amax <= 3.4e38f;  // false for NaN
    r = fast ? __frcp_rn(s) : 0.f;
  }
  __device__ __forceinline__ uint32_t pair(uint32_t w) const {  // two bf16 -> two e4m3
    const float x0 = bf16lo(w), x1 = bf16hi(w);
    if (fast) {
      const float q0 = x0 * r, q1 = x1 * r;
      return e4m3x2(fmaf(fmaf(-q0, s, x0), r, q0), fmaf(fmaf(-q1, s, x1), r, q1));
    }
    return e4m3x2(__fdiv_rn(x0, s), __fdiv_rn(x1, s));
  }
  __device__ __forceinline__ uint2 eight(const uint4& v) const {
    return make_uint2(pair(v.x) | (pair(v.y) << 16), pair(v.z) | (pair(v.w) << 16));
  }
};

// 8 bf16 at x, the first `left` of which exist (others read as zero)
__device__ __forceinline__ uint4 quant_load8(const uint16_t* x, int64_t left) {
  if (left >= 8) return ldg_nc_v4(x);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < left) w[e >> 1] |= static_cast<uint32_t>(__ldg(x + e)) << ((e & 1) * 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void quant_store8(uint8_t* q, uint2 v, int64_t left) {
  if (left >= 8) {
    *reinterpret_cast<uint2*>(q) = v;
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < left) q[e] = static_cast<uint8_t>((e < 4 ? v.x : v.y) >> ((e & 3) * 8));
}

// 16 teams of 16 lanes; a team takes U blocks of one row.  R = 16: the teams
// take 16 consecutive rows, whose scales are neighbours in memory; R = 1 (fewer
// than 16 rows): the teams take consecutive blocks of one row.
template <int R, int U>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const QuantParams p) {
  const int team = threadIdx.x >> 4, tl = threadIdx.x & 15;
  constexpr int TB = 16 / R;  // teams side by side along the blocks
  const int64_t row = static_cast<int64_t>(blockIdx.x) * R + team / TB;
  const int64_t b0 = static_cast<int64_t>(blockIdx.y) * (TB * U) + team % TB;
  wait_prior_kernels();
  uint4 v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t col = (b0 + u * TB) * 128 + tl * 8;
    v[u] = (row < p.n && col < p.d) ? quant_load8(p.x + row * p.ldx + col, p.d - col) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t m = absmax_words(v[u], 0u);
#pragma unroll
    for (int k = 8; k >= 1; k /= 2) m = absmax_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, k));
    const QuantDiv dv(max_nan(bf16lo(m), bf16hi(m)));
    const int64_t blk = b0 + u * TB;
    const int64_t col = blk * 128 + tl * 8;
    if (row < p.n && col < p.d) {
      quant_store8(p.q + row * p.ldq + col, dv.eight(v[u]), p.d - col);
      if (tl == 0) p.s[blk * p.lds + row] = dv.s;
    }
  }
}

// One 128 x 128 block per CTA: 16 rows per pass, 16 lanes x 8 columns per row.
__global__ void __launch_bounds__(256) quantize_blocks_kernel(const QuantParams p) {
  __shared__ float warp_max[8];
  const int64_t blk = blockIdx.x;
  const int mb = static_cast<int>(blk % p.mblocks);
  const int64_t rest = blk / p.mblocks;
  const int db = static_cast<int>(rest % p.dblocks);
  const int64_t mat = rest / p.dblocks;
  const int64_t row0 = static_cast<int64_t>(db) * 128 + (threadIdx.x >> 4);
  const int64_t col = static_cast<int64_t>(mb) * 128 + (threadIdx.x & 15) * 8;
  const uint16_t* x = p.x + mat * p.xstride + row0 * p.ldx + col;
  uint8_t* q = p.q + mat * p.qstride + row0 * p.ldq + col;
  wait_prior_kernels();
  uint4 v[8];
#pragma unroll
  for (int u = 0; u < 8; ++u)
    v[u] = (row0 + u * 16 < p.n && col < p.d) ? quant_load8(x + u * 16 * p.ldx, p.d - col) : make_uint4(0u, 0u, 0u, 0u);
  uint32_t m = 0u;
#pragma unroll
  for (int u = 0; u < 8; ++u) m = absmax_words(v[u], m);
#pragma unroll
  for (int k = 16; k >= 1; k /= 2) m = absmax_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, k));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = max_nan(bf16lo(m), bf16hi(m));
  __syncthreads();
  float a = warp_max[0];
#pragma unroll
  for (int w = 1; w < 8; ++w) a = max_nan(a, warp_max[w]);
  const QuantDiv dv(a);
#pragma unroll
  for (int u = 0; u < 8; ++u)
    if (row0 + u * 16 < p.n && col < p.d) quant_store8(q + u * 16 * p.ldq, dv.eight(v[u]), p.d - col);
  if (threadIdx.x == 0) p.s[blk] = dv.s;
}

}  // namespace rmm
