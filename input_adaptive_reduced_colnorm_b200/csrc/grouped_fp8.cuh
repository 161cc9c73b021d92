// The e4m3 product with block scales for groups of many rows (see grouped.cuh for
// the formula and the group bounds): tiles of 256 rows of X x 256 columns of W on
// CTA pairs, rows on the M side.
//
// Why not swapped as the narrow tiles: every 128-deep block's accumulator passes
// through the epilogue threads, 128 x 256 fp32 per CTA, while the tensor cores
// spend 512 cycles on the next one.  With rows of X on the lanes a thread's 128
// columns share ONE scale (its row's times the weight block's), kept in a
// register, and tensor memory is read in the 32 x 32-bit shape (128 bytes per
// cycle and warp scheduler: 256 of the 512 cycles; the 16 x 256-bit shape that the
// swapped form needs reads half as fast, 546 cycles).  What it costs is a group's
// last tile, 256 rows however few are left.
//
// Roles (384 threads): warp 0 TMA producer, warp 1 MMA issuer (even CTA), warps
// 4-11 epilogue: warp w reads lanes 32 (w % 4) .. + 31 and one half of the columns.
// The tiles of a partial last wave are cut along W into 128- or 64-column pieces.
#pragma once
#include "grouped.cuh"

namespace rmm {

struct GroupedFp8Cfg {
  static constexpr int X_BYTES = 128 * 128;  // this CTA's 128 rows x 128 contraction indices
  static constexpr int W_BYTES = 128 * 128;  // its 128 of the 256 columns
  static constexpr int STAGES = 6;
  static constexpr int THREADS = 384;
  // registers per thread at launch, and the split after the set-up: 128 sums and
  // two 32-column loads in flight per epilogue thread (the host checks that the
  // kernel was compiled to LAUNCH_REGS, on which the split draws)
  static constexpr int LAUNCH_REGS = 168, OTHER_REGS = 56, EPI_REGS = 224;
  static_assert(OTHER_REGS + 2 * EPI_REGS <= 3 * LAUNCH_REGS, "three warpgroups share what was launched");
  static int smem_bytes(int groups) { return 1024 + STAGES * (X_BYTES + W_BYTES) + 256 + (2 * groups + 2) * 4; }
  static_assert(8 * (2 * STAGES + 5) + 8 <= 256, "barrier area");
};

struct GroupedFp8Units {
  const int *off, *pre;
  int groups, n_tiles, whole, cut, count;
  __device__ __forceinline__ GroupedFp8Units(const GroupedParams& p, const int* off_, const int* pre_, int workers)
      : off(off_), pre(pre_), groups(p.groups), n_tiles(p.m_tiles), cut(1) {
    const int tiles = pre[groups] * n_tiles;
    const int rest = tiles % workers;
    if (rest > 0)
      while (cut < 4 && 2 * cut * rest <= workers) cut *= 2;
    whole = tiles - rest;
    count = whole + rest * cut;
  }
  // t.mtile: first column of the piece; t.w: its columns (256, 128 or 64)
  __device__ __forceinline__ GroupedTile get(int unit) const {
    int tile = unit, part = 0;
    GroupedTile t;
    t.w = 256;
    if (unit >= whole) {
      tile = whole + (unit - whole) / cut;
      part = (unit - whole) % cut;
      t.w = 256 / cut;
    }
    int lo = 0, hi = groups - 1;  // the last group whose first tile is <= tile
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] * n_tiles <= tile) lo = mid;
      else hi = mid - 1;
    }
    const int rt = pre[lo + 1] - pre[lo];
    const int r = tile - pre[lo] * n_tiles;
    t.group = lo;
    t.mtile = (r / rt) * 256 + part * t.w;
    t.row0 = off[lo] + (r % rt) * 256;
    t.row_end = off[lo + 1];
    return t;
  }
};

__global__ void __launch_bounds__(GroupedFp8Cfg::THREADS, 1)
    grouped_fp8_rows_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                            const GroupedParams p) {
  using C = GroupedFp8Cfg;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t grouped_fp8_smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(grouped_fp8_smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sX = smem;
  uint8_t* sW = smem + STAGES * C::X_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(sW + STAGES * C::W_BYTES);  // used in the even CTA
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;  // used in the even CTA
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* off = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(full) + 256);
  int* pre = off + p.groups + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // 0: the CTA that issues the MMAs
  const int worker = static_cast<int>(blockIdx.x >> 1), workers = static_cast<int>(gridDim.x >> 1);
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 16);  // eight epilogue warps of each CTA
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&tmW);
    prefetch_tensormap(&tmX);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  wait_prior_kernels();  // bounds, operands and the output are touched only after this
  if (warp == 2) grouped_bounds<256>(p, off, pre, lane);
  tc_fence_before();
  cluster_sync();  // barriers of both CTAs initialised, tensor memory allocated
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const GroupedFp8Units units(p, off, pre, workers);

  if (warp < 4) set_max_regs_down<C::OTHER_REGS>();
  if (warp == 0) {
    // ------------------------------------------------------------ producer (both CTAs)
    if (lane == 0) {
      const uint32_t full_even = map_shared_rank(smem_u32(&full[0]), 0u);
      int stage = 0;
      uint32_t phase = 0, issued = 0;
      bool ok = true;
      for (int unit = worker; ok && unit < units.count; unit += workers) {
        const GroupedTile t = units.get(unit);
        const int row = t.row0 + static_cast<int>(rank) * 128;
        const int col = t.mtile + static_cast<int>(rank) * (t.w / 2);
        for (int kb = 0; kb < p.num_kb; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, kDevErrTimeoutProducer)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * (C::X_BYTES + C::W_BYTES));
          const uint32_t bar = full_even + 8u * static_cast<uint32_t>(stage);
          tma_load_2d_pair(sX + stage * C::X_BYTES, &tmX, bar, kb * 128, row);
          // (a narrow piece uses the first t.w / 2 of the 128 columns loaded)
          tma_load_3d_pair(sW + stage * C::W_BYTES, &tmW, bar, col, kb * 128, t.group);
          ++issued;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && rank == 0) {
        // wait (bounded) for the stages filled so far, so no copy lands after exit
        for (int s = 0; s < STAGES; ++s) {
          const uint32_t uses = (issued + STAGES - 1 - s) / STAGES;
          if (uses == 0) continue;
          const uint32_t a = smem_u32(&full[s]);
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait(a, (uses - 1) & 1u) && globaltimer_ns() - t0 < kWaitTimeoutNs) {
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (rank == 0 && lane == 0) {
      int stage = 0;
      uint32_t phase = 0, acc_i = 0;
      bool ok = true;
      for (int unit = worker; ok && unit < units.count; unit += workers) {
        const uint32_t idesc = make_idesc_e4m3(256, 0, 0, 1) | (static_cast<uint32_t>(units.get(unit).w >> 3) << 17);
        for (int kb = 0; kb < p.num_kb; ++kb, ++acc_i) {
          const uint32_t acc = acc_i & 1u;
          if (!mbar_wait(&tempty[acc], ((acc_i >> 1) & 1u) ^ 1u, abort_flag, kDevErrTimeoutMma, 0, kMbarClusterRelaxed) ||
              !mbar_wait(&full[stage], phase, abort_flag, kDevErrTimeoutMma)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t x0 = smem_u32(sX + stage * C::X_BYTES);
          const uint32_t w0 = smem_u32(sW + stage * C::W_BYTES);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_e4m3_pair(tmem_base + acc * 256, make_sw128_desc(x0 + kk * 32, 16, 1024),
                           make_sw128_desc(w0 + kk * 4096, 16384, 1024), idesc, kk != 0 ? 1u : 0u);
          umma_commit_pair(&empty[stage], 0x3);
          umma_commit_pair(&tfull[acc], 0x3);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // every MMA issued by this thread is complete once `drain` flips
      umma_commit_pair(drain, 0x1);
      const uint32_t a = smem_u32(drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(a, 0) && globaltimer_ns() - t0 < kWaitTimeoutNs) {
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue (both CTAs)
    set_max_regs_up<C::EPI_REGS>();
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t tempty_even = map_shared_rank(smem_u32(&tempty[0]), 0u);
    uint32_t acc_i = 0;
    bool ok = true;
    for (int unit = worker; ok && unit < units.count; unit += workers) {
      const GroupedTile t = units.get(unit);
      const int row = t.row0 + static_cast<int>(rank) * 128 + quarter * 32 + lane;
      const int hw = t.w / 2;                    // columns of this thread: 128, 64 or 32
      const int col0 = t.mtile + half * hw;      // they lie in one 128-column block of scales
      const bool row_ok = row < t.row_end, cols_ok = col0 < p.m;
      const float* sx = p.sx + (row_ok ? row : 0);
      const float* sw = p.sw + static_cast<int64_t>(t.group) * p.num_kb * p.sw_cols + (cols_ok ? col0 / 128 : 0);
      const uint32_t base = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(half * hw);
      uint64_t sum[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) sum[i] = 0;
      float nx = ldg_f32_pinned(sx), nw = ldg_f32_pinned(sw);  // scales, loaded one block ahead
      for (int kb = 0; kb < p.num_kb; ++kb, ++acc_i) {
        const uint32_t acc = acc_i & 1u;
        const float s = nx * nw;
        if (kb + 1 < p.num_kb) {
          sx += p.lds;
          sw += p.sw_cols;
          nx = ldg_f32_pinned(sx);
          nw = ldg_f32_pinned(sw);
        }
        const uint64_t s2 = pack_u64(__float_as_uint(s), __float_as_uint(s));
        if (!mbar_wait(&tfull[acc], (acc_i >> 1) & 1u, abort_flag, kDevErrTimeoutEpilogue)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // 32 columns at a time, the next 32 on their way (a narrow piece reads past
        // its columns, inside the accumulator; those sums are not stored)
        uint32_t r[2][32];
        tmem_ld32(base + acc * 256, r[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tmem_ld_wait();
          if (c < 3) {
            tmem_ld32(base + acc * 256 + (c + 1) * 32, r[(c + 1) & 1]);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if (rank == 0) mbar_arrive(&tempty[acc]);
              else mbar_arrive_cluster_relaxed(tempty_even + 8u * acc);
            }
          }
#pragma unroll
          for (int e = 0; e < 16; ++e)
            sum[c * 16 + e] = grouped_fma2(pack_u64(r[c & 1][2 * e], r[c & 1][2 * e + 1]), s2, sum[c * 16 + e]);
        }
      }
      if (!ok) break;
      if (row_ok) {
        uint16_t* y = p.Y + static_cast<int64_t>(row) * p.ldy + col0;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const int left = min(hw, p.m - col0) - c * 8;  // columns of this 16-byte piece that exist
          if (left <= 0) break;
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint64_t v = sum[c * 4 + e];
            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(static_cast<uint32_t>(v)),
                                                           __uint_as_float(static_cast<uint32_t>(v >> 32)));
            w[e] = *reinterpret_cast<const uint32_t*>(&b);
          }
          if (left >= 8) {
            *reinterpret_cast<uint4*>(y + c * 8) = make_uint4(w[0], w[1], w[2], w[3]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (e < left) y[c * 8 + e] = static_cast<uint16_t>(w[e >> 1] >> ((e & 1) * 16));
          }
        }
      }
    }
  }

  tc_fence_before();
  cluster_sync();  // both CTAs are done with every MMA, copy and accumulator
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

}  // namespace rmm
