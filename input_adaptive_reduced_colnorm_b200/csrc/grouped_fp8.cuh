// The e4m3 product with block scales for groups of many rows (see grouped.cuh for
// the formula and the group bounds): tiles of 128 rows of X x 256 columns of W, rows
// on the M side.
//
// Why not swapped as the narrow tiles: every 128-deep block's accumulator passes
// through the epilogue threads, 128 x 256 fp32, while the tensor cores spend 512
// cycles on the next one.  With rows of X on the lanes a thread's 128 columns share
// ONE scale (its row's times the weight block's), kept in a register, and tensor
// memory is read in the 32 x 32-bit shape (128 bytes per cycle and warp scheduler:
// 256 of the 512 cycles; the 16 x 256-bit shape that the swapped form needs reads half
// as fast, 546 cycles).  What it costs is a group's last tile, 128 rows however few
// are left.  One CTA, not a pair: a pair stages a third less (32 KB a block and CTA
// against 48), but its accumulators' round trip is longer, and its 256-row tiles leave
// more of a group's last one empty (measured when the choice was made: 1024 x 4096 x
// 14336 of 8 groups 123 us against 152; 8192 x 4096 x 14336 of 8 566 against 600;
// 8192 x 8192 x 8192 635 against 625).
//
// A block's product is issued as two of half the columns with barriers of their
// own, so that the two epilogue warps of a scheduler work out of step (one loads
// and waits while the other multiplies); each takes the next block's first columns
// out of tensor memory before it adds the last ones of this block.
//
// 4096 x 4096 x 14336: 234-284 us, 1690-2060 TFLOP/s at 1.36-1.6 GHz (the power cap);
// 840-910 cycles a block, tile changes included, where the product takes 512.  The
// product cannot bound this tile: staging alone (48 KB a block; copies alone reach 77
// bytes a cycle) takes some 640.  Nor does one other thing: of 880 cycles a quarter of
// the products left 850, no additions 790, neither 730 -- staging and the accumulators'
// round trip (product, commit, epilogue, hand-back) on the two accumulators of 256
// columns that tensor memory holds; ~2500 cycles a tile.  The power cap takes the rest:
// 8192 x 14336 x 4096 of 8 runs at 866 cycles a block and 1.57 GHz in a burst (503 us),
// at 848 and 1.31 GHz for seconds (576 us).
//
// Roles (384 threads): warp 0 TMA producer, warps 1 and 2 MMA issuers, one for each
// product, warps 4-11 epilogue: warp w reads lanes 32 (w % 4) .. + 31 of one of the two
// products.  Results go through 4 KB of shared memory per warp: 32 rows x 64 columns
// that all belong to the group and the matrix leave as one TMA store, others row by
// row, 128 bytes at a time.  The tiles of a partial last wave are cut along W into
// 128- or 64-column pieces.
#pragma once
#include "grouped.cuh"

namespace rmm {

struct GroupedFp8Cfg {
  static constexpr int X_BYTES = 128 * 128;  // 128 rows x 128 contraction indices
  static constexpr int W_BYTES = 256 * 128;  // 128 contraction indices x 256 columns, two boxes of 128
  static constexpr int STAGES = 3;           // (four measured the same)
  static constexpr int OUT_BYTES = 8 * 32 * 128;  // 32 rows x 64 bf16 columns for each epilogue warp
  static constexpr int THREADS = 384;
  // registers per thread at launch, and the split after the set-up: 128 sums and
  // two 32-column loads in flight per epilogue thread (the host checks that the
  // kernel was compiled to LAUNCH_REGS, on which the split draws)
  static constexpr int LAUNCH_REGS = 168, OTHER_REGS = 40, EPI_REGS = 232;
  static_assert(OTHER_REGS + 2 * EPI_REGS <= 3 * LAUNCH_REGS, "three warpgroups share what was launched");
  static int smem_bytes(int groups) { return 1024 + STAGES * (X_BYTES + W_BYTES) + OUT_BYTES + 256 + (2 * groups + 2) * 4; }
  static_assert(8 * (2 * STAGES + 9) + 8 <= 256, "barrier area");
};

// sum[0..15] += v[0..15] * s between the question whether a phase of a barrier is
// complete and its answer, which takes some 200 cycles even when it is.
__device__ __forceinline__ uint32_t test_wait_fma16(uint32_t bar, uint32_t parity, float* sum, const uint32_t (&v)[16], float s) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%17], %18;\n\t"
      "fma.rn.f32 %1, %19, %35, %1;\n\tfma.rn.f32 %2, %20, %35, %2;\n\t"
      "fma.rn.f32 %3, %21, %35, %3;\n\tfma.rn.f32 %4, %22, %35, %4;\n\t"
      "fma.rn.f32 %5, %23, %35, %5;\n\tfma.rn.f32 %6, %24, %35, %6;\n\t"
      "fma.rn.f32 %7, %25, %35, %7;\n\tfma.rn.f32 %8, %26, %35, %8;\n\t"
      "fma.rn.f32 %9, %27, %35, %9;\n\tfma.rn.f32 %10, %28, %35, %10;\n\t"
      "fma.rn.f32 %11, %29, %35, %11;\n\tfma.rn.f32 %12, %30, %35, %12;\n\t"
      "fma.rn.f32 %13, %31, %35, %13;\n\tfma.rn.f32 %14, %32, %35, %14;\n\t"
      "fma.rn.f32 %15, %33, %35, %15;\n\tfma.rn.f32 %16, %34, %35, %16;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok), "+f"(sum[0]), "+f"(sum[1]), "+f"(sum[2]), "+f"(sum[3]), "+f"(sum[4]), "+f"(sum[5]), "+f"(sum[6]),
        "+f"(sum[7]), "+f"(sum[8]), "+f"(sum[9]), "+f"(sum[10]), "+f"(sum[11]), "+f"(sum[12]), "+f"(sum[13]),
        "+f"(sum[14]), "+f"(sum[15])
      : "r"(bar), "r"(parity), "f"(__uint_as_float(v[0])), "f"(__uint_as_float(v[1])), "f"(__uint_as_float(v[2])),
        "f"(__uint_as_float(v[3])), "f"(__uint_as_float(v[4])), "f"(__uint_as_float(v[5])), "f"(__uint_as_float(v[6])),
        "f"(__uint_as_float(v[7])), "f"(__uint_as_float(v[8])), "f"(__uint_as_float(v[9])), "f"(__uint_as_float(v[10])),
        "f"(__uint_as_float(v[11])), "f"(__uint_as_float(v[12])), "f"(__uint_as_float(v[13])),
        "f"(__uint_as_float(v[14])), "f"(__uint_as_float(v[15])), "f"(s)
      : "memory");
  return ok;
}

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
    t.row0 = off[lo] + (r % rt) * 128;
    t.row_end = off[lo + 1];
    return t;
  }
};

__global__ void __launch_bounds__(GroupedFp8Cfg::THREADS, 1)
    grouped_fp8_rows_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                            const __grid_constant__ CUtensorMap tmY, const GroupedParams p) {
  using C = GroupedFp8Cfg;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t grouped_fp8_smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(grouped_fp8_smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sX = smem;
  uint8_t* sW = smem + STAGES * C::X_BYTES;
  uint8_t* sOut = sW + STAGES * C::W_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(sOut + C::OUT_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 4;  // both [accumulator][half]
  uint64_t* drain = tempty + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* off = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(full) + 256);
  int* pre = off + p.groups + 1;

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int worker = static_cast<int>(blockIdx.x), workers = static_cast<int>(gridDim.x);
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], p.expire_producer_waits ? 3 : 2);  // both issuers
    }
    for (int a = 0; a < 4; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 4);  // four epilogue warps
    }
    mbar_init(drain, 2);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&tmW);
    prefetch_tensormap(&tmX);
    prefetch_tensormap(&tmY);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  wait_prior_kernels();  // bounds, operands and the output are touched only after this
  grouped_bounds<128>(p, off, pre, warp, lane);
  tc_fence_before();
  __syncthreads();  // barriers initialised, bounds there, tensor memory allocated
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const GroupedFp8Units units(p, off, pre, workers);

  if (warp < 4) set_max_regs_down<C::OTHER_REGS>();
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // (elected lane of a warp that runs the loop together, as below)
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    const uint64_t limit_ns = p.expire_producer_waits ? kGroupedHookWaitNs : kWaitTimeoutNs;
    bool ok = true;
    for (int unit = worker; ok && unit < units.count; unit += workers) {
      const GroupedTile t = units.get(unit);
      for (int kb = 0; kb < p.num_kb; ++kb) {
        if (!__all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1u, abort_flag, kDevErrTimeoutProducer, 0, kMbarCta,
                                               limit_ns))) {
          ok = false;
          break;
        }
        if (elect_one()) {
          // (a narrow piece's columns are all in the first box of W)
          mbar_arrive_expect_tx(&full[stage], C::X_BYTES + (t.w == 256 ? C::W_BYTES : C::W_BYTES / 2));
          uint8_t* w = sW + stage * C::W_BYTES;
          tma_load_2d(sX + stage * C::X_BYTES, &tmX, &full[stage], kb * 128, t.row0);
          tma_load_3d(w, &tmW, &full[stage], t.mtile, kb * 128, t.group);
          if (t.w == 256) tma_load_3d(w + 16384, &tmW, &full[stage], t.mtile + 128, kb * 128, t.group);
        }
        ++issued;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) {
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
    __syncwarp();
  } else if (warp <= 2) {
    // ------------------------------------------------------------ MMA issuers
    // warp 1 issues the product of the first half of the columns, warp 2 that of the
    // second (one warp's waits for both, 3 of about 100 cycles a block, left the
    // tensor cores idle).  The warp runs the loop together and elects the issuing
    // lane, so that the descriptors stay in uniform registers.
    const int h = warp - 1;
    const uint64_t xd0 = make_sw128_desc(smem_u32(sX), 16, 1024), wd0 = make_sw128_desc(smem_u32(sW), 16384, 1024);
    int stage = 0;
    uint32_t phase = 0, acc_i = 0;
    bool ok = true;
    for (int unit = worker; ok && unit < units.count; unit += workers) {
      const int w = units.get(unit).w;
      const uint32_t idesc = make_idesc_e4m3(128, 0, 0, 1) | (static_cast<uint32_t>(w >> 4) << 17);  // N = w / 2
      const int first = w == 256 ? h * 16384 : h * (w >> 1);  // a piece's columns are all in the first box
      for (int kb = 0; kb < p.num_kb; ++kb, ++acc_i) {
        const uint32_t buf = (acc_i & 1u) * 2 + h;
        const uint64_t xd = xd0 + static_cast<uint64_t>(stage * (C::X_BYTES >> 4));
        const uint64_t wd = wd0 + static_cast<uint64_t>((stage * C::W_BYTES + first) >> 4);
        // (the operands are there long before the accumulator: asked first, off the
        // path from one block's epilogue to the next but one's product)
        const bool go = mbar_wait(&full[stage], phase, abort_flag, kDevErrTimeoutMma) &&
                        mbar_wait(&tempty[buf], ((acc_i >> 1) & 1u) ^ 1u, abort_flag, kDevErrTimeoutMma);
        if (!__all_sync(0xffffffffu, go)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_e4m3(tmem_base + buf * 128, xd + static_cast<uint64_t>(kk * (32 >> 4)),
                      wd + static_cast<uint64_t>(kk * (4096 >> 4)), idesc, kk != 0 ? 1u : 0u);
          umma_commit(&tfull[buf]);
          umma_commit(&empty[stage]);
        }
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (elect_one()) {
      // every MMA issued by this warp is complete once `drain` flips
      umma_commit(drain);
      const uint32_t a = smem_u32(drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(a, 0) && globaltimer_ns() - t0 < kWaitTimeoutNs) {
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    set_max_regs_up<C::EPI_REGS>();
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t base = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(half * 128);
    uint8_t* out = sOut + (warp - 4) * 4096;
    uint32_t acc_i = 0;
    bool ok = true;
    // the tile at hand; the scale s of its next block and the row's of the two after;
    // the weight blocks' scales of 32 blocks and of the 32 after, one per lane (uniform
    // over the warp, they are passed on by shuffles: a load a block less)
    GroupedTile t;
    const float *px = nullptr, *pw = nullptr;
    float s, x1, x2, u, u_next;
    auto next_x = [&](int kb) {  // of block kb; past the last one its own again
      const float x = ld_f32_pinned(px);
      px += kb + 1 < p.num_kb ? p.lds : 0;
      return x;
    };
    auto load_w = [&](int kb) {  // of blocks kb .. kb + 31
      u_next = ld_f32_pinned(pw + static_cast<int64_t>(min(kb + lane, p.num_kb - 1)) * p.sw_cols);
    };
    auto begin = [&](int unit) {
      t = units.get(unit);
      const int row = t.row0 + quarter * 32 + lane;
      px = p.sx + (row < t.row_end ? row : 0);
      // this warp's columns lie in one 128-column block of scales (past the edge: any)
      const int block = min((t.mtile + half * (t.w / 2)) / 128, p.sw_cols - 1);
      pw = p.sw + static_cast<int64_t>(t.group) * p.num_kb * p.sw_cols + block;
      s = next_x(0);
      x1 = next_x(1);
      x2 = next_x(2);
      load_w(0);
    };
    if (worker < units.count) begin(worker);
    for (int unit = worker; unit < units.count; unit += workers) {
      u = u_next;
      s *= __shfl_sync(0xffffffffu, u, 0);
      if (p.num_kb > 32) load_w(32);
      float sum[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) sum[i] = 0.f;
      uint32_t r[2][16];
      ok = __all_sync(0xffffffffu, mbar_wait(&tfull[(acc_i & 1u) * 2 + half], (acc_i >> 1) & 1u, abort_flag,
                                             kDevErrTimeoutEpilogue));
      if (!ok) break;
      tc_fence_after();
      tmem_ld16(base + (acc_i & 1u) * 256, r[0]);
      for (int kb = 0; ok && kb < p.num_kb; ++kb) {
        const uint32_t acc = acc_i & 1u;
        ++acc_i;
        if ((kb & 31) == 31) {
          u = u_next;
          if (kb + 33 < p.num_kb) load_w(kb + 33);
        }
        float s_next = 0.f;
        // 16 columns at a time, the next 16 on their way (a narrow piece reads past
        // its columns, inside the accumulator; those sums are not stored).  The
        // loads stand outside every branch, and the additions keep their place:
        // left to itself the compiler moved them past the waits, 1.2x the time.
        uint64_t* next_full = &tfull[(acc ^ 1u) * 2 + half];
        uint32_t ready = 0;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          tmem_ld_wait();
          if (c < 7) {
            tmem_ld16(base + acc * 256 + (c + 1) * 16, r[(c + 1) & 1]);
            if (c == 1) s_next = x1 * __shfl_sync(0xffffffffu, u, (kb + 1) & 31);
            if (c == 3) {
              x1 = x2;
              x2 = next_x(kb + 3);
            }
          } else {
            tc_fence_before();
            __syncwarp();
            if (elect_one()) mbar_arrive(&tempty[acc * 2 + half]);
            if (kb + 1 < p.num_kb && __any_sync(0xffffffffu, !ready))
              ok = __all_sync(0xffffffffu, mbar_wait(next_full, (acc_i >> 1) & 1u, abort_flag, kDevErrTimeoutEpilogue));
            tc_fence_after();
            tmem_ld16(base + (acc ^ 1u) * 256, r[0]);  // (after the last block: not used)
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            if (c == 5 && e == 0) ready = test_wait_fma16(smem_u32(next_full), (acc_i >> 1) & 1u, &sum[c * 16], r[c & 1], s);
            if (c != 5) fma_pinned(sum[c * 16 + e], __uint_as_float(r[c & 1][e]), s);
          }
        }
        s = s_next;
      }
      tmem_ld_wait();
      if (!ok) break;
      const int hw = t.w / 2;                 // this warp's columns: 128, 64 or 32
      const int col0 = t.mtile + half * hw;
      const int row0 = t.row0 + quarter * 32;
      const int row_end = t.row_end;
#pragma unroll
      for (int q = 0; q < 2; ++q) {  // columns 64 q .. 64 q + 63 of them
        if (q == 1) {
          // the next tile's scales come while this one is written
          if (unit + workers < units.count) begin(unit + workers);
          if (hw <= 64) break;
        }
        if (lane == 0) bulk_wait_group_read<0>();  // the last store has left the buffer
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(sum[q * 64 + k * 8 + 2 * e], sum[q * 64 + k * 8 + 2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t*>(&b);
          }
          *reinterpret_cast<uint4*>(out + lane * 128 + ((k ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        // (a store that crosses column m would write zeros up to the next 16 bytes)
        const int first = col0 + q * 64;
        if (hw >= 64 && row0 + 32 <= row_end && first + 64 <= p.m) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&tmY, out, first, row0, 0);
            bulk_commit_group();
          }
          continue;
        }
        __syncwarp();
        const int k = lane & 7;  // 8 columns of this thread's rows lane / 8, + 4, ...
        const int col = first + k * 8;
        const int left = q * 64 + k * 8 < hw ? p.m - col : 0;  // columns that exist
#pragma unroll
        for (int it = 0; it < 8; ++it) {
          const int i = it * 4 + (lane >> 3);
          const uint4 v = *reinterpret_cast<const uint4*>(out + i * 128 + ((k ^ (i & 7)) << 4));
          if (row0 + i < row_end && left > 0) {
            uint16_t* y = p.Y + static_cast<int64_t>(row0 + i) * p.ldy + col;
            if (left >= 8) {
              *reinterpret_cast<uint4*>(y) = v;
            } else {
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (e < left) y[e] = static_cast<uint16_t>(w[e >> 1] >> ((e & 1) * 16));
            }
          }
        }
      }
    }
    if (lane == 0) bulk_wait_group<0>();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();  // every MMA, copy and accumulator is done with
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

}  // namespace rmm
