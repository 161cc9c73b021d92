// Products grouped by expert, in bf16 and in e4m3 with block scales:
//   Y[i, :] = X[i, :] . W[e]          for offsets[e] <= i < offsets[e + 1]
// with W[e] d x m (contraction index as the row).  With e4m3 operands
//   Y[i, c] = sum_b sx[b, i] sw[e, b, c / 128] sum_{j in block b} X[i, j] W[e][j, c],
// b running over blocks of 128 contraction indices.  A plain product is the case
// of one group.
//
// The operands are swapped, D = W^T X^T: the weights' columns fill the M side of
// the tensor cores (128 lanes of tensor memory), the rows of X the N side, whose
// width (16 to 256) follows the rows an expert has.  With the rows on the M side
// an expert with 4 rows would pay for 128.
//
// A stage holds 128 bytes of the contraction (64 bf16 or 128 e4m3 indices) for
// MT x 128 columns of W (MN-major, 128-byte swizzle) and N rows of X (K-major),
// brought by TMA; what lies past a matrix's edge reads as zeros.  A tile's rows
// past its group's end belong to the next group: they are multiplied, not stored.
//
// Block scales: each 128-deep block gets an accumulator of its own (of two), and
// the epilogue threads add it, scaled, into fp32 registers.  They read tensor
// memory in the 16 x 256-bit shape: a thread gets 2 neighbouring rows of X for 4
// columns of W out of each 8 x 32, so one pair of row scales (times the weight
// block's, kept by each warp in shared memory) serves 4 packed multiply-adds.
// (With a lane's whole row per thread, every multiply-add needed a scale of its own
// from shared memory, twice the time of the block's tensor work; 380 TFLOP/s at
// 4096 x 4096 x 14336, on tiles of 256 x 256.)
//
// Bound by HBM with few rows (bf16 64 x 4096 x 14336 of 8 groups: 139 us, the copy
// bandwidth; e4m3 8 x 8192 x 28672: 40-41 us, 0.88 of it) and by the tensor cores at the
// power cap with many (8192 x 4096 x 14336 of 8: 690-890 us, 530 cycles a stage of
// 512 at 1.3-1.45 GHz).
//
// Tiles are cut to the rows that are there: the N of a tile's instructions is
// its row count rounded up to 16 (32 for a pair), and one CTA copies only the runs of
// 32 rows that hold some (a pair copies all: with four copies of 32 rows in place of one
// 2048 x 4096 x 14336 of 8 took 1.3 times as long).  When the tiles do not fill a whole
// number of waves, those of the last wave are cut into narrower ones.
//
// Few tiles (decoding): the contraction of a tile is split over the 2 to 8 CTAs of
// a cluster; they leave their fp32 sums in shared memory and each adds up, in the
// order of the ranks, some of the columns of all of them (no atomics, no workspace,
// the same result every time).
//
// Group bounds are read on the device (the call does not synchronise): every CTA
// clamps them to 0 <= ... <= n, non-decreasing, and sums the row tiles of the
// groups before it starts; a tile number is looked up by bisection.
//
// Roles: warp 0 TMA producer, warp 1 (and for e4m3 the last warp) MMA issuer, warps from
// 2 on epilogue: 8, and 16 for the e4m3 tiles of 128 accumulator columns, whose every
// block goes through them (64 x 4096 x 14336: 17.4 us, 0.82 of the time with 8; 4096 x
// 2048 x 1408 of 64 groups 46 against 48; each waits for its loads of tensor memory, and two
// warps a scheduler do not cover that).  CG = 2 (bf16): two CTAs of a cluster form one
// M = 256 product (256 columns of W x 256 rows of X), each staging its own 128 columns of
// W and half of the rows.
//
// Every role asks after a wait whether all its lanes had it fulfilled: when one runs
// out, lanes may see the barrier, the timer and the abort word at different polls, and a
// warp of which some lanes left would hang in its next shuffle or tensor-memory load.
#pragma once
#include <cuda_bf16.h>
#include "ptx.cuh"

namespace rmm {

constexpr int kGroupedMaxGroups = 1024;

struct GroupedParams {
  const int32_t* offsets;  // [groups + 1] on the device, or null: one group of n rows
  int groups;
  int n, m;
  int num_kb;              // 128-byte blocks of the contraction
  int m_tiles;             // tiles of CG * MT * 128 columns
  int splits;              // CTAs of a cluster that share one tile's contraction (CG = 1); 1: none
  uint16_t* Y;
  int64_t ldy;
  // block scales (e4m3)
  const float* sx;         // [num_kb][lds]
  int64_t lds;
  const float* sw;         // [groups][num_kb][sw_cols]
  int sw_cols;
  // test hook (0 in every product call): 1 makes the barriers of empty stages expect one
  // arrival more than they get and limits the producers' waits to 1 ms, so that the wait
  // for a stage's second use runs out and the kernel takes its timeout path
  int expire_producer_waits;
};

constexpr uint64_t kGroupedHookWaitNs = 1000ull * 1000ull;

template <bool FP8, int N, int MT, int CG, int OCC>
struct GroupedCfg {
  static constexpr int A_BYTES = MT * 128 * 128;
  static constexpr int X_ROWS = N / CG;
  static constexpr int X_BYTES = X_ROWS * 128;
  static constexpr int X_BOX = CG == 1 && X_ROWS > 32 ? 32 : X_ROWS;  // rows of a copy
  static constexpr int COLS = MT * N;          // accumulator columns of one tile
  static constexpr int EW = FP8 && COLS >= 128 ? 16 : 8;  // epilogue warps
  static constexpr int THREADS = (2 + EW + (FP8 ? 1 : 0)) * 32;
  static constexpr int HC = COLS / (EW / 4);   // columns of one epilogue thread
  static constexpr int TMEM_COLS = 2 * COLS;
  static constexpr int SCALE_BYTES = FP8 ? EW * 2 * HC * 4 : 0;
  static constexpr int OUT_BYTES = EW * 512;   // results on their way, 512 bytes per epilogue warp
  // OCC CTAs share an SM (with the bounds of up to 128 groups; more lower it to one)
  static constexpr int BOUND_GROUPS = OCC == 1 ? kGroupedMaxGroups : 128;
  static constexpr int STAGES_FIT =
      (233472 / OCC - 1024 - 1024 - 256 - SCALE_BYTES - OUT_BYTES - (2 * BOUND_GROUPS + 2) * 4) / (A_BYTES + X_BYTES);
  static constexpr int STAGES = STAGES_FIT > 8 ? 8 : STAGES_FIT;
  static_assert(!(FP8 && CG == 2), "pairs are bf16's (see grouped_fp8.cuh for the e4m3 tiles of large groups)");
  static_assert(STAGES >= 3, "at least three stages");
  static_assert(TMEM_COLS >= 32 && TMEM_COLS <= 512 && (TMEM_COLS & (TMEM_COLS - 1)) == 0, "tensor memory");
  static_assert(8 * (2 * STAGES + 5) + 8 <= 256, "barrier area");
  static int smem_bytes(int groups) {
    return 1024 + STAGES * (A_BYTES + X_BYTES) + SCALE_BYTES + OUT_BYTES + 256 + (2 * groups + 2) * 4;
  }
};

// Clamped group bounds off[0..groups] and the running count of N-row tiles
// pre[0..groups], by the whole CTA: all bounds are fetched at once, then one warp
// scans them, a run of neighbours per lane (fetched by the scan, 32 at a time, 114
// groups cost 5 us).
template <int N>
__device__ __forceinline__ void grouped_bounds(const GroupedParams& p, int* off, int* pre, int warp, int lane) {
  if (p.offsets == nullptr) {
    if (threadIdx.x == 0) {
      off[0] = 0;
      off[1] = p.n;
      pre[0] = 0;
      pre[1] = (p.n + N - 1) / N;
    }
    return;
  }
  for (int i = threadIdx.x; i <= p.groups; i += blockDim.x) off[i] = min(max(p.offsets[i], 0), p.n);
  __syncthreads();
  if (warp != 2) return;
  const int run = (p.groups + 32) / 32;  // entries per lane of groups + 1
  const int lo = min(lane * run, p.groups + 1), hi = min(lo + run, p.groups + 1);
  int top = 0;  // the largest bound so far: this lane's, then with those of the lanes before
  for (int i = lo; i < hi; ++i) top = max(top, off[i]);
#pragma unroll
  for (int s = 1; s < 32; s *= 2) {
    const int u = __shfl_up_sync(0xffffffffu, top, s);
    if (lane >= s) top = max(top, u);
  }
  top = __shfl_up_sync(0xffffffffu, top, 1);
  if (lane == 0) top = 0;
  int tiles = 0, last = top;  // of the groups that end at this lane's bounds
  for (int i = lo; i < hi; ++i) {
    const int v = max(off[i], last);
    off[i] = v;
    if (i > 0) tiles += (v - last + N - 1) / N;
    last = v;
    pre[i] = tiles;
  }
  int before = tiles;
#pragma unroll
  for (int s = 1; s < 32; s *= 2) {
    const int u = __shfl_up_sync(0xffffffffu, before, s);
    if (lane >= s) before += u;
  }
  before -= tiles;
  for (int i = lo; i < hi; ++i) pre[i] += before;
}

// One piece of work: rows [row0, row_end) (at most w of them) of group `group`
// times column tile mtile of its weights.
struct GroupedTile {
  int group, row0, row_end, mtile, w;
};

// The tiles of a call as units of work.  Tile order: group, then column tile,
// then row tile fastest, so that the row tiles of one piece of the weights run
// side by side and share it through L2.  The tiles past the last whole wave are
// cut into `cut` pieces of N / cut rows where that lets more workers take part.
template <int N, int CG>
struct GroupedUnits {
  const int *off, *pre;
  int groups, m_tiles, whole, cut, count;
  __device__ __forceinline__ GroupedUnits(const GroupedParams& p, const int* off_, const int* pre_, int workers)
      : off(off_), pre(pre_), groups(p.groups), m_tiles(p.m_tiles), cut(1) {
    const int tiles = pre[groups] * m_tiles;
    const int rest = tiles % workers;
    if (N >= 128 && rest > 0)
      while (N / cut > 32 * CG && 2 * cut * rest <= workers) cut *= 2;
    whole = tiles - rest;
    count = whole + rest * cut;
  }
  __device__ __forceinline__ GroupedTile get(int unit) const {
    int tile = unit, part = 0;
    if (N >= 128 && unit >= whole) {
      tile = whole + (unit - whole) / cut;
      part = (unit - whole) % cut;
    }
    const int width = (N >= 128 && unit >= whole) ? N / cut : N;
    int lo = 0, hi = groups - 1;  // the last group whose first tile is <= tile
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] * m_tiles <= tile) lo = mid;
      else hi = mid - 1;
    }
    const int rt = pre[lo + 1] - pre[lo];
    const int r = tile - pre[lo] * m_tiles;
    GroupedTile t;
    t.group = lo;
    t.mtile = r / rt;
    t.row0 = off[lo] + (r - t.mtile * rt) * N + part * width;
    t.row_end = min(off[lo + 1], t.row0 + width);
    constexpr int STEP = 16 * CG;
    t.w = t.row_end > t.row0 ? (t.row_end - t.row0 + STEP - 1) / STEP * STEP : 0;
    return t;
  }
};

__device__ __forceinline__ uint64_t grouped_fma2(uint64_t a, uint64_t b, uint64_t c) {  // a * b + c, two fp32
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t pack_u64(uint32_t lo, uint32_t hi) {
  return static_cast<uint64_t>(lo) | (static_cast<uint64_t>(hi) << 32);
}

// 16 lanes x 16 columns of tensor memory: thread T gets lanes T / 4 (r[0], r[1],
// r[4], r[5]) and T / 4 + 8 (r[2], r[3], r[6], r[7]), columns 2 (T % 4) + {0, 1}
// of the first (r[0..3]) and second (r[4..7]) eight.
__device__ __forceinline__ void tmem_ld_16x16(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}

// Writes an 8-row x 32-column piece of Y.  v[j]: fp32 pairs of columns T / 4 + 8 j
// of W for rows 2 (T % 4) + {0, 1} of X.  Rounded to bf16 and transposed on their
// way to 512 bytes of shared memory of this warp (`buf`), read back as 8
// neighbouring columns of row T / 4 per thread: one 16-byte store, 64 bytes of a row
// per four threads.  (Transposed by moves and shuffles inside the warp instead, it
// took three times the instructions.)
__device__ __forceinline__ void grouped_store(const GroupedParams& p, uint8_t* buf, const uint64_t (&v)[4], int row_base,
                                              int row_end, int col_base, int lane) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(__uint_as_float(static_cast<uint32_t>(v[j])),
                                                   __uint_as_float(static_cast<uint32_t>(v[j] >> 32)));
    w[j] = *reinterpret_cast<const uint32_t*>(&t);
  }
  // 8 x 8 matrix j: lane 8 j + i names where its i-th row of X goes; a row's four
  // 16-byte columns are rotated by half the row number, against bank conflicts
  const int i = lane & 7, j = lane >> 3;
  const uint32_t at = smem_u32(buf) + static_cast<uint32_t>(i * 64 + (((j + (i >> 1)) & 3) << 4));
  __syncwarp();  // the last piece has been read
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3])
               : "memory");
  __syncwarp();
  const int r = lane >> 2, q = lane & 3;
  const uint4 x = lds_v4(smem_u32(buf) + static_cast<uint32_t>(r * 64 + (((q + (r >> 1)) & 3) << 4)));
  const int row = row_base + r;
  const int col = col_base + q * 8;
  if (row < row_end && col < p.m) {
    uint16_t* y = p.Y + static_cast<int64_t>(row) * p.ldy + col;
    if (col + 8 <= p.m) {
      *reinterpret_cast<uint4*>(y) = x;
    } else {
      const uint32_t c[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (col + e < p.m) y[e] = static_cast<uint16_t>(c[e >> 1] >> ((e & 1) * 16));
    }
  }
}

// Row of the tile and 128-column tile of W of accumulator column share * HC + i (one
// of HC and N is a multiple of the other).
template <int N, int HC>
__device__ __forceinline__ int grouped_r(int share, int i) {
  return HC >= N ? i % N : share % (N / HC > 0 ? N / HC : 1) * HC + i;
}
template <int N, int HC>
__device__ __forceinline__ int grouped_mt(int share, int i) {
  return HC >= N ? share * (HC / N) + i / N : share / (N / HC > 0 ? N / HC : 1);
}

template <bool FP8, int N, int MT, int CG, int OCC>
__global__ void __launch_bounds__(GroupedCfg<FP8, N, MT, CG, OCC>::THREADS, OCC)
    grouped_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                   const GroupedParams p) {
  using C = GroupedCfg<FP8, N, MT, CG, OCC>;
  constexpr int STAGES = C::STAGES, HC = C::HC, EW = C::EW;
  constexpr int BK = FP8 ? 128 : 64;
  // the instructions' N is set per tile
  constexpr uint32_t IDESC0 = FP8 ? make_idesc_e4m3(128 * CG, 0, 1, 0) : make_idesc_bf16(128 * CG, 0, 1, 0);
  // bytes between the k-steps of W in a stage (16 bf16 or 32 e4m3 rows of 128 bytes)
  constexpr uint32_t A_STEP = FP8 ? 4096 : 2048;

  extern __shared__ uint8_t grouped_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(grouped_smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sX = smem + STAGES * C::A_BYTES;
  float* sScale = reinterpret_cast<float*>(sX + STAGES * C::X_BYTES);  // [EW warps][2][HC]
  uint8_t* sOut = reinterpret_cast<uint8_t*>(sScale) + C::SCALE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(sOut + C::OUT_BYTES);  // even CTA
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;  // even CTA
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* off = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(full) + 256);
  int* pre = off + p.groups + 1;

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;  // 0: the CTA that issues the MMAs
  const int splits = CG == 2 ? 1 : p.splits;
  const uint32_t part = splits > 1 ? cluster_ctarank() : 0u;
  // with splits every cluster has one tile at most
  const int worker = static_cast<int>(blockIdx.x) / (CG * splits), workers = static_cast<int>(gridDim.x) / (CG * splits);
  const int kb_begin = splits > 1 ? static_cast<int>(static_cast<int64_t>(part) * p.num_kb / splits) : 0;
  const int kb_end = splits > 1 ? static_cast<int>(static_cast<int64_t>(part + 1) * p.num_kb / splits) : p.num_kb;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], p.expire_producer_waits ? 2 : 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], EW * CG);
    }
    mbar_init(drain, FP8 ? 2 : 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&tmW);
    prefetch_tensormap(&tmX);
  }
  if (warp == 1) {
    if (CG == 2) {
      tmem_alloc_pair(tmem_slot, C::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, C::TMEM_COLS);
      tmem_relinquish();
    }
  }
  wait_prior_kernels();  // bounds, operands and the output are touched only after this
  grouped_bounds<N>(p, off, pre, warp, lane);
  tc_fence_before();
  if (CG == 2) cluster_sync();  // barriers of both CTAs initialised, tensor memory allocated
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const GroupedUnits<N, CG> units(p, off, pre, workers);

  if (warp == 0) {
    // ------------------------------------------------------------ producer (both CTAs)
    // (the warp runs the loop together and elects the lane that issues, as the MMA
    // issuers do: the copies' operands then stay in uniform registers; bf16 1 x 4096 x
    // 14336 21.8 us against 22.4 with one lane in the loop, 1024 x 4096 x 14336 of 8 167
    // against 174, 1000 x 6000 x 500 of 20 53 against 58; 8192 x 4096 x 14336 of 8, at the
    // power cap for seconds, 795 and 794)
    const uint32_t full_even = CG == 2 ? map_shared_rank(smem_u32(&full[0]), 0u) : 0u;
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    const uint64_t limit_ns = p.expire_producer_waits ? kGroupedHookWaitNs : kWaitTimeoutNs;
    bool ok = true;
    for (int unit = worker; ok && unit < units.count; unit += workers) {
      const GroupedTile t = units.get(unit);
      if (t.w == 0) continue;
      const int f0 = (t.mtile * CG + static_cast<int>(rank)) * MT * 128;
      const int row = t.row0 + static_cast<int>(rank) * (t.w / 2);  // half of a pair's rows
      const int x_boxes = CG == 2 ? 1 : (t.w + C::X_BOX - 1) / C::X_BOX;  // those that hold rows of the tile
      for (int kb = kb_begin; kb < kb_end; ++kb) {
        if (!__all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1u, abort_flag, kDevErrTimeoutProducer, 0, kMbarCta,
                                               limit_ns))) {
          ok = false;
          break;
        }
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], CG * (C::A_BYTES + x_boxes * C::X_BOX * 128));
          uint8_t* a = sA + stage * C::A_BYTES;
          uint8_t* x = sX + stage * C::X_BYTES;
          constexpr int BOXES = FP8 ? MT : 2 * MT;     // boxes of 128 bytes of columns
          constexpr int BOX_COLS = FP8 ? 128 : 64;
          if (CG == 2) {
            const uint32_t bar = full_even + 8u * static_cast<uint32_t>(stage);
#pragma unroll
            for (int j = 0; j < BOXES; ++j)
              tma_load_3d_pair(a + j * (BK * 128), &tmW, bar, f0 + j * BOX_COLS, kb * BK, t.group);
            tma_load_2d_pair(x, &tmX, bar, kb * BK, row);
          } else {
#pragma unroll
            for (int j = 0; j < BOXES; ++j)
              tma_load_3d(a + j * (BK * 128), &tmW, &full[stage], f0 + j * BOX_COLS, kb * BK, t.group);
            for (int j = 0; j < x_boxes; ++j)
              tma_load_2d(x + j * (C::X_BOX * 128), &tmX, &full[stage], kb * BK, row + j * C::X_BOX);
          }
        }
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
    __syncwarp();
  } else if (warp == 1 || warp == 2 + EW) {
    // ------------------------------------------------------------ MMA issuers (even CTA)
    // e4m3: warp 1 issues the even blocks' products, the last warp the odd ones', each to an
    // accumulator of its own.  Issuing takes about as long as the products, and one
    // warp's waits between them (accumulator, operands: 400 cycles a block) would leave
    // the tensor cores idle.  bf16 adds to one accumulator and waits once a tile.
    // The warp runs the loop together and elects the issuing lane: the descriptors
    // then stay in uniform registers (with one lane in the loop an instruction took
    // 90 cycles to issue, with the warp 20).
    if (rank == 0) {
      const uint64_t ad0 = make_sw128_desc(smem_u32(sA), 8192, 1024), xd0 = make_sw128_desc(smem_u32(sX), 16, 1024);
      int stage = 0;
      uint32_t phase = 0;
      uint32_t acc_i = 0;
      bool ok = true;
      for (int unit = worker; ok && unit < units.count; unit += workers) {
        const int w = units.get(unit).w;
        if (w == 0) continue;
        const uint32_t idesc = IDESC0 | (static_cast<uint32_t>(w >> 3) << 17);
        for (int kb = kb_begin; kb < kb_end; ++kb) {
          const uint32_t acc = acc_i & 1u;
          if (FP8 && acc != (warp == 1 ? 0u : 1u)) {  // the other warp's
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
            ++acc_i;
            continue;
          }
          // The accumulator first: once the epilogue has handed back block kb - 2's, every
          // block up to it has been loaded and read, block kb - STAGES among them, so that
          // the stage's barrier is in this block's phase or past it when it is asked.  (A
          // warp that skips blocks and asks the stage first may meet the phase before the
          // last, whose parity is the same.)
          static_assert(STAGES > 2, "the stage's last block is before kb - 2");
          bool go = true;
          if (FP8 || kb == kb_begin)
            go = mbar_wait(&tempty[acc], ((acc_i >> 1) & 1u) ^ 1u, abort_flag, kDevErrTimeoutMma, 0,
                           CG == 2 ? kMbarClusterRelaxed : kMbarCta);
          go = go && mbar_wait(&full[stage], phase, abort_flag, kDevErrTimeoutMma);
          if (!__all_sync(0xffffffffu, go)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const bool last = FP8 || kb == kb_end - 1;
          if (elect_one()) {
            const uint32_t d_tmem = tmem_base + acc * C::COLS;
            const uint64_t ad = ad0 + static_cast<uint64_t>(stage * (C::A_BYTES >> 4));
            const uint64_t xd = xd0 + static_cast<uint64_t>(stage * (C::X_BYTES >> 4));
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint32_t add = (kk != 0 || (!FP8 && kb != kb_begin)) ? 1u : 0u;
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                const uint64_t am = ad + static_cast<uint64_t>((mt * 16384 + kk * A_STEP) >> 4);
                const uint64_t xm = xd + static_cast<uint64_t>((kk * 32) >> 4);
                const uint32_t d = d_tmem + static_cast<uint32_t>(mt * N);
                if (CG == 2) umma_bf16_pair(d, am, xm, idesc, add);
                else if (FP8) umma_e4m3(d, am, xm, idesc, add);
                else umma_bf16(d, am, xm, idesc, add);
              }
            }
            if (CG == 2) umma_commit_pair(&empty[stage], 0x3);
            else umma_commit(&empty[stage]);
            if (last) {
              if (CG == 2) umma_commit_pair(&tfull[acc], 0x3);
              else umma_commit(&tfull[acc]);
            }
          }
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
          if (last) ++acc_i;
        }
      }
      if (elect_one()) {
        // every MMA issued by this warp is complete once `drain` flips
        if (CG == 2) umma_commit_pair(drain, 0x1);
        else umma_commit(drain);
        const uint32_t a = smem_u32(drain);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(a, 0) && globaltimer_ns() - t0 < kWaitTimeoutNs) {
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int quarter = warp & 3;         // lanes of tensor memory a warp may read
    const int share = (warp - 2) >> 2;
    // this thread's accumulator columns [share * HC, share * HC + HC): rows r_of(i)
    // of the tile, columns of W in its 128-column tile mt_of(i)
    auto mt_of = [&](int i) { return grouped_mt<N, HC>(share, i); };
    auto r_of = [&](int i) { return grouped_r<N, HC>(share, i); };
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(share * HC);
    const uint32_t tempty_even = CG == 2 ? map_shared_rank(smem_u32(&tempty[0]), 0u) : 0u;
    float* my_scale = sScale + (warp - 2) * 2 * HC;
    uint8_t* out = sOut + (warp - 2) * 512;
    // this thread's sums with splits, [HC / 2][32 lanes] per warp, over the stages
    // (every copy and product of the one tile is complete when they are written)
    uint64_t* my_part = reinterpret_cast<uint64_t*>(smem) + (warp - 2) * (HC / 2) * 32 + lane;
    uint32_t acc_i = 0;
    bool ok = true;
    auto release = [&](uint32_t acc) {  // this warp has read the accumulator
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) mbar_arrive(&tempty[acc]);
        else mbar_arrive_cluster_relaxed(tempty_even + 8u * acc);
      }
    };
    for (int unit = worker; ok && unit < units.count; unit += workers) {
      const GroupedTile t = units.get(unit);
      if (t.w == 0) continue;
      const int mblock0 = (t.mtile * CG + static_cast<int>(rank)) * MT;  // first 128-column tile
      if (FP8) {
        // sum[g][j]: columns T / 4 + 8 j of the warp's 32, rows 8 g + 2 (T % 4) + {0, 1}
        uint64_t sum[HC / 8][4];
#pragma unroll
        for (int g = 0; g < HC / 8; ++g)
#pragma unroll
          for (int j = 0; j < 4; ++j) sum[g][j] = 0;
        // scales of this warp's HC rows (lane, lane + 32, ...) and of the weight
        // blocks, loaded two blocks ahead (a trip to L2 takes longer than a block)
        constexpr int SC = (HC + 31) / 32;
        float nx[2][SC], nw[2][SC];
        auto load_scales = [&](int kb, float (&nx)[SC], float (&nw)[SC]) {
#pragma unroll
          for (int i = 0; i < SC; ++i) {
            const int row = t.row0 + r_of(i * 32 + lane);
            const int mb = mblock0 + mt_of(i * 32 + lane);
            const bool there = i * 32 + lane < HC && row < t.row_end && mb < p.sw_cols;
            nx[i] = there ? p.sx[kb * p.lds + row] : 0.f;
            nw[i] = there ? p.sw[(static_cast<int64_t>(t.group) * p.num_kb + kb) * p.sw_cols + mb] : 0.f;
          }
        };
        load_scales(kb_begin, nx[0], nw[0]);
        if (kb_begin + 1 < kb_end) load_scales(kb_begin + 1, nx[1], nw[1]);
        auto add_block = [&](int kb, float (&nx)[SC], float (&nw)[SC]) {
          const uint32_t acc = acc_i & 1u;
          float* sc = my_scale + acc * HC;
#pragma unroll
          for (int i = 0; i < SC; ++i)
            if (i * 32 + lane < HC) sc[i * 32 + lane] = nx[i] * nw[i];
          __syncwarp();
          if (kb + 2 < kb_end) load_scales(kb + 2, nx, nw);
          if (!__all_sync(0xffffffffu, mbar_wait(&tfull[acc], (acc_i >> 1) & 1u, abort_flag, kDevErrTimeoutEpilogue)))
            return false;
          tc_fence_after();
          const uint32_t base = lane_base + acc * C::COLS;
          // two 8-column groups at a time, the next two on their way
          uint32_t r[2][2][8];
          tmem_ld_16x16(base, r[0][0]);
          tmem_ld_16x16(base + (16u << 16), r[0][1]);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < HC / 16; ++c) {
            if (c + 1 < HC / 16) {
              tmem_ld_16x16(base + (c + 1) * 16, r[(c + 1) & 1][0]);
              tmem_ld_16x16(base + (c + 1) * 16 + (16u << 16), r[(c + 1) & 1][1]);
            }
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const uint64_t s2 = *reinterpret_cast<const uint64_t*>(sc + c * 16 + g * 8 + 2 * (lane & 3));
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t* v = &r[c & 1][j >> 1][g * 4 + (j & 1) * 2];
                sum[2 * c + g][j] = grouped_fma2(pack_u64(v[0], v[1]), s2, sum[2 * c + g][j]);
              }
            }
            if (c + 1 < HC / 16) tmem_ld_wait();
            if (c + 2 == HC / 16 || (HC == 16 && c == 0)) release(acc);
          }
          ++acc_i;
          return true;
        };
        for (int kb = kb_begin; ok && kb < kb_end; kb += 2) {
          ok = add_block(kb, nx[0], nw[0]);
          if (ok && kb + 1 < kb_end) ok = add_block(kb + 1, nx[1], nw[1]);
        }
        if (!ok) break;
        if (splits > 1) {
#pragma unroll
          for (int i = 0; i < HC / 2; ++i) my_part[i * 32] = sum[i / 4][i % 4];
          break;
        }
#pragma unroll
        for (int g = 0; g < HC / 8; ++g)
          grouped_store(p, out, sum[g], t.row0 + r_of(g * 8), t.row_end, (mblock0 + mt_of(g * 8)) * 128 + quarter * 32, lane);
      } else {
        const uint32_t acc = acc_i & 1u;
        if (!__all_sync(0xffffffffu, mbar_wait(&tfull[acc], (acc_i >> 1) & 1u, abort_flag, kDevErrTimeoutEpilogue, 64)))
          break;
        tc_fence_after();
        const uint32_t base = lane_base + acc * C::COLS;
#pragma unroll 4
        for (int c = 0; c < HC / 16; ++c) {
          uint32_t r[2][8];
          tmem_ld_16x16(base + c * 16, r[0]);
          tmem_ld_16x16(base + c * 16 + (16u << 16), r[1]);
          tmem_ld_wait();
          if (c == HC / 16 - 1) release(acc);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            uint64_t v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = pack_u64(r[j >> 1][g * 4 + (j & 1) * 2], r[j >> 1][g * 4 + (j & 1) * 2 + 1]);
            if (splits > 1) {
#pragma unroll
              for (int j = 0; j < 4; ++j) my_part[((c * 2 + g) * 4 + j) * 32] = v[j];
              continue;
            }
            grouped_store(p, out, v, t.row0 + r_of(c * 16 + g * 8), t.row_end,
                          (mblock0 + mt_of(c * 16 + g * 8)) * 128 + quarter * 32, lane);
          }
        }
        ++acc_i;
      }
    }
  }

  if (CG == 1 && splits > 1) {
    cluster_sync();  // every CTA's sums are there
    if (warp >= 2 && warp < 2 + EW && worker < units.count) {
      const GroupedTile t = units.get(worker);
      const int quarter = warp & 3, share = (warp - 2) >> 2;
      uint8_t* out = sOut + (warp - 2) * 512;
      const uint32_t at = smem_u32(smem) + static_cast<uint32_t>((((warp - 2) * (HC / 2)) * 32 + lane) * 8);
#pragma unroll
      for (int g = 0; g < HC / 8; ++g) {
        if (g % splits != static_cast<int>(part)) continue;
        float2 s[4] = {};
        for (int r = 0; r < splits; ++r) {
          const uint32_t from = map_shared_rank(at, static_cast<uint32_t>(r));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 v = ld_shared_cluster_f32x2(from + static_cast<uint32_t>((g * 4 + j) * 32 * 8));
            s[j].x += v.x;
            s[j].y += v.y;
          }
        }
        uint64_t v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = pack_u64(__float_as_uint(s[j].x), __float_as_uint(s[j].y));
        grouped_store(p, out, v, t.row0 + grouped_r<N, HC>(share, g * 8), t.row_end,
                      (t.mtile * MT + grouped_mt<N, HC>(share, g * 8)) * 128 + quarter * 32, lane);
      }
    }
  }
  tc_fence_before();
  // both CTAs of a pair are done with every MMA, copy and accumulator, the CTAs of
  // a split tile with one another's sums
  if (CG == 2 || splits > 1) cluster_sync();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if (CG == 2) tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    else tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

}  // namespace rmm
