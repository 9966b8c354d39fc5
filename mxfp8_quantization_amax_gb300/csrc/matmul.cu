// matmul.cu -- the product of blockwise FP8 tensors on the tensor cores: one
// matrix product, the products of rows sorted by expert, and the experts'
// weight gradients.
//
//   D[m, n] = sum_kb sa[m, kb] * sb(n, kb) * P_kb[m, n],
//   P_kb[m, n] = sum over the 128 values k of block kb of A[m, k] * B[n, k],
//
// with A and B the 8-bit codes (both K-major, as fp8q_quantize_blockwise
// leaves them) and sa, sb their scale_inv ("混合精度与 FP8 训练" 10.2-10.5).
// The scales change every 128 values of K, so the tensor core sums one block
// at a time into tensor memory (exact products, FP32 sums), and warps of sums
// read each block back, scale it and add it in FP32 registers.
//
// A tile is 256 rows x 256 columns over a pair of CTAs (or 128 x 256 over one):
// the widest that two blocks of tensor memory and 128 sums a thread hold, and
// a pair, because each of its CTAs feeds its tensor core half of B only.  Warps
// by role: eight hold the sums (216 registers a thread), one loads by TMA, one
// issues the products, one or two bring the scales.
//
// Bound, 9728 x 4096 x 4096: the chain around the two blocks of tensor memory,
// not a rate (tensor pipe 54% busy, L2 37%, DRAM 11%).  From the issue of a
// block's products to the sums' warps 870 cycles, 600 to 800 until its place
// is free again, 250 until the next issue: 830 cycles a block of K, of which
// the products are 512.  A packed multiply a value for column scales makes it
// 1390; their kernels also spill (56 to 246 bytes a thread).  Measured: 12345 x
// 4096 x 14336 604 to 620 us (2.3 to 2.4 PFLOP/s, at the power limit), FP32 14336
// x 4096 x 16384 with column scales 1115 to 1130 us, 65536 rows over 64 experts
// of 4096 x 7168 1800 to 1870 us, 128 rows over them 234 to 253 us (6.3 to 6.8
// TB/s of the weights that some row reaches).  128-column tiles with four blocks in tensor memory
// were slower (174 against 118 us at 4864 x 2048 x 16384): a warp of sums
// needs some 600 cycles a block whatever its columns.
#include "fp8q_device.cuh"
#include "internal.h"
#include "umma.cuh"

namespace fp8q {

constexpr int kMmBlock = 128;  // values of K that share a scale
constexpr int kMmRows = 128;   // rows of A of one CTA in a tile
constexpr int kMmCols = 256;   // columns of a tile
constexpr int kMmEpiWarps = 8;
constexpr int kMmThreads = (kMmEpiWarps + 4) * 32;
// Registers a thread: 168 at launch, moved from the warpgroup of the loads
// and the tensor core to the two that hold the sums (128 of them each).
constexpr int kMmRegsLaunch = 168, kMmRegsEpi = 216, kMmRegsLoad = 72;
static_assert(kMmEpiWarps * 32 * kMmRegsEpi + 128 * kMmRegsLoad <= kMmThreads * kMmRegsLaunch, "register split");
constexpr int kMmScaleSlots = 3;  // ring of scales, four blocks of K each
constexpr uint64_t kMmDrainNs = 2000000000ull;

__device__ unsigned int g_mm_error;
__device__ unsigned long long g_mm_wait_budget_ns = 1000000000ull;
__device__ int g_mm_stall_loads;  // test hook: issue no loads

// Waits that mostly last a few hundred cycles: the clock is looked at only
// once some 100 us of tries have failed, 64 by a whole warp or 8192 by the one
// thread that polls, the tensor core's (it is the quicker to see a barrier).
// From there on the wait has its whole budget.
constexpr uint32_t kMmTries = 64, kMmPolls = 8192;
__device__ __forceinline__ uint64_t mm_budget() { return *(volatile unsigned long long*)&g_mm_wait_budget_ns; }
__device__ __forceinline__ bool mm_wait(uint64_t* bar, uint32_t parity, uint32_t tries = kMmTries) {
  return mbar_try_loop(bar, parity, tries) || mbar_wait(bar, parity, mm_budget());
}

// Notes the time of this warp's n = kMmTries; tells of a later n whether the
// budget is over since then.
__device__ __forceinline__ bool mm_late(volatile uint64_t* since, uint32_t n) {
  if (n < kMmTries) return false;
  const uint64_t now = globaltimer_ns();
  since += threadIdx.x >> 5;
  if (n == kMmTries) *since = now;
  return now - *since > mm_budget();
}

// What the groups divide: nothing, the rows of A and D, or K.
enum : int { kMmDense = 0, kMmRowGroups = 1, kMmKGroups = 2 };

struct MmParams {
  int64_t m, n, k;   // rows of A, rows of B (of one group), values along K
  const float* sa;   // [m][sa_ld]
  const float* sb;   // 1x128: [n][sb_ld]; 128x128: [groups][ceil(n / 128)][sb_ld]
  int64_t sa_ld, sb_ld;
  const int64_t* off;
  int groups;
  int tiles_n;
  int accumulate;
  uint32_t idesc;
  void* out;         // [m][n]; K groups: [groups][m][n]
};

// A tile is 128 * CG rows x 256 columns, CG the CTAs that work on it: one, or a
// pair, whose CTAs each hold 128 rows of A and half of B's.
template <int CG>
struct MmShape {
  static constexpr int kTileRows = kMmRows * CG;
  static constexpr int kABytes = kMmRows * kMmBlock;
  static constexpr int kBBytes = kMmCols / CG * kMmBlock;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = 196608 / kStageBytes;  // 192 KB
};

struct MmTile {
  int g;
  int64_t row0, row_end;  // rows of A and D
  int64_t n0;
  int64_t k0;             // first value of K
  int nkb;                // blocks of K
};

__device__ __forceinline__ int64_t mm_clamped(const int64_t* off, int g, int64_t hi) {
  const int64_t v = __ldg(off + g);
  return v < 0 ? 0 : v > hi ? hi : v;
}

// Tile t of the grid-wide list.  Inside a group, bands of 16 row tiles are
// walked row tile first, so the CTAs of one wave read few distinct tiles of
// A and of B and find them in L2.
template <int CG, int MODE>
__device__ __forceinline__ MmTile mm_tile(const MmParams& p, const unsigned* first, uint32_t t) {
  constexpr int ROWS = MmShape<CG>::kTileRows;
  MmTile r;
  r.g = 0;
  int64_t lo = 0, hi = p.m;
  uint32_t mt_all;
  if constexpr (MODE == kMmRowGroups) {
    int a = 0, b = p.groups;  // last g whose first tile is <= t
    while (b - a > 1) {
      const int mid = (a + b) >> 1;
      if ((uint64_t)first[mid] * p.tiles_n <= t) a = mid; else b = mid;
    }
    r.g = a;
    t -= first[a] * p.tiles_n;
    mt_all = first[a + 1] - first[a];
    lo = mm_clamped(p.off, a, p.m);
    hi = mm_clamped(p.off, a + 1, p.m);
  } else {
    mt_all = (uint32_t)((p.m + ROWS - 1) / ROWS);
    if constexpr (MODE == kMmKGroups) {
      const uint32_t per = mt_all * p.tiles_n;
      r.g = (int)(t / per);
      t -= r.g * per;
    }
  }
  const uint32_t per_band = 16u * p.tiles_n, band = t / per_band;
  const uint32_t in_band = t - band * per_band, rest = mt_all - band * 16u, height = rest < 16u ? rest : 16u;
  r.row0 = lo + (int64_t)(band * 16u + in_band % height) * ROWS;
  r.row_end = hi;
  r.n0 = (int64_t)(in_band / height) * kMmCols;
  r.k0 = 0;
  int64_t k1 = p.k;
  if constexpr (MODE == kMmKGroups) {
    // a start off the 128 grid breaks the caller's promise; rounded down it
    // still makes an aligned TMA coordinate
    r.k0 = mm_clamped(p.off, r.g, p.k) & ~(int64_t)(kMmBlock - 1);
    k1 = mm_clamped(p.off, r.g + 1, p.k);
  }
  r.nkb = k1 > r.k0 ? (int)((k1 - r.k0 + kMmBlock - 1) / kMmBlock) : 0;
  return r;
}

// first[g] = row tiles of the groups before g, first[groups] = all of them.
template <int ROWS>
__device__ __forceinline__ void mm_scan_groups(const MmParams& p, unsigned* first, unsigned* sums) {
  const int tid = threadIdx.x, per = (p.groups + 255) / 256;
  const int g0 = min(tid * per, p.groups), g1 = min(g0 + per, p.groups);
  uint64_t mine = 0;
  if (tid < 256) {
    for (int g = g0; g < g1; g++) {
      const int64_t n = mm_clamped(p.off, g + 1, p.m) - mm_clamped(p.off, g, p.m);
      mine += n > 0 ? (uint64_t)((n + ROWS - 1) / ROWS) : 0;
    }
    sums[tid] = (unsigned)(mine < 0x7FFFFFu ? mine : 0x7FFFFFu);
  }
  __syncthreads();
  if (tid < 32) {  // exclusive scan of 256 sums: 8 per lane
    unsigned s[8], total = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      s[i] = total;
      total += sums[tid * 8 + i];
    }
    unsigned incl = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (tid >= o) incl += v;
    }
#pragma unroll
    for (int i = 0; i < 8; i++) sums[tid * 8 + i] = incl - total + s[i];
    if (tid == 31) first[p.groups] = incl;
  }
  __syncthreads();
  if (tid < 256) {
    unsigned at = sums[tid];
    for (int g = g0; g < g1; g++) {
      first[g] = at;
      const int64_t n = mm_clamped(p.off, g + 1, p.m) - mm_clamped(p.off, g, p.m);
      at += n > 0 ? (unsigned)((n + ROWS - 1) / ROWS) : 0;
    }
  }
  __syncthreads();
}

// Stores COLS consecutive values of one row, those below column n.
template <int COLS, bool F32>
__device__ __forceinline__ void mm_store_row(const MmParams& p, int64_t row, int64_t c0, const uint64_t (&acc)[COLS / 2]) {
  const int64_t left = p.n - c0;
  if constexpr (F32) {
    float* o = (float*)p.out + row * p.n + c0;
    if (p.n % 8 == 0 && ((uintptr_t)p.out & 31) == 0) {
#pragma unroll
      for (int c = 0; c < COLS; c += 8) {
        if (c < left) {
          float v[8];
#pragma unroll
          for (int i = 0; i < 4; i++) unpack2(acc[c / 2 + i], v[2 * i], v[2 * i + 1]);
          if (p.accumulate) {
            const float4 a = *(const float4*)(o + c), b = *(const float4*)(o + c + 4);
            v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w, v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
          }
          uint32_t d[8];
#pragma unroll
          for (int i = 0; i < 8; i++) d[i] = __float_as_uint(v[i]);
          st32B(o + c, d);
        }
      }
    } else {
#pragma unroll
      for (int c = 0; c < COLS; c += 2) {
        float x, y;
        unpack2(acc[c / 2], x, y);
        if (c < left) o[c] = p.accumulate ? o[c] + x : x;
        if (c + 1 < left) o[c + 1] = p.accumulate ? o[c + 1] + y : y;
      }
    }
  } else {
    uint16_t* o = (uint16_t*)p.out + row * p.n + c0;
    if (p.n % 16 == 0 && ((uintptr_t)p.out & 31) == 0) {
#pragma unroll
      for (int c = 0; c < COLS; c += 16) {
        if (c < left) {
          uint32_t d[8];
#pragma unroll
          for (int i = 0; i < 8; i++) {
            float x, y;
            unpack2(acc[c / 2 + i], x, y);
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d[i]) : "f"(y), "f"(x));
          }
          st32B(o + c, d);
        }
      }
    } else {
#pragma unroll
      for (int c = 0; c < COLS; c += 2) {
        float x, y;
        uint32_t d;
        unpack2(acc[c / 2], x, y);
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(y), "f"(x));
        if (c < left) o[c] = (uint16_t)d;
        if (c + 1 < left) o[c + 1] = (uint16_t)(d >> 16);
      }
    }
  }
}

// Adds a tile's sums over the CTAs of a cluster, in the order of their ranks,
// and stores them.  Each CTA writes its sums into its own stages (free by
// then; rows of 1 KB, 16-byte chunks permuted by the row) and takes a slice of
// the columns from all of them: a warp reads whole lines of the others' shared
// memory.  (Written there 16 bytes a row instead, 128 rows took 20 us.)
// Called by the warps of sums; the others join its two barriers.
template <int COLS, bool F32>
__device__ __forceinline__ void mm_store_split(const MmParams& p, const MmTile& w, unsigned char* stages, int r, int half,
                                               const uint64_t (&acc)[COLS / 2]) {
  constexpr int kMost = 8;  // CTAs of a cluster
  const uint32_t part = cluster_rank(), parts = cluster_size();
  const int64_t there = w.row_end - w.row0;
  const int rows = there < kMmRows ? (int)there : kMmRows;
  if (r < rows) {
#pragma unroll
    for (int c = 0; c < COLS; c += 4) {
      float4 v;
      unpack2(acc[c / 2], v.x, v.y);
      unpack2(acc[c / 2 + 1], v.z, v.w);
      *(float4*)(stages + r * 1024 + ((((half * COLS + c) >> 2) ^ (r & 7)) << 4)) = v;
    }
  }
  cluster_sync();
  const int chunks = kMmCols / 4 / (int)parts;  // of a row of the slice
  uint32_t at[kMost];
#pragma unroll
  for (uint32_t q = 0; q < kMost; q++) at[q] = cluster_addr(stages, q < parts ? q : 0);
  const bool wide = p.n % 4 == 0 && ((uintptr_t)p.out & (F32 ? 15 : 7)) == 0;
  for (int i = threadIdx.x; i < rows * chunks; i += kMmEpiWarps * 32) {
    const int row = i / chunks, chunk = (int)part * chunks + i % chunks;
    float4 u[kMost];
#pragma unroll
    for (uint32_t q = 0; q < kMost; q++)
      if (q < parts) u[q] = ld_cluster4(at[q] + row * 1024 + ((chunk ^ (row & 7)) << 4));
    float4 v = u[0];
#pragma unroll
    for (uint32_t q = 1; q < kMost; q++)
      if (q < parts) v.x += u[q].x, v.y += u[q].y, v.z += u[q].z, v.w += u[q].w;
    const int64_t c0 = w.n0 + 4 * chunk, o = (w.row0 + row) * p.n + c0;
    if (c0 >= p.n) continue;
    const float x[4] = {v.x, v.y, v.z, v.w};
    if constexpr (F32) {
      float* out = (float*)p.out + o;
      if (wide) {
        if (p.accumulate) {
          const float4 y = *(const float4*)out;
          v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
        }
        *(float4*)out = v;
      } else {
#pragma unroll
        for (int k = 0; k < 4; k++)
          if (c0 + k < p.n) out[k] = p.accumulate ? out[k] + x[k] : x[k];
      }
    } else {
      uint16_t* out = (uint16_t*)p.out + o;
      uint32_t d[2];
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d[0]) : "f"(x[1]), "f"(x[0]));
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d[1]) : "f"(x[3]), "f"(x[2]));
      if (wide) {
        *(uint2*)out = make_uint2(d[0], d[1]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; k++)
          if (c0 + k < p.n) out[k] = (uint16_t)(d[k >> 1] >> (16 * (k & 1)));
      }
    }
  }
  cluster_sync();  // no CTA leaves while another reads from it
}

// SPLIT: the CTAs of a cluster share one tile's blocks of K and add their sums
// at the end.  COLSCALE: B has a scale for each of its rows
// (1x128 groups), else one for each 128 of them.
template <int CG, bool SPLIT, bool COLSCALE, bool F32, int MODE>
__global__ void __launch_bounds__(kMmThreads, 1)
    matmul_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, MmParams p) {
  using S = MmShape<CG>;
  constexpr int COLS = kMmCols / 2;  // of one warp of sums
  // scales of one block of K: the rows', and the columns' or the halves' two
  constexpr int NS = kMmRows + (COLSCALE ? kMmCols : 32);
  constexpr int SW = COLSCALE ? 2 : 1;  // warps that load them
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t full[S::kStages], empty[S::kStages], done[2], taken[2], drained;
  __shared__ uint64_t sfull[kMmScaleSlots], sempty[kMmScaleSlots];
  __shared__ uint32_t tmem_base;
  __shared__ unsigned sums[MODE == kMmRowGroups ? 256 : 1];
  __shared__ __align__(16) float scale[kMmScaleSlots][4][NS];
  __shared__ volatile int abort_flag;
  __shared__ uint64_t since[kMmEpiWarps];  // when the sums' warps began to wait long
  unsigned char* stages = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  unsigned* first = (unsigned*)(stages + S::kStages * S::kStageBytes);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < S::kStages; s++) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; b++) {
      mbar_init(&done[b], 1);
      mbar_init(&taken[b], kMmEpiWarps * CG);
    }
    mbar_init(&drained, 1);
    for (int i = 0; i < kMmScaleSlots; i++) {
      mbar_init(&sfull[i], SW);
      mbar_init(&sempty[i], kMmEpiWarps);
    }
    abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kMmEpiWarps) {
    tmem_alloc<CG>(&tmem_base, 512);
    tc_fence_before();
    if (lane == 0) {
      prefetch_tensormap(&map_a);
      prefetch_tensormap(&map_b);
    }
  }
  pdl_wait();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();  // the leader's barriers, before the other CTA uses them
  tc_fence_after();
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;
  const uint32_t tile0 = blockIdx.x / (SPLIT ? cluster_size() : CG);
  const uint32_t tile_step = SPLIT ? 0x40000000u : gridDim.x / CG;  // a split has one tile a cluster
  const uint32_t tmem = tmem_base;

  uint32_t tiles;
  const auto tile_of = [&](uint32_t t) {
    MmTile w = mm_tile<CG, MODE>(p, first, t);
    if constexpr (SPLIT) {  // this CTA's share of the blocks
      const uint32_t part = cluster_rank(), parts = cluster_size(), n = (uint32_t)w.nkb;
      const uint32_t kb0 = n * part / parts;
      w.k0 += (int64_t)kb0 * kMmBlock;
      w.nkb = (int)(n * (part + 1) / parts - kb0);
    }
    return w;
  };
  if constexpr (MODE == kMmRowGroups) {
    mm_scan_groups<S::kTileRows>(p, first, sums);
    tiles = first[p.groups] * (uint32_t)p.tiles_n;
  } else {
    tiles = (uint32_t)((p.m + S::kTileRows - 1) / S::kTileRows) * (uint32_t)p.tiles_n * (uint32_t)p.groups;
  }

  if (warp >= kMmEpiWarps) {
    regs_dec<kMmRegsLoad>();
    if (warp == kMmEpiWarps) {
      // ---------------- loads: one thread ----------------
      if (elect_one()) {
        uint32_t it = 0;  // blocks of K issued
        for (uint32_t t = g_mm_stall_loads ? tiles : tile0; t < tiles && !abort_flag; t += tile_step) {
          const MmTile w = tile_of(t);
          const int arow = (int)w.row0 + rank * kMmRows;
          const int brow = (int)(w.n0 + (MODE == kMmRowGroups ? (int64_t)w.g * p.n : 0)) + rank * (kMmCols / CG);
          int at = (int)w.k0;
          for (int kb = 0; kb < w.nkb; kb++, it++, at += kMmBlock) {
            const uint32_t s = it % S::kStages, round = it / S::kStages;
            if (round > 0 && !mm_wait(&empty[s], (round - 1) & 1u, kMmPolls)) {
              abort_flag = 1;
              break;
            }
            unsigned char* st = stages + s * S::kStageBytes;
            if constexpr (CG == 1) {
              mbar_arrive_expect_tx(&full[s], S::kStageBytes);
              tma_load_2d(st, &map_a, at, arow, &full[s]);
              tma_load_2d(st + S::kABytes, &map_b, at, brow, &full[s]);
            } else {
              // the leader's barrier counts the bytes of both CTAs
              if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * S::kStageBytes);
              const uint32_t bar = cluster_addr(&full[s], 0);
              tma_load_2d_pair(st, &map_a, at, arow, bar);
              tma_load_2d_pair(st + S::kABytes, &map_b, at, brow, bar);
            }
          }
        }
        // Every issued copy lands before the CTA (the pair) can exit (fixed 2 s
        // bound), and every block is used or the flag that tells of a failure up.
        const uint32_t tail = it > S::kStages ? it - S::kStages : 0;
        if (rank == 0)
          for (uint32_t j = tail; j < it; j++) mbar_wait(&full[j % S::kStages], (j / S::kStages) & 1u, kMmDrainNs);
        for (uint32_t j = tail; j < it && !abort_flag; j++)
          if (!mm_wait(&empty[j % S::kStages], (j / S::kStages) & 1u, kMmPolls)) abort_flag = 1;
        if (abort_flag) atomicOr(&g_mm_error, 1u);
      }
      __syncwarp();
      pdl_launch_dependents();
    } else if (warp == kMmEpiWarps + 1) {
      // ---------------- tensor core: one thread of the leader ----------------
      if (rank == 0 && elect_one()) {
        uint32_t it = 0;
        for (uint32_t t = tile0; t < tiles && !abort_flag; t += tile_step) {
          const MmTile w = tile_of(t);
          for (int kb = 0; kb < w.nkb; kb++, it++) {
            const uint32_t s = it % S::kStages, round = it / S::kStages, b = it & 1u, use = it >> 1;
            if (!mm_wait(&full[s], round & 1u, kMmPolls) || (use > 0 && !mm_wait(&taken[b], (use - 1) & 1u, kMmPolls))) {
              atomicOr(&g_mm_error, 1u);
              abort_flag = 1;
              break;
            }
            tc_fence_after();
            const uint32_t st = smem_u32(stages + s * S::kStageBytes);
            const uint64_t da = smem_desc_sw128(st), db = smem_desc_sw128(st + S::kABytes);
#pragma unroll
            for (int k = 0; k < kMmBlock / 32; k++)
              mma_f8<CG>(tmem + b * kMmCols, da + 2 * k, db + 2 * k, p.idesc, k > 0);
            mma_commit<CG>(&done[b]);
            mma_commit<CG>(&empty[s]);
          }
        }
        // nothing is in flight when the tensor memory is freed
        mma_commit<CG>(&drained);
        mbar_wait(&drained, 0, kMmDrainNs);
      }
      __syncwarp();
    } else if (warp < kMmEpiWarps + 2 + SW) {
      // ---------------- scales: SW warps, four blocks of K at a time ----------------
      // Quads of blocks are aligned in the scale rows, so that with rows of a
      // multiple of four a quad is one 16-byte load (a line a row: four times
      // fewer than a load a block).
      const bool vec = ((p.sa_ld | p.sb_ld) & 3) == 0 && (((uintptr_t)p.sa | (uintptr_t)p.sb) & 15) == 0;
      const auto quad = [&](const float* row, int64_t ld, int64_t q) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (vec) {
          v = __ldg((const float4*)(row + 4 * q));
        } else {
          v.x = __ldg(row + 4 * q);
          if (4 * q + 1 < ld) v.y = __ldg(row + 4 * q + 1);
          if (4 * q + 2 < ld) v.z = __ldg(row + 4 * q + 2);
          if (4 * q + 3 < ld) v.w = __ldg(row + 4 * q + 3);
        }
        return v;
      };
      const auto put = [&](float* at, const float4& v) {  // the four blocks of one row or column
        at[0] = v.x, at[NS] = v.y, at[2 * NS] = v.z, at[3 * NS] = v.w;
      };
      uint32_t it = 0;
      bool ok = true;
      for (uint32_t t = tile0; t < tiles && ok; t += tile_step) {
        const MmTile w = tile_of(t);
        if (w.nkb == 0) continue;
        const int64_t kb0 = w.k0 / kMmBlock;
        for (int64_t q = kb0 >> 2; q <= (kb0 + w.nkb - 1) >> 2; q++, it++) {
          const uint32_t s = it % kMmScaleSlots, round = it / kMmScaleSlots;
          float* at = &scale[s][0][0];
          constexpr int N = NS / 32 / SW;
          const int e0 = (warp - (kMmEpiWarps + 2)) * N * 32 + lane;  // of the rows, then of the columns
          float4 v[N];
#pragma unroll
          for (int i = 0; i < N; i++) {
            const int e = e0 + i * 32;
            if (e < kMmRows) {
              const int64_t r = w.row0 + rank * kMmRows + e;
              v[i] = quad(p.sa + (r < p.m ? r : p.m - 1) * p.sa_ld, p.sa_ld, q);
            } else if constexpr (COLSCALE) {
              const int64_t c = w.n0 + e - kMmRows;
              v[i] = quad(p.sb + (c < p.n ? c : p.n - 1) * p.sb_ld, p.sb_ld, q);
            } else {
              const int64_t nb = (p.n + kMmBlock - 1) / kMmBlock, c = w.n0 / kMmBlock + (lane & 1);
              v[i] = quad(p.sb + ((MODE == kMmRowGroups ? (int64_t)w.g * nb : 0) + (c < nb ? c : nb - 1)) * p.sb_ld, p.sb_ld, q);
            }
          }
          if (!__all_sync(0xFFFFFFFFu, round == 0 || mm_wait(&sempty[s], (round - 1) & 1u))) {
            ok = false;
            break;
          }
#pragma unroll
          for (int i = 0; i < N; i++) put(at + e0 + i * 32, v[i]);
          __syncwarp();
          if (lane == 0) mbar_arrive(&sfull[s]);
        }
      }
      if (!ok) {
        if (lane == 0) atomicOr(&g_mm_error, 1u);
        abort_flag = 1;
      }
    }
  } else {
    regs_inc<kMmRegsEpi>();
    // ---------------- sums over the blocks and the epilogue ----------------
    const int half = warp >> 2;                         // columns [half * COLS, half * COLS + COLS)
    const int quarter = warp & 3;                       // this warp's 32 lanes of tensor memory
    const uint32_t taddr = tmem + ((uint32_t)quarter << 21) + half * COLS;
    const uint32_t taken_at = CG == 1 ? 0 : cluster_addr(&taken[0], 0);
    uint32_t it = 0, sit = 0;  // blocks of K and quads of scales taken
    int kq = 0;                // the next block's place in its quad
    float next = 0.0f, next_col = 0.0f;  // its row's scale, and its half's
    uint32_t r[2][32];
    bool dead = false;
    // A wait of mm_wait's rule that ends with the other warps', too.  Its start is
    // kept in shared memory, for want of registers, and nothing is asked before
    // kMmTries (14336 x 4096 x 16384 with column scales: 1130 us, 1142 with a look
    // at abort_flag each time, 1164 with the clock in registers).  After one that
    // ran out the warp goes on without waiting, since its loads are collective;
    // its tile loop ends, and the error word tells that the output is worthless.
    const auto wait = [&](uint64_t* bar, uint32_t parity) {
      for (uint32_t n = dead ? kMmTries : 0; !mbar_try_wait(bar, parity); n++)
        if (n >= kMmTries && (abort_flag || mm_late(since, n))) {
          abort_flag = 1;
          dead = true;
          break;
        }
    };
    // Waits for a block of K and starts its way from tensor memory to registers.
    const auto fetch = [&](bool new_quad) {
      const uint32_t slot = sit % kMmScaleSlots, b = it & 1u;
      wait(&done[b], (it >> 1) & 1u);
      if (new_quad) wait(&sfull[slot], (sit / kMmScaleSlots) & 1u);
      tc_fence_after();
      __syncwarp();
      tmem_load32(r[0], taddr + b * kMmCols);
      // not multiplied here: that would hold the warp until they have come
      next = scale[slot][kq][quarter * 32 + lane];
      if constexpr (!COLSCALE) next_col = scale[slot][kq][kMmRows + half];
    };
    for (uint32_t t = tile0; t < tiles && !__any_sync(0xFFFFFFFFu, dead); t += tile_step) {
      int nkb;
      {
        const MmTile w = tile_of(t);
        nkb = w.nkb;
        kq = (int)(w.k0 / kMmBlock) & 3;
      }
      uint64_t acc[COLS / 2];
#pragma unroll
      for (int i = 0; i < COLS / 2; i++) acc[i] = 0;
      // Chunks of 32 columns, the next one (of the next block, too) on its
      // way from tensor memory while this one is added.
      if (nkb > 0) fetch(true);
      for (; nkb > 0; nkb--) {
        const uint32_t b = it & 1u, slot = sit % kMmScaleSlots;
        const float* sc = scale[slot][kq];
        const float f = COLSCALE ? next : __fmul_rn(next, next_col);
        const uint64_t s2 = pack2(__float_as_uint(f), __float_as_uint(f));
        const bool quad_ends = kq == 3 || nkb == 1;
        it++;
        kq = (kq + 1) & 3;
        sit += quad_ends;
#pragma unroll
        for (int c = 0; c < COLS; c += 32) {
          uint32_t(&v)[32] = r[(c / 32) & 1];
          tmem_wait_loads(v);
          if (c + 32 < COLS) {
            tmem_load32(r[(c / 32 + 1) & 1], taddr + b * kMmCols + c + 32);
          } else {
            // everything of this block is in registers
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if constexpr (CG == 1) mbar_arrive(&taken[b]); else mbar_arrive_cluster(taken_at + 8 * b);
            }
            if (nkb > 1) fetch(quad_ends);
          }
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            uint64_t f0 = s2, f1 = s2;
            if constexpr (COLSCALE) {
              const ulonglong2 cs = *(const ulonglong2*)&sc[kMmRows + half * COLS + c + i];
              f0 = mul2p(cs.x, s2);
              f1 = mul2p(cs.y, s2);
            }
            acc[(c + i) / 2] = fma2(pack2(v[i], v[i + 1]), f0, acc[(c + i) / 2]);
            acc[(c + i) / 2 + 1] = fma2(pack2(v[i + 2], v[i + 3]), f1, acc[(c + i) / 2 + 1]);
          }
        }
        if (quad_ends) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sempty[slot]);
        }
      }
      // the tile again, rather than its values kept through the loop
      uint32_t t2 = t;
      asm volatile("" : "+r"(t2));
      const MmTile w = tile_of(t2);
      const int64_t row = w.row0 + rank * kMmRows + quarter * 32 + lane;
      if constexpr (SPLIT)
        mm_store_split<COLS, F32>(p, w, stages, quarter * 32 + lane, half, acc);
      else if (row < w.row_end)
        mm_store_row<COLS, F32>(p, (MODE == kMmKGroups ? (int64_t)w.g * p.m : 0) + row, w.n0 + half * COLS, acc);
    }
    if (dead) {
      atomicOr(&g_mm_error, 1u);
      abort_flag = 1;
    }
    pdl_launch_dependents();
  }
  if (SPLIT && warp >= kMmEpiWarps && tile0 < tiles) {  // the barriers of mm_store_split
    __syncwarp();
    cluster_sync();
    cluster_sync();
  }
  tc_fence_before();
  __syncthreads();
  // in a pair, neither leaves while the other's copies, products or arrivals
  // may still reach its shared memory; every wait before this one is bounded
  if constexpr (CG == 2) cluster_sync();
  if (warp == kMmEpiWarps) {
    __syncwarp();
    tc_fence_after();
    tmem_free<CG>(tmem, 512);
  }
}

// Groups whose reduction is empty: zeros for their rows, which follow one
// another from the first group's first to the last one's last.
template <typename T>
__global__ void zero_groups_kernel(T* out, const int64_t* off, int groups, int64_t rows, int64_t n) {
  pdl_wait();
  const int64_t lo = mm_clamped(off, 0, rows) * n, hi = mm_clamped(off, groups, rows) * n;
  for (int64_t i = lo + (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < hi; i += (int64_t)gridDim.x * blockDim.x) out[i] = T(0);
  pdl_launch_dependents();
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// Codes [rows][k], boxes of 128 codes x box_rows.
static fp8q_status mm_map(CUtensorMap* map, const void* q, int64_t rows, int64_t k, int box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return fail(FP8Q_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)k};
  cuuint32_t box[2] = {kMmBlock, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(q), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FP8Q_OK : fail(FP8Q_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
}

template <int CG, int MODE>
static size_t mm_smem(int groups) {
  return 1024 + (size_t)MmShape<CG>::kStages * MmShape<CG>::kStageBytes + (MODE == kMmRowGroups ? 4 * ((size_t)groups + 1) : 0);
}

// Clusters of `size` CTAs of a kernel that the GPU holds at a time (a GB300: 76
// of 2, 36 of 4, 15 of 8, since a cluster stays inside one part of the chip).
template <int CG, bool SPLIT, bool COLSCALE, bool F32, int MODE>
static int mm_clusters(int size) {
  static PerDevice<int> found[9];
  int clusters;
  const bool known = found[size].get(current_device(), &clusters, [&](int* n) {
    const auto kernel = matmul_kernel<CG, SPLIT, COLSCALE, F32, MODE>;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = size;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(sm_count() / size * size));
    cfg.blockDim = dim3(kMmThreads);
    cfg.dynamicSmemBytes = mm_smem<CG, MODE>(MODE == kMmRowGroups ? FP8Q_MAX_GROUPS : 1);
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cfg.dynamicSmemBytes) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(n, kernel, &cfg) == cudaSuccess)
      return *n > 0;
    cudaGetLastError();
    return false;
  });
  return known ? clusters : 1;
}

template <int CG, bool SPLIT, bool COLSCALE, bool F32, int MODE>
static fp8q_status launch_mm_t(const void* a, const void* b, MmParams p, int fmt_a, int fmt_b, int parts, cudaStream_t s) {
  using S = MmShape<CG>;
  CUtensorMap ma, mb;
  fp8q_status r = mm_map(&ma, a, p.m, p.k, kMmRows);
  if (r != FP8Q_OK) return r;
  if ((r = mm_map(&mb, b, MODE == kMmRowGroups ? p.n * p.groups : p.n, p.k, kMmCols / CG)) != FP8Q_OK) return r;
  p.idesc = instr_desc_f8(fmt_a, fmt_b, S::kTileRows, kMmCols);
  p.tiles_n = (int)((p.n + kMmCols - 1) / kMmCols);
  const size_t smem = mm_smem<CG, MODE>(p.groups);
  const auto kernel = matmul_kernel<CG, SPLIT, COLSCALE, F32, MODE>;
  static PerDevice<bool> allowed;
  const cudaError_t attr = allow_smem(allowed, kernel, mm_smem<CG, MODE>(FP8Q_MAX_GROUPS));
  if (attr != cudaSuccess) return cuda_fail(attr, "matmul shared memory");
  // the kernel moves registers between its warpgroups: they must be there
  static PerDevice<int> launch_regs;
  int regs = 0;
  if (!launch_regs.get(current_device(), &regs, [&](int* n) {
        cudaFuncAttributes f;
        const cudaError_t e = cudaFuncGetAttributes(&f, kernel);
        *n = e == cudaSuccess ? f.numRegs : 0;
        return e == cudaSuccess;
      }))
    return cuda_fail(cudaGetLastError(), "cudaFuncGetAttributes(matmul)");
  if (regs < kMmRegsLaunch) return fail(FP8Q_ERR_CUDA, "matmul kernel built with %d registers a thread", regs);
  const int64_t per = (p.m + S::kTileRows - 1) / S::kTileRows;
  const int64_t tiles = (MODE == kMmRowGroups ? per + p.groups : MODE == kMmKGroups ? per * p.groups : per) * p.tiles_n;
  if (tiles > INT32_MAX) return fail(FP8Q_ERR_UNSUPPORTED, "product too large: %lld output tiles", (long long)tiles);
  // a persistent grid leaves no pair for later, a split no cluster
  int64_t grid = CG == 1 ? sm_count() : mm_clusters<CG, SPLIT, COLSCALE, F32, MODE>(CG);
  if (SPLIT || grid > tiles) grid = tiles;
  const unsigned cluster = SPLIT ? parts : CG;
  const cudaError_t e = launch_cluster(kernel, dim3((unsigned)grid * cluster), dim3(kMmThreads), cluster, smem, s, ma, mb, p);
  if (e != cudaSuccess) return cuda_fail(e, "matmul kernel launch");
  return check_launch("matmul kernel");
}

// Which form.  A split over K where every tile can have a cluster of 2, 4 or 8
// CTAs at once and each CTA two blocks of K: few rows.  (1 x 4096 x 4096: 20.1
// us unsplit, 14.5 by 2, 10.0 by 4; 8, of which only 15 run at a time, 15.1.)
// Pairs where a tile's 256 rows are there (row groups: on average).  Else
// single CTAs.
template <bool COLSCALE, bool F32, int MODE>
static fp8q_status launch_mm_form(const void* a, const void* b, const MmParams& p, int fmt_a, int fmt_b, cudaStream_t s) {
  if constexpr (MODE != kMmKGroups) {
    const int64_t cols = (p.n + kMmCols - 1) / kMmCols, rows = (p.m + kMmRows - 1) / kMmRows;
    const int64_t tiles = (MODE == kMmRowGroups ? rows + p.groups : rows) * cols, kb = (p.k + kMmBlock - 1) / kMmBlock;
    int parts = 1;
    while (parts < 8 && kb >= parts * 4 && tiles <= mm_clusters<1, true, COLSCALE, F32, MODE>(parts * 2)) parts *= 2;
    if (parts > 1) return launch_mm_t<1, true, COLSCALE, F32, MODE>(a, b, p, fmt_a, fmt_b, parts, s);
  }
  if ((MODE == kMmRowGroups ? p.m / p.groups : p.m) > kMmRows)
    return launch_mm_t<2, false, COLSCALE, F32, MODE>(a, b, p, fmt_a, fmt_b, 1, s);
  return launch_mm_t<1, false, COLSCALE, F32, MODE>(a, b, p, fmt_a, fmt_b, 1, s);
}

template <bool COLSCALE, int MODE>
static fp8q_status launch_mm_out(const void* a, const void* b, const MmParams& p, int fmt_a, int fmt_b, int out_dt,
                                 cudaStream_t s) {
  return out_dt == FP8Q_OUT_FP32 ? launch_mm_form<COLSCALE, true, MODE>(a, b, p, fmt_a, fmt_b, s)
                                 : launch_mm_form<COLSCALE, false, MODE>(a, b, p, fmt_a, fmt_b, s);
}

fp8q_status launch_matmul(const MatmulLaunch& L) {
  MmParams p{};
  p.m = L.m;
  p.n = L.n;
  p.k = L.k;
  p.sa = L.sa;
  p.sb = L.sb;
  p.sa_ld = p.sb_ld = (L.k + kMmBlock - 1) / kMmBlock;
  p.off = L.off;
  p.groups = L.groups;
  p.accumulate = L.accumulate;
  p.out = L.out;
  if (L.kind == kMatmulRowGroups) return launch_mm_out<false, kMmRowGroups>(L.a, L.b, p, L.a_fmt, L.b_fmt, L.out_dt, L.stream);
  if (L.kind == kMatmulKGroups) return launch_mm_out<true, kMmKGroups>(L.a, L.b, p, L.a_fmt, L.b_fmt, L.out_dt, L.stream);
  return L.b_block == FP8Q_BLOCK_128X128
             ? launch_mm_out<false, kMmDense>(L.a, L.b, p, L.a_fmt, L.b_fmt, L.out_dt, L.stream)
             : launch_mm_out<true, kMmDense>(L.a, L.b, p, L.a_fmt, L.b_fmt, L.out_dt, L.stream);
}

fp8q_status launch_matmul_zero_groups(const MatmulLaunch& L) {
  const int64_t ctas = (L.m * L.n + 255) / 256, most = (int64_t)sm_count() * 8;
  const dim3 grid((unsigned)(ctas < most ? ctas : most)), block(256);
  const cudaError_t e =
      L.out_dt == FP8Q_OUT_FP32
          ? launch_kernel(zero_groups_kernel<float>, grid, block, 0, L.stream, (float*)L.out, L.off, L.groups, L.m, L.n)
          : launch_kernel(zero_groups_kernel<uint16_t>, grid, block, 0, L.stream, (uint16_t*)L.out, L.off, L.groups, L.m, L.n);
  if (e != cudaSuccess) return cuda_fail(e, "zero kernel launch");
  return check_launch("zero kernel");
}

fp8q_status mm_device_status(bool clear, unsigned* word) {
  unsigned v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_mm_error, sizeof(v));
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpyFromSymbol");
  if (clear && v) {
    const unsigned z = 0;
    e = cudaMemcpyToSymbol(g_mm_error, &z, sizeof(z));
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpyToSymbol");
  }
  *word = v;
  return FP8Q_OK;
}

fp8q_status mm_set_stall_loads(bool on) {
  const int v = on ? 1 : 0;
  const cudaError_t e = cudaMemcpyToSymbol(g_mm_stall_loads, &v, sizeof(v));
  return e == cudaSuccess ? FP8Q_OK : cuda_fail(e, "cudaMemcpyToSymbol(stall hook)");
}

fp8q_status mm_set_wait_budget(unsigned long long ns) {
  cudaError_t e = cudaMemcpyToSymbol(g_mm_wait_budget_ns, &ns, sizeof(ns));
  return e == cudaSuccess ? FP8Q_OK : cuda_fail(e, "cudaMemcpyToSymbol(wait budget)");
}

}  // namespace fp8q
