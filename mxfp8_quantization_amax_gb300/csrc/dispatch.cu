// dispatch.cu -- the order of the experts' rows, and the rows gathered in that
// order and quantized.
//
// Slot t * top_k + j is token t's j-th expert.  The plan is a stable counting
// sort of the slots by expert, each expert's segment padded to a multiple of
// `align` rows: offsets[e] (segment starts), row_of[slot], src[row] (-1 for
// padding).  A slot whose id is no expert's is dropped (row_of -1).
//
// Each CTA takes a contiguous piece of the slots, each warp a contiguous part
// of the piece.  A first pass counts the piece's slots per expert; the second
// adds the counts of the pieces before it and the padded totals of the
// experts before each, and places the slots, lanes of one expert in lane
// order.  Only integers are counted, so the result does not depend on timing.
#include "fp8q_device.cuh"
#include "internal.h"
#include "tma.cuh"

namespace fp8q {

constexpr int kPlanMaxExperts = 1024;
constexpr int kPlanThreads = 256;
constexpr int kPlanWarps = kPlanThreads / 32;
// Slots of one CTA.  One piece needs no counts before it: one launch (1536
// slots, 64 experts: one CTA 5.9 us, two launches 6.3; 4096: 8.5 and 5.7).
// Of 512, 1024 and 2048, 65536 slots take 8.7, 6.9 and 7.1 us.
constexpr int kPlanPiece = 1024;
// Pieces grow beyond 128 of them, since each CTA reads all pieces' counts
// (262144 slots, 256 experts: 12.0 us, 16.4 with 256).
constexpr int kPlanMaxPieces = 128;

struct PlanParams {
  const int* ids;
  int64_t slots;
  int64_t piece;
  int pieces;
  int experts, align;
  int64_t rows;
  int64_t* offsets;
  int* row_of;
  int* src;
  int* counts;  // [pieces][experts]
};

__device__ __forceinline__ int plan_id(const PlanParams& p, int64_t slot, int64_t end) {
  if (slot >= end) return -1;
  const int id = __ldg(p.ids + slot);
  return id >= 0 && id < p.experts ? id : -1;
}

__global__ void __launch_bounds__(kPlanThreads) plan_count_kernel(PlanParams p) {
  __shared__ int hist[kPlanMaxExperts];
  pdl_wait();
  for (int e = threadIdx.x; e < p.experts; e += kPlanThreads) hist[e] = 0;
  __syncthreads();
  const int64_t lo = blockIdx.x * p.piece, hi = min(lo + p.piece, p.slots);
  for (int64_t s = lo + threadIdx.x; s < hi; s += kPlanThreads) {
    const int id = plan_id(p, s, hi);
    if (id >= 0) atomicAdd(&hist[id], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.experts; e += kPlanThreads) p.counts[(int64_t)blockIdx.x * p.experts + e] = hist[e];
  pdl_launch_dependents();
}

// Exclusive sum over the CTA of one value per thread; *all gets the total.
__device__ __forceinline__ int64_t plan_scan(int64_t v, int64_t* sh, int64_t* all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) sh[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kPlanWarps; w++) {
    if (w < warp) before += sh[w];
    total += sh[w];
  }
  __syncthreads();
  *all = total;
  return before + incl - v;
}

__global__ void __launch_bounds__(kPlanThreads) plan_place_kernel(PlanParams p) {
  extern __shared__ int next[];  // [warps][experts]: the next row of each expert for each warp
  __shared__ int64_t sh[kPlanWarps];
  __shared__ int2 pad[kPlanMaxExperts];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  for (int i = tid; i < kPlanWarps * p.experts; i += kPlanThreads) next[i] = 0;
  __syncthreads();
  const int64_t lo = blockIdx.x * p.piece, hi = min(lo + p.piece, p.slots);
  const int64_t part = (p.piece / kPlanWarps + 31) / 32 * 32;
  const int64_t w0 = min(lo + warp * part, hi), w1 = min(w0 + part, hi);
  int* mine = next + warp * p.experts;
  for (int64_t s = w0 + lane; s < w1; s += 32) {
    const int id = plan_id(p, s, w1);
    if (id >= 0) atomicAdd(&mine[id], 1);
  }
  __syncthreads();
  // experts in chunks of one per thread: padded totals of those before
  int64_t base = 0;
  for (int e0 = 0; e0 < p.experts; e0 += kPlanThreads) {
    const int e = e0 + tid;
    int64_t total = 0, before = 0;
    if (e < p.experts) {
      if (p.pieces == 1) {
        for (int w = 0; w < kPlanWarps; w++) total += next[w * p.experts + e];
      } else {
#pragma unroll 8
        for (int b = 0; b < p.pieces; b++) {
          const int c = __ldg(p.counts + (int64_t)b * p.experts + e);
          if (b < (int)blockIdx.x) before += c;
          total += c;
        }
      }
    }
    const int64_t padded = (total + p.align - 1) / p.align * p.align;
    int64_t all;
    const int64_t start = base + plan_scan(padded, sh, &all);
    base += all;
    if (e < p.experts) {
      int64_t at = start + before;
      for (int w = 0; w < kPlanWarps; w++) {
        const int c = next[w * p.experts + e];
        next[w * p.experts + e] = (int)at;
        at += c;
      }
      if (blockIdx.x == 0) p.offsets[e] = start;
      pad[e] = make_int2((int)(start + total), (int)(start + padded));
    }
  }
  if (blockIdx.x == 0 && tid == 0) p.offsets[p.experts] = base;
  __syncthreads();
  for (int e = blockIdx.x + warp * p.pieces; e < p.experts; e += kPlanWarps * p.pieces)  // the segments' padding
    for (int r = pad[e].x + lane; r < pad[e].y; r += 32) p.src[r] = -1;
  for (int64_t r = base + blockIdx.x * kPlanThreads + tid; r < p.rows; r += (int64_t)p.pieces * kPlanThreads) p.src[r] = -1;
  __syncthreads();
  for (int64_t s0 = w0; s0 < w1; s0 += 32) {
    const int64_t s = s0 + lane;
    const int id = plan_id(p, s, w1);
    const unsigned same = __match_any_sync(0xFFFFFFFFu, id);
    const int rank = __popc(same & ((1u << lane) - 1u));
    int row = -1;
    if (id >= 0) {
      row = mine[id] + rank;
      p.src[row] = (int)s;
    }
    __syncwarp();
    if (id >= 0 && rank == 0) mine[id] += __popc(same);
    __syncwarp();
    if (s < w1) p.row_of[s] = row;
  }
  pdl_launch_dependents();
}

// ---------------------------------------------------------------------------
// gather and quantize
//
// A CTA takes 128 gathered rows and a run of 128-column tiles of them; both
// copies' groups are whole in a tile.  The next tile comes into shared memory
// by cp.async while this one is quantized.  The CTAs running at a time walk
// the columns together, so that the part of x they gather from (each row is
// read top_k times) stays in L2.  The arithmetic is fp8q_quantize_blockwise's:
// per group scale = fl32(F8max / amax) with the per-tensor special cases, code
// = RNE_sat(fl32(x * scale)), and fl32(1 / scale) stored.
//
// Instructions and the gather's L2 reads matter as much as memory here (65536
// rows of 7168, both copies: 291 us, of which 71 go when nothing is stored; 170
// us of HBM traffic): each group's division is done by one lane, the maxima are
// packed pairs, a row's maximum takes one shuffle a row and lane, and whole
// tiles without NaN ask for nothing value by value.
// ---------------------------------------------------------------------------
constexpr int kDpTile = 128;
constexpr int kDpThreads = 256;
constexpr int kDpBoxBytes = kDpTile * 128;  // 64 columns of the tile's rows
constexpr int kDpTileBytes = 2 * kDpBoxBytes;

struct DispatchParams {
  const uint16_t* x;
  const int* src;
  int64_t slots;
  int top_k;
  int64_t rows, cols;
  int tiles_r, tiles_c;
  int run;        // column tiles of a CTA
  int pow2;
  uint8_t* q;     // [rows][cols]
  float* s;       // [rows][tiles_c]
  uint8_t* q_t;   // [cols][rows]
  float* s_t;     // [cols][tiles_r]
};

// Byte offset in the tile of row r, column c (c even): two boxes of 64
// columns, 128 bytes a row, whose 16-byte chunks are permuted by the row so
// that eight rows of one chunk, and one row's chunks, lie in different banks.
__device__ __forceinline__ uint32_t dp_off(int r, int c) {
  const int b = (c & 63) * 2;
  return (uint32_t)((c >> 6) * kDpBoxBytes + r * 128 + ((((b >> 4) ^ (r & 7)) << 4) | (b & 15)));
}

template <int FMT>
__device__ __forceinline__ float dp_scale(uint32_t amax_bits, int pow2) {
  const float s = scale_from_amax(amax_bits, Fmt<FMT>::kMax, 0);
  return pow2 ? __uint_as_float(__float_as_uint(s) & 0xFF800000u) : s;  // s is a positive normal float
}

// The halves of a BF16 pair as FP32: a mixed addition of -0, exact, which runs
// beside the integer pipe that masks and shifts would fill (3% of the kernel).
__device__ __forceinline__ float dp_flo(uint32_t w) {
  float r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tadd.rn.f32.bf16 %0, a, %2;\n\t}" : "=f"(r) : "r"(w), "f"(-0.0f));
  return r;
}
__device__ __forceinline__ float dp_fhi(uint32_t w) {
  float r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tadd.rn.f32.bf16 %0, b, %2;\n\t}" : "=f"(r) : "r"(w), "f"(-0.0f));
  return r;
}

// Four codes of (a, b, c, d) * s.
template <int FMT>
__device__ __forceinline__ uint32_t dp_codes(float a, float b, float c, float d, float s) {
  mul2(a, b, s, s);
  mul2(c, d, s, s);
  return cvt4<FMT>(a, b, c, d);
}

// Magnitude bits (as FP32 bits) of both halves of a packed maximum.
__device__ __forceinline__ uint32_t dp_lo(uint32_t m) { return (m & 0x7FFFu) << 16; }
__device__ __forceinline__ uint32_t dp_hi(uint32_t m) { return m & 0x7FFF0000u; }

// The packed maxima of 8 rows over the 16 lanes of a half-warp: at each step a
// lane hands half of its rows over and keeps the other half, so that 8
// shuffles do.  Lane hl ends with row dp_row_of(hl).
__device__ __forceinline__ int dp_row_of(int hl) { return (hl >> 1) & 7; }
__device__ __forceinline__ uint32_t dp_row_max(uint32_t (&m)[8], int hl) {
#pragma unroll
  for (int n = 4; n >= 1; n >>= 1) {  // lane distance 2 n
    const bool up = hl & (2 * n);
#pragma unroll
    for (int i = 0; i < n; i++) {
      const uint32_t give = up ? m[i] : m[i + n], keep = up ? m[i + n] : m[i];
      m[i] = absmax_nan_bf16x2(keep, __shfl_xor_sync(0xFFFFFFFFu, give, 2 * n));
    }
  }
  return absmax_nan_bf16x2(m[0], __shfl_xor_sync(0xFFFFFFFFu, m[0], 1));
}

// Row groups: 16 lanes a row, 8 rows (16 apart) a lane; nr, nc: rows and
// columns of the tile that are there.
template <int FMT>
__device__ __forceinline__ void dp_rows(const DispatchParams& p, const unsigned char* tile, int64_t r0, int tc, int nr,
                                        int nc) {
  const int hl = threadIdx.x & 15, half = threadIdx.x & 16, r = threadIdx.x >> 4;
  const unsigned char* from = tile + dp_off(r, hl * 8);  // 16 rows further: 2048 bytes, the same permutation
  uint4 v[8];
  uint32_t m[8];
#pragma unroll
  for (int i = 0; i < 8; i++) {
    v[i] = *(const uint4*)(from + 2048 * i);
    m[i] = absmax_nan_bf16x2(absmax_nan_bf16x2(v[i].x, v[i].y), absmax_nan_bf16x2(v[i].z, v[i].w));
  }
  const uint32_t packed = dp_row_max(m, hl);
  const uint32_t a = max(dp_lo(packed), dp_hi(packed));
  const float s = dp_scale<FMT>(a, p.pow2);
  const int mine = r + 16 * dp_row_of(hl);
  if (!(hl & 1) && mine < nr) p.s[(r0 + mine) * p.tiles_c + tc] = __frcp_rn(s);
  const bool nan = __any_sync(0xFFFFFFFFu, a > 0x7F800000u);
  uint8_t* at = p.q + (r0 + r) * p.cols + (int64_t)tc * kDpTile + hl * 8;
  const int64_t step = 16 * p.cols;
  const auto codes = [&](int i) {
    const float si = __shfl_sync(0xFFFFFFFFu, s, half | 2 * i);
    return make_uint2(dp_codes<FMT>(dp_flo(v[i].x), dp_fhi(v[i].x), dp_flo(v[i].y), dp_fhi(v[i].y), si),
                      dp_codes<FMT>(dp_flo(v[i].z), dp_fhi(v[i].z), dp_flo(v[i].w), dp_fhi(v[i].w), si));
  };
  if (nr == kDpTile && nc == kDpTile && !nan) {  // nearly every tile: nothing to ask for each row
#pragma unroll
    for (int i = 0; i < 8; i++, at += step) *(uint2*)at = codes(i);  // 6% faster than st_stream
  } else {
    const int there = hl * 8 < nc ? nr - r : 0;
#pragma unroll
    for (int i = 0; i < 8; i++, at += step) {
      uint2 o = codes(i);
      if (nan) o = make_uint2(canon_nan4<FMT>(o.x), canon_nan4<FMT>(o.y));
      if (16 * i < there) st_stream(at, o);
    }
  }
}

// 32 codes of one column group: one 32-byte store where the column's length
// allows, else 16 at a time, as many as there are.
__device__ __forceinline__ void dp_store(uint8_t* at, const uint32_t (&d)[8], bool wide, int left) {
  if (wide) {
    st32B(at, d);
  } else {
    st_stream(at, make_uint4(d[0], d[1], d[2], d[3]));
    if (left > 16) st_stream(at + 16, make_uint4(d[4], d[5], d[6], d[7]));
  }
}

// Column groups: a thread takes a column pair over 32 rows; the quarters of
// the rows meet in shared memory, where one thread a column divides.
template <int FMT>
__device__ __forceinline__ void dp_cols(const DispatchParams& p, const unsigned char* tile, int64_t r0, int tc, int nr,
                                        int nc, uint32_t (*quarters)[64], float* scale) {
  const int tid = threadIdx.x, pair = tid & 63, h = tid >> 6, c = 2 * pair;
  const int64_t c0 = (int64_t)tc * kDpTile;
  uint32_t w[32], m = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) {  // 8 rows further: 1024 bytes, the same permutation
    const unsigned char* from = tile + dp_off(32 * h + i, c);
#pragma unroll
    for (int j = 0; j < 4; j++) w[8 * j + i] = *(const uint32_t*)(from + 1024 * j);
  }
#pragma unroll
  for (int i = 0; i < 32; i++) m = absmax_nan_bf16x2(m, w[i]);
  quarters[h][pair] = m;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; k++) m = absmax_nan_bf16x2(m, quarters[k][pair]);
  if (tid < kDpTile) {
    // column c + h: the pairs' even columns by the first 64 threads, the odd by the next
    const float s = dp_scale<FMT>(h ? dp_hi(m) : dp_lo(m), p.pow2);
    scale[c + h] = s;
    if (c + h < nc) p.s_t[(c0 + c + h) * p.tiles_r + r0 / kDpTile] = __frcp_rn(s);
  }
  __syncthreads();
  const int left = nr - 32 * h;
  if (c >= nc || left <= 0) return;
  const bool wide = (p.rows & 31) == 0 && ((uintptr_t)p.q_t & 31) == 0;
  const float s0 = scale[c], s1 = scale[c + 1];
  uint32_t d0[8], d1[8];
#pragma unroll
  for (int k = 0; k < 8; k++) {
    d0[k] = dp_codes<FMT>(dp_flo(w[4 * k]), dp_flo(w[4 * k + 1]), dp_flo(w[4 * k + 2]), dp_flo(w[4 * k + 3]), s0);
    d1[k] = dp_codes<FMT>(dp_fhi(w[4 * k]), dp_fhi(w[4 * k + 1]), dp_fhi(w[4 * k + 2]), dp_fhi(w[4 * k + 3]), s1);
  }
  if (max(dp_lo(m), dp_hi(m)) > 0x7F800000u) {  // a NaN in a group
#pragma unroll
    for (int k = 0; k < 8; k++) {
      d0[k] = canon_nan4<FMT>(d0[k]);
      d1[k] = canon_nan4<FMT>(d1[k]);
    }
  }
  uint8_t* at = p.q_t + (c0 + c) * p.rows + r0 + 32 * h;
  dp_store(at, d0, wide, left);
  dp_store(at + p.rows, d1, wide, left);
}

template <int FMT, int DIR>
__global__ void __launch_bounds__(kDpThreads, 3) dispatch_kernel(DispatchParams p) {
  extern __shared__ __align__(128) unsigned char tiles[];  // two
  __shared__ uint32_t quarters[4][64];
  __shared__ float scale[kDpTile];
  const int part = threadIdx.x & 15, r = threadIdx.x >> 4;  // 16 lanes fetch one row's 256 bytes
  const int64_t r0 = (int64_t)blockIdx.x * kDpTile;
  const int tc0 = blockIdx.y * p.run, tc1 = min(tc0 + p.run, p.tiles_c);
  pdl_wait();
  const int nr = (int)min((int64_t)kDpTile, p.rows - r0);
  const uint16_t* from[8];  // the rows' values of this lane's column; padding: size 0
  uint32_t there = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int s = r + 16 * i < nr ? __ldg(p.src + r0 + r + 16 * i) : -1;
    const bool real = s >= 0 && s < p.slots;
    from[i] = p.x + (real ? (int64_t)(s / p.top_k) * p.cols + (int64_t)tc0 * kDpTile + part * 8 : 0);
    there |= (uint32_t)real << i;
  }
  const uint32_t to = smem_u32(tiles) + dp_off(r, part * 8);
  const auto load = [&](int tc) {
    const uint32_t dst = to + ((tc - tc0) & 1) * kDpTileBytes;
    const int64_t ahead = (int64_t)(tc - tc0) * kDpTile;
    // past the last column: size 0, and the row's start for an address
    const bool column = (int64_t)tc * kDpTile + part * 8 < p.cols;
    const uint32_t real = column ? there : 0;
#pragma unroll
    for (int i = 0; i < 8; i++)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + 2048 * i), "l"(from[i] + (column ? ahead : 0)),
                   "r"((real >> i & 1u) << 4)
                   : "memory");
  };
  load(tc0);
  asm volatile("cp.async.commit_group;" ::: "memory");
  for (int tc = tc0; tc < tc1; tc++) {
    if (tc + 1 < tc1) load(tc + 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    const unsigned char* tile = tiles + ((tc - tc0) & 1) * kDpTileBytes;
    const int nc = (int)min((int64_t)kDpTile, p.cols - (int64_t)tc * kDpTile);
    if constexpr (DIR & MXFP8_ROW) dp_rows<FMT>(p, tile, r0, tc, nr, nc);
    if constexpr (DIR & MXFP8_COL) dp_cols<FMT>(p, tile, r0, tc, nr, nc, quarters, scale);
    __syncthreads();  // the tile's place is loaded into next
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  pdl_launch_dependents();
}

template <int FMT, int DIR>
static fp8q_status launch_dispatch_d(DispatchParams p, cudaStream_t s) {
  static PerDevice<bool> allowed;
  const cudaError_t attr = allow_smem(allowed, dispatch_kernel<FMT, DIR>, 2 * kDpTileBytes);
  if (attr != cudaSuccess) return cuda_fail(attr, "dispatch shared memory");
  // Runs as long as leave every SM 12 CTAs, at most 16 tiles (65536 rows of
  // 7168, both copies, an earlier form: 311 us; runs of one tile 409, of a whole
  // row 346).
  const int64_t tiles = (int64_t)p.tiles_r * p.tiles_c, ctas = (int64_t)sm_count() * 12;
  p.run = (int)(tiles / ctas < 1 ? 1 : tiles / ctas > 16 ? 16 : tiles / ctas);
  const dim3 grid((unsigned)p.tiles_r, (unsigned)((p.tiles_c + p.run - 1) / p.run));
  const cudaError_t e = launch_kernel(dispatch_kernel<FMT, DIR>, grid, dim3(kDpThreads), 2 * kDpTileBytes, s, p);
  if (e != cudaSuccess) return cuda_fail(e, "dispatch kernel launch");
  return check_launch("dispatch kernel");
}

template <int FMT>
static fp8q_status launch_dispatch_f(const DispatchParams& p, int dir, cudaStream_t s) {
  if (dir == MXFP8_ROW) return launch_dispatch_d<FMT, MXFP8_ROW>(p, s);
  if (dir == MXFP8_COL) return launch_dispatch_d<FMT, MXFP8_COL>(p, s);
  return launch_dispatch_d<FMT, MXFP8_BOTH>(p, s);
}

static void plan_pieces(int64_t slots, int64_t* piece, int* pieces) {
  int64_t n = (slots + kPlanPiece - 1) / kPlanPiece;
  n = n < 1 ? 1 : n > kPlanMaxPieces ? kPlanMaxPieces : n;
  *piece = ((slots + n - 1) / n + 255) / 256 * 256;  // 32 slots a step for each of the warps
  *pieces = slots > 0 ? (int)((slots + *piece - 1) / *piece) : 1;
}

static fp8q_status check_plan(int64_t slots, int32_t experts, int32_t align) {
  if (slots < 0) return fail(FP8Q_ERR_INVALID_ARG, "slots must be >= 0");
  if (experts < 1) return fail(FP8Q_ERR_INVALID_ARG, "experts must be >= 1");
  if (experts > kPlanMaxExperts) return fail(FP8Q_ERR_UNSUPPORTED, "a plan serves at most %d experts", kPlanMaxExperts);
  if (align < 1 || align > 4096) return fail(FP8Q_ERR_INVALID_ARG, "align must be in [1, 4096]");
  if (slots > INT32_MAX - (int64_t)experts * align) return fail(FP8Q_ERR_UNSUPPORTED, "too many slots");
  return FP8Q_OK;
}

}  // namespace fp8q

using namespace fp8q;

extern "C" int64_t fp8q_moe_rows(int64_t slots, int32_t experts, int32_t align) {
  if (slots < 0 || experts < 1 || align < 1) return -1;
  const int64_t used = slots < experts ? slots : experts;
  return (slots + used * (align - 1)) / align * align;
}

extern "C" size_t fp8q_moe_plan_workspace_bytes(int64_t slots, int32_t experts) {
  if (slots < 0 || experts < 1) return 0;
  int64_t piece;
  int pieces;
  plan_pieces(slots, &piece, &pieces);
  return pieces > 1 ? (size_t)pieces * experts * sizeof(int) : 0;
}

extern "C" fp8q_status fp8q_moe_plan(const int32_t* ids, int64_t slots, int32_t experts, int32_t align, int64_t rows,
                                     int64_t* offsets, int32_t* row_of, int32_t* src, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  clear_error();
  const fp8q_status r = check_plan(slots, experts, align);
  if (r != FP8Q_OK) return r;
  if (rows < fp8q_moe_rows(slots, experts, align))
    return fail(FP8Q_ERR_INVALID_ARG, "rows (%lld) is below fp8q_moe_rows() = %lld", (long long)rows,
                (long long)fp8q_moe_rows(slots, experts, align));
  if (rows > INT32_MAX) return fail(FP8Q_ERR_UNSUPPORTED, "too many rows");
  if (!offsets || ((uintptr_t)offsets & 7)) return fail(FP8Q_ERR_INVALID_ARG, "offsets must be an 8-byte aligned device pointer");
  if (slots > 0 && (!ids || !row_of || ((uintptr_t)ids & 3) || ((uintptr_t)row_of & 3)))
    return fail(FP8Q_ERR_INVALID_ARG, "ids and row_of must be 4-byte aligned device pointers");
  if (rows > 0 && (!src || ((uintptr_t)src & 3))) return fail(FP8Q_ERR_INVALID_ARG, "src must be a 4-byte aligned device pointer");
  const size_t need = fp8q_moe_plan_workspace_bytes(slots, experts);
  if (need > 0 && (!workspace || ((uintptr_t)workspace & 3) || workspace_bytes < need))
    return fail(FP8Q_ERR_INVALID_ARG, "workspace must be a 4-byte aligned device pointer to %zu bytes", need);
  PlanParams p{};
  p.ids = ids;
  p.slots = slots;
  plan_pieces(slots, &p.piece, &p.pieces);
  p.experts = experts;
  p.align = align;
  p.rows = rows;
  p.offsets = offsets;
  p.row_of = row_of;
  p.src = src;
  p.counts = (int*)workspace;
  const cudaStream_t s = (cudaStream_t)stream;
  if (p.pieces > 1) {
    const cudaError_t e = launch_kernel(plan_count_kernel, dim3(p.pieces), dim3(kPlanThreads), 0, s, p);
    if (e != cudaSuccess) return cuda_fail(e, "plan kernel launch");
  }
  const cudaError_t e = launch_kernel(plan_place_kernel, dim3(p.pieces), dim3(kPlanThreads),
                                      (size_t)kPlanWarps * experts * sizeof(int), s, p);
  if (e != cudaSuccess) return cuda_fail(e, "plan kernel launch");
  return check_launch("plan kernel");
}

extern "C" fp8q_status fp8q_moe_dispatch(const void* x, int32_t dt, int64_t tokens, int64_t cols, int32_t top_k,
                                         const int32_t* src, int64_t rows, int32_t fmt, int32_t pow2_scales,
                                         int32_t dir, uint8_t* q, float* scale_inv, uint8_t* q_t, float* scale_inv_t,
                                         void* stream) {
  clear_error();
  if (dt != FP8Q_IN_BF16 && dt != FP8Q_IN_FP32) return fail(FP8Q_ERR_INVALID_ARG, "dt must be FP8Q_IN_BF16 or FP8Q_IN_FP32");
  if (dt != FP8Q_IN_BF16) return fail(FP8Q_ERR_UNSUPPORTED, "dispatch takes BF16 input");
  if (fmt != FP8Q_E4M3 && fmt != FP8Q_E5M2) return fail(FP8Q_ERR_INVALID_ARG, "fmt must be FP8Q_E4M3 or FP8Q_E5M2");
  if (dir != MXFP8_ROW && dir != MXFP8_COL && dir != MXFP8_BOTH)
    return fail(FP8Q_ERR_INVALID_ARG, "dir must be MXFP8_ROW, MXFP8_COL or MXFP8_BOTH");
  if (tokens < 0 || cols < 0 || rows < 0) return fail(FP8Q_ERR_INVALID_ARG, "tokens, cols and rows must be >= 0");
  if (top_k < 1) return fail(FP8Q_ERR_INVALID_ARG, "top_k must be >= 1");
  if (cols % 16 != 0) return fail(FP8Q_ERR_UNSUPPORTED, "dispatch needs cols %% 16 == 0");
  if ((dir & MXFP8_COL) && rows % 16 != 0) return fail(FP8Q_ERR_UNSUPPORTED, "the transposed copy needs rows %% 16 == 0");
  if (rows > INT32_MAX || tokens > INT32_MAX / top_k || cols > 65535 * (int64_t)kDpTile)
    return fail(FP8Q_ERR_UNSUPPORTED, "tokens, cols or rows too large");
  if (rows * cols == 0) return FP8Q_OK;
  if ((tokens > 0 && !x) || ((uintptr_t)x & 15)) return fail(FP8Q_ERR_INVALID_ARG, "x must be a 16-byte aligned device pointer");
  if (!src || ((uintptr_t)src & 3)) return fail(FP8Q_ERR_INVALID_ARG, "src must be a 4-byte aligned device pointer");
  if ((dir & MXFP8_ROW) && (!q || !scale_inv || ((uintptr_t)q & 15) || ((uintptr_t)scale_inv & 3)))
    return fail(FP8Q_ERR_INVALID_ARG, "q (16-byte aligned) and scale_inv are required for the rowwise copy");
  if ((dir & MXFP8_COL) && (!q_t || !scale_inv_t || ((uintptr_t)q_t & 15) || ((uintptr_t)scale_inv_t & 3)))
    return fail(FP8Q_ERR_INVALID_ARG, "q_t (16-byte aligned) and scale_inv_t are required for the transposed copy");
  DispatchParams p{};
  p.rows = rows;
  p.cols = cols;
  p.tiles_r = (int)((rows + kDpTile - 1) / kDpTile);
  p.tiles_c = (int)((cols + kDpTile - 1) / kDpTile);
  p.pow2 = pow2_scales ? 1 : 0;
  p.q = q;
  p.s = scale_inv;
  p.q_t = q_t;
  p.s_t = scale_inv_t;
  p.x = (const uint16_t*)x;
  p.src = src;
  p.slots = tokens * top_k;
  p.top_k = top_k;
  return fmt == FP8Q_E4M3 ? launch_dispatch_f<kE4M3>(p, dir, (cudaStream_t)stream)
                          : launch_dispatch_f<kE5M2>(p, dir, (cudaStream_t)stream);
}
