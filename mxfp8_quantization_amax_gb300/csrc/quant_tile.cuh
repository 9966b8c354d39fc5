// quant_tile.cuh -- blockwise FP8 copies of values that a kernel computes on
// the way, for the norm and the gated activation: FP32 values in registers go
// straight to codes, with the arithmetic of the blockwise quantizer.  Per group
// of 128: scale = fl32(F8max / amax) with the per-tensor special cases, code =
// RNE_sat(fl32(v * scale)), fl32(1 / scale) stored.
//
// Two shapes.  Rows alone: 16 lanes hold a group, 8 values each.  Both copies
// (or the transposed one): a CTA of 256 threads holds a tile of 128 x 128, a
// thread 8 x 8 of it, so that row groups meet in a half-warp and column groups
// in shared memory, and neither copy needs the values a second time.
#pragma once

#include "fp8q_device.cuh"
#include "internal.h"

namespace fp8q {

template <int FMT>
__device__ __forceinline__ float qt_scale(float amax, int pow2) {
  const float s = scale_from_amax(__float_as_uint(amax) & 0x7FFFFFFFu, Fmt<FMT>::kMax, 0);
  return pow2 ? __uint_as_float(__float_as_uint(s) & 0xFF800000u) : s;  // s is a positive normal float
}

// The largest of two magnitudes (sign bit 0, NaN above all else), of three values' magnitudes.
__device__ __forceinline__ float qt_max(float a, float b) {
  return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
}
__device__ __forceinline__ float qt_max(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float qt_max8(const float (&v)[8]) {
  return qt_max(qt_max(qt_max(v[0], v[1], v[2]), v[3], v[4]), qt_max(v[5], v[6], v[7]));
}

// V consecutive values of type DT (kBF16, kFP32) as FP32, read once.  V = 8
// takes 16-byte loads, V = 1 any place.
template <int DT, int V>
struct QtRaw {
  uint4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    if constexpr (V == 8) {
      if constexpr (DT == kBF16) {
        a = ld_stream((const uint16_t*)p + i);
      } else {
        a = ld_stream((const float*)p + i);
        b = ld_stream((const float*)p + i + 4);
      }
    } else {
      a.x = DT == kBF16 ? (uint32_t)__ldg((const uint16_t*)p + i) << 16 : __ldg((const uint32_t*)p + i);
    }
  }
  __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&v)[V]) const {
    if constexpr (V == 8 && DT == kBF16) {
      v[0] = bf16_lo(a.x), v[1] = bf16_hi(a.x), v[2] = bf16_lo(a.y), v[3] = bf16_hi(a.y);
      v[4] = bf16_lo(a.z), v[5] = bf16_hi(a.z), v[6] = bf16_lo(a.w), v[7] = bf16_hi(a.w);
    } else if constexpr (V == 8) {
      v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
      v[4] = __uint_as_float(b.x), v[5] = __uint_as_float(b.y), v[6] = __uint_as_float(b.z), v[7] = __uint_as_float(b.w);
    } else {
      v[0] = __uint_as_float(a.x);
    }
  }
};

__device__ __forceinline__ uint32_t qt_pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// V consecutive values to type DT, one rounding; with `back`, v gets what was stored.
template <int DT, int V>
__device__ __forceinline__ void qt_store(void* p, int64_t i, float (&v)[V], bool back = false) {
  if constexpr (DT == kBF16) {
    uint16_t* q = (uint16_t*)p + i;
    if constexpr (V == 8) {
      const uint4 u = make_uint4(qt_pack(v[0], v[1]), qt_pack(v[2], v[3]), qt_pack(v[4], v[5]), qt_pack(v[6], v[7]));
      st_stream(q, u);
      if (back) {
        v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
        v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
      }
    } else {
      const uint32_t u = qt_pack(v[0], 0.0f);
      *q = (uint16_t)u;
      if (back) v[0] = bf16_lo(u);
    }
  } else {
    float* q = (float*)p + i;
    if constexpr (V == 8) {
      st_stream(q, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
      st_stream(q + 4, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
    } else {
      *q = v[0];
    }
  }
}

template <int FMT>
__device__ __forceinline__ uint32_t qt_codes4(float a, float b, float c, float d, float s) {
  mul2(a, b, s, s);
  mul2(c, d, s, s);
  return cvt4<FMT>(a, b, c, d);
}

// One row group: 16 lanes (hl = lane & 15) of 8 values each.  All lanes of the
// warp come here; `there`: the lane's values lie in the matrix (others are 0).
template <int FMT>
__device__ __forceinline__ void qt_group(const float (&v)[8], int pow2, uint8_t* q, float* scale_inv, bool there, int hl) {
  float m = qt_max8(v);
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) m = qt_max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  const float s = qt_scale<FMT>(m, pow2);
  uint2 c = make_uint2(qt_codes4<FMT>(v[0], v[1], v[2], v[3], s), qt_codes4<FMT>(v[4], v[5], v[6], v[7], s));
  if (!(m <= 3.40282346638528859812e+38f)) c = make_uint2(canon_nan4<FMT>(c.x), canon_nan4<FMT>(c.y));
  if (there) {
    st_stream(q, c);
    if (hl == 0) *scale_inv = __frcp_rn(s);
  }
}

// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------
constexpr int kQtTile = 128;
constexpr int kQtThreads = 256;

struct QtOut {
  int64_t rows, cols;  // of the quantized matrix
  int tiles_r, tiles_c;
  int pow2;
  int apart;    // tile columns are taken in the order 0, half, 1, half + 1, ...: two halves of the columns share inputs
  void* dense;  // the values in the source's type, or NULL
  uint8_t* q;   // row copy, or NULL
  float* s;
  uint8_t* q_t;
  float* s_t;
};

// A source gives the values of 8 columns of 8 rows; its type is that of the
// dense output:
//   static constexpr int kType;
//   void tile(float (&v)[8][8], int64_t row, int64_t col, int64_t rows) const;   // rows from `rows` on are 0
template <class Src, int FMT, bool ROW>
__global__ void __launch_bounds__(kQtThreads, 2) quant_tile_kernel(Src src, QtOut o) {
  __shared__ float part[kQtThreads / 32][kQtTile];
  __shared__ float scale[kQtTile];
  __shared__ int odd[1];                               // some group holds Inf or NaN
  __shared__ __align__(16) uint8_t stage[kQtTile * 128];  // codes of the transposed tile
  const int tid = threadIdx.x, lane = tid & 31, hl = tid & 15, ty = tid >> 4;
  pdl_wait();
  const int64_t tr = blockIdx.x / o.tiles_c;
  int tc = (int)(blockIdx.x - tr * o.tiles_c);
  if (o.apart) tc = (tc & 1) ? (o.tiles_c + 1) / 2 + tc / 2 : tc / 2;
  const int64_t r0 = tr * kQtTile + ty * 8, c0 = (int64_t)tc * kQtTile, c = c0 + hl * 8;
  const bool col_ok = c < o.cols;
  float v[8][8];
  if (col_ok) {
    src.tile(v, r0, c, o.rows);
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++)
#pragma unroll
      for (int k = 0; k < 8; k++) v[i][k] = 0.0f;
  }
  if (tid == 0) odd[0] = 0;
  // columns: 8 rows of a thread, 16 of a warp, 128 of the CTA
  {
    float m[8];
#pragma unroll
    for (int k = 0; k < 8; k++)
      m[k] = qt_max(qt_max(qt_max(v[0][k], v[1][k], v[2][k]), v[3][k], v[4][k]), qt_max(v[5][k], v[6][k], v[7][k]));
    const bool up = lane & 16;  // each half-warp keeps four of the columns
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const float give = up ? m[k] : m[k + 4], keep = up ? m[k + 4] : m[k];
      m[k] = qt_max(keep, __shfl_xor_sync(0xFFFFFFFFu, give, 16));
    }
    *(float4*)&part[tid >> 5][hl * 8 + (up ? 4 : 0)] = make_float4(m[0], m[1], m[2], m[3]);
  }
  if (o.dense != nullptr && col_ok) {
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (r0 + i < o.rows) qt_store<Src::kType, 8>(o.dense, (r0 + i) * o.cols + c, v[i]);
  }
  __syncthreads();
  if (tid < kQtTile) {
    float m = part[0][tid];
#pragma unroll
    for (int w = 1; w < kQtThreads / 32; w++) m = qt_max(m, part[w][tid]);
    const float s = qt_scale<FMT>(m, o.pow2);
    scale[tid] = s;
    if (!(m <= 3.40282346638528859812e+38f)) odd[0] = 1;
    if (c0 + tid < o.cols) o.s_t[(c0 + tid) * o.tiles_r + tr] = __frcp_rn(s);
  }
  if constexpr (ROW) {
    // rows: at each step a lane hands half of its rows over and keeps the other
    // half; lane hl ends with row (hl >> 1) & 7 of the thread's 8
    float m[8];
#pragma unroll
    for (int i = 0; i < 8; i++) m[i] = qt_max8(v[i]);
#pragma unroll
    for (int n = 4; n >= 1; n >>= 1) {
      const bool up = hl & (2 * n);
#pragma unroll
      for (int i = 0; i < n; i++) {
        const float give = up ? m[i] : m[i + n], keep = up ? m[i + n] : m[i];
        m[i] = qt_max(keep, __shfl_xor_sync(0xFFFFFFFFu, give, 2 * n));
      }
    }
    m[0] = qt_max(m[0], __shfl_xor_sync(0xFFFFFFFFu, m[0], 1));
    const float s = qt_scale<FMT>(m[0], o.pow2);
    const int64_t mine = r0 + ((hl >> 1) & 7);
    if (!(hl & 1) && mine < o.rows) o.s[mine * o.tiles_c + tc] = __frcp_rn(s);
    const bool nan = __any_sync(0xFFFFFFFFu, !(m[0] <= 3.40282346638528859812e+38f));
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float si = __shfl_sync(0xFFFFFFFFu, s, (lane & 16) | 2 * i);
      uint2 u = make_uint2(qt_codes4<FMT>(v[i][0], v[i][1], v[i][2], v[i][3], si),
                           qt_codes4<FMT>(v[i][4], v[i][5], v[i][6], v[i][7], si));
      if (nan) u = make_uint2(canon_nan4<FMT>(u.x), canon_nan4<FMT>(u.y));
      if (col_ok && r0 + i < o.rows) *(uint2*)(o.q + (r0 + i) * o.cols + c) = u;
    }
  }
  __syncthreads();
  {
    const float4 a = *(const float4*)&scale[hl * 8], b = *(const float4*)&scale[hl * 8 + 4];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      mul2(v[i][0], v[i][1], a.x, a.y);
      mul2(v[i][2], v[i][3], a.z, a.w);
      mul2(v[i][4], v[i][5], b.x, b.y);
      mul2(v[i][6], v[i][7], b.z, b.w);
    }
    const bool nan = odd[0];
#pragma unroll
    for (int k = 0; k < 8; k++) {
      uint2 u = make_uint2(cvt4<FMT>(v[0][k], v[1][k], v[2][k], v[3][k]), cvt4<FMT>(v[4][k], v[5][k], v[6][k], v[7][k]));
      if (nan) u = make_uint2(canon_nan4<FMT>(u.x), canon_nan4<FMT>(u.y));
      // 8-byte piece ty of the column's 128 rows, permuted by the thread's columns: 16 lanes hit 16 places
      *(uint2*)(stage + (hl * 8 + k) * 128 + ((ty ^ hl) << 3)) = u;
    }
  }
  __syncthreads();
  const int64_t rt = tr * kQtTile;
  const bool wide = o.rows % 32 == 0 && ((uintptr_t)o.q_t & 31) == 0;
#pragma unroll
  for (int n = 0; n < 2; n++) {  // 32 rows of a column: four threads a column
    const int col = (tid >> 2) + 64 * n, at = tid & 3, flip = col >> 3;
    const int64_t row = rt + 32 * at;
    if (c0 + col >= o.cols || row >= o.rows) continue;
    uint4 a = *(const uint4*)(stage + col * 128 + (((2 * at) ^ (flip >> 1)) << 4));
    uint4 b = *(const uint4*)(stage + col * 128 + (((2 * at + 1) ^ (flip >> 1)) << 4));
    if (flip & 1) {
      a = make_uint4(a.z, a.w, a.x, a.y);
      b = make_uint4(b.z, b.w, b.x, b.y);
    }
    uint8_t* to = o.q_t + (c0 + col) * o.rows + row;
    if (wide) {
      const uint32_t d[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      st32B(to, d);
    } else {
      st_stream(to, a);
      if (row + 16 < o.rows) st_stream(to + 16, b);
    }
  }
  pdl_launch_dependents();
}

template <class Src, int FMT>
cudaError_t launch_quant_tiles(const Src& src, const QtOut& o, cudaStream_t s) {
  const dim3 grid((unsigned)((int64_t)o.tiles_r * o.tiles_c));
  return o.q ? launch_kernel(quant_tile_kernel<Src, FMT, true>, grid, dim3(kQtThreads), 0, s, src, o)
             : launch_kernel(quant_tile_kernel<Src, FMT, false>, grid, dim3(kQtThreads), 0, s, src, o);
}

// Checks of the copies' arguments, for cols columns.
inline fp8q_status qt_check(int64_t rows, int64_t cols, int32_t fmt, int32_t dir, const uint8_t* q, const float* s,
                            const uint8_t* q_t, const float* s_t) {
  const auto off = [](const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) != 0; };
  if (fmt != FP8Q_E4M3 && fmt != FP8Q_E5M2) return fail(FP8Q_ERR_INVALID_ARG, "fmt must be FP8Q_E4M3 or FP8Q_E5M2");
  if (dir < 0 || dir > MXFP8_BOTH) return fail(FP8Q_ERR_INVALID_ARG, "dir must be 0, MXFP8_ROW, MXFP8_COL or MXFP8_BOTH");
  if (dir && cols % 16 != 0) return fail(FP8Q_ERR_UNSUPPORTED, "the copies need a multiple of 16 columns");
  if ((dir & MXFP8_COL) && rows % 16 != 0) return fail(FP8Q_ERR_UNSUPPORTED, "the transposed copy needs rows %% 16 == 0");
  if (rows * cols == 0) return FP8Q_OK;
  if ((dir & MXFP8_ROW) && (!q || !s || off(q, 16) || off(s, 4)))
    return fail(FP8Q_ERR_INVALID_ARG, "q (16-byte aligned) and scale_inv are required for the rowwise copy");
  if ((dir & MXFP8_COL) && (!q_t || !s_t || off(q_t, 16) || off(s_t, 4)))
    return fail(FP8Q_ERR_INVALID_ARG, "q_t (16-byte aligned) and scale_inv_t are required for the transposed copy");
  return FP8Q_OK;
}

}  // namespace fp8q
