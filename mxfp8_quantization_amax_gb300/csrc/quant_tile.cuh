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
//
// Bound by memory and issue together: the activation of 65536 x 2048 in both
// copies 128 us (6.3 TB/s); an earlier form 158 with a CTA a tile, 124 with CTAs
// that stay and have the next inputs on their way.
#pragma once

#include "fp8q_device.cuh"
#include "internal.h"

namespace fp8q {

template <int FMT>
__device__ __forceinline__ float qt_scale(float amax, int pow2) {
  const float s = scale_from_amax(__float_as_uint(amax) & 0x7FFFFFFFu, Fmt<FMT>::kMax, 0);
  return pow2 ? __uint_as_float(__float_as_uint(s) & 0xFF800000u) : s;  // s is a positive normal float
}

// Every NaN becomes code 0x7F in both formats: what the conversion itself gives
// for all payloads and signs.

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

// The halves of a BF16 pair as FP32: a mixed addition of -0, exact, which leaves
// the integer pipe to the conversions and maxima.
__device__ __forceinline__ void qt_halves(uint32_t w, float& lo, float& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tadd.rn.f32.bf16 %0, a, %3;\n\tadd.rn.f32.bf16 %1, b, %3;\n\t}"
      : "=f"(lo), "=f"(hi) : "r"(w), "f"(-0.0f));
}

// V consecutive values of type DT (kBF16, kFP32), read once.  V = 8 takes
// 16-byte loads, V = 1 any place.
template <int DT, int V>
struct QtRaw {
  static constexpr int kPair = V == 8 ? DT : kFP32;  // how pair() gives two values
  uint4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    if constexpr (V == 8) {
      if constexpr (DT == kBF16) {
        a = ld_stream((const uint16_t*)p + i);
      } else {
        const float* q = (const float*)p + i;
        if (((uintptr_t)q & 31) == 0) {  // whole sectors
          asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                       : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                       : "l"(q));
        } else {
          a = ld_stream(q);
          b = ld_stream(q + 4);
        }
      }
    } else {
      a.x = DT == kBF16 ? (uint32_t)__ldg((const uint16_t*)p + i) << 16 : __ldg((const uint32_t*)p + i);
    }
  }
  __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
  // values 2 k and 2 k + 1: a BF16 pair in x, or FP32 bits in both
  __device__ __forceinline__ uint2 pair(int k) const {
    if constexpr (V == 1) return make_uint2(a.x, a.x);
    if constexpr (DT == kBF16) return make_uint2(k == 0 ? a.x : k == 1 ? a.y : k == 2 ? a.z : a.w, 0);
    return k == 0 ? make_uint2(a.x, a.y) : k == 1 ? make_uint2(a.z, a.w) : k == 2 ? make_uint2(b.x, b.y) : make_uint2(b.z, b.w);
  }
  __device__ __forceinline__ void get(float (&v)[V]) const {
    if constexpr (V == 8 && DT == kBF16) {
      qt_halves(a.x, v[0], v[1]);
      qt_halves(a.y, v[2], v[3]);
      qt_halves(a.z, v[4], v[5]);
      qt_halves(a.w, v[6], v[7]);
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
      const uint32_t u[8] = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]),
                             __float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
      if (((uintptr_t)q & 31) == 0) {  // whole sectors
        st32B(q, u);
      } else {
        st_stream(q, make_uint4(u[0], u[1], u[2], u[3]));
        st_stream(q + 4, make_uint4(u[4], u[5], u[6], u[7]));
      }
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

// 16 bytes into shared memory while other work goes on.
__device__ __forceinline__ void qt_ask(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
// The first `bytes` of them, zeros behind.
__device__ __forceinline__ void qt_ask(uint32_t to, const void* from, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void qt_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void qt_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}
__device__ __forceinline__ uint4 qt_taken(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

// Eight values for each of G consecutive lanes of a warp (lane g of them), which
// lie side by side from value i of p on and of which `left` are there: asked
// for in whole sectors, so that FP32 lanes read what others asked for (with a
// __syncwarp between, both ways).  ENDS: the run may end anywhere.
template <int DT>
constexpr int kQtRunBytes = DT == kBF16 ? 16 : 32;  // of a lane

template <int DT, int G, bool ENDS = false>
__device__ __forceinline__ void qt_ask8(const void* p, int64_t i, int64_t left, uint32_t place, int g) {
  const uint8_t* from = (const uint8_t*)p + i * (DT == kBF16 ? 2 : 4);
#pragma unroll
  for (int k = 0; k < kQtRunBytes<DT> / 16; k++) {
    const int u = k * G + g;
    if (u * (DT == kBF16 ? 8 : 4) < left) {
      if constexpr (ENDS) qt_ask(place + 16 * u, from + 16 * u, (int)min((int64_t)16, left * (DT == kBF16 ? 2 : 4) - 16 * u));
      else qt_ask(place + 16 * u, from + 16 * u);
    }
  }
}
template <int DT>
__device__ __forceinline__ void qt_taken8(uint32_t place, int g, QtRaw<DT, 8>& raw) {
  raw.a = qt_taken(place + kQtRunBytes<DT> * g);
  if constexpr (DT == kFP32) raw.b = qt_taken(place + 32 * g + 16);
}

// The maxima of R row groups over the 16 lanes of a half-warp: at each step a
// lane hands half of its groups over and keeps the other half, until 16 / R
// lanes share one.  Lane hl ends with the maximum of group hl / (16 / R), and
// one division serves a group.
template <int R>
__device__ __forceinline__ float qt_group_max(float (&m)[R], int hl) {
  constexpr int kLanes = 16 / R;
#pragma unroll
  for (int n = R / 2; n >= 1; n >>= 1) {
    const bool up = hl & (kLanes * n);
#pragma unroll
    for (int i = 0; i < n; i++) {
      const float give = up ? m[i] : m[i + n], keep = up ? m[i + n] : m[i];
      m[i] = qt_max(keep, __shfl_xor_sync(0xFFFFFFFFu, give, kLanes * n));
    }
  }
#pragma unroll
  for (int n = kLanes / 2; n >= 1; n >>= 1) m[0] = qt_max(m[0], __shfl_xor_sync(0xFFFFFFFFu, m[0], n));
  return m[0];
}

// R row groups: 16 lanes (hl = lane & 15) of 8 values each.  All lanes of the
// warp come here.  codes(i) is where group i's go and scale(i) its 1 / scale;
// there(i): the lane's values of group i lie in the matrix (others are 0).
template <int FMT, int R, class Codes, class Scale, class There>
__device__ __forceinline__ void qt_groups(const float (&v)[R][8], int pow2, Codes codes, Scale scale, There there) {
  constexpr int kLanes = 16 / R;
  const int lane = threadIdx.x & 31, hl = lane & 15;
  float m[R];
#pragma unroll
  for (int i = 0; i < R; i++) m[i] = qt_max8(v[i]);
  const float s = qt_scale<FMT>(qt_group_max<R>(m, hl), pow2), inv = __frcp_rn(s);
#pragma unroll
  for (int i = 0; i < R; i++) {
    const float si = __shfl_sync(0xFFFFFFFFu, s, (lane & 16) | kLanes * i), vi = __shfl_sync(0xFFFFFFFFu, inv, (lane & 16) | kLanes * i);
    if (there(i)) {
      *(uint2*)codes(i) = make_uint2(qt_codes4<FMT>(v[i][0], v[i][1], v[i][2], v[i][3], si), qt_codes4<FMT>(v[i][4], v[i][5], v[i][6], v[i][7], si));
      if (hl == 0) *scale(i) = vi;
    }
  }
}

// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------
constexpr int kQtTile = 128;
constexpr int kQtRows = 8;                                // rows of a thread (4: 3 to 6% slower)
constexpr int kQtThreads = kQtTile * kQtTile / 8 / kQtRows;

struct QtOut {
  int64_t rows, cols;  // of the quantized matrix
  int tiles_r, tiles_c;
  int pow2;
  void* dense;  // the values in the source's type, or NULL
  uint8_t* q;   // row copy, or NULL
  float* s;
  uint8_t* q_t;
  float* s_t;
};

// A source gives 8 values of a row (columns come in multiples of 16, and for the transposed copy rows do)
// from kInputs runs of 8 inputs of type kType, which is the dense output's too:
//   bool needs(int input, int col) const;
//   const void* at(int input, int row, int col) const;
//   int pitch(int input) const;                             // values from a row to the next
//   void begin(int row, int col);                           // of kQtRows rows
//   void values(const QtRaw<kType, 8> (&in)[kInputs], int i, int col, float (&v)[8]) const;   // of row + i
// and, where both halves of the columns have the same inputs (kHalves),
//   void both(const QtRaw<kType, 8> (&in)[kInputs], float (&first)[8], float (&second)[8]) const;
template <class Src>
constexpr size_t kQtSmem = (size_t)kQtRows * Src::kInputs * kQtThreads * kQtRunBytes<Src::kType>;

// What a half-warp asks for: the values of its `rows` rows (ALL: kQtRows or none)
// from column col on.
template <class Src, bool ALL>
__device__ __forceinline__ void qt_ask_tile(const Src& src, int row, int col, int cols, int rows, uint32_t place, int hl) {
  constexpr int kSize = Src::kType == kBF16 ? 2 : 4, kRun = kQtRunBytes<Src::kType>;
  if (rows > 0) {
#pragma unroll
    for (int n = 0; n < Src::kInputs; n++) {
#pragma unroll
      for (int k = 0; k < kRun / 16; k++) {
        // (a half-warp's columns may lie in two halves with different inputs: each lane asks for its own then)
        const int c = col + (k * 16 + hl) * (16 / kSize);
        if (c < cols && src.needs(n, c)) {
          const uint8_t* from = (const uint8_t*)src.at(n, row, c);
          const int64_t pitch = (int64_t)src.pitch(n) * kSize;
#pragma unroll
          for (int i = 0; i < kQtRows; i++)
            if (ALL || i < rows) qt_ask(place + (i * Src::kInputs + n) * kQtThreads * kRun + (k * 16 + hl) * 16, from + i * pitch);
        }
      }
    }
  }
  qt_commit();
}

// Persistent: the inputs of a CTA's next tile come while it works on this one.
// PAIR: the tiles of both halves come from one set of inputs; the second half's
// values wait where its inputs were.  Without COL (any number of rows) no barrier
// is left: a half-warp has its rows to itself.
template <class Src, int FMT, bool ROW, bool COL, bool PAIR>
__global__ void __launch_bounds__(kQtThreads, 2) quant_tile_kernel(Src src, QtOut o) {
  extern __shared__ __align__(16) uint8_t inputs[];  // [rows of a thread][inputs][threads] of 8 values
  __shared__ float scale[COL ? kQtTile : 1];
  __shared__ __align__(16) uint8_t stage[COL ? kQtTile * 128 : 16];  // codes of the transposed tile; the warps' column maxima before
  float(*part)[kQtTile] = (float(*)[kQtTile])stage;
  constexpr int kRun = kQtRunBytes<Src::kType>;
  const int tid = threadIdx.x, lane = tid & 31, hl = tid & 15, ty = tid >> 4, all_rows = (int)o.rows, all_cols = (int)o.cols;
  const uint32_t place = (uint32_t)__cvta_generic_to_shared(inputs) + ty * 16 * kRun;  // of the half-warp
  const int items_c = PAIR ? o.tiles_c / 2 : o.tiles_c, items = o.tiles_r * items_c, cols = PAIR ? all_cols / 2 : all_cols;
  const bool wide = all_rows % 32 == 0 && ((uintptr_t)o.q_t & 31) == 0;
  pdl_wait();
  const auto place_of = [&](int item, int& tr, int& tc) {
    tr = item / items_c;
    tc = item - tr * items_c;
    if (Src::kHalves && !PAIR) tc = (tc & 1) ? (items_c + 1) / 2 + tc / 2 : tc / 2;
  };
  const auto ask = [&](int tr, int tc) {
    const int row = tr * kQtTile + ty * kQtRows;
    qt_ask_tile<Src, COL>(src, row, tc * kQtTile, cols, all_rows - row, place, hl);
  };
  // where the second half's values of row i wait: 32 bytes of the thread's own
  const auto waits = [&](int i, int k) {
    return kRun == 32 ? place + i * Src::kInputs * kQtThreads * 32 + hl * 32 + k * 16 : place + (i * Src::kInputs + k) * kQtThreads * 16 + hl * 16;
  };
  int tr, tc, half = 0, item = blockIdx.x;
  place_of(item, tr, tc);
  ask(tr, tc);
  while (item < items) {
    const int this_r = tr, this_c = tc + half * items_c;
    const int rt = tr * kQtTile, r0 = rt + ty * kQtRows, c0 = this_c * kQtTile, c = c0 + hl * 8;
    const bool there = c < all_cols && r0 < all_rows;
    const int rows = COL ? kQtRows : all_rows - r0;  // of the thread's; of others the values are anything
    float v[kQtRows][8];
    if (there) src.begin(r0, c);
    if (!PAIR || half == 0) {
      qt_wait<0>();
      __syncwarp();
      if (there) {
#pragma unroll
        for (int i = 0; i < kQtRows; i++) {
          QtRaw<Src::kType, 8> in[Src::kInputs];
#pragma unroll
          for (int n = 0; n < Src::kInputs; n++)
            if (PAIR || src.needs(n, c)) qt_taken8<Src::kType>(place + (i * Src::kInputs + n) * kQtThreads * kRun, hl, in[n]);
          if constexpr (PAIR) {
            float second[8];
            src.both(in, v[i], second);
#pragma unroll
            for (int k = 0; k < 2; k++)
              asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(waits(i, k)), "f"(second[4 * k]), "f"(second[4 * k + 1]),
                           "f"(second[4 * k + 2]), "f"(second[4 * k + 3])
                           : "memory");
          } else {
            src.values(in, i, c, v[i]);
          }
        }
      }
    } else if (there) {
#pragma unroll
      for (int i = 0; i < kQtRows; i++) {
        const uint4 a = qt_taken(waits(i, 0)), b = qt_taken(waits(i, 1));
        v[i][0] = __uint_as_float(a.x), v[i][1] = __uint_as_float(a.y), v[i][2] = __uint_as_float(a.z), v[i][3] = __uint_as_float(a.w);
        v[i][4] = __uint_as_float(b.x), v[i][5] = __uint_as_float(b.y), v[i][6] = __uint_as_float(b.z), v[i][7] = __uint_as_float(b.w);
      }
    }
    if (!there) {
#pragma unroll
      for (int i = 0; i < kQtRows; i++)
#pragma unroll
        for (int k = 0; k < 8; k++) v[i][k] = 0.0f;
    }
    __syncwarp();
    if (PAIR && half == 0) {
      half = 1;
    } else {
      half = 0;
      item += gridDim.x;
      if (item < items) {
        place_of(item, tr, tc);
        ask(tr, tc);
      }
    }
    if constexpr (COL) {  // columns: the rows of a thread, twice as many of a warp, 128 of the CTA
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
    if (o.dense != nullptr && there) {
#pragma unroll
      for (int i = 0; i < kQtRows; i++)
        if (COL || i < rows) qt_store<Src::kType, 8>(o.dense, (int64_t)(r0 + i) * all_cols + c, v[i]);
    }
    if constexpr (COL) __syncthreads();
    if (COL && tid < kQtTile) {
      float m = part[0][tid];
#pragma unroll
      for (int w = 1; w < kQtThreads / 32; w++) m = qt_max(m, part[w][tid]);
      const float s = qt_scale<FMT>(m, o.pow2);
      scale[tid] = s;
      if (c0 + tid < all_cols) o.s_t[(int64_t)(c0 + tid) * o.tiles_r + this_r] = __frcp_rn(s);
    }
    if constexpr (ROW) {
      uint8_t* to = o.q + (int64_t)r0 * all_cols + c;
      float* scale_to = o.s + (int64_t)r0 * o.tiles_c + this_c;
      qt_groups<FMT, kQtRows>(
          v, o.pow2, [&](int i) { return to + (int64_t)i * all_cols; }, [&](int i) { return scale_to + (int64_t)i * o.tiles_c; },
          [&](int i) { return there && (COL || i < rows); });
    }
    if constexpr (COL) {
      __syncthreads();
      {
        const float4 a = *(const float4*)&scale[hl * 8], b = *(const float4*)&scale[hl * 8 + 4];
#pragma unroll
        for (int i = 0; i < kQtRows; i++) {
          mul2(v[i][0], v[i][1], a.x, a.y);
          mul2(v[i][2], v[i][3], a.z, a.w);
          mul2(v[i][4], v[i][5], b.x, b.y);
          mul2(v[i][6], v[i][7], b.z, b.w);
        }
        // 8-byte pieces of the column's 128 rows, permuted by the thread's columns: 16 lanes hit 16 places
        uint8_t* to = stage + hl * 8 * 128 + ((ty ^ hl) << 3);
#pragma unroll
        for (int k = 0; k < 8; k++)
          *(uint2*)(to + k * 128) = make_uint2(cvt4<FMT>(v[0][k], v[1][k], v[2][k], v[3][k]), cvt4<FMT>(v[4][k], v[5][k], v[6][k], v[7][k]));
      }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < 512 / kQtThreads; n++) {  // 32 rows of a column: four threads a column
        const int col = (tid + n * kQtThreads) >> 2, at = tid & 3, flip = col >> 3;
        const int row = rt + 32 * at;
        if (c0 + col >= all_cols || row >= all_rows) continue;
        uint4 a = *(const uint4*)(stage + col * 128 + (((2 * at) ^ (flip >> 1)) << 4));
        uint4 b = *(const uint4*)(stage + col * 128 + (((2 * at + 1) ^ (flip >> 1)) << 4));
        if (flip & 1) {
          a = make_uint4(a.z, a.w, a.x, a.y);
          b = make_uint4(b.z, b.w, b.x, b.y);
        }
        uint8_t* to = o.q_t + (int64_t)(c0 + col) * all_rows + row;
        if (wide) {
          const uint32_t d[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
          st32B(to, d);
        } else {
          st_stream(to, a);
          if (row + 16 < all_rows) st_stream(to + 16, b);
        }
      }
      __syncthreads();  // the codes have been read
    }
  }
  pdl_launch_dependents();
}

template <class Src, int FMT, bool ROW, bool COL, bool PAIR>
cudaError_t launch_quant_tiles_t(const Src& src, const QtOut& o, cudaStream_t s) {
  const auto kernel = quant_tile_kernel<Src, FMT, ROW, COL, PAIR>;
  static PerDevice<bool> allowed;
  const cudaError_t e = allow_smem(allowed, kernel, kQtSmem<Src>);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)o.tiles_r * o.tiles_c / (PAIR ? 2 : 1), fit = (kQtSmem<Src> > 96 * 1024 ? 1 : 2) * (int64_t)sm_count();
  return launch_kernel(kernel, dim3((unsigned)(tiles < fit ? tiles : fit)), dim3(kQtThreads), kQtSmem<Src>, s, src, o);
}

// Halves with the same inputs: where they are whole tiles one CTA makes both
// tiles of them; else tile columns are taken in the order 0, half, 1, half + 1, ...
template <class Src, int FMT, bool ROW, bool COL>
cudaError_t launch_quant_tiles(const Src& src, const QtOut& o, cudaStream_t s) {
  if constexpr (Src::kHalves) {
    if (o.cols % (2 * kQtTile) == 0) return launch_quant_tiles_t<Src, FMT, ROW, COL, true>(src, o, s);
  }
  return launch_quant_tiles_t<Src, FMT, ROW, COL, false>(src, o, s);
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
