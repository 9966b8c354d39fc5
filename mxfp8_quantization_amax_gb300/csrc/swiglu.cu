// swiglu.cu -- the gated activation between the two products of a block, its
// 8-bit copies, and its gradient's.
//
//   h = [gate | up],  s = 1 / (1 + exp(-gate)),  a = gate * s * up
//   d_up = d_a * gate * s,   d_gate = d_a * up * s * (1 + gate * (1 - s))
//
// With e = exp(-gate), s = 1 / (1 + e) and 1 - s = e s: no difference of near
// values.  exp(-g) = 2^(-g log2 e), the product as a sum of two FP32 numbers:
// the larger goes to the exponential instruction, the smaller, l, comes in as
// 1 + l ln 2.  In the exponential a gate counts as one within [-88.5, 127]; s is
// 0 where it would be below 2^-126 (gates below -87.3).  FP32 throughout;
// codes are made from the FP32 values, a dense output is rounded once.
//
// Both copies: tiles (quant_tile.cuh).  65536 x 2048 128 us (6.3 TB/s), the
// gradient of 16384 x 14336 419 us (5.7 TB/s; an earlier form 690 with a sigmoid
// and a read of the inputs for each half, 486 with one for both).  The row copy
// alone 101 us (6.7 TB/s) and 286 us (6.6 TB/s).  128 rows of 2048: 1.4 us, in a
// call of 17.
#include "quant_tile.cuh"

namespace fp8q {

__device__ __forceinline__ void fma2(float& a, float& b, float x, float y, float c, float d) {  // a, b = a x + c, b y + d
  unsigned long long u, v, w;
  asm("mov.b64 %0, {%1, %2};" : "=l"(u) : "f"(a), "f"(b));
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(w) : "f"(c), "f"(d));
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(u) : "l"(v), "l"(w));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(u));
}

// Pairs of inputs as QtRaw::pair gives them: their values, those within [-88.5, 127].
template <int P>
__device__ __forceinline__ void sg_values(uint2 w, float& x0, float& x1) {
  if constexpr (P == kBF16) qt_halves(w.x, x0, x1);
  else x0 = __uint_as_float(w.x), x1 = __uint_as_float(w.y);
}
template <int P>
__device__ __forceinline__ void sg_within(uint2 w, float& x0, float& x1) {
  if constexpr (P == kBF16) {
    uint32_t c;
    asm("{\n\t.reg .b32 t;\n\tmin.bf16x2 t, %1, %2;\n\tmax.bf16x2 %0, t, %3;\n\t}" : "=r"(c) : "r"(w.x), "r"(0x42FE42FEu), "r"(0xC2B1C2B1u));
    qt_halves(c, x0, x1);
  } else {
    x0 = fmaxf(fminf(__uint_as_float(w.x), 127.0f), -88.5f);
    x1 = fmaxf(fminf(__uint_as_float(w.y), 127.0f), -88.5f);
  }
}
// The larger magnitude of each of two pairs with the sign of their product, and the smaller magnitude; NaN stays.
template <int P>
__device__ __forceinline__ void sg_order(uint2 a, uint2 b, uint2& big, uint2& small) {
  if constexpr (P == kBF16) {
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(big.x) : "r"(a.x), "r"(b.x));
    asm("min.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(small.x) : "r"(a.x), "r"(b.x));
    small.x &= 0x7FFF7FFFu;
  } else {
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=r"(big.x) : "r"(a.x), "r"(b.x));
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=r"(big.y) : "r"(a.y), "r"(b.y));
    asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=r"(small.x) : "r"(a.x), "r"(b.x));
    asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=r"(small.y) : "r"(a.y), "r"(b.y));
    small.x &= 0x7FFFFFFFu, small.y &= 0x7FFFFFFFu;
  }
}

// s and e of two gates.
template <int P>
__device__ __forceinline__ void sg_sigmoid(uint2 gate, float& s0, float& s1, float& e0, float& e1) {
  constexpr float kLog2e = 1.44269502f, kRest = 1.92596299e-8f, kLn2 = 0.693147181f;  // log2 e = kLog2e + kRest
  float g0, g1, x0, x1;
  sg_within<P>(gate, g0, g1);
  float t0 = g0, t1 = g1, l0 = g0, l1 = g1;
  mul2(t0, t1, -kLog2e, -kLog2e);
  fma2(l0, l1, kLog2e, kLog2e, t0, t1);  // what the rounding of t took, exactly
  fma2(g0, g1, kRest, kRest, l0, l1);
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(x0) : "f"(t0));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(x1) : "f"(t1));
  mul2(g0, g1, -kLn2, -kLn2);
  fma2(g0, g1, x0, x1, x0, x1);
  e0 = g0, e1 = g1;
  fma2(g0, g1, 1.0f, 1.0f, 1.0f, 1.0f);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s0) : "f"(g0));  // within one unit
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s1) : "f"(g1));
}

// x0, x1 = values of w times x0, x1.
template <int P>
__device__ __forceinline__ void sg_times(uint2 w, float& x0, float& x1) {
  float v0, v1;
  sg_values<P>(w, v0, v1);
  mul2(x0, x1, v0, v1);
}

// The sigmoid comes first in every product, so that none leaves FP32's range
// where the result does not: gate * s lies between -0.28 and the gate.
template <int P>
__device__ __forceinline__ void sg_forward(uint2 gate, uint2 up, float& a0, float& a1) {
  float s0, s1, e0, e1;
  sg_sigmoid<P>(gate, s0, s1, e0, e1);
  sg_values<P>(gate, a0, a1);
  mul2(a0, a1, s0, s1);
  sg_times<P>(up, a0, a1);
}

// The slope of gate * s, s (1 + gate (1 - s)), lies between -0.1 and 1.1; of up and
// d_a the larger comes first, as slope * smaller could fall below the range.  (The
// products of two inputs first, again with the sigmoid first where that gave Inf
// or NaN: no faster, 131 us against 128 for 65536 x 2048 in both copies.)
template <int P>
__device__ __forceinline__ void sg_slope(uint2 up, uint2 d, float g0, float g1, float s0, float s1, float e0, float e1, float& o0, float& o1) {
  mul2(e0, e1, s0, s1);
  fma2(g0, g1, e0, e1, 1.0f, 1.0f);
  mul2(g0, g1, s0, s1);
  uint2 big, small;
  sg_order<P>(up, d, big, small);
  sg_times<P>(big, g0, g1);
  sg_times<P>(small, g0, g1);
  o0 = g0, o1 = g1;
}

// One half of d_h: of the gate (UP false) or of the up branch.
template <bool UP, int P>
__device__ __forceinline__ void sg_backward(uint2 gate, uint2 up, uint2 d, float& o0, float& o1) {
  float s0, s1, e0, e1, g0, g1;
  sg_sigmoid<P>(gate, s0, s1, e0, e1);
  sg_values<P>(gate, g0, g1);
  if constexpr (UP) {
    mul2(g0, g1, s0, s1);
    sg_times<P>(d, g0, g1);
    o0 = g0, o1 = g1;
  } else {
    sg_slope<P>(up, d, g0, g1, s0, s1, e0, e1, o0, o1);
  }
}

// Both.
template <int P>
__device__ __forceinline__ void sg_both(uint2 gate, uint2 up, uint2 d, float& g0, float& g1, float& u0, float& u1) {
  float s0, s1, e0, e1, x0, x1;
  sg_sigmoid<P>(gate, s0, s1, e0, e1);
  sg_values<P>(gate, x0, x1);
  float y0 = x0, y1 = x1;
  mul2(y0, y1, s0, s1);
  sg_times<P>(d, y0, y1);
  sg_slope<P>(up, d, x0, x1, s0, s1, e0, e1, g0, g1);
  u0 = y0, u1 = y1;
}

template <int DT>
struct SwigluForward {
  static constexpr int kType = DT;
  const void* h;
  int64_t inner;
  template <int V>
  __device__ __forceinline__ void row(float (&a)[V], int64_t r, int64_t c) const {
    QtRaw<DT, V> g, u;
    g.load(h, r * 2 * inner + c);
    u.load(h, r * 2 * inner + inner + c);
    values<V>(g, u, a);
  }
  static constexpr int kInputs = 2;
  static constexpr bool kHalves = false;
  __device__ __forceinline__ bool needs(int, int) const { return true; }
  __device__ __forceinline__ const void* at(int n, int row, int col) const {
    return (const uint8_t*)h + (row * 2 * inner + n * inner + col) * (DT == kBF16 ? 2 : 4);
  }
  __device__ __forceinline__ int pitch(int) const { return (int)(2 * inner); }
  __device__ __forceinline__ void begin(int, int) {}
  __device__ __forceinline__ void values(const QtRaw<DT, 8> (&in)[2], int, int, float (&v)[8]) const { values<8>(in[0], in[1], v); }
  template <int V>
  static __device__ __forceinline__ void values(const QtRaw<DT, V>& g, const QtRaw<DT, V>& u, float (&a)[V]) {
#pragma unroll
    for (int k = 0; k < (V + 1) / 2; k++) {
      float a0, a1;
      sg_forward<QtRaw<DT, V>::kPair>(g.pair(k), u.pair(k), a0, a1);
      a[2 * k] = a0;
      if constexpr (V > 1) a[2 * k + 1] = a1;
    }
  }
};

// Columns [0, inner) are the gate's gradient, [inner, 2 inner) the up branch's.
template <int DT>
struct SwigluBackward {
  static constexpr int kType = DT;
  const void* h;
  const void* d_a;
  int64_t inner;
  template <int V>
  __device__ __forceinline__ void row(float (&o)[V], int64_t r, int64_t c) const {
    const bool up = c >= inner;
    const int64_t j = up ? c - inner : c;
    QtRaw<DT, V> g, u, d;
    g.load(h, r * 2 * inner + j);
    if (!up) u.load(h, r * 2 * inner + inner + j);
    d.load(d_a, r * inner + j);
    if (up) values<true, V>(g, g, d, o);
    else values<false, V>(g, u, d, o);
  }
  static constexpr int kInputs = 3;
  static constexpr bool kHalves = true;
  __device__ __forceinline__ bool needs(int n, int col) const { return n != 1 || col < inner; }
  __device__ __forceinline__ const void* at(int n, int row, int col) const {
    const int64_t j = col >= inner ? col - inner : col, size = DT == kBF16 ? 2 : 4;
    return n == 2 ? (const uint8_t*)d_a + (row * inner + j) * size : (const uint8_t*)h + (row * 2 * inner + n * inner + j) * size;
  }
  __device__ __forceinline__ int pitch(int n) const { return (int)(n == 2 ? inner : 2 * inner); }
  __device__ __forceinline__ void begin(int, int) {}
  __device__ __forceinline__ void values(const QtRaw<DT, 8> (&in)[3], int, int col, float (&v)[8]) const {
    if (col >= inner) values<true, 8>(in[0], in[0], in[2], v);
    else values<false, 8>(in[0], in[1], in[2], v);
  }
  static __device__ __forceinline__ void both(const QtRaw<DT, 8> (&in)[3], float (&o_g)[8], float (&o_u)[8]) {
#pragma unroll
    for (int k = 0; k < 4; k++)
      sg_both<DT>(in[0].pair(k), in[1].pair(k), in[2].pair(k), o_g[2 * k], o_g[2 * k + 1], o_u[2 * k], o_u[2 * k + 1]);
  }
  // both halves of a row's columns c .. c + 7
  __device__ __forceinline__ void row_both(float (&o_g)[8], float (&o_u)[8], int64_t r, int64_t c) const {
    QtRaw<DT, 8> in[3];
    in[0].load(h, r * 2 * inner + c);
    in[1].load(h, r * 2 * inner + inner + c);
    in[2].load(d_a, r * inner + c);
    both(in, o_g, o_u);
  }
  template <bool UP, int V>
  static __device__ __forceinline__ void values(const QtRaw<DT, V>& g, const QtRaw<DT, V>& u, const QtRaw<DT, V>& d, float (&o)[V]) {
#pragma unroll
    for (int k = 0; k < (V + 1) / 2; k++) {
      float o0, o1;
      sg_backward<UP, QtRaw<DT, V>::kPair>(g.pair(k), u.pair(k), d.pair(k), o0, o1);
      o[2 * k] = o0;
      if constexpr (V > 1) o[2 * k + 1] = o1;
    }
  }
};

// Few rows, or no copy: a half-warp takes a row's group of 128 columns (without a
// copy: 16 V columns); PAIR: that group and its partner in the other half.
constexpr int kSgThreads = 256;

template <class Src, int FMT, int V, bool PAIR>
__global__ void __launch_bounds__(kSgThreads) swiglu_rows_kernel(Src src, QtOut o, uint32_t per_row, uint32_t items) {
  constexpr int U = PAIR ? 2 : 1;
  const int hl = threadIdx.x & 15;
  const uint32_t item = blockIdx.x * (kSgThreads / 16) + threadIdx.x / 16, r = item / per_row, group = item - r * per_row;
  const int64_t cols = PAIR ? o.cols / 2 : o.cols, c = (int64_t)(group * 16 + hl) * V;
  const bool ok = item < items && c < cols;
  pdl_wait();
  float v[U][V] = {};
  if (ok) {
    if constexpr (PAIR) src.row_both(v[0], v[1], r, c);
    else src.template row<V>(v[0], r, c);
  }
  if constexpr (V == 8) {
    if (o.q != nullptr) {
      uint8_t* q = o.q + r * o.cols + c;
      float* s = o.s + (int64_t)r * o.tiles_c + c / 128;
      qt_groups<FMT, U>(
          v, o.pow2, [&](int i) { return q + i * cols; }, [&](int i) { return s + i * cols / 128; }, [&](int) { return ok; });
    }
  }
  if (o.dense != nullptr && ok) {
#pragma unroll
    for (int i = 0; i < U; i++) qt_store<Src::kType, V>(o.dense, r * o.cols + i * cols + c, v[i]);
  }
  pdl_launch_dependents();
}

template <class Src, int FMT, int V, bool PAIR>
static fp8q_status launch_swiglu_rows(const Src& src, const QtOut& o, cudaStream_t s) {
  const int64_t cols = PAIR ? o.cols / 2 : o.cols, per_row = (cols + V * 16 - 1) / (V * 16), items = o.rows * per_row;
  if (items > UINT32_MAX - kSgThreads) return fail(FP8Q_ERR_UNSUPPORTED, "rows * inner too large");
  const dim3 grid((unsigned)((items + kSgThreads / 16 - 1) / (kSgThreads / 16)));
  const cudaError_t e = launch_kernel(swiglu_rows_kernel<Src, FMT, V, PAIR>, grid, dim3(kSgThreads), 0, s, src, o, (uint32_t)per_row, (uint32_t)items);
  return e == cudaSuccess ? check_launch("swiglu kernel") : cuda_fail(e, "swiglu kernel launch");
}

template <class Src, int FMT>
static fp8q_status launch_swiglu(const Src& src, const QtOut& o, bool vec, cudaStream_t s) {
  // The row copy alone by tiles from 3 an SM on, else a half-warp a group (us: 2000 x 2048 4.9 and 4.8, 4096 x 2048 8.1 and 8.4,
  // 65536 x 2048 101 and 127; the gradient of 4099 x 1936 17.2 and 18.1).  Where one set of inputs gives two tiles the
  // half-warp saves the second read too, and tiles win from 8 pairs an SM on (gradient of 4096 x 2048 13.4 and 12.0,
  // 8192 x 2048 27.2 and 26.3, 10000 x 2048 31.9 and 32.1, 24576 x 2048 67 and 75).
  const int64_t tiles = (int64_t)o.tiles_r * o.tiles_c;
  const bool pairs = Src::kHalves && o.cols % (2 * kQtTile) == 0, many = pairs ? tiles / 2 >= 8 * sm_count() : tiles >= 3 * sm_count();
  if (o.q_t || (o.q && many)) {
    const cudaError_t e = !o.q_t ? launch_quant_tiles<Src, FMT, true, false>(src, o, s)
                          : o.q  ? launch_quant_tiles<Src, FMT, true, true>(src, o, s)
                                 : launch_quant_tiles<Src, FMT, false, true>(src, o, s);
    return e == cudaSuccess ? check_launch("swiglu kernel") : cuda_fail(e, "swiglu kernel launch");
  }
  if (!vec) return launch_swiglu_rows<Src, FMT, 1, false>(src, o, s);
  if constexpr (Src::kHalves) {
    if (o.cols % 256 == 0) return launch_swiglu_rows<Src, FMT, 8, true>(src, o, s);
  }
  return launch_swiglu_rows<Src, FMT, 8, false>(src, o, s);
}

template <class Src>
static fp8q_status launch_swiglu_fmt(const Src& src, const QtOut& o, int fmt, bool vec, cudaStream_t s) {
  return fmt == kE4M3 ? launch_swiglu<Src, kE4M3>(src, o, vec, s) : launch_swiglu<Src, kE5M2>(src, o, vec, s);
}

static bool off(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

// Forward where d_a is NULL.
static fp8q_status swiglu(const void* h, const void* d_a, bool backward, int32_t dt, int64_t rows, int64_t inner, int32_t fmt,
                          int32_t dir, int32_t pow2, void* dense, uint8_t* q, float* s, uint8_t* q_t, float* s_t,
                          void* stream) {
  if (dt != FP8Q_IN_BF16 && dt != FP8Q_IN_FP32) return fail(FP8Q_ERR_INVALID_ARG, "dt must be FP8Q_IN_BF16 or FP8Q_IN_FP32");
  if (rows < 0 || inner < 0) return fail(FP8Q_ERR_INVALID_ARG, "rows and inner must be >= 0");
  if (rows > INT32_MAX / 2 || inner > INT32_MAX / 4) return fail(FP8Q_ERR_UNSUPPORTED, "rows or inner too large");
  const int64_t cols = backward ? 2 * inner : inner;
  const fp8q_status r = qt_check(rows, cols, fmt, dir, q, s, q_t, s_t);
  if (r != FP8Q_OK) return r;
  if (!dir && !dense && rows * cols > 0) return fail(FP8Q_ERR_INVALID_ARG, "no output is asked for");
  if (rows * cols == 0) return FP8Q_OK;
  const size_t size = dt == FP8Q_IN_BF16 ? 2 : 4, need = dir ? 16 : size;
  if (!h || off(h, need)) return fail(FP8Q_ERR_INVALID_ARG, "h must be a device pointer, 16-byte aligned for a copy");
  if (backward && (!d_a || off(d_a, need)))
    return fail(FP8Q_ERR_INVALID_ARG, "d_a must be a device pointer, 16-byte aligned for a copy");
  if (off(dense, need)) return fail(FP8Q_ERR_INVALID_ARG, "the dense output must be aligned as h is");
  const bool vec = inner % 8 == 0 && !off(h, 16) && !off(d_a, 16) && !off(dense, 16);
  QtOut o{};
  o.rows = rows;
  o.cols = cols;
  const int64_t tiles_r = (rows + kQtTile - 1) / kQtTile, tiles_c = (cols + kQtTile - 1) / kQtTile;
  if (tiles_r * tiles_c > INT32_MAX) return fail(FP8Q_ERR_UNSUPPORTED, "rows * inner too large");
  o.tiles_r = (int)tiles_r;
  o.tiles_c = (int)tiles_c;
  o.pow2 = pow2 ? 1 : 0;
  o.dense = dense;
  if (dir & MXFP8_ROW) o.q = q, o.s = s;
  if (dir & MXFP8_COL) o.q_t = q_t, o.s_t = s_t;
  const cudaStream_t st = (cudaStream_t)stream;
  if (backward) {
    if (dt == FP8Q_IN_BF16) return launch_swiglu_fmt(SwigluBackward<kBF16>{h, d_a, inner}, o, fmt, vec, st);
    return launch_swiglu_fmt(SwigluBackward<kFP32>{h, d_a, inner}, o, fmt, vec, st);
  }
  if (dt == FP8Q_IN_BF16) return launch_swiglu_fmt(SwigluForward<kBF16>{h, inner}, o, fmt, vec, st);
  return launch_swiglu_fmt(SwigluForward<kFP32>{h, inner}, o, fmt, vec, st);
}

}  // namespace fp8q

using namespace fp8q;

extern "C" fp8q_status fp8q_swiglu(const void* h, int32_t dt, int64_t rows, int64_t inner, int32_t fmt, int32_t dir,
                                   int32_t pow2_scales, void* a, uint8_t* q, float* scale_inv, uint8_t* q_t,
                                   float* scale_inv_t, void* stream) {
  clear_error();
  return swiglu(h, nullptr, false, dt, rows, inner, fmt, dir, pow2_scales, a, q, scale_inv, q_t, scale_inv_t, stream);
}

extern "C" fp8q_status fp8q_swiglu_backward(const void* h, const void* d_a, int32_t dt, int64_t rows, int64_t inner,
                                            int32_t fmt, int32_t dir, int32_t pow2_scales, void* d_h, uint8_t* q,
                                            float* scale_inv, uint8_t* q_t, float* scale_inv_t, void* stream) {
  clear_error();
  return swiglu(h, d_a, true, dt, rows, inner, fmt, dir, pow2_scales, d_h, q, scale_inv, q_t, scale_inv_t, stream);
}
