// swiglu.cu -- the gated activation between the two products of a block, its
// 8-bit copies, and its gradient's.
//
//   h = [gate | up],  s = 1 / (1 + exp(-gate)),  a = gate * s * up
//   d_up = d_a * gate * s,   d_gate = d_a * up * s * (1 + gate * (1 - s))
//
// With e = exp(-gate), s = 1 / (1 + e) and 1 - s = e s: no difference of near
// values.  exp(-g) = 2^(-g log2 e), the product as a sum of two FP32 numbers:
// the larger goes to the exponential instruction, the smaller, l, comes in as
// 1 + l ln 2.  Where a gate of a thread's eight is beyond +-87 (or is not
// finite), e = exp(-|gate|) and r = 1 / (1 + e) give s and 1 - s as r and e r, or
// the other way round, for all eight.  FP32 throughout; codes are made from the
// FP32 values, a dense output is rounded once.
#include "quant_tile.cuh"

namespace fp8q {

// Two values of s and e = (1 - s) / s at a time: packed products and sums.
__device__ __forceinline__ void fma2(float& a, float& b, float x, float y, float c, float d) {  // a, b = a x + c, b y + d
  unsigned long long u, v, w;
  asm("mov.b64 %0, {%1, %2};" : "=l"(u) : "f"(a), "f"(b));
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(w) : "f"(c), "f"(d));
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(u) : "l"(v), "l"(w));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(u));
}

// s and 1 - s (without it, t holds e) of V gates.
template <bool T, int V>
__device__ __forceinline__ void sg_sigmoid(const float (&g)[V], float (&s)[V], float (&t)[V]) {
  constexpr float kLog2e = 1.44269502f, kRest = 1.92596299e-8f, kLn2 = 0.693147181f;  // log2 e = kLog2e + kRest
  float m;
  if constexpr (V == 8) m = qt_max8(g);
  else m = fabsf(g[0]);
  if (m <= 87.0f) {
#pragma unroll
    for (int k = 0; k < V; k += 2) {
      constexpr int n = V > 1;
      float t0 = g[k], t1 = g[k + n], l0 = t0, l1 = t1, e0, e1;
      mul2(t0, t1, -kLog2e, -kLog2e);
      fma2(l0, l1, kLog2e, kLog2e, t0, t1);  // what the rounding of t took, exactly
      float r0 = g[k], r1 = g[k + n];
      fma2(r0, r1, kRest, kRest, l0, l1);
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(t0));
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(t1));
      mul2(r0, r1, -kLn2, -kLn2);
      fma2(r0, r1, e0, e1, e0, e1);
      float d0 = r0, d1 = r1;
      fma2(d0, d1, 1.0f, 1.0f, 1.0f, 1.0f);
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d0) : "f"(d0));  // of 1 to 2^126: within one unit
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d1) : "f"(d1));
      if (T) mul2(r0, r1, d0, d1);
      s[k] = d0, s[k + n] = d1;
      t[k] = r0, t[k + n] = r1;
    }
  } else {
#pragma unroll
    for (int k = 0; k < V; k++) {
      const float e = expf(-fabsf(g[k])), r = __frcp_rn(1.0f + e), er = __fmul_rn(e, r);
      s[k] = g[k] >= 0.0f ? r : er;
      t[k] = g[k] >= 0.0f ? er : r;
    }
  }
}

template <int V>
__device__ __forceinline__ void sg_forward(const float (&g)[V], const float (&u)[V], float (&a)[V]) {
  float s[V], t[V];
  sg_sigmoid<false>(g, s, t);
#pragma unroll
  for (int k = 0; k < V; k += 2) {
    constexpr int n = V > 1;
    float a0 = g[k], a1 = g[k + n];
    mul2(a0, a1, s[k], s[k + n]);
    mul2(a0, a1, u[k], u[k + n]);
    a[k + n] = a1;
    a[k] = a0;
  }
}

// One half of d_h: of the gate (UP false) or of the up branch.
template <bool UP, int V>
__device__ __forceinline__ void sg_backward(const float (&g)[V], const float (&u)[V], const float (&d)[V], float (&o)[V]) {
  float s[V], t[V];
  sg_sigmoid<!UP>(g, s, t);
#pragma unroll
  for (int k = 0; k < V; k += 2) {
    constexpr int n = V > 1;
    float o0 = g[k], o1 = g[k + n];
    if (!UP) {
      fma2(o0, o1, t[k], t[k + n], 1.0f, 1.0f);
      mul2(o0, o1, u[k], u[k + n]);
    }
    mul2(o0, o1, s[k], s[k + n]);
    mul2(o0, o1, d[k], d[k + n]);
    o[k + n] = o1;
    o[k] = o0;
  }
}

template <int DT>
struct SwigluForward {
  static constexpr int kType = DT;
  const void* h;
  int64_t inner;
  template <int V>
  __device__ __forceinline__ void row(float (&a)[V], int64_t r, int64_t c) const {
    QtRaw<DT, V> g, u;
    float gv[V], uv[V];
    g.load(h, r * 2 * inner + c);
    u.load(h, r * 2 * inner + inner + c);
    g.get(gv);
    u.get(uv);
    sg_forward<V>(gv, uv, a);
  }
  __device__ __forceinline__ void tile(float (&v)[8][8], int64_t row, int64_t col, int64_t rows) const {
    QtRaw<DT, 8> g[8], u[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      if (row + i < rows) {
        g[i].load(h, (row + i) * 2 * inner + col);
        u[i].load(h, (row + i) * 2 * inner + inner + col);
      } else {
        g[i].zero();
        u[i].zero();
      }
    }
#pragma unroll
    for (int i = 0; i < 8; i++) {
      float gv[8], uv[8];
      g[i].get(gv);
      u[i].get(uv);
      sg_forward<8>(gv, uv, v[i]);
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
    float gv[V], uv[V], dv[V];
    g.load(h, r * 2 * inner + j);
    u.load(h, r * 2 * inner + inner + j);
    d.load(d_a, r * inner + j);
    g.get(gv);
    u.get(uv);
    d.get(dv);
    if (up) sg_backward<true>(gv, uv, dv, o);
    else sg_backward<false>(gv, uv, dv, o);
  }
  __device__ __forceinline__ void tile(float (&v)[8][8], int64_t row, int64_t col, int64_t rows) const {
    const bool up = col >= inner;
    const int64_t j = up ? col - inner : col;
#pragma unroll
    for (int n = 0; n < 8; n += 4) {  // four rows on their way at a time
      QtRaw<DT, 8> g[4], u[4], d[4];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int64_t r = row + n + i;
        g[i].zero();
        u[i].zero();
        d[i].zero();
        if (r < rows) {
          g[i].load(h, r * 2 * inner + j);
          if (!up) u[i].load(h, r * 2 * inner + inner + j);
          d[i].load(d_a, r * inner + j);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; i++) {
        float gv[8], uv[8], dv[8];
        g[i].get(gv);
        u[i].get(uv);
        d[i].get(dv);
        if (up) sg_backward<true>(gv, uv, dv, v[n + i]);
        else sg_backward<false>(gv, uv, dv, v[n + i]);
      }
    }
  }
};

// Rows alone: the dense output, the row copy or both.  A half-warp takes a row
// group of 128 columns (without a copy: any V * 16 columns).
constexpr int kSgThreads = 256;

template <class Src, int FMT, int V>
__global__ void __launch_bounds__(kSgThreads) swiglu_rows_kernel(Src src, QtOut o, int64_t groups, int per_row) {
  const int hl = threadIdx.x & 15;
  pdl_wait();
  for (int64_t g0 = (int64_t)blockIdx.x * (kSgThreads / 16); g0 < groups; g0 += (int64_t)gridDim.x * (kSgThreads / 16)) {
    const int64_t g = g0 + threadIdx.x / 16;
    const int64_t r = g / per_row;
    const int64_t c = ((g - r * per_row) * 16 + hl) * V;
    const bool there = g < groups && c < o.cols;
    float v[V];
#pragma unroll
    for (int k = 0; k < V; k++) v[k] = 0.0f;
    if (there) src.template row<V>(v, r, c);
    if constexpr (V == 8) {
      if (o.q != nullptr) qt_group<FMT>(v, o.pow2, o.q + r * o.cols + c, o.s + g, there, hl);
    }
    if (o.dense != nullptr && there) qt_store<Src::kType, V>(o.dense, r * o.cols + c, v);
  }
  pdl_launch_dependents();
}

template <class Src, int FMT>
static fp8q_status launch_swiglu(const Src& src, const QtOut& o, bool vec, cudaStream_t s) {
  cudaError_t e;
  if (o.q_t) {
    e = launch_quant_tiles<Src, FMT>(src, o, s);
  } else {
    const int per_row = (int)((o.cols + (vec ? 128 : 16) - 1) / (vec ? 128 : 16));
    const int64_t groups = o.rows * per_row, ctas = (groups + kSgThreads / 16 - 1) / (kSgThreads / 16);
    const dim3 grid((unsigned)(ctas < INT32_MAX ? ctas : INT32_MAX));
    e = vec ? launch_kernel(swiglu_rows_kernel<Src, FMT, 8>, grid, dim3(kSgThreads), 0, s, src, o, groups, per_row)
            : launch_kernel(swiglu_rows_kernel<Src, FMT, 1>, grid, dim3(kSgThreads), 0, s, src, o, groups, per_row);
  }
  if (e != cudaSuccess) return cuda_fail(e, "swiglu kernel launch");
  return check_launch("swiglu kernel");
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
  o.apart = backward;
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
