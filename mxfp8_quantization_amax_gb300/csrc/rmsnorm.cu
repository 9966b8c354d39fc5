// rmsnorm.cu -- root-mean-square norm with the residual's addition, the 8-bit
// copies of its output, and its gradients.
//
//   h = x + residual (rounded to the residual's type: the stream that goes on), or x
//   rstd = 1 / sqrt(mean(h^2) + eps),   y = h * rstd * weight
//   with g = d_y * weight and u = h * rstd:
//   d_x = rstd * (g - u * mean(g * u)) + d_h,   d_weight = sum over the rows of d_y * u
//
// Sums are FP32 in a fixed order.  The norm is of h as it is stored, so that
// the gradient, which reads h again, differentiates what was computed.
//
// Bound by memory where rows are many: CTAs stay and have the next rows' inputs
// on their way.  16384 x 4096 BF16 with the residual: row copy 71 us (6.6 TB/s;
// 120 with a CTA a row), gradients 87 us (6.2 TB/s), the transposed copy 34 us
// more: it needs the statistics of 128 rows, and 128 rows of 4096 do not fit an
// SM, so h is read again.  12345 x 7168, FP32 stream, y and row copy 188 us (6.1
// TB/s).  Without a residual dependent chains on 16 warps an SM bound it
// (16384 x 7168 78 us, 4.5 TB/s; issue 62%).  Odd
// columns: 12345 x 4097 80 us (5.0 TB/s), gradients 107 us (2.8 TB/s); value by
// value, as unaligned tensors are taken, 159 and 295.  One row of 7168: 2.8 us,
// latency.
#include "quant_tile.cuh"

namespace fp8q {

constexpr int kRnMaxCols = 32768;
constexpr int kRnThreads = 256;      // of a CTA at least
constexpr int kRnMaxPartials = 608;  // rows of the weight gradient's partial sums: one a CTA
constexpr int kNone = -1;

struct RmsNorm {
  const void* x;
  const void* residual;  // its type: RT
  const void* weight;
  int weight_dt;
  int64_t rows, cols;
  int lanes;  // threads of a row
  float eps, one_over_cols;
  int fmt, pow2, tiles_c;
  void* h;
  float* rstd;
  void* y;
  uint8_t* q;
  float* s;
};

// V values that the kernel may write in place.
template <int DT, int V>
__device__ __forceinline__ void rn_load_plain(const void* p, int64_t i, QtRaw<DT, V>& r) {
  if constexpr (V == 8 && DT == kBF16) {
    r.a = *(const uint4*)((const uint16_t*)p + i);
  } else if constexpr (V == 8) {
    r.a = *(const uint4*)((const float*)p + i);
    r.b = *(const uint4*)((const float*)p + i + 4);
  } else {
    r.a.x = DT == kBF16 ? (uint32_t) * ((const uint16_t*)p + i) << 16 : *((const uint32_t*)p + i);
  }
}

// V weights; every row reads them, so they may stay in L1.
template <int V>
__device__ __forceinline__ void rn_weight(const void* w, int dt, int64_t i, float (&v)[V]) {
  if (dt == kFP32) {
    const float* q = (const float*)w + i;
    if constexpr (V == 8) {
      const float4 a = __ldg((const float4*)q), b = __ldg((const float4*)q + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      v[0] = __ldg(q);
    }
  } else {
    const uint16_t* q = (const uint16_t*)w + i;
    if constexpr (V == 8) {
      const uint4 a = __ldg((const uint4*)q);
      v[0] = bf16_lo(a.x), v[1] = bf16_hi(a.x), v[2] = bf16_lo(a.y), v[3] = bf16_hi(a.y);
      v[4] = bf16_lo(a.z), v[5] = bf16_hi(a.z), v[6] = bf16_lo(a.w), v[7] = bf16_hi(a.w);
    } else {
      v[0] = __uint_as_float((uint32_t)__ldg(q) << 16);
    }
  }
}

// The sum over the `lanes` threads of a row (a multiple of 32; rows of a CTA
// lie side by side).  Every thread of the CTA comes here; calls in a row take
// the halves of sh in turn.
__device__ __forceinline__ float rn_row_sum(float v, int lanes, float* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (lanes == 32) return v;
  const int warp = threadIdx.x >> 5, per = lanes >> 5, first = warp / per * per;
  if ((threadIdx.x & 31) == 0) sh[warp] = v;
  __syncthreads();
  v = 0.0f;
  for (int w = 0; w < per; w++) v += sh[first + w];
  return v;
}

// Rows of any number of columns: a thread's chunks of eight lie on multiples of
// eight values of memory, so the first starts `shift` = (r * cols) % 8 columns
// before the row and the last may end behind it.  A group of threads whose rows
// are a multiple of eight apart has one shift, and so the same columns in every row.
// What of a chunk that starts at column c is not the row's becomes 0.
template <bool ODD>
__device__ __forceinline__ void rn_clear(int c, int cols, float (&v)[8]) {
  if (ODD && (c < 0 || c + 8 > cols)) {
#pragma unroll
    for (int k = 0; k < 8; k++)
      if (c + k < 0 || c + k >= cols) v[k] = 0.0f;
  }
}
template <int DT, bool ODD, int V>
__device__ __forceinline__ void rn_store(void* to, int64_t row, int c, int cols, float (&v)[V], bool back = false) {
  if (ODD && (c < 0 || c + V > cols)) {
#pragma unroll
    for (int k = 0; k < V; k++) {
      float one[1] = {v[k]};
      if (c + k >= 0 && c + k < cols) qt_store<DT, 1>(to, row + c + k, one, back);
      v[k] = one[0];
    }
  } else {
    qt_store<DT, V>(to, row + c, v, back);
  }
}

template <int V>
__device__ __forceinline__ void rn_add(float (&v)[V], const float (&b)[V]) {
#pragma unroll
  for (int k = 0; k < V; k++) v[k] = __fadd_rn(v[k], b[k]);
}

// The outputs of a row whose h is in the registers of p.lanes threads, V values in each of N chunks.
template <int DT, int V, int N, bool ODD, class Weight>
__device__ __forceinline__ void rn_row(const RmsNorm& p, float (&v)[N][V], int64_t r, bool row_ok, int t, int shift, float* sh, Weight weight) {
  float sum = 0.0f;
#pragma unroll
  for (int n = 0; n < N; n++)
#pragma unroll
    for (int k = 0; k < V; k++) sum = __fmaf_rn(v[n][k], v[n][k], sum);
  // rsqrtf is within two units
  const float rstd = rsqrtf(__fadd_rn(__fmul_rn(rn_row_sum(sum, p.lanes, sh), p.one_over_cols), p.eps));
  if (row_ok && t == 0) p.rstd[r] = rstd;
  if (p.y == nullptr && p.q == nullptr) return;
#pragma unroll
  for (int n = 0; n < N; n++) {
    if (!row_ok || (n * p.lanes + t) * V - shift >= p.cols) continue;
    float w[V];
    weight(n, w);
    if constexpr (V == 8) {
#pragma unroll
      for (int k = 0; k < V; k += 2) {
        mul2(v[n][k], v[n][k + 1], rstd, rstd);
        mul2(v[n][k], v[n][k + 1], w[k], w[k + 1]);
      }
    } else {
      v[n][0] = __fmul_rn(__fmul_rn(v[n][0], rstd), w[0]);
    }
  }
  if constexpr (V == 8 && !ODD) {
    if (p.q != nullptr) {  // 16 threads hold a group of 128 columns, N of them
      uint8_t* q = p.q + r * p.cols + 8 * t;
      float* s = p.s + r * p.tiles_c + t / 16;
      const auto codes = [&](int n) { return q + (int64_t)n * p.lanes * 8; };
      const auto scale = [&](int n) { return s + n * p.lanes / 16; };
      const auto there = [&](int n) { return row_ok && (n * p.lanes + t) * 8 < p.cols; };
      if (p.fmt == kE4M3) qt_groups<kE4M3, N>(v, p.pow2, codes, scale, there);
      else qt_groups<kE5M2, N>(v, p.pow2, codes, scale, there);
    }
  }
  if (p.y != nullptr) {
#pragma unroll
    for (int n = 0; n < N; n++) {
      const int c = (n * p.lanes + t) * V - shift;
      if (row_ok && c < p.cols) rn_store<DT, ODD, V>(p.y, r * p.cols, c, (int)p.cols, v[n]);
    }
  }
}

// A CTA a row, or a few short rows.
template <int DT, int RT, int V, int N, int T>
__global__ void __launch_bounds__(T) rmsnorm_kernel(RmsNorm p) {
  __shared__ float sh[64];
  const int t = threadIdx.x % p.lanes;
  const int64_t r = (int64_t)blockIdx.x * (blockDim.x / p.lanes) + threadIdx.x / p.lanes;
  const bool row_ok = r < p.rows;
  // all loads before the first store: where nothing is there the first values are read
  QtRaw<DT, V> raw[N];
  QtRaw<RT == kNone ? DT : RT, V> res[N];
  float v[N][V];
  const auto at = [&](int n) { return row_ok && (n * p.lanes + t) * V < p.cols ? r * p.cols + (n * p.lanes + t) * V : 0; };
  pdl_wait();
#pragma unroll
  for (int n = 0; n < N; n++) {
    raw[n].load(p.x, at(n));
    if constexpr (RT != kNone) rn_load_plain<RT, V>(p.residual, at(n), res[n]);
  }
#pragma unroll
  for (int n = 0; n < N; n++) {
    if (row_ok && (n * p.lanes + t) * V < p.cols) {
      raw[n].get(v[n]);
      if constexpr (RT != kNone) {
        float b[V];
        res[n].get(b);
        rn_add<V>(v[n], b);
        qt_store<RT, V>(p.h, at(n), v[n], true);
      }
    } else {
#pragma unroll
      for (int k = 0; k < V; k++) v[n][k] = 0.0f;
    }
  }
  rn_row<DT, V, N, false>(p, v, r, row_ok, t, 0, sh, [&](int n, float (&w)[V]) { rn_weight<V>(p.weight, p.weight_dt, (int64_t)(n * p.lanes + t) * V, w); });
  pdl_launch_dependents();
}

// Many rows: CTAs stay, keep the weights in registers and have the next rows on
// their way.  (More rows on their way, more CTAs with the weights in L1 instead:
// slower.)
constexpr int kRnChunks = 4;
template <int DT>
constexpr int kRnBytes = DT == kNone ? 0 : 32 * kQtRunBytes<DT>;  // of a warp's chunk of one input

template <int DT, int RT, int T, bool ODD>
__global__ void __launch_bounds__(T, T == kRnThreads ? 2 : 1) rmsnorm_stream_kernel(RmsNorm p) {
  constexpr int kChunk = kRnBytes<DT> + kRnBytes<RT>;
  // Without a residual a row's chain of instructions bounds it: addresses go from row to row, and chunks behind the row are 0 from the start.
  constexpr bool kLean = RT == kNone && !ODD;
  extern __shared__ __align__(16) uint8_t inputs[];  // [warps][chunks][kChunk]
  __shared__ float sh[64];
  const int t = threadIdx.x % p.lanes, lane = threadIdx.x & 31, per = blockDim.x / p.lanes, cols = (int)p.cols;
  const uint32_t place = (uint32_t)__cvta_generic_to_shared(inputs) + (threadIdx.x >> 5) * kRnChunks * kChunk;
  const int64_t step = (int64_t)gridDim.x * per;
  int64_t r0 = (int64_t)blockIdx.x * per;
  const int shift = ODD ? (int)((r0 + threadIdx.x / p.lanes) * cols & 7) : 0;
  constexpr int kSize = DT == kBF16 ? 2 : 4;
  const uint8_t* from = (const uint8_t*)p.x + ((r0 + threadIdx.x / p.lanes) * cols + (t - lane) * 8) * kSize + lane * 16;
  const int64_t from_step = step * cols * kSize;
  const auto ask = [&](int64_t r) {
    if (kLean) {
      if (r < p.rows) {
#pragma unroll
        for (int n = 0; n < kRnChunks; n++)
#pragma unroll
          for (int k = 0; k < kSize / 2; k++)
            if ((n * p.lanes + t - lane) * 8 + (k * 32 + lane) * (16 / kSize) < cols)
              qt_ask(place + n * kChunk + (k * 32 + lane) * 16, from + n * p.lanes * 8 * kSize + k * 512);
        from += from_step;
      }
    } else if (r < p.rows) {
#pragma unroll
      for (int n = 0; n < kRnChunks; n++) {
        const int c = (n * p.lanes + t - lane) * 8 - shift;
        qt_ask8<DT, 32, ODD>(p.x, r * cols + c, cols - c, place + n * kChunk, lane);
        if constexpr (RT != kNone) qt_ask8<RT, 32, ODD>(p.residual, r * cols + c, cols - c, place + n * kChunk + kRnBytes<DT>, lane);
      }
    }
    qt_commit();
  };
  pdl_wait();
  if constexpr (kLean) {
    for (unsigned i = threadIdx.x; i < blockDim.x / 32 * kRnChunks * kChunk / 16; i += blockDim.x) ((uint4*)inputs)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }
  ask(r0 + threadIdx.x / p.lanes);
  float w[kRnChunks][8];
#pragma unroll
  for (int n = 0; n < kRnChunks; n++) {
    const int c = (n * p.lanes + t) * 8 - shift;
    if (ODD) {
#pragma unroll
      for (int k = 0; k < 8; k++) {
        float one[1] = {0.0f};
        if (c + k >= 0 && c + k < cols) rn_weight<1>(p.weight, p.weight_dt, c + k, one);
        w[n][k] = one[0];
      }
    } else if (c < cols) {
      rn_weight<8>(p.weight, p.weight_dt, c, w[n]);
    }
  }
  int turn = 0;
  for (; r0 < p.rows; r0 += step) {
    const int64_t r = r0 + threadIdx.x / p.lanes;
    const bool row_ok = r < p.rows;
    float v[kRnChunks][8];
    qt_wait<0>();
    __syncwarp();
#pragma unroll
    for (int n = 0; n < kRnChunks; n++) {
      const int c = (n * p.lanes + t) * 8 - shift;
#pragma unroll
      for (int k = 0; k < 8; k++) v[n][k] = 0.0f;
      if (kLean || (row_ok && c < cols)) {
        QtRaw<DT, 8> raw;
        qt_taken8<DT>(place + n * kChunk, lane, raw);
        raw.get(v[n]);
        if constexpr (RT != kNone) {
          QtRaw<RT, 8> res;
          float b[8];
          qt_taken8<RT>(place + n * kChunk + kRnBytes<DT>, lane, res);
          res.get(b);
          rn_add<8>(v[n], b);
          rn_store<RT, ODD, 8>(p.h, r * cols, c, cols, v[n], true);
        }
        rn_clear<ODD>(c, cols, v[n]);
      }
    }
    __syncwarp();
    ask(r + step);
    rn_row<DT, 8, kRnChunks, ODD>(p, v, r, row_ok, t, shift, sh + (turn ^= 32), [&](int n, float (&u)[8]) {
#pragma unroll
      for (int k = 0; k < 8; k++) u[k] = w[n][k];
    });
  }
  pdl_launch_dependents();
}

// The transposed copy needs 128 rows' statistics at a time: a second pass over h.
template <int DT>
struct RmsNormTile {
  static constexpr int kType = DT;
  const void* h;
  const void* weight;
  int weight_dt;
  const float* rstd;
  int64_t cols;
  float s[kQtRows], w[8];
  static constexpr int kInputs = 1;
  static constexpr bool kHalves = false;
  __device__ __forceinline__ bool needs(int, int) const { return true; }
  __device__ __forceinline__ const void* at(int, int row, int col) const {
    return (const uint8_t*)h + (row * cols + col) * (DT == kBF16 ? 2 : 4);
  }
  __device__ __forceinline__ int pitch(int) const { return (int)cols; }
  __device__ __forceinline__ void begin(int row, int col) {
#pragma unroll
    for (int i = 0; i < kQtRows; i++) s[i] = rstd[row + i];  // written by the kernel before: no read-only load
    rn_weight<8>(weight, weight_dt, col, w);
  }
  __device__ __forceinline__ void values(const QtRaw<DT, 8> (&in)[1], int i, int, float (&v)[8]) const {
    in[0].get(v);
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      mul2(v[k], v[k + 1], s[i], s[i]);
      mul2(v[k], v[k + 1], w[k], w[k + 1]);
    }
  }
};

// ---------------------------------------------------------------------------
// gradients
// ---------------------------------------------------------------------------
struct RmsNormBackward {
  const void* d_y;
  const void* h;
  const void* weight;
  int weight_dt;
  const float* rstd;
  const void* d_h;  // or NULL
  int64_t rows, cols;
  int lanes;
  float one_over_cols;
  void* d_x;
  float* partial;  // [groups of threads][cols]
};

// The sums of the CTA's groups of threads, in their order, as one row of partial sums.
template <int N, bool ODD>
__device__ __forceinline__ void rn_partial(const RmsNormBackward& p, const float (&acc)[N][8], int t, int per, int shift, float* sh) {
  float* to = p.partial + (int64_t)blockIdx.x * p.cols;
  __syncthreads();
  if (per > 1) {  // p.lanes * 8 * N values, of which cols are there, for each group
#pragma unroll
    for (int n = 0; n < N; n++)
#pragma unroll
      for (int k = 0; k < 8; k++) sh[(threadIdx.x / p.lanes * N + n) * p.lanes * 8 + t * 8 + k] = acc[n][k];
    __syncthreads();
    for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
      float sum = 0.0f;
      for (int i = 0; i < per; i++) sum += sh[i * N * p.lanes * 8 + c + (ODD ? (int)(((int64_t)blockIdx.x * per + i) * p.cols & 7) : 0)];
      to[c] = sum;
    }
  } else {
#pragma unroll
    for (int n = 0; n < N; n++)
#pragma unroll
      for (int k = 0; k < 8; k++) {
        const int c = (n * p.lanes + t) * 8 + k - shift;
        if (c < p.cols && (!ODD || c >= 0)) to[c] = acc[n][k];
      }
  }
}

// Each group of p.lanes threads takes every gridDim.x-th set of rows and keeps
// its columns' sums of the weight gradient.  Eight values a chunk; the next
// rows' inputs are on their way.
template <int DT, int HT, int T, bool ODD>
__global__ void __launch_bounds__(T, T == kRnThreads ? 2 : 1) rmsnorm_backward_kernel(RmsNormBackward p) {
  constexpr int N = kRnChunks, kFirst = kRnBytes<DT> + kRnBytes<HT>, kChunk = kFirst + kRnBytes<HT>;
  extern __shared__ __align__(16) uint8_t inputs[];  // [warps][chunks][kChunk]
  __shared__ float sh[64];
  const int t = threadIdx.x % p.lanes, lane = threadIdx.x & 31, per = blockDim.x / p.lanes, cols = (int)p.cols;
  const uint32_t place = (uint32_t)__cvta_generic_to_shared(inputs) + (threadIdx.x >> 5) * N * kChunk;
  const int64_t step = (int64_t)gridDim.x * per;
  int64_t r = (int64_t)blockIdx.x * per + threadIdx.x / p.lanes;
  const int shift = ODD ? (int)(r * cols & 7) : 0;
  float* weights = (float*)(inputs + (T / 32) * N * kChunk) + (threadIdx.x - t) * N * 8;  // ODD: of the group's columns
  const auto weight = [&](int n, int c, float (&w)[8]) {
    if constexpr (ODD) {
      const float4 a = *(const float4*)(weights + (n * p.lanes + t) * 8), b = *(const float4*)(weights + (n * p.lanes + t) * 8 + 4);
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    } else {
      rn_weight<8>(p.weight, p.weight_dt, c, w);
    }
  };
  const auto ask = [&](int64_t r, bool past) {  // d_y and h, or d_h
    if (r < p.rows && (!past || p.d_h != nullptr)) {
#pragma unroll
      for (int n = 0; n < N; n++) {
        const int c = (n * p.lanes + t - lane) * 8 - shift;
        if (past) {
          qt_ask8<HT, 32, ODD>(p.d_h, r * cols + c, cols - c, place + n * kChunk + kFirst, lane);
        } else {
          qt_ask8<DT, 32, ODD>(p.d_y, r * cols + c, cols - c, place + n * kChunk, lane);
          qt_ask8<HT, 32, ODD>(p.h, r * cols + c, cols - c, place + n * kChunk + kRnBytes<DT>, lane);
        }
      }
    }
    qt_commit();
  };
  pdl_wait();
  ask(r, false);
  ask(r, true);
  if constexpr (ODD) {
    for (int i = t; i < N * p.lanes * 8; i += p.lanes) {
      float one[1] = {0.0f};
      if (i >= shift && i - shift < cols) rn_weight<1>(p.weight, p.weight_dt, i - shift, one);
      weights[i] = one[0];
    }
    __syncthreads();
  }
  float next_rstd = r < p.rows ? __ldg(p.rstd + r) : 0.0f;
  int turn = 0;
  float acc[N][8] = {};
  for (int64_t r0 = (int64_t)blockIdx.x * per; r0 < p.rows; r0 += step, r += step) {
    const bool row_ok = r < p.rows;
    const float rstd = next_rstd;
    QtRaw<DT, 8> d[N];
    QtRaw<HT, 8> h[N];
    qt_wait<1>();
    __syncwarp();
#pragma unroll
    for (int n = 0; n < N; n++) {
      d[n].zero();
      h[n].zero();
      if (row_ok && (n * p.lanes + t) * 8 - shift < cols) {
        qt_taken8<DT>(place + n * kChunk, lane, d[n]);
        qt_taken8<HT>(place + n * kChunk + kRnBytes<DT>, lane, h[n]);
      }
    }
    __syncwarp();
    ask(r + step, false);
    if (r + step < p.rows) next_rstd = __ldg(p.rstd + r + step);
    float sum = 0.0f;
#pragma unroll
    for (int n = 0; n < N; n++) {
      const int c = (n * p.lanes + t) * 8 - shift;
      if (c >= p.cols) continue;
      float dv[8], u[8], w[8];
      weight(n, c, w);
      d[n].get(dv);
      h[n].get(u);
      rn_clear<ODD>(c, cols, dv);
      rn_clear<ODD>(c, cols, u);
#pragma unroll
      for (int k = 0; k < 8; k++) {
        u[k] = __fmul_rn(u[k], rstd);
        sum = __fmaf_rn(__fmul_rn(dv[k], w[k]), u[k], sum);
        acc[n][k] = __fmaf_rn(dv[k], u[k], acc[n][k]);
      }
    }
    const float mean = __fmul_rn(rn_row_sum(sum, p.lanes, sh + (turn ^= 32)), p.one_over_cols);
    qt_wait<1>();
    __syncwarp();
#pragma unroll
    for (int n = 0; n < N; n++) {
      const int c = (n * p.lanes + t) * 8 - shift;
      if (!row_ok || c >= p.cols) continue;
      float dv[8], u[8], w[8];
      weight(n, c, w);
      d[n].get(dv);
      h[n].get(u);
#pragma unroll
      for (int k = 0; k < 8; k++) {
        u[k] = __fmul_rn(u[k], rstd);
        dv[k] = __fmul_rn(rstd, __fmaf_rn(-u[k], mean, __fmul_rn(dv[k], w[k])));
      }
      if (p.d_h != nullptr) {
        QtRaw<HT, 8> past;
        qt_taken8<HT>(place + n * kChunk + kFirst, lane, past);
        past.get(u);
#pragma unroll
        for (int k = 0; k < 8; k++) dv[k] = __fadd_rn(dv[k], u[k]);
      }
      rn_store<HT, ODD, 8>(p.d_x, r * p.cols, c, cols, dv);
    }
    __syncwarp();
    ask(r + step, true);
  }
  qt_wait<0>();
  rn_partial<N, ODD>(p, acc, t, per, shift, (float*)inputs);
  pdl_launch_dependents();
}

// Any alignment, and rows too wide for the kernel before: value by value, kRnBatch of a thread on their way at
// a time, each row read twice; the columns' sums in shared memory, for each
// group of threads its own.
constexpr int kRnBatch = 4;
constexpr int kRnAnyLanes = 128;

template <int DT, int HT>
__global__ void __launch_bounds__(kRnThreads) rmsnorm_backward_any_kernel(RmsNormBackward p) {
  extern __shared__ float acc_sh[];  // [groups of threads][cols]
  __shared__ float sh[64];
  const int t = threadIdx.x % p.lanes, per = blockDim.x / p.lanes, cols = (int)p.cols;
  float* mine = acc_sh + threadIdx.x / p.lanes * cols;
  // the row's values of columns c, c + lanes, ...: where nothing is, the first is read
  const auto values = [&](int64_t row, int c, float rstd, float (&d)[kRnBatch], float (&g)[kRnBatch], float (&u)[kRnBatch]) {
    QtRaw<DT, 1> draw[kRnBatch];
    QtRaw<HT, 1> hraw[kRnBatch];
    float w[kRnBatch][1];
#pragma unroll
    for (int i = 0; i < kRnBatch; i++) {
      const int at = c + i * p.lanes < cols ? c + i * p.lanes : 0;
      draw[i].load(p.d_y, row + at);
      hraw[i].load(p.h, row + at);
      rn_weight<1>(p.weight, p.weight_dt, at, w[i]);
    }
#pragma unroll
    for (int i = 0; i < kRnBatch; i++) {
      float v[1];
      draw[i].get(v);
      d[i] = v[0];
      g[i] = __fmul_rn(v[0], w[i][0]);
      hraw[i].get(v);
      u[i] = __fmul_rn(v[0], rstd);
    }
  };
  pdl_wait();
  int turn = 0;
  for (int c = t; c < cols; c += p.lanes) mine[c] = 0.0f;
  for (int64_t r0 = (int64_t)blockIdx.x * per; r0 < p.rows; r0 += (int64_t)gridDim.x * per) {
    const int64_t r = r0 + threadIdx.x / p.lanes;
    const bool row_ok = r < p.rows;
    const int64_t row = row_ok ? r * cols : 0;
    const float rstd = row_ok ? __ldg(p.rstd + r) : 0.0f;
    float sum = 0.0f, d[kRnBatch], g[kRnBatch], u[kRnBatch];
    for (int c = t; c < cols; c += kRnBatch * p.lanes) {
      values(row, c, rstd, d, g, u);
#pragma unroll
      for (int i = 0; i < kRnBatch; i++) {
        if (c + i * p.lanes >= cols || !row_ok) continue;
        sum = __fmaf_rn(g[i], u[i], sum);
        mine[c + i * p.lanes] = __fmaf_rn(d[i], u[i], mine[c + i * p.lanes]);
      }
    }
    const float mean = __fmul_rn(rn_row_sum(sum, p.lanes, sh + (turn ^= 32)), p.one_over_cols);
    for (int c = t; c < cols && row_ok; c += kRnBatch * p.lanes) {
      float past[kRnBatch][1];
      values(row, c, rstd, d, g, u);
#pragma unroll
      for (int i = 0; i < kRnBatch; i++) {
        past[i][0] = 0.0f;
        if (p.d_h != nullptr) {
          QtRaw<HT, 1> raw;
          rn_load_plain<HT, 1>(p.d_h, row + (c + i * p.lanes < cols ? c + i * p.lanes : t), raw);
          raw.get(past[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < kRnBatch; i++) {
        float o[1] = {__fmul_rn(rstd, __fmaf_rn(-u[i], mean, g[i]))};
        if (p.d_h != nullptr) o[0] = __fadd_rn(o[0], past[i][0]);
        if (c + i * p.lanes < cols) qt_store<HT, 1>(p.d_x, row + c + i * p.lanes, o);
      }
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < cols; c += blockDim.x) {
    float sum = 0.0f;
    for (int i = 0; i < per; i++) sum += acc_sh[i * cols + c];
    p.partial[(int64_t)blockIdx.x * cols + c] = sum;
  }
  pdl_launch_dependents();
}

// d_weight[c] = the sum of `parts` rows of partial sums, kRnSumWarps warps to 32 columns in a fixed order.
constexpr int kRnSumWarps = 32;  // 8: 2 us slower

__global__ void __launch_bounds__(32 * kRnSumWarps) rmsnorm_weight_kernel(const float* partial, int parts, int64_t cols,
                                                                           float* d_weight) {
  __shared__ float sh[kRnSumWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  pdl_wait();
  float sum = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int i = warp; i < parts; i += kRnSumWarps) sum += partial[(int64_t)i * cols + c];
  }
  sh[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && c < cols) {
#pragma unroll
    for (int w = 1; w < kRnSumWarps; w++) sum += sh[w][lane];
    d_weight[c] = sum;
  }
  pdl_launch_dependents();
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
static bool off(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) != 0; }
static size_t size_of(int32_t dt) { return dt == FP8Q_IN_BF16 ? 2 : 4; }
static bool type_ok(int32_t dt) { return dt == FP8Q_IN_BF16 || dt == FP8Q_IN_FP32; }

// Threads of a row of which each has N chunks of V values at most: whole warps.
static int row_lanes(int64_t cols, int v, int n) { return (int)((cols + 32 * v * n - 1) / (32 * v * n)) * 32; }
// CTAs of kernels that stay; odd columns: groups of threads keep their shift.
static int64_t stream_grid(int64_t sets, int64_t fit) { return sets < fit ? sets : fit & ~(int64_t)7; }
// Rows side by side in a CTA of about `threads` threads.
static int row_groups(int lanes, int threads) { return lanes < threads ? threads / lanes : 1; }

template <int DT, int RT, int V, int N>
static cudaError_t launch_norm_rows(RmsNorm& p, cudaStream_t s) {
  p.lanes = row_lanes(p.cols, V, N);
  const int per = row_groups(p.lanes, kRnThreads), threads = p.lanes * per;
  const dim3 grid((unsigned)((p.rows + per - 1) / per));
  return launch_kernel(threads <= kRnThreads ? rmsnorm_kernel<DT, RT, V, N, kRnThreads> : rmsnorm_kernel<DT, RT, V, N, 1024>, grid,
                       dim3(threads), 0, s, p);
}

template <int DT, int RT, int T, bool ODD>
static cudaError_t launch_norm_stream(RmsNorm& p, cudaStream_t s) {
  constexpr size_t kEach = (size_t)kRnChunks * (kRnBytes<DT> + kRnBytes<RT>) / 32;  // of a thread
  p.lanes = row_lanes(p.cols + (ODD ? 7 : 0), 8, kRnChunks);
  const int per = row_groups(p.lanes, kRnThreads), threads = p.lanes * per;
  static PerDevice<bool> allowed;
  const cudaError_t e = allow_smem(allowed, rmsnorm_stream_kernel<DT, RT, T, ODD>, kEach * T);
  if (e != cudaSuccess) return e;
  const int64_t sets = (p.rows + per - 1) / per, fit = (T == kRnThreads ? 2 : 1) * (int64_t)sm_count();
  return launch_kernel(rmsnorm_stream_kernel<DT, RT, T, ODD>, dim3((unsigned)stream_grid(sets, fit)), dim3(threads), kEach * threads, s, p);
}

// Which kernel; each edge with both sides measured (us, BF16, in a graph).
// Few short rows: a row in as many threads as it has chunks, nothing on its way;
//   row copy, residual: 64 x 2048 2.1 (2.8 by CTAs that stay), 304 x 2048 2.4 (2.7),
//   608 x 2048 2.9 (2.9), 64 x 4096 2.4 (2.7), 304 x 4096 3.2 (2.9), 64 x 5120 2.7 (2.7),
//   64 x 7168 3.2 (2.7), 1 x 7168 3.0 (2.6);
//   y of odd columns: 304 x 1001 4.0 (4.7), 304 x 4097 5.5 (4.9), 64 x 8185 6.1 (4.7).
// More than 8192 columns: 512 threads that stay, against 1024 that go, 4000 rows, residual
//   (without): 8208 49 and 57 (35 and 29), 12288 58 and 86 (37 and 44), 16384 70 and 105 (43 and 54).
// More than 16384 columns: 1024 threads, whose 64 registers spill: 4000 x 32768 228 (floor 138).
// Unaligned, or odd columns beyond 8185: value by value (y of 4000 x 32767 651, floor 157).
template <int DT, int RT>
static cudaError_t launch_norm(RmsNorm& p, bool aligned, cudaStream_t s) {
  const bool few = p.rows <= 2 * sm_count() && p.cols <= 4096;
  if (!aligned || p.cols % 8 != 0) {
    if (aligned && !few && p.cols + 7 <= 8 * kRnChunks * kRnThreads) return launch_norm_stream<DT, RT, kRnThreads, true>(p, s);
    return p.cols <= 8192 ? launch_norm_rows<DT, RT, 1, 8>(p, s) : launch_norm_rows<DT, RT, 1, 32>(p, s);
  }
  if (few) return launch_norm_rows<DT, RT, 8, 1>(p, s);
  if (p.cols <= 8 * kRnChunks * kRnThreads) return launch_norm_stream<DT, RT, kRnThreads, false>(p, s);
  if (p.cols <= 8 * kRnChunks * 512) return launch_norm_stream<DT, RT, 512, false>(p, s);
  return launch_norm_rows<DT, RT, 8, 4>(p, s);
}

static int64_t backward_grid(int64_t rows, int per, int ctas) {
  const int64_t sets = (rows + per - 1) / per, fit = (int64_t)sm_count() * ctas, most = fit < kRnMaxPartials ? fit : kRnMaxPartials;
  return stream_grid(sets, most);
}

template <int DT, int HT, int T, bool ODD>
static cudaError_t launch_norm_backward_vec(RmsNormBackward& p, int* parts, cudaStream_t s) {
  constexpr size_t kInputs = (size_t)kRnChunks * (kRnBytes<DT> + 2 * kRnBytes<HT>) / 32;  // of a thread; > the partial sums' 4 * 8 * kRnChunks
  constexpr size_t kEach = kInputs + (ODD ? kRnChunks * 8 * sizeof(float) : 0);
  p.lanes = row_lanes(p.cols + (ODD ? 7 : 0), 8, kRnChunks);
  const int per = row_groups(p.lanes, kRnThreads), threads = p.lanes * per;
  static PerDevice<bool> allowed;
  const cudaError_t e = allow_smem(allowed, rmsnorm_backward_kernel<DT, HT, T, ODD>, kEach * T);
  if (e != cudaSuccess) return e;
  const int64_t grid = backward_grid(p.rows, per, T == kRnThreads ? 2 : 1);
  *parts = (int)grid;
  return launch_kernel(rmsnorm_backward_kernel<DT, HT, T, ODD>, dim3((unsigned)grid), dim3(threads), ODD ? kEach * T : kEach * threads, s, p);
}

template <int DT, int HT>
static cudaError_t launch_norm_backward_any(RmsNormBackward& p, int* parts, cudaStream_t s) {
  const int per = p.cols <= kRnMaxCols / 4 ? kRnThreads / kRnAnyLanes : 1;
  p.lanes = kRnThreads / per;
  const size_t smem = (size_t)per * p.cols * sizeof(float);
  static PerDevice<bool> allowed;
  const cudaError_t e = allow_smem(allowed, rmsnorm_backward_any_kernel<DT, HT>, kRnMaxCols * sizeof(float));
  if (e != cudaSuccess) return e;
  const int64_t grid = backward_grid(p.rows, per, 4);
  *parts = (int)grid;
  return launch_kernel(rmsnorm_backward_any_kernel<DT, HT>, dim3((unsigned)grid), dim3(kRnThreads), smem, s, p);
}

template <int DT, int HT>
static cudaError_t launch_norm_backward(RmsNormBackward& p, bool aligned, int* parts, cudaStream_t s) {
  const bool vec = aligned && p.cols % 8 == 0;
  if (aligned && !vec && p.cols + 7 <= 8 * kRnChunks * kRnThreads) return launch_norm_backward_vec<DT, HT, kRnThreads, true>(p, parts, s);
  if (vec && p.cols <= 8 * kRnChunks * kRnThreads) return launch_norm_backward_vec<DT, HT, kRnThreads, false>(p, parts, s);
  if (vec && p.cols <= 8 * kRnChunks * 512) return launch_norm_backward_vec<DT, HT, 512, false>(p, parts, s);
  return launch_norm_backward_any<DT, HT>(p, parts, s);
}

}  // namespace fp8q

using namespace fp8q;

extern "C" fp8q_status fp8q_rmsnorm(const void* x, int32_t dt, const void* residual, int32_t residual_dt,
                                    const void* weight, int32_t weight_dt, int64_t rows, int64_t cols, float eps,
                                    int32_t fmt, int32_t dir, int32_t pow2_scales, void* h, float* rstd, void* y,
                                    uint8_t* q, float* scale_inv, uint8_t* q_t, float* scale_inv_t, void* stream) {
  clear_error();
  if (!type_ok(dt) || !type_ok(weight_dt) || (residual && !type_ok(residual_dt)))
    return fail(FP8Q_ERR_INVALID_ARG, "dt, residual_dt and weight_dt must be FP8Q_IN_BF16 or FP8Q_IN_FP32");
  if (rows < 0 || cols < 1) return fail(FP8Q_ERR_INVALID_ARG, "rows must be >= 0 and cols >= 1");
  if (rows > INT32_MAX / 2 || cols > kRnMaxCols) return fail(FP8Q_ERR_UNSUPPORTED, "rows too large, or cols > %d", kRnMaxCols);
  if (!(eps >= 0.0f) || eps > 3.4e38f) return fail(FP8Q_ERR_INVALID_ARG, "eps must be finite and >= 0");
  const fp8q_status r = qt_check(rows, cols, fmt, dir, q, scale_inv, q_t, scale_inv_t);
  if (r != FP8Q_OK) return r;
  if (rows == 0) return FP8Q_OK;
  const bool copy = dir != 0;
  const size_t a_x = copy ? 16 : size_of(dt), a_r = copy ? 16 : size_of(residual_dt), a_w = copy ? 16 : size_of(weight_dt);
  if (!x || off(x, a_x)) return fail(FP8Q_ERR_INVALID_ARG, "x must be a device pointer, 16-byte aligned for a copy");
  if (residual && (off(residual, a_r) || !h || off(h, a_r)))
    return fail(FP8Q_ERR_INVALID_ARG, "a residual needs h, both 16-byte aligned for a copy");
  if (!weight || off(weight, a_w)) return fail(FP8Q_ERR_INVALID_ARG, "weight must be a device pointer, 16-byte aligned for a copy");
  if (!rstd || off(rstd, 4)) return fail(FP8Q_ERR_INVALID_ARG, "rstd must be a 4-byte aligned device pointer");
  if (off(y, a_x)) return fail(FP8Q_ERR_INVALID_ARG, "y must be aligned as x is");
  RmsNorm p{};
  p.x = x;
  p.residual = residual;
  p.weight = weight;
  p.weight_dt = weight_dt;
  p.rows = rows;
  p.cols = cols;
  p.eps = eps;
  p.one_over_cols = 1.0f / (float)cols;
  p.fmt = fmt;
  p.pow2 = pow2_scales ? 1 : 0;
  p.tiles_c = (int)((cols + kQtTile - 1) / kQtTile);
  p.h = h;
  p.rstd = rstd;
  p.y = y;
  if (dir & MXFP8_ROW) p.q = q, p.s = scale_inv;
  const cudaStream_t s = (cudaStream_t)stream;
  const bool aligned = !off(x, 16) && !off(residual, 16) && !off(residual ? h : nullptr, 16) &&
                   !off(weight, 16) && !off(y, 16);
  const int rt = residual ? residual_dt : kNone;
  cudaError_t e;
  if (dt == FP8Q_IN_BF16)
    e = rt == kNone ? launch_norm<kBF16, kNone>(p, aligned, s) : rt == kBF16 ? launch_norm<kBF16, kBF16>(p, aligned, s) : launch_norm<kBF16, kFP32>(p, aligned, s);
  else
    e = rt == kNone ? launch_norm<kFP32, kNone>(p, aligned, s) : rt == kBF16 ? launch_norm<kFP32, kBF16>(p, aligned, s) : launch_norm<kFP32, kFP32>(p, aligned, s);
  if (e != cudaSuccess) return cuda_fail(e, "rmsnorm kernel launch");
  if (dir & MXFP8_COL) {
    QtOut o{};
    o.rows = rows;
    o.cols = cols;
    const int64_t tiles_r = (rows + kQtTile - 1) / kQtTile;
    if (tiles_r * p.tiles_c > INT32_MAX) return fail(FP8Q_ERR_UNSUPPORTED, "rows * cols too large");
    o.tiles_r = (int)tiles_r;
    o.tiles_c = p.tiles_c;
    o.pow2 = p.pow2;
    o.q_t = q_t;
    o.s_t = scale_inv_t;
    const int ht = residual ? residual_dt : dt;
    const void* from = residual ? h : x;
    if (ht == FP8Q_IN_BF16) {
      const RmsNormTile<kBF16> src{from, weight, weight_dt, rstd, cols, {}, {}};
      e = fmt == FP8Q_E4M3 ? launch_quant_tiles<RmsNormTile<kBF16>, kE4M3, false, true>(src, o, s)
                           : launch_quant_tiles<RmsNormTile<kBF16>, kE5M2, false, true>(src, o, s);
    } else {
      const RmsNormTile<kFP32> src{from, weight, weight_dt, rstd, cols, {}, {}};
      e = fmt == FP8Q_E4M3 ? launch_quant_tiles<RmsNormTile<kFP32>, kE4M3, false, true>(src, o, s)
                           : launch_quant_tiles<RmsNormTile<kFP32>, kE5M2, false, true>(src, o, s);
    }
    if (e != cudaSuccess) return cuda_fail(e, "rmsnorm transposed copy launch");
  }
  return check_launch("rmsnorm kernel");
}

extern "C" size_t fp8q_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows < 1 || cols < 1 || cols > kRnMaxCols) return 0;
  const int64_t parts = rows < kRnMaxPartials ? rows : kRnMaxPartials;
  return (size_t)parts * cols * sizeof(float);
}

extern "C" fp8q_status fp8q_rmsnorm_backward(const void* d_y, int32_t dt, const void* h, int32_t h_dt, const void* weight,
                                             int32_t weight_dt, const float* rstd, const void* d_h, int64_t rows,
                                             int64_t cols, void* d_x, float* d_weight, void* workspace,
                                             size_t workspace_bytes, void* stream) {
  clear_error();
  if (!type_ok(dt) || !type_ok(h_dt) || !type_ok(weight_dt))
    return fail(FP8Q_ERR_INVALID_ARG, "dt, h_dt and weight_dt must be FP8Q_IN_BF16 or FP8Q_IN_FP32");
  if (rows < 0 || cols < 1) return fail(FP8Q_ERR_INVALID_ARG, "rows must be >= 0 and cols >= 1");
  if (rows > INT32_MAX / 2 || cols > kRnMaxCols) return fail(FP8Q_ERR_UNSUPPORTED, "rows too large, or cols > %d", kRnMaxCols);
  if (!d_weight || off(d_weight, 4)) return fail(FP8Q_ERR_INVALID_ARG, "d_weight must be a 4-byte aligned device pointer");
  const cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  int parts = 0;
  if (rows > 0) {
    if (!d_y || off(d_y, size_of(dt))) return fail(FP8Q_ERR_INVALID_ARG, "d_y must be a device pointer aligned to its type");
    if (!h || off(h, size_of(h_dt)) || !d_x || off(d_x, size_of(h_dt)) || off(d_h, size_of(h_dt)))
      return fail(FP8Q_ERR_INVALID_ARG, "h, d_h and d_x must be device pointers aligned to their type");
    if (!weight || off(weight, size_of(weight_dt)) || !rstd || off(rstd, 4))
      return fail(FP8Q_ERR_INVALID_ARG, "weight and rstd must be device pointers aligned to their type");
    if (!workspace || off(workspace, 16) || workspace_bytes < fp8q_rmsnorm_backward_workspace_bytes(rows, cols))
      return fail(FP8Q_ERR_INVALID_ARG, "workspace must be 16-byte aligned and of fp8q_rmsnorm_backward_workspace_bytes()");
    RmsNormBackward p{};
    p.d_y = d_y;
    p.h = h;
    p.weight = weight;
    p.weight_dt = weight_dt;
    p.rstd = rstd;
    p.d_h = d_h;
    p.rows = rows;
    p.cols = cols;
    p.one_over_cols = 1.0f / (float)cols;
    p.d_x = d_x;
    p.partial = (float*)workspace;
    const bool aligned = !off(d_y, 16) && !off(h, 16) && !off(weight, 16) && !off(d_h, 16) && !off(d_x, 16);
    if (dt == FP8Q_IN_BF16)
      e = h_dt == FP8Q_IN_BF16 ? launch_norm_backward<kBF16, kBF16>(p, aligned, &parts, s) : launch_norm_backward<kBF16, kFP32>(p, aligned, &parts, s);
    else
      e = h_dt == FP8Q_IN_BF16 ? launch_norm_backward<kFP32, kBF16>(p, aligned, &parts, s) : launch_norm_backward<kFP32, kFP32>(p, aligned, &parts, s);
    if (e != cudaSuccess) return cuda_fail(e, "rmsnorm gradient launch");
  }
  e = launch_kernel(rmsnorm_weight_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(32 * kRnSumWarps), 0, s,
                    (const float*)workspace, parts, cols, d_weight);
  if (e != cudaSuccess) return cuda_fail(e, "rmsnorm weight gradient launch");
  return check_launch("rmsnorm gradient kernel");
}
