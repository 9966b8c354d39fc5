// combine.cu -- the experts' rows back to the tokens: a weighted sum, and the
// gradients of the rows and of the weights.
//
//   out[t] = sum_j w[t, j] * y[row_of[t, j]]         (w = 1 without weights)
//   d_y[row_of[t, j]] = w[t, j] * d_out[t],   d_w[t, j] = <d_out[t], y[row_of[t, j]]>
//
// Sums are FP32, over j in order and over columns in a fixed order; each row
// belongs to one slot, so nothing is added by two threads.  Without weights
// the sum is the gradient of the dispatch.  Padding rows of d_y are zeroed.
//
// Bound by memory: each row is read once, wherever it lies, 16 bytes a thread
// and four rows on their way.  65536 rows of 7168 BF16, 8 a token: the sum 181
// us (5.8 TB/s), the gradients 337 us (6.1 TB/s), 399 with one row at a time.
#include "fp8q_device.cuh"
#include "internal.h"

namespace fp8q {

constexpr int kCbThreads = 128;
constexpr int kCbBackThreads = 256;
constexpr int kCbBatch = 4;     // rows a thread has on their way at a time (a missing one reads row 0)
constexpr int kCbPadRows = 64;  // rows whose padding one CTA of the backward grid looks for

struct CbParams {
  const void* y;
  const int* row_of;
  const float* w;
  int64_t tokens, cols, rows;
  int top_k;
  void* out;
  const void* d_out;
  const int* src;
  void* d_y;
  float* d_w;
};

// V consecutive values of type DT as FP32.
template <int DT, int V>
__device__ __forceinline__ void cb_load(const void* p, int64_t i, float (&v)[V]) {
  if constexpr (DT == kBF16) {
    const uint16_t* q = (const uint16_t*)p + i;
    if constexpr (V == 8) {
      const uint4 u = __ldg((const uint4*)q);
      v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
      v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
    } else {
#pragma unroll
      for (int k = 0; k < V; k++) v[k] = __uint_as_float((uint32_t)__ldg(q + k) << 16);
    }
  } else {
    const float* q = (const float*)p + i;
    if constexpr (V == 8) {
      const float4 a = __ldg((const float4*)q), b = __ldg((const float4*)q + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
      for (int k = 0; k < V; k++) v[k] = __ldg(q + k);
    }
  }
}

template <int DT, int V>
__device__ __forceinline__ void cb_store(void* p, int64_t i, const float (&v)[V]) {
  if constexpr (DT == kBF16) {
    uint16_t* q = (uint16_t*)p + i;
    if constexpr (V == 8) {
      uint4 u;
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.x) : "f"(v[1]), "f"(v[0]));
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.y) : "f"(v[3]), "f"(v[2]));
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.z) : "f"(v[5]), "f"(v[4]));
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.w) : "f"(v[7]), "f"(v[6]));
      st_stream(q, u);
    } else {
#pragma unroll
      for (int k = 0; k < V; k++) {
        uint16_t h;
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(v[k]));
        q[k] = h;
      }
    }
  } else {
    float* q = (float*)p + i;
#pragma unroll
    for (int k = 0; k < V; k += 4) {
      if constexpr (V == 8)
        st_stream(q + k, make_uint4(__float_as_uint(v[k]), __float_as_uint(v[k + 1]), __float_as_uint(v[k + 2]),
                                    __float_as_uint(v[k + 3])));
      else
        q[k] = v[k];
    }
  }
}

__device__ __forceinline__ int64_t cb_row(const CbParams& p, int64_t slot) {
  const int r = __ldg(p.row_of + slot);
  return r >= 0 && r < p.rows ? r : -1;
}

template <int DT, int V>
__global__ void __launch_bounds__(kCbThreads) combine_kernel(CbParams p) {
  pdl_wait();
  const int64_t t = blockIdx.x;
  const int64_t c = ((int64_t)blockIdx.y * kCbThreads + threadIdx.x) * V;
  if (c < p.cols) {
    float acc[V];
#pragma unroll
    for (int k = 0; k < V; k++) acc[k] = 0.0f;
    for (int j0 = 0; j0 < p.top_k && p.rows > 0; j0 += kCbBatch) {
      int64_t r[kCbBatch];
      float v[kCbBatch][V];
#pragma unroll
      for (int i = 0; i < kCbBatch; i++) r[i] = j0 + i < p.top_k ? cb_row(p, t * p.top_k + j0 + i) : -1;
#pragma unroll
      for (int i = 0; i < kCbBatch; i++) cb_load<DT, V>(p.y, (r[i] < 0 ? 0 : r[i]) * p.cols + c, v[i]);
#pragma unroll
      for (int i = 0; i < kCbBatch; i++) {
        if (r[i] < 0) continue;
        const float w = p.w ? __ldg(p.w + t * p.top_k + j0 + i) : 1.0f;
#pragma unroll
        for (int k = 0; k < V; k++) acc[k] = __fmaf_rn(w, v[i][k], acc[k]);
      }
    }
    cb_store<DT, V>(p.out, t * p.cols + c, acc);
  }
  pdl_launch_dependents();
}

// CTA t < tokens: one token.  The others zero the padding of kCbPadRows rows.
template <int DT, int V, int KMAX>
__global__ void __launch_bounds__(kCbBackThreads) combine_backward_kernel(CbParams p) {
  __shared__ float part[kCbBackThreads / 32][KMAX];
  __shared__ int64_t rows[KMAX];
  __shared__ float weights[KMAX];
  pdl_wait();
  const int tid = threadIdx.x;
  if (blockIdx.x >= p.tokens) {
    const int64_t r0 = (blockIdx.x - p.tokens) * kCbPadRows;
    float zero[V];
#pragma unroll
    for (int k = 0; k < V; k++) zero[k] = 0.0f;
    for (int64_t r = r0; r < min(r0 + kCbPadRows, p.rows); r++) {
      const int s = __ldg(p.src + r);
      if (s >= 0 && s < p.tokens * p.top_k) continue;
      for (int64_t c = (int64_t)tid * V; c < p.cols; c += kCbBackThreads * V) cb_store<DT, V>(p.d_y, r * p.cols + c, zero);
    }
  } else {
    const int64_t t = blockIdx.x;
    if (tid < KMAX) {
      rows[tid] = tid < p.top_k ? cb_row(p, t * p.top_k + tid) : -1;
      weights[tid] = tid < p.top_k ? __ldg(p.w + t * p.top_k + tid) : 0.0f;
    }
    __syncthreads();
    float dot[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; j++) dot[j] = 0.0f;
    for (int64_t c = (int64_t)tid * V; c < p.cols; c += kCbBackThreads * V) {
      float d[V];
      cb_load<DT, V>(p.d_out, t * p.cols + c, d);
#pragma unroll
      for (int j0 = 0; j0 < KMAX; j0 += kCbBatch) {
        if (j0 >= p.top_k || p.rows == 0) break;
        float v[kCbBatch][V];
#pragma unroll
        for (int i = 0; i < kCbBatch; i++) {
          const int64_t r = rows[j0 + i];
          cb_load<DT, V>(p.y, (r < 0 ? 0 : r) * p.cols + c, v[i]);
        }
#pragma unroll
        for (int i = 0; i < kCbBatch; i++) {
          const int64_t r = rows[j0 + i];
          if (r < 0) continue;
          const float w = weights[j0 + i];
          float o[V];
#pragma unroll
          for (int k = 0; k < V; k++) {
            dot[j0 + i] = __fmaf_rn(d[k], v[i][k], dot[j0 + i]);
            o[k] = __fmul_rn(w, d[k]);
          }
          cb_store<DT, V>(p.d_y, r * p.cols + c, o);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < KMAX; j++) {
      if (j >= p.top_k) break;
      float v = dot[j];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      if ((tid & 31) == 0) part[tid >> 5][j] = v;
    }
    __syncthreads();
    if (tid < p.top_k) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kCbBackThreads / 32; w++) v += part[w][tid];
      p.d_w[t * p.top_k + tid] = v;
    }
  }
  pdl_launch_dependents();
}

template <int DT>
static fp8q_status launch_combine(const CbParams& p, bool backward, bool vec, cudaStream_t s) {
  cudaError_t e;
  if (!backward) {
    const int64_t per = (int64_t)kCbThreads * (vec ? 8 : 1);
    const dim3 grid((unsigned)p.tokens, (unsigned)((p.cols + per - 1) / per));
    e = launch_kernel(vec ? combine_kernel<DT, 8> : combine_kernel<DT, 1>, grid, dim3(kCbThreads), 0, s, p);
  } else {
    const dim3 grid((unsigned)(p.tokens + (p.rows + kCbPadRows - 1) / kCbPadRows));
    const auto kernel = p.top_k <= 8 ? (vec ? combine_backward_kernel<DT, 8, 8> : combine_backward_kernel<DT, 1, 8>)
                                     : (vec ? combine_backward_kernel<DT, 8, 32> : combine_backward_kernel<DT, 1, 32>);
    e = launch_kernel(kernel, grid, dim3(kCbBackThreads), 0, s, p);
  }
  if (e != cudaSuccess) return cuda_fail(e, "combine kernel launch");
  return check_launch("combine kernel");
}

static fp8q_status check_combine(int32_t dt, int64_t tokens, int64_t cols, int32_t top_k, int64_t rows) {
  if (dt != FP8Q_IN_BF16 && dt != FP8Q_IN_FP32) return fail(FP8Q_ERR_INVALID_ARG, "dt must be FP8Q_IN_BF16 or FP8Q_IN_FP32");
  if (tokens < 0 || cols < 0 || rows < 0) return fail(FP8Q_ERR_INVALID_ARG, "tokens, cols and rows must be >= 0");
  if (top_k < 1 || top_k > 32) return fail(FP8Q_ERR_UNSUPPORTED, "top_k must be in [1, 32]");
  if (rows > INT32_MAX || tokens > INT32_MAX / top_k || cols > 65535 * (int64_t)kCbThreads)
    return fail(FP8Q_ERR_UNSUPPORTED, "tokens, cols or rows too large");
  return FP8Q_OK;
}

static bool off(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

}  // namespace fp8q

using namespace fp8q;

extern "C" fp8q_status fp8q_moe_combine(const void* y, int32_t dt, int64_t rows, int64_t cols, const int32_t* row_of,
                                        const float* weights, int64_t tokens, int32_t top_k, void* out, void* stream) {
  clear_error();
  const fp8q_status r = check_combine(dt, tokens, cols, top_k, rows);
  if (r != FP8Q_OK) return r;
  if (tokens * cols == 0) return FP8Q_OK;
  const size_t size = dt == FP8Q_IN_BF16 ? 2 : 4;
  if ((rows > 0 && !y) || off(y, size)) return fail(FP8Q_ERR_INVALID_ARG, "y must be a device pointer aligned to its type");
  if (!out || off(out, size)) return fail(FP8Q_ERR_INVALID_ARG, "out must be a device pointer aligned to its type");
  if (!row_of || off(row_of, 4) || off(weights, 4))
    return fail(FP8Q_ERR_INVALID_ARG, "row_of and weights must be 4-byte aligned device pointers");
  CbParams p{};
  p.y = y;
  p.row_of = row_of;
  p.w = weights;
  p.tokens = tokens;
  p.cols = cols;
  p.rows = rows;
  p.top_k = top_k;
  p.out = out;
  const bool vec = cols % 8 == 0 && !off(y, 16) && !off(out, 16);
  return dt == FP8Q_IN_BF16 ? launch_combine<kBF16>(p, false, vec, (cudaStream_t)stream)
                            : launch_combine<kFP32>(p, false, vec, (cudaStream_t)stream);
}

extern "C" fp8q_status fp8q_moe_combine_backward(const void* d_out, const void* y, int32_t dt, int64_t rows,
                                                 int64_t cols, const int32_t* row_of, const int32_t* src,
                                                 const float* weights, int64_t tokens, int32_t top_k, void* d_y,
                                                 float* d_weights, void* stream) {
  clear_error();
  const fp8q_status r = check_combine(dt, tokens, cols, top_k, rows);
  if (r != FP8Q_OK) return r;
  const size_t size = dt == FP8Q_IN_BF16 ? 2 : 4;
  if (tokens > 0 && cols > 0 && (!d_out || off(d_out, size)))
    return fail(FP8Q_ERR_INVALID_ARG, "d_out must be a device pointer aligned to its type");
  if (rows * cols > 0 && (!y || off(y, size) || !d_y || off(d_y, size)))
    return fail(FP8Q_ERR_INVALID_ARG, "y and d_y must be device pointers aligned to their type");
  if (rows > 0 && (!src || off(src, 4))) return fail(FP8Q_ERR_INVALID_ARG, "src must be a 4-byte aligned device pointer");
  if (tokens > 0 && (!row_of || off(row_of, 4) || !weights || off(weights, 4) || !d_weights || off(d_weights, 4)))
    return fail(FP8Q_ERR_INVALID_ARG, "row_of, weights and d_weights must be 4-byte aligned device pointers");
  if (tokens == 0 && rows * cols == 0) return FP8Q_OK;
  CbParams p{};
  p.y = y;
  p.row_of = row_of;
  p.w = weights;
  p.tokens = tokens;
  p.cols = cols;
  p.rows = rows;
  p.top_k = top_k;
  p.d_out = d_out;
  p.src = src;
  p.d_y = d_y;
  p.d_w = d_weights;
  const bool vec = cols % 8 == 0 && !off(y, 16) && !off(d_out, 16) && !off(d_y, 16);
  return dt == FP8Q_IN_BF16 ? launch_combine<kBF16>(p, true, vec, (cudaStream_t)stream)
                            : launch_combine<kFP32>(p, true, vec, (cudaStream_t)stream);
}
