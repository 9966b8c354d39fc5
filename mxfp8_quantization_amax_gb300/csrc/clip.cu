// clip.cu -- the norm of many gradients together, and their scaling to a
// largest norm.
//
//   norm = sqrt(sum over all tensors of g^2),  scale = min(1, max_norm / (norm + 1e-6))
//   out = g * scale
//
// The tensors of a launch come as a table in the kernel's parameters, cut into
// pieces of 32 KB; a CTA takes pieces by index, so that every sum has a fixed
// order.  Squares are added in FP32 over at most 64 values of a thread, then in
// FP64: across pieces, CTAs and launches.  The CTAs that write add the partial
// sums up themselves, all in the same order, and take the pieces from the last
// on: those are still in L2.
//
// Bound by memory: the norm has to be known before the first value is written,
// so that all but what L2 keeps is read twice.  705M FP32 values 1230 us (385 to
// read, 7.3 TB/s; 845 to read and write, 6.7 TB/s), 180M BF16 values 163 us.
#include <math.h>

#include <algorithm>
#include <new>

#include "quant_tile.cuh"

namespace fp8q {

constexpr int kClThreads = 256;
constexpr int kClPieceBytes = 32768;
constexpr int kClTensors = 256;   // of one launch
constexpr int64_t kClMost = INT64_C(1) << 42;  // values in all: their pieces are counted in 32 bits
constexpr int kClParts = 1216;    // partial sums of one launch: 8 CTAs on each of 152 SMs

struct ClTable {
  const void* g[kClTensors];
  void* out[kClTensors];
  int64_t n[kClTensors];
  int first[kClTensors + 1];  // first piece of each tensor
  uint8_t wide[kClTensors];   // type | aligned << 1
  int tensors;
  bool in_place;              // every tensor is its own output
};

struct ClPiece {
  const void* g;
  void* out;
  int64_t lo, hi;
  int type;
  bool vec;
};

__device__ __forceinline__ ClPiece cl_piece(const ClTable& t, int piece) {
  int lo = 0, hi = t.tensors;  // the last tensor whose first piece is not behind this one
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= piece) lo = mid; else hi = mid;
  }
  ClPiece p;
  p.type = t.wide[lo] & 1;
  p.vec = t.wide[lo] & 2;
  const int64_t per = kClPieceBytes / (p.type == kBF16 ? 2 : 4);
  p.g = t.g[lo];
  p.out = t.out[lo];
  p.lo = (piece - t.first[lo]) * per;
  p.hi = min(p.lo + per, t.n[lo]);
  return p;
}

__device__ __forceinline__ double cl_block_sum(double v, double* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < kClThreads / 32; w++) v += sh[w];
  __syncthreads();
  return v;
}

// FP32 sum of the squares of this thread's values of a piece.
template <int DT>
__device__ __forceinline__ float cl_squares(const ClPiece& p) {
  float s[4] = {};
  if (p.vec) {
    constexpr int kPer = kClThreads * 8, kN = kClPieceBytes / (DT == kBF16 ? 2 : 4) / kPer;
    QtRaw<DT, 8> r[kN];
#pragma unroll
    for (int i = 0; i < kN; i++) {
      const int64_t at = p.lo + i * kPer + threadIdx.x * 8;
      r[i].zero();
      if (at + 8 <= p.hi) {
        r[i].load(p.g, at);
      }
    }
#pragma unroll
    for (int i = 0; i < kN; i++) {
      float v[8];
      r[i].get(v);
#pragma unroll
      for (int k = 0; k < 8; k++) s[k & 3] = __fmaf_rn(v[k], v[k], s[k & 3]);
    }
  }
  // what is left of the last eight, or all of an unaligned tensor
  for (int64_t at = (p.vec ? p.lo + (p.hi - p.lo) / 8 * 8 : p.lo) + threadIdx.x; at < p.hi; at += kClThreads) {
    QtRaw<DT, 1> r;
    float v[1];
    r.load(p.g, at);
    r.get(v);
    s[0] = __fmaf_rn(v[0], v[0], s[0]);
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

__global__ void __launch_bounds__(kClThreads) clip_norm_kernel(const __grid_constant__ ClTable t, double* part) {
  __shared__ double sh[kClThreads / 32];
  pdl_wait();
  double sum = 0.0;
  for (int i = blockIdx.x; i < t.first[t.tensors]; i += gridDim.x) {
    const ClPiece p = cl_piece(t, i);
    sum += (double)(p.type == kBF16 ? cl_squares<kBF16>(p) : cl_squares<kFP32>(p));
  }
  sum = cl_block_sum(sum, sh);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
  pdl_launch_dependents();
}

// Every thread of the CTA gets the norm.
__device__ __forceinline__ float cl_norm(const double* part, int parts, double* sh) {
  double sum = 0.0;
#pragma unroll 4
  for (int i = threadIdx.x; i < parts; i += kClThreads) sum += part[i];  // written by the kernel before: no read-only load
  return (float)sqrt(cl_block_sum(sum, sh));
}
__device__ __forceinline__ float cl_scale(float norm, float max_norm) {
  const float s = __fdiv_rn(max_norm, __fadd_rn(norm, 1e-6f));
  return s > 1.0f ? 1.0f : s;  // NaN stays
}

__global__ void __launch_bounds__(kClThreads) clip_scale_kernel(const double* part, int parts, float max_norm, float* norm,
                                                                 float* scale) {
  __shared__ double sh[kClThreads / 32];
  pdl_wait();
  const float n = cl_norm(part, parts, sh);
  if (threadIdx.x == 0) {
    *norm = n;
    if (scale != nullptr) *scale = cl_scale(n, max_norm);
  }
  pdl_launch_dependents();
}

template <int DT>
__device__ __forceinline__ void cl_write(const ClPiece& p, float scale) {
  if (p.vec) {
    constexpr int kPer = kClThreads * 8, kN = kClPieceBytes / (DT == kBF16 ? 2 : 4) / kPer;
    QtRaw<DT, 8> r[kN];
#pragma unroll
    for (int i = 0; i < kN; i++) {
      const int64_t at = p.lo + i * kPer + threadIdx.x * 8;
      if (at + 8 <= p.hi) {
        if constexpr (DT == kBF16) {
          r[i].a = *(const uint4*)((const uint16_t*)p.g + at);
        } else {
          r[i].a = *(const uint4*)((const float*)p.g + at);
          r[i].b = *(const uint4*)((const float*)p.g + at + 4);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kN; i++) {
      const int64_t at = p.lo + i * kPer + threadIdx.x * 8;
      if (at + 8 <= p.hi) {
        float v[8];
        r[i].get(v);
#pragma unroll
        for (int k = 0; k < 8; k++) v[k] = __fmul_rn(v[k], scale);
        qt_store<DT, 8>(p.out, at, v);
      }
    }
  }
  for (int64_t at = (p.vec ? p.lo + (p.hi - p.lo) / 8 * 8 : p.lo) + threadIdx.x; at < p.hi; at += kClThreads) {
    float v[1];
    v[0] = DT == kBF16 ? __uint_as_float((uint32_t)((const uint16_t*)p.g)[at] << 16) : ((const float*)p.g)[at];
    v[0] = __fmul_rn(v[0], scale);
    qt_store<DT, 1>(p.out, at, v);
  }
}

// In place a scale of 1 leaves nothing to do (NaN payloads apart).
__global__ void __launch_bounds__(kClThreads) clip_write_kernel(const __grid_constant__ ClTable t, const double* part, int parts,
                                                                 float max_norm, float* norm, float* scale_at, bool first) {
  __shared__ double sh[kClThreads / 32];
  pdl_wait();
  float scale;
  if (parts > 0) {
    const float n = cl_norm(part, parts, sh);
    scale = cl_scale(n, max_norm);
    if (first && blockIdx.x == 0 && threadIdx.x == 0) *norm = n, *scale_at = scale;
  } else {
    scale = *scale_at;
  }
  if (!(t.in_place && scale == 1.0f)) {
    for (int i = t.first[t.tensors] - 1 - (int)blockIdx.x; i >= 0; i -= gridDim.x) {
      const ClPiece p = cl_piece(t, i);
      if (scale == 1.0f && p.g == p.out) continue;
      if (p.type == kBF16) cl_write<kBF16>(p, scale);
      else cl_write<kFP32>(p, scale);
    }
  }
  pdl_launch_dependents();
}

static bool off(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

// Tables of up to kClTensors tensors at a time.
struct ClWalk {
  const void* const* g;
  void* const* out;
  const int64_t* n;
  const int32_t* dt;
  int count, at;
  bool next(ClTable* t) {
    if (at >= count) return false;
    t->tensors = 0;
    t->first[0] = 0;
    t->in_place = true;
    for (; at < count && t->tensors < kClTensors; at++) {
      if (n[at] == 0) continue;
      const int i = t->tensors;
      const int64_t per = kClPieceBytes / (dt[at] == FP8Q_IN_BF16 ? 2 : 4), pieces = (n[at] + per - 1) / per;
      t->g[i] = g[at];
      t->out[i] = out ? out[at] : nullptr;
      t->n[i] = n[at];
      t->in_place = t->in_place && t->g[i] == t->out[i];
      t->wide[i] = (uint8_t)(dt[at] | (off(g[at], 16) || (out && off(out[at], 16)) ? 0 : 2));
      t->first[i + 1] = t->first[i] + (int)pieces;
      t->tensors++;
    }
    return t->tensors > 0;
  }
};

// Bytes of a gradient, of an output, or of a tensor that is both.
struct ClRange {
  uintptr_t lo, hi;
  bool out;
};

// Whether an output overlaps another tensor.  In the order of their starts a
// range overlaps one before it if that one ends behind its start.
static bool overlapping(const void* const* g, void* const* out, const int64_t* n, const int32_t* dt, int count, ClRange* r) {
  int ranges = 0;
  for (int i = 0; i < count; i++) {
    if (n[i] == 0) continue;
    const uintptr_t bytes = (uintptr_t)n[i] * (dt[i] == FP8Q_IN_BF16 ? 2 : 4), from = (uintptr_t)g[i], to = (uintptr_t)out[i];
    r[ranges++] = ClRange{to, to + bytes, true};
    if (from != to) r[ranges++] = ClRange{from, from + bytes, false};
  }
  std::sort(r, r + ranges, [](const ClRange& a, const ClRange& b) { return a.lo < b.lo; });
  uintptr_t read = 0, written = 0;  // ends of the ranges so far
  for (int i = 0; i < ranges; i++) {
    if (r[i].lo < written || (r[i].out && r[i].lo < read)) return true;
    uintptr_t& end = r[i].out ? written : read;
    end = std::max(end, r[i].hi);
  }
  return false;
}

}  // namespace fp8q

using namespace fp8q;

extern "C" size_t fp8q_clip_grads_workspace_bytes(int32_t count) {
  if (count < 0) return 0;
  return ((size_t)count / kClTensors + 2) * kClParts * sizeof(double);
}

extern "C" fp8q_status fp8q_clip_grads(const void* const* grads, const int64_t* sizes, const int32_t* dts, int32_t count,
                                       float max_norm, void* const* out, float* norm, float* scale, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  clear_error();
  if (count < 0 || count > (1 << 20)) return fail(FP8Q_ERR_INVALID_ARG, "count must be in [0, 2^20]");
  if (count > 0 && (!grads || !sizes || !dts)) return fail(FP8Q_ERR_INVALID_ARG, "grads, sizes and dts are required");
  if (!norm || off(norm, 4)) return fail(FP8Q_ERR_INVALID_ARG, "norm must be a 4-byte aligned device pointer");
  if (out && !scale) return fail(FP8Q_ERR_INVALID_ARG, "scale is required with out");
  if (off(scale, 4)) return fail(FP8Q_ERR_INVALID_ARG, "scale must be a 4-byte aligned device pointer");
  if (scale && !(max_norm >= 0.0f)) return fail(FP8Q_ERR_INVALID_ARG, "max_norm must be >= 0");
  int64_t total = 0;
  for (int i = 0; i < count; i++) {
    if (dts[i] != FP8Q_IN_BF16 && dts[i] != FP8Q_IN_FP32) return fail(FP8Q_ERR_INVALID_ARG, "dts must be FP8Q_IN_BF16 or FP8Q_IN_FP32");
    const size_t size = dts[i] == FP8Q_IN_BF16 ? 2 : 4;
    if (sizes[i] < 0) return fail(FP8Q_ERR_INVALID_ARG, "sizes must be >= 0");
    total += sizes[i] < kClMost ? sizes[i] : kClMost + 1;
    if (total > kClMost) return fail(FP8Q_ERR_UNSUPPORTED, "more than 2^42 values");
    if (sizes[i] > 0 && (!grads[i] || off(grads[i], size) || (out && (!out[i] || off(out[i], size)))))
      return fail(FP8Q_ERR_INVALID_ARG, "gradient %d: device pointers aligned to their type are required", i);
  }
  if (!workspace || off(workspace, 8) || workspace_bytes < fp8q_clip_grads_workspace_bytes(count))
    return fail(FP8Q_ERR_INVALID_ARG, "workspace must be 8-byte aligned and of fp8q_clip_grads_workspace_bytes()");
  if (out) {
    ClRange few[128], *ranges = count <= 64 ? few : new (std::nothrow) ClRange[2 * (size_t)count];
    if (!ranges) return fail(FP8Q_ERR_UNSUPPORTED, "no host memory for %d tensors", count);
    const bool bad = overlapping(grads, out, sizes, dts, count, ranges);
    if (ranges != few) delete[] ranges;
    if (bad) return fail(FP8Q_ERR_INVALID_ARG, "an output overlaps another tensor");
  }
  const cudaStream_t s = (cudaStream_t)stream;
  const int most = 8 * sm_count() < kClParts ? 8 * sm_count() : kClParts;
  ClTable t;
  int parts = 0;
  cudaError_t e;
  for (ClWalk w{grads, nullptr, sizes, dts, count, 0}; w.next(&t);) {
    const int grid = t.first[t.tensors] < most ? t.first[t.tensors] : most;
    e = launch_kernel(clip_norm_kernel, dim3(grid), dim3(kClThreads), 0, s, t, (double*)workspace + parts);
    if (e != cudaSuccess) return cuda_fail(e, "clip norm launch");
    parts += grid;
  }
  // up to this many partial sums every writing CTA adds up (10 us for all of them)
  const bool apart = !out || parts == 0 || parts > 4 * kClParts;
  if (apart) {
    e = launch_kernel(clip_scale_kernel, dim3(1), dim3(kClThreads), 0, s, (const double*)workspace, parts, max_norm, norm, scale);
    if (e != cudaSuccess) return cuda_fail(e, "clip scale launch");
  }
  if (out) {
    bool first = true;
    for (ClWalk w{grads, out, sizes, dts, count, 0}; w.next(&t); first = false) {
      const int grid = t.first[t.tensors] < most ? t.first[t.tensors] : most;
      e = launch_kernel(clip_write_kernel, dim3(grid), dim3(kClThreads), 0, s, t, (const double*)workspace, apart ? 0 : parts, max_norm, norm,
                        scale, first);
      if (e != cudaSuccess) return cuda_fail(e, "clip write launch");
    }
  }
  return check_launch("clip kernel");
}
