// route.cu -- routing of tokens to experts, and its gradient.
//
// A token's logits x[e] give scores s = softmax(x) or 1 / (1 + exp(-x)) and
// keys to choose by: s[e] + bias[e], or, with neither bias nor groups, x[e]
// itself (the same order without the rounding of s).  With groups, a group
// of E / groups consecutive experts is worth the sum of its two best keys
// and only the best groups stay.  The top_k best keys are chosen, equal keys
// from the lowest index, and weigh
//   w_j = c * s_j / sum_i s_i    (renormalised)    or    c * s_j.
// A logit of -inf or NaN is never chosen (id -1, weight 0 where too few are
// left); a NaN, under softmax also +inf, makes the token's weights NaN.
//
// Gradient, with d_j the gradient of w_j and g_j that of s_j:
//   renormalised  g_j = c * (d_j - sum_i d_i s_i / S) / S,  S = sum_i s_i
//                 (d less that of an expert with more than half of S: nothing
//                 cancels where it has nearly all)
//   else          g_j = c * d_j
//   sigmoid       dx_j = g_j s_j (1 - s_j),  0 for experts not chosen
//   softmax       dx_e = p_e (g_e - sum_j g_j p_j); renormalised, the last
//                 sum is zero and p_j / S a softmax over the chosen alone.
// The bias and the choice have no gradient.  A token whose weights are NaN has
// NaN for the gradient of each of its logits.
//
// One warp takes one token, expert e = lane + 32 i in register i.  A choice is
// one warp-wide integer maximum of the order-preserving bits of the lanes'
// best and a ballot of who has it (a minimum of the indices where several do);
// that lane writes its expert to shared memory.
// Up to 256 experts each lane sorts its keys first (52 to 54 us for 65536
// tokens over 256 experts, 8 each, 31 over 64; a search of all registers for each choice
// takes 63).  Bound by instructions (77% of the issue slots), five times the
// 10 us that reading FP32 logits takes.  The gradient of the chosen, 24 us with
// inputs beyond L2, is near what reading the logits and writing theirs takes
// (20 us); that of plain softmax, 52 us, is bound by instructions again (70%).
#include "fp8q_device.cuh"
#include "internal.h"

namespace fp8q {

constexpr int kRtWarps = 8;
constexpr int kRtMaxExperts = 1024;
constexpr unsigned kFull = 0xFFFFFFFFu;

struct RtParams {
  const void* logits;
  int64_t tokens;
  int experts, top_k;
  int renorm;
  float weight_scale;
  const float* bias;
  int groups, top_groups;
  float* weights;
  int* ids;
  const int* ids_in;
  const float* d_weights;
  void* d_logits;
};

template <int DT>
__device__ __forceinline__ float rt_load(const void* p, int64_t i) {
  if constexpr (DT == kBF16)
    return __uint_as_float((uint32_t)__ldg((const uint16_t*)p + i) << 16);
  else
    return __ldg((const float*)p + i);
}

// A token's logits, -inf beyond them; no load waits for a branch.
template <int DT, int V>
__device__ __forceinline__ void rt_load_row(const RtParams& p, int64_t t, int lane, float (&x)[V]) {
  const int64_t row = t * p.experts;
  if (p.experts == 32 * V) {
#pragma unroll
    for (int i = 0; i < V; i++) x[i] = rt_load<DT>(p.logits, row + lane + 32 * i);
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) x[i] = rt_load<DT>(p.logits, row + min(lane + 32 * i, p.experts - 1));
#pragma unroll
    for (int i = 0; i < V; i++)
      if (lane + 32 * i >= p.experts) x[i] = __uint_as_float(0xFF800000u);
  }
}

template <int DT>
__device__ __forceinline__ void rt_store(void* p, int64_t i, float v) {
  if constexpr (DT == kBF16) {
    uint16_t h;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(v));
    ((uint16_t*)p)[i] = h;
  } else {
    ((float*)p)[i] = v;
  }
}

__device__ __forceinline__ float rt_sigmoid(float x) { return __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-x))); }

// Unsigned integers in the order of the floats (-0 as +0); always above 0.
__device__ __forceinline__ uint32_t rt_order(float v) {
  const uint32_t u = __float_as_uint(__fadd_rn(v, 0.0f));
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float rt_value(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

__device__ __forceinline__ float rt_warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ float rt_warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

// Zeroes the keys (in shared memory, order-preserving bits) outside the best
// groups.  32 / 2^ceil(log2 groups) lanes share a group.
__device__ __forceinline__ void rt_keep_groups(uint32_t* keys, const RtParams& p, int lane) {
  const int size = p.experts / p.groups;
  int lanes = 32;
  while (lanes * p.groups > 32) lanes >>= 1;
  const int g = lane / lanes, j = lane % lanes;
  uint32_t a = 0, b = 0;  // best and second best
  if (g < p.groups) {
    for (int i = j; i < size; i += lanes) {
      const int e = g * size + i;
      const uint32_t v = keys[e + (e >> 5)];
      b = max(b, min(a, v));
      a = max(a, v);
    }
  }
  for (int o = 1; o < lanes; o <<= 1) {
    const uint32_t a2 = __shfl_xor_sync(kFull, a, o), b2 = __shfl_xor_sync(kFull, b, o);
    b = max(min(a, a2), max(b, b2));
    a = max(a, a2);
  }
  const float none = __uint_as_float(0xFF800000u);
  const float va = a ? rt_value(a) : none, vb = b ? rt_value(b) : none;
  const uint32_t worth = g < p.groups && j == 0 ? rt_order(size > 1 ? __fadd_rn(va, vb) : va) : 0u;
  uint32_t mine = worth;
  bool keep = false;
  for (int i = 0; i < p.top_groups; i++) {
    const uint32_t best = __reduce_max_sync(kFull, mine);
    const unsigned who = __ballot_sync(kFull, mine == best);
    if (lane == __ffs(who) - 1) {
      keep = true;
      mine = 0;
    }
  }
  const unsigned kept = __ballot_sync(kFull, keep);
  for (int e = lane; e < p.experts; e += 32)
    if (!((kept >> (e / size * lanes)) & 1u)) keys[e + (e >> 5)] = 0;
  __syncwarp();
}

// The order-preserving bits of +inf and of -inf, and what stands for a NaN.
constexpr uint32_t kRtInf = 0xFF800000u, kRtNan = 0xFFFFFFFFu, kRtNone = 0x007FFFFFu;

// BYLOGIT: no bias and no groups, so the logits are the keys.
template <int DT, bool SOFTMAX, bool BYLOGIT, int V>
__global__ void __launch_bounds__(kRtWarps * 32) route_kernel(RtParams p) {
  extern __shared__ uint32_t rt_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ int picks[kRtWarps][32];
  uint32_t* sh = rt_smem + warp * (V * 33);
  const float none = __uint_as_float(0xFF800000u);
  pdl_wait();
  for (int64_t t = (int64_t)blockIdx.x * kRtWarps + warp; t < p.tokens; t += (int64_t)gridDim.x * kRtWarps) {
    float x[V];
    if constexpr (V > 8) {  // 1024 experts, BF16: 163 us, 360 with a question before each load; 256 experts: 54, 53
      rt_load_row<DT, V>(p, t, lane, x);
    } else {
#pragma unroll
      for (int i = 0; i < V; i++) {
        const int e = lane + 32 * i;
        x[i] = e < p.experts ? rt_load<DT>(p.logits, t * p.experts + e) : none;
      }
    }
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; i++) key[i] = x[i] == x[i] ? rt_order(x[i]) : kRtNan;
    // the largest key tells of a NaN or (under softmax) an infinity
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < V; i++) top = max(top, key[i]);
    top = __reduce_max_sync(kFull, top);
    const bool poison = SOFTMAX ? top >= kRtInf : top == kRtNan;
    if (top == kRtNan) {  // the maximum of the others
      top = 0;
#pragma unroll
      for (int i = 0; i < V; i++) {
        if (key[i] == kRtNan) key[i] = 0;
        top = max(top, key[i]);
      }
      top = __reduce_max_sync(kFull, top);
    }
    const float most = top ? rt_value(top) : none;
    float sum = 1.0f;
    if (SOFTMAX && !(BYLOGIT && p.renorm)) {
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < V; i++) sum += x[i] == x[i] ? expf(x[i] - most) : 0.0f;
      sum = rt_warp_sum(sum);
    }
    const auto score = [&](float v) { return SOFTMAX ? __fdiv_rn(expf(v - most), sum) : rt_sigmoid(v); };
    if constexpr (!BYLOGIT) {
#pragma unroll
      for (int i = 0; i < V; i++) {
        const int e = lane + 32 * i;
        float k = score(x[i]);
        if (p.bias != nullptr && e < p.experts) k = __fadd_rn(k, __ldg(p.bias + e));
        key[i] = x[i] > none && k > none ? rt_order(k) : 0u;
      }
      if (p.groups > 1) {
#pragma unroll
        for (int i = 0; i < V; i++) sh[lane + 33 * i] = key[i];
        __syncwarp();
        rt_keep_groups(sh, p, lane);
#pragma unroll
        for (int i = 0; i < V; i++) key[i] = sh[lane + 33 * i];
        __syncwarp();
      }
    }
    // Each lane's best first, so that a choice is one maximum of the heads and
    // one shift of the chosen lane's queue.  Equal keys keep their order.
    uint32_t place = 0x76543210u;  // register of each queue entry, 4 bits each
    if constexpr (V <= 8 && V > 1) {
      uint32_t at[V];
#pragma unroll
      for (int i = 0; i < V; i++) at[i] = i;
#pragma unroll
      for (int n = V - 1; n > 0; n--)
#pragma unroll
        for (int i = 0; i < n; i++) {
          const bool swap = key[i + 1] > key[i];
          const uint32_t k0 = max(key[i], key[i + 1]), k1 = min(key[i], key[i + 1]);
          const uint32_t a0 = swap ? at[i + 1] : at[i], a1 = swap ? at[i] : at[i + 1];
          key[i] = k0, key[i + 1] = k1, at[i] = a0, at[i + 1] = a1;
        }
      place = 0;
#pragma unroll
      for (int i = 0; i < V; i++) place |= at[i] << (4 * i);
    }
    int j = 0;
    for (; j < p.top_k; j++) {
      uint32_t best = 0;
      int at = 0;
      if constexpr (V <= 8) {
        best = key[0];
        at = place & 15;
      } else {
#pragma unroll
        for (int i = 0; i < V; i++)
          if (key[i] > best) {
            best = key[i];
            at = i;
          }
      }
      const uint32_t chosen = j == 0 && BYLOGIT ? top : __reduce_max_sync(kFull, best);
      if (chosen <= kRtNone) break;
      bool mine = best == chosen;
      const unsigned who = __ballot_sync(kFull, mine);
      if (who & (who - 1)) mine = lane == (int)(__reduce_min_sync(kFull, mine ? (unsigned)(lane + 32 * at) : kFull) & 31);
      if (mine) {
        picks[warp][j] = lane + 32 * at;
        if constexpr (V <= 8) {
#pragma unroll
          for (int i = 0; i + 1 < V; i++) key[i] = key[i + 1];
          key[V - 1] = 0;
          place >>= 4;
        } else {
#pragma unroll
          for (int i = 0; i < V; i++)
            if (i == at) key[i] = 0;
        }
      }
    }
    __syncwarp();
    const int id = lane < j ? picks[warp][lane] : -1;
    __syncwarp();
    float w = 0.0f;
    if (id >= 0) w = score(rt_load<DT>(p.logits, t * p.experts + id));
    if (p.renorm) {
      float s = rt_warp_sum(w);
      // Experts that a bias or a group chose far below the best logit: their
      // scores run out of FP32, the softmax over them alone does not
      if (SOFTMAX && !BYLOGIT && s < 0x1p-60f) {
        const float v = id >= 0 ? rt_load<DT>(p.logits, t * p.experts + id) : none;
        const float top_v = rt_warp_max(v);
        w = id >= 0 ? expf(v - top_v) : 0.0f;
        s = rt_warp_sum(w);
      }
      w = s > 0.0f ? __fdiv_rn(w, s) : s == 0.0f ? 0.0f : s;
    }
    w = __fmul_rn(w, p.weight_scale);
    if (poison) w = __uint_as_float(0x7FC00000u);
    if (lane < p.top_k) {
      p.weights[t * p.top_k + lane] = w;
      p.ids[t * p.top_k + lane] = id;
    }
  }
  pdl_launch_dependents();
}

// A logit that makes routing's weights NaN.
template <bool SOFTMAX>
__device__ __forceinline__ bool rt_poison(float x) {
  return SOFTMAX ? !(x < __uint_as_float(0x7F800000u)) : x != x;
}

// The gradient where it reaches the chosen experts alone (sigmoid scores, or
// renormalised softmax): L = 8, 16 or 32 lanes take a token, a slot each, after
// the warp has cleared its tokens' rows.  All logits are read nevertheless: one
// that is NaN is never chosen, and must not pass unseen.
template <int DT, bool SOFTMAX, int L>
__global__ void __launch_bounds__(kRtWarps * 32) route_backward_chosen_kernel(RtParams p) {
  constexpr int N = 32 / L;  // tokens of a warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane % L;
  const auto total = [](float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
  };
  pdl_wait();
  for (int64_t t0 = ((int64_t)blockIdx.x * kRtWarps + warp) * N; t0 < p.tokens; t0 += (int64_t)gridDim.x * kRtWarps * N) {
    const int64_t t = t0 + lane / L;
    int id = -1;
    float d = 0.0f, x = __uint_as_float(0xFF800000u);
    if (t < p.tokens && j < p.top_k) {
      id = __ldg(p.ids_in + t * p.top_k + j);
      if (id < 0 || id >= p.experts) id = -1;
      if (id >= 0) {
        d = __ldg(p.d_weights + t * p.top_k + j);
        x = rt_load<DT>(p.logits, t * p.experts + id);
      }
    }
    // the rows: looked through and cleared, 16 bytes at a time where they allow it
    const int size = DT == kBF16 ? 2 : 4, n = (int)min((int64_t)N, p.tokens - t0) * p.experts;
    const char* from = (const char*)p.logits + t0 * p.experts * size;
    char* row = (char*)p.d_logits + t0 * p.experts * size;
    uint32_t bad = 0;  // bit i: token t0 + i
    if ((((uintptr_t)row | (uintptr_t)from | (uintptr_t)(n * size)) & 15) == 0) {
      constexpr int kBatch = 4;  // loads on their way
      for (int i0 = lane * 16; i0 < n * size; i0 += kBatch * 512) {
        uint4 v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; k++)
          v[k] = i0 + 512 * k < n * size ? __ldg((const uint4*)(from + i0 + 512 * k)) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < kBatch; k++) {
          const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
          uint32_t which = 0;  // of the values of these 16 bytes
#pragma unroll
          for (int q = 0; q < 4; q++) {
            if constexpr (DT == kBF16) {
              which |= (uint32_t)rt_poison<SOFTMAX>(bf16_lo(u[q])) << (2 * q);
              which |= (uint32_t)rt_poison<SOFTMAX>(bf16_hi(u[q])) << (2 * q + 1);
            } else {
              which |= (uint32_t)rt_poison<SOFTMAX>(__uint_as_float(u[q])) << q;
            }
          }
          for (; which; which &= which - 1) bad |= 1u << (((i0 + 512 * k) / size + __ffs(which) - 1) / p.experts);
          if (i0 + 512 * k < n * size) *(uint4*)(row + i0 + 512 * k) = make_uint4(0, 0, 0, 0);
        }
      }
    } else {
      for (int i = lane; i < n; i += 32) {
        if (rt_poison<SOFTMAX>(rt_load<DT>(from, i))) bad |= 1u << (i / p.experts);
        rt_store<DT>(row, i, 0.0f);
      }
    }
    float s = 0.0f, dx;
    if constexpr (SOFTMAX) {
      float most = x;
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(kFull, most, o));
      if (id >= 0) s = expf(x - most);
    } else if (id >= 0) {
      s = rt_sigmoid(x);
    }
    if (p.renorm) {
      const float all = total(s);
      const float share = all != 0.0f ? __fdiv_rn(s, all) : 0.0f;
      // Less the d of the one expert that may have more than half, so that what
      // it has of the mean is exactly 0: of its d - mean nothing would be left
      // where its share is nearly 1.  (Taken off always, one more rounding
      // makes usual gradients a quarter less exact.)
      const float r = total(share > 0.5f ? d : 0.0f);
      d = id >= 0 ? __fsub_rn(d, r) : 0.0f;
      const float mean = total(__fmul_rn(d, share));
      // p_j g_j (softmax) and g_j s_j (sigmoid) are both c (d_j - mean) s_j / S
      dx = __fmul_rn(__fmul_rn(p.weight_scale, __fsub_rn(d, mean)), share);
    } else {
      dx = __fmul_rn(__fmul_rn(p.weight_scale, d), s);
    }
    // 1 - s is the score of -x: of a rounded s near 1 the difference keeps few
    // digits (x = 12: off by 0.9%; x = 17: 0 instead of 4e-8)
    if (!SOFTMAX) dx = __fmul_rn(dx, rt_sigmoid(-x));
    __syncwarp();
    if (id >= 0) rt_store<DT>(p.d_logits, t * p.experts + id, dx);
    bad = __reduce_or_sync(kFull, bad);
    if (bad) {
      __syncwarp();  // after the chosen logits' gradients
      for (int i = lane; i < n; i += 32)
        if (bad >> (i / p.experts) & 1u) rt_store<DT>(row, i, __uint_as_float(0x7FC00000u));
    }
  }
  pdl_launch_dependents();
}

// The gradient of softmax weights that are not renormalised: every expert's.
template <int DT, int V>
__global__ void __launch_bounds__(kRtWarps * 32) route_backward_all_kernel(RtParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float none = __uint_as_float(0xFF800000u);
  pdl_wait();
  for (int64_t t = (int64_t)blockIdx.x * kRtWarps + warp; t < p.tokens; t += (int64_t)gridDim.x * kRtWarps) {
    int id = -1;
    float g = 0.0f, xj = none;
    if (lane < p.top_k) {
      id = __ldg(p.ids_in + t * p.top_k + lane);
      if (id < 0 || id >= p.experts) id = -1;
      if (id >= 0) {
        g = __fmul_rn(p.weight_scale, __ldg(p.d_weights + t * p.top_k + lane));
        xj = rt_load<DT>(p.logits, t * p.experts + id);
      }
    }
    float x[V], most = none, others = 0.0f;
    int peaks = 0;  // logits equal to the largest: their exponentials are 1
    bool bad = false;  // a NaN beside -inf alone would leave the maximum at -inf
#pragma unroll
    for (int i = 0; i < V; i++) {
      const int e = lane + 32 * i;
      x[i] = e < p.experts ? rt_load<DT>(p.logits, t * p.experts + e) : none;
      bad |= rt_poison<true>(x[i]);
      most = fmaxf(most, x[i]);
    }
    most = rt_warp_max(most);
    if (__any_sync(kFull, bad)) {
      for (int e = lane; e < p.experts; e += 32) rt_store<DT>(p.d_logits, t * p.experts + e, __uint_as_float(0x7FC00000u));
      continue;
    }
#pragma unroll
    for (int i = 0; i < V; i++) {
      const bool peak = most > none && x[i] == most;
      x[i] = most > none ? expf(x[i] - most) : 0.0f;
      others += peak ? 0.0f : x[i];
      peaks += peak;
    }
    others = rt_warp_sum(others);
    peaks = __reduce_add_sync(kFull, peaks);
    const float sum = __fadd_rn(others, (float)peaks);
    const float s = id >= 0 ? __fdiv_rn(expf(xj - most), sum) : 0.0f;
    // sum_j g_j p_j, and g - that.  Alone at the top an expert's p may be nearly
    // 1, and its g (1 - p) - (the others' sum) is taken from the others
    const float gs = __fmul_rn(g, s);
    const bool lone = id >= 0 && peaks == 1 && xj == most;
    const unsigned who = __ballot_sync(kFull, lone);
    const float rest = rt_warp_sum(lone ? 0.0f : gs);
    const float dot = who ? __fadd_rn(rest, __shfl_sync(kFull, gs, __ffs(who) - 1)) : rest;
    const float left = lone ? __fsub_rn(__fmul_rn(g, __fdiv_rn(others, sum)), rest) : __fsub_rn(g, dot);
#pragma unroll
    for (int i = 0; i < V; i++) {
      const int e = lane + 32 * i;
      if (e < p.experts)
        rt_store<DT>(p.d_logits, t * p.experts + e, most > none ? -__fmul_rn(__fdiv_rn(x[i], sum), dot) : 0.0f);
    }
    __syncwarp();
    if (id >= 0) rt_store<DT>(p.d_logits, t * p.experts + id, __fmul_rn(s, left));
  }
  pdl_launch_dependents();
}

// One warp for each `per` tokens, at most 8 CTAs of warps an SM.
static fp8q_status launch_rt(void (*kernel)(RtParams), const RtParams& p, int per, size_t smem, cudaStream_t s) {
  int64_t grid = (p.tokens + per * kRtWarps - 1) / (per * kRtWarps);
  const int64_t cap = (int64_t)sm_count() * 8;
  if (grid > cap) grid = cap;
  const cudaError_t e = launch_kernel(kernel, dim3((unsigned)grid), dim3(kRtWarps * 32), smem, s, p);
  if (e != cudaSuccess) return cuda_fail(e, "route kernel launch");
  return check_launch("route kernel");
}

template <int DT, bool SOFTMAX, int V>
static fp8q_status launch_route_v(const RtParams& p, bool backward, cudaStream_t s) {
  if (backward) return launch_rt(route_backward_all_kernel<DT, V>, p, 1, 0, s);  // softmax only
  if (p.bias == nullptr && p.groups == 1) return launch_rt(route_kernel<DT, SOFTMAX, true, V>, p, 1, 0, s);
  const size_t smem = p.groups > 1 ? (size_t)kRtWarps * V * 33 * 4 : 0;
  return launch_rt(route_kernel<DT, SOFTMAX, false, V>, p, 1, smem, s);
}

template <int DT, bool SOFTMAX>
static fp8q_status launch_route_e(const RtParams& p, bool backward, cudaStream_t s) {
  if (backward && (!SOFTMAX || p.renorm)) {
    if (p.top_k <= 8) return launch_rt(route_backward_chosen_kernel<DT, SOFTMAX, 8>, p, 4, 0, s);
    if (p.top_k <= 16) return launch_rt(route_backward_chosen_kernel<DT, SOFTMAX, 16>, p, 2, 0, s);
    return launch_rt(route_backward_chosen_kernel<DT, SOFTMAX, 32>, p, 1, 0, s);
  }
  if (p.experts <= 32) return launch_route_v<DT, SOFTMAX, 1>(p, backward, s);
  if (p.experts <= 64) return launch_route_v<DT, SOFTMAX, 2>(p, backward, s);
  if (p.experts <= 128) return launch_route_v<DT, SOFTMAX, 4>(p, backward, s);
  if (p.experts <= 256) return launch_route_v<DT, SOFTMAX, 8>(p, backward, s);
  if (p.experts <= 512) return launch_route_v<DT, SOFTMAX, 16>(p, backward, s);
  return launch_route_v<DT, SOFTMAX, 32>(p, backward, s);
}

static fp8q_status launch_route(const RtParams& p, int dt, int score, bool backward, cudaStream_t s) {
  if (dt == FP8Q_IN_BF16)
    return score == FP8Q_SCORE_SOFTMAX ? launch_route_e<kBF16, true>(p, backward, s) : launch_route_e<kBF16, false>(p, backward, s);
  return score == FP8Q_SCORE_SOFTMAX ? launch_route_e<kFP32, true>(p, backward, s) : launch_route_e<kFP32, false>(p, backward, s);
}

static fp8q_status check_route(const void* logits, int32_t dt, int64_t tokens, int32_t experts, int32_t top_k, int32_t score) {
  if (dt != FP8Q_IN_BF16 && dt != FP8Q_IN_FP32) return fail(FP8Q_ERR_INVALID_ARG, "dt must be FP8Q_IN_BF16 or FP8Q_IN_FP32");
  if (score != FP8Q_SCORE_SOFTMAX && score != FP8Q_SCORE_SIGMOID)
    return fail(FP8Q_ERR_INVALID_ARG, "score must be FP8Q_SCORE_SOFTMAX or FP8Q_SCORE_SIGMOID");
  if (tokens < 0) return fail(FP8Q_ERR_INVALID_ARG, "tokens must be >= 0");
  if (experts < 1) return fail(FP8Q_ERR_INVALID_ARG, "experts must be >= 1");
  if (experts > kRtMaxExperts) return fail(FP8Q_ERR_UNSUPPORTED, "routing serves at most %d experts", kRtMaxExperts);
  if (top_k < 1 || top_k > experts) return fail(FP8Q_ERR_INVALID_ARG, "top_k must be in [1, experts]");
  if (top_k > 32) return fail(FP8Q_ERR_UNSUPPORTED, "routing serves at most 32 experts a token");
  if (tokens > INT64_MAX / 8 / experts) return fail(FP8Q_ERR_INVALID_ARG, "tokens * experts too large");
  if (tokens > 0 && (!logits || ((uintptr_t)logits & (dt == FP8Q_IN_BF16 ? 1 : 3))))
    return fail(FP8Q_ERR_INVALID_ARG, "logits must be a device pointer aligned to its type");
  return FP8Q_OK;
}

}  // namespace fp8q

using namespace fp8q;

extern "C" fp8q_status fp8q_moe_route(const void* logits, int32_t dt, int64_t tokens, int32_t experts, int32_t top_k,
                                      int32_t score, const float* bias, int32_t num_groups, int32_t top_groups,
                                      int32_t renormalize, float weight_scale, float* weights, int32_t* ids,
                                      void* stream) {
  clear_error();
  const fp8q_status r = check_route(logits, dt, tokens, experts, top_k, score);
  if (r != FP8Q_OK) return r;
  if (num_groups < 1 || num_groups > 32 || experts % num_groups != 0)
    return fail(FP8Q_ERR_INVALID_ARG, "num_groups must be in [1, 32] and divide experts");
  if (top_groups < 1 || top_groups > num_groups) return fail(FP8Q_ERR_INVALID_ARG, "top_groups must be in [1, num_groups]");
  if (top_k > experts / num_groups * top_groups)
    return fail(FP8Q_ERR_INVALID_ARG, "top_k exceeds the experts of top_groups groups");
  if ((uintptr_t)bias & 3) return fail(FP8Q_ERR_INVALID_ARG, "bias must be 4-byte aligned");
  if (tokens == 0) return FP8Q_OK;
  if (!weights || !ids || ((uintptr_t)weights & 3) || ((uintptr_t)ids & 3))
    return fail(FP8Q_ERR_INVALID_ARG, "weights and ids must be 4-byte aligned device pointers");
  RtParams p{};
  p.logits = logits;
  p.tokens = tokens;
  p.experts = experts;
  p.top_k = top_k;
  p.renorm = renormalize ? 1 : 0;
  p.weight_scale = weight_scale;
  p.bias = bias;
  p.groups = num_groups;
  p.top_groups = top_groups;
  p.weights = weights;
  p.ids = ids;
  return launch_route(p, dt, score, false, (cudaStream_t)stream);
}

extern "C" fp8q_status fp8q_moe_route_backward(const void* logits, int32_t dt, int64_t tokens, int32_t experts,
                                               int32_t top_k, int32_t score, int32_t renormalize, float weight_scale,
                                               const int32_t* ids, const float* d_weights, void* d_logits,
                                               void* stream) {
  clear_error();
  const fp8q_status r = check_route(logits, dt, tokens, experts, top_k, score);
  if (r != FP8Q_OK) return r;
  if (tokens == 0) return FP8Q_OK;
  if (!ids || !d_weights || ((uintptr_t)ids & 3) || ((uintptr_t)d_weights & 3))
    return fail(FP8Q_ERR_INVALID_ARG, "ids and d_weights must be 4-byte aligned device pointers");
  if (!d_logits || ((uintptr_t)d_logits & (dt == FP8Q_IN_BF16 ? 1 : 3)))
    return fail(FP8Q_ERR_INVALID_ARG, "d_logits must be a device pointer aligned to its type");
  RtParams p{};
  p.logits = logits;
  p.tokens = tokens;
  p.experts = experts;
  p.top_k = top_k;
  p.renorm = renormalize ? 1 : 0;
  p.weight_scale = weight_scale;
  p.ids_in = ids;
  p.d_weights = d_weights;
  p.d_logits = d_logits;
  p.groups = 1;
  return launch_route(p, dt, score, true, (cudaStream_t)stream);
}
