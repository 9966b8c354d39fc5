// decode.cu -- the expert layer for a few tokens, both products in two kernels.
//
//   out[t] = sum_j w[t, j] * W2[e] a,   a = silu(G) * U,  [G; U] = W1[e] x_t,  e = ids[t, j]
//
// The weights are FP8 codes with one scale for each 128 x 128 block; the tokens
// and the inner values are not quantized.  With few tokens the weights of the
// experts that some token chose are nearly all that moves, and each is read
// once.  A warp takes 32 weight rows against 8 tokens by mma.m16n8k16 in FP16
// with FP32 sums: a code is an FP16 value as it is, and a BF16 token row
// becomes FP16 exactly after a power of two for each 128 of it (values 2^-32
// below their group's largest lose digits).  The inner values are split into
// two FP16 parts, 22 bits, with a power of two for each 16 of them.
//
// K is taken in an order that suits the loads: of a block of 128 values the
// lanes q = 0..3 of a row take 16 q .. 16 q + 15 and 64 beyond, and step s of
// eight multiplies the four-byte words s & 3 of both, so that 16 K values of a
// step are {64 (s >> 2) + 16 q + 4 (s & 3) + j}.  The first product's units are
// those 16 inner values, which is how the second finds them with one scale.
//
// First kernel: a unit is 16 inner values of one expert (16 rows of G and of U)
// for up to 8 of its tokens; the 8 warps of a CTA share K.  Second kernel: a CTA
// takes 32 output columns of all tokens and sums over the experts, so that every
// sum has a fixed order; the warps share the experts' blocks of K.
#include "fp8q_device.cuh"
#include "internal.h"

namespace fp8q {

constexpr int kMdThreads = 256;
constexpr int kMdWarps = kMdThreads / 32;
constexpr int kMdTokens = 64;
constexpr int kMdTopK = 32;
constexpr int kMdExperts = 1024;
constexpr int kMdPairs = kMdTokens * kMdTopK;
constexpr int kMdCols = 8;                                   // tokens of one job
constexpr int kMdJobs = kMdExperts + kMdPairs / kMdCols;
constexpr int kMdPitch = 20;                                 // floats of a column of partial sums (16 rows)
constexpr int kMdRows = 32;                                  // output columns of a CTA of the second kernel
constexpr int kMdOutPitch = 36;

struct MdParams {
  const uint16_t* x;  // [tokens][hidden] BF16
  const int* ids;     // [tokens][top_k]
  const float* weights;
  const uint8_t* w1;  // [experts][2 inner][hidden]
  const float* s1;    // [experts][nb1][kb1]
  const uint8_t* w2;  // [experts][hidden][inner]
  const float* s2;    // [experts][nb2][kb2]
  int tokens, top_k, experts, hidden, inner;
  int kb1, kb2, nb1, nb2;
  uint16_t* a_hi;  // [pairs][128 kb2] FP16
  uint16_t* a_lo;
  float* a_s;      // [pairs][kb2][8]
  int out_dt;
  void* out;
};

// The (token, expert) pairs in order of expert, and jobs of up to 8 of one expert's.
struct MdLists {
  uint32_t mask[2 * kMdExperts];  // tokens of each expert
  uint32_t job[kMdJobs];          // expert | tokens << 16
  uint16_t first[kMdJobs];        // first pair
  uint8_t token[kMdPairs];
  int warp_sum[kMdWarps];
  int jobs, pairs;
};

__device__ __forceinline__ void md_lists(const MdParams& p, MdLists& l) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < 2 * p.experts; i += kMdThreads) l.mask[i] = 0;
  __syncthreads();
  for (int i = tid; i < p.tokens * p.top_k; i += kMdThreads) {
    const int e = __ldg(p.ids + i), t = i / p.top_k;
    if (e >= 0 && e < p.experts) atomicOr(&l.mask[2 * e + (t >> 5)], 1u << (t & 31));
  }
  __syncthreads();
  const int per = (p.experts + kMdThreads - 1) / kMdThreads, e0 = tid * per, e1 = min(e0 + per, p.experts);
  int mine = 0;  // jobs << 16 | pairs
  for (int e = e0; e < e1; e++) {
    const int n = __popc(l.mask[2 * e]) + __popc(l.mask[2 * e + 1]);
    mine += ((n + kMdCols - 1) / kMdCols << 16) + n;
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) l.warp_sum[warp] = incl;
  __syncthreads();
  int at = incl - mine, all = 0;
#pragma unroll
  for (int w = 0; w < kMdWarps; w++) {
    if (w < warp) at += l.warp_sum[w];
    all += l.warp_sum[w];
  }
  for (int e = e0; e < e1; e++) {
    uint64_t m = (uint64_t)l.mask[2 * e + 1] << 32 | l.mask[2 * e];
    int n = __popcll(m), pair = at & 0xFFFF, job = at >> 16;
    at += ((n + kMdCols - 1) / kMdCols << 16) + n;
    for (int i = pair; m; m &= m - 1, i++) l.token[i] = (uint8_t)(__ffsll((long long)m) - 1);
    for (; n > 0; n -= kMdCols, pair += kMdCols, job++) {
      l.job[job] = (uint32_t)e | (uint32_t)min(n, kMdCols) << 16;
      l.first[job] = (uint16_t)pair;
    }
  }
  if (tid == 0) l.jobs = all >> 16, l.pairs = all & 0xFFFF;
  __syncthreads();
}

// Two codes -> two FP16 values, exactly.
template <int FMT>
__device__ __forceinline__ void md_codes(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == kE4M3)
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
  else
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e5m2x2 %0, a;\n\tcvt.rn.f16x2.e5m2x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
}

__device__ __forceinline__ void md_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t md_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The power of two that brings magnitudes up to `bits` (FP32) below 2^15, as
// its exponent field; 254 minus it is its reciprocal's.
__device__ __forceinline__ uint32_t md_exponent(uint32_t bits) { return min(268u - (bits >> 23), 253u); }

// 128 bytes of K of 32 weight rows: this lane's 32 bytes of rows g and g + 8 of two sets of 16.
struct MdTile {
  uint4 v[2][2][2];  // [set][row g, g + 8][K 16 q, 64 + 16 q]
};

__device__ __forceinline__ uint32_t md_word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// ---------------------------------------------------------------------------
// first product and the activation
// ---------------------------------------------------------------------------
// Rows of unit `unit`'s sets (0: gate, 1: up) and where they lie.
struct MdUnit {
  int expert, count, first, inner0;  // inner value of row 0; row m is inner0 + 16 (m >> 2) + (m & 3)
};

__device__ __forceinline__ MdUnit md_unit(const MdParams& p, const MdLists& l, int unit) {
  const int per = p.kb2 * 8, job = unit / per, at = unit - job * per, s = at & 7;
  MdUnit u;
  u.expert = l.job[job] & 0xFFFF;
  u.count = l.job[job] >> 16;
  u.first = l.first[job];
  u.inner0 = (at >> 3) * 128 + 64 * (s >> 2) + 4 * (s & 3);
  return u;
}

__device__ __forceinline__ void md_load1(const MdParams& p, const MdUnit& u, int kb, MdTile& t, float (&sc)[2][2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3, k = kb * 128 + 16 * q;
#pragma unroll
  for (int set = 0; set < 2; set++)
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const int m = g + 8 * h, i = u.inner0 + 16 * (m >> 2) + (m & 3), row = set * p.inner + i;
      const bool ok = i < p.inner && kb < p.kb1;
      const uint8_t* at = p.w1 + ((int64_t)u.expert * 2 * p.inner + row) * p.hidden + k;
      t.v[set][h][0] = ok && k < p.hidden ? ld_stream(at) : make_uint4(0, 0, 0, 0);
      t.v[set][h][1] = ok && k + 64 < p.hidden ? ld_stream(at + 64) : make_uint4(0, 0, 0, 0);
      sc[set][h] = ok ? __ldg(p.s1 + ((int64_t)u.expert * p.nb1 + (row >> 7)) * p.kb1 + kb) : 0.0f;
    }
}

template <int FMT>
__global__ void __launch_bounds__(kMdThreads, 2) decode_first_kernel(MdParams p) {
  __shared__ MdLists l;
  __shared__ float part[kMdWarps][2][kMdCols * kMdPitch];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  pdl_wait();
  md_lists(p, l);
  const int units = l.jobs * p.kb2 * 8;
  int unit = blockIdx.x, kb = warp;
  if (unit < units) {
    MdUnit u = md_unit(p, l, unit);
    MdTile next;
    float next_sc[2][2];
    md_load1(p, u, kb, next, next_sc);
    for (; unit < units; unit += gridDim.x) {
      float acc[2][4] = {};
      const int token = g < u.count ? l.token[u.first + g] : -1;
      for (kb = warp; kb - warp < p.kb1; kb += kMdWarps) {
        const MdTile tile = next;
        const float sc[2][2] = {{next_sc[0][0], next_sc[0][1]}, {next_sc[1][0], next_sc[1][1]}};
        // the tokens' part of this block of K
        const int k = kb * 128 + 16 * q;
        uint4 x[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int at = k + 64 * (i >> 1) + 8 * (i & 1);
          x[i] = token >= 0 && at < p.hidden ? __ldg((const uint4*)(p.x + (int64_t)token * p.hidden + at)) : make_uint4(0, 0, 0, 0);
        }
        // the next block, of this unit or the next one
        if (kb - warp + kMdWarps < p.kb1) {
          md_load1(p, u, kb + kMdWarps, next, next_sc);
        } else if (unit + gridDim.x < units) {
          md_load1(p, md_unit(p, l, unit + gridDim.x), warp, next, next_sc);
        }
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; i++) m = absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(m, x[i].x), x[i].y), x[i].z), x[i].w);
        m = max_u16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = max_u16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        const uint32_t f = md_exponent(max(m << 16, m & 0xFFFF0000u));
        const float up = __uint_as_float(f << 23);
        const uint32_t inv = (254u - f) << 23;
        const float inv0 = __uint_as_float(__shfl_sync(0xFFFFFFFFu, inv, 8 * q)), inv1 = __uint_as_float(__shfl_sync(0xFFFFFFFFu, inv, 8 * q + 4));
        float d[2][4] = {};
#pragma unroll
        for (int s = 0; s < 8; s++) {
          const uint4& xv = x[s >> 1];
          const uint32_t x0 = s & 1 ? xv.z : xv.x, x1 = s & 1 ? xv.w : xv.y;
          const uint32_t b0 = md_half2(__fmul_rn(bf16_lo(x0), up), __fmul_rn(bf16_hi(x0), up));
          const uint32_t b1 = md_half2(__fmul_rn(bf16_lo(x1), up), __fmul_rn(bf16_hi(x1), up));
#pragma unroll
          for (int set = 0; set < 2; set++) {
            uint32_t a0, a1, a2, a3;
            md_codes<FMT>(md_word(tile.v[set][0][s >> 2], s & 3), a0, a2);
            md_codes<FMT>(md_word(tile.v[set][1][s >> 2], s & 3), a1, a3);
            md_mma(d[set], a0, a1, a2, a3, b0, b1);
          }
        }
#pragma unroll
        for (int set = 0; set < 2; set++)
#pragma unroll
          for (int c = 0; c < 4; c++)
            acc[set][c] = __fmaf_rn(__fmul_rn(sc[set][c >> 1], c & 1 ? inv1 : inv0), d[set][c], acc[set][c]);
      }
      __syncthreads();  // the last unit's sums have been read
#pragma unroll
      for (int set = 0; set < 2; set++)
#pragma unroll
        for (int c = 0; c < 4; c++) part[warp][set][(2 * q + (c & 1)) * kMdPitch + g + 8 * (c >> 1)] = acc[set][c];
      __syncthreads();
      if (tid < kMdCols * 16) {  // inner value tid & 15 of token tid / 16
        const int m = tid & 15, n = tid >> 4;
        float gate = 0.0f, up = 0.0f;
#pragma unroll
        for (int w = 0; w < kMdWarps; w++) {
          gate += part[w][0][n * kMdPitch + m];
          up += part[w][1][n * kMdPitch + m];
        }
        const float e = expf(-fabsf(gate)), r = __frcp_rn(1.0f + e);
        const float a = __fmul_rn(__fmul_rn(gate, gate >= 0.0f ? r : __fmul_rn(e, r)), up);
        uint32_t big = __float_as_uint(a) & 0x7FFFFFFFu;
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, o));
        const uint32_t f = md_exponent(big);
        const float v = __fmul_rn(a, __uint_as_float(f << 23));
        const uint32_t hi = md_half2(v, 0.0f) & 0xFFFFu;
        float back;
        asm("{\n\t.reg .b16 h, z;\n\tmov.b32 {h, z}, %1;\n\tcvt.f32.f16 %0, h;\n\t}" : "=f"(back) : "r"(hi));
        const uint32_t lo = md_half2((hi & 0x7C00u) == 0x7C00u ? 0.0f : v - back, 0.0f) & 0xFFFFu;
        if (n < u.count) {
          const int64_t pair = u.first + n, at = pair * p.kb2 * 128 + u.inner0 + 16 * (m >> 2) + (m & 3);
          p.a_hi[at] = (uint16_t)hi;
          p.a_lo[at] = (uint16_t)lo;
          if (m == 0) p.a_s[(pair * p.kb2 + (u.inner0 >> 7)) * 8 + ((u.inner0 >> 4) & 4) + ((u.inner0 >> 2) & 3)] = __uint_as_float((254u - f) << 23);
        }
      }
      if (unit + gridDim.x < units) u = md_unit(p, l, unit + gridDim.x);
    }
  }
  pdl_launch_dependents();
}

// ---------------------------------------------------------------------------
// second product and the weighted sum
// ---------------------------------------------------------------------------
__device__ __forceinline__ void md_load2(const MdParams& p, const MdLists& l, int at, int row0, MdTile& t, float& sc) {
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3, job = at / p.kb2, kb = at - job * p.kb2;
  const int e = l.job[job] & 0xFFFF, k = kb * 128 + 16 * q;
#pragma unroll
  for (int set = 0; set < 2; set++)
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const int row = row0 + 16 * set + g + 8 * h;
      const uint8_t* from = p.w2 + ((int64_t)e * p.hidden + row) * p.inner + k;
      const bool ok = row < p.hidden;
      t.v[set][h][0] = ok && k < p.inner ? ld_stream(from) : make_uint4(0, 0, 0, 0);
      t.v[set][h][1] = ok && k + 64 < p.inner ? ld_stream(from + 64) : make_uint4(0, 0, 0, 0);
    }
  sc = __ldg(p.s2 + ((int64_t)e * p.nb2 + (row0 >> 7)) * p.kb2 + kb);
}

template <int FMT>
__global__ void __launch_bounds__(kMdThreads, 2) decode_second_kernel(MdParams p) {
  extern __shared__ float sums[];  // [warps][tokens][kMdOutPitch]
  __shared__ MdLists l;
  __shared__ float weight[kMdPairs];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const int row0 = blockIdx.x * kMdRows;
  // The first kernel has waited for all before it and writes none of what is read here: only its inner values are waited for below.
  md_lists(p, l);
  for (int i = tid; i < l.pairs; i += kMdThreads) {  // a pair's weight: an expert that a token names twice counts twice
    const int t = l.token[i];
    int j = 0;  // the pair's expert: the last whose first pair is not behind it
    for (int lo = 0, hi = l.jobs; hi - lo > 1;) {
      const int mid = (lo + hi) >> 1;
      if (l.first[mid] <= i) lo = mid; else hi = mid;
      j = lo;
    }
    const int e = l.job[j] & 0xFFFF;
    float w = 0.0f;
    for (int k = 0; k < p.top_k; k++)
      if (__ldg(p.ids + t * p.top_k + k) == e) w += __ldg(p.weights + t * p.top_k + k);
    weight[i] = w;
  }
  for (int i = tid; i < kMdWarps * p.tokens * kMdOutPitch; i += kMdThreads) sums[i] = 0.0f;
  float* mine = sums + warp * p.tokens * kMdOutPitch;
  const int all = l.jobs * p.kb2;
  const int lo = (int)((int64_t)all * warp / kMdWarps), hi = (int)((int64_t)all * (warp + 1) / kMdWarps);
  MdTile next;
  float next_sc = 0.0f;
  if (lo < hi) md_load2(p, l, lo, row0, next, next_sc);
  __syncthreads();
  pdl_wait();
  float acc[2][4] = {};
  for (int at = lo; at < hi; at++) {
    const int job = at / p.kb2, kb = at - job * p.kb2, count = l.job[job] >> 16, first = l.first[job];
    const MdTile tile = next;
    const float sc = next_sc;
    if (at + 1 < hi) md_load2(p, l, at + 1, row0, next, next_sc);
    const int64_t from = (int64_t)(first + g) * p.kb2 * 128 + kb * 128 + 16 * q;
#pragma unroll
    for (int half = 0; half < 2; half++) {
      uint4 bh[2], bl[2];
      float4 s0 = make_float4(0, 0, 0, 0), s1 = s0;
#pragma unroll
      for (int i = 0; i < 2; i++) {
        bh[i] = g < count ? *(const uint4*)(p.a_hi + from + 64 * half + 8 * i) : make_uint4(0, 0, 0, 0);
        bl[i] = g < count ? *(const uint4*)(p.a_lo + from + 64 * half + 8 * i) : make_uint4(0, 0, 0, 0);
      }
      if (2 * q < count) s0 = *(const float4*)(p.a_s + ((int64_t)(first + 2 * q) * p.kb2 + kb) * 8 + 4 * half);
      if (2 * q + 1 < count) s1 = *(const float4*)(p.a_s + ((int64_t)(first + 2 * q + 1) * p.kb2 + kb) * 8 + 4 * half);
#pragma unroll
      for (int s = 0; s < 4; s++) {
        const uint4 &h4 = bh[s >> 1], &l4 = bl[s >> 1];
        const uint32_t h0 = s & 1 ? h4.z : h4.x, h1 = s & 1 ? h4.w : h4.y, l0 = s & 1 ? l4.z : l4.x, l1 = s & 1 ? l4.w : l4.y;
        const float f0 = __fmul_rn(sc, s == 0 ? s0.x : s == 1 ? s0.y : s == 2 ? s0.z : s0.w);
        const float f1 = __fmul_rn(sc, s == 0 ? s1.x : s == 1 ? s1.y : s == 2 ? s1.z : s1.w);
#pragma unroll
        for (int set = 0; set < 2; set++) {
          uint32_t a0, a1, a2, a3;
          float d[4] = {};
          md_codes<FMT>(md_word(tile.v[set][0][half], s), a0, a2);
          md_codes<FMT>(md_word(tile.v[set][1][half], s), a1, a3);
          md_mma(d, a0, a1, a2, a3, l0, l1);
          md_mma(d, a0, a1, a2, a3, h0, h1);
#pragma unroll
          for (int c = 0; c < 4; c++) acc[set][c] = __fmaf_rn(c & 1 ? f1 : f0, d[c], acc[set][c]);
        }
      }
    }
    if (kb == p.kb2 - 1 || at + 1 == hi) {  // on to another job: its tokens' sums leave the registers
#pragma unroll
      for (int n = 0; n < 2; n++) {
        if (2 * q + n < count) {
          const float w = weight[first + 2 * q + n];
          float* to = mine + l.token[first + 2 * q + n] * kMdOutPitch + g;
#pragma unroll
          for (int set = 0; set < 2; set++)
#pragma unroll
            for (int h = 0; h < 2; h++) to[16 * set + 8 * h] = __fmaf_rn(w, acc[set][2 * h + n], to[16 * set + 8 * h]);
        }
      }
      __syncwarp();
#pragma unroll
      for (int set = 0; set < 2; set++)
#pragma unroll
        for (int c = 0; c < 4; c++) acc[set][c] = 0.0f;
    }
  }
  __syncthreads();
  for (int i = tid; i < p.tokens * kMdRows; i += kMdThreads) {
    const int t = i / kMdRows, r = i % kMdRows;
    if (row0 + r >= p.hidden) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kMdWarps; w++) v += sums[(w * p.tokens + t) * kMdOutPitch + r];
    const int64_t at = (int64_t)t * p.hidden + row0 + r;
    if (p.out_dt == FP8Q_OUT_BF16) {
      uint16_t h;
      asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(v));
      ((uint16_t*)p.out)[at] = h;
    } else {
      ((float*)p.out)[at] = v;
    }
  }
  pdl_launch_dependents();
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
static bool off(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

static size_t decode_workspace(int64_t pairs, int64_t inner) {
  const int64_t kb2 = (inner + 127) / 128;
  return (size_t)(pairs * kb2 * (2 * 2 * 128 + 8 * 4));
}

template <int FMT>
static fp8q_status launch_decode(const MdParams& p, cudaStream_t s) {
  const int pairs = p.tokens * p.top_k;
  int64_t units = (int64_t)(pairs < p.experts ? pairs : p.experts + pairs / kMdCols) * p.kb2 * 8;
  const int64_t fit = 2 * (int64_t)sm_count();
  if (units > fit) units = fit;
  cudaError_t e = launch_kernel(decode_first_kernel<FMT>, dim3((unsigned)units), dim3(kMdThreads), 0, s, p);
  if (e != cudaSuccess) return cuda_fail(e, "decode first kernel launch");
  static PerDevice<bool> allowed;
  e = allow_smem(allowed, decode_second_kernel<FMT>, (size_t)kMdWarps * kMdTokens * kMdOutPitch * sizeof(float));
  if (e != cudaSuccess) return cuda_fail(e, "decode shared memory");
  e = launch_kernel(decode_second_kernel<FMT>, dim3((unsigned)((p.hidden + kMdRows - 1) / kMdRows)), dim3(kMdThreads),
                    (size_t)kMdWarps * p.tokens * kMdOutPitch * sizeof(float), s, p);
  if (e != cudaSuccess) return cuda_fail(e, "decode second kernel launch");
  return check_launch("decode kernel");
}

}  // namespace fp8q

using namespace fp8q;

extern "C" size_t fp8q_moe_decode_workspace_bytes(int64_t tokens, int32_t top_k, int64_t inner) {
  if (tokens < 0 || tokens > kMdTokens || top_k < 1 || top_k > kMdTopK || inner < 0 || inner > INT32_MAX / 4) return 0;
  return decode_workspace(tokens * top_k, inner);
}

extern "C" fp8q_status fp8q_moe_decode(const void* x, int64_t tokens, int64_t hidden, int64_t inner, int32_t experts,
                                       int32_t top_k, const int32_t* ids, const float* weights, const uint8_t* w1,
                                       const float* w1_scale_inv, const uint8_t* w2, const float* w2_scale_inv,
                                       int32_t w_fmt, int32_t out_dt, void* out, void* workspace, size_t workspace_bytes,
                                       void* stream) {
  clear_error();
  if (tokens < 0 || hidden < 1 || inner < 1) return fail(FP8Q_ERR_INVALID_ARG, "tokens must be >= 0, hidden and inner >= 1");
  if (tokens > kMdTokens) return fail(FP8Q_ERR_UNSUPPORTED, "at most %d tokens: the grouped products take more", kMdTokens);
  if (experts < 1) return fail(FP8Q_ERR_INVALID_ARG, "experts must be >= 1");
  if (experts > kMdExperts) return fail(FP8Q_ERR_UNSUPPORTED, "at most %d experts", kMdExperts);
  if (top_k < 1 || top_k > kMdTopK) return fail(FP8Q_ERR_UNSUPPORTED, "top_k must be in [1, %d]", kMdTopK);
  if (hidden % 16 != 0 || inner % 16 != 0) return fail(FP8Q_ERR_UNSUPPORTED, "hidden and inner must be multiples of 16");
  if (hidden > (1 << 20) || inner > (1 << 20)) return fail(FP8Q_ERR_UNSUPPORTED, "hidden or inner too large");
  if (w_fmt != FP8Q_E4M3 && w_fmt != FP8Q_E5M2) return fail(FP8Q_ERR_INVALID_ARG, "w_fmt must be FP8Q_E4M3 or FP8Q_E5M2");
  if (out_dt != FP8Q_OUT_BF16 && out_dt != FP8Q_OUT_FP32) return fail(FP8Q_ERR_INVALID_ARG, "out_dt must be FP8Q_OUT_BF16 or FP8Q_OUT_FP32");
  if (tokens == 0) return FP8Q_OK;
  if (!x || off(x, 16)) return fail(FP8Q_ERR_INVALID_ARG, "x must be a 16-byte aligned device pointer");
  if (!ids || off(ids, 4) || !weights || off(weights, 4)) return fail(FP8Q_ERR_INVALID_ARG, "ids and weights must be 4-byte aligned device pointers");
  if (!w1 || off(w1, 16) || !w2 || off(w2, 16)) return fail(FP8Q_ERR_INVALID_ARG, "w1 and w2 must be 16-byte aligned device pointers");
  if (!w1_scale_inv || off(w1_scale_inv, 4) || !w2_scale_inv || off(w2_scale_inv, 4))
    return fail(FP8Q_ERR_INVALID_ARG, "the scales must be 4-byte aligned device pointers");
  if (!out || off(out, out_dt == FP8Q_OUT_BF16 ? 2 : 4)) return fail(FP8Q_ERR_INVALID_ARG, "out must be a device pointer aligned to its type");
  const int64_t pairs = tokens * top_k;
  if (!workspace || off(workspace, 16) || workspace_bytes < decode_workspace(pairs, inner))
    return fail(FP8Q_ERR_INVALID_ARG, "workspace must be 16-byte aligned and of fp8q_moe_decode_workspace_bytes()");
  MdParams p{};
  p.x = (const uint16_t*)x;
  p.ids = ids;
  p.weights = weights;
  p.w1 = w1;
  p.s1 = w1_scale_inv;
  p.w2 = w2;
  p.s2 = w2_scale_inv;
  p.tokens = (int)tokens;
  p.top_k = top_k;
  p.experts = experts;
  p.hidden = (int)hidden;
  p.inner = (int)inner;
  p.kb1 = (int)((hidden + 127) / 128);
  p.kb2 = (int)((inner + 127) / 128);
  p.nb1 = (int)((2 * inner + 127) / 128);
  p.nb2 = (int)((hidden + 127) / 128);
  p.a_hi = (uint16_t*)workspace;
  p.a_lo = p.a_hi + pairs * p.kb2 * 128;
  p.a_s = (float*)(p.a_lo + pairs * p.kb2 * 128);
  p.out_dt = out_dt;
  p.out = out;
  return w_fmt == FP8Q_E4M3 ? launch_decode<kE4M3>(p, (cudaStream_t)stream) : launch_decode<kE5M2>(p, (cudaStream_t)stream);
}
