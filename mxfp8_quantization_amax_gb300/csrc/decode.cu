// decode.cu -- the expert layer for a few tokens, both products in two kernels.
//
//   out[t] = sum_j w[t, j] * W2[e] a,   a = silu(G) * U,  [G; U] = W1[e] x_t,  e = ids[t, j]
//
// The weights are FP8 codes with one scale for each 128 x 128 block; the tokens
// and the inner values are not quantized.  With few tokens the weights of the
// experts that some token chose are nearly all that moves, and each is read
// once.  A warp takes 32 weight rows and 128 of K against 8 tokens by
// mma.m16n8k16 in FP16 with FP32 sums: a code is an FP16 value as it is, and a
// BF16 token row becomes FP16 exactly after a power of two for each 128 of it
// (values 2^-32 below their group's largest lose digits).  The inner values
// are FP16 with a power of two for each 32 of them; for FP32 output a
// second FP16 number holds what the first one's rounding (2^-11) left.  BF16
// output, which rounds by 2^-8 at the end, does without: the second number's
// products and loads are 12 to 16% of the layer (16 tokens 431 us against 382).
//
// First kernel: a unit is 32 inner values of one expert (rows of G and of U)
// for up to 8 of its tokens; 8 or 4 warps of a CTA share K.  Second kernel: a
// CTA takes 32 output columns of all tokens and a share of the experts' blocks
// of K, and its warps share those; the CTAs of a cluster have the same columns
// and add up through distributed shared memory.  Every sum has a fixed order.
//
// Bound by the weights' bytes.  64 experts of 7168 x 2048, 8 a token, BF16 (FP32)
// output: 1 token 61 us (69; 352 MB, 5.8 TB/s; some 7 us are the two kernels'
// start, lists and end), 4 tokens 185 (210), 16 tokens 382 (431; 6.6 TB/s).
// Beyond 8 tokens an expert its weights are read again, from L2, and converted
// again: 64 tokens 557 (646; floor 421).  Sizes whose K leaves warps idle cost
// more: 61 tokens, 40 experts of 2064 x 1360 98 (110; floor 50).  Jobs of 16
// tokens were slower everywhere (64 tokens 767 then against 677): their
// registers leave one CTA an SM.
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
constexpr int kMdUnit = 32;                                  // inner values of one unit
constexpr int kMdPitch = 20;                                 // floats of a column of partial sums (16 rows)
constexpr int kMdSetFloats = kMdCols * kMdPitch + 16;        // of a set of 16 rows
constexpr int kMdRows = 32;                                  // output columns of a CTA of the second kernel
constexpr int kMdOutPitch = 36;
constexpr size_t kMdHalfSm = 112 * 1024;                     // shared memory of a CTA of which two fit an SM

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
  uint16_t* a_lo;  // or NULL
  float* a_s;      // [pairs][kb2][4]
  void* out;
};

// The (token, expert) pairs in order of expert, and jobs of up to 8 of one
// expert's.  Where the lists lie in shared memory, for `slots` slots:
struct MdLists {
  uint32_t* job;     // expert | tokens << 16 | place among the expert's jobs << 20 | their number << 24
  uint16_t* first;   // first pair of a job
  uint8_t* token;    // of a pair
  float* weight;     // of a pair (an expert that a token names twice counts twice); second kernel only
  int jobs, pairs;
};

__host__ __device__ constexpr size_t md_list_bytes(int slots) { return (size_t)slots * (4 + 4 + 2 + 1) + 16; }

__device__ __forceinline__ MdLists md_list_places(uint8_t* at, int slots) {
  MdLists l;
  l.job = (uint32_t*)at;
  l.weight = (float*)(at + 4 * slots);
  l.first = (uint16_t*)(at + 8 * slots);
  l.token = at + 10 * slots;
  return l;
}

// `scratch`: 4 * 2 * experts + 10 * slots bytes that are free again afterwards.
template <bool WEIGHTS>
__device__ __forceinline__ void md_lists(const MdParams& p, MdLists& l, uint8_t* scratch, int* warp_sum) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, slots = p.tokens * p.top_k;
  uint32_t* mask = (uint32_t*)scratch;  // tokens of each expert
  int* ids = (int*)(mask + 2 * p.experts);
  float* weights = (float*)(ids + slots);
  uint16_t* expert = (uint16_t*)(weights + slots);  // of a pair
  for (int i = tid; i < 2 * p.experts; i += kMdThreads) mask[i] = 0;
  for (int i = tid; i < slots; i += kMdThreads) {
    ids[i] = __ldg(p.ids + i);
    if (WEIGHTS) weights[i] = __ldg(p.weights + i);
  }
  __syncthreads();
  for (int i = tid; i < slots; i += kMdThreads) {
    const int e = ids[i], t = i / p.top_k;
    if (e >= 0 && e < p.experts) atomicOr(&mask[2 * e + (t >> 5)], 1u << (t & 31));
  }
  __syncthreads();
  const int per = (p.experts + kMdThreads - 1) / kMdThreads, e0 = tid * per, e1 = min(e0 + per, p.experts);
  int mine = 0;  // jobs << 16 | pairs
  for (int e = e0; e < e1; e++) {
    const int n = __popc(mask[2 * e]) + __popc(mask[2 * e + 1]);
    mine += ((n + kMdCols - 1) / kMdCols << 16) + n;
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int at = incl - mine, all = 0;
#pragma unroll
  for (int w = 0; w < kMdWarps; w++) {
    if (w < warp) at += warp_sum[w];
    all += warp_sum[w];
  }
  l.jobs = all >> 16;
  l.pairs = all & 0xFFFF;
  for (int e = e0; e < e1; e++) {
    uint64_t m = (uint64_t)mask[2 * e + 1] << 32 | mask[2 * e];
    int n = __popcll(m), pair = at & 0xFFFF, job = at >> 16;
    at += ((n + kMdCols - 1) / kMdCols << 16) + n;
    for (int i = pair; m; m &= m - 1, i++) {
      l.token[i] = (uint8_t)(__ffsll((long long)m) - 1);
      if (WEIGHTS) expert[i] = (uint16_t)e;
    }
    const uint32_t jobs = (n + kMdCols - 1) / kMdCols;
    for (uint32_t place = 0; n > 0; n -= kMdCols, pair += kMdCols, job++, place++) {
      l.job[job] = (uint32_t)e | (uint32_t)min(n, kMdCols) << 16 | place << 20 | jobs << 24;
      l.first[job] = (uint16_t)pair;
    }
  }
  __syncthreads();
  if (WEIGHTS) {
    for (int i = tid; i < l.pairs; i += kMdThreads) {
      const int e = expert[i], from = l.token[i] * p.top_k;
      float w = 0.0f;
      for (int k = 0; k < p.top_k; k++) w += ids[from + k] == e ? weights[from + k] : 0.0f;
      l.weight[i] = w;
    }
    __syncthreads();  // the scratch is free
  }
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

// The halves of a BF16 pair times a BF16 power of two: the products are exact.
__device__ __forceinline__ uint32_t md_scaled(uint32_t w, uint32_t power) {
  float lo, hi;
  asm("{\n\t.reg .b16 a, b, c;\n\tmov.b32 {a, b}, %2;\n\tcvt.u16.u32 c, %3;\n\t"
      "fma.rn.f32.bf16 %0, a, c, %4;\n\tfma.rn.f32.bf16 %1, b, c, %4;\n\t}"
      : "=f"(lo), "=f"(hi) : "r"(w), "r"(power), "f"(-0.0f));
  return md_half2(lo, hi);
}

// The power of two that brings magnitudes up to `bits` (FP32) below 2^15, as
// its exponent field; 254 minus it is its reciprocal's.
__device__ __forceinline__ uint32_t md_exponent(uint32_t bits) { return min(268u - (bits >> 23), 253u); }

// A tile: 32 rows of 128 bytes of weights, whose 16-byte chunks are permuted by
// the row so that the eight rows of a matrix load lie in different banks.  A
// warp's tiles come by cp.async into a ring of its own; a place is asked for
// again as soon as its tile has been read.  Step s of a tile multiplies chunk s
// of all rows: lane q of a row has K values 16 s + 4 q .. 4 q + 3.
constexpr int kMdStages = 2;
constexpr int kMdTileBytes = 32 * 128;
constexpr int kMdRingBytes = kMdStages * kMdTileBytes;  // of one warp

__device__ __forceinline__ void md_copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
// 16 bytes, or zeros: nothing is asked for where nothing is there.
__device__ __forceinline__ void md_copy16(uint32_t to, const void* from, bool there) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "@p cp.async.cg.shared.global [%0], [%1], 16;\n\t"
      "@!p st.shared.v4.u32 [%0], {%3, %3, %3, %3};\n\t}" ::"r"(to),
      "l"(from), "r"((uint32_t)there), "r"(0)
      : "memory");
}
__device__ __forceinline__ void md_copy4(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void md_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void md_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t md_smem(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// Asks for rows 0 .. 31 of a tile: 16 rows from `lo` on and 16 from `hi` on, of
// which n_lo and n_hi are there, and `k` bytes of each (all of 128: most tiles).
__device__ __forceinline__ void md_tile(uint32_t to, const uint8_t* lo, const uint8_t* hi, int64_t pitch, int n_lo, int n_hi, int k) {
  const int lane = threadIdx.x & 31, r = lane >> 3, c = lane & 7;
  const uint32_t even = to + r * 128 + ((c ^ r) << 4), odd = to + r * 128 + ((c ^ (r + 4)) << 4);
  lo += r * pitch + 16 * c;
  hi += r * pitch + 16 * c;
  if (n_lo >= 16 && n_hi >= 16 && k >= 128) {
#pragma unroll
    for (int i = 0; i < 8; i++) md_copy16((i & 1 ? odd : even) + i * 512, (i < 4 ? lo : hi) + (i & 3) * 4 * pitch);
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const bool there = (i & 3) * 4 + r < (i < 4 ? n_lo : n_hi) && 16 * c < k;
      md_copy16((i & 1 ? odd : even) + i * 512, (i < 4 ? lo : hi) + (i & 3) * 4 * pitch, there);
    }
  }
}

// Chunk s of the tile: this lane's four codes of rows g, g + 8, g + 16, g + 24.
// `at`: the tile's start + 128 * lane + 16 * (lane & 7).
__device__ __forceinline__ void md_chunk(uint32_t at, int s, uint32_t (&w)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(at ^ (s << 4))
               : "memory");
}

// ---------------------------------------------------------------------------
// first product and the activation
// ---------------------------------------------------------------------------
// This lane's BF16 values of a block of K of one token: 4 of each 16.
__device__ __forceinline__ void md_token(const uint16_t* x, int left, bool there, uint32_t (&v)[16]) {
  if (there && left >= 128) {
#pragma unroll
    for (int s = 0; s < 8; s++) {
      const uint2 u = __ldg((const uint2*)(x + 16 * s));
      v[2 * s] = u.x, v[2 * s + 1] = u.y;
    }
  } else {
#pragma unroll
    for (int s = 0; s < 8; s++) {
      const uint2 u = there && 16 * s < left ? __ldg((const uint2*)(x + 16 * s)) : make_uint2(0, 0);
      v[2 * s] = u.x, v[2 * s + 1] = u.y;
    }
  }
}

// 32 inner values of an expert from inner0 on, for `count` of its tokens.
struct MdUnit {
  int expert, count, first, inner0;
};

__device__ __forceinline__ MdUnit md_unit(const MdParams& p, const MdLists& l, int unit) {
  const int per = p.kb2 * (128 / kMdUnit), job = unit / per;
  MdUnit u;
  u.expert = l.job[job] & 0xFFFF;
  u.count = l.job[job] >> 16 & 15;
  u.first = l.first[job];
  u.inner0 = (unit - job * per) * kMdUnit;
  return u;
}

// What a warp asks for next: of one unit after the other the blocks of K warp,
// warp + 8, ..., of each a tile of gate rows and one of up rows.
struct MdFeed {
  int unit, kb, up, rows;  // rows: how many of a tile are there
  const uint8_t* gate;     // the unit's first gate row
  const float* scale;      // lane i < 4: of rows 0, 16 (gate), 0, 16 (up)
};

__device__ __forceinline__ void md_feed_unit(const MdParams& p, const MdLists& l, MdFeed& f) {
  const int lane = threadIdx.x & 31;
  const MdUnit u = md_unit(p, l, f.unit);
  f.rows = p.inner - u.inner0;
  f.gate = p.w1 + ((int64_t)u.expert * 2 * p.inner + min(u.inner0, p.inner - 16)) * p.hidden;
  const int row = u.inner0 + 16 * (lane & 1) + (lane & 2 ? p.inner : 0);
  f.scale = p.s1 + ((int64_t)u.expert * p.nb1 + min(row >> 7, p.nb1 - 1)) * p.kb1;
}

// Asks for the next tile, into `to` (the warp's) and, a block's first, `scales`;
// `warp`, `warps`: the warp's place among those that share K.
__device__ __forceinline__ void md_feed(const MdParams& p, const MdLists& l, MdFeed& f, int units, int step, int warp, int warps,
                                        uint32_t to, uint32_t scales) {
  if (f.unit < units) {
    if (f.kb < p.kb1) {
      const int lane = threadIdx.x & 31, k = f.kb * 128;
      const int64_t pitch = p.hidden;
      const uint8_t* from = f.gate + k + (f.up ? p.inner * pitch : 0);
      md_tile(to, from, from + 16 * pitch, pitch, f.rows, f.rows - 16, p.hidden - k);
      if (!f.up && lane < 4) md_copy4(scales + 4 * lane, f.scale + f.kb);
    }
    f.up ^= 1;
    if (!f.up) {
      f.kb += warps;
      if (f.kb - warp >= p.kb1) {
        f.kb = warp;
        f.unit += step;
        if (f.unit < units) md_feed_unit(p, l, f);
      }
    }
  }
  md_commit();
}

// WARPS share a unit's K: a CTA works on 8 / WARPS units at a time.
template <int FMT, int WARPS>
__global__ void __launch_bounds__(kMdThreads, 2) decode_first_kernel(MdParams p) {
  extern __shared__ uint8_t dynamic[];  // [warps][kMdRingBytes], from a multiple of 128 on, then the lists
  __shared__ float part[kMdWarps][4 * kMdSetFloats];
  __shared__ __align__(16) float scales[kMdWarps][kMdStages][4];
  __shared__ int warp_sum[kMdWarps];
  const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const int cta_warp = tid >> 5, group = cta_warp / WARPS, warp = cta_warp % WARPS;
  uint8_t* rings = dynamic + (-md_smem(dynamic) & 127u);
  MdLists l = md_list_places(rings + kMdWarps * kMdRingBytes, p.tokens * p.top_k);
  pdl_wait();
  // The second kernel's CTAs may come as soon as there is room: they ask for
  // their first weights and wait for this kernel's end before they go on.
  pdl_launch_dependents();
  md_lists<false>(p, l, rings, warp_sum);
  // units are dealt out evenly: to fewer groups of warps rather than in a last round of a few
  const int units = l.jobs * p.kb2 * (128 / kMdUnit), groups = gridDim.x * (kMdWarps / WARPS), rounds = (units + groups - 1) / groups;
  const int step = rounds ? (units + rounds - 1) / rounds : 0, mine_first = blockIdx.x + group * gridDim.x;
  if (mine_first >= step) return;
  const auto meet = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(32 * WARPS) : "memory"); };  // the group's warps
  const uint32_t ring = md_smem(rings) + cta_warp * kMdRingBytes, sc_at = md_smem(&scales[cta_warp][0][0]);
  const uint32_t mine = ring + lane * 128 + ((lane & 7) << 4);
  MdFeed f;
  f.unit = mine_first;
  f.kb = warp;
  f.up = 0;
  md_feed_unit(p, l, f);
#pragma unroll
  for (int i = 0; i < kMdStages; i++) md_feed(p, l, f, units, step, warp, WARPS, ring + i * kMdTileBytes, sc_at + i * 16);
  int stage = 0;
  for (int unit = mine_first; unit < units; unit += step) {
    const MdUnit u = md_unit(p, l, unit);
    float acc[4][4] = {};
    const bool there = g < u.count;
    const uint16_t* xt = p.x + (int64_t)(there ? l.token[u.first + g] : 0) * p.hidden + 4 * q;
    uint32_t x[16];
    md_token(xt + warp * 128, p.hidden - warp * 128, there, x);
    for (int kb = warp; kb - warp < p.kb1; kb += WARPS) {
      // the tokens' part of this block of K
      uint32_t b[16], m = 0;
#pragma unroll
      for (int i = 0; i < 16; i++) m = absmax_bf16x2(m, x[i]);
      m = max_u16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = max_u16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      const uint32_t power = md_exponent(max(m << 16, m & 0xFFFF0000u)), back = (254u - power) << 23;
      const float inv0 = __uint_as_float(__shfl_sync(0xFFFFFFFFu, back, 8 * q));
      const float inv1 = __uint_as_float(__shfl_sync(0xFFFFFFFFu, back, 8 * q + 4));
#pragma unroll
      for (int i = 0; i < 16; i++) b[i] = md_scaled(x[i], power << 7);
      const int k = (kb + WARPS) * 128;  // the next block's come while this one is multiplied
      md_token(xt + k, p.hidden - k, there, x);
      float4 sc = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int tile = 0; tile < 2; tile++) {
        md_wait<kMdStages - 1>();
        __syncwarp();
        if (tile == 0) sc = *(const float4*)scales[cta_warp][stage];
        float d[2][4] = {};
        if (kb < p.kb1) {  // else the rest of the warps' last round
#pragma unroll
          for (int s = 0; s < 8; s++) {
            uint32_t w[4];
            md_chunk(mine + stage * kMdTileBytes, s, w);
#pragma unroll
            for (int set = 0; set < 2; set++) {
              uint32_t a0, a1, a2, a3;
              md_codes<FMT>(w[2 * set], a0, a2);
              md_codes<FMT>(w[2 * set + 1], a1, a3);
              md_mma(d[set], a0, a1, a2, a3, b[2 * s], b[2 * s + 1]);
            }
          }
        }
        __syncwarp();  // all lanes have their codes
        md_feed(p, l, f, units, step, warp, WARPS, ring + stage * kMdTileBytes, sc_at + stage * 16);
        stage = stage + 1 == kMdStages ? 0 : stage + 1;
        if (kb < p.kb1) {
#pragma unroll
          for (int set = 0; set < 2; set++) {
            const float s = tile ? (set ? sc.w : sc.z) : (set ? sc.y : sc.x);
            const float f0 = __fmul_rn(s, inv0), f1 = __fmul_rn(s, inv1);
#pragma unroll
            for (int c = 0; c < 4; c++) acc[2 * tile + set][c] = __fmaf_rn(c & 1 ? f1 : f0, d[set][c], acc[2 * tile + set][c]);
          }
        }
      }
    }
    meet();  // the last unit's sums have been read
#pragma unroll
    for (int set = 0; set < 4; set++)
#pragma unroll
      for (int c = 0; c < 4; c++) part[cta_warp][set * kMdSetFloats + (2 * q + (c & 1)) * kMdPitch + g + 8 * (c >> 1)] = acc[set][c];
    meet();
#pragma unroll
    for (int n = warp; n < kMdCols; n += WARPS) {  // inner value m for token n: a warp each token
      const int m = lane, at = n * kMdPitch + (m & 15) + (m >> 4) * kMdSetFloats;
      float gate = 0.0f, up = 0.0f;
#pragma unroll
      for (int w = 0; w < WARPS; w++) {
        gate += part[group * WARPS + w][at];
        up += part[group * WARPS + w][2 * kMdSetFloats + at];
      }
      const float e = expf(-fabsf(gate)), r = __frcp_rn(1.0f + e);
      const float a = __fmul_rn(__fmul_rn(gate, gate >= 0.0f ? r : __fmul_rn(e, r)), up);
      const uint32_t power = md_exponent(warp_max_u32(__float_as_uint(a) & 0x7FFFFFFFu));
      const float v = __fmul_rn(a, __uint_as_float(power << 23));
      const uint32_t hi = md_half2(v, 0.0f) & 0xFFFFu;
      if (n < u.count) {
        // in the order of the second kernel's lanes: value 16 s + 4 q + j of 128 at 32 q + 4 s + j
        const int i = u.inner0 + m;
        const int64_t pair = u.first + n, to = pair * p.kb2 * 128 + (i & ~127) + (i >> 2 & 3) * 32 + (i >> 4 & 7) * 4 + (i & 3);
        p.a_hi[to] = (uint16_t)hi;
        if (p.a_lo != nullptr) {
          float back;
          asm("{\n\t.reg .b16 h, z;\n\tmov.b32 {h, z}, %1;\n\tcvt.f32.f16 %0, h;\n\t}" : "=f"(back) : "r"(hi));
          p.a_lo[to] = (uint16_t)md_half2((hi & 0x7C00u) == 0x7C00u ? 0.0f : v - back, 0.0f);
        }
        if (m == 0) p.a_s[pair * p.kb2 * 4 + u.inner0 / kMdUnit] = __uint_as_float((254u - power) << 23);
      }
    }
  }
  md_wait<0>();
}

// ---------------------------------------------------------------------------
// second product and the weighted sum
// ---------------------------------------------------------------------------
// A place in the list of all jobs' blocks of K.  The jobs of one expert take
// turns every kMdTurn blocks, so that the second finds the weights in L2: all
// warps together read some 150 MB in 16 blocks (64 tokens, 64 experts of 7168 x 2048
// 548 us, 562 without turns, 553 with 4 blocks each).
constexpr int kMdTurn = 8;

struct MdPlace {
  int job, kb, count, first;
  __device__ __forceinline__ void start(const MdParams& p, const MdLists& l, int at) {
    job = at / p.kb2;
    const int place = l.job[job] >> 20 & 15, jobs = l.job[job] >> 24;
    job -= place;
    at -= job * p.kb2;  // among the expert's
    kb = 0;
    if (jobs > 1) kb = at / (jobs * kMdTurn) * kMdTurn;
    at -= kb * jobs;
    const int turn = jobs > 1 ? min(kMdTurn, p.kb2 - kb) : p.kb2;
    job += at / turn;
    kb += at % turn;
  }
  __device__ __forceinline__ void at_job(const MdLists& l) {
    count = l.job[job] >> 16 & 15;
    first = l.first[job];
  }
  // to the next block; whether that is another job's
  __device__ __forceinline__ bool next(const MdParams& p, const MdLists& l) {
    kb++;
    if (kb < p.kb2 && kb % kMdTurn != 0) return false;
    const uint32_t place = l.job[job] >> 20 & 15, jobs = l.job[job] >> 24;
    if (place + 1 < jobs) {  // the expert's next job, from where this turn began
      job++;
      kb = (kb - 1) / kMdTurn * kMdTurn;
    } else if (kb < p.kb2) {  // the expert's next turn
      job -= place;
      return jobs > 1;
    } else {
      job++;
      kb = 0;
    }
    return true;
  }
};

// What a warp asks for next of rows row0 .. row0 + 31: `left` blocks from `at` on.
struct MdFeed2 {
  MdPlace at;
  int left;
  const uint8_t* from;
  const float* scale;
};

__device__ __forceinline__ void md_feed2_job(const MdParams& p, const MdLists& l, int row0, MdFeed2& f) {
  const int64_t e = l.job[f.at.job] & 0xFFFF;
  f.from = p.w2 + (e * p.hidden + row0) * p.inner + f.at.kb * 128;
  f.scale = p.s2 + (e * p.nb2 + (row0 >> 7)) * p.kb2 + f.at.kb;
}

__device__ __forceinline__ void md_feed2(const MdParams& p, const MdLists& l, int row0, MdFeed2& f, uint32_t to, uint32_t scale) {
  if (f.left > 0) {
    md_tile(to, f.from, f.from + 16 * (int64_t)p.inner, p.inner, p.hidden - row0, p.hidden - row0 - 16, p.inner - f.at.kb * 128);
    if ((threadIdx.x & 31) == 0) md_copy4(scale, f.scale);
    f.from += 128;
    f.scale++;
    if (f.at.next(p, l) && f.left > 1) md_feed2_job(p, l, row0, f);
    f.left--;
  }
  md_commit();
}

// The inner values of token g and the scales of tokens 2 q, 2 q + 1 for one block of K.
template <bool LO>
struct MdInner {
  uint4 hi[4], lo[LO ? 4 : 1];
  float4 s[2];
  __device__ __forceinline__ void load(const MdParams& p, const MdPlace& at) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3, kb = at.kb, count = at.count, first = at.first;
    const int64_t from = (int64_t)(first + g) * p.kb2 * 128 + kb * 128 + 32 * q;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      hi[i] = g < count ? *(const uint4*)(p.a_hi + from + 8 * i) : make_uint4(0, 0, 0, 0);
      if (LO) lo[i] = g < count ? *(const uint4*)(p.a_lo + from + 8 * i) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int c = 0; c < 2; c++)
      s[c] = 2 * q + c < count ? *(const float4*)(p.a_s + ((int64_t)(first + 2 * q + c) * p.kb2 + kb) * 4) : make_float4(0, 0, 0, 0);
  }
};

__device__ __forceinline__ void md_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// STAGES: tiles of a warp's ring.
template <int FMT, bool LO, int STAGES>
__global__ void __launch_bounds__(kMdThreads, 2) decode_second_kernel(MdParams p, int shares) {
  constexpr int kRing = STAGES * kMdTileBytes;
  extern __shared__ uint8_t dynamic[];  // [warps][kRing], from a multiple of 128 on, then the lists and the sums
  __shared__ float scales[kMdWarps][STAGES];
  __shared__ int warp_sum[kMdWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const int row0 = blockIdx.x / shares * kMdRows, rank = blockIdx.x % shares;
  uint8_t* rings = dynamic + (-md_smem(dynamic) & 127u);
  float* sums = (float*)(rings + kMdWarps * kRing);  // [warps][tokens][kMdOutPitch]
  MdLists l = md_list_places((uint8_t*)(sums + kMdWarps * p.tokens * kMdOutPitch), p.tokens * p.top_k);
  // The first kernel has waited for all before it and writes none of what is
  // read here: only its inner values are waited for below.
  md_lists<true>(p, l, rings, warp_sum);
  const int64_t all = (int64_t)l.jobs * p.kb2;
  const int parts = kMdWarps * shares, part = rank * kMdWarps + warp;
  const int begin = (int)(all * part / parts), end = (int)(all * (part + 1) / parts);
  const uint32_t ring = md_smem(rings) + warp * kRing, sc_at = md_smem(&scales[warp][0]);
  const uint32_t tile_at = ring + lane * 128 + ((lane & 7) << 4);
  MdPlace at;  // of the inner values asked for last
  MdFeed2 f;
  f.left = end - begin;
  if (begin < end) {
    at.start(p, l, begin);
    at.at_job(l);
    f.at = at;
    md_feed2_job(p, l, row0, f);
  }
#pragma unroll
  for (int i = 0; i < STAGES; i++) md_feed2(p, l, row0, f, ring + i * kMdTileBytes, sc_at + i * 4);
  float* mine = sums + warp * p.tokens * kMdOutPitch;
  for (int i = lane; i < p.tokens * kMdOutPitch; i += 32) mine[i] = 0.0f;
  __syncwarp();
  pdl_wait();
  int stage = 0;
  float acc[2][4] = {};
  MdInner<LO> next;
  if (begin < end) next.load(p, at);
  for (int left = end - begin; left > 0; left--) {
    const MdInner<LO> a = next;
    const int count = at.count, first = at.first;
    const bool last = at.next(p, l);  // of its job's turn
    if (left > 1) {
      if (last) at.at_job(l);
      next.load(p, at);
    }
    md_wait<STAGES - 1>();
    __syncwarp();
    const float sc = scales[warp][stage];
#pragma unroll
    for (int group = 0; group < 4; group++) {  // 32 inner values with one scale
      float d[2][4] = {};
#pragma unroll
      for (int s = 2 * group; s < 2 * group + 2; s++) {
        uint32_t w[4];
        md_chunk(tile_at + stage * kMdTileBytes, s, w);
#pragma unroll
        for (int set = 0; set < 2; set++) {
          uint32_t a0, a1, a2, a3;
          md_codes<FMT>(w[2 * set], a0, a2);
          md_codes<FMT>(w[2 * set + 1], a1, a3);
          if constexpr (LO) {
            const uint4& v = a.lo[s >> 1];
            md_mma(d[set], a0, a1, a2, a3, s & 1 ? v.z : v.x, s & 1 ? v.w : v.y);
          }
          const uint4& h = a.hi[s >> 1];
          md_mma(d[set], a0, a1, a2, a3, s & 1 ? h.z : h.x, s & 1 ? h.w : h.y);
        }
      }
      const float f0 = __fmul_rn(sc, group == 0 ? a.s[0].x : group == 1 ? a.s[0].y : group == 2 ? a.s[0].z : a.s[0].w);
      const float f1 = __fmul_rn(sc, group == 0 ? a.s[1].x : group == 1 ? a.s[1].y : group == 2 ? a.s[1].z : a.s[1].w);
#pragma unroll
      for (int set = 0; set < 2; set++)
#pragma unroll
        for (int c = 0; c < 4; c++) acc[set][c] = __fmaf_rn(c & 1 ? f1 : f0, d[set][c], acc[set][c]);
    }
    __syncwarp();  // all lanes have their codes
    md_feed2(p, l, row0, f, ring + stage * kMdTileBytes, sc_at + stage * 4);
    stage = stage + 1 == STAGES ? 0 : stage + 1;
    if (last || left == 1) {  // on to another job: its tokens' sums leave the registers
#pragma unroll
      for (int c = 0; c < 2; c++) {
        const int col = 2 * q + c;
        if (col < count) {
          const float w = l.weight[first + col];
          float* to = mine + l.token[first + col] * kMdOutPitch + g;
#pragma unroll
          for (int set = 0; set < 2; set++)
#pragma unroll
            for (int h = 0; h < 2; h++) to[16 * set + 8 * h] = __fmaf_rn(w, acc[set][2 * h + c], to[16 * set + 8 * h]);
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
  const int values = p.tokens * kMdRows;
  if (shares > 1) {  // this CTA's sums into its first warp's place, where the others read them
    for (int i = tid; i < values; i += kMdThreads) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kMdWarps; w++) v += sums[(w * p.tokens + i / kMdRows) * kMdOutPitch + i % kMdRows];
      sums[i / kMdRows * kMdOutPitch + i % kMdRows] = v;
    }
    md_cluster_sync();
  }
  const int copies = shares > 1 ? shares : kMdWarps;
  for (int i = rank * kMdThreads + tid; i < values; i += shares * kMdThreads) {
    const int t = i / kMdRows, r = i % kMdRows;
    float v = 0.0f;
    for (int c = 0; c < copies; c++) {
      if (shares > 1) {
        uint32_t from;
        float u;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(md_smem(&sums[t * kMdOutPitch + r])), "r"(c));
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(u) : "r"(from) : "memory");
        v += u;
      } else {
        v += sums[(c * p.tokens + t) * kMdOutPitch + r];
      }
    }
    if (row0 + r >= p.hidden) continue;
    const int64_t at = (int64_t)t * p.hidden + row0 + r;
    if (LO) {
      ((float*)p.out)[at] = v;
    } else {
      uint16_t h;
      asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(v));
      ((uint16_t*)p.out)[at] = h;
    }
  }
  pdl_launch_dependents();
  __syncwarp();
  if (shares > 1) md_cluster_sync();  // no CTA leaves while others read its sums
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
static bool off(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

static size_t decode_workspace(int64_t pairs, int64_t inner) {
  const int64_t kb2 = (inner + 127) / 128;
  return (size_t)(pairs * kb2 * (2 * 2 * 128 + 4 * 4));
}

// The second kernel with STAGES tiles a warp on their way.
template <int FMT, bool LO, int STAGES>
static cudaError_t launch_second(const MdParams& p, cudaStream_t s) {
  constexpr size_t kRings = (size_t)kMdWarps * STAGES * kMdTileBytes + 128, kSums = (size_t)kMdWarps * kMdOutPitch * sizeof(float);
  const size_t smem = kRings + md_list_bytes(p.tokens * p.top_k) + p.tokens * kSums;
  static PerDevice<bool> allowed;
  const cudaError_t e = allow_smem(allowed, decode_second_kernel<FMT, LO, STAGES>, kRings + md_list_bytes(kMdPairs) + kMdTokens * kSums);
  if (e != cudaSuccess) return e;
  // CTAs of one column tile: as many as there is room for side by side
  const int tiles = (p.hidden + kMdRows - 1) / kMdRows;
  const int room = (smem > kMdHalfSm ? 1 : 2) * sm_count();
  int shares = 1;
  while (shares < 8 && tiles * 2 * shares <= room) shares *= 2;
  return launch_cluster(decode_second_kernel<FMT, LO, STAGES>, dim3((unsigned)(tiles * shares)), dim3(kMdThreads), shares, smem, s, p, shares);
}

// The first kernel, WARPS warps a unit.
template <int FMT, int WARPS>
static cudaError_t launch_first(const MdParams& p, int64_t units, cudaStream_t s) {
  constexpr size_t kRings = (size_t)kMdWarps * kMdRingBytes + 128;
  static PerDevice<bool> allowed;
  const cudaError_t e = allow_smem(allowed, decode_first_kernel<FMT, WARPS>, kRings + md_list_bytes(kMdPairs));
  if (e != cudaSuccess) return e;
  const int64_t fit = 2 * (int64_t)sm_count(), ctas = (units + kMdWarps / WARPS - 1) / (kMdWarps / WARPS);  // two an SM have room
  return launch_kernel(decode_first_kernel<FMT, WARPS>, dim3((unsigned)(ctas < fit ? ctas : fit)), dim3(kMdThreads),
                       kRings + md_list_bytes(p.tokens * p.top_k), s, p);
}

template <int FMT, bool LO>
static fp8q_status launch_decode(const MdParams& p, cudaStream_t s) {
  const int slots = p.tokens * p.top_k;
  const int64_t per_job = (int64_t)p.kb2 * (128 / kMdUnit);
  const int64_t units = (slots < p.experts ? slots : p.experts + slots / kMdCols) * per_job;  // at most
  // Half the warps a unit where K's blocks leave many of 8 warps idle and there are units enough (BF16 output: 61 tokens, 40
  // experts of 2064 x 1360: 17 blocks, 97 us, 106 with 8; 16 tokens, 64 experts of 7168 x 2048: 56 blocks, 387 us, 380 with 8)
  const int idle8 = (8 - p.kb1 % 8) % 8, idle4 = (4 - p.kb1 % 4) % 4;
  const bool four = (idle8 - idle4) * 8 > p.kb1 && (slots < p.experts ? slots : p.experts) * per_job >= 8 * (int64_t)sm_count();
  cudaError_t e = four ? launch_first<FMT, 4>(p, units, s) : launch_first<FMT, 8>(p, units, s);
  if (e != cudaSuccess) return cuda_fail(e, "decode first kernel launch");
  // two CTAs an SM matter more than a second tile of each warp on its way
  const size_t smem = (size_t)kMdWarps * kMdRingBytes + 128 + md_list_bytes(slots) + (size_t)kMdWarps * p.tokens * kMdOutPitch * sizeof(float);
  e = smem <= kMdHalfSm ? launch_second<FMT, LO, 2>(p, s) : launch_second<FMT, LO, 1>(p, s);
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
  p.a_lo = out_dt == FP8Q_OUT_FP32 ? p.a_hi + pairs * p.kb2 * 128 : nullptr;
  p.a_s = (float*)(p.a_hi + 2 * pairs * p.kb2 * 128);
  p.out = out;
  const cudaStream_t s = (cudaStream_t)stream;
  if (out_dt == FP8Q_OUT_FP32) return w_fmt == FP8Q_E4M3 ? launch_decode<kE4M3, true>(p, s) : launch_decode<kE5M2, true>(p, s);
  return w_fmt == FP8Q_E4M3 ? launch_decode<kE4M3, false>(p, s) : launch_decode<kE5M2, false>(p, s);
}
