// blockwise.cuh -- quantization of one 128 x 128 tile of BF16 values in shared
// memory to blockwise FP8, shared by the kernels that load such a tile: with
// TMA from consecutive rows, or row by row from anywhere.
#pragma once

#include "fp8q_device.cuh"
#include "tma.cuh"

namespace fp8q {

constexpr int kBwTile = 128;
constexpr int kBwBoxCols = 64;
constexpr int kBwBoxBytes = kBwTile * 128;      // 128 rows x 128 bytes
constexpr int kBwStageBytes = 2 * kBwBoxBytes;  // 32 KB
constexpr int kBwConsumers = 256;
constexpr int kBwBarCons = 1;  // named barrier ids among the consumers

struct BwParams {
  int64_t rows, cols;
  int64_t tiles_r, tiles_c;  // ceil(rows / 128), ceil(cols / 128)
  int pow2;
  uint8_t* q;     // [rows][cols]
  float* s;       // 1x128: [rows][tiles_c]; 128x128: [tiles_r][tiles_c]
  uint8_t* q_t;   // [cols][rows]
  float* s_t;     // 128x1: [cols][tiles_r]; 128x128: [tiles_c][tiles_r]
};

// Byte offset in a stage of the 16-byte chunk part holding row r, column c
// (c even): box c / 64, then the 128-byte row line with its chunks swizzled.
__device__ __forceinline__ uint32_t bw_off(int r, int c) {
  const int b = (c & 63) * 2;
  return (uint32_t)((c >> 6) * kBwBoxBytes + r * 128 + ((((b >> 4) ^ (r & 7)) << 4) | (b & 15)));
}

template <int FMT>
__device__ __forceinline__ float bw_scale(uint32_t amax_bits, int pow2) {
  float s = scale_from_amax(amax_bits, Fmt<FMT>::kMax, 0);
  if (pow2) s = __uint_as_float(__float_as_uint(s) & 0xFF800000u);  // s is a positive normal float
  return s;
}

// Magnitude bits (as FP32 bits) of the largest of 8 BF16 values.
__device__ __forceinline__ uint32_t amax8(const uint4& v) {
  const uint32_t m = absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(absmax_bf16x2(0u, v.x), v.y), v.z), v.w);
  return max(m << 16, m & 0xFFFF0000u);
}

template <int FMT>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float s) {
  return canon_nan4<FMT>(cvt4<FMT>(__fmul_rn(a, s), __fmul_rn(b, s), __fmul_rn(c, s), __fmul_rn(d, s)));
}

// Row pass: rows of the tile in 8 sweeps of 16 (a warp takes 2 rows, one
// per half-warp).  BLOCK 1: each row is a group; 128: every row uses s_tile.
template <int FMT, int BLOCK>
__device__ __forceinline__ void bw_rows(const BwParams& p, const unsigned char* st, int64_t r0, int64_t c0,
                                        float s_tile, int ctid) {
  const int w = ctid >> 5, l = ctid & 31, half = l >> 4, hl = l & 15;
  const int c = hl * 8;
  const bool col_ok = c0 + c < p.cols;
#pragma unroll 2
  for (int pass = 0; pass < kBwTile / 16; pass++) {
    const int r = pass * 16 + w * 2 + half;
    const uint4 v = *(const uint4*)(st + bw_off(r, c));
    float s = s_tile;
    if constexpr (BLOCK == 1) {
      uint32_t a = amax8(v);
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) a = max(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
      s = bw_scale<FMT>(a, p.pow2);
      if (hl == 0 && r0 + r < p.rows) p.s[(r0 + r) * p.tiles_c + c0 / kBwTile] = __frcp_rn(s);
    }
    if (r0 + r < p.rows && col_ok) {
      uint2 o;
      o.x = codes4<FMT>(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y), s);
      o.y = codes4<FMT>(bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w), s);
      st_stream(p.q + (r0 + r) * p.cols + c0 + c, o);
    }
  }
}

// Column pass: thread = (column pair, row quarter).  BLOCK 1: each column is
// a group of 128 rows; 128: both columns use s_tile (the transposed block).
template <int FMT, int BLOCK>
__device__ __forceinline__ void bw_cols(const BwParams& p, const unsigned char* st, int64_t r0, int64_t c0,
                                        float s_tile, int ctid, uint32_t* sh_amax) {
  const int pp = ctid & 63, h = ctid >> 6;
  const int c = 2 * pp;
  uint32_t w[32];
#pragma unroll
  for (int i = 0; i < 32; i++) {
    const int r = 32 * h + i;
    w[i] = *(const uint32_t*)(st + bw_off(r, c));
  }
  float s0 = s_tile, s1 = s_tile;
  if constexpr (BLOCK == 1) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 32; i++) m = absmax_bf16x2(m, w[i]);
    sh_amax[h * kBwTile + c] = (m & 0xFFFFu) << 16;
    sh_amax[h * kBwTile + c + 1] = m & 0xFFFF0000u;
    named_barrier_sync(kBwBarCons, kBwConsumers);
    uint32_t a0 = 0, a1 = 0;
#pragma unroll
    for (int k = 0; k < 4; k++) {
      a0 = max(a0, sh_amax[k * kBwTile + c]);
      a1 = max(a1, sh_amax[k * kBwTile + c + 1]);
    }
    named_barrier_sync(kBwBarCons, kBwConsumers);  // sh_amax is rewritten by the next tile
    s0 = bw_scale<FMT>(a0, p.pow2);
    s1 = bw_scale<FMT>(a1, p.pow2);
    if (h == 0 && c0 + c < p.cols) {
      p.s_t[(c0 + c) * p.tiles_r + r0 / kBwTile] = __frcp_rn(s0);
      p.s_t[(c0 + c + 1) * p.tiles_r + r0 / kBwTile] = __frcp_rn(s1);
    }
  }
  if (c0 + c >= p.cols) return;
  uint32_t d0[8], d1[8];
#pragma unroll
  for (int k = 0; k < 8; k++) {
    d0[k] = codes4<FMT>(bf16_lo(w[4 * k]), bf16_lo(w[4 * k + 1]), bf16_lo(w[4 * k + 2]), bf16_lo(w[4 * k + 3]), s0);
    d1[k] = codes4<FMT>(bf16_hi(w[4 * k]), bf16_hi(w[4 * k + 1]), bf16_hi(w[4 * k + 2]), bf16_hi(w[4 * k + 3]), s1);
  }
  const int64_t rr = r0 + 32 * h;
  uint8_t* t0 = p.q_t + (c0 + c) * p.rows + rr;
  uint8_t* t1 = t0 + p.rows;
  if (rr < p.rows) {
    st_stream(t0, make_uint4(d0[0], d0[1], d0[2], d0[3]));
    st_stream(t1, make_uint4(d1[0], d1[1], d1[2], d1[3]));
  }
  if (rr + 16 < p.rows) {
    st_stream(t0 + 16, make_uint4(d0[4], d0[5], d0[6], d0[7]));
    st_stream(t1 + 16, make_uint4(d1[4], d1[5], d1[6], d1[7]));
  }
}

}  // namespace fp8q
