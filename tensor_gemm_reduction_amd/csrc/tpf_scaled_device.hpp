// Device pieces shared by the 8-bit products: the scaled matrix instruction and
// the experts' rows.
#pragma once

#include "tpf_gauss.hpp"
#include "tpf_scaled.hpp"

namespace tpf {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

// c + 2^(wb - 127 + xb - 127) w x over one block of 128.
__device__ __forceinline__ f32x4_t sc_mfma(i32x8_t w, i32x8_t x, f32x4_t c, int wb, int xb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, 0, 0, 0, wb, 0, xb);
}

// 32 codes as four operands of the bf16 instruction.
struct ScFine {
  bf16x8_t k[4];
};
__device__ __forceinline__ ScFine sc_fine(i32x8_t c) {
  ScFine f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    typedef uint32_t u32x4v_t __attribute__((ext_vector_type(4)));
    u32x4v_t w;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      w[2 * j] = __builtin_bit_cast(uint32_t, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[2 * i + j], 1.0f, false));
      w[2 * j + 1] = __builtin_bit_cast(uint32_t, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[2 * i + j], 1.0f, true));
    }
    f.k[i] = __builtin_bit_cast(bf16x8_t, w);
  }
  return f;
}
// w x over one block of 128.
__device__ __forceinline__ f32x4_t sc_mfma_fine(const ScFine& w, const ScFine& x) {
  f32x4_t c = f32x4_t{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.k[i], x.k[i], c, 0, 0, 0);
  return c;
}
// GeLU, x Phi(x).  For bf16 results the density's exponent x^2 / 2 is rounded to
// fp32, which costs up to 2^-17 of the result by x = -13.  For fp32 results what the
// square and its product with log2(e) / 2 lose is carried into the density: 2^-20 of
// the result at most (mills' sum and reciprocal, exp2 and four products: 7.4 half
// steps with exact reciprocals and exp2).  Results below the least normal number may
// be zeros.
template <int OUT>
__device__ __forceinline__ float sc_gelu1(float x) {
  if constexpr (OUT == OUT_F32) {
    const float a = fabsf(x);
    if (a > 32.0f) return x > 0.0f ? x : x * 0.0f;
    constexpr float kHalf = -0x1.715476p-1f, kHalfLow = -0x1.4ae0cp-27f;        // -log2(e) / 2
    const float square = a * a, low = __builtin_fmaf(a, a, -square), t = square * kHalf;
    const float rest = __builtin_fmaf(low, kHalf, __builtin_fmaf(square, kHalfLow, __builtin_fmaf(square, kHalf, -t)));
    const float e = __builtin_amdgcn_exp2f(t);
    const float tail = mills<1>(a) * __builtin_fmaf(e, rest * 0.69314718f, e) * a;
    return x < 0.0f ? -tail : x - tail;
  } else {
    return x * gauss<1>(x).cdf;
  }
}
template <int OUT>
__device__ __forceinline__ f32x4_t sc_gelu(f32x4_t v) {
  return f32x4_t{sc_gelu1<OUT>(v[0]), sc_gelu1<OUT>(v[1]), sc_gelu1<OUT>(v[2]), sc_gelu1<OUT>(v[3])};
}
// 2^(e - 127), NaN for 255 as the matrix instruction takes it
__device__ __forceinline__ float exp_byte(int e) {
  return __uint_as_float((uint32_t)e << 23 | ((uint32_t)e - 1u >= 254u ? 0x400000u : 0u));
}

// Number `t` of the tiles of BM rows that the experts' rows are cut into, each
// expert's from its first row on: the expert, the tile's first row and its
// rows (0: there is no such tile).  "Expert" E: the rows behind the last one's.
struct RowTile {
  int e, row0, rows;
};
template <int BM>
__device__ __forceinline__ RowTile expert_tile(const int* offsets, int E, int R, int t, int lane) {
  int before = 0;
  for (int base = 0; base <= E; base += 64) {
    const int i = base + lane;
    int lo = 0, hi = 0;
    if (i <= E) {
      lo = min(max(offsets[i], 0), R);
      hi = i < E ? min(max(offsets[i + 1], lo), R) : R;
    }
    const int tiles = (hi - lo + BM - 1) / BM;
    int upto = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(upto, d);
      if (lane >= d) upto += v;
    }
    const uint64_t past = __ballot(before + upto > t);
    if (past) {
      const int at = __builtin_ctzll(past);
      const int skip = max(t - (before + __builtin_amdgcn_readlane(upto - tiles, at)), 0);
      const int first = __builtin_amdgcn_readlane(lo, at) + skip * BM;
      return RowTile{base + at, first, min(BM, __builtin_amdgcn_readlane(hi, at) - first)};
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  return RowTile{0, 0, 0};
}
// The most tiles that any loads of the experts can need.
inline int expert_tiles(int64_t R, int64_t E, int BM) {
  return (int)((R + (int64_t)(BM - 1) * (E + 1 < R ? E + 1 : R)) / BM);
}

// Expert e's blocks of 128 columns in a packed transpose that holds `blocks`.
struct BlockRange {
  int first, n;
};
__device__ __forceinline__ BlockRange expert_blocks(const int* offsets, int E, int e, int blocks, int lane) {
  int before = 0, mine = 0;
  for (int base = 0; base <= e; base += 64) {
    const int i = base + lane;
    const int n = i <= e && i < E ? (max(offsets[i + 1] - offsets[i], 0) + kScaleBlock - 1) / kScaleBlock : 0;
    if (i == e) mine = n;
    before += i < e ? n : 0;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    before += __shfl_xor(before, d);
    mine = max(mine, __shfl_xor(mine, d));
  }
  before = __builtin_amdgcn_readfirstlane(min(max(before, 0), blocks));
  mine = __builtin_amdgcn_readfirstlane(mine);
  return BlockRange{before, min(mine, blocks - before)};
}

}  // namespace tpf
