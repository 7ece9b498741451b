// Activations packed for 8-bit products: e4m3 codes with one power of two for
// each 128 values along a row, and the same of the transpose.
//
// A block shares the least power of two s >= 2^-117 with max|finite u| <= 448 s;
// codes are e4m3(u / s), round to nearest even, and NaN where u is not finite.
// A power of two costs a floating-point code nothing (its relative step is the
// same at every scale), the matrix cores apply it by themselves, and u / s is
// exact, so the one rounding is the code's.
#include <algorithm>

#include "tpf_scaled.hpp"

namespace tpf {
namespace {

// Largest finite magnitude of eight bf16 values, as bf16 bits.
__device__ __forceinline__ uint32_t top_of(u32x4_t w) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t lo = w[j] & 0x7fffu, hi = (w[j] >> 16) & 0x7fffu;
    if (lo < 0x7f80u) top = max(top, lo);
    if (hi < 0x7f80u) top = max(top, hi);
  }
  return top;
}

// Exponent byte of the scale of a block with this largest magnitude: 448 =
// 1.75 2^8 holds everything up to 1.75 of its binade, one more is needed above.
__device__ __forceinline__ int scale_byte(uint32_t top) { return max(10, (int)(((top << 16) + 0x1fffffu) >> 23) - 8); }

// Code of u / s; the conversion saturates, so values that are not finite are
// given the code of NaN here.
__device__ __forceinline__ float scaled(uint32_t bits, float inv) {
  return (bits & 0x7f800000u) == 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float(bits) * inv;
}
__device__ __forceinline__ uint32_t codes4(uint32_t w0, uint32_t w1, float inv) {
  uint32_t c = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(scaled(w0 << 16, inv), scaled(w0 & 0xffff0000u, inv), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(scaled(w1 << 16, inv), scaled(w1 & 0xffff0000u, inv), (int)c, true);
}
__device__ __forceinline__ float inverse(int e) { return __uint_as_float((uint32_t)(254 - e) << 23); }

// One wave packs 512 values of a row: lane l holds the eight from 8 l, a block
// is 16 lanes wide, and the four blocks' scales are one word.  Memory bounds it (8 x
// 2048 x 6144: 60 us, 5.0 TB/s).
__global__ __launch_bounds__(256) void scaled_pack_rows_kernel(PackArgs args) {
  (void)args;
  const PackArgs& a = *(const PackArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  const int lane = threadIdx.x & 63;
  const int width = ((a.K + 127) / 128 + 3) >> 2;        // words of scales a row
  const int k = blockIdx.y;
  for (int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); unit < (int64_t)a.M * width;
       unit += (int64_t)gridDim.x * 4) {
    const int row = __builtin_amdgcn_readfirstlane((int)(unit / width));
    const int quad = __builtin_amdgcn_readfirstlane((int)(unit - (int64_t)row * width));
    const int col = quad * 512 + lane * 8;
    const bool ok = col < a.K;
    u32x4_t w = u32x4_t{0, 0, 0, 0};
    const int64_t at = (int64_t)row * a.K + col;
    if (ok) w = *reinterpret_cast<const u32x4_t*>(reinterpret_cast<const uint16_t*>(a.u[k]) + at);
    uint32_t top = top_of(w);
#pragma unroll
    for (int d = 1; d <= 8; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    const int e = scale_byte(top);
    const float inv = inverse(e);
    if (ok) *reinterpret_cast<u32x2_t*>(a.codes[k] + at) = u32x2_t{codes4(w[0], w[1], inv), codes4(w[2], w[3], inv)};
    const uint32_t word = (uint32_t)__shfl(e, 0) | (uint32_t)__shfl(e, 16) << 8 | (uint32_t)__shfl(e, 32) << 16 |
                          (uint32_t)__shfl(e, 48) << 24;
    if (lane == 0) *reinterpret_cast<uint32_t*>(a.scales[k] + ((int64_t)row * width + quad) * 4) = word;
  }
}

// Rows [first, first + n) of the block of 128 columns number `blk` of a packed
// transpose: the experts' rows, each expert's from a block of its own, or the
// rows as they are.
struct RowRange {
  int first, n;
};
__device__ __forceinline__ RowRange block_rows(const PackArgs& a, int blk, int lane) {
  if ((int64_t)blk * kScaleBlock >= a.columns) return RowRange{0, 0};
  if (!a.offsets) return RowRange{blk * kScaleBlock, max(0, min(kScaleBlock, a.R - blk * kScaleBlock))};
  int before = 0;
  for (int base = 0; base < a.E; base += 64) {
    const int i = base + lane;
    int lo = 0, hi = 0;
    if (i < a.E) {
      lo = min(max(a.offsets[i], 0), a.R);
      hi = min(max(a.offsets[i + 1], lo), a.R);
    }
    const int blocks = (hi - lo + kScaleBlock - 1) / kScaleBlock;
    int upto = blocks;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int t = __shfl_up(upto, d);
      if (lane >= d) upto += t;
    }
    const uint64_t past = __ballot(before + upto > blk);
    if (past) {
      const int at = __builtin_ctzll(past);
      const int skip = max(blk - (before + __shfl(upto - blocks, at)), 0);
      const int f = __shfl(lo, at) + skip * kScaleBlock;
      return RowRange{f, min(kScaleBlock, __shfl(hi, at) - f)};
    }
    before += __shfl(upto, 63);
  }
  return RowRange{0, 0};
}

// A workgroup packs a block of 128 rows x 128 columns of u down the columns, and
// with ROWS along the rows as well, so that u is read once.  Thread (q, c) holds
// rows 8 q .. 8 q + 7 of columns 8 c .. 8 c + 7: a row's largest value takes the
// exchange of 16 lanes, a column's that of the wave's four q and the four waves.
// The transpose's codes go through LDS, eight rows of a column at a time, their
// places XORed with c so that 16 lanes write to all banks.
// 4096 x 4096 both ways: rows and columns packed in passes of their own 26 us, in
// one 22 (with two waves a SIMD, as the registers fall out by themselves, 31).  All
// workgroups of that size run at once, so that loads and stores, 7 us each at
// memory's rate, lie one behind the other; larger sizes overlap them.
template <int ROWS>
__global__ __launch_bounds__(256, 4) void scaled_pack_columns_kernel(PackArgs args) {
  (void)args;
  const PackArgs& a = *(const PackArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  __shared__ __attribute__((aligned(16))) uint8_t turned[128 * 128];
  __shared__ uint16_t tops[4][128];
  const int k = blockIdx.z, blk = blockIdx.x, c0 = blockIdx.y * 128;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = threadIdx.x & 15, q = threadIdx.x >> 4;
  const uint16_t* u = reinterpret_cast<const uint16_t*>(a.u[k]);
  const RowRange r = block_rows(a, blk, lane);
  const int col = c0 + c * 8;
  u32x4_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int local = q * 8 + i;
    w[i] = u32x4_t{0, 0, 0, 0};
    if (local < r.n && col < a.K) {
      int row = r.first + local;
      if (a.src) row = a.src[row] / a.top;
      if ((uint32_t)row < (uint32_t)a.M) w[i] = *reinterpret_cast<const u32x4_t*>(u + (int64_t)row * a.K + col);
    }
  }
  const int xwidth = ((a.K + 127) / 128 + 3) >> 2 << 2, twidth = (a.columns / kScaleBlock + 3) >> 2 << 2;
  if constexpr (ROWS) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t top = top_of(w[i]);
#pragma unroll
      for (int d = 1; d <= 8; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
      const int e = scale_byte(top);
      const float inv = inverse(e);
      if (q * 8 + i < r.n) {
        const int64_t row = r.first + q * 8 + i;
        if (col < a.K)
          *reinterpret_cast<u32x2_t*>(a.codes[k] + row * a.K + col) =
              u32x2_t{codes4(w[i][0], w[i][1], inv), codes4(w[i][2], w[i][3], inv)};
        if (c == 0) a.scales[k][row * xwidth + blockIdx.y] = (uint8_t)e;
      }
    }
  }
  // The columns' largest values: of the thread's rows, the wave's, then all.
  uint32_t even[4] = {}, odd[4] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = w[i][j] & 0x7fffu, hi = (w[i][j] >> 16) & 0x7fffu;
      if (lo < 0x7f80u) even[j] = max(even[j], lo);
      if (hi < 0x7f80u) odd[j] = max(odd[j], hi);
    }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int d = 16; d <= 32; d <<= 1) {
      even[j] = max(even[j], (uint32_t)__shfl_xor((int)even[j], d));
      odd[j] = max(odd[j], (uint32_t)__shfl_xor((int)odd[j], d));
    }
    if (lane < 16) *reinterpret_cast<uint32_t*>(&tops[wave][c * 8 + 2 * j]) = even[j] | odd[j] << 16;
  }
  __syncthreads();
  int e[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const uint32_t t = *reinterpret_cast<const uint32_t*>(&tops[v][c * 8 + 2 * j]);
      lo = max(lo, t & 0xffffu);
      hi = max(hi, t >> 16);
    }
    e[2 * j] = scale_byte(lo);
    e[2 * j + 1] = scale_byte(hi);
  }
  if (q == 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col + j < a.K) a.scales_t[k][(int64_t)(col + j) * twidth + blk] = (uint8_t)e[j];
  }
  if (blk * kScaleBlock >= a.columns) return;            // a word's bytes behind the last block
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float inv = inverse(e[j]);
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = j & 1 ? w[i][j >> 1] & 0xffff0000u : w[i][j >> 1] << 16;
    u32x2_t codes;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t t = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(scaled(v[4 * h], inv), scaled(v[4 * h + 1], inv), 0, false);
      codes[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(scaled(v[4 * h + 2], inv), scaled(v[4 * h + 3], inv), (int)t, true);
    }
    *reinterpret_cast<u32x2_t*>(&turned[(c * 8 + j) * 128 + (q ^ c) * 8]) = codes;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = i * 256 + threadIdx.x, tc = at >> 3, part = at & 7;      // 16 rows of one column
    if (c0 + tc >= a.K) continue;
    const u32x2_t lo = *reinterpret_cast<const u32x2_t*>(&turned[tc * 128 + ((2 * part) ^ (tc >> 3)) * 8]);
    const u32x2_t hi = *reinterpret_cast<const u32x2_t*>(&turned[tc * 128 + ((2 * part + 1) ^ (tc >> 3)) * 8]);
    *reinterpret_cast<u32x4_t*>(a.codes_t[k] + (int64_t)(c0 + tc) * a.columns + blk * 128 + part * 16) =
        u32x4_t{lo[0], lo[1], hi[0], hi[1]};
  }
}

}  // namespace

hipError_t launch_scaled_pack(const PackArgs& a, hipStream_t s) {
  // One read of u where the columns' rows are the rows as they lie; experts' blocks begin inside the rows' own and end
  // before the rows of no expert, so theirs are two passes (32768 x 4096 of 64 experts: 171 us; plain rows 145).
  const bool together = a.codes[0] && a.codes_t[0] && !a.offsets;
  if (a.codes[0] && !together) {
    const int64_t units = (int64_t)a.M * (scale_width(a.K) / 4);
    hipLaunchKernelGGL(scaled_pack_rows_kernel, dim3((unsigned)std::min<int64_t>((units + 3) / 4, 1 << 22), a.p), dim3(256),
                       0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.codes_t[0]) {
    // Words of scales end with the bytes of blocks that are not there: those too have a workgroup.
    const dim3 grid((unsigned)scale_width(a.columns), (unsigned)(together ? scale_width(a.K) : scale_blocks(a.K)), a.p);
    if (together) hipLaunchKernelGGL(scaled_pack_columns_kernel<1>, grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(scaled_pack_columns_kernel<0>, grid, dim3(256), 0, s, a);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace tpf
