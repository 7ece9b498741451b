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
// is 16 lanes wide, and the four blocks' scales are one word.
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
      const int skip = blk - (before + __shfl(upto - blocks, at));
      const int f = __shfl(lo, at) + skip * kScaleBlock;
      return RowRange{f, min(kScaleBlock, __shfl(hi, at) - f)};
    }
    before += __shfl(upto, 63);
  }
  return RowRange{0, 0};
}

// A workgroup packs 512 columns of the transpose (four blocks of rows of u) of
// 32 rows (columns of u): each block's 128 x 32 values go through LDS, turned.
// The four blocks' scales of a row are one word, their codes 512 bytes.
constexpr int kPackK = 32;
__global__ __launch_bounds__(256) void scaled_pack_columns_kernel(PackArgs args) {
  (void)args;
  const PackArgs& a = *(const PackArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  __shared__ uint32_t codes[kPackK][129];     // 512 codes a row, one word of padding
  __shared__ uint8_t exps[kPackK][4];
  const int k = blockIdx.z, quad = blockIdx.x, c0 = blockIdx.y * kPackK;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint16_t* u = reinterpret_cast<const uint16_t*>(a.u[k]);
  // Wave w packs block w: lane l holds rows 2 (l / 4) + 32 i and the one after
  // them, columns 8 (l % 4) .. + 7.
  const int blk = quad * 4 + wave;
  RowRange r{0, 0};
  if (blk * kScaleBlock < a.columns) r = block_rows(a, blk, lane);
  const int col = c0 + (lane & 3) * 8;
  u32x4_t w[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int local = i * 32 + (lane >> 2) * 2 + h;
      w[i][h] = u32x4_t{0, 0, 0, 0};
      if (local < r.n && col < a.K) {
        int row = r.first + local;
        if (a.src) row = a.src[row] / a.top;
        if ((uint32_t)row < (uint32_t)a.M) w[i][h] = *reinterpret_cast<const u32x4_t*>(u + (int64_t)row * a.K + col);
      }
    }
  // Each of the lane's eight columns: the largest of its 8 rows, then over the 16 lanes of the column.
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t v = (c & 1 ? w[i][h][c >> 1] >> 16 : w[i][h][c >> 1]) & 0x7fffu;
        if (v < 0x7f80u) top = max(top, v);
      }
#pragma unroll
    for (int d = 4; d <= 32; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    const int e = scale_byte(top);
    const float inv = inverse(e);
    const int kr = (lane & 3) * 8 + c;
    if (lane < 4) exps[kr][wave] = (uint8_t)e;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b0 = c & 1 ? w[i][0][c >> 1] & 0xffff0000u : w[i][0][c >> 1] << 16;
      const uint32_t b1 = c & 1 ? w[i][1][c >> 1] & 0xffff0000u : w[i][1][c >> 1] << 16;
      const uint32_t two = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(scaled(b0, inv), scaled(b1, inv), 0, false);
      reinterpret_cast<uint16_t*>(&codes[kr][wave * 32])[i * 16 + (lane >> 2)] = (uint16_t)two;
    }
  }
  __syncthreads();
  const int width = (a.columns / kScaleBlock + 3) >> 2;
  for (int i = threadIdx.x; i < kPackK * 32; i += 256) {
    const int kr = i >> 5, part = i & 31;               // 16 bytes each
    const int x = quad * 512 + part * 16;
    if (c0 + kr < a.K && x < a.columns) {
      const uint32_t* from = &codes[kr][part * 4];
      *reinterpret_cast<u32x4_t*>(a.codes_t[k] + (int64_t)(c0 + kr) * a.columns + x) =
          u32x4_t{from[0], from[1], from[2], from[3]};
    }
  }
  if (threadIdx.x < kPackK && c0 + (int)threadIdx.x < a.K)
    reinterpret_cast<uint32_t*>(a.scales_t[k])[(int64_t)(c0 + threadIdx.x) * width + quad] =
        *reinterpret_cast<const uint32_t*>(exps[threadIdx.x]);
}

}  // namespace

hipError_t launch_scaled_pack(const PackArgs& a, hipStream_t s) {
  if (a.codes[0]) {
    const int64_t units = (int64_t)a.M * (scale_width(a.K) / 4);
    hipLaunchKernelGGL(scaled_pack_rows_kernel, dim3((unsigned)std::min<int64_t>((units + 3) / 4, 1 << 22), a.p), dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.codes_t[0]) {
    const int quads = (a.columns / kScaleBlock + 3) / 4;
    hipLaunchKernelGGL(scaled_pack_columns_kernel, dim3(quads, (a.K + kPackK - 1) / kPackK, a.p), dim3(256), 0, s, a);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace tpf
