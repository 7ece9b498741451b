// Products with 4-bit weights for a few rows: Y = sum_k X_k W_k^T with
// W_k[n][j] = (q - z) s, one scale s and zero point z per `group` j of a row.
//
// A code byte 0..15, read as e4m3, is q 2^-9 (0..7 are its subnormals, 8..15
// its first binade), so one conversion instruction turns two codes into exact
// bf16 integers.  A group's product runs on the matrix cores over the
// integers, and the scale and zero point enter once a group in fp32:
//   y += s (sum_j x q - z sum_j x).
#include "tpf_block.hpp"

namespace tpf {

__device__ __forceinline__ const QweightArgs& qw_kernarg() {
  return *(const QweightArgs*)__builtin_amdgcn_kernarg_segment_ptr();
}

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// Eight consecutive weights of four code bytes: byte j holds code j (low half)
// and code j + 4 (high half).
__device__ __forceinline__ bf16x8_t unpack8(uint32_t w) {
  const uint32_t lo = w & 0x0f0f0f0fu, hi = (w >> 4) & 0x0f0f0f0fu;
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 512.0f, false);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 512.0f, true);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 512.0f, false);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 512.0f, true);
  return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

constexpr int kQwWaves = 8;

// One workgroup computes 16 columns of Y for 16 MB rows; its waves split the
// groups of all shards and join through LDS.
template <int MB>
__global__ __launch_bounds__(64 * kQwWaves) void qweight_kernel(QweightArgs args) {
  (void)args;
  const QweightArgs& a = qw_kernarg();
  __shared__ float part[kQwWaves][MB * 16][17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n15 = lane & 15, q = lane >> 4;
  const int n = blockIdx.x * 16 + n15;
  const int m0 = blockIdx.y * (MB * 16);
  const int nc = min(n, a.N - 1);          // columns past the end repeat the last one and are not stored
  const int gps = a.K / a.group;           // groups per shard
  const int total = gps * a.p;
  const int g0 = (int)((int64_t)total * wave / kQwWaves), g1 = (int)((int64_t)total * (wave + 1) / kQwWaves);
  f32x4_t acc[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) acc[i] = f32x4_t{0, 0, 0, 0};
  bf16x8_t ones;
#pragma unroll
  for (int i = 0; i < 8; ++i) ones[i] = (__bf16)1.0f;
  for (int g = g0; g < g1; ++g) {
    const int k = __builtin_amdgcn_readfirstlane(g / gps);
    const int gi = g - k * gps;
    const uint8_t* codes = a.codes[k] + (int64_t)nc * (a.K / 2);
    const __bf16* x = a.X[k];
    f32x4_t d[MB], xs[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) d[i] = xs[i] = f32x4_t{0, 0, 0, 0};
    for (int j = gi * a.group; j < (gi + 1) * a.group; j += 32) {
      const bf16x8_t b = unpack8(*reinterpret_cast<const uint32_t*>(codes + j / 2 + 4 * q));
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        const int m = min(m0 + i * 16 + n15, a.M - 1);
        const bf16x8_t xv = *reinterpret_cast<const bf16x8_t*>(x + (int64_t)m * a.K + j + 8 * q);
        d[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, b, d[i], 0, 0, 0);
        xs[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, ones, xs[i], 0, 0, 0);
      }
    }
    const int64_t at = (int64_t)nc * gps + gi;
    const float s = __uint_as_float((uint32_t)a.scales[k][at] << 16);
    const float sz = s * (a.zeros[0] ? (float)a.zeros[k][at] : 8.0f);
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        acc[i][v] = __builtin_fmaf(s, d[i][v], __builtin_fmaf(-sz, xs[i][v], acc[i][v]));
  }
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) part[wave][i * 16 + 4 * q + v][n15] = acc[i][v];
  __syncthreads();
  for (int e = threadIdx.x; e < MB * 256; e += 64 * kQwWaves) {
    const int r = e >> 4, c = e & 15;
    float y = part[0][r][c];
#pragma unroll
    for (int w = 1; w < kQwWaves; ++w) y += part[w][r][c];
    const int m = m0 + r, col = blockIdx.x * 16 + c;
    if (m >= a.M || col >= a.N) continue;
    if (a.gelu) y = gelu_f32(y);
    const int64_t o = (int64_t)m * a.N + col;
    if (a.out == OUT_F32) reinterpret_cast<float*>(a.Y)[o] = y;
    else reinterpret_cast<__bf16*>(a.Y)[o] = (__bf16)y;
  }
}

hipError_t launch_qweight(const QweightArgs& a, hipStream_t s) {
  const unsigned gx = (unsigned)((a.N + 15) / 16);
  const int rows = a.M < kQwMaxRows ? a.M : kQwMaxRows;
  if (rows <= 16) hipLaunchKernelGGL(qweight_kernel<1>, dim3(gx, (a.M + 15) / 16), dim3(64 * kQwWaves), 0, s, a);
  else if (rows <= 32) hipLaunchKernelGGL(qweight_kernel<2>, dim3(gx, (a.M + 31) / 32), dim3(64 * kQwWaves), 0, s, a);
  else hipLaunchKernelGGL(qweight_kernel<4>, dim3(gx, (a.M + 63) / 64), dim3(64 * kQwWaves), 0, s, a);
  return hipGetLastError();
}

}  // namespace tpf
