// Activations kept in 8 bits for the backward pass: pack (with the forward's
// GeLU) and GeLU's gradient from them.
//
// A block of 32 x 32 values shares the least power of two s >= 2^-117 with
// max|finite u| <= 448 s; codes are e4m3(u / s), round to nearest even, and
// NaN where u is not finite.  s >= 2^-117 makes code * s a normal bf16 or
// zero, so every stored value is exact in bf16.
#include <algorithm>

#include "tpf_block.hpp"

namespace tpf {

template <int STREAM, class V>
__device__ __forceinline__ void put(V* p, V v) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, p);
  else *p = v;
}
template <int STREAM, class V>
__device__ __forceinline__ V get(const V* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(p);
  else return *p;
}

typedef u32x2_t u32x2a4_t __attribute__((aligned(4)));   // codes rows are 8-byte aligned at least

template <class A>
__device__ __forceinline__ const A& stash_kernarg() {
  return *(const A*)__builtin_amdgcn_kernarg_segment_ptr();
}

// Phi(-a) / exp(-a^2 / 2) for a >= 0 as a polynomial in 1 / (1 + c a), fitted
// here to the least largest relative error over [0, 14].  The value alone,
// u Phi(u), is rounded to bf16 as it stands, and a fit to 4.8e-6 is far below
// half a step of that (2^-9).  The slope's two terms cancel near u = -0.75,
// where that fit left 1.4e-3 of the result, so the backward takes three terms
// more and 1.2e-8, a fifth of half an fp32 step: the same time there, while the
// pack, nearer to its arithmetic, takes 82 us with them instead of 75.  One
// reciprocal and one exp2 serve the value and the density, where erff and expf
// took about twice the instructions.
struct Gauss {
  float cdf;      // Phi(u)
  float bell;     // exp(-u^2 / 2)
};
template <int FINE>
__device__ __forceinline__ float mills(float a) {
  if constexpr (FINE) {
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.265f, a, 1.0f));
    float q = 0.0308207776f;
    q = __builtin_fmaf(q, t, -0.144228257f);
    q = __builtin_fmaf(q, t, 0.217814239f);
    q = __builtin_fmaf(q, t, -0.116361839f);
    q = __builtin_fmaf(q, t, 0.137952611f);
    q = __builtin_fmaf(q, t, 0.0603132998f);
    q = __builtin_fmaf(q, t, 0.102700938f);
    q = __builtin_fmaf(q, t, 0.10524667f);
    q = __builtin_fmaf(q, t, 0.105741564f);
    return q * t;
  } else {
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.31f, a, 1.0f));
    float q = -0.0739293803f;
    q = __builtin_fmaf(q, t, 0.180450903f);
    q = __builtin_fmaf(q, t, 0.0157443031f);
    q = __builtin_fmaf(q, t, 0.133429849f);
    q = __builtin_fmaf(q, t, 0.12044131f);
    q = __builtin_fmaf(q, t, 0.123860693f);
    return q * t;
  }
}
template <int FINE>
__device__ __forceinline__ Gauss gauss(float u) {
  const float ratio = mills<FINE>(fabsf(u));
  const float bell = __builtin_amdgcn_exp2f(u * u * -0.72134752044f);
  const float tail = ratio * bell;
  return Gauss{u < 0.0f ? tail : 1.0f - tail, bell};
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  const bf16x2_t v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}

// One wave packs 32 rows x 128 columns: lane l holds the eight columns
// 8 (l % 16) of rows l / 16 + 4 i, so a 32-column block is four lanes wide and
// its largest value takes the lane's own maximum and four exchanges.  The codes
// are not read before the backward pass and go past the caches, and so does u
// where its GeLU is what the next product reads.  Without GeLU the next products
// read u itself: smaller than half the memory-side cache it is loaded through
// the caches (pack of 4096 x 4096 and four products of it 365 us, past them 370),
// larger it is not (8192 x 8192: 944 us either way, the pack alone 39 against 37).
// Bound by memory: 4 x 4096 x 4096 with GeLU in 63 us a call, 5.3 TB/s, a large
// copy's rate and more (10 us longer with u and the codes through the caches).
template <int GELU, int STREAM>
__global__ __launch_bounds__(256) void stash_pack_kernel(StashArgs args) {
  (void)args;
  const StashArgs& a = stash_kernarg<StashArgs>();
  const int lane = threadIdx.x & 63;
  const uint32_t rows = a.M;      // unsigned: a band's last row can be past 31 bits
  const int strips = (a.F + 127) / 128, bands = (int)((rows + 31) / 32);
  const int nsc = (a.F + 31) / 32;
  const int64_t units = (int64_t)strips * bands;
  const int64_t unit = a.unit0 + (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (unit >= units * a.p) return;
  const int k = __builtin_amdgcn_readfirstlane((int)(unit / units));
  const int64_t r = unit - k * units;
  const int band = (int)(r / strips), strip = (int)(r % strips);
  const int col = strip * 128 + (lane & 15) * 8;
  const uint32_t row0 = (uint32_t)band * 32 + (lane >> 4);
  const uint16_t* u = reinterpret_cast<const uint16_t*>(a.u[k]);
  const bool cok = col < a.F;
  u32x4_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t row = row0 + 4 * i;
    w[i] = u32x4_t{0, 0, 0, 0};
    if (cok && row < rows) w[i] = get<GELU || STREAM>(reinterpret_cast<const u32x4_t*>(u + (int64_t)row * a.F + col));
  }
  // Largest finite magnitude, as bf16 bits.
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = w[i][j] & 0x7fffu, hi = (w[i][j] >> 16) & 0x7fffu;
      if (lo < 0x7f80u) top = max(top, lo);
      if (hi < 0x7f80u) top = max(top, hi);
    }
#pragma unroll
  for (int d = 1; d <= 32; d <<= 1)
    if (d != 4 && d != 8) top = max(top, (uint32_t)__shfl_xor((int)top, d));
  // The exponent byte of the least power of two that brings the largest value
  // to 448 = 1.75 2^8 or below (one more above 1.75); at least 2^-117.
  const int e = max(10, (int)(((top << 16) + 0x1fffffu) >> 23) - 8);
  const float inv = __uint_as_float((uint32_t)(254 - e) << 23);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t row = row0 + 4 * i;
    if (!cok || row >= rows) continue;
    u32x2_t c;
    u32x4_t hv;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float lo = bf_lo(w[i][j]), hi = bf_hi(w[i][j]);
      int two = __builtin_amdgcn_cvt_pk_fp8_f32(lo * inv, hi * inv, 0, false) & 0xffff;
      if ((w[i][j] & 0x7f80u) == 0x7f80u) two = (two & 0xff00) | 0x7f;
      if ((w[i][j] & 0x7f800000u) == 0x7f800000u) two = (two & 0x00ff) | 0x7f00;
      if (j & 1) c[j >> 1] |= (uint32_t)two << 16;
      else c[j >> 1] = (uint32_t)two;
      if constexpr (GELU) hv[j] = pack_bf16(lo * gauss<0>(lo).cdf, hi * gauss<0>(hi).cdf);
    }
    const int64_t at = (int64_t)row * a.F + col;
    put<1>(reinterpret_cast<u32x2_t*>(a.codes[k] + at), c);
    if constexpr (GELU) put<STREAM>(reinterpret_cast<u32x4_t*>(reinterpret_cast<uint16_t*>(a.h[k]) + at), hv);
  }
  if (cok && (lane & 51) == 0) a.scales[k][(int64_t)band * nsc + (col >> 5)] = (uint8_t)e;
}

hipError_t launch_stash_pack(const StashArgs& a, int gelu, hipStream_t s) {
  const int64_t units = (int64_t)((a.F + 127) / 128) * (((int64_t)a.M + 31) / 32) * a.p;
  const int64_t most = (int64_t)UINT32_MAX / 256 * 4;      // a grid has fewer than 2^32 threads
  for (int64_t u = 0; u < units; u += most) {
    StashArgs part = a;
    part.unit0 = u;
    const dim3 grid((unsigned)((std::min(units - u, most) + 3) / 4));
    const int64_t bytes = (int64_t)a.p * a.M * a.F * 2;
    if (!gelu && bytes >= kStreamBytes / 2) hipLaunchKernelGGL((stash_pack_kernel<0, 1>), grid, dim3(256), 0, s, part);
    else if (!gelu) hipLaunchKernelGGL((stash_pack_kernel<0, 0>), grid, dim3(256), 0, s, part);
    else if (bytes >= kStreamBytes) hipLaunchKernelGGL((stash_pack_kernel<1, 1>), grid, dim3(256), 0, s, part);
    else hipLaunchKernelGGL((stash_pack_kernel<1, 0>), grid, dim3(256), 0, s, part);
  }
  return hipGetLastError();
}

// du = dh (Phi(u) + u phi(u)) and h = u Phi(u) from the stored values, eight
// columns a lane.  Bound by memory: 8 x 2048 x 6144 in 122 to 124 us a call, 5.7 TB/s.
template <int STREAM>
__global__ __launch_bounds__(256) void stash_backward_kernel(StashArgs args) {
  (void)args;
  const StashArgs& a = stash_kernarg<StashArgs>();
  const int k = blockIdx.y;
  const int fv = a.F / 8, nsc = (a.F + 31) / 32;
  const int64_t total = (int64_t)a.M * fv;
  const uint8_t* codes = a.codes[k];
  const uint8_t* scales = a.scales[k];
  const uint16_t* dh = reinterpret_cast<const uint16_t*>(a.dh[k]);
  uint16_t* du = reinterpret_cast<uint16_t*>(a.du[k]);
  uint16_t* h = reinterpret_cast<uint16_t*>(a.h[k]);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int row = (int)(i / fv), v = (int)(i - (int64_t)row * fv);
    const u32x2_t c = *reinterpret_cast<const u32x2a4_t*>(codes + i * 8);
    const u32x4_t g = get<STREAM>(reinterpret_cast<const u32x4_t*>(dh + i * 8));
    const float scale = __uint_as_float((uint32_t)scales[(int64_t)(row >> 5) * nsc + (v >> 2)] << 23);
    u32x4_t o, y;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      typedef float f32x2_t __attribute__((ext_vector_type(2)));
      const f32x2_t two = (j & 1) ? __builtin_amdgcn_cvt_pk_f32_fp8((int)c[j >> 1], true)
                                  : __builtin_amdgcn_cvt_pk_f32_fp8((int)c[j >> 1], false);
      const float u0 = two[0] * scale, u1 = two[1] * scale;
      const Gauss g0 = gauss<1>(u0), g1 = gauss<1>(u1);
      const float d0 = bf_lo(g[j]) * __builtin_fmaf(u0 * 0.3989422804f, g0.bell, g0.cdf);
      const float d1 = bf_hi(g[j]) * __builtin_fmaf(u1 * 0.3989422804f, g1.bell, g1.cdf);
      o[j] = pack_bf16(d0, d1);
      y[j] = pack_bf16(u0 * g0.cdf, u1 * g1.cdf);
    }
    put<STREAM>(reinterpret_cast<u32x4_t*>(du + i * 8), o);
    put<STREAM>(reinterpret_cast<u32x4_t*>(h + i * 8), y);
  }
}

hipError_t launch_stash_backward(const StashArgs& a, int num_cus, hipStream_t s) {
  const int64_t groups = ((int64_t)a.M * (a.F / 8) + 255) / 256;
  const int64_t cap = std::max<int64_t>(1, (int64_t)num_cus * 32 / a.p);
  const dim3 grid((unsigned)std::min(groups, cap), (unsigned)a.p);
  if ((int64_t)a.p * a.M * a.F * 4 >= kStreamBytes) hipLaunchKernelGGL(stash_backward_kernel<1>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(stash_backward_kernel<0>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace tpf
