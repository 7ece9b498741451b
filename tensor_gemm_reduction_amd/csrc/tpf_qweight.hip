// Products with 4-bit weights for a few rows: Y = sum_k X_k W_k^T with
// W_k[n][j] = (q - z) s, one scale s and zero point z per group of j.
//
// A code byte 0..15, read as e4m3, is q 2^-9 (0..7 are its subnormals, 8..15
// its first binade), so one conversion instruction turns two codes into exact
// bf16 integers: seven instructions for eight weights.  A group's product runs
// on the matrix cores over the integers, and the scale and zero point enter
// once a group in fp32:
//   y += s (sum_j x q - z sum_j x),
// the second sum from a product with ones, shared by all columns of a wave.
//
// The codes are read in units of 128 along a row, 16 bytes a lane: the 16
// lanes of each quarter wave hold 16 columns, the four quarters the unit's
// four runs of 32.  An MFMA contracts one run at a time (a run never leaves
// its group), so the four registers are exchanged between the quarters, a 4 x 4
// transposition in four instructions, and X is read in its own order, 64
// contiguous bytes a row.
#include <algorithm>
#include <type_traits>

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

// Lanes 32..63 of a and lanes 0..31 of b change places.
__device__ __forceinline__ void swap_halves(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
// In each half wave, lanes 16..31 of a and lanes 0..15 of b change places.
__device__ __forceinline__ void swap_rows(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

// Quarter q of register j becomes quarter j of register q.
__device__ __forceinline__ void transpose4(u32x4_t& d) {
  uint32_t a = d[0], b = d[1], c = d[2], e = d[3];
  swap_halves(a, c);
  swap_halves(b, e);
  swap_rows(a, b);
  swap_rows(c, e);
  d = u32x4_t{a, b, c, e};
}

// Quarter r of w in all quarters of out[r] (RUNS = 1: w is the same in all
// quarters; RUNS = 2: in each pair).
template <int GROUPS>
__device__ __forceinline__ void spread(uint32_t w, uint32_t (&out)[GROUPS]) {
  if constexpr (GROUPS == 1) {
    out[0] = w;
  } else {
    uint32_t lo = w, hi = w;
    swap_halves(lo, hi);
    if constexpr (GROUPS == 2) {
      out[0] = lo;
      out[1] = hi;
    } else {
      out[0] = out[1] = lo;
      swap_rows(out[0], out[1]);
      out[2] = out[3] = hi;
      swap_rows(out[2], out[3]);
    }
  }
}

// One workgroup: 16 MB rows of X, 16 NB columns, the units of part blockIdx.z
// dealt to its W waves in turn (neighbouring waves read neighbouring 64-byte
// pieces of the same rows) and joined through LDS in wave order.  RUNS: runs of
// 32 a group.
template <int MB, int NB, int W, int RUNS>
__global__ __launch_bounds__(64 * W) void qweight_kernel(QweightArgs args) {
  (void)args;
  const QweightArgs& a = qw_kernarg();
  constexpr int GROUPS = 4 / RUNS;            // groups a unit
  constexpr int XD = MB == 4 && RUNS != 2 ? 2 : 4;   // runs of X held or on their way
  __shared__ float part[W][MB * 16][16 * NB + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n15 = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * (16 * NB), m0 = blockIdx.y * (MB * 16);
  const int per = (a.K + 127) / 128;          // units a shard
  const int gps = a.K / (32 * RUNS);          // groups a shard
  const int total = per * a.p;
  const int u0 = (int)((int64_t)total * blockIdx.z / gridDim.z), u1 = (int)((int64_t)total * (blockIdx.z + 1) / gridDim.z);
  // Rows and columns past the end repeat the last one and are not stored.
  uint32_t row[MB], col[NB];
#pragma unroll
  for (int i = 0; i < MB; ++i) row[i] = (uint32_t)min(m0 + i * 16 + n15, a.M - 1) * (uint32_t)a.K * 2u + 16u * q;
#pragma unroll
  for (int b = 0; b < NB; ++b) col[b] = (uint32_t)min(n0 + b * 16 + n15, a.N - 1);

  struct Unit {
    const char* x;          // the unit's first column of X
    const uint8_t* codes;
    const uint16_t* scales;
    const uint8_t* zeros;
    int runs;               // 4, or fewer at the end of a shard's rows
    uint32_t code_off;      // this lane's bytes within the unit
    uint32_t group;         // this lane's group
  };
  auto unit = [&](int u) {
    u = min(u, u1 - 1);
    const int k = __builtin_amdgcn_readfirstlane(u / per);
    const int i = __builtin_amdgcn_readfirstlane(u - k * per);
    Unit o;
    o.x = reinterpret_cast<const char*>(a.X[k]) + (int64_t)i * 256;
    o.codes = a.codes[k] + (int64_t)i * 64;
    o.scales = a.scales[k];
    o.zeros = a.zeros[k];
    o.runs = min(4, (a.K - i * 128) / 32);
    const int mine = min(q, o.runs - 1);
    o.code_off = 16u * mine;
    o.group = (uint32_t)((i * 4 + mine) / RUNS);
    return o;
  };
  auto load_codes = [&](const Unit& o, u32x4_t (&c)[NB], uint32_t (&sz)[NB]) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      c[b] = *reinterpret_cast<const u32x4_t*>(o.codes + (col[b] * (uint32_t)(a.K / 2) + o.code_off));
      const uint32_t at = col[b] * (uint32_t)gps + o.group;
      sz[b] = ((uint32_t)o.scales[at] << 16) | (o.zeros ? o.zeros[at] : 8u);
    }
  };
  auto load_x = [&](const Unit& o, int r, bf16x8_t (&x)[MB]) {
#pragma unroll
    for (int i = 0; i < MB; ++i)
      x[i] = *reinterpret_cast<const bf16x8_t*>(o.x + (row[i] + 64u * (uint32_t)min(r, o.runs - 1)));
  };

  f32x4_t acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[i][b] = f32x4_t{0, 0, 0, 0};
  bf16x8_t ones;
#pragma unroll
  for (int i = 0; i < 8; ++i) ones[i] = (__bf16)1.0f;

  if (u0 + wave < u1) {
    Unit cur = unit(u0 + wave), next = cur;
    u32x4_t c[NB], cn[NB];
    uint32_t sz[NB], sn[NB];
    bf16x8_t x[XD][MB];
    load_codes(cur, c, sz);
#pragma unroll
    for (int r = 0; r < XD; ++r) load_x(cur, r, x[r]);
    const f32x4_t none = {0, 0, 0, 0};
    // A unit's products: FULL when all its four runs are inside the row.
    auto products = [&](auto full) {
      constexpr bool FULL = decltype(full)::value;
      uint32_t g[NB][GROUPS];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        transpose4(c[b]);
        spread<GROUPS>(sz[b], g[b]);
      }
      auto refill = [&](int r) {
        if (r + XD < 4) load_x(cur, r + XD, x[r % XD]);
        else load_x(next, r + XD - 4, x[r % XD]);
      };
      auto join = [&](int b, int i, uint32_t w, const f32x4_t& dv, const f32x4_t& xv) {
        const float s = __uint_as_float(w & 0xffff0000u);
        const float z = -s * (float)(w & 0xffu);
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][b][v] = __builtin_fmaf(s, dv[v], __builtin_fmaf(z, xv[v], acc[i][b][v]));
      };
#pragma unroll
      for (int gi = 0; gi < GROUPS; ++gi) {
        if (!FULL && gi * RUNS >= cur.runs) {
#pragma unroll
          for (int r = gi * RUNS; r < (gi + 1) * RUNS; ++r) refill(r);
          continue;
        }
        f32x4_t xs[MB];
        if constexpr (RUNS <= 2) {
          // One column block at a time, so that few sums are live.
#pragma unroll
          for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int r = 0; r < RUNS; ++r)
              xs[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[(gi * RUNS + r) % XD][i], ones, r ? xs[i] : none, 0, 0, 0);
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            f32x4_t d[MB];
#pragma unroll
            for (int r = 0; r < RUNS; ++r) {
              const bf16x8_t w = unpack8(c[b][gi * RUNS + r]);
#pragma unroll
              for (int i = 0; i < MB; ++i)
                d[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[(gi * RUNS + r) % XD][i], w, r ? d[i] : none, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < MB; ++i) join(b, i, g[b][gi], d[i], xs[i]);
          }
#pragma unroll
          for (int r = gi * RUNS; r < (gi + 1) * RUNS; ++r) refill(r);
        } else {
          // One run at a time, so that X's registers are free for the next early.
          f32x4_t d[MB][NB];
#pragma unroll
          for (int r = 0; r < RUNS; ++r) {
#pragma unroll
            for (int i = 0; i < MB; ++i)
              xs[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[r % XD][i], ones, r ? xs[i] : none, 0, 0, 0);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              const bf16x8_t w = unpack8(c[b][r]);
#pragma unroll
              for (int i = 0; i < MB; ++i)
                d[i][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[r % XD][i], w, r ? d[i][b] : none, 0, 0, 0);
            }
            refill(r);
          }
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < MB; ++i) join(b, i, g[b][0], d[i][b], xs[i]);
        }
        // With 64 rows two groups' sums do not fit the registers side by side.
        if constexpr (MB == 4) __builtin_amdgcn_sched_barrier(0);
      }
    };
    for (int u = u0 + wave; u < u1; u += W) {
      next = unit(u + W);
      load_codes(next, cn, sn);
      if (cur.runs == 4) products(std::true_type{});
      else products(std::false_type{});
      cur = next;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        c[b] = cn[b];
        sz[b] = sn[b];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int v = 0; v < 4; ++v) part[wave][i * 16 + 4 * q + v][b * 16 + n15] = acc[i][b][v];
  __syncthreads();
  for (int e = threadIdx.x; e < MB * 16 * 16 * NB; e += 64 * W) {
    const int r = e / (16 * NB), c = e % (16 * NB);
    float y = part[0][r][c];
#pragma unroll
    for (int w = 1; w < W; ++w) y += part[w][r][c];
    const int m = m0 + r, n = n0 + c;
    if (m >= a.M || n >= a.N) continue;
    const int64_t o = (int64_t)m * a.N + n;
    if (gridDim.z > 1) {
      a.partial[(int64_t)blockIdx.z * a.M * a.N + o] = y;
      continue;
    }
    if (a.gelu) y = gelu_f32(y);
    if (a.out == OUT_F32) reinterpret_cast<float*>(a.Y)[o] = y;
    else reinterpret_cast<__bf16*>(a.Y)[o] = (__bf16)y;
  }
}

// The parts of a cut contraction, added in order.
__global__ __launch_bounds__(256) void qweight_sum_kernel(QweightArgs args) {
  (void)args;
  const QweightArgs& a = qw_kernarg();
  const int64_t n = (int64_t)a.M * a.N, e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= n) return;
  float y = 0.0f;
  for (int i = 0; i < a.splits; ++i) y += a.partial[(int64_t)i * n + e];
  if (a.gelu) y = gelu_f32(y);
  if (a.out == OUT_F32) reinterpret_cast<float*>(a.Y)[e] = y;
  else reinterpret_cast<__bf16*>(a.Y)[e] = (__bf16)y;
}

// Rows and columns of a workgroup, by M and N.
struct QwShape {
  int mb, nb;
};
static QwShape qw_shape(int64_t M, int64_t N) {
  const int mb = M <= 16 ? 1 : M <= 32 ? 2 : 4;
  const int64_t blocks = (N + 15) / 16 * ((M + 63) / 64);
  const int nb = mb == 4 || blocks >= 512 ? 2 : 1;
  return {mb, nb};
}

int qweight_splits(int p, int64_t M, int64_t K, int64_t N) {
  const QwShape t = qw_shape(M, N);
  const int64_t wgs = (N + 16 * t.nb - 1) / (16 * t.nb) * ((M + 63) / 64);
  const int64_t units = p * ((K + 127) / 128);
  if (t.mb < 4) return 1;
  return (int)std::max<int64_t>(1, std::min<int64_t>(256 / wgs, units / 32));
}

template <int MB, int NB, int W>
static void launch_qw(const QweightArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.N + 16 * NB - 1) / (16 * NB)), (unsigned)((a.M + 16 * MB - 1) / (16 * MB)), (unsigned)a.splits);
  if (a.group == 32) hipLaunchKernelGGL((qweight_kernel<MB, NB, W, 1>), grid, dim3(64 * W), 0, s, a);
  else if (a.group == 64) hipLaunchKernelGGL((qweight_kernel<MB, NB, W, 2>), grid, dim3(64 * W), 0, s, a);
  else hipLaunchKernelGGL((qweight_kernel<MB, NB, W, 4>), grid, dim3(64 * W), 0, s, a);
}

hipError_t launch_qweight(const QweightArgs& a, hipStream_t s) {
  const QwShape t = qw_shape(a.M, a.N);
  if (t.mb == 1) {
    if (t.nb == 1) launch_qw<1, 1, 16>(a, s);
    else launch_qw<1, 2, 8>(a, s);
  } else if (t.mb == 2) {
    if (t.nb == 1) launch_qw<2, 1, 8>(a, s);
    else launch_qw<2, 2, 8>(a, s);
  } else {
    launch_qw<4, 2, 8>(a, s);
  }
  if (a.splits > 1) {
    const int64_t n = (int64_t)a.M * a.N;
    hipLaunchKernelGGL(qweight_sum_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace tpf
