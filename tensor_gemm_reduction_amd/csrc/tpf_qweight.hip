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
// Where x is infinite both sums are, and their difference is NaN though the
// definition, x (q - z) s, may be infinite; where x is near the largest float,
// x q can pass it though x (q - z) s does not.  Neither leaves a finite sum, so
// an element whose sum is not finite is summed again, term by term.
//
// The codes are read in units of 128 along a row, 16 bytes a lane: the 16
// lanes of each quarter wave hold 16 columns, the four quarters the unit's
// four runs of 32.  An MFMA contracts one run at a time (a run never leaves
// its group), so the four registers are exchanged between the quarters, a 4 x 4
// transposition in four instructions, and X is read in its own order, 64
// contiguous bytes a row.
#include <algorithm>

#include "tpf_block.hpp"
#include "tpf_gemm.hpp"

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

// ---------------------------------------------------------------------------
// Units of 128 codes, numbered through the shards.
// ---------------------------------------------------------------------------
struct UnitPos {
  int k, i;                 // shard, unit within its rows
};
__device__ __forceinline__ UnitPos unit_at(const QweightArgs& a, int u, int per) {
  const int k = min(__builtin_amdgcn_readfirstlane(u / per), a.p - 1);
  return UnitPos{k, __builtin_amdgcn_readfirstlane(u - k * per)};
}
// The next unit; true where it is in another shard.
__device__ __forceinline__ bool advance(UnitPos& o, const QweightArgs& a, int per) {
  if (++o.i != per || o.k + 1 == a.p) return false;
  o.i = 0;
  ++o.k;
  return true;
}

// ORed into an offset (below 2^31): leaves it or puts it outside any buffer.
__device__ __forceinline__ uint32_t outside(bool in) { return in ? 0u : kOOB; }

// A wave's stream of codes of 16 NB columns, one unit after the other.  Loads
// outside the part, a row or the columns go to an offset outside the buffer:
// they return zero without touching memory.
template <int NB>
struct CodeStream {
  UnitPos at;
  int left;                       // units before the part's end
  const uint8_t* codes;           // the shard's
  uint32_t code0[NB];
  int per, q;

  __device__ __forceinline__ void init(const QweightArgs& a, int u, int count, int n0, int lane) {
    per = (a.K + 127) / 128;
    at = unit_at(a, u, per);
    codes = a.codes[at.k];
    left = count;
    q = lane >> 4;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int n = n0 + b * 16 + (lane & 15);
      code0[b] = n < a.N ? (uint32_t)n * (uint32_t)(a.K / 2) + 16u * q : kOOB;
    }
  }
  __device__ __forceinline__ void load(const QweightArgs& a, u32x4_t (&c)[NB]) {
    const auto rc = make_rsrc(codes, (int64_t)a.N * (a.K / 2));
    const uint32_t out = outside((left > 0) & ((at.i * 4 + q) * 32 < a.K));
#pragma unroll
    for (int b = 0; b < NB; ++b)
      c[b] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                             rc, (int)((code0[b] + 64u * (uint32_t)at.i) | out), 0, 0));
    if (advance(at, a, per)) codes = a.codes[at.k];
    --left;
  }
};

// Scales and zero points of a wave's next kBlockUnits units of 16 NB columns.
// An operand needs one of each per lane and group, two bytes here and there of
// 16 rows: loaded so, they cost the cache four times the codes' lines.  A block
// is loaded along the rows instead (neighbouring lanes neighbouring groups),
// one block ahead, and laid out in the wave's own LDS by group and column.
// Past the part's or a row's end the scale is zero and adds nothing.
constexpr int kBlockUnits = 4;
template <int NB, int RUNS>
struct ScaleStream {
  static constexpr int GROUPS = 4 / RUNS, GB = kBlockUnits * GROUPS;   // groups a block
  static constexpr int COLS = 16 * NB, PITCH = COLS + 1, EACH = COLS * GB / 64;
  static constexpr int WORDS = GB * PITCH;
  UnitPos at;
  int left, per, gps;
  const uint16_t* scales;
  const uint8_t* zeros;
  uint32_t s[EACH], z[EACH];

  __device__ __forceinline__ void init(const QweightArgs& a, int u, int count) {
    per = (a.K + 127) / 128;
    gps = a.K / (32 * RUNS);
    at = unit_at(a, u, per);
    left = count;
    shard(a);
  }
  __device__ __forceinline__ void shard(const QweightArgs& a) {
    scales = a.scales[at.k];
    zeros = a.zeros[at.k];
  }
  __device__ __forceinline__ void load(const QweightArgs& a, int n0, int lane) {
    const int j = lane % GB, unit = j / GROUPS;
    const bool mine = unit < left;
    if (at.i + kBlockUnits <= per || at.k + 1 == a.p) {   // one shard's
      const auto rs = make_rsrc(scales, (int64_t)a.N * gps * 2);
      const auto rz = make_rsrc(zeros, zeros ? (int64_t)a.N * gps : 0);
      const int g = at.i * GROUPS + j;
      const uint32_t out = outside(mine & (g < gps));
#pragma unroll
      for (int e = 0; e < EACH; ++e) {
        const int n = n0 + (e * 64 + lane) / GB;
        const uint32_t o = (uint32_t)n * (uint32_t)gps + (uint32_t)g, skip = out | outside(n < a.N);
        s[e] = __builtin_amdgcn_raw_buffer_load_b16(rs, (int)((o * 2u) | skip), 0, 0);
        z[e] = __builtin_amdgcn_raw_buffer_load_b8(rz, (int)(o | skip), 0, 0);
      }
    } else {
      int k = at.k, i = at.i + unit;
      while (i >= per && k + 1 < a.p) {
        i -= per;
        ++k;
      }
      const int g = i * GROUPS + j % GROUPS;
      const uint16_t* sk = a.scales[k];
      const uint8_t* zk = a.zeros[k];
#pragma unroll
      for (int e = 0; e < EACH; ++e) {
        const int n = n0 + (e * 64 + lane) / GB;
        const bool in = mine && g < gps && n < a.N;
        const uint32_t o = (uint32_t)n * (uint32_t)gps + (uint32_t)g;
        s[e] = in ? sk[o] : 0;
        z[e] = in && zk ? zk[o] : 0;
      }
    }
    bool moved = false;
#pragma unroll
    for (int u = 0; u < kBlockUnits; ++u) moved |= advance(at, a, per);
    if (moved) shard(a);
    left -= kBlockUnits;
  }
  // Leaves the loaded block in `lds` for its wave; `eight` is the zero point of
  // weights that have none.  A wave's LDS accesses are carried out in order, so
  // its lanes need no barrier between them, only the compiler's order.
  __device__ __forceinline__ void publish(uint32_t* lds, uint32_t eight, int lane) const {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int e = 0; e < EACH; ++e) lds[(lane % GB) * PITCH + (e * 64 + lane) / GB] = (s[e] << 16) | z[e] | eight;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
};

__device__ __forceinline__ f32x4_t qw_mfma(const bf16x8_t& x, const bf16x8_t& w, const f32x4_t& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w, c, 0, 0, 0);
}
// y += s (d - z xs) for a scale and zero point packed in w.
__device__ __forceinline__ void qw_join(f32x4_t& y, uint32_t w, const f32x4_t& d, const f32x4_t& xs) {
  const float s = __uint_as_float(w & 0xffff0000u);
  const float z = -s * (float)(w & 0xffu);
#pragma unroll
  for (int v = 0; v < 4; ++v) y[v] = __builtin_fmaf(s, d[v], __builtin_fmaf(z, xs[v], y[v]));
  asm volatile("" : "+v"(y));   // here: left to itself the compiler sinks the sums of several units and spills
}
__device__ __forceinline__ bf16x8_t bf16_ones() {
  bf16x8_t o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = (__bf16)1.0f;
  return o;
}
// One element over units u0 .. u1 - 1 by the definition; (q - z) s is exact in
// fp32.  Rare and bound by latency: one infinity in 16 rows over 8 shards of 1024
// makes 22 us 290; a NaN at the end of each of 64 rows over 8 of 3584 makes 69 us
// 5.8 ms.
__device__ __forceinline__ float qw_term_by_term(const QweightArgs& a, int m, int n, int u0, int u1) {
  const int per = (a.K + 127) / 128, gps = a.K / a.group;
  float y = 0.0f;
#pragma unroll 1
  for (int u = u0; u < u1; ++u) {
    const int k = u / per, first = (u - k * per) * 128, end = min(first + 128, a.K);
    const uint8_t* codes = a.codes[k] + (int64_t)n * (a.K / 2);
    const __bf16* x = a.X[k] + (int64_t)m * a.K;
#pragma unroll 1
    for (int j = first; j < end; j += 8) {
      const int64_t g = (int64_t)n * gps + j / a.group;
      const float s = __uint_as_float((uint32_t)a.scales[k][g] << 16);
      const float z = a.zeros[k] ? (float)a.zeros[k][g] : 8.0f;
      const uint32_t c = *reinterpret_cast<const uint32_t*>(codes + j / 2);
      const bf16x8_t xv = *reinterpret_cast<const bf16x8_t*>(x + j);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float q = (float)((c >> (8 * (i & 3) + (i & 4))) & 15u);
        y = __builtin_fmaf((float)xv[i], (q - z) * s, y);
      }
    }
    if (y != y) return y;   // and stays so
  }
  return y;
}

__device__ __forceinline__ void qw_store(const QweightArgs& a, int m, int n, float y, int u0, int u1) {
  if (m >= a.M || n >= a.N) return;
  if (!(fabsf(y) <= 3.402823466e38f)) y = qw_term_by_term(a, m, n, u0, u1);
  const int64_t o = (int64_t)m * a.N + n;
  if (gridDim.z > 1) {
    a.partial[(int64_t)blockIdx.z * a.M * a.N + o] = y;
    return;
  }
  if (a.gelu) y = gelu_f32(y);
  if (a.out == OUT_F32) reinterpret_cast<float*>(a.Y)[o] = y;
  else reinterpret_cast<__bf16*>(a.Y)[o] = (__bf16)y;
}

// ---------------------------------------------------------------------------
// Up to 16 rows: a workgroup has 16 NB columns, each of its W waves a
// contiguous share of the units, joined through LDS in wave order.  A wave
// keeps D units of codes and X on their way.
//
// Bound by the cache accesses, not by the bytes or the arithmetic: a read of
// the codes alone in this pattern takes 6.6 us for 8192 x 8192, the same kernel
// without X's loads 3 us less, without the unpacking the same.  One row, groups
// of 128: 11.9 us a call (2.9 TB/s); 16 rows over 8 shards of 1024, groups of 32
// with zero points: 17.9 us (6.5 more with a scale and zero point loaded per lane),
// in a call of 21.5.
// ---------------------------------------------------------------------------
template <int NB, int W, int D, int RUNS>
__global__ __launch_bounds__(64 * W) void qweight_few_kernel(QweightArgs args) {
  (void)args;
  const QweightArgs& a = qw_kernarg();
  using Scales = ScaleStream<NB, RUNS>;
  constexpr int GROUPS = Scales::GROUPS, JOIN = 16 * (16 * NB + 1);
  static_assert(kBlockUnits % D == 0, "slots of a block");
  __shared__ uint32_t lds[W][Scales::WORDS > JOIN ? Scales::WORDS : JOIN];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n15 = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * (16 * NB);
  const int per = (a.K + 127) / 128, total = per * a.p;
  const int u0 = (int)((int64_t)total * wave / W), n = (int)((int64_t)total * (wave + 1) / W) - u0;

  f32x4_t acc[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) acc[b] = f32x4_t{0, 0, 0, 0};
  if (n > 0) {
    Scales sc;
    sc.init(a, u0, n);
    sc.load(a, n0, lane);
    CodeStream<NB> cs;
    cs.init(a, u0, n, n0, lane);
    u32x4_t c[D][NB];
    bf16x8_t x[D][4];
    const uint32_t eight = a.zeros[0] ? 0u : 8u;
    UnitPos xp = cs.at;
    const __bf16* xk = a.X[xp.k];
    int xleft = n;
    const uint32_t x0 = n15 < a.M ? (uint32_t)n15 * (uint32_t)a.K * 2u + 16u * q : kOOB;
    auto load_x = [&](bf16x8_t (&o)[4]) {
      const auto rx = make_rsrc(xk, (int64_t)a.M * a.K * 2);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t out = outside((xleft > 0) & ((xp.i * 4 + r) * 32 < a.K));
        o[r] = __builtin_bit_cast(bf16x8_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                rx, (int)((x0 + 256u * (uint32_t)xp.i + 64u * r) | out), 0, 0));
      }
      if (advance(xp, a, per)) xk = a.X[xp.k];
      --xleft;
    };
#pragma unroll
    for (int d = 0; d < D; ++d) {
      cs.load(a, c[d]);
      load_x(x[d]);
    }
    const bf16x8_t ones = bf16_ones();
    const f32x4_t none = {0, 0, 0, 0};
    for (int u = 0; u < n; u += kBlockUnits) {
      sc.publish(lds[wave], eight, lane);
      sc.load(a, n0, lane);
#pragma unroll
      for (int v = 0; v < kBlockUnits; ++v) {
        const int d = v % D;
#pragma unroll
        for (int b = 0; b < NB; ++b) transpose4(c[d][b]);
#pragma unroll
        for (int gi = 0; gi < GROUPS; ++gi) {
          f32x4_t xs, dv[NB];
#pragma unroll
          for (int r = 0; r < RUNS; ++r) {
            xs = qw_mfma(x[d][gi * RUNS + r], ones, r ? xs : none);
#pragma unroll
            for (int b = 0; b < NB; ++b)
              dv[b] = qw_mfma(x[d][gi * RUNS + r], unpack8(c[d][b][gi * RUNS + r]), r ? dv[b] : none);
          }
#pragma unroll
          for (int b = 0; b < NB; ++b)
            qw_join(acc[b], lds[wave][(v * GROUPS + gi) * Scales::PITCH + b * 16 + n15], dv[b], xs);
          // Two groups at a time: all four would take the registers of the loads on their way.
          if (GROUPS == 4 && gi == 1) __builtin_amdgcn_sched_barrier(0);
        }
        cs.load(a, c[d]);
        load_x(x[d]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  __syncthreads();
  float (*part)[JOIN] = reinterpret_cast<float (*)[JOIN]>(&lds[0][0]);
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int v = 0; v < 4; ++v) part[wave][(4 * q + v) * (16 * NB + 1) + b * 16 + n15] = acc[b][v];
  __syncthreads();
  for (int e = threadIdx.x; e < 16 * 16 * NB; e += 64 * W) {
    const int r = e / (16 * NB), col = e % (16 * NB);
    float y = part[0][r * (16 * NB + 1) + col];
#pragma unroll
    for (int w = 1; w < W; ++w) y += part[w][r * (16 * NB + 1) + col];
    qw_store(a, r, n0 + col, y, 0, total);
  }
}

// ---------------------------------------------------------------------------
// More rows: a workgroup has 16 MB rows and 128 columns, its eight waves four
// column blocks of 32 times the two halves of the part's units.  X would be
// read once for every 32 columns from the cache, eight times the codes' bytes
// at 64 rows, so a unit's X (rows x 256 bytes) is staged in LDS, two slots, for
// the four waves that need it; its 16-byte chunks are swizzled by the row, so
// that the 16 rows of an operand read hit every bank.
//
// 64 rows, 8 shards of 3584 x 8192, groups of 64: 67 us a call, 5 of them for the
// sum of the four parts, where one 32-column block a wave with X from the cache
// took 141; bound by the waits between a unit's operand reads, products and sums at
// two waves a SIMD (four waves' registers do not hold 64 rows: 266 us).
// ---------------------------------------------------------------------------
template <int MB, int RUNS>
__global__ __launch_bounds__(512) void qweight_rows_kernel(QweightArgs args) {
  (void)args;
  const QweightArgs& a = qw_kernarg();
  using Scales = ScaleStream<2, RUNS>;
  constexpr int NB = 2, D = 2, GROUPS = Scales::GROUPS;
  __shared__ __attribute__((aligned(1024))) char lds[2][2][MB * 16 * 256];
  __shared__ uint32_t szs[8][Scales::WORDS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n15 = lane & 15, q = lane >> 4;
  const int half = wave >> 2, cw = wave & 3;
  const int n0 = blockIdx.x * 128 + cw * 32, m0 = blockIdx.y * (MB * 16);
  const int per = (a.K + 127) / 128, total = per * a.p;
  const int u0 = (int)((int64_t)total * blockIdx.z / gridDim.z), u1 = (int)((int64_t)total * (blockIdx.z + 1) / gridDim.z);
  const int steps = (u1 - u0 + 1) / 2;                  // of the first half; the other may have one less
  const int first = u0 + half * steps, count = half ? u1 - u0 - steps : steps;

  // This wave's quarter of its half's X: 4 MB rows, 16 chunks each.
  UnitPos xp = unit_at(a, min(first, total - 1), per);
  const __bf16* xk = a.X[xp.k];
  int xleft = count;
  uint32_t x0[MB], xd[MB];
  const int chunk = lane & 15;
#pragma unroll
  for (int j = 0; j < MB; ++j) {
    const int row = cw * 4 * MB + j * 4 + (lane >> 4), m = m0 + row;
    x0[j] = m < a.M ? (uint32_t)m * (uint32_t)a.K * 2u + 16u * chunk : kOOB;
    xd[j] = (uint32_t)row * 256u + 16u * (uint32_t)(chunk ^ (row & 15));
  }
  u32x4_t xr[MB];
  auto load_x = [&]() {
    const auto rx = make_rsrc(xk, (int64_t)a.M * a.K * 2);
    const uint32_t out = outside((xleft > 0) & (xp.i * 128 + chunk * 8 < a.K));
#pragma unroll
    for (int j = 0; j < MB; ++j)
      xr[j] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                              rx, (int)((x0[j] + 256u * (uint32_t)xp.i) | out), 0, 0));
    if (advance(xp, a, per)) xk = a.X[xp.k];
    --xleft;
  };
  auto store_x = [&](int slot) {
#pragma unroll
    for (int j = 0; j < MB; ++j) *reinterpret_cast<u32x4_t*>(lds[slot][half] + xd[j]) = xr[j];
  };

  f32x4_t acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[i][b] = f32x4_t{0, 0, 0, 0};
  Scales sc;
  sc.init(a, min(first, total - 1), count);
  sc.load(a, n0, lane);
  CodeStream<NB> cs;
  cs.init(a, min(first, total - 1), count, n0, lane);
  u32x4_t c[D][NB];
  const uint32_t eight = a.zeros[0] ? 0u : 8u;
  load_x();
#pragma unroll
  for (int d = 0; d < D; ++d) cs.load(a, c[d]);
  store_x(0);
  load_x();
  lds_barrier();
  const bf16x8_t ones = bf16_ones();
  const f32x4_t none = {0, 0, 0, 0};
  const uint32_t xrow = (uint32_t)n15 * 256u;
  for (int t = 0; t < steps; t += kBlockUnits) {
    sc.publish(szs[wave], eight, lane);
    sc.load(a, n0, lane);
#pragma unroll
    for (int v = 0; v < kBlockUnits; ++v) {
      const int d = v % D, slot = v % 2;
      // The other slot was left by every wave before the last barrier.
      store_x(slot ^ 1);
      load_x();
#pragma unroll
      for (int b = 0; b < NB; ++b) transpose4(c[d][b]);
      const char* xl = lds[slot][half] + xrow;
#pragma unroll
      for (int gi = 0; gi < GROUPS; ++gi) {
        f32x4_t xs[MB], dv[MB][NB];
#pragma unroll
        for (int r = 0; r < RUNS; ++r) {
          const int run = gi * RUNS + r;
          bf16x8_t w[NB];
#pragma unroll
          for (int b = 0; b < NB; ++b) w[b] = unpack8(c[d][b][run]);
#pragma unroll
          for (int i = 0; i < MB; ++i) {
            const bf16x8_t x = *reinterpret_cast<const bf16x8_t*>(xl + i * 4096 + 16 * ((run * 4 + q) ^ n15));
            xs[i] = qw_mfma(x, ones, r ? xs[i] : none);
#pragma unroll
            for (int b = 0; b < NB; ++b) dv[i][b] = qw_mfma(x, w[b], r ? dv[i][b] : none);
          }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint32_t w = szs[wave][(v * GROUPS + gi) * Scales::PITCH + b * 16 + n15];
#pragma unroll
          for (int i = 0; i < MB; ++i) qw_join(acc[i][b], w, dv[i][b], xs[i]);
        }
        // With 64 rows two groups' sums do not fit the registers side by side.
        if (MB == 4 && GROUPS > 1) __builtin_amdgcn_sched_barrier(0);
      }
      cs.load(a, c[d]);
      lds_barrier();
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // Both halves' sums through LDS, the first half's plus the second's.
  __syncthreads();
  float* join = reinterpret_cast<float*>(lds);
  constexpr int ROWS = MB * 16;
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (half == 1) join[(i * 16 + 4 * q + v) * 128 + cw * 32 + b * 16 + n15] = acc[i][b][v];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (half == 0) join[(i * 16 + 4 * q + v) * 128 + cw * 32 + b * 16 + n15] += acc[i][b][v];
  __syncthreads();
#pragma unroll 1
  for (int e = threadIdx.x; e < ROWS * 128; e += 512) 
    qw_store(a, m0 + e / 128, blockIdx.x * 128 + e % 128, join[e], u0, u1);
}

// The parts of a cut contraction, added in order, V elements a thread.
template <int V>
__global__ __launch_bounds__(256) void qweight_sum_kernel(QweightArgs args) {
  (void)args;
  const QweightArgs& a = qw_kernarg();
  const int64_t n = (int64_t)a.M * a.N, e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V;
  if (e >= n) return;
  typedef float vec_t __attribute__((ext_vector_type(V)));
  vec_t y = 0.0f;
#pragma unroll 4
  for (int i = 0; i < a.splits; ++i) y += *reinterpret_cast<const vec_t*>(a.partial + (int64_t)i * n + e);
  if (a.gelu) {
#pragma unroll
    for (int v = 0; v < V; ++v) y[v] = gelu_f32(y[v]);
  }
  if (a.out == OUT_F32) {
    *reinterpret_cast<vec_t*>(reinterpret_cast<float*>(a.Y) + e) = y;
  } else {
    typedef __bf16 out_t __attribute__((ext_vector_type(V)));
    out_t o;
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = (__bf16)y[v];
    *reinterpret_cast<out_t*>(reinterpret_cast<__bf16*>(a.Y) + e) = o;
  }
}

// Columns of a workgroup of the kernel for few rows: 16 while that leaves at most
// one workgroup a compute unit (4096 columns: 9.2 us against 11.1 with 32), else 32,
// which read X half as often (16384 columns, 16 rows: 23.0 us with 16, 16.2 with 32).
static bool qw_few_wide(int64_t N) { return N > 16 * 256; }

// The kernel for more rows cuts the units into parts until every compute unit
// has a workgroup, of at least four units a half (one part of 8 x 3584 x 8192
// takes 203 us, two 106, four 64, eight 75 and twice the partial sums).
int qweight_splits(int p, int64_t M, int64_t K, int64_t N) {
  if (M <= 16) return 1;
  const int64_t wgs = (N + 127) / 128 * ((M + 63) / 64);
  const int64_t steps = (p * ((K + 127) / 128) + 1) / 2;
  return (int)std::max<int64_t>(1, std::min<int64_t>(256 / wgs, steps / 4));
}

template <int NB, int W, int D>
static void launch_qw_few(const QweightArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.N + 16 * NB - 1) / (16 * NB)));
  if (a.group == 32) hipLaunchKernelGGL((qweight_few_kernel<NB, W, D, 1>), grid, dim3(64 * W), 0, s, a);
  else if (a.group == 64) hipLaunchKernelGGL((qweight_few_kernel<NB, W, D, 2>), grid, dim3(64 * W), 0, s, a);
  else hipLaunchKernelGGL((qweight_few_kernel<NB, W, D, 4>), grid, dim3(64 * W), 0, s, a);
}

template <int MB>
static void launch_qw_rows(const QweightArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.N + 127) / 128), (unsigned)((a.M + 16 * MB - 1) / (16 * MB)), (unsigned)a.splits);
  if (a.group == 32) hipLaunchKernelGGL((qweight_rows_kernel<MB, 1>), grid, dim3(512), 0, s, a);
  else if (a.group == 64) hipLaunchKernelGGL((qweight_rows_kernel<MB, 2>), grid, dim3(512), 0, s, a);
  else hipLaunchKernelGGL((qweight_rows_kernel<MB, 4>), grid, dim3(512), 0, s, a);
}

hipError_t launch_qweight(const QweightArgs& a, hipStream_t s) {
  if (a.M <= 16) {
    if (qw_few_wide(a.N)) launch_qw_few<2, 8, 1>(a, s);
    else launch_qw_few<1, 8, 2>(a, s);
  } else if (a.M <= 32) {
    launch_qw_rows<2>(a, s);
  } else {
    launch_qw_rows<4>(a, s);
  }
  if (a.splits > 1) {
    const int64_t n = (int64_t)a.M * a.N;
    if (n % 4 == 0) hipLaunchKernelGGL(qweight_sum_kernel<4>, dim3((unsigned)((n + 1023) / 1024)), dim3(256), 0, s, a);
    else hipLaunchKernelGGL(qweight_sum_kernel<1>, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace tpf
