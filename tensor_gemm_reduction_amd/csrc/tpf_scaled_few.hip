// Products of 8-bit operands for a few rows (a decode step): the weights are
// streamed once from memory into registers.
//
// A workgroup owns 16 TM rows and 16 TN columns of the result; its W waves take
// the blocks of 128 along the contraction (and over the shards) in turn, each U of
// its own ahead, and their sums are joined in LDS in the order of the waves.
// A lane's 32 codes of a block are two 16-byte loads of one weight row, so four
// lanes read whole 64-byte halves of its 128.  Codes become bf16 (exact) and go to
// the bf16 instructions, whose sums keep fp32's bits: next to memory the
// conversions are small (192 cycles of a SIMD's 1260 that a block's 4 KB take at
// 8 TB/s).  16 x 8 x 1024 x 8192: 15.7 us, 4.3 TB/s, one round of workgroups whose
// streams start and end together; 16 tokens to 8 of 64 experts, K 4096, N 1024: 46
// us, 5.1 TB/s.
#include <algorithm>
#include <type_traits>

#include "tpf_gemm.hpp"
#include "tpf_scaled.hpp"
#include "tpf_scaled_device.hpp"

namespace tpf {
namespace {

// U: loads of about 8 KB a wave in flight, as the registers allow.
constexpr int few_ahead(int TM) { return TM == 1 ? 4 : TM == 2 ? 3 : 2; }

template <int TM, int TN>
struct FewBlock {
  i32x8_t x[TM], w[TN];
  int xs[TM];
  float ws;
};

template <int TM, int TN, int W, int EXPERTS, int WS, int OUT>
__global__ __launch_bounds__(64 * W) void scaled_few_kernel(ScaledArgs args) {
  (void)args;
  const ScaledArgs& a = *(const ScaledArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  __shared__ f32x4_t part[W][TM * TN][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int unit = blockIdx.x / a.tiles_n, n0 = (int)(blockIdx.x - unit * a.tiles_n) * 16 * TN;
  int e = 0, row0 = unit * 16 * TM, rows = min(16 * TM, a.M - row0);
  const int kbs = (a.K + kScaleBlock - 1) / kScaleBlock;
  int blocks = a.p * kbs;
  if constexpr (EXPERTS) {
    const RowTile t = expert_tile<16 * TM>(a.offsets, a.E, a.M, unit, lane);
    if (t.rows <= 0) return;
    row0 = t.row0;
    rows = t.rows;
    e = t.e;
    if (e == a.E) e = 0, blocks = 0;                 // rows of no expert: zeros
  }
  // This lane's rows of both operands, as offsets from the first (of gathered rows: from the first token); rows and
  // columns past the last repeat it and are not stored.
  constexpr int U = few_ahead(TM);
  const int r16 = lane & 15, chunk = 16 * (lane >> 4);
  const bool gather = EXPERTS && a.top;
  uint32_t x_at[TM], w_at[TN], xs_at[TM];
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    int r = min(m * 16 + r16, rows - 1);
    if (gather) r = min(max(a.src[row0 + r], 0) / a.top, a.xrows - 1);
    x_at[m] = (uint32_t)r * (uint32_t)a.K + chunk;
    xs_at[m] = (uint32_t)r * (uint32_t)a.xsw;
  }
#pragma unroll
  for (int n = 0; n < TN; ++n) w_at[n] = (uint32_t)min(n * 16 + r16, a.N - 1 - n0) * (uint32_t)a.K + chunk;
  const int64_t x_row = gather ? 0 : row0, w_row = (int64_t)e * a.N + n0;
  const int64_t x_bytes = (int64_t)(gather ? a.xrows : rows) * a.K, w_bytes = (int64_t)min(16 * TN, a.N - n0) * a.K;
  const int64_t ws_at = ((int64_t)e * ((a.N + kScaleBlock - 1) / kScaleBlock) + n0 / kScaleBlock) * a.wsw;

  // The next block to be loaded.  Tiles start at blocks of their own, W + 1 apart: from the same one, or from the few
  // that steps of W leave of a power of two, rows of such a length would all be read from the same few memory channels
  // (8192 x 8192, 1 row: steps of W 21.2 us, of W + 1 15.1; 4096 x 8192 11.2 and 9.0; 28672 x 2048, four waves, 14.2
  // and 15.1).
  const int b0 = blocks ? (int)((uint32_t)(wave + (n0 / (16 * TN) + unit) * (W + 1)) % (uint32_t)blocks) : 0;
  int s = b0 / kbs, kb = b0 - s * kbs;
  const auto load = [&](FewBlock<TM, TN>& b) {
    const int k0 = kb * kScaleBlock;
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x[s] + x_row * a.K, x_bytes), rw = make_rsrc(a.w[s] + w_row * a.K, w_bytes);
    // codes past the end of a row read as zeros
    const bool tail = k0 + kScaleBlock > a.K;
    const uint32_t lo = tail && k0 + chunk >= a.K ? kOOB : 0, hi = tail && k0 + chunk + 64 >= a.K ? kOOB : 0;
    const auto codes = [&](const __amdgpu_buffer_rsrc_t& r, uint32_t at) {
      const i32x4_t c0 = __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)(at | lo), k0, 0));
      const i32x4_t c1 = __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)((at + 64) | hi), k0, 0));
      return __builtin_shufflevector(c0, c1, 0, 1, 2, 3, 4, 5, 6, 7);
    };
#pragma unroll
    for (int n = 0; n < TN; ++n) b.w[n] = codes(rw, w_at[n]);
#pragma unroll
    for (int m = 0; m < TM; ++m) b.x[m] = codes(rx, x_at[m]);
    const uint8_t* xs = a.xs[s] + x_row * a.xsw + kb;
#pragma unroll
    for (int m = 0; m < TM; ++m) b.xs[m] = xs[xs_at[m]];
    if constexpr (WS == WS_F32) b.ws = reinterpret_cast<const float*>(a.ws[s])[ws_at + kb];
    else b.ws = exp_byte(a.ws[s][ws_at + kb]);
    kb += W;
    while (kb >= kbs) {
      kb -= kbs;
      if (++s == a.p) s = 0;
    }
  };
  f32x4_t acc[TM][TN];
#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int n = 0; n < TN; ++n) acc[m][n] = f32x4_t{0, 0, 0, 0};
  const int mine = blocks > wave ? (blocks - wave + W - 1) / W : 0;
  FewBlock<TM, TN> ring[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u < mine) load(ring[u]);
  for (int i = 0; i < mine; i += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u >= mine) break;
      ScFine w[TN];
#pragma unroll
      for (int n = 0; n < TN; ++n) w[n] = sc_fine(ring[u].w[n]);
#pragma unroll
      for (int m = 0; m < TM; ++m) {
        const ScFine x = sc_fine(ring[u].x[m]);
        const float f = exp_byte(ring[u].xs[m]) * ring[u].ws;
#pragma unroll
        for (int n = 0; n < TN; ++n) {
          const f32x4_t v = sc_mfma_fine(w[n], x);
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[m][n][q] = __builtin_fmaf(v[q], f, acc[m][n][q]);
        }
      }
      if (i + u + U < mine) load(ring[u]);
    }
  }
#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int n = 0; n < TN; ++n) part[wave][m * TN + n][lane] = acc[m][n];
  __syncthreads();
  for (int i = threadIdx.x; i < TM * TN * 64; i += 64 * W) {
    const int t = i >> 6, l = i & 63;
    f32x4_t v = part[0][t][l];
#pragma unroll
    for (int w = 1; w < W; ++w) v += part[w][t][l];
    const int row = t / TN * 16 + (l & 15), col = n0 + t % TN * 16 + 4 * (l >> 4);
    if (row >= rows || col >= a.N) continue;
    if (a.gelu) v = sc_gelu<OUT>(v);
    const int64_t at = (int64_t)(row0 + row) * a.N + col;
    if constexpr (OUT == OUT_F32)
      *reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(a.y[0]) + at) = v;
    else
      *reinterpret_cast<u32x2_t*>(reinterpret_cast<uint16_t*>(a.y[0]) + at) =
          u32x2_t{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
  }
}

template <int TM, int TN, int W, int EXPERTS, int WS>
hipError_t launch_few(ScaledArgs a, hipStream_t s) {
  a.tiles_n = (a.N + 16 * TN - 1) / (16 * TN);
  a.tiles_m = EXPERTS ? expert_tiles(a.M, a.E, 16 * TM) : (a.M + 16 * TM - 1) / (16 * TM);
  if (a.out == OUT_F32)
    hipLaunchKernelGGL((scaled_few_kernel<TM, TN, W, EXPERTS, WS, OUT_F32>), dim3(a.tiles_n * a.tiles_m), dim3(64 * W),
                       0, s, a);
  else
    hipLaunchKernelGGL((scaled_few_kernel<TM, TN, W, EXPERTS, WS, OUT_BF16>), dim3(a.tiles_n * a.tiles_m), dim3(64 * W),
                       0, s, a);
  return hipGetLastError();
}

// Eight waves a workgroup where each compute unit has one at most, four where they
// are more: three then share a compute unit, and one's start and end lie beside the
// others' streams.  us, four and eight waves, 1 row and 16: 8192 x 8192 (256
// workgroups) 20.3 and 15.1, 21.7 and 17.1; 8192 x 8 x 1024 19.5 and 14.9, 20.3 and
// 16.2; 7168 x 7168 17.2 and 12.7, 18.2 and 14.8; 8192 x 4096 10.4 and 9.0, 11.3 and
// 10.4; more of them: 10240 x 8192 24.7 and 25.0, 30.2 and 31.0; 12288 x 4096 13.4 and
// 15.1, 17.3 and 18.0; 16384 x 8 x 1024 26.6 and 27.5, 29.8 and 30.7; 16384 x 1024 5.8
// and 6.7, 6.1 and 7.2; 28672 x 8192 54.1 and 50.3, 59.1 and 60.7.  From a block a wave
// on: 4096 x 1024 (8 blocks) 4.2 and 4.1, 4.7 and 4.5; 4096 x 512 (4) 2.9 and 3.0, 3.1
// and 3.2.  Experts' workgroups are more than the compute units as a rule: 16 tokens to
// 8 of 64, K 4096, N 1024: 49, with eight waves 62.
template <int TM, int EXPERTS, int WS>
hipError_t launch_few_sized(const ScaledArgs& a, hipStream_t s) {
  if constexpr (!EXPERTS) {
    const int64_t groups = ((int64_t)a.M + 16 * TM - 1) / (16 * TM) * ((a.N + 31) / 32);
    if (a.p * scale_blocks(a.K) >= 8 && groups <= 256) return launch_few<TM, 2, 8, EXPERTS, WS>(a, s);
  }
  return launch_few<TM, 2, 4, EXPERTS, WS>(a, s);
}

}  // namespace

// Against the tiles, whose rows and columns of 128 leave compute units idle where
// there are few of both (us, this kernel and the tiles; weights N x K, M rows):
// with a workgroup a compute unit or fewer this kernel wins, of its forms the one
// of fewest rows (4096 x 4096: M 1 9.9 and 20.4, M 32 10.2 and 20.1, M 64 13.4 and
// 20.3, M 128 18.6 and 21.0, M 192 would be two rounds; 1024 x 8192, M 256: 21.7
// and 36.6); with two, weights read again by each are most of the time (8192 x
// 8192, M 96: 55 and 52; 16384 x 4096, M 48: 38 and 29), but for a form that reads
// them once (16384 x 4096, M 32: 23 and 29).  Up to 16 rows read them once whatever
// their width (28672 x 8192: 52 and 58 at M 1, 60 and 59 at M 16).
//
// Of experts at most M have rows.  Up to 8 rows an expert this kernel wins with 32
// blocks or more along the contraction (64 x 1024 x 4096: 2 rows each 51 and 58, 8 57
// and 67, 12 63 and 67; of 5120: 2 61 and 63, 6 69 and 67, 8 72 and 67; 64 x 2048 x 4096: 8
// 109 and 130; 16 x 2048 x 4096: 8 36 and 37, 12 37 and 37); with fewer, while its
// workgroups, whose streams are short, are not many more than run at once: 2048 of the
// experts that can have rows (64 x 1024 x 3968, 31 blocks: 1024 of them 32 and 33, 2048
// 53 and 52, with 8 rows each 56 and 52; of 2048: 1024 18 and 19, 2048 30 and 29; 8 x 8192
// x 1024: 2048 17 and 23; 64 x 4096 x 1024: 1024 12 and 17, 2048 19 and 18, 4096 34 and
// 30; 256 x 512 x 2048: 512 12 and 19, 2048 34 and 29, 4096 61 and 54).  Between the sizes
// that it fits, the rule is up to 17 % off.
int scaled_few_tiles(int64_t M, int64_t N, int64_t blocks, int64_t E) {
  const int64_t across = (N + 31) / 32;
  if (E) return M <= 8 * E && (blocks >= 32 || std::min(M, E) * across <= 2048) ? 1 : 0;
  const auto groups = [&](int tm) { return (M + 16 * tm - 1) / (16 * tm) * across; };
  if (M <= 16 || groups(1) <= 256) return 1;
  if (groups(2) <= (M <= 32 ? 512 : 256)) return 2;
  return groups(4) <= 256 ? 4 : 0;
}

hipError_t launch_scaled_few(const ScaledArgs& a, int wscale, int tm, hipStream_t s) {
  const auto go = [&](auto ws) {
    constexpr int WS = decltype(ws)::value;
    if (a.E) return launch_few_sized<1, 1, WS>(a, s);
    return tm == 1 ? launch_few_sized<1, 0, WS>(a, s) : tm == 2 ? launch_few_sized<2, 0, WS>(a, s) : launch_few_sized<4, 0, WS>(a, s);
  };
  return wscale == WS_F32 ? go(std::integral_constant<int, WS_F32>()) : go(std::integral_constant<int, WS_BYTE>());
}

}  // namespace tpf
