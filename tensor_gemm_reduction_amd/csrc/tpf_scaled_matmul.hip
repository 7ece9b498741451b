// Products of 8-bit operands with a scale for each block of 128 along the
// contraction, on matrix-core tiles.
//
// v_mfma_scale_f32_16x16x128 multiplies 16 x 128 codes by 128 x 16 and applies
// a power of two to each operand's block: exactly one block of 128, so packed
// rows' exponent bytes go into the instruction and a product of two of them
// costs nothing beside it.  Weights with fp32 scales take the block's partial
// sum from the instruction and one fused multiply-add an element more.
//
// Lane l of the instruction holds 32 codes of row (or column) l % 16.  Which 32
// of the block's 128 each group of 16 lanes holds is free, as long as both
// operands agree and the scale is the same for all: group g takes the 16-byte
// chunks g and g + 4, so that each is one 16-byte LDS read.
//
// The 8-bit instructions add eight products at a time with 13 binary places
// below the largest of the eight and drop the rest (measured; all forms of them
// do): about 2^-16 of a sum's size, far below half a step of bf16 (2^-9), so
// results in bf16 take them.  Results in fp32 take the bf16 instructions, at
// half the rate: codes are exact in bf16 and those sums keep fp32's bits.
//
// The weights are the instruction's first operand: lane l's four results are
// then y[m = l % 16][n = 4 (l / 16) .. + 3], stored together.
#include "tpf_gemm.hpp"
#include "tpf_scaled.hpp"
#include "tpf_scaled_device.hpp"
#include "tpf_tiles.hpp"

namespace tpf {
namespace {

enum Mode : int { PLAIN = 0, GRAD = 1, EXPERTS = 2, EXPERTS_GRAD = 3 };

// BM x BN results a workgroup of WAVES_M x WAVES_N waves; both operands' tiles
// of one block of 128 in two LDS slots each.
template <int BM_, int BN_, int WAVES_M_, int WAVES_N_>
struct ScCfg {
  static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_;
  static constexpr int NW = WAVES_M * WAVES_N, THREADS = 64 * NW;
  static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N, TM = WM / 16, TN = WN / 16;
  static constexpr int X_LOADS = BM / 8 / NW, W_LOADS = BN / 8 / NW;   // 1 KiB each: 8 rows of 128 codes
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "loads must split evenly over the waves");
  static_assert(128 % WN == 0, "a wave's columns lie in one block of scales");
};

template <class Cfg, int S>
__device__ __forceinline__ char* x_slot() {
  __shared__ __attribute__((aligned(1024))) char buf[Cfg::BM * 128];
  return buf;
}
template <class Cfg, int S>
__device__ __forceinline__ char* w_slot() {
  __shared__ __attribute__((aligned(1024))) char buf[Cfg::BN * 128];
  return buf;
}

// Rows of 128 bytes, two to a span of the LDS banks: chunks are XORed with the
// row's number over two, so that 16 rows' same chunk lies in all banks once.
__device__ __forceinline__ int sc_swz(int row) { return (row >> 1) & 7; }

// What one workgroup computes.
struct ScJob {
  int e;               // expert
  int64_t xrow, wrow;  // first rows of the operands (in codes: xrow * K)
  int row0, rows;      // first row of the result, valid rows
  int n0;              // first column
  int s0, kb0;         // first shard and block
  int steps, kbs;      // steps in all; blocks of a shard (the weight gradients: a bound never reached)
};

template <class Cfg, int MODE>
struct ScLoader {
  uint32_t x_off[Cfg::X_LOADS], w_off[Cfg::W_LOADS];   // byte offsets at block 0, kOOB: reads as zeros
  int64_t x_base, w_base, x_bytes, w_bytes;
  int K;

  __device__ __forceinline__ void init(const ScaledArgs& a, const ScJob& j) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    K = a.K;
    const bool gather = MODE == EXPERTS && a.top;
    x_base = gather ? 0 : j.xrow * K;
    x_bytes = gather ? (int64_t)a.xrows * K : (int64_t)j.rows * K;
    w_base = j.wrow * K;
    const int cols = min(Cfg::BN, a.N - j.n0);
    w_bytes = (int64_t)cols * K;
#pragma unroll
    for (int i = 0; i < Cfg::X_LOADS; ++i) {
      const int row = (wave * Cfg::X_LOADS + i) * 8 + (lane >> 3);
      int at = row < j.rows ? row : -1;
      if (gather && at >= 0) {
        at = a.src[j.row0 + row] / a.top;
        if ((uint32_t)at >= (uint32_t)a.xrows) at = -1;
      }
      x_off[i] = at >= 0 ? (uint32_t)at * (uint32_t)K + 16 * ((lane & 7) ^ sc_swz(row)) : kOOB;
    }
#pragma unroll
    for (int i = 0; i < Cfg::W_LOADS; ++i) {
      const int row = (wave * Cfg::W_LOADS + i) * 8 + (lane >> 3);
      w_off[i] = row < cols ? (uint32_t)row * (uint32_t)K + 16 * ((lane & 7) ^ sc_swz(row)) : kOOB;
    }
  }

  // Block kb of shard s into a slot.  Codes past the end of a row read as zeros.
  __device__ __forceinline__ void issue(const ScaledArgs& a, int s, int kb, char* lx, char* lw) const {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x[s] + x_base, x_bytes);
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.w[s] + w_base, w_bytes);
    const int k0 = kb * kScaleBlock;
    const bool tail = k0 + kScaleBlock > K;
#pragma unroll
    for (int i = 0; i < Cfg::X_LOADS; ++i) {
      const int row = (wave * Cfg::X_LOADS + i) * 8 + (lane >> 3);
      uint32_t off = x_off[i];
      if (tail && k0 + 16 * ((lane & 7) ^ sc_swz(row)) >= K) off = kOOB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void_t*)(lx + (wave * Cfg::X_LOADS + i) * 1024), 16, (int)off,
                                               k0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < Cfg::W_LOADS; ++i) {
      const int row = (wave * Cfg::W_LOADS + i) * 8 + (lane >> 3);
      uint32_t off = w_off[i];
      if (tail && k0 + 16 * ((lane & 7) ^ sc_swz(row)) >= K) off = kOOB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void_t*)(lw + (wave * Cfg::W_LOADS + i) * 1024), 16, (int)off,
                                               k0, 0, 0);
    }
  }
};

// A wave's scales of one block.
template <class Cfg, int WS>
struct ScScales {
  int x[Cfg::TM];
  int w[WS == WS_ROW ? Cfg::TN : 1];
  float f;
};

template <class Cfg, int MODE, int WS>
struct ScScaleLoader {
  int x_off[Cfg::TM], w_off[WS == WS_ROW ? Cfg::TN : 1];
  int64_t x_base, w_base;
  __device__ __forceinline__ void init(const ScaledArgs& a, const ScJob& j) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int wm = wave / Cfg::WAVES_N, wn = wave % Cfg::WAVES_N;
    const bool gather = MODE == EXPERTS && a.top;
    x_base = gather ? 0 : j.xrow * a.xsw;
#pragma unroll
    for (int i = 0; i < Cfg::TM; ++i) {
      int row = min(wm * Cfg::WM + i * 16 + (lane & 15), j.rows - 1);     // rows past the last are not stored
      if (gather) row = min(max(a.src[j.row0 + row], 0) / a.top, a.xrows - 1);
      x_off[i] = row * a.xsw;
    }
    if constexpr (WS == WS_ROW) {
      w_base = j.wrow * a.wsw;
#pragma unroll
      for (int i = 0; i < Cfg::TN; ++i)
        w_off[i] = min(wn * Cfg::WN + i * 16 + (lane & 15), a.N - 1 - j.n0) * a.wsw;
    } else {
      const int nb = (a.N + kScaleBlock - 1) / kScaleBlock;
      w_base = ((int64_t)j.e * nb + min((j.n0 + wn * Cfg::WN) / kScaleBlock, nb - 1)) * a.wsw;
    }
  }
  __device__ __forceinline__ void load(const ScaledArgs& a, int s, int kb, ScScales<Cfg, WS>& r) const {
    const uint8_t* x = a.xs[s] + x_base;
#pragma unroll
    for (int i = 0; i < Cfg::TM; ++i) r.x[i] = x[x_off[i] + kb];
    if constexpr (WS == WS_ROW) {
      const uint8_t* w = a.ws[s] + w_base;
#pragma unroll
      for (int i = 0; i < Cfg::TN; ++i) r.w[i] = w[w_off[i] + kb];
    } else if constexpr (WS == WS_BYTE) {
      r.w[0] = a.ws[s][w_base + kb];
    } else {
      r.f = reinterpret_cast<const float*>(a.ws[s])[w_base + kb];
    }
  }
};

// Row `row` of a slot: the lane's 32 codes.
__device__ __forceinline__ i32x8_t sc_read(const char* l, int row, int lane) {
  const int g = lane >> 4, z = sc_swz(row);
  const i32x4_t lo = *reinterpret_cast<const i32x4_t*>(l + row * 128 + 16 * (g ^ z));
  const i32x4_t hi = *reinterpret_cast<const i32x4_t*>(l + row * 128 + 16 * ((g + 4) ^ z));
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// One block's products on the 8-bit instructions.
template <class Cfg, int WS>
__device__ __forceinline__ void sc_compute(f32x4_t (&acc)[Cfg::TM][Cfg::TN], const char* lx, const char* lw,
                                           const ScScales<Cfg, WS>& sc) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int wm = wave / Cfg::WAVES_N, wn = wave % Cfg::WAVES_N;
  i32x8_t w[Cfg::TN];
#pragma unroll
  for (int i = 0; i < Cfg::TN; ++i) w[i] = sc_read(lw, wn * Cfg::WN + i * 16 + (lane & 15), lane);
  if constexpr (WS == WS_F32) {
    // The partial sums of one row of blocks are added while the next row's are
    // computed; the barriers keep the compiler from holding more of them.
    f32x4_t part[2][Cfg::TN];
#pragma unroll
    for (int m = 0; m <= Cfg::TM; ++m) {
      if (m < Cfg::TM) {
        const i32x8_t x = sc_read(lx, wm * Cfg::WM + m * 16 + (lane & 15), lane);
#pragma unroll
        for (int n = 0; n < Cfg::TN; ++n) part[m & 1][n] = sc_mfma(w[n], x, f32x4_t{0, 0, 0, 0}, 127, sc.x[m]);
      }
      if (m > 0) {
#pragma unroll
        for (int n = 0; n < Cfg::TN; ++n)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            acc[m - 1][n][v] = __builtin_fmaf(part[(m - 1) & 1][n][v], sc.f, acc[m - 1][n][v]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  } else {
#pragma unroll
    for (int m = 0; m < Cfg::TM; ++m) {
      const i32x8_t x = sc_read(lx, wm * Cfg::WM + m * 16 + (lane & 15), lane);
#pragma unroll
      for (int n = 0; n < Cfg::TN; ++n) acc[m][n] = sc_mfma(w[n], x, acc[m][n], sc.w[WS == WS_ROW ? n : 0], sc.x[m]);
    }
  }
}

// The same on the bf16 instructions, whose sums keep fp32's bits: every code is
// exact in bf16, a block's partial sum is scaled once.
template <class Cfg, int WS>
__device__ __forceinline__ void sc_compute_fine(f32x4_t (&acc)[Cfg::TM][Cfg::TN], const char* lx, const char* lw,
                                                const ScScales<Cfg, WS>& sc) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int wm = wave / Cfg::WAVES_N, wn = wave % Cfg::WAVES_N;
  ScFine w[Cfg::TN];
#pragma unroll
  for (int n = 0; n < Cfg::TN; ++n) w[n] = sc_fine(sc_read(lw, wn * Cfg::WN + n * 16 + (lane & 15), lane));
  float ws[WS == WS_ROW ? Cfg::TN : 1][4];
  if constexpr (WS == WS_ROW) {
#pragma unroll
    for (int n = 0; n < Cfg::TN; ++n)
#pragma unroll
      for (int v = 0; v < 4; ++v) ws[n][v] = exp_byte(__shfl(sc.w[n], 4 * (lane >> 4) + v));
  } else {
    ws[0][0] = WS == WS_F32 ? sc.f : exp_byte(sc.w[0]);
  }
#pragma unroll
  for (int m = 0; m < Cfg::TM; ++m) {
    const ScFine x = sc_fine(sc_read(lx, wm * Cfg::WM + m * 16 + (lane & 15), lane));
    const float xs = exp_byte(sc.x[m]);
#pragma unroll
    for (int n = 0; n < Cfg::TN; ++n) {
      const f32x4_t part = sc_mfma_fine(w[n], x);
#pragma unroll
      for (int v = 0; v < 4; ++v)
        acc[m][n][v] = __builtin_fmaf(part[v], xs * (WS == WS_ROW ? ws[n][v] : ws[0][0]), acc[m][n][v]);
    }
  }
}

template <class Cfg, int MODE, int WS, int OUT>
__global__ __launch_bounds__(Cfg::THREADS) void scaled_tile_kernel(ScaledArgs args) {
  (void)args;
  const ScaledArgs& a = *(const ScaledArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / Cfg::WAVES_N, wn = wave % Cfg::WAVES_N;
  ScJob j{};
  int outer, tm, tn;
  tile_coords(xcd_task(blockIdx.x, a.tasks), a.tiles_m, a.tiles_n, outer, tm, tn);
  const int kbs = (a.K + kScaleBlock - 1) / kScaleBlock;
  j.n0 = tn * Cfg::BN;
  j.kbs = kbs;
  j.steps = a.p * kbs;
  j.row0 = tm * Cfg::BM;
  j.rows = min(Cfg::BM, a.M - j.row0);
  j.wrow = j.n0;
  void* out = a.y[0];
  int64_t out_row = 0;
  if constexpr (MODE == GRAD) {
    j.s0 = outer;
    j.steps = kbs;
    out = a.y[outer];
  }
  if constexpr (MODE == EXPERTS) {
    const RowTile t = expert_tile<Cfg::BM>(a.offsets, a.E, a.M, tm, lane);
    if (t.rows <= 0) return;
    j.e = t.e;
    j.row0 = t.row0;
    j.rows = t.rows;
    if (t.e == a.E) j.steps = 0, j.e = 0;          // rows of no expert: zeros
    j.wrow = (int64_t)j.e * a.N + j.n0;
  }
  if constexpr (MODE == EXPERTS_GRAD) {
    j.s0 = outer / a.E;
    const int e = outer % a.E;
    const BlockRange b = expert_blocks(a.offsets, a.E, e, a.K / kScaleBlock, lane);
    j.kb0 = b.first;
    j.steps = b.n;
    out = a.y[j.s0];
    out_row = (int64_t)e * a.M;
  }
  j.xrow = j.row0;
  f32x4_t acc[Cfg::TM][Cfg::TN];
#pragma unroll
  for (int m = 0; m < Cfg::TM; ++m)
#pragma unroll
    for (int n = 0; n < Cfg::TN; ++n) acc[m][n] = f32x4_t{0, 0, 0, 0};

  if (j.steps > 0) {
    ScLoader<Cfg, MODE> ld;
    ScScaleLoader<Cfg, MODE, WS> sl;
    ld.init(a, j);
    sl.init(a, j);
    int s = j.s0, kb = j.kb0;                       // of the next step to be loaded
    ScScales<Cfg, WS> sc[2];
    sl.load(a, s, kb, sc[0]);
    ld.issue(a, s, kb, x_slot<Cfg, 0>(), w_slot<Cfg, 0>());
    const auto step = [&](int t, char* lx, char* lw, char* nx, char* nw, ScScales<Cfg, WS>& cur,
                          ScScales<Cfg, WS>& next) {
      if (++kb == j.kbs) kb = 0, ++s;
      wait_vmcnt(0);
      lds_barrier();
      if (t + 1 < j.steps) {
        sl.load(a, s, kb, next);
        ld.issue(a, s, kb, nx, nw);
      }
      if constexpr (OUT == OUT_F32) sc_compute_fine<Cfg, WS>(acc, lx, lw, cur);
      else sc_compute<Cfg, WS>(acc, lx, lw, cur);
    };
    for (int t = 0; t < j.steps; t += 2) {
      step(t, x_slot<Cfg, 0>(), w_slot<Cfg, 0>(), x_slot<Cfg, 1>(), w_slot<Cfg, 1>(), sc[0], sc[1]);
      if (t + 1 >= j.steps) break;
      step(t + 1, x_slot<Cfg, 1>(), w_slot<Cfg, 1>(), x_slot<Cfg, 0>(), w_slot<Cfg, 0>(), sc[1], sc[0]);
    }
  }

  constexpr int ES = OUT == OUT_F32 ? 4 : 2;
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(
      reinterpret_cast<char*>(out) + ((out_row + j.row0) * a.N + j.n0) * ES, (int64_t)j.rows * a.N * ES);
#pragma unroll
  for (int m = 0; m < Cfg::TM; ++m)
#pragma unroll
    for (int n = 0; n < Cfg::TN; ++n) {
      const int row = wm * Cfg::WM + m * 16 + (lane & 15), col = wn * Cfg::WN + n * 16 + 4 * (lane >> 4);
      const int off = row < j.rows && j.n0 + col < a.N ? (row * a.N + col) * ES : (int)kOOB;
      f32x4_t v = acc[m][n];
      if (a.gelu) v = f32x4_t{gelu_f32(v[0]), gelu_f32(v[1]), gelu_f32(v[2]), gelu_f32(v[3])};
      if constexpr (OUT == OUT_F32)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), rs, off, 0, 0);
      else
        __builtin_amdgcn_raw_buffer_store_b64(
            u32x2_t{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])}, rs, off, 0, 0);
    }
}

using Big = ScCfg<256, 256, 2, 4>;
using Mid = ScCfg<128, 128, 2, 2>;

template <class Cfg, int MODE, int WS, int OUT>
hipError_t launch_cfg(ScaledArgs a, hipStream_t s) {
  a.tiles_n = (a.N + Cfg::BN - 1) / Cfg::BN;
  a.tiles_m = (a.M + Cfg::BM - 1) / Cfg::BM;
  if (MODE == EXPERTS) a.tiles_m = expert_tiles(a.M, a.E, Cfg::BM);
  int64_t tasks = (int64_t)a.tiles_m * a.tiles_n;
  if (MODE == GRAD || MODE == EXPERTS_GRAD) tasks *= a.p * (MODE == EXPERTS_GRAD ? a.E : 1);
  if (tasks > 1 << 23) return hipErrorInvalidConfiguration;
  a.tasks = (int)tasks;
  hipLaunchKernelGGL((scaled_tile_kernel<Cfg, MODE, WS, OUT>), dim3(a.tasks), dim3(Cfg::THREADS), 0, s, a);
  return hipGetLastError();
}

template <int MODE, int WS>
hipError_t launch_mode(const ScaledArgs& a, int64_t rows, int64_t outs, hipStream_t s) {
  const int64_t big = (rows + 255) / 256 * ((a.N + 255) / 256) * outs;
  if (a.out == OUT_F32) return launch_cfg<Mid, MODE, WS, OUT_F32>(a, s);
  if constexpr (WS == WS_F32) return launch_cfg<Mid, MODE, WS, OUT_BF16>(a, s);
  else return big >= 192 ? launch_cfg<Big, MODE, WS, OUT_BF16>(a, s) : launch_cfg<Mid, MODE, WS, OUT_BF16>(a, s);
}

}  // namespace

hipError_t launch_scaled_matmul(ScaledArgs a, int wscale, hipStream_t s) {
  if (const int few = scaled_few_tiles(a.M, a.E)) return launch_scaled_few(a, wscale, few, s);
  if (a.E) {
    return wscale == WS_F32 ? launch_mode<EXPERTS, WS_F32>(a, a.M, 1, s) : launch_mode<EXPERTS, WS_BYTE>(a, a.M, 1, s);
  }
  return wscale == WS_F32 ? launch_mode<PLAIN, WS_F32>(a, a.M, 1, s) : launch_mode<PLAIN, WS_BYTE>(a, a.M, 1, s);
}

hipError_t launch_scaled_weight_grad(ScaledArgs a, hipStream_t s) {
  return a.E ? launch_mode<EXPERTS_GRAD, WS_ROW>(a, a.M, (int64_t)a.p * a.E, s)
             : launch_mode<GRAD, WS_ROW>(a, a.M, a.p, s);
}

}  // namespace tpf
