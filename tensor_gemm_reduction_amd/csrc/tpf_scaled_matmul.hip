// Products of 8-bit operands with a scale for each block of 128 along the
// contraction, on matrix-core tiles.
//
// v_mfma_scale_f32_16x16x128 multiplies 16 x 128 codes by 128 x 16 and applies
// a power of two to each operand's block: exactly one block of 128, so packed
// rows' exponent bytes go into the instruction and a product of two of them
// costs nothing beside it.  Of a weight's fp32 scale the power of two goes into the
// instruction as well, so that no partial sum leaves fp32's range where the scales'
// product lies within it (4096^3: 79 us as with the whole scale afterwards); its other
// part, 1 to 2, takes one fused multiply-add an element more.
//
// Lane l of the instruction holds 32 codes of row (or column) l % 16.  Which 32
// of the block's 128 each group of 16 lanes holds is free, as long as both
// operands agree and the scale is the same for all: group g takes the 16-byte
// chunks g and g + 4, so that each is one 16-byte LDS read.
//
// The 8-bit instructions add eight products at a time with 13 binary places
// below the largest of the eight and drop the rest (measured; all forms of them
// do): less than 2^-10 of the products' magnitudes, about 2^-16 of them as a rule,
// far below half a step of bf16 (2^-9) unless products cancel, so results in bf16
// take them.  Results in fp32, and those in bf16 that are asked for with sums in
// fp32 (FINE), take the bf16 instructions, at half the rate: codes are exact in
// bf16 and those sums keep fp32's bits.
//
// What bounds them: 4 x 4096 x 4096 x 4096 take 209 us, 2630 TFLOP/s; the matrix
// cores are busy 64 % of the time at the 1.9 GHz that the board holds them to (a
// library's product with one scale a tensor: 0.83 of the time).  With few steps a
// tile (64 experts, K 1024) its start, first loads and stores are as long as its
// products: 195 us, matrix cores 29 %.  Four waves of 128 x 128 would read a third
// less of LDS, but their sums leave too few registers (3.3 times as long).
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

// BM x BN results a workgroup of WAVES_M x WAVES_N waves, one block of 128 a step;
// W_SLOTS tiles of w in LDS.
template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int W_SLOTS_>
struct ScCfg {
  static constexpr int W_SLOTS = W_SLOTS_, UNROLL = W_SLOTS == 1 ? 3 : 6;      // steps until the slots' turn is over
  static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_;
  static constexpr int NW = WAVES_M * WAVES_N, THREADS = 64 * NW;
  static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N, TM = WM / 16, TN = WN / 16;
  static constexpr int SLICES = TM / 2;                                // two rows of 16 x 16 blocks each
  static constexpr int X_LOADS = BM / 8 / NW, W_LOADS = BN / 8 / NW;   // 1 KiB each: 8 rows of 128 codes
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "loads must split evenly over the waves");
  static_assert(WM % 64 == 0 && WN == 64, "a wave's scales: 64 rows a word load, columns in one block");
  static_assert(SLICES % 2 == 0, "slices alternate between two sets of registers");
};

// Three slots of x's tiles and one or two of w's, each an object of its own, so that the
// compiler sees that loads in flight into one do not touch what is read.
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
  int steps, kbs;      // steps in all; blocks of a shard
};

// Where a step's block lies: counts on from step to step, staying at the last.
struct ScAt {
  int s, kb, left;     // steps after this one
  __device__ __forceinline__ bool next(int kbs) {      // whether the shard changed
    if (left == 0) return false;
    --left;
    if (++kb < kbs) return false;
    kb = 0;
    ++s;
    return true;
  }
};

template <class Cfg, int MODE>
struct ScLoader {
  uint32_t x_off[Cfg::X_LOADS], w_off[Cfg::W_LOADS];   // byte offsets at block 0, kOOB: reads as zeros
  int64_t x_base, w_base;
  int x_bytes, w_bytes;
  __amdgpu_buffer_rsrc_t rx, rw;
  ScAt at;
  int k0, wave, kc[2];                                 // kc: the lane's byte within a block, of even and odd loads

  __device__ __forceinline__ void init(const ScaledArgs& a, const ScJob& j) {
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const bool gather = MODE == EXPERTS && a.top;
    x_base = gather ? 0 : j.xrow * a.K;
    x_bytes = (int)(gather ? (int64_t)a.xrows * a.K : (int64_t)j.rows * a.K);
    w_base = j.wrow * a.K;
    const int cols = min(Cfg::BN, a.N - j.n0);
    w_bytes = cols * a.K;
    // load i's rows are 8 more than load i - 1's: the swizzle differs by 4
#pragma unroll
    for (int i = 0; i < 2; ++i) kc[i] = 16 * ((lane & 7) ^ sc_swz(i * 8 + (lane >> 3)));
#pragma unroll
    for (int i = 0; i < Cfg::X_LOADS; ++i) {
      const int row = (wave * Cfg::X_LOADS + i) * 8 + (lane >> 3);
      int from = row < j.rows ? row : -1;
      if (gather && from >= 0) {
        from = a.src[j.row0 + row] / a.top;
        if ((uint32_t)from >= (uint32_t)a.xrows) from = -1;
      }
      x_off[i] = from >= 0 ? (uint32_t)from * (uint32_t)a.K + 16 * ((lane & 7) ^ sc_swz(row)) : kOOB;
    }
#pragma unroll
    for (int i = 0; i < Cfg::W_LOADS; ++i) {
      const int row = (wave * Cfg::W_LOADS + i) * 8 + (lane >> 3);
      w_off[i] = row < cols ? (uint32_t)row * (uint32_t)a.K + 16 * ((lane & 7) ^ sc_swz(row)) : kOOB;
    }
    at = ScAt{j.s0, j.kb0, j.steps - 1};
    operands(a);
  }
  __device__ __forceinline__ void operands(const ScaledArgs& a) {
    rx = make_rsrc(a.x[at.s] + x_base, x_bytes);
    rw = make_rsrc(a.w[at.s] + w_base, w_bytes);
    k0 = at.kb * kScaleBlock;
  }
  __device__ __forceinline__ void next(const ScaledArgs& a, int kbs) {
    if (at.next(kbs)) operands(a);
    k0 = at.kb * kScaleBlock;
  }
  // Codes past the end of a row read as zeros.
  __device__ __forceinline__ uint32_t within(uint32_t off, int row8, int K) const {
    return k0 + kc[row8 & 1] < K ? off : kOOB;
  }
  __device__ __forceinline__ void x_load(int i, int K, char* to) const {
    const int q = wave * Cfg::X_LOADS + i;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void_t*)(to + q * 1024), 16,
                                             (int)within(x_off[i], Cfg::X_LOADS % 2 ? q : i, K), k0, 0, 0);
  }
  __device__ __forceinline__ void w_load(int i, int K, char* to) const {
    const int q = wave * Cfg::W_LOADS + i;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void_t*)(to + q * 1024), 16,
                                             (int)within(w_off[i], Cfg::W_LOADS % 2 ? q : i, K), k0, 0, 0);
  }
};

// An fp32 factor as the byte of its power of two and what is left: +-[1, 2), [0, 2)
// below the least normal number, infinities and NaN as they are.
struct ScFactor {
  int byte;
  float part;
};
__device__ __forceinline__ ScFactor sc_factor(float f) {
  const int byte = min((int)(__float_as_uint(f) >> 23 & 255), 254);
  return ScFactor{byte, __builtin_amdgcn_ldexpf(f, 127 - byte)};
}

// A wave's scales.  Lane l loads the word of row l (and l + 64), four blocks'
// exponent bytes; rows of 16 lanes then spread over the wave, so that lane l
// holds row l % 16 of every block of 16 rows, as the matrix instruction takes it.
__device__ __forceinline__ void spread(uint32_t v, uint32_t (&out)[4]) {
  const auto halves = __builtin_amdgcn_permlane32_swap(v, v, false, false);           // [0 1 0 1], [2 3 2 3]
  const auto lo = __builtin_amdgcn_permlane16_swap(halves[0], halves[0], false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap(halves[1], halves[1], false, false);
  out[0] = lo[0];
  out[1] = lo[1];
  out[2] = hi[0];
  out[3] = hi[1];
}

template <class Cfg, int MODE, int WS>
struct ScScales {
  int x_off[Cfg::WM / 64], w_off;       // of the rows whose words the lane loads
  int64_t x_base, w_base;
  ScAt at;                              // the step after the current one
  const uint8_t *xs, *ws;               // its shard's scales, held: a scalar load would wait for the LDS reads as well
  uint32_t raw[Cfg::WM / 64], raww;     // words of the next four blocks
  uint32_t x[Cfg::TM], w[4];            // words of the current four
  uint32_t w_byte, w_next;              // WS_BYTE: the block's byte
  float f, f_next;                      // WS_F32: its factor
  int shift;
  int lane0;                            // 0, unknown to the compiler: vector loads of what is the same in all lanes

  __device__ __forceinline__ void init(const ScaledArgs& a, const ScJob& j) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int wm = wave / Cfg::WAVES_N, wn = wave % Cfg::WAVES_N;
    lane0 = 0;
    asm volatile("" : "+v"(lane0));
    const bool gather = MODE == EXPERTS && a.top;
    x_base = gather ? 0 : j.xrow * a.xsw;
#pragma unroll
    for (int i = 0; i < Cfg::WM / 64; ++i) {
      int row = min(wm * Cfg::WM + i * 64 + lane, j.rows - 1);            // rows past the last are not stored
      if (gather) row = min(max(a.src[j.row0 + row], 0) / a.top, a.xrows - 1);
      x_off[i] = row * a.xsw;
    }
    if constexpr (WS == WS_ROW) {
      w_base = j.wrow * a.wsw;
      w_off = min(wn * Cfg::WN + lane, a.N - 1 - j.n0) * a.wsw;
    } else {
      const int nb = (a.N + kScaleBlock - 1) / kScaleBlock;
      w_base = ((int64_t)j.e * nb + min((j.n0 + wn * Cfg::WN) / kScaleBlock, nb - 1)) * a.wsw;
    }
    at = ScAt{j.s0, j.kb0, j.steps - 1};
    shard(a);
    load_words();
    load_block();
    take();
    take_block();
    step(a, j.kbs);
  }
  __device__ __forceinline__ void shard(const ScaledArgs& a) {
    xs = a.xs[at.s] + x_base;
    ws = a.ws[at.s] + w_base * (WS == WS_F32 ? 4 : 1);
  }
  __device__ __forceinline__ void load_words() {
    const uint8_t* p = xs + (at.kb & ~3);
#pragma unroll
    for (int i = 0; i < Cfg::WM / 64; ++i) raw[i] = *reinterpret_cast<const uint32_t*>(p + x_off[i]);
    if constexpr (WS == WS_ROW) raww = *reinterpret_cast<const uint32_t*>(ws + (at.kb & ~3) + w_off);
  }
  __device__ __forceinline__ void load_block() {
    if constexpr (WS == WS_BYTE) w_next = ws[at.kb + lane0];
    if constexpr (WS == WS_F32) f_next = reinterpret_cast<const float*>(ws)[at.kb + lane0];
  }
  __device__ __forceinline__ void take() {
#pragma unroll
    for (int i = 0; i < Cfg::WM / 64; ++i) {
      uint32_t four[4];
      spread(raw[i], four);
#pragma unroll
      for (int q = 0; q < 4; ++q) x[4 * i + q] = four[q];
    }
    if constexpr (WS == WS_ROW) spread(raww, w);
  }
  __device__ __forceinline__ void take_block() {
    w_byte = w_next;
    f = f_next;
    shift = 8 * (at.kb & 3);
  }
  bool words;                           // the next step's words are not the current ones
  // Loads for the step after the current one, at the current one's start.
  __device__ __forceinline__ void step(const ScaledArgs& a, int kbs) {
    words = at.left > 0;
    if (at.next(kbs)) shard(a);
    words = words && (at.kb & 3) == 0;
  }
  __device__ __forceinline__ void load() {
    if (words) load_words();
    load_block();
  }
  // The next step becomes the current one.
  __device__ __forceinline__ void advance(const ScaledArgs& a, int kbs) {
    if (words) take();
    take_block();
    step(a, kbs);
  }
};

// Where the lane's 32 codes of a wave's first 16 rows lie in a slot: rows 16
// further on are 2 KiB further on, their swizzle being the same.  One offset and a
// constant a read: through longer chains of address arithmetic the compiler loses
// which slot a read is of, and then waits for every load in flight.
struct ScPlace {
  int lo, hi;
  __device__ __forceinline__ ScPlace(int row0, int lane) {
    const int row = row0 + (lane & 15), g = lane >> 4, z = sc_swz(row);
    lo = row * 128 + 16 * (g ^ z);
    hi = row * 128 + 16 * ((g + 4) ^ z);
    asm volatile("" : "+v"(lo), "+v"(hi));
  }
};
__device__ __forceinline__ i32x8_t sc_read(const char* slot, const ScPlace& at, int rows) {
  const i32x4_t lo = *reinterpret_cast<const i32x4_t*>(slot + (at.lo + rows * 128));
  const i32x4_t hi = *reinterpret_cast<const i32x4_t*>(slot + (at.hi + rows * 128));
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// A wave's operands: of x two rows of blocks at a time, of w all columns.
template <class Cfg, int FINE>
struct ScOperands {
  i32x8_t x[2][2];
  i32x8_t w[Cfg::TN];
};
template <class Cfg>
struct ScOperands<Cfg, 1> {
  i32x8_t x[2][2];
  ScFine w[Cfg::TN];
};
__device__ __forceinline__ void sc_take(i32x8_t& to, i32x8_t v) { to = v; }
__device__ __forceinline__ void sc_take(ScFine& to, i32x8_t v) { to = sc_fine(v); }

// One step.  On entry the registers hold the step's w and its first slice of x.
// Each slice's instructions run while the next slice of x is read.  The tile of x
// for the step after the next goes into the slot that the step before left,
// between the instructions of all slices but the last; before the last slice the
// wave waits for the next step's tiles (loads issued since may stay in flight) and
// passes a barrier; between the last slice's instructions it reads the next step's
// w, column by column, and loads the tile of w for the step after into the slot
// that this step's w was read from a step ago.
// With one slot of w (two workgroups then share a compute unit) a barrier at the
// step's start says that all waves hold w; the next step's tile replaces it during
// the first slice, x's loads follow in the second.
template <class Cfg, int MODE, int WS, int FINE, int T>
__device__ __forceinline__ void sc_step(f32x4_t (&acc)[Cfg::TM][Cfg::TN], ScOperands<Cfg, FINE>& o,
                                        ScLoader<Cfg, MODE>& ld, ScScales<Cfg, MODE, WS>& sc, const ScPlace& px,
                                        const ScPlace& pw, const ScaledArgs& a, int kbs) {
  const int lane = threadIdx.x & 63;
  constexpr int SX = T % 3, SW = T % Cfg::W_SLOTS, S = Cfg::SLICES;
  constexpr int XL = Cfg::X_LOADS, PER = (XL + S - 2) / (S - 1);
  constexpr bool ONE = Cfg::W_SLOTS == 1;
  if constexpr (ONE) lds_barrier();
  sc.load();
  float wf[WS == WS_ROW && FINE ? Cfg::TN : 1][4];
  if constexpr (FINE && WS == WS_ROW) {
#pragma unroll
    for (int n = 0; n < Cfg::TN; ++n) {
      const float own = exp_byte((int)(sc.w[n] >> sc.shift) & 255);
#pragma unroll
      for (int v = 0; v < 4; ++v) wf[n][v] = __shfl(own, 4 * (lane >> 4) + v);
    }
  } else if constexpr (FINE) {
    wf[0][0] = WS == WS_F32 ? sc.f : exp_byte(sc.w_byte);
  }
  ScFactor factor{};
  if constexpr (!FINE && WS == WS_F32) factor = sc_factor(sc.f);
  if constexpr (!ONE) ld.next(a, kbs);
#pragma unroll
  for (int s = 0; s < S; ++s) {
    if (ONE && s == 1) ld.next(a, kbs);
    if (s < S - 1) {
#pragma unroll
      for (int i = 0; i < 2; ++i) o.x[(s + 1) & 1][i] = sc_read(x_slot<Cfg, SX>(), px, (2 * s + 2 + i) * 16);
    } else {
      wait_vmcnt(XL);
      lds_barrier();
#pragma unroll
      for (int i = 0; i < 2; ++i) o.x[0][i] = sc_read(x_slot<Cfg, (SX + 1) % 3>(), px, i * 16);
    }
    ScFine xf[2];
    if constexpr (FINE) {
#pragma unroll
      for (int i = 0; i < 2; ++i) xf[i] = sc_fine(o.x[s & 1][i]);
    }
#pragma unroll
    for (int n = 0; n < Cfg::TN; ++n) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int m = 2 * s + i;
        const uint32_t xb = sc.x[m] >> sc.shift;
        if constexpr (FINE) {
          const f32x4_t part = sc_mfma_fine(o.w[n], xf[i]);
          const float xs = exp_byte(xb & 255);
#pragma unroll
          for (int v = 0; v < 4; ++v)
            acc[m][n][v] = __builtin_fmaf(part[v], xs * (WS == WS_ROW ? wf[n][v] : wf[0][0]), acc[m][n][v]);
        } else if constexpr (WS == WS_F32) {
          const f32x4_t part = sc_mfma(o.w[n], o.x[s & 1][i], f32x4_t{0, 0, 0, 0}, factor.byte, (int)xb);
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[m][n][v] = __builtin_fmaf(part[v], factor.part, acc[m][n][v]);
        } else {
          acc[m][n] = sc_mfma(o.w[n], o.x[s & 1][i], acc[m][n],
                              (int)(WS == WS_ROW ? sc.w[n] >> sc.shift : sc.w_byte), (int)xb);
        }
      }
      if (s < S - 1) {
#pragma unroll
        for (int q = 0; q < XL; ++q)      // slice s issues loads PER s .. PER (s + 1) - 1, spread over its columns
          if (ONE ? s == 1 && q * Cfg::TN / XL == n : q / PER == s && (q % PER) * Cfg::TN / PER == n)
            ld.x_load(q, a.K, x_slot<Cfg, (SX + 2) % 3>());
        if constexpr (ONE) {
#pragma unroll
          for (int q = 0; q < Cfg::W_LOADS; ++q)
            if (s == 0 && q * Cfg::TN / Cfg::W_LOADS == n) ld.w_load(q, a.K, w_slot<Cfg, 0>());
        }
      } else {
        sc_take(o.w[n], sc_read(w_slot<Cfg, (SW + 1) % Cfg::W_SLOTS>(), pw, n * 16));
        if constexpr (!ONE) {
#pragma unroll
          for (int q = 0; q < Cfg::W_LOADS; ++q)
            if (q * Cfg::TN / Cfg::W_LOADS == n) ld.w_load(q, a.K, w_slot<Cfg, SW>());
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);     // reads of later slices would need more registers than there are
  }
  // The compiler would move the instructions down, past the barrier and the next step's reads, to where their
  // results are used: 60 registers more than there are.
#pragma unroll
  for (int m = 0; m < Cfg::TM; ++m)
    asm volatile("" : "+v"(acc[m][0]), "+v"(acc[m][1]), "+v"(acc[m][2]), "+v"(acc[m][3]));
  sc.advance(a, kbs);
}

template <class Cfg, int MODE, int WS, int FINE, int T>
__device__ __forceinline__ void sc_steps(f32x4_t (&acc)[Cfg::TM][Cfg::TN], ScOperands<Cfg, FINE>& o,
                                         ScLoader<Cfg, MODE>& ld, ScScales<Cfg, MODE, WS>& sc, const ScPlace& px,
                                         const ScPlace& pw, const ScaledArgs& a, const ScJob& j, int t) {
  if constexpr (T < Cfg::UNROLL) {
    if (t + T < j.steps) {
      sc_step<Cfg, MODE, WS, FINE, T>(acc, o, ld, sc, px, pw, a, j.kbs);
      sc_steps<Cfg, MODE, WS, FINE, T + 1>(acc, o, ld, sc, px, pw, a, j, t);
    }
  }
}

template <class Cfg, int MODE, int WS, int OUT, int FINE>
__global__ __launch_bounds__(Cfg::THREADS, 2) void scaled_tile_kernel(ScaledArgs args) {
  (void)args;
  const ScaledArgs& a = *(const ScaledArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane & 15;
  const int wm = wave / Cfg::WAVES_N, wn = wave % Cfg::WAVES_N;
  ScJob j{};
  int outer, tm, tn;
  if constexpr (MODE == EXPERTS) {
    // Pairs of row tiles go to the XCDs in turn, so that the tiles behind the last rows, which end at once, are spread
    // over them; within a pair column by column, so that both read a tile of w at the same time.
    const int x = blockIdx.x % kXcds, i = blockIdx.x / kXcds;
    const int pair = i / (2 * a.tiles_n), in = i - pair * 2 * a.tiles_n;
    outer = 0;
    tm = (pair * kXcds + x) * 2 + (in & 1);
    tn = in >> 1;
  } else if constexpr (MODE == EXPERTS_GRAD) {
    // Each expert's tiles over all XCDs: the experts' lengths differ.
    const int per = a.tiles_m * a.tiles_n;
    outer = blockIdx.x / per;
    int shard;
    tile_coords(xcd_task(blockIdx.x - outer * per, per), a.tiles_m, a.tiles_n, shard, tm, tn);
  } else {
    tile_coords(xcd_task(blockIdx.x, a.tasks), a.tiles_m, a.tiles_n, outer, tm, tn);
  }
  j.n0 = tn * Cfg::BN;
  j.kbs = (a.K + kScaleBlock - 1) / kScaleBlock;
  j.steps = a.p * j.kbs;
  j.row0 = tm * Cfg::BM;
  j.rows = min(Cfg::BM, a.M - j.row0);
  j.wrow = j.n0;
  void* out = a.y[0];
  int64_t out_row = 0;
  if constexpr (MODE == GRAD) {
    j.s0 = outer;
    j.steps = j.kbs;
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
    ScScales<Cfg, MODE, WS> sc;
    ld.init(a, j);
    // Tiles of steps 0 and 1 (past the end the last step again, here as in the loop).
#pragma unroll
    for (int q = 0; q < Cfg::X_LOADS; ++q) ld.x_load(q, a.K, x_slot<Cfg, 0>());
#pragma unroll
    for (int q = 0; q < Cfg::W_LOADS; ++q) ld.w_load(q, a.K, w_slot<Cfg, 0>());
    ld.next(a, j.kbs);
#pragma unroll
    for (int q = 0; q < Cfg::X_LOADS; ++q) ld.x_load(q, a.K, x_slot<Cfg, 1>());
    if constexpr (Cfg::W_SLOTS == 2) {
#pragma unroll
      for (int q = 0; q < Cfg::W_LOADS; ++q) ld.w_load(q, a.K, w_slot<Cfg, 1>());
    }
    sc.init(a, j);                                 // behind the tiles' loads: one latency covers both
    wait_vmcnt(Cfg::X_LOADS + (Cfg::W_SLOTS == 2 ? Cfg::W_LOADS : 0));
    lds_barrier();
    ScOperands<Cfg, FINE> o;
    const ScPlace px(wm * Cfg::WM, lane), pw(wn * Cfg::WN, lane);
#pragma unroll
    for (int n = 0; n < Cfg::TN; ++n) sc_take(o.w[n], sc_read(w_slot<Cfg, 0>(), pw, n * 16));
#pragma unroll
    for (int i = 0; i < 2; ++i) o.x[0][i] = sc_read(x_slot<Cfg, 0>(), px, i * 16);
    for (int t = 0; t < j.steps; t += Cfg::UNROLL) sc_steps<Cfg, MODE, WS, FINE, 0>(acc, o, ld, sc, px, pw, a, j, t);
    wait_vmcnt(0);                                 // the repeated loads past the last step
  }

  constexpr int ES = OUT == OUT_F32 ? 4 : 2;
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(
      reinterpret_cast<char*>(out) + ((out_row + j.row0) * a.N + j.n0) * ES, (int64_t)j.rows * a.N * ES);
#pragma unroll
  for (int m = 0; m < Cfg::TM; ++m) {
    const int row = wm * Cfg::WM + m * 16 + r16;
    const int at = row < j.rows ? row * a.N : -1;
#pragma unroll
    for (int n = 0; n < Cfg::TN; n += 2) {
      f32x4_t v[2] = {acc[m][n], acc[m][n + 1]};
      if ((MODE == PLAIN || MODE == EXPERTS) && a.gelu) v[0] = sc_gelu<OUT>(v[0]), v[1] = sc_gelu<OUT>(v[1]);
      const int col0 = wn * Cfg::WN + n * 16;
      if constexpr (OUT == OUT_F32) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int col = col0 + i * 16 + 4 * (lane >> 4);
          const int off = at >= 0 && j.n0 + col < a.N ? (at + col) * ES : (int)kOOB;
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v[i]), rs, off, 0, 0);
        }
      } else {
        // Rows of 16 lanes exchange halves of two blocks, so that a lane stores eight columns: of the first block
        // lanes 0-15 the first eight and 32-47 the others, of the second lanes 16-31 and 48-63.
        const auto lo = __builtin_amdgcn_permlane16_swap(bf16_pair(v[0][0], v[0][1]), bf16_pair(v[1][0], v[1][1]), false, false);
        const auto hi = __builtin_amdgcn_permlane16_swap(bf16_pair(v[0][2], v[0][3]), bf16_pair(v[1][2], v[1][3]), false, false);
        const int col = col0 + (lane & 16) + 8 * (lane >> 5);
        const int off = at >= 0 && j.n0 + col < a.N ? (at + col) * ES : (int)kOOB;
        __builtin_amdgcn_raw_buffer_store_b128(u32x4_t{lo[0], hi[0], lo[1], hi[1]}, rs, off, 0, 0);
      }
    }
  }
}

using Big = ScCfg<256, 256, 2, 4, 2>;
using Tall = ScCfg<128, 256, 1, 4, 1>;
using Mid = ScCfg<128, 128, 2, 2, 2>;

template <class Cfg, int MODE, int WS, int OUT, int FINE = OUT == OUT_F32>
hipError_t launch_cfg(ScaledArgs a, hipStream_t s) {
  a.tiles_n = (a.N + Cfg::BN - 1) / Cfg::BN;
  a.tiles_m = (a.M + Cfg::BM - 1) / Cfg::BM;
  if (MODE == EXPERTS) a.tiles_m = (expert_tiles(a.M, a.E, Cfg::BM) + 2 * kXcds - 1) / (2 * kXcds) * (2 * kXcds);
  int64_t tasks = (int64_t)a.tiles_m * a.tiles_n;
  if (MODE == GRAD || MODE == EXPERTS_GRAD) tasks *= a.p * (MODE == EXPERTS_GRAD ? a.E : 1);
  if (tasks * Cfg::THREADS >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;
  a.tasks = (int)tasks;
  hipLaunchKernelGGL((scaled_tile_kernel<Cfg, MODE, WS, OUT, FINE>), dim3(a.tasks), dim3(Cfg::THREADS), 0, s, a);
  return hipGetLastError();
}

// Which tiles, by what their rounds over the compute units cost, in times of a
// 128 x 128 tile when they fill the chip:
//   256 x 256, one a compute unit, 750 a round of 256: half the LDS reads of four
//     small ones, 30 % faster where they fill the rounds;
//   128 x 256, two a compute unit, for experts, 825 a round of 512: as few LDS
//     reads but half as many rows lost at an expert's end, and a tile's start and
//     end beside the other's steps (so 700 where an expert's gradient sums up to
//     1024 rows), against half again the loads;
//   128 x 128, two a compute unit: 1 each and 110 for the start and the end.
// An expert's last tile counts as half full.  Where gradients change from 128 x 256 to
// 256 x 256, at 1024 rows an expert (us, 256 x 256 and 128 x 256): 16 of 4096 x 1024, 768
// rows 89 and 83, 1024 106 and 103, 1152 112 and 112, 1280 119 and 120, 2048 164 and 166;
// 64 of 1024 x 1024, 512 81 and 79, 1024 115 and 116, 1280 130 and 134, 2048 177 and 184; 4 of
// 4096 x 4096, 1024 85 and 82, 1280 96 and 95, 1536 112 and 116; but 8 of 2048 x 2048, 1280
// 56 and 52, 2560 89 and 89, 4096 138 and 148.  Measured, us, in this order: 4096 x
// 4096 x 4096: 60, 69, 77; 2560 x 4096: 53, 58, 58; 2048 x 4096: 52, 46, 42; 4352 x
// 4096, two rounds: 97, 88, 89.  64 experts of K 1024, N 4096, rows drawn evenly,
// 128 each: 103, 96, 107, 512: 219, 209, 257, drawn with a power of -0.7: 226, 207,
// 251; 16 experts of K and N 4096, 512: 170, 190, 194.  Gradients 16 x 4096 x 1024,
// rows an expert 512: 74, 69, 81, 4096: 283, 292, 352.
// The first two have no registers for partial sums: bf16 results and scales of
// powers of two only.
template <int MODE, int WS>
hipError_t launch_mode(const ScaledArgs& a, int64_t rows, int64_t outs, hipStream_t s) {
  if (a.out == OUT_F32) return launch_cfg<Mid, MODE, WS, OUT_F32>(a, s);
  if (a.fine) return launch_cfg<Mid, MODE, WS, OUT_BF16, 1>(a, s);
  if constexpr (WS != WS_F32) {
    constexpr bool TALL = MODE == EXPERTS || MODE == EXPERTS_GRAD;
    const auto tiles = [&](int64_t bm, int64_t bn) {
      const int64_t down = MODE == EXPERTS ? rows / bm + a.E / 2 : (rows + bm - 1) / bm;
      return down * ((a.N + bn - 1) / bn) * outs;
    };
    const int64_t big = (tiles(256, 256) + 255) / 256 * 750, mid = tiles(128, 128) + 110;
    if constexpr (TALL) {
      const bool brief = MODE == EXPERTS_GRAD && a.K <= (int64_t)1152 * a.E;      // 1024 rows and what fills their last block
      const int64_t tall = (tiles(128, 256) + 511) / 512 * (brief ? 700 : 825);
      if (tall < big && tall <= mid) return launch_cfg<Tall, MODE, WS, OUT_BF16>(a, s);
    }
    if (big <= mid) return launch_cfg<Big, MODE, WS, OUT_BF16>(a, s);
  }
  return launch_cfg<Mid, MODE, WS, OUT_BF16>(a, s);
}

}  // namespace

hipError_t launch_scaled_matmul(ScaledArgs a, int wscale, hipStream_t s) {
  if (const int few = scaled_few_tiles(a.M, a.N, a.p * scale_blocks(a.K), a.E)) return launch_scaled_few(a, wscale, few, s);
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
