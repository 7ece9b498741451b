// Weight gradients from 8-bit activations: dW_k = U_k^T dY_k, U = code * scale.
//
// The bf16 tile of tpf_gemm.hpp with its transposed A operand kept in 8 bits
// up to the registers: a step's A tile is 64 rows x BM bytes of codes (half a
// bf16 tile's LDS and global traffic), ds_read_b64_tr_b8 hands lane i of each
// 16-lane group the eight consecutive k of column i, and four conversions with
// the block's power of two make them the exact bf16 operand.  A 32-row MFMA
// operand lies within one 32 x 32 block, so its scale is the same for all lanes.
//
// The smaller A tile leaves LDS for three slots of both operands: the loads of
// step t + 2 go out between the MFMAs of step t's first three slices, one or
// two at a time, into the slot that step t - 1 left.
//
// 4 shards of 4096^3: 441 us a call, 1246 TFLOP/s, where a large library product of
// bf16 reaches 1259 on the same card: bound by the matrix cores at the clock they
// are held to (under a profiler 462 us there, 481 on a card whose library product
// reaches 1202).
// 2 x [1003, 1352 x 2056]: 19.0 us a call (586 TFLOP/s): 374 tiles of 128 x 128 leave
// 138 of 256 compute units with one tile and 118 with two, 0.8 us a step of 64 rows,
// and about 8 us go to the start, the first loads and the stores (10 with two-byte
// stores).
#include <algorithm>

#include "tpf_block.hpp"
#include "tpf_gemm.hpp"
#include "tpf_tiles.hpp"

namespace tpf {

__device__ __forceinline__ const StashGradArgs& sg_kernarg() {
  return *(const StashGradArgs*)__builtin_amdgcn_kernarg_segment_ptr();
}

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef int i32x2_t __attribute__((ext_vector_type(2)));

constexpr int kSgSteps = 512;    // steps whose scales are held in LDS at a time

template <class Cfg>
struct SgCfg {
  static_assert(Cfg::BK == 64 && (Cfg::BM == 256 || Cfg::BM == 128), "tile shape");
  static constexpr int LDS_Q = Cfg::BM * 64;
  static constexpr int Q_PER_WAVE = LDS_Q / 1024 / Cfg::NW;
  static constexpr int LOADS = Q_PER_WAVE + Cfg::B_PER_WAVE;
  static constexpr int RB = Cfg::BM / 32;          // scale blocks across the tile
  static_assert(LDS_Q % (1024 * Cfg::NW) == 0 && LOADS <= 2 * 3, "loads per slice");
  // 16-byte chunks of a row of codes are swizzled by k so that the eight rows
  // and two chunks of a 32-lane pass of the transposing read hit every bank once.
  __device__ __forceinline__ static int swz(int k) { return Cfg::BM == 256 ? 2 * (k & 7) : 2 * ((k >> 1) & 3); }
};

template <class Cfg, int S>
__device__ __forceinline__ char* q_slot() {
  __shared__ __attribute__((aligned(1024))) char buf[SgCfg<Cfg>::LDS_Q];
  return buf;
}
template <class Cfg>
__device__ __forceinline__ uint8_t* scale_slot() {
  __shared__ __attribute__((aligned(16))) uint8_t buf[(kSgSteps + 1) * 2 * (Cfg::BM / 32)];
  return buf;
}

template <class Cfg>
struct SgLoader {
  using S = SgCfg<Cfg>;
  __amdgpu_buffer_rsrc_t rq, rb;
  uint32_t q_off[S::Q_PER_WAVE], b_off[Cfg::B_PER_WAVE];   // byte offsets at step 0 (kOOB when out of range)
  uint32_t q_step, b_step;                                 // bytes from one step to the next
  int last;                                                // last step of the part

  __device__ __forceinline__ void init(const StashGradArgs& a, int k, int r0, int c0) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    rq = make_rsrc(a.codes[k], (int64_t)a.M * a.R);
    rb = make_rsrc(a.dY[k], (int64_t)a.M * a.C * 2);
    q_step = 64u * (uint32_t)a.R;
    b_step = 128u * (uint32_t)a.C;
    // Rows past M are out of the buffer's range by themselves; with fewer than
    // 64 rows the row's offset could pass 32 bits, so it is checked here.
#pragma unroll
    for (int i = 0; i < S::Q_PER_WAVE; ++i) {
      const int byte = (wave * S::Q_PER_WAVE + i) * 1024 + lane * 16;
      const int row = byte / Cfg::BM, c = ((byte % Cfg::BM) / 16) ^ S::swz(row);
      const int r = r0 + c * 16;
      q_off[i] = row < a.M && r < a.R ? (uint32_t)((int64_t)row * a.R + r) : kOOB;
    }
#pragma unroll
    for (int i = 0; i < Cfg::B_PER_WAVE; ++i) {
      constexpr int ROW_BYTES = Cfg::BN * 2;
      const int byte = (wave * Cfg::B_PER_WAVE + i) * 1024 + lane * 16;
      const int row = byte / ROW_BYTES, pchunk = (byte % ROW_BYTES) / 16;
      const int c = ((pchunk >> 1) ^ (Cfg::SWB * (row & 3))) * 2 + (pchunk & 1);
      const int n = c0 + c * 8;
      b_off[i] = row < a.M && n < a.C ? (uint32_t)(((int64_t)row * a.C + n) * 2) : kOOB;
    }
  }
  // Load q of step `step` (past the part's end its last step again, which
  // nothing reads): codes first, then dY.  The offset is a lane register, so
  // that the range check covers all of it.
  __device__ __forceinline__ void load(char* lq, char* lb, int step, int q) const {
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t st = (uint32_t)min(step, last);
    if (q < S::Q_PER_WAVE) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rq, (lds_void_t*)(lq + (wv * S::Q_PER_WAVE + q) * 1024), 16,
                                               (int)(q_off[q] + st * q_step), 0, 0, 0);
    } else {
      const int i = q - S::Q_PER_WAVE;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void_t*)(lb + (wv * Cfg::B_PER_WAVE + i) * 1024), 16,
                                               (int)(b_off[i] + st * b_step), 0, 0, 0);
    }
  }
};

// Operands of one 16-wide k slice: codes as read, dY in bf16.
template <class Cfg>
struct SgSlice {
  i32x2_t q[Cfg::TM];
  Operands<Cfg> o;
};

template <class Cfg>
__device__ __forceinline__ void sg_read(SgSlice<Cfg>& d, const char* lq, const char* lb, int s, int wm, int wn,
                                        int lane) {
  const int g = lane >> 4, jl = lane & 15;
  const int k = s * 16 + (g >> 1) * 8 + (jl >> 1);
#pragma unroll
  for (int i = 0; i < Cfg::TM; ++i) {
    const int c = (wm * Cfg::WM + i * 32) / 16 + (g & 1);
    const int off = k * Cfg::BM + ((c ^ SgCfg<Cfg>::swz(k)) * 16) + (jl & 1) * 8;
    d.q[i] = __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2_t*)((lds_void_t*)(lq + off)));
  }
  read_b<Cfg, B_KN>(d.o, lb, s, wm, wn, lane);
}

__device__ __forceinline__ float sg_scale(uint32_t word, int i) {
  return __uint_as_float(((word >> (8 * i)) & 0xffu) << 23);
}

// One slice's MFMAs, with loads Q0 .. Q1 - 1 of step `ahead` between them.
template <class Cfg, int Q0, int Q1>
__device__ __forceinline__ void sg_mfma(Frag<Cfg>& f, SgSlice<Cfg>& d, uint32_t scales, const SgLoader<Cfg>& ld,
                                        char* lq, char* lb, int ahead) {
#pragma unroll
  for (int i = 0; i < Cfg::TM; ++i) {
    const float sc = sg_scale(scales, i);
    const bf16x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d.q[i][0], sc, false);
    const bf16x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d.q[i][0], sc, true);
    const bf16x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d.q[i][1], sc, false);
    const bf16x2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d.q[i][1], sc, true);
    const bf16x8_t av = {p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
#pragma unroll
    for (int jn = 0; jn < Cfg::TN; ++jn)
      f.acc[i][jn] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(av, d.o.b[jn], f.acc[i][jn], 0, 0, 0);
    if (Q0 + i < Q1) ld.load(lq, lb, ahead, Q0 + i);
  }
}

template <class Cfg>
__device__ __forceinline__ uint32_t sg_words(int kb, int wm) {
  const uint8_t* p = scale_slot<Cfg>() + kb * SgCfg<Cfg>::RB + wm * Cfg::TM;
  if constexpr (Cfg::TM == 4) return *reinterpret_cast<const uint32_t*>(p);
  else return *reinterpret_cast<const uint16_t*>(p);
}

// Step kt on slot T; on entry d[0] holds its first slice and w its two words
// of scales.
template <class Cfg, int T>
__device__ __forceinline__ void sg_step(Frag<Cfg>& f, SgSlice<Cfg> (&d)[2], uint32_t (&w)[2], const SgLoader<Cfg>& ld,
                                        int kt, int kb, int wm, int wn, int lane) {
  constexpr int L = SgCfg<Cfg>::LOADS;
  constexpr int N1 = (L + 2) / 3, N2 = (2 * L + 2) / 3;
  const char* cq = q_slot<Cfg, T>();
  const char* cb = b_slot<Cfg, T>();
  char* fq = q_slot<Cfg, (T + 2) % 3>();
  char* fb = b_slot<Cfg, (T + 2) % 3>();
  sg_read<Cfg>(d[1], cq, cb, 1, wm, wn, lane);
  sg_mfma<Cfg, 0, N1>(f, d[0], w[0], ld, fq, fb, kt + 2);
  sg_read<Cfg>(d[0], cq, cb, 2, wm, wn, lane);
  sg_mfma<Cfg, N1, N2>(f, d[1], w[0], ld, fq, fb, kt + 2);
  sg_read<Cfg>(d[1], cq, cb, 3, wm, wn, lane);
  sg_mfma<Cfg, N2, L>(f, d[0], w[1], ld, fq, fb, kt + 2);
  wait_vmcnt(L);            // step kt + 1 has landed; only step kt + 2's loads are newer
  lds_barrier();
  sg_read<Cfg>(d[0], q_slot<Cfg, (T + 1) % 3>(), b_slot<Cfg, (T + 1) % 3>(), 0, wm, wn, lane);
  const uint32_t w1 = w[1];
  w[0] = sg_words<Cfg>(kb + 2, wm);
  w[1] = sg_words<Cfg>(kb + 3, wm);
  sg_mfma<Cfg, 0, 0>(f, d[1], w1, ld, fq, fb, 0);
}

// store_tile for bf16, two columns a store: neighbouring lanes hold neighbouring
// columns and exchange one of two rows, so that the even lane stores the first
// row and the odd lane the second.  C is even, so both columns are inside or not.
template <class Cfg>
__device__ __forceinline__ void store_tile_bf16(const Frag<Cfg>& f, const TileJob& j, void* out, int64_t ldo) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int wm = wave / Cfg::WAVES_N, wn = wave % Cfg::WAVES_N;
  const bool odd = lane & 1;
  const auto rs = make_rsrc(reinterpret_cast<char*>(out) + ((int64_t)j.m0 * ldo + j.n0) * 2, (int64_t)j.rows * ldo * 2);
  const int pitch = __builtin_amdgcn_readfirstlane((int)ldo * 2);
#pragma unroll
  for (int i = 0; i < Cfg::TM; ++i) {
#pragma unroll
    for (int jn = 0; jn < Cfg::TN; ++jn) {
      const int col = wn * Cfg::WN + jn * 32 + (lane & 30);
      const int row0 = wm * Cfg::WM + i * 32 + 4 * (lane >> 5) + odd;
#pragma unroll
      for (int v = 0; v < 16; v += 2) {
        const float a = f.acc[i][jn][v], b = f.acc[i][jn][v + 1];
        const float other = __int_as_float(
            __builtin_amdgcn_mov_dpp(__float_as_int(odd ? a : b), 0xB1, 0xf, 0xf, true));   // lanes 2 n and 2 n + 1
        const bf16x2_t two = {(__bf16)(odd ? other : a), (__bf16)(odd ? b : other)};
        const int row = row0 + 8 * (v >> 2) + (v & 3);
        const int off = row < j.rows && j.n0 + col < j.N ? row * pitch + col * 2 : (int)kOOB;
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, two), rs, off, 0, 0);
      }
    }
  }
}

template <class Cfg>
__global__ __launch_bounds__(Cfg::THREADS) void stash_grad_kernel(StashGradArgs args) {
  (void)args;
  using S = SgCfg<Cfg>;
  const StashGradArgs& a = sg_kernarg();
  const int part = blockIdx.y;
  const int u = xcd_task(blockIdx.x, a.tasks);
  int k, tm, tn;
  tile_coords(u, a.tiles_m, a.tiles_n, k, tm, tn);
  const int r0 = tm * Cfg::BM, c0 = tn * Cfg::BN;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int wm = wave / Cfg::WAVES_N, wn = wave % Cfg::WAVES_N;
  const int s0 = (int)((int64_t)a.steps * part / a.splits), s1 = (int)((int64_t)a.steps * (part + 1) / a.splits);
  Frag<Cfg> f;
#pragma unroll
  for (int i = 0; i < Cfg::TM; ++i)
#pragma unroll
    for (int jn = 0; jn < Cfg::TN; ++jn)
#pragma unroll
      for (int v = 0; v < 16; ++v) f.acc[i][jn][v] = 0.0f;
  SgLoader<Cfg> ld;
  ld.init(a, k, r0, c0);
  const int bands = (a.M + 31) / 32, nsc = (a.R + 31) / 32;
  // The scales of up to kSgSteps steps at a time; almost every call has one round.
  for (int b0 = s0; b0 < s1; b0 += kSgSteps) {
    const int b1 = min(b0 + kSgSteps, s1);
    ld.last = b1 - 1;
#pragma unroll
    for (int q = 0; q < S::LOADS; ++q) ld.load(q_slot<Cfg, 0>(), b_slot<Cfg, 0>(), b0, q);
#pragma unroll
    for (int q = 0; q < S::LOADS; ++q) ld.load(q_slot<Cfg, 1>(), b_slot<Cfg, 1>(), b0 + 1, q);
    // Behind the first tiles' loads, so that one latency covers both.
    const int words = (b1 - b0 + 1) * 2 * S::RB;     // a step more: its words are fetched, not used
    for (int i = threadIdx.x; i < words; i += Cfg::THREADS) {
      const int band = b0 * 2 + i / S::RB, col = (r0 >> 5) + i % S::RB;
      scale_slot<Cfg>()[i] = band < bands && col < nsc ? a.scales[k][(int64_t)band * nsc + col] : 0;
    }
    wait_vmcnt(S::LOADS);
    lds_barrier();
    SgSlice<Cfg> d[2];
    uint32_t w[2] = {sg_words<Cfg>(0, wm), sg_words<Cfg>(1, wm)};
    sg_read<Cfg>(d[0], q_slot<Cfg, 0>(), b_slot<Cfg, 0>(), 0, wm, wn, lane);
    for (int kt = b0; kt < b1; kt += 3) {
      const int kb = (kt - b0) * 2;
      sg_step<Cfg, 0>(f, d, w, ld, kt, kb, wm, wn, lane);
      if (kt + 1 >= b1) break;
      sg_step<Cfg, 1>(f, d, w, ld, kt + 1, kb + 2, wm, wn, lane);
      if (kt + 2 >= b1) break;
      sg_step<Cfg, 2>(f, d, w, ld, kt + 2, kb + 4, wm, wn, lane);
    }
    wait_vmcnt(0);   // the repeated loads past the last step
    __syncthreads();
  }
  TileJob j{};
  j.m0 = r0;
  j.rows = min(Cfg::BM, a.R - r0);
  j.n0 = c0;
  j.N = a.C;
  if (a.splits > 1)
    store_tile<Cfg, OUT_F32>(f, j, a.partial + ((int64_t)part * a.p + k) * a.R * a.C, a.C);
  else if (a.out == OUT_F32)
    store_tile<Cfg, OUT_F32>(f, j, a.dW[k], a.C);
  else
    store_tile_bf16<Cfg>(f, j, a.dW[k], a.C);
}

// The parts of a cut contraction, added in order, four elements a thread.
__global__ __launch_bounds__(256) void stash_grad_sum_kernel(StashGradArgs args) {
  (void)args;
  const StashGradArgs& a = sg_kernarg();
  const int k = blockIdx.y;
  const int64_t n = (int64_t)a.R * a.C, e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (e >= n) return;
  f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int i = 0; i < a.splits; ++i)
    s += *reinterpret_cast<const f32x4_t*>(a.partial + ((int64_t)i * a.p + k) * n + e);
  if (a.out == OUT_F32) {
    *reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(a.dW[k]) + e) = s;
  } else {
    u32x2_t w;
    w[0] = f32_to_bf16_bits(s[0]) | (f32_to_bf16_bits(s[1]) << 16);
    w[1] = f32_to_bf16_bits(s[2]) | (f32_to_bf16_bits(s[3]) << 16);
    *reinterpret_cast<u32x2_t*>(reinterpret_cast<uint16_t*>(a.dW[k]) + e) = w;
  }
}

using SgLarge = TileCfg<256, 256, 2, 4, 2, 64>;
using SgSmall = TileCfg<128, 128, 2, 2, 2, 64>;

static int64_t sg_tiles(int p, int64_t R, int64_t C, int b) { return p * ((R + b - 1) / b) * ((C + b - 1) / b); }

// 256 x 256 tiles when they come close to one a compute unit, else 128 x 128
// tiles, two of which share a unit.
static bool sg_large(int p, int64_t R, int64_t C) { return sg_tiles(p, R, C, 256) >= 192; }

int stash_grad_splits(int p, int64_t M, int64_t R, int64_t C) {
  if (sg_large(p, R, C)) return 1;
  const int64_t tiles = sg_tiles(p, R, C, 128), steps = (M + 63) / 64;
  return (int)std::max<int64_t>(1, std::min<int64_t>(512 / tiles, steps / 4));
}

template <class Cfg>
static void launch_sg(StashGradArgs& a, hipStream_t s) {
  a.tiles_m = (a.R + Cfg::BM - 1) / Cfg::BM;
  a.tiles_n = (a.C + Cfg::BN - 1) / Cfg::BN;
  a.tasks = a.p * a.tiles_m * a.tiles_n;
  hipLaunchKernelGGL(stash_grad_kernel<Cfg>, dim3((unsigned)a.tasks, (unsigned)a.splits), dim3(Cfg::THREADS), 0, s, a);
}

hipError_t launch_stash_weight_grad(StashGradArgs a, hipStream_t s) {
  a.steps = (a.M + 63) / 64;
  if (sg_large(a.p, a.R, a.C)) launch_sg<SgLarge>(a, s);
  else launch_sg<SgSmall>(a, s);
  if (a.splits > 1) {
    const int64_t n = (int64_t)a.R * a.C;
    hipLaunchKernelGGL(stash_grad_sum_kernel, dim3((unsigned)((n + 1023) / 1024), (unsigned)a.p), dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace tpf
