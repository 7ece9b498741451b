// The MLP block's operators around its matrix products: the norms before and
// after it, its activations kept in 8 bits, its products with 4-bit weights.
// Plain structs passed by value as kernel arguments.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tpf_device.hpp"
#include "tpf_internal.hpp"

namespace tpf {

enum GateKind : int { GATE_NONE = 0, GATE_CHANNEL = 1, GATE_TOKEN = 2 };

constexpr int kNormMaxH = 32768;     // a row is held in one workgroup's registers
constexpr int kStashBlock = 32;      // 8-bit activations: one scale per 32 x 32 values

// Outputs of this many bytes and more, the memory-side cache's size, are stored
// past the caches: no reader finds them there, and on their way through they
// cost lines still to be read (norm backward of 8192 x 8192 160 -> 155 us, GeLU
// backward of 8 x 2048 x 6144 128 -> 122 us).  Smaller ones stay for the kernel that
// reads them next: past the caches a norm of 4096 x 4096 takes 24.5 us by itself
// instead of 28.1, but norm, matrix product and norm of 2048 x 8192 216 instead of
// 204 and of 4096 x 8192 270 instead of 259.
constexpr int64_t kStreamBytes = (int64_t)256 << 20;

// ---------------------------------------------------------------------------
// Norms.
// ---------------------------------------------------------------------------
struct NormArgs {
  const void* x;                     // [M][H] residual stream (backward: after the block)
  const void* blocks[kMaxShards];    // [M][H] each: the block's output, or its p partial sums
  const void* w_pre;                 // [H]
  const void* w_post;                // [H]
  const void* gate;                  // [H], [M] or NULL
  void* x_out;                       // forward: [M][H]; backward: dx
  void* y;                           // forward: [M][H] bf16; backward: db
  float* stats;                      // [2][M]: 1/rms of the block's output, then of x_out (forward: may be NULL)
  const void* dy;                    // backward: [M][H] bf16
  const void* dx_out;                // backward: [M][H] (NULL: zeros)
  float* dw_pre;                     // backward: [H]
  float* dw_post;                    // backward: [H]
  float* dgate;                      // backward: [H], [M] or NULL
  float* partial;                    // backward: [groups][2][H] column sums
  int p, M, H;
  int x_f32, b_f32, w_f32;           // 1: fp32, 0: bf16
  int gate_kind;
  float alpha, beta, eps, offset;    // offset: 1 where the weights are stored as offsets from 1
  int groups;                        // backward: workgroups, each summing rows group, group + groups, ...
  uint32_t row0;                     // forward: the launch's first row
};

// Workgroups of the backward's row pass: a pure function of M and H, so that the
// workspace can be asked for without a GPU and the sums' order is the same on all.
int norm_backward_groups(int64_t M, int64_t H);
hipError_t launch_block_norm(const NormArgs& a, hipStream_t s);
hipError_t launch_block_norm_backward(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_columns(const NormArgs& a, hipStream_t s);

// ---------------------------------------------------------------------------
// Activations in 8 bits: e4m3 codes [M][F] and one power of two (its binary32
// exponent byte) per 32 x 32 block, [ceil(M / 32)][ceil(F / 32)].
// ---------------------------------------------------------------------------
struct StashArgs {
  const void* u[kMaxShards];         // pack: [M][F] bf16
  void* h[kMaxShards];               // [M][F] bf16: GeLU(u) (pack without GeLU: unused)
  uint8_t* codes[kMaxShards];
  uint8_t* scales[kMaxShards];
  const void* dh[kMaxShards];        // backward: [M][F] bf16
  void* du[kMaxShards];              // backward: [M][F] bf16
  int64_t unit0;                     // pack: the launch's first unit of 32 x 128
  int p, M, F;
};
hipError_t launch_stash_pack(const StashArgs& a, int gelu, hipStream_t s);
hipError_t launch_stash_backward(const StashArgs& a, int num_cus, hipStream_t s);

struct StashGradArgs {
  const uint8_t* codes[kMaxShards];  // [M][R]
  const uint8_t* scales[kMaxShards];
  const __bf16* dY[kMaxShards];      // [M][C]
  void* dW[kMaxShards];              // [R][C]
  int p, M, R, C;
  int out;                           // OUT_F32 or OUT_BF16
  float* partial;                    // splits > 1: [splits][p][R][C]
  int splits, steps;                 // the contraction's K steps, and the parts they are cut into
  int tiles_m, tiles_n, tasks;
};
// Parts that the contraction is cut into for these sizes (1: no workspace).
int stash_grad_splits(int p, int64_t M, int64_t R, int64_t C);
hipError_t launch_stash_weight_grad(StashGradArgs a, hipStream_t s);

// ---------------------------------------------------------------------------
// 4-bit weights: W_k[n][j] = (q - z) * s with one scale s (bf16) and zero
// point z (one byte, or 8 everywhere) per `group` consecutive j of a row.
// ---------------------------------------------------------------------------
struct QweightArgs {
  const __bf16* X[kMaxShards];       // [M][K]
  const uint8_t* codes[kMaxShards];  // [N][K / 2]
  const uint16_t* scales[kMaxShards];  // [N][K / group] bf16
  const uint8_t* zeros[kMaxShards];  // [N][K / group], or NULL: 8
  void* Y;                           // [M][N]
  int p, M, K, N, group;
  int gelu, out;
  float* partial;                    // splits > 1: [splits][M][N]
  int splits;
};
// Parts that the contraction is cut into for these sizes (1: no workspace).
int qweight_splits(int p, int64_t M, int64_t K, int64_t N);
hipError_t launch_qweight(const QweightArgs& a, hipStream_t s);

}  // namespace tpf
