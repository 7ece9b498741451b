// Products of operands in 8 bits with a scale for each block of 128, and the
// MLP block of experts.  Plain structs passed by value as kernel arguments.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tpf_device.hpp"
#include "tpf_internal.hpp"

namespace tpf {

constexpr int kScaleBlock = 128;      // values along the contraction that share a scale
constexpr int kExpertMaxE = 1024;     // experts
constexpr int kExpertMaxK = 16;       // experts of one token
constexpr int kExpertMaxGroups = 16;

enum ScoreKind : int { SCORE_SOFTMAX = 0, SCORE_SIGMOID = 1 };

// Two values rounded to bf16 (nearest even), the first in the low half.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  const bf16x2_t v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}

constexpr int64_t scale_blocks(int64_t n) { return (n + kScaleBlock - 1) / kScaleBlock; }
// Scale bytes of a packed row of n values: whole words, so that one word load
// brings four blocks' scales.
constexpr int64_t scale_width(int64_t n) { return (scale_blocks(n) + 3) / 4 * 4; }
// Columns of a packed transpose whose R rows belong to E experts, each expert's
// padded to whole blocks: the most that any loads of the experts can need.
constexpr int64_t expert_columns(int64_t R, int64_t E) {
  return (R + (kScaleBlock - 1) * (E < R ? E : R)) / kScaleBlock * kScaleBlock;
}

// ---------------------------------------------------------------------------
// Packing: e4m3 codes and one exponent byte per 128 values along a row (or,
// transposed, down a column).
// ---------------------------------------------------------------------------
struct PackArgs {
  const void* u[kMaxShards];         // [rows of u][K] bf16
  uint8_t* codes[kMaxShards];        // [M][K], or NULL
  uint8_t* scales[kMaxShards];       // [M][width]
  uint8_t* codes_t[kMaxShards];      // [K][columns], or NULL
  uint8_t* scales_t[kMaxShards];     // [K][width of columns]
  const int* offsets;                // experts' first rows [E + 1], or NULL: rows as they are
  const int* src;                    // slot of each row: row r is u[src / top]; NULL: u[r]
  int p, M, K;                       // M: rows of u
  int R;                             // rows of the transpose's layout
  int E, top;
  int columns;                       // multiple of 128
};
hipError_t launch_scaled_pack(const PackArgs& a, hipStream_t s);

// ---------------------------------------------------------------------------
// Products.  y[m][n] = sum over blocks b of 2^(xs - 127) * ws * sum x w over the
// block, both operands stored along the contraction.
// ---------------------------------------------------------------------------
enum WScale : int { WS_BYTE = 0, WS_F32 = 1, WS_ROW = 2 };   // one per 128 x 128 (byte, fp32), or as x's

struct ScaledArgs {
  const uint8_t* x[kMaxShards];      // [rows][K] codes
  const uint8_t* xs[kMaxShards];     // [rows][xsw] exponent bytes
  const uint8_t* w[kMaxShards];      // [N][K] codes; experts: [E][N][K]
  const uint8_t* ws[kMaxShards];     // [ceil(N / 128)][wsw] (experts: [E] of them), or [N][wsw] as x's
  void* y[kMaxShards];
  const int* offsets;                // experts' first rows [E + 1]
  const int* src;                    // slot of each row
  int p;                             // shards summed; weight gradients: outputs
  int M, K, N;                       // rows of the result, length of an operand's rows, columns
  int xrows;                         // rows of x
  int xsw, wsw;
  int E, top;                        // top: slots a token where x's rows are tokens (0: x's rows are the result's)
  int gelu, out;
  int fine;                          // sums in fp32 whatever the result's type
  int tiles_m, tiles_n, tasks;
};
// Tiles of 16 rows that the kernel for few rows takes for M rows (of E experts),
// 0: the large tiles take them.
int scaled_few_tiles(int64_t M, int64_t N, int64_t blocks, int64_t E);
hipError_t launch_scaled_few(const ScaledArgs& a, int wscale, int tiles, hipStream_t s);
hipError_t launch_scaled_matmul(ScaledArgs a, int wscale, hipStream_t s);        // E > 0: experts' rows
hipError_t launch_scaled_weight_grad(ScaledArgs a, hipStream_t s);               // E > 0: experts' gradients

// ---------------------------------------------------------------------------
// Routing.
// ---------------------------------------------------------------------------
struct RouteArgs {
  const void* logits;                // [T][E]
  const float* bias;                 // [E] or NULL
  const uint8_t* mask;               // [T] or NULL
  int* ids;                          // [T][k]
  float* weights;                    // [T][k]
  int* offsets;                      // [E + 1]
  int* src;                          // [T k]
  int* pos;                          // [T][k]
  uint16_t* hist;                    // [E][pad]: rows of each expert in each part
  int T, E, k;
  int score, groups, top_groups, renorm;
  double scale;
  int logits_f32;
  int chunks, chunk, pad;            // parts of the tokens, tokens in each; chunks rounded up to 4
};
// Parts that T tokens are cut into: each counts its experts' rows by itself.
int route_chunks(int64_t T, int64_t* chunk);
hipError_t launch_expert_route(const RouteArgs& a, hipStream_t s);

struct RouteGradArgs {
  const void* logits;                // [T][E]
  const int* ids;                    // [T][k]
  const float* weights;              // [T][k]
  const float* dweights;             // [T][k]
  void* dlogits;                     // [T][E], the logits' type
  int T, E, k;
  int score, renorm;
  double scale;
  int logits_f32;
};
hipError_t launch_expert_route_backward(const RouteGradArgs& a, hipStream_t s);

struct CombineArgs {
  const void* rows;                  // [T k][H]
  const float* weights;              // [T][k]
  const int* pos;                    // [T][k]
  const int* offsets;                // backward: [E + 1]
  void* y;                           // forward: [T][H]
  const void* dy;                    // backward: [T][H]
  void* drows;                       // backward: [T k][H]
  float* dweights;                   // backward: [T][k]
  int T, k, H, E;
  int rows_f32, y_f32;               // 1: fp32, 0: bf16 (dy and y: y_f32; drows: rows_f32)
};
hipError_t launch_expert_combine(const CombineArgs& a, hipStream_t s);
hipError_t launch_expert_combine_backward(const CombineArgs& a, hipStream_t s);

}  // namespace tpf
