// C ABI of the MLP block's operators around its matrix products: argument
// checks and launches.
#include <hip/hip_runtime.h>

#include <string>

#include "../../include/tpfuse.h"
#include "tpf_block.hpp"
#include "tpf_host.hpp"

using namespace tpf;

static_assert(TPF_NORM_MAX_H == kNormMaxH, "row limit mismatch");
static_assert(TPF_GATE_NONE == GATE_NONE && TPF_GATE_CHANNEL == GATE_CHANNEL && TPF_GATE_TOKEN == GATE_TOKEN,
              "gate kinds mismatch");

namespace {

int check_norm(int p, int64_t M, int64_t H, int x_dtype, int b_dtype, int w_dtype, const void* gate, int gate_kind) {
  int st;
  if ((st = check_shards(p))) return st;
  if ((st = check_sizes(M, H, 1, "M and H"))) return st;
  if (H % 8 != 0) return fail(TPF_ERR_ALIGNMENT, "H must be a multiple of 8");
  if (H > kNormMaxH) return fail(TPF_ERR_UNSUPPORTED, "H must be at most " + std::to_string(kNormMaxH));
  if (!valid_dtype(x_dtype) || !valid_dtype(b_dtype) || !valid_dtype(w_dtype))
    return fail(TPF_ERR_INVALID_ARG, "unknown dtype");
  if (gate_kind < TPF_GATE_NONE || gate_kind > TPF_GATE_TOKEN)
    return fail(TPF_ERR_INVALID_ARG, "unknown gate kind");
  if (gate_kind != TPF_GATE_NONE && (st = check_ptr(gate, "gate"))) return st;
  return TPF_OK;
}

NormArgs norm_args(int p, int64_t M, int64_t H, const void* x, int x_dtype, const void* const* blocks, int b_dtype,
                   const void* w_pre, const void* w_post, const void* gate, int gate_kind, int w_dtype, float alpha,
                   float beta, int unit_offset) {
  NormArgs a{};
  a.x = x;
  for (int k = 0; k < p; ++k) a.blocks[k] = blocks[k];
  a.w_pre = w_pre;
  a.w_post = w_post;
  a.gate = gate_kind == TPF_GATE_NONE ? nullptr : gate;
  a.p = p;
  a.M = (int)M;
  a.H = (int)H;
  a.x_f32 = x_dtype == TPF_F32;
  a.b_f32 = b_dtype == TPF_F32;
  a.w_f32 = w_dtype == TPF_F32;
  a.gate_kind = gate_kind;
  a.alpha = alpha;
  a.beta = beta;
  a.offset = unit_offset ? 1.0f : 0.0f;
  return a;
}

int check_stash(int p, int64_t M, int64_t F) {
  int st;
  if ((st = check_shards(p))) return st;
  if ((st = check_sizes(M, F, 1, "M and F"))) return st;
  if (F % 8 != 0) return fail(TPF_ERR_ALIGNMENT, "F must be a multiple of 8");
  if (M * F > (int64_t)1 << 36) return fail(TPF_ERR_UNSUPPORTED, "operand too large");
  return TPF_OK;
}

int check_stash_grad(int p, int64_t M, int64_t R, int64_t C) {
  int st;
  if ((st = check_shards(p))) return st;
  if ((st = check_sizes(M, R, C, "M, R and C"))) return st;
  if (R % 8 != 0 || C % 8 != 0) return fail(TPF_ERR_ALIGNMENT, "R and C must be multiples of 8");
  const int64_t lim = ((int64_t)1 << 31) - 1;
  if (M * R * 2 > lim || M * C * 2 > lim || R * C * 4 > lim)
    return fail(TPF_ERR_UNSUPPORTED, "each operand (in bf16) and each output must be smaller than 2 GiB");
  return TPF_OK;
}

int check_qweight(int p, int64_t M, int64_t K, int64_t N, int group) {
  int st;
  if ((st = check_shards(p))) return st;
  if ((st = check_sizes(M, K, N, "M, K and N"))) return st;
  if (group != 32 && group != 64 && group != 128)
    return fail(TPF_ERR_UNSUPPORTED, "the group must be 32, 64 or 128");
  if (K % group != 0) return fail(TPF_ERR_SHAPE, "K must be a multiple of the group");
  const int64_t lim = ((int64_t)1 << 31) - 1;
  if (M * K * 2 > lim || N * (K / 2) > lim || M * N * 4 > lim)
    return fail(TPF_ERR_UNSUPPORTED, "each operand and the output must be smaller than 2 GiB");
  if ((M + 15) / 16 > 65535) return fail(TPF_ERR_UNSUPPORTED, "M must be at most 16 * 65535");
  return TPF_OK;
}

}  // namespace

extern "C" {

int tpf_block_norm(tpf_handle h, int p, int64_t M, int64_t H, const void* x, int x_dtype,
                   const void* const* blocks, int b_dtype, const void* w_pre, const void* w_post,
                   const void* gate, int gate_kind, int w_dtype, float alpha, float beta, float eps,
                   int unit_offset, void* x_out, void* y, float* stats, void* stream) {
  return guarded([&]() -> int {
    int st;
    if ((st = check_norm(p, M, H, x_dtype, b_dtype, w_dtype, gate, gate_kind))) return st;
    if ((st = check_ptr(x, "x"))) return st;
    if ((st = check_ptrs(blocks, p, "blocks"))) return st;
    if ((st = check_ptr(w_pre, "w_pre"))) return st;
    if ((st = check_ptr(w_post, "w_post"))) return st;
    if ((st = check_ptr(x_out, "x_out"))) return st;
    if ((st = check_ptr(y, "y"))) return st;
    if (stats && !aligned(stats, 4)) return fail(TPF_ERR_ALIGNMENT, "stats is not 4-byte aligned");
    if ((st = check_handle(h))) return st;
    if ((st = set_device(h))) return st;
    NormArgs a = norm_args(p, M, H, x, x_dtype, blocks, b_dtype, w_pre, w_post, gate, gate_kind, w_dtype, alpha, beta,
                           unit_offset);
    a.eps = eps;
    a.x_out = x_out;
    a.y = y;
    a.stats = stats;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    TPF_TIMED(h, s, launch_block_norm(a, s));
    return TPF_OK;
  });
}

size_t tpf_block_norm_backward_ws(int64_t M, int64_t H) {
  if (M <= 0 || H <= 0 || M > INT32_MAX || H > kNormMaxH || H % 8 != 0) return 0;
  return (size_t)norm_backward_groups(M, H) * 2 * (size_t)H * sizeof(float);
}

int tpf_block_norm_backward(tpf_handle h, int p, int64_t M, int64_t H, const void* dy, const void* dx_out,
                            const void* x, int x_dtype, const void* const* blocks, int b_dtype,
                            const float* stats, const void* w_pre, const void* w_post, const void* gate,
                            int gate_kind, int w_dtype, float alpha, float beta, int unit_offset, void* dx,
                            void* db, float* dw_pre, float* dw_post, float* dgate, void* ws, size_t ws_bytes,
                            void* stream) {
  return guarded([&]() -> int {
    int st;
    if ((st = check_norm(p, M, H, x_dtype, b_dtype, w_dtype, gate, gate_kind))) return st;
    if ((st = check_ptr(dy, "dy"))) return st;
    if (dx_out && (st = check_ptr(dx_out, "dx_out"))) return st;
    if ((st = check_ptr(x, "x"))) return st;
    if ((st = check_ptrs(blocks, p, "blocks"))) return st;
    if ((st = check_ptr(stats, "stats"))) return st;
    if ((st = check_ptr(w_pre, "w_pre"))) return st;
    if ((st = check_ptr(w_post, "w_post"))) return st;
    if ((st = check_ptr(dx, "dx"))) return st;
    if ((st = check_ptr(db, "db"))) return st;
    if ((st = check_ptr(dw_pre, "dw_pre"))) return st;
    if ((st = check_ptr(dw_post, "dw_post"))) return st;
    if (gate_kind != TPF_GATE_NONE && (st = check_ptr(dgate, "dgate"))) return st;
    if ((st = check_ws(ws, ws_bytes, tpf_block_norm_backward_ws(M, H)))) return st;
    if ((st = check_handle(h))) return st;
    if ((st = set_device(h))) return st;
    NormArgs a = norm_args(p, M, H, x, x_dtype, blocks, b_dtype, w_pre, w_post, gate, gate_kind, w_dtype, alpha, beta,
                           unit_offset);
    a.stats = const_cast<float*>(stats);
    a.dy = dy;
    a.dx_out = dx_out;
    a.x_out = dx;
    a.y = db;
    a.dw_pre = dw_pre;
    a.dw_post = dw_post;
    a.dgate = dgate;
    a.partial = reinterpret_cast<float*>(ws);
    a.groups = norm_backward_groups(M, H);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    TPF_TIMED(h, s, launch_block_norm_backward(a, s));
    TPF_HIP(launch_norm_columns(a, s));
    return TPF_OK;
  });
}

int tpf_stash_pack(tpf_handle h, int p, int64_t M, int64_t F, const void* const* u, int gelu, void* const* act,
                   void* const* codes, void* const* scales, void* stream) {
  return guarded([&]() -> int {
    int st;
    if ((st = check_stash(p, M, F))) return st;
    if ((st = check_ptrs(u, p, "u"))) return st;
    if (gelu && (st = check_outs(act, p, "act", 16))) return st;
    if ((st = check_outs(codes, p, "codes", 8))) return st;
    if ((st = check_outs(scales, p, "scales", 1))) return st;
    if ((st = check_handle(h))) return st;
    if ((st = set_device(h))) return st;
    StashArgs a{};
    for (int k = 0; k < p; ++k) {
      a.u[k] = u[k];
      a.h[k] = gelu ? act[k] : nullptr;
      a.codes[k] = reinterpret_cast<uint8_t*>(codes[k]);
      a.scales[k] = reinterpret_cast<uint8_t*>(scales[k]);
    }
    a.p = p;
    a.M = (int)M;
    a.F = (int)F;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    TPF_TIMED(h, s, launch_stash_pack(a, gelu, s));
    return TPF_OK;
  });
}

int tpf_stash_backward(tpf_handle h, int p, int64_t M, int64_t F, const void* const* codes,
                       const void* const* scales, const void* const* dh, void* const* du, void* const* act,
                       void* stream) {
  return guarded([&]() -> int {
    int st;
    if ((st = check_stash(p, M, F))) return st;
    if ((st = check_ptrs_at(codes, p, "codes", 8))) return st;
    if ((st = check_ptrs_at(scales, p, "scales", 1))) return st;
    if ((st = check_ptrs(dh, p, "dh"))) return st;
    if ((st = check_outs(du, p, "du", 16))) return st;
    if ((st = check_outs(act, p, "act", 16))) return st;
    if ((st = check_handle(h))) return st;
    if ((st = set_device(h))) return st;
    StashArgs a{};
    for (int k = 0; k < p; ++k) {
      a.codes[k] = const_cast<uint8_t*>(reinterpret_cast<const uint8_t*>(codes[k]));
      a.scales[k] = const_cast<uint8_t*>(reinterpret_cast<const uint8_t*>(scales[k]));
      a.dh[k] = dh[k];
      a.du[k] = du[k];
      a.h[k] = act[k];
    }
    a.p = p;
    a.M = (int)M;
    a.F = (int)F;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    TPF_TIMED(h, s, launch_stash_backward(a, h->num_cus, s));
    return TPF_OK;
  });
}

size_t tpf_stash_weight_grad_ws(int p, int64_t M, int64_t R, int64_t C) {
  return guarded_size([&]() -> size_t {
    if (check_stash_grad(p, M, R, C) != TPF_OK) return 0;
    const int splits = stash_grad_splits(p, M, R, C);
    return splits > 1 ? (size_t)splits * p * R * C * sizeof(float) : 0;
  });
}

int tpf_stash_weight_grad(tpf_handle h, int p, int64_t M, int64_t R, int64_t C, const void* const* codes,
                          const void* const* scales, const void* const* dY, void* const* dW, int dw_dtype,
                          void* ws, size_t ws_bytes, void* stream) {
  return guarded([&]() -> int {
    int st;
    if ((st = check_stash_grad(p, M, R, C))) return st;
    if (!valid_dtype(dw_dtype)) return fail(TPF_ERR_INVALID_ARG, "unknown output dtype");
    if ((st = check_ptrs_at(codes, p, "codes", 8))) return st;
    if ((st = check_ptrs_at(scales, p, "scales", 1))) return st;
    if ((st = check_ptrs(dY, p, "dY"))) return st;
    if ((st = check_outs(dW, p, "dW", 16))) return st;
    if ((st = check_ws(ws, ws_bytes, tpf_stash_weight_grad_ws(p, M, R, C)))) return st;
    if ((st = check_handle(h))) return st;
    if ((st = set_device(h))) return st;
    StashGradArgs a{};
    for (int k = 0; k < p; ++k) {
      a.codes[k] = reinterpret_cast<const uint8_t*>(codes[k]);
      a.scales[k] = reinterpret_cast<const uint8_t*>(scales[k]);
      a.dY[k] = reinterpret_cast<const __bf16*>(dY[k]);
      a.dW[k] = dW[k];
    }
    a.p = p;
    a.M = (int)M;
    a.R = (int)R;
    a.C = (int)C;
    a.out = out_kind(dw_dtype);
    a.partial = reinterpret_cast<float*>(ws);
    a.splits = stash_grad_splits(p, M, R, C);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    TPF_TIMED(h, s, launch_stash_weight_grad(a, s));
    return TPF_OK;
  });
}

size_t tpf_qweight_matmul_ws(int p, int64_t M, int64_t K, int64_t N, int group) {
  return guarded_size([&]() -> size_t {
    if (check_qweight(p, M, K, N, group) != TPF_OK) return 0;
    const int splits = qweight_splits(p, M, K, N);
    return splits > 1 ? (size_t)splits * M * N * sizeof(float) : 0;
  });
}

int tpf_qweight_matmul(tpf_handle h, int p, int64_t M, int64_t K, int64_t N, int group, const void* const* X,
                       const void* const* codes, const void* const* scales, const void* const* zeros, int gelu,
                       void* Y, int y_dtype, void* ws, size_t ws_bytes, void* stream) {
  return guarded([&]() -> int {
    int st;
    if ((st = check_qweight(p, M, K, N, group))) return st;
    if (!valid_dtype(y_dtype)) return fail(TPF_ERR_INVALID_ARG, "unknown output dtype");
    if ((st = check_ptrs(X, p, "X"))) return st;
    if ((st = check_ptrs(codes, p, "codes"))) return st;
    if ((st = check_ptrs_at(scales, p, "scales", 2))) return st;
    if (zeros && (st = check_ptrs_at(zeros, p, "zeros", 1))) return st;
    if ((st = check_ptr(Y, "Y"))) return st;
    if ((st = check_ws(ws, ws_bytes, tpf_qweight_matmul_ws(p, M, K, N, group)))) return st;
    if ((st = check_handle(h))) return st;
    if ((st = set_device(h))) return st;
    QweightArgs a{};
    for (int k = 0; k < p; ++k) {
      a.X[k] = reinterpret_cast<const __bf16*>(X[k]);
      a.codes[k] = reinterpret_cast<const uint8_t*>(codes[k]);
      a.scales[k] = reinterpret_cast<const uint16_t*>(scales[k]);
      a.zeros[k] = zeros ? reinterpret_cast<const uint8_t*>(zeros[k]) : nullptr;
    }
    a.Y = Y;
    a.p = p;
    a.M = (int)M;
    a.K = (int)K;
    a.N = (int)N;
    a.group = group;
    a.gelu = gelu;
    a.out = out_kind(y_dtype);
    a.partial = reinterpret_cast<float*>(ws);
    a.splits = qweight_splits(p, M, K, N);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    TPF_TIMED(h, s, launch_qweight(a, s));
    return TPF_OK;
  });
}

}  // extern "C"
