// C ABI of the 8-bit Linears and of the MLP block of experts: argument checks and
// launches.
#include <hip/hip_runtime.h>

#include <cmath>
#include <string>

#include "../../include/tpfuse.h"
#include "tpf_host.hpp"
#include "tpf_scaled.hpp"

using namespace tpf;

static_assert(TPF_SCALE_BYTE == WS_BYTE && TPF_SCALE_F32 == WS_F32, "scale types mismatch");
static_assert(TPF_SCORE_SOFTMAX == SCORE_SOFTMAX && TPF_SCORE_SIGMOID == SCORE_SIGMOID, "scores mismatch");
static_assert(TPF_EXPERT_MAX_E == kExpertMaxE && TPF_EXPERT_MAX_K == kExpertMaxK &&
              TPF_EXPERT_MAX_GROUPS == kExpertMaxGroups, "limits mismatch");

namespace {

// The handle's device for one call; the thread's current one afterwards.
struct OnDevice {
  int before = -1;
  hipError_t error;
  explicit OnDevice(int device) {
    error = hipGetDevice(&before);
    if (error == hipSuccess && before != device) error = hipSetDevice(device);
    else before = -1;
  }
  ~OnDevice() {
    if (before >= 0) (void)hipSetDevice(before);
  }
};

#define TPF_ON_DEVICE(h)                \
  if (int st_ = check_handle(h)) return st_; \
  OnDevice on_device_((h)->device);     \
  TPF_HIP(on_device_.error)

int check_packed(int64_t rows, int64_t K, const char* names) {
  int st;
  if ((st = check_sizes(rows, K, 1, names))) return st;
  if (K % 16 != 0) return fail(TPF_ERR_ALIGNMENT, "a packed row's length must be a multiple of 16");
  if (K > 1 << 22) return fail(TPF_ERR_UNSUPPORTED, "a packed row's length must be at most 2^22");
  if (rows * K > (int64_t)1 << 40) return fail(TPF_ERR_UNSUPPORTED, "operand too large");
  return TPF_OK;
}

// Rows and columns of a product and the number of them in one launch.
int check_product(int64_t M, int64_t N, int64_t outs) {
  if (int st = check_sizes(M, N, 1, "the result's sizes")) return st;
  if (N % 8 != 0) return fail(TPF_ERR_ALIGNMENT, "the result's width must be a multiple of 8");
  if (N > 1 << 20) return fail(TPF_ERR_UNSUPPORTED, "the result's width must be at most 2^20");
  // a launch's limit of 2^32 threads, 512 to 256 x 256 results
  if ((double)((M + 255) / 256) * (double)((N + 255) / 256) * (double)outs > 8.0e6)
    return fail(TPF_ERR_UNSUPPORTED, "too many results for one call");
  return TPF_OK;
}

int check_experts(int64_t E) {
  if (E < 1 || E > kExpertMaxE)
    return fail(TPF_ERR_UNSUPPORTED, "the experts must be 1 to " + std::to_string(kExpertMaxE));
  return TPF_OK;
}

// Rows that are slots of tokens: `top` slots each, 0 where rows are taken as they lie.
int check_slots(int64_t R, int top, const int32_t* src) {
  if (top < 0 || top > kExpertMaxK) return fail(TPF_ERR_SHAPE, "top must be 0 to " + std::to_string(kExpertMaxK));
  if (top && R % top != 0) return fail(TPF_ERR_SHAPE, "the rows must be a multiple of top");
  if (top && !src) return fail(TPF_ERR_INVALID_ARG, "src is NULL");
  if (top && !aligned(src, 4)) return fail(TPF_ERR_ALIGNMENT, "src is not 4-byte aligned");
  return TPF_OK;
}

int check_ints(const void* p, const char* name) {
  if (!p) return fail(TPF_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if (!aligned(p, 4)) return fail(TPF_ERR_ALIGNMENT, std::string(name) + " is not 4-byte aligned");
  return TPF_OK;
}

int check_scale_type(int t) {
  if (t != TPF_SCALE_BYTE && t != TPF_SCALE_F32) return fail(TPF_ERR_INVALID_ARG, "unknown scale type");
  return TPF_OK;
}

int check_route(int64_t T, int64_t E, int k, int dtype, int score, double scale) {
  int st;
  if ((st = check_sizes(T, E, 1, "T and E"))) return st;
  if ((st = check_experts(E))) return st;
  if (k < 1 || k > kExpertMaxK || k > E)
    return fail(TPF_ERR_SHAPE, "k must be 1 to " + std::to_string(kExpertMaxK) + " and at most E");
  // parts of the tokens are counted in 32 bits up to the end of the last one
  if (T > INT32_MAX - (1 << 17) || T * k > INT32_MAX) return fail(TPF_ERR_SHAPE, "T k must fit in 31 bits, T within 2^31 - 2^17");
  if (!valid_dtype(dtype)) return fail(TPF_ERR_INVALID_ARG, "unknown dtype");
  if (score != TPF_SCORE_SOFTMAX && score != TPF_SCORE_SIGMOID) return fail(TPF_ERR_INVALID_ARG, "unknown score");
  if (!std::isfinite(scale) || scale == 0.0) return fail(TPF_ERR_INVALID_ARG, "scale must be finite and not 0");
  return TPF_OK;
}

int check_combine(int64_t T, int k, int64_t H, int rows_dtype, int y_dtype) {
  int st;
  if ((st = check_sizes(T, H, 1, "T and H"))) return st;
  if (k < 1 || k > kExpertMaxK) return fail(TPF_ERR_SHAPE, "k must be 1 to " + std::to_string(kExpertMaxK));
  if (T * k > INT32_MAX) return fail(TPF_ERR_SHAPE, "T k must fit in 31 bits");
  if (H % 8 != 0) return fail(TPF_ERR_ALIGNMENT, "H must be a multiple of 8");
  if (H > 1 << 24) return fail(TPF_ERR_UNSUPPORTED, "H must be at most 2^24");
  if (!valid_dtype(rows_dtype) || !valid_dtype(y_dtype)) return fail(TPF_ERR_INVALID_ARG, "unknown dtype");
  return TPF_OK;
}

void set_operands(ScaledArgs& a, int p, const void* const* X, const void* const* xs, const void* const* W,
                  const void* const* ws) {
  for (int k = 0; k < p; ++k) {
    a.x[k] = reinterpret_cast<const uint8_t*>(X[k]);
    a.xs[k] = reinterpret_cast<const uint8_t*>(xs[k]);
    a.w[k] = reinterpret_cast<const uint8_t*>(W[k]);
    a.ws[k] = reinterpret_cast<const uint8_t*>(ws[k]);
  }
  a.p = p;
}

// E = 0: a plain product of M rows; otherwise the experts'.
int scaled_matmul(tpf_handle h, int p, int64_t M, int64_t K, int64_t N, int64_t E, const void* const* X,
                  const void* const* x_scales, const void* const* W, const void* const* w_scales, int w_scale_type,
                  const int32_t* offsets, const int32_t* src, int top, int gelu, void* Y, int y_dtype, void* stream) {
  int st;
  if ((st = check_shards(p))) return st;
  if ((st = check_packed(M, K, "the rows and K"))) return st;
  if ((st = check_product(M + (E ? 256 * (E + 1) : 0), N, 1))) return st;
  if (N * K > (int64_t)1 << 40) return fail(TPF_ERR_UNSUPPORTED, "operand too large");
  if (E) {
    if ((st = check_slots(M, top, src))) return st;
    if (top && M / top * K > ((int64_t)1 << 31) - 1)
      return fail(TPF_ERR_UNSUPPORTED, "the rows that are gathered must be smaller than 2 GiB");
    if ((st = check_ints(offsets, "offsets"))) return st;
  }
  if ((st = check_scale_type(w_scale_type))) return st;
  const int fine = y_dtype & TPF_SUMS_F32;
  y_dtype -= fine;
  if (!valid_dtype(y_dtype)) return fail(TPF_ERR_INVALID_ARG, "unknown output dtype");
  if ((st = check_ptrs(X, p, "X"))) return st;
  if ((st = check_ptrs_at(x_scales, p, "x_scales", 4))) return st;
  if ((st = check_ptrs(W, p, "W"))) return st;
  if ((st = check_ptrs_at(w_scales, p, "w_scales", w_scale_type == TPF_SCALE_F32 ? 4 : 1))) return st;
  if ((st = check_ptr(Y, "Y"))) return st;
  TPF_ON_DEVICE(h);
  ScaledArgs a{};
  set_operands(a, p, X, x_scales, W, w_scales);
  a.y[0] = Y;
  a.M = (int)M;
  a.K = (int)K;
  a.N = (int)N;
  a.xrows = (int)(top ? M / top : M);
  a.xsw = (int)scale_width(K);
  a.wsw = (int)scale_blocks(K);
  a.E = (int)E;
  a.top = top;
  a.offsets = offsets;
  a.src = src;
  a.gelu = gelu;
  a.out = out_kind(y_dtype);
  a.fine = fine;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  TPF_TIMED(h, s, launch_scaled_matmul(a, w_scale_type, s));
  return TPF_OK;
}

int scaled_weight_grad(tpf_handle h, int p, int64_t Mt, int64_t R, int64_t C, int64_t E, const void* const* A,
                       const void* const* a_scales, const void* const* B, const void* const* b_scales,
                       const int32_t* offsets, void* const* dW, int dw_dtype, void* stream) {
  int st;
  if ((st = check_shards(p))) return st;
  if ((st = check_packed(R, Mt, "R and Mt"))) return st;
  if (Mt % kScaleBlock != 0) return fail(TPF_ERR_SHAPE, "Mt must be a multiple of 128");
  if ((st = check_packed(C, Mt, "C and Mt"))) return st;
  if ((st = check_product(R, C, (int64_t)p * (E ? E : 1)))) return st;
  if (E && (st = check_ints(offsets, "offsets"))) return st;
  const int fine = dw_dtype & TPF_SUMS_F32;
  dw_dtype -= fine;
  if (!valid_dtype(dw_dtype)) return fail(TPF_ERR_INVALID_ARG, "unknown output dtype");
  if ((st = check_ptrs(A, p, "A"))) return st;
  if ((st = check_ptrs_at(a_scales, p, "a_scales", 4))) return st;
  if ((st = check_ptrs(B, p, "B"))) return st;
  if ((st = check_ptrs_at(b_scales, p, "b_scales", 4))) return st;
  if ((st = check_outs(dW, p, "dW", 16))) return st;
  TPF_ON_DEVICE(h);
  ScaledArgs a{};
  set_operands(a, p, A, a_scales, B, b_scales);
  for (int k = 0; k < p; ++k) a.y[k] = dW[k];
  a.M = (int)R;
  a.K = (int)Mt;
  a.N = (int)C;
  a.xrows = (int)R;
  a.xsw = a.wsw = (int)scale_width(Mt);
  a.E = (int)E;
  a.offsets = offsets;
  a.out = out_kind(dw_dtype);
  a.fine = fine;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  TPF_TIMED(h, s, launch_scaled_weight_grad(a, s));
  return TPF_OK;
}

}  // namespace

extern "C" {

int64_t tpf_expert_columns(int64_t R, int64_t E) {
  if (R < 1 || R > INT32_MAX || E < 1 || E > kExpertMaxE) return 0;
  return expert_columns(R, E);
}

int tpf_scaled_pack(tpf_handle h, int p, int64_t M, int64_t K, const void* const* u, void* const* codes,
                    void* const* scales, void* const* codes_t, void* const* scales_t, int64_t E,
                    const int32_t* offsets, const int32_t* src, int top, void* stream) {
  return guarded([&]() -> int {
    int st;
    if ((st = check_shards(p))) return st;
    if ((st = check_packed(M, K, "M and K"))) return st;
    if ((st = check_ptrs(u, p, "u"))) return st;
    if (!codes != !scales) return fail(TPF_ERR_INVALID_ARG, "codes and scales go together");
    if (!codes_t != !scales_t) return fail(TPF_ERR_INVALID_ARG, "codes_t and scales_t go together");
    if (!codes && !codes_t) return fail(TPF_ERR_INVALID_ARG, "no output is asked for");
    if (codes && (st = check_outs(codes, p, "codes", 16))) return st;
    if (codes && (st = check_outs(scales, p, "scales", 4))) return st;
    int64_t R = M, columns = scale_blocks(M) * kScaleBlock;
    if (codes_t) {
      if ((st = check_outs(codes_t, p, "codes_t", 16))) return st;
      if ((st = check_outs(scales_t, p, "scales_t", 4))) return st;
      if (E) {
        if ((st = check_experts(E))) return st;
        if (top) R = M * top;
        if ((st = check_slots(R, top, src))) return st;
        if ((st = check_ints(offsets, "offsets"))) return st;
        if (R > INT32_MAX) return fail(TPF_ERR_SHAPE, "the experts' rows must fit in 31 bits");
        columns = expert_columns(R, E);
      }
      if (columns > 1 << 22) return fail(TPF_ERR_UNSUPPORTED, "the transpose must have at most 2^22 columns");
      if (K > 1 << 20) return fail(TPF_ERR_UNSUPPORTED, "the transpose must have at most 2^20 rows");
    }
    TPF_ON_DEVICE(h);
    PackArgs a{};
    for (int k = 0; k < p; ++k) {
      a.u[k] = u[k];
      a.codes[k] = codes ? reinterpret_cast<uint8_t*>(codes[k]) : nullptr;
      a.scales[k] = codes ? reinterpret_cast<uint8_t*>(scales[k]) : nullptr;
      a.codes_t[k] = codes_t ? reinterpret_cast<uint8_t*>(codes_t[k]) : nullptr;
      a.scales_t[k] = codes_t ? reinterpret_cast<uint8_t*>(scales_t[k]) : nullptr;
    }
    a.offsets = E ? offsets : nullptr;
    a.src = E && top ? src : nullptr;
    a.p = p;
    a.M = (int)M;
    a.K = (int)K;
    a.R = (int)R;
    a.E = (int)E;
    a.top = top;
    a.columns = (int)columns;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    TPF_TIMED(h, s, launch_scaled_pack(a, s));
    return TPF_OK;
  });
}

int tpf_scaled_matmul(tpf_handle h, int p, int64_t M, int64_t K, int64_t N, const void* const* X,
                      const void* const* x_scales, const void* const* W, const void* const* w_scales,
                      int w_scale_type, int gelu, void* Y, int y_dtype, void* stream) {
  return guarded([&]() -> int {
    return scaled_matmul(h, p, M, K, N, 0, X, x_scales, W, w_scales, w_scale_type, nullptr, nullptr, 0, gelu, Y,
                         y_dtype, stream);
  });
}

int tpf_scaled_weight_grad(tpf_handle h, int p, int64_t Mt, int64_t R, int64_t C, const void* const* A,
                           const void* const* a_scales, const void* const* B, const void* const* b_scales,
                           void* const* dW, int dw_dtype, void* stream) {
  return guarded([&]() -> int {
    return scaled_weight_grad(h, p, Mt, R, C, 0, A, a_scales, B, b_scales, nullptr, dW, dw_dtype, stream);
  });
}

int tpf_expert_matmul(tpf_handle h, int p, int64_t R, int64_t K, int64_t N, int64_t E, const void* const* X,
                      const void* const* x_scales, const void* const* W, const void* const* w_scales,
                      int w_scale_type, const int32_t* offsets, const int32_t* src, int top, int gelu, void* Y,
                      int y_dtype, void* stream) {
  return guarded([&]() -> int {
    if (int st = check_experts(E)) return st;
    return scaled_matmul(h, p, R, K, N, E, X, x_scales, W, w_scales, w_scale_type, offsets, src, top, gelu, Y, y_dtype,
                         stream);
  });
}

int tpf_expert_weight_grad(tpf_handle h, int p, int64_t Mt, int64_t R, int64_t C, int64_t E, const void* const* A,
                           const void* const* a_scales, const void* const* B, const void* const* b_scales,
                           const int32_t* offsets, void* const* dW, int dw_dtype, void* stream) {
  return guarded([&]() -> int {
    if (int st = check_experts(E)) return st;
    return scaled_weight_grad(h, p, Mt, R, C, E, A, a_scales, B, b_scales, offsets, dW, dw_dtype, stream);
  });
}

size_t tpf_expert_route_ws(int64_t T, int64_t E) {
  if (T < 1 || T > INT32_MAX || E < 1 || E > kExpertMaxE) return 0;
  return (size_t)((route_chunks(T, nullptr) + 3) / 4 * 4) * (size_t)E * sizeof(uint16_t);
}

int tpf_expert_route(tpf_handle h, int64_t T, int64_t E, int k, const void* logits, int dtype, int score,
                     const float* bias, int groups, int top_groups, int renorm, double scale, const uint8_t* mask,
                     int32_t* ids, float* weights, int32_t* offsets, int32_t* src, int32_t* pos, void* ws,
                     size_t ws_bytes, void* stream) {
  return guarded([&]() -> int {
    int st;
    if ((st = check_route(T, E, k, dtype, score, scale))) return st;
    if (groups < 1 || groups > kExpertMaxGroups || E % groups != 0)
      return fail(TPF_ERR_SHAPE, "groups must be 1 to " + std::to_string(kExpertMaxGroups) + " and divide E");
    if (top_groups < 1 || top_groups > groups) return fail(TPF_ERR_SHAPE, "top_groups must be 1 to groups");
    if (k > E / groups * top_groups) return fail(TPF_ERR_SHAPE, "k must be at most the experts of top_groups groups");
    if ((st = check_ptr(logits, "logits"))) return st;
    if (bias && (st = check_ints(bias, "bias"))) return st;
    if ((st = check_ints(ids, "ids"))) return st;
    if ((st = check_ints(weights, "weights"))) return st;
    if ((st = check_ints(offsets, "offsets"))) return st;
    if ((st = check_ints(src, "src"))) return st;
    if ((st = check_ints(pos, "pos"))) return st;
    if ((st = check_ws(ws, ws_bytes, tpf_expert_route_ws(T, E)))) return st;
    TPF_ON_DEVICE(h);
    RouteArgs a{};
    a.logits = logits;
    a.bias = bias;
    a.mask = mask;
    a.ids = ids;
    a.weights = weights;
    a.offsets = offsets;
    a.src = src;
    a.pos = pos;
    a.hist = reinterpret_cast<uint16_t*>(ws);
    a.T = (int)T;
    a.E = (int)E;
    a.k = k;
    a.score = score;
    a.groups = groups;
    a.top_groups = top_groups;
    a.renorm = renorm;
    a.scale = scale;
    a.logits_f32 = dtype == TPF_F32;
    int64_t chunk;
    a.chunks = route_chunks(T, &chunk);
    a.chunk = (int)chunk;
    a.pad = (a.chunks + 3) / 4 * 4;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    TPF_TIMED(h, s, launch_expert_route(a, s));
    return TPF_OK;
  });
}

int tpf_expert_route_backward(tpf_handle h, int64_t T, int64_t E, int k, const void* logits, int dtype, int score,
                              int renorm, double scale, const int32_t* ids, const float* weights,
                              const float* dweights, void* dlogits, void* stream) {
  return guarded([&]() -> int {
    int st;
    if ((st = check_route(T, E, k, dtype, score, scale))) return st;
    if ((st = check_ptr(logits, "logits"))) return st;
    if ((st = check_ints(ids, "ids"))) return st;
    if ((st = check_ints(weights, "weights"))) return st;
    if ((st = check_ints(dweights, "dweights"))) return st;
    if ((st = check_ptr(dlogits, "dlogits"))) return st;
    TPF_ON_DEVICE(h);
    RouteGradArgs a{};
    a.logits = logits;
    a.ids = ids;
    a.weights = weights;
    a.dweights = dweights;
    a.dlogits = dlogits;
    a.T = (int)T;
    a.E = (int)E;
    a.k = k;
    a.score = score;
    a.renorm = renorm;
    a.scale = scale;
    a.logits_f32 = dtype == TPF_F32;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    TPF_TIMED(h, s, launch_expert_route_backward(a, s));
    return TPF_OK;
  });
}

int tpf_expert_combine(tpf_handle h, int64_t T, int k, int64_t H, const void* rows, int rows_dtype,
                       const float* weights, const int32_t* pos, void* y, int y_dtype, void* stream) {
  return guarded([&]() -> int {
    int st;
    if ((st = check_combine(T, k, H, rows_dtype, y_dtype))) return st;
    if ((st = check_ptr(rows, "rows"))) return st;
    if ((st = check_ints(weights, "weights"))) return st;
    if ((st = check_ints(pos, "pos"))) return st;
    if ((st = check_ptr(y, "y"))) return st;
    TPF_ON_DEVICE(h);
    CombineArgs a{};
    a.rows = rows;
    a.weights = weights;
    a.pos = pos;
    a.y = y;
    a.T = (int)T;
    a.k = k;
    a.H = (int)H;
    a.rows_f32 = rows_dtype == TPF_F32;
    a.y_f32 = y_dtype == TPF_F32;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    TPF_TIMED(h, s, launch_expert_combine(a, s));
    return TPF_OK;
  });
}

int tpf_expert_combine_backward(tpf_handle h, int64_t T, int k, int64_t H, int64_t E, const void* dy, int dy_dtype,
                                const void* rows, int rows_dtype, const float* weights, const int32_t* pos,
                                const int32_t* offsets, void* drows, float* dweights, void* stream) {
  return guarded([&]() -> int {
    int st;
    if ((st = check_combine(T, k, H, rows_dtype, dy_dtype))) return st;
    if ((st = check_experts(E))) return st;
    if ((st = check_ptr(dy, "dy"))) return st;
    if ((st = check_ptr(rows, "rows"))) return st;
    if ((st = check_ints(weights, "weights"))) return st;
    if ((st = check_ints(pos, "pos"))) return st;
    if ((st = check_ints(offsets, "offsets"))) return st;
    if ((st = check_ptr(drows, "drows"))) return st;
    if ((st = check_ints(dweights, "dweights"))) return st;
    TPF_ON_DEVICE(h);
    CombineArgs a{};
    a.rows = rows;
    a.weights = weights;
    a.pos = pos;
    a.offsets = offsets;
    a.dy = dy;
    a.drows = drows;
    a.dweights = dweights;
    a.T = (int)T;
    a.k = k;
    a.H = (int)H;
    a.E = (int)E;
    a.rows_f32 = rows_dtype == TPF_F32;
    a.y_f32 = dy_dtype == TPF_F32;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    TPF_TIMED(h, s, launch_expert_combine_backward(a, s));
    return TPF_OK;
  });
}

}  // extern "C"
