// Norms before and after a block, fused with its gate, residual scale and
// residual add.
//
//   b      = (B_0 + B_1) + ... + B_{p-1}            fp32, shard order
//   r_b    = (mean(b^2) + eps)^-1/2
//   x_out  = alpha x + beta gate b r_b (w_post + o)  rounded once to x's type
//   r_x    = (mean(x_out^2) + eps)^-1/2              of the stored values
//   y      = x_out r_x (w_pre + o)                   rounded once to bf16
//
// Each row is read once: it stays in the registers of its T threads between
// the two means.  Sums, statistics and weight gradients are fp32.
#include <algorithm>

#include "tpf_block.hpp"

namespace tpf {

struct F8 {
  float v[8];
};

// Eight consecutive elements at element e (16-byte aligned), widened exactly.
template <int F32>
__device__ __forceinline__ F8 load8(const void* base, int64_t e) {
  F8 o;
  if constexpr (F32) {
    const f32x4_t* q = reinterpret_cast<const f32x4_t*>(reinterpret_cast<const float*>(base) + e);
    const f32x4_t a = q[0], b = q[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o.v[i] = a[i];
      o.v[i + 4] = b[i];
    }
  } else {
    const u32x4_t w = *reinterpret_cast<const u32x4_t*>(reinterpret_cast<const uint16_t*>(base) + e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o.v[2 * i] = __uint_as_float(w[i] << 16);
      o.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  return o;
}

__device__ __forceinline__ F8 load8_any(const void* base, int64_t e, int f32) {
  return f32 ? load8<1>(base, e) : load8<0>(base, e);
}

__device__ __forceinline__ u32x4_t to_bf16x8(const F8& x) {
  bf16x8_t h;
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = (__bf16)x.v[i];
  return __builtin_bit_cast(u32x4_t, h);
}

template <int F32>
__device__ __forceinline__ void store8(void* base, int64_t e, const F8& x) {
  if constexpr (F32) {
    f32x4_t* q = reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(base) + e);
    q[0] = f32x4_t{x.v[0], x.v[1], x.v[2], x.v[3]};
    q[1] = f32x4_t{x.v[4], x.v[5], x.v[6], x.v[7]};
  } else {
    *reinterpret_cast<u32x4_t*>(reinterpret_cast<uint16_t*>(base) + e) = to_bf16x8(x);
  }
}

// The left fold over the p shards of eight elements, loads four at a time.
template <int F32>
__device__ __forceinline__ F8 load_sum8(const NormArgs& a, int64_t e) {
  F8 s = load8<F32>(a.blocks[0], e);
  for (int k = 1; k < a.p; k += 3) {
    F8 t[3];
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (k + j < a.p) t[j] = load8<F32>(a.blocks[k + j], e);
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (k + j < a.p) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s.v[i] += t[j].v[i];
      }
  }
  return s;
}

// Sums of N values over a row's T threads; every thread gets them, added in
// the same order whatever the number of rows.
template <int T, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* lds) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], d);
  if constexpr (T > 64) {
    constexpr int W = T / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) lds[i * W + wave] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += lds[i * W + w];
      v[i] = s;
    }
  }
}

template <class A>
__device__ __forceinline__ const A& norm_kernarg() {
  return *(const A*)__builtin_amdgcn_kernarg_segment_ptr();
}

// T threads a row, V vectors of eight elements a thread; workgroups of at
// least 256 threads, so short rows share one.
template <int T>
constexpr int norm_rows() {
  return T < 256 ? (T == 64 ? 4 : 1) : 1;
}

template <int XF, int BF, int T, int V>
__global__ __launch_bounds__(T * norm_rows<T>()) void block_norm_kernel(NormArgs args) {
  (void)args;
  const NormArgs& a = norm_kernarg<NormArgs>();
  __shared__ float lds[2][T / 64];
  const int t = threadIdx.x % T;
  const int m = blockIdx.x * norm_rows<T>() + threadIdx.x / T;
  if (norm_rows<T>() > 1 && m >= a.M) return;
  const int64_t row = (int64_t)m * a.H;
  F8 b[V], x[V];
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int h = (i * T + t) * 8;
    if (h < a.H) {
      b[i] = load_sum8<BF>(a, row + h);
      x[i] = load8<XF>(a.x, row + h);
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if ((i * T + t) * 8 < a.H) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] += b[i].v[j] * b[i].v[j];
    }
  row_sums<T, 1>(s, lds[0]);
  const float inv_h = 1.0f / (float)a.H;
  const float rb = 1.0f / sqrtf(s[0] * inv_h + a.eps);
  const float g_row = a.gate_kind == GATE_TOKEN ? (a.w_f32 ? reinterpret_cast<const float*>(a.gate)[m]
                                                           : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(a.gate)[m] << 16))
                                                : 1.0f;
  const float scale = a.beta * g_row;
  s[0] = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int h = (i * T + t) * 8;
    if (h < a.H) {
      const F8 w = load8_any(a.w_post, h, a.w_f32);
      F8 g;
      if (a.gate_kind == GATE_CHANNEL) g = load8_any(a.gate, h, a.w_f32);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float n = b[i].v[j] * rb * (w.v[j] + a.offset);
        if (a.gate_kind == GATE_CHANNEL) n *= g.v[j];
        float o = a.alpha * x[i].v[j] + scale * n;
        if constexpr (!XF) o = (float)(__bf16)o;   // the next norm is of the stored stream
        x[i].v[j] = o;
        s[0] += o * o;
      }
      store8<XF>(a.x_out, row + h, x[i]);
    }
  }
  row_sums<T, 1>(s, lds[1]);
  const float rx = 1.0f / sqrtf(s[0] * inv_h + a.eps);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int h = (i * T + t) * 8;
    if (h < a.H) {
      const F8 w = load8_any(a.w_pre, h, a.w_f32);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i].v[j] = x[i].v[j] * rx * (w.v[j] + a.offset);
      store8<0>(a.y, row + h, x[i]);
    }
  }
  if (a.stats && t == 0) {
    a.stats[m] = rb;
    a.stats[a.M + m] = rx;
  }
}

// Backward of one row, with xh = x_out r_x and bh = b r_b:
//   u  = dy (w_pre + o)
//   dt = dx_out + r_x (u - xh mean(u xh))
//   v  = beta dt,  z = v gate (w_post + o)
//   db = r_b (z - bh mean(z bh)),  dx = alpha dt
// mean(z bh) needs dt and so mean(u xh); written out, it is the difference of
// two row sums that need neither, so one round of sums serves both:
//   sum(z bh) = beta (A - mean(u xh) B),
//   A = sum((dx_out + r_x u) gate w bh),  B = sum(r_x xh gate w bh).
// Column sums over the rows: P = sum dy xh (dw_pre) and Q = sum v g bh, g the
// token's gate or 1.  dw_post is Q (times a channel's gate) and a channel's
// gate gradient is Q (w_post + o), so two sums serve three gradients.
// Workgroup i adds rows i, i + groups, ... in registers; norm_columns_kernel
// adds the workgroups in a fixed order.
template <int XF, int BF, int T, int V>
__global__ __launch_bounds__(T) void block_norm_backward_kernel(NormArgs args) {
  (void)args;
  const NormArgs& a = norm_kernarg<NormArgs>();
  __shared__ float lds[2][3 * (T / 64)];
  const int t = threadIdx.x;
  const float inv_h = 1.0f / (float)a.H;
  F8 sp[V], sq[V];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) sp[i].v[j] = sq[i].v[j] = 0.0f;
  int par = 0;
  for (int m = blockIdx.x; m < a.M; m += a.groups, par ^= 1) {
    const int64_t row = (int64_t)m * a.H;
    const float rb = a.stats[m], rx = a.stats[a.M + m];
    const float g_row = a.gate_kind == GATE_TOKEN ? (a.w_f32 ? reinterpret_cast<const float*>(a.gate)[m]
                                                             : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(a.gate)[m] << 16))
                                                  : 1.0f;
    F8 bh[V], xh[V], e[V], dy[V];   // e = dx_out + r_x u
    float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int h = (i * T + t) * 8;
      if (h < a.H) {
        bh[i] = load_sum8<BF>(a, row + h);
        xh[i] = load8<XF>(a.x, row + h);
        dy[i] = load8<0>(a.dy, row + h);
        if (a.dx_out) {
          e[i] = load8<XF>(a.dx_out, row + h);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) e[i].v[j] = 0.0f;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int h = (i * T + t) * 8;
      if (h < a.H) {
        const F8 wq = load8_any(a.w_pre, h, a.w_f32), wp = load8_any(a.w_post, h, a.w_f32);
        F8 g;
        if (a.gate_kind == GATE_CHANNEL) g = load8_any(a.gate, h, a.w_f32);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          bh[i].v[j] *= rb;
          xh[i].v[j] *= rx;
          const float u = dy[i].v[j] * (wq.v[j] + a.offset);
          e[i].v[j] += rx * u;
          float k = (wp.v[j] + a.offset) * bh[i].v[j];
          if (a.gate_kind == GATE_CHANNEL) k *= g.v[j];
          s[0] += u * xh[i].v[j];
          s[1] += e[i].v[j] * k;
          s[2] += rx * xh[i].v[j] * k;
        }
      }
    }
    row_sums<T, 3>(s, lds[par]);   // the other half is still read by slower waves
    const float c1 = s[0] * inv_h;
    const float vk = a.beta * (s[1] - c1 * s[2]);     // sum(v gate_h w bh), before the token's gate
    const float c2 = vk * g_row * inv_h;
    const float bg = a.beta * g_row;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int h = (i * T + t) * 8;
      if (h < a.H) {
        const F8 wp = load8_any(a.w_post, h, a.w_f32);
        F8 g;
        if (a.gate_kind == GATE_CHANNEL) g = load8_any(a.gate, h, a.w_f32);
        F8 dx, db;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float dt = e[i].v[j] - rx * c1 * xh[i].v[j];
          const float v = bg * dt;
          float z = v * (wp.v[j] + a.offset);
          if (a.gate_kind == GATE_CHANNEL) z *= g.v[j];
          dx.v[j] = a.alpha * dt;
          db.v[j] = rb * (z - bh[i].v[j] * c2);
          sp[i].v[j] += dy[i].v[j] * xh[i].v[j];
          sq[i].v[j] += v * bh[i].v[j];
        }
        store8<XF>(a.x_out, row + h, dx);
        store8<0>(a.y, row + h, db);
      }
    }
    if (a.gate_kind == GATE_TOKEN && t == 0) a.dgate[m] = vk;
  }
  float* out = a.partial + (int64_t)blockIdx.x * 2 * a.H;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int h = (i * T + t) * 8;
    if (h < a.H) {
      store8<1>(out, h, sp[i]);
      store8<1>(out + a.H, h, sq[i]);
    }
  }
}

// Columns 4 c .. 4 c + 3 of both sums over the workgroups of the row pass: 16
// threads along the columns, 16 strips of workgroups, joined through LDS.
__global__ __launch_bounds__(256) void norm_columns_kernel(NormArgs args) {
  (void)args;
  const NormArgs& a = norm_kernarg<NormArgs>();
  __shared__ f32x4_t lds[16][17];
  const int c = threadIdx.x & 15, strip = threadIdx.x >> 4;
  const int h = (blockIdx.x * 16 + c) * 4;
  const int which = blockIdx.y;
  f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
  if (h < a.H)
    for (int g = strip; g < a.groups; g += 16)
      s += *reinterpret_cast<const f32x4_t*>(a.partial + ((int64_t)g * 2 + which) * a.H + h);
  lds[strip][c] = s;
  __syncthreads();
  if (strip != 0 || h >= a.H) return;
#pragma unroll
  for (int k = 1; k < 16; ++k) s += lds[k][c];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i = h + j;
    if (which == 0) {
      a.dw_pre[i] = s[j];
    } else if (a.gate_kind == GATE_CHANNEL) {
      const float w = (a.w_f32 ? reinterpret_cast<const float*>(a.w_post)[i]
                               : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(a.w_post)[i] << 16)) +
                      a.offset;
      const float g = a.w_f32 ? reinterpret_cast<const float*>(a.gate)[i]
                              : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(a.gate)[i] << 16);
      a.dw_post[i] = g * s[j];
      a.dgate[i] = w * s[j];
    } else {
      a.dw_post[i] = s[j];
    }
  }
}

template <int XF, int BF>
static void launch_norm_t(const NormArgs& a, hipStream_t s) {
#define TPF_NORM(T, V)                                                                                          \
  hipLaunchKernelGGL((block_norm_kernel<XF, BF, T, V>), dim3((a.M + norm_rows<T>() - 1) / norm_rows<T>()),     \
                     dim3(T * norm_rows<T>()), 0, s, a)
  if (a.H <= 512) TPF_NORM(64, 1);
  else if (a.H <= 1024) TPF_NORM(64, 2);
  else if (a.H <= 2048) TPF_NORM(256, 1);
  else if (a.H <= 4096) TPF_NORM(256, 2);
  else if (a.H <= 8192) TPF_NORM(512, 2);
  else if (a.H <= 16384) TPF_NORM(1024, 2);
  else TPF_NORM(1024, 4);
#undef TPF_NORM
}

hipError_t launch_block_norm(const NormArgs& a, hipStream_t s) {
  if (a.x_f32) {
    if (a.b_f32) launch_norm_t<1, 1>(a, s);
    else launch_norm_t<1, 0>(a, s);
  } else {
    if (a.b_f32) launch_norm_t<0, 1>(a, s);
    else launch_norm_t<0, 0>(a, s);
  }
  return hipGetLastError();
}

int norm_backward_groups(int64_t M, int64_t H) {
  (void)H;
  return (int)std::min<int64_t>(M, 512);
}

template <int XF, int BF>
static void launch_norm_bwd_t(const NormArgs& a, hipStream_t s) {
#define TPF_NORM(T, V) \
  hipLaunchKernelGGL((block_norm_backward_kernel<XF, BF, T, V>), dim3(a.groups), dim3(T), 0, s, a)
  if (a.H <= 512) TPF_NORM(64, 1);
  else if (a.H <= 2048) TPF_NORM(256, 1);
  else if (a.H <= 4096) TPF_NORM(512, 1);
  else if (a.H <= 8192) TPF_NORM(1024, 1);
  else if (a.H <= 16384) TPF_NORM(1024, 2);
  else TPF_NORM(1024, 4);
#undef TPF_NORM
}

hipError_t launch_block_norm_backward(const NormArgs& a, hipStream_t s) {
  if (a.x_f32) {
    if (a.b_f32) launch_norm_bwd_t<1, 1>(a, s);
    else launch_norm_bwd_t<1, 0>(a, s);
  } else {
    if (a.b_f32) launch_norm_bwd_t<0, 1>(a, s);
    else launch_norm_bwd_t<0, 0>(a, s);
  }
  return hipGetLastError();
}

hipError_t launch_norm_columns(const NormArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(norm_columns_kernel, dim3((a.H + 63) / 64, 2), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace tpf
