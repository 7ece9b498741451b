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
//
// Bound by memory, at the rate of a large copy (4.75 TB/s) or above: forward of
// 4096 x 4096 bf16 28 us a call (4.7 TB/s), of 2048 x 12288 fp32 from four partials
// 126 (5.2 TB/s), of 2048 x 32768 bf16 134 (4.0 TB/s).  A decode step's 16 x 8192
// takes 5.6 us of the GPU, of which a launch alone is 2.3: the rest is one row's
// chain of load, sum, exchange, sum, store.
#include <algorithm>

#include "tpf_block.hpp"

namespace tpf {

struct F8 {
  float v[8];
};

// Eight consecutive elements as loaded, and widened exactly.
template <int F32>
struct Raw8 {
  u32x4_t w[F32 ? 2 : 1];
};
template <int F32>
__device__ __forceinline__ Raw8<F32> load_raw(const void* base, int64_t e) {
  Raw8<F32> r;
  const u32x4_t* q = reinterpret_cast<const u32x4_t*>(reinterpret_cast<const char*>(base) + e * (F32 ? 4 : 2));
  r.w[0] = q[0];
  if constexpr (F32) r.w[1] = q[1];
  return r;
}
template <int F32>
__device__ __forceinline__ F8 widen(const Raw8<F32>& r) {
  F8 o;
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o.v[i] = __uint_as_float(r.w[0][i]);
      o.v[i + 4] = __uint_as_float(r.w[1][i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o.v[2 * i] = __uint_as_float(r.w[0][i] << 16);
      o.v[2 * i + 1] = __uint_as_float(r.w[0][i] & 0xffff0000u);
    }
  }
  return o;
}
template <int F32>
__device__ __forceinline__ F8 load8(const void* base, int64_t e) {
  return widen<F32>(load_raw<F32>(base, e));
}

__device__ __forceinline__ F8 load8_any(const void* base, int64_t e, int f32) {
  return f32 ? load8<1>(base, e) : load8<0>(base, e);
}
__device__ __forceinline__ float load1_any(const void* base, int64_t e, int f32) {
  return f32 ? reinterpret_cast<const float*>(base)[e]
             : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(base)[e] << 16);
}

template <int STREAM, class V>
__device__ __forceinline__ void put(V* p, V v) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, p);
  else *p = v;
}

template <int F32, int STREAM>
__device__ __forceinline__ void store8(void* base, int64_t e, const F8& x) {
  if constexpr (F32) {
    f32x4_t* q = reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(base) + e);
    put<STREAM>(q, f32x4_t{x.v[0], x.v[1], x.v[2], x.v[3]});
    put<STREAM>(q + 1, f32x4_t{x.v[4], x.v[5], x.v[6], x.v[7]});
  } else {
    bf16x8_t h;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = (__bf16)x.v[i];
    put<STREAM>(reinterpret_cast<u32x4_t*>(reinterpret_cast<uint16_t*>(base) + e), __builtin_bit_cast(u32x4_t, h));
  }
}

// Adds shards 1 .. p-1 to s in order, loads three at a time.
template <int F32>
__device__ __forceinline__ void add_shards(F8& s, const NormArgs& a, int64_t e) {
  for (int k = 1; k < a.p; k += 3) {
    Raw8<F32> t[3];
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (k + j < a.p) t[j] = load_raw<F32>(a.blocks[k + j], e);
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (k + j < a.p) {
        const F8 f = widen<F32>(t[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) s.v[i] += f.v[i];
      }
  }
}

// Sums of N values over the waves of a row (at most 16); every thread gets
// them, added in an order that depends on the row's length alone.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*lds)[16], int waves, int wave) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], d);
  if (waves == 1) return;
  const int lane = threadIdx.x & 63;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) lds[i][wave] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = (lane & 15) < waves ? lds[i][lane & 15] : 0.0f;
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) v[i] += __shfl_xor(v[i], d);
  }
}

template <class A>
__device__ __forceinline__ const A& norm_kernarg() {
  return *(const A*)__builtin_amdgcn_kernarg_segment_ptr();
}

// A row takes the fewest whole waves that hold it at V vectors of eight
// elements a thread (odd widths leave at most a wave's worth idle); rows of
// one wave share workgroups of four.
constexpr int kNormRows = 4;
template <int V>
static int norm_threads(int H) {
  return (H + 512 * V - 1) / (512 * V) * 64;
}

template <int XF, int BF, int V, int STREAM>
__global__ __launch_bounds__(1024) void block_norm_kernel(NormArgs args) {
  (void)args;
  const NormArgs& a = norm_kernarg<NormArgs>();
  __shared__ float lds[2][1][16];
  const int T = blockDim.x, t = threadIdx.x, waves = T / 64, wave = t >> 6;
  const uint32_t m = a.row0 + blockIdx.x * blockDim.y + threadIdx.y;
  if (m >= (uint32_t)a.M) return;      // only where a row is one wave: no barrier follows
  const int64_t row = (int64_t)m * a.H;
  F8 b[V];
  Raw8<XF> xr[V];
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int h = (i * T + t) * 8;
    if (h < a.H) {
      b[i] = load8<BF>(a.blocks[0], row + h);
      xr[i] = load_raw<XF>(a.x, row + h);
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int h = (i * T + t) * 8;
    if (h < a.H) {
      add_shards<BF>(b[i], a, row + h);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] += b[i].v[j] * b[i].v[j];
    }
  }
  row_sums<1>(s, lds[0], waves, wave);
  const float inv_h = 1.0f / (float)a.H;
  const float rb = 1.0f / sqrtf(s[0] * inv_h + a.eps);
  const float scale = a.gate_kind == GATE_TOKEN ? a.beta * load1_any(a.gate, m, a.w_f32) : a.beta;
  F8 x[V];
  s[0] = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int h = (i * T + t) * 8;
    if (h < a.H) {
      x[i] = widen<XF>(xr[i]);
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
      store8<XF, STREAM>(a.x_out, row + h, x[i]);
    }
  }
  row_sums<1>(s, lds[1], waves, wave);
  const float rx = 1.0f / sqrtf(s[0] * inv_h + a.eps);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int h = (i * T + t) * 8;
    if (h < a.H) {
      const F8 w = load8_any(a.w_pre, h, a.w_f32);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i].v[j] = x[i].v[j] * rx * (w.v[j] + a.offset);
      store8<0, STREAM>(a.y, row + h, x[i]);
    }
  }
  if (a.stats && t == 0) {
    a.stats[m] = rb;
    a.stats[a.M + (int64_t)m] = rx;
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
// Bound by memory for long columns (8192 x 8192 bf16: 147 us and 7 for the column
// sums, 5.2 TB/s).  1003 x 5000 with fp32 rows and vectors takes 27 and 4 us
// (3.1 TB/s): four rows a workgroup one after the other, each with its vectors read
// again in both halves, and the start of both launches.
// With V = 1 (rows of up to 8192) a thread loads the next row before it joins
// the current one, so that the row's barrier does not leave the memory idle,
// and keeps its columns' bf16 weights and gate.  The bound of 16 waves leaves 128
// registers a thread, in shorter rows too: rows past 8192 are read again from the
// cache after the sums instead of being held, and so are fp32 weights.  That does
// not keep every instance within the registers: the ones with bf16 rows and V = 1
// spill two at most, those with fp32 rows or V = 2 up to 25, those with V = 4 from
// 105 to 148 (200 to 268 bytes a lane), which bounds them: 2048 x 32768 takes
// 474 us in bf16 (1.7 TB/s) and 636 in fp32, 2048 x 12288 in fp32 162 (3.1 TB/s).
template <int XF, int BF, int WF, int V, int STREAM>
__global__ __launch_bounds__(1024) void block_norm_backward_kernel(NormArgs args) {
  (void)args;
  const NormArgs& a = norm_kernarg<NormArgs>();
  __shared__ float lds[2][3][16];
  const int T = blockDim.x, t = threadIdx.x, waves = T / 64, wave = t >> 6;
  constexpr bool HOLD = V == 1, HOLDW = V == 1 && !WF;
  const float inv_h = 1.0f / (float)a.H;
  struct Row {
    Raw8<BF> b[V];
    Raw8<XF> x[V], e[V];
    Raw8<0> dy[V];
    float rb, rx, g;
  };
  auto load_part = [&](Row& r, uint32_t m, int i) {
    const int64_t at = (int64_t)m * a.H + (i * T + t) * 8;
    r.b[i] = load_raw<BF>(a.blocks[0], at);
    r.x[i] = load_raw<XF>(a.x, at);
    r.dy[i] = load_raw<0>(a.dy, at);
    if (a.dx_out) r.e[i] = load_raw<XF>(a.dx_out, at);
  };
  auto load_row = [&](Row& r, uint32_t m) {
    if constexpr (HOLD) {
      if (t * 8 < a.H) load_part(r, m, 0);
    }
    r.rb = a.stats[m];
    r.rx = a.stats[a.M + (int64_t)m];
    r.g = a.gate_kind == GATE_TOKEN ? load1_any(a.gate, m, a.w_f32) : 1.0f;
  };
  const bool channel = a.gate_kind == GATE_CHANNEL;
  F8 sp[V], sq[V];
  Raw8<WF> hq, hp, hg;
  if constexpr (HOLDW) {
    if (t * 8 < a.H) {
      hq = load_raw<WF>(a.w_pre, t * 8);
      hp = load_raw<WF>(a.w_post, t * 8);
      if (channel) hg = load_raw<WF>(a.gate, t * 8);
    }
  }
  auto w_pre = [&](int h) { return widen<WF>(HOLDW ? hq : load_raw<WF>(a.w_pre, h)); };
  auto w_post = [&](int h) { return widen<WF>(HOLDW ? hp : load_raw<WF>(a.w_post, h)); };
  auto gate = [&](int h) { return widen<WF>(HOLDW ? hg : load_raw<WF>(a.gate, h)); };
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) sp[i].v[j] = sq[i].v[j] = 0.0f;
  // bh, xh and e = dx_out + r_x u of one part of the row.
  auto terms = [&](const Row& r, int64_t at, int h, int i, F8& bh, F8& xh, F8& e, F8& u) {
    bh = widen<BF>(r.b[i]);
    add_shards<BF>(bh, a, at);
    xh = widen<XF>(r.x[i]);
    u = widen<0>(r.dy[i]);
    const F8 q = w_pre(h);
    if (a.dx_out) e = widen<XF>(r.e[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      bh.v[j] *= r.rb;
      xh.v[j] *= r.rx;
      u.v[j] *= q.v[j] + a.offset;
      e.v[j] = (a.dx_out ? e.v[j] : 0.0f) + r.rx * u.v[j];
    }
  };
  int par = 0;
  Row next;
  load_row(next, blockIdx.x);
  // Row numbers are unsigned: the last one plus `groups` can pass 31 bits.
  for (uint32_t m = blockIdx.x; m < (uint32_t)a.M; m += a.groups, par ^= 1) {
    const int64_t row = (int64_t)m * a.H;
    Row r = next;
    if (m + a.groups < (uint32_t)a.M) load_row(next, m + a.groups);
    F8 bh, xh, e;
    float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int h = (i * T + t) * 8;
      if (h < a.H) {
        if constexpr (!HOLD) load_part(r, m, i);
        F8 u;
        terms(r, row + h, h, i, bh, xh, e, u);
        if constexpr (!HOLDW) asm volatile("" ::: "memory");   // the next weights after these are used
        const F8 w = w_post(h), dy = widen<0>(r.dy[i]);
        F8 g;
        if (channel) g = gate(h);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float k = (w.v[j] + a.offset) * bh.v[j];
          if (channel) k *= g.v[j];
          s[0] += u.v[j] * xh.v[j];
          s[1] += e.v[j] * k;
          s[2] += r.rx * xh.v[j] * k;
          sp[i].v[j] += dy.v[j] * xh.v[j];
        }
        if constexpr (!HOLD) asm volatile("" ::: "memory");    // one part's loads at a time
      }
    }
    row_sums<3>(s, lds[par], waves, wave);   // the other half is still read by slower waves
    const float c1 = s[0] * inv_h;
    const float vk = a.beta * (s[1] - c1 * s[2]);     // sum(v gate_h w bh), before the token's gate
    const float c2 = vk * r.g * inv_h;
    const float bg = a.beta * r.g;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int h = (i * T + t) * 8;
      if (h < a.H) {
        if constexpr (!HOLD) {
          F8 u;
          load_part(r, m, i);
          terms(r, row + h, h, i, bh, xh, e, u);
        }
        const F8 w = w_post(h);
        F8 g, dx, db;
        if (channel) g = gate(h);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float dt = e.v[j] - r.rx * c1 * xh.v[j];
          const float v = bg * dt;
          float z = v * (w.v[j] + a.offset);
          if (channel) z *= g.v[j];
          dx.v[j] = a.alpha * dt;
          db.v[j] = r.rb * (z - bh.v[j] * c2);
          sq[i].v[j] += v * bh.v[j];
        }
        store8<XF, STREAM>(a.x_out, row + h, dx);
        store8<0, STREAM>(a.y, row + h, db);
        if constexpr (!HOLD) asm volatile("" ::: "memory");
      }
    }
    if (a.gate_kind == GATE_TOKEN && t == 0) a.dgate[m] = vk;
  }
  float* out = a.partial + (int64_t)blockIdx.x * 2 * a.H;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int h = (i * T + t) * 8;
    if (h < a.H) {
      store8<1, 0>(out, h, sp[i]);
      store8<1, 0>(out + a.H, h, sq[i]);
    }
  }
}

// Columns 4 c .. 4 c + 3 of both sums over the workgroups of the row pass: 16
// threads along the columns, 64 strips of workgroups, joined through LDS.
__global__ __launch_bounds__(1024) void norm_columns_kernel(NormArgs args) {
  (void)args;
  const NormArgs& a = norm_kernarg<NormArgs>();
  __shared__ f32x4_t lds[64][17];
  const int c = threadIdx.x & 15, strip = threadIdx.x >> 4;
  const int h = (blockIdx.x * 16 + c) * 4;
  const int which = blockIdx.y;
  f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
  if (h < a.H) {
    const float* base = a.partial + (int64_t)which * a.H + h;
    const int64_t stride = (int64_t)2 * a.H;
#pragma unroll 4
    for (int g = strip; g < a.groups; g += 64) s += *reinterpret_cast<const f32x4_t*>(base + g * stride);
  }
  lds[strip][c] = s;
  __syncthreads();
  if (strip < 8) {
#pragma unroll
    for (int k = 1; k < 8; ++k) s += lds[strip + 8 * k][c];
    lds[strip][c] = s;
  }
  __syncthreads();
  if (strip != 0 || h >= a.H) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) s += lds[k][c];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i = h + j;
    if (which == 0) {
      a.dw_pre[i] = s[j];
    } else if (a.gate_kind == GATE_CHANNEL) {
      a.dw_post[i] = load1_any(a.gate, i, a.w_f32) * s[j];
      a.dgate[i] = (load1_any(a.w_post, i, a.w_f32) + a.offset) * s[j];
    } else {
      a.dw_post[i] = s[j];
    }
  }
}

// Whether both [M][H] outputs are stored past the caches.
template <int XF>
static bool norm_streams(const NormArgs& a) {
  return (int64_t)a.M * a.H * (XF ? 6 : 4) >= kStreamBytes;
}

template <int XF, int BF, int V>
static void launch_norm_v(const NormArgs& a, hipStream_t s) {
  const int T = norm_threads<V>(a.H), rows = T == 64 ? kNormRows : 1;
  const int64_t most = UINT32_MAX / T, groups = ((int64_t)a.M + rows - 1) / rows;   // a grid has fewer than 2^32 threads
  for (int64_t g = 0; g < groups; g += most) {
    NormArgs part = a;
    part.row0 = (uint32_t)(g * rows);
    const dim3 grid((unsigned)std::min(groups - g, most)), block(T, rows);
    if (norm_streams<XF>(a)) hipLaunchKernelGGL((block_norm_kernel<XF, BF, V, 1>), grid, block, 0, s, part);
    else hipLaunchKernelGGL((block_norm_kernel<XF, BF, V, 0>), grid, block, 0, s, part);
  }
}

template <int XF, int BF>
static void launch_norm_t(const NormArgs& a, hipStream_t s) {
  if (a.H <= 8192) launch_norm_v<XF, BF, 1>(a, s);
  else if (a.H <= 16384) launch_norm_v<XF, BF, 2>(a, s);
  else launch_norm_v<XF, BF, 4>(a, s);
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

// As many workgroups as the GPU's 256 compute units hold at 16 waves each,
// but at least eight rows a workgroup once every unit has one: each workgroup
// leaves 8 H bytes of column sums.
int norm_backward_groups(int64_t M, int64_t H) {
  const int waves = std::min<int>(16, norm_threads<1>((int)H) / 64);
  const int64_t cap = 256 * (16 / waves);
  return (int)std::max(std::min<int64_t>(M, 256), std::min(cap, M / 8));
}

template <int XF, int BF, int WF>
static void launch_norm_bwd_w(const NormArgs& a, hipStream_t s) {
#define TPF_NORM(V)                                                                                         \
  if (norm_streams<XF>(a))                                                                                  \
    hipLaunchKernelGGL((block_norm_backward_kernel<XF, BF, WF, V, 1>), dim3(a.groups),                      \
                       dim3(norm_threads<V>(a.H)), 0, s, a);                                                \
  else                                                                                                      \
    hipLaunchKernelGGL((block_norm_backward_kernel<XF, BF, WF, V, 0>), dim3(a.groups),                      \
                       dim3(norm_threads<V>(a.H)), 0, s, a)
  if (a.H <= 8192) {
    TPF_NORM(1);
  } else if (a.H <= 16384) {
    TPF_NORM(2);
  } else {
    TPF_NORM(4);
  }
#undef TPF_NORM
}

template <int XF, int BF>
static void launch_norm_bwd_t(const NormArgs& a, hipStream_t s) {
  if (a.w_f32) launch_norm_bwd_w<XF, BF, 1>(a, s);
  else launch_norm_bwd_w<XF, BF, 0>(a, s);
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
  hipLaunchKernelGGL(norm_columns_kernel, dim3((a.H + 63) / 64, 2), dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace tpf
