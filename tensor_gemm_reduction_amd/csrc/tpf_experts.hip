// The MLP block of experts around its products: routing of tokens (scores,
// choice, weights, the order of the experts' rows), the router's gradient, and
// the sum of each token's rows with its gradient.
#include <algorithm>

#include "tpf_scaled.hpp"

namespace tpf {
namespace {

template <class A>
__device__ __forceinline__ const A& kernarg() {
  return *(const A*)__builtin_amdgcn_kernarg_segment_ptr();
}

__device__ __forceinline__ float bf16_at(const void* p, int64_t i) {
  return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << 16);
}
template <int F32>
__device__ __forceinline__ float value_at(const void* p, int64_t i) {
  return F32 ? reinterpret_cast<const float*>(p)[i] : bf16_at(p, i);
}

constexpr int kRouteThreads = 1024;
constexpr int kRouteTokens = 64;       // tokens of a part of the order, at least
constexpr double kNone = -__builtin_huge_val();

template <int L>
__device__ __forceinline__ double max_over(double v) {
#pragma unroll
  for (int d = 1; d < L; d <<= 1) v = fmax(v, __shfl_xor(v, d));
  return v;
}
template <int L>
__device__ __forceinline__ double sum_over(double v) {
#pragma unroll
  for (int d = 1; d < L; d <<= 1) v += __shfl_xor(v, d);
  return v;
}
// The largest value's index, the lowest among equals; index INT_MAX: nothing.
template <int L>
__device__ __forceinline__ int best_over(double v, int at) {
#pragma unroll
  for (int d = 1; d < L; d <<= 1) {
    const double ov = __shfl_xor(v, d);
    const int oa = __shfl_xor(at, d);
    if (ov > v || (ov == v && oa < at)) v = ov, at = oa;
  }
  return at;
}

// The order of the experts' rows, part b of the tokens: each expert's rows
// follow those of the experts before it and of its own in earlier parts, in the
// order of the slots.  One thread an expert walks the part's slots, so the order
// needs no atomics.
constexpr int kOrderSlots = 4096;
__device__ void order_part(const RouteArgs& a, int b, int* lds_total, uint16_t* lds_ids) {
  const int tid = threadIdx.x, nt = blockDim.x;
  const int lane = tid & 63;
  // Rows of every expert, then the first row of each (one wave, 64 at a time).
  for (int e = tid; e < a.E; e += nt) {
    int total = 0;
    for (int c = 0; c < a.chunks; ++c) total += a.hist[(int64_t)c * a.E + e];
    lds_total[e] = total;
  }
  __syncthreads();
  if (tid < 64) {
    int before = 0;
    for (int base = 0; base < a.E; base += 64) {
      const int e = base + lane;
      const int n = e < a.E ? lds_total[e] : 0;
      int upto = n;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(upto, d);
        if (lane >= d) upto += v;
      }
      if (e < a.E) lds_total[e] = before + upto - n;
      before += __shfl(upto, 63);
    }
    if (lane == 0) lds_total[a.E] = before;
  }
  __syncthreads();
  if (b == 0)
    for (int e = tid; e <= a.E; e += nt) a.offsets[e] = lds_total[e];
  const int R = a.T * a.k;
  // Rows behind the last expert's have no slot.
  for (int64_t r = (int64_t)lds_total[a.E] + (int64_t)b * nt + tid; r < R; r += (int64_t)a.chunks * nt) a.src[r] = -1;
  const int64_t first = (int64_t)b * a.chunk * a.k;
  const int64_t last = min((int64_t)R, first + (int64_t)a.chunk * a.k);
  for (int e0 = 0; e0 < a.E; e0 += nt) {
    const int e = e0 + tid;
    int row = 0;
    if (e < a.E) {
      row = lds_total[e];
      for (int c = 0; c < b; ++c) row += a.hist[(int64_t)c * a.E + e];
    }
    for (int64_t s0 = first; s0 < last; s0 += kOrderSlots) {
      const int n = (int)min((int64_t)kOrderSlots, last - s0);
      __syncthreads();
      for (int i = tid; i < n; i += nt) {
        const int id = a.ids[s0 + i];
        lds_ids[i] = (uint16_t)id;
        if (id < 0) a.pos[s0 + i] = -1;
      }
      __syncthreads();
      if (e < a.E)
        for (int i = 0; i < n; ++i)
          if (lds_ids[i] == e) {
            a.pos[s0 + i] = row;
            a.src[row] = (int)(s0 + i);
            ++row;
          }
    }
  }
}

__global__ __launch_bounds__(kRouteThreads) void expert_order_kernel(RouteArgs args) {
  (void)args;
  __shared__ int total[kExpertMaxE + 1];
  __shared__ uint16_t ids[kOrderSlots];
  order_part(kernarg<RouteArgs>(), blockIdx.x, total, ids);
}

// Routes one part of the tokens.  L lanes share a token, lane l holding the
// experts l, l + L, ...; choices are compared in 64 bits, so that the order of
// nearly equal values is the definition's.  With one part the order of the
// experts' rows follows in the same launch.
template <int L, int V, int F32>
__global__ __launch_bounds__(kRouteThreads) void expert_route_kernel(RouteArgs args) {
  (void)args;
  const RouteArgs& a = kernarg<RouteArgs>();
  __shared__ int hist[kExpertMaxE + 1];
  __shared__ uint16_t order_ids[kOrderSlots];
  const int b = blockIdx.x, lane = threadIdx.x & 63, li = lane & (L - 1);
  for (int e = threadIdx.x; e < a.E; e += kRouteThreads) hist[e] = 0;
  __syncthreads();
  constexpr int PASS = kRouteThreads / L;
  const int t_end = min(a.T, (b + 1) * a.chunk);
  for (int t0 = b * a.chunk; t0 < t_end; t0 += PASS) {
    const int t = t0 + (int)threadIdx.x / L;
    const bool routed = t < t_end && (!a.mask || a.mask[t]);
    const int64_t row = (int64_t)(t < t_end ? t : t0) * a.E;
    float x[V];
    double v[V];
    double top = kNone;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * L + li;
      x[i] = e < a.E ? value_at<F32>(a.logits, row + e) : -__builtin_huge_valf();
      v[i] = x[i];
      top = fmax(top, v[i]);
    }
    if (a.score == SCORE_SOFTMAX) top = max_over<L>(top);
    double sum = 1.0;
    const bool scores = a.bias || a.groups > 1;
    if (a.score == SCORE_SOFTMAX && (scores || !a.renorm)) {
      sum = 0.0;
#pragma unroll
      for (int i = 0; i < V; ++i) sum += top == kNone ? 0.0 : exp((double)x[i] - top);
      sum = sum_over<L>(sum);
    }
    uint32_t taken = 0;               // the lane's experts that cannot be chosen (any more)
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i * L + li >= a.E) taken |= 1u << i;
    if (scores) {
      double biased[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = i * L + li;
        const double s = a.score == SCORE_SIGMOID ? 1.0 / (1.0 + exp(-(double)x[i]))
                                                  : (top == kNone ? 0.0 : exp((double)x[i] - top) / sum);
        biased[i] = s + (a.bias && e < a.E ? (double)a.bias[e] : 0.0);
        if (!(biased[i] == biased[i])) biased[i] = kNone;
        if (a.bias) v[i] = biased[i];
      }
      if (a.groups > 1) {
        const int gs = a.E / a.groups;
        double mine = kNone;          // lane g's: the sum of the two largest of group g
        for (int g = 0; g < a.groups; ++g) {
          double t1 = kNone, t2 = kNone;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const int e = i * L + li;
            if (e >= g * gs && e < (g + 1) * gs) {
              t2 = fmax(t2, fmin(t1, biased[i]));
              t1 = fmax(t1, biased[i]);
            }
          }
#pragma unroll
          for (int d = 1; d < L; d <<= 1) {
            const double o1 = __shfl_xor(t1, d), o2 = __shfl_xor(t2, d);
            t2 = fmax(fmin(t1, o1), fmax(t2, o2));
            t1 = fmax(t1, o1);
          }
          if (li == g) mine = gs > 1 ? t1 + t2 : t1;
        }
        if (!(mine == mine)) mine = kNone;
        uint32_t allowed = 0;
        bool free_group = li < a.groups;
        for (int g = 0; g < a.top_groups; ++g) {
          const int at = best_over<L>(free_group ? mine : kNone, free_group ? li : INT32_MAX);
          allowed |= 1u << at;
          if (li == at) free_group = false;
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (!(allowed >> min((i * L + li) / gs, 31) & 1)) taken |= 1u << i;
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (!(v[i] == v[i])) v[i] = kNone;
    int id = -1;                      // lane j's: the token's j-th expert
    for (int j = 0; j < a.k; ++j) {
      double best = kNone;
      int at = INT32_MAX;
#pragma unroll
      for (int i = 0; i < V; ++i)     // a lane's experts rise with i: the first of equals stays
        if (!(taken >> i & 1) && (v[i] > best || at == INT32_MAX)) best = v[i], at = i * L + li;
      at = best_over<L>(best, at);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i * L + li == at) taken |= 1u << i;
      if (li == j) id = at;
    }
    const bool mine = routed && li < a.k && (uint32_t)id < (uint32_t)a.E;
    double s = 0.0;
    if (mine) {
      const double l = value_at<F32>(a.logits, row + id);
      s = a.score == SCORE_SIGMOID ? 1.0 / (1.0 + exp(-l)) : (top == kNone ? 0.0 : exp(l - top));
    }
    if (a.renorm) sum = sum_over<L>(s);
    if (t < t_end && li < a.k) {
      double w = 0.0;
      if (mine) w = a.renorm ? (sum == 0.0 ? 0.0 : a.scale * (s / sum)) :
                    a.scale * (a.score == SCORE_SIGMOID || sum == 0.0 ? s : s / sum);
      a.ids[(int64_t)t * a.k + li] = mine ? id : -1;
      a.weights[(int64_t)t * a.k + li] = (float)w;
      if (mine) atomicAdd(&hist[id], 1);
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kRouteThreads) a.hist[(int64_t)b * a.E + e] = hist[e];
  if (a.chunks == 1) {
    __syncthreads();
    order_part(a, 0, hist, order_ids);
  }
}

// The router's gradient: one wave a token, lane l holding the experts l, l + 64, ...
// Through renormalised weights w = c s / sum s:  dl = w (dw - sum_i w_i dw_i / c),
// times 1 - s for sigmoid scores; otherwise through w = c s.
template <int F32>
__global__ __launch_bounds__(256) void expert_route_backward_kernel(RouteGradArgs args) {
  (void)args;
  const RouteGradArgs& a = kernarg<RouteGradArgs>();
  const int lane = threadIdx.x & 63;
  for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < a.T; t += (int64_t)gridDim.x * 4) {
    const int64_t row = t * a.E;
    int id = -1;
    double d = 0.0, w = 0.0, g = 0.0;
    if (lane < a.k) {
      id = a.ids[t * a.k + lane];
      if ((uint32_t)id >= (uint32_t)a.E) id = -1;
      if (id >= 0) {
        w = a.weights[t * a.k + lane];
        g = a.dweights[t * a.k + lane];
      }
    }
    const bool routed = __ballot(id >= 0) != 0;
    const bool dense = a.score == SCORE_SOFTMAX && !a.renorm;
    const double l = id >= 0 ? (double)value_at<F32>(a.logits, row + id) : 0.0;
    const double total = sum_over<64>(w * g);
    if (id >= 0) {
      if (a.renorm) {
        d = w * (g - total / a.scale);
        if (a.score == SCORE_SIGMOID) d = d / (1.0 + exp(l));
      } else if (a.score == SCORE_SIGMOID) {
        d = w * g / (1.0 + exp(l));
      } else {
        d = w * g;
      }
    }
    const float df = (float)d;
    double top = kNone, sum = 0.0;
    if (dense && routed) {
      for (int e = lane; e < a.E; e += 64) top = fmax(top, (double)value_at<F32>(a.logits, row + e));
      top = max_over<64>(top);
      for (int e = lane; e < a.E; e += 64) sum += exp((double)value_at<F32>(a.logits, row + e) - top);
      sum = sum_over<64>(sum);
    }
    for (int e0 = 0; e0 < a.E; e0 += 64) {
      const int e = e0 + lane;
      float out = 0.0f;
      for (int j = 0; j < a.k; ++j) {
        const int ej = __builtin_amdgcn_readlane(id, j);
        const float dj = __uint_as_float(__builtin_amdgcn_readlane((int)__float_as_uint(df), j));
        if (e == ej) out = dj;
      }
      if (e < a.E) {
        if (dense && routed && top != kNone) out -= (float)(exp((double)value_at<F32>(a.logits, row + e) - top) / sum * total);
        if (F32) reinterpret_cast<float*>(a.dlogits)[row + e] = out;
        else reinterpret_cast<uint16_t*>(a.dlogits)[row + e] = (uint16_t)f32_to_bf16_bits(out);
      }
    }
  }
}

// Eight consecutive values.
template <int F32>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&v)[8]) {
  if constexpr (F32) {
    const f32x4_t* q = reinterpret_cast<const f32x4_t*>(reinterpret_cast<const float*>(p) + at);
    const f32x4_t lo = q[0], hi = q[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = lo[i], v[4 + i] = hi[i];
  } else {
    const u32x4_t w = *reinterpret_cast<const u32x4_t*>(reinterpret_cast<const uint16_t*>(p) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
template <int F32>
__device__ __forceinline__ void store8(void* p, int64_t at, const float (&v)[8]) {
  if constexpr (F32) {
    f32x4_t* q = reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(p) + at);
    q[0] = f32x4_t{v[0], v[1], v[2], v[3]};
    q[1] = f32x4_t{v[4], v[5], v[6], v[7]};
  } else {
    u32x4_t w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f32_to_bf16_bits(v[2 * i]) | f32_to_bf16_bits(v[2 * i + 1]) << 16;
    *reinterpret_cast<u32x4_t*>(reinterpret_cast<uint16_t*>(p) + at) = w;
  }
}

// y[t] = sum_j w[t][j] rows[pos[t][j]], in the order of j: eight values a thread.
template <int ROWS_F32, int Y_F32>
__global__ __launch_bounds__(256) void expert_combine_kernel(CombineArgs args) {
  (void)args;
  const CombineArgs& a = kernarg<CombineArgs>();
  const int per = a.H / 8;
  const int64_t units = (int64_t)a.T * per, R = (int64_t)a.T * a.k;
  for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < units; u += (int64_t)gridDim.x * 256) {
    const int64_t t = u / per;
    const int c = (int)(u - t * per) * 8;
    float acc[8] = {};
#pragma unroll 4
    for (int j = 0; j < a.k; ++j) {
      const int r = a.pos[t * a.k + j];
      if ((uint32_t)r >= (uint64_t)R) continue;
      const float w = a.weights[t * a.k + j];
      float v[8];
      load8<ROWS_F32>(a.rows, (int64_t)r * a.H + c, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(w, v[i], acc[i]);
    }
    store8<Y_F32>(a.y, t * a.H + c, acc);
  }
}

// Its gradient: a workgroup takes a token, writes w dy into each of its rows and
// sums dy . row.  Rows behind the last expert's become zeros.
template <int ROWS_F32, int Y_F32>
__global__ __launch_bounds__(256) void expert_combine_backward_kernel(CombineArgs args) {
  (void)args;
  const CombineArgs& a = kernarg<CombineArgs>();
  __shared__ float part[4][kExpertMaxK];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int64_t R = (int64_t)a.T * a.k;
  const int64_t used = min(max((int64_t)a.offsets[a.E], (int64_t)0), R);
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    float dot[kExpertMaxK];
#pragma unroll
    for (int j = 0; j < kExpertMaxK; ++j) dot[j] = 0.0f;
    for (int c = threadIdx.x * 8; c < a.H; c += blockDim.x * 8) {
      float dy[8];
      load8<Y_F32>(a.dy, t * a.H + c, dy);
#pragma unroll
      for (int j = 0; j < kExpertMaxK; ++j) {
        if (j < a.k) {
          const int r = a.pos[t * a.k + j];
          if ((uint32_t)r < (uint64_t)R) {
            const float w = a.weights[t * a.k + j];
            float v[8], o[8];
            load8<ROWS_F32>(a.rows, (int64_t)r * a.H + c, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              dot[j] = __builtin_fmaf(dy[i], v[i], dot[j]);
              o[i] = w * dy[i];
            }
            store8<ROWS_F32>(a.drows, (int64_t)r * a.H + c, o);
          }
          if (t * a.k + j >= used) {
            const float zero[8] = {};
            store8<ROWS_F32>(a.drows, (t * a.k + j) * a.H + c, zero);
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kExpertMaxK; ++j) {
      if (j < a.k) {
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) dot[j] += __shfl_xor(dot[j], d);
        if (lane == 0) part[wave][j] = dot[j];
      }
    }
    __syncthreads();
    if ((int)threadIdx.x < a.k) {
      float s = part[0][threadIdx.x];
      for (int w = 1; w < waves; ++w) s += part[w][threadIdx.x];
      a.dweights[t * a.k + threadIdx.x] = s;
    }
    __syncthreads();
  }
}

template <int L, int V>
hipError_t launch_route_sized(const RouteArgs& a, hipStream_t s) {
  if (a.logits_f32)
    hipLaunchKernelGGL((expert_route_kernel<L, V, 1>), dim3(a.chunks), dim3(kRouteThreads), 0, s, a);
  else
    hipLaunchKernelGGL((expert_route_kernel<L, V, 0>), dim3(a.chunks), dim3(kRouteThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace

int route_chunks(int64_t T, int64_t* chunk) {
  int64_t c = (T + 255) / 256;                              // at most 256 parts
  c = std::max<int64_t>(kRouteTokens, (c + kRouteTokens - 1) / kRouteTokens * kRouteTokens);
  if (chunk) *chunk = c;
  return (int)((T + c - 1) / c);
}

hipError_t launch_expert_route(const RouteArgs& a, hipStream_t s) {
  hipError_t e;
  if (a.E <= 64) e = launch_route_sized<16, 4>(a, s);
  else if (a.E <= 256) e = launch_route_sized<16, 16>(a, s);
  else e = launch_route_sized<64, 16>(a, s);
  if (e != hipSuccess || a.chunks == 1) return e;
  hipLaunchKernelGGL(expert_order_kernel, dim3(a.chunks), dim3(kRouteThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_expert_route_backward(const RouteGradArgs& a, hipStream_t s) {
  const unsigned blocks = (unsigned)std::min<int64_t>(((int64_t)a.T + 3) / 4, 1 << 20);
  if (a.logits_f32) hipLaunchKernelGGL(expert_route_backward_kernel<1>, dim3(blocks), dim3(256), 0, s, a);
  else hipLaunchKernelGGL(expert_route_backward_kernel<0>, dim3(blocks), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_expert_combine(const CombineArgs& a, hipStream_t s) {
  const unsigned blocks = (unsigned)std::min<int64_t>(((int64_t)a.T * (a.H / 8) + 255) / 256, 1 << 22);
  const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(blocks), dim3(256), 0, s, a); };
  if (a.rows_f32) a.y_f32 ? go(expert_combine_kernel<1, 1>) : go(expert_combine_kernel<1, 0>);
  else a.y_f32 ? go(expert_combine_kernel<0, 1>) : go(expert_combine_kernel<0, 0>);
  return hipGetLastError();
}

hipError_t launch_expert_combine_backward(const CombineArgs& a, hipStream_t s) {
  const unsigned blocks = (unsigned)std::min<int64_t>(a.T, 1 << 22);
  const unsigned threads = (unsigned)std::min(256, (a.H / 8 + 63) / 64 * 64);
  const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(blocks), dim3(threads), 0, s, a); };
  if (a.rows_f32) a.y_f32 ? go(expert_combine_backward_kernel<1, 1>) : go(expert_combine_backward_kernel<1, 0>);
  else a.y_f32 ? go(expert_combine_backward_kernel<0, 1>) : go(expert_combine_backward_kernel<0, 0>);
  return hipGetLastError();
}

}  // namespace tpf
