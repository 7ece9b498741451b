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

constexpr int kRouteThreads = 1024, kRouteWaves = kRouteThreads / 64;
constexpr int kRouteTokens = 64;       // tokens of a part of the order, at least
constexpr double kNone = -__builtin_huge_val();

// Data-parallel moves within rows of 16 lanes: one vector instruction for each 32
// bits, where an exchange through the LDS crossbar takes over 100 cycles.
constexpr int kRowShr = 0x110, kRowRor = 0x120, kRowBcast = 0x150;
template <int CTRL, class T>
__device__ __forceinline__ T dpp(T v) {
  if constexpr (sizeof(T) == 8) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xf, 0xf, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xf, 0xf, true);
    return __builtin_bit_cast(T, (uint64_t)hi << 32 | lo);
  } else {
    return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
  }
}
// f over the L lanes (16 or 64) that share a token, in all of them.
template <int L, class T, class F>
__device__ __forceinline__ T over(T v, F f) {
  static_assert(L == 16 || L == 64, "rows of 16 lanes, or all");
  v = f(v, dpp<kRowRor + 8>(v));
  v = f(v, dpp<kRowRor + 4>(v));
  v = f(v, dpp<kRowRor + 2>(v));
  v = f(v, dpp<kRowRor + 1>(v));
  if constexpr (L == 64) {
    v = f(v, __shfl_xor(v, 16));
    v = f(v, __shfl_xor(v, 32));
  }
  return v;
}
template <int L, class T>
__device__ __forceinline__ T max_over(T v) {
  return over<L>(v, [](T x, T y) { return max(x, y); });
}
template <int L, class T>
__device__ __forceinline__ T min_over(T v) {
  return over<L>(v, [](T x, T y) { return min(x, y); });
}
template <int L, class T>
__device__ __forceinline__ T sum_over(T v) {
  return over<L>(v, [](T x, T y) { return x + y; });
}
// The sum up to and with this lane.
template <int L>
__device__ __forceinline__ int sum_upto(int v, int li) {
  v += dpp<kRowShr + 1>(v);
  v += dpp<kRowShr + 2>(v);
  v += dpp<kRowShr + 4>(v);
  v += dpp<kRowShr + 8>(v);
  if constexpr (L == 64) {
    int o = __shfl(v, (li & 48) - 1);
    if (li & 16) v += o;
    o = __shfl(v, 31);
    if (li & 32) v += o;
  }
  return v;
}
// f(j, v of lane j) for the L lanes that share a token.
template <int L, int J = 0, class T, class F>
__device__ __forceinline__ void each_lane(T v, F f) {
  if constexpr (J < L) {
    if constexpr (L == 16) f(J, dpp<kRowBcast + J>(v));
    else f(J, __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), J)));
    each_lane<L, J + 1>(v, f);
  }
}
// The largest value's index, the lowest among equals; index INT_MAX: nothing.
__device__ __forceinline__ int best_over(double v, int at) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double ov = __shfl_xor(v, d);
    const int oa = __shfl_xor(at, d);
    if (ov > v || (ov == v && oa < at)) v = ov, at = oa;
  }
  return at;
}
// Lanes of one wave exchange values through LDS: its accesses stay in order.
__device__ __forceinline__ void wave_lds() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ---------------------------------------------------------------------------
// The order of the experts' rows.
//
// Each part of the tokens has counted its rows of every expert (hist[e][part],
// 16 bits).  An expert's rows of part b begin behind those of the experts before
// it and its own of earlier parts; within a part, waves take 64 slots at a time:
// ballots over the expert numbers' bits give each slot the number of equal ones
// before it in its wave, a count a wave and expert the number in the waves
// before.  No atomics, so the order is always that of the slots.  16384 x 8 slots of
// 256 experts: 12 us (one part's slots after another's 127), half of it the chain of
// loads from counts to ids to rows.
// ---------------------------------------------------------------------------
struct OrderLds {
  int base[kExpertMaxE + 1];                     // rows of every expert; then its next row
  int before[kExpertMaxE];                       // rows of every expert in earlier parts
  uint16_t wave[kRouteWaves][kExpertMaxE];       // rows of the waves before
};

__device__ void order_part(const RouteArgs& a, int b, OrderLds& lds) {
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  if (tid < 64) {                                // totals -> first rows, 64 experts at a time
    int before = 0;
    for (int base = 0; base < a.E; base += 64) {
      const int e = base + lane;
      const int n = e < a.E ? lds.base[e] : 0;
      const int upto = sum_upto<64>(n, lane);
      if (e < a.E) lds.base[e] = before + upto - n;
      before += __builtin_amdgcn_readlane(upto, 63);
    }
    if (lane == 0) lds.base[a.E] = before;
  }
  __syncthreads();
  const int R = a.T * a.k, used = lds.base[a.E];
  if (b == 0)
    for (int e = tid; e <= a.E; e += kRouteThreads) a.offsets[e] = lds.base[e];
  for (int64_t r = (int64_t)used + (int64_t)b * kRouteThreads + tid; r < R; r += (int64_t)a.chunks * kRouteThreads)
    a.src[r] = -1;                               // rows behind the last expert's have no slot
  if (a.chunks > 1) {
    __syncthreads();
    for (int e = tid; e < a.E; e += kRouteThreads) lds.base[e] += lds.before[e];
  }
  const int64_t first = (int64_t)b * a.chunk * a.k;
  const int64_t last = min((int64_t)R, first + (int64_t)a.chunk * a.k);
  int id_bits = 0;
  while (1 << id_bits < a.E) ++id_bits;
  for (int64_t s0 = first; s0 < last; s0 += kRouteThreads) {
    __syncthreads();
    for (int i = tid; i < kRouteWaves * kExpertMaxE / 8; i += kRouteThreads)
      reinterpret_cast<u32x4_t*>(lds.wave)[i] = u32x4_t{0, 0, 0, 0};
    __syncthreads();
    const int64_t slot = s0 + tid;
    const int id = slot < last ? a.ids[slot] : -1;
    uint64_t peers = __ballot(id >= 0);
    for (int i = 0; i < id_bits; ++i) {
      const uint64_t set = __ballot(id >> i & 1);
      peers &= id >> i & 1 ? set : ~set;
    }
    const int rank = __popcll(peers & ((1ull << lane) - 1));
    if (id >= 0 && rank == 0) lds.wave[w][id] = (uint16_t)__popcll(peers);
    __syncthreads();
    int total = 0;
    if (tid < a.E)
#pragma unroll
      for (int i = 0; i < kRouteWaves; ++i) {
        const int n = lds.wave[i][tid];
        lds.wave[i][tid] = (uint16_t)total;
        total += n;
      }
    __syncthreads();
    if (id >= 0) {
      const int row = lds.base[id] + lds.wave[w][id] + rank;
      a.pos[slot] = row;
      a.src[row] = (int)slot;
    } else if (slot < last) {
      a.pos[slot] = -1;
    }
    __syncthreads();
    if (tid < a.E) lds.base[tid] += total;
  }
}

__global__ __launch_bounds__(kRouteThreads) void expert_order_kernel(RouteArgs args) {
  (void)args;
  const RouteArgs& a = kernarg<RouteArgs>();
  __shared__ OrderLds lds;
  const int lane = threadIdx.x & 63;
  // One wave an expert, four parts' counts a lane, eight experts' loads at a time.
  const int wave = threadIdx.x >> 6;
  for (int e0 = wave; e0 < a.E; e0 += 8 * kRouteWaves) {
    int all[8] = {}, before[8] = {};
    for (int c = lane * 4; c < a.chunks; c += 256) {
      u32x2_t v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = *reinterpret_cast<const u32x2_t*>(a.hist + (int64_t)min(e0 + j * kRouteWaves, a.E - 1) * a.pad + c);
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = i & 1 ? (int)(v[j][i >> 1] >> 16) : (int)(v[j][i >> 1] & 0xffffu);
          all[j] += c + i < a.chunks ? n : 0;
          before[j] += c + i < (int)blockIdx.x ? n : 0;
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      all[j] = sum_over<64>(all[j]);
      before[j] = sum_over<64>(before[j]);
      if (lane == 0 && e0 + j * kRouteWaves < a.E) {
        lds.base[e0 + j * kRouteWaves] = all[j];
        lds.before[e0 + j * kRouteWaves] = before[j];
      }
    }
  }
  __syncthreads();
  order_part(a, blockIdx.x, lds);
}

// ---------------------------------------------------------------------------
// Scores, choice and weights.
// ---------------------------------------------------------------------------
__device__ __forceinline__ double sigmoid64(double x) { return 1.0 / (1.0 + exp(-x)); }

// A token's experts and weights once the choice is made: lane j < k of the L that
// share the token holds the j-th expert.  top and sum: the softmax's (64 bits); a sum
// of NaN makes the weights NaN.
template <int L, int F32>
__device__ __forceinline__ void put_choice(const RouteArgs& a, int t, int li, int id, bool routed, double top, double sum,
                                           int* hist) {
  const bool mine = routed && li < a.k && (uint32_t)id < (uint32_t)a.E;
  double s = 0.0;
  if (mine) {
    const double l = value_at<F32>(a.logits, (int64_t)t * a.E + id);
    s = a.score == SCORE_SIGMOID ? sigmoid64(l) : (top == kNone ? 0.0 : exp(l - top));
    if (!(sum == sum)) s = sum;
  }
  if (a.renorm) sum = sum_over<L>(s);
  if (li < a.k) {
    double w = 0.0;
    if (mine) w = a.renorm ? (sum == 0.0 ? 0.0 : a.scale * (s / sum)) :
                  a.scale * (a.score == SCORE_SIGMOID || sum == 0.0 ? s : s / sum);
    a.ids[(int64_t)t * a.k + li] = mine ? id : -1;
    a.weights[(int64_t)t * a.k + li] = (float)w;
    if (mine) atomicAdd(&hist[id], 1);
  }
}

template <int L, int F32>
__device__ __forceinline__ double softmax_sum(const RouteArgs& a, int64_t row, int li, double top) {
  double sum = 0.0;
#pragma unroll 1
  for (int e = li; e < a.E; e += L) sum += exp((double)value_at<F32>(a.logits, row + e) - top);
  return sum_over<L>(sum);
}

// One token by a whole wave, everything in 64 bits: the definition as it stands.
// values: LDS of E numbers.
template <int F32>
__device__ __forceinline__ void route_token(const RouteArgs& a, int t, int lane, int* hist, double* values) {
  const int64_t row = (int64_t)t * a.E;
  const bool softmax = a.score == SCORE_SOFTMAX, scores = a.bias || a.groups > 1;
  double top = kNone, sum = 1.0;
#pragma unroll 1
  for (int e = lane; e < a.E; e += 64) {
    const double l = value_at<F32>(a.logits, row + e);
    if (!(l == l)) sum = l;
    top = max(top, l);
  }
  top = max_over<64>(top);
  if (softmax) {                    // over a NaN or +inf it is NaN throughout, renormalised or not
    if (__ballot(!(sum == sum)) || top == -kNone) sum = __builtin_nan("");
    else if (scores || !a.renorm) sum = top == kNone ? 0.0 : softmax_sum<64, F32>(a, row, lane, top);
  } else {
    sum = 1.0;
  }
  wave_lds();
#pragma unroll 1
  for (int e = lane; e < a.E; e += 64) {
    const double l = value_at<F32>(a.logits, row + e);
    double v = l;
    if (scores) v = softmax ? (sum == 0.0 ? 0.0 : exp(l - top) / sum) : sigmoid64(l);
    if (a.bias) v += (double)a.bias[e];
    values[e] = v == v ? v : kNone;
  }
  wave_lds();
  uint32_t allowed = ~0u;
  const int gs = a.E / a.groups;
  if (a.groups > 1) {
    double t1 = kNone, t2 = kNone;  // lane g's: the two largest of group g
    if (lane < a.groups)
#pragma unroll 4
      for (int i = 0; i < gs; ++i) {
        const double v = values[lane * gs + i];
        t2 = max(t2, min(t1, v));
        t1 = max(t1, v);
      }
    double mine = gs > 1 ? t1 + t2 : t1;
    if (!(mine == mine)) mine = kNone;
    allowed = 0;
    bool free_group = lane < a.groups;
    for (int g = 0; g < a.top_groups; ++g) {
      const int at = best_over(free_group ? mine : kNone, free_group ? lane : INT32_MAX);
      allowed |= 1u << at;
      if (lane == at) free_group = false;
    }
    if (!a.bias) {                  // ordered by the logit
      wave_lds();
      for (int e = lane; e < a.E; e += 64) {
        const double l = value_at<F32>(a.logits, row + e);
        values[e] = l == l ? l : kNone;
      }
      wave_lds();
    }
  }
  uint32_t taken = 0;               // the lane's experts that cannot be chosen (any more)
  for (int i = 0; i * 64 < a.E; ++i) {
    const int e = i * 64 + lane;
    if (e >= a.E || (a.groups > 1 && !(allowed >> (e / gs) & 1))) taken |= 1u << i;
  }
  int id = -1;                      // lane j's: the token's j-th expert
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) {
    double best = kNone;
    int at = INT32_MAX;
#pragma unroll 1
    for (int i = 0; i * 64 < a.E; ++i) {        // a lane's experts rise with i: the first of equals stays
      const int e = i * 64 + lane;
      if (taken >> i & 1) continue;
      const double v = values[e];
      if (v > best || at == INT32_MAX) best = v, at = e;
    }
    at = best_over(best, at);
    if ((at & 63) == lane) taken |= 1u << (at >> 6);
    if (lane == j) id = at;
  }
  put_choice<64, F32>(a, t, lane, id, true, top, sum, hist);
}

// Routes one part of the tokens, L lanes a token, lane l holding experts 4 l to
// 4 l + 3 of every 4 L (so loads are 16 bytes and a group of experts is whole
// fours).
//
// Scores are computed in fp32 with a bound on their error.  The k-th largest of
// the lanes' maxima is not above the token's k-th largest value; what reaches it
// within the bound, a dozen values as a rule, goes into a list, and an entry's
// place is the number of entries before it.  Where two entries lie closer than the
// bound, places are taken from the list's values in 64 bits, and so are the groups
// where one taken and one that is not lie so close; where more than 32
// values reach the list, fewer than k do or something is not finite, the token is
// routed again by the whole wave in 64 bits: the choice is always the definition's.
// Without bias values are the logits themselves and nothing is uncertain.  Where fewer
// than k lanes hold an expert that can be chosen (k above the fours of E or of the
// groups taken), every finite value reaches the list: up to 32 of them that is the fast
// way still (choice and order of 16384 tokens to 8 of 16: 14 us, in 64 bits 48), with
// more experts (k from 14 on of 60: 55 to 78 us) it is not.
// 16384 tokens, 256 experts in 8 groups with bias: 88 us with everything in 64 bits
// and a round over all values for each choice, 20 this way (bound by vector
// instructions of about 5100 cycles a wave and by their first fetch).
constexpr int kRouteList = 32;
// A value and its expert as one number that is compared: larger values first, the
// lower number first among equals.
__device__ __forceinline__ int64_t route_key(float v, int e) {
  const int bits = __builtin_bit_cast(int, v + 0.0f);          // no -0
  return (int64_t)((uint64_t)(uint32_t)(bits ^ (bits >> 31 & 0x7fffffff)) << 32 | (uint32_t)~e);
}
__device__ __forceinline__ float key_value(int64_t key) {
  const int bits = (int)(key >> 32);
  return __builtin_bit_cast(float, bits ^ (bits >> 31 & 0x7fffffff));
}
__device__ __forceinline__ int key_expert(int64_t key) { return ~(int)(uint32_t)key; }
template <int L, int V>
struct ChoiceLds {
  static constexpr int kValues = L == 64 ? L * V : V == 4 ? 128 : 32 * V;     // 64 V / 4 pairs, 64 / L lists, E
  static_assert(kValues >= 32 * V && kValues >= 64 / L * kRouteList && kValues >= L * V, "values of a wave");
  double values[kRouteWaves][kValues];            // also: the two largest of each four experts of the wave's tokens
  int64_t list[kRouteWaves][64 / L * kRouteList];
  int64_t sorted[kRouteWaves][64 / L * kRouteList];
};
typedef f32x4_t f32x4a4_t __attribute__((aligned(4)));      // the bias lies at any float
template <int L, int V>
union RouteLds {
  ChoiceLds<L, V> choice;
  OrderLds order;
};

// Which groups are taken: lane g's `in` for group g.  quads: LDS, the two largest of
// each four experts.  Values v are off by up to slack / 2 (1 + |v|), and so are a
// group's two largest, whose sum may be far smaller than they are; `sure`: the sums
// taken lie above the others by more than that.
template <int L, class T>
__device__ __forceinline__ void choose_groups(const RouteArgs& a, const T (*quads)[2], int li, T slack, bool& in,
                                              bool& sure) {
  const T none = -(T)__builtin_huge_val();
  wave_lds();
  T t1 = none, t2 = none;
  const int n = a.E / a.groups / 4;
  if (li < a.groups)
    for (int i0 = 0; i0 < n; i0 += 4) {
      T o[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int q = li * n + min(i0 + i, n - 1);
        o[i][0] = quads[q][0];
        o[i][1] = quads[q][1];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i0 + i < n) {
          t2 = max(min(t1, o[i][0]), max(t2, o[i][1]));
          t1 = max(t1, o[i][0]);
        }
    }
  T mine = t1 + t2;
  if (!(li < a.groups && mine == mine)) mine = none;
  int place = 0;
  each_lane<16>(L == 16 ? mine : __shfl(mine, li & 15), [&](int g, T o) { place += o > mine || (o == mine && g < li); });
  in = li < a.groups && place < a.top_groups;
  const T off = slack * (T(1) + fabs(t1) + fabs(t2));     // both values', the sum's rounding and that of what follows
  T low = mine - off, high = mine + off;
  if (!(low == low)) low = none;
  if (!(high == high)) high = -none;
  sure = min_over<L>(in ? low : -none) > max_over<L>(in || li >= a.groups ? none : high);
}

template <int L, int V, int F32>
__global__ __launch_bounds__(kRouteThreads) void expert_route_kernel(RouteArgs args) {
  (void)args;
  const RouteArgs& a = kernarg<RouteArgs>();
  __shared__ RouteLds<L, V> lds;
  __shared__ int hist[kExpertMaxE];
  constexpr int TOKENS = 64 / L, LIST = kRouteList;
  constexpr float kLog2e = 1.44269504089f;
  const int b = blockIdx.x, wave = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < a.E; e += kRouteThreads) hist[e] = 0;
  __syncthreads();
  const bool softmax = a.score == SCORE_SOFTMAX, scores = a.bias || a.groups > 1;
  const int gs = a.E / a.groups, gs_inv = ((1 << 20) + gs - 1) / gs;
  // Groups of whole fours take the fast way, and any number of experts without groups (but see k above); other groups
  // are routed in 64 bits by the whole wave (16384 tokens: 6 of 128 17 us, of 129 by single loads 19, in 64 bits 47;
  // 6 of 64 in 4 groups 17, of 60 49).
  const bool whole = a.E % 4 == 0, fours = a.groups == 1 || (whole && gs % 4 == 0);
  // Twice the largest error of an fp32 value v is below bound (1 + |v|): sigmoid 4e-7 (exp2, reciprocal and sum
  // round by 1.2e-7 at most, the argument's rounding counts s (1 - s) |x| 2^-24), softmax 2.4e-6 (a sum of 1024).
  const float bound = !a.bias ? 0.0f : softmax ? 0x1p-17f : 0x1p-20f;
  const float gslack = softmax ? 0x1p-17f : 0x1p-20f;
  const int t_end = min(a.T, (b + 1) * a.chunk);
  for (int t0 = b * a.chunk + wave * TOKENS; t0 < t_end; t0 += kRouteWaves * TOKENS) {
    // Hidden from the compiler, which would hold what follows from the lane's number in registers over the loop.
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int li = lane & (L - 1), lt = lane / L, lane0 = lane & ~(L - 1);
    double(*quads)[2] = reinterpret_cast<double(*)[2]>(lds.choice.values[wave]) + lt * (L * V / 4);
    int64_t* list = lds.choice.list[wave] + lt * LIST;
    int64_t* sorted = lds.choice.sorted[wave] + lt * LIST;
    // Number of the lane's q-th four: turned from q to q, so that groups of experts spread over the lanes.
    const auto four = [&](int q) { return q * L + ((li + q * (L / 4)) & (L - 1)); };
    const int t = t0 + lt;
    const bool routed = t < t_end && (!a.mask || a.mask[t]);
    const int64_t row = (int64_t)min(t, t_end - 1) * a.E;
    bool unsure = !fours;
    int id = -1;
    double top64 = kNone, sum64 = 1.0;
    if (fours) {
      float x[V], v[V];
      float top = -__builtin_huge_valf();
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        const int e = four(q) * 4;
        f32x4_t w = f32x4_t{top, top, top, top};       // past the last expert: -inf
        if (!whole) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (e + i < a.E) w[i] = value_at<F32>(a.logits, row + e + i);
        } else if (e < a.E) {
          if constexpr (F32) {
            w = *reinterpret_cast<const f32x4_t*>(reinterpret_cast<const float*>(a.logits) + row + e);
          } else {
            const u32x2_t h = *reinterpret_cast<const u32x2_t*>(reinterpret_cast<const uint16_t*>(a.logits) + row + e);
            w = f32x4_t{__uint_as_float(h[0] << 16), __uint_as_float(h[0] & 0xffff0000u), __uint_as_float(h[1] << 16),
                        __uint_as_float(h[1] & 0xffff0000u)};
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) x[4 * q + i] = w[i];
      }
      bool lost = false;            // to be routed in 64 bits
#pragma unroll
      for (int i = 0; i < V; ++i) lost |= !(x[i] == x[i]);
      if (softmax) {
#pragma unroll
        for (int i = 0; i < V; ++i) top = max(top, x[i]);
        top = max_over<L>(top);
        lost |= !(fabsf(top) < __builtin_huge_valf());
        top64 = top;
        if (!a.renorm) sum64 = softmax_sum<L, F32>(a, row, li, top64);
      }
      if (scores) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          v[i] = __builtin_amdgcn_exp2f((softmax ? x[i] - top : -x[i]) * kLog2e);
          if (softmax) sum += v[i];
        }
        const float inv = softmax ? __builtin_amdgcn_rcpf(sum_over<L>(sum)) : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = softmax ? v[i] * inv : __builtin_amdgcn_rcpf(1.0f + v[i]);
        if (a.bias)
#pragma unroll
          for (int q = 0; q < V / 4; ++q)
            if (four(q) * 4 + 3 < a.E) {
              const f32x4a4_t c = *reinterpret_cast<const f32x4a4_t*>(a.bias + four(q) * 4);
#pragma unroll
              for (int i = 0; i < 4; ++i) v[4 * q + i] += c[i];
            } else if (!whole) {
#pragma unroll
              for (int i = 0; i < 3; ++i)
                if (four(q) * 4 + i < a.E) v[4 * q + i] += a.bias[four(q) * 4 + i];
            }
        // a bias that is NaN: what follows counts on values that are ordered
#pragma unroll
        for (int i = 0; i < V; ++i) lost |= !(v[i] == v[i]);
      }
      if (a.groups > 1) {
        bool in, sure;
        float(*pairs)[2] = reinterpret_cast<float(*)[2]>(quads);
        wave_lds();
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
          const float a0 = max(v[4 * q], v[4 * q + 1]), a1 = min(v[4 * q], v[4 * q + 1]);
          const float b0 = max(v[4 * q + 2], v[4 * q + 3]), b1 = min(v[4 * q + 2], v[4 * q + 3]);
          pairs[four(q)][0] = max(a0, b0);
          pairs[four(q)][1] = max(min(a0, b0), max(a1, b1));
        }
        choose_groups<L>(a, pairs, li, gslack, in, sure);
        if (__ballot(a.top_groups < a.groups && !sure)) {
          if (softmax && a.renorm) sum64 = softmax_sum<L, F32>(a, row, li, top64);
          wave_lds();
#pragma unroll 1
          for (int q = li; q < a.E / 4; q += L) {
            double t1 = kNone, t2 = kNone;
#pragma unroll 1
            for (int e = q * 4; e < q * 4 + 4; ++e) {
              const double l = value_at<F32>(a.logits, row + e);
              const double s = (softmax ? exp(l - top64) / sum64 : sigmoid64(l)) + (a.bias ? (double)a.bias[e] : 0.0);
              t2 = max(t2, min(t1, s));
              t1 = max(t1, s);
            }
            quads[q][0] = t1;
            quads[q][1] = t2;
          }
          choose_groups<L>(a, quads, li, 0.0, in, sure);
        }
        const uint32_t allowed = (uint32_t)(__ballot(in) >> lane0) & 0xffffu;
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
          const int g = (int)((uint32_t)(four(q) * 4) * (uint32_t)gs_inv >> 20);
          const bool in = g < a.groups && (allowed >> g & 1);
#pragma unroll
          for (int i = 4 * q; i < 4 * q + 4; ++i) v[i] = in ? (a.bias ? v[i] : x[i]) : -__builtin_huge_valf();
        }
      } else if (!a.bias) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = x[i];
      } else {
#pragma unroll
        for (int q = 0; q < V / 4; ++q)
          if (four(q) * 4 + 3 >= a.E)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (four(q) * 4 + i >= a.E) v[4 * q + i] = -__builtin_huge_valf();
      }
      // The k-th largest of the lanes' maxima.
      float m = v[0];
#pragma unroll
      for (int i = 1; i < V; ++i) m = max(m, v[i]);
      int place = 0;
      each_lane<L>(m, [&](int j, float o) { place += o > m || (o == m && j < li); });
      const uint64_t kth = __ballot(place == a.k - 1) >> lane0 & (L == 64 ? ~0ull : (1ull << L) - 1);
      float least = __shfl(m, lane0 + (kth ? __builtin_ctzll(kth) : 0));
      least = max(least - 2.0f * bound * (1.0f + fabsf(least)), -0x1.fffffep127f);     // fewer lanes: all that is finite
      int n = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) n += v[i] >= least;
      const int upto = sum_upto<L>(n, li);
      const int total = max_over<L>(upto);
      lost |= total > LIST || total < a.k;
      int at = upto - n;
      wave_lds();
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (v[i] >= least) {
          if (at < LIST) list[at] = route_key(v[i], four(i / 4) * 4 + i % 4);
          ++at;
        }
      wave_lds();
      const int held = min(total, LIST);
      int most = held;
#pragma unroll
      for (int d = L; d < 64; d <<= 1) most = max(most, __shfl_xor(most, d));
      most = __builtin_amdgcn_readfirstlane(most);
      // Entries li and (where 16 lanes share the token) li + 16: their places.
      constexpr int PER = LIST > L ? LIST / L : 1;
      int64_t own[PER];
      int before[PER] = {};
#pragma unroll
      for (int i = 0; i < PER; ++i) own[i] = list[min(li + i * L, LIST - 1)];
      for (int j0 = 0; j0 < most; j0 += 4) {
        int64_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = list[j0 + j];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < PER; ++i) before[i] += j0 + j < held && o[j] > own[i];
      }
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (li + i * L < held) sorted[before[i]] = own[i];
      wave_lds();
      bool close = false;           // lane j: entry j and the one after it
      if (a.bias && li < a.k && li + 1 < held) {
        const float v0 = key_value(sorted[li]), v1 = key_value(sorted[li + 1]);
        close = !(v0 - v1 > bound * (1.0f + fabsf(v0)));
      }
      if (__ballot(close)) {        // places by the values in 64 bits
        if (softmax && a.renorm) sum64 = softmax_sum<L, F32>(a, row, li, top64);
        double* values = lds.choice.values[wave] + lt * LIST;
#pragma unroll 1
        for (int j = li; j < held; j += L) {
          const int e = key_expert(list[j]);
          const double l = value_at<F32>(a.logits, row + e);
          values[j] = (softmax ? exp(l - top64) / sum64 : sigmoid64(l)) + (double)a.bias[e];
        }
        wave_lds();
#pragma unroll 1
        for (int i = li; i < held; i += L) {
          const double mine = values[i];
          const int64_t key = list[i];
          int n = 0;
#pragma unroll 1
          for (int j = 0; j < held; ++j) n += values[j] > mine || (values[j] == mine && key_expert(list[j]) < key_expert(key));
          sorted[n] = key;
        }
        wave_lds();
      }
      if (li < a.k) id = key_expert(sorted[li]);
      unsure = (__ballot(lost) >> lane0 & (L == 64 ? ~0ull : (1ull << L) - 1)) != 0;
    }
    if (t < t_end && !(unsure && routed)) put_choice<L, F32>(a, t, li, id, routed, top64, sum64, hist);
    uint64_t again = __ballot(unsure && routed && li == 0);
    while (again) {
      const int at = __builtin_ctzll(again);
      again &= again - 1;
      route_token<F32>(a, __builtin_amdgcn_readlane(t, at), lane, hist, lds.choice.values[wave]);
    }
  }
  __syncthreads();
  if (a.chunks == 1) {
    for (int e = threadIdx.x; e < a.E; e += kRouteThreads) lds.order.base[e] = hist[e];
    __syncthreads();
    order_part(a, 0, lds.order);
  } else {
    for (int e = threadIdx.x; e < a.E; e += kRouteThreads) a.hist[(int64_t)e * a.pad + b] = (uint16_t)hist[e];
  }
}

// The router's gradient.  Through renormalised weights w = c s / sum s it is
// dl = w (dw - sum_i w_i dw_i / c), times 1 - s for sigmoid scores.  The weights sum to
// c, so that is w sum_i w_i (dw - dw_i) / c, which does not cancel where one weight is
// close to c and its difference to c lost in its rounding to fp32.  Otherwise
// dl = w dw (1 - s) through w = c s of a sigmoid: nothing but the chosen experts'
// logits matter.  16 lanes take a token's choices and lay its row out in LDS, so that
// the gradient is written once, whole (16384 tokens, 256 experts: 7 us; with a wave a
// token that goes over all of its logits 16).
constexpr int kGradTokens = 16;
template <int F32>
__global__ __launch_bounds__(256) void expert_route_backward_kernel(RouteGradArgs args) {
  (void)args;
  const RouteGradArgs& a = kernarg<RouteGradArgs>();
  extern __shared__ __attribute__((aligned(16))) float rows[];      // [kGradTokens][E rounded up to 8]
  const int lane = threadIdx.x & 63, li = lane & 15, tok = threadIdx.x >> 4, width = (a.E + 7) & ~7;
  float* mine = rows + tok * width;
  for (int64_t t0 = (int64_t)blockIdx.x * kGradTokens; t0 < a.T; t0 += (int64_t)gridDim.x * kGradTokens) {
    const int64_t t = t0 + tok;
    for (int e = li * 4; e < width; e += 64) *reinterpret_cast<f32x4_t*>(mine + e) = f32x4_t{0, 0, 0, 0};
    int id = -1;
    float w = 0.0f, g = 0.0f;
    if (t < a.T && li < a.k) {
      id = a.ids[t * a.k + li];
      if ((uint32_t)id >= (uint32_t)a.E) id = -1;
      if (id >= 0) {
        w = a.weights[t * a.k + li];
        g = a.dweights[t * a.k + li];
      }
    }
    double d = g;
    if (a.renorm) {
      double sum = 0.0;
      each_lane<16>((uint64_t)__float_as_uint(g) << 32 | __float_as_uint(w), [&](int, uint64_t o) {
        sum += (double)__uint_as_float((uint32_t)o) * ((double)g - (double)__uint_as_float((uint32_t)(o >> 32)));
      });
      d = sum / a.scale;
    }
    d *= w;
    if (a.score == SCORE_SIGMOID && id >= 0) d = d / (1.0 + exp((double)value_at<F32>(a.logits, t * a.E + id)));
    wave_lds();
    if (id >= 0) mine[id] = (float)d;
    wave_lds();
    if (t < a.T && a.E % 8 == 0) {                        // rows of the gradient are whole 16 bytes
      for (int e = li * 8; e < a.E; e += 128) {
        const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(mine + e);
        const f32x4_t hi = *reinterpret_cast<const f32x4_t*>(mine + e + 4);
        if constexpr (F32) {
          f32x4_t* out = reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(a.dlogits) + t * a.E + e);
          out[0] = lo;
          out[1] = hi;
        } else {
          *reinterpret_cast<u32x4_t*>(reinterpret_cast<uint16_t*>(a.dlogits) + t * a.E + e) =
              u32x4_t{bf16_pair(lo[0], lo[1]), bf16_pair(lo[2], lo[3]), bf16_pair(hi[0], hi[1]), bf16_pair(hi[2], hi[3])};
        }
      }
    } else if (t < a.T) {
      for (int e = li; e < a.E; e += 16) {
        if constexpr (F32) reinterpret_cast<float*>(a.dlogits)[t * a.E + e] = mine[e];
        else reinterpret_cast<uint16_t*>(a.dlogits)[t * a.E + e] = (uint16_t)f32_to_bf16_bits(mine[e]);
      }
    }
    wave_lds();
  }
}

// Lane j's, j the same in all lanes.
__device__ __forceinline__ double lane_value(double v, int j) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, j);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), j);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Through softmax scores that are not renormalised every logit has a gradient:
// dl = s (g - sum_i s_i g_i), g = c dw at the chosen, 0 elsewhere.  At a chosen j the
// difference is taken apart, sum_i s_i (g_j - g_i) + g_j (the others' s): near s_j = 1 it
// is that much smaller than its terms, and is left with their full precision this way.
// The scores are those of the logits in 64 bits, not the weights' rounded ones.  One
// wave a token; lane j < k holds the j-th expert.  Two 64-bit exponentials an expert
// bound it: 16384 tokens to 8 of 64 13 us, 8 of 256 26, 16 of 1024 85.
template <int F32>
__global__ __launch_bounds__(256) void expert_route_dense_backward_kernel(RouteGradArgs args) {
  (void)args;
  const RouteGradArgs& a = kernarg<RouteGradArgs>();
  const int lane = threadIdx.x & 63;
  const auto put = [&](int64_t at, double v) {
    if constexpr (F32) reinterpret_cast<float*>(a.dlogits)[at] = (float)v;
    else reinterpret_cast<uint16_t*>(a.dlogits)[at] = (uint16_t)f32_to_bf16_bits((float)v);
  };
  for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < a.T; t += (int64_t)gridDim.x * 4) {
    const int64_t row = t * a.E;
    int id = -1;
    double g = 0.0, l = kNone;
    if (lane < a.k) {
      id = a.ids[t * a.k + lane];
      if ((uint32_t)id >= (uint32_t)a.E) id = -1;
      if (id >= 0) {
        g = a.scale * a.dweights[t * a.k + lane];
        l = value_at<F32>(a.logits, row + id);
      }
    }
    uint32_t chosen = 0;                                // of the experts 64 i + lane: bit i
    for (int j = 0; j < a.k; ++j) {
      const int ej = __builtin_amdgcn_readlane(id, j);
      if (ej >= 0 && (ej & 63) == lane) chosen |= 1u << (ej >> 6);
    }
    double top = kNone, others = 0.0, x = 0.0;
    if (__ballot(id >= 0)) {
      for (int e = lane; e < a.E; e += 64) top = max(top, (double)value_at<F32>(a.logits, row + e));
      top = max_over<64>(top);
    }
    // No logit above -inf: the scores are 0, as the router has them (but NaN if there is nothing else).
    const bool any = top != kNone || __ballot(!(l == l));
    if (any) {
      for (int e0 = 0; e0 < a.E; e0 += 64) {
        const int e = e0 + lane;
        const double v = e < a.E ? exp((double)value_at<F32>(a.logits, row + e) - top) : 0.0;
        if (!(chosen >> (e0 >> 6) & 1)) others += v;
        const double mine = __shfl(v, id & 63);
        if (id >= 0 && id >> 6 == e0 >> 6) x = mine;
      }
      others = sum_over<64>(others);
    }
    const double part = any ? 1.0 / (others + sum_over<64>(x)) : 0.0, total = sum_over<64>(x * g) * part * part;
    double d = g * others;
#pragma unroll 1
    for (int j = 0; j < a.k; ++j) d += lane_value(x, j) * (g - lane_value(g, j));
    if (id >= 0) put(row + id, x * part * (d * part));
    for (int e = lane; e < a.E; e += 64)
      if (!(chosen >> (e >> 6) & 1))
        put(row + e, any ? -(exp((double)value_at<F32>(a.logits, row + e) - top) * total) : 0.0);
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
// Past the caches: on their way through them the stores cost rows still to be read
// (the gradient of 1003 tokens, 6 slots, H 5000, its outputs kept: 48 us, past them
// 28; with the packing of what it wrote behind it 98 either way).
template <int F32>
__device__ __forceinline__ void store8(void* p, int64_t at, const float (&v)[8]) {
  if constexpr (F32) {
    f32x4_t* q = reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(p) + at);
    __builtin_nontemporal_store(f32x4_t{v[0], v[1], v[2], v[3]}, q);
    __builtin_nontemporal_store(f32x4_t{v[4], v[5], v[6], v[7]}, q + 1);
  } else {
    u32x4_t w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
    __builtin_nontemporal_store(w, reinterpret_cast<u32x4_t*>(reinterpret_cast<uint16_t*>(p) + at));
  }
}

// y[t] = sum_j w[t][j] rows[pos[t][j]], in the order of j: eight values a thread.
// Memory bounds it: 4096 tokens, 8 slots, H 4096: 64 us, 4.7 TB/s.
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
    for (int j0 = 0; j0 < a.k; j0 += 8) {       // the slots' rows first, then all their loads
      int r[8];
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t at = t * a.k + min(j0 + j, a.k - 1);
        r[j] = j0 + j < a.k ? a.pos[at] : -1;
        w[j] = a.weights[at];
      }
      float v[8][8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if ((uint32_t)r[j] < (uint64_t)R) load8<ROWS_F32>(a.rows, (int64_t)r[j] * a.H + c, v[j]);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if ((uint32_t)r[j] < (uint64_t)R)
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(w[j], v[j][i], acc[i]);
    }
    store8<Y_F32>(a.y, t * a.H + c, acc);
  }
}

// Its gradient: a workgroup takes a token, writes w dy into each of its rows and
// sums dy . row.  Rows behind the last expert's become zeros.  1003 tokens, 6 slots,
// H 5000: 28 us, 4.4 TB/s.
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
      // Four slots' loads before their stores, which the compiler could not move them across.
#pragma unroll
      for (int j0 = 0; j0 < kExpertMaxK; j0 += 4) {
        if (j0 < a.k) {
          int r[4];
          float v[4][8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            r[j] = j0 + j < a.k ? a.pos[t * a.k + j0 + j] : -1;
            if ((uint32_t)r[j] < (uint64_t)R) load8<ROWS_F32>(a.rows, (int64_t)r[j] * a.H + c, v[j]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if ((uint32_t)r[j] < (uint64_t)R) {
              const float w = a.weights[t * a.k + j0 + j];
              float o[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                dot[j0 + j] = __builtin_fmaf(dy[i], v[j][i], dot[j0 + j]);
                o[i] = w * dy[i];
              }
              store8<ROWS_F32>(a.drows, (int64_t)r[j] * a.H + c, o);
            }
            if (j0 + j < a.k && t * a.k + j0 + j >= used) {
              const float zero[8] = {};
              store8<ROWS_F32>(a.drows, (t * a.k + j0 + j) * a.H + c, zero);
            }
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
  int64_t c = (T + 255) / 256;                              // 256 parts, one a compute unit
  c = std::max<int64_t>(kRouteTokens, (c + kRouteTokens - 1) / kRouteTokens * kRouteTokens);
  c = std::min<int64_t>(c, 1023 * kRouteTokens);            // a part's counts are held in 16 bits
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
  if (a.score == SCORE_SOFTMAX && !a.renorm) {
    const unsigned blocks = (unsigned)std::min<int64_t>(((int64_t)a.T + 3) / 4, 1 << 20);
    if (a.logits_f32) hipLaunchKernelGGL(expert_route_dense_backward_kernel<1>, dim3(blocks), dim3(256), 0, s, a);
    else hipLaunchKernelGGL(expert_route_dense_backward_kernel<0>, dim3(blocks), dim3(256), 0, s, a);
    return hipGetLastError();
  }
  const unsigned blocks = (unsigned)std::min<int64_t>(((int64_t)a.T + kGradTokens - 1) / kGradTokens, 1 << 22);
  const unsigned lds = kGradTokens * ((a.E + 7) / 8 * 8) * sizeof(float);      // at most 64 KiB
  if (a.logits_f32) hipLaunchKernelGGL(expert_route_backward_kernel<1>, dim3(blocks), dim3(256), lds, s, a);
  else hipLaunchKernelGGL(expert_route_backward_kernel<0>, dim3(blocks), dim3(256), lds, s, a);
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
