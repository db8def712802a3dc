// moe_route.cu -- routing of tokens to experts: scores, group-limited top-k,
// weights, and the gradient of the logits.
//
// For the E logits x of a token (bf16 or fp32; x <= kRouteOff marks an expert
// as off):
//   s_e = exp(x_e) / sum_live exp(x)  or  1 / (1 + exp(-x_e)),  0 where off
//   v_e = s_e + bias_e                (bias optional; -inf where off)
//   groups of E / groups consecutive experts: a group's score is the sum of
//   its `group_best` (1 or 2) largest v (off experts count 0; -inf if all are
//   off); the top_groups best groups stay, the others' v become -inf
//   chosen: the top_k largest v > -inf in descending order, ties to the lower
//   index; slots left over get expert -1 and weight 0
//   w_i = scale * s_i / (renorm ? sum of the chosen s : 1)
//
// Ranking.  Sums of two close scores may differ by less than fp32 arithmetic
// tells apart, and which expert wins is a whole number.  Where the ranking
// follows the logits themselves (no bias, and no sum over a group's best two)
// the logits are compared, which is exact.  Otherwise the scores are computed
// in fp32 together with a bound on their error; if every gap that decides
// something (between neighbours among the chosen and the first expert left
// out, and at the border of the kept groups) exceeds the bound, the ranking
// is that of the exact scores.  (Equal logits with equal biases have no gap to
// decide; at the border of the chosen ones the next expert behind such an equal is
// looked at instead.)  If one does not (about one token in a thousand
// for 256 sigmoid scores with a random bias), the candidates are ranked in fp64,
// one per lane; a border of groups, a softmax row or a third close candidate
// takes the whole token through fp64.  (All such tokens in fp64 throughout cost
// 9 of 32 us at 16384 tokens of 256 experts.)
//
// One warp per token, E/32 logits per lane in registers; each of the top_k
// rounds is one warp-wide integer maximum over order-preserving keys and one
// minimum over the indices that hold it; a lane keeps its two best candidates,
// so it seldom looks through its keys again.  Bound by its instructions (about
// 1200 per token of 256 experts in groups): 16384 tokens 23 us, 32 tokens 4.3 us
// on GB300, sigmoid scores with a bias, 4 of 8 groups, top 8.  Loading the next
// token ahead in fewer, longer-lived warps was slower (35 us).
#include <type_traits>

#include "wst.h"
#include "wst_common.cuh"
#include "wst_host.h"

namespace wst {

namespace {

constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopK = 16;
constexpr int kRouteMaxGroups = 32;
constexpr float kRouteOff = -3.0e38f;

struct RouteArgs {
  int T, E, top_k;
  const void* logits;
  long long ld;
  const float* bias;
  int groups, top_groups, group_best;
  int group_size;
  int group_shift;       // 2^group_shift lanes share the scan of a group
  uint32_t group_magic;  // e / group_size == e * group_magic >> 20 for e < 1024
  int renorm;
  float scale;
  int* experts;
  float* weights;
};

__device__ __forceinline__ float load_logit(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(__ldg(p)); }

// Order-preserving keys: larger value, larger key; NaN above +inf (as
// torch.topk ranks it), -0 equal to +0; 0 stands for "not a candidate".
// (The addition makes -0 +0 and any NaN the one with bits 0x7fffffff.)
__device__ __forceinline__ uint32_t order_key(float v) {
  const int32_t b = __float_as_int(v + 0.0f);
  return (uint32_t)(b ^ ((b >> 31) | (int32_t)0x80000000));
}
__device__ __forceinline__ uint64_t order_key(double v) {
  if (v != v) return ~0ull;
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  return (b >> 63) ? ~b : (b | (1ull << 63));
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ double key_value(uint64_t k) {
  return __longlong_as_double((long long)((k >> 63) ? (k & ~(1ull << 63)) : ~k));
}

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return ((uint64_t)hi << 32) | lo;
}
template <typename R>
__device__ __forceinline__ R warp_sum(R v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float route_exp(float x) { return expf(x); }
__device__ __forceinline__ double route_exp(double x) { return exp(x); }

// Sums over a row that every score of the row needs (softmax).
template <typename R>
struct RowStats {
  R top;  // largest live logit
  R sum;  // sum_live exp(x - top)
};

template <bool SOFTMAX, typename R>
__device__ __forceinline__ R route_score(float x, const RowStats<R>& st) {
  R s;
  if constexpr (SOFTMAX) s = route_exp(R(x) - st.top) / st.sum;
  else if constexpr (sizeof(R) == 4) s = __fdividef(1.0f, 1.0f + expf(-x));  // (two units off at most)
  else s = R(1) / (R(1) + route_exp(-R(x)));
  return x <= kRouteOff ? R(0) : s;
}

// Bound on the error of an fp32 score s of logit x.  sigmoid: expf 2^-22, the
// sum 2^-24, the approximate quotient 2^-22.  softmax: the sum of up to 1024 terms in a
// tree of at most 37 additions, expf and the quotient below 2^-18; the rounded
// difference x - top adds |x - top| 2^-24, and s |x - top| <= max s / e.
template <bool SOFTMAX>
__device__ __forceinline__ float score_error(float s, float s_max_if_softmax, const RowStats<float>& st) {
  if constexpr (SOFTMAX) return 0x1p-18f * fminf(s, s_max_if_softmax / st.sum) + 0x1p-24f / st.sum;
  else return 0x1.4p-21f * s;
}

template <typename R>
struct KeyOf { using type = uint32_t; };
template <>
struct KeyOf<double> { using type = uint64_t; };

constexpr int route_warps(int vpl) { return vpl <= 8 ? 8 : 4; }
// One row of keys per warp; 4 words of padding per 32 spread the groups over
// the banks.
constexpr int route_row(int vpl) { return vpl * 36; }
__device__ __forceinline__ int row_at(int e) { return e + 4 * (e >> 5); }

// Chooses the top_k + 2 best experts of a row into lanes 0 .. top_k + 1 (-1: none
// left).  BY_LOGIT ranks by the logits, else by v in arithmetic R.  Returns
// whether the kept groups are certain (always, in fp64 and by logits).
template <int VPL, bool SOFTMAX, bool BY_LOGIT, typename R>
__device__ __forceinline__ bool choose(const RouteArgs& a, const float (&x)[VPL], const RowStats<R>& st, bool row_nan,
                                       void* row_mem, int lane, int& mine) {
  using K = typename KeyOf<R>::type;
  K key[VPL];
  float bias[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) bias[j] = !BY_LOGIT && a.bias && j * 32 + lane < a.E ? __ldg(a.bias + j * 32 + lane) : 0.0f;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    R v;
    if constexpr (BY_LOGIT) v = SOFTMAX && row_nan ? R(NAN) : R(x[j]);
    else v = route_score<SOFTMAX, R>(x[j], st) + R(bias[j]);
    // (a bias of -inf turns an expert off too; x past the last expert is -inf)
    const bool off = x[j] <= kRouteOff || v == R(-INFINITY);
    const K k = order_key(v);
    key[j] = off ? K(0) : k;
  }
  bool sure = true;
  if (a.groups > 1) {
    K* row = static_cast<K*>(row_mem);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int e = j * 32 + lane;
      if (e < a.E) row[row_at(e)] = key[j];
    }
    __syncwarp();
    // `lpg` lanes scan each group's members for its two largest keys.
    const int size = a.group_size, lpg = 1 << a.group_shift;
    const int g = lane >> a.group_shift, part = lane & (lpg - 1);
    K k1 = 0, k2 = 0;
    if (g < a.groups) {
      for (int i = part; i < size; i += lpg) {
        const K k = row[row_at(g * size + i)];
        k2 = max(k2, min(k1, k));
        k1 = max(k1, k);
      }
    }
    for (int o = 1; o < lpg; o <<= 1) {
      const K p1 = __shfl_xor_sync(0xffffffffu, k1, o), p2 = __shfl_xor_sync(0xffffffffu, k2, o);
      k2 = max(min(k1, p1), max(k2, p2));
      k1 = max(k1, p1);
    }
    K gk = k1;
    float gerr = 0.0f;  // bound on the error of a group's score in fp32
    if constexpr (!BY_LOGIT && sizeof(R) == 4) {
      if (k1 != 0) gerr = score_error<SOFTMAX>(1.0f, 1.0f, st) + 0x1p-23f * fabsf(key_value(k1));
      if (a.group_best == 2 && k2 != 0) gerr = 2.0f * gerr + 0x1p-22f * fabsf(key_value(k2));
    }
    // (an order key is never 0, so a group with a live expert ranks above one without)
    if (a.group_best == 2 && k1 != 0 && k2 != 0) gk = order_key(R(key_value(k1) + key_value(k2)));
    // Rank of each group; ties go to the lower index.
    int rank = 0;
    for (int o = 0; o < a.groups; ++o) {
      const K other = __shfl_sync(0xffffffffu, gk, o * lpg);
      rank += (other > gk || (other == gk && o < g)) ? 1 : 0;
    }
    const bool first = part == 0 && g < a.groups;
    const uint32_t kept_lanes = __ballot_sync(0xffffffffu, first && rank < a.top_groups);
    if constexpr (!BY_LOGIT && sizeof(R) == 4) {
      // Neighbours in rank at the border of the kept groups.
      const uint32_t in = __ballot_sync(0xffffffffu, first && rank == a.top_groups - 1);
      const uint32_t out = __ballot_sync(0xffffffffu, first && rank == a.top_groups);
      if (out) {
        const int li = __ffs(in) - 1, lo = __ffs(out) - 1;
        const K ki = __shfl_sync(0xffffffffu, gk, li), ko = __shfl_sync(0xffffffffu, gk, lo);
        // (any group may lie behind the border with the largest error)
        const float tol = 2.0f * __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(gerr)));
        if (ko != 0 && ko != 0xffffffffu) sure = key_value(ki) - key_value(ko) > tol;
      }
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int e = j * 32 + lane;
      const int ge = (int)(((uint32_t)e * a.group_magic) >> 20);
      if (e < a.E && !((kept_lanes >> (ge * lpg)) & 1u)) key[j] = 0;
    }
  }
  // Every lane keeps its two best candidates and looks through its keys again
  // only when both are taken.
  mine = -1;
  uint32_t taken = 0;
  K b1, b2;
  int j1, j2, have;
  auto look = [&](auto first) {
    b1 = b2 = 0;
    j1 = j2 = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const K k = !decltype(first)::value && ((taken >> j) & 1u) ? K(0) : key[j];
      const bool g1 = k > b1, g2 = k > b2;
      b2 = g1 ? b1 : g2 ? k : b2;
      j2 = g1 ? j1 : g2 ? j : j2;
      b1 = g1 ? k : b1;
      j1 = g1 ? j : j1;
    }
    have = 2;
  };
  look(std::true_type());
  for (int r = 0; r < a.top_k + (BY_LOGIT ? 0 : 2); ++r) {
    const K top = warp_max(b1);
    if (top == 0) break;
    const unsigned e = b1 == top ? (unsigned)(j1 * 32 + lane) : 0xffffffffu;
    const unsigned win = __reduce_min_sync(0xffffffffu, e);
    if (lane == r) mine = (int)win;
    if (e == win) {
      taken |= 1u << j1;
      b1 = b2;
      j1 = j2;
      if (--have == 0) look(std::false_type());
    }
  }
  return sure;
}

template <int VPL, bool SOFTMAX, bool BY_LOGIT, typename L>
__global__ void __launch_bounds__(32 * route_warps(VPL)) k_route(const RouteArgs a) {
  constexpr int kWarps = route_warps(VPL);
  __shared__ uint64_t rows[kWarps][route_row(VPL)];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kWarps + warp;
  if (t >= a.T) return;
  const L* src = static_cast<const L*>(a.logits) + (long long)t * a.ld;
  float x[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = j * 32 + lane;
    x[j] = e < a.E ? load_logit(src + e) : -INFINITY;
  }
  RowStats<float> st{0.0f, 1.0f};
  bool row_nan = false;
  if constexpr (SOFTMAX) {
    uint32_t k = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (!(x[j] <= kRouteOff)) k = max(k, order_key(x[j]));
    k = warp_max(k);
    st.top = k ? key_value(k) : 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (!(x[j] <= kRouteOff)) sum += expf(x[j] - st.top);
    st.sum = warp_sum(sum);
    row_nan = st.sum != st.sum;
    if (k == 0) st.sum = 1.0f;  // no live expert
  }
  int mine;
  bool sure = choose<VPL, SOFTMAX, BY_LOGIT, float>(a, x, st, row_nan, rows[warp], lane, mine);
  float xe = mine >= 0 ? load_logit(src + mine) : -INFINITY;
  float s = route_score<SOFTMAX, float>(xe, st);
  if constexpr (!BY_LOGIT) {
    // Is every neighbour's gap above its error?  (Equal logits with equal
    // biases are equal exactly; NaN ranks by its index.)
    const float be = (a.bias && mine >= 0) ? __ldg(a.bias + mine) : 0.0f;
    const float v = s + be;
    const float err = score_error<SOFTMAX>(s, 1.0f, st) + 0x1p-23f * fabsf(v);
    const int next = __shfl_down_sync(0xffffffffu, mine, 1);
    const float nx = __shfl_down_sync(0xffffffffu, xe, 1), nb = __shfl_down_sync(0xffffffffu, be, 1);
    const float nv = __shfl_down_sync(0xffffffffu, v, 1);
    float ne = __shfl_down_sync(0xffffffffu, err, 1);
    // Behind the last chosen one any expert may follow: one with the largest score
    // (and a bias that nearly cancels it) has the largest error.
    if (lane == a.top_k - 1) ne = fmaxf(ne, score_error<SOFTMAX>(1.0f, 1.0f, st) + 0x1p-22f * fabsf(v));
    const bool equal = nx == xe && nb == be;
    bool decides = lane < a.top_k && next >= 0 && !equal && nv == nv;
    float gap = v - nv;
    // The last chosen one and an exact equal left out: their order is certain, but
    // the expert behind the two may be larger than both.
    const bool more = __shfl_sync(0xffffffffu, mine, a.top_k + 1) >= 0;
    const float v_more = __shfl_sync(0xffffffffu, v, a.top_k + 1);
    if (lane == a.top_k - 1 && next >= 0 && equal) {
      decides = more;
      gap = v - v_more;
    }
    const bool groups_sure = sure;
    sure = sure && !__any_sync(0xffffffffu, decides && !(gap > err + ne) && v == v);
    if (!SOFTMAX && !sure && groups_sure) {
      // Sigmoid scores: only the candidates are computed in fp64, one per lane.
      // They hold the chosen ones if the second expert left out lies certainly
      // below every chosen one.
      const float most = score_error<SOFTMAX>(1.0f, 1.0f, st) +
                         0x1p-22f * fmaxf(fabsf(__shfl_sync(0xffffffffu, v, 0)), fabsf(v_more));
      const float left = __shfl_sync(0xffffffffu, v, a.top_k - 1) - v_more;
      if (!more || left > 2.0f * most) {
        const bool candidate = lane <= a.top_k && mine >= 0;
        const RowStats<double> sd{0.0, 1.0};
        const uint64_t key = candidate ? order_key(route_score<SOFTMAX, double>(xe, sd) + (double)be) : 0ull;
        int rank = 0;
        for (int i = 0; i <= a.top_k; ++i) {
          const uint64_t other = __shfl_sync(0xffffffffu, key, i);
          const int oe = __shfl_sync(0xffffffffu, mine, i);
          rank += other > key || (other == key && oe < mine) ? 1 : 0;
        }
        int* order = reinterpret_cast<int*>(rows[warp]);
        __syncwarp();
        if (lane <= a.top_k) order[lane] = -1;
        __syncwarp();
        if (candidate) order[rank] = mine;
        __syncwarp();
        mine = lane <= a.top_k ? order[lane] : -1;
        __syncwarp();
        xe = mine >= 0 ? load_logit(src + mine) : -INFINITY;
        s = route_score<SOFTMAX, float>(xe, st);
        sure = true;
      }
    }
    if (!sure) {
      RowStats<double> sd{(double)st.top, 1.0};
      if constexpr (SOFTMAX) {
        double sum = 0.0;
#pragma unroll
        for (int j = 0; j < VPL; ++j)
          if (!(x[j] <= kRouteOff)) sum += exp((double)x[j] - sd.top);
        sum = warp_sum(sum);
        if (sum > 0.0) sd.sum = sum;
      }
      choose<VPL, SOFTMAX, false, double>(a, x, sd, row_nan, rows[warp], lane, mine);
      xe = mine >= 0 ? load_logit(src + mine) : -INFINITY;
      s = route_score<SOFTMAX, float>(xe, st);
    }
  }
  // Weights, lane i the i-th chosen expert.
  const bool live = lane < a.top_k && mine >= 0;
  float w = live ? s : 0.0f;
  if (a.renorm) {
    // Shares of the chosen scores, by differences to the largest chosen
    // logit: small scores keep their ratios where they underflow.
    float m = live ? xe : -INFINITY;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (live && !(row_nan && SOFTMAX)) {
      if (SOFTMAX) w = expf(xe - m);
      else if (m <= 0.0f) w = expf(xe - m) * ((1.0f + expf(m)) / (1.0f + expf(xe)));
    }
    const float sum = warp_sum(w);
    w = live ? w / sum : 0.0f;
  }
  if (lane < a.top_k) {
    const long long o = (long long)t * a.top_k + lane;
    a.experts[o] = mine;
    a.weights[o] = a.scale * w;
  }
}

// ----------------------------------------------------------------------------
// gradient of the logits
// ----------------------------------------------------------------------------
struct RouteBwdArgs {
  int T, E, top_k;
  const void* logits;
  long long ld;
  int renorm;
  float scale;
  const int* experts;
  const float* dweights;
  void* dlogits;
  long long ldd;
};

__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// With p_i = s_i / sum of the chosen s (renormalised) and D = sum_j p_j dw_j:
//   softmax:           dx_e = s_e (g_e - sum_j s_j g_j),  g_e = scale * (sum of dw over slots that chose e)
//   softmax, renorm:   dx_i = scale p_i (dw_i - D)        at the chosen, 0 elsewhere
//   sigmoid:           dx_i = scale dw_i s_i (1 - s_i)
//   sigmoid, renorm:   dx_i = scale p_i (1 - s_i) (dw_i - D)
// One warp per token; the slots' values are added to the row in slot order, so
// an expert that occurs in two slots gets both.  Bound by the row in and out.
template <int VPL, bool SOFTMAX, typename L>
__global__ void __launch_bounds__(32 * route_warps(VPL)) k_route_backward(const RouteBwdArgs a) {
  constexpr int kWarps = route_warps(VPL);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kWarps + warp;
  if (t >= a.T) return;
  const L* src = static_cast<const L*>(a.logits) + (long long)t * a.ld;
  int mine = -1;
  float dw = 0.0f;
  if (lane < a.top_k) {
    mine = __ldg(a.experts + (long long)t * a.top_k + lane);
    dw = __ldg(a.dweights + (long long)t * a.top_k + lane);
  }
  const bool dense = SOFTMAX && !a.renorm;
  float x[VPL];
  RowStats<float> st{0.0f, 1.0f};
  if (dense) {
    uint32_t k = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int e = j * 32 + lane;
      x[j] = e < a.E ? load_logit(src + e) : -INFINITY;
      if (!(x[j] <= kRouteOff)) k = max(k, order_key(x[j]));
    }
    k = warp_max(k);
    st.top = k ? key_value(k) : 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      x[j] = x[j] <= kRouteOff ? 0.0f : expf(x[j] - st.top);
      sum += x[j];
    }
    sum = warp_sum(sum);
    st.sum = k ? sum : 1.0f;
  }
  const bool named = mine >= 0 && mine < a.E;  // a slot without an expert has no gradient
  const float xe = named ? load_logit(src + mine) : -INFINITY;
  const bool live = named && !(xe <= kRouteOff);
  float val = 0.0f, dot = 0.0f;
  if (a.renorm) {
    float m = live ? xe : -INFINITY;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float p = 0.0f, left = 1.0f;  // share, and 1 - s for sigmoid scores
    if (live) {
      if constexpr (SOFTMAX) {
        p = expf(xe - m);
      } else {
        p = m <= 0.0f ? expf(xe - m) * ((1.0f + expf(m)) / (1.0f + expf(xe))) : 1.0f / (1.0f + expf(-xe));
        left = 1.0f / (1.0f + expf(xe));
      }
    }
    const float sum = warp_sum(p);
    p = live ? p / sum : 0.0f;
    const float mean = warp_sum(live ? p * dw : 0.0f);
    val = live ? a.scale * p * left * (dw - mean) : 0.0f;
  } else if constexpr (SOFTMAX) {
    const float s = live ? expf(xe - st.top) / st.sum : 0.0f;
    val = live ? a.scale * dw : 0.0f;
    dot = warp_sum(live ? s * val : 0.0f);
  } else {
    val = live ? a.scale * dw * (1.0f / (1.0f + expf(-xe))) * (1.0f / (1.0f + expf(xe))) : 0.0f;
  }
  float g[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) g[j] = 0.0f;
  for (int i = 0; i < a.top_k; ++i) {
    const int e = __shfl_sync(0xffffffffu, live ? mine : -1, i);
    const float v = __shfl_sync(0xffffffffu, val, i);
    if (e >= 0 && (e & 31) == lane) {
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (j == (e >> 5)) g[j] += v;
    }
  }
  L* dst = static_cast<L*>(a.dlogits) + (long long)t * a.ldd;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = j * 32 + lane;
    if (e < a.E) store_logit(dst + e, dense ? (x[j] / st.sum) * (g[j] - dot) : g[j]);
  }
}

template <int VPL, typename L>
void launch_route(const RouteArgs& a, bool softmax, bool by_logit, cudaStream_t stream) {
  const int warps = route_warps(VPL);
  const dim3 grid((unsigned)((a.T + warps - 1) / warps)), block(32 * warps);
  if (softmax) {
    if (by_logit) k_route<VPL, true, true, L><<<grid, block, 0, stream>>>(a);
    else k_route<VPL, true, false, L><<<grid, block, 0, stream>>>(a);
  } else {
    if (by_logit) k_route<VPL, false, true, L><<<grid, block, 0, stream>>>(a);
    else k_route<VPL, false, false, L><<<grid, block, 0, stream>>>(a);
  }
}

template <int VPL, typename L>
void launch_route_backward(const RouteBwdArgs& a, bool softmax, cudaStream_t stream) {
  const int warps = route_warps(VPL);
  const dim3 grid((unsigned)((a.T + warps - 1) / warps)), block(32 * warps);
  if (softmax) k_route_backward<VPL, true, L><<<grid, block, 0, stream>>>(a);
  else k_route_backward<VPL, false, L><<<grid, block, 0, stream>>>(a);
}

// Calls f with the number of logits a lane holds as a compile-time constant.
template <typename F>
void by_width(int E, F f) {
  if (E <= 32) f(std::integral_constant<int, 1>());
  else if (E <= 64) f(std::integral_constant<int, 2>());
  else if (E <= 128) f(std::integral_constant<int, 4>());
  else if (E <= 256) f(std::integral_constant<int, 8>());
  else if (E <= 512) f(std::integral_constant<int, 16>());
  else f(std::integral_constant<int, 32>());
}

int check_route_sizes(const char* what, int T, int E, int top_k, long ld, int type, int score, float scale) {
  if (T < 0 || E < 1 || top_k < 1 || top_k > E)
    return reject(ST_INVALID_ARG, "%s: sizes out of range (T=%d E=%d top_k=%d)", what, T, E, top_k);
  if (E > kRouteMaxExperts || top_k > kRouteMaxTopK)
    return reject(ST_UNSUPPORTED, "%s: E=%d, top_k=%d: this build supports E <= %d, top_k <= %d", what, E, top_k,
                  kRouteMaxExperts, kRouteMaxTopK);
  // (a block of tokens past the last one fits 32 bits)
  if (T > 0x7fffffff - 1024) return reject(ST_UNSUPPORTED, "%s: T=%d: too many tokens", what, T);
  if (ld < E) return reject(ST_INVALID_ARG, "%s: leading dimension %ld < E", what, ld);
  if (type != WST_F32 && type != WST_BF16) return reject(ST_INVALID_ARG, "%s: unknown type %d", what, type);
  if (score != WST_SCORE_SOFTMAX && score != WST_SCORE_SIGMOID)
    return reject(ST_INVALID_ARG, "%s: unknown score %d", what, score);
  if (!(scale >= -3.0e38f && scale <= 3.0e38f)) return reject(ST_INVALID_ARG, "%s: scale must be finite", what);
  return ST_OK;
}

}  // namespace
}  // namespace wst

using namespace wst;

#define WST_TRY(expr)                  \
  do {                                 \
    int st__ = (expr);                 \
    if (st__) return (wst_status)st__; \
  } while (0)

extern "C" {

wst_status wst_moe_route(int T, int E, int top_k, const void* logits, long ld, wst_dtype logits_type, wst_score score,
                         const float* bias, int groups, int top_groups, int group_best, int renorm, float scale,
                         int* experts, float* weights, void* stream) {
  set_error("%s", "");
  WST_TRY(check_route_sizes("route", T, E, top_k, ld, logits_type, score, scale));
  if (groups < 1 || E % groups || top_groups < 1 || top_groups > groups || group_best < 1 || group_best > 2)
    return (wst_status)reject(ST_INVALID_ARG, "route: groups out of range (E=%d groups=%d top_groups=%d group_best=%d)",
                              E, groups, top_groups, group_best);
  if (groups > kRouteMaxGroups)
    return (wst_status)reject(ST_UNSUPPORTED, "route: groups=%d: this build supports up to %d", groups, kRouteMaxGroups);
  if ((long long)top_groups * (E / groups) < top_k)
    return (wst_status)reject(ST_INVALID_ARG, "route: %d groups of %d experts hold fewer than top_k=%d", top_groups,
                              E / groups, top_k);
  if ((long long)T * top_k > 0x7fffffffLL - (1 << 20)) return (wst_status)reject(ST_INVALID_ARG, "route: too many pairs");
  if (T && (!logits || !experts || !weights)) return (wst_status)reject(ST_INVALID_ARG, "route: NULL array");
  if (!aligned_to(logits, logits_type == WST_F32 ? 4 : 2) || !aligned_to(bias, 4) || !aligned_to(experts, 4) ||
      !aligned_to(weights, 4))
    return (wst_status)reject(ST_ALIGNMENT, "route: arrays must be aligned to their elements");
  if (T == 0) return WST_OK;
  WST_TRY(check_operand(logits, "logits"));
  WST_TRY(check_operand(experts, "experts"));
  WST_TRY(check_operand(weights, "weights"));
  if (bias) WST_TRY(check_operand(bias, "bias"));
  DeviceInfo dev;
  WST_TRY(current_device_info(&dev));
  RouteArgs a{};
  a.T = T;
  a.E = E;
  a.top_k = top_k;
  a.logits = logits;
  a.ld = ld;
  a.bias = bias;
  // all groups kept: no group is left out
  a.groups = top_groups == groups ? 1 : groups;
  a.top_groups = a.groups == 1 ? 1 : top_groups;
  a.group_best = group_best;
  const int size = E / a.groups;
  a.group_size = size;
  while ((2 << a.group_shift) * a.groups <= 32) ++a.group_shift;
  a.group_magic = (uint32_t)(((1 << 20) + size - 1) / size);
  a.renorm = renorm != 0;
  a.scale = scale;
  a.experts = experts;
  a.weights = weights;
  const bool by_logit = !bias && (a.groups == 1 || group_best == 1);
  const bool softmax = score == WST_SCORE_SOFTMAX;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  by_width(E, [&](auto vpl) {
    if (logits_type == WST_F32) launch_route<decltype(vpl)::value, float>(a, softmax, by_logit, s);
    else launch_route<decltype(vpl)::value, __nv_bfloat16>(a, softmax, by_logit, s);
  });
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? WST_OK : (wst_status)cuda_fail(e, "launch k_route");
}

wst_status wst_moe_route_backward(int T, int E, int top_k, const void* logits, long ld, wst_dtype logits_type,
                                  wst_score score, int renorm, float scale, const int* experts, const float* dweights,
                                  void* dlogits, long ldd, void* stream) {
  set_error("%s", "");
  WST_TRY(check_route_sizes("route backward", T, E, top_k, ld < ldd ? ld : ldd, logits_type, score, scale));
  if (T && (!logits || !experts || !dweights || !dlogits))
    return (wst_status)reject(ST_INVALID_ARG, "route backward: NULL array");
  const size_t es = logits_type == WST_F32 ? 4 : 2;
  if (!aligned_to(logits, es) || !aligned_to(dlogits, es) || !aligned_to(experts, 4) || !aligned_to(dweights, 4))
    return (wst_status)reject(ST_ALIGNMENT, "route backward: arrays must be aligned to their elements");
  if (T == 0) return WST_OK;
  WST_TRY(check_operand(logits, "logits"));
  WST_TRY(check_operand(experts, "experts"));
  WST_TRY(check_operand(dweights, "dweights"));
  WST_TRY(check_operand(dlogits, "dlogits"));
  DeviceInfo dev;
  WST_TRY(current_device_info(&dev));
  RouteBwdArgs a{T, E, top_k, logits, ld, renorm != 0, scale, experts, dweights, dlogits, ldd};
  const bool softmax = score == WST_SCORE_SOFTMAX;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  by_width(E, [&](auto vpl) {
    if (logits_type == WST_F32) launch_route_backward<decltype(vpl)::value, float>(a, softmax, s);
    else launch_route_backward<decltype(vpl)::value, __nv_bfloat16>(a, softmax, s);
  });
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? WST_OK : (wst_status)cuda_fail(e, "launch k_route_backward");
}

}  // extern "C"
