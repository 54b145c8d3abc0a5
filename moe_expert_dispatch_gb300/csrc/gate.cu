// gate.cu - moe_route_gate and its backward: the top-k gate with softmax or
// sigmoid scores, a balance bias, groups and renormalised weights.
#include <climits>

#include "common.cuh"
#include "internal.h"

namespace moe {

int* device_error_word();

namespace {

constexpr int kMaxGroups = 32;
constexpr int kMaxCluster = 8;
constexpr float kFloatMax = 3.402823466e38f;
constexpr unsigned kAll = 0xffffffffu;

struct GateParams {
  const void* logits;
  const float* bias;
  int64_t T;
  int E, k, score, n_group, topk_group, group_topk, renorm;
  float scale;
  int vec;                   // rows start on 16 bytes and E is a multiple of a vector
};

template <typename L>
__device__ __forceinline__ float load_logit(const L* p);
template <>
__device__ __forceinline__ float load_logit<float>(const float* p) {
  return __ldg(p);
}
template <>
__device__ __forceinline__ float load_logit<__nv_bfloat16>(const __nv_bfloat16* p) {
  return __bfloat162float(*p);
}

// NaN counts as -inf, +inf as the largest float.
// (fmaxf drops a NaN)
__device__ __forceinline__ float clean(float l) { return fminf(fmaxf(l, -INFINITY), kFloatMax); }

// W consecutive lanes share a token: sums, maxima over them.
template <int W, typename V>
__device__ __forceinline__ V seg_sum(V v) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
template <int W>
__device__ __forceinline__ float seg_max(float v) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <int W>
__device__ __forceinline__ unsigned seg_max_key(unsigned v) {
  if (W == 32) return __reduce_max_sync(kAll, v);
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

// Unsigned keys in the order of the floats (-0.0 below +0.0), and back. Below
// the lowest finite one's there is room for what is masked, and 0 for nothing.
constexpr unsigned kLeastKey = 0x00800000u;
__device__ __forceinline__ unsigned key_of(float v) {
  const int b = __float_as_int(v);
  return static_cast<unsigned>(b) ^ (static_cast<unsigned>(b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float float_of(unsigned k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// 1 / (1 + exp(-l)) from the hardware's 2^x and reciprocal (for the choice:
// off by 2^-21.8 at most, see gate_kernel) and from expf and a division (for
// the weights: a few units in the last place).
__device__ __forceinline__ float fast_exp(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
}
__device__ __forceinline__ float fast_sigmoid(float l) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + fast_exp(-l)));
  return r;
}
__device__ __forceinline__ float sigmoid(float l) { return __fdividef(1.0f, 1.0f + expf(-l)); }

// Whether x, that ranks before y, is larger by more than both may be off.
__device__ __forceinline__ bool apart(float x, float y, float abs_off, float rel_off) {
  return y == -INFINITY ? x != -INFINITY : x - y > abs_off + (fabsf(x) + fabsf(y)) * rel_off;
}

// Half of a group's score, which stays in float's range, from the group's best
// two values (the second -inf: one counts), and half of what these measure: a
// sum of opposite signs is as far off as they are, not as it is itself.
struct GroupScore {
  float half, size;
};
__device__ __forceinline__ GroupScore group_score(float best, float next) {
  GroupScore r = {0.5f * best, best == -INFINITY ? 0.0f : 0.5f * fabsf(best)};
  if (next != -INFINITY) {
    r.half = fmaf(0.5f, next, r.half);
    r.size = fmaf(0.5f, fabsf(next), r.size);
  }
  return r;
}
// How far half of a score may be off: both values by off and 2^-24 of
// themselves, their sum by 2^-24 of it, and what compares it by as much again.
__device__ __forceinline__ float group_off(float size, float off) {
  return fmaf(size, 0x1p-22f, off);
}

// Batcher's odd-even merge sort, descending, over registers: a[kLo .. kLo + kN).
template <int kLo, int kN, int kStep, int N>
__device__ __forceinline__ void merge_desc(unsigned (&a)[N]) {
  if constexpr (2 * kStep < kN) {
    merge_desc<kLo, kN, 2 * kStep>(a);
    merge_desc<kLo + kStep, kN, 2 * kStep>(a);
#pragma unroll
    for (int i = kLo + kStep; i + kStep < kLo + kN; i += 2 * kStep) {
      const unsigned x = a[i], y = a[i + kStep];
      a[i] = max(x, y);
      a[i + kStep] = min(x, y);
    }
  } else {
    const unsigned x = a[kLo], y = a[kLo + kStep];
    a[kLo] = max(x, y);
    a[kLo + kStep] = min(x, y);
  }
}
template <int kLo, int kN, int N>
__device__ __forceinline__ void sort_desc(unsigned (&a)[N]) {
  if constexpr (kN > 1) {
    sort_desc<kLo, kN / 2>(a);
    sort_desc<kLo + kN / 2, kN / 2>(a);
    merge_desc<kLo, kN, 1>(a);
  }
}

// ------------------------------------------------------------------ one token in double

// One chosen expert: its key in the order, whose low bits count the lane's
// experts down, and its lane's first expert.
struct Pick {
  unsigned key;
  int e;
};
template <int C>
__device__ __forceinline__ int expert_of(const Pick& q) {
  return q.e + static_cast<int>(C - 1u - (q.key & (C - 1u)));
}

// Signed keys in the order of the doubles (-0.0 entered as +0.0).
__device__ __forceinline__ long long order_of(double v) {
  const long long b = __double_as_longlong(v + 0.0);
  return b ^ static_cast<long long>(static_cast<unsigned long long>(b >> 63) >> 1);
}
constexpr long long kLowest = LLONG_MIN;

__device__ __forceinline__ void warp_argmax(long long& v, int& e) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const long long ov = __shfl_xor_sync(kAll, v, o);
    const int oe = __shfl_xor_sync(kAll, e, o);
    if (ov > v || (ov == v && oe < e)) {
      v = ov;
      e = oe;
    }
  }
}

// The choice of one token by a whole warp with every value in double (v: E
// values of shared memory): for the few tokens that neither reorder nor
// groups_in_double can settle. Some 20 us, most of it the exponentials: double
// precision runs at 1/64 of float's rate here.
template <typename L>
__device__ __noinline__ void choose_in_double(const GateParams& p, const L* row, double* v,
                                              Pick* pick) {
  const int lane = lane_id();
  const int size = p.E / p.n_group;
  const bool soft = p.score == MOE_SCORE_SOFTMAX;
  const bool scored = p.bias != nullptr || p.n_group > 1;      // else the logits' own order
  // one exponential for all experts where their logits are the same (of a router
  // whose weights are still zero, say)
  float m = -INFINITY, least = INFINITY;
  int open = 0;
  for (int e = lane; e < p.E; e += 32) {
    const float l = clean(load_logit(row + e));
    m = fmaxf(m, l);
    if (l == -INFINITY) continue;
    least = fminf(least, l);
    ++open;
  }
  m = seg_max<32>(m);
  const bool level = -seg_max<32>(-least) >= m;
  double inv = 1.0, top = 0.0;
  if (soft && scored) {
    top = m == -INFINITY ? 0.0 : static_cast<double>(m);
    double sum = open;
    if (!level) {
      sum = 0.0;
#pragma unroll 4
      for (int e = lane; e < p.E; e += 32) sum += exp(clean(load_logit(row + e)) - top);
    }
    sum = seg_sum<32>(sum);
    inv = sum > 0.0 ? 1.0 / sum : 0.0;
  }
  auto score = [&](float l) {
    const double ex = exp(soft ? l - top : -static_cast<double>(l));
    return soft ? ex * inv : 1.0 / (1.0 + ex);
  };
  const double same = scored && level ? score(m) : 0.0;
  __syncwarp();
#pragma unroll 4
  for (int e = lane; e < p.E; e += 32) {
    const float l = clean(load_logit(row + e));
    const float b = p.bias ? clean(__ldg(p.bias + e)) : 0.0f;
    v[e] = l == -INFINITY || b == -INFINITY ? -INFINITY : (scored && !level ? score(l) : same) + b;
  }
  __syncwarp();
  unsigned kept = kAll;
  if (p.n_group > 1) {
    double g = -INFINITY;
    if (lane < p.n_group) {
      double a = -INFINITY, b = -INFINITY;
#pragma unroll 4
      for (int i = 0; i < size; ++i) {
        const double x = v[lane * size + i];
        b = order_of(x) > order_of(a) ? a : order_of(x) > order_of(b) ? x : b;
        a = order_of(x) > order_of(a) ? x : a;
      }
      g = a;
      if (p.group_topk == 2 && b != -INFINITY) g += b;
    }
    kept = 0u;
    for (int j = 0; j < p.topk_group; ++j) {
      const bool open = lane < p.n_group && !((kept >> lane) & 1u);
      long long bv = open ? order_of(g) : kLowest;
      int be = open ? lane : INT_MAX;
      warp_argmax(bv, be);
      kept |= 1u << be;                             // topk_group <= n_group: one is open
    }
  }
  __syncwarp();
  // the values' order in place of the values
  long long* o = reinterpret_cast<long long*>(v);
  for (int e = lane; e < p.E; e += 32) {
    const double x = v[e] == -INFINITY || p.bias ? v[e]
                                                 : static_cast<double>(clean(load_logit(row + e)));
    o[e] = (kept >> (e / size)) & 1u ? order_of(x) : kLowest;
  }
  __syncwarp();
  for (int j = 0; j < p.k; ++j) {
    long long bv = kLowest;
    int be = INT_MAX;
#pragma unroll 4
    for (int e = lane; e < p.E; e += 32)
      if (o[e] > bv) {
        bv = o[e];
        be = e;
      }
    warp_argmax(bv, be);                            // k experts at least are kept
    if ((be & 31) == lane) o[be] = kLowest;
    if (lane == 0) pick[j] = Pick{kAll, be};         // low bits all set: nothing to add
    __syncwarp();
  }
}

// The groups that a token keeps (a bit each), by a whole warp, where sigmoid
// scores leave two groups at the border too close for float: only the groups
// there, and of them only the experts that may be among their best, are
// computed in double, one by each lane. 0 with more of them than lanes.
// row_v: 2 E floats of shared memory; off: what a score may be off.
template <typename L>
__device__ __noinline__ unsigned groups_in_double(const GateParams& p, const L* row, float* row_v,
                                                  float off) {
  const int lane = lane_id(), size = p.E / p.n_group;
  int* list = reinterpret_cast<int*>(row_v + p.E);
  __syncwarp();
  for (int e = lane; e < p.E; e += 32) {
    const float l = clean(load_logit(row + e));
    const float b = p.bias ? clean(__ldg(p.bias + e)) : 0.0f;
    row_v[e] = l == -INFINITY || b == -INFINITY ? -INFINITY : fast_sigmoid(l) + b;
  }
  __syncwarp();
  float a = -INFINITY, c = -INFINITY;
  if (lane < p.n_group)
    for (int i = 0, at = lane % size; i < size; ++i, at = at + 1 == size ? 0 : at + 1) {
      const float x = row_v[lane * size + at];
      c = fmaxf(c, fminf(a, x));
      a = fmaxf(a, x);
    }
  const bool two = p.group_topk == 2 && c != -INFINITY;
  const GroupScore mine_of = group_score(a, two ? c : -INFINITY);
  const float g = mine_of.half, may_be = group_off(mine_of.size, off);
  int rank = 0;
  for (int j = 0; j < p.n_group; ++j) {
    const float o = __shfl_sync(kAll, g, j);
    rank += o > g || (o == g && j < lane);
  }
  const bool in = lane < p.n_group && rank < p.topk_group;
  // certain: above whatever those outside may be, or below whatever those inside may be
  const float low = -seg_max<32>(in ? may_be - g : -INFINITY);
  const float high = seg_max<32>(in || lane >= p.n_group ? -INFINITY : g + may_be);
  const bool open = lane < p.n_group && !(in ? g - may_be > high : g + may_be < low);
  const unsigned opens = __ballot_sync(kAll, open);
  unsigned kept = __ballot_sync(kAll, in && !open);
  const float least = two ? c : a;                 // what a group's best may be level with
  int n = 0;
  for (int e1 = 0; e1 < p.E; e1 += 32) {
    const int e = e1 + lane;
    const int of = e < p.E ? e / size : 0;
    const float bar = __shfl_sync(kAll, least, of);
    const bool may = e < p.E && ((opens >> of) & 1u) && row_v[e] != -INFINITY &&
                     !apart(bar, row_v[e], 2.0f * off, 0x1p-22f);
    const unsigned m = __ballot_sync(kAll, may);
    const int at = n + __popc(m & ((1u << lane) - 1u));
    if (may && at < 32) list[at] = e;
    n += __popc(m);
  }
  __syncwarp();
  if (n > 32) return 0u;
  int mine = -1;
  double x = 0.0;
  if (lane < n) {
    const int e = list[lane];
    mine = e / size;
    x = 1.0 / (1.0 + exp(-static_cast<double>(clean(load_logit(row + e))))) +
        (p.bias ? clean(__ldg(p.bias + e)) : 0.0f);
  }
  double best = -INFINITY, next = -INFINITY;
  for (int j = 0; j < n; ++j) {
    const double o = __shfl_sync(kAll, x, j);
    const int of = __shfl_sync(kAll, mine, j);
    if (of != lane) continue;
    next = o > best ? best : o > next ? o : next;
    best = o > best ? o : best;
  }
  if (p.group_topk == 2 && next != -INFINITY) best += next;
  for (int j = __popc(kept); j < p.topk_group; ++j) {
    const bool free = open && !((kept >> lane) & 1u);
    long long bv = free ? order_of(best) : kLowest;
    int be = free ? lane : INT_MAX;
    warp_argmax(bv, be);
    kept |= 1u << be;                              // the open groups are enough
  }
  __syncwarp();
  return kept;
}

// The first k of n <= 32 candidates in their right order, by a whole warp.
// Where neighbours that are close are all the same pair of logit and bias,
// only their indices tell them apart; else every value is computed in double,
// one by each lane. False where that would need the softmax's sum.
template <typename L, int C>
__device__ __noinline__ bool reorder(const GateParams& p, const L* row, Pick* pick, int n,
                                     float abs_off) {
  const int lane = lane_id();
  const bool soft = p.score == MOE_SCORE_SOFTMAX;
  unsigned key = 0u;
  int e = INT_MAX;
  float l = -INFINITY, b = 0.0f;
  if (lane < n && pick[lane].key != 0u) {
    key = pick[lane].key & ~(C - 1u);
    e = expert_of<C>(pick[lane]);
    l = clean(load_logit(row + e));
    if (p.bias) b = clean(__ldg(p.bias + e));
  }
  const unsigned next = __shfl_down_sync(kAll, key, 1);
  const float nl = __shfl_down_sync(kAll, l, 1), nb = __shfl_down_sync(kAll, b, 1);
  const bool differ = lane + 1 < n && next >= kLeastKey && !(l == nl && b == nb) &&
                      !apart(float_of(key), float_of(next), abs_off, C * 0x1.2p-23f);
  const bool compute = __any_sync(kAll, differ);
  if (compute && soft && p.bias) return false;
  long long v = key;                                // equal for the same pair
  if (compute && key != 0u) {
    double x = l;
    if (p.bias) x = 1.0 / (1.0 + exp(-static_cast<double>(l))) + b;
    v = order_of(l == -INFINITY || b == -INFINITY ? -INFINITY : x);
  } else if (compute) {
    v = kLowest;
  }
  int rank = 0;
  for (int j = 0; j < n; ++j) {
    const long long ov = __shfl_sync(kAll, v, j);
    const int oe = __shfl_sync(kAll, e, j);
    rank += ov > v || (ov == v && oe < e);
  }
  __syncwarp();
  if (rank < p.k && lane < n) pick[rank] = Pick{kAll, e};
  __syncwarp();
  return true;
}

// ------------------------------------------------------------------ weights of the chosen

__device__ __noinline__ double sigmoid_in_double(float l) {
  return l == -INFINITY ? 0.0 : 1.0 / (1.0 + exp(-static_cast<double>(l)));
}
__device__ __noinline__ float share_in_double(float l, double total) {
  return total > 0.0 ? static_cast<float>(sigmoid_in_double(l) / total) : 0.0f;
}

// u_j of the slots j = sub + W i of a token, i < S: its weight before the
// scale. l: the logit, -inf for a masked slot; top, inv: of the softmax that
// is not renormalised.
template <int W, int S>
__device__ __forceinline__ void slot_weights(const GateParams& p, const float (&l)[S], float top,
                                             float inv, float (&u)[S]) {
  if (!p.renorm) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      u[i] = 0.0f;
      if (W * i >= p.k) continue;                   // the same for every lane
      u[i] = l[i] == -INFINITY               ? 0.0f
             : p.score == MOE_SCORE_SOFTMAX  ? expf(l[i] - top) * inv
                                             : sigmoid(l[i]);
    }
    return;
  }
  float sum = 0.0f;
  bool low = false;
  if (p.score == MOE_SCORE_SOFTMAX) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < S; ++i) m = fmaxf(m, l[i]);
    m = seg_max<W>(m);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      u[i] = 0.0f;
      if (W * i >= p.k) continue;
      u[i] = l[i] == -INFINITY ? 0.0f : expf(l[i] - m);
      sum += u[i];
    }
    sum = seg_sum<W>(sum);
  } else {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      u[i] = 0.0f;
      if (W * i >= p.k) continue;
      u[i] = l[i] == -INFINITY ? 0.0f : sigmoid(l[i]);
      sum += u[i];
    }
    sum = seg_sum<W>(sum);
    // a token whose scores lie near the end of float's range (masked slots alone
    // do not): their ratios in double, and no other token's of the warp
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < S; ++i) m = fmaxf(m, l[i]);
    m = __any_sync(kAll, sum < 1e-30f) ? seg_max<W>(m) : 0.0f;
    low = sum < 1e-30f && m > -INFINITY;
    if (__any_sync(kAll, low)) {
      double total = 0.0;
#pragma unroll
      for (int i = 0; i < S; ++i) total += low ? sigmoid_in_double(l[i]) : 0.0;
      total = seg_sum<W>(total);
#pragma unroll
      for (int i = 0; i < S; ++i)
        if (low) u[i] = share_in_double(l[i], total);
    }
  }
#pragma unroll
  for (int i = 0; i < S; ++i)
    if (W * i < p.k && !low) u[i] = sum > 0.0f ? __fdividef(u[i], sum) : 0.0f;
}

// The softmax's largest logit (0 for a row of -inf) and the reciprocal of
// its sum, over the C logits of each of a token's W lanes.
template <int W, int C>
__device__ __forceinline__ void softmax_of(const float (&l)[C], float* top, float* inv) {
  float m = l[0];
#pragma unroll
  for (int i = 1; i < C; ++i) m = fmaxf(m, l[i]);
  m = seg_max<W>(m);
  *top = m == -INFINITY ? 0.0f : m;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < C; ++i) sum += fast_exp(l[i] - *top);
  sum = seg_sum<W>(sum);
  *inv = sum > 0.0f ? 1.0f / sum : 0.0f;
}

// C consecutive values of a row from expert e0 on; `past` beyond E.
template <int C, typename L>
__device__ __forceinline__ void load_row(const L* row, int e0, int E, int vec, float past,
                                         float (&l)[C]) {
  if (vec && e0 + C <= E) {
    if constexpr (sizeof(L) == 4) {
#pragma unroll
      for (int i = 0; i < C; i += 4) {
        const float4 q = __ldg(reinterpret_cast<const float4*>(row + e0 + i));
        l[i] = q.x;
        l[i + 1] = q.y;
        l[i + 2] = q.z;
        l[i + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < C; i += 8) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(row + e0 + i));
        const unsigned w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          l[i + 2 * h] = __uint_as_float(w[h] << 16);
          l[i + 2 * h + 1] = __uint_as_float(w[h] & 0xffff0000u);
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) l[i] = e0 + i < E ? load_logit(row + e0 + i) : past;
  }
}

// Shapes of the two kernels: W lanes of C experts each share a token.
template <int W, int C>
struct GateShape {
  static constexpr int kWarps = C > 16 ? 4 : 8;
  static constexpr int kTokens = 32 / W;                       // of a warp
  static constexpr int kMost = W * C < 32 ? W * C : 32;        // the largest k
  static constexpr int kPicks = kMost + 1;                     // and the first one left out
  static constexpr int kSlots = (kMost + W - 1) / W;           // k over W lanes
  static constexpr int kCtas = C > 16 ? 2 : 4;                 // of an SM, by registers
};

// ------------------------------------------------------------------ forward

// W lanes share a token, each with C consecutive experts in registers, so
// that the lowest lane of equal values holds the lowest expert. The values'
// order-preserving keys, with the index inside the lane in their low bits,
// are sorted in every lane; k + 1 rounds of a maximum over the lanes' heads
// then pick the experts, the winner shifting its list up.
//
// Which order is right is decided in double, but rarely computed there: a
// score in float is off by at most 2^-21 of the largest score (ex2.approx
// and rcp.approx within 2^-22 and 2^-23, and s (1 - s) <= 1/4), a choice
// value by 2^-24 of itself more, and its key by the C - 1 units that its low
// bits hold; a group's score as group_off says. Only tokens with two
// neighbours in the order closer than that (some 0.3% with scores of 256
// experts) are looked at again: for ties and most others in the order of the
// candidates alone (reorder). bf16 logits that rank by themselves leave room
// for the whole index in the key, and need no second look at all (kScored
// false: no bias and no groups).
//
// Bound by instruction issue: 65536 tokens x 256 experts (sigmoid, bias, 8
// groups) take 62 us, 690 warp instructions a token with two thirds of the
// issue slots busy, where their 71 MB take 10.5; 50 us without groups, 36 for
// bf16 logits ranked by themselves. 8192 x 128 take 7.6 us and 32 x 256 7.7,
// most of it launch and latency. Four CTAs an SM measured 60 against 67 for
// three.
//
// The bound on a score is absolute, so that scores far below the largest look
// closer than they are, and the time then depends on the values. 65536 x 256,
// k 8, where 50 to 70 us are usual: softmax scores with a bias of zeros and
// logits of a spread of 5 141 us, of 7 274 (reorder needs the row's sum there, and
// leaves them to choose_in_double); sigmoid scores with a bias of zeros and logits
// around -12 103 us, around -15 344, around +12 (scores that are all 1 in
// float) 994; groups without a bias and logits around -12 109. Rows whose logits
// and bias are all the same tie beyond 32 candidates: 342 to 364 us. A bias whose
// values differ keeps saturated scores apart (50 us).
template <typename L, int W, int C, bool kScored>
__global__ void __launch_bounds__((GateShape<W, C>::kWarps * 32), (GateShape<W, C>::kCtas))
    gate_kernel(const __grid_constant__ GateParams p, int32_t* __restrict__ ids, float* __restrict__ probs,
                int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
                int32_t* __restrict__ scratch, int clustered) {
  using G = GateShape<W, C>;
  extern __shared__ __align__(16) unsigned char smem[];
  double* sh_v = reinterpret_cast<double*>(smem);              // [warps][E]
  int* hist = reinterpret_cast<int*>(sh_v + static_cast<size_t>(G::kWarps) * p.E);   // [E]
  __shared__ __align__(16) float sh_bias[kScored ? W * C : 4];
  __shared__ Pick sh_pick[G::kWarps][G::kTokens][G::kPicks];
  __shared__ float sh_group[kScored ? G::kWarps : 1][G::kTokens][G::kMost];
  const int lane = lane_id(), w = threadIdx.x >> 5;
  const int sub = lane & (W - 1), tok = lane / W, e0 = sub * C;
  const unsigned seg = static_cast<unsigned>((1ull << W) - 1ull) << (lane & ~(W - 1));
  const unsigned before = (1u << lane) - 1u;                   // lower lanes
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) hist[e] = 0;
  if (kScored && p.bias)                                       // out of E: masked
    for (int e = threadIdx.x; e < W * C; e += blockDim.x)
      sh_bias[e] = e < p.E ? clean(__ldg(p.bias + e)) : -INFINITY;
  __syncthreads();

  const bool biased = kScored && p.bias != nullptr, grouped = kScored && p.n_group > 1;
  const bool soft = p.score == MOE_SCORE_SOFTMAX;
  constexpr bool exact = sizeof(L) == 2 && !kScored;           // keys that hold the index whole
  const int size = p.E / p.n_group;
  Pick* pick = sh_pick[w][tok];
  const int64_t step = static_cast<int64_t>(gridDim.x) * G::kWarps * G::kTokens;
  // the trip count is the same for every lane of a warp
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * G::kWarps + w) * G::kTokens; t0 < p.T;
       t0 += step) {
    const int64_t t = min(t0 + tok, p.T - 1);                  // past the end: the last token again
    const L* row = static_cast<const L*>(p.logits) + t * p.E;
    float l[C];
    load_row<C>(row, e0, p.E, p.vec, -INFINITY, l);
    unsigned key[C];
    if (exact) {
#pragma unroll
      for (int i = 0; i < C; ++i)
        key[i] = (key_of(fmaxf(l[i], -INFINITY) + 0.0f) & 0xffff0000u) | (0xffffu - e0 - i);
    }
#pragma unroll
    for (int i = 0; i < C; ++i) l[i] = clean(l[i]);
    float top = 0.0f, inv = 1.0f;
    if (soft && (kScored || !p.renorm)) softmax_of<W, C>(l, &top, &inv);
    float v[C];
    if (kScored) {
      if (soft) {
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] = fast_exp(l[i] - top) * inv;
      } else {
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] = fast_sigmoid(l[i]);
      }
      if (biased) {
#pragma unroll
        for (int i = 0; i < C; i += 4) {
          const float4 b = *reinterpret_cast<const float4*>(sh_bias + e0 + i);
          v[i] += b.x;
          v[i + 1] += b.y;
          v[i + 2] += b.z;
          v[i + 3] += b.w;
        }
      }
    }
    bool masks = false;                                        // in any of the warp's tokens
    if (!exact) {
      float least = l[0];
#pragma unroll
      for (int i = 1; i < C; ++i) least = fminf(least, l[i]);
      if (biased) {
#pragma unroll
        for (int i = 0; i < C; ++i) least = fminf(least, v[i]);
      }
      masks = __any_sync(kAll, least == -INFINITY);
      if (kScored && masks) {
#pragma unroll
        for (int i = 0; i < C; ++i)
          if (l[i] == -INFINITY) v[i] = -INFINITY;
      }
    }
    if (!exact) {
#pragma unroll
      for (int i = 0; i < C; ++i)
        key[i] = (key_of((biased ? v[i] : l[i]) + 0.0f) & ~(C - 1u)) | (C - 1u - i);   // one zero
      if (masks) {
        // what is masked ranks after every float, the lower expert first
#pragma unroll
        for (int i = 0; i < C; ++i)
          if ((biased ? v[i] : l[i]) == -INFINITY) key[i] = C * (W - sub) + (C - 1u - i);
      }
    }
    // how far a score may be off (logits that rank by themselves: only by their key)
    const float off = soft ? inv * 0x1p-19f : 0x1p-21f;
    bool open_set = false;                                     // the k experts are not certain
    // the groups of the warp's tokens that opens names, in double; 0: not settled
    auto settle_groups = [&](unsigned opens) {
      unsigned right = 0u;
      for (int q = 0; q < G::kTokens && !soft; ++q) {
        const unsigned mine = static_cast<unsigned>((1ull << W) - 1ull) << (q * W);
        if (!(opens & mine)) continue;
        const unsigned kept =
            groups_in_double(p, static_cast<const L*>(p.logits) + min(t0 + q, p.T - 1) * p.E,
                             reinterpret_cast<float*>(sh_v + static_cast<size_t>(w) * p.E), off);
        if (tok == q) right = kept;
      }
      return right;
    };
    if (grouped) {
      // a group's score, its rank, and the lanes' experts that it leaves out
      if (p.E == W * C && p.n_group <= W) {
        const int lanes = W / p.n_group;                       // of a group
        float a = -INFINITY, c = -INFINITY;
#pragma unroll
        for (int i = 0; i < C; ++i) {
          c = fmaxf(c, fminf(a, v[i]));
          a = fmaxf(a, v[i]);
        }
        for (int o = 1; o < lanes; o <<= 1) {
          const float oa = __shfl_xor_sync(kAll, a, o), oc = __shfl_xor_sync(kAll, c, o);
          c = fmaxf(fminf(a, oa), fmaxf(c, oc));
          a = fmaxf(a, oa);
        }
        const GroupScore score = group_score(a, p.group_topk == 2 ? c : -INFINITY);
        const float g = score.half;
        // topk_group rounds of the largest; groups of one score go together,
        // and are then too close to be certain (masked ones go by their index)
        unsigned gk = g == -INFINITY ? W - (sub & ~(lanes - 1)) : key_of(g + 0.0f);
        unsigned low = 0u, high = 0u;
        for (int j = 0; j <= p.topk_group; ++j) {
          low = high;
          high = seg_max_key<W>(gk);
          if (j < p.topk_group && gk == high) gk = 0u;
        }
        bool kept = gk == 0u;
        const int of = __popc(__ballot_sync(kAll, kept) & seg);
        const float size_most = __uint_as_float(seg_max_key<W>(__float_as_uint(score.size)));
        open_set = of != p.topk_group * lanes ||
                   (high >= kLeastKey &&
                    !(float_of(low) - float_of(high) > 2.0f * group_off(size_most, off)));
        if (const unsigned opens = __ballot_sync(kAll, open_set)) {
          const unsigned right = settle_groups(opens);
          if (right) {
            kept = (right >> (sub / lanes)) & 1u;
            open_set = false;
          }
        }
        if (!kept) {
#pragma unroll
          for (int i = 0; i < C; ++i) key[i] = 0u;
        }
      } else {
        // groups that lie across the lanes: through shared memory
        float* row_v = reinterpret_cast<float*>(sh_v + static_cast<size_t>(w) * p.E);
        float* score = sh_group[w][tok];
        unsigned kept = 0u;
        float low = INFINITY, high = -INFINITY, size_most = 0.0f;
        for (int q = 0; q < G::kTokens; ++q) {                 // the warp's tokens in turn
          __syncwarp();
          if (tok == q) {
#pragma unroll
            for (int i = 0; i < C; ++i)
              if (e0 + i < p.E) row_v[e0 + i] = v[i];
          }
          __syncwarp();
          unsigned most = 0u;
          if (lane < p.n_group) {
            float a = -INFINITY, c = -INFINITY;
            for (int i = 0, at = lane % size; i < size; ++i, at = at + 1 == size ? 0 : at + 1) {
              const float x = row_v[lane * size + at];         // rotated: other banks
              c = fmaxf(c, fminf(a, x));
              a = fmaxf(a, x);
            }
            const GroupScore r = group_score(a, p.group_topk == 2 ? c : -INFINITY);
            sh_group[w][q][lane] = r.half;
            most = __float_as_uint(r.size);
          }
          most = __reduce_max_sync(kAll, most);
          if (tok == q) size_most = __uint_as_float(most);
        }
        __syncwarp();
        for (int g = sub; g < p.n_group; g += W) {
          int rank = 0;
          const float mine = score[g];
          for (int o = 0; o < p.n_group; ++o)
            rank += score[o] > mine || (score[o] == mine && o < g);
          if (rank < p.topk_group) {
            kept |= 1u << g;
            low = fminf(low, mine);
          } else {
            high = fmaxf(high, mine);
          }
        }
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1) kept |= __shfl_xor_sync(kAll, kept, o);
        low = -seg_max<W>(-low);
        high = seg_max<W>(high);
        open_set = high != -INFINITY && !(low - high > 2.0f * group_off(size_most, off));
        if (const unsigned opens = __ballot_sync(kAll, open_set)) {
          const unsigned right = settle_groups(opens);
          if (right) {
            kept = right;
            open_set = false;
          }
        }
#pragma unroll
        for (int i = 0; i < C; ++i)
          if (e0 + i >= p.E || !((kept >> ((e0 + i) / size)) & 1u)) key[i] = 0u;
        __syncwarp();
      }
    }
    if (p.E != W * C) {
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (e0 + i >= p.E) key[i] = 0u;
    }
    sort_desc<0, C>(key);
    __syncwarp();                                              // the last token's picks are read
    auto pop = [&](int j) {
      const unsigned best = seg_max_key<W>(key[0]);
      bool won = key[0] == best;
      if (!exact) {
        const unsigned same = __ballot_sync(kAll, won);        // every lane votes
        won = won && !(same & seg & before);                   // the lowest of equal lanes
      }
      if (won) {
        pick[j] = Pick{best, e0};
#pragma unroll
        for (int i = 0; i + 1 < C; ++i) key[i] = key[i + 1];
        key[C - 1] = 0u;
      }
    };
    for (int j = 0; j <= p.k; ++j) pop(j);
    __syncwarp();
    if (!exact) {
      // neighbours too close for float: among the k, or at their end
      const float abs_off = biased ? 2.0f * off : 1e-43f;
      auto close = [&](int i, int j) {
        const unsigned ka = pick[i].key & ~(C - 1u), kb = pick[j].key & ~(C - 1u);
        return kb >= kLeastKey && !apart(float_of(ka), float_of(kb), abs_off, C * 0x1.2p-23f);
      };
      bool open_order = false, open_end = false;
      for (int j = sub; j < p.k; j += W)
        if (close(j, j + 1)) (j + 1 < p.k ? open_order : open_end) = true;
      if (__any_sync(kAll, open_order || open_end || open_set)) {
        int n = p.k;
        if (unsigned ends = __ballot_sync(kAll, open_end)) {
          // more candidates, until one is apart from the k-th
          const int most = G::kPicks < 32 ? G::kPicks : 32;
          for (n = p.k + 1; ends && n < most; ++n) {
            pop(n);
            __syncwarp();
            ends = __ballot_sync(kAll, (ends & seg) && close(p.k - 1, n));
          }
          if (ends & seg) open_set = true;
          n = min(n, 32);
        }
        const unsigned sets = __ballot_sync(kAll, open_set);
        const unsigned orders = __ballot_sync(kAll, open_order || open_end);
        for (int q = 0; q < G::kTokens; ++q) {
          const unsigned mine = static_cast<unsigned>((1ull << W) - 1ull) << (q * W);
          if (!((sets | orders) & mine)) continue;
          const L* its = static_cast<const L*>(p.logits) + min(t0 + q, p.T - 1) * p.E;
          if ((sets & mine) || !reorder<L, C>(p, its, sh_pick[w][q], n, abs_off))
            choose_in_double(p, its, sh_v + static_cast<size_t>(w) * p.E, sh_pick[w][q]);
        }
      }
    }
    // weights
    float lj[G::kSlots], u[G::kSlots];
    int ej[G::kSlots];
#pragma unroll
    for (int i = 0; i < G::kSlots; ++i) {
      const int j = sub + W * i;
      lj[i] = -INFINITY;
      if (W * i < p.k && j < p.k) {
        ej[i] = exact ? static_cast<int>(0xffffu - (pick[j].key & 0xffffu)) : expert_of<C>(pick[j]);
        lj[i] = clean(load_logit(row + ej[i]));
        if (biased && sh_bias[ej[i]] == -INFINITY) lj[i] = -INFINITY;
      }
    }
    slot_weights<W>(p, lj, top, inv, u);
#pragma unroll
    for (int i = 0; i < G::kSlots; ++i) {
      const int j = sub + W * i;
      if (W * i < p.k && j < p.k && t0 + tok < p.T) {
        ids[t * p.k + j] = ej[i];
        probs[t * p.k + j] = p.scale * u[i];
        atomicAdd(hist + ej[i], 1);
      }
    }
  }

  // counts and offsets: one cluster adds up its CTAs' histograms; more CTAs
  // than that add theirs to the workspace, and the last one scans
  __syncthreads();
  if (clustered) {
    cluster_sync();
    const int ctas = gridDim.x;
    if (blockIdx.x == 0)
      for (int e = threadIdx.x; e < p.E; e += blockDim.x)
        for (int c = 1; c < ctas; ++c) hist[e] += ld_cluster_s32(smem_u32(hist + e), c);
    cluster_sync();
    if (blockIdx.x != 0) return;
  } else {
    __shared__ int is_last;
    int* total = scratch + 64;
    asm volatile("griddepcontrol.wait;" ::: "memory");         // gate_zero_kernel's zeros
    for (int e = threadIdx.x; e < p.E; e += blockDim.x)
      if (hist[e]) atomicAdd(total + e, hist[e]);
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) is_last = atomicAdd(scratch, 1) == static_cast<int>(gridDim.x) - 1;
    __syncthreads();
    if (!is_last) return;
    __threadfence();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) hist[e] = __ldcg(total + e);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) counts[e] = hist[e];
  if (threadIdx.x < 32) {
    int run = 0;
    for (int e1 = 0; e1 < p.E; e1 += 32) {
      const int e = e1 + lane;
      const int c = e < p.E ? hist[e] : 0;
      int inc = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(kAll, inc, o);
        if (lane >= o) inc += n;
      }
      if (e < p.E) offsets[e] = run + inc - c;
      run += __shfl_sync(kAll, inc, 31);
    }
    if (lane == 0) offsets[p.E] = run;
  }
}

// Zeroes the ticket and the totals while gate_kernel already runs beside it.
__global__ void __launch_bounds__(256) gate_zero_kernel(int32_t* scratch, int n) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int i = threadIdx.x; i < n; i += blockDim.x) scratch[i] = 0;
}

// ------------------------------------------------------------------ backward

// W lanes of C experts share a token, as forward. The slots' gradients go
// through a row of shared memory, zero between tokens, to the lanes that own
// their experts; every lane then writes its C columns. 16384 x 64 (dense
// softmax): 6.0 us, half of it a launch's latency, against 1.4 for its 9.2 MB.
// 65536 x 256: 54 us dense, 43 where only the chosen have a gradient (71 MB
// written and read, 10.5).
template <typename L, int W, int C>
__global__ void __launch_bounds__((GateShape<W, C>::kWarps * 32), (C > 8 ? 2 : 4))
    gate_backward_kernel(const __grid_constant__ GateParams p, const float* __restrict__ dprobs,
                         const int32_t* __restrict__ ids, L* __restrict__ dlogits, int vec_out,
                         int* err) {
  using G = GateShape<W, C>;
  __shared__ float sh_row[G::kWarps][G::kTokens][W * C + 1];   // + 1: tokens on other banks
  const int lane = lane_id(), w = threadIdx.x >> 5;
  const int sub = lane & (W - 1), tok = lane / W, e0 = sub * C;
  float* mine = sh_row[w][tok];
  for (int e = sub; e < W * C; e += W) mine[e] = 0.0f;
  __syncwarp();
  const bool biased = p.bias != nullptr;
  const bool sigm = p.score == MOE_SCORE_SIGMOID;
  const bool dense = !sigm && !p.renorm;
  const int64_t step = static_cast<int64_t>(gridDim.x) * G::kWarps * G::kTokens;
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * G::kWarps + w) * G::kTokens; t0 < p.T;
       t0 += step) {
    const bool live_row = t0 + tok < p.T;
    const int64_t t = min(t0 + tok, p.T - 1);
    const L* row = static_cast<const L*>(p.logits) + t * p.E;
    float l[C];
    float top = 0.0f, inv = 1.0f;
    if (dense) {
      load_row<C>(row, e0, p.E, p.vec, -INFINITY, l);
#pragma unroll
      for (int i = 0; i < C; ++i) l[i] = clean(l[i]);
      softmax_of<W, C>(l, &top, &inv);
    }
    float lj[G::kSlots], dp[G::kSlots], u[G::kSlots];
    int ej[G::kSlots];
#pragma unroll
    for (int i = 0; i < G::kSlots; ++i) {
      const int j = sub + W * i;
      lj[i] = -INFINITY;
      dp[i] = 0.0f;
      ej[i] = -1;
      if (W * i < p.k && j < p.k) {
        ej[i] = __ldg(ids + t * p.k + j);
        if (ej[i] < 0 || ej[i] >= p.E) {
          report_error(err, kErrBadId);
          ej[i] = -1;
        } else {
          dp[i] = __ldg(dprobs + t * p.k + j);
          lj[i] = clean(load_logit(row + ej[i]));
          if (biased && clean(__ldg(p.bias + ej[i])) == -INFINITY) lj[i] = -INFINITY;
        }
      }
    }
    slot_weights<W>(p, lj, top, inv, u);
    float d = 0.0f;
#pragma unroll
    for (int i = 0; i < G::kSlots; ++i)
      if (lj[i] != -INFINITY) d = fmaf(dp[i], u[i], d);
    d = seg_sum<W>(d);
    // an expert in two slots of a token (no gate chooses so) adds up in slot order
    bool twice = false;
#pragma unroll
    for (int i = 0; i < G::kSlots; ++i)
      if (ej[i] >= 0) mine[ej[i]] = static_cast<float>(sub + W * i + 1);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < G::kSlots; ++i)
      if (ej[i] >= 0) twice |= mine[ej[i]] != static_cast<float>(sub + W * i + 1);
    const bool any_twice = __any_sync(kAll, twice);
    __syncwarp();
    float g[G::kSlots];
#pragma unroll
    for (int i = 0; i < G::kSlots; ++i) {
      if (W * i >= p.k) continue;
      const float far = sigm ? 1.0f / (1.0f + expf(lj[i])) : 1.0f;     // 1 - s
      g[i] = lj[i] == -INFINITY ? 0.0f : u[i] * far * (p.renorm ? dp[i] - d : dp[i]);
      if (ej[i] >= 0) mine[ej[i]] = any_twice ? 0.0f : g[i];
    }
    __syncwarp();
    if (any_twice) {
      for (int j = 0; j < p.k; ++j) {
#pragma unroll
        for (int i = 0; i < G::kSlots; ++i)
          if (sub + W * i == j && ej[i] >= 0) mine[ej[i]] += g[i];
        __syncwarp();
      }
    }
    float out[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      out[i] = mine[e0 + i];
      if (dense) out[i] = fmaf(-d * inv, fast_exp(l[i] - top), out[i]);
      out[i] *= p.scale;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < G::kSlots; ++i)
      if (ej[i] >= 0) mine[ej[i]] = 0.0f;
    __syncwarp();
    if (live_row) {
      L* to = dlogits + t * p.E + e0;
      if (vec_out && e0 + C <= p.E) {
        if constexpr (sizeof(L) == 4) {
#pragma unroll
          for (int i = 0; i < C; i += 4)
            *reinterpret_cast<float4*>(to + i) =
                make_float4(out[i], out[i + 1], out[i + 2], out[i + 3]);
        } else {
#pragma unroll
          for (int i = 0; i < C; i += 8)
            *reinterpret_cast<uint4*>(to + i) =
                make_uint4(pack_bf16x2(out[i], out[i + 1]), pack_bf16x2(out[i + 2], out[i + 3]),
                           pack_bf16x2(out[i + 4], out[i + 5]), pack_bf16x2(out[i + 6], out[i + 7]));
        }
      } else {
#pragma unroll
        for (int i = 0; i < C; ++i)
          if (e0 + i < p.E) {
            if constexpr (sizeof(L) == 4)
              to[i] = out[i];
            else
              to[i] = __float2bfloat16_rn(out[i]);
          }
      }
    }
  }
}

moe_status gate_params(GateParams* p, const void* logits, int type, const float* bias, int64_t T,
                       int E, int k, const moe_gate_config* cfg) {
  moe_gate_config c;
  moe_gate_config_init(&c);
  if (cfg) c = *cfg;
  if (T < 0 || E < 1 || E > kMaxExperts || k < 1 || k > E || k > kMaxTopK ||
      T > ((static_cast<int64_t>(1) << 31) - 1) / k)
    return MOE_ERR_INVALID_ARG;
  if (type != MOE_TYPE_F32 && type != MOE_TYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (c.score != MOE_SCORE_SOFTMAX && c.score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (c.n_group < 1 || c.n_group > kMaxGroups || E % c.n_group != 0 || c.topk_group < 1 ||
      c.topk_group > c.n_group || c.topk_group * (E / c.n_group) < k)
    return MOE_ERR_INVALID_ARG;
  if (c.group_topk < 1 || c.group_topk > 2 || !(c.scale - c.scale == 0.0f))
    return MOE_ERR_INVALID_ARG;
  const uintptr_t mask = type == MOE_TYPE_F32 ? 3 : 1;
  if (reinterpret_cast<uintptr_t>(logits) & mask) return MOE_ERR_INVALID_ARG;
  const int vec = (reinterpret_cast<uintptr_t>(logits) & 15) == 0 &&
                  E % (type == MOE_TYPE_F32 ? 4 : 8) == 0;
  *p = GateParams{logits,       bias,         T,             E,       k,  c.score, c.n_group,
                  c.topk_group, c.group_topk, c.renormalise, c.scale, vec};
  return MOE_OK;
}

// Head of the workspace (the ticket, 256 bytes) and one total per expert.
size_t gate_scratch_bytes(int E) { return 256 + static_cast<size_t>(E) * sizeof(int32_t); }

// CTAs that hold all tokens at once.
struct GateCtas {
  int64_t T;
  template <int W, int C>
  int64_t operator()() const {
    const int64_t per = GateShape<W, C>::kWarps * GateShape<W, C>::kTokens;
    return T > 0 ? (T + per - 1) / per : 1;
  }
};

template <typename L, int W, int C>
cudaError_t launch_gate(const GateParams& p, int32_t* ids, float* probs, int32_t* counts,
                        int32_t* offsets, int32_t* scratch, cudaStream_t st) {
  using G = GateShape<W, C>;
  const int64_t want = GateCtas{p.T}.operator()<W, C>();
  const size_t smem = static_cast<size_t>(G::kWarps) * p.E * sizeof(double) + p.E * sizeof(int);
  auto* kernel = p.bias || p.n_group > 1 ? gate_kernel<L, W, C, true> : gate_kernel<L, W, C, false>;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.blockDim = dim3(G::kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (want <= kMaxCluster) {
    cfg.gridDim = dim3(static_cast<unsigned>(want));
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(want);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, ids, probs, counts, offsets, scratch, 1);
  }
  gate_zero_kernel<<<1, 256, 0, st>>>(scratch, static_cast<int>(gate_scratch_bytes(p.E) / 4));
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // beside the zeroing; it waits for it before it counts
  const int64_t cap = static_cast<int64_t>(device_sm_count()) * G::kCtas;
  cfg.gridDim = dim3(static_cast<unsigned>(want < cap ? want : cap));
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, ids, probs, counts, offsets, scratch, 0);
}

template <typename L, int W, int C>
cudaError_t launch_gate_backward(const GateParams& p, const float* dprobs, const int32_t* ids,
                                 void* dlogits, cudaStream_t st) {
  using G = GateShape<W, C>;
  const int64_t per = G::kWarps * G::kTokens;
  const int64_t want = (p.T + per - 1) / per;
  const int64_t cap = static_cast<int64_t>(device_sm_count()) * 8;
  const int vec_out = (reinterpret_cast<uintptr_t>(dlogits) & 15) == 0 &&
                      p.E % (sizeof(L) == 4 ? 4 : 8) == 0;
  gate_backward_kernel<L, W, C>
      <<<static_cast<unsigned>(want < cap ? want : cap), G::kWarps * 32, 0, st>>>(
          p, dprobs, ids, static_cast<L*>(dlogits), vec_out, device_error_word());
  return cudaGetLastError();
}

// Calls f with the lanes per token and the experts per lane that hold E. Most
// instructions are a token's, not an expert's, and a warp issues them once for
// all its tokens: sixteen experts a lane where there are that many to hold
// (65536 x 256: 63 us, with eight 72). Where latency counts eight are the shorter
// way (32 x 256: 7.3 us, with eight 6.0; the gradient 3.7 against 2.9): the shape
// goes by E alone.
template <typename F>
auto with_shape(int E, F&& f) {
  if (E <= 8) return f.template operator()<1, 8>();
  if (E <= 16) return f.template operator()<2, 8>();
  if (E <= 32) return f.template operator()<4, 8>();
  if (E <= 64) return f.template operator()<4, 16>();
  if (E <= 128) return f.template operator()<8, 16>();
  if (E <= 256) return f.template operator()<16, 16>();
  if (E <= 512) return f.template operator()<32, 16>();
  return f.template operator()<32, 32>();
}

template <typename L>
struct GateLauncher {
  const GateParams& p;
  int32_t* ids;
  float* probs;
  int32_t *counts, *offsets, *scratch;
  cudaStream_t st;
  template <int W, int C>
  cudaError_t operator()() const {
    return launch_gate<L, W, C>(p, ids, probs, counts, offsets, scratch, st);
  }
};

template <typename L>
struct GateBackwardLauncher {
  const GateParams& p;
  const float* dprobs;
  const int32_t* ids;
  void* dlogits;
  cudaStream_t st;
  template <int W, int C>
  cudaError_t operator()() const {
    return launch_gate_backward<L, W, C>(p, dprobs, ids, dlogits, st);
  }
};

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

void moe_gate_config_init(moe_gate_config* cfg) {
  if (!cfg) return;
  *cfg = moe_gate_config{MOE_SCORE_SOFTMAX, 1, 1, 1, 1, 1.0f};
}

size_t moe_route_gate_workspace_size(int64_t T, int k, int E) {
  if (T < 0 || k < 1 || E < 1 || T > ((static_cast<int64_t>(1) << 31) - 1) / k) return 0;
  return with_shape(E, GateCtas{T}) <= kMaxCluster ? 0 : gate_scratch_bytes(E);
}

moe_status moe_route_gate(const void* logits, int logits_type, const float* bias, int64_t T, int E,
                          int k, const moe_gate_config* cfg, int32_t* expert_ids, float* probs,
                          int32_t* counts, int32_t* offsets, void* workspace, size_t ws_bytes,
                          void* stream) {
  MOE_ENTRY_RANGE();
  GateParams p;
  const moe_status s = gate_params(&p, logits, logits_type, bias, T, E, k, cfg);
  if (s != MOE_OK) return s;
  if ((T > 0 && (!logits || !expert_ids || !probs)) || !counts || !offsets)
    return MOE_ERR_INVALID_ARG;
  const size_t need = moe_route_gate_workspace_size(T, k, E);
  if (need > 0 && (!workspace || ws_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 15)))
    return MOE_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int32_t* scratch = static_cast<int32_t*>(workspace);
  const cudaError_t e =
      logits_type == MOE_TYPE_F32
          ? with_shape(E, GateLauncher<float>{p, expert_ids, probs, counts, offsets, scratch, st})
          : with_shape(E, GateLauncher<__nv_bfloat16>{p, expert_ids, probs, counts, offsets,
                                                      scratch, st});
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_route_gate_backward(const float* dprobs, const void* logits, int logits_type,
                                   const float* bias, const int32_t* expert_ids, int64_t T, int E,
                                   int k, const moe_gate_config* cfg, void* dlogits, void* stream) {
  MOE_ENTRY_RANGE();
  GateParams p;
  const moe_status s = gate_params(&p, logits, logits_type, bias, T, E, k, cfg);
  if (s != MOE_OK) return s;
  if (T == 0) return MOE_OK;
  if (!dprobs || !logits || !expert_ids || !dlogits) return MOE_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(dlogits) & (logits_type == MOE_TYPE_F32 ? 3 : 1))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      logits_type == MOE_TYPE_F32
          ? with_shape(E, GateBackwardLauncher<float>{p, dprobs, expert_ids, dlogits, st})
          : with_shape(E, GateBackwardLauncher<__nv_bfloat16>{p, dprobs, expert_ids, dlogits, st});
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
