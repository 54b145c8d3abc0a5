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
__device__ __forceinline__ float clean(float l) { return isnan(l) ? -INFINITY : fminf(l, kFloatMax); }

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

// Unsigned keys in the order of the floats (-0.0 entered as +0.0), and back.
__device__ __forceinline__ unsigned key_of(float v) {
  const int b = __float_as_int(v + 0.0f);
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
__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// Whether x, that ranks before y, is larger by more than both may be off.
__device__ __forceinline__ bool apart(float x, float y, float abs_off, float rel_off) {
  return y == -INFINITY ? x != -INFINITY : x - y > abs_off + (fabsf(x) + fabsf(y)) * rel_off;
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

__device__ __forceinline__ double warp_sum(double v) { return seg_sum<32>(v); }

// The larger value first, equal values to the lower index.
__device__ __forceinline__ void warp_argmax(double& v, int& e) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double ov = __shfl_xor_sync(kAll, v, o);
    const int oe = __shfl_xor_sync(kAll, e, o);
    if (ov > v || (ov == v && oe < e)) {
      v = ov;
      e = oe;
    }
  }
}

struct Pick {                // one chosen expert: its key in the order, and its index
  unsigned key;
  int e;
};

// The choice of one token by a whole warp with every value in double (v: E
// doubles of shared memory): for the tokens whose order float leaves open.
template <typename L>
__device__ __noinline__ void choose_in_double(const GateParams& p, const L* row, double* v,
                                              Pick* pick) {
  const int lane = lane_id();
  const int size = p.E / p.n_group;
  double inv = 1.0, top = 0.0;
  if (p.score == MOE_SCORE_SOFTMAX) {
    float m = -INFINITY;
    for (int e = lane; e < p.E; e += 32) m = fmaxf(m, clean(load_logit(row + e)));
    m = seg_max<32>(m);
    top = m == -INFINITY ? 0.0 : static_cast<double>(m);
    double sum = 0.0;
    for (int e = lane; e < p.E; e += 32) sum += exp(clean(load_logit(row + e)) - top);
    sum = warp_sum(sum);
    inv = sum > 0.0 ? 1.0 / sum : 0.0;
  }
  __syncwarp();
  for (int e = lane; e < p.E; e += 32) {
    const float l = clean(load_logit(row + e));
    const float b = p.bias ? clean(__ldg(p.bias + e)) : 0.0f;
    v[e] = l == -INFINITY || b == -INFINITY   ? -INFINITY
           : p.score == MOE_SCORE_SOFTMAX     ? exp(l - top) * inv + b
                                              : 1.0 / (1.0 + exp(-static_cast<double>(l))) + b;
  }
  __syncwarp();
  unsigned kept = kAll;
  if (p.n_group > 1) {
    double g = -INFINITY;
    if (lane < p.n_group) {
      double a = -INFINITY, b = -INFINITY;
      for (int e = lane * size; e < (lane + 1) * size; ++e) {
        const double x = v[e];
        if (x > a) {
          b = a;
          a = x;
        } else if (x > b) {
          b = x;
        }
      }
      g = a;
      if (p.group_topk == 2 && b != -INFINITY) g += b;
    }
    kept = 0u;
    for (int j = 0; j < p.topk_group; ++j) {
      const bool open = lane < p.n_group && !((kept >> lane) & 1u);
      double bv = open ? g : -INFINITY;
      int be = open ? lane : INT_MAX;
      warp_argmax(bv, be);
      kept |= 1u << be;                             // topk_group <= n_group: one is open
    }
  }
  unsigned taken = 0u;                              // bit i: expert lane + 32 i
  for (int j = 0; j < p.k; ++j) {
    double bv = -INFINITY;
    int be = INT_MAX;
    for (int i = 0, e = lane; e < p.E; ++i, e += 32) {
      if (((taken >> i) & 1u) || !((kept >> (e / size)) & 1u)) continue;
      const double x = v[e] == -INFINITY ? -INFINITY
                       : p.bias          ? v[e]
                                         : static_cast<double>(clean(load_logit(row + e)));
      if (x > bv || be == INT_MAX) {
        bv = x;
        be = e;
      }
    }
    warp_argmax(bv, be);
    if ((be & 31) == lane) taken |= 1u << (be >> 5);
    if (lane == 0) pick[j].e = be;
  }
  __syncwarp();
}

// The same k experts in the order of their values in double: where only the
// order among them is open, and a value needs no sum over the others.
template <typename L>
__device__ __noinline__ void reorder_in_double(const GateParams& p, const L* row, Pick* pick) {
  const int lane = lane_id();
  int e = INT_MAX;
  double v = -INFINITY;
  if (lane < p.k) {
    e = pick[lane].e;
    const float l = clean(load_logit(row + e));
    const float b = p.bias ? clean(__ldg(p.bias + e)) : 0.0f;
    if (l != -INFINITY && b != -INFINITY)
      v = p.bias ? 1.0 / (1.0 + exp(-static_cast<double>(l))) + b : static_cast<double>(l);
  }
  int rank = 0;
  for (int j = 0; j < p.k; ++j) {
    const double ov = __shfl_sync(kAll, v, j);
    const int oe = __shfl_sync(kAll, e, j);
    rank += ov > v || (ov == v && oe < e);
  }
  __syncwarp();
  if (lane < p.k) pick[rank].e = e;
  __syncwarp();
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
    for (int i = 0; i < S; ++i)
      u[i] = l[i] == -INFINITY               ? 0.0f
             : p.score == MOE_SCORE_SOFTMAX  ? expf(l[i] - top) * inv
                                             : sigmoid(l[i]);
    return;
  }
  float sum = 0.0f;
  if (p.score == MOE_SCORE_SOFTMAX) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < S; ++i) m = fmaxf(m, l[i]);
    m = seg_max<W>(m);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      u[i] = l[i] == -INFINITY ? 0.0f : expf(l[i] - m);
      sum += u[i];
    }
    sum = seg_sum<W>(sum);
  } else {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      u[i] = l[i] == -INFINITY ? 0.0f : sigmoid(l[i]);
      sum += u[i];
    }
    sum = seg_sum<W>(sum);
    // scores near the end of float's range: their ratios in double
    if (__any_sync(kAll, sum < 1e-30f)) {
      double total = 0.0;
#pragma unroll
      for (int i = 0; i < S; ++i) total += sigmoid_in_double(l[i]);
      total = seg_sum<W>(total);
#pragma unroll
      for (int i = 0; i < S; ++i) u[i] = share_in_double(l[i], total);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < S; ++i) u[i] = sum > 0.0f ? u[i] / sum : 0.0f;
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
  static constexpr int kPicks = (W * C < 32 ? W * C : 32) + 1; // k, and the first one left out
  static constexpr int kSlots = 32 / W < 8 ? 32 / W : 8;       // k <= min(32, W * C) over W lanes
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
// bits hold. Only tokens with two neighbours in the order closer than that
// (some 0.2% with scores of 256 experts) are ordered again in double. bf16
// logits that rank by themselves leave room for the whole index in the key,
// and need no second look at all (kScored false: no bias and no groups).
//
// Bound by instruction issue (some 400 warp instructions for 256 experts).
template <typename L, int W, int C, bool kScored>
__global__ void __launch_bounds__((GateShape<W, C>::kWarps * 32), (C > 8 ? 2 : 4))
    gate_kernel(const __grid_constant__ GateParams p, int32_t* __restrict__ ids, float* __restrict__ probs,
                int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
                int32_t* __restrict__ scratch, int clustered) {
  using G = GateShape<W, C>;
  extern __shared__ __align__(16) unsigned char smem[];
  double* sh_v = reinterpret_cast<double*>(smem);              // [warps][E]
  int* hist = reinterpret_cast<int*>(sh_v + static_cast<size_t>(G::kWarps) * p.E);   // [E]
  __shared__ Pick sh_pick[G::kWarps][G::kTokens][G::kPicks];
  __shared__ float sh_group[G::kWarps][G::kTokens][G::kPicks - 1];
  const int lane = lane_id(), w = threadIdx.x >> 5;
  const int sub = lane & (W - 1), tok = lane / W, e0 = sub * C;
  const unsigned seg = static_cast<unsigned>((1ull << W) - 1ull) << (lane & ~(W - 1));
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) hist[e] = 0;
  __syncthreads();

  const bool biased = kScored && p.bias != nullptr, grouped = kScored && p.n_group > 1;
  const bool soft = p.score == MOE_SCORE_SOFTMAX;
  constexpr bool exact = sizeof(L) == 2 && !kScored;           // keys that hold the index whole
  const int size = p.E / p.n_group;
  float b[C];
  if (biased) {
    load_row<C>(p.bias, e0, p.E, (reinterpret_cast<uintptr_t>(p.bias) & 15) == 0 && p.E % 4 == 0,
                -INFINITY, b);
#pragma unroll
    for (int i = 0; i < C; ++i) b[i] = clean(b[i]);
  }
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
        key[i] = (key_of(isnan(l[i]) ? -INFINITY : l[i]) & 0xffff0000u) | (0xffffu - e0 - i);
    }
#pragma unroll
    for (int i = 0; i < C; ++i) l[i] = clean(l[i]);
    float top = 0.0f, inv = 1.0f;
    if (soft && (kScored || !p.renorm)) softmax_of<W, C>(l, &top, &inv);
    float v[C];
    if (kScored) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        v[i] = soft ? fast_exp(l[i] - top) * inv : fast_sigmoid(l[i]);
        if (biased) v[i] = b[i] == -INFINITY ? -INFINITY : v[i] + b[i];
        if (l[i] == -INFINITY) v[i] = -INFINITY;
      }
    }
    if (!exact) {
#pragma unroll
      for (int i = 0; i < C; ++i)
        key[i] = (key_of(biased ? v[i] : l[i]) & ~(C - 1u)) | (C - 1u - i);
    }
    // how far a score may be off (logits that rank by themselves: only by their key)
    const float off = soft ? inv * 0x1p-19f : 0x1p-21f;
    bool open_set = false;                                     // the k experts are not certain
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
        const float g = p.group_topk == 2 && c != -INFINITY ? a + c : a;
        int rank = 0;
        for (int o = lanes; o < W; o += lanes) {
          const int from = sub ^ o;                            // every other group once
          const float og = __shfl_xor_sync(kAll, g, o);
          rank += og > g || (og == g && from < sub);
        }
        const bool kept = rank < p.topk_group;
        const float low = -seg_max<W>(kept ? -g : -INFINITY);
        const float high = seg_max<W>(kept ? -INFINITY : g);
        open_set = p.topk_group < p.n_group && !apart(low, high, 4.0f * off, 0x1p-22f);
        if (!kept) {
#pragma unroll
          for (int i = 0; i < C; ++i) key[i] = 0u;
        }
      } else {
        // groups that lie across the lanes: through shared memory
        float* row_v = reinterpret_cast<float*>(sh_v + static_cast<size_t>(w) * p.E);
        float* score = sh_group[w][tok];
        unsigned kept = 0u;
        float low = INFINITY, high = -INFINITY;
        for (int q = 0; q < G::kTokens; ++q) {                 // the warp's tokens in turn
          __syncwarp();
          if (tok == q) {
#pragma unroll
            for (int i = 0; i < C; ++i)
              if (e0 + i < p.E) row_v[e0 + i] = v[i];
          }
          __syncwarp();
          if (lane < p.n_group) {
            float a = -INFINITY, c = -INFINITY;
            for (int i = 0, at = lane % size; i < size; ++i, at = at + 1 == size ? 0 : at + 1) {
              const float x = row_v[lane * size + at];         // rotated: other banks
              c = fmaxf(c, fminf(a, x));
              a = fmaxf(a, x);
            }
            sh_group[w][q][lane] = p.group_topk == 2 && c != -INFINITY ? a + c : a;
          }
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
        open_set = p.topk_group < p.n_group && !apart(low, high, 4.0f * off, 0x1p-22f);
#pragma unroll
        for (int i = 0; i < C; ++i)
          if (e0 + i >= p.E || !((kept >> ((e0 + i) / size)) & 1u)) key[i] = 0u;
        __syncwarp();
      }
    }
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (e0 + i >= p.E) key[i] = 0u;
    sort_desc<0, C>(key);
    __syncwarp();                                              // the last token's picks are read
    for (int j = 0; j <= p.k; ++j) {
      const unsigned best = seg_max_key<W>(key[0]);
      const unsigned same = __ballot_sync(kAll, key[0] == best) & seg;
      if (lane == __ffs(same) - 1) {
        pick[j].key = best;
        pick[j].e = exact ? static_cast<int>(0xffffu - (best & 0xffffu))
                          : e0 + static_cast<int>(C - 1u - (best & (C - 1u)));
#pragma unroll
        for (int i = 0; i + 1 < C; ++i) key[i] = key[i + 1];
        key[C - 1] = 0u;
      }
    }
    __syncwarp();
    // neighbours too close for float
    bool open_order = false;
    if (!exact) {
      for (int j = sub; j < p.k; j += W) {
        const unsigned ka = pick[j].key & ~(C - 1u), kb = pick[j + 1].key & ~(C - 1u);
        if (kb == 0u) continue;                                // nothing is left out
        const float x = float_of(ka), y = float_of(kb);
        const bool close = !apart(x, y, biased ? 2.0f * off : 1e-43f, C * 0x1.2p-23f);
        if (close && j + 1 == p.k) open_set = true;
        if (close && j + 1 < p.k) open_order = true;
      }
    }
    const unsigned sets = __ballot_sync(kAll, open_set || (open_order && soft && biased));
    const unsigned orders = __ballot_sync(kAll, open_order);
    if (sets | orders) {
      for (int q = 0; q < G::kTokens; ++q) {
        const unsigned mine = static_cast<unsigned>((1ull << W) - 1ull) << (q * W);
        const L* its = static_cast<const L*>(p.logits) + min(t0 + q, p.T - 1) * p.E;
        if (sets & mine)
          choose_in_double(p, its, sh_v + static_cast<size_t>(w) * p.E, sh_pick[w][q]);
        else if (orders & mine)
          reorder_in_double(p, its, sh_pick[w][q]);
      }
    }
    // weights
    float lj[G::kSlots], u[G::kSlots];
    int ej[G::kSlots];
#pragma unroll
    for (int i = 0; i < G::kSlots; ++i) {
      const int j = sub + W * i;
      lj[i] = -INFINITY;
      if (j < p.k) {
        ej[i] = pick[j].e;
        lj[i] = clean(load_logit(row + ej[i]));
        if (biased && clean(__ldg(p.bias + ej[i])) == -INFINITY) lj[i] = -INFINITY;
      }
    }
    slot_weights<W>(p, lj, top, inv, u);
#pragma unroll
    for (int i = 0; i < G::kSlots; ++i) {
      const int j = sub + W * i;
      if (j < p.k && t0 + tok < p.T) {
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

// ------------------------------------------------------------------ backward

// W lanes of C experts share a token, as forward. The slots' gradients go
// through a row of shared memory, zero between tokens, to the lanes that own
// their experts; every lane then writes its C columns.
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
      if (j < p.k) {
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

template <typename L, int W, int C>
cudaError_t launch_gate(const GateParams& p, int32_t* ids, float* probs, int32_t* counts,
                        int32_t* offsets, int32_t* scratch, cudaStream_t st) {
  using G = GateShape<W, C>;
  const int64_t per = G::kWarps * G::kTokens;
  const int64_t want = p.T > 0 ? (p.T + per - 1) / per : 1;
  const size_t smem = static_cast<size_t>(G::kWarps) * p.E * sizeof(double) + p.E * sizeof(int);
  auto* kernel = p.bias || p.n_group > 1 ? gate_kernel<L, W, C, true> : gate_kernel<L, W, C, false>;
  if (want <= kMaxCluster) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(want);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(want));
    cfg.blockDim = dim3(G::kWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, ids, probs, counts, offsets, scratch, 1);
  }
  cudaError_t e = cudaMemsetAsync(scratch, 0, gate_scratch_bytes(p.E), st);
  if (e != cudaSuccess) return e;
  const int64_t cap = static_cast<int64_t>(device_sm_count()) * 4;
  kernel<<<static_cast<unsigned>(want < cap ? want : cap), G::kWarps * 32, smem, st>>>(
      p, ids, probs, counts, offsets, scratch, 0);
  return cudaGetLastError();
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

// Calls f with the lanes per token and the experts per lane that hold E:
// eight experts a lane, as many tokens a warp as that leaves room for.
template <typename F>
cudaError_t with_shape(int E, F&& f) {
  if (E <= 8) return f.template operator()<1, 8>();
  if (E <= 16) return f.template operator()<2, 8>();
  if (E <= 32) return f.template operator()<4, 8>();
  if (E <= 64) return f.template operator()<8, 8>();
  if (E <= 128) return f.template operator()<16, 8>();
  if (E <= 256) return f.template operator()<32, 8>();
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
  return gate_scratch_bytes(E);
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
  if (!workspace || ws_bytes < moe_route_gate_workspace_size(T, k, E) ||
      (reinterpret_cast<uintptr_t>(workspace) & 15))
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
