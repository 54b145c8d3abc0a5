// gate.cu - moe_route_gate and its backward: the top-k gate with softmax or
// sigmoid scores, a balance bias, groups and renormalised weights.
#include <climits>

#include "common.cuh"
#include "internal.h"

namespace moe {

int* device_error_word();

namespace {

constexpr int kMaxGroups = 32;
constexpr int kGateWarps = 4;              // tokens in flight per CTA
constexpr float kFloatMax = 3.402823466e38f;

struct GateParams {
  const void* logits;
  const float* bias;
  int64_t T;
  int E, k, score, n_group, topk_group, group_topk, renorm;
  float scale;
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

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// The larger value first, equal values to the lower index.
__device__ __forceinline__ void warp_argmax(double& v, int& e) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double ov = __shfl_xor_sync(0xffffffffu, v, o);
    const int oe = __shfl_xor_sync(0xffffffffu, e, o);
    if (ov > v || (ov == v && oe < e)) {
      v = ov;
      e = oe;
    }
  }
}

// One warp per token, everything in double: scores and choice values in
// shared memory, the groups by one lane each, then k rounds of a warp
// arg-max in rank order.
template <typename L>
__global__ void __launch_bounds__(kGateWarps * 32)
    gate_kernel(GateParams p, int32_t* __restrict__ ids, float* __restrict__ probs,
                int32_t* __restrict__ counts) {
  extern __shared__ double sh_v[];                 // [warps][E] choice values
  __shared__ int sh_hist[kMaxExperts];
  const int lane = lane_id(), w = threadIdx.x >> 5;
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) sh_hist[e] = 0;
  __syncthreads();
  double* v = sh_v + static_cast<size_t>(w) * p.E;
  const int size = p.E / p.n_group;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kGateWarps + w; t < p.T;
       t += static_cast<int64_t>(gridDim.x) * kGateWarps) {
    const L* row = static_cast<const L*>(p.logits) + t * p.E;
    double inv = 1.0, top = 0.0;
    if (p.score == MOE_SCORE_SOFTMAX) {
      float m = -INFINITY;
      for (int e = lane; e < p.E; e += 32) m = fmaxf(m, clean(load_logit(row + e)));
      m = warp_max(m);
      top = m == -INFINITY ? 0.0 : static_cast<double>(m);
      double sum = 0.0;
      for (int e = lane; e < p.E; e += 32) sum += exp(clean(load_logit(row + e)) - top);
      sum = warp_sum(sum);
      inv = sum > 0.0 ? 1.0 / sum : 0.0;
    }
    auto score_of = [&](float l) {
      return p.score == MOE_SCORE_SOFTMAX ? exp(l - top) * inv
                                          : 1.0 / (1.0 + exp(-static_cast<double>(l)));
    };
    __syncwarp();
    for (int e = lane; e < p.E; e += 32) {
      const float l = clean(load_logit(row + e));
      const float b = p.bias ? clean(__ldg(p.bias + e)) : 0.0f;
      v[e] = l == -INFINITY || b == -INFINITY ? -INFINITY : score_of(l) + b;
    }
    __syncwarp();
    unsigned kept = 0xffffffffu;
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
        double bv = (lane < p.n_group && !((kept >> lane) & 1u)) ? g : -INFINITY;
        int be = (lane < p.n_group && !((kept >> lane) & 1u)) ? lane : INT_MAX;
        warp_argmax(bv, be);
        kept |= 1u << be;                           // topk_group <= n_group: one is left
      }
    }
    unsigned taken = 0u;                            // bit i: expert lane + 32 i
    double my_s = 0.0;
    float my_l = -INFINITY;
    int my_e = 0;
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
      if (lane == j) {
        my_e = be;
        const float l = clean(load_logit(row + be));
        if (v[be] != -INFINITY) {
          my_l = l;
          my_s = score_of(l);
        }
      }
    }
    double u = my_s;
    if (p.renorm) {
      if (p.score == MOE_SCORE_SOFTMAX) {
        const float m = warp_max(lane < p.k ? my_l : -INFINITY);
        u = my_l == -INFINITY ? 0.0 : exp(static_cast<double>(my_l) - m);
      }
      const double sum = warp_sum(lane < p.k ? u : 0.0);
      u = sum > 0.0 ? u / sum : 0.0;
    }
    if (lane < p.k) {
      ids[t * p.k + lane] = my_e;
      probs[t * p.k + lane] = static_cast<float>(p.scale * u);
      atomicAdd(&sh_hist[my_e], 1);
    }
    __syncwarp();
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += blockDim.x)
    if (sh_hist[e]) atomicAdd(counts + e, sh_hist[e]);
}

__global__ void __launch_bounds__(32) gate_offsets_kernel(const int32_t* __restrict__ counts, int E,
                                                          int32_t* __restrict__ offsets) {
  int run = 0;
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane_id();
    const int c = e < E ? counts[e] : 0;
    int inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane_id() >= o) inc += n;
    }
    if (e < E) offsets[e] = run + inc - c;
    run += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (threadIdx.x == 0) offsets[E] = run;
}

template <typename L>
__device__ __forceinline__ void store_grad(L* p, float v);
template <>
__device__ __forceinline__ void store_grad<float>(float* p, float v) {
  *p = v;
}
template <>
__device__ __forceinline__ void store_grad<__nv_bfloat16>(__nv_bfloat16* p, float v) {
  *p = __float2bfloat16_rn(v);
}

// One warp per token; lane j holds slot j.
template <typename L>
__global__ void __launch_bounds__(kGateWarps * 32)
    gate_backward_kernel(GateParams p, const float* __restrict__ dprobs,
                         const int32_t* __restrict__ ids, L* __restrict__ dlogits, int* err) {
  extern __shared__ double sh_g[];                 // [warps][E]
  const int lane = lane_id(), w = threadIdx.x >> 5;
  double* g = sh_g + static_cast<size_t>(w) * p.E;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kGateWarps + w; t < p.T;
       t += static_cast<int64_t>(gridDim.x) * kGateWarps) {
    const L* row = static_cast<const L*>(p.logits) + t * p.E;
    int e = -1;
    float l = -INFINITY;
    double dp = 0.0;
    if (lane < p.k) {
      e = ids[t * p.k + lane];
      if (e < 0 || e >= p.E) {
        report_error(err, kErrBadId);
        e = -1;
      } else {
        dp = dprobs[t * p.k + lane];
        l = clean(load_logit(row + e));
        if (p.bias && clean(__ldg(p.bias + e)) == -INFINITY) l = -INFINITY;
      }
    }
    const bool live = l != -INFINITY;
    const bool dense = p.score == MOE_SCORE_SOFTMAX && !p.renorm;
    double top = 0.0, inv = 1.0;
    if (dense) {
      float m = -INFINITY;
      for (int i = lane; i < p.E; i += 32) m = fmaxf(m, clean(load_logit(row + i)));
      m = warp_max(m);
      top = m == -INFINITY ? 0.0 : static_cast<double>(m);
      double sum = 0.0;
      for (int i = lane; i < p.E; i += 32) sum += exp(clean(load_logit(row + i)) - top);
      sum = warp_sum(sum);
      inv = sum > 0.0 ? 1.0 / sum : 0.0;
    }
    double u = 0.0, far = 1.0;
    if (live) {
      if (p.score == MOE_SCORE_SIGMOID) {
        u = 1.0 / (1.0 + exp(-static_cast<double>(l)));
        far = 1.0 / (1.0 + exp(static_cast<double>(l)));
      } else if (dense) {
        u = exp(l - top) * inv;
      }
    }
    if (p.renorm) {
      if (p.score == MOE_SCORE_SOFTMAX) {
        const float m = warp_max(l);
        u = live ? exp(static_cast<double>(l) - m) : 0.0;
      }
      const double sum = warp_sum(u);
      u = sum > 0.0 ? u / sum : 0.0;
    }
    const double d = warp_sum(live ? dp * u : 0.0);
    double mine = 0.0;
    if (live) mine = dense ? u * dp : p.renorm ? u * far * (dp - d) : u * far * dp;
    for (int i = lane; i < p.E; i += 32)
      g[i] = dense ? -exp(clean(load_logit(row + i)) - top) * inv * d : 0.0;
    __syncwarp();
    for (int j = 0; j < p.k; ++j) {                // in slot order: a repeated id adds up
      if (lane == j && live) g[e] += mine;
      __syncwarp();
    }
    for (int i = lane; i < p.E; i += 32)
      store_grad(dlogits + t * p.E + i, static_cast<float>(p.scale * g[i]));
    __syncwarp();
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
  *p = GateParams{logits,    bias,         T,            E,           k, c.score,
                  c.n_group, c.topk_group, c.group_topk, c.renormalise, c.scale};
  return MOE_OK;
}

int gate_grid(int64_t T) {
  const int64_t want = (T + kGateWarps - 1) / kGateWarps;
  const int64_t cap = static_cast<int64_t>(device_sm_count()) * 8;
  return static_cast<int>(want < cap ? want : cap);
}

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
  return 256;
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
  if (cudaMemsetAsync(counts, 0, E * sizeof(int32_t), st) != cudaSuccess) return MOE_ERR_CUDA;
  const size_t smem = static_cast<size_t>(kGateWarps) * E * sizeof(double);
  if (T > 0) {
    if (logits_type == MOE_TYPE_F32)
      gate_kernel<float><<<gate_grid(T), kGateWarps * 32, smem, st>>>(p, expert_ids, probs, counts);
    else
      gate_kernel<__nv_bfloat16>
          <<<gate_grid(T), kGateWarps * 32, smem, st>>>(p, expert_ids, probs, counts);
  }
  gate_offsets_kernel<<<1, 32, 0, st>>>(counts, E, offsets);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
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
  const size_t smem = static_cast<size_t>(kGateWarps) * E * sizeof(double);
  int* err = device_error_word();
  if (logits_type == MOE_TYPE_F32)
    gate_backward_kernel<float><<<gate_grid(T), kGateWarps * 32, smem, st>>>(
        p, dprobs, expert_ids, static_cast<float*>(dlogits), err);
  else
    gate_backward_kernel<__nv_bfloat16><<<gate_grid(T), kGateWarps * 32, smem, st>>>(
        p, dprobs, expert_ids, static_cast<__nv_bfloat16*>(dlogits), err);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
