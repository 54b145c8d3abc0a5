// clip.cu - moe_clip_grad_norm: one norm over many gradients, and all of
// them scaled by it.
#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kClipThreads = 256;
constexpr int kClipChunk = 16384;          // elements of one work item
constexpr int kClipTensors = 256;          // tensors of one launch's table
constexpr int kClipMaxCtas = 2048;         // partial results in the workspace

struct ClipTable {
  const void* src[kClipTensors];
  void* dst[kClipTensors];
  int64_t numel[kClipTensors];
  int64_t chunk0[kClipTensors + 1];        // first work item of each tensor
  uint8_t type[kClipTensors];
  int n;
};

// The tensor whose work items hold c.
__device__ __forceinline__ int clip_find(const ClipTable& t, int64_t c) {
  int lo = 0, hi = t.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.chunk0[mid] <= c)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ float clip_load(const ClipTable& t, int i, int64_t at) {
  return t.type[i] == MOE_TYPE_F32
             ? static_cast<const float*>(t.src[i])[at]
             : __bfloat162float(static_cast<const __nv_bfloat16*>(t.src[i])[at]);
}

// The larger of two magnitudes as bit patterns: a NaN is above every number.
__device__ __forceinline__ unsigned max_bits(unsigned m, float g) {
  return max(m, __float_as_uint(g) & 0x7fffffffu);
}

// Every CTA's part of the sum of squares (or of the largest magnitude, as
// the value of its bits) into partial[blockIdx.x]; a later launch of the
// same call (first = 0) adds to it, in the same order every time.
__global__ void __launch_bounds__(kClipThreads)
    clip_norm_kernel(const __grid_constant__ ClipTable t, int kind, int first,
                     double* __restrict__ partial) {
  __shared__ double sh[kClipThreads];
  double sum = 0.0;
  unsigned big = 0u;
  const int64_t items = t.chunk0[t.n];
  for (int64_t c = blockIdx.x; c < items; c += gridDim.x) {
    const int i = clip_find(t, c);
    const int64_t lo = (c - t.chunk0[i]) * kClipChunk;
    const int64_t hi = min(t.numel[i], lo + kClipChunk);
    float part = 0.0f;
    for (int64_t at = lo + threadIdx.x; at < hi; at += kClipThreads) {
      const float g = clip_load(t, i, at);
      part = fmaf(g, g, part);
      big = max_bits(big, g);
    }
    sum += part;
  }
  sh[threadIdx.x] = kind == 0 ? sum : static_cast<double>(big);
  for (int o = kClipThreads / 2; o > 0; o >>= 1) {
    __syncthreads();
    if (threadIdx.x < o)
      sh[threadIdx.x] = kind == 0 ? sh[threadIdx.x] + sh[threadIdx.x + o]
                                  : fmax(sh[threadIdx.x], sh[threadIdx.x + o]);
  }
  if (threadIdx.x == 0) {
    double v = sh[0];
    if (!first) v = kind == 0 ? v + partial[blockIdx.x] : fmax(v, partial[blockIdx.x]);
    partial[blockIdx.x] = v;
  }
}

__global__ void __launch_bounds__(32) clip_finish_kernel(const double* __restrict__ partial, int n,
                                                         int kind, float max_norm, float eps,
                                                         float* __restrict__ norm_coef) {
  double v = 0.0;
  for (int i = threadIdx.x; i < n; i += 32) v = kind == 0 ? v + partial[i] : fmax(v, partial[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double x = __shfl_xor_sync(0xffffffffu, v, o);
    v = kind == 0 ? v + x : fmax(v, x);
  }
  if (threadIdx.x == 0) {
    const double norm = kind == 0 ? sqrt(v) : __uint_as_float(static_cast<unsigned>(v));
    const double c = max_norm / (norm + eps);
    norm_coef[0] = static_cast<float>(norm);
    norm_coef[1] = max_norm < 0.0f || c >= 1.0 ? 1.0f : static_cast<float>(c);
  }
}

__global__ void __launch_bounds__(kClipThreads)
    clip_scale_kernel(const __grid_constant__ ClipTable t, int in_place,
                      const float* __restrict__ norm_coef) {
  const float coef = norm_coef[1];
  if (in_place && coef == 1.0f) return;
  const int64_t items = t.chunk0[t.n];
  for (int64_t c = blockIdx.x; c < items; c += gridDim.x) {
    const int i = clip_find(t, c);
    const int64_t lo = (c - t.chunk0[i]) * kClipChunk;
    const int64_t hi = min(t.numel[i], lo + kClipChunk);
    for (int64_t at = lo + threadIdx.x; at < hi; at += kClipThreads) {
      const float g = clip_load(t, i, at) * coef;
      if (t.type[i] == MOE_TYPE_F32)
        static_cast<float*>(t.dst[i])[at] = g;
      else
        static_cast<__nv_bfloat16*>(t.dst[i])[at] = __float2bfloat16_rn(g);
    }
  }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_clip_grad_norm_workspace_size(void) { return kClipMaxCtas * sizeof(double); }

moe_status moe_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* numels,
                              const int* types, int64_t n_tensors, float max_norm, int norm_kind,
                              float eps, float* norm_coef, void* workspace, size_t ws_bytes,
                              void* stream) {
  MOE_ENTRY_RANGE();
  if (n_tensors < 0 || n_tensors > (1 << 20) || (norm_kind != 0 && norm_kind != 1) ||
      !(eps >= 0.0f) || max_norm != max_norm || !norm_coef)
    return MOE_ERR_INVALID_ARG;
  if (n_tensors > 0 && (!grads || !numels || !types)) return MOE_ERR_INVALID_ARG;
  for (int64_t i = 0; i < n_tensors; ++i) {
    if (numels[i] < 0 || numels[i] > (static_cast<int64_t>(1) << 48) ||
        (types[i] != MOE_TYPE_F32 && types[i] != MOE_TYPE_BF16))
      return MOE_ERR_INVALID_ARG;
    if (numels[i] == 0) continue;
    const uintptr_t mask = types[i] == MOE_TYPE_F32 ? 3 : 1;
    if (!grads[i] || (reinterpret_cast<uintptr_t>(grads[i]) & mask)) return MOE_ERR_INVALID_ARG;
    if (outs && (!outs[i] || (reinterpret_cast<uintptr_t>(outs[i]) & mask)))
      return MOE_ERR_INVALID_ARG;
  }
  if (!workspace || ws_bytes < moe_clip_grad_norm_workspace_size() ||
      (reinterpret_cast<uintptr_t>(workspace) & 15))
    return MOE_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  double* partial = static_cast<double*>(workspace);
  ClipTable t;
  const int cap = device_sm_count() * 8 < kClipMaxCtas ? device_sm_count() * 8 : kClipMaxCtas;
  for (int pass = 0; pass < 2; ++pass) {
    if (pass == 1 && max_norm < 0.0f && !outs) break;
    int launches = 0;
    int64_t i = 0;
    do {
      t.n = 0;
      t.chunk0[0] = 0;
      for (; i < n_tensors && t.n < kClipTensors; ++i) {
        if (numels[i] == 0) continue;
        t.src[t.n] = grads[i];
        t.dst[t.n] = outs ? outs[i] : const_cast<void*>(grads[i]);
        t.numel[t.n] = numels[i];
        t.type[t.n] = static_cast<uint8_t>(types[i]);
        t.chunk0[t.n + 1] = t.chunk0[t.n] + (numels[i] + kClipChunk - 1) / kClipChunk;
        ++t.n;
      }
      // every norm launch has the whole grid, so that all partials are written
      if (pass == 0)
        clip_norm_kernel<<<cap, kClipThreads, 0, st>>>(t, norm_kind, launches == 0, partial);
      else if (t.n > 0)
        clip_scale_kernel<<<cap, kClipThreads, 0, st>>>(t, outs == nullptr, norm_coef);
      ++launches;
    } while (i < n_tensors);
    if (pass == 0)
      clip_finish_kernel<<<1, 32, 0, st>>>(partial, cap, norm_kind, max_norm, eps, norm_coef);
  }
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
