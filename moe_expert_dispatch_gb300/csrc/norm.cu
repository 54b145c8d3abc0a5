// norm.cu - moe_norm_residual and its backward: the norm after the block,
// its gate, the scaled residual and the norm before the next block.
#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kNormThreads = 256;
constexpr int kMaxNormH = 65536;

struct NormParams {
  const void* x;        // forward: the stream; backward: d_out (may be null)
  const void* out;      // backward: the forward's out
  const __nv_bfloat16* y;
  const __nv_bfloat16* d_n;
  const void* w_post;
  const void* gate;
  const void* w_next;
  const float* rstd_y;
  const float* rstd_out;
  int64_t T;
  int64_t gate_span;    // tokens that share a gate row
  int H;
  float eps, a, b;
  float inv_h;
};

template <typename E>
__device__ __forceinline__ float ld(const void* p, int64_t i);
// plain loads: out may be x, and dx may be d_out
template <>
__device__ __forceinline__ float ld<float>(const void* p, int64_t i) {
  return static_cast<const float*>(p)[i];
}
template <>
__device__ __forceinline__ float ld<__nv_bfloat16>(const void* p, int64_t i) {
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void st(float* p, float v) { *p = v; }
__device__ __forceinline__ void st(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// The sum of v over the CTA, to every thread; red holds one float per warp.
__device__ __forceinline__ float cta_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (lane_id() == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) s += red[i];
  return s;
}

// ------------------------------------------------------------------ any H, any alignment

// One CTA per row, three passes over it (the later two from L1/L2).
template <typename ST, typename WT>
__global__ void __launch_bounds__(kNormThreads)
    norm_rows_kernel(NormParams p, ST* out, __nv_bfloat16* __restrict__ n, float* rstd_y,
                     float* rstd_out) {
  __shared__ float red[kNormThreads / 32];
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    const int64_t at = t * p.H;
    float ry = 1.0f;
    if (p.w_post) {
      float s = 0.0f;
      for (int h = threadIdx.x; h < p.H; h += kNormThreads) {
        const float v = ld<__nv_bfloat16>(p.y, at + h);
        s = fmaf(v, v, s);
      }
      ry = 1.0f / sqrtf(cta_sum(s, red) * p.inv_h + p.eps);
      if (threadIdx.x == 0 && rstd_y) rstd_y[t] = ry;
    }
    const int64_t gat = p.gate ? t / p.gate_span * p.H : 0;
    auto row = [&](int h) {
      const float xv = ld<ST>(p.x, at + h);
      if (!p.y) return xv;
      float z = ld<__nv_bfloat16>(p.y, at + h);
      if (p.w_post) z = z * ry * ld<WT>(p.w_post, h);
      if (p.gate) z *= ld<WT>(p.gate, gat + h);
      return fmaf(p.a, xv, p.b * z);
    };
    float ro = 1.0f;
    if (p.w_next) {
      float s = 0.0f;
      for (int h = threadIdx.x; h < p.H; h += kNormThreads) {
        const float o = row(h);
        s = fmaf(o, o, s);
      }
      ro = 1.0f / sqrtf(cta_sum(s, red) * p.inv_h + p.eps);
      if (threadIdx.x == 0 && rstd_out) rstd_out[t] = ro;
    }
    for (int h = threadIdx.x; h < p.H; h += kNormThreads) {
      const float o = row(h);                      // before out, which may be x, is written
      if (out) st(out + at + h, o);
      if (p.w_next) st(n + at + h, o * ro * ld<WT>(p.w_next, h));
    }
  }
}

// D_t at column h, from the row's mean c = m(q * o).
template <typename ST, typename WT>
__device__ __forceinline__ float total_grad(const NormParams& p, int64_t at, int h, float ro,
                                            float c) {
  float d = p.x ? ld<ST>(p.x, at + h) : 0.0f;
  if (p.d_n) {
    const float q = ld<__nv_bfloat16>(p.d_n, at + h) * ld<WT>(p.w_next, h);
    d = fmaf(ro, q - ld<ST>(p.out, at + h) * ro * c, d);
  }
  return d;
}

// One CTA per row. kMean: the row's mean c, for the column sums that follow;
// else dx and dy from it. Two launches around the column sums, because these
// read d_out and dx may be d_out itself.
template <typename ST, typename WT, bool kMean>
__global__ void __launch_bounds__(kNormThreads)
    norm_rows_backward_kernel(NormParams p, ST* dx, __nv_bfloat16* __restrict__ dy,
                              float* __restrict__ c_of) {
  __shared__ float red[kNormThreads / 32];
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    const int64_t at = t * p.H;
    const float ro = p.d_n ? p.rstd_out[t] : 0.0f;
    if (kMean) {
      float s = 0.0f;
      if (p.d_n)
        for (int h = threadIdx.x; h < p.H; h += kNormThreads)
          s = fmaf(ld<__nv_bfloat16>(p.d_n, at + h) * ld<WT>(p.w_next, h),
                   ld<ST>(p.out, at + h) * ro, s);
      s = cta_sum(s, red);
      if (threadIdx.x == 0) c_of[t] = s * p.inv_h;
      continue;
    }
    const float c = c_of[t];
    const int64_t gat = p.gate ? t / p.gate_span * p.H : 0;
    const float ry = p.y && p.w_post ? p.rstd_y[t] : 1.0f;
    auto grad_z = [&](int h) {                     // of the normalised y, times w_post
      float q = p.b * total_grad<ST, WT>(p, at, h, ro, c);
      if (p.gate) q *= ld<WT>(p.gate, gat + h);
      if (p.w_post) q *= ld<WT>(p.w_post, h);
      return q;
    };
    float m = 0.0f;
    if (p.y && p.w_post) {
      float s = 0.0f;
      for (int h = threadIdx.x; h < p.H; h += kNormThreads)
        s = fmaf(grad_z(h), ld<__nv_bfloat16>(p.y, at + h) * ry, s);
      m = cta_sum(s, red) * p.inv_h;
    }
    for (int h = threadIdx.x; h < p.H; h += kNormThreads) {
      const float d = total_grad<ST, WT>(p, at, h, ro, c);
      if (p.y) {
        float q = grad_z(h);
        if (p.w_post) q = ry * (q - ld<__nv_bfloat16>(p.y, at + h) * ry * m);
        st(dy + at + h, q);
      }
      st(dx + at + h, p.y ? p.a * d : d);          // last: dx may be d_out
    }
  }
}

// Rows of strip i of n: [i T / n, (i + 1) T / n); the strip of a row.
__host__ __device__ __forceinline__ int64_t strip_row(int64_t T, int n, int64_t i) {
  return i * T / n;
}
__device__ __forceinline__ int64_t strip_of(int64_t T, int n, int64_t row) {
  return ((row + 1) * n - 1) / T;
}

// Column sums of a strip of rows (blockIdx.y), one column per thread: dw_next
// and dw_post into part[strip], and S = sum D yh of every gate row: straight
// to dgate where the strip holds all of the row's tokens, else into one of
// the strip's two pieces (0: the row began in an earlier strip, 1: in this one).
template <typename ST, typename WT>
__global__ void __launch_bounds__(128)
    norm_cols_backward_kernel(NormParams p, const float* __restrict__ c_of,
                              float* __restrict__ part_post, float* __restrict__ part_next,
                              float* __restrict__ part_gate, float* __restrict__ dgate,
                              int accumulate) {
  const int h = blockIdx.x * 128 + threadIdx.x;
  if (h >= p.H) return;
  const int64_t strip = blockIdx.y;
  const int64_t lo = strip_row(p.T, gridDim.y, strip), hi = strip_row(p.T, gridDim.y, strip + 1);
  const float wp = p.w_post ? ld<WT>(p.w_post, h) : 1.0f;
  float sum_post = 0.0f, sum_next = 0.0f, s = 0.0f, g = 1.0f;
  int64_t first = 0;                               // the current gate row's first token
  for (int64_t t = lo; t < hi; ++t) {
    if (p.gate && (t == lo || t % p.gate_span == 0)) {
      first = t / p.gate_span * p.gate_span;
      g = ld<WT>(p.gate, t / p.gate_span * p.H + h);
      s = 0.0f;
    }
    const float ro = p.d_n ? p.rstd_out[t] : 0.0f;
    if (p.y) {
      const float d = p.b * total_grad<ST, WT>(p, t * p.H, h, ro, c_of[t]);
      const float yh = ld<__nv_bfloat16>(p.y, t * p.H + h) * (p.w_post ? p.rstd_y[t] : 1.0f);
      sum_post = fmaf(g * d, yh, sum_post);
      s = fmaf(d, yh, s);
    }
    if (p.d_n)
      sum_next = fmaf(ld<__nv_bfloat16>(p.d_n, t * p.H + h), ld<ST>(p.out, t * p.H + h) * ro,
                      sum_next);
    if (p.gate && (t + 1 == hi || (t + 1) % p.gate_span == 0)) {
      if (first >= lo && first + p.gate_span <= hi) {
        float* to = dgate + t / p.gate_span * p.H + h;
        *to = accumulate ? *to + s * wp : s * wp;
      } else {
        part_gate[(strip * 2 + (first >= lo)) * p.H + h] = s;
      }
    }
  }
  if (part_post) part_post[strip * p.H + h] = sum_post;
  if (part_next) part_next[strip * p.H + h] = sum_next;
}

// The strips' parts, in order. blockIdx.y 0: dw_post, 1: dw_next, 2 + r: gate row r.
template <typename WT>
__global__ void __launch_bounds__(128)
    norm_finish_kernel(NormParams p, int strips, const float* __restrict__ part_post,
                       const float* __restrict__ part_next, const float* __restrict__ part_gate,
                       float* __restrict__ dw_post, float* __restrict__ dw_next,
                       float* __restrict__ dgate, int64_t gate_rows, int accumulate) {
  const int h = blockIdx.x * 128 + threadIdx.x;
  if (h >= p.H) return;
  for (int64_t what = blockIdx.y; what < 2 + gate_rows; what += gridDim.y) {
    float s = 0.0f;
    float* to;
    if (what < 2) {
      const float* part = what == 0 ? part_post : part_next;
      to = what == 0 ? dw_post : dw_next;
      if (!to) continue;
      if (part)
        for (int i = 0; i < strips; ++i) s += part[static_cast<int64_t>(i) * p.H + h];
      to += h;
    } else {
      const int64_t r = what - 2, a = r * p.gate_span, b = a + p.gate_span;
      to = dgate + r * p.H + h;
      if (strips > 0) {
        const int64_t i0 = strip_of(p.T, strips, a), i1 = strip_of(p.T, strips, b - 1);
        if (i0 == i1) continue;                    // written by its strip
        for (int64_t i = i0; i <= i1; ++i) s += part_gate[(i * 2 + (i == i0)) * p.H + h];
      }
      if (p.w_post) s *= ld<WT>(p.w_post, h);
    }
    *to = accumulate ? *to + s : s;
  }
}

int norm_strips(int64_t T) {
  const int64_t most = static_cast<int64_t>(device_sm_count()) * 2;
  return static_cast<int>(T < most ? T : most);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

moe_status norm_config_of(moe_norm_config* c, const moe_norm_config* cfg, int64_t T, int H) {
  moe_norm_config_init(c);
  if (cfg) *c = *cfg;
  if (T < 0 || H < 1 || T > (static_cast<int64_t>(1) << 40)) return MOE_ERR_INVALID_ARG;
  if (H > kMaxNormH) return MOE_ERR_UNSUPPORTED;
  if (!(c->eps >= 0.0f) || !(c->residual_scale - c->residual_scale == 0.0f) ||
      !(c->branch_scale - c->branch_scale == 0.0f))
    return MOE_ERR_INVALID_ARG;
  if ((c->stream_type != MOE_TYPE_F32 && c->stream_type != MOE_TYPE_BF16) ||
      (c->weight_type != MOE_TYPE_F32 && c->weight_type != MOE_TYPE_BF16))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

bool gate_rows_ok(const void* gate, int64_t rows, int64_t T) {
  return gate ? rows >= 1 && (T == 0 || T % rows == 0) : rows == 0;
}

int rows_grid(int64_t T) {
  const int64_t most = static_cast<int64_t>(device_sm_count()) * 8;
  return static_cast<int>(T < most ? T : most);
}

template <typename ST, typename WT>
cudaError_t forward(const NormParams& p, void* out, void* n, float* rstd_y, float* rstd_out,
                    cudaStream_t s) {
  norm_rows_kernel<ST, WT><<<rows_grid(p.T), kNormThreads, 0, s>>>(
      p, static_cast<ST*>(out), static_cast<__nv_bfloat16*>(n), rstd_y, rstd_out);
  return cudaGetLastError();
}

struct NormGrads {
  void *dx, *dy;
  float *dw_post, *dgate, *dw_next;
  int64_t gate_rows;
  int accumulate;
};

template <typename ST, typename WT>
cudaError_t backward(const NormParams& p, const NormGrads& g, void* ws, cudaStream_t s) {
  const int strips = p.T > 0 ? norm_strips(p.T) : 0;
  float* c_of = static_cast<float*>(ws);
  float* part = c_of + (p.T + 63) / 64 * 64;
  const int64_t one = static_cast<int64_t>(strips) * p.H;
  float* part_post = g.dw_post && strips ? part : nullptr;
  float* part_next = g.dw_next && strips ? part + one : nullptr;
  float* part_gate = part + 2 * one;
  const unsigned cols = static_cast<unsigned>((p.H + 127) / 128);
  if (p.T > 0) {
    norm_rows_backward_kernel<ST, WT, true><<<rows_grid(p.T), kNormThreads, 0, s>>>(
        p, static_cast<ST*>(g.dx), static_cast<__nv_bfloat16*>(g.dy), c_of);
    if (part_post || part_next || g.dgate)
      norm_cols_backward_kernel<ST, WT><<<dim3(cols, strips), 128, 0, s>>>(
          p, c_of, part_post, part_next, part_gate, g.dgate, g.accumulate);
    norm_rows_backward_kernel<ST, WT, false><<<rows_grid(p.T), kNormThreads, 0, s>>>(
        p, static_cast<ST*>(g.dx), static_cast<__nv_bfloat16*>(g.dy), c_of);
  }
  if (g.dw_post || g.dw_next || g.dgate) {
    const int64_t want = 2 + g.gate_rows;
    norm_finish_kernel<WT><<<dim3(cols, static_cast<unsigned>(want < 1024 ? want : 1024)), 128, 0,
                             s>>>(p, strips, part_post, part_next, part_gate, g.dw_post, g.dw_next,
                                  g.dgate, g.dgate ? g.gate_rows : 0, g.accumulate);
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

void moe_norm_config_init(moe_norm_config* cfg) {
  if (!cfg) return;
  *cfg = moe_norm_config{1e-6f, 1.0f, 1.0f, MOE_TYPE_BF16, MOE_TYPE_BF16};
}

moe_status moe_norm_residual(const void* x, const void* y, const void* w_post, const void* gate,
                             int64_t gate_rows, const void* w_next, int64_t T, int H,
                             const moe_norm_config* cfg, void* out, void* n, float* rstd_y,
                             float* rstd_out, void* stream) {
  MOE_ENTRY_RANGE();
  moe_norm_config c;
  const moe_status s = norm_config_of(&c, cfg, T, H);
  if (s != MOE_OK) return s;
  if (!gate_rows_ok(gate, gate_rows, T)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;                       // empty tensors may come as null pointers
  if (!y && (w_post || gate || out || !w_next)) return MOE_ERR_INVALID_ARG;
  if (!x || (y && !out) || (w_next && !n)) return MOE_ERR_INVALID_ARG;
  for (const void* q : {x, y, w_post, gate, w_next, static_cast<const void*>(out),
                        static_cast<const void*>(n)})
    if (!aligned16(q)) return MOE_ERR_INVALID_ARG;
  NormParams p = {};
  p.x = x;
  p.y = static_cast<const __nv_bfloat16*>(y);
  p.w_post = w_post;
  p.gate = gate;
  p.w_next = w_next;
  p.T = T;
  p.gate_span = gate ? T / gate_rows : T;
  p.H = H;
  p.eps = c.eps;
  p.a = c.residual_scale;
  p.b = c.branch_scale;
  p.inv_h = 1.0f / H;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool sf = c.stream_type == MOE_TYPE_F32, wf = c.weight_type == MOE_TYPE_F32;
  auto* run = sf ? (wf ? forward<float, float> : forward<float, __nv_bfloat16>)
                 : (wf ? forward<__nv_bfloat16, float> : forward<__nv_bfloat16, __nv_bfloat16>);
  return run(p, out, n, rstd_y, rstd_out, st) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_norm_residual_backward_workspace_size(int64_t T, int H, int64_t gate_rows) {
  if (T < 0 || H < 1 || H > kMaxNormH || gate_rows < 0 || T > (static_cast<int64_t>(1) << 40))
    return 0;
  return static_cast<size_t>((T + 63) / 64 * 64) * sizeof(float) +
         4 * static_cast<size_t>(norm_strips(T)) * H * sizeof(float) + 256;
}

moe_status moe_norm_residual_backward(const void* d_out, const void* d_n, const void* out,
                                      const void* y, const void* w_post, const void* gate,
                                      int64_t gate_rows, const void* w_next, const float* rstd_y,
                                      const float* rstd_out, int64_t T, int H,
                                      const moe_norm_config* cfg, void* dx, void* dy,
                                      float* dw_post, float* dgate, float* dw_next,
                                      int accumulate_dw, void* workspace, size_t ws_bytes,
                                      void* stream) {
  MOE_ENTRY_RANGE();
  moe_norm_config c;
  const moe_status s = norm_config_of(&c, cfg, T, H);
  if (s != MOE_OK) return s;
  if (!gate_rows_ok(gate, gate_rows, T)) return MOE_ERR_INVALID_ARG;
  // with no tokens, empty tensors may come as null pointers
  if (T > 0 && ((!y && (w_post || gate || dy)) || (!d_out && !d_n) || (d_n && !w_next) ||
                (d_n && !dw_next) || (!d_n && dw_next)))
    return MOE_ERR_INVALID_ARG;
  if ((w_post && !dw_post) || (gate && !dgate) || (!w_post && dw_post) || (!gate && dgate) ||
      (!w_next && dw_next))
    return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!dx || (y && !dy) || (d_n && (!out || !rstd_out)) || (w_post && !rstd_y)))
    return MOE_ERR_INVALID_ARG;
  for (const void* q : {d_out, d_n, out, y, w_post, gate, w_next, static_cast<const void*>(dx),
                        static_cast<const void*>(dy), static_cast<const void*>(dw_post),
                        static_cast<const void*>(dgate), static_cast<const void*>(dw_next)})
    if (!aligned16(q)) return MOE_ERR_INVALID_ARG;
  if (!workspace || ws_bytes < moe_norm_residual_backward_workspace_size(T, H, gate_rows) ||
      !aligned16(workspace))
    return MOE_ERR_WORKSPACE;
  NormParams p = {};
  p.x = d_out;
  p.out = out;
  p.y = static_cast<const __nv_bfloat16*>(y);
  p.d_n = static_cast<const __nv_bfloat16*>(d_n);
  p.w_post = w_post;
  p.gate = gate;
  p.w_next = w_next;
  p.rstd_y = rstd_y;
  p.rstd_out = rstd_out;
  p.T = T;
  p.gate_span = gate && T ? T / gate_rows : (T ? T : 1);
  p.H = H;
  p.eps = c.eps;
  p.a = c.residual_scale;
  p.b = c.branch_scale;
  p.inv_h = 1.0f / H;
  const NormGrads g{dx, dy, dw_post, dgate, dw_next, gate_rows, accumulate_dw};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool sf = c.stream_type == MOE_TYPE_F32, wf = c.weight_type == MOE_TYPE_F32;
  auto* run = sf ? (wf ? backward<float, float> : backward<float, __nv_bfloat16>)
                 : (wf ? backward<__nv_bfloat16, float> : backward<__nv_bfloat16, __nv_bfloat16>);
  return run(p, g, workspace, st) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
