// norm.cu - moe_norm_residual and its backward: the norm after the block,
// its gate, the scaled residual and the norm before the next block. The entry
// points, and the kernels for rows that those of norm_ring.cu do not take.
#include "norm.cuh"

#include <type_traits>

namespace moe {
namespace {

constexpr int kNormThreads = 256;
constexpr int kMaxNormH = 65536;
constexpr int64_t kMaxTokens = (static_cast<int64_t>(1) << 32) - 1;

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

// ------------------------------------------------------------------ forward, rows in registers

// W consecutive elements of one of the two types, through 8- or 16-byte words.
template <int W>
struct Raw {
  unsigned u[W / 2];
};
template <int W>
__device__ __forceinline__ Raw<W> load_bf16(const void* p, int64_t i) {
  Raw<W> r;
  const char* at = static_cast<const char*>(p) + i * 2;
  if constexpr (W == 8)
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.u[0]), "=r"(r.u[1]), "=r"(r.u[2]), "=r"(r.u[3])
                 : "l"(at)
                 : "memory");
  else
    asm volatile("ld.global.L1::no_allocate.v2.b32 {%0, %1}, [%2];"
                 : "=r"(r.u[0]), "=r"(r.u[1])
                 : "l"(at)
                 : "memory");
  return r;
}
template <int W>
__device__ __forceinline__ void unpack(const Raw<W>& r, float (&f)[W]) {
#pragma unroll
  for (int i = 0; i < W / 2; ++i) {
    f[2 * i] = __uint_as_float(r.u[i] << 16);
    f[2 * i + 1] = __uint_as_float(r.u[i] & 0xffff0000u);
  }
}
template <int W>
__device__ __forceinline__ void store_bf16(__nv_bfloat16* p, const float (&f)[W]) {
  if constexpr (W == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                              pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
}
// Weights: read by every row, so they stay in L1.
template <typename WT, int W>
__device__ __forceinline__ void load_weights(const void* p, int64_t i, float (&f)[W]) {
  if constexpr (sizeof(WT) == 4) {
#pragma unroll
    for (int h = 0; h < W; h += 4) {
      const float4 q = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i + h));
      f[h] = q.x;
      f[h + 1] = q.y;
      f[h + 2] = q.z;
      f[h + 3] = q.w;
    }
  } else {
    Raw<W> r;
    const uint2* q = reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + i);
#pragma unroll
    for (int h = 0; h < W / 4; ++h) {
      const uint2 v = __ldg(q + h);
      r.u[2 * h] = v.x;
      r.u[2 * h + 1] = v.y;
    }
    unpack<W>(r, f);
  }
}

// The sum of v over the CTA to every thread, with one barrier; red: one float
// for each of up to 32 warps, not written again before the barrier after.
__device__ __forceinline__ float cta_sum_once(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane_id() == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane_id() < static_cast<int>(blockDim.x >> 5) ? red[lane_id()] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One CTA per row, the whole row in its registers: V vectors of W elements a
// thread (16-byte loads of the stream, coalesced for both types), loaded
// before the first of the two reductions, so that x and y are read once. For
// few rows (1 x 7168: 3.1 us, a launch and two reductions; the ring kernel 3.4)
// and for rows longer than the ring kernels take (4096 x 10240: 74 us, bound by
// the latency between its reductions; their bytes take 49).
template <typename ST, typename WT, int V>
__global__ void __launch_bounds__(1024)
    norm_forward_kernel(NormParams p, ST* out, __nv_bfloat16* __restrict__ n, float* rstd_y,
                        float* rstd_out) {
  constexpr int W = sizeof(ST) == 4 ? 4 : 8;
  __shared__ float red[2][2][32];
  const int nvec = p.H / W;
  int odd = 0;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, odd ^= 1) {
    const int64_t at = t * p.H;
    Raw<W> y[V];
    float x[V][W];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = threadIdx.x + v * blockDim.x;
      if (i >= nvec) continue;
      if (p.y) y[v] = load_bf16<W>(p.y, at + i * W);
      if constexpr (W == 4) {
        const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(p.x) + at +
                                                          i * W);
        x[v][0] = q.x;
        x[v][1] = q.y;
        x[v][2] = q.z;
        x[v][3] = q.w;
      } else {
        unpack<W>(load_bf16<W>(p.x, at + i * W), x[v]);
      }
    }
    if (p.y) {
      float ry = 1.0f;
      if (p.w_post) {
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (threadIdx.x + v * blockDim.x >= nvec) continue;
          float f[W];
          unpack<W>(y[v], f);
#pragma unroll
          for (int h = 0; h < W; ++h) s = fmaf(f[h], f[h], s);
        }
        ry = 1.0f / sqrtf(cta_sum_once(s, red[odd][0]) * p.inv_h + p.eps);
        if (threadIdx.x == 0 && rstd_y) rstd_y[t] = ry;
      }
      const int64_t gat = p.gate ? t / p.gate_span * p.H : 0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int i = threadIdx.x + v * blockDim.x;
        if (i >= nvec) continue;
        float f[W], w[W];
        unpack<W>(y[v], f);
        if (p.w_post) {
          load_weights<WT, W>(p.w_post, i * W, w);
#pragma unroll
          for (int h = 0; h < W; ++h) f[h] = f[h] * ry * w[h];
        }
        if (p.gate) {
          load_weights<WT, W>(p.gate, gat + i * W, w);
#pragma unroll
          for (int h = 0; h < W; ++h) f[h] *= w[h];
        }
#pragma unroll
        for (int h = 0; h < W; ++h) x[v][h] = fmaf(p.a, x[v][h], p.b * f[h]);
        if constexpr (W == 4)
          *reinterpret_cast<float4*>(out + at + i * W) =
              make_float4(x[v][0], x[v][1], x[v][2], x[v][3]);
        else
          store_bf16<W>(out + at + i * W, x[v]);
      }
    }
    if (p.w_next) {
      float s = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (threadIdx.x + v * blockDim.x >= nvec) continue;
#pragma unroll
        for (int h = 0; h < W; ++h) s = fmaf(x[v][h], x[v][h], s);
      }
      const float ro = 1.0f / sqrtf(cta_sum_once(s, red[odd][1]) * p.inv_h + p.eps);
      if (threadIdx.x == 0 && rstd_out) rstd_out[t] = ro;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int i = threadIdx.x + v * blockDim.x;
        if (i >= nvec) continue;
        float w[W];
        load_weights<WT, W>(p.w_next, i * W, w);
#pragma unroll
        for (int h = 0; h < W; ++h) w[h] *= x[v][h] * ro;
        store_bf16<W>(n + at + i * W, w);
      }
    }
  }
}

// ------------------------------------------------------------------ any H

// V elements: one, or four through 8- or 16-byte words. Plain accesses: out may be
// x, and dx may be d_out.
template <typename E, int V>
__device__ __forceinline__ void ldv(const void* p, int64_t i, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = ld<E>(p, i);
  } else if constexpr (sizeof(E) == 4) {
    const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    f[0] = q.x;
    f[1] = q.y;
    f[2] = q.z;
    f[3] = q.w;
  } else {
    const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + i);
    unpack<4>(Raw<4>{q.x, q.y}, f);
  }
}
template <typename E, int V>
__device__ __forceinline__ void stv(E* p, const float (&f)[V]) {
  if constexpr (V == 1)
    st(p, f[0]);
  else if constexpr (sizeof(E) == 4)
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  else
    store_bf16<4>(p, f);
}

// The threads that share a row: a warp up to kWarpH elements, else the CTA; V
// elements a thread at once.
constexpr int kWarpH = 1024;
template <bool kWarp, int V>
struct RowGroup {
  static constexpr int kThreads = kWarp ? 32 : kNormThreads;
  static constexpr int kRows = kNormThreads / kThreads;      // of a CTA at once
  static constexpr int kStep = kThreads * V;
  static constexpr int kUnroll = V == 1 ? 4 : 1;       // of the loops along a row
  int tid, h0;
  int64_t first;
  float* red;
  __device__ __forceinline__ explicit RowGroup(float* shared)
      : tid(threadIdx.x % kThreads),
        h0(tid * V),
        first(static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kThreads),
        red(shared) {}
  __device__ __forceinline__ float sum(float v) const {
    if (!kWarp) return cta_sum(v, red);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
};

// A warp or a CTA per row, three passes over it (the later two from L1/L2):
// lengths that are no multiple of eight, and very long rows. 16384 x 333: 20 us
// (a CTA per row: 63), 4096 x 4095: 84, 4096 x 10236: 103 (single elements: 250),
// bound by the latency of the three passes.
template <typename ST, typename WT, bool kWarp, int V>
__global__ void __launch_bounds__(kNormThreads, V == 1 ? 6 : 8)
    norm_rows_kernel(NormParams p, ST* out, __nv_bfloat16* __restrict__ n, float* rstd_y,
                     float* rstd_out) {
  using Group = RowGroup<kWarp, V>;
  __shared__ float red[kNormThreads / 32];
  const Group w(red);
  for (int64_t t = w.first; t < p.T; t += static_cast<int64_t>(gridDim.x) * w.kRows) {
    const int64_t at = t * p.H;
    float ry = 1.0f;
    if (p.w_post) {
      float s = 0.0f;
#pragma unroll(Group::kUnroll)
      for (int h = w.h0; h < p.H; h += w.kStep) {
        float y[V];
        ldv<__nv_bfloat16>(p.y, at + h, y);
#pragma unroll
        for (int i = 0; i < V; ++i) s = fmaf(y[i], y[i], s);
      }
      ry = 1.0f / sqrtf(w.sum(s) * p.inv_h + p.eps);
      if (w.tid == 0 && rstd_y) rstd_y[t] = ry;
    }
    const int64_t gat = p.gate ? t / p.gate_span * p.H : 0;
    auto row = [&](int h, float (&o)[V]) {
      ldv<ST>(p.x, at + h, o);
      if (!p.y) return;
      float z[V], f[V];
      ldv<__nv_bfloat16>(p.y, at + h, z);
      if (p.w_post) {
        ldv<WT>(p.w_post, h, f);
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = z[i] * ry * f[i];
      }
      if (p.gate) {
        ldv<WT>(p.gate, gat + h, f);
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] *= f[i];
      }
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = fmaf(p.a, o[i], p.b * z[i]);
    };
    float ro = 1.0f;
    if (p.w_next) {
      float s = 0.0f;
#pragma unroll(Group::kUnroll)
      for (int h = w.h0; h < p.H; h += w.kStep) {
        float o[V];
        row(h, o);
#pragma unroll
        for (int i = 0; i < V; ++i) s = fmaf(o[i], o[i], s);
      }
      ro = 1.0f / sqrtf(w.sum(s) * p.inv_h + p.eps);
      if (w.tid == 0 && rstd_out) rstd_out[t] = ro;
    }
#pragma unroll(Group::kUnroll)
    for (int h = w.h0; h < p.H; h += w.kStep) {
      float o[V], f[V];
      row(h, o);                                   // before out, which may be x, is written
      if (out) stv<ST>(out + at + h, o);
      if (p.w_next) {
        ldv<WT>(p.w_next, h, f);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] *= o[i] * ro;
        stv<__nv_bfloat16>(n + at + h, f);
      }
    }
  }
}

// D_t at the columns from h, from the row's mean c = m(q * o).
template <typename ST, typename WT, int V>
__device__ __forceinline__ void total_grad(const NormParams& p, int64_t at, int h, float ro,
                                           float c, float (&d)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) d[i] = 0.0f;
  if (p.x) ldv<ST>(p.x, at + h, d);
  if (p.d_n) {
    float q[V], f[V], o[V];
    ldv<__nv_bfloat16>(p.d_n, at + h, q);
    ldv<WT>(p.w_next, h, f);
    ldv<ST>(p.out, at + h, o);
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = fmaf(ro, q[i] * f[i] - o[i] * ro * c, d[i]);
  }
}

// A warp or a CTA per row. kMean: the row's mean c, for the column sums that follow;
// else dx and dy from it. Two launches around the column sums, because these
// read d_out and dx may be d_out itself. The three together: 16384 x 333 54 us
// (a CTA per row: 100), 4096 x 10240 296 us (single elements: 630), of which the
// four readings of the rows are the most.
template <typename ST, typename WT, bool kMean, bool kWarp, int V>
__global__ void __launch_bounds__(kNormThreads, V == 1 ? 5 : 1)
    norm_rows_backward_kernel(NormParams p, ST* dx, __nv_bfloat16* __restrict__ dy,
                              float* __restrict__ c_of) {
  using Group = RowGroup<kWarp, V>;
  __shared__ float red[kNormThreads / 32];
  const Group w(red);
  for (int64_t t = w.first; t < p.T; t += static_cast<int64_t>(gridDim.x) * w.kRows) {
    const int64_t at = t * p.H;
    const float ro = p.d_n ? p.rstd_out[t] : 0.0f;
    if (kMean) {
      float s = 0.0f;
      if (p.d_n)
#pragma unroll(Group::kUnroll)
        for (int h = w.h0; h < p.H; h += w.kStep) {
          float q[V], f[V], o[V];
          ldv<__nv_bfloat16>(p.d_n, at + h, q);
          ldv<WT>(p.w_next, h, f);
          ldv<ST>(p.out, at + h, o);
#pragma unroll
          for (int i = 0; i < V; ++i) s = fmaf(q[i] * f[i], o[i] * ro, s);
        }
      s = w.sum(s);
      if (w.tid == 0) c_of[t] = s * p.inv_h;
      continue;
    }
    const float c = c_of[t];
    const int64_t gat = p.gate ? t / p.gate_span * p.H : 0;
    const float ry = p.y && p.w_post ? p.rstd_y[t] : 1.0f;
    auto grad_z = [&](int h, float (&q)[V]) {      // of the normalised y, times w_post, from D
      float f[V];
#pragma unroll
      for (int i = 0; i < V; ++i) q[i] *= p.b;
      if (p.gate) {
        ldv<WT>(p.gate, gat + h, f);
#pragma unroll
        for (int i = 0; i < V; ++i) q[i] *= f[i];
      }
      if (p.w_post) {
        ldv<WT>(p.w_post, h, f);
#pragma unroll
        for (int i = 0; i < V; ++i) q[i] *= f[i];
      }
    };
    float m = 0.0f;
    if (p.y && p.w_post) {
      float s = 0.0f;
#pragma unroll(Group::kUnroll)
      for (int h = w.h0; h < p.H; h += w.kStep) {
        float q[V], y[V];
        ldv<__nv_bfloat16>(p.y, at + h, y);
        total_grad<ST, WT>(p, at, h, ro, c, q);
        grad_z(h, q);
#pragma unroll
        for (int i = 0; i < V; ++i) s = fmaf(q[i], y[i] * ry, s);
      }
      m = w.sum(s) * p.inv_h;
    }
#pragma unroll(Group::kUnroll)
    for (int h = w.h0; h < p.H; h += w.kStep) {
      float d[V];
      total_grad<ST, WT>(p, at, h, ro, c, d);
      if (p.y) {
        float q[V], y[V];
#pragma unroll
        for (int i = 0; i < V; ++i) q[i] = d[i];
        grad_z(h, q);
        if (p.w_post) {
          ldv<__nv_bfloat16>(p.y, at + h, y);
#pragma unroll
          for (int i = 0; i < V; ++i) q[i] = ry * (q[i] - y[i] * ry * m);
        }
        stv<__nv_bfloat16>(dy + at + h, q);
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] *= p.a;
      }
      stv<ST>(dx + at + h, d);                     // last: dx may be d_out
    }
  }
}

// Column sums of a strip of rows (blockIdx.y), V columns per thread: dw_next
// and dw_post into part[strip], and S = sum D yh of every gate row: straight
// to dgate where the strip holds all of the row's tokens, else into one of
// the strip's two pieces (0: the row began in an earlier strip, 1: in this
// one). All without b, and with one gate row without it, as the fast kernel.
template <typename ST, typename WT, int V>
__global__ void __launch_bounds__(128)
    norm_cols_backward_kernel(NormParams p, const float* __restrict__ c_of,
                              float* __restrict__ part_post, float* __restrict__ part_next,
                              float* __restrict__ part_gate, int one_gate,
                              float* __restrict__ dgate, int accumulate) {
  const int h = (blockIdx.x * 128 + threadIdx.x) * V;
  if (h >= p.H) return;
  const int64_t strip = blockIdx.y;
  const int64_t lo = strip_row(p.T, gridDim.y, strip), hi = strip_row(p.T, gridDim.y, strip + 1);
  float sum_post[V] = {}, sum_next[V] = {};
  const bool many = p.gate && !one_gate;
  // the gate row of the token, and the token after its last one
  int64_t r = many ? lo / p.gate_span : 0, end = many ? (r + 1) * p.gate_span : hi;
  for (int64_t t0 = lo; t0 < hi;) {
    const int64_t stop = min(hi, end);
    float s[V] = {};
#pragma unroll 4
    for (int64_t t = t0; t < stop; ++t) {
      const float ro = p.d_n ? p.rstd_out[t] : 0.0f;
      if (p.y) {
        const float ry = p.w_post ? p.rstd_y[t] : 1.0f;
        float d[V], y[V];
        ldv<__nv_bfloat16>(p.y, t * p.H + h, y);
        total_grad<ST, WT>(p, t * p.H, h, ro, c_of[t], d);
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = fmaf(d[i], y[i] * ry, s[i]);
      }
      if (p.d_n) {
        float q[V], o[V];
        ldv<__nv_bfloat16>(p.d_n, t * p.H + h, q);
        ldv<ST>(p.out, t * p.H + h, o);
#pragma unroll
        for (int i = 0; i < V; ++i) sum_next[i] = fmaf(q[i], o[i] * ro, sum_next[i]);
      }
    }
    if (many) {
      float g[V];
      ldv<WT>(p.gate, r * p.H + h, g);
#pragma unroll
      for (int i = 0; i < V; ++i) sum_post[i] = fmaf(g[i], s[i], sum_post[i]);
      const int64_t first = end - p.gate_span;
      if (first >= lo && end <= hi) {
        float* to = dgate + r * p.H + h;
        float old[V] = {}, wp[V];
#pragma unroll
        for (int i = 0; i < V; ++i) wp[i] = 1.0f;
        if (accumulate) ldv<float>(to, 0, old);
        if (p.w_post) ldv<WT>(p.w_post, h, wp);
#pragma unroll
        for (int i = 0; i < V; ++i) old[i] += s[i] * wp[i] * p.b;
        stv<float>(to, old);
      } else {
        stv<float>(part_gate + (strip * 2 + (first >= lo)) * p.H + h, s);
      }
      ++r;
      end += p.gate_span;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) sum_post[i] += s[i];
    }
    t0 = stop;
  }
  if (part_post) stv<float>(part_post + strip * p.H + h, sum_post);
  if (part_next) stv<float>(part_next + strip * p.H + h, sum_next);
}

// The partial sums, in order: 128 columns a CTA, its warps taking the parts in
// turn. blockIdx.y 0: dw_post, 1: dw_next, beyond: a gate row, from the pieces of
// the strips that share it. Bound by latency: 5 us, of which two are hidden by
// its launch while the last rows are worked on.
struct FinishParams {
  const float *part_post, *part_next, *part_gate;
  float *dw_post, *dw_next, *dgate;
  const void *w_post, *gate;           // factors of dgate and (one gate row) of dw_post
  int64_t T, gate_span, gate_rows;
  int H, parts, strips, one_gate, accumulate, weights_f32;
  float b;
};

// Gate rows, or strips' ends, that the kernel looks at.
__host__ __device__ __forceinline__ int64_t finish_gates(const FinishParams& p) {
  if (!p.dgate) return 0;
  return !p.one_gate && p.strips > 0 && p.strips - 1 < p.gate_rows ? p.strips - 1 : p.gate_rows;
}

__global__ void __launch_bounds__(256) norm_finish_kernel(const __grid_constant__ FinishParams p) {
  constexpr int kWarps = 8, kLoads = 10;
  __shared__ float4 sh[kWarps][32];
  const int lane = lane_id(), w = threadIdx.x >> 5;
  const int h = blockIdx.x * 128 + lane * 4;       // the lane's four columns
  const bool vec = p.H % 4 == 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // one gate row: its sum is the one behind dw_post. Several: those that lie
  // across strips (the others are written by their strips), found from the rows
  // or, if there are fewer, from the strips' ends: a row counts at its first one
  const bool across = !p.one_gate && p.strips > 0, by_end = across && p.strips - 1 < p.gate_rows;
  for (int64_t what = blockIdx.y; what < 2 + finish_gates(p); what += gridDim.y) {
    const bool of_gate = what >= 2;
    if (!of_gate && !(what == 0 ? p.dw_post : p.dw_next)) continue;
    const bool pieces = of_gate && !p.one_gate;
    const float* part = what == 1 ? p.part_next : pieces ? p.part_gate : p.part_post;
    int64_t r = what - 2;
    int i0 = 0, i1 = p.parts;
    if (of_gate && across) {
      const int64_t end = by_end ? strip_row(p.T, p.strips, what - 1) : 0;
      if (by_end) r = (end - 1) / p.gate_span;
      i0 = static_cast<int>(strip_of(p.T, p.strips, r * p.gate_span));
      if (by_end && i0 != what - 2) continue;
      i1 = static_cast<int>(strip_of(p.T, p.strips, (r + 1) * p.gate_span - 1)) + 1;
      if (i1 - i0 == 1) continue;
    }
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i = i0 + w; i < i1; i += kWarps * kLoads) {
      float4 f[kLoads];                            // as many loads on their way
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const int j = i + kWarps * u;
        const float* at = part + static_cast<int64_t>(pieces ? j * 2 + (j == i0) : j) * p.H + h;
        f[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (j < i1 && h < p.H) {
          if (vec) {
            f[u] = *reinterpret_cast<const float4*>(at);
          } else {
            f[u].x = at[0];
            if (h + 1 < p.H) f[u].y = at[1];
            if (h + 2 < p.H) f[u].z = at[2];
            if (h + 3 < p.H) f[u].w = at[3];
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        s.x += f[u].x;
        s.y += f[u].y;
        s.z += f[u].z;
        s.w += f[u].w;
      }
    }
    __syncthreads();
    sh[w][lane] = s;
    __syncthreads();
    const int c = blockIdx.x * 128 + threadIdx.x;
    if (threadIdx.x < 128 && c < p.H) {
      const float* all = reinterpret_cast<const float*>(sh);
      float z = 0.0f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) z += all[i * 128 + threadIdx.x];
      float* to = (of_gate ? p.dgate + r * p.H : what == 0 ? p.dw_post : p.dw_next) + c;
      if (what != 1) z *= p.b;
      if (of_gate && p.w_post) z *= weight_at(p.w_post, p.weights_f32, c);
      if (what == 0 && p.one_gate) z *= weight_at(p.gate, p.weights_f32, c);
      *to = p.accumulate ? *to + z : z;
    }
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

moe_status norm_config_of(moe_norm_config* c, const moe_norm_config* cfg, int64_t T, int H) {
  moe_norm_config_init(c);
  if (cfg) *c = *cfg;
  if (T < 0 || H < 1 || T > kMaxTokens) return MOE_ERR_INVALID_ARG;
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

// Bytes of the gate in a row of the ring: a token's own.
int token_gate_bytes(const NormParams& p) {
  return p.gate && p.gate_span == 1 && p.T > 1 ? p.H * (p.weights_f32 ? 4 : 2) : 0;
}

// Threads of a forward CTA that hold a row in V vectors each (0: too long).
int forward_threads(int H, int W, int V) {
  const int threads = (H / W + 32 * V - 1) / (32 * V) * 32;
  return threads <= 1024 ? threads : 0;
}

// f(kWarp, V) of the kernels that take any length of a row.
template <typename F>
void with_rows_of(int H, F f) {
  using std::integral_constant;
  if (H <= kWarpH && H % 4 == 0)
    f(std::true_type(), integral_constant<int, 4>());
  else if (H <= kWarpH)
    f(std::true_type(), integral_constant<int, 1>());
  else if (H % 4 == 0)
    f(std::false_type(), integral_constant<int, 4>());
  else
    f(std::false_type(), integral_constant<int, 1>());
}

template <typename ST, typename WT>
cudaError_t forward(const NormParams& p, void* out, void* n, float* rstd_y, float* rstd_out,
                    cudaStream_t s) {
  // up to one row an SM the kernel without a ring is shorter (152 x 7168: 3.4
  // against 3.7 us); beyond, rows through shared memory (300 x 7168: 5.2 against
  // 5.8, 4096 x 4096 in bf16: 23.4 against 28.9). Not for every shape between:
  // 300 x 2048 3.5 against 3.0, 600 x 7168 7.8 against 6.9, 4096 x 4096 with a
  // float stream 36.9 against 35.6
  const int row_bytes = p.H * static_cast<int>(sizeof(ST) + (p.y ? 2 : 0)) + token_gate_bytes(p);
  const RingShape r = ring_shape(p.T, p.H, row_bytes, false, false);
  if (r.groups > 0 && p.T > device_sm_count()) {
    RingOut ro = {};
    ro.stream = out;
    ro.branch = static_cast<__nv_bfloat16*>(n);
    ro.rstd_y = rstd_y;
    ro.rstd_out = rstd_out;
    return launch_norm_ring(p, r, ro, sizeof(ST) == 4, false, row_bytes, s);
  }
  constexpr int W = sizeof(ST) == 4 ? 4 : 8;
  ST* o = static_cast<ST*>(out);
  __nv_bfloat16* nn = static_cast<__nv_bfloat16*>(n);
  if (p.H % 8 == 0 && forward_threads(p.H, W, 4)) {
    // few rows: every vector a thread of its own, for the shortest way through a
    // row (1 x 7168: 3.1 us, with two vectors a thread 3.5, with four 5.0); many:
    // more loads in flight a thread (4096 x 16384: 115 with four, 135 with two)
    const int nvec = p.H / W;
    int V = p.T <= device_sm_count() * 2 || nvec < 256 ? 1 : nvec < 512 ? 2 : 4;
    while (!forward_threads(p.H, W, V)) V *= 2;
    auto* kernel = V == 1   ? norm_forward_kernel<ST, WT, 1>
                   : V == 2 ? norm_forward_kernel<ST, WT, 2>
                            : norm_forward_kernel<ST, WT, 4>;
    const int64_t most = 1 << 30;
    kernel<<<static_cast<unsigned>(p.T < most ? p.T : most), forward_threads(p.H, W, V), 0, s>>>(
        p, o, nn, rstd_y, rstd_out);
    return cudaGetLastError();
  }
  with_rows_of(p.H, [&](auto warp, auto width) {
    constexpr bool kWarp = decltype(warp)::value;
    constexpr int V = decltype(width)::value;
    norm_rows_kernel<ST, WT, kWarp, V>
        <<<rows_grid(kWarp ? (p.T + 7) / 8 : p.T), kNormThreads, 0, s>>>(p, o, nn, rstd_y, rstd_out);
  });
  return cudaGetLastError();
}

struct NormGrads {
  void *dx, *dy;
  float *dw_post, *dgate, *dw_next;
  int64_t gate_rows;
  int accumulate;
};

int row_bytes_of(const NormParams& p, int stream_size) {
  return p.H * ((p.x ? stream_size : 0) + (p.d_n ? stream_size + 2 : 0) + (p.y ? 2 : 0)) +
         token_gate_bytes(p);
}

template <typename ST, typename WT>
cudaError_t backward(const NormParams& p, const NormGrads& g, void* ws, cudaStream_t s) {
  const bool one_gate = p.gate && p.T > 0 && p.gate_span == p.T;
  const int row_bytes = row_bytes_of(p, sizeof(ST));
  RingShape b = ring_shape(p.T, p.H, row_bytes, true,
                           p.gate && !one_gate && p.gate_span > 1);
  if (b.groups == 0) {
    const int64_t most = static_cast<int64_t>(device_sm_count()) * 2;
    b.strips = b.ctas = static_cast<int>(p.T < most ? p.T : most);
  }
  float* c_of = static_cast<float*>(ws);
  float* part = c_of + (p.T + 63) / 64 * 64;
  const int64_t one = static_cast<int64_t>(b.ctas) * p.H;
  float* part_post = (g.dw_post || one_gate) && b.strips ? part : nullptr;
  float* part_next = g.dw_next && b.strips ? part + one : nullptr;
  float* part_gate = part + 2 * one;
  cudaError_t e = cudaSuccess;
  if (b.groups > 0) {
    RingOut o = {};
    o.stream = g.dx;
    o.branch = static_cast<__nv_bfloat16*>(g.dy);
    o.dgate = g.dgate;
    o.part_post = part_post;
    o.part_next = part_next;
    o.part_gate = part_gate;
    o.accumulate = g.accumulate;
    e = launch_norm_ring(p, b, o, sizeof(ST) == 4, true, row_bytes, s);
  } else if (p.T > 0) {
    ST* dx = static_cast<ST*>(g.dx);
    __nv_bfloat16* dy = static_cast<__nv_bfloat16*>(g.dy);
    with_rows_of(p.H, [&](auto warp, auto width) {
      constexpr bool kWarp = decltype(warp)::value;
      constexpr int V = decltype(width)::value;
      const int rows = rows_grid(kWarp ? (p.T + 7) / 8 : p.T);
      norm_rows_backward_kernel<ST, WT, true, kWarp, V><<<rows, kNormThreads, 0, s>>>(p, dx, dy,
                                                                                    c_of);
      if (part_post || part_next || g.dgate) {
        const unsigned cols = static_cast<unsigned>((p.H + 128 * V - 1) / (128 * V));
        norm_cols_backward_kernel<ST, WT, V><<<dim3(cols, b.strips), 128, 0, s>>>(
            p, c_of, part_post, part_next, part_gate, one_gate, g.dgate, g.accumulate);
      }
      norm_rows_backward_kernel<ST, WT, false, kWarp, V><<<rows, kNormThreads, 0, s>>>(p, dx, dy,
                                                                                     c_of);
    });
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || !(g.dw_post || g.dw_next || g.dgate)) return e;
  FinishParams f = {part_post, part_next,   part_gate, g.dw_post, g.dw_next, g.dgate,
                    p.w_post,  p.gate,      p.T,       p.gate_span, g.dgate ? g.gate_rows : 0,
                    p.H,       b.ctas,      b.strips,  one_gate,  g.accumulate, sizeof(WT) == 4,
                    p.b};
  // a row for each token (and with fewer tokens than strips, none across them)
  if (p.T > 0 && p.gate_span == 1 && !one_gate) f.dgate = nullptr;
  const int64_t want = 2 + finish_gates(f);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  // its CTAs may come up while the last rows are still worked on; they wait
  // for the whole grid before they read
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>((p.H + 127) / 128),
                     static_cast<unsigned>(want < 1024 ? want : 1024));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_finish_kernel, f);
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
  p.weights_f32 = c.weight_type == MOE_TYPE_F32;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool sf = c.stream_type == MOE_TYPE_F32, wf = c.weight_type == MOE_TYPE_F32;
  auto* run = sf ? (wf ? forward<float, float> : forward<float, __nv_bfloat16>)
                 : (wf ? forward<__nv_bfloat16, float> : forward<__nv_bfloat16, __nv_bfloat16>);
  return run(p, out, n, rstd_y, rstd_out, st) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_norm_residual_backward_workspace_size(int64_t T, int H, int64_t gate_rows) {
  if (T < 0 || H < 1 || H > kMaxNormH || gate_rows < 0 || T > kMaxTokens)
    return 0;
  // the layout with the most CTAs and strips, whatever a call's tensors are
  const int64_t sms = device_sm_count(), groups = most_ring_groups(H);
  const int64_t ctas = T < 2 * sms ? T : 2 * sms;
  const int64_t most = sms * (groups > 2 ? groups : 2), strips = T < most ? T : most;
  return static_cast<size_t>((T + 63) / 64 * 64) * sizeof(float) +
         2 * static_cast<size_t>(ctas + (gate_rows > 1 ? strips : 0)) * H * sizeof(float) + 256;
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
  p.weights_f32 = c.weight_type == MOE_TYPE_F32;
  const NormGrads g{dx, dy, dw_post, dgate, dw_next, gate_rows, accumulate_dw};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool sf = c.stream_type == MOE_TYPE_F32, wf = c.weight_type == MOE_TYPE_F32;
  auto* run = sf ? (wf ? backward<float, float> : backward<float, __nv_bfloat16>)
                 : (wf ? backward<__nv_bfloat16, float> : backward<__nv_bfloat16, __nv_bfloat16>);
  return run(p, g, workspace, st) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
