// norm_ring.cu - the norms around the block for rows of up to 8192 elements:
// forward and backward over strips of rows that bulk copies bring into shared
// memory.
//
// A group of threads (whole warps) walks a strip of consecutive rows, every
// thread with 4 V fixed columns (V vectors of four, so that all accesses are
// coalesced for float and for bf16): V = 2 forward, V = 4 backward, where the
// registers of the pointers and counters would leave too few for the columns
// of a thread with eight. What belongs to a column stays in its registers from
// row to row: the weights, b w_post g as one factor, and the column sums of the
// weight gradients. A row's tensors lie in one stage of the group's ring, which
// its first thread fills with bulk copies up to three rows ahead; each is read
// from HBM once. A CTA has as many groups as its threads hold, one CTA an SM,
// so that short rows too have enough bytes on their way, and the groups'
// column sums are added up in shared memory: the finishing kernel finds one
// row of partial sums an SM.
//
// Bound by HBM, 8 bytes an element forward and 12 backward in bf16 (18 with a
// float stream), where a row's instructions stay below its bytes' time: pairs
// of columns go through the packed float instructions (fma.rn.f32x2), which
// round each half as the single ones do.
#include "norm.cuh"

namespace moe {

int* device_error_word();

namespace {

constexpr int kSharedBytes = 216 * 1024;  // of the rings, and what lies behind them
constexpr int kMaxStages = 4;
constexpr int kForwardVecs = 2, kBackwardVecs = 4;
constexpr int ring_threads(int V) { return 2048 / V; }

struct RingParams {
  NormParams n;
  RingOut o;
  RingShape r;
  int row_bytes;
  int* err;
};

// ------------------------------------------------------------------ pairs of floats

typedef unsigned long long Pair;

__device__ __forceinline__ Pair pair(float lo, float hi) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
  return p;
}
__device__ __forceinline__ Pair pair(float v) { return pair(v, v); }
__device__ __forceinline__ float2 halves(Pair p) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
  return f;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float sum2(Pair a) {
  const float2 f = halves(a);
  return f.x + f.y;
}

struct Four {
  Pair p[2];
};

__device__ __forceinline__ Pair widen(unsigned q) {
  return pair(__uint_as_float(q << 16), __uint_as_float(q & 0xffff0000u));
}
__device__ __forceinline__ Four widen(uint2 q) { return Four{{widen(q.x), widen(q.y)}}; }

// Four elements in shared memory, and to global memory.
template <typename T>
__device__ __forceinline__ Four get4(const unsigned char* p) {
  if constexpr (sizeof(T) == 4) {
    const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(p);
    return Four{{q.x, q.y}};
  } else {
    return widen(*reinterpret_cast<const uint2*>(p));
  }
}
template <typename T>
__device__ __forceinline__ void put4(unsigned char* p, const Four& v) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(v.p[0], v.p[1]);
  } else {
    const float2 a = halves(v.p[0]), b = halves(v.p[1]);
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(b.x, b.y));
  }
}

// ------------------------------------------------------------------ groups and rings

// The sum of v over a group to each of its threads; warps: of the group. The
// barrier in it also tells that the group has read what it had to.
template <int kWarps>
__device__ __forceinline__ float group_sum(float v, float* red, int warp, int bar, int group) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (group == 32) return v;
  if (lane_id() == 0) red[warp] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(group) : "memory");
  const int at = lane_id() & (kWarps - 1);
  v = at < (group >> 5) ? red[at] : 0.0f;
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void group_barrier(int bar, int group) {
  if (group == 32)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(group) : "memory");
}

// A group's place in its CTA, its strip and its ring.
template <int V>
struct Walk {
  int g, tid, warp, H;
  int64_t lo, hi;
  unsigned char* ring;
  uint32_t full;               // mbarriers of its stages
  int col0, step;              // columns col0 + v step .. + 3 are the thread's
  bool has[V];
};

// kFull: every thread has all its columns.
template <int V, bool kFull>
__device__ __forceinline__ Walk<V> walk_of(const RingParams& p, unsigned char* ring_all,
                                           uint64_t (*full_all)[kMaxStages], int* abort_wait) {
  Walk<V> w;
  w.g = threadIdx.x / p.r.group;
  w.tid = threadIdx.x - w.g * p.r.group;
  w.warp = w.tid >> 5;
  w.H = p.n.H;
  const int strip = blockIdx.x * p.r.groups + w.g;
  w.lo = w.hi = 0;
  if (strip < p.r.strips) {
    w.lo = strip_row(p.n.T, p.r.strips, strip);
    w.hi = strip_row(p.n.T, p.r.strips, strip + 1);
  }
  w.ring = ring_all + static_cast<size_t>(w.g) * p.r.stages * p.row_bytes;
  w.full = smem_u32(&full_all[w.g][0]);
  w.col0 = 4 * w.tid;
  w.step = 4 * p.r.group;
#pragma unroll
  for (int v = 0; v < V; ++v) w.has[v] = kFull || w.col0 + v * w.step < w.H;
  if (threadIdx.x == 0) *abort_wait = 0;
  if (w.tid == 0) {
    for (int i = 0; i < p.r.stages; ++i) mbar_init(w.full + 8 * i, 1);
    fence_mbar_init();
  }
  __syncthreads();
  return w;
}

// f[columns] *= weights[row + columns]
template <int V>
__device__ __forceinline__ void times(const RingParams& p, const Walk<V>& w, const void* weights,
                                      int64_t row, Pair (&f)[2 * V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (!w.has[v]) continue;
    const int64_t at = row + w.col0 + v * w.step;
    Four m;
    if (p.n.weights_f32) {
      const float4 q = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(weights) + at));
      m = Four{{pair(q.x, q.y), pair(q.z, q.w)}};
    } else {
      m = widen(__ldg(
          reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(weights) + at)));
    }
    f[2 * v] = mul2(f[2 * v], m.p[0]);
    f[2 * v + 1] = mul2(f[2 * v + 1], m.p[1]);
  }
}

// Waits for a stage. No wait as long as the limit is legitimate: it is
// reported, and the waits after it are given up at once.
template <int V>
__device__ __forceinline__ void wait_stage(const RingParams& p, const Walk<V>& w, int stage,
                                           int parity, unsigned long long* limit,
                                           int* abort_wait) {
  if (!mbar_wait(w.full + 8 * stage, parity, *limit, abort_wait)) {
    report_error(p.err, kErrTimeout);
    *limit = 0;
  }
}

// ------------------------------------------------------------------ forward

template <typename ST, bool kMany, bool kFull>
__global__ void __launch_bounds__(ring_threads(kForwardVecs), 1)
    norm_ring_kernel(const __grid_constant__ RingParams p) {
  constexpr int V = kForwardVecs, kWarps = ring_threads(V) / 32;
  extern __shared__ __align__(128) unsigned char ring_all[];
  __shared__ float red_all[kMaxRingGroups][4][kWarps];
  __shared__ __align__(8) uint64_t full_all[kMaxRingGroups][kMaxStages];
  __shared__ int abort_wait;
  const Walk<V> w = walk_of<V, kFull>(p, ring_all, full_all, &abort_wait);
  const NormParams& q = p.n;
  const bool branch = q.y, post = q.w_post, next = q.w_next;
  constexpr int kSize = sizeof(ST);
  const int wide = w.H * kSize, half = w.H * 2;
  auto issue = [&](int64_t t, int stage) {
    const uint32_t bar = w.full + 8 * stage, to = smem_u32(w.ring) + stage * p.row_bytes;
    mbar_arrive_expect_tx(bar, p.row_bytes);
    bulk_copy_g2s(to, static_cast<const ST*>(q.x) + t * w.H, wide, bar);
    if (branch) bulk_copy_g2s(to + wide, q.y + t * w.H, half, bar);
  };
  if (w.tid == 0)
    for (int i = 0; i < p.r.stages && w.lo + i < w.hi; ++i) issue(w.lo + i, i);

  Pair gw[2 * V], wn[2 * V];
#pragma unroll
  for (int i = 0; i < 2 * V; ++i) {
    gw[i] = pair(q.b);
    wn[i] = pair(1.0f);
  }
  if (next) times(p, w, q.w_next, 0, wn);
  if (!kMany) {
    if (post) times(p, w, q.w_post, 0, gw);
    if (q.gate) times(p, w, q.gate, 0, gw);
  }
  int64_t gate_row = -1, gate_end = w.lo;
  if (kMany && w.lo < w.hi) gate_row = w.lo / q.gate_span - 1;
  unsigned long long limit = kDefaultWaitNs;
  int stage = 0, parity = 0, odd = 0;
  unsigned char* to_out = static_cast<unsigned char*>(p.o.stream) + (w.lo * w.H + w.col0) * kSize;
  unsigned char* to_n = reinterpret_cast<unsigned char*>(p.o.branch) + (w.lo * w.H + w.col0) * 2;
  const unsigned char* row_x = w.ring + w.col0 * kSize;
  const unsigned char* row_y = w.ring + wide + w.col0 * 2;
  const Pair a = pair(q.a);
  for (int64_t t = w.lo; t < w.hi; ++t, to_out += wide, to_n += half) {
    if (kMany && t == gate_end) {
      ++gate_row;
      gate_end = (gate_row + 1) * q.gate_span;
#pragma unroll
      for (int i = 0; i < 2 * V; ++i) gw[i] = pair(q.b);
      if (post) times(p, w, q.w_post, 0, gw);
      times(p, w, q.gate, gate_row * w.H, gw);
    }
    wait_stage(p, w, stage, parity, &limit, &abort_wait);
    const int base = stage * p.row_bytes;
    Four x[V], y[V];
    Pair s = pair(0.0f);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!w.has[v]) continue;
      x[v] = get4<ST>(row_x + (base + v * w.step * kSize));
      if (branch) {
        y[v] = get4<__nv_bfloat16>(row_y + (base + v * w.step * 2));
        s = fma2(y[v].p[0], y[v].p[0], s);
        s = fma2(y[v].p[1], y[v].p[1], s);
      }
    }
    float ry = 1.0f;
    if (post) {
      const float m = group_sum<kWarps>(sum2(s), red_all[w.g][odd], w.warp, w.g + 1, p.r.group);
      ry = 1.0f / sqrtf(fmaf(m, q.inv_h, q.eps));
      if (w.tid == 0 && p.o.rstd_y) p.o.rstd_y[t] = ry;
    }
    if (!post || p.r.group == 32) group_barrier(w.g + 1, p.r.group);
    // every thread has the row in registers: its stage takes another
    if (w.tid == 0 && t + p.r.stages < w.hi) issue(t + p.r.stages, stage);
    s = pair(0.0f);
    const Pair r = pair(ry);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!w.has[v]) continue;
      if (branch) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          x[v].p[h] = fma2(mul2(y[v].p[h], r), gw[2 * v + h], mul2(a, x[v].p[h]));
        put4<ST>(to_out + v * w.step * kSize, x[v]);
      }
      s = fma2(x[v].p[0], x[v].p[0], s);
      s = fma2(x[v].p[1], x[v].p[1], s);
    }
    if (next) {
      const float m =
          group_sum<kWarps>(sum2(s), red_all[w.g][2 + odd], w.warp, w.g + 1, p.r.group);
      const float ro = 1.0f / sqrtf(fmaf(m, q.inv_h, q.eps));
      if (w.tid == 0 && p.o.rstd_out) p.o.rstd_out[t] = ro;
      const Pair o = pair(ro);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (!w.has[v]) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) x[v].p[h] = mul2(mul2(x[v].p[h], o), wn[2 * v + h]);
        put4<__nv_bfloat16>(to_n + v * w.step * 2, x[v]);
      }
    }
    odd ^= 1;
    if (++stage == p.r.stages) {
      stage = 0;
      parity ^= 1;
    }
  }
}

// ------------------------------------------------------------------ backward

// With r = rstd_out, t = d_n out: dw_next += r t,
//   D = d_out + r (d_n w_next - out (r^2 m(t w_next)));
// with r = rstd_y, u = D y, gw = b g w_post: S += r u (dw_post = b g S and
// dgate = b w_post S for one gate row; kMany keeps S for a row's tokens, and
// its sum over rows times g in shared memory),
//   dy = r (gw D - y (r^2 m(u gw))).
// No product of three r: a row of 1e15 stays in float's range.
template <typename ST, bool kMany, bool kFull>
__global__ void __launch_bounds__(ring_threads(kBackwardVecs), 1)
    norm_ring_backward_kernel(const __grid_constant__ RingParams p) {
  constexpr int V = kBackwardVecs, kWarps = ring_threads(V) / 32;
  extern __shared__ __align__(128) unsigned char ring_all[];
  __shared__ float red_all[kMaxRingGroups][4][kWarps];
  __shared__ __align__(8) uint64_t full_all[kMaxRingGroups][kMaxStages];
  __shared__ int abort_wait;
  const Walk<V> w = walk_of<V, kFull>(p, ring_all, full_all, &abort_wait);
  const NormParams& q = p.n;
  const bool branch = q.y, post = q.w_post, next = q.d_n, has_d = q.x;
  constexpr int kSize = sizeof(ST);
  // a stage: d_out, out, y, d_n, as far as there are any
  const int wide = w.H * kSize, half = w.H * 2;
  const int at_out = has_d ? wide : 0, at_y = at_out + (next ? wide : 0),
            at_dn = at_y + (branch ? half : 0);
  auto issue = [&](int64_t t, int stage) {
    const uint32_t bar = w.full + 8 * stage, to = smem_u32(w.ring) + stage * p.row_bytes;
    const int64_t at = t * w.H;
    mbar_arrive_expect_tx(bar, p.row_bytes);
    if (has_d) bulk_copy_g2s(to, static_cast<const ST*>(q.x) + at, wide, bar);
    if (next) bulk_copy_g2s(to + at_out, static_cast<const ST*>(q.out) + at, wide, bar);
    if (branch) bulk_copy_g2s(to + at_y, q.y + at, half, bar);
    if (next) bulk_copy_g2s(to + at_dn, q.d_n + at, half, bar);
  };
  if (w.tid == 0)
    for (int i = 0; i < p.r.stages && w.lo + i < w.hi; ++i) issue(w.lo + i, i);

  // kMany: the group's sum of g S, behind the rings
  float* sum_w = reinterpret_cast<float*>(ring_all + static_cast<size_t>(p.r.groups) * p.r.stages *
                                                         p.row_bytes) +
                 w.g * w.H + w.col0;
  Pair gw[2 * V], wn[2 * V], sum_s[2 * V], sum_n[2 * V];
#pragma unroll
  for (int i = 0; i < 2 * V; ++i) {
    gw[i] = pair(q.b);
    wn[i] = pair(1.0f);
    sum_s[i] = sum_n[i] = pair(0.0f);
  }
  if (next) times(p, w, q.w_next, 0, wn);
  if (kMany) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (w.has[v])
        *reinterpret_cast<float4*>(sum_w + v * w.step) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  } else {
    if (post) times(p, w, q.w_post, 0, gw);
    if (q.gate) times(p, w, q.gate, 0, gw);
  }
  int64_t gate_row = -1, gate_end = w.lo;
  if (kMany && w.lo < w.hi) gate_row = w.lo / q.gate_span - 1;
  unsigned long long limit = kDefaultWaitNs;
  float next_ro = 0.0f, next_ry = 1.0f;
  if (w.lo < w.hi) {
    if (next) next_ro = q.rstd_out[w.lo];
    if (post) next_ry = q.rstd_y[w.lo];
  }
  int stage = 0, parity = 0, odd = 0;
  unsigned char* to_dx = static_cast<unsigned char*>(p.o.stream) + (w.lo * w.H + w.col0) * kSize;
  unsigned char* to_dy = reinterpret_cast<unsigned char*>(p.o.branch) + (w.lo * w.H + w.col0) * 2;
  const unsigned char* row_wide = w.ring + w.col0 * kSize;
  const unsigned char* row_half = w.ring + w.col0 * 2;
  const Pair a = pair(branch ? q.a : 1.0f);
  for (int64_t t = w.lo; t < w.hi; ++t, to_dx += wide, to_dy += half) {
    const float ro = next_ro, ry = next_ry;
    if (t + 1 < w.hi) {
      if (next) next_ro = q.rstd_out[t + 1];
      if (post) next_ry = q.rstd_y[t + 1];
    }
    if (kMany && t == gate_end) {
      ++gate_row;
      gate_end = (gate_row + 1) * q.gate_span;
#pragma unroll
      for (int i = 0; i < 2 * V; ++i) {
        gw[i] = pair(q.b);
        sum_s[i] = pair(0.0f);
      }
      if (post) times(p, w, q.w_post, 0, gw);
      times(p, w, q.gate, gate_row * w.H, gw);
    }
    wait_stage(p, w, stage, parity, &limit, &abort_wait);
    const int base = stage * p.row_bytes;
    Four d[V];
    if (next) {
      Pair s = pair(0.0f);
      const Pair r = pair(ro);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (!w.has[v]) continue;
        const Four f = get4<__nv_bfloat16>(row_half + (base + at_dn + v * w.step * 2));
        const Four out = get4<ST>(row_wide + (base + at_out + v * w.step * kSize));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const Pair u = mul2(f.p[h], out.p[h]);
          s = fma2(u, wn[2 * v + h], s);
          sum_n[2 * v + h] = fma2(u, r, sum_n[2 * v + h]);
        }
      }
      const float m = group_sum<kWarps>(sum2(s), red_all[w.g][odd], w.warp, w.g + 1, p.r.group);
      const Pair k = pair(-ro * (ro * (m * q.inv_h)));
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (!w.has[v]) continue;
        // read again: shared memory is cheaper here than registers
        const Four f = get4<__nv_bfloat16>(row_half + (base + at_dn + v * w.step * 2));
        const Four out = get4<ST>(row_wide + (base + at_out + v * w.step * kSize));
        Four e = {{0, 0}};
        if (has_d) e = get4<ST>(row_wide + (base + v * w.step * kSize));
#pragma unroll
        for (int h = 0; h < 2; ++h)
          d[v].p[h] = fma2(r, fma2(k, out.p[h], mul2(f.p[h], wn[2 * v + h])), e.p[h]);
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (w.has[v]) d[v] = get4<ST>(row_wide + (base + v * w.step * kSize));
    }
    uint2 y[V];
    Pair s = pair(0.0f);
    const Pair r = pair(ry);
    if (branch) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (!w.has[v]) continue;
        y[v] = *reinterpret_cast<const uint2*>(row_half + (base + at_y + v * w.step * 2));
        const Four f = widen(y[v]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const Pair u = mul2(d[v].p[h], f.p[h]);
          sum_s[2 * v + h] = fma2(u, r, sum_s[2 * v + h]);
          s = fma2(u, gw[2 * v + h], s);
        }
      }
    }
    float m = 0.0f;
    if (post) m = group_sum<kWarps>(sum2(s), red_all[w.g][2 + odd], w.warp, w.g + 1, p.r.group);
    if (!post || p.r.group == 32) group_barrier(w.g + 1, p.r.group);
    // every thread has the row in registers: its stage takes another
    if (w.tid == 0 && t + p.r.stages < w.hi) issue(t + p.r.stages, stage);
    const Pair k = pair(-ry * (ry * (m * q.inv_h)));
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!w.has[v]) continue;
      if (branch) {
        const Four f = widen(y[v]);
        Four g;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          g.p[h] = mul2(gw[2 * v + h], d[v].p[h]);
          if (post) g.p[h] = mul2(r, fma2(k, f.p[h], g.p[h]));
        }
        put4<__nv_bfloat16>(to_dy + v * w.step * 2, g);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) d[v].p[h] = mul2(a, d[v].p[h]);
      put4<ST>(to_dx + v * w.step * kSize, d[v]);
    }
    if (kMany && (t + 1 == gate_end || t + 1 == w.hi)) {
      // S of the gate row: whole to dgate, else a piece (0: begun in an earlier
      // strip, 1: in this one); its share of dw_post stays
      const int64_t first = gate_row * q.gate_span;
      const bool whole = first >= w.lo && t + 1 == gate_end;
      const int64_t strip = static_cast<int64_t>(blockIdx.x) * p.r.groups + w.g;
      float* to = (whole ? p.o.dgate + gate_row * w.H
                         : p.o.part_gate + (strip * 2 + (first >= w.lo)) * w.H) +
                  w.col0;
      Pair f[2 * V];
#pragma unroll
      for (int i = 0; i < 2 * V; ++i) f[i] = sum_s[i];
      times(p, w, q.gate, gate_row * w.H, f);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (!w.has[v]) continue;
        float4* at = reinterpret_cast<float4*>(sum_w + v * w.step);
        const float2 lo = halves(f[2 * v]), hi = halves(f[2 * v + 1]);
        const float4 z = *at;
        *at = make_float4(z.x + lo.x, z.y + lo.y, z.z + hi.x, z.w + hi.y);
      }
#pragma unroll
      for (int i = 0; i < 2 * V; ++i) f[i] = whole ? mul2(pair(q.b), sum_s[i]) : sum_s[i];
      if (whole && post) times(p, w, q.w_post, 0, f);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (!w.has[v]) continue;
        float4* at = reinterpret_cast<float4*>(to + v * w.step);
        const float2 lo = halves(f[2 * v]), hi = halves(f[2 * v + 1]);
        float4 z = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (whole && p.o.accumulate) z = *at;
        *at = make_float4(z.x + lo.x, z.y + lo.y, z.z + hi.x, z.w + hi.y);
      }
    }
    odd ^= 1;
    if (++stage == p.r.stages) {
      stage = 0;
      parity ^= 1;
    }
  }

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // the groups' sums, in order
  auto add_up = [&](const float* all, float* part) {
    __syncthreads();
    for (int h = threadIdx.x; h < w.H; h += blockDim.x) {
      float z = 0.0f;
      for (int i = 0; i < p.r.groups; ++i) z += all[i * w.H + h];
      part[static_cast<int64_t>(blockIdx.x) * w.H + h] = z;
    }
  };
  auto share = [&](const Pair (&sum)[2 * V]) {
    float* all = reinterpret_cast<float*>(ring_all) + w.g * w.H + w.col0;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (w.has[v])
        *reinterpret_cast<ulonglong2*>(all + v * w.step) =
            make_ulonglong2(sum[2 * v], sum[2 * v + 1]);
    return reinterpret_cast<const float*>(ring_all);
  };
  if (p.o.part_post) add_up(kMany ? sum_w - w.g * w.H - w.col0 : share(sum_s), p.o.part_post);
  if (p.o.part_next) add_up(share(sum_n), p.o.part_next);
}

// ------------------------------------------------------------------ launches

// Threads that share a row of H, V vectors of four each; 0: more than a CTA has.
int group_of(int H, int V) {
  const int group = (H + 128 * V - 1) / (128 * V) * 32;
  return H % 8 == 0 && group <= ring_threads(V) ? group : 0;
}

template <typename K>
cudaError_t launch(K* kernel, const RingParams& p, size_t smem, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  kernel<<<p.r.ctas, p.r.groups * p.r.group, smem, st>>>(p);
  return cudaGetLastError();
}

template <typename ST>
cudaError_t launch_of(const RingParams& p, bool backward, bool many, size_t smem, cudaStream_t st) {
  const bool full = p.n.H == 4 * (backward ? kBackwardVecs : kForwardVecs) * p.r.group;
  auto* kernel =
      backward ? (many ? (full ? norm_ring_backward_kernel<ST, true, true>
                               : norm_ring_backward_kernel<ST, true, false>)
                       : (full ? norm_ring_backward_kernel<ST, false, true>
                               : norm_ring_backward_kernel<ST, false, false>))
               : (many ? (full ? norm_ring_kernel<ST, true, true> : norm_ring_kernel<ST, true, false>)
                       : (full ? norm_ring_kernel<ST, false, true>
                               : norm_ring_kernel<ST, false, false>));
  return launch(kernel, p, smem, st);
}

}  // namespace

int most_ring_groups(int H) {
  const int group = group_of(H, kBackwardVecs);
  const int groups = group ? ring_threads(kBackwardVecs) / group : 0;
  return groups < kMaxRingGroups ? groups : kMaxRingGroups;
}

RingShape ring_shape(int64_t T, int H, int row_bytes, bool backward, bool many) {
  RingShape r = {};
  const int V = backward ? kBackwardVecs : kForwardVecs;
  r.group = group_of(H, V);
  r.tail_bytes = backward && many ? H * static_cast<int>(sizeof(float)) : 0;
  if (T == 0 || r.group == 0 || 2 * row_bytes + r.tail_bytes > kSharedBytes) return r;
  const int sms = device_sm_count();
  // as many groups as there are threads and two stages of memory for, unless
  // the rows run out first
  r.groups = ring_threads(V) / r.group;
  if (r.groups > kMaxRingGroups) r.groups = kMaxRingGroups;
  while (r.groups > 1 && (r.groups * (2 * row_bytes + r.tail_bytes) > kSharedBytes ||
                          T <= static_cast<int64_t>(sms) * (r.groups - 1)))
    --r.groups;
  r.stages = (kSharedBytes / r.groups - r.tail_bytes) / row_bytes;
  if (r.stages > kMaxStages) r.stages = kMaxStages;
  const int64_t most = static_cast<int64_t>(sms) * r.groups;
  r.strips = static_cast<int>(T < most ? T : most);
  r.ctas = (r.strips + r.groups - 1) / r.groups;
  return r;
}

cudaError_t launch_norm_ring(const NormParams& n, const RingShape& r, const RingOut& o,
                             bool stream_f32, bool backward, int row_bytes, cudaStream_t st) {
  const RingParams p = {n, o, r, row_bytes, device_error_word()};
  const bool many = n.gate && n.gate_span < n.T;
  const size_t rings = static_cast<size_t>(r.groups) * (r.stages * row_bytes + r.tail_bytes);
  const size_t sums = backward ? static_cast<size_t>(r.groups) * n.H * sizeof(float) : 0;
  const size_t smem = rings > sums ? rings : sums;
  return stream_f32 ? launch_of<float>(p, backward, many, smem, st)
                    : launch_of<__nv_bfloat16>(p, backward, many, smem, st);
}

}  // namespace moe
