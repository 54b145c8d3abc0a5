// norm_ring.cu - the norms around the block for rows of up to 8192 elements:
// forward and backward over strips of rows that bulk copies bring into shared
// memory.
//
// A group of threads (whole warps) walks a strip of consecutive rows, every
// thread with sixteen fixed columns: two vectors of eight in bf16, four of four
// with a float stream, so that all accesses are 16 bytes and coalesced. What
// belongs to a column stays in its registers from row to row: the weights,
// b w_post g as one factor, and the column sums of the weight gradients. A
// row's tensors lie in one stage of the group's ring, which its first thread
// fills with bulk copies up to three rows ahead; each is read from HBM once. A
// CTA has as many groups as 512 threads hold, one CTA an SM, so that short rows
// too have enough bytes on their way, and the groups' column sums are added up
// in shared memory: the finishing kernel finds one row of partial sums an SM.
//
// Bound by HBM, 8 bytes an element forward and 12 backward in bf16 (18 with a
// float stream), where a row's instructions stay below its bytes' time: pairs
// of columns go through the packed float instructions (fma.rn.f32x2), which
// round each half as the single ones do, and the backward's two means, of which
// the second needs the first, come from one reduction of three sums.
#include "norm.cuh"

#include <stdlib.h>

namespace moe {

int* device_error_word();

namespace {

constexpr int kSharedBytes = 208 * 1024;  // of the rings, and what lies behind them
constexpr int kMaxStages = 4;
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kCols = 16;                 // of a thread

// How tokens share gate rows: one row (or none), whose factors stay in
// registers; several rows of several tokens each, loaded as a strip comes to
// them; a row for each token, which comes through the ring.
enum Gate { kOneGate, kManyGates, kTokenGates };

struct RingParams {
  NormParams n;
  RingOut o;
  RingShape r;
  int row_bytes;
  int* err;
#ifdef MOE_DEBUG
  bool give_up;                            // every wait is given up
#endif
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

// W columns, as floats and (bf16) as they are stored.
template <int W>
struct Vec {
  Pair p[W / 2];
};
template <int W>
struct Half {
  unsigned u[W / 2];
};

template <int W>
__device__ __forceinline__ Vec<W> widen(const Half<W>& h) {
  Vec<W> v;
#pragma unroll
  for (int i = 0; i < W / 2; ++i)
    v.p[i] = pair(__uint_as_float(h.u[i] << 16), __uint_as_float(h.u[i] & 0xffff0000u));
  return v;
}
template <int W>
__device__ __forceinline__ Half<W> get_half(const unsigned char* p) {
  if constexpr (W == 8) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    return Half<W>{{q.x, q.y, q.z, q.w}};
  } else {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    return Half<W>{{q.x, q.y}};
  }
}

// A vector of the stream as it is stored: floats (W = 4) or bf16.
template <typename ST>
struct Stream {
  static constexpr int W = sizeof(ST) == 4 ? 4 : 8;
  static constexpr int V = kCols / W;
  ulonglong2 f;
  Half<W> h;
  static __device__ __forceinline__ Stream get(const unsigned char* p) {
    Stream s;
    if constexpr (W == 4)
      s.f = *reinterpret_cast<const ulonglong2*>(p);
    else
      s.h = get_half<W>(p);
    return s;
  }
  __device__ __forceinline__ Vec<W> wide() const {
    if constexpr (W == 4)
      return Vec<W>{{f.x, f.y}};
    else
      return widen<W>(h);
  }
};

template <int W>
__device__ __forceinline__ void put_half(unsigned char* p, const Vec<W>& v) {
  unsigned u[W / 2];
#pragma unroll
  for (int i = 0; i < W / 2; ++i) {
    const float2 f = halves(v.p[i]);
    u[i] = pack_bf16x2(f.x, f.y);
  }
  if constexpr (W == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
}
template <typename ST, int W>
__device__ __forceinline__ void put_stream(unsigned char* p, const Vec<W>& v) {
  if constexpr (sizeof(ST) == 4)
    *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(v.p[0], v.p[1]);
  else
    put_half<W>(p, v);
}

// ------------------------------------------------------------------ groups and rings

// The sums of N values over a group to each of its threads. The barrier in it
// also tells that the group has read what it had to.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float4* red, int warp, int bar, int group) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (group == 32) {
    __syncwarp();
    return;
  }
  if (lane_id() == 0)
    red[warp] = make_float4(v[0], N > 1 ? v[N > 1 ? 1 : 0] : 0.0f, N > 2 ? v[N > 2 ? 2 : 0] : 0.0f,
                            0.0f);
  asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(group) : "memory");
  const int at = lane_id() & (kWarps - 1);
  float4 r = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (at < (group >> 5)) r = red[at];
  v[0] = r.x;
  if (N > 1) v[N > 1 ? 1 : 0] = r.y;
  if (N > 2) v[N > 2 ? 2 : 0] = r.z;
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
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
  int col0, step;              // columns col0 + v step .. + W - 1 are the thread's
  bool has[V];
};

// Waits that were given up: in the CTA, and in each group (1; 2: and its copies
// were waited for).
struct GaveUp {
  int cta, group[kMaxRingGroups];
};

// kFull: every thread has all its columns.
template <int V, bool kFull>
__device__ __forceinline__ Walk<V> walk_of(const RingParams& p, unsigned char* ring_all,
                                           uint64_t (*full_all)[kMaxStages], GaveUp* gave_up) {
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
  w.col0 = (kCols / V) * w.tid;
  w.step = (kCols / V) * p.r.group;
#pragma unroll
  for (int v = 0; v < V; ++v) w.has[v] = kFull || w.col0 + v * w.step < w.H;
  if (threadIdx.x == 0) gave_up->cta = 0;
  if (w.tid == 0) {
    gave_up->group[w.g] = 0;
    for (int i = 0; i < p.r.stages; ++i) mbar_init(w.full + 8 * i, 1);
    fence_mbar_init();
  }
  __syncthreads();
  return w;
}

// f[columns] *= weights[row + columns]
template <int V>
__device__ __forceinline__ void times(const RingParams& p, const Walk<V>& w, const void* weights,
                                      int64_t row, Pair (&f)[kCols / 2]) {
  constexpr int W = kCols / V;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (!w.has[v]) continue;
    const int64_t at = row + w.col0 + v * w.step;
    Vec<W> m;
    if (p.n.weights_f32) {
#pragma unroll
      for (int i = 0; i < W / 4; ++i) {
        const float4 q = __ldg(
            reinterpret_cast<const float4*>(static_cast<const float*>(weights) + at) + i);
        m.p[2 * i] = pair(q.x, q.y);
        m.p[2 * i + 1] = pair(q.z, q.w);
      }
    } else {
      Half<W> h;
#pragma unroll
      for (int i = 0; i < W / 4; ++i) {
        const uint2 q = __ldg(
            reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(weights) + at) + i);
        h.u[2 * i] = q.x;
        h.u[2 * i + 1] = q.y;
      }
      m = widen<W>(h);
    }
#pragma unroll
    for (int i = 0; i < W / 2; ++i) f[v * (W / 2) + i] = mul2(f[v * (W / 2) + i], m.p[i]);
  }
}

// A gate row's vector in shared memory.
template <int W>
__device__ __forceinline__ Vec<W> gate_of(const RingParams& p, const unsigned char* row, int col) {
  if (!p.n.weights_f32) return widen<W>(get_half<W>(row + col * 2));
  Vec<W> v;
#pragma unroll
  for (int i = 0; i < W / 4; ++i) {
    const ulonglong2 q = reinterpret_cast<const ulonglong2*>(row + col * 4)[i];
    v.p[2 * i] = q.x;
    v.p[2 * i + 1] = q.y;
  }
  return v;
}

// Waits for a stage. No wait as long as the limit is legitimate: it is reported,
// and what the thread computes from there on is no result, but it keeps to the
// group's barriers to the last one. Its own later waits and the CTA's others
// are given up with it, each after the few microseconds that a try_wait lasts.
template <int V>
__device__ __forceinline__ void wait_stage(const RingParams& p, const Walk<V>& w, int stage,
                                           int parity, bool* gave_up, GaveUp* all) {
  const uint32_t bar = w.full + 8 * stage;
  volatile int *cta = &all->cta, *group = &all->group[w.g];
#ifdef MOE_DEBUG
  const bool unseen = p.give_up;           // whether or not the copies have come
#else
  const bool unseen = false;
#endif
  if (!unseen && mbar_try_wait(bar, parity)) return;
  if (!unseen && mbar_wait(bar, parity, *gave_up ? 0 : kDefaultWaitNs, cta)) return;
  report_error(p.err, kErrTimeout);
  *cta = 1;
  if (*group == 0) *group = 1;
  *gave_up = true;
}

// Waits, once more with a limit, for the copies of a group that are still on their
// way: from the row of this stage on, of which `left` are to come.
__device__ __noinline__ void drain(uint32_t full, int stages, int left, int stage, int parity) {
  const unsigned long long t0 = global_timer_ns();
  for (int i = 0; i < stages && i < left; ++i) {
    while (!mbar_try_wait(full + 8 * stage, parity))
      if (global_timer_ns() - t0 > kDefaultWaitNs) return;
    if (++stage == stages) {
      stage = 0;
      parity ^= 1;
    }
  }
}

// Whether the group's first thread may fill a stage again, behind the barrier that
// the group came to with that stage's row. Once a wait was given up it fills
// none: it has waited for what was on its way, and nothing is when the CTA ends.
template <int V>
__device__ __forceinline__ bool may_refill(const RingParams& p, const Walk<V>& w, int left,
                                           int stage, int parity, GaveUp* all) {
  const int was = *static_cast<volatile int*>(&all->group[w.g]);
  if (was == 1) {
    drain(w.full, p.r.stages, left, stage, parity);
    all->group[w.g] = 2;
  }
  return was == 0;
}

// ------------------------------------------------------------------ forward

// kAll: with y, w_post and w_next. 4096 x 4096 in bf16 takes 23.5 us where L2 has
// some of it, and 26.7 (134 MB: 5.0 TB/s), of which 4 are launch and the first
// rows' way; 16384 x 7168 145 us (6.5 TB/s), with a float stream 247 (5.7 TB/s).
// Other forms: 16384 x 7168 in bf16 without w_post 164 us (5.7 TB/s), the norm
// alone 97 (4.8 TB/s).
template <typename ST, int kGate, bool kFull, bool kAll>
__global__ void __launch_bounds__(kThreads, 1)
    norm_ring_kernel(const __grid_constant__ RingParams p) {
  constexpr int W = Stream<ST>::W, V = Stream<ST>::V, P = W / 2, kSize = sizeof(ST);
  extern __shared__ __align__(128) unsigned char ring_all[];
  __shared__ float4 red_all[kMaxRingGroups][4][kWarps];
  __shared__ __align__(8) uint64_t full_all[kMaxRingGroups][kMaxStages];
  __shared__ GaveUp gave_up_all;
  const Walk<V> w = walk_of<V, kFull>(p, ring_all, full_all, &gave_up_all);
  const NormParams& q = p.n;
  const bool branch = kAll || q.y, post = kAll || q.w_post, next = kAll || q.w_next;
  constexpr bool kMany = kGate == kManyGates, kToken = kGate == kTokenGates;
  const int wide = w.H * kSize, half = w.H * 2;
  const int at_g = wide + half, gate_bytes = q.weights_f32 ? w.H * 4 : half;
  auto issue = [&](int64_t t, int stage) {
    const uint32_t bar = w.full + 8 * stage, to = smem_u32(w.ring) + stage * p.row_bytes;
    mbar_arrive_expect_tx(bar, p.row_bytes);
    bulk_copy_g2s(to, static_cast<const ST*>(q.x) + t * w.H, wide, bar);
    if (branch) bulk_copy_g2s(to + wide, q.y + t * w.H, half, bar);
    if (kToken)
      bulk_copy_g2s(to + at_g, static_cast<const char*>(q.gate) + t * gate_bytes, gate_bytes, bar);
  };
  if (w.tid == 0)
    for (int i = 0; i < p.r.stages && w.lo + i < w.hi; ++i) issue(w.lo + i, i);

  Pair gw[kCols / 2], wn[kCols / 2];
#pragma unroll
  for (int i = 0; i < kCols / 2; ++i) {
    gw[i] = pair(q.b);
    wn[i] = pair(1.0f);
  }
  if (next) times(p, w, q.w_next, 0, wn);
  if (!kMany) {
    if (post) times(p, w, q.w_post, 0, gw);
    if (kGate == kOneGate && q.gate) times(p, w, q.gate, 0, gw);
  }
  int64_t gate_row = -1;
  int to_gate = 0;                                 // rows until another gate row
  if (kMany && w.lo < w.hi) gate_row = w.lo / q.gate_span - 1;
  bool gave_up = false;
  int stage = 0, parity = 0, odd = 0;
  unsigned char* to_out = static_cast<unsigned char*>(p.o.stream) + (w.lo * w.H + w.col0) * kSize;
  unsigned char* to_n = reinterpret_cast<unsigned char*>(p.o.branch) + (w.lo * w.H + w.col0) * 2;
  const int rows = static_cast<int>(w.hi - w.lo);
  const Pair a = pair(q.a);
  for (int t = 0; t < rows; ++t, to_out += wide, to_n += half) {
    if (kMany && to_gate-- == 0) {
      ++gate_row;
      to_gate = static_cast<int>((gate_row + 1) * q.gate_span - (w.lo + t)) - 1;
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) gw[i] = pair(q.b);
      if (post) times(p, w, q.w_post, 0, gw);
      times(p, w, q.gate, gate_row * w.H, gw);
    }
    wait_stage(p, w, stage, parity, &gave_up, &gave_up_all);
    const unsigned char* row_x = w.ring + (stage * p.row_bytes + w.col0 * kSize);
    const unsigned char* row_y = w.ring + (stage * p.row_bytes + wide + w.col0 * 2);
    Vec<W> x[V], y[V];
    Pair s = pair(0.0f);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!w.has[v]) continue;
      x[v] = Stream<ST>::get(row_x + v * w.step * kSize).wide();
      if (branch) {
        y[v] = widen<W>(get_half<W>(row_y + v * w.step * 2));
#pragma unroll
        for (int h = 0; h < P; ++h) s = fma2(y[v].p[h], y[v].p[h], s);
        if (kToken) {
          const Vec<W> g = gate_of<W>(p, w.ring + stage * p.row_bytes + at_g, w.col0 + v * w.step);
#pragma unroll
          for (int h = 0; h < P; ++h) y[v].p[h] = mul2(y[v].p[h], g.p[h]);
        }
      }
    }
    float ry = 1.0f;
    if (post) {
      float m[1] = {sum2(s)};
      group_sum(m, red_all[w.g][odd], w.warp, w.g + 1, p.r.group);
      ry = 1.0f / sqrtf(fmaf(m[0], q.inv_h, q.eps));
    } else {
      group_barrier(w.g + 1, p.r.group);
    }
    // every thread has the row in registers: its stage takes another
    if (w.tid == 0) {
      if (may_refill(p, w, rows - t, stage, parity, &gave_up_all) && t + p.r.stages < rows)
        issue(w.lo + t + p.r.stages, stage);
      if (post && p.o.rstd_y) p.o.rstd_y[w.lo + t] = ry;
    }
    s = pair(0.0f);
    const Pair r = pair(ry);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!w.has[v]) continue;
      if (branch) {
#pragma unroll
        for (int h = 0; h < P; ++h)
          x[v].p[h] = fma2(mul2(y[v].p[h], r), gw[P * v + h], mul2(a, x[v].p[h]));
        put_stream<ST, W>(to_out + v * w.step * kSize, x[v]);
      }
#pragma unroll
      for (int h = 0; h < P; ++h) s = fma2(x[v].p[h], x[v].p[h], s);
    }
    if (next) {
      float m[1] = {sum2(s)};
      group_sum(m, red_all[w.g][2 + odd], w.warp, w.g + 1, p.r.group);
      const float ro = 1.0f / sqrtf(fmaf(m[0], q.inv_h, q.eps));
      if (w.tid == 0 && p.o.rstd_out) p.o.rstd_out[w.lo + t] = ro;
      const Pair o = pair(ro);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (!w.has[v]) continue;
#pragma unroll
        for (int h = 0; h < P; ++h) x[v].p[h] = mul2(mul2(x[v].p[h], o), wn[P * v + h]);
        put_half<W>(to_n + v * w.step * 2, x[v]);
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

// With r = rstd_out: dw_next += r d_n out, and D = A + k out with
//   A = d_out + r d_n w_next,  k = -r (r (r m(d_n w_next out))).
// The gradient of y's norm needs m(gw D y), gw = b g w_post, which is
// m(gw A y) + k m(gw out y): three sums of one pass over the row, one barrier.
// With r = rstd_y: S += r D y, and dy = r (gw D - y (r^2 m(gw D y))). One gate
// row: dw_post = b g S and dgate = b w_post S; kManyGates keeps S for a row's
// tokens, and its sum over rows times g in shared memory; kTokenGates sums g
// times it and writes dgate at once (16384 x 2048 in bf16: 105 us at a floor of 89;
// by kManyGates' way of leaving a row 409).
// kAll: with d_out, d_n, y and w_post. 16384 x 7168 with a float stream takes
// 327 us (2.1 GB: 6.5 TB/s, 95% of a copy's rate), in bf16 242 us (5.8 TB/s);
// 4083 x 2048 in bf16 with three gate rows 32.9 us (3.1 TB/s), of which some 9 are
// launches, the first rows' way and the strips' sums. Other forms choose at run
// time and spill more: 16384 x 7168 in bf16 without w_post and gate 371 us (y is
// read and summed up for a gradient that nobody takes: 10 of its 12 bytes an
// element are needed, 173 us), the norm alone 318 (138); with a float stream 421
// (277) and 260 (242).
template <typename ST, int kGate, bool kFull, bool kAll>
__global__ void __launch_bounds__(kThreads, 1)
    norm_ring_backward_kernel(const __grid_constant__ RingParams p) {
  constexpr int W = Stream<ST>::W, V = Stream<ST>::V, P = W / 2, kSize = sizeof(ST);
  extern __shared__ __align__(128) unsigned char ring_all[];
  __shared__ float4 red_all[kMaxRingGroups][2][kWarps];
  __shared__ __align__(8) uint64_t full_all[kMaxRingGroups][kMaxStages];
  __shared__ GaveUp gave_up_all;
  const Walk<V> w = walk_of<V, kFull>(p, ring_all, full_all, &gave_up_all);
  const NormParams& q = p.n;
  const bool branch = kAll || q.y, post = kAll || q.w_post, next = kAll || q.d_n,
             has_d = kAll || q.x;
  constexpr bool kMany = kGate == kManyGates, kToken = kGate == kTokenGates;
  // a stage: d_out, out, y, d_n, as far as there are any
  const int wide = w.H * kSize, half = w.H * 2;
  const int at_out = has_d ? wide : 0, at_y = at_out + (next ? wide : 0),
            at_dn = at_y + (branch ? half : 0), at_g = at_dn + (next ? half : 0);
  const int gate_bytes = q.weights_f32 ? w.H * 4 : half;
  auto issue = [&](int64_t t, int stage) {
    const uint32_t bar = w.full + 8 * stage, to = smem_u32(w.ring) + stage * p.row_bytes;
    const int64_t at = t * w.H;
    mbar_arrive_expect_tx(bar, p.row_bytes);
    if (has_d) bulk_copy_g2s(to, static_cast<const ST*>(q.x) + at, wide, bar);
    if (next) bulk_copy_g2s(to + at_out, static_cast<const ST*>(q.out) + at, wide, bar);
    if (branch) bulk_copy_g2s(to + at_y, q.y + at, half, bar);
    if (next) bulk_copy_g2s(to + at_dn, q.d_n + at, half, bar);
    if (kToken)
      bulk_copy_g2s(to + at_g, static_cast<const char*>(q.gate) + t * gate_bytes, gate_bytes, bar);
  };
  if (w.tid == 0)
    for (int i = 0; i < p.r.stages && w.lo + i < w.hi; ++i) issue(w.lo + i, i);

  // kMany: the group's sum of g S, behind the rings; the only group's is the
  // CTA's partial sum itself
  auto sum_of_groups = [&]() {
    return p.r.tail_bytes ? reinterpret_cast<float*>(ring_all + static_cast<size_t>(p.r.groups) *
                                                                    p.r.stages * p.row_bytes)
                          : p.o.part_post + static_cast<int64_t>(blockIdx.x) * w.H;
  };
  const bool keep_w = kMany && p.o.part_post;
  Pair gw[kCols / 2], wn[kCols / 2], sum_s[kCols / 2], sum_n[kCols / 2];
#pragma unroll
  for (int i = 0; i < kCols / 2; ++i) {
    gw[i] = pair(q.b);
    wn[i] = pair(1.0f);
    sum_s[i] = sum_n[i] = pair(0.0f);
  }
  if (next) times(p, w, q.w_next, 0, wn);
  if (kMany) {
    float* sum_w = keep_w ? sum_of_groups() + (p.r.tail_bytes ? w.g * w.H : 0) + w.col0 : nullptr;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (w.has[v] && keep_w)
#pragma unroll
        for (int i = 0; i < W; i += 4)
          *reinterpret_cast<float4*>(sum_w + v * w.step + i) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  } else {
    if (post) times(p, w, q.w_post, 0, gw);
    if (kGate == kOneGate && q.gate) times(p, w, q.gate, 0, gw);
  }
  int64_t gate_row = -1;
  int to_gate = 0;                                 // rows until another gate row
  if (kMany && w.lo < w.hi) gate_row = w.lo / q.gate_span - 1;
  bool gave_up = false;
  int stage = 0, parity = 0;
  const int rows = static_cast<int>(w.hi - w.lo);
  const Pair a = pair(branch ? q.a : 1.0f);
  float ro32 = 0.0f, ry32 = 1.0f;                  // of 32 rows, a lane each
  for (int t = 0; t < rows; ++t) {
    if ((t & 31) == 0) {
      const int64_t at = min(w.lo + t + lane_id(), w.hi - 1);
      if (next) ro32 = q.rstd_out[at];
      if (post) ry32 = q.rstd_y[at];
    }
    const float ro = __shfl_sync(0xffffffffu, ro32, t & 31);
    const float ry = __shfl_sync(0xffffffffu, ry32, t & 31);
    if (kMany && to_gate == 0) {
      ++gate_row;
      to_gate = static_cast<int>((gate_row + 1) * q.gate_span - (w.lo + t));
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) {
        gw[i] = pair(q.b);
        sum_s[i] = pair(0.0f);
      }
      if (post) times(p, w, q.w_post, 0, gw);
      times(p, w, q.gate, gate_row * w.H, gw);
    }
    wait_stage(p, w, stage, parity, &gave_up, &gave_up_all);
    const unsigned char* row_wide = w.ring + (stage * p.row_bytes + w.col0 * kSize);
    const unsigned char* row_half = w.ring + (stage * p.row_bytes + w.col0 * 2);
    Vec<W> d[V];                                   // A, then D
    Half<W> y[V];
    Pair s0 = pair(0.0f), s1 = s0, s2 = s0;
    const Pair r = pair(ro);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!w.has[v]) continue;
      if (has_d) d[v] = Stream<ST>::get(row_wide + v * w.step * kSize).wide();
      if (next) {
        const Vec<W> dn = widen<W>(get_half<W>(row_half + (at_dn + v * w.step * 2)));
        const Vec<W> o = Stream<ST>::get(row_wide + (at_out + v * w.step * kSize)).wide();
#pragma unroll
        for (int h = 0; h < P; ++h) {
          const int i = P * v + h;
          const Pair u = mul2(dn.p[h], wn[i]);
          s0 = fma2(u, o.p[h], s0);
          sum_n[i] = fma2(mul2(dn.p[h], o.p[h]), r, sum_n[i]);
          d[v].p[h] = has_d ? fma2(u, r, d[v].p[h]) : mul2(u, r);
        }
      }
      if (branch) {
        y[v] = get_half<W>(row_half + (at_y + v * w.step * 2));
        if (post) {
          Vec<W> f = widen<W>(y[v]), o;
          if (kToken) {
            const Vec<W> g = gate_of<W>(p, w.ring + stage * p.row_bytes + at_g,
                                        w.col0 + v * w.step);
#pragma unroll
            for (int h = 0; h < P; ++h) f.p[h] = mul2(f.p[h], g.p[h]);
          }
          if (next) o = Stream<ST>::get(row_wide + (at_out + v * w.step * kSize)).wide();
#pragma unroll
          for (int h = 0; h < P; ++h) {
            const Pair u = mul2(f.p[h], gw[P * v + h]);
            s1 = fma2(u, d[v].p[h], s1);
            if (next) s2 = fma2(u, o.p[h], s2);
          }
        }
      }
    }
    float m[3] = {sum2(s0), sum2(s1), sum2(s2)};
    if (post || next) group_sum(m, red_all[w.g][t & 1], w.warp, w.g + 1, p.r.group);
    const float k0 = next ? -ro * (ro * (ro * (m[0] * q.inv_h))) : 0.0f;
    const Pair k = pair(k0), l = pair(-ry * (ry * (fmaf(k0, m[2], m[1]) * q.inv_h)));
    const Pair e = pair(ry);
    if (next) {
      // out once more: registers to keep it would be spilled, and with this much
      // shared memory L1 is too small to spill to
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (!w.has[v]) continue;
        const Vec<W> o = Stream<ST>::get(row_wide + (at_out + v * w.step * kSize)).wide();
#pragma unroll
        for (int h = 0; h < P; ++h) d[v].p[h] = fma2(k, o.p[h], d[v].p[h]);
      }
    }
    // every thread has the row in registers: its stage takes another (after the
    // gate's row has been read too)
    auto refill = [&]() {
      group_barrier(w.g + 1, p.r.group);
      if (w.tid == 0 && may_refill(p, w, rows - t, stage, parity, &gave_up_all) &&
          t + p.r.stages < rows)
        issue(w.lo + t + p.r.stages, stage);
    };
    if (!kToken) refill();
    const int64_t first_col = (w.lo + t) * w.H + w.col0;
    unsigned char* to_dx = static_cast<unsigned char*>(p.o.stream) + first_col * kSize;
    unsigned char* to_dy = reinterpret_cast<unsigned char*>(p.o.branch) + first_col * 2;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!w.has[v]) continue;
      if (branch) {
        const Vec<W> f = widen<W>(y[v]);
        Vec<W> g, z;
        if (kToken)
          z = gate_of<W>(p, w.ring + stage * p.row_bytes + at_g, w.col0 + v * w.step);
#pragma unroll
        for (int h = 0; h < P; ++h) {
          const int i = P * v + h;
          Pair u = mul2(d[v].p[h], f.p[h]);        // D y
          g.p[h] = mul2(gw[i], d[v].p[h]);
          if (kToken) {
            u = mul2(u, e);
            sum_s[i] = fma2(u, z.p[h], sum_s[i]);
            g.p[h] = mul2(g.p[h], z.p[h]);
            z.p[h] = mul2(u, gw[i]);               // this token's dgate
          } else {
            sum_s[i] = fma2(u, e, sum_s[i]);
          }
          if (post) g.p[h] = mul2(e, fma2(l, f.p[h], g.p[h]));
        }
        put_half<W>(to_dy + v * w.step * 2, g);
        if (kToken) {
          float* to = p.o.dgate + first_col + v * w.step;
#pragma unroll
          for (int i = 0; i < W; i += 4) {
            const float2 lo = halves(z.p[i / 2]), hi = halves(z.p[i / 2 + 1]);
            float4 old = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (p.o.accumulate) old = *reinterpret_cast<const float4*>(to + i);
            *reinterpret_cast<float4*>(to + i) =
                make_float4(old.x + lo.x, old.y + lo.y, old.z + hi.x, old.w + hi.y);
          }
        }
      }
#pragma unroll
      for (int h = 0; h < P; ++h) d[v].p[h] = mul2(a, d[v].p[h]);
      put_stream<ST, W>(to_dx + v * w.step * kSize, d[v]);
    }
    if (kToken) refill();
    if (kMany && (--to_gate == 0 || t + 1 == rows)) {
      // S of the gate row: whole to dgate, else a piece (0: begun in an earlier
      // strip, 1: in this one); its share of dw_post stays
      const int64_t first = gate_row * q.gate_span;
      const bool whole = first >= w.lo && to_gate == 0;
      const int64_t strip = static_cast<int64_t>(blockIdx.x) * p.r.groups + w.g;
      float* to = (whole ? p.o.dgate + gate_row * w.H
                         : p.o.part_gate + (strip * 2 + (first >= w.lo)) * w.H) +
                  w.col0;
      Pair f[kCols / 2];
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) f[i] = sum_s[i];
      times(p, w, q.gate, gate_row * w.H, f);
      auto add4 = [&](float* at, int i, bool old) {
        const float2 lo = halves(f[i]), hi = halves(f[i + 1]);
        float4 z = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (old) z = *reinterpret_cast<const float4*>(at);
        *reinterpret_cast<float4*>(at) =
            make_float4(z.x + lo.x, z.y + lo.y, z.z + hi.x, z.w + hi.y);
      };
      float* sum_w = keep_w ? sum_of_groups() + (p.r.tail_bytes ? w.g * w.H : 0) + w.col0 : nullptr;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (w.has[v] && keep_w)
#pragma unroll
          for (int i = 0; i < W; i += 4) add4(sum_w + v * w.step + i, P * v + i / 2, true);
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) f[i] = whole ? mul2(pair(q.b), sum_s[i]) : sum_s[i];
      if (whole && post) times(p, w, q.w_post, 0, f);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (w.has[v])
#pragma unroll
          for (int i = 0; i < W; i += 4)
            add4(to + v * w.step + i, P * v + i / 2, whole && p.o.accumulate);
    }
    if (++stage == p.r.stages) {
      stage = 0;
      parity ^= 1;
    }
  }

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // with a wait given up there are no sums, and perhaps a copy that never came to
  // where they would lie
  __syncthreads();
  if (gave_up_all.cta) return;
  // the groups' sums, in order
  auto add_up = [&](const float* all, float* part) {
    __syncthreads();
    for (int h = threadIdx.x; h < w.H; h += blockDim.x) {
      float z = 0.0f;
      for (int i = 0; i < p.r.groups; ++i) z += all[i * w.H + h];
      part[static_cast<int64_t>(blockIdx.x) * w.H + h] = z;
    }
  };
  auto share = [&](const Pair (&sum)[kCols / 2]) {
    float* all = reinterpret_cast<float*>(ring_all) + w.g * w.H + w.col0;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (w.has[v])
#pragma unroll
        for (int i = 0; i < W; i += 4)
          *reinterpret_cast<ulonglong2*>(all + v * w.step + i) =
              make_ulonglong2(sum[P * v + i / 2], sum[P * v + i / 2 + 1]);
    return reinterpret_cast<const float*>(ring_all);
  };
  if (p.o.part_post && !(kMany && p.r.tail_bytes == 0))
    add_up(kMany ? sum_of_groups() : share(sum_s), p.o.part_post);
  if (p.o.part_next) add_up(share(sum_n), p.o.part_next);
}

// ------------------------------------------------------------------ launches

// Threads that share a row; 0: more than a CTA has.
int group_of(int H) {
  const int group = (H + 32 * kCols - 1) / (32 * kCols) * 32;
  return H % 8 == 0 && group <= kThreads ? group : 0;
}

// A call's shared memory follows from its rows, types and gate; the kernel's limit
// is set once per device, to the most of any call, and never lowered: a call
// from another thread may lie between its setting and this launch.
template <void (*kKernel)(RingParams)>
cudaError_t launch(const RingParams& p, size_t smem, cudaStream_t st) {
  static bool configured[kMaxDevices] = {};
  const int d = current_device();
  if (d < 0 || d >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!configured[d]) {
    const cudaError_t e = cudaFuncSetAttribute(
        kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedBytes);
    if (e != cudaSuccess) return e;
    configured[d] = true;
  }
  kKernel<<<p.r.ctas, p.r.groups * p.r.group, smem, st>>>(p);
  return cudaGetLastError();
}

template <typename ST, int kGate, bool kFull, bool kAll>
cudaError_t launch_of(const RingParams& p, bool backward, size_t smem, cudaStream_t st) {
  return backward ? launch<norm_ring_backward_kernel<ST, kGate, kFull, kAll>>(p, smem, st)
                  : launch<norm_ring_kernel<ST, kGate, kFull, kAll>>(p, smem, st);
}

template <typename ST, bool kFull, bool kAll>
cudaError_t launch_of(const RingParams& p, bool backward, int gate, size_t smem, cudaStream_t st) {
  return gate == kTokenGates  ? launch_of<ST, kTokenGates, kFull, kAll>(p, backward, smem, st)
         : gate == kManyGates ? launch_of<ST, kManyGates, kFull, kAll>(p, backward, smem, st)
                              : launch_of<ST, kOneGate, kFull, kAll>(p, backward, smem, st);
}

// Rows of a multiple of 512 with all the tensors are what layers have; any
// other takes the kernels that look at each run.
template <typename ST>
cudaError_t launch_of(const RingParams& p, bool backward, size_t smem, cudaStream_t st) {
  const NormParams& n = p.n;
  const int gate = !n.gate || n.gate_span == n.T ? kOneGate
                   : n.gate_span == 1            ? kTokenGates
                                                 : kManyGates;
  const bool full = n.H == kCols * p.r.group;
  const bool all = n.y && n.w_post && (backward ? n.x && n.d_n : n.w_next != nullptr);
  return full ? (all ? launch_of<ST, true, true>(p, backward, gate, smem, st)
                     : launch_of<ST, true, false>(p, backward, gate, smem, st))
              : (all ? launch_of<ST, false, true>(p, backward, gate, smem, st)
                     : launch_of<ST, false, false>(p, backward, gate, smem, st));
}

}  // namespace

int most_ring_groups(int H) {
  const int group = group_of(H);
  const int groups = group ? kThreads / group : 0;
  return groups < kMaxRingGroups ? groups : kMaxRingGroups;
}

RingShape ring_shape(int64_t T, int H, int row_bytes, bool backward, bool many) {
  RingShape r = {};
  r.group = group_of(H);
  if (T == 0 || r.group == 0 || 2 * row_bytes > kSharedBytes) return r;
  const int sms = device_sm_count();
  // as many groups as there are threads and two stages of memory for, unless
  // the rows run out first
  r.groups = kThreads / r.group;
  if (r.groups > kMaxRingGroups) r.groups = kMaxRingGroups;
  const int tail = backward && many ? H * static_cast<int>(sizeof(float)) : 0;
  while (r.groups > 1 && (r.groups * (2 * row_bytes + tail) > kSharedBytes ||
                          T <= static_cast<int64_t>(sms) * (r.groups - 1)))
    --r.groups;
  r.tail_bytes = r.groups > 1 ? tail : 0;
  r.stages = (kSharedBytes / r.groups - r.tail_bytes) / row_bytes;
  if (r.stages > kMaxStages) r.stages = kMaxStages;
  const int64_t most = static_cast<int64_t>(sms) * r.groups;
  r.strips = static_cast<int>(T < most ? T : most);
  r.ctas = (r.strips + r.groups - 1) / r.groups;
  return r;
}

cudaError_t launch_norm_ring(const NormParams& n, const RingShape& r, const RingOut& o,
                             bool stream_f32, bool backward, int row_bytes, cudaStream_t st) {
  RingParams p = {n, o, r, row_bytes, device_error_word()};
#ifdef MOE_DEBUG
  // for tests of what a wait given up leaves behind
  p.give_up = getenv("MOE_GB300_GIVE_UP_WAITS") != nullptr;
#endif
  const size_t rings = static_cast<size_t>(r.groups) * (r.stages * row_bytes + r.tail_bytes);
  const size_t sums = backward ? static_cast<size_t>(r.groups) * n.H * sizeof(float) : 0;
  const size_t smem = rings > sums ? rings : sums;
  return stream_f32 ? launch_of<float>(p, backward, smem, st)
                    : launch_of<__nv_bfloat16>(p, backward, smem, st);
}

}  // namespace moe
