// norm_ring.cu - the norms around the block for rows of up to 8192 elements:
// forward and backward over strips of rows that bulk copies bring into shared
// memory.
//
// A group of threads (whole warps) walks a strip of consecutive rows, every
// thread with sixteen fixed columns (four vectors of four, so that all accesses
// are coalesced for float and for bf16; with eight a thread, the registers of
// the pointers and counters left too few for the columns). What belongs to a column stays in its
// registers from row to row: the weights, b w_post g as one factor, and the
// column sums of the weight gradients. A row's tensors lie in one stage of the
// group's ring, which its first thread fills with bulk copies up to three rows
// ahead; each is read from HBM once. A CTA has as many groups as 512 threads
// hold, one CTA an SM, so that short rows too have enough bytes on their way,
// and the groups' column sums are added up in shared memory: the finishing
// kernel finds one row of partial sums an SM.
//
// Both are bound by HBM, 8 bytes an element forward and 12 backward in bf16
// (18 with a float stream), as long as a row's instructions stay below its
// bytes' time: about 12 operations an element and two barriers a row.
#include "norm.cuh"

namespace moe {

int* device_error_word();

namespace {

constexpr int kRingBytes = 216 * 1024;
constexpr int kMaxStages = 4;
constexpr int kRingThreads = 512;
constexpr int kVecs = 4;                  // vectors of four columns a thread
constexpr int kCols = 4 * kVecs;

struct RingParams {
  NormParams n;
  RingOut o;
  RingShape r;
  int row_bytes;
  int* err;
};

__device__ __forceinline__ float warp_add(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void group_barrier(int bar, int group) {
  asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(group) : "memory");
}

// The sum of v over a group to each of its threads; warp: the thread's in it.
__device__ __forceinline__ float group_sum(float v, float* red, int warp, int bar, int group) {
  v = warp_add(v);
  if (lane_id() == 0) red[warp] = v;
  group_barrier(bar, group);
  v = lane_id() < (group >> 5) ? red[lane_id()] : 0.0f;
  return warp_add(v);
}

struct Four {
  float f[4];
};

__device__ __forceinline__ Four widen(uint2 q) {
  return Four{{__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xffff0000u),
               __uint_as_float(q.y << 16), __uint_as_float(q.y & 0xffff0000u)}};
}

// Four elements of a row in shared memory.
template <typename T>
__device__ __forceinline__ Four row4(const unsigned char* row, int col) {
  if constexpr (sizeof(T) == 4) {
    const float4 q = *reinterpret_cast<const float4*>(row + col * 4);
    return Four{{q.x, q.y, q.z, q.w}};
  } else {
    return widen(*reinterpret_cast<const uint2*>(row + col * 2));
  }
}

template <typename T>
__device__ __forceinline__ void put4(T* p, const Four& v) {
  if constexpr (sizeof(T) == 4)
    *reinterpret_cast<float4*>(p) = make_float4(v.f[0], v.f[1], v.f[2], v.f[3]);
  else
    *reinterpret_cast<uint2*>(p) =
        make_uint2(pack_bf16x2(v.f[0], v.f[1]), pack_bf16x2(v.f[2], v.f[3]));
}

// A group's place in its CTA, its strip and its ring.
struct Walk {
  int g, tid, warp, H;
  int64_t lo, hi;
  unsigned char* ring;
  uint32_t full;               // mbarriers of its stages
  int col[kVecs];
  bool has[kVecs];
};

// kFull: every thread has all sixteen columns (H a multiple of 512).
template <bool kFull>
__device__ __forceinline__ Walk walk_of(const RingParams& p, unsigned char* ring_all,
                                        uint64_t (*full_all)[kMaxStages], int* abort_wait) {
  Walk w;
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
#pragma unroll
  for (int v = 0; v < kVecs; ++v) {
    w.col[v] = 4 * (w.tid + v * p.r.group);
    w.has[v] = kFull || w.col[v] < w.H;
  }
  if (threadIdx.x == 0) *abort_wait = 0;
  if (w.tid == 0) {
    for (int i = 0; i < p.r.stages; ++i) mbar_init(w.full + 8 * i, 1);
    fence_mbar_init();
  }
  __syncthreads();
  return w;
}

__device__ __forceinline__ void times(const RingParams& p, const Walk& w, const void* weights,
                                      int64_t row, float (&f)[kCols]) {
#pragma unroll
  for (int v = 0; v < kVecs; ++v) {
    if (!w.has[v]) continue;
    Four m;
    if (p.n.weights_f32) {
      const float4 q =
          __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(weights) + row + w.col[v]));
      m = Four{{q.x, q.y, q.z, q.w}};
    } else {
      m = widen(__ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(weights) +
                                                     row + w.col[v])));
    }
#pragma unroll
    for (int h = 0; h < 4; ++h) f[4 * v + h] *= m.f[h];
  }
}

// Waits for a stage. No wait as long as the limit is legitimate: it is
// reported, and the waits after it are given up at once.
__device__ __forceinline__ void wait_stage(const RingParams& p, const Walk& w, int stage, int parity,
                                           unsigned long long* limit, int* abort_wait) {
  if (!mbar_wait(w.full + 8 * stage, parity, *limit, abort_wait)) {
    report_error(p.err, kErrTimeout);
    *limit = 0;
  }
}

// ------------------------------------------------------------------ forward

template <typename ST, bool kMany, bool kFull>
__global__ void __launch_bounds__(kRingThreads, 1)
    norm_ring_kernel(const __grid_constant__ RingParams p) {
  extern __shared__ __align__(128) unsigned char ring_all[];
  __shared__ float red_all[kMaxRingGroups][4][kRingThreads / 32];
  __shared__ __align__(8) uint64_t full_all[kMaxRingGroups][kMaxStages];
  __shared__ int abort_wait;
  const Walk w = walk_of<kFull>(p, ring_all, full_all, &abort_wait);
  const NormParams& q = p.n;
  const bool branch = q.y, post = q.w_post, next = q.w_next;
  const int wide = w.H * static_cast<int>(sizeof(ST)), half = w.H * 2;
  auto issue = [&](int64_t t, int stage) {
    const uint32_t bar = w.full + 8 * stage, to = smem_u32(w.ring) + stage * p.row_bytes;
    mbar_arrive_expect_tx(bar, p.row_bytes);
    bulk_copy_g2s(to, static_cast<const ST*>(q.x) + t * w.H, wide, bar);
    if (branch) bulk_copy_g2s(to + wide, q.y + t * w.H, half, bar);
  };
  if (w.tid == 0)
    for (int i = 0; i < p.r.stages && w.lo + i < w.hi; ++i) issue(w.lo + i, i);

  float gw[kCols], wn[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) {
    gw[i] = q.b;
    wn[i] = 1.0f;
  }
  if (next) times(p, w, q.w_next, 0, wn);
  if (!kMany) {
    if (post) times(p, w, q.w_post, 0, gw);
    if (q.gate) times(p, w, q.gate, 0, gw);
  }
  unsigned long long limit = kDefaultWaitNs;
  int stage = 0, parity = 0, odd = 0;
  int64_t gate_row = -1, gate_end = w.lo;
  if (kMany && w.lo < w.hi) gate_row = w.lo / q.gate_span - 1;
  ST* to_out = static_cast<ST*>(p.o.stream) + w.lo * w.H;
  __nv_bfloat16* to_n = p.o.branch + w.lo * w.H;
  for (int64_t t = w.lo; t < w.hi; ++t, to_out += w.H, to_n += w.H) {
    if (kMany && t == gate_end) {
      ++gate_row;
      gate_end = (gate_row + 1) * q.gate_span;
#pragma unroll
      for (int i = 0; i < kCols; ++i) gw[i] = q.b;
      if (post) times(p, w, q.w_post, 0, gw);
      times(p, w, q.gate, gate_row * w.H, gw);
    }
    wait_stage(p, w, stage, parity, &limit, &abort_wait);
    const unsigned char* row = w.ring + stage * p.row_bytes;
    Four x[kVecs], y[kVecs];
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      if (!w.has[v]) continue;
      x[v] = row4<ST>(row, w.col[v]);
      if (branch) {
        y[v] = row4<__nv_bfloat16>(row + wide, w.col[v]);
#pragma unroll
        for (int h = 0; h < 4; ++h) s = fmaf(y[v].f[h], y[v].f[h], s);
      }
    }
    float ry = 1.0f;
    if (post) {
      s = group_sum(s, red_all[w.g][odd], w.warp, w.g + 1, p.r.group);
      ry = 1.0f / sqrtf(fmaf(s, q.inv_h, q.eps));
      if (w.tid == 0 && p.o.rstd_y) p.o.rstd_y[t] = ry;
    } else {
      group_barrier(w.g + 1, p.r.group);
    }
    // every thread has the row in registers: its stage takes another
    if (w.tid == 0 && t + p.r.stages < w.hi) issue(t + p.r.stages, stage);
    s = 0.0f;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      if (!w.has[v]) continue;
      if (branch) {
#pragma unroll
        for (int h = 0; h < 4; ++h)
          x[v].f[h] = fmaf(y[v].f[h] * ry, gw[4 * v + h], q.a * x[v].f[h]);
        put4(to_out + w.col[v], x[v]);
      }
#pragma unroll
      for (int h = 0; h < 4; ++h) s = fmaf(x[v].f[h], x[v].f[h], s);
    }
    if (next) {
      s = group_sum(s, red_all[w.g][2 + odd], w.warp, w.g + 1, p.r.group);
      const float ro = 1.0f / sqrtf(fmaf(s, q.inv_h, q.eps));
      if (w.tid == 0 && p.o.rstd_out) p.o.rstd_out[t] = ro;
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        if (!w.has[v]) continue;
#pragma unroll
        for (int h = 0; h < 4; ++h) x[v].f[h] *= ro * wn[4 * v + h];
        put4(to_n + w.col[v], x[v]);
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
// dgate = b w_post S for one gate row; kMany keeps S for a row's tokens and its
// sum over rows times g),
//   dy = r (gw D - y (r^2 m(u gw))).
// No product of three r: a row of 1e15 stays in float's range.
template <typename ST, bool kMany, bool kFull>
__global__ void __launch_bounds__(kRingThreads, 1)
    norm_ring_backward_kernel(const __grid_constant__ RingParams p) {
  extern __shared__ __align__(128) unsigned char ring_all[];
  __shared__ float red_all[kMaxRingGroups][4][kRingThreads / 32];
  __shared__ __align__(8) uint64_t full_all[kMaxRingGroups][kMaxStages];
  __shared__ int abort_wait;
  const Walk w = walk_of<kFull>(p, ring_all, full_all, &abort_wait);
  const NormParams& q = p.n;
  const bool branch = q.y, post = q.w_post, next = q.d_n, has_d = q.x;
  // a stage: d_out, out, y, d_n, as far as there are any
  const int wide = w.H * static_cast<int>(sizeof(ST)), half = w.H * 2;
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

  float gw[kCols], wn[kCols], sum_s[kCols], sum_n[kCols], sum_w[kMany ? kCols : 1];
#pragma unroll
  for (int i = 0; i < kCols; ++i) {
    gw[i] = q.b;
    wn[i] = 1.0f;
    sum_s[i] = sum_n[i] = 0.0f;
    if (kMany) sum_w[i] = 0.0f;
  }
  if (next) times(p, w, q.w_next, 0, wn);
  if (!kMany) {
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
  ST* to_dx = static_cast<ST*>(p.o.stream) + w.lo * w.H;
  __nv_bfloat16* to_dy = p.o.branch + w.lo * w.H;
  for (int64_t t = w.lo; t < w.hi; ++t, to_dx += w.H, to_dy += w.H) {
    const float ro = next_ro, ry = next_ry;
    if (t + 1 < w.hi) {
      if (next) next_ro = q.rstd_out[t + 1];
      if (post) next_ry = q.rstd_y[t + 1];
    }
    if (kMany && t == gate_end) {
      ++gate_row;
      gate_end = (gate_row + 1) * q.gate_span;
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        gw[i] = q.b;
        sum_s[i] = 0.0f;
      }
      if (post) times(p, w, q.w_post, 0, gw);
      times(p, w, q.gate, gate_row * w.H, gw);
    }
    wait_stage(p, w, stage, parity, &limit, &abort_wait);
    const unsigned char* row = w.ring + stage * p.row_bytes;
    Four d[kVecs];
    if (next) {
      float s = 0.0f;
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        if (!w.has[v]) continue;
        const Four f = row4<__nv_bfloat16>(row + at_dn, w.col[v]);
        const Four out = row4<ST>(row + at_out, w.col[v]);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int i = 4 * v + h;
          const float u = f.f[h] * out.f[h];
          s = fmaf(u, wn[i], s);
          sum_n[i] = fmaf(u, ro, sum_n[i]);
        }
      }
      s = group_sum(s, red_all[w.g][odd], w.warp, w.g + 1, p.r.group);
      const float k = ro * (ro * (s * q.inv_h));
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        if (!w.has[v]) continue;
        // read again: shared memory is cheaper here than registers
        const Four f = row4<__nv_bfloat16>(row + at_dn, w.col[v]);
        const Four out = row4<ST>(row + at_out, w.col[v]);
#pragma unroll
        for (int h = 0; h < 4; ++h)
          d[v].f[h] = fmaf(-k, out.f[h], f.f[h] * wn[4 * v + h]);
        const Four e = has_d ? row4<ST>(row, w.col[v]) : Four{};
#pragma unroll
        for (int h = 0; h < 4; ++h) d[v].f[h] = fmaf(ro, d[v].f[h], e.f[h]);
      }
    } else {
#pragma unroll
      for (int v = 0; v < kVecs; ++v)
        if (w.has[v]) d[v] = row4<ST>(row, w.col[v]);
    }
    uint2 y[kVecs];
    float m = 0.0f;
    if (branch) {
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        if (!w.has[v]) continue;
        y[v] = *reinterpret_cast<const uint2*>(row + at_y + w.col[v] * 2);
        const Four f = widen(y[v]);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int i = 4 * v + h;
          const float u = d[v].f[h] * f.f[h];
          sum_s[i] = fmaf(u, ry, sum_s[i]);
          m = fmaf(u, gw[i], m);
        }
      }
    }
    if (post)
      m = group_sum(m, red_all[w.g][2 + odd], w.warp, w.g + 1, p.r.group);
    else
      group_barrier(w.g + 1, p.r.group);
    // every thread has the row in registers: its stage takes another
    if (w.tid == 0 && t + p.r.stages < w.hi) issue(t + p.r.stages, stage);
    const float k = ry * (ry * (m * q.inv_h));
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      if (!w.has[v]) continue;
      if (branch) {
        const Four f = widen(y[v]);
        Four g;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          g.f[h] = gw[4 * v + h] * d[v].f[h];
          if (post) g.f[h] = ry * fmaf(-k, f.f[h], g.f[h]);
          d[v].f[h] *= q.a;
        }
        put4(to_dy + w.col[v], g);
      }
      put4(to_dx + w.col[v], d[v]);
    }
    if (kMany && (t + 1 == gate_end || t + 1 == w.hi)) {
      // S of the gate row: whole to dgate, else a piece (0: begun in an earlier
      // strip, 1: in this one); its share of dw_post stays
      const int64_t first = gate_row * q.gate_span;
      const bool whole = first >= w.lo && t + 1 == gate_end;
      const int64_t strip = static_cast<int64_t>(blockIdx.x) * p.r.groups + w.g;
      float* to = whole ? p.o.dgate + gate_row * w.H
                        : p.o.part_gate + (strip * 2 + (first >= w.lo)) * w.H;
      float gt[kCols], wp[kCols];
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        gt[i] = 1.0f;
        wp[i] = q.b;
      }
      times(p, w, q.gate, gate_row * w.H, gt);
      if (post) times(p, w, q.w_post, 0, wp);
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        if (!w.has[v]) continue;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int i = 4 * v + h;
          sum_w[i] = fmaf(gt[i], sum_s[i], sum_w[i]);
          float z = whole ? sum_s[i] * wp[i] : sum_s[i];
          if (whole && p.o.accumulate) z += to[w.col[v] + h];
          to[w.col[v] + h] = z;
        }
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
  auto add_up = [&](const float* sum, float* part) {
    float* all = reinterpret_cast<float*>(ring_all);
    __syncthreads();
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
      if (w.has[v])
        *reinterpret_cast<float4*>(all + w.g * w.H + w.col[v]) =
            make_float4(sum[4 * v], sum[4 * v + 1], sum[4 * v + 2], sum[4 * v + 3]);
    __syncthreads();
    for (int h = threadIdx.x; h < w.H; h += blockDim.x) {
      float z = 0.0f;
      for (int i = 0; i < p.r.groups; ++i) z += all[i * w.H + h];
      part[static_cast<int64_t>(blockIdx.x) * w.H + h] = z;
    }
  };
  if (p.o.part_post) add_up(kMany ? sum_w : sum_s, p.o.part_post);
  if (p.o.part_next) add_up(sum_n, p.o.part_next);
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
cudaError_t launch_of(const RingParams& p, bool backward, size_t smem, cudaStream_t st) {
  const bool many = p.n.gate && p.n.gate_span < p.n.T, full = p.n.H == kCols * p.r.group;
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

int ring_group(int H) {
  const int group = (H + 32 * kCols - 1) / (32 * kCols) * 32;
  return H % 8 == 0 && group <= kRingThreads ? group : 0;
}

int max_ring_groups(int group) {
  return group == 0 ? 0 : kRingThreads / group < kMaxRingGroups ? kRingThreads / group : kMaxRingGroups;
}

RingShape ring_shape(int64_t T, int H, int row_bytes) {
  RingShape r = {};
  const int group = ring_group(H);
  if (T == 0 || group == 0 || 2 * row_bytes > kRingBytes) return r;
  const int sms = device_sm_count();
  r.group = group;
  // as many groups as there are threads and two stages of memory for, unless
  // the rows run out first
  r.groups = max_ring_groups(group);
  while (r.groups > 1 && (r.groups * 2 * row_bytes > kRingBytes ||
                          T <= static_cast<int64_t>(sms) * (r.groups - 1)))
    --r.groups;
  r.stages = kRingBytes / (r.groups * row_bytes);
  if (r.stages > kMaxStages) r.stages = kMaxStages;
  const int64_t most = static_cast<int64_t>(sms) * r.groups;
  r.strips = static_cast<int>(T < most ? T : most);
  r.ctas = (r.strips + r.groups - 1) / r.groups;
  return r;
}

cudaError_t launch_norm_ring(const NormParams& n, const RingShape& r, const RingOut& o,
                             bool stream_f32, bool backward, int row_bytes, cudaStream_t st) {
  const RingParams p = {n, o, r, row_bytes, device_error_word()};
  const size_t ring = static_cast<size_t>(r.groups) * r.stages * row_bytes;
  const size_t sums = backward ? static_cast<size_t>(r.groups) * n.H * sizeof(float) : 0;
  const size_t smem = ring > sums ? ring : sums;
  return stream_f32 ? launch_of<float>(p, backward, smem, st)
                    : launch_of<__nv_bfloat16>(p, backward, smem, st);
}

}  // namespace moe
