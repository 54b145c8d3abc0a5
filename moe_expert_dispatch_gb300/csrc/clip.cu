// clip.cu - moe_clip_grad_norm: one norm over many gradients, and all of them
// scaled by it.
//
// Two launches: clip_norm_kernel reads every gradient and leaves one partial
// result a CTA, clip_scale_kernel adds these up in every CTA, each for itself
// (a few hundred values, one warp), and scales. Both walk the same items, 16 KB
// of one tensor each in short runs, the second in the opposite order: what the
// first read last is still in L2. The tensors' table travels in the kernels' parameters.
// Up to 16 items (256 KB) are one launch of one cluster, clip_small_kernel,
// which keeps them in registers between the norm and the scaling.
//
// Bound by HBM: a gradient is read twice and written once (12 bytes an element
// in float), the second read from L2 as far as the 129 MB hold. Double
// precision runs at 1/64 of float's rate here, so the long sums are kept as
// pairs of floats (a sum and what its roundings lost), and only sums that would
// leave float's range go on in double.
//
// 5.6 GB in float: 2.47 to 2.53 ms for its three passes over HBM (16.9 GB: 6.8 TB/s;
// read once and written once it would be 1.66 ms). 50 MB: 22 us on the GPU. 300
// packed bf16 tensors, 100 MB: 50 to 52 us. 45 thousand elements: 5 us, one launch.
// One cooperative launch for both passes was slower: 28 us (50 MB) and 3.0 ms.
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kClipThreads = 256;
constexpr int kClipCtas = 4;               // of an SM: 3 to 5, 256 or 512 threads and items of 16
                                           // or 32 KB measured within 5% of each other
constexpr int kItemBytes = 16384;
constexpr int kLoads = kItemBytes / 16 / kClipThreads;   // 16-byte words of a thread
constexpr int kClipMaxCtas = 1024;         // partial results in the workspace
constexpr int kSmallCtas = 8, kSmallItems = 2;   // the one cluster's
constexpr int64_t kMaxNumel = static_cast<int64_t>(1) << 40;

template <int N>
struct ClipTable {
  const void* src[N];
  void* dst[N];
  int64_t numel[N];
  int item0[N + 1];                        // first item of each tensor
  uint8_t type[N];
  int n;
};

// The tensor that item c belongs to.
template <int N>
__device__ __forceinline__ int clip_find(const ClipTable<N>& t, int c) {
  int lo = 0, hi = t.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.item0[mid] <= c)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Elements before the first 16-byte boundary (all of a short tensor): they go
// with the tensor's first item.
__host__ __device__ __forceinline__ int64_t head_of(const void* p, int shift, int64_t numel) {
  const int64_t head = ((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) >> shift;
  return head < numel ? head : numel;
}
__host__ __device__ __forceinline__ int64_t items_of(const void* p, int shift, int64_t numel) {
  const int64_t body = (numel - head_of(p, shift, numel)) << shift;
  return body > kItemBytes ? (body + kItemBytes - 1) / kItemBytes : 1;
}

// A sum of squares: a float, what its roundings lost (Knuth's two-sum), and in
// double what would leave float's range, which no usual gradient comes near: a
// share of an item adds less than kFar to it, so that s stays finite unless a
// square is not. An infinite sum stays one, a NaN too.
constexpr float kFar = 1e38f;
struct Sum {
  float s, lost;
  double far;
  __device__ __forceinline__ void add(float x) {
    const float t = s + x, b = t - s;
    lost += (s - (t - b)) + (x - b);
    s = t;
  }
  __device__ __forceinline__ void settle() {
    if (!(s > kFar)) return;
    far += s;
    if (isinf(s)) lost = 0.0f;
    s = 0.0f;
  }
  __device__ __forceinline__ double value() const {
    return (isfinite(s) ? static_cast<double>(s) + lost : static_cast<double>(s)) + far;
  }
};

// The larger of two magnitudes as bit patterns: a NaN is above every number.
__device__ __forceinline__ unsigned max_bits(unsigned m, float g) {
  return max(m, __float_as_uint(g) & 0x7fffffffu);
}

// One thread's share of an item: kLoads words, all on their way at once; from L2
// alone, since no word is read twice by an SM (by L1's way the same within 1%).
struct Words {
  uint4 w[kLoads];
  bool has[kLoads];
};
__device__ __forceinline__ Words load_words(const char* p, int words) {
  Words r;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int at = threadIdx.x + i * kClipThreads;
    r.has[i] = at < words;
    r.w[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r.has[i])
      r.w[i] = __ldcg(reinterpret_cast<const uint4*>(p + static_cast<int64_t>(at) * 16));
  }
  return r;
}

// An item: its words, and the elements before (first item) and after (last
// item) the tensor's words.
struct Item {
  const char* src;
  char* dst;
  int64_t body;              // byte offset of the words in the tensor
  int words, head, tail;     // tail: elements after the words
  int f32;
};
// The tensor of a run of items: looked up once, then followed to its neighbours.
struct Tensor {
  const char* src;
  char* dst;
  int64_t bytes;             // after the head
  int item0, item1, i;       // its items; its place in the table
  int head, f32;
  template <int N>
  __device__ __forceinline__ void load(const ClipTable<N>& t, int at) {
    i = at;
    src = static_cast<const char*>(t.src[i]);
    dst = static_cast<char*>(t.dst[i]);
    f32 = t.type[i] == MOE_TYPE_F32;
    const int shift = f32 ? 2 : 1;
    head = static_cast<int>(head_of(src, shift, t.numel[i]));
    bytes = (t.numel[i] - head) << shift;
    item0 = t.item0[i];
    item1 = t.item0[i + 1];
  }
  template <int N>
  __device__ __forceinline__ Item item(const ClipTable<N>& t, int c) {
    if (c >= item1) load(t, i + 1);
    if (c < item0) load(t, i - 1);
    Item it;
    it.src = src;
    it.dst = dst;
    it.f32 = f32;
    const int shift = f32 ? 2 : 1;
    const int64_t lo = static_cast<int64_t>(c - item0) * kItemBytes, left = bytes - lo;
    it.body = (head << shift) + lo;
    it.words = static_cast<int>((left < kItemBytes ? left : kItemBytes) >> 4);
    it.head = c == item0 ? head : 0;
    it.tail = left < kItemBytes ? static_cast<int>(left & 15) >> shift : 0;
    return it;
  }
};
// Items go to the CTAs in waves of kRun for each: a run of neighbours, which
// share a tensor for the most part, while the CTAs stay close together (a search
// for every item: 1.6 GB in 100 bf16 tensors 848 us against 747; one run a CTA:
// 5.6 GB 2.65 against 2.60 ms). The last wave's are as long as one another or one
// longer.
constexpr int kRun = 8;
struct Run {
  int c0, c1;
};
__device__ __forceinline__ Run run_of(int items, int64_t base) {
  const int64_t wave = static_cast<int64_t>(gridDim.x) * kRun;
  const int64_t n = items - base < wave ? items - base : wave;
  return Run{static_cast<int>(base + n * blockIdx.x / gridDim.x),
             static_cast<int>(base + n * (blockIdx.x + 1) / gridDim.x)};
}

__device__ __forceinline__ float element(const char* p, int f32, int64_t at) {
  return f32 ? reinterpret_cast<const float*>(p)[at]
             : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[at]);
}

template <bool kF32, typename F>
__device__ __forceinline__ void each(const uint4& q, F&& f) {
  const unsigned w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kF32) {
      f(__uint_as_float(w[i]));
    } else {
      f(__uint_as_float(w[i] << 16));
      f(__uint_as_float(w[i] & 0xffff0000u));
    }
  }
}

// One thread's squares (kInf: largest magnitude) of an item.
template <bool kInf>
__device__ __forceinline__ void take_item(const Item& it, const Words& q, Sum* sum, unsigned* big) {
  float part[4] = {};
  auto take = [&](float g, int k) {
    if (kInf)
      *big = max_bits(*big, g);
    else
      part[k] = fmaf(g, g, part[k]);
  };
  auto take_words = [&](auto f32) {
    int k = 0;
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
      each<decltype(f32)::value>(q.w[u], [&](float g) { take(g, k++ & 3); });
  };
  if (it.f32)
    take_words(std::true_type());
  else
    take_words(std::false_type());
  if (threadIdx.x < it.head) take(element(it.src, it.f32, threadIdx.x), 0);
  if (threadIdx.x < it.tail)
    take(element(it.src + it.body + it.words * 16, it.f32, threadIdx.x), 1);
  if (!kInf) {
    sum->add((part[0] + part[1]) + (part[2] + part[3]));
    sum->settle();
  }
}

// The CTA's result from its threads', in thread 0; sh: one value a warp.
template <bool kInf>
__device__ __forceinline__ double cta_result(Sum sum, unsigned big, double* sh) {
  double all = 0.0;
  if (kInf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
    all = static_cast<double>(big);
  } else if (__any_sync(0xffffffffu, sum.s > kFar / 32 || sum.far != 0.0)) {
    // 32 lanes together may leave float's range
    all = sum.value();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
  } else {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float s = __shfl_xor_sync(0xffffffffu, sum.s, o);
      const float l = __shfl_xor_sync(0xffffffffu, sum.lost, o);
      sum.add(s);
      sum.lost += l;
    }
    all = sum.value();
  }
  if (lane_id() == 0) sh[threadIdx.x >> 5] = all;
  __syncthreads();
  double v = 0.0;
  if (threadIdx.x == 0)
#pragma unroll
    for (int w = 0; w < kClipThreads / 32; ++w) v = kInf ? fmax(v, sh[w]) : v + sh[w];
  return v;
}

// Every CTA's part of the sum of squares (kInf: of the largest magnitude, as
// the value of its bits) into partial[blockIdx.x]; a later launch of the same
// call (first = 0) adds to it, in the same order every time.
template <int N, bool kInf>
__global__ void __launch_bounds__(kClipThreads, kClipCtas)
    clip_norm_kernel(const __grid_constant__ ClipTable<N> t, int first,
                     double* __restrict__ partial) {
  __shared__ double sh[kClipThreads / 32];
  Sum sum = {0.0f, 0.0f, 0.0};
  unsigned big = 0u;
  const int items = t.item0[t.n];
  const int64_t wave = static_cast<int64_t>(gridDim.x) * kRun;
  for (int64_t base = 0; base < items; base += wave) {
    const Run r = run_of(items, base);
    if (r.c0 == r.c1) break;
    Tensor tensor;
    tensor.load(t, clip_find(t, r.c0));
    for (int c = r.c0; c < r.c1; ++c) {
      const Item it = tensor.item(t, c);
      take_item<kInf>(it, load_words(it.src + it.body, it.words), &sum, &big);
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const double v = cta_result<kInf>(sum, big, sh);
  if (threadIdx.x == 0) {
    const double old = first ? 0.0 : partial[blockIdx.x];
    partial[blockIdx.x] = kInf ? fmax(old, v) : old + v;
  }
}

struct ClipHow {
  const double* partial;
  float* norm_coef;
  int parts, inf, in_place;
  float max_norm, eps;
};

// norm and coef from the whole sum of squares (or the largest magnitude's bits).
__device__ __forceinline__ float2 norm_and_coef(const ClipHow& h, double s) {
  float norm;
  if (h.inf)
    norm = __uint_as_float(static_cast<unsigned>(s));
  else                       // a sum beyond float's range, but with a root in it
    norm = s > 1e38 ? sqrtf(static_cast<float>(s * 0x1p-60)) * 0x1p30f
                    : sqrtf(static_cast<float>(s));
  const float c = h.max_norm / (norm + h.eps);
  return make_float2(norm, h.max_norm < 0.0f || c >= 1.0f ? 1.0f : c);     // a NaN stays one
}

// The coefficient from the partial results, by the first warp, to every thread.
__device__ __forceinline__ float clip_coef(const ClipHow& h, bool write) {
  __shared__ float sh;
  if (threadIdx.x < 32) {
    double v[4] = {};
    for (int i = threadIdx.x; i < h.parts; i += 128)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = i + 32 * u;
        const double x = j < h.parts ? __ldcg(h.partial + j) : 0.0;
        v[u] = h.inf ? fmax(v[u], x) : v[u] + x;
      }
    double s = h.inf ? fmax(fmax(v[0], v[1]), fmax(v[2], v[3])) : (v[0] + v[1]) + (v[2] + v[3]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double x = __shfl_xor_sync(0xffffffffu, s, o);
      s = h.inf ? fmax(s, x) : s + x;
    }
    if (threadIdx.x == 0) {
      const float2 r = norm_and_coef(h, s);
      sh = r.y;
      if (write) {
        h.norm_coef[0] = r.x;
        h.norm_coef[1] = r.y;
      }
    }
  }
  __syncthreads();
  return sh;
}

// An item times coef, to its tensor's destination.
template <bool kF32>
__device__ __forceinline__ void scale_item(const Item& it, const Words& q, float coef) {
  using E = std::conditional_t<kF32, float, __nv_bfloat16>;
  E* dst = reinterpret_cast<E*>(it.dst);
  auto put = [&](int64_t at, float g) {
    if constexpr (kF32)
      dst[at] = g * coef;
    else
      dst[at] = __float2bfloat16_rn(g * coef);
  };
  constexpr int kShift = kF32 ? 2 : 1;
  const bool alike =
      ((reinterpret_cast<uintptr_t>(it.dst) ^ reinterpret_cast<uintptr_t>(it.src)) & 15) == 0;
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    if (!q.has[u]) continue;
    const int64_t at = it.body + (threadIdx.x + u * kClipThreads) * 16;
    if (alike) {
      float g[8];
      int k = 0;
      each<kF32>(q.w[u], [&](float x) { g[k++] = x * coef; });
      uint4 w;
      if (kF32)
        w = make_uint4(__float_as_uint(g[0]), __float_as_uint(g[1]), __float_as_uint(g[2]),
                       __float_as_uint(g[3]));
      else
        w = make_uint4(pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]), pack_bf16x2(g[4], g[5]),
                       pack_bf16x2(g[6], g[7]));
      // first to leave L2: what is still to be read there stays (50 MB 21.4 us
      // against 22.7, 100 MB 50.4 against 51.2, 5.6 GB the same)
      __stcs(reinterpret_cast<uint4*>(it.dst + at), w);
    } else {
      int64_t e = at >> kShift;                    // another alignment: element by element
      each<kF32>(q.w[u], [&](float x) { put(e++, x); });
    }
  }
  if (threadIdx.x < it.head) put(threadIdx.x, element(it.src, kF32, threadIdx.x));
  if (threadIdx.x < it.tail) {
    const int64_t at = ((it.body + it.words * 16) >> kShift) + threadIdx.x;
    put(at, element(it.src, kF32, at));
  }
}
__device__ __forceinline__ void scale_item(const Item& it, const Words& q, float coef) {
  if (it.f32)
    scale_item<true>(it, q, coef);
  else
    scale_item<false>(it, q, coef);
}

template <int N>
__global__ void __launch_bounds__(kClipThreads, kClipCtas)
    clip_scale_kernel(const __grid_constant__ ClipTable<N> t, const __grid_constant__ ClipHow h) {
  const int items = t.item0[t.n];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const float coef = clip_coef(h, blockIdx.x == 0);
  if (h.in_place && coef == 1.0f) return;
  const int64_t wave = static_cast<int64_t>(gridDim.x) * kRun;
  for (int64_t base = (items - 1) / wave * wave; base >= 0 && items > 0; base -= wave) {
    const Run r = run_of(items, base);
    if (r.c0 == r.c1) continue;
    Tensor tensor;
    tensor.load(t, clip_find(t, r.c1 - 1));
    for (int c = r.c1 - 1; c >= r.c0; --c) {
      const Item it = tensor.item(t, c);
      scale_item(it, load_words(it.src + it.body, it.words), coef);
    }
  }
}

// The whole call by one cluster: every CTA keeps its items in registers while
// the CTAs' sums meet.
template <int N, bool kInf>
__global__ void __launch_bounds__(kClipThreads, 1)
    clip_small_kernel(const __grid_constant__ ClipTable<N> t, const __grid_constant__ ClipHow h) {
  __shared__ double sh[kClipThreads / 32];
  __shared__ double mine;
  __shared__ float sh_coef;
  const int items = t.item0[t.n];
  Sum sum = {0.0f, 0.0f, 0.0};
  unsigned big = 0u;
  Item it[kSmallItems];
  Words q[kSmallItems];
#pragma unroll
  for (int i = 0; i < kSmallItems; ++i) {
    const int c = blockIdx.x + i * gridDim.x;
    it[i] = Item{};
    if (c < items) {
      Tensor tensor;
      tensor.load(t, clip_find(t, c));
      it[i] = tensor.item(t, c);
    }
    q[i] = load_words(it[i].src + it[i].body, it[i].words);
  }
#pragma unroll
  for (int i = 0; i < kSmallItems; ++i) take_item<kInf>(it[i], q[i], &sum, &big);
  const double v = cta_result<kInf>(sum, big, sh);
  if (threadIdx.x == 0) mine = v;
  cluster_sync();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (unsigned c = 0; c < gridDim.x; ++c) {
      const double x = ld_cluster_f64(smem_u32(&mine), c);
      s = kInf ? fmax(s, x) : s + x;
    }
    const float2 r = norm_and_coef(h, s);
    sh_coef = r.y;
    if (blockIdx.x == 0) {
      h.norm_coef[0] = r.x;
      h.norm_coef[1] = r.y;
    }
  }
  cluster_sync();
  const float coef = sh_coef;
  if (h.in_place && coef == 1.0f) return;
#pragma unroll
  for (int i = 0; i < kSmallItems; ++i)
    if (blockIdx.x + i * gridDim.x < items) scale_item(it[i], q[i], coef);
}

struct ClipCall {
  const void* const* grads;
  void* const* outs;
  const int64_t* numels;
  const int* types;
  int64_t n;
  float max_norm, eps;
  int inf;
  float* norm_coef;
  double* partial;
  cudaStream_t st;
};

// The next table of up to N tensors from i on, empty ones left out.
template <int N>
void fill_table(const ClipCall& c, int64_t* i, ClipTable<N>* t) {
  int n = 0;
  int64_t items = 0;
  t->item0[0] = 0;
  for (; *i < c.n && n < N; ++*i) {
    const int64_t numel = c.numels[*i];
    if (numel == 0) continue;
    const int64_t more = items_of(c.grads[*i], c.types[*i] == MOE_TYPE_F32 ? 2 : 1, numel);
    if (items + more > INT32_MAX) break;           // the next launch's
    items += more;
    t->src[n] = c.grads[*i];
    t->dst[n] = c.outs ? c.outs[*i] : const_cast<void*>(c.grads[*i]);
    t->numel[n] = numel;
    t->type[n] = static_cast<uint8_t>(c.types[*i]);
    t->item0[++n] = static_cast<int>(items);
  }
  t->n = n;
}

template <int N>
cudaError_t clip(const ClipCall& c) {
  ClipTable<N> t;
  const int most = device_sm_count() * kClipCtas < kClipMaxCtas ? device_sm_count() * kClipCtas
                                                                 : kClipMaxCtas;
  int64_t i = 0;
  fill_table(c, &i, &t);
  const bool one = i >= c.n;                       // the whole call in one table
  const int all = t.item0[t.n];
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.blockDim = dim3(kClipThreads);
  cfg.stream = c.st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  ClipHow h = {c.partial, c.norm_coef, 0, c.inf, c.outs == nullptr, c.max_norm, c.eps};
  if (one && all <= kSmallCtas * kSmallItems) {
    const int ctas = all < kSmallCtas ? (all > 0 ? all : 1) : kSmallCtas;
    cfg.gridDim = dim3(ctas);
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    return c.inf ? cudaLaunchKernelEx(&cfg, clip_small_kernel<N, true>, t, h)
                 : cudaLaunchKernelEx(&cfg, clip_small_kernel<N, false>, t, h);
  }
  // one partial result a CTA; with several tables each launch has them all
  const int parts = h.parts = one && all < most ? all : most;
  for (bool first = true;; first = false) {
    if (c.inf)
      clip_norm_kernel<N, true><<<parts, kClipThreads, 0, c.st>>>(t, first, c.partial);
    else
      clip_norm_kernel<N, false><<<parts, kClipThreads, 0, c.st>>>(t, first, c.partial);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (i >= c.n) break;
    fill_table(c, &i, &t);
  }
  const bool norm_only = c.max_norm < 0.0f && !c.outs;
  // comes up while the norm's last CTAs still run, and waits for all of them
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  if (!one) i = 0;
  do {
    if (!one) fill_table(c, &i, &t);
    if (norm_only) t.n = t.item0[0] = 0;
    const int ctas = t.item0[t.n] < most ? t.item0[t.n] : most;
    cfg.gridDim = dim3(static_cast<unsigned>(ctas > 0 ? ctas : 1));
    const cudaError_t e = cudaLaunchKernelEx(&cfg, clip_scale_kernel<N>, t, h);
    if (e != cudaSuccess || norm_only) return e;
    cfg.numAttrs = 0;
  } while (i < c.n);
  return cudaSuccess;
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
    if (numels[i] < 0 || numels[i] > kMaxNumel ||
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
  const ClipCall c = {grads, outs, numels,   types,     n_tensors, max_norm,
                      eps,   norm_kind, norm_coef, static_cast<double*>(workspace),
                      static_cast<cudaStream_t>(stream)};
  // a table that holds them: its bytes go with every launch. 300 tensors in three
  // tables of 100 take 78 us for 50 (100 MB); the small tables spare the launches
  // of few tensors some 28 KB of parameters (0.1 to 0.2 us of 4.7)
  const cudaError_t e = n_tensors <= 8     ? clip<8>(c)
                        : n_tensors <= 100 ? clip<100>(c)
                                           : clip<960>(c);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
