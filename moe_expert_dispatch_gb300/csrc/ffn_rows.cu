// ffn_rows.cu - the gated feed-forward block for few rows (a decoding step, a short
// batch): its products with the weights, all bound by reading those once.
//
//   Gated     h from x, W_gate and W_up        Down    y from h and W_down
//   GatedBwd  h, dA_g, dA_u from dy, W_down    InGrad  dx from dA_g, dA_u, W_gate, W_up
//
// The roles of the operands are exchanged: 128 columns of the result are the M of a
// tile and the tokens its N (16 to 128), so that a tile is full of weights however
// few the tokens are. Of a Gated tile the 128 are 64 columns of W_gate and the same
// 64 of W_up, and it ends with A_g and A_u of 64 columns of h.
//
// The weights arrive by TMA, 64 of K at a time (16 KB), into a ring that keeps 100
// KB of loads under way in each of two CTAs an SM: 30 MB over the GPU, where the
// memory's rate times its latency asks for about 8. K is split over the CTAs of a
// cluster (up to 8) so that narrow layers fill the GPU too; the cluster adds its
// sums up through shared memory in the order of the ranks, each CTA finishing every
// C-th token, and no sum depends on timing. The second product of a pass is launched
// while the first runs (programmatic dependent launch): its rings fill with weights
// before it waits for the first one's results.
//
// Bound by the weights: 64 rows of 4096 x 14336 read 352 MB in 64 us, 5.5 TB/s (W_gate and
// W_up at 5.6, W_down at 4.6, with its ring's start overlapped); 16 rows of 2048 x 768 (9.4
// MB, which stay in L2) take 11 us, the latency of two launches. Without the split of K
// these are 110 and 19 us, without the overlapped launch 65 and 12.6, and 67 and 11 where
// the weights are not marked as the first to leave L2.
#include "act.cuh"
#include "common.cuh"
#include "ffn.h"
#include "internal.h"

namespace moe {

namespace {

constexpr int BK = 64;
constexpr int kWBytes = 128 * BK * 2;            // 16 KB: 128 columns of weights x 64 of K
constexpr int kBox = 64 * BK * 2;
constexpr int kThreads = 192;
constexpr int kMaxStages = 6;
constexpr int kRingBytes = 108 * 1024;           // of a CTA: two share an SM
constexpr unsigned long long kDrainNs = 1000000000ull;

struct Smem {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t done;
  uint32_t tmem_base;
  int abort;
  int zero;
};

enum class Op { Gated, Down, GatedBwd, InGrad };
// weights with the columns of the result contiguous (MN-major), or with K (K-major)
constexpr bool w_mn(Op op) { return op == Op::Gated || op == Op::Down; }

struct Maps {
  CUtensorMap w[2], x[2];
};

struct Args {
  int T, tn;             // rows, and rounded up to the MMA's N
  int N, kb0, kb;        // columns of the result; k-blocks of the first operands, of both
  int split;             // CTAs of a cluster
  int stages;
  int tmem_cols;
  int act;
  const __nv_bfloat16* add;
  __nv_bfloat16* out;    // h, y, h again or dx
  __nv_bfloat16* a_gate; // Gated: A_g and A_u where they are kept; GatedBwd: as they were kept
  __nv_bfloat16* a_up;
  __nv_bfloat16* da_gate;
  __nv_bfloat16* da_up;
  int* err;
  unsigned long long wait_ns;
};

__device__ __forceinline__ float act_any(int act, float z) {
  switch (act) {
    case MOE_ACT_SILU: return act_f<MOE_ACT_SILU>(z);
    case MOE_ACT_GELU: return act_f<MOE_ACT_GELU>(z);
    case MOE_ACT_GELU_TANH: return act_f<MOE_ACT_GELU_TANH>(z);
    default: return act_f<MOE_ACT_RELU>(z);
  }
}

__device__ __forceinline__ void act_both_any(int act, float z, float& f, float& d) {
  switch (act) {
    case MOE_ACT_SILU: act_both<MOE_ACT_SILU>(z, f, d); break;
    case MOE_ACT_GELU: act_both<MOE_ACT_GELU>(z, f, d); break;
    case MOE_ACT_GELU_TANH: act_both<MOE_ACT_GELU_TANH>(z, f, d); break;
    default: act_both<MOE_ACT_RELU>(z, f, d); break;
  }
}

__device__ __forceinline__ float4 bf16x4(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                     __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
}

__device__ __forceinline__ void put_bf16x4(__nv_bfloat16* p, float a, float b, float c, float d) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
}

// A cluster takes one tile of columns, each of its CTAs a run of k-blocks.
template <Op op>
__global__ void __launch_bounds__(kThreads)
    rows_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Smem* sm = reinterpret_cast<Smem*>(ring + kRingBytes);
  const int warp = threadIdx.x >> 5, lane = lane_id();
  const uint32_t rank = cluster_ctarank();
  constexpr bool kGated = op == Op::Gated, kMn = w_mn(op);
  const int tile = static_cast<int>(blockIdx.x) / p.split;
  const int n0 = tile * (kGated ? 64 : 128);
  const int per = (p.kb + p.split - 1) / p.split;
  const int kb0 = min(p.kb, static_cast<int>(rank) * per), kb1 = min(p.kb, kb0 + per);
  const int S = p.stages, stage_bytes = kWBytes + p.tn * BK * 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&sm->full[s]), 1);
      mbar_init(smem_u32(&sm->empty[s]), 1);
    }
    mbar_init(smem_u32(&sm->done), 1);
    sm->abort = 0;
    sm->zero = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sm->tmem_base), p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm->tmem_base;
  volatile int* abort_flag = &sm->abort;
  if (kGated || op == Op::GatedBwd) grid_dependents_launch();

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t ring0 = smem_u32(ring);
      const uint64_t pol = l2_policy_evict_first();     // weights are read once
      auto load_w = [&](int kb, int s) {
        const uint32_t bar = smem_u32(&sm->full[s]), sa = ring0 + s * stage_bytes;
        mbar_arrive_expect_tx(bar, stage_bytes);
        if (kMn) {
          tma_load_2d_hint(sa, &maps.w[0], bar, n0, kb * BK, pol);
          tma_load_2d_hint(sa + kBox, &maps.w[kGated ? 1 : 0], bar, kGated ? n0 : n0 + 64, kb * BK,
                           pol);
        } else {
          const bool second = op == Op::InGrad && kb >= p.kb0;
          tma_load_2d_hint(sa, &maps.w[second ? 1 : 0], bar, (second ? kb - p.kb0 : kb) * BK, n0,
                           pol);
        }
      };
      auto load_x = [&](int kb, int s) {
        const bool second = op == Op::InGrad && kb >= p.kb0;
        tma_load_2d(ring0 + s * stage_bytes + kWBytes, &maps.x[second ? 1 : 0],
                    smem_u32(&sm->full[s]), (second ? kb - p.kb0 : kb) * BK, 0);
      };
      // weights fill the ring before the rows are there
      const int first = min(S, kb1 - kb0);
      for (int i = 0; i < first; ++i) load_w(kb0 + i, i);
      grid_dependency_wait();
      fence_proxy_async();
      for (int i = 0; i < first; ++i) load_x(kb0 + i, i);
      int stage = first == S ? 0 : first;
      uint32_t phase = first == S ? 1 : 0;
      bool ok = true;
      int issued = first;
      for (int kb = kb0 + first; kb < kb1; ++kb) {
        if (!mbar_wait(smem_u32(&sm->empty[stage]), phase ^ 1, p.wait_ns, abort_flag)) {
          ok = false;
          break;
        }
        load_w(kb, stage);
        load_x(kb, stage);
        ++issued;
        if (++stage == S) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (!ok) {
        sm->abort = 1;
        report_error(p.err, kErrTimeout);
      }
      // every copy lands before the CTA goes on to use the ring for its sums, or exits
      for (int i = issued > S ? issued - S : 0; i < issued; ++i)
        mbar_wait(smem_u32(&sm->full[i % S]), (i / S) & 1, kDrainNs, &sm->zero);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // weights: MN-major atoms of 64 columns, 8 KB apart, or K-major like the rows
      const uint32_t idesc = idesc_bf16(128, p.tn, kMn, false);
      const uint32_t ring0 = smem_u32(ring);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(smem_u32(&sm->full[stage]), phase, p.wait_ns, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sa = ring0 + stage * stage_bytes;
        const uint64_t ad = sdesc_sw128(sa, kMn ? kBox : 16, 1024);
        const uint64_t bd = sdesc_sw128(sa + kWBytes, 16, 1024);
#pragma unroll
        for (int ks = 0; ks < BK / 16; ++ks)
          umma_bf16(tmem, ad + ks * (kMn ? 2048 >> 4 : 32 >> 4), bd + ks * (32 >> 4), idesc,
                    (kb > kb0 || ks) ? 1u : 0u);
        umma_commit(smem_u32(&sm->empty[stage]));
        if (++stage == S) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (!ok) {
        sm->abort = 1;
        report_error(p.err, kErrTimeout);
      }
      umma_commit(smem_u32(&sm->done));
    }
  } else {
    const bool got = mbar_wait(smem_u32(&sm->done), 0, p.wait_ns, abort_flag);
    if (!__all_sync(0xffffffffu, got)) {
      sm->abort = 1;
      if (lane == 0) {
        report_error(p.err, kErrTimeout);
        mbar_wait(smem_u32(&sm->done), 0, kDrainNs, &sm->zero);
      }
    }
    tc_fence_after();
  }
  __syncthreads();               // the MMAs have read the ring, and every copy has landed

  // this CTA's sums as [token][column of the tile]; a run of no k-blocks is 0
  float* part = reinterpret_cast<float*>(ring);
  if (warp >= 2) {
    const int q = warp & 3, c = q * 32 + lane;
    for (int t0 = 0; t0 < p.tn; t0 += 16) {
      uint32_t v[16];
      tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(q * 32) << 16) + t0, v);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) part[(t0 + i) * 128 + c] = kb0 < kb1 ? __uint_as_float(v[i]) : 0.0f;
    }
    tc_fence_before();
  }
  if (p.split > 1) cluster_sync();
  else __syncthreads();

  // tokens rank, rank + split, ...: a warp a token, four columns a lane
  const uint32_t part0 = smem_u32(part);
  const bool broken = sm->abort != 0;
  for (int t = static_cast<int>(rank) + p.split * warp; t < p.T && !broken;
       t += p.split * (kThreads / 32)) {
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int r = 0; r < p.split; ++r) {
      const float4 v = p.split > 1 ? ld_cluster_f32x4(part0 + (t * 128 + lane * 4) * 4, r)
                                   : *reinterpret_cast<const float4*>(part + t * 128 + lane * 4);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    if (kGated) {
      // lanes 0-15 hold A_g of 64 columns, lanes 16-31 A_u of the same
      const int col = n0 + (lane & 15) * 4;
      const int64_t at = static_cast<int64_t>(t) * p.N + col;
      const bool up = lane >= 16;
      if (p.a_gate && col < p.N) put_bf16x4((up ? p.a_up : p.a_gate) + at, s.x, s.y, s.z, s.w);
      const float ux = __shfl_down_sync(0xffffffffu, s.x, 16);
      const float uy = __shfl_down_sync(0xffffffffu, s.y, 16);
      const float uz = __shfl_down_sync(0xffffffffu, s.z, 16);
      const float uw = __shfl_down_sync(0xffffffffu, s.w, 16);
      if (!up && col < p.N)
        put_bf16x4(p.out + at, act_any(p.act, s.x) * ux, act_any(p.act, s.y) * uy,
                   act_any(p.act, s.z) * uz, act_any(p.act, s.w) * uw);
      continue;
    }
    const int col = n0 + lane * 4;
    if (col >= p.N) continue;
    const int64_t at = static_cast<int64_t>(t) * p.N + col;
    if (op == Op::GatedBwd) {
      const float4 g = bf16x4(p.a_gate + at), u = bf16x4(p.a_up + at);
      float4 f, d;
      act_both_any(p.act, g.x, f.x, d.x);
      act_both_any(p.act, g.y, f.y, d.y);
      act_both_any(p.act, g.z, f.z, d.z);
      act_both_any(p.act, g.w, f.w, d.w);
      put_bf16x4(p.out + at, f.x * u.x, f.y * u.y, f.z * u.z, f.w * u.w);
      put_bf16x4(p.da_gate + at, s.x * u.x * d.x, s.y * u.y * d.y, s.z * u.z * d.z,
                 s.w * u.w * d.w);
      put_bf16x4(p.da_up + at, s.x * f.x, s.y * f.y, s.z * f.z, s.w * f.w);
    } else {
      if (p.add) {
        const float4 a = bf16x4(p.add + at);
        s.x += a.x;
        s.y += a.y;
        s.z += a.z;
        s.w += a.w;
      }
      put_bf16x4(p.out + at, s.x, s.y, s.z, s.w);
    }
  }
  if (p.split > 1) cluster_sync();               // the others have read this CTA's sums
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
}

constexpr size_t kSmemBytes = 1024 + kRingBytes + sizeof(Smem);
static_assert(2 * (kSmemBytes + 1024) <= 233472, "two CTAs an SM");
static_assert(kFewRows * 128 * sizeof(float) <= kRingBytes, "the sums take the ring's place");
static_assert(kFewRows <= 128, "columns of tensor memory");

// CTAs to a cluster: as many as two an SM take, each with a k-block at least.
int pick_split(int tiles, int kb) {
  int s = 1;
  while (s < 8 && 2 * s <= kb && tiles * 2 * s <= 2 * device_sm_count()) s *= 2;
  return s;
}

template <Op op>
cudaError_t launch(const Maps& maps, Args p, cudaStream_t st) {
  auto kern = rows_kernel<op>;
  static bool configured[kMaxDevices] = {};
  const int d = current_device();
  if (d < 0 || d >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!configured[d]) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(kSmemBytes));
    if (e != cudaSuccess) return e;
    configured[d] = true;
  }
  p.tn = (p.T + 15) / 16 * 16;
  p.tmem_cols = p.tn <= 32 ? 32 : p.tn <= 64 ? 64 : 128;
  const int stage_bytes = kWBytes + p.tn * BK * 2;
  p.stages = kRingBytes / stage_bytes < kMaxStages ? kRingBytes / stage_bytes : kMaxStages;
  const int cols = op == Op::Gated ? 64 : 128, tiles = (p.N + cols - 1) / cols;
  p.split = pick_split(tiles, p.kb);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(tiles * p.split);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = op == Op::Down || op == Op::InGrad ? 2 : 1;   // those run beside the one before
  return cudaLaunchKernelEx(&cfg, kern, maps, p);
}

bool rows_map(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint32_t box_outer) {
  return make_tmap_bf16_2d(m, base, inner, outer, inner * 2, BK, box_outer);
}

}  // namespace

cudaError_t ffn_few_rows(const void* x, const void* w_gate, const void* w_up, const void* w_down,
                         const void* add, int T, int H, int F, int act, void* y, void* a_gate,
                         void* a_up, void* h, int* err, cudaStream_t st) {
  Maps m1{}, m2{};
  const uint32_t rows = static_cast<uint32_t>((T + 15) / 16 * 16);
  if (!rows_map(&m1.w[0], w_gate, F, H, BK) || !rows_map(&m1.w[1], w_up, F, H, BK) ||
      !rows_map(&m1.x[0], x, H, T, rows) || !rows_map(&m2.w[0], w_down, H, F, BK) ||
      !rows_map(&m2.x[0], h, F, T, rows))
    return cudaErrorInvalidValue;
  Args p{};
  p.T = T;
  p.N = F;
  p.kb = p.kb0 = (H + BK - 1) / BK;
  p.act = act;
  p.out = static_cast<__nv_bfloat16*>(h);
  p.a_gate = static_cast<__nv_bfloat16*>(a_gate);
  p.a_up = static_cast<__nv_bfloat16*>(a_up);
  p.err = err;
  p.wait_ns = kDefaultWaitNs;
  const cudaError_t e = launch<Op::Gated>(m1, p, st);
  if (e != cudaSuccess) return e;
  p.N = H;
  p.kb = p.kb0 = (F + BK - 1) / BK;
  p.add = static_cast<const __nv_bfloat16*>(add);
  p.out = static_cast<__nv_bfloat16*>(y);
  return launch<Op::Down>(m2, p, st);
}

cudaError_t ffn_few_rows_backward(const void* dy, const void* w_gate, const void* w_up,
                                  const void* w_down, const void* a_gate, const void* a_up,
                                  const void* add, int T, int H, int F, int act, void* dx, void* h,
                                  void* da_gate, void* da_up, int* err, cudaStream_t st) {
  Maps m1{}, m2{};
  const uint32_t rows = static_cast<uint32_t>((T + 15) / 16 * 16);
  if (!rows_map(&m1.w[0], w_down, H, F, 128) || !rows_map(&m1.x[0], dy, H, T, rows) ||
      !rows_map(&m2.w[0], w_gate, F, H, 128) || !rows_map(&m2.w[1], w_up, F, H, 128) ||
      !rows_map(&m2.x[0], da_gate, F, T, rows) || !rows_map(&m2.x[1], da_up, F, T, rows))
    return cudaErrorInvalidValue;
  Args p{};
  p.T = T;
  p.N = F;
  p.kb = p.kb0 = (H + BK - 1) / BK;
  p.act = act;
  p.out = static_cast<__nv_bfloat16*>(h);
  p.a_gate = static_cast<__nv_bfloat16*>(const_cast<void*>(a_gate));
  p.a_up = static_cast<__nv_bfloat16*>(const_cast<void*>(a_up));
  p.da_gate = static_cast<__nv_bfloat16*>(da_gate);
  p.da_up = static_cast<__nv_bfloat16*>(da_up);
  p.err = err;
  p.wait_ns = kDefaultWaitNs;
  const cudaError_t e = launch<Op::GatedBwd>(m1, p, st);
  if (e != cudaSuccess) return e;
  p.N = H;
  p.kb0 = (F + BK - 1) / BK;
  p.kb = 2 * p.kb0;
  p.add = static_cast<const __nv_bfloat16*>(add);
  p.out = static_cast<__nv_bfloat16*>(dx);
  return launch<Op::InGrad>(m2, p, st);
}

}  // namespace moe
