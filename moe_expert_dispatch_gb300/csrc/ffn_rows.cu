// ffn_rows.cu - the forward of the gated feed-forward block for few rows (a
// decoding step): both products bound by reading the weights once.
//
// The roles of the operands are exchanged: 128 columns of the weights are the M of
// a tile and the tokens its N (16 to 128), so that a tile is full of weights however
// few the tokens are. In the first product the 128 are 64 columns of W_gate and the
// same 64 of W_up, and the tile ends with A_g and A_u of 64 columns of h.
//
// The weights arrive by TMA, 64 of K at a time (16 KB), into a ring that keeps 100
// KB of loads under way in each of two CTAs an SM: 30 MB over the GPU, where the
// memory's rate times its latency asks for about 8. K is split over the CTAs of a
// cluster (up to 8) so that narrow layers fill the GPU too; the cluster adds its
// sums up through shared memory in the order of the ranks, each CTA finishing every
// C-th token, and no sum depends on timing. The second product is launched while the
// first runs (programmatic dependent launch): its rings fill with W_down before it
// waits for h.
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

struct Maps {
  CUtensorMap w[2], x;
};

struct Args {
  int T, tn;             // rows, and rounded up to the MMA's N
  int N, kb;             // columns of the result, k-blocks
  int split;             // CTAs of a cluster
  int stages;
  int tmem_cols;
  int act;
  const __nv_bfloat16* add;
  __nv_bfloat16* out;    // h or y
  __nv_bfloat16* a_gate;
  __nv_bfloat16* a_up;
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

// A cluster takes one tile of weight columns, each of its CTAs a run of k-blocks.
template <bool kGated>
__global__ void __launch_bounds__(kThreads)
    rows_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Smem* sm = reinterpret_cast<Smem*>(ring + kRingBytes);
  const int warp = threadIdx.x >> 5, lane = lane_id();
  const uint32_t rank = cluster_ctarank();
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
  if (kGated) grid_dependents_launch();

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t ring0 = smem_u32(ring);
      const uint64_t pol = l2_policy_evict_first();     // weights are read once
      auto load_w = [&](int kb, int s) {
        const uint32_t bar = smem_u32(&sm->full[s]), sa = ring0 + s * stage_bytes;
        mbar_arrive_expect_tx(bar, stage_bytes);
        tma_load_2d_hint(sa, &maps.w[0], bar, n0, kb * BK, pol);
        tma_load_2d_hint(sa + kBox, &maps.w[kGated ? 1 : 0], bar, kGated ? n0 : n0 + 64, kb * BK,
                         pol);
      };
      auto load_x = [&](int kb, int s) {
        tma_load_2d(ring0 + s * stage_bytes + kWBytes, &maps.x, smem_u32(&sm->full[s]), kb * BK, 0);
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
      // weights: MN-major atoms of 64 columns, 8 KB apart; rows of x: K-major
      const uint32_t idesc = idesc_bf16(128, p.tn, true, false);
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
        const uint64_t ad = sdesc_sw128(sa, kBox, 1024), bd = sdesc_sw128(sa + kWBytes, 16, 1024);
#pragma unroll
        for (int ks = 0; ks < BK / 16; ++ks)
          umma_bf16(tmem, ad + ks * (2048 >> 4), bd + ks * (32 >> 4), idesc,
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
      if (p.a_gate && col < p.N)
        *reinterpret_cast<uint2*>((up ? p.a_up : p.a_gate) + at) =
            make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
      const float ux = __shfl_down_sync(0xffffffffu, s.x, 16);
      const float uy = __shfl_down_sync(0xffffffffu, s.y, 16);
      const float uz = __shfl_down_sync(0xffffffffu, s.z, 16);
      const float uw = __shfl_down_sync(0xffffffffu, s.w, 16);
      if (!up && col < p.N)
        *reinterpret_cast<uint2*>(p.out + at) =
            make_uint2(pack_bf16x2(act_any(p.act, s.x) * ux, act_any(p.act, s.y) * uy),
                       pack_bf16x2(act_any(p.act, s.z) * uz, act_any(p.act, s.w) * uw));
    } else {
      const int col = n0 + lane * 4;
      if (col < p.N) {
        const int64_t at = static_cast<int64_t>(t) * p.N + col;
        if (p.add) {
          const uint2 a = *reinterpret_cast<const uint2*>(p.add + at);
          s.x += __uint_as_float(a.x << 16);
          s.y += __uint_as_float(a.x & 0xFFFF0000u);
          s.z += __uint_as_float(a.y << 16);
          s.w += __uint_as_float(a.y & 0xFFFF0000u);
        }
        *reinterpret_cast<uint2*>(p.out + at) =
            make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
      }
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

// CTAs to a cluster: as many as two an SM take, each with a k-block at least.
int pick_split(int tiles, int kb) {
  int s = 1;
  while (s < 8 && 2 * s <= kb && tiles * 2 * s <= 2 * device_sm_count()) s *= 2;
  return s;
}

template <bool kGated>
cudaError_t launch(const Maps& maps, Args p, cudaStream_t st) {
  auto kern = rows_kernel<kGated>;
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
  const int cols = kGated ? 64 : 128, tiles = (p.N + cols - 1) / cols;
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
  cfg.numAttrs = kGated ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, kern, maps, p);
}

}  // namespace

cudaError_t ffn_few_rows(const void* x, const void* w_gate, const void* w_up, const void* w_down,
                         const void* add, int T, int H, int F, int act, void* y, void* a_gate,
                         void* a_up, void* h, int* err, cudaStream_t st) {
  Maps m1, m2;
  const uint32_t rows = static_cast<uint32_t>((T + 15) / 16 * 16);
  const uint64_t rF = static_cast<uint64_t>(F) * 2, rH = static_cast<uint64_t>(H) * 2;
  if (!make_tmap_bf16_2d(&m1.w[0], w_gate, F, H, rF, 64, BK) ||
      !make_tmap_bf16_2d(&m1.w[1], w_up, F, H, rF, 64, BK) ||
      !make_tmap_bf16_2d(&m1.x, x, H, T, rH, BK, rows) ||
      !make_tmap_bf16_2d(&m2.w[0], w_down, H, F, rH, 64, BK) ||
      !make_tmap_bf16_2d(&m2.x, h, F, T, rF, BK, rows))
    return cudaErrorInvalidValue;
  m2.w[1] = m2.w[0];
  Args p{};
  p.T = T;
  p.N = F;
  p.kb = (H + BK - 1) / BK;
  p.act = act;
  p.out = static_cast<__nv_bfloat16*>(h);
  p.a_gate = static_cast<__nv_bfloat16*>(a_gate);
  p.a_up = static_cast<__nv_bfloat16*>(a_up);
  p.err = err;
  p.wait_ns = kDefaultWaitNs;
  const cudaError_t e = launch<true>(m1, p, st);
  if (e != cudaSuccess) return e;
  p.N = H;
  p.kb = (F + BK - 1) / BK;
  p.add = static_cast<const __nv_bfloat16*>(add);
  p.out = static_cast<__nv_bfloat16*>(y);
  return launch<false>(m2, p, st);
}

}  // namespace moe
