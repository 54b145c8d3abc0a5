// lora.cu - low-rank adapters of many requests beside a shared projection
// (moe_lora_plan, moe_lora, moe_lora_backward).
//
// With A and B both stored rank-major ([n, r, H] and [n, r, N]), forward and
// backward need three products only, each over the rows of one adapter:
//   shrink  V[t, j]   = sum_c in[t, c] P[j, c]              v from x, A; dv from dy, B
//   expand  out[t, c] = base[t, c] + sum_j s V[t, j] Q[j, c]   out from v, B; dx from dv, A
//   grad    G[j, c]   = sum_t s V[t, j] in[t, c]            dA from dv, x; dB from v, dy
// The widths are thousands and the rank is at most 128, so all three are bound by
// the rows that they read and write; the products go through tcgen05.mma, which
// leaves the SMs to move rows.
//
// Rows are taken in the order of the plan, 128 of one adapter at a time (a unit).
// A plan comes from the caller: every row number is checked against T before use.
//
// V is float. Where it enters a product it is a sum of bf16 numbers: two of them
// (16 bits) for expand, whose result is rounded to bf16, and three (24 bits) for
// grad, whose result is float. The shrink kernel writes them as images: the parts of
// a unit's rows side by side, parts * R columns in atoms of 64 rows x 64 columns, in
// the swizzled order in which the tensor cores read shared memory, so that bulk
// copies bring them in, as a K-major operand to expand and as an MN-major one to
// grad. Rows past the end of an adapter are zeros there.
//
// The tensor cores add their products up in float but cut off what does not fit;
// over thousands of terms that bias shows in float results. So shrink and grad
// take their accumulators out of tensor memory every 128 or 64 terms and add them up
// in float registers, which round.
#include <string.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

int* device_error_word();

namespace {

constexpr int kRows = 128;          // rows of a unit: one adapter's
constexpr int kMaxAdapters = 1024;
constexpr int kMaxRank = 128;
// Offsets that overlap can name every row 512 times: with so many rows the sums of
// units and chunks stay below 2^31 whatever a plan holds.
constexpr int64_t kMaxRows = 1 << 27;
constexpr unsigned long long kDrainNs = 1000000000ull;
constexpr int kAtom = kRows * 128;  // 16 KB: 128 rows x 64 columns of an image or a tile
// 64-wide atoms of an image of so many parts
__host__ __device__ constexpr int atoms(int parts, int R) { return (parts * R + 63) / 64; }

// 16 bytes global -> shared, or 16 zero bytes where ok is false (src is then
// any valid address and nothing is read).
__device__ __forceinline__ void cp_async_16z(uint32_t dst, const void* src, bool ok) {
  const int n = ok ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(n)
               : "memory");
}

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(addr, rank)) : "memory");
  return v;
}

// The next bf16 part of two values, packed; what is left of them stays. What is not
// finite is in the first part alone.
__device__ __forceinline__ uint32_t take_part(float& v0, float& v1) {
  const uint32_t w = pack_bf16x2(v0, v1);
  const float h0 = __uint_as_float(w << 16), h1 = __uint_as_float(w & 0xFFFF0000u);
  v0 = fabsf(h0) < INFINITY ? v0 - h0 : 0.0f;
  v1 = fabsf(h1) < INFINITY ? v1 - h1 : 0.0f;
  return w;
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// R consecutive accumulator columns of this lane added to sum.
template <int R>
__device__ __forceinline__ void add_columns(uint32_t taddr, float* sum) {
#pragma unroll
  for (int c = 0; c < R; c += 16) {
    uint32_t v[16];
    tmem_ld_32x32b_x16(taddr + c, v);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) sum[c + i] += __uint_as_float(v[i]);
  }
}

// ------------------------------------------------------------------ plan

struct Plan {
  const int32_t* order;
  const int32_t* offsets;
  int64_t T;
  int n;
  int* err;
};

// The rows of adapter a (a = n: those without one), as [lo, hi) of the order; an
// offset that does not fit is reported and cut.
__device__ __forceinline__ void segment(const Plan& p, int a, int& lo, int& hi) {
  const int T = static_cast<int>(p.T);
  const int l = __ldg(p.offsets + a), h = a < p.n ? __ldg(p.offsets + a + 1) : T;
  lo = min(max(l, 0), T);
  hi = min(max(h, lo), T);
  if (lo != l || hi != h || (a == 0 && l != 0)) report_error(p.err, kErrBadId);
}

// A row number of the order, or -1 (reported) where it is no row.
__device__ __forceinline__ int checked_row(const Plan& p, int r) {
  if (r >= 0 && r < p.T) return r;
  report_error(p.err, kErrBadId);
  return -1;
}

struct Unit { int a, lo, rows; };   // adapter, first entry of the order, rows (0: none)

// Unit u of the batch: the adapters' units one after the other, those of rows without
// an adapter last. Called by a whole warp.
__device__ __forceinline__ Unit find_unit(const Plan& p, int u) {
  const int lane = lane_id();
  Unit b = {-1, 0, 0};
  int before = 0;
  for (int a0 = 0; a0 <= p.n; a0 += 32) {
    int lo = 0, hi = 0;
    const int a = a0 + lane;
    if (a <= p.n) segment(p, a, lo, hi);
    const int mine = (hi - lo + kRows - 1) / kRows;
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += o;
    }
    const int first = before + sum - mine;
    const unsigned hit = __ballot_sync(0xffffffffu, u >= first && u < first + mine);
    if (hit) {
      const int src = __ffs(hit) - 1;
      b.a = a0 + src;
      const int l = __shfl_sync(0xffffffffu, lo, src), h = __shfl_sync(0xffffffffu, hi, src);
      b.lo = l + (u - __shfl_sync(0xffffffffu, first, src)) * kRows;
      b.rows = min(kRows, h - b.lo);
      return b;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  return b;
}

// The units of a batch, those of rows without an adapter where none is set. Called by a
// whole warp.
__device__ __forceinline__ int count_units(const Plan& p, bool none) {
  int sum = 0;
  for (int a = lane_id(); a < p.n + (none ? 1 : 0); a += 32) {
    int lo, hi;
    segment(p, a, lo, hi);
    sum += (hi - lo + kRows - 1) / kRows;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  return sum;
}

// Stable counting sort by adapter in one cluster: each warp counts a run of rows, one
// scan over adapters, CTAs and warps gives every run its places, and each warp then
// deals its rows out, 32 at a time: which of them share an adapter comes from a ballot
// for each bit of the id. Eight loads of a lane are under way at once; what bounds it is
// the ballots' issue, which eight CTAs share.
constexpr int kIdLoads = 8;
constexpr int kPlanCtas = 8;
// Rows up to which one CTA sorts alone, spared the cluster's two barriers. 64 rows of 8
// adapters take 2.8 us so and 4.2 by eight CTAs, 4096 5.0 both ways; 65536 of 64 47 and 10.
constexpr int64_t kPlanRows = 4096;

// The ids of rows t, t + 32, ... below t1 as they are.
__device__ __forceinline__ void plan_keys(const int32_t* ids, int64_t t, int64_t t1, int* key) {
#pragma unroll
  for (int i = 0; i < kIdLoads; ++i) key[i] = t + 32 * i < t1 ? __ldg(ids + t + 32 * i) : -1;
}

__global__ void __launch_bounds__(1024, 1)
    plan_kernel(const int32_t* ids, int64_t T64, int n, int32_t* order, int32_t* offsets, int* err) {
  extern __shared__ int plan_smem[];
  const int keys = n + 1, T = static_cast<int>(T64);
  int* place = plan_smem;                       // [32][keys]: of a warp, before it in the CTA
  int* count = place + 32 * keys;               // [keys]: the CTA's
  const int rank = static_cast<int>(cluster_ctarank()), ctas = static_cast<int>(gridDim.x);
  int* total = ctas > 1 ? count + keys : count; // [keys]: of all CTAs, then where they begin
  const int warp = threadIdx.x >> 5, lane = lane_id();
  for (int i = threadIdx.x; i < 32 * keys; i += 1024) place[i] = 0;
  __syncthreads();
  const int64_t run = (T64 + 1024 * ctas - 1) / (1024 * ctas) * 32;   // rows of a warp
  const int64_t t0 = (rank * 32 + warp) * run, t1 = min(t0 + run, T64);
  int* mine = place + warp * keys;
  for (int64_t t = t0 + lane; t - lane < t1; t += 32 * kIdLoads) {
    int key[kIdLoads];
    plan_keys(ids, t, t1, key);
#pragma unroll
    for (int i = 0; i < kIdLoads; ++i) {
      if (t + 32 * i >= t1) break;
      if (key[i] < -1 || key[i] >= n) report_error(err, kErrBadId);
      atomicAdd(mine + (key[i] < 0 || key[i] >= n ? n : key[i]), 1);   // counts: no order
    }
  }
  __syncthreads();
  for (int k = threadIdx.x; k < keys; k += 1024) {
    int sum = 0;
    for (int w = 0; w < 32; ++w) {
      const int c = place[w * keys + k];
      place[w * keys + k] = sum;
      sum += c;
    }
    count[k] = sum;
  }
  if (ctas > 1) {
    cluster_sync();
    for (int k = threadIdx.x; k < keys; k += 1024) {
      int sum = 0, before = 0;                   // over the CTAs, and those before this one
      for (int q = 0; q < ctas; ++q) {
        const int c = __float_as_int(ld_cluster_f32(smem_u32(count + k), q));
        if (q < rank) before += c;
        sum += c;
      }
      total[k] = sum;
      for (int w = 0; w < 32; ++w) place[w * keys + k] += before;
    }
    cluster_sync();                              // the others have read this CTA's counts
  } else {
    __syncthreads();
  }
  if (warp == 0) {
    int before = 0;
    for (int k0 = 0; k0 < keys; k0 += 32) {
      const int c = k0 + lane < keys ? total[k0 + lane] : 0;
      int sum = c;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += o;
      }
      if (k0 + lane < keys) {
        total[k0 + lane] = before + sum - c;
        // keys = n + 1 offsets: the last is where none begin
        if (rank == 0) offsets[k0 + lane] = before + sum - c;
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
  __syncthreads();
  const int bits = 32 - __clz(n);                // of the keys 0 to n
  for (int64_t t = t0 + lane; t - lane < t1; t += 32 * kIdLoads) {
    int key[kIdLoads];
    plan_keys(ids, t, t1, key);
#pragma unroll
    for (int i = 0; i < kIdLoads; ++i) {
      if (t - lane + 32 * i >= t1) break;        // the whole warp
      const bool row = t + 32 * i < t1;
      const int k = key[i] < 0 || key[i] >= n ? n : key[i];
      unsigned same = __ballot_sync(0xffffffffu, row);
      for (int b = 0; b < bits; ++b) {
        const bool set = (k >> b) & 1;
        const unsigned m = __ballot_sync(0xffffffffu, set);
        same &= set ? m : ~m;
      }
      int at = T;
      if (row) at = total[k] + mine[k] + __popc(same & ((1u << lane) - 1));
      __syncwarp();
      if (at < T) order[at] = static_cast<int32_t>(t + 32 * i);
      if (row && lane == __ffs(same) - 1) mine[k] += __popc(same);
      __syncwarp();
    }
  }
}

// ------------------------------------------------------------------ shrink

// A cluster takes a unit, each of its CTAs a run of 64-wide k-blocks; the sums are
// added over the cluster in the order of the ranks, and each CTA splits and writes
// its share. Warps: 0 loads P by TMA, 1 issues the MMAs, then 4 (a quarter of the
// accumulators' rows each) or 8 (and half of their columns) drain the accumulators,
// and 4 gather the rows (cp.async, 128 bytes a row and k-block). Boxes by TMA where the
// rows follow one another were no faster (16384 rows of 4096, r = 64: 164 us the whole
// backward both ways). Bound by the rows: 8192 of 4096, r = 16, take 19.5 us, 3.4 TB/s,
// 16384 with r = 64 and the images of both V 37 us, 4.0 TB/s; what is missing to the
// memory's rate is the start and end of CTAs that live for 30 k-blocks or fewer.
constexpr int kBlocks = 2;          // k-blocks that an accumulator takes up

template <int R>
struct Shrink {
  static constexpr int kStages = R <= 16 ? 6 : R <= 32 ? 5 : 4;   // two CTAs an SM up to 64
  static constexpr int kStage = kAtom + R * 128;
  static constexpr int kAcc = R > 64 ? 2 : 4;       // accumulators in flight
  static constexpr int kTmem = R <= 16 ? 64 : R <= 32 ? 128 : 256;
  static constexpr int kRing = kStages * kStage;
  static constexpr int kBytes = 1024 + (kRing > kRows * R * 4 ? kRing : kRows * R * 4);
  static constexpr int kGroups = R > 32 ? 2 : 1;    // draining warps to a quarter of the rows
  static constexpr int kOwn = R / kGroups;          // columns of such a warp
  static constexpr int kThreads = 32 * (2 + 4 * kGroups + 4);
};

struct ShrinkArgs {
  const __nv_bfloat16* in;     // [T, K]
  const float* scales;         // or NULL
  float* V;                    // [T, r] or NULL: the sums, without the scale
  uint8_t* img;                // images of s V
  const float* kept;           // [T, r] or NULL: another V that is split as well
  uint8_t* img_kept;
  int parts;                   // of each image: 2 or 3
  int K, r, split;
  unsigned long long wait_ns;
  Plan plan;
};

// Columns 8 c to 8 c + 7 of a row of V into the image of its unit, part by part.
template <int R>
__device__ __forceinline__ void put_parts(uint8_t* img, int unit, int row, int c, int parts, float* v) {
  const int64_t at = (static_cast<int64_t>(unit) * 2 + (row >> 6)) * atoms(parts, R) * (kAtom / 2) +
                     (row & 63) * 128;
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (k < parts) {
      const int piece = k * (R / 8) + c;         // of 16 bytes, of the row
      uint4 w;
      w.x = take_part(v[0], v[1]);
      w.y = take_part(v[2], v[3]);
      w.z = take_part(v[4], v[5]);
      w.w = take_part(v[6], v[7]);
      *reinterpret_cast<uint4*>(img + at + (piece >> 3) * (kAtom / 2) +
                                (((piece & 7) ^ (row & 7)) << 4)) = w;
    }
}

template <int R>
__global__ void __launch_bounds__(Shrink<R>::kThreads, R > 64 ? 1 : 2)
    shrink_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ ShrinkArgs p) {
  using S = Shrink<R>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int rows[kRows];
  __shared__ uint64_t full[S::kStages], empty[S::kStages], tfull[S::kAcc], tempty[S::kAcc];
  __shared__ uint32_t tmem_at;
  __shared__ int stop, zero;
  uint8_t* ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t rank = cluster_ctarank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int unit = static_cast<int>(blockIdx.x) / p.split;
  const Unit u = find_unit(p.plan, unit);
  // on its way while the barriers are made
  const int raw = tid < u.rows ? __ldg(p.plan.order + u.lo + tid) : 0;
  if (u.rows == 0 || u.a == p.plan.n) {         // the whole cluster leaves together
    if (tid < kRows) rows[tid] = tid < u.rows ? checked_row(p.plan, raw) : -1;
    __syncthreads();
    if (rank == 0 && p.V)
      for (int i = tid; i < u.rows * p.r; i += S::kThreads)
        if (rows[i / p.r] >= 0) p.V[static_cast<int64_t>(rows[i / p.r]) * p.r + i % p.r] = 0.0f;
    return;
  }
  if (tid == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1 + 128);   // P's bytes, and a lane of the gathering warps each
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int a = 0; a < S::kAcc; ++a) {
      mbar_init(smem_u32(&tfull[a]), 1);
      mbar_init(smem_u32(&tempty[a]), 4 * S::kGroups);
    }
    stop = 0;
    zero = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_at), S::kTmem);
    tmem_relinquish();
  }
  if (tid < kRows) rows[tid] = tid < u.rows ? checked_row(p.plan, raw) : -1;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_at;
  const int kblocks = (p.K + 63) / 64, per = (kblocks + p.split - 1) / p.split;
  const int kb0 = min(kblocks, static_cast<int>(rank) * per), kb1 = min(kblocks, kb0 + per);
  const int steps = kb1 - kb0;
  const float f = p.scales ? __ldg(p.scales + u.a) : 1.0f;
  volatile int* stopped = &stop;
  bool ok = true;
  float sum[S::kOwn];                            // of a draining warp's lane
  const int j0 = ((warp - 2) >> 2) * S::kOwn;    // and its first column
#pragma unroll
  for (int j = 0; j < S::kOwn; ++j) sum[j] = 0.0f;

  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < steps; ++i) {
        const int s = i % S::kStages;
        ok = mbar_wait(smem_u32(&empty[s]), ((i / S::kStages) & 1) ^ 1, p.wait_ns, stopped);
        if (!ok) break;
        mbar_arrive_expect_tx(smem_u32(&full[s]), R * 128);
        tma_load_3d(smem_u32(ring) + s * S::kStage + kAtom, &map_p, smem_u32(&full[s]),
                    (kb0 + i) * 64, 0, u.a);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16(128, R, false, false);
      for (int i = 0; i < steps; ++i) {
        const int s = i % S::kStages, d = i / kBlocks, a = d % S::kAcc;
        ok = (i % kBlocks || mbar_wait(smem_u32(&tempty[a]), ((d / S::kAcc) & 1) ^ 1, p.wait_ns,
                                       stopped)) &&
             mbar_wait(smem_u32(&full[s]), (i / S::kStages) & 1, p.wait_ns, stopped);
        if (!ok) break;
        fence_proxy_async_shared();              // the gathered rows came through the generic proxy
        tc_fence_after();
        const uint32_t sa = smem_u32(ring) + s * S::kStage;
        const uint64_t ad = sdesc_sw128(sa, 16, 1024), bd = sdesc_sw128(sa + kAtom, 16, 1024);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          umma_bf16(tmem + a * R, ad + ks * 2, bd + ks * 2, idesc, (i % kBlocks || ks) ? 1u : 0u);
        umma_commit(smem_u32(&empty[s]));
        if (i % kBlocks == kBlocks - 1 || i + 1 == steps) umma_commit(smem_u32(&tfull[a]));
      }
    }
  } else if (warp < 2 + 4 * S::kGroups) {
    const uint32_t taddr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + j0;
    for (int d = 0; d * kBlocks < steps; ++d) {
      const int a = d % S::kAcc;
      const bool got = mbar_wait(smem_u32(&tfull[a]), (d / S::kAcc) & 1, p.wait_ns, stopped);
      ok = __all_sync(0xffffffffu, got);
      if (!ok) break;
      tc_fence_after();
      add_columns<S::kOwn>(taddr + a * R, sum);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&tempty[a]));
    }
  } else {
    const int g = tid - (S::kThreads - 128), ch = g & 7, r0 = g >> 3;
    const __nv_bfloat16* src[8];
    bool live[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = rows[r0 + 16 * i];
      live[i] = row >= 0;
      src[i] = p.in + static_cast<int64_t>(live[i] ? row : 0) * p.K + ch * 8;
    }
    for (int i = 0; i < steps; ++i) {
      const int s = i % S::kStages, k0 = (kb0 + i) * 64;
      const bool got = mbar_wait(smem_u32(&empty[s]), ((i / S::kStages) & 1) ^ 1, p.wait_ns, stopped);
      ok = __all_sync(0xffffffffu, got);
      if (!ok) break;
      const uint32_t sa = smem_u32(ring) + s * S::kStage;
      const bool in_k = k0 + ch * 8 < p.K;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int row = r0 + 16 * j;
        const bool here = live[j] && in_k;
        cp_async_16z(sa + row * 128 + ((ch ^ (row & 7)) << 4), here ? src[j] + k0 : p.in, here);
      }
      cp_async_arrive_noinc(smem_u32(&full[s]));
    }
    // the other V, while the last rows come in
    if (p.kept) {
#pragma unroll 2
      for (int e = static_cast<int>(rank) + p.split * g; e < kRows * (R / 8); e += p.split * 128) {
        const int row = e / (R / 8), c = e % (R / 8), t = rows[row];
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[j] = (t >= 0 && c * 8 + j < p.r)
                     ? f * __ldg(p.kept + static_cast<int64_t>(t) * p.r + c * 8 + j)
                     : 0.0f;
        put_parts<R>(p.img_kept, unit, row, c, p.parts, v);
      }
    }
    cp_commit();
    cp_wait<0>();
  }
  if (!ok) {
    stop = 1;
    report_error(p.plan.err, kErrTimeout);
    // what is under way lands (or is given up on) before the CTA goes on
    if (warp == 0 && lane == 0)
      for (int s = 0; s < S::kStages; ++s) mbar_wait(smem_u32(&full[s]), 0, kDrainNs / 8, &zero);
  }
  __syncthreads();                               // the ring has been read

  // sums as [row][column], 16-byte piece c of row i at c ^ (i & kMix)
  constexpr int kMix = R >= 32 ? 7 : 3;
  float* part = reinterpret_cast<float*>(ring);
  if (warp >= 2 && warp < 2 + 4 * S::kGroups) {
    const int row = (warp & 3) * 32 + lane;
#pragma unroll
    for (int j = 0; j < S::kOwn; j += 4)
      *reinterpret_cast<float4*>(part + row * R + ((((j0 + j) >> 2) ^ (row & kMix)) << 2)) =
          make_float4(sum[j], sum[j + 1], sum[j + 2], sum[j + 3]);
  }
  if (p.split > 1) cluster_sync();
  else __syncthreads();
  const uint32_t part0 = smem_u32(part);
  // eight columns of a row at a time, dealt out over the cluster
  for (int e = static_cast<int>(rank) + p.split * tid; e < kRows * (R / 8);
       e += p.split * S::kThreads) {
    const int row = e / (R / 8), c = e % (R / 8);
    const int g = rows[row];
    const uint32_t at0 = part0 + (row * R + (((2 * c) ^ (row & kMix)) << 2)) * 4;
    const uint32_t at1 = part0 + (row * R + (((2 * c + 1) ^ (row & kMix)) << 2)) * 4;
    float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int q0 = 0; q0 < 8; q0 += 4)
      if (q0 < p.split) {
        float4 a[4], b[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {            // all of them on their way at once
          a[q] = b[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (q0 + q < p.split) {
            a[q] = ld_cluster_f32x4(at0, q0 + q);
            b[q] = ld_cluster_f32x4(at1, q0 + q);
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          v[0] += a[q].x;
          v[1] += a[q].y;
          v[2] += a[q].z;
          v[3] += a[q].w;
          v[4] += b[q].x;
          v[5] += b[q].y;
          v[6] += b[q].z;
          v[7] += b[q].w;
        }
      }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (g < 0 || c * 8 + j >= p.r) {
        v[j] = 0.0f;                             // whatever the scale is
      } else {
        if (p.V) p.V[static_cast<int64_t>(g) * p.r + c * 8 + j] = v[j];
        v[j] *= f;
      }
    }
    put_parts<R>(p.img, unit, row, c, p.parts, v);
  }
  tc_fence_before();
  if (p.split > 1) cluster_sync();               // the others have read this CTA's sums
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmem);
  }
}

// ------------------------------------------------------------------ expand

// The work is a list of items (unit, tile of 64 columns), the tiles running fastest, of
// which two CTAs an SM (one for more than 64 ranks) take equal runs, however many units
// the plan has; warp 0 prepares the next unit of a run while the last one's tiles are
// finished. CTAs dealt out by the number of units that there may be took 258 us instead of
// 160 for 16384 mixed rows of 32 adapters, 4096 x 6144 (one CTA a unit: half of the GPU),
// 51 and 48 for 8192 rows of 16, and 24.0 and 25.5 for 700 of 32.
// Warps: 0 loads the image and Q, 1 issues the MMAs, 2 to 5 finish every second tile and 6
// to 9 the others: base comes in by runs of 128 bytes a row, a tile ahead in registers,
// and goes through 4 KB of shared memory a warp, in which each lane adds its row of the
// accumulator, back into runs of 128 bytes. Bound by base and out, and by the instructions
// of that way: 8192 rows of 4096, r = 16, take 28 us, 4.8 TB/s; 16384, r = 64, 50 us, 5.4
// TB/s. Launched beside the shrink kernel (as far as its results let it) both were slower,
// the 8192 53 us in all against 49: its CTAs take the room in which shrink's next ones start.
constexpr int kCols = 64;
constexpr int kPiece = 32 * 128;
constexpr int kExpandThreads = 320;
constexpr int kExpandAcc = 4;                     // accumulators: two to each half of the warps

template <int R>
struct Expand {
  static constexpr int kImg = atoms(2, R) * kAtom;
  static constexpr int kQ = R * 128;
  static constexpr int kStages = 3;
  static constexpr int kBytes = 1024 + kImg + kStages * kQ + 8 * kPiece;
};

// Where the items of CTA b of all begin. Tensors that fit in memory have fewer than 2^32.
__device__ __forceinline__ uint32_t items_begin(uint32_t items, uint32_t all, uint32_t b) {
  return items / all * b + min(b, items % all);
}

// What a CTA does of one unit: steps tiles from t0 on.
struct Part { int unit, a, rows, t0, steps; };

struct ExpandArgs {
  const uint8_t* img;
  int parts;                      // of the image; the first two are used
  const __nv_bfloat16* base;      // or NULL
  __nv_bfloat16* out;
  int N;
  int units;                      // that the images have room for
  unsigned long long wait_ns;
  Plan plan;
};

template <int R>
__global__ void __launch_bounds__(kExpandThreads, R > 64 ? 1 : 2)
    expand_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ ExpandArgs p) {
  using S = Expand<R>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int rows_of[2][kRows];               // of this part and of the next
  __shared__ Part parts[2];
  __shared__ uint32_t at, past;                   // items that no part has yet
  __shared__ uint64_t full[S::kStages], empty[S::kStages], tfull[kExpandAcc], tempty[kExpandAcc],
      image;
  __shared__ uint32_t tmem_at;
  __shared__ int stop, zero;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t tiles = (p.N + kCols - 1) / kCols;
  // the next part, by warp 0; no steps: there is none
  auto prepare = [&](int k) {
    if (at >= past) {
      if (lane == 0) parts[k].steps = 0;
      return;
    }
    const uint32_t unit = at / tiles, t0 = at - unit * tiles, steps = min(tiles - t0, past - at);
    const Unit u = find_unit(p.plan, static_cast<int>(unit));
#pragma unroll
    for (int r = 0; r < kRows; r += 32)
      rows_of[k][r + lane] =
          r + lane < u.rows ? checked_row(p.plan, __ldg(p.plan.order + u.lo + r + lane)) : -1;
    __syncwarp();
    if (lane == 0) {
      parts[k] = {static_cast<int>(unit), u.a, u.rows, static_cast<int>(t0), static_cast<int>(steps)};
      at += steps;
    }
  };
  if (warp == 0) {
    // in place the rows without an adapter stay as they are; the plan's offsets may overlap
    const uint32_t items = min(count_units(p.plan, p.base != p.out), p.units) * tiles;
    if (lane == 0) {
      at = items_begin(items, gridDim.x, blockIdx.x);
      past = items_begin(items, gridDim.x, blockIdx.x + 1);
    }
    __syncwarp();
    prepare(0);
  }
  if (tid == 64) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int a = 0; a < kExpandAcc; ++a) {
      mbar_init(smem_u32(&tfull[a]), 1);
      mbar_init(smem_u32(&tempty[a]), 4);
    }
    mbar_init(smem_u32(&image), 1);
    stop = 0;
    zero = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_at), kExpandAcc * kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_at, img0 = smem_u32(smem), q0 = img0 + S::kImg;
  volatile int* stopped = &stop;
  bool ok = true;

  int before = 0;                                // steps of the units before, and their number
  for (uint32_t turn = 0, units = 0; parts[turn & 1].steps > 0; ++turn) {
    const int* rows = rows_of[turn & 1];
    const Part& u = parts[turn & 1];
    const int steps = u.steps, t0 = u.t0;
    if (u.a == p.plan.n) {                       // base as it is, or zeros
      for (int i = warp; i < u.rows; i += kExpandThreads / 32) {
        if (rows[i] < 0) continue;
        const int64_t at = static_cast<int64_t>(rows[i]) * (p.N / 8);
        for (int e = lane; e < steps * (kCols / 8); e += 32) {
          const int c = t0 * (kCols / 8) + e;
          if (c < p.N / 8)
            reinterpret_cast<uint4*>(p.out)[at + c] =
                p.base ? reinterpret_cast<const uint4*>(p.base)[at + c] : make_uint4(0, 0, 0, 0);
        }
      }
    } else if (warp == 0) {
      if (lane == 0) {
        int i = before;
        for (; i < before + steps; ++i) {
          const int s = i % S::kStages;
          ok = mbar_wait(smem_u32(&empty[s]), ((i / S::kStages) & 1) ^ 1, p.wait_ns, stopped);
          if (!ok) break;
          mbar_arrive_expect_tx(smem_u32(&full[s]), S::kQ);
          tma_load_3d(q0 + s * S::kQ, &map_q, smem_u32(&full[s]), (t0 + i - before) * kCols, 0, u.a);
          if (i == before) {                     // the last unit's MMAs have read their image
            mbar_arrive_expect_tx(smem_u32(&image), S::kImg);
            const uint8_t* src = p.img + static_cast<int64_t>(u.unit) * atoms(p.parts, R) * kAtom;
            for (int k = 0; k < S::kImg / kAtom; ++k)
              for (int h = 0; h < 2; ++h)        // rows of the unit's halves
                bulk_copy_g2s(img0 + k * kAtom + h * (kAtom / 2),
                              src + (h * atoms(p.parts, R) + k) * (kAtom / 2), kAtom / 2,
                              smem_u32(&image));
          }
        }
        for (int k = i > S::kStages ? i - S::kStages : 0; k < i; ++k)
          mbar_wait(smem_u32(&full[k % S::kStages]), (k / S::kStages) & 1, kDrainNs, &zero);
      }
    } else if (warp == 1) {
      if (lane == 0) {
        const uint32_t idesc = idesc_bf16(128, kCols, false, true);
        ok = mbar_wait(smem_u32(&image), units & 1, p.wait_ns, stopped);
        for (int i = before; i < before + steps && ok; ++i) {
          const int s = i % S::kStages, a = i % kExpandAcc;
          ok = mbar_wait(smem_u32(&tempty[a]), ((i / kExpandAcc) & 1) ^ 1, p.wait_ns, stopped) &&
               mbar_wait(smem_u32(&full[s]), (i / S::kStages) & 1, p.wait_ns, stopped);
          if (!ok) break;
          tc_fence_after();
          const uint64_t bd = sdesc_sw128(q0 + s * S::kQ, S::kQ, 1024);
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int ks = 0; ks < R / 16; ++ks) {
              const int at = k * (R / 16) + ks;  // of the image's columns, in 16s
              const uint64_t ad = sdesc_sw128(img0 + (at >> 2) * kAtom, 16, 1024) + (at & 3) * 2;
              umma_bf16(tmem + a * kCols, ad, bd + ks * (2048 >> 4), idesc, (k | ks) ? 1u : 0u);
            }
          umma_commit(smem_u32(&empty[s]));
          umma_commit(smem_u32(&tfull[a]));
        }
      }
    } else {
      const int q = warp & 3, half = (warp - 2) >> 2;
      uint8_t* st = smem + S::kImg + S::kStages * S::kQ + (warp - 2) * kPiece;
      const int ch = lane & 7, r0 = lane >> 3;   // of the runs: rows r0, r0 + 4, ... of 32
      const int end = before + steps, first = before + ((half ^ before) & 1);
      // rows and a bit for each that is there; where its run begins is one product away
      uint32_t g[8], here = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int row = rows[q * 32 + r0 + 4 * j];
        g[j] = row < 0 ? 0 : row;
        here |= row < 0 ? 0 : 1u << j;
      }
      const uint32_t pitch = static_cast<uint32_t>(p.N) * 2;
      auto at = [&](int j) { return static_cast<uint64_t>(g[j]) * pitch; };
      const bool any = __any_sync(0xffffffffu, rows[q * 32 + lane] >= 0);
      uint4 next[8];
      auto load = [&](int i) {                   // base of step i
        const int col = (t0 + i - before) * kCols + ch * 8;
        const uint8_t* src = reinterpret_cast<const uint8_t*>(p.base) + static_cast<int64_t>(col) * 2;
        const uint32_t on = p.base && i < end && col < p.N ? here : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          next[j] = on & (1u << j) ? __ldcs(reinterpret_cast<const uint4*>(src + at(j)))
                                   : make_uint4(0, 0, 0, 0);
      };
      load(first);
      for (int i = first; i < end; i += 2) {
        const int a = i % kExpandAcc;
        if (any) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int row = r0 + 4 * j;
            *reinterpret_cast<uint4*>(st + row * 128 + ((ch ^ (row & 7)) << 4)) = next[j];
          }
          __syncwarp();
          load(i + 2);
        }
        const bool got = mbar_wait(smem_u32(&tfull[a]), (i / kExpandAcc) & 1, p.wait_ns, stopped);
        ok = __all_sync(0xffffffffu, got);
        if (!ok) break;
        tc_fence_after();
        const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + a * kCols;
        if (any) {                               // else no row of the quarter is there
#pragma unroll
          for (int c0 = 0; c0 < 8; c0 += 2) {
            uint32_t v[16];
            tmem_ld_32x32b_x16(taddr + c0 * 8, v);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint4* w = reinterpret_cast<uint4*>(st + lane * 128 + (((c0 + c) ^ (lane & 7)) << 4));
              const uint4 o = *w;
              const float* x = reinterpret_cast<const float*>(v + c * 8);
              *w = make_uint4(pack_bf16x2(x[0] + lo_f(o.x), x[1] + hi_f(o.x)),
                              pack_bf16x2(x[2] + lo_f(o.y), x[3] + hi_f(o.y)),
                              pack_bf16x2(x[4] + lo_f(o.z), x[5] + hi_f(o.z)),
                              pack_bf16x2(x[6] + lo_f(o.w), x[7] + hi_f(o.w)));
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&tempty[a]));
        const int col = (t0 + i - before) * kCols + ch * 8;
        uint8_t* to = reinterpret_cast<uint8_t*>(p.out) + static_cast<int64_t>(col) * 2;
        if (any && col < p.N) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int row = r0 + 4 * j;
            if (here & (1u << j))
              __stcs(reinterpret_cast<uint4*>(to + at(j)),
                     *reinterpret_cast<const uint4*>(st + row * 128 + ((ch ^ (row & 7)) << 4)));
          }
        }
        __syncwarp();                            // the piece may be filled again
      }
    }
    if (warp == 0) {
      __syncwarp();
      prepare((turn + 1) & 1);
    }
    if (u.a != p.plan.n) {
      before += steps;
      ++units;
    }
    if (!ok) {
      stop = 1;
      report_error(p.plan.err, kErrTimeout);
      if (warp == 1 && lane == 0) mbar_wait(smem_u32(&image), (units - 1) & 1, kDrainNs, &zero);
    }
    tc_fence_before();
    if (__syncthreads_or(!ok)) break;            // every tile of the part has been finished
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kExpandAcc * kCols);
  }
}

// ------------------------------------------------------------------ grad

// Both gradients in one launch. Their work is a list of items: (tile of columns, 64
// rows of one adapter), the rows running fastest. One CTA an SM takes an equal run of
// items whatever the adapters' shares are; where a run ends inside an output, its sums
// go to a slot of the CTA, and grad_finish_kernel adds the slots up in order.
// Warps: 0 loads images, 1 issues the MMAs, then 8 draining warps (one for each 32
// columns, or 32 columns and half of the rank) and 4 gathering rows of the input, each
// row's columns of the tile in one run of 512 (256) bytes, where warp 0 cannot load the
// 64 rows as boxes. The accumulators take up two chunks of an output; those of one half
// of a tile are taken out while the other half's MMAs run. Bound by the input's rows, and
// by what one warp issues for a stage: 16384 rows of twice 4096, r = 64, take 62 us, 4.8
// TB/s, and the finish 9; with the rows gathered by cp.async throughout the whole backward
// takes 191 us instead of 164.
struct GradJob {
  CUtensorMap map;             // of in: boxes of 64 columns x 64 rows
  const uint8_t* img;          // three parts
  const __nv_bfloat16* in;     // [T, N]
  float* G;                    // [n, r, N]
  int N, tiles;
};

struct GradArgs {
  GradJob job[2];
  float* partial;              // [2 * CTAs][R][kTile]
  int* chunks;                 // [n + 1]: 64-row chunks before each adapter, for the finish
  int r, accumulate;
  int units;                   // that the images have room for
  unsigned long long wait_ns;
  Plan plan;
};

template <int R>
struct Grad {
  static constexpr int kHalves = R > 64 ? 1 : 2;
  static constexpr int kTile = 128 * kHalves;
  static constexpr int kIn = kHalves * kAtom;                 // 64 rows of the tile's columns
  static constexpr int kImg = atoms(3, R) * kAtom / 2;        // 64 rows of three parts
  static constexpr int kStage = kIn + kImg;
  static constexpr int kStages = R <= 16 ? 5 : R <= 32 ? 4 : 3;
  static constexpr int kDrain = 8;
  static constexpr int kOwn = R > 64 ? 64 : R;                // ranks of a draining warp
  static constexpr int kThreads = 32 * (2 + kDrain + 4);
  static constexpr int kTmem = R <= 16 ? 128 : R <= 32 ? 256 : 512;   // kHalves * 3 R
  static constexpr int kBytes = 1024 + kStages * kStage;
};

// What of the list CTA b has: items [first(b), first(b + 1)).
__device__ __forceinline__ int64_t first_item(int64_t items, int ctas, int b) {
  return items * b / ctas;
}

// A walk over items: tile, chunk c within the tile, adapter a with the chunks from c0 to
// c1 (kept here: every role takes a step for every stage).
struct Walk {
  int tile, c, a, c0, c1;
  __device__ __forceinline__ void start(int64_t item, int total, int n, const int* chunks) {
    tile = static_cast<int>(item / total);
    c = static_cast<int>(item - static_cast<int64_t>(tile) * total);
    int lo = 0, hi = n - 1;                      // the last adapter that begins at or before c
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (chunks[mid] <= c) lo = mid; else hi = mid - 1;
    }
    a = lo;
    c0 = chunks[a];
    c1 = chunks[a + 1];
  }
  __device__ __forceinline__ bool last() const { return c + 1 == c1; }   // of its output
  // Whether accumulators with so many chunks are full, or their output complete.
  __device__ __forceinline__ bool ends_group(int held) const { return held == 2 || last(); }
  __device__ __forceinline__ void next(int total, const int* chunks) {
    if (++c < c1) return;
    if (c == total) {
      ++tile;
      c = 0;
      a = -1;
    }
    do ++a; while (chunks[a + 1] <= c);          // adapters without rows have no chunk
    c0 = chunks[a];
    c1 = chunks[a + 1];
  }
};

template <int R>
__global__ void __launch_bounds__(Grad<R>::kThreads, 1)
    grad_kernel(const __grid_constant__ GradArgs p) {
  using S = Grad<R>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int chunks[kMaxAdapters + 1], units[kMaxAdapters + 1], begin[kMaxAdapters], end[kMaxAdapters];
  __shared__ uint64_t full[S::kStages], empty[S::kStages], tfull[2], tempty[2];
  __shared__ uint32_t tmem_at;
  __shared__ int ends[S::kStages];               // whether the accumulators end with a stage
  __shared__ int stop, zero;
  uint8_t* ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = p.plan.n, b = blockIdx.x, ctas = gridDim.x;
  grid_dependents_launch();
  if (warp == 0) {
    int c_sum = 0, u_sum = 0;
    for (int a0 = 0; a0 < n; a0 += 32) {
      int lo = 0, hi = 0;
      if (a0 + lane < n) segment(p.plan, a0 + lane, lo, hi);
      int c = (hi - lo + 63) >> 6, u = (hi - lo + kRows - 1) / kRows;
      const int c_own = c, u_own = u;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int oc = __shfl_up_sync(0xffffffffu, c, d), ou = __shfl_up_sync(0xffffffffu, u, d);
        if (lane >= d) {
          c += oc;
          u += ou;
        }
      }
      if (a0 + lane < n) {
        chunks[a0 + lane] = c_sum + c - c_own;
        units[a0 + lane] = u_sum + u - u_own;
        begin[a0 + lane] = lo;
        end[a0 + lane] = hi;
      }
      c_sum += __shfl_sync(0xffffffffu, c, 31);
      u_sum += __shfl_sync(0xffffffffu, u, 31);
    }
    if (lane == 0) chunks[n] = c_sum;
  }
  if (tid == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1 + 128);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int m = 0; m < S::kHalves; ++m) {
      mbar_init(smem_u32(&tfull[m]), 1);
      mbar_init(smem_u32(&tempty[m]), S::kDrain / S::kHalves);
    }
    stop = 0;
    zero = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_at), S::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_at;
  const int total = chunks[n];
  if (b == 0)
    for (int a = tid; a <= n; a += S::kThreads) p.chunks[a] = chunks[a];
  const int64_t items = static_cast<int64_t>(p.job[0].tiles + p.job[1].tiles) * total;
  const int64_t i0 = first_item(items, ctas, b);
  const int steps = static_cast<int>(first_item(items, ctas, b + 1) - i0);
  volatile int* stopped = &stop;
  bool ok = true;
  Walk w = {0, 0, 0, 0, 0};
  if (steps > 0) w.start(i0, total, n, chunks);
  const int t0 = p.job[0].tiles;

  // a chunk's rows as the plan has them, two a lane (checked when they are used, so that
  // nothing waits for them before); -1 past the adapter
  auto plan_rows = [&](const Walk& x, int& o0, int& o1) {
    const int at = begin[x.a] + (x.c - x.c0) * 64 + lane, past = end[x.a];
    o0 = at < past ? __ldg(p.plan.order + at) : -1;
    o1 = at + 32 < past ? __ldg(p.plan.order + at + 32) : -1;
  };
  // 64 rows that follow one another: the same answer in every warp
  auto is_box = [&](int o0, int o1) {
    const int first = __shfl_sync(0xffffffffu, o0, 0);
    return __all_sync(0xffffffffu, first >= 0 && first <= p.plan.T - 64 && o0 == first + lane &&
                                       o1 == first + 32 + lane);
  };

  if (steps == 0) {
    // nothing of the list
  } else if (warp == 0) {
    int o0, o1, held = 0;
    plan_rows(w, o0, o1);
    for (int i = 0; i < steps; ++i) {
      const int s = i % S::kStages;
      const Walk x = w;
      const bool last = w.ends_group(++held) || i + 1 == steps;
      if (last) held = 0;
      const bool box = is_box(o0, o1);
      const int row = __shfl_sync(0xffffffffu, o0, 0);
      if (i + 1 < steps) {
        w.next(total, chunks);
        plan_rows(w, o0, o1);
      }
      const bool got = mbar_wait(smem_u32(&empty[s]), ((i / S::kStages) & 1) ^ 1, p.wait_ns, stopped);
      ok = __all_sync(0xffffffffu, got);
      if (!ok) break;
      const uint32_t bar = smem_u32(&full[s]), dst = smem_u32(ring) + s * S::kStage;
      const bool second = x.tile >= t0;
      const int col = (second ? x.tile - t0 : x.tile) * S::kTile;
      if (lane == 0) {
        ends[s] = last;
        mbar_arrive_expect_tx(bar, S::kImg + (box ? S::kIn : 0));
        const int c = x.c - x.c0;                // chunk of the adapter: half a unit
        const int unit = min(units[x.a] + (c >> 1), p.units - 1);   // offsets may overlap
        bulk_copy_g2s(dst + S::kIn,
                      (second ? p.job[1].img : p.job[0].img) +
                          (static_cast<int64_t>(unit) * 2 + (c & 1)) * S::kImg, S::kImg, bar);
      }
      __syncwarp();
      if (box && lane < S::kTile / 64)           // a lane a box
        tma_load_2d(dst + lane * (kAtom / 2), second ? &p.job[1].map : &p.job[0].map, bar,
                    col + 64 * lane, row);
      __syncwarp();
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // the parts side by side are one N of 3 R, or of 256 and 128
      constexpr int kN0 = 3 * R > 256 ? 256 : 3 * R, kN1 = 3 * R - kN0;
      const uint32_t idesc0 = idesc_bf16(128, kN0, true, true);
      const uint32_t idesc1 = idesc_bf16(128, kN1 > 0 ? kN1 : 16, true, true);
      const uint64_t ad0 = sdesc_sw128(smem_u32(ring), kAtom / 2, 1024);
      const uint64_t bd0 = sdesc_sw128(smem_u32(ring) + S::kIn, kAtom / 2, 1024);
      uint32_t held = 0, turn = 0;               // the accumulators hold something; turns so far
      int s = 0;
      uint32_t phase = 0;
      for (int i = 0; i < steps; ++i) {
        ok = mbar_wait(smem_u32(&full[s]), phase, p.wait_ns, stopped);
        if (!ok) break;
        const bool last = ends[s] != 0;
        fence_proxy_async_shared();
        tc_fence_after();
        const uint64_t off = static_cast<uint64_t>(s) * (S::kStage >> 4);
#pragma unroll
        for (int m = 0; m < S::kHalves; ++m) {
          if (held == 0) {                       // the half's last sums have been taken out
            ok = mbar_wait(smem_u32(&tempty[m]), turn ^ 1, p.wait_ns, stopped);
            if (!ok) break;
            tc_fence_after();
          }
          const uint64_t ad = ad0 + off + m * (kAtom >> 4), bd = bd0 + off;
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint32_t to = tmem + m * 3 * R, on = ks ? 1u : held;
            umma_bf16(to, ad + ks * (2048 >> 4), bd + ks * (2048 >> 4), idesc0, on);
            if (kN1 > 0)
              umma_bf16(to + kN0, ad + ks * (2048 >> 4),
                        bd + (kN0 / 64) * (kAtom / 2 >> 4) + ks * (2048 >> 4), idesc1, on);
          }
          if (last) umma_commit(smem_u32(&tfull[m]));
        }
        if (!ok) break;
        umma_commit(smem_u32(&empty[s]));
        held = last ? 0 : 1;
        turn ^= last ? 1 : 0;
        if (++s == S::kStages) {
          s = 0;
          phase ^= 1;
        }
      }
    }
  } else if (warp < 2 + S::kDrain) {
    const int m = S::kHalves == 2 ? (warp - 2) >> 2 : 0, q = warp & 3;
    const int j0 = S::kHalves == 2 ? 0 : ((warp - 2) >> 2) * S::kOwn;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + m * 3 * R + j0;
    const int in_tile = m * 128 + q * 32 + lane;
    float sum[S::kOwn];
#pragma unroll
    for (int j = 0; j < S::kOwn; ++j) sum[j] = 0.0f;
    bool from_first = w.c == w.c0;               // the run began with its output's first chunk
    bool first_run = true;
    int held = 0, d = 0;
    for (int i = 0; i < steps; ++i) {
      const bool last = w.last();
      if (w.ends_group(++held) || i + 1 == steps) {
        const bool got = mbar_wait(smem_u32(&tfull[m]), d & 1, p.wait_ns, stopped);
        ok = __all_sync(0xffffffffu, got);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < S::kOwn; j += 16) {        // the smallest part first
          uint32_t v0[16], v1[16], v2[16];
          tmem_ld_32x32b_x16(taddr + j, v0);
          tmem_ld_32x32b_x16(taddr + R + j, v1);
          tmem_ld_32x32b_x16(taddr + 2 * R + j, v2);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 16; ++k)
            sum[j + k] += __uint_as_float(v0[k]) + (__uint_as_float(v1[k]) + __uint_as_float(v2[k]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&tempty[m]));
        held = 0;
        ++d;
      }
      if (last || i + 1 == steps) {              // the run's end
        const GradJob& job = p.job[w.tile >= t0];
        const int col = (w.tile >= t0 ? w.tile - t0 : w.tile) * S::kTile + in_tile;
        if (last && from_first) {
          if (col < job.N) {
            float* at = job.G + (static_cast<int64_t>(w.a) * p.r + j0) * job.N + col;
#pragma unroll
            for (int j = 0; j < S::kOwn; ++j) {
              if (j0 + j < p.r) *at = p.accumulate ? *at + sum[j] : sum[j];
              at += job.N;
            }
          }
        } else {
          float* slot = p.partial + static_cast<int64_t>(2 * b + (first_run ? 0 : 1)) * R * S::kTile;
#pragma unroll
          for (int j = 0; j < S::kOwn; ++j) slot[(j0 + j) * S::kTile + in_tile] = sum[j];
        }
#pragma unroll
        for (int j = 0; j < S::kOwn; ++j) sum[j] = 0.0f;
        first_run = false;
        from_first = true;
      }
      if (i + 1 < steps) w.next(total, chunks);
    }
  } else {
    const int g = warp - 2 - S::kDrain;          // rows g, g + 4, ... of a chunk
    constexpr int kVec = S::kTile / 8;           // 16-byte pieces of a row: 32 or 16
    constexpr int kPer = 32 / kVec;              // rows of a warp's instruction
    const int ch = lane % kVec, sub = lane / kVec;
    int o0, o1;
    plan_rows(w, o0, o1);
    for (int i = 0; i < steps; ++i) {
      const int s = i % S::kStages;
      const Walk x = w;
      const bool box = is_box(o0, o1);
      int h0 = o0, h1 = o1;
      if (i + 1 < steps) {
        w.next(total, chunks);
        plan_rows(w, o0, o1);
      }
      const bool got = mbar_wait(smem_u32(&empty[s]), ((i / S::kStages) & 1) ^ 1, p.wait_ns, stopped);
      ok = __all_sync(0xffffffffu, got);
      if (!ok) break;
      if (box) {
        mbar_arrive(smem_u32(&full[s]));
        continue;
      }
      const int left = end[x.a] - begin[x.a] - (x.c - x.c0) * 64;   // rows of the adapter
      if ((lane < left && (h0 < 0 || h0 >= p.plan.T)) ||
          (lane + 32 < left && (h1 < 0 || h1 >= p.plan.T)))
        report_error(p.plan.err, kErrBadId);
      if (h0 >= p.plan.T) h0 = -1;
      if (h1 >= p.plan.T) h1 = -1;
      const GradJob& job = p.job[x.tile >= t0];
      const int col = (x.tile >= t0 ? x.tile - t0 : x.tile) * S::kTile + ch * 8;
      const bool in_n = col < job.N;
      const uint32_t dst = smem_u32(ring) + s * S::kStage + (ch >> 3) * (kAtom / 2);
#pragma unroll
      for (int j = 0; j < 16 / kPer; ++j) {
        const int row = 4 * (j * kPer + sub) + g;
        const int t_lo = __shfl_sync(0xffffffffu, h0, row & 31);
        const int t_hi = __shfl_sync(0xffffffffu, h1, row & 31);
        const int t = row < 32 ? t_lo : t_hi;
        const bool live = t >= 0 && in_n;
        cp_async_16z(dst + row * 128 + (((ch & 7) ^ (row & 7)) << 4),
                     live ? job.in + static_cast<int64_t>(t) * job.N + col : job.in, live);
      }
      cp_async_arrive_noinc(smem_u32(&full[s]));
    }
    cp_commit();
    cp_wait<0>();
  }
  if (!ok) {
    stop = 1;
    report_error(p.plan.err, kErrTimeout);
    if (warp == 0 && lane == 0)
      for (int s = 0; s < S::kStages; ++s) mbar_wait(smem_u32(&full[s]), 0, kDrainNs / 8, &zero);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmem);
  }
}

// The outputs that more than one CTA added to, in the order of the CTAs, and those of
// adapters without rows; kFinishRanks ranks of a tile to a CTA.
constexpr int kFinishRanks = 8;

template <int R>
__global__ void __launch_bounds__(Grad<R>::kTile)
    grad_finish_kernel(const __grid_constant__ GradArgs p, int ctas) {
  using S = Grad<R>;
  const int a = blockIdx.y, n = p.plan.n, tile = blockIdx.x, t0 = p.job[0].tiles;
  const GradJob& job = p.job[tile >= t0];
  const int col = (tile >= t0 ? tile - t0 : tile) * S::kTile + threadIdx.x;
  grid_dependency_wait();
  const int total = p.chunks[n], c0 = p.chunks[a], c1 = p.chunks[a + 1];
  float* g = job.G + static_cast<int64_t>(a) * p.r * job.N + col;
  const int j0 = blockIdx.z * kFinishRanks, j1 = min(p.r, j0 + kFinishRanks);
  if (col >= job.N) return;
  if (c0 == c1) {
    if (!p.accumulate)
      for (int j = j0; j < j1; ++j) g[static_cast<int64_t>(j) * job.N] = 0.0f;
    return;
  }
  const int64_t items = static_cast<int64_t>(t0 + p.job[1].tiles) * total;
  const int64_t i0 = static_cast<int64_t>(tile) * total + c0, i1 = i0 + (c1 - c0);
  // the CTA of an item, the last one that begins at or before it: items b / ctas <= i
  auto owner = [&](int64_t i) { return static_cast<int>(((i + 1) * ctas - 1) / items); };
  const int b0 = owner(i0), b1 = owner(i1 - 1);
  if (b0 == b1) return;
  float v[kFinishRanks];
#pragma unroll
  for (int j = 0; j < kFinishRanks; ++j) v[j] = 0.0f;
  for (int b = b0; b <= b1; ++b) {
    const int64_t first = first_item(items, ctas, b);
    if (first == first_item(items, ctas, b + 1)) continue;        // a CTA without items
    const int slot = 2 * b + (first >= i0 ? 0 : 1);
    const float* src = p.partial + (static_cast<int64_t>(slot) * R + j0) * S::kTile + threadIdx.x;
#pragma unroll
    for (int j = 0; j < kFinishRanks; ++j) v[j] += src[j * S::kTile];
  }
#pragma unroll
  for (int j = 0; j < kFinishRanks; ++j)
    if (j0 + j < j1) {
      float* at = g + static_cast<int64_t>(j0 + j) * job.N;
      *at = p.accumulate ? *at + v[j] : v[j];
    }
}

// ------------------------------------------------------------------ few rows

constexpr int kFewCtas = 8;         // CTAs of a row's cluster
constexpr int kFewThreads = 256;
constexpr int kFewAhead = 44 * 1024;   // bytes of B that are fetched before v is known

// One cluster a row: each CTA takes an eighth of H for v and, once the cluster has
// added v up, an eighth of N for out. What the CTA needs of B is on its way into shared
// memory (as much as kFewAhead holds) and base in registers before v is known. No plan,
// one launch; what bounds it is the latency of three loads and two cluster barriers: one
// row takes 4.1 us, 64 rows of as many adapters (23 MB) 8.1, 2.8 TB/s.
__global__ void __launch_bounds__(kFewThreads, 4)
    few_kernel(const __nv_bfloat16* __restrict__ x, const __nv_bfloat16* __restrict__ A,
               const __nv_bfloat16* __restrict__ B, const int32_t* __restrict__ ids,
               const float* __restrict__ scales, const __nv_bfloat16* base, __nv_bfloat16* out,
               float* __restrict__ v, int H, int N, int n, int r, int* err) {
  extern __shared__ uint4 ahead[];                // [ranks][vectors of this CTA]
  __shared__ float part[kMaxRank];                // this CTA's share of v
  __shared__ float whole[kMaxRank];
  __shared__ float red[kFewThreads * 8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int64_t t = blockIdx.x / kFewCtas;
  const int id = __ldg(ids + t);
  const bool on = id >= 0 && id < n;
  if (!on && id != -1 && tid == 0 && rank == 0) report_error(err, kErrBadId);
  // columns in vectors of eight
  const int hv = H / 8, hper = (hv + kFewCtas - 1) / kFewCtas;
  const int h0 = min(hv, static_cast<int>(rank) * hper), h1 = min(hv, h0 + hper);
  const int nv = N / 8, nper = (nv + kFewCtas - 1) / kFewCtas;
  const int n0 = min(nv, static_cast<int>(rank) * nper), n1 = min(nv, n0 + nper);
  const int vecs = n1 - n0;
  const uint4* xr = reinterpret_cast<const uint4*>(x + t * H);
  const uint4* Aa = reinterpret_cast<const uint4*>(A + static_cast<int64_t>(on ? id : 0) * r * H);
  const uint4* Ba = reinterpret_cast<const uint4*>(B + static_cast<int64_t>(on ? id : 0) * r * N);
  auto dot8 = [](const uint4& p, const uint4& q, float acc) {
    const uint32_t a[4] = {p.x, p.y, p.z, p.w}, b[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc = fmaf(lo_f(a[i]), lo_f(b[i]), acc);
      acc = fmaf(hi_f(a[i]), hi_f(b[i]), acc);
    }
    return acc;
  };
  const int fetched = on && vecs > 0 ? min(r, kFewAhead / 16 / vecs) : 0;
  if (on) {
    // the ranks of a warp two at a time, so that their loads overlap
    for (int j = warp; j < r; j += kFewThreads / 16) {
      const int k = min(j + kFewThreads / 32, r - 1);
      float s0 = 0.0f, s1 = 0.0f;
#pragma unroll 2
      for (int h = h0 + lane; h < h1; h += 32) {
        const uint4 xv = __ldg(xr + h);
        const uint4 a0 = __ldg(Aa + static_cast<int64_t>(j) * hv + h);
        const uint4 a1 = __ldg(Aa + static_cast<int64_t>(k) * hv + h);
        s0 = dot8(xv, a0, s0);
        s1 = dot8(xv, a1, s1);
      }
      if (j == warp) {                             // behind the first loads of A
        for (int e = tid; e < fetched * vecs; e += kFewThreads)
          cp_async_16(smem_u32(ahead + e), Ba + static_cast<int64_t>(e / vecs) * nv + n0 + e % vecs);
        cp_commit();
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) {
        s0 += __shfl_xor_sync(0xffffffffu, s0, d);
        s1 += __shfl_xor_sync(0xffffffffu, s1, d);
      }
      if (lane == 0) {
        part[j] = s0;
        part[k] = s1;
      }
    }
    if (warp >= r) {                               // warps without a rank fetch their share too
      for (int e = tid; e < fetched * vecs; e += kFewThreads)
        cp_async_16(smem_u32(ahead + e), Ba + static_cast<int64_t>(e / vecs) * nv + n0 + e % vecs);
      cp_commit();
    }
  }
  // groups of threads share the ranks where a CTA's columns are few
  int groups = 1;
  while (groups < 32 && 2 * groups * vecs <= kFewThreads) groups *= 2;
  const int width = kFewThreads / groups;          // threads of a group
  const int grp = tid / width, col = tid % width;
  uint4 first = make_uint4(0, 0, 0, 0);            // base of the first columns
  if (base && grp == 0 && n0 + col < n1)
    first = *(reinterpret_cast<const uint4*>(base + t * N) + n0 + col);
  if (on) {
    cluster_sync();
    const float f = scales ? __ldg(scales + id) : 1.0f;
    for (int j = tid; j < r; j += kFewThreads) {
      float s[kFewCtas];
#pragma unroll
      for (int q = 0; q < kFewCtas; ++q) s[q] = ld_cluster_f32(smem_u32(part + j), q);
      float sum = s[0];
#pragma unroll
      for (int q = 1; q < kFewCtas; ++q) sum += s[q];
      if (rank == 0) v[t * r + j] = sum;
      whole[j] = f * sum;
    }
    cp_wait<0>();
    cluster_sync();                                // part has been read; whole and B are there
  } else if (rank == 0) {
    for (int j = tid; j < r; j += kFewThreads) v[t * r + j] = 0.0f;
  }
  for (int c0 = n0; c0 < n1; c0 += width) {
    const int c = c0 + col;
    const bool live = c < n1;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
    auto add = [&](const uint4& q, float w) {
      const uint32_t b[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] = fmaf(w, lo_f(b[i]), acc[2 * i]);
        acc[2 * i + 1] = fmaf(w, hi_f(b[i]), acc[2 * i + 1]);
      }
    };
    if (on && live) {
      int j = grp;
#pragma unroll 4
      for (; j < fetched; j += groups) add(ahead[j * vecs + c - n0], whole[j]);
#pragma unroll 4
      for (; j < r; j += groups) add(__ldg(Ba + static_cast<int64_t>(j) * nv + c), whole[j]);
    }
    if (groups > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) red[i * kFewThreads + tid] = acc[i];
      __syncthreads();
      if (grp == 0)
        for (int g = 1; g < groups; ++g)
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] += red[i * kFewThreads + g * width + col];
    }
    if (grp == 0 && live) {
      if (base) {
        const uint4 o = c0 == n0 ? first : *(reinterpret_cast<const uint4*>(base + t * N) + c);
        const uint32_t b[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[2 * i] += lo_f(b[i]);
          acc[2 * i + 1] += hi_f(b[i]);
        }
      }
      *(reinterpret_cast<uint4*>(out + t * N) + c) =
          make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                     pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7]));
    }
  }
}

// ------------------------------------------------------------------ host

// A launch with clusters of `cluster` CTAs; beside: beside the kernel before it.
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kern)(KArgs...), dim3 grid, int threads, int smem, int cluster,
                   bool beside, bool* configured, cudaStream_t st, Args... args) {
  const int d = current_device();
  if (d < 0 || d >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!configured[d]) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured[d] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = beside ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, KArgs(args)...);
}

int64_t max_units(int64_t T, int n) { return (T + kRows - 1) / kRows + n; }
// The kernels' R: 8192 rows with r = 16 take 51 us by R = 16 and 54 by 32.
int rank_up(int r) { return r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128; }
size_t up256(size_t b) { return (b + 255) / 256 * 256; }
size_t image_bytes(int64_t T, int n, int r, int parts) {
  return static_cast<size_t>(max_units(T, n)) * atoms(parts, rank_up(r)) * kAtom;
}

template <int R>
cudaError_t shrink(const __nv_bfloat16* P, ShrinkArgs p, cudaStream_t st) {
  static bool configured[kMaxDevices] = {};
  CUtensorMap map;
  if (!make_tmap_bf16_3d(&map, P, p.K, p.r, p.plan.n, 64, R)) return cudaErrorInvalidValue;
  const int64_t units = max_units(p.plan.T, p.plan.n);
  const int kblocks = (p.K + 63) / 64;
  // CTAs to a cluster: as many as two an SM take at once, each with four k-blocks at least
  // (300 rows of 16 adapters, 4096 x 4096: the call takes 18 us, 38 with one CTA a unit)
  p.split = 1;
  while (p.split < 8 && kblocks / (p.split + 1) >= 4 &&
         units * (p.split + 1) <= 2 * device_sm_count())
    ++p.split;
  p.wait_ns = kDefaultWaitNs;
  return launch(shrink_kernel<R>, dim3(static_cast<unsigned>(units * p.split)), Shrink<R>::kThreads,
                Shrink<R>::kBytes, p.split, false, configured, st, map, p);
}

template <int R>
cudaError_t expand(const __nv_bfloat16* Q, int r, ExpandArgs p, cudaStream_t st) {
  static bool configured[kMaxDevices] = {};
  CUtensorMap map;
  if (!make_tmap_bf16_3d(&map, Q, p.N, r, p.plan.n, 64, R)) return cudaErrorInvalidValue;
  p.units = static_cast<int>(max_units(p.plan.T, p.plan.n));
  p.wait_ns = kDefaultWaitNs;
  return launch(expand_kernel<R>, dim3(device_sm_count() * (R > 64 ? 1 : 2)), kExpandThreads,
                Expand<R>::kBytes, 1, false, configured, st, map, p);
}

template <int R>
cudaError_t grad(GradArgs p, cudaStream_t st) {
  static bool configured[kMaxDevices] = {}, configured_finish[kMaxDevices] = {};
  for (GradJob& j : p.job) {
    j.tiles = (j.N + Grad<R>::kTile - 1) / Grad<R>::kTile;
    if (!make_tmap_bf16_2d(&j.map, j.in, j.N, p.plan.T, static_cast<uint64_t>(j.N) * 2, 64, 64))
      return cudaErrorInvalidValue;
  }
  p.wait_ns = kDefaultWaitNs;
  const int ctas = device_sm_count();
  const cudaError_t e = launch(grad_kernel<R>, dim3(ctas), Grad<R>::kThreads, Grad<R>::kBytes, 1,
                               false, configured, st, p);
  if (e != cudaSuccess) return e;
  return launch(grad_finish_kernel<R>, dim3(p.job[0].tiles + p.job[1].tiles, p.plan.n, (p.r + kFinishRanks - 1) / kFinishRanks),
                Grad<R>::kTile, 0, 1, true, configured_finish, st, p, ctas);
}

#define MOE_BY_RANK(r, call)       \
  ((r) <= 16   ? call<16>          \
   : (r) <= 32 ? call<32>          \
   : (r) <= 64 ? call<64>          \
               : call<128>)

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

moe_status check_sizes(int64_t T, int H, int N, int n, int r) {
  if (T < 0 || T > INT32_MAX - 1024 || H <= 0 || N <= 0 || H > (1 << 30) || N > (1 << 30) ||
      n < 1 || n > kMaxAdapters || r < 1)
    return MOE_ERR_INVALID_ARG;
  return (H % 8 || N % 8 || r > kMaxRank || T > kMaxRows) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// Whether one cluster takes each row, without a plan: every row then reads its adapter
// whole, which the rows of a unit share otherwise, but a unit costs as much for one row as
// for 128. In units of 2 ns at 4096 x 4096 a row takes 25 + r, the two launches 6000 + 100
// r and a unit 135, one at least to an adapter in use. How many are is known on the device
// alone: all of up to 32 are taken to be, and of more some half. By clusters and by units,
// with every adapter in use: r = 16 and 32 adapters, 128 rows 11 and 22 us, 256 20 and 23,
// 512 35 and 23; 128 adapters, 512 rows 36 and 47, 1024 68 and 47; 512 adapters, 512 rows 41
// and 160, 1024 75 and 145, 1800 129 and 161; 1024 adapters, 1800 rows 131 and 280; r = 64
// and 32 adapters, 128 rows 20 and 34, 256 36 and 34; of 4096 x 14336 with r = 16, 128
// adapters, 512 rows 52 and 87, 1024 98 and 93. With one or 16 in use, r = 16: of 16, 256
// rows 19 and 15 to 19; of 256, 512 rows 36 and 41 to 46, 1000 66 and 41 to 47; of 512, 1000
// rows 66 and 45 to 54, 1800 116 and 51 to 55; of 1024, 1800 rows 116 and 89 to 104, 4096
// 278 and 95 to 99; r = 64, of 512, 512 rows 66 and 52 to 58, 1000 124 and 49 to 60. (Every
// adapter taken to be in use sent 1800 rows of one among 512 to the clusters.)
bool few_rows(int64_t T, int n, int r) {
  const int64_t likely = n <= 32 ? n : 16 + n / 2;
  return T * (25 + r) <= 6000 + 100 * r + 135 * (T < likely ? T : likely);
}

// What the backward has in its workspace.
struct BwdLayout {
  size_t dv, v, partial, chunks, total;
};
BwdLayout bwd_layout(int64_t T, int n, int r) {
  BwdLayout L;
  const size_t img = up256(image_bytes(T, n, r, 3));
  L.dv = 0;
  L.v = img;
  L.partial = 2 * img;
  const size_t tile = r > 64 ? 128 : 256;
  L.chunks = L.partial + up256(static_cast<size_t>(2) * device_sm_count() * rank_up(r) * tile * 4);
  L.total = L.chunks + up256((n + 1) * sizeof(int));
  return L;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_lora_plan(const int32_t* adapter_ids, int64_t T, int n, int32_t* order,
                         int32_t* offsets, void* stream) {
  MOE_ENTRY_RANGE();
  if (T < 0 || T > INT32_MAX - 1024 || n < 1 || n > kMaxAdapters || !offsets ||
      (T > 0 && (!adapter_ids || !order)))
    return MOE_ERR_INVALID_ARG;
  static bool configured[kMaxDevices] = {};
  const int d = current_device();
  if (d < 0 || d >= kMaxDevices) return MOE_ERR_CUDA;
  auto bytes = [](int keys) { return 34 * keys * static_cast<int>(sizeof(int)); };
  if (!configured[d] &&
      cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           bytes(kMaxAdapters + 1)) != cudaSuccess)
    return MOE_ERR_CUDA;
  configured[d] = true;
  const int ctas = T <= kPlanRows ? 1 : kPlanCtas;
  return launch(plan_kernel, dim3(ctas), 1024, bytes(n + 1), ctas, false, configured,
                static_cast<cudaStream_t>(stream), adapter_ids, T, n, order, offsets,
                device_error_word()) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

size_t moe_lora_workspace_size(int64_t T, int n, int r) {
  if (check_sizes(T, 8, 8, n, r) != MOE_OK || T == 0 || few_rows(T, n, r)) return 0;
  return up256(image_bytes(T, n, r, 2));
}

moe_status moe_lora(const void* x, const void* a, const void* b, const int32_t* adapter_ids,
                    const int32_t* order, const int32_t* offsets, const float* scales,
                    const void* base, int64_t T, int H, int N, int n, int r, void* out, float* v,
                    void* workspace, size_t ws_bytes, void* stream) {
  MOE_ENTRY_RANGE();
  const moe_status s = check_sizes(T, H, N, n, r);
  if (s != MOE_OK) return s;
  if (T == 0) return MOE_OK;
  if (!x || !a || !b || !adapter_ids || !order || !offsets || !out || !v || !aligned16(x) ||
      !aligned16(a) || !aligned16(b) || !aligned16(base) || !aligned16(out))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const auto* xb = static_cast<const __nv_bfloat16*>(x);
  const auto* ab = static_cast<const __nv_bfloat16*>(a);
  const auto* bb = static_cast<const __nv_bfloat16*>(b);
  const auto* yb = static_cast<const __nv_bfloat16*>(base);
  auto* ob = static_cast<__nv_bfloat16*>(out);
  if (few_rows(T, n, r)) {
    static bool configured[kMaxDevices] = {};
    return launch(few_kernel, dim3(static_cast<unsigned>(T) * kFewCtas), kFewThreads,
                  kFewAhead, kFewCtas,
                  false, configured, st, xb, ab, bb, adapter_ids, scales, yb, ob, v, H, N, n, r,
                  device_error_word()) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
  }
  if (!workspace || ws_bytes < moe_lora_workspace_size(T, n, r) || !aligned16(workspace))
    return MOE_ERR_WORKSPACE;
  const Plan plan = {order, offsets, T, n, device_error_word()};
  ShrinkArgs sh{};
  sh.in = xb;
  sh.scales = scales;
  sh.V = v;
  sh.img = static_cast<uint8_t*>(workspace);
  sh.parts = 2;
  sh.K = H;
  sh.r = r;
  sh.plan = plan;
  ExpandArgs ex{};
  ex.img = sh.img;
  ex.parts = 2;
  ex.base = yb;
  ex.out = ob;
  ex.N = N;
  ex.plan = plan;
  if (MOE_BY_RANK(r, shrink)(ab, sh, st) != cudaSuccess ||
      MOE_BY_RANK(r, expand)(bb, r, ex, st) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_OK;
}

size_t moe_lora_backward_workspace_size(int64_t T, int n, int r) {
  if (check_sizes(T, 8, 8, n, r) != MOE_OK || T == 0) return 0;
  return bwd_layout(T, n, r).total;
}

moe_status moe_lora_backward(const void* dy, const void* x, const float* v, const void* a,
                             const void* b, const int32_t* order, const int32_t* offsets,
                             const float* scales, const void* base, int64_t T, int H, int N, int n,
                             int r, void* dx, float* da, float* db, int accumulate,
                             void* workspace, size_t ws_bytes, void* stream) {
  MOE_ENTRY_RANGE();
  const moe_status s = check_sizes(T, H, N, n, r);
  if (s != MOE_OK) return s;
  if (!da || !db || !aligned16(da) || !aligned16(db)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    if (accumulate) return MOE_OK;
    const size_t each = static_cast<size_t>(n) * r * sizeof(float);
    return cudaMemsetAsync(da, 0, each * H, st) == cudaSuccess &&
                   cudaMemsetAsync(db, 0, each * N, st) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
  }
  if (!dy || !x || !v || !a || !b || !order || !offsets || !dx || dx == dy || dx == x ||
      !aligned16(dy) ||
      !aligned16(x) || !aligned16(a) || !aligned16(b) || !aligned16(base) || !aligned16(dx))
    return MOE_ERR_INVALID_ARG;
  const BwdLayout L = bwd_layout(T, n, r);
  if (!workspace || ws_bytes < L.total || !aligned16(workspace)) return MOE_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const Plan plan = {order, offsets, T, n, device_error_word()};
  const auto* gb = static_cast<const __nv_bfloat16*>(dy);
  const auto* xb = static_cast<const __nv_bfloat16*>(x);
  ShrinkArgs sh{};
  sh.in = gb;
  sh.scales = scales;
  sh.img = ws + L.dv;
  sh.kept = v;
  sh.img_kept = ws + L.v;
  sh.parts = 3;
  sh.K = N;
  sh.r = r;
  sh.plan = plan;
  ExpandArgs ex{};
  ex.img = sh.img;
  ex.parts = 3;
  ex.base = static_cast<const __nv_bfloat16*>(base);
  ex.out = static_cast<__nv_bfloat16*>(dx);
  ex.N = H;
  ex.plan = plan;
  GradArgs gr{};
  gr.job[0] = {{}, ws + L.dv, xb, da, H, 0};
  gr.job[1] = {{}, ws + L.v, gb, db, N, 0};
  gr.partial = reinterpret_cast<float*>(ws + L.partial);
  gr.chunks = reinterpret_cast<int*>(ws + L.chunks);
  gr.r = r;
  gr.accumulate = accumulate;
  gr.units = static_cast<int>(max_units(T, n));
  gr.plan = plan;
  if (MOE_BY_RANK(r, shrink)(static_cast<const __nv_bfloat16*>(b), sh, st) != cudaSuccess ||
      MOE_BY_RANK(r, expand)(static_cast<const __nv_bfloat16*>(a), r, ex, st) != cudaSuccess ||
      MOE_BY_RANK(r, grad)(gr, st) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_OK;
}

}  // extern "C"
