// lora.cu - low-rank adapters of many requests beside a shared projection
// (moe_lora_plan, moe_lora, moe_lora_backward).
//
// With A and B both stored rank-major ([n, r, H] and [n, r, N]), forward and
// backward need three products only, each over the rows of one adapter:
//   shrink  V[t, j]   = s sum_c in[t, c] P[j, c]      v from x, A; dv from dy, B
//   expand  out[t, c] = base[t, c] + sum_j V[t, j] Q[j, c]   out from v, B; dx from dv, A
//   grad    G[j, c]   = sum_t V[t, j] in[t, c]        dA from dv, x; dB from v, dy
// The rank is at most 128 and the widths are thousands, so all three are bound
// by the rows that they read and write. The products go through mma.sync
// m16n8k16: a tile of 64 rows and one adapter's rank fills it as it is, where a
// tcgen05 tile would be mostly padding, and its rate is far above what the
// memory delivers.
//
// V is float. Where it enters a product it is the sum of two bf16 numbers, 16
// bits of its 24 (rounding to one would cost as much as rounding the result to
// bf16 once more). Sums over long axes leave the tensor cores every 64 terms and
// are added up in float registers, because the accumulation there truncates.
//
// Rows are taken in the order of the plan, 64 of one adapter at a time. A plan
// comes from the caller: every row number is checked against T before use.
#include <string.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

int* device_error_word();

namespace {

constexpr int kRows = 64;           // rows of a block: one adapter's
constexpr int kMaxAdapters = 1024;
constexpr int kMaxRank = 128;

// ------------------------------------------------------------------ mma.sync

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void mma_bf16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

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

// v = hi + lo in bf16, packed by pairs; what is not finite is in hi alone.
__device__ __forceinline__ void split2(float v0, float v1, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(v0, v1);
  const float h0 = __uint_as_float(hi << 16), h1 = __uint_as_float(hi & 0xFFFF0000u);
  const float l0 = v0 - h0, l1 = v1 - h1;
  lo = pack_bf16x2(fabsf(h0) < INFINITY ? l0 : 0.0f, fabsf(h1) < INFINITY ? l1 : 0.0f);
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

// Row i of the order, or -1 (reported) where it is no row.
__device__ __forceinline__ int plan_row(const Plan& p, int i) {
  const int r = __ldg(p.order + i);
  if (r >= 0 && r < p.T) return r;
  report_error(p.err, kErrBadId);
  return -1;
}

struct Block { int a, lo, rows; };   // adapter, first entry of the order, rows (0: none)

// Block u of the batch: the adapters' blocks one after the other, those without an
// adapter last. Called by a whole warp.
__device__ __forceinline__ Block find_block(const Plan& p, int u) {
  const int lane = lane_id();
  Block b = {-1, 0, 0};
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

// Stable counting sort by adapter in one CTA: each of 32 warps counts a run of
// rows, one scan over adapters and warps gives every run its places, and each warp
// then deals its rows out.
__global__ void __launch_bounds__(1024, 1)
    plan_kernel(const int32_t* ids, int64_t T64, int n, int32_t* order, int32_t* offsets, int* err) {
  extern __shared__ int plan_smem[];
  const int keys = n + 1, T = static_cast<int>(T64);
  int* place = plan_smem;                       // [32][keys]
  int* total = place + 32 * keys;               // [keys + 1]
  const int warp = threadIdx.x >> 5, lane = lane_id();
  for (int i = threadIdx.x; i < 32 * keys; i += 1024) place[i] = 0;
  __syncthreads();
  const int64_t run = (T64 + 1023) / 1024 * 32;             // rows of a warp, a multiple of 32
  const int64_t t0 = warp * run, t1 = min(t0 + run, T64);
  int* mine = place + warp * keys;
  for (int64_t t = t0 + lane; t - lane < t1; t += 32) {
    int key = -1;
    if (t < t1) {
      key = ids[t];
      if (key < -1 || key >= n) report_error(err, kErrBadId);
      if (key < 0 || key >= n) key = n;
    }
    const unsigned same = __match_any_sync(0xffffffffu, key);
    if (key >= 0 && lane == __ffs(same) - 1) mine[key] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  for (int k = threadIdx.x; k < keys; k += 1024) {
    int sum = 0;
    for (int w = 0; w < 32; ++w) {
      const int c = place[w * keys + k];
      place[w * keys + k] = sum;
      sum += c;
    }
    total[k] = sum;
  }
  __syncthreads();
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
        offsets[k0 + lane] = before + sum - c;   // keys = n + 1 offsets: the last is where none begin
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
  __syncthreads();
  for (int64_t t = t0 + lane; t - lane < t1; t += 32) {
    int key = -1;
    if (t < t1) {
      key = ids[t];
      if (key < 0 || key >= n) key = n;
    }
    const unsigned same = __match_any_sync(0xffffffffu, key);
    int at = 0;
    if (key >= 0) at = total[key] + mine[key] + __popc(same & ((1u << lane) - 1));
    if (key >= 0 && at < T) order[at] = static_cast<int32_t>(t);
    __syncwarp();
    if (key >= 0 && lane == __ffs(same) - 1) mine[key] += __popc(same);
    __syncwarp();
  }
}

// ------------------------------------------------------------------ shrink

// x tile and P tile: rows of 64 columns (128 bytes), 16-byte chunk c of row i at c ^ (i & 7).
template <int R>
struct Shrink {
  static constexpr int kStages = 4;
  static constexpr int kX = kRows * 128, kP = R * 128;
  static constexpr int kStage = kX + kP;
  static constexpr int kPartial = kRows * R * 4;
  static constexpr int kBytes = kStages * kStage > kPartial ? kStages * kStage : kPartial;
};

// A cluster of CTAs takes a block of rows, each CTA a run of 64-wide k-blocks;
// their sums are added over the cluster in the order of the ranks. Four warps of
// 16 rows each.
template <int R>
__global__ void __launch_bounds__(128)
    shrink_kernel(const __nv_bfloat16* __restrict__ in, const __nv_bfloat16* __restrict__ P,
                  const float* __restrict__ scales, float* __restrict__ V, int K, int r, int split,
                  Plan plan) {
  using S = Shrink<R>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int rows[kRows];
  const uint32_t rank = cluster_ctarank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Block blk = find_block(plan, static_cast<int>(blockIdx.x / split));
  if (tid < kRows) rows[tid] = tid < blk.rows ? plan_row(plan, blk.lo + tid) : -1;
  __syncthreads();
  if (blk.rows == 0 || blk.a == plan.n) {       // the whole cluster leaves together
    if (rank == 0)
      for (int i = tid; i < blk.rows * r; i += 128)
        if (rows[i / r] >= 0) V[static_cast<int64_t>(rows[i / r]) * r + i % r] = 0.0f;
    return;
  }
  const int kblocks = (K + 63) / 64, per = (kblocks + split - 1) / split;
  const int kb0 = static_cast<int>(rank) * per, kb1 = min(kblocks, kb0 + per);
  const __nv_bfloat16* Pa = P + static_cast<int64_t>(blk.a) * r * K;
  const uint32_t base = smem_u32(smem);
  // this thread's chunk column and rows of the copies
  const int ch = tid & 7, r0 = tid >> 3;
  const __nv_bfloat16* src[4];
  bool live[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = rows[r0 + 16 * i];
    live[i] = row >= 0;
    src[i] = in + static_cast<int64_t>(live[i] ? row : 0) * K + ch * 8;
  }
  auto load = [&](int kb, int s) {
    const int col = kb * 64 + ch * 8;
    const bool in_k = col < K;
    const uint32_t sx = base + s * S::kStage, sp = sx + S::kX;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = r0 + 16 * i;
      const bool ok = live[i] && in_k;
      cp_async_16z(sx + row * 128 + ((ch ^ (row & 7)) << 4), ok ? src[i] + kb * 64 : in, ok);
    }
#pragma unroll
    for (int i = 0; i < R / 16; ++i) {
      const int j = r0 + 16 * i;
      const bool ok = j < r && in_k;
      cp_async_16z(sp + j * 128 + ((ch ^ (j & 7)) << 4),
                   ok ? Pa + static_cast<int64_t>(j) * K + col : P, ok);
    }
  };
  float sum[R / 8][4];
#pragma unroll
  for (int i = 0; i < R / 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[i][j] = 0.0f;
#pragma unroll
  for (int s = 0; s < S::kStages - 1; ++s) {
    if (kb0 + s < kb1) load(kb0 + s, s);
    cp_commit();
  }
  for (int kb = kb0; kb < kb1; ++kb) {
    const int s = (kb - kb0) % S::kStages;
    cp_wait<S::kStages - 2>();
    __syncthreads();
    if (kb + S::kStages - 1 < kb1) load(kb + S::kStages - 1, (s + S::kStages - 1) % S::kStages);
    cp_commit();
    const uint32_t sx = base + s * S::kStage, sp = sx + S::kX;
    float acc[R / 8][4];
#pragma unroll
    for (int i = 0; i < R / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      uint32_t a[4];
      const int row = warp * 16 + (lane & 15), ca = 2 * ks + (lane >> 4);
      ldsm4(sx + row * 128 + ((ca ^ (row & 7)) << 4), a);
#pragma unroll
      for (int nt = 0; nt < R / 16; ++nt) {
        uint32_t b[4];
        const int j = nt * 16 + (lane & 7) + ((lane >> 4) << 3), cb = 2 * ks + ((lane >> 3) & 1);
        ldsm4(sp + j * 128 + ((cb ^ (j & 7)) << 4), b);
        mma_bf16(acc[2 * nt], a, b[0], b[1]);
        mma_bf16(acc[2 * nt + 1], a, b[2], b[3]);
      }
    }
#pragma unroll
    for (int i = 0; i < R / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[i][j] += acc[i][j];
  }
  cp_wait<0>();
  __syncthreads();
  // partial sums of the block, then each rank adds its share of the entries
  float* part = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int i = 0; i < R / 8; ++i) {
    const int row = warp * 16 + (lane >> 2), c = i * 8 + (lane & 3) * 2;
    part[row * R + c] = sum[i][0];
    part[row * R + c + 1] = sum[i][1];
    part[(row + 8) * R + c] = sum[i][2];
    part[(row + 8) * R + c + 1] = sum[i][3];
  }
  const float f = scales ? __ldg(scales + blk.a) : 1.0f;
  if (split > 1) cluster_sync();
  else __syncthreads();
  const int share = kRows * R / split;            // split divides it: a power of two up to 8
  for (int i = tid; i < share; i += 128) {
    const int e = static_cast<int>(rank) * share + i, row = e / R, j = e % R;
    float v = 0.0f;
    if (split > 1) {
      for (int q = 0; q < split; ++q) v += ld_cluster_f32(base + e * 4, q);
    } else {
      v = part[e];
    }
    if (j < r && rows[row] >= 0) V[static_cast<int64_t>(rows[row]) * r + j] = f * v;
  }
  if (split > 1) cluster_sync();                  // the others' sums have been read
}

// ------------------------------------------------------------------ expand

constexpr int kCols = 128;          // columns of a tile: rows of 256 bytes

template <int R>
struct Expand {
  static constexpr int kStages = R >= 128 ? 2 : 3;
  static constexpr int kT = kRows * 256, kQ = R * 256;
  static constexpr int kStage = kT + kQ;
  static constexpr int kBytes = kStages * kStage;
};

template <int R>
__global__ void __launch_bounds__(128)
    expand_kernel(const float* __restrict__ V, const __nv_bfloat16* __restrict__ Q,
                  const float* __restrict__ scales, const __nv_bfloat16* base, __nv_bfloat16* out,
                  int N, int r, Plan plan) {
  using S = Expand<R>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int rows[kRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Block blk = find_block(plan, static_cast<int>(blockIdx.x));
  if (blk.rows == 0) return;
  const bool none = blk.a == plan.n;
  if (none && base == out) return;                // base stays as it is
  if (tid < kRows) rows[tid] = tid < blk.rows ? plan_row(plan, blk.lo + tid) : -1;
  __syncthreads();
  const uint32_t sb = smem_u32(smem);
  const int tiles = (N + kCols - 1) / kCols;
  const int t0 = blockIdx.y, dt = gridDim.y;
  const __nv_bfloat16* Qa = Q + static_cast<int64_t>(none ? 0 : blk.a) * r * N;
  // this lane's chunk and rows of its warp's part of a tile: two rows a step
  const int ch = lane & 15, w0 = warp * 16 + (lane >> 4);
  auto load = [&](int t, int s) {
    const int col = t * kCols + ch * 8;
    const bool in_n = col < N;
    const uint32_t st = sb + s * S::kStage, sq = st + S::kT;
    if (base) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = w0 + 2 * i, g = rows[row];
        const bool ok = in_n && g >= 0;
        cp_async_16z(st + row * 256 + ((ch ^ (row & 7)) << 4),
                     ok ? base + static_cast<int64_t>(g) * N + col : base, ok);
      }
    }
    if (!none) {
#pragma unroll
      for (int i = 0; i < R / 8; ++i) {
        const int j = (tid >> 4) + 8 * i;
        const bool ok = in_n && j < r;
        cp_async_16z(sq + j * 256 + ((ch ^ (j & 7)) << 4),
                     ok ? Qa + static_cast<int64_t>(j) * N + col : Q, ok);
      }
    }
  };
#pragma unroll
  for (int s = 0; s < S::kStages - 1; ++s) {
    if (t0 + s * dt < tiles) load(t0 + s * dt, s);
    cp_commit();
  }
  // V of this warp's rows as the A operand, high and low parts
  uint32_t hi[R / 16][4], lo[R / 16][4];
  {
    const float f = (scales && !none) ? __ldg(scales + blk.a) : 1.0f;
    auto at = [&](int row, int j) {
      const int g = rows[row];
      return (!none && g >= 0 && j < r) ? f * __ldg(V + static_cast<int64_t>(g) * r + j) : 0.0f;
    };
#pragma unroll
    for (int ks = 0; ks < R / 16; ++ks)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = warp * 16 + (lane >> 2) + (i & 1) * 8;
        const int j = ks * 16 + (lane & 3) * 2 + (i >> 1) * 8;
        split2(at(row, j), at(row, j + 1), hi[ks][i], lo[ks][i]);
      }
  }
  int it = 0;
  for (int t = t0; t < tiles; t += dt, ++it) {
    const int s = it % S::kStages;
    cp_wait<S::kStages - 2>();
    __syncthreads();
    if (t + (S::kStages - 1) * dt < tiles)
      load(t + (S::kStages - 1) * dt, (s + S::kStages - 1) % S::kStages);
    cp_commit();
    uint8_t* st = smem + s * S::kStage;
    const uint32_t sq = sb + s * S::kStage + S::kT;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float acc[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
      if (!none) {
#pragma unroll
        for (int ks = 0; ks < R / 16; ++ks)
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            uint32_t b[4];
            const int j = ks * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
            const int c = half * 8 + nt * 2 + (lane >> 4);
            ldsm4_t(sq + j * 256 + ((c ^ (j & 7)) << 4), b);
            mma_bf16(acc[2 * nt], hi[ks], b[0], b[1]);
            mma_bf16(acc[2 * nt + 1], hi[ks], b[2], b[3]);
            mma_bf16(acc[2 * nt], lo[ks], b[0], b[1]);
            mma_bf16(acc[2 * nt + 1], lo[ks], b[2], b[3]);
          }
      }
#pragma unroll
      for (int nt = 0; nt < 8; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = warp * 16 + (lane >> 2) + i * 8, c = half * 8 + nt;
          uint32_t* w = reinterpret_cast<uint32_t*>(st + row * 256 + ((c ^ (row & 7)) << 4) +
                                                    (lane & 3) * 4);
          float v0 = acc[nt][2 * i], v1 = acc[nt][2 * i + 1];
          if (base) {
            const uint32_t o = *w;
            v0 += __uint_as_float(o << 16);
            v1 += __uint_as_float(o & 0xFFFF0000u);
          }
          *w = pack_bf16x2(v0, v1);
        }
    }
    __syncwarp();                                  // the warp's 16 rows are its own
    const int col = t * kCols + ch * 8;
    if (col < N) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = w0 + 2 * i, g = rows[row];
        if (g >= 0)
          __stcs(reinterpret_cast<uint4*>(out + static_cast<int64_t>(g) * N + col),
                 *reinterpret_cast<const uint4*>(st + row * 256 + ((ch ^ (row & 7)) << 4)));
      }
    }
  }
  cp_wait<0>();
}

// ------------------------------------------------------------------ grad

struct GradJob {
  const float* V;              // [T, r]
  const __nv_bfloat16* in;     // [T, N]
  const float* scales;         // or NULL
  float* G;                    // [n, r, N]
  int N;
};

template <int R>
struct Grad {
  static constexpr int kStages = 3;
  static constexpr int kIn = kRows * 256;
  static constexpr int kVRow = R * 2 + 16;                  // padded: eight rows hit all banks
  static constexpr int kV = 2 * kRows * kVRow;              // high and low parts
  static constexpr int kRing = kStages * kIn + 2 * kV;
  static constexpr int kPartial = R * kCols * 4;
  static constexpr int kBytes = kRing > kPartial ? kRing : kPartial;
};

// A cluster takes (adapter, 128 columns), each of its CTAs a run of the adapter's
// 64-row chunks; eight warps of 16 columns and the whole rank each. blockIdx.z:
// which of the two gradients.
template <int R>
__global__ void __launch_bounds__(256)
    grad_kernel(GradJob job0, GradJob job1, int r, int split, int accumulate, Plan plan) {
  using S = Grad<R>;
  extern __shared__ __align__(128) uint8_t smem[];
  const GradJob job = blockIdx.z ? job1 : job0;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int tile = static_cast<int>(blockIdx.x / split), a = blockIdx.y;
  if (tile * kCols >= job.N) return;               // the whole cluster
  int lo, hi;
  segment(plan, a, lo, hi);
  const int chunks = (hi - lo + kRows - 1) / kRows, per = (chunks + split - 1) / split;
  const int c0 = min(chunks, static_cast<int>(rank) * per), c1 = min(chunks, c0 + per);
  const int N = job.N, col0 = tile * kCols;
  const uint32_t sb = smem_u32(smem), sv = sb + S::kStages * S::kIn;
  const float f = job.scales ? __ldg(job.scales + a) : 1.0f;
  const int ch = tid & 15, w0 = tid >> 4;          // chunk and first row of the copies
  const bool in_n = col0 + ch * 8 < N;
  auto load = [&](int c, int s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = w0 + 16 * i, at = lo + c * kRows + row;
      const int g = at < hi ? plan_row(plan, at) : -1;
      const bool ok = in_n && g >= 0;
      cp_async_16z(sb + s * S::kIn + row * 256 + ((ch ^ (row & 7)) << 4),
                   ok ? job.in + static_cast<int64_t>(g) * N + col0 + ch * 8 : job.in, ok);
    }
  };
  // V of a chunk: 64 x R values, R / 8 pairs a thread
  float2 vr[R / 8];
  auto load_v = [&](int c) {
#pragma unroll
    for (int i = 0; i < R / 8; ++i) {
      const int e = (tid + 256 * i) * 2, row = e / R, j = e % R, at = lo + c * kRows + row;
      const int g = at < hi ? plan_row(plan, at) : -1;
      const float* src = job.V + static_cast<int64_t>(g < 0 ? 0 : g) * r + j;
      vr[i].x = (g >= 0 && j < r) ? f * __ldg(src) : 0.0f;
      vr[i].y = (g >= 0 && j + 1 < r) ? f * __ldg(src + 1) : 0.0f;
    }
  };
  auto store_v = [&](int b) {
#pragma unroll
    for (int i = 0; i < R / 8; ++i) {
      const int e = (tid + 256 * i) * 2, row = e / R, j = e % R;
      uint32_t h, l;
      split2(vr[i].x, vr[i].y, h, l);
      uint8_t* p = smem + S::kStages * S::kIn + b * S::kV + row * S::kVRow + j * 2;
      *reinterpret_cast<uint32_t*>(p) = h;
      *reinterpret_cast<uint32_t*>(p + kRows * S::kVRow) = l;
    }
  };
  float sum[R / 16][2][4];
#pragma unroll
  for (int m = 0; m < R / 16; ++m)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[m][i][j] = 0.0f;
#pragma unroll
  for (int s = 0; s < S::kStages - 1; ++s) {
    if (c0 + s < c1) load(c0 + s, s);
    cp_commit();
  }
  if (c0 < c1) {
    load_v(c0);
    store_v(0);
  }
  for (int c = c0; c < c1; ++c) {
    const int it = c - c0, s = it % S::kStages, vb = it & 1;
    cp_wait<S::kStages - 2>();
    __syncthreads();
    if (c + S::kStages - 1 < c1) load(c + S::kStages - 1, (s + S::kStages - 1) % S::kStages);
    cp_commit();
    if (c + 1 < c1) load_v(c + 1);
    const uint32_t si = sb + s * S::kIn, sh = sv + vb * S::kV, sl = sh + kRows * S::kVRow;
    float acc[R / 16][2][4];
#pragma unroll
    for (int m = 0; m < R / 16; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[m][i][j] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      uint32_t b[4];
      const int k = ks * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, cc = warp * 2 + (lane >> 4);
      ldsm4_t(si + k * 256 + ((cc ^ (k & 7)) << 4), b);
      const int kv = ks * 16 + (lane & 7) + ((lane >> 4) << 3), mc = ((lane >> 3) & 1) * 16;
#pragma unroll
      for (int m = 0; m < R / 16; ++m) {
        uint32_t h[4], l[4];
        ldsm4_t(sh + kv * S::kVRow + m * 32 + mc, h);
        ldsm4_t(sl + kv * S::kVRow + m * 32 + mc, l);
        mma_bf16(acc[m][0], h, b[0], b[1]);
        mma_bf16(acc[m][1], h, b[2], b[3]);
        mma_bf16(acc[m][0], l, b[0], b[1]);
        mma_bf16(acc[m][1], l, b[2], b[3]);
      }
    }
#pragma unroll
    for (int m = 0; m < R / 16; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[m][i][j] += acc[m][i][j];
    if (c + 1 < c1) store_v(vb ^ 1);               // read by nobody until the next barrier
  }
  cp_wait<0>();
  __syncthreads();
  float* part = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int m = 0; m < R / 16; ++m)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = m * 16 + (lane >> 2), c = warp * 16 + i * 8 + (lane & 3) * 2;
      part[j * kCols + c] = sum[m][i][0];
      part[j * kCols + c + 1] = sum[m][i][1];
      part[(j + 8) * kCols + c] = sum[m][i][2];
      part[(j + 8) * kCols + c + 1] = sum[m][i][3];
    }
  if (split > 1) cluster_sync();
  else __syncthreads();
  const int share = R * kCols / split;
  for (int i = tid; i < share; i += 256) {
    const int e = static_cast<int>(rank) * share + i, j = e / kCols, c = e % kCols;
    float v = 0.0f;
    if (split > 1) {
      for (int q = 0; q < split; ++q) v += ld_cluster_f32(sb + e * 4, q);
    } else {
      v = part[e];
    }
    if (j < r && col0 + c < N) {
      float* g = job.G + (static_cast<int64_t>(a) * r + j) * N + col0 + c;
      *g = accumulate ? *g + v : v;
    }
  }
  if (split > 1) cluster_sync();
}

// ------------------------------------------------------------------ few rows

constexpr int kFewCtas = 8;         // CTAs of a row's cluster
constexpr int kFewThreads = 256;

// One cluster a row: each CTA takes an eighth of H for v and, once the cluster has
// added v up, an eighth of N for out. The first values of B are on their way
// before v is known. No plan, one launch.
__global__ void __launch_bounds__(kFewThreads)
    few_kernel(const __nv_bfloat16* __restrict__ x, const __nv_bfloat16* __restrict__ A,
               const __nv_bfloat16* __restrict__ B, const int32_t* __restrict__ ids,
               const float* __restrict__ scales, const __nv_bfloat16* base, __nv_bfloat16* out,
               float* __restrict__ v, int H, int N, int n, int r, int* err) {
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
  const __nv_bfloat16* xr = x + t * H;
  const __nv_bfloat16* Aa = A + static_cast<int64_t>(on ? id : 0) * r * H;
  const __nv_bfloat16* Ba = B + static_cast<int64_t>(on ? id : 0) * r * N;
  auto dot8 = [](const uint4& p, const uint4& q, float acc) {
    const uint32_t a[4] = {p.x, p.y, p.z, p.w}, b[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc = fmaf(__uint_as_float(a[i] << 16), __uint_as_float(b[i] << 16), acc);
      acc = fmaf(__uint_as_float(a[i] & 0xFFFF0000u), __uint_as_float(b[i] & 0xFFFF0000u), acc);
    }
    return acc;
  };
  // groups of threads share the rank where a CTA's columns are few
  int groups = 1;
  while (groups < 32 && 2 * groups * (n1 - n0) <= kFewThreads) groups *= 2;
  const int width = kFewThreads / groups;          // threads of a group
  const int grp = tid / width, col = tid % width;
  constexpr int kAhead = 8;
  uint4 ahead[kAhead];
  const bool early = on && n0 + col < n1;
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int j = grp + i * groups;
    ahead[i] = (early && j < r)
                   ? __ldg(reinterpret_cast<const uint4*>(Ba + static_cast<int64_t>(j) * N) + n0 + col)
                   : make_uint4(0, 0, 0, 0);
  }
  if (on) {
    for (int j = warp; j < r; j += kFewThreads / 32) {
      float s = 0.0f;
#pragma unroll 4
      for (int h = h0 + lane; h < h1; h += 32)
        s = dot8(__ldg(reinterpret_cast<const uint4*>(xr) + h),
                 __ldg(reinterpret_cast<const uint4*>(Aa + static_cast<int64_t>(j) * H) + h), s);
#pragma unroll
      for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      if (lane == 0) part[j] = s;
    }
    cluster_sync();
    const float f = scales ? __ldg(scales + id) : 1.0f;
    for (int j = tid; j < r; j += kFewThreads) {
      float s = 0.0f;
#pragma unroll
      for (int q = 0; q < kFewCtas; ++q) s += ld_cluster_f32(smem_u32(part + j), q);
      if (rank == 0) v[t * r + j] = s;
      whole[j] = f * s;
    }
    cluster_sync();                                // part has been read, whole is there
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
        acc[2 * i] = fmaf(w, __uint_as_float(b[i] << 16), acc[2 * i]);
        acc[2 * i + 1] = fmaf(w, __uint_as_float(b[i] & 0xFFFF0000u), acc[2 * i + 1]);
      }
    };
    if (on && live) {
      int i0 = 0;
      if (c0 == n0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          if (grp + i * groups < r) add(ahead[i], whole[grp + i * groups]);
        i0 = kAhead;
      }
#pragma unroll 8
      for (int j = grp + i0 * groups; j < r; j += groups)
        add(__ldg(reinterpret_cast<const uint4*>(Ba + static_cast<int64_t>(j) * N) + c), whole[j]);
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
        const uint4 o = *(reinterpret_cast<const uint4*>(base + t * N) + c);
        const uint32_t b[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[2 * i] += __uint_as_float(b[i] << 16);
          acc[2 * i + 1] += __uint_as_float(b[i] & 0xFFFF0000u);
        }
      }
      *(reinterpret_cast<uint4*>(out + t * N) + c) =
          make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                     pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7]));
    }
  }
}

// ------------------------------------------------------------------ host

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kern)(KArgs...), dim3 grid, int threads, int smem, int cluster,
                           bool* configured, cudaStream_t st, Args... args) {
  const int d = current_device();
  if (d < 0 || d >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!configured[d]) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured[d] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, KArgs(args)...);
}

// CTAs to a cluster: as many as leave each of them `least` steps of `steps`, while
// `units` clusters do not fill the GPU four CTAs deep.
int pick_split(int64_t units, int64_t steps, int least) {
  int s = 1;
  while (s < 8 && steps / (2 * s) >= least && units * s < 4 * device_sm_count()) s *= 2;
  return s;
}

int64_t max_blocks(const Plan& p) { return (p.T + kRows - 1) / kRows + p.n; }

template <int R>
cudaError_t shrink(const __nv_bfloat16* in, const __nv_bfloat16* P, const float* scales, float* V,
                   int K, int r, const Plan& plan, cudaStream_t st) {
  static bool configured[kMaxDevices] = {};
  const int64_t blocks = max_blocks(plan);
  const int split = pick_split(blocks, (K + 63) / 64, 4);
  return launch_cluster(shrink_kernel<R>, dim3(static_cast<unsigned>(blocks * split)), 128,
                        Shrink<R>::kBytes, split, configured, st, in, P, scales, V, K, r, split,
                        plan);
}

template <int R>
cudaError_t expand(const float* V, const __nv_bfloat16* Q, const float* scales,
                   const __nv_bfloat16* base, __nv_bfloat16* out, int N, int r, const Plan& plan,
                   cudaStream_t st) {
  static bool configured[kMaxDevices] = {};
  const int64_t blocks = max_blocks(plan);
  const int tiles = (N + kCols - 1) / kCols;
  int split = 1;
  while (2 * split <= tiles && tiles / (2 * split) >= 2 && blocks * split < 8 * device_sm_count())
    split *= 2;
  return launch_cluster(expand_kernel<R>, dim3(static_cast<unsigned>(blocks), split), 128,
                        Expand<R>::kBytes, 1, configured, st, V, Q, scales, base, out, N, r, plan);
}

template <int R>
cudaError_t grad(const GradJob& j0, const GradJob& j1, int r, int accumulate, const Plan& plan,
                 cudaStream_t st) {
  static bool configured[kMaxDevices] = {};
  const int wide = j0.N > j1.N ? j0.N : j1.N;
  const int tiles = (wide + kCols - 1) / kCols;
  const int split = pick_split(static_cast<int64_t>(tiles) * plan.n, plan.T / plan.n / kRows, 2);
  return launch_cluster(grad_kernel<R>, dim3(tiles * split, plan.n, 2), 256, Grad<R>::kBytes, split,
                        configured, st, j0, j1, r, split, accumulate, plan);
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
  return (H % 8 || N % 8 || r > kMaxRank) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// The rows that one cluster each takes without a plan: every row reads its adapter
// whole, which 64 rows of a block share otherwise.
bool few_rows(int64_t T, int r) { return T <= 128 && T * r <= 4096; }

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
  auto bytes = [](int keys) { return (33 * keys + 1) * static_cast<int>(sizeof(int)); };
  if (!configured[d]) {
    if (cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             bytes(kMaxAdapters + 1)) != cudaSuccess)
      return MOE_ERR_CUDA;
    configured[d] = true;
  }
  plan_kernel<<<1, 1024, bytes(n + 1), static_cast<cudaStream_t>(stream)>>>(
      adapter_ids, T, n, order, offsets, device_error_word());
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_lora(const void* x, const void* a, const void* b, const int32_t* adapter_ids,
                    const int32_t* order, const int32_t* offsets, const float* scales,
                    const void* base, int64_t T, int H, int N, int n, int r, void* out, float* v,
                    void* stream) {
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
  if (few_rows(T, r)) {
    static bool configured[kMaxDevices] = {};
    return launch_cluster(few_kernel, dim3(static_cast<unsigned>(T) * kFewCtas), kFewThreads, 0,
                          kFewCtas, configured, st, xb, ab, bb, adapter_ids, scales, yb, ob, v, H,
                          N, n, r, device_error_word()) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
  }
  const Plan plan = {order, offsets, T, n, device_error_word()};
  if (MOE_BY_RANK(r, shrink)(xb, ab, nullptr, v, H, r, plan, st) != cudaSuccess ||
      MOE_BY_RANK(r, expand)(v, bb, scales, yb, ob, N, r, plan, st) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_OK;
}

size_t moe_lora_backward_workspace_size(int64_t T, int r) {
  if (T < 0 || T > INT32_MAX - 1024 || r < 1 || r > kMaxRank) return 0;
  return (static_cast<size_t>(T) * r * sizeof(float) + 255) / 256 * 256;
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
  if (!dy || !x || !v || !a || !b || !order || !offsets || !dx || !aligned16(dy) ||
      !aligned16(x) || !aligned16(a) || !aligned16(b) || !aligned16(base) || !aligned16(dx))
    return MOE_ERR_INVALID_ARG;
  if (!workspace || ws_bytes < moe_lora_backward_workspace_size(T, r) || !aligned16(workspace))
    return MOE_ERR_WORKSPACE;
  const Plan plan = {order, offsets, T, n, device_error_word()};
  const auto* gb = static_cast<const __nv_bfloat16*>(dy);
  const auto* xb = static_cast<const __nv_bfloat16*>(x);
  const auto* ab = static_cast<const __nv_bfloat16*>(a);
  const auto* bb = static_cast<const __nv_bfloat16*>(b);
  float* dv = static_cast<float*>(workspace);
  const GradJob ja = {dv, xb, nullptr, da, H}, jb = {v, gb, scales, db, N};
  if (MOE_BY_RANK(r, shrink)(gb, bb, scales, dv, N, r, plan, st) != cudaSuccess ||
      MOE_BY_RANK(r, expand)(dv, ab, nullptr, static_cast<const __nv_bfloat16*>(base),
                             static_cast<__nv_bfloat16*>(dx), H, r, plan, st) != cudaSuccess ||
      MOE_BY_RANK(r, grad)(ja, jb, r, accumulate, plan, st) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_OK;
}

}  // extern "C"
