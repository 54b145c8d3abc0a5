// ffn.cu - the gated feed-forward block of a dense layer (moe_gated_ffn and
// its backward): persistent GEMMs on the 5th-generation tensor cores with the
// activation, the product and its gradient in their epilogues.
//
//   Gated     [A_g | A_u] = x [W_gate | W_up],  h = bf16(act(A_g) A_u)
//   Down      y = bf16(add + h W_down)
//   GatedBwd  dh = dy W_down^T; h, dA_g, dA_u from it and the kept A_g, A_u
//   InGrad    dx = bf16(add + dA_g W_gate^T + dA_u W_up^T), one accumulator
//   WGrad     dW_down = h^T dy, and [dW_gate | dW_up] = x^T [dA_g | dA_u]
//
// One kernel body serves the five. A cluster of two CTAs shares a tile of 256
// rows and kBN columns (tcgen05.mma.cta_group::2): each CTA loads its own 128
// rows of A and half of the tile's columns of B, the leader issues the MMAs,
// and each CTA finishes its own 128 rows. Of a Gated tile one CTA loads columns
// of W_gate and the other the same columns of W_up, so that the accumulator
// holds A_g and A_u of a row in one lane. Warps: 0 the TMA producer, 1 the MMA
// issuer, 2 to 5 the epilogue; two accumulators, so that the epilogue of a tile
// runs beside the MMAs of the next.
//
// Nothing is padded: rows and columns past the matrices are the zeros that TMA
// fills in, they add nothing, and the stores are clipped (or, where a whole
// piece lies outside, left out). What the epilogues read besides the
// accumulator (A_g and A_u, or add) arrives by TMA in pieces of 32 rows x 32
// columns, one step ahead.
#include "act.cuh"
#include "common.cuh"
#include "ffn.h"
#include "internal.h"

namespace moe {

int* device_error_word();

namespace {

enum class Op { Gated, Down, GatedBwd, InGrad, WGradB16, WGradF32 };

constexpr int BK = 64;                         // k-block: 128 bytes of bf16
constexpr int kABytes = kTileM * BK * 2;       // 16 KB: this CTA's rows of A
constexpr int kBox = 64 * BK * 2;              // 8 KB: 64 columns x 64 of K
constexpr int kStageBytes = 2 * kABytes;       // A and up to 128 columns of B
constexpr int kThreads = 192;
constexpr uint32_t kTmemCols = 512;
constexpr int kPieceBytes = 32 * 64;           // 32 rows x 64 bytes, 64-byte swizzle
constexpr unsigned long long kDrainNs = 1000000000ull;
constexpr unsigned long long kPairDrainNs = 50000000ull;

// pieces that a warp reads for 32 columns, out slots per warp, ring depth: what
// 227 KB hold
template <Op op>
constexpr int loads() { return op == Op::GatedBwd ? 2 : (op == Op::Down || op == Op::InGrad) ? 1 : 0; }
template <Op op>
constexpr int out_slots() { return loads<op>() == 1 ? 2 : 3; }
template <Op op>
constexpr int stages() { return loads<op>() == 2 ? 5 : 6; }
constexpr int kMaxStages = 6;

template <Op op>
constexpr bool a_mn() { return op == Op::WGradB16 || op == Op::WGradF32; }
template <Op op>
constexpr bool b_mn() { return op != Op::GatedBwd && op != Op::InGrad; }

struct Smem {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t in[4][2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int zero;
};

template <Op op>
constexpr int pieces_bytes() { return 4 * (out_slots<op>() + 2 * loads<op>()) * kPieceBytes; }
template <Op op>
constexpr size_t smem_bytes() {
  return 1024 + static_cast<size_t>(stages<op>()) * kStageBytes + pieces_bytes<op>() + sizeof(Smem);
}
static_assert(smem_bytes<Op::Gated>() <= 232448 && smem_bytes<Op::Down>() <= 232448 &&
              smem_bytes<Op::GatedBwd>() <= 232448, "shared memory of one CTA");

struct Maps {
  CUtensorMap a[2], b[2], out[3], in[2];
};

struct Args {
  int M, N;          // rows and (per output) columns of the result
  int mt, nt;        // tiles; nt of both outputs of a WGrad together
  int nt0;           // WGrad: tiles of the first output
  int kb0, kb;       // k-blocks of the first pair of operands, and of both
  int group;         // row tiles that one column tile is walked over
  int act;           // Gated, GatedBwd
  int keep;          // Gated: A_g and A_u are stored
  int add;           // Down, InGrad: in[0] is added
  int accumulate;    // WGradF32
  int* err;
  unsigned long long wait_ns;
};

struct Tile { int m, n; };

// Column tiles follow one another over groups of row tiles: a group's rows of A
// stay in L2 while the columns of B stream by once a group.
__device__ __forceinline__ Tile decode(int t, const Args& p) {
  const int per = p.group * p.nt;
  const int g = t / per, local = t - g * per;
  const int rows = min(p.group, p.mt - g * p.group);
  Tile r;
  r.n = local / rows;
  r.m = g * p.group + local - r.n * rows;
  return r;
}

// 32 accumulator columns of A_g and A_u -> 16 words of h.
template <int kAct>
__device__ __forceinline__ void gated_words(const uint32_t* g, const uint32_t* u, uint32_t* w) {
#pragma unroll
  for (int i = 0; i < 16; ++i)
    w[i] = pack_bf16x2(act_f<kAct>(__uint_as_float(g[2 * i])) * __uint_as_float(u[2 * i]),
                       act_f<kAct>(__uint_as_float(g[2 * i + 1])) * __uint_as_float(u[2 * i + 1]));
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// 32 columns of dh and the kept A_g, A_u (16 words each) -> dA_g over g, dA_u over u,
// and h.
template <int kAct>
__device__ __forceinline__ void gated_bwd_words(const uint32_t* dh, uint32_t* g, uint32_t* u,
                                                uint32_t* h) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float f0, f1, d0, d1;
    act_both<kAct>(lo_f(g[i]), f0, d0);
    act_both<kAct>(hi_f(g[i]), f1, d1);
    const float u0 = lo_f(u[i]), u1 = hi_f(u[i]);
    const float e0 = __uint_as_float(dh[2 * i]), e1 = __uint_as_float(dh[2 * i + 1]);
    h[i] = pack_bf16x2(f0 * u0, f1 * u1);
    g[i] = pack_bf16x2(e0 * u0 * d0, e1 * u1 * d1);
    u[i] = pack_bf16x2(e0 * f0, e1 * f1);
  }
}

// ------------------------------------------------------------------ the kernel

template <Op op, int kBN>
__global__ void __launch_bounds__(kThreads, 1)
    dense_gemm_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args p) {
  extern __shared__ uint8_t smem_raw[];
  constexpr bool kAmn = a_mn<op>(), kBmn = b_mn<op>();
  constexpr bool kWGrad = op == Op::WGradB16 || op == Op::WGradF32;
  constexpr int S = stages<op>(), kLoads = loads<op>(), kSlots = out_slots<op>();
  constexpr int kHalfN = kBN / 2;              // columns of B that a CTA loads
  constexpr int kOutN = op == Op::Gated ? kBN / 2 : kBN;   // columns of the result in a tile
  uint8_t* ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* pieces = ring + S * kStageBytes;
  Smem* sm = reinterpret_cast<Smem*>(pieces + pieces_bytes<op>());
  const int warp = threadIdx.x >> 5, lane = lane_id();
  const uint32_t rank = cluster_ctarank();
  const int walk0 = static_cast<int>(blockIdx.x >> 1);
  const int step = static_cast<int>(gridDim.x >> 1);
  const int total = p.mt * p.nt;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&sm->full[s]), 1);
      mbar_init(smem_u32(&sm->empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&sm->tfull[a]), 1);
      mbar_init(smem_u32(&sm->tempty[a]), 8);   // the epilogue warps of both CTAs
      for (int q = 0; q < 4; ++q) mbar_init(smem_u32(&sm->in[q][a]), 1);
    }
    mbar_init(smem_u32(&sm->drain), 1);
    sm->abort = 0;
    sm->zero = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&sm->tmem_base), kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();            // both CTAs' barriers exist before either signals the other
  tc_fence_after();
  const uint32_t tmem_base = sm->tmem_base;
  volatile int* abort_flag = &sm->abort;

  if (warp == 0) {
    // ---------------------------------------------------------- producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, fills = 0;
      bool ok = true;
      const uint64_t pol = l2_policy_evict_normal();
      const uint32_t ring0 = smem_u32(ring);
      for (int t = walk0; t < total && ok; t += step) {
        const Tile tl = decode(t, p);
        const int m0 = (2 * tl.m + static_cast<int>(rank)) * kTileM;
        const bool second = kWGrad && tl.n >= p.nt0;        // WGrad: the second output
        int n0 = (kWGrad && second ? tl.n - p.nt0 : tl.n) * kOutN;
        if (op != Op::Gated) n0 += static_cast<int>(rank) * kHalfN;
        for (int kb = 0; kb < p.kb; ++kb) {
          const uint32_t full = smem_u32(&sm->full[stage]);
          if (!mbar_wait(smem_u32(&sm->empty[stage]), phase ^ 1, p.wait_ns, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t sa = ring0 + stage * kStageBytes, sb = sa + kABytes;
          // both CTAs' copies complete on the leader's barrier
          const uint32_t full_l = mapa_shared(full, 0);
          if (rank == 0) mbar_arrive_expect_tx(full, 2 * (kABytes + kHalfN * BK * 2));
          const bool part1 = op == Op::InGrad && kb >= p.kb0;
          const int k0 = (part1 ? kb - p.kb0 : kb) * BK;
          const CUtensorMap* ma = &maps.a[part1 ? 1 : 0];
          const CUtensorMap* mb =
              &maps.b[(op == Op::Gated ? rank == 1 : op == Op::InGrad ? part1 : second) ? 1 : 0];
          if (kAmn) {
            tma_load_2d_pair(sa, ma, full_l, m0, k0, pol);
            tma_load_2d_pair(sa + kBox, ma, full_l, m0 + 64, k0, pol);
          } else {
            tma_load_2d_pair(sa, ma, full_l, k0, m0, pol);
          }
          if (kBmn) {
#pragma unroll
            for (int j = 0; j < kHalfN / 64; ++j)
              tma_load_2d_pair(sb + j * kBox, mb, full_l, n0 + 64 * j, k0, pol);
          } else {
            tma_load_2d_pair(sb, mb, full_l, k0, n0, pol);
          }
          ++fills;
          if (++stage == S) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok) {
        sm->abort = 1;
        report_error(p.err, kErrTimeout);
      }
      // the last S fills have to land, and the MMAs that read them to be done, before
      // the CTA may exit: a slot is released only after both CTAs' copies into it
      // landed. After an abort the MMAs may never come, so the waits are short: a copy
      // lands within microseconds
      for (uint32_t i = fills > S ? fills - S : 0; i < fills; ++i)
        mbar_wait(smem_u32(&sm->empty[i % S]), (i / S) & 1, kPairDrainNs, &sm->zero);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = idesc_bf16(2 * kTileM, kBN, kAmn, kBmn);
      const uint32_t ring0 = smem_u32(ring);
      // K-major, 128-byte swizzle: groups of 8 rows 1 KB apart, 32 bytes a step of K = 16.
      // MN-major: atoms of 64 columns 8 KB apart, groups of 8 of K 1 KB apart, 2 KB a step
      const uint64_t ad0 = sdesc_sw128(ring0, kAmn ? kBox : 16, 1024);
      const uint64_t bd0 = sdesc_sw128(ring0 + kABytes, kBmn ? kBox : 16, 1024);
      constexpr uint64_t kAStep = kAmn ? (2048 >> 4) : (32 >> 4);
      constexpr uint64_t kBStep = kBmn ? (2048 >> 4) : (32 >> 4);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true, issued = false;
      for (int t = walk0; t < total && ok; t += step) {
        if (!mbar_wait(smem_u32(&sm->tempty[acc]), acc_phase ^ 1, p.wait_ns, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + acc * 256;
        for (int kb = 0; kb < p.kb; ++kb) {
          if (!mbar_wait(smem_u32(&sm->full[stage]), phase, p.wait_ns, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t off = static_cast<uint64_t>(stage) * (kStageBytes >> 4);
#pragma unroll
          for (int ks = 0; ks < BK / 16; ++ks)
            umma_bf16_pair(d, ad0 + off + ks * kAStep, bd0 + off + ks * kBStep, idesc,
                           (kb | ks) ? 1u : 0u);
          umma_commit_pair_mc(smem_u32(&sm->empty[stage]), 0x3);   // the slot, in both CTAs
          issued = true;
          if (++stage == S) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        umma_commit_pair_mc(smem_u32(&sm->tfull[acc]), 0x3);       // both CTAs' epilogues
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
      }
      if (!ok) {
        sm->abort = 1;
        report_error(p.err, kErrTimeout);
      }
      if (issued) {
        umma_commit_pair_mc(smem_u32(&sm->drain), 0x1);
        mbar_wait(smem_u32(&sm->drain), 0, kDrainNs, &sm->zero);
      }
    }
  } else {
    // ---------------------------------------------------------- epilogue
    const int q = warp & 3;                    // TMEM lane quadrant of this warp
    const uint32_t out0 = smem_u32(pieces) + q * kSlots * kPieceBytes;
    const uint32_t in0 = smem_u32(pieces) + 4 * kSlots * kPieceBytes + q * 2 * kLoads * kPieceBytes;
    const uint32_t my_row = lane * 64, sw = (lane >> 1) & 3;
    int npiece = 0;
    uint32_t n_asked = 0, n_got = 0;           // steps of 32 columns asked for, and waited for
    // 16-byte chunk j of row r of a piece lies at chunk j ^ ((r >> 1) & 3)
    auto put = [&](const uint32_t* w, const CUtensorMap* map, int x, int y, bool add) {
      if (lane == 0) bulk_wait_group_read<kSlots - 1>();
      __syncwarp();
      const uint32_t slot = out0 + (npiece % kSlots) * kPieceBytes;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(slot + my_row + ((j ^ sw) << 4)),
                     "r"(w[4 * j]), "r"(w[4 * j + 1]), "r"(w[4 * j + 2]), "r"(w[4 * j + 3])
                     : "memory");
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) {
        if (add) tma_reduce_add_2d(map, slot, x, y);
        else tma_store_2d(map, slot, x, y);
        bulk_commit_group();
      }
      ++npiece;
    };
    auto get = [&](uint32_t slot, uint32_t* w) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[4 * j]), "=r"(w[4 * j + 1]), "=r"(w[4 * j + 2]), "=r"(w[4 * j + 3])
                     : "r"(slot + my_row + ((j ^ sw) << 4))
                     : "memory");
    };
    const bool reads = kLoads == 2 || (kLoads == 1 && p.add != 0);
    auto ask = [&](int x, int y) {             // the pieces of the next 32 columns
      if (lane == 0) {
        const int b = n_asked & 1;
        const uint32_t bar = smem_u32(&sm->in[q][b]);
        mbar_arrive_expect_tx(bar, kLoads * kPieceBytes);
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          tma_load_2d(in0 + (b * kLoads + i) * kPieceBytes, &maps.in[i], bar, x, y);
      }
      ++n_asked;
    };
    int acc = 0;
    uint32_t acc_phase = 0;
    const uint32_t tempty0 = mapa_shared(smem_u32(&sm->tempty[0]), 0);
    bool ok = true;
    for (int t = walk0; t < total && ok; t += step) {
      const Tile tl = decode(t, p);
      const bool second = kWGrad && tl.n >= p.nt0;
      const int n0 = (second ? tl.n - p.nt0 : tl.n) * kOutN;
      const int y = (2 * tl.m + static_cast<int>(rank)) * kTileM + q * 32;
      const int cols = y < p.M ? min(kOutN, p.N - n0) : 0;     // 0: nothing of this warp's
      if (reads && cols > 0) ask(n0, y);
      const bool got = mbar_wait(smem_u32(&sm->tfull[acc]), acc_phase, p.wait_ns, abort_flag);
      // tcgen05.ld is warp-collective: the whole warp goes on or stops together
      if (!__all_sync(0xffffffffu, got)) {
        sm->abort = 1;
        if (lane == 0) report_error(p.err, kErrTimeout);
        break;
      }
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * 256;
#pragma unroll 1
      for (int c = 0; c < cols; c += 32) {
        uint32_t v[32], g[16], u[16];
        if (reads) {
          if (c + 32 < cols) ask(n0 + c + 32, y);
          const int b = n_got & 1;
          const bool here = mbar_wait(smem_u32(&sm->in[q][b]), (n_got >> 1) & 1, p.wait_ns,
                                      abort_flag);
          if (!__all_sync(0xffffffffu, here)) {
            sm->abort = 1;
            if (lane == 0) report_error(p.err, kErrTimeout);
            ok = false;
            break;
          }
          ++n_got;
          get(in0 + b * kLoads * kPieceBytes, g);
          if (kLoads == 2) get(in0 + (b * kLoads + 1) * kPieceBytes, u);
        }
        tmem_ld_32x32b_x32(taddr + c, v);
        if (op == Op::Gated) {
          uint32_t up[32], w[16];
          tmem_ld_32x32b_x32(taddr + kBN / 2 + c, up);
          tmem_ld_wait();
          switch (p.act) {
            case MOE_ACT_SILU: gated_words<MOE_ACT_SILU>(v, up, w); break;
            case MOE_ACT_GELU: gated_words<MOE_ACT_GELU>(v, up, w); break;
            case MOE_ACT_GELU_TANH: gated_words<MOE_ACT_GELU_TANH>(v, up, w); break;
            default: gated_words<MOE_ACT_RELU>(v, up, w); break;
          }
          put(w, &maps.out[0], n0 + c, y, false);
          if (p.keep) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              w[i] = pack_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
            put(w, &maps.out[1], n0 + c, y, false);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              w[i] = pack_bf16x2(__uint_as_float(up[2 * i]), __uint_as_float(up[2 * i + 1]));
            put(w, &maps.out[2], n0 + c, y, false);
          }
        } else if (op == Op::GatedBwd) {
          uint32_t h[16];
          tmem_ld_wait();
          switch (p.act) {
            case MOE_ACT_SILU: gated_bwd_words<MOE_ACT_SILU>(v, g, u, h); break;
            case MOE_ACT_GELU: gated_bwd_words<MOE_ACT_GELU>(v, g, u, h); break;
            case MOE_ACT_GELU_TANH: gated_bwd_words<MOE_ACT_GELU_TANH>(v, g, u, h); break;
            default: gated_bwd_words<MOE_ACT_RELU>(v, g, u, h); break;
          }
          put(h, &maps.out[0], n0 + c, y, false);
          put(g, &maps.out[1], n0 + c, y, false);
          put(u, &maps.out[2], n0 + c, y, false);
        } else if (op == Op::WGradF32) {
          tmem_ld_wait();
          const CUtensorMap* map = &maps.out[second ? 1 : 0];
          put(v, map, n0 + c, y, p.accumulate != 0);
          if (c + 16 < cols) put(v + 16, map, n0 + c + 16, y, p.accumulate != 0);
        } else {
          uint32_t w[16];
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float a = __uint_as_float(v[2 * i]), b = __uint_as_float(v[2 * i + 1]);
            if (reads) {
              a += lo_f(g[i]);
              b += hi_f(g[i]);
            }
            w[i] = pack_bf16x2(a, b);
          }
          put(w, &maps.out[second ? 1 : 0], n0 + c, y, false);
        }
        __syncwarp();       // this step's pieces are read before they are asked for again
      }
      if (!ok) break;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(tempty0 + acc * static_cast<uint32_t>(sizeof(uint64_t)));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    }
    // what was asked for lands, and every store has been made, before the CTA exits
    for (; n_got != n_asked; ++n_got)
      mbar_wait(smem_u32(&sm->in[q][n_got & 1]), (n_got >> 1) & 1, kDrainNs, &sm->zero);
    if (lane == 0) bulk_wait_group_all();
  }

  tc_fence_before();
  __syncthreads();
  // neither CTA leaves while the other may still signal its barriers, read its slots
  // (the leader's MMAs) or write its accumulators
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

template <Op op, int kBN>
cudaError_t launch_bn(const Maps& maps, const Args& p, cudaStream_t st) {
  auto kern = dense_gemm_kernel<op, kBN>;
  static bool configured[kMaxDevices] = {};
  static int max_pairs[kMaxDevices] = {};       // clusters of two that fit at once
  const int d = current_device();
  if (d < 0 || d >= kMaxDevices) return cudaErrorInvalidDevice;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<op>();
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (!configured[d]) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem_bytes<op>()));
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(2 * kMaxDevices);        // any even size: the query asks how many fit
    e = cudaOccupancyMaxActiveClusters(&max_pairs[d], kern, &cfg);
    if (e != cudaSuccess) return e;
    if (max_pairs[d] < 1) return cudaErrorInvalidConfiguration;
    configured[d] = true;
  }
  const int64_t total = static_cast<int64_t>(p.mt) * p.nt;
  cfg.gridDim = dim3(2 * static_cast<int>(total < max_pairs[d] ? total : max_pairs[d]));
  return cudaLaunchKernelEx(&cfg, kern, maps, p);
}

int up_div(int64_t a, int b) { return static_cast<int>((a + b - 1) / b); }

// Tiles of a [M, N] result with tiles of 256 x bn, N columns in each of n_out outputs.
void set_tiles(Args& p, int64_t M, int N, int bn, int n_out) {
  p.M = static_cast<int>(M);
  p.N = N;
  p.mt = up_div(M, 2 * kTileM);
  p.nt0 = up_div(N, bn);
  p.nt = n_out * p.nt0;
  p.group = p.mt < 16 ? p.mt : 16;
}

// Tiles half as wide where whole ones (of bn columns) would leave clusters without one.
bool narrow(int64_t M, int N, int bn, int n_out) {
  return static_cast<int64_t>(up_div(M, 2 * kTileM)) * up_div(N, bn) * n_out <
         device_sm_count() / 2;
}

template <Op op>
cudaError_t launch(Maps& maps, Args& p, int64_t M, int N, int n_out, cudaStream_t st) {
  constexpr int bn = op == Op::Gated ? 128 : 256;
  if (narrow(M, N, bn, n_out)) {
    set_tiles(p, M, N, bn / 2, n_out);
    return launch_bn<op, 128>(maps, p, st);
  }
  set_tiles(p, M, N, bn, n_out);
  return launch_bn<op, 256>(maps, p, st);
}

bool in_map(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint32_t box_outer) {
  return make_tmap_bf16_2d(m, base, inner, outer, inner * 2, BK, box_outer);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
size_t up256(size_t b) { return (b + 255) / 256 * 256; }

moe_status check_sizes(int64_t T, int H, int F, int act) {
  if (T < 0 || T > INT32_MAX - 1024 || H <= 0 || F <= 0 || H > (1 << 30) || F > (1 << 30) ||
      act < MOE_ACT_SILU || act > MOE_ACT_RELU)
    return MOE_ERR_INVALID_ARG;
  return (H % 8 || F % 8) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// mt * nt stays below 2^31 where the tensors fit in memory at all; refuse the rest
bool tiles_fit(int64_t M, int N) {
  return static_cast<int64_t>(up_div(M, 2 * kTileM)) * up_div(N, 64) * 2 < INT32_MAX;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_gated_ffn_workspace_size(int64_t T, int H, int F) {
  if (check_sizes(T, H, F, 0) != MOE_OK) return 0;
  return up256(static_cast<size_t>(T) * F * 2);
}

moe_status moe_gated_ffn(const void* x, const void* w_gate, const void* w_up, const void* w_down,
                         const void* add, int64_t T, int H, int F, int act, void* y, void* a_gate,
                         void* a_up, void* workspace, size_t ws_bytes, void* stream) {
  MOE_ENTRY_RANGE();
  const moe_status s = check_sizes(T, H, F, act);
  if (s != MOE_OK) return s;
  if (T == 0) return MOE_OK;
  if (!x || !w_gate || !w_up || !w_down || !y || !a_gate != !a_up) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w_gate) || !aligned16(w_up) || !aligned16(w_down) ||
      !aligned16(add) || !aligned16(y) || !aligned16(a_gate) || !aligned16(a_up) ||
      !tiles_fit(T, F) || !tiles_fit(T, H))
    return MOE_ERR_INVALID_ARG;
  if (!workspace || ws_bytes < moe_gated_ffn_workspace_size(T, H, F) || !aligned16(workspace))
    return MOE_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T <= kFewRows)
    return ffn_few_rows(x, w_gate, w_up, w_down, add, static_cast<int>(T), H, F, act, y, a_gate,
                        a_up, workspace, device_error_word(), st) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
  Args p{};
  p.act = act;
  p.err = device_error_word();
  p.wait_ns = kDefaultWaitNs;
  Maps m1{}, m2{};
  const uint64_t rF = static_cast<uint64_t>(F) * 2, rH = static_cast<uint64_t>(H) * 2;
  if (!in_map(&m1.a[0], x, H, T, kTileM) || !in_map(&m1.b[0], w_gate, F, H, BK) ||
      !in_map(&m1.b[1], w_up, F, H, BK) || !make_out_tmap(&m1.out[0], workspace, F, T, rF, false) ||
      (a_gate && (!make_out_tmap(&m1.out[1], a_gate, F, T, rF, false) ||
                  !make_out_tmap(&m1.out[2], a_up, F, T, rF, false))) ||
      !in_map(&m2.a[0], workspace, F, T, kTileM) || !in_map(&m2.b[0], w_down, H, F, BK) ||
      !make_out_tmap(&m2.out[0], y, H, T, rH, false) ||
      (add && !make_out_tmap(&m2.in[0], add, H, T, rH, false)))
    return MOE_ERR_CUDA;
  Args p1 = p, p2 = p;
  p1.keep = a_gate != nullptr;
  p1.kb = p1.kb0 = up_div(H, BK);
  p2.add = add != nullptr;
  p2.kb = p2.kb0 = up_div(F, BK);
  if (launch<Op::Gated>(m1, p1, T, F, 1, st) != cudaSuccess ||
      launch<Op::Down>(m2, p2, T, H, 1, st) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_OK;
}

size_t moe_gated_ffn_backward_workspace_size(int64_t T, int H, int F) {
  if (check_sizes(T, H, F, 0) != MOE_OK) return 0;
  return 3 * up256(static_cast<size_t>(T) * F * 2);
}

moe_status moe_gated_ffn_backward(const void* dy, const void* x, const void* w_gate,
                                  const void* w_up, const void* w_down, const void* a_gate,
                                  const void* a_up, const void* add, int64_t T, int H, int F,
                                  int act, void* dx, void* dw_gate, void* dw_up, void* dw_down,
                                  int dw_type, int accumulate_dw, void* workspace, size_t ws_bytes,
                                  void* stream) {
  MOE_ENTRY_RANGE();
  const moe_status s = check_sizes(T, H, F, act);
  if (s != MOE_OK) return s;
  if (!dw_gate != !dw_up || !dw_gate != !dw_down || !aligned16(dw_gate) || !aligned16(dw_up) ||
      !aligned16(dw_down) || (dw_type != MOE_TYPE_F32 && dw_type != MOE_TYPE_BF16))
    return MOE_ERR_INVALID_ARG;
  const bool f32 = dw_type == MOE_TYPE_F32;
  if (dw_gate && accumulate_dw && !f32) return MOE_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    if (!dw_gate || accumulate_dw) return MOE_OK;
    const size_t bytes = static_cast<size_t>(H) * F * (f32 ? 4 : 2);
    return cudaMemsetAsync(dw_gate, 0, bytes, st) == cudaSuccess &&
                   cudaMemsetAsync(dw_up, 0, bytes, st) == cudaSuccess &&
                   cudaMemsetAsync(dw_down, 0, bytes, st) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
  }
  if (!dy || !x || !w_gate || !w_up || !w_down || !a_gate || !a_up || !dx)
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(dy) || !aligned16(x) || !aligned16(w_gate) || !aligned16(w_up) ||
      !aligned16(w_down) || !aligned16(a_gate) || !aligned16(a_up) || !aligned16(add) ||
      !aligned16(dx) || !tiles_fit(T, F) || !tiles_fit(T, H) || !tiles_fit(H, F) ||
      !tiles_fit(F, H))
    return MOE_ERR_INVALID_ARG;
  if (!workspace || ws_bytes < moe_gated_ffn_backward_workspace_size(T, H, F) ||
      !aligned16(workspace))
    return MOE_ERR_WORKSPACE;
  const size_t each = up256(static_cast<size_t>(T) * F * 2);
  void* h = workspace;
  void* da_g = static_cast<char*>(workspace) + each;
  void* da_u = static_cast<char*>(workspace) + 2 * each;
  const uint64_t rF = static_cast<uint64_t>(F) * 2, rH = static_cast<uint64_t>(H) * 2;
  Args p{};
  p.act = act;
  p.err = device_error_word();
  p.wait_ns = kDefaultWaitNs;
  Maps m2{}, m1{};
  if (T <= kFewRows) {
    if (ffn_few_rows_backward(dy, w_gate, w_up, w_down, a_gate, a_up, add, static_cast<int>(T), H,
                              F, act, dx, h, da_g, da_u, p.err, st) != cudaSuccess)
      return MOE_ERR_CUDA;
  } else {
    // K-major B: one box of the columns that a CTA loads
    const uint32_t box_h = narrow(T, F, 256, 1) ? 64 : 128, box_x = narrow(T, H, 256, 1) ? 64 : 128;
    Maps mh{}, mx{};
    if (!in_map(&mh.a[0], dy, H, T, kTileM) || !in_map(&mh.b[0], w_down, H, F, box_h) ||
        !make_out_tmap(&mh.in[0], a_gate, F, T, rF, false) ||
        !make_out_tmap(&mh.in[1], a_up, F, T, rF, false) ||
        !make_out_tmap(&mh.out[0], h, F, T, rF, false) ||
        !make_out_tmap(&mh.out[1], da_g, F, T, rF, false) ||
        !make_out_tmap(&mh.out[2], da_u, F, T, rF, false) ||
        !in_map(&mx.a[0], da_g, F, T, kTileM) || !in_map(&mx.a[1], da_u, F, T, kTileM) ||
        !in_map(&mx.b[0], w_gate, F, H, box_x) || !in_map(&mx.b[1], w_up, F, H, box_x) ||
        !make_out_tmap(&mx.out[0], dx, H, T, rH, false) ||
        (add && !make_out_tmap(&mx.in[0], add, H, T, rH, false)))
      return MOE_ERR_CUDA;
    Args ph = p, px = p;
    ph.kb = ph.kb0 = up_div(H, BK);
    px.kb0 = up_div(F, BK);
    px.kb = 2 * px.kb0;
    px.add = add != nullptr;
    if (launch<Op::GatedBwd>(mh, ph, T, F, 1, st) != cudaSuccess ||
        launch<Op::InGrad>(mx, px, T, H, 1, st) != cudaSuccess)
      return MOE_ERR_CUDA;
  }
  if (!dw_gate) return MOE_OK;
  const uint64_t z = f32 ? 4 : 2;
  if (!in_map(&m2.a[0], h, F, T, BK) || !in_map(&m2.b[0], dy, H, T, BK) ||
      !make_out_tmap(&m2.out[0], dw_down, H, F, static_cast<uint64_t>(H) * z, f32) ||
      !in_map(&m1.a[0], x, H, T, BK) || !in_map(&m1.b[0], da_g, F, T, BK) ||
      !in_map(&m1.b[1], da_u, F, T, BK) ||
      !make_out_tmap(&m1.out[0], dw_gate, F, H, static_cast<uint64_t>(F) * z, f32) ||
      !make_out_tmap(&m1.out[1], dw_up, F, H, static_cast<uint64_t>(F) * z, f32))
    return MOE_ERR_CUDA;
  Args pw = p;
  pw.kb = pw.kb0 = up_div(T, BK);
  pw.accumulate = accumulate_dw;
  Args pw1 = pw;
  const cudaError_t e2 = f32 ? launch<Op::WGradF32>(m2, pw, F, H, 1, st)
                             : launch<Op::WGradB16>(m2, pw, F, H, 1, st);
  if (e2 != cudaSuccess) return MOE_ERR_CUDA;
  const cudaError_t e1 = f32 ? launch<Op::WGradF32>(m1, pw1, H, F, 2, st)
                             : launch<Op::WGradB16>(m1, pw1, H, F, 2, st);
  return e1 == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
