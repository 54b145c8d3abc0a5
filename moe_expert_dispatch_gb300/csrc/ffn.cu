// ffn.cu - the gated feed-forward block of a dense layer (moe_gated_ffn and
// its backward): persistent GEMMs on the 5th-generation tensor cores with the
// activation, the product and its gradient in their epilogues.
//
//   Gated     [A_g | A_u] = x [W_gate | W_up],  h = bf16(act(A_g) A_u)
//   Down      y = bf16(add + h W_down)
//   GatedBwd  dh = dy W_down^T; h, dA_g, dA_u from it and the kept A_g, A_u
//   Joint     dx = bf16(add + dA_g W_gate^T + dA_u W_up^T), one accumulator, and
//             dW_down = h^T dy, dW_gate = x^T dA_g, dW_up = x^T dA_u: nothing of
//             these waits for another, so their tiles are one launch
//
// h, dA_g and dA_u are rounded to bf16 because the next product takes them as operands: in
// two parts each they would cost it a second pass of MMAs. Each is off by up to 2^-8, which
// averages over a sum to about what the result's own rounding is off by: on Gaussian inputs
// the results are 0.0024 (root mean square) off float64's, 0.0017 with all three in float.
//
// One kernel body serves the four. A cluster of two CTAs shares a tile of 256
// rows and 256 columns (tcgen05.mma.cta_group::2): each CTA loads its own 128
// rows of A and half of the tile's columns of B, the leader issues the MMAs, and
// each CTA finishes its own 128 rows. Of a Gated tile one CTA loads columns of
// W_gate and the other the same columns of W_up, so that the accumulator holds A_g
// and A_u of a row in one lane. Warps: 0 the TMA producer, 1 the MMA issuer, 2 to 9
// the epilogue (two to a quarter of the rows, taking turns at 32 columns); two
// accumulators, so that the epilogue of a tile runs beside the MMAs of the next (or of
// the next run of rows of a weight gradient).
//
// Nothing is padded: rows and columns past the matrices are the zeros that TMA
// fills in, they add nothing, and the stores are clipped (or, where a whole piece
// lies outside, left out). What the epilogues read besides the accumulator (A_g and
// A_u, or add) arrives by TMA in pieces of 32 rows x 32 columns, a step ahead.
//
// Where a product has fewer tiles than the GPU has room for clusters and a long K
// (short batches), K is split: the parts of a tile leave their accumulators as they
// are, in float, and a small kernel adds them up in their order and does what the
// epilogue would have done. The split is chosen from the sizes alone, so that the
// same call gives the same bits.
#include "act.cuh"
#include "common.cuh"
#include "ffn.h"
#include "internal.h"

namespace moe {

int* device_error_word();

namespace {

enum class Op { Gated, Down, GatedBwd, Joint };
// What a tile of Joint is; Main is the product of the other three, and dx.
enum Kind { kNone = -1, kMain = 0, kDwDown = 1, kDwGate = 2, kDwUp = 3 };

constexpr int BK = 64;                         // k-block: 128 bytes of bf16
constexpr int BN = 256;                        // columns of an accumulator
constexpr int kABytes = kTileM * BK * 2;       // 16 KB: this CTA's rows of A
constexpr int kBox = 64 * BK * 2;              // 8 KB: 64 columns x 64 of K
constexpr int kStageBytes = 2 * kABytes;       // A and 128 columns of B
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr uint32_t kTmemCols = 512;
constexpr int kPieceBytes = 32 * 64;           // 32 rows x 64 bytes, 64-byte swizzle
constexpr int kSlots = 2;                      // pieces on their way out, of a warp
constexpr unsigned long long kDrainNs = 1000000000ull;
constexpr unsigned long long kPairDrainNs = 50000000ull;
constexpr int kMaxSplit = 8;
// The tensor cores cut off what does not fit in their float sums, so that a long sum of
// one sign ends too small: by 2^-20.1 of itself over 512 rows, 2^-14.8 over 8192, 2^-13.6
// over 16384. A weight gradient sums over the rows; its accumulators are therefore taken out
// every so many k-blocks and added up in registers, which round. In float every 512 rows,
// in bf16 every 8192, where 2^-14.8 is far below its rounding. The float gradients of 8192
// rows of 4096 x 14336 take 3743 us so (every 256 rows some 4100) and 3555 to 3680 by one
// accumulator, those of 1024 rows 508 and 480, of 2048 rows of 2048 x 768 45 and 43.
constexpr int kRunF32 = 8;
constexpr int kRunBf16 = 128;

// Pieces that a warp reads for 32 columns: one goes out again in its own place, two have
// places beside those of the pieces that go out. The ring depth that 227 KB leave.
template <Op op>
constexpr int loads() { return op == Op::GatedBwd ? 2 : op == Op::Gated ? 0 : 1; }
template <Op op>
constexpr int in_slots() { return op == Op::GatedBwd ? 2 : 0; }
template <Op op>
constexpr int stages() { return op == Op::GatedBwd ? 5 : 6; }
constexpr int kMaxStages = 6;

struct Smem {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t in[kEpiWarps];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int zero;
};

template <Op op>
constexpr int pieces_bytes() { return kEpiWarps * (kSlots + in_slots<op>()) * kPieceBytes; }
template <Op op>
constexpr size_t smem_bytes() {
  return 1024 + static_cast<size_t>(stages<op>()) * kStageBytes + pieces_bytes<op>() + sizeof(Smem);
}
static_assert(smem_bytes<Op::Gated>() <= 232448 && smem_bytes<Op::Down>() <= 232448 &&
              smem_bytes<Op::GatedBwd>() <= 232448 && smem_bytes<Op::Joint>() <= 232448,
              "shared memory of one CTA");

// Operands by kind: Main a[0], b[0] (a[1], b[1]: W_up, or dA_u with W_up), the
// weight gradients from [2] on.
struct Maps {
  CUtensorMap a[4], b[5];
  CUtensorMap out[4], in[2], part;
};

// n / d for n below 2^31 by a product and a shift (Granlund and Montgomery: "Division by
// invariant integers using multiplication", 1994): a tile's place takes four divisions,
// which the hardware has to go through step by step.
struct Divisor {
  uint32_t d, m, l;
};

__device__ __forceinline__ int quotient(int n, const Divisor& v) {
  return static_cast<int>((__umulhi(static_cast<uint32_t>(n), v.m) + static_cast<uint32_t>(n)) >> v.l);
}

struct Grid {
  int M, N;          // rows and columns of the result
  int mt, nt;        // tiles
  int group;         // row tiles that one column tile is walked over
  Divisor per, whole, last;    // tiles of a group; row tiles of a whole one, of the last
};

struct Args {
  Grid main, down, gate;       // Joint: dW_down; dW_gate and dW_up
  int kb0, kb;                 // Main: k-blocks of the first pair of operands, and of both
  int kb_rows;                 // weight gradients: k-blocks (of rows)
  int split, per;              // Main: parts of K, k-blocks of a part
  int units;                   // of Main: tiles times parts
  Divisor tiles;               // of Main
  int rounds, rest;            // units = rounds * clusters + rest
  int dw_units;                // tiles of the weight gradients
  int skip;                    // their rounds that clusters with a unit of Main stay out of
  int act;
  int keep;                    // Gated: A_g and A_u are stored
  int add;                     // Down, Joint: in[0] is added
  int f32, accumulate;         // weight gradients
  int run;                     // their k-blocks to an accumulator
  int* err;
  unsigned long long wait_ns;
};

struct Unit {
  int kind, m, n, part, kb0, kb1;              // tiles below 2^26, parts up to kMaxSplit
};

// Column tiles follow one another over groups of row tiles: a group's rows of A
// stay in L2 while the columns of B stream by once a group.
__device__ __forceinline__ void place(int t, const Grid& g, Unit& u) {
  const int i = quotient(t, g.per), local = t - i * static_cast<int>(g.per.d);
  const Divisor& rows = (i + 1) * g.group <= g.mt ? g.whole : g.last;
  u.n = quotient(local, rows);
  u.m = i * g.group + local - u.n * static_cast<int>(rows.d);
}

// The i-th unit of a cluster (its tile and part). Units of Main go round the clusters. Weight gradients
// follow: where Main has fewer units than there are clusters, those with one join in
// when the others have done as much.
template <Op op>
__device__ __forceinline__ Unit unit_at(int i, const Args& p, int cluster, int clusters) {
  Unit u = {kNone, 0, 0, 0, 0, 0};
  int t = cluster + i * clusters;
  if (t < p.units) {
    u.kind = kMain;
    u.part = quotient(t, p.tiles);
    place(t - u.part * static_cast<int>(p.tiles.d), p.main, u);
    return u;
  }
  if (op != Op::Joint) return u;
  const int r = i - p.rounds - (cluster < p.rest ? 1 : 0);
  if (p.units < clusters) {
    const int rest = clusters - p.units;
    if (cluster >= p.units && r < p.skip) t = r * rest + cluster - p.units;
    else t = p.skip * rest + (cluster >= p.units ? r - p.skip : r) * clusters + cluster;
  } else {
    t = r * clusters + cluster - p.rest + (cluster < p.rest ? clusters : 0);
  }
  if (t >= p.dw_units) return u;
  const int down = p.down.mt * p.down.nt, gate = p.gate.mt * p.gate.nt;
  if (t < down) {
    u.kind = kDwDown;
    place(t, p.down, u);
  } else {
    u.kind = t - down < gate ? kDwGate : kDwUp;
    place(t - down - (u.kind == kDwUp ? gate : 0), p.gate, u);
  }
  return u;
}

// The units of a cluster in turn, for a whole warp: 32 of them are worked out at once,
// one a lane, and dealt out by shuffles: worked out one by one they took half the time
// of a weight gradient over few rows.
template <Op op>
struct Units {
  const Args& p;
  int cluster, clusters;
  uint32_t where, what;        // row tile and kind + 1; column tile and part
  __device__ __forceinline__ Unit get(int i) {
    if ((i & 31) == 0) {
      const Unit u = unit_at<op>(i + lane_id(), p, cluster, clusters);
      where = static_cast<uint32_t>(u.m) | static_cast<uint32_t>(u.kind + 1) << 28;
      what = static_cast<uint32_t>(u.n) | static_cast<uint32_t>(u.part) << 28;
    }
    const uint32_t a = __shfl_sync(0xffffffffu, where, i & 31);
    const uint32_t b = __shfl_sync(0xffffffffu, what, i & 31);
    Unit u;
    u.kind = static_cast<int>(a >> 28) - 1;
    u.m = static_cast<int>(a & 0xFFFFFFFu);
    u.n = static_cast<int>(b & 0xFFFFFFFu);
    u.part = static_cast<int>(b >> 28);
    u.kb0 = u.kind == kMain ? min(p.kb, u.part * p.per) : 0;
    u.kb1 = u.kind == kMain ? min(p.kb, u.kb0 + p.per) : p.kb_rows;
    return u;
  }
};

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

// 2 n columns of dh and the kept A_g, A_u (n words each) -> dA_g over g, dA_u over u,
// and h.
template <int kAct, int n>
__device__ __forceinline__ void gated_bwd_words(const uint32_t* dh, uint32_t* g, uint32_t* u,
                                                uint32_t* h) {
#pragma unroll
  for (int i = 0; i < n; ++i) {
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

template <int n>
__device__ __forceinline__ void gated_bwd_any(int act, const uint32_t* dh, uint32_t* g, uint32_t* u,
                                              uint32_t* h) {
  switch (act) {
    case MOE_ACT_SILU: gated_bwd_words<MOE_ACT_SILU, n>(dh, g, u, h); break;
    case MOE_ACT_GELU: gated_bwd_words<MOE_ACT_GELU, n>(dh, g, u, h); break;
    case MOE_ACT_GELU_TANH: gated_bwd_words<MOE_ACT_GELU_TANH, n>(dh, g, u, h); break;
    default: gated_bwd_words<MOE_ACT_RELU, n>(dh, g, u, h); break;
  }
}

// ------------------------------------------------------------------ the kernel

// kRuns (of Joint): the rows of a weight gradient are more than one run of k-blocks. A
// kernel of its own, because the 128 sums of a thread take all registers: in one kernel for
// both, the gradients of 256 rows of 2048 x 768 took 25 us instead of 23.6.
template <Op op, bool kRuns>
__global__ void __launch_bounds__(kThreads, 1)
    dense_gemm_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args p) {
  extern __shared__ uint8_t smem_raw[];
  constexpr int S = stages<op>(), kLoads = loads<op>();
  uint8_t* ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* pieces = ring + S * kStageBytes;
  Smem* sm = reinterpret_cast<Smem*>(pieces + pieces_bytes<op>());
  const int warp = threadIdx.x >> 5, lane = lane_id();
  const uint32_t rank = cluster_ctarank();
  const int cluster = static_cast<int>(blockIdx.x >> 1);
  const int clusters = static_cast<int>(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&sm->full[s]), 1);
      mbar_init(smem_u32(&sm->empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&sm->tfull[a]), 1);
      mbar_init(smem_u32(&sm->tempty[a]), 2 * kEpiWarps);   // the epilogue warps of both CTAs
    }
    for (int e = 0; e < kEpiWarps; ++e) mbar_init(smem_u32(&sm->in[e]), 1);
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
  grid_dependency_wait();    // Joint and Down run beside the launch before them
  grid_dependents_launch();
  Units<op> units = {p, cluster, clusters, 0, 0};

  if (warp == 0) {
    // ---------------------------------------------------------- producer
    int stage = 0;
    uint32_t phase = 0, fills = 0;
    bool ok = true;
    const uint64_t pol = l2_policy_evict_normal();
    const uint32_t ring0 = smem_u32(ring);
    if (lane == 0) fence_proxy_async();
    for (int i = 0; __shfl_sync(0xffffffffu, ok, 0); ++i) {
      const Unit u = units.get(i);
      if (u.kind == kNone) break;
      if (lane == 0) {
        const bool wgrad = op == Op::Joint && u.kind != kMain;
        const int m0 = (2 * u.m + static_cast<int>(rank)) * kTileM;
        const int n0 = op == Op::Gated ? u.n * (BN / 2)
                                       : u.n * BN + static_cast<int>(rank) * (BN / 2);
        for (int kb = u.kb0; kb < u.kb1; ++kb) {
          const uint32_t full = smem_u32(&sm->full[stage]);
          if (!mbar_wait(smem_u32(&sm->empty[stage]), phase ^ 1, p.wait_ns, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t sa = ring0 + stage * kStageBytes, sb = sa + kABytes;
          // both CTAs' copies complete on the leader's barrier
          const uint32_t full_l = mapa_shared(full, 0);
          if (rank == 0) mbar_arrive_expect_tx(full, 2 * kStageBytes);
          if (wgrad) {                         // both operands MN-major: boxes of 64 columns
            const CUtensorMap* ma = &maps.a[u.kind == kDwDown ? 2 : 3];
            const CUtensorMap* mb = &maps.b[1 + u.kind];
            tma_load_2d_pair(sa, ma, full_l, m0, kb * BK, pol);
            tma_load_2d_pair(sa + kBox, ma, full_l, m0 + 64, kb * BK, pol);
            tma_load_2d_pair(sb, mb, full_l, n0, kb * BK, pol);
            tma_load_2d_pair(sb + kBox, mb, full_l, n0 + 64, kb * BK, pol);
          } else {
            const int second = op == Op::Joint && kb >= p.kb0 ? 1 : 0;
            const int k0 = (second ? kb - p.kb0 : kb) * BK;
            tma_load_2d_pair(sa, &maps.a[second], full_l, k0, m0, pol);
            if (op == Op::Gated || op == Op::Down) {
              const CUtensorMap* mb = &maps.b[op == Op::Gated ? rank : 0];
              tma_load_2d_pair(sb, mb, full_l, n0, k0, pol);
              tma_load_2d_pair(sb + kBox, mb, full_l, n0 + 64, k0, pol);
            } else {
              tma_load_2d_pair(sb, &maps.b[second], full_l, k0, n0, pol);
            }
          }
          ++fills;
          if (++stage == S) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
    }
    if (lane == 0) {
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
    if (rank == 0) {
      constexpr bool kBmnMain = op == Op::Gated || op == Op::Down;
      // K-major, 128-byte swizzle: groups of 8 rows 1 KB apart, 32 bytes a step of K = 16.
      // MN-major: atoms of 64 columns 8 KB apart, groups of 8 of K 1 KB apart, 2 KB a step
      const uint32_t ring0 = smem_u32(ring);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true, issued = false;
      for (int i = 0; __shfl_sync(0xffffffffu, ok, 0); ++i) {
        const Unit u = units.get(i);
        if (u.kind == kNone) break;
        if (lane != 0) continue;
        const bool wgrad = op == Op::Joint && u.kind != kMain, bmn = kBmnMain || wgrad;
        const uint32_t idesc = idesc_bf16(2 * kTileM, BN, wgrad, bmn);
        const uint64_t ad0 = sdesc_sw128(ring0, wgrad ? kBox : 16, 1024);
        const uint64_t bd0 = sdesc_sw128(ring0 + kABytes, bmn ? kBox : 16, 1024);
        const uint64_t a_step = wgrad ? 2048 >> 4 : 32 >> 4, b_step = bmn ? 2048 >> 4 : 32 >> 4;
        // an accumulator takes up a unit's k-blocks, a weight gradient's by runs
        for (int kb = u.kb0; ok;) {
          const int first = kb, end = kRuns && wgrad ? min(kb + p.run, u.kb1) : u.kb1;
          if (!mbar_wait(smem_u32(&sm->tempty[acc]), acc_phase ^ 1, p.wait_ns, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + acc * BN;
          for (; kb < end; ++kb) {
            if (!mbar_wait(smem_u32(&sm->full[stage]), phase, p.wait_ns, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t off = static_cast<uint64_t>(stage) * (kStageBytes >> 4);
#pragma unroll
            for (int ks = 0; ks < BK / 16; ++ks)
              umma_bf16_pair(d, ad0 + off + ks * a_step, bd0 + off + ks * b_step, idesc,
                             (kb > first || ks) ? 1u : 0u);
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
          if (kb >= u.kb1) break;
        }
      }
      if (!ok) {
        sm->abort = 1;
        report_error(p.err, kErrTimeout);
      }
      if (issued) {                            // of lane 0 alone
        umma_commit_pair_mc(smem_u32(&sm->drain), 0x1);
        mbar_wait(smem_u32(&sm->drain), 0, kDrainNs, &sm->zero);
      }
    }
  } else {
    // ---------------------------------------------------------- epilogue
    const int e = warp - 2, q = warp & 3;      // q: TMEM lane quadrant of this warp
    const int c_first = (e >> 2) * 32;         // its first columns; the next are 64 on
    const uint32_t out0 = smem_u32(pieces) + e * (kSlots + in_slots<op>()) * kPieceBytes;
    const uint32_t in_bar = smem_u32(&sm->in[e]);
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
    // The same of 128 bytes a row, by both slots: chunk j of row r at chunk j ^ (r & 7).
    // Weight gradients, which follow all other pieces of a cluster, leave so: with few
    // rows they are bound by these stores (the gradients of 64 rows of 4096 x 14336 take
    // 161 us, by pieces of 64 bytes a row 168; two such places and a stage less 161).
    auto put_wide = [&](const uint32_t* w, const CUtensorMap* map, int x, int y, bool add) {
      if (lane == 0) bulk_wait_group_read<0>();
      __syncwarp();
      const uint32_t slot = out0;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(slot + lane * 128 +
                                                                     ((j ^ (lane & 7)) << 4)),
                     "r"(w[4 * j]), "r"(w[4 * j + 1]), "r"(w[4 * j + 2]), "r"(w[4 * j + 3])
                     : "memory");
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) {
        if (add) tma_reduce_add_2d(map, slot, x, y);
        else tma_store_2d(map, slot, x, y);
        bulk_commit_group();
      }
    };
    auto put_rounded = [&](const uint32_t* v, const CUtensorMap* map, int x, int y) {
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        w[i] = pack_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
      put(w, map, x, y, false);
    };
    auto get = [&](uint32_t slot, uint32_t* w) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[4 * j]), "=r"(w[4 * j + 1]), "=r"(w[4 * j + 2]), "=r"(w[4 * j + 3])
                     : "r"(slot + my_row + ((j ^ sw) << 4))
                     : "memory");
    };
    // the pieces of 32 columns: two into places of their own, one into the place from
    // which piece k will go out, once the one before it there has been read
    auto in_place = [&](int k) {
      return out0 + (kLoads == 2 ? kSlots : k % kSlots) * kPieceBytes;
    };
    auto ask = [&](int x, int y, int k) {
      if (lane == 0) {
        if (kLoads == 1) bulk_wait_group_read<0>();
        mbar_arrive_expect_tx(in_bar, kLoads * kPieceBytes);
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          tma_load_2d(in_place(k) + i * kPieceBytes, &maps.in[i], in_bar, x, y);
      }
      ++n_asked;
    };
    if (lane == 0) fence_proxy_async();
    int acc = 0;
    uint32_t acc_phase = 0;
    const uint32_t tempty0 = mapa_shared(smem_u32(&sm->tempty[0]), 0);
    bool ok = true;
    // the next accumulator is full: tcgen05.ld is warp-collective, so the whole warp goes on
    // or stops together
    auto wait_full = [&]() {
      const bool got = mbar_wait(smem_u32(&sm->tfull[acc]), acc_phase, p.wait_ns, abort_flag);
      if (!__all_sync(0xffffffffu, got)) {
        sm->abort = 1;
        if (lane == 0) report_error(p.err, kErrTimeout);
        return false;
      }
      tc_fence_after();
      return true;
    };
    // and may be filled again
    auto hand_back = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(tempty0 + acc * static_cast<uint32_t>(sizeof(uint64_t)));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    };
    for (int i = 0; ok; ++i) {
      const Unit u = units.get(i);
      if (u.kind == kNone) break;
      const bool main = op != Op::Joint || u.kind == kMain;
      const Grid& g = main ? p.main : u.kind == kDwDown ? p.down : p.gate;
      const bool part = main && p.split > 1;   // the accumulator leaves as it is
      const bool reads = !part && (kLoads == 2 || (kLoads == 1 && main && p.add != 0));
      const int y = (2 * u.m + static_cast<int>(rank)) * kTileM + q * 32;
      const int width = op == Op::Gated && !part ? BN / 2 : BN;
      const int n0 = u.n * width;
      const int cols = y >= g.M ? 0 : part ? BN : min(width, g.N - n0);   // 0: nothing to finish
      if (kRuns && !main) {
        // one run of k-blocks after another: columns c0 to c0 + 63 and the same 128 on,
        // those past the matrix too
        const int c0 = (e >> 2) * 64;
        float sum[128];
#pragma unroll
        for (int j = 0; j < 128; ++j) sum[j] = 0.0f;
        for (int kb = u.kb0; kb < u.kb1; kb += p.run) {
          ok = wait_full();
          if (!ok) break;
          const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * BN + c0;
#pragma unroll
          for (int j = 0; j < 128; j += 32) {
            uint32_t v[16], w[16];
            tmem_ld_32x32b_x16(taddr + j / 64 * 128 + j % 64, v);
            tmem_ld_32x32b_x16(taddr + j / 64 * 128 + j % 64 + 16, w);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k) sum[j + k] += __uint_as_float(v[k]);
#pragma unroll
            for (int k = 0; k < 16; ++k) sum[j + 16 + k] += __uint_as_float(w[k]);
          }
          hand_back();
        }
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int c = c0 + i * 128;
          uint32_t w[32];
          if (p.f32) {
#pragma unroll
            for (int j = 0; j < 64; j += 32) {
#pragma unroll
              for (int k = 0; k < 32; ++k) w[k] = __float_as_uint(sum[i * 64 + j + k]);
              if (c + j < cols) put_wide(w, &maps.out[u.kind], n0 + c + j, y, p.accumulate != 0);
            }
          } else if (c < cols) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              w[k] = pack_bf16x2(sum[i * 64 + 2 * k], sum[i * 64 + 2 * k + 1]);
            put_wide(w, &maps.out[u.kind], n0 + c, y, p.accumulate != 0);
          }
        }
        continue;
      }
      if (reads && c_first < cols) ask(n0 + c_first, y, npiece);
      if (!wait_full()) break;
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * BN;
      if (op == Op::Joint && !kRuns && !main) {
        const int wide = p.f32 ? 32 : 64;      // columns of a piece
#pragma unroll 1
        for (int c = (e >> 2) * wide; c < cols; c += 2 * wide) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(taddr + c, v);
          if (!p.f32) {
            uint32_t more[32];
            tmem_ld_32x32b_x32(taddr + c + 32, more);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              v[j] = pack_bf16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
              more[j] = pack_bf16x2(__uint_as_float(more[2 * j]), __uint_as_float(more[2 * j + 1]));
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) v[16 + j] = more[j];
          } else {
            tmem_ld_wait();
          }
          put_wide(v, &maps.out[u.kind], n0 + c, y, p.accumulate != 0);
        }
      }
#pragma unroll 1
      for (int c = op == Op::Joint && !kRuns && !main ? cols : c_first; c < cols; c += 64) {
        uint32_t v[32], a[16], b[16];
        if (reads) {
          const bool here = mbar_wait(in_bar, n_got & 1, p.wait_ns, abort_flag);
          if (!__all_sync(0xffffffffu, here)) {
            sm->abort = 1;
            if (lane == 0) report_error(p.err, kErrTimeout);
            ok = false;
            break;
          }
          ++n_got;
          get(in_place(npiece), a);
          if (kLoads == 2) get(in_place(npiece) + kPieceBytes, b);
          __syncwarp();                        // read before the place is filled again
          if (c + 64 < cols) ask(n0 + c + 64, y, npiece + 1);
        }
        tmem_ld_32x32b_x32(taddr + c, v);
        if (part) {
          tmem_ld_wait();
          const int py = y + u.part * p.main.mt * 2 * kTileM;
          put(v, &maps.part, n0 + c, py, false);
          put(v + 16, &maps.part, n0 + c + 16, py, false);
        } else if (op == Op::Gated) {
          uint32_t up[32], w[16];
          tmem_ld_32x32b_x32(taddr + BN / 2 + c, up);
          tmem_ld_wait();
          switch (p.act) {
            case MOE_ACT_SILU: gated_words<MOE_ACT_SILU>(v, up, w); break;
            case MOE_ACT_GELU: gated_words<MOE_ACT_GELU>(v, up, w); break;
            case MOE_ACT_GELU_TANH: gated_words<MOE_ACT_GELU_TANH>(v, up, w); break;
            default: gated_words<MOE_ACT_RELU>(v, up, w); break;
          }
          put(w, &maps.out[0], n0 + c, y, false);
          if (p.keep) {
            put_rounded(v, &maps.out[1], n0 + c, y);
            put_rounded(up, &maps.out[2], n0 + c, y);
          }
        } else if (op == Op::GatedBwd) {
          uint32_t h[16];
          tmem_ld_wait();
          gated_bwd_any<16>(p.act, v, a, b, h);
          put(h, &maps.out[0], n0 + c, y, false);
          put(a, &maps.out[1], n0 + c, y, false);
          put(b, &maps.out[2], n0 + c, y, false);
        } else {
          tmem_ld_wait();
          if (reads)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              v[2 * j] = __float_as_uint(__uint_as_float(v[2 * j]) + lo_f(a[j]));
              v[2 * j + 1] = __float_as_uint(__uint_as_float(v[2 * j + 1]) + hi_f(a[j]));
            }
          put_rounded(v, &maps.out[kMain], n0 + c, y);
        }
      }
      if (!ok) break;
      hand_back();
    }
    // what was asked for lands, and every store has been made, before the CTA exits
    if (n_got != n_asked) mbar_wait(in_bar, n_got & 1, kDrainNs, &sm->zero);
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

// ------------------------------------------------------------------ parts of K added up

struct FinishArgs {
  const float* part;           // [split][mpad][ncols]
  int64_t mpad;
  int ncols, split, N, act;
  int64_t T;
  const __nv_bfloat16 *in0, *in1;     // add, or A_g and A_u
  __nv_bfloat16 *out0, *out1, *out2;  // the epilogue's outputs
};

__device__ __forceinline__ void add_parts(const FinishArgs& p, int64_t at, float* v) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  for (int s = 0; s < p.split; ++s) {
    const float4* q = reinterpret_cast<const float4*>(p.part + s * p.mpad * p.ncols + at);
    const float4 a = __ldcs(q), b = __ldcs(q + 1);
    v[0] += a.x;
    v[1] += a.y;
    v[2] += a.z;
    v[3] += a.w;
    v[4] += b.x;
    v[5] += b.y;
    v[6] += b.z;
    v[7] += b.w;
  }
}

__device__ __forceinline__ uint4 rounded(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

__device__ __forceinline__ float act_any(int act, float z) {
  switch (act) {
    case MOE_ACT_SILU: return act_f<MOE_ACT_SILU>(z);
    case MOE_ACT_GELU: return act_f<MOE_ACT_GELU>(z);
    case MOE_ACT_GELU_TANH: return act_f<MOE_ACT_GELU_TANH>(z);
    default: return act_f<MOE_ACT_RELU>(z);
  }
}

// Eight columns of a row a thread: the parts in their order, then what the epilogue of
// op does with a whole sum (Joint: dx).
template <Op op>
__global__ void __launch_bounds__(256) finish_kernel(const __grid_constant__ FinishArgs p) {
  grid_dependency_wait();
  const int vecs = p.N / 8;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= p.T * vecs) return;
  const int64_t t = i / vecs;
  const int c = static_cast<int>(i - t * vecs) * 8;
  const int64_t to = t * p.N + c;
  float v[8];
  if (op == Op::Gated) {
    float up[8];
    const int64_t at = t * p.ncols + c / (BN / 2) * BN + c % (BN / 2);
    add_parts(p, at, v);
    add_parts(p, at + BN / 2, up);
    if (p.out1) {
      *reinterpret_cast<uint4*>(p.out1 + to) = rounded(v);
      *reinterpret_cast<uint4*>(p.out2 + to) = rounded(up);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = act_any(p.act, v[j]) * up[j];
    *reinterpret_cast<uint4*>(p.out0 + to) = rounded(v);
    return;
  }
  add_parts(p, t * p.ncols + c, v);
  if (op == Op::GatedBwd) {
    const uint4 a = *reinterpret_cast<const uint4*>(p.in0 + to);
    const uint4 b = *reinterpret_cast<const uint4*>(p.in1 + to);
    uint32_t g[4] = {a.x, a.y, a.z, a.w}, u[4] = {b.x, b.y, b.z, b.w}, h[4], dh[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) dh[j] = __float_as_uint(v[j]);
    gated_bwd_any<4>(p.act, dh, g, u, h);
    *reinterpret_cast<uint4*>(p.out0 + to) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(p.out1 + to) = make_uint4(g[0], g[1], g[2], g[3]);
    *reinterpret_cast<uint4*>(p.out2 + to) = make_uint4(u[0], u[1], u[2], u[3]);
    return;
  }
  if (p.in0) {
    const uint4 a = *reinterpret_cast<const uint4*>(p.in0 + to);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] += lo_f(w[j]);
      v[2 * j + 1] += hi_f(w[j]);
    }
  }
  *reinterpret_cast<uint4*>(p.out0 + to) = rounded(v);
}

// ------------------------------------------------------------------ host

int up_div(int64_t a, int b) { return static_cast<int>((a + b - 1) / b); }

Divisor divisor(int64_t d) {
  Divisor v = {static_cast<uint32_t>(d), 0, 0};
  while ((1ull << v.l) < v.d) ++v.l;
  v.m = static_cast<uint32_t>(((1ull << 32) * ((1ull << v.l) - v.d)) / (v.d ? v.d : 1) + 1);
  return v;
}

// Tiles of an [M, N] result whose rows of A are kb k-blocks long. The clusters that run
// at one time take a patch of tiles and move through K together, so that the squarest
// patch reads least (8 row tiles by 9 or 10); where the rows of A of 16 row tiles fit in
// half of L2, they stay there and the columns of B are what the patch has to spare.
// Measured on 4096 x 14336 under the power cap: the gradients of 8192 rows 3740 us, by
// 16 throughout 3784; the forward of 4096 rows 888 us, by 8 throughout 892.
Grid make_grid(int64_t M, int N, int cols, int kb) {
  Grid g;
  const int most = kb < 128 ? 16 : 8;          // 16 times 32 KB a k-block
  g.M = static_cast<int>(M);
  g.N = N;
  g.mt = up_div(M, 2 * kTileM);
  g.nt = up_div(N, cols);
  g.group = g.mt < most ? g.mt : most;
  g.per = divisor(static_cast<int64_t>(g.group) * g.nt);
  g.whole = divisor(g.group);
  g.last = divisor(g.group > 0 ? (g.mt - 1) % g.group + 1 : 0);
  return g;
}

int clusters() { return device_sm_count() > 1 ? device_sm_count() / 2 : 1; }

// Parts of K for a product alone in its launch: as many as the clusters that its tiles
// leave idle, each with 8 k-blocks at least (what a tile's start and end cost). Measured,
// split and not: the forward of 4096 x 14336, 160 rows 80 and 114 us, 512 rows 113 and
// 135, 1024 198 both ways; dh of 2048 x 768 in the gradients of 256 rows, 24 and 33.
int pick_split(const Grid& g, int kb) {
  const int64_t tiles = static_cast<int64_t>(g.mt) * g.nt;
  int s = 1;
  while (s < kMaxSplit && tiles * (s + 1) <= clusters() && kb / (s + 1) >= 8) ++s;
  return s;
}

// Parts of K of dx beside the weight gradients, by what the launch would take in k-blocks
// of a cluster: a tile costs its own and some 8 more; the clusters without a unit of dx
// take gradient tiles meanwhile, as unit_at deals them out, and all of them the rest. The
// kernel that adds the parts up costs about 9, and their way out and in again one for
// three parts. Measured, split and not: 160 rows of 1024 x 8192 50 and 98 us, 1024 rows 96
// and 111, 512 rows of 2048 x 8192 100 and 110; not worth it where the gradients are the
// most of it or a split needs another round, 256 rows of 2048 x 768 27 (in two) and 25,
// 2048 of 512 x 2048 45 (in two) and 40.
constexpr int kTileCost = 8;
int pick_split_joint(const Grid& g, int kb, int64_t dw_units, int kb_rows) {
  if (dw_units == 0) return pick_split(g, kb);
  const int64_t tiles = static_cast<int64_t>(g.mt) * g.nt, all = clusters(), dw = kb_rows + kTileCost;
  int best = 1;
  int64_t least = 0;
  for (int s = 1; s <= kMaxSplit && (s == 1 || (kb / s >= 8 && tiles * s < all)); ++s) {
    const int64_t own = up_div(kb, s) + kTileCost, idle = all - tiles * s;
    int64_t cost;
    if (idle <= 0) {
      cost = (tiles * own + dw_units * dw) / all;
    } else {
      const int64_t left = dw_units - idle * (own / dw), rounds = (dw_units + idle - 1) / idle;
      if (left > 0) cost = own + (left + all - 1) / all * dw;
      else cost = own > rounds * dw ? own : rounds * dw;
    }
    if (s > 1) cost += 9 + tiles * s / 3;
    if (s == 1 || cost < least) {
      best = s;
      least = cost;
    }
  }
  return best;
}

void set_main(Args& p, const Grid& g, int kb0, int kb, int split) {
  p.main = g;
  p.kb0 = kb0;
  p.kb = kb;
  p.split = split;
  p.per = up_div(kb, split);
  p.units = g.mt * g.nt * split;
  p.tiles = divisor(static_cast<int64_t>(g.mt) * g.nt);
}

size_t part_bytes(const Grid& g, int split) {
  return split > 1 ? static_cast<size_t>(split) * g.mt * 2 * kTileM * g.nt * BN * sizeof(float) : 0;
}

bool part_map(CUtensorMap* m, void* base, const Grid& g, int split) {
  if (split <= 1) return true;
  const uint64_t cols = static_cast<uint64_t>(g.nt) * BN;
  return make_out_tmap(m, base, cols, static_cast<uint64_t>(split) * g.mt * 2 * kTileM, cols * 4,
                       true);
}

// beside: beside the launch before it, as far as its waits let it.
template <typename K, typename A, typename... B>
cudaError_t launch_beside(K kern, dim3 grid, int threads, size_t smem, int cluster, cudaStream_t st,
                          const A& a, const B&... b) {
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
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a, b...);
}

template <Op op, bool kRuns = false>
cudaError_t launch(const Maps& maps, Args p, cudaStream_t st) {
  auto kern = dense_gemm_kernel<op, kRuns>;
  static bool configured[kMaxDevices] = {};
  static int max_pairs[kMaxDevices] = {};       // clusters of two that fit at once
  const int d = current_device();
  if (d < 0 || d >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!configured[d]) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem_bytes<op>()));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(2 * kMaxDevices);        // any even size: the query asks how many fit
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes<op>();
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&max_pairs[d], kern, &cfg);
    if (e != cudaSuccess) return e;
    if (max_pairs[d] < 1) return cudaErrorInvalidConfiguration;
    configured[d] = true;
  }
  const int64_t units = static_cast<int64_t>(p.units) + p.dw_units;
  const int n = static_cast<int>(units < max_pairs[d] ? units : max_pairs[d]);
  if (n == 0) return cudaSuccess;
  p.rounds = p.units / n;
  p.rest = p.units % n;
  return launch_beside(kern, dim3(2 * n), kThreads, smem_bytes<op>(), 2, st, maps, p);
}

template <Op op>
cudaError_t finish(const Args& p, const float* part, int64_t T, const void* in0, const void* in1,
                   void* out0, void* out1, void* out2, cudaStream_t st) {
  if (p.split <= 1) return cudaSuccess;
  FinishArgs f;
  f.part = part;
  f.mpad = static_cast<int64_t>(p.main.mt) * 2 * kTileM;
  f.ncols = p.main.nt * BN;
  f.split = p.split;
  f.N = p.main.N;
  f.act = p.act;
  f.T = T;
  f.in0 = static_cast<const __nv_bfloat16*>(in0);
  f.in1 = static_cast<const __nv_bfloat16*>(in1);
  f.out0 = static_cast<__nv_bfloat16*>(out0);
  f.out1 = static_cast<__nv_bfloat16*>(out1);
  f.out2 = static_cast<__nv_bfloat16*>(out2);
  const int64_t ctas = (T * (f.N / 8) + 255) / 256;
  return launch_beside(finish_kernel<op>, dim3(static_cast<unsigned>(ctas)), 256, 0, 1, st, f);
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

// Units stay below 2^30 where the tensors fit in memory at all; refuse the rest.
bool tiles_fit(int64_t M, int N) {
  return static_cast<int64_t>(up_div(M, 2 * kTileM)) * up_div(N, BN / 2) < (1 << 26);
}

// The forward's workspace: h, then the parts of whichever product is being split.
struct FwdPlan {
  Grid gated, down;
  int s_gated, s_down;
  size_t part, total;
};
FwdPlan fwd_plan(int64_t T, int H, int F) {
  FwdPlan f;
  f.gated = make_grid(T, F, BN / 2, up_div(H, BK));
  f.down = make_grid(T, H, BN, up_div(F, BK));
  const bool few = T <= kFewRows;
  f.s_gated = few ? 1 : pick_split(f.gated, up_div(H, BK));
  f.s_down = few ? 1 : pick_split(f.down, up_div(F, BK));
  f.part = up256(static_cast<size_t>(T) * F * 2);
  const size_t a = part_bytes(f.gated, f.s_gated), b = part_bytes(f.down, f.s_down);
  f.total = f.part + up256(a > b ? a : b);
  return f;
}

// The backward's: h, dA_g, dA_u, then the parts.
struct BwdPlan {
  Grid dh, dx, down, gate;
  int s_dh, s_dx, kb_rows;
  int64_t dw_units;
  size_t each, part, total;
};
BwdPlan bwd_plan(int64_t T, int H, int F, bool dw) {
  BwdPlan b;
  b.kb_rows = up_div(T, BK);
  b.dh = make_grid(T, F, BN, up_div(H, BK));
  b.dx = make_grid(T, H, BN, 2 * up_div(F, BK));
  b.down = make_grid(F, H, BN, b.kb_rows);
  b.gate = make_grid(H, F, BN, b.kb_rows);
  b.dw_units = dw ? static_cast<int64_t>(b.down.mt) * b.down.nt +
                        2 * static_cast<int64_t>(b.gate.mt) * b.gate.nt
                  : 0;
  const bool few = T <= kFewRows;
  b.s_dh = few ? 1 : pick_split(b.dh, up_div(H, BK));
  b.s_dx = few ? 1 : pick_split_joint(b.dx, 2 * up_div(F, BK), b.dw_units, b.kb_rows);
  b.each = up256(static_cast<size_t>(T) * F * 2);
  b.part = 3 * b.each;
  const size_t x = part_bytes(b.dh, b.s_dh), y = part_bytes(b.dx, b.s_dx);
  b.total = b.part + up256(x > y ? x : y);
  return b;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_gated_ffn_workspace_size(int64_t T, int H, int F) {
  if (check_sizes(T, H, F, 0) != MOE_OK || !tiles_fit(T, F) || !tiles_fit(T, H)) return 0;
  return fwd_plan(T, H, F).total;
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
  const FwdPlan f = fwd_plan(T, H, F);
  if (!workspace || ws_bytes < f.total || !aligned16(workspace)) return MOE_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T <= kFewRows)
    return ffn_few_rows(x, w_gate, w_up, w_down, add, static_cast<int>(T), H, F, act, y, a_gate,
                        a_up, workspace, device_error_word(), st) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
  float* part = reinterpret_cast<float*>(static_cast<char*>(workspace) + f.part);
  Args p1{};
  p1.act = act;
  p1.err = device_error_word();
  p1.wait_ns = kDefaultWaitNs;
  Args p2 = p1;
  p1.keep = a_gate != nullptr;
  p2.add = add != nullptr;
  set_main(p1, f.gated, up_div(H, BK), up_div(H, BK), f.s_gated);
  set_main(p2, f.down, up_div(F, BK), up_div(F, BK), f.s_down);
  Maps m1{}, m2{};
  const uint64_t rF = static_cast<uint64_t>(F) * 2, rH = static_cast<uint64_t>(H) * 2;
  if (!in_map(&m1.a[0], x, H, T, kTileM) || !in_map(&m1.b[0], w_gate, F, H, BK) ||
      !in_map(&m1.b[1], w_up, F, H, BK) || !make_out_tmap(&m1.out[0], workspace, F, T, rF, false) ||
      (a_gate && (!make_out_tmap(&m1.out[1], a_gate, F, T, rF, false) ||
                  !make_out_tmap(&m1.out[2], a_up, F, T, rF, false))) ||
      !part_map(&m1.part, part, f.gated, f.s_gated) ||
      !in_map(&m2.a[0], workspace, F, T, kTileM) || !in_map(&m2.b[0], w_down, H, F, BK) ||
      !make_out_tmap(&m2.out[0], y, H, T, rH, false) ||
      (add && !make_out_tmap(&m2.in[0], add, H, T, rH, false)) ||
      !part_map(&m2.part, part, f.down, f.s_down))
    return MOE_ERR_CUDA;
  if (launch<Op::Gated>(m1, p1, st) != cudaSuccess ||
      finish<Op::Gated>(p1, part, T, nullptr, nullptr, workspace, a_gate, a_up, st) != cudaSuccess ||
      launch<Op::Down>(m2, p2, st) != cudaSuccess ||
      finish<Op::Down>(p2, part, T, add, nullptr, y, nullptr, nullptr, st) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_OK;
}

size_t moe_gated_ffn_backward_workspace_size(int64_t T, int H, int F) {
  if (check_sizes(T, H, F, 0) != MOE_OK || !tiles_fit(T, F) || !tiles_fit(T, H)) return 0;
  // dx alone is split the more, for want of weight gradients beside it
  const size_t a = bwd_plan(T, H, F, true).total, b = bwd_plan(T, H, F, false).total;
  return a > b ? a : b;
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
  if (!dy || !x || !w_gate || !w_up || !w_down || !a_gate || !a_up || !dx || dx == dy || dx == x)
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(dy) || !aligned16(x) || !aligned16(w_gate) || !aligned16(w_up) ||
      !aligned16(w_down) || !aligned16(a_gate) || !aligned16(a_up) || !aligned16(add) ||
      !aligned16(dx) || !tiles_fit(T, F) || !tiles_fit(T, H) || !tiles_fit(H, F) ||
      !tiles_fit(F, H))
    return MOE_ERR_INVALID_ARG;
  if (!workspace || ws_bytes < moe_gated_ffn_backward_workspace_size(T, H, F) ||
      !aligned16(workspace))
    return MOE_ERR_WORKSPACE;
  const BwdPlan b = bwd_plan(T, H, F, dw_gate != nullptr);
  char* ws = static_cast<char*>(workspace);
  void *h = ws, *da_g = ws + b.each, *da_u = ws + 2 * b.each;
  float* part = reinterpret_cast<float*>(ws + b.part);
  const uint64_t rF = static_cast<uint64_t>(F) * 2, rH = static_cast<uint64_t>(H) * 2;
  Args ph{};
  ph.act = act;
  ph.err = device_error_word();
  ph.wait_ns = kDefaultWaitNs;
  Args pj = ph;
  Maps mh{}, mj{};
  if (T <= kFewRows) {
    if (ffn_few_rows_backward(dy, w_gate, w_up, w_down, a_gate, a_up, add, static_cast<int>(T), H,
                              F, act, dx, h, da_g, da_u, ph.err, st) != cudaSuccess)
      return MOE_ERR_CUDA;
    pj.split = 1;
  } else {
    set_main(ph, b.dh, up_div(H, BK), up_div(H, BK), b.s_dh);
    set_main(pj, b.dx, up_div(F, BK), 2 * up_div(F, BK), b.s_dx);
    pj.add = add != nullptr;
    if (!in_map(&mh.a[0], dy, H, T, kTileM) || !in_map(&mh.b[0], w_down, H, F, 128) ||
        !make_out_tmap(&mh.in[0], a_gate, F, T, rF, false) ||
        !make_out_tmap(&mh.in[1], a_up, F, T, rF, false) ||
        !make_out_tmap(&mh.out[0], h, F, T, rF, false) ||
        !make_out_tmap(&mh.out[1], da_g, F, T, rF, false) ||
        !make_out_tmap(&mh.out[2], da_u, F, T, rF, false) ||
        !part_map(&mh.part, part, b.dh, b.s_dh) ||
        !in_map(&mj.a[0], da_g, F, T, kTileM) || !in_map(&mj.a[1], da_u, F, T, kTileM) ||
        !in_map(&mj.b[0], w_gate, F, H, 128) || !in_map(&mj.b[1], w_up, F, H, 128) ||
        !make_out_tmap(&mj.out[kMain], dx, H, T, rH, false) ||
        (add && !make_out_tmap(&mj.in[0], add, H, T, rH, false)) ||
        !part_map(&mj.part, part, b.dx, b.s_dx))
      return MOE_ERR_CUDA;
    if (launch<Op::GatedBwd>(mh, ph, st) != cudaSuccess ||
        finish<Op::GatedBwd>(ph, part, T, a_gate, a_up, h, da_g, da_u, st) != cudaSuccess)
      return MOE_ERR_CUDA;
  }
  if (dw_gate) {
    const uint64_t z = f32 ? 4 : 2;
    if (!in_map(&mj.a[2], h, F, T, BK) || !in_map(&mj.b[1 + kDwDown], dy, H, T, BK) ||
        !make_out_tmap(&mj.out[kDwDown], dw_down, H, F, static_cast<uint64_t>(H) * z, f32,
                       true) ||
        !in_map(&mj.a[3], x, H, T, BK) || !in_map(&mj.b[1 + kDwGate], da_g, F, T, BK) ||
        !in_map(&mj.b[1 + kDwUp], da_u, F, T, BK) ||
        !make_out_tmap(&mj.out[kDwGate], dw_gate, F, H, static_cast<uint64_t>(F) * z, f32,
                       true) ||
        !make_out_tmap(&mj.out[kDwUp], dw_up, F, H, static_cast<uint64_t>(F) * z, f32, true))
      return MOE_ERR_CUDA;
    pj.down = b.down;
    pj.gate = b.gate;
    pj.dw_units = static_cast<int>(b.dw_units);
    pj.kb_rows = b.kb_rows;
    pj.f32 = f32;
    pj.run = f32 ? kRunF32 : kRunBf16;
    pj.accumulate = accumulate_dw;
    // as many rounds as the gradient tiles that take as long as a unit of dx (the
    // gradients of 300 rows of 4096 x 14336: 253 us, with everyone in every round 304)
    pj.skip = pj.units > 0 ? (pj.per + kTileCost) / (b.kb_rows + kTileCost) : 0;
  }
  const bool runs = dw_gate && b.kb_rows > pj.run;
  if ((runs ? launch<Op::Joint, true>(mj, pj, st) : launch<Op::Joint>(mj, pj, st)) != cudaSuccess ||
      finish<Op::Joint>(pj, part, T, add, nullptr, dx, nullptr, nullptr, st) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_OK;
}

}  // extern "C"
