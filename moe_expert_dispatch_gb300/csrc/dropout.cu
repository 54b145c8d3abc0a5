// dropout.cu - moe_dropout_residual and its backward: dropout of a branch with
// a mask that is never stored, and the scaled residual that it joins.
//
// The mask comes from Philox 4x32 with ten rounds (Salmon, Moraes, Dror, Shaw:
// "Parallel random numbers: as easy as 1, 2, 3", 2011): a bijection of a 128-bit
// counter under a 64-bit key, so that element i's number is a function of (seed,
// draw, i) alone and the backward makes it again. A block of 128 bits serves
// eight elements with 16 bits each; the probability is then a multiple of 2^-16,
// and the factor of what is kept is that of the multiple, which keeps the
// expectation exact. 32 bits an element would take twice the rounds.
//
// A thread owns a block: one 16-byte load (two for float) of each input, ten
// rounds of two 32 x 32 -> 64 bit products, and the stores. Seed and draw are
// read by the kernel, so that a replayed graph takes the draw of its replay.
// Bound by memory: 117 M elements of a bf16 branch into a float stream move 1.17
// GB in 165 us, 7.1 TB/s, as fast as a copy.
#include <math.h>
#include <string.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kThreads = 256;

struct DropArgs {
  int64_t numel;
  const int64_t* rng;
  uint32_t threshold;      // of the upper half of a word: t << 16
  float a, f;
};

struct Key { uint32_t lo, hi; };

__device__ __forceinline__ uint4 philox(uint64_t block, uint64_t draw, Key k) {
  uint32_t c0 = static_cast<uint32_t>(block), c1 = static_cast<uint32_t>(block >> 32);
  uint32_t c2 = static_cast<uint32_t>(draw), c3 = static_cast<uint32_t>(draw >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p = static_cast<uint64_t>(c0) * 0xD2511F53u;
    const uint64_t q = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(q >> 32) ^ c1 ^ (k.lo + i * 0x9E3779B9u);
    c1 = static_cast<uint32_t>(q);
    c2 = static_cast<uint32_t>(p >> 32) ^ c3 ^ (k.hi + i * 0xBB67AE85u);
    c3 = static_cast<uint32_t>(p);
  }
  return make_uint4(c0, c1, c2, c3);
}

// Eight elements, as they lie: 16 bytes of bf16, 32 of float.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    v = __ldcs(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void put(__nv_bfloat16* p, const float* f) {
    __stcs(reinterpret_cast<uint4*>(p),
           make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7])));
  }
};
template <>
struct Eight<float> {
  float4 v[2];
  __device__ __forceinline__ void load(const float* p) {
    v[0] = __ldcs(reinterpret_cast<const float4*>(p));
    v[1] = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[4 * i] = v[i].x;
      f[4 * i + 1] = v[i].y;
      f[4 * i + 2] = v[i].z;
      f[4 * i + 3] = v[i].w;
    }
  }
  static __device__ __forceinline__ void put(float* p, const float* f) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
  }
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float* p, float v) { *p = v; }
__device__ __forceinline__ void from_f(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Whether element j of a block is kept: the low or the high half of word j / 2.
__device__ __forceinline__ bool kept(const uint32_t* w, int j, uint32_t t) {
  return ((j & 1) ? w[j >> 1] : (w[j >> 1] << 16)) >= t;
}

// Forward: in = y, res = x (or none), out. Backward: in = d_out, out = dy, and dx
// with kDx. kWide: whole blocks go 16 bytes at a time.
template <typename TIn, typename TOut, bool kRes, bool kDx, bool kWide>
__global__ void __launch_bounds__(kThreads)
    dropout_kernel(const TIn* in, const TOut* res, TOut* out, TIn* dx, DropArgs p) {
  const int64_t blocks = (p.numel + 7) >> 3;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  const uint64_t seed = static_cast<uint64_t>(__ldg(p.rng));
  const uint64_t draw = static_cast<uint64_t>(__ldg(p.rng + 1));
  const Key key = {static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32)};
  for (int64_t b = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; b < blocks;
       b += step) {
    const int64_t at = b * 8;
    if (kWide && at + 8 <= p.numel) {
      Eight<TIn> e;
      Eight<TOut> r;
      e.load(in + at);
      if (kRes) r.load(res + at);
      const uint4 u = philox(b, draw, key);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
      float v[8], x[8], o[8];
      e.get(v);
      if (kRes) r.get(x);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float base = kRes ? p.a * x[j] : 0.0f;
        o[j] = kept(w, j, p.threshold) ? fmaf(p.f, v[j], base) : base;
      }
      Eight<TOut>::put(out + at, o);
      if (kDx) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= p.a;
        Eight<TIn>::put(dx + at, v);
      }
    } else {
      const uint4 u = philox(b, draw, key);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t i = at + j;
        if (i >= p.numel) break;
        const float v = to_f(in[i]), base = kRes ? p.a * to_f(res[i]) : 0.0f;
        from_f(out + i, kept(w, j, p.threshold) ? fmaf(p.f, v, base) : base);
        if (kDx) from_f(dx + i, p.a * v);
      }
    }
  }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <typename TIn, typename TOut, bool kRes, bool kDx>
cudaError_t launch_typed(const void* in, const void* res, void* out, void* dx, const DropArgs& p,
                         cudaStream_t st) {
  // 16 bytes at a time: 16.8 M elements of bf16 take 12.4 us so, one by one 48
  const bool wide = aligned(in, 16) && aligned(res, 16) && aligned(out, 16) && aligned(dx, 16);
  const int64_t ctas = ((p.numel + 7) / 8 + kThreads - 1) / kThreads;
  // One wave of CTAs that step through the tensor spares the others their start (seed and
  // draw are loads of their own); past some eight waves a CTA for every 256 blocks is
  // faster, as no SM has to wait for the slowest. 16.8 M elements of bf16: 12.4 us by one
  // wave, 14.3 by all; 117 M of a float stream: 192 and 165.
  const int64_t wave = static_cast<int64_t>(device_sm_count()) * 8;
  const unsigned grid = static_cast<unsigned>(ctas <= wave || ctas > 8 * wave ? ctas : wave);
  const TIn* i = static_cast<const TIn*>(in);
  const TOut* r = static_cast<const TOut*>(res);
  if (wide)
    dropout_kernel<TIn, TOut, kRes, kDx, true><<<grid, kThreads, 0, st>>>(
        i, r, static_cast<TOut*>(out), static_cast<TIn*>(dx), p);
  else
    dropout_kernel<TIn, TOut, kRes, kDx, false><<<grid, kThreads, 0, st>>>(
        i, r, static_cast<TOut*>(out), static_cast<TIn*>(dx), p);
  return cudaGetLastError();
}

template <bool kRes, bool kDx>
cudaError_t launch(int in_type, int out_type, const void* in, const void* res, void* out, void* dx,
                   const DropArgs& p, cudaStream_t st) {
  if (in_type == MOE_TYPE_F32)
    return out_type == MOE_TYPE_F32
               ? launch_typed<float, float, kRes, kDx>(in, res, out, dx, p, st)
               : launch_typed<float, __nv_bfloat16, kRes, kDx>(in, res, out, dx, p, st);
  return out_type == MOE_TYPE_F32
             ? launch_typed<__nv_bfloat16, float, kRes, kDx>(in, res, out, dx, p, st)
             : launch_typed<__nv_bfloat16, __nv_bfloat16, kRes, kDx>(in, res, out, dx, p, st);
}

bool is_type(int t) { return t == MOE_TYPE_F32 || t == MOE_TYPE_BF16; }
uintptr_t width(int t) { return t == MOE_TYPE_F32 ? 4 : 2; }

// The checks that both directions share, and the kernel's scalars.
moe_status prepare(int64_t numel, const int64_t* rng, const moe_dropout_config& c, DropArgs& p) {
  if (numel < 0 || numel >= (static_cast<int64_t>(1) << 40) || !(c.p >= 0.0f && c.p < 1.0f) ||
      !isfinite(c.residual_scale) || !isfinite(c.branch_scale) || !is_type(c.stream_type) ||
      !is_type(c.branch_type))
    return MOE_ERR_INVALID_ARG;
  if (numel > 0 && (!rng || !aligned(rng, 8))) return MOE_ERR_INVALID_ARG;
  const double t = fmin(65535.0, rint(static_cast<double>(c.p) * 65536.0));
  p.numel = numel;
  p.rng = rng;
  p.threshold = static_cast<uint32_t>(t) << 16;
  p.a = c.residual_scale;
  p.f = static_cast<float>(c.branch_scale / (1.0 - t / 65536.0));
  return isfinite(p.f) ? MOE_OK : MOE_ERR_INVALID_ARG;   // inf * 0 where y is 0
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

void moe_dropout_config_init(moe_dropout_config* cfg) {
  if (!cfg) return;
  memset(cfg, 0, sizeof(*cfg));
  cfg->p = 0.1f;
  cfg->residual_scale = 1.0f;
  cfg->branch_scale = 1.0f;
  cfg->stream_type = MOE_TYPE_BF16;
  cfg->branch_type = MOE_TYPE_BF16;
}

moe_status moe_dropout_residual(const void* y, const void* x, int64_t numel, const int64_t* rng,
                                const moe_dropout_config* cfg, void* out, void* stream) {
  MOE_ENTRY_RANGE();
  moe_dropout_config c;
  moe_dropout_config_init(&c);
  if (cfg) c = *cfg;
  DropArgs p;
  const moe_status s = prepare(numel, rng, c, p);
  if (s != MOE_OK || numel == 0) return s;
  if (!y || !out || !aligned(y, width(c.branch_type)) || !aligned(x, width(c.stream_type)) ||
      !aligned(out, width(c.stream_type)) || (out == y && c.stream_type != c.branch_type))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      x ? launch<true, false>(c.branch_type, c.stream_type, y, x, out, nullptr, p, st)
        : launch<false, false>(c.branch_type, c.stream_type, y, nullptr, out, nullptr, p, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_dropout_residual_backward(const void* d_out, int64_t numel, const int64_t* rng,
                                         const moe_dropout_config* cfg, void* dx, void* dy,
                                         void* stream) {
  MOE_ENTRY_RANGE();
  moe_dropout_config c;
  moe_dropout_config_init(&c);
  if (cfg) c = *cfg;
  DropArgs p;
  const moe_status s = prepare(numel, rng, c, p);
  if (s != MOE_OK || numel == 0) return s;
  if (!d_out || !dy || !aligned(d_out, width(c.stream_type)) || !aligned(dx, width(c.stream_type)) ||
      !aligned(dy, width(c.branch_type)) || dy == dx ||
      (dy == d_out && (dx || c.stream_type != c.branch_type)))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      dx ? launch<false, true>(c.stream_type, c.branch_type, d_out, nullptr, dy, dx, p, st)
         : launch<false, false>(c.stream_type, c.branch_type, d_out, nullptr, dy, nullptr, p, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
