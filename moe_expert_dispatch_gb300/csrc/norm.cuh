// norm.cuh - what the kernels of the norms around the block share.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace moe {

struct NormParams {
  const void* x;        // forward: the stream; backward: d_out (may be null)
  const void* out;      // backward: the forward's out
  const __nv_bfloat16* y;
  const __nv_bfloat16* d_n;
  const void* w_post;
  const void* gate;
  const void* w_next;
  const float* rstd_y;
  const float* rstd_out;
  int64_t T;
  int64_t gate_span;    // tokens that share a gate row
  int H;
  int weights_f32;
  float eps, a, b;
  float inv_h;
};

// Rows of strip i of n: [i T / n, (i + 1) T / n); the strip of a row.
__host__ __device__ __forceinline__ int64_t strip_row(int64_t T, int n, int64_t i) {
  return i * T / n;
}
__device__ __forceinline__ int64_t strip_of(int64_t T, int n, int64_t row) {
  return ((row + 1) * n - 1) / T;
}

// How a call's rows lie on the ring kernels; groups 0: another length of a row.
struct RingShape {
  int groups, group, stages, ctas, strips, tail_bytes;
};
constexpr int kMaxRingGroups = 15;       // a named barrier each, beside the CTA's own
RingShape ring_shape(int64_t T, int H, int row_bytes, bool backward, bool many);
int most_ring_groups(int H);             // of a CTA of the backward; 0: not on the ring kernels

struct RingOut {
  void* stream;                  // out, or dx
  __nv_bfloat16* branch;         // n, or dy
  float *rstd_y, *rstd_out;      // forward
  float* dgate;                  // backward
  float* part_post;              // [CTAs, H] sum of D yh (of g D yh with more than one gate row)
  float* part_next;              // [CTAs, H] sum of d_n o
  float* part_gate;              // two pieces of [H] for every strip
  int accumulate;
};
cudaError_t launch_norm_ring(const NormParams& p, const RingShape& r, const RingOut& o,
                             bool stream_f32, bool backward, int row_bytes, cudaStream_t st);

__device__ __forceinline__ float weight_at(const void* w, int f32, int64_t i) {
  return f32 ? __ldg(static_cast<const float*>(w) + i)
             : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
}

}  // namespace moe
