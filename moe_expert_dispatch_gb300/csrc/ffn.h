// ffn.h - what the two forms of the gated feed-forward block share: tiles of 256
// rows (ffn.cu) and the few rows of a decoding step (ffn_rows.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

// Rows up to which the block takes the form of ffn_rows.cu. Measured by that form and by
// tiles of 256 rows: the forward of 4096 x 14336, 16 rows 60 and 87 us, 64 rows 65 and 84,
// 128 rows 80 and 81; its gradients, 64 rows 162 and 180, 128 rows 187 and 200; the forward
// of 2048 x 768, 16 rows 11 and 21, 128 rows 18 and 20. So by 128 rows the wide layer's
// forward takes as long both ways. The MMA's N would allow 256 rows; the ring, three stages
// at 128 rows, would have two from 176 on, and the sums that take its place at the end
// (512 bytes a row) would not fit it past 216.
constexpr int kFewRows = 128;

// h [T, F] and, where a_gate is given, A_g and A_u; then y = bf16(add + h W_down).
// T from 1 to kFewRows, the rest as moe_gated_ffn.
cudaError_t ffn_few_rows(const void* x, const void* w_gate, const void* w_up, const void* w_down,
                         const void* add, int T, int H, int F, int act, void* y, void* a_gate,
                         void* a_up, void* h, int* err, cudaStream_t st);

// h, dA_g and dA_u [T, F], then dx = bf16(add + dA_g W_gate^T + dA_u W_up^T).
cudaError_t ffn_few_rows_backward(const void* dy, const void* w_gate, const void* w_up,
                                  const void* w_down, const void* a_gate, const void* a_up,
                                  const void* add, int T, int H, int F, int act, void* dx, void* h,
                                  void* da_gate, void* da_up, int* err, cudaStream_t st);

}  // namespace moe
