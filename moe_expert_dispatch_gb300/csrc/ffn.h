// ffn.h - what the two forms of the gated feed-forward block share: tiles of 256
// rows (ffn.cu) and the few rows of a decoding step (ffn_rows.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

// Rows up to which the block takes the form of ffn_rows.cu. Measured by that form and by
// tiles of 256 rows: the forward of 4096 x 14336, 16 rows 59 and 86 us, 64 rows 64 and 83,
// 128 rows 80 both ways; its gradients, 64 rows 168 and 188, 128 rows 197 both ways; the
// forward of 2048 x 768, 16 rows 11 and 24, 128 rows 22 both ways. Past 128 rows the tiles
// win (their N here would be two MMAs' worth).
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
