// ffn.h - what the two forms of the gated feed-forward block share: tiles of 256
// rows (ffn.cu) and the few rows of a decoding step (ffn_rows.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

// Rows up to which the block's forward takes the form of ffn_rows.cu.
constexpr int kFewRows = 128;

// h [T, F] and, where a_gate is given, A_g and A_u; then y = bf16(add + h W_down).
// T from 1 to kFewRows, the rest as moe_gated_ffn.
cudaError_t ffn_few_rows(const void* x, const void* w_gate, const void* w_up, const void* w_down,
                         const void* add, int T, int H, int F, int act, void* y, void* a_gate,
                         void* a_up, void* h, int* err, cudaStream_t st);

}  // namespace moe
