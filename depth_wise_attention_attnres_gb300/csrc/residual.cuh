// What the two files of the gated residual share.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace attnres {

// sigmoid(g) and its slope from e = exp(-|g|), which neither overflows nor
// loses the small factor of the slope e / (1 + e)^2 to cancellation.
__device__ __forceinline__ float sigmoid(float g, float* slope) {
  const float e = expf(-fabsf(g)), r = 1.0f / (1.0f + e);
  *slope = e * r * r;
  return g < 0.f ? e * r : r;
}

// Whether runs of tokens, but not all of them, share gate rows whose gradient
// is wanted; and whether all tokens share one.
inline bool residual_bwd_shares_gates(const ResidualBwdArgs& a) {
  return a.dgate && a.gate_rows > 1 && a.gate_rows < a.T;
}
inline bool residual_bwd_sums_gate(const ResidualBwdArgs& a) {
  return a.dgate && a.gate_rows > 1 && a.gate_rows >= a.T;
}

// residual_fast.cu
bool residual_fast_ok(const ResidualArgs& a);
bool residual_bwd_fast_ok(const ResidualBwdArgs& a);
int64_t residual_bwd_fast_scratch(int64_t T, int d, int64_t gate_rows);
int residual_bwd_parts(const ResidualBwdArgs& a);
cudaError_t launch_residual_fast(const ResidualArgs& a, cudaStream_t s);
cudaError_t launch_residual_bwd_fast(const ResidualBwdArgs& a, cudaStream_t s);
cudaError_t launch_residual_bwd_join_gate(const ResidualBwdArgs& a, cudaStream_t s);

}  // namespace attnres
