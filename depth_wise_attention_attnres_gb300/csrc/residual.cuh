// What the files of the gated residual share.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace attnres {

// sigmoid(g) and its slope from e = exp(-|g|), which neither overflows nor
// loses the small factor of the slope e / (1 + e)^2 to cancellation. e is the
// square of 2^(t/2), so that it may be subnormal where 2^(t/2) is not; t =
// -|g| log2(e) is taken in two parts, as Cody and Waite reduce arguments, and
// the power of the second one to first order. e^-110 is 0 in fp32. With 2^t and
// the reciprocal within 3 and 2 x 2^-24 both results are within 20 x 2^-24,
// relative (e: 2 x (3 + 2) and its product; the rest: two roundings each).
__device__ __forceinline__ float sigmoid(float g, float* slope) {
  float m = fabsf(g);
  m = m > 110.f ? 110.f : m;  // a NaN stays
  const float t = m * -0.72134752f;                      // -log2(e) / 2
  const float rest = fmaf(m, -0.72134752f, -t) - m * 9.62981e-9f;  // and what fp32 leaves of it
  float y, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(t));
  y = fmaf(y, rest * 0.69314718f, y);
  const float e = y * y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  const float er = e * r;
  *slope = er * r;
  return g < 0.f ? er : r;
}

// Whether runs of tokens, but not all of them, share gate rows whose gradient
// is wanted; and whether all tokens share one.
inline bool residual_bwd_shares_gates(const ResidualBwdArgs& a) {
  return a.dgate && a.gate_rows > 1 && a.gate_rows < a.T;
}
inline bool residual_bwd_sums_gate(const ResidualBwdArgs& a) {
  return a.dgate && a.gate_rows > 1 && a.gate_rows >= a.T;
}

// How the gate rows whose tokens several teams had are summed from the teams'
// parts ([teams][2][d]: of a row that began before the team's tokens, and of one
// that goes on after them): a block for each gate row and 32 features, or a
// block for each team's first row and 1024 features.
struct ResidualJoin {
  const float* part = nullptr;
  int64_t teams = 0, blocks = 0;
  int by_group = 0;
};

// residual_fwd.cu, residual_bwd.cu
bool residual_fast_ok(const ResidualArgs& a);
bool residual_bwd_fast_ok(const ResidualBwdArgs& a);
int64_t residual_bwd_fast_scratch(int64_t T, int d, int64_t gate_rows);
int residual_bwd_parts(const ResidualBwdArgs& a);
cudaError_t launch_residual_fast(const ResidualArgs& a, cudaStream_t s);
cudaError_t launch_residual_bwd_fast(const ResidualBwdArgs& a, cudaStream_t s);
ResidualJoin residual_bwd_join(const ResidualBwdArgs& a);

}  // namespace attnres
