// What the files of the gated residual share.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace attnres {

// sigmoid(g) and its slope, of two values, from e = exp(-|g|), which neither
// overflows nor loses the small factor of the slope e / (1 + e)^2 to cancellation.
// e is the square of 2^(t/2), so that it may be subnormal where 2^(t/2) is not; t =
// -|g| log2(e) is taken in two parts, as Cody and Waite reduce arguments, and
// the power of the second one to first order. e^-110 is 0 in fp32. With 2^t and
// the reciprocal within 3 and 2 x 2^-24 both results are within 20 x 2^-24,
// relative (e: 2 x (3 + 2) and its product; the rest: two roundings each).
__device__ __forceinline__ float2 sigmoid2(float2 g, float2* slope) {
  float2 m, y, r;
  asm("min.NaN.f32 %0, %1, 0f42DC0000;" : "=f"(m.x) : "f"(fabsf(g.x)));  // 110; a NaN stays
  asm("min.NaN.f32 %0, %1, 0f42DC0000;" : "=f"(m.y) : "f"(fabsf(g.y)));
  const float2 h = fmul2(m, make_float2(0.72134752f, 0.72134752f));  // log2(e) / 2
  // What fp32 leaves of -m log2(e) / 2 when -h is taken.
  float2 rest = ffma2(m, make_float2(-0.72134752f, -0.72134752f), h);
  rest = ffma2(m, make_float2(-9.62981e-9f, -9.62981e-9f), rest);
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(-h.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(-h.y));
  y = ffma2(y, fmul2(rest, make_float2(0.69314718f, 0.69314718f)), y);
  const float2 e = fmul2(y, y), d = ffma2(y, y, make_float2(1.f, 1.f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
  const float2 er = fmul2(e, r);
  *slope = fmul2(er, r);
  return make_float2(g.x < 0.f ? er.x : r.x, g.y < 0.f ? er.y : r.y);
}
__device__ __forceinline__ float sigmoid(float g, float* slope) {
  float2 s;
  const float2 a = sigmoid2(make_float2(g, 0.f), &s);
  *slope = s.x;
  return a.x;
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
