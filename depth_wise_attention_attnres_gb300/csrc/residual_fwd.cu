// The gated residual for d a multiple of 8 up to 8192 with aligned rows (the
// formulas stand at the top of residual.cu, the teams in residual_team.cuh).
//
// Bound by memory: each row is read and written once. A thread holds 8 features
// of the row and of the gains. The sum of squares of row r's result and that of
// row r + 1's f go through the team together, so a row costs one barrier.
#include "residual_team.cuh"

namespace attnres {
namespace {

__device__ unsigned int g_timeout = 0;

constexpr int kMaxWarps = 32;

// F: the type of f and normed; X: of x and x_out.
template <typename F, typename X, int GATE>
__global__ void __launch_bounds__(kMaxWarps * 32, 1)
    residual_fast_kernel(ResidualArgs a, const __grid_constant__ TeamGeom g) {
  extern __shared__ __align__(128) unsigned char smem[];
  init_bars(g, smem);
  Team m = make_team(g, a.T, smem);
  pdl_trigger();
  pdl_wait();
  fill_ring(m, g);
  const int d = a.d, k = m.tid * 8;
  const bool mine = k < d;
  const float inv_d = 1.0f / static_cast<float>(d);
  // Without a post-norm its gain is 1; scale rides on it.
  V8 gpost = fill8(a.scale), gpre = fill8(0.f);
  if (mine && a.gpost) gpost = mul8(ld8(a.gpost + k), a.scale);
  if (mine && a.gpre) gpre = ld8(a.gpre + k);
  // The shared gate row of the current token, and the first token of the next one.
  int64_t group = 0, group_end = a.T;
  V8 gate = fill8(1.f), unused;
  if (GATE == kSharedGate) {
    group = m.r0 / a.gate_rows;
    if (a.gate_rows < a.T) group_end = (group + 1) * a.gate_rows;
    if (mine && m.rows > 0) {
      gate = ld8(a.gate, group * d + k, a.g_bf16);
      activate8<false>(gate, unused, a.sigmoid);
    }
  }

  // Waits for row r and takes its part of sum f^2.
  int stage = 0;
  uint32_t parity = 0;
  auto begin_row = [&](float* sum) {
    const bool ok = mbar_wait(m.bars + stage * 8, parity);
    if (ok && mine && a.gpost) {
      const V8 f = ld8(reinterpret_cast<const F*>(m.ring + stage * g.stage_bytes + g.f) + k);
      *sum = dot8(f, f);
    }
    return ok;
  };
  float s[2] = {0.f, 0.f};  // sum x_out^2 of a row, sum f^2 of the next
  bool ok = m.rows == 0 || begin_row(&s[1]);
  ok = team_sum(m, s, 1, ok);
  if (!ok) give_up(m, g, 0, &g_timeout);
  for (int r = 0; ok && r < m.rows; ++r) {
    const int64_t row = m.r0 + r;
    if (GATE == kSharedGate && row == group_end) {
      ++group;
      group_end += a.gate_rows;
      if (mine) {
        gate = ld8(a.gate, group * d + k, a.g_bf16);
        activate8<false>(gate, unused, a.sigmoid);
      }
    }
    const unsigned char* st = m.ring + stage * g.stage_bytes;
    V8 x = fill8(0.f);
    const float rf = a.gpost ? rsqrtf(s[1] * inv_d + a.eps_post) : 1.f;
    s[0] = s[1] = 0.f;
    if (mine) {
      const V8 f = ld8(reinterpret_cast<const F*>(st + g.f) + k);
      if (a.x) x = ld8(reinterpret_cast<const X*>(st + g.x) + k);
      V8 w = mul8(gpost, rf);
      if (GATE == kTokenGate) {
        gate = ld8(st + g.gate, k, a.g_bf16);
        activate8<false>(gate, unused, a.sigmoid);
      }
      if (GATE != kNoGate) w = mul8(w, gate);
      x = fma8(w, f, x);
      st8(static_cast<X*>(a.x_out) + row * d + k, x);
      s[0] = dot8(x, x);
    }
    if (++stage == m.nst) stage = 0, parity ^= 1u;
    if (r + 1 < m.rows) ok = begin_row(&s[1]);
    ok = team_sum(m, s, r & 1, ok);
    if (!ok) {
      give_up(m, g, r + 1, &g_timeout);
      break;
    }
    // Every thread has what it needs of row r: its stage is free.
    if (m.tid == 0 && m.issued < m.rows) issue_row(m, g);
    if (a.normed && mine)
      st8(static_cast<F*>(a.normed) + row * d + k, mul8(mul8(gpre, rsqrtf(s[0] * inv_d + a.eps_pre)), x));
  }
}

bool geom_of(const ResidualArgs& a, TeamGeom* g) {
  *g = TeamGeom{};
  const int es = a.f_bf16 ? 2 : 4, xs = a.x_bf16 ? 2 : 4;
  add_input(*g, a.f, a.d * es, &g->f);
  add_input(*g, a.x, a.d * xs, &g->x);
  add_input(*g, a.gate && a.gate_rows == 1 ? a.gate : nullptr, a.d * (a.g_bf16 ? 2 : 4), &g->gate);
  return finish_geom(*g, team_shape(a.d, kMaxWarps), 0, 2);
}

template <typename F, typename X>
cudaError_t launch_typed(const ResidualArgs& a, const TeamGeom& g, int64_t ctas, cudaStream_t s) {
  if (!a.gate) return launch_teams(residual_fast_kernel<F, X, kNoGate>, g, ctas, s, a, g);
  if (a.gate_rows == 1) return launch_teams(residual_fast_kernel<F, X, kTokenGate>, g, ctas, s, a, g);
  return launch_teams(residual_fast_kernel<F, X, kSharedGate>, g, ctas, s, a, g);
}

}  // namespace

bool residual_fast_ok(const ResidualArgs& a) {
  TeamGeom g;
  return a.T > 0 && a.d % 8 == 0 && a.d <= kMaxTeamD && aligned16(a.f) && aligned16(a.x) && aligned16(a.gate) &&
         aligned16(a.gpost) && aligned16(a.gpre) && aligned16(a.x_out) && aligned16(a.normed) && geom_of(a, &g);
}

cudaError_t launch_residual_fast(const ResidualArgs& a, cudaStream_t s) {
  TeamGeom g;
  if (!geom_of(a, &g)) return cudaErrorInvalidValue;
  const int64_t ctas = team_ctas(a.T, team_shape(a.d, kMaxWarps), cta_cap());
  if (!a.f_bf16) return launch_typed<float, float>(a, g, ctas, s);
  return a.x_bf16 ? launch_typed<bf16, bf16>(a, g, ctas, s) : launch_typed<bf16, float>(a, g, ctas, s);
}

cudaError_t take_timeout_residual_fwd(unsigned int* flag) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(flag, g_timeout, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_timeout, &zero, sizeof(unsigned int));
}

}  // namespace attnres
