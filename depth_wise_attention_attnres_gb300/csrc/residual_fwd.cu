// The gated residual for d a multiple of 8 up to 8192 with aligned rows (the
// formulas stand at the top of residual.cu, the teams in residual_team.cuh).
//
// Bound by memory: each row is read and written once (131072 x 2048 bf16 in 317
// to 324 us by machine, 98 to 100 % of the copy bandwidth). Rows of few bytes are
// bound by a row's fixed work instead: bf16 rows of 384 features run at 53 to 62 %,
// of 5120 at 65 to 69, of 896 without x and normed at 51. A thread holds its 8 or
// 16 features of the row and of the gains. The sum of squares of row r's result
// and that of row r + 1's f go through the team together, so a row costs one
// barrier. With 16 features a thread the teams take rows in turn (131072 x 2048
// takes 9 % less by it than with a run of rows each); with 8 a run each was better
// (104857 x 640: 92 % of the copy bandwidth against 86).
#include "residual_team.cuh"

namespace attnres {
namespace {

__device__ unsigned int g_timeout = 0;

// 28 warps of 72 registers (which spills 4 to 20 bytes), 16 of 128 for 16 features a
// thread, 12 of 168 for 24: with 32 of 64 and 20 of 96 the spills cost more than the
// warps brought (131072 x 2048 took 14 % longer).
constexpr int max_warps(int vectors) { return vectors == 1 ? 28 : vectors == 2 ? 16 : 12; }
// Rows in flight per SM: with all of the 227 KB the reads crowd out the writes,
// the wider ones of an fp32 stream sooner (65536 x 1024 with a gate at 84 % of the
// copy bandwidth, with 146 and 120 KB at 98; without one at 86 with 146, at 96 with
// 120). bf16 rows gain by the deeper ring (32768 x 1024 with a gate 86 against 83).
// A team alone wants a third row (6553 x 5120 fp32 with bf16 gates at 92 % of the copy
// bandwidth, with two 67; only 4096 x 8192 with an fp32 stream and bf16 gates lost by
// it, 83 against 87), and so do single warps of fp32 (131072 x 256: 87 % with
// 168 KB, 77 with 120).
constexpr int kRingF32 = 120 * 1024, kRingBf16 = 146 * 1024, kWarpF32Third = 168 * 1024;

// F: the type of f and normed; X: of x and x_out. GATE kNoGate also takes the
// one gate row of all tokens, which then rides on the gain.
template <typename F, typename X, int GATE, int VPT>
__global__ void __launch_bounds__(max_warps(VPT) * 32, 1)
    residual_fast_kernel(ResidualArgs a, const __grid_constant__ TeamGeom g) {
  extern __shared__ __align__(128) unsigned char smem[];
  init_bars(g, smem);
  Team m = make_team<VPT >= 2 && GATE != kSharedGate>(g, a.T, smem);
  pdl_trigger();
  pdl_wait();
  fill_ring(m, g);
  const int d = a.d, k0 = m.tid * 8, step = m.warps * 256;
  const float inv_d = 1.0f / static_cast<float>(d);
  V8 gain[VPT], gpre[VPT], f[VPT], x[VPT];
  // scale * gamma_post (1 without a post-norm), with a shared gate times its value too.
  auto load_gain = [&](int64_t group) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int k = k0 + v * step;
      gain[v] = fill8(0.f);
      if (k < d) {
        gain[v] = a.gpost ? mul8(ld8(a.gpost + k), a.scale) : fill8(a.scale);
        if (GATE != kTokenGate && a.gate) {
          V8 gate = ld8(a.gate, group * d + k, a.g_bf16), unused;
          activate8<false>(gate, unused, a.sigmoid);
          gain[v] = mul8(gain[v], gate);
        }
      }
    }
  };
  if (GATE != kSharedGate) load_gain(0);
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    gpre[v] = f[v] = fill8(0.f);
    if (k0 + v * step < d && a.gpre) gpre[v] = ld8(a.gpre + k0 + v * step);
  }

  // Waits for a row and takes its part of f and of sum f^2.
  int stage = 0;
  uint32_t parity = 0;
  auto begin_row = [&]() {
    const bool ok = mbar_wait(m.bars + stage * 8, parity);
    float s = 0.f;
    if (ok) {
#pragma unroll
      for (int v = 0; v < VPT; ++v)
        if (k0 + v * step < d) {
          f[v] = ld8(reinterpret_cast<const F*>(m.ring + stage * g.stage_bytes + g.f) + k0 + v * step);
          s += dot8(f[v], f[v]);
        }
    }
    return ok ? s : -1.f;
  };
  float s[2] = {0.f, m.rows == 0 ? 0.f : begin_row()};  // sum x_out^2 of a row, sum f^2 of the next
  bool ok = !(s[1] < 0.f);
  ok = team_sum(m, s, 1, ok);
  if (!ok) give_up(m, g, 0, &g_timeout);
  // Runs of tokens with one gate row (without such rows: the one run).
  for (int r = 0; ok && r < m.rows;) {
    int run_end = m.rows;
    if (GATE == kSharedGate) {
      const int64_t group = (m.r0 + r) / a.gate_rows;
      const int64_t end = (group + 1) * a.gate_rows - m.r0;
      if (end < run_end) run_end = static_cast<int>(end);
      load_gain(group);
    }
    for (; r < run_end; ++r) {
      const int64_t row = (m.r0 + static_cast<int64_t>(r) * m.stride) * d;
      const unsigned char* st = m.ring + stage * g.stage_bytes;
      const float rf = a.gpost ? rsqrtf(s[1] * inv_d + a.eps_post) : 1.f;
      s[0] = s[1] = 0.f;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int k = k0 + v * step;
        if (k < d) {
          x[v] = a.x ? ld8(reinterpret_cast<const X*>(st + g.x) + k) : fill8(0.f);
          V8 w = mul8(gain[v], rf);
          if (GATE == kTokenGate) {
            V8 gate = ld8(st + g.gate, k, a.g_bf16), unused;
            activate8<false>(gate, unused, a.sigmoid);
            w = mul8(w, gate);
          }
          x[v] = fma8(w, f[v], x[v]);
          out8(static_cast<X*>(a.x_out) + row + k, x[v]);
          s[0] += dot8(x[v], x[v]);
        }
      }
      if (++stage == m.nst) stage = 0, parity ^= 1u;
      if (r + 1 < m.rows) s[1] = begin_row();
      ok = !(s[1] < 0.f);
      ok = team_sum(m, s, r & 1, ok);
      if (!ok) {
        give_up(m, g, r + 1, &g_timeout);
        break;
      }
      // Every thread has what it needs of row r: its stage is free.
      if (m.tid == 0 && m.issued < m.rows) issue_row(m, g);
      if (a.normed) {
        const float rx = rsqrtf(s[0] * inv_d + a.eps_pre);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
          const int k = k0 + v * step;
          if (k < d) out8(static_cast<F*>(a.normed) + row + k, mul8(mul8(gpre[v], rx), x[v]));
        }
      }
    }
  }
}

// Rows that three warps of 8 features a thread would leave partly idle go to one
// warp with 24: no barrier, and no lanes without work (104857 x 640 bf16 at 94 %
// of the copy bandwidth, with three warps 71; at d = 768 three were better).
TeamShape shape_of(int64_t T, int d) {
  const int v = d > 512 && d <= 704 ? 3 : (d > 256 * max_warps(1) || (d > 512 && sixteen_pay(d)) ? 2 : 1);
  return team_shape(T, d, v, max_warps(v));
}

bool geom_of(const ResidualArgs& a, TeamGeom* g) {
  *g = TeamGeom{};
  const int es = a.f_bf16 ? 2 : 4, xs = a.x_bf16 ? 2 : 4;
  add_input(*g, a.f, a.d * es, &g->f);
  add_input(*g, a.x, a.d * xs, &g->x);
  add_input(*g, a.gate && a.gate_rows == 1 ? a.gate : nullptr, a.d * (a.g_bf16 ? 2 : 4), &g->gate);
  const TeamShape s = shape_of(a.T, a.d);
  const int third = s.warps == 1 && !a.f_bf16 ? kWarpF32Third : s.teams == 1 ? kTeamSmem : 0;
  return finish_geom(*g, s, 0, 2, a.x_bf16 ? kRingBf16 : kRingF32, third);
}

template <typename F, typename X, int VPT>
cudaError_t launch_typed(const ResidualArgs& a, const TeamGeom& g, int64_t ctas, cudaStream_t s) {
  if (!a.gate || (a.gate_rows >= a.T && a.gate_rows > 1))
    return launch_teams(residual_fast_kernel<F, X, kNoGate, VPT>, g, ctas, s, a, g);
  if (a.gate_rows == 1) return launch_teams(residual_fast_kernel<F, X, kTokenGate, VPT>, g, ctas, s, a, g);
  return launch_teams(residual_fast_kernel<F, X, kSharedGate, VPT>, g, ctas, s, a, g);
}

template <int VPT>
cudaError_t launch_vectors(const ResidualArgs& a, const TeamGeom& g, int64_t ctas, cudaStream_t s) {
  if (!a.f_bf16) return launch_typed<float, float, VPT>(a, g, ctas, s);
  return a.x_bf16 ? launch_typed<bf16, bf16, VPT>(a, g, ctas, s) : launch_typed<bf16, float, VPT>(a, g, ctas, s);
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
  const TeamShape t = shape_of(a.T, a.d);
  const int64_t ctas = team_ctas(a.T, t, cta_cap());
  return t.vectors == 1 ? launch_vectors<1>(a, g, ctas, s)
                        : (t.vectors == 2 ? launch_vectors<2>(a, g, ctas, s) : launch_vectors<3>(a, g, ctas, s));
}

cudaError_t take_timeout_residual_fwd(unsigned int* flag) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(flag, g_timeout, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_timeout, &zero, sizeof(unsigned int));
}

}  // namespace attnres
