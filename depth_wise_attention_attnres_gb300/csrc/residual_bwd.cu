// Backward of the gated residual, and of RMSNorm, for d a multiple of 8 up to
// 8192 with aligned rows (the formulas stand at the top of residual.cu, the
// teams in residual_team.cuh).
//
// Bound by memory: each row is read and written once. The sums over tokens stay
// in registers for the whole run of rows (a thread's features never change),
// are added over the CTA's teams in shared memory and leave one partial row per
// CTA; a gate row that some tokens share is written by the team that has all of
// them, or left in two parts per team for one more kernel. The sums of row r's
// second mean and of row r + 1's first ones go through the team together, so a
// row costs one barrier.
#include "residual_team.cuh"

namespace attnres {
namespace {

__device__ unsigned int g_timeout = 0;

// 20 warps of 96 registers, 32 of 64; past d = 5120 the gated kernel's threads
// take 16 features and 128 registers (a row is then 11 to 16 warps).
constexpr int kNormWarps = 32, kGatedWarps = 20, kWideWarps = 16;
int max_warps(const ResidualBwdArgs& a) { return a.f ? kGatedWarps : kNormWarps; }

// 8 features of a gate row that tokens share: act(gate), and its slope.
__device__ __forceinline__ V8 shared_act(const ResidualBwdArgs& a, int64_t group, int k, V8& slope) {
  V8 gate = ld8(a.gate, group * a.d + k, a.g_bf16);
  activate8<true>(gate, slope, a.sigmoid);
  return gate;
}
// scale * gamma_post (1 without a post-norm).
__device__ __forceinline__ V8 scaled_gain(const ResidualBwdArgs& a, int k) {
  return a.gpost ? mul8(ld8(a.gpost + k), a.scale) : fill8(a.scale);
}

// The end of a run of tokens that share a gate row, at 8 features, with acc the
// sum of q D over the team's tokens of it: their part of sum act q D, and the
// gate row's gradient, slope scale gamma_post acc, written where the team has all
// of the row's tokens, or kept for the kernel that joins the teams' parts.
// part nullptr: the gradient is not wanted; all: one row for all tokens (its
// gradient goes with the other sums over tokens, in acc).
__device__ __forceinline__ void flush_gate(const ResidualBwdArgs& a, const Team& m, float* part, int teams, bool all,
                                           int64_t group, int k, V8& acc, V8& post) {
  V8 slope;
  post = fma8(shared_act(a, group, k, slope), acc, post);
  const V8 sum = mul8(mul8(slope, scaled_gain(a, k)), acc);
  acc = all ? sum : fill8(0.f);
  if (!part) return;
  const int64_t start = group * a.gate_rows;
  const int64_t end = a.gate_rows < a.T - start ? start + a.gate_rows : a.T;
  if (start >= m.r0 && end <= m.r0 + m.rows) {
    st8(a.dgate, group * a.d + k, a.g_bf16, sum);
    return;
  }
  const int64_t id = static_cast<int64_t>(blockIdx.x) * teams + m.team;
  part += (id * 2 + (start < m.r0 ? 0 : 1)) * a.d + k;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    part[2 * i] = sum.p[i].x;
    part[2 * i + 1] = sum.p[i].y;
  }
}

// A thread's part of a sum over tokens, for its team.
template <int VPT>
__device__ __forceinline__ void park(float* buf, const Team& m, int d, const V8 (&t)[VPT], float scale) {
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int k = (v * m.warps * 32 + m.tid) * 8;
    if (k < d) st8(buf + m.team * d + k, mul8(t[v], scale));
  }
}

// The CTA's partial rows, its teams added in order: sums [3][gridDim.x][d]
// (dgamma_post, dgamma_pre, the one gate row of all tokens). The rings are
// free: every copy has landed and been read.
template <int VPT>
__device__ __forceinline__ void write_sums(const ResidualBwdArgs& a, const Team& m, const TeamGeom& g, float* buf,
                                           float* sums, bool with_post, bool with_gate, const V8 (&post)[VPT],
                                           const V8 (&pre)[VPT], const V8 (&gate)[VPT]) {
  for (int which = 0; which < 3; ++which) {
    if (which == 0 ? !with_post : (which == 1 ? !(a.dn && a.dgpre) : !with_gate)) continue;
    __syncthreads();
    if (which == 0)
      park(buf, m, a.d, post, a.scale);
    else
      park(buf, m, a.d, which == 1 ? pre : gate, 1.f);
    __syncthreads();
    float* part = sums + (static_cast<int64_t>(which) * gridDim.x + blockIdx.x) * a.d;
    for (int k = threadIdx.x; k < a.d; k += blockDim.x) {
      float t = 0.f;
      for (int i = 0; i < g.teams; ++i) t += buf[i * a.d + k];
      part[k] = t;
    }
  }
}

// F: the type of f, dnormed and df; X: of x_out; G: of dx_out and dx. HAS_F:
// with the sublayer's side; without, the backward of RMSNorm.
template <typename F, typename X, typename G, int GATE, bool HAS_F>
__global__ void __launch_bounds__((HAS_F ? kGatedWarps : kNormWarps) * 32, 1)
    residual_bwd_kernel(ResidualBwdArgs a, const __grid_constant__ TeamGeom g, float* sums, float* shared_part) {
  extern __shared__ __align__(128) unsigned char smem[];
  init_bars(g, smem);
  Team m = make_team(g, a.T, smem);
  pdl_trigger();
  pdl_wait();
  fill_ring(m, g);
  const int d = a.d, k = m.tid * 8;
  const bool mine = k < d, post_norm = HAS_F && a.gpost != nullptr;
  const float inv_d = 1.0f / static_cast<float>(d);
  // scale * gamma_post, with a shared gate times its value too.
  V8 gain = mine && HAS_F ? scaled_gain(a, k) : fill8(0.f), gpre = fill8(0.f), slope;
  if (mine && a.dn) gpre = ld8(a.gpre + k);
  // The shared gate row of the current token, and the first token of the next one.
  int64_t group = 0, group_end = a.T;
  if (GATE == kSharedGate) {
    group = m.r0 / a.gate_rows;
    if (a.gate_rows < a.T) group_end = (group + 1) * a.gate_rows;
    if (mine && m.rows > 0) gain = mul8(gain, shared_act(a, group, k, slope));
  }
  // Sums over tokens: act q D (dgamma_post / scale), dn u, and of the current
  // shared gate row q D.
  V8 post[1] = {fill8(0.f)}, pre[1] = {fill8(0.f)}, gsum[1] = {fill8(0.f)};

  // Waits for a row and takes its part of sum x^2, sum h x and sum f^2.
  int stage = 0;
  uint32_t parity = 0;
  constexpr int kSums = HAS_F ? 4 : 2;
  float s[kSums] = {};  // those of a row, and last sum gamma_post dy q of the row before
  auto begin_row = [&]() {
    const bool ok = mbar_wait(m.bars + stage * 8, parity);
    if (ok && mine) {
      const unsigned char* st = m.ring + stage * g.stage_bytes;
      if (a.dn) {
        const V8 x = ld8(reinterpret_cast<const X*>(st + g.x) + k);
        s[0] = dot8(x, x);
        s[1] = dot8(mul8(gpre, ld8(reinterpret_cast<const F*>(st + g.dn) + k)), x);
      }
      if constexpr (HAS_F) {
        const V8 f = ld8(reinterpret_cast<const F*>(st + g.f) + k);
        s[2] = dot8(f, f);
      }
    }
    return ok;
  };
  bool ok = m.rows == 0 || begin_row();
  ok = team_sum(m, s, 1, ok);
  if (!ok) give_up(m, g, 0, &g_timeout);
  for (int r = 0; ok && r < m.rows; ++r) {
    const int64_t row = m.r0 + r;
    if (GATE == kSharedGate && row == group_end) {
      ++group;
      group_end += a.gate_rows;
      if (mine) gain = mul8(scaled_gain(a, k), shared_act(a, group, k, slope));
    }
    const unsigned char* st = m.ring + stage * g.stage_bytes;
    const float rx = a.dn ? rsqrtf(s[0] * inv_d + a.eps_pre) : 0.f, mx = rx * (s[1] * inv_d);
    float rf = 1.f;
    if constexpr (HAS_F) {
      if (post_norm) rf = rsqrtf(s[2] * inv_d + a.eps_post);
    }
#pragma unroll
    for (int i = 0; i < kSums; ++i) s[i] = 0.f;
    V8 q, t;  // t = gamma_post dy = scale gamma_post act D
    if (mine) {
      V8 D = a.dxo ? ld8(reinterpret_cast<const G*>(st + g.dxo) + k) : fill8(0.f);
      if (a.dn) {
        const V8 x = mul8(ld8(reinterpret_cast<const X*>(st + g.x) + k), rx);
        const V8 h = ld8(reinterpret_cast<const F*>(st + g.dn) + k);
        pre[0] = fma8(h, x, pre[0]);
        D = fma8(fma8(x, -mx, mul8(gpre, h)), rx, D);
      }
      if (a.dx) st8(static_cast<G*>(a.dx) + row * d + k, D);
      if constexpr (HAS_F) {
        q = mul8(ld8(reinterpret_cast<const F*>(st + g.f) + k), rf);
        if (GATE == kTokenGate) {
          V8 act = ld8(st + g.gate, k, a.g_bf16);
          activate8<true>(act, slope, a.sigmoid);
          const V8 qD = mul8(q, D);
          post[0] = fma8(act, qD, post[0]);
          if (a.dgate) st8(a.dgate, row * d + k, a.g_bf16, mul8(slope, mul8(gain, qD)));
          t = mul8(mul8(gain, act), D);
        } else {
          V8& sum = GATE == kSharedGate ? gsum[0] : post[0];
          sum = fma8(q, D, sum);
          t = mul8(gain, D);
        }
        s[3] = dot8(t, q);
      }
    }
    if (++stage == m.nst) stage = 0, parity ^= 1u;
    if (r + 1 < m.rows) ok = begin_row();
    ok = team_sum(m, s, r & 1, ok);
    if (!ok) {
      give_up(m, g, r + 1, &g_timeout);
      break;
    }
    // Every thread has what it needs of row r: its stage is free.
    if (m.tid == 0 && m.issued < m.rows) issue_row(m, g);
    if constexpr (HAS_F) {
      if (mine && a.df)
        st8(static_cast<F*>(a.df) + row * d + k, post_norm ? mul8(fma8(q, -(s[3] * inv_d), t), rf) : t);
      if (GATE == kSharedGate && mine && (r + 1 == m.rows || row + 1 == group_end))
        flush_gate(a, m, shared_part, g.teams, a.gate_rows >= a.T, group, k, gsum[0], post[0]);
    }
  }
  write_sums<1>(a, m, g, reinterpret_cast<float*>(smem + g.stages), sums, post_norm && a.dgpost,
                GATE == kSharedGate && a.dgate && a.gate_rows >= a.T, post, pre, gsum);
}

// The gated backward past d = 5120: 16 features a thread, so only D and the
// sums over tokens stay in registers; the row is read from its stage again in
// each step, and the gains from shared memory. A stage is refilled after the
// next row's first sum, when every thread is past its last read of it.
template <int GATE>
__global__ void __launch_bounds__(kWideWarps * 32, 1)
    residual_bwd_wide_kernel(ResidualBwdArgs a, const __grid_constant__ TeamGeom g, float* sums, float* shared_part) {
  constexpr int kV = 2;
  extern __shared__ __align__(128) unsigned char smem[];
  init_bars(g, smem);
  Team m = make_team(g, a.T, smem);
  pdl_trigger();
  pdl_wait();
  fill_ring(m, g);
  const int d = a.d, step = m.warps * 256;
  const bool post_norm = a.gpost != nullptr;
  const float inv_d = 1.0f / static_cast<float>(d);
  float* gains = reinterpret_cast<float*>(smem + g.gain);  // scale * gamma_post, gamma_pre
  for (int k = threadIdx.x; k < d; k += blockDim.x) {
    gains[k] = post_norm ? a.gpost[k] * a.scale : a.scale;
    gains[d + k] = a.dn ? a.gpre[k] : 0.f;
  }
  __syncthreads();
  int64_t group = 0, group_end = a.T;
  if (GATE == kSharedGate) {
    group = m.r0 / a.gate_rows;
    if (a.gate_rows < a.T) group_end = (group + 1) * a.gate_rows;
  }
  V8 post[kV], pre[kV], gsum[kV];
#pragma unroll
  for (int v = 0; v < kV; ++v) post[v] = pre[v] = gsum[v] = fill8(0.f);

  int stage = 0;
  uint32_t parity = 0;
  for (int r = 0; r < m.rows; ++r) {
    const int64_t row = m.r0 + r;
    if (GATE == kSharedGate && row == group_end) {
      ++group;
      group_end += a.gate_rows;
    }
    const unsigned char* st = m.ring + stage * g.stage_bytes;
    bool ok = mbar_wait(m.bars + stage * 8, parity);
    if (++stage == m.nst) stage = 0, parity ^= 1u;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (ok) {
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        const int k = v * step + m.tid * 8;
        if (k < d) {
          if (a.dn) {
            const V8 x = ld8(st + g.x, k, a.x_bf16);
            s[0] += dot8(x, x);
            s[1] += dot8(mul8(ld8(gains + d + k), ld8(st + g.dn, k, a.f_bf16)), x);
          }
          if (post_norm) {
            const V8 f = ld8(st + g.f, k, a.f_bf16);
            s[2] += dot8(f, f);
          }
        }
      }
    }
    ok = team_sum(m, s, 0, ok);
    if (!ok) {
      give_up(m, g, r, &g_timeout);
      break;
    }
    if (m.tid == 0 && r > 0 && m.nst > 1 && m.issued < m.rows) issue_row(m, g);
    const float rx = a.dn ? rsqrtf(s[0] * inv_d + a.eps_pre) : 0.f, mx = rx * (s[1] * inv_d);
    const float rf = post_norm ? rsqrtf(s[2] * inv_d + a.eps_post) : 1.f;
    // act(gate) at 8 features, and a token's own gate's slope.
    auto act_at = [&](V8& slope, int k) {
      if (GATE == kSharedGate) return shared_act(a, group, k, slope);
      if (GATE == kNoGate) return fill8(1.f);
      V8 act = ld8(st + g.gate, k, a.g_bf16);
      activate8<true>(act, slope, a.sigmoid);
      return act;
    };

    V8 D[kV], slope;
    float q[1] = {0.f};
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      const int k = v * step + m.tid * 8;
      if (k < d) {
        D[v] = a.dxo ? ld8(st + g.dxo, k, a.dx_bf16) : fill8(0.f);
        if (a.dn) {
          const V8 x = mul8(ld8(st + g.x, k, a.x_bf16), rx), h = ld8(st + g.dn, k, a.f_bf16);
          pre[v] = fma8(h, x, pre[v]);
          D[v] = fma8(fma8(x, -mx, mul8(ld8(gains + d + k), h)), rx, D[v]);
        }
        if (a.dx) st8(a.dx, row * d + k, a.dx_bf16, D[v]);
        if (post_norm)
          q[0] += dot8(mul8(ld8(gains + k), mul8(act_at(slope, k), D[v])), mul8(ld8(st + g.f, k, a.f_bf16), rf));
      }
    }
    (void)team_sum(m, q, 1, true);
    const float mf = post_norm ? q[0] * inv_d : 0.f;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      const int k = v * step + m.tid * 8;
      if (k < d) {
        const V8 f = mul8(ld8(st + g.f, k, a.f_bf16), rf), c = ld8(gains + k), qD = mul8(f, D[v]);
        const V8 act = act_at(slope, k);
        if (GATE == kSharedGate) {
          gsum[v] = fma8(f, D[v], gsum[v]);
        } else {
          post[v] = fma8(act, qD, post[v]);
          if (GATE == kTokenGate && a.dgate) st8(a.dgate, row * d + k, a.g_bf16, mul8(slope, mul8(c, qD)));
        }
        if (a.df) {
          const V8 t = mul8(mul8(c, act), D[v]);
          st8(a.df, row * d + k, a.f_bf16, post_norm ? mul8(fma8(f, -mf, t), rf) : t);
        }
        if (GATE == kSharedGate && (r + 1 == m.rows || row + 1 == group_end))
          flush_gate(a, m, shared_part, g.teams, a.gate_rows >= a.T, group, k, gsum[v], post[v]);
      }
    }
    // A ring of one stage: the next row's copies start when all are done with this one.
    if (m.nst == 1 && r + 1 < m.rows) {
      team_sync(m);
      if (m.tid == 0) issue_row(m, g);
    }
  }
  write_sums<kV>(a, m, g, reinterpret_cast<float*>(smem + g.stages), sums, post_norm && a.dgpost,
                 GATE == kSharedGate && a.dgate && a.gate_rows >= a.T, post, pre, gsum);
}

// Gate rows whose tokens lie in several teams' runs: the sums of those teams,
// in order. A thread block takes a team and a block of features and acts if
// the team's first row is the first of its gate row's tokens outside the run
// of the team that has the row's first token.
__global__ void __launch_bounds__(256)
    residual_bwd_join_gate_kernel(ResidualBwdArgs a, const float* shared_part, int64_t teams) {
  pdl_trigger();
  pdl_wait();
  const int64_t t = blockIdx.x + 1;
  const int64_t k = static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x;
  const int64_t row = a.T * t / teams;
  const int64_t group = row / a.gate_rows, start = group * a.gate_rows;
  if (row == a.T * (t + 1) / teams || start == row || k >= a.d) return;
  const int64_t first = ((start + 1) * teams - 1) / a.T;  // the team with the row's first token
  if (a.T * (first + 1) / teams != row) return;
  const int64_t end = a.gate_rows < a.T - start ? start + a.gate_rows : a.T;
  const int64_t last = (end * teams - 1) / a.T;           // and the one with its last
  const float* part = shared_part + k;
  float s = part[(first * 2 + 1) * a.d];
  if (a.T >= teams) {
#pragma unroll 8
    for (int64_t u = t; u <= last; ++u) s += part[u * 2 * a.d];
  } else {  // some teams have no rows, and have written nothing
    for (int64_t u = t; u <= last; ++u)
      if (a.T * u / teams < a.T * (u + 1) / teams) s += part[u * 2 * a.d];
  }
  if (a.g_bf16)
    static_cast<bf16*>(a.dgate)[group * a.d + k] = from_f32<bf16>(s);
  else
    static_cast<float*>(a.dgate)[group * a.d + k] = s;
}

bool geom_of(const ResidualBwdArgs& a, TeamGeom* g) {
  *g = TeamGeom{};
  const int es = a.f_bf16 ? 2 : 4, xs = a.x_bf16 ? 2 : 4;
  add_input(*g, a.f, a.d * es, &g->f);
  add_input(*g, a.dn ? a.xo : nullptr, a.d * xs, &g->x);
  add_input(*g, a.dxo, a.d * (a.dx_bf16 ? 2 : 4), &g->dxo);
  add_input(*g, a.dn, a.d * es, &g->dn);
  add_input(*g, a.gate && a.gate_rows == 1 ? a.gate : nullptr, a.d * (a.g_bf16 ? 2 : 4), &g->gate);
  const TeamShape s = team_shape(a.d, max_warps(a));
  // The teams' sums go through the rings' space: 4 bytes a feature and team.
  return finish_geom(*g, s, s.vectors > 1 ? 8 * a.d : 0, s.vectors > 1 ? 1 : 2) && g->nst * g->stage_bytes >= 4 * a.d;
}

struct Plan {
  TeamGeom g;
  int64_t ctas;
  float* sums;
  float* shared;
  cudaStream_t s;
};

template <typename F, typename X, typename G>
cudaError_t launch_typed(const ResidualBwdArgs& a, const Plan& p) {
  if (!a.gate) return launch_teams(residual_bwd_kernel<F, X, G, kNoGate, true>, p.g, p.ctas, p.s, a, p.g, p.sums, p.shared);
  if (a.gate_rows == 1)
    return launch_teams(residual_bwd_kernel<F, X, G, kTokenGate, true>, p.g, p.ctas, p.s, a, p.g, p.sums, p.shared);
  return launch_teams(residual_bwd_kernel<F, X, G, kSharedGate, true>, p.g, p.ctas, p.s, a, p.g, p.sums, p.shared);
}
template <typename F, typename G>
cudaError_t launch_norm(const ResidualBwdArgs& a, const Plan& p) {
  return launch_teams(residual_bwd_kernel<F, F, G, kNoGate, false>, p.g, p.ctas, p.s, a, p.g, p.sums, p.shared);
}

}  // namespace

bool residual_bwd_fast_ok(const ResidualBwdArgs& a) {
  TeamGeom g;
  return a.T > 0 && a.d % 8 == 0 && a.d <= kMaxTeamD && aligned16(a.f) && aligned16(a.gate) && aligned16(a.gpost) &&
         aligned16(a.xo) && aligned16(a.gpre) && aligned16(a.dxo) && aligned16(a.dn) && aligned16(a.df) &&
         aligned16(a.dx) && aligned16(a.dgate) && geom_of(a, &g);
}

// Enough for either shape of a CTA (the gated one has more teams to a CTA's
// partial rows of shared gates, the other more CTAs to none).
int64_t residual_bwd_fast_scratch(int64_t T, int d, int64_t gate_rows) {
  if (T == 0 || d % 8 != 0 || d > kMaxTeamD) return 0;
  const TeamShape s = team_shape(d, kGatedWarps);
  const int64_t ctas = team_ctas(T, s, kMaxCtas);
  return 3 * ctas * d + (gate_rows > 1 && gate_rows < T ? ctas * s.teams * 2 * d : 0);
}

int residual_bwd_parts(const ResidualBwdArgs& a) {
  return static_cast<int>(team_ctas(a.T, team_shape(a.d, max_warps(a)), cta_cap()));
}

cudaError_t launch_residual_bwd_fast(const ResidualBwdArgs& a, cudaStream_t s) {
  Plan p{{}, residual_bwd_parts(a), a.scratch, nullptr, s};
  if (!geom_of(a, &p.g)) return cudaErrorInvalidValue;
  if (residual_bwd_shares_gates(a)) p.shared = p.sums + 3 * p.ctas * a.d;
  if (!a.f) {
    if (!a.f_bf16) return launch_norm<float, float>(a, p);
    return a.dx_bf16 ? launch_norm<bf16, bf16>(a, p) : launch_norm<bf16, float>(a, p);
  }
  if (team_shape(a.d, kGatedWarps).vectors > 1) {
    if (!a.gate) return launch_teams(residual_bwd_wide_kernel<kNoGate>, p.g, p.ctas, s, a, p.g, p.sums, p.shared);
    if (a.gate_rows == 1)
      return launch_teams(residual_bwd_wide_kernel<kTokenGate>, p.g, p.ctas, s, a, p.g, p.sums, p.shared);
    return launch_teams(residual_bwd_wide_kernel<kSharedGate>, p.g, p.ctas, s, a, p.g, p.sums, p.shared);
  }
  if (!a.f_bf16) return launch_typed<float, float, float>(a, p);
  if (a.x_bf16) return a.dx_bf16 ? launch_typed<bf16, bf16, bf16>(a, p) : launch_typed<bf16, bf16, float>(a, p);
  return a.dx_bf16 ? launch_typed<bf16, float, bf16>(a, p) : launch_typed<bf16, float, float>(a, p);
}

cudaError_t launch_residual_bwd_join_gate(const ResidualBwdArgs& a, cudaStream_t s) {
  const int64_t ctas = residual_bwd_parts(a), teams = ctas * team_shape(a.d, kGatedWarps).teams;
  const float* shared = a.scratch + 3 * ctas * a.d;
  if (teams < 2) return cudaSuccess;
  return launch_pdl_grid(residual_bwd_join_gate_kernel, dim3(static_cast<unsigned>(teams - 1), (a.d - 1) / 256 + 1), 256, 0,
                         s, a, shared, teams);
}

cudaError_t take_timeout_residual_bwd(unsigned int* flag) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(flag, g_timeout, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_timeout, &zero, sizeof(unsigned int));
}

}  // namespace attnres
