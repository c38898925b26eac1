// Backward of the gated residual, and of RMSNorm, for d a multiple of 8 up to
// 8192 with aligned rows (the formulas stand at the top of residual.cu, the
// teams in residual_team.cuh).
//
// Each row is read and written once, which bounds rows with an fp32 stream or
// gradient (64M elements with a gate per token at 90 to 95 % of the copy bandwidth
// from 512 to 5120 features). Rows of bf16 throughout take the same time for 1.4
// times fewer bytes (32768 x 896 in 109 us, 63 %; 63 to 79 % from 512 to 8192
// features, 58 at 384): a row's instructions and its barrier bound them, not its
// bytes. Short runs of shared gate rows pay for their ends (32768 x 896 with an fp32
// stream: 139 us with runs of 2 tokens, 108 with 8, 109 with a row each).
//
// The sums over tokens stay in registers for the whole run of rows (a thread's
// features never change), are added over the CTA's teams in shared memory and
// leave one partial row per CTA; a gate row that some tokens share is written by
// the team that has all of them, or left in two parts per team for one more
// kernel. The sums of row r's second mean and of row r + 1's first ones go through
// the team together, so a row costs one barrier.
#include "residual_team.cuh"

namespace attnres {
namespace {

__device__ unsigned int g_timeout = 0;

// Warps of a CTA. The backward of RMSNorm: 28 of 72 registers, 16 of 128 for
// 16 features a thread, 12 of 168 for 24. The gated one: 20 of 96 (8192 x 896 takes
// 4 % less than with 16 of 128, 32749 x 640 with shared gate rows 6 %), 8 of 255 for
// 24 features a thread; past the width that 8 features cover its threads take 16, and
// 128 registers. (With shared gate rows these spill 8 and 16 to 32 bytes.)
constexpr int norm_warps(int vectors) { return vectors == 1 ? 28 : vectors == 2 ? 16 : 12; }
constexpr int gated_warps(int vectors) { return vectors == 1 ? 20 : vectors == 2 ? 16 : 8; }
// Rows in flight per SM, held as the forward's to what leaves the writes room
// (ungated, an fp32 stream: 131072 x 256 at 91 % of the copy bandwidth with 146 KB,
// 80 with 190). Fewer than 10 teams want a third row, of up to 196 KB (16384 x 2048
// fp32: 90 % against 82; with 215 KB 1024 and 1536 lose 4 to 5), a team alone
// wherever it fits (8192 x 4096 fp32 with gates: 89 % with 221 KB, 75 with two rows).
// The RMSNorm backward's single warps want a third row each where rows are long
// enough that 120 KB hold only two (262144 x 256: 94 % with 180 KB, 75 with 120;
// other widths lose 2 to 8 % by it), and past 512 features all-bf16 rows gain up to
// 2.7 % by 146 KB (9362 x 3584: 83 % against 81).
constexpr int kNormRing = 120 * 1024, kNarrowNormRing = 180 * 1024, kBf16NormRing = 146 * 1024;
constexpr int kGatedRing = 146 * 1024, kGatedThird = 196 * 1024;

// The gate of a call: none or one row for all tokens, one per token, or rows
// that runs of tokens share.
int gate_kind(int64_t T, int64_t gate_rows, bool gate) {
  if (!gate || (gate_rows > 1 && gate_rows >= T)) return kNoGate;
  return gate_rows == 1 ? kTokenGate : kSharedGate;
}
// Where three warps of 8 features a thread would be short of instructions, one
// warp takes the row with 24 (104857 x 640, all bf16, at 91 % of the copy bandwidth,
// with three 71; with fp32 gradients, which give them more time, 86 against 94).
TeamShape norm_shape(int64_t T, int d, bool all_bf16) {
  const int v = d > 512 && d <= 768 && all_bf16 ? 3 : (d > 256 * norm_warps(1) || (d > 512 && sixteen_pay(d)) ? 2 : 1);
  return team_shape(T, d, v, norm_warps(v));
}
TeamShape gated_shape(int64_t T, int d, int gate) {
  // (Not with shared gates: 32749 x 640 in runs of 2048 tokens took 77 us by single
  // warps, 72 by three.)
  const int v = d > 512 && d <= 704 && gate != kSharedGate ? 3 : (d > 256 * gated_warps(1) ? 2 : 1);
  return team_shape(T, d, v, gated_warps(v));
}
TeamShape shape_of(const ResidualBwdArgs& a) {
  return a.f ? gated_shape(a.T, a.d, gate_kind(a.T, a.gate_rows, a.gate != nullptr)) : norm_shape(a.T, a.d, a.f_bf16 && a.dx_bf16);
}

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
// sum of q D over the team's tokens of it: returns their part of sum act q D,
// and makes acc the gate row's gradient, slope scale gamma_post acc, which is
// written where the team has all of the row's tokens, or kept for the kernel
// that joins the teams' parts (part nullptr: neither).
__device__ __forceinline__ V8 flush_gate(const ResidualBwdArgs& a, const Team& m, float* part, int teams, int64_t group,
                                         int k, V8& acc) {
  V8 slope;
  const V8 post = mul8(shared_act(a, group, k, slope), acc);
  acc = mul8(mul8(slope, scaled_gain(a, k)), acc);
  if (!part) return post;
  const int64_t start = group * a.gate_rows;
  const int64_t end = a.gate_rows < a.T - start ? start + a.gate_rows : a.T;
  if (start >= m.r0 && end <= m.r0 + m.rows) {
    out8(a.dgate, group * a.d + k, a.g_bf16, acc);
    return post;
  }
  const int64_t id = static_cast<int64_t>(blockIdx.x) * teams + m.team;
  part += (id * 2 + (start < m.r0 ? 0 : 1)) * a.d + k;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    part[2 * i] = acc.p[i].x;
    part[2 * i + 1] = acc.p[i].y;
  }
  return post;
}

// The CTA's partial rows, its teams added in order: sums [3][gridDim.x][d]
// (dgamma_post, dgamma_pre, the one gate row of all tokens). The rings are
// free: every copy has landed and been read.
template <int VPT>
__device__ __forceinline__ void write_sums(const ResidualBwdArgs& a, const Team& m, const TeamGeom& g, float* buf,
                                           float* sums, bool with_post, bool with_gate, const V8 (&post)[VPT],
                                           const V8 (&pre)[VPT], const V8 (&gate)[VPT]) {
  const bool direct = g.teams == 1 && (reinterpret_cast<uintptr_t>(sums) & 15) == 0;
  for (int which = 0; which < 3; ++which) {
    if (which == 0 ? !with_post : (which == 1 ? !(a.dn && a.dgpre) : !with_gate)) continue;
    float* const part = sums + (static_cast<int64_t>(which) * gridDim.x + blockIdx.x) * a.d;
    if (!direct) __syncthreads();
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int k = (v * m.warps * 32 + m.tid) * 8;
      if (k < a.d)
        st8((direct ? part : buf + m.team * a.d) + k,
            which == 0 ? mul8(post[v], a.scale) : (which == 1 ? pre[v] : gate[v]));
    }
    if (direct) continue;
    __syncthreads();
    for (int k = threadIdx.x; k < a.d; k += blockDim.x) {
      float t = 0.f;
      for (int i = 0; i < g.teams; ++i) t += buf[i * a.d + k];
      part[k] = t;
    }
  }
}

// The backward of RMSNorm. F: the type of x and dy; G: of dres and dx.
template <typename F, typename G, int VPT>
__global__ void __launch_bounds__(norm_warps(VPT) * 32, 1)
    rmsnorm_bwd_kernel(ResidualBwdArgs a, const __grid_constant__ TeamGeom g, float* sums) {
  extern __shared__ __align__(128) unsigned char smem[];
  init_bars(g, smem);
  Team m = make_team<false>(g, a.T, smem);
  pdl_trigger();
  pdl_wait();
  fill_ring(m, g);
  const int d = a.d, k0 = m.tid * 8, step = m.warps * 256;
  const float inv_d = 1.0f / static_cast<float>(d);
  V8 gain[VPT], sum[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    gain[v] = sum[v] = fill8(0.f);
    if (k0 + v * step < d) gain[v] = ld8(a.gpre + k0 + v * step);
  }
  int stage = 0;
  uint32_t parity = 0;
  for (int r = 0; r < m.rows; ++r) {
    const unsigned char* st = m.ring + stage * g.stage_bytes;
    bool ok = mbar_wait(m.bars + stage * 8, parity);
    if (++stage == m.nst) stage = 0, parity ^= 1u;
    V8 x[VPT], h[VPT], D[VPT];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int k = k0 + v * step;
      if (ok && k < d) {
        x[v] = ld8(reinterpret_cast<const F*>(st + g.x) + k);
        h[v] = ld8(reinterpret_cast<const F*>(st + g.dn) + k);
        s[0] += dot8(x[v], x[v]);
        s[1] += dot8(mul8(gain[v], h[v]), x[v]);
        D[v] = a.dxo ? ld8(reinterpret_cast<const G*>(st + g.dxo) + k) : fill8(0.f);
      }
    }
    ok = team_sum(m, s, r & 1, ok);
    if (!ok) {
      give_up(m, g, r, &g_timeout);
      break;
    }
    // Every thread has its part of the row in registers: the stage is free.
    if (m.tid == 0 && m.issued < m.rows) issue_row(m, g);
    const float rx = rsqrtf(s[0] * inv_d + a.eps_pre), mx = rx * (s[1] * inv_d);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int k = k0 + v * step;
      if (k < d) {
        const V8 u = mul8(x[v], rx);
        sum[v] = fma8(h[v], u, sum[v]);
        out8(static_cast<G*>(a.dx) + (m.r0 + r) * d + k, fma8(fma8(u, -mx, mul8(gain[v], h[v])), rx, D[v]));
      }
    }
  }
  write_sums<VPT>(a, m, g, reinterpret_cast<float*>(smem + g.stages), sums, false, false, sum, sum, sum);
}

// The gated backward. F: the type of f, dnormed and df; X: of x_out; G: of
// dx_out and dx. GATE kNoGate also takes the one gate row of all tokens, which
// rides on the gain. VPT: 8 or 24 features a thread, with the gains in registers,
// or for the widest rows 16 (one team a CTA), with the gains in shared memory
// and rings that may hold a single row. FAR: gamma_pre is read from the L2 for each
// row, which leaves room for a second one (a switch while running cost the
// others up to 6 %).
template <typename F, typename X, typename G, int GATE, int VPT, bool FAR = false>
__global__ void __launch_bounds__(gated_warps(VPT) * 32, 1)
    residual_bwd_kernel(ResidualBwdArgs a, const __grid_constant__ TeamGeom g, float* sums, float* shared_part) {
  extern __shared__ __align__(128) unsigned char smem[];
  init_bars(g, smem);
  Team m = make_team<false>(g, a.T, smem);
  pdl_trigger();
  pdl_wait();
  fill_ring(m, g);
  const int d = a.d, k0 = m.tid * 8, step = m.warps * 256;
  const bool post_norm = a.gpost != nullptr;
  const float inv_d = 1.0f / static_cast<float>(d);
  // scale * gamma_post, with a shared gate times its value too; gamma_pre; the
  // sums over the tokens of earlier runs (of the widest rows, whose one team needs
  // the room for a row, in the CTA's partial row: 4096 x 8192 bf16 with shared gate
  // rows at 51 % of the copy bandwidth, in shared memory 39). What is in memory is
  // each thread's own part.
  constexpr bool kWide = VPT == 2;
  V8 gain_reg[VPT] = {}, gpre_reg[VPT] = {}, slope;
  auto kept = [&](int which) { return reinterpret_cast<float*>(smem + g.gain) + which * d; };
  auto ld_earlier = [&](int k) {
    if constexpr (!kWide) return ld8(kept(0) + static_cast<int>(threadIdx.x) / (g.warps * 32) * d + k);
    const float* p = sums + static_cast<int64_t>(blockIdx.x) * d + k;
    V8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i] = make_float2(p[2 * i], p[2 * i + 1]);
    return r;
  };
  auto st_earlier = [&](int k, const V8& x) {
    if constexpr (!kWide) {
      st8(kept(0) + static_cast<int>(threadIdx.x) / (g.warps * 32) * d + k, x);
    } else {
      float* p = sums + static_cast<int64_t>(blockIdx.x) * d + k;
#pragma unroll
      for (int i = 0; i < 4; ++i) p[2 * i] = x.p[i].x, p[2 * i + 1] = x.p[i].y;
    }
  };
  auto gain = [&](int v, int k) {
    if constexpr (kWide) return ld8(kept(0) + k);
    else return gain_reg[v];
  };
  auto gpre = [&](int v, int k) {
    if constexpr (kWide) return ld8((FAR ? a.gpre : kept(1)) + k);
    else return gpre_reg[v];
  };
  auto set_gain = [&](int64_t group) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int k = k0 + v * step;
      gain_reg[v] = fill8(0.f);
      if (k < d) {
        V8 c = scaled_gain(a, k);
        if (GATE != kTokenGate && a.gate) c = mul8(c, shared_act(a, group, k, slope));
        if (kWide)
          st8(kept(0) + k, c);
        else
          gain_reg[v] = c;
      }
    }
  };
  if (GATE != kSharedGate) set_gain(0);
  // Sums over tokens: q D (with a gate per token act q D), of the current run of
  // a shared gate row; dn u.
  V8 acc[VPT], pre[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int k = k0 + v * step;
    acc[v] = pre[v] = gpre_reg[v] = fill8(0.f);
    if (k < d) {
      if (a.dn) {
        gpre_reg[v] = ld8(a.gpre + k);
        if (kWide && !FAR) st8(kept(1) + k, gpre_reg[v]);
      }
      if (GATE == kSharedGate) st_earlier(k, acc[v]);
    }
  }

  // Waits for a row and takes its part of sum x^2, sum h x and sum f^2.
  int stage = 0;
  uint32_t parity = 0;
  float s[4] = {};  // those of a row, and last sum gamma_post dy q of the row before
  auto begin_row = [&]() {
    const bool ok = mbar_wait(m.bars + stage * 8, parity);
    const unsigned char* st = m.ring + stage * g.stage_bytes;
    if (ok) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int k = k0 + v * step;
        if (k < d) {
          if (a.dn) {
            const V8 x = ld8(reinterpret_cast<const X*>(st + g.x) + k);
            s[0] += dot8(x, x);
            s[1] += dot8(mul8(gpre(v, k), ld8(reinterpret_cast<const F*>(st + g.dn) + k)), x);
          }
          const V8 f = ld8(reinterpret_cast<const F*>(st + g.f) + k);
          s[2] += dot8(f, f);
        }
      }
    }
    return ok;
  };
  bool ok = m.rows == 0 || begin_row();
  ok = team_sum(m, s, 1, ok);
  if (!ok) give_up(m, g, 0, &g_timeout);
  // Runs of tokens with one gate row (without such rows: the one run).
  for (int r = 0; ok && r < m.rows;) {
    int run_end = m.rows;
    if (GATE == kSharedGate) {
      const int64_t group = (m.r0 + r) / a.gate_rows;
      const int64_t end = (group + 1) * a.gate_rows - m.r0;
      if (end < run_end) run_end = static_cast<int>(end);
      set_gain(group);
    }
    for (; r < run_end; ++r) {
      const int64_t row = (m.r0 + r) * d;
      const unsigned char* st = m.ring + stage * g.stage_bytes;
      const float rx = a.dn ? rsqrtf(s[0] * inv_d + a.eps_pre) : 0.f, mx = rx * (s[1] * inv_d);
      const float rf = post_norm ? rsqrtf(s[2] * inv_d + a.eps_post) : 1.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = 0.f;
      V8 q[VPT], t[VPT];  // t = gamma_post dy = scale gamma_post act D
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int k = k0 + v * step;
        if (k < d) {
          V8 D = a.dxo ? ld8(reinterpret_cast<const G*>(st + g.dxo) + k) : fill8(0.f);
          if (a.dn) {
            const V8 u = mul8(ld8(reinterpret_cast<const X*>(st + g.x) + k), rx);
            const V8 h = ld8(reinterpret_cast<const F*>(st + g.dn) + k);
            pre[v] = fma8(h, u, pre[v]);
            D = fma8(fma8(u, -mx, mul8(gpre(v, k), h)), rx, D);
          }
          if (a.dx) out8(static_cast<G*>(a.dx) + row + k, D);
          q[v] = mul8(ld8(reinterpret_cast<const F*>(st + g.f) + k), rf);
          if (GATE == kTokenGate) {
            V8 act = ld8(st + g.gate, k, a.g_bf16);
            activate8<true>(act, slope, a.sigmoid);
            const V8 qD = mul8(q[v], D), c = gain(v, k);
            acc[v] = fma8(act, qD, acc[v]);
            if (a.dgate) out8(a.dgate, row + k, a.g_bf16, mul8(slope, mul8(c, qD)));
            t[v] = mul8(mul8(c, act), D);
          } else {
            acc[v] = fma8(q[v], D, acc[v]);
            t[v] = mul8(gain(v, k), D);
          }
          s[3] += dot8(t[v], q[v]);
        }
      }
      if (++stage == m.nst) stage = 0, parity ^= 1u;
      if (r + 1 < m.rows) {
        if (kWide && m.nst == 1) {  // a ring of one row: the next one comes when all are past this one
          team_sync(m);
          if (m.tid == 0) issue_row(m, g);
        }
        ok = begin_row();
      }
      ok = team_sum(m, s, r & 1, ok);
      if (!ok) {
        give_up(m, g, r + 1, &g_timeout);
        break;
      }
      // Every thread has what it needs of row r: its stage is free.
      if ((!kWide || m.nst > 1) && m.tid == 0 && m.issued < m.rows) issue_row(m, g);
      if (a.df)
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
          const int k = k0 + v * step;
          if (k < d)
            out8(static_cast<F*>(a.df) + row + k, post_norm ? mul8(fma8(q[v], -(s[3] * inv_d), t[v]), rf) : t[v]);
        }
    }
    if (GATE == kSharedGate) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int k = k0 + v * step;
        if (k < d) {
          const V8 post = flush_gate(a, m, shared_part, g.teams, (m.r0 + run_end - 1) / a.gate_rows, k, acc[v]);
          st_earlier(k, add8(ld_earlier(k), post));
          acc[v] = fill8(0.f);
        }
      }
    }
  }
  V8 post[VPT], gate[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int k = k0 + v * step;
    post[v] = gate[v] = acc[v];
    if (k < d) {
      if (GATE == kSharedGate) post[v] = ld_earlier(k);
      if (GATE == kNoGate && a.gate) post[v] = flush_gate(a, m, nullptr, g.teams, 0, k, gate[v]);
    }
  }
  write_sums<VPT>(a, m, g, reinterpret_cast<float*>(smem + g.stages), sums, post_norm && a.dgpost,
                  GATE == kNoGate && a.gate && a.dgate, post, pre, gate);
}

bool geom_of(const ResidualBwdArgs& a, TeamGeom* g) {
  *g = TeamGeom{};
  const int es = a.f_bf16 ? 2 : 4, xs = a.x_bf16 ? 2 : 4;
  add_input(*g, a.f, a.d * es, &g->f);
  add_input(*g, a.dn ? a.xo : nullptr, a.d * xs, &g->x);
  add_input(*g, a.dxo, a.d * (a.dx_bf16 ? 2 : 4), &g->dxo);
  add_input(*g, a.dn, a.d * es, &g->dn);
  add_input(*g, a.gate && a.gate_rows == 1 ? a.gate : nullptr, a.d * (a.g_bf16 ? 2 : 4), &g->gate);
  const TeamShape s = shape_of(a);
  // With 16 features a thread the gated kernel's gains; else, where runs of tokens
  // share gate rows, the sums of earlier runs.
  int gain_bytes = a.f && s.vectors == 2 ? 8 * a.d : 0;
  // Where two rows fit only without it, gamma_pre is read from the L2 for each row
  // (4096 x 8192 ungated with an fp32 stream at 72 % of the copy bandwidth, by single
  // rows 57).
  if (gain_bytes && a.dn && kTeamSmem - rows_offset(s) - gain_bytes < 2 * g->stage_bytes &&
      kTeamSmem - rows_offset(s) - gain_bytes / 2 >= 2 * g->stage_bytes) {
    g->far_gain = 1;
    gain_bytes /= 2;
  }
  if (a.f && s.vectors != 2 && gate_kind(a.T, a.gate_rows, a.gate != nullptr) == kSharedGate)
    gain_bytes = 4 * s.teams * a.d;
  const bool all_bf16 = a.f_bf16 && a.dx_bf16;
  const int ring = a.f                            ? kGatedRing
                   : a.d > 200 && a.d <= 256      ? kNarrowNormRing
                   : all_bf16 && a.d > 512        ? kBf16NormRing
                                                  : kNormRing;
  const int third = !a.f ? 0 : s.teams == 1 ? kTeamSmem : s.teams < 10 ? kGatedThird : 0;
  // The teams' sums go through the rings' space: 4 bytes a feature and team.
  return finish_geom(*g, s, gain_bytes, a.f && s.vectors == 2 ? 1 : 2, ring, third) &&
         g->nst * g->stage_bytes >= 4 * a.d;
}

struct Plan {
  TeamGeom g;
  int64_t ctas;
  float* sums;
  float* shared;
  cudaStream_t s;
  int gate;
};

template <typename F, typename X, typename G, int GATE>
cudaError_t launch_gate(const ResidualBwdArgs& a, const Plan& p) {
  const int v = shape_of(a).vectors;
  if (v == 1) return launch_teams(residual_bwd_kernel<F, X, G, GATE, 1>, p.g, p.ctas, p.s, a, p.g, p.sums, p.shared);
  // (Rows of fewer bytes leave room for two beside both gains.)
  if constexpr (GATE == kTokenGate || 2 * sizeof(F) + sizeof(X) + sizeof(G) > 10)
    if (p.g.far_gain)
      return launch_teams(residual_bwd_kernel<F, X, G, GATE, 2, true>, p.g, p.ctas, p.s, a, p.g, p.sums, p.shared);
  if (p.g.far_gain) return cudaErrorInvalidValue;
  if (v == 2) return launch_teams(residual_bwd_kernel<F, X, G, GATE, 2>, p.g, p.ctas, p.s, a, p.g, p.sums, p.shared);
  if constexpr (GATE != kSharedGate)
    return launch_teams(residual_bwd_kernel<F, X, G, GATE, 3>, p.g, p.ctas, p.s, a, p.g, p.sums, p.shared);
  return cudaErrorInvalidValue;
}
template <typename F, typename X, typename G>
cudaError_t launch_typed(const ResidualBwdArgs& a, const Plan& p) {
  if (p.gate == kNoGate) return launch_gate<F, X, G, kNoGate>(a, p);
  return p.gate == kTokenGate ? launch_gate<F, X, G, kTokenGate>(a, p) : launch_gate<F, X, G, kSharedGate>(a, p);
}
template <typename F, typename G>
cudaError_t launch_norm(const ResidualBwdArgs& a, const Plan& p) {
  const int v = shape_of(a).vectors;
  if (v == 1) return launch_teams(rmsnorm_bwd_kernel<F, G, 1>, p.g, p.ctas, p.s, a, p.g, p.sums);
  if (v == 2) return launch_teams(rmsnorm_bwd_kernel<F, G, 2>, p.g, p.ctas, p.s, a, p.g, p.sums);
  if constexpr (sizeof(F) == 2 && sizeof(G) == 2)
    return launch_teams(rmsnorm_bwd_kernel<F, G, 3>, p.g, p.ctas, p.s, a, p.g, p.sums);
  return cudaErrorInvalidValue;
}

}  // namespace

bool residual_bwd_fast_ok(const ResidualBwdArgs& a) {
  TeamGeom g;
  return a.T > 0 && a.d % 8 == 0 && a.d <= kMaxTeamD && aligned16(a.f) && aligned16(a.gate) && aligned16(a.gpost) &&
         aligned16(a.xo) && aligned16(a.gpre) && aligned16(a.dxo) && aligned16(a.dn) && aligned16(a.df) &&
         aligned16(a.dx) && aligned16(a.dgate) && geom_of(a, &g);
}

// Enough for any gate of these rows, and with gate_rows 1 for the backward of
// RMSNorm: that of the shape with the fewest teams, so the most CTAs.
int64_t residual_bwd_fast_scratch(int64_t T, int d, int64_t gate_rows) {
  if (T == 0 || d % 8 != 0 || d > kMaxTeamD) return 0;
  const int gate = gate_kind(T, gate_rows, true);
  TeamShape s = gated_shape(T, d, gate);
  for (const bool all_bf16 : {false, true}) {
    const TeamShape n = norm_shape(T, d, all_bf16);
    if (gate == kTokenGate && n.teams < s.teams) s = n;
  }
  const int64_t ctas = team_ctas(T, s, kMaxCtas);
  return 3 * ctas * d + (gate == kSharedGate ? ctas * s.teams * 2 * d : 0);
}

int residual_bwd_parts(const ResidualBwdArgs& a) {
  return static_cast<int>(team_ctas(a.T, shape_of(a), cta_cap()));
}

cudaError_t launch_residual_bwd_fast(const ResidualBwdArgs& a, cudaStream_t s) {
  Plan p{{}, residual_bwd_parts(a), a.scratch, nullptr, s, gate_kind(a.T, a.gate_rows, a.gate != nullptr)};
  if (!geom_of(a, &p.g)) return cudaErrorInvalidValue;
  if (residual_bwd_shares_gates(a)) p.shared = p.sums + 3 * p.ctas * a.d;
  if (!a.f) {
    if (!a.f_bf16) return launch_norm<float, float>(a, p);
    return a.dx_bf16 ? launch_norm<bf16, bf16>(a, p) : launch_norm<bf16, float>(a, p);
  }
  if (!a.f_bf16) return launch_typed<float, float, float>(a, p);
  if (a.x_bf16) return a.dx_bf16 ? launch_typed<bf16, bf16, bf16>(a, p) : launch_typed<bf16, bf16, float>(a, p);
  return a.dx_bf16 ? launch_typed<bf16, float, bf16>(a, p) : launch_typed<bf16, float, float>(a, p);
}

ResidualJoin residual_bwd_join(const ResidualBwdArgs& a) {
  ResidualJoin j;
  if (!residual_bwd_shares_gates(a)) return j;
  const int64_t ctas = residual_bwd_parts(a), groups = (a.T - 1) / a.gate_rows + 1;
  j.part = a.scratch + 3 * ctas * a.d;
  j.teams = ctas * shape_of(a).teams;
  // Rows that many teams had tokens of take many lanes to a sum; where they are
  // many themselves, that is more blocks than it gains (32768 x 896 with rows of 256
  // tokens: 126 us by rows, 96 by teams).
  j.by_group = groups <= j.teams / 16;
  j.blocks = j.by_group ? groups * ((a.d - 1) / 32 + 1) : (j.teams - 1) * ((a.d - 1) / 1024 + 1);
  return j;
}

cudaError_t take_timeout_residual_bwd(unsigned int* flag) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(flag, g_timeout, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_timeout, &zero, sizeof(unsigned int));
}

}  // namespace attnres
