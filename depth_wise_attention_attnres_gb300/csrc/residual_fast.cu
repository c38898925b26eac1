// The gated residual and its backward for d a multiple of 8 up to 8192 with
// aligned rows (the formulas stand at the top of residual.cu).
//
// Both are bound by memory: every row is read once and written once, and the
// two means per row need nothing that is not in the row. A CTA holds several
// teams of warps; each team takes a run of consecutive rows, one at a time,
// with 8 features (16 past d = 4096) per thread. The team's first thread keeps
// a ring of rows in flight with bulk copies (one per input array and row), so
// the loads of the next rows pass under the two sums over the team of this
// one, and no thread holds registers for loads that are still on their way.
// A stage is refilled after the next row's first sum: by then every thread of
// the team has passed its last read of it, so the ring needs no barriers of
// its own.
//
// Backward: the sums over tokens stay in registers for the whole run of rows
// (a thread's features never change), are added over the CTA's teams in shared
// memory and leave one partial row per CTA.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "residual.cuh"

namespace attnres {
namespace {

__device__ unsigned int g_residual_timeout = 0;

constexpr int kMaxWarps = 16;          // of a CTA
constexpr int kMaxCtas = 152;          // one per SM of a GB300; bounds the scratch
constexpr int kMaxD = 8192;
constexpr int kMaxStages = 8;
constexpr int kRedOff = 1024;          // after the barriers (at most 16 teams x 8 stages)
constexpr int kStageOff = 2048;        // after the teams' sums (3 x 16 warps x 4 floats)
constexpr int kSmem = 227 * 1024;

struct TeamGeom {
  int warps, teams, nst, stage_bytes, total;
  int n;                      // input arrays of a stage
  const unsigned char* src[5];
  int bytes[5], off[5];       // of one row
  int f, x, dxo, dn, gate;    // offsets in a stage of what is there
  int64_t withhold;
};

int vectors_of(int d) { return d <= 4096 ? 1 : 2; }
int warps_of(int d) { return (d - 1) / (256 * vectors_of(d)) + 1; }
// Teams of several warps meet at named barriers, of which there are 15 to use.
int teams_of(int d) {
  const int t = kMaxWarps / warps_of(d);
  return t < 1 ? 1 : t;
}
unsigned ctas_of(int64_t T, int d) {
  const int64_t want = (T - 1) / teams_of(d) + 1;
  const int64_t cap = sm_count() < kMaxCtas ? sm_count() : kMaxCtas;
  return static_cast<unsigned>(want < cap ? want : cap);
}

void add_input(TeamGeom& g, const void* p, int bytes, int* at) {
  *at = g.stage_bytes;
  if (!p) return;
  g.src[g.n] = static_cast<const unsigned char*>(p);
  g.bytes[g.n] = bytes;
  g.off[g.n++] = g.stage_bytes;
  g.stage_bytes += bytes;
}
// Splits `smem` bytes into the teams' rings; false if not even one row fits.
bool finish_geom(TeamGeom& g, int d, int smem) {
  g.warps = warps_of(d);
  g.teams = teams_of(d);
  g.nst = (smem - kStageOff) / (g.teams * g.stage_bytes);
  if (g.nst > kMaxStages) g.nst = kMaxStages;
  g.total = kStageOff + g.nst * g.teams * g.stage_bytes;
  g.withhold = withhold_for(kWithholdResidual);
  return g.nst >= 1;
}

// ---------------------------------------------------------------- a team ----

// Whether every thread of `count` (a named barrier's) passes ok.
__device__ __forceinline__ bool named_all(int id, int count, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n"
      " setp.ne.u32 p, %1, 0;\n"
      " barrier.cta.red.and.pred q, %2, %3, p;\n"
      " selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(ok)), "r"(id), "r"(count)
      : "memory");
  return r != 0;
}

struct Team {
  int warps, team, tid, nst;
  float4* red;                 // [3][warps]
  uint32_t bars;
  unsigned char* ring;
  int64_t r0;                  // first row
  int rows;
  int issued, next;            // rows whose copies were started; the next one's stage
};

__device__ __forceinline__ Team make_team(const TeamGeom& g, int64_t T, unsigned char* smem) {
  Team m;
  m.warps = g.warps;
  m.team = static_cast<int>(threadIdx.x) / (g.warps * 32);
  m.tid = static_cast<int>(threadIdx.x) % (g.warps * 32);
  m.nst = g.nst;
  m.red = reinterpret_cast<float4*>(smem + kRedOff) + m.team * 3 * g.warps;
  m.bars = smem_u32(smem) + m.team * g.nst * 8;
  m.ring = smem + kStageOff + static_cast<size_t>(m.team) * g.nst * g.stage_bytes;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * g.teams + m.team;
  const int64_t all = static_cast<int64_t>(gridDim.x) * g.teams;
  m.r0 = T * id / all;
  m.rows = static_cast<int>(T * (id + 1) / all - m.r0);
  m.issued = m.next = 0;
  return m;
}

// Starts the copies of the next row of the team's run (its first thread only).
__device__ __forceinline__ void issue_row(Team& m, const TeamGeom& g) {
  const int s = m.next;
  m.next = s + 1 == m.nst ? 0 : s + 1;
  if (m.issued != g.withhold) {  // the test hook leaves this row out
    const uint32_t bar = m.bars + s * 8, dst = smem_u32(m.ring) + s * g.stage_bytes;
    mbar_arrive_expect_tx(bar, g.stage_bytes);
    for (int i = 0; i < g.n; ++i)
      bulk_g2s(dst + g.off[i], g.src[i] + (m.r0 + m.issued) * g.bytes[i], g.bytes[i], bar);
  }
  ++m.issued;
}

// After a wait for row r that ran out: records it and lets the copies in flight land.
__device__ __forceinline__ void give_up(const Team& m, const TeamGeom& g, int r) {
  if (m.tid != 0) return;
  atomicOr(&g_residual_timeout, 1u);
  for (; r < m.issued; ++r)
    if (r != g.withhold) (void)mbar_wait(m.bars + r % m.nst * 8, static_cast<uint32_t>(r / m.nst & 1));
}

// Sums over the team; every thread gets them. Also a barrier of the team, which
// agrees on `ok`. Consecutive calls take different `buf`s (0..2).
__device__ __forceinline__ bool team_sum(const Team& m, float4& v, int n, int buf, bool ok) {
  v.x = warp_sum(v.x);
  if (n > 1) {
    v.y = warp_sum(v.y);
    v.z = warp_sum(v.z);
  }
  if (m.warps == 1) return __all_sync(0xffffffffu, ok);
  float4* red = m.red + buf * m.warps;
  if ((m.tid & 31) == 0) red[m.tid >> 5] = v;
  ok = named_all(m.team + 1, m.warps * 32, ok);
  v = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int w = 0; w < m.warps; ++w) {
    const float4 o = red[w];
    v.x += o.x;
    v.y += o.y;
    v.z += o.z;
  }
  return ok;
}
__device__ __forceinline__ void team_sync(const Team& m) {
  if (m.warps == 1)
    __syncwarp();
  else
    named_sync(m.team + 1, m.warps * 32);
}

// 8 consecutive elements of either type.
__device__ __forceinline__ void load8(const void* base, int k, int is_bf16, float (&x)[8]) {
  if (is_bf16) {
    lds16(static_cast<const bf16*>(base) + k, x);
  } else {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + k);
    const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + k + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
}
__device__ __forceinline__ void store8(void* base, int64_t i, int is_bf16, const float (&x)[8]) {
  if (is_bf16) {
    *reinterpret_cast<uint4*>(static_cast<bf16*>(base) + i) =
        make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  } else {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// The gate's values (and slopes) at 8 features.
enum GateKind { kNoGate = 0, kTokenGate = 1, kSharedGate = 2 };
template <bool SLOPE>
__device__ __forceinline__ void activate(float (&g)[8], float (&slope)[8], int is_sigmoid) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (is_sigmoid) {
      float s;
      g[e] = sigmoid(g[e], &s);
      if (SLOPE) slope[e] = s;
    } else if (SLOPE) {
      slope[e] = 1.f;
    }
  }
}

__device__ __forceinline__ void init_bars(const TeamGeom& g, unsigned char* smem) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < g.teams * g.nst; ++i) mbar_init(smem_u32(smem) + i * 8, 1);
    mbar_fence_init();
  }
  __syncthreads();
}

// --------------------------------------------------------------- forward ----

template <int VPT, int GATE>
__global__ void __launch_bounds__(kMaxWarps * 32, 1) residual_fast_kernel(ResidualArgs a, const __grid_constant__ TeamGeom g) {
  extern __shared__ __align__(128) unsigned char smem[];
  init_bars(g, smem);
  Team m = make_team(g, a.T, smem);
  pdl_trigger();
  pdl_wait();
  if (m.tid == 0)
    while (m.issued < m.rows && m.issued < m.nst) issue_row(m, g);
  const int d = a.d, step = m.warps * 256;
  const float inv_d = 1.0f / static_cast<float>(d);
  // The shared gate row of the current token, and the first token of the next one.
  int64_t group = GATE == kSharedGate ? m.r0 / a.gate_rows : 0;
  int64_t group_end = GATE == kSharedGate && a.gate_rows < a.T ? (group + 1) * a.gate_rows : a.T;

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
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (ok && a.gpost) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int k = v * step + m.tid * 8;
        if (k < d) {
          float f[8];
          load8(st + g.f, k, a.f_bf16, f);
#pragma unroll
          for (int e = 0; e < 8; ++e) s.x = fmaf(f[e], f[e], s.x);
        }
      }
    }
    ok = team_sum(m, s, 1, r & 1, ok);
    if (!ok) {
      give_up(m, g, r);
      break;
    }
    // The stage of the row before is free: every thread is past that row.
    if (m.tid == 0 && r > 0 && m.nst > 1 && m.issued < m.rows) issue_row(m, g);
    const float rf = a.gpost ? rsqrtf(s.x * inv_d + a.eps_post) : 1.f;

    float x[VPT][8];
    s.x = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int k = v * step + m.tid * 8;
      if (k < d) {
        float f[8], c[8], unused[8];
        load8(st + g.f, k, a.f_bf16, f);
        if (a.gpost) {
          load8(a.gpost, k, 0, c);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] *= rf * c[e];
        }
        if (a.x) {
          load8(st + g.x, k, a.x_bf16, x[v]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[v][e] = 0.f;
        }
        if (GATE != kNoGate) {
          if (GATE == kTokenGate)
            load8(st + g.gate, k, a.g_bf16, c);
          else
            load8(static_cast<const unsigned char*>(a.gate) + group * d * (a.g_bf16 ? 2 : 4), k, a.g_bf16, c);
          activate<false>(c, unused, a.sigmoid);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[v][e] = fmaf(a.scale * c[e], f[e], x[v][e]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[v][e] = fmaf(a.scale, f[e], x[v][e]);
        }
        store8(a.x_out, row * d + k, a.x_bf16, x[v]);
#pragma unroll
        for (int e = 0; e < 8; ++e) s.x = fmaf(x[v][e], x[v][e], s.x);
      }
    }
    if (a.normed) {
      (void)team_sum(m, s, 1, 2, true);
      const float rx = rsqrtf(s.x * inv_d + a.eps_pre);
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int k = v * step + m.tid * 8;
        if (k < d) {
          float c[8];
          load8(a.gpre, k, 0, c);
#pragma unroll
          for (int e = 0; e < 8; ++e) c[e] *= x[v][e] * rx;
          store8(a.normed, row * d + k, a.f_bf16, c);
        }
      }
    }
    // A ring of one stage: the next row's copies start when all are done with this one.
    if (m.nst == 1 && r + 1 < m.rows) {
      team_sync(m);
      if (m.tid == 0) issue_row(m, g);
    }
  }
}

// -------------------------------------------------------------- backward ----

// Writes (or keeps, for the kernel that joins them) the sum of a gate row over
// the team's rows [from, to) of it.
template <int VPT>
__device__ __forceinline__ void flush_gate(const ResidualBwdArgs& a, const Team& m, float* shared_part, int teams,
                                           int64_t group, float (&acc)[VPT][8]) {
  const int64_t start = group * a.gate_rows;
  const int64_t end = a.gate_rows < a.T - start ? start + a.gate_rows : a.T;
  const bool whole = start >= m.r0 && end <= m.r0 + m.rows;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * teams + m.team;
  float* part = shared_part + (id * 2 + (start < m.r0 ? 0 : 1)) * a.d;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int k = v * m.warps * 256 + m.tid * 8;
    if (k < a.d) {
      if (whole) {
        store8(a.dgate, group * a.d + k, a.g_bf16, acc[v]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) part[k + e] = acc[v][e];
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[v][e] = 0.f;
  }
}

// sums: partial rows [3][gridDim.x][d] (dgamma_post, dgamma_pre, the one gate
// row of all tokens); shared_part: [teams of the grid][2][d] for gate rows that
// runs of tokens share (nullptr when there are none to sum).
template <int VPT, int GATE, bool HAS_F>
__global__ void __launch_bounds__(kMaxWarps * 32, 1)
    residual_bwd_fast_kernel(ResidualBwdArgs a, const __grid_constant__ TeamGeom g, float* sums, float* shared_part) {
  extern __shared__ __align__(128) unsigned char smem[];
  init_bars(g, smem);
  Team m = make_team(g, a.T, smem);
  pdl_trigger();
  pdl_wait();
  if (m.tid == 0)
    while (m.issued < m.rows && m.issued < m.nst) issue_row(m, g);
  const int d = a.d, step = m.warps * 256;
  const float inv_d = 1.0f / static_cast<float>(d);
  float post[VPT][8] = {}, pre[VPT][8] = {}, gsum[VPT][8] = {};
  const bool post_norm = HAS_F && a.gpost != nullptr;
  // The shared gate row of the current token, and the first token of the next one.
  int64_t group = GATE == kSharedGate ? m.r0 / a.gate_rows : 0;
  int64_t group_end = GATE == kSharedGate && a.gate_rows < a.T ? (group + 1) * a.gate_rows : a.T;

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
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (ok) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int k = v * step + m.tid * 8;
        if (k < d) {
          if (a.dn) {
            float x[8], h[8], c[8];
            load8(st + g.x, k, a.x_bf16, x);
            load8(st + g.dn, k, a.f_bf16, h);
            load8(a.gpre, k, 0, c);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              s.x = fmaf(x[e], x[e], s.x);
              s.y = fmaf(c[e] * h[e], x[e], s.y);
            }
          }
          if (post_norm) {
            float f[8];
            load8(st + g.f, k, a.f_bf16, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) s.z = fmaf(f[e], f[e], s.z);
          }
        }
      }
    }
    ok = team_sum(m, s, 3, r & 1, ok);
    if (!ok) {
      give_up(m, g, r);
      break;
    }
    // The stage of the row before is free: every thread is past that row.
    if (m.tid == 0 && r > 0 && m.nst > 1 && m.issued < m.rows) issue_row(m, g);
    const float rx = a.dn ? rsqrtf(s.x * inv_d + a.eps_pre) : 0.f;
    const float mx = rx * (s.y * inv_d);
    const float rf = post_norm ? rsqrtf(s.z * inv_d + a.eps_post) : 1.f;
    const void* gate_row = nullptr;
    if (GATE == kTokenGate) gate_row = st + g.gate;
    if (GATE == kSharedGate)
      gate_row = static_cast<const unsigned char*>(a.gate) + group * d * (a.g_bf16 ? 2 : 4);

    float D[VPT][8];
    s.x = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int k = v * step + m.tid * 8;
      if (k < d) {
        if (a.dxo) {
          load8(st + g.dxo, k, a.dx_bf16, D[v]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) D[v][e] = 0.f;
        }
        if (a.dn) {
          float x[8], h[8], c[8];
          load8(st + g.x, k, a.x_bf16, x);
          load8(st + g.dn, k, a.f_bf16, h);
          load8(a.gpre, k, 0, c);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float u = x[e] * rx;
            D[v][e] = fmaf(rx, c[e] * h[e] - u * mx, D[v][e]);
            pre[v][e] = fmaf(h[e], u, pre[v][e]);
          }
        }
        if (a.dx) store8(a.dx, row * d + k, a.dx_bf16, D[v]);
        if (post_norm) {
          float f[8], c[8], act[8], slope[8];
          load8(st + g.f, k, a.f_bf16, f);
          load8(a.gpost, k, 0, c);
          if (GATE != kNoGate) {
            load8(gate_row, k, a.g_bf16, act);
            activate<false>(act, slope, a.sigmoid);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float dy = (GATE != kNoGate ? a.scale * act[e] : a.scale) * D[v][e];
            s.x = fmaf(c[e] * dy, f[e] * rf, s.x);
          }
        }
      }
    }
    if (HAS_F) {
      float mf = 0.f;
      if (post_norm) {
        (void)team_sum(m, s, 1, 2, true);
        mf = s.x * inv_d;
      }
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int k = v * step + m.tid * 8;
        if (k < d) {
          float f[8], c[8], act[8], slope[8], df[8];
          load8(st + g.f, k, a.f_bf16, f);
          if (a.gpost) {
            load8(a.gpost, k, 0, c);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) c[e] = 1.f;
          }
          if (GATE != kNoGate) {
            load8(gate_row, k, a.g_bf16, act);
            activate<true>(act, slope, a.sigmoid);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float q = f[e] * rf, cq = c[e] * q;
            const float dy = (GATE != kNoGate ? a.scale * act[e] : a.scale) * D[v][e];
            df[e] = rf * (c[e] * dy - q * mf);
            post[v][e] = fmaf(dy, q, post[v][e]);
            if (GATE == kTokenGate) act[e] = a.scale * slope[e] * cq * D[v][e];
            if (GATE == kSharedGate) gsum[v][e] = fmaf(a.scale * slope[e] * cq, D[v][e], gsum[v][e]);
          }
          if (a.df) store8(a.df, row * d + k, a.f_bf16, df);
          if (GATE == kTokenGate && a.dgate) store8(a.dgate, row * d + k, a.g_bf16, act);
        }
      }
      if (GATE == kSharedGate && shared_part) {
        if (r + 1 == m.rows || row + 1 == group_end) flush_gate<VPT>(a, m, shared_part, g.teams, group, gsum);
      }
    }
    // A ring of one stage: the next row's copies start when all are done with this one.
    if (m.nst == 1 && r + 1 < m.rows) {
      team_sync(m);
      if (m.tid == 0) issue_row(m, g);
    }
  }

  // The CTA's partial rows, its teams added in order. The rings are free: every
  // copy has landed and been read.
  float* buf = reinterpret_cast<float*>(smem + kStageOff);
#pragma unroll
  for (int which = 0; which < 3; ++which) {
    if (which == 0 && !(post_norm && a.dgpost)) continue;
    if (which == 1 && !(a.dn && a.dgpre)) continue;
    if (which == 2 && !(GATE == kSharedGate && a.dgate && !shared_part)) continue;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int k = v * step + m.tid * 8;
      if (k < d) {
        float4* p = reinterpret_cast<float4*>(buf + m.team * d + k);
        const float(&t)[8] = which == 0 ? post[v] : (which == 1 ? pre[v] : gsum[v]);
        p[0] = make_float4(t[0], t[1], t[2], t[3]);
        p[1] = make_float4(t[4], t[5], t[6], t[7]);
      }
    }
    __syncthreads();
    float* part = sums + (static_cast<int64_t>(which) * gridDim.x + blockIdx.x) * d;
    for (int k = threadIdx.x; k < d; k += blockDim.x) {
      float t = 0.f;
      for (int i = 0; i < g.teams; ++i) t += buf[i * d + k];
      part[k] = t;
    }
  }
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
  float s = shared_part[(first * 2 + 1) * a.d + k];
  for (int64_t u = t; u < teams; ++u) {
    const int64_t u0 = a.T * u / teams, u1 = a.T * (u + 1) / teams;
    if (u0 >= end) break;
    if (u0 < u1) s += shared_part[u * 2 * a.d + k];
  }
  if (a.g_bf16)
    static_cast<bf16*>(a.dgate)[group * a.d + k] = from_f32<bf16>(s);
  else
    static_cast<float*>(a.dgate)[group * a.d + k] = s;
}

bool fwd_geom(const ResidualArgs& a, TeamGeom* g) {
  *g = TeamGeom{};
  const int es = a.f_bf16 ? 2 : 4, xs = a.x_bf16 ? 2 : 4;
  add_input(*g, a.f, a.d * es, &g->f);
  add_input(*g, a.x, a.d * xs, &g->x);
  add_input(*g, a.gate && a.gate_rows == 1 ? a.gate : nullptr, a.d * (a.g_bf16 ? 2 : 4), &g->gate);
  return finish_geom(*g, a.d, kSmem);
}

bool bwd_geom(const ResidualBwdArgs& a, TeamGeom* g) {
  *g = TeamGeom{};
  const int es = a.f_bf16 ? 2 : 4, xs = a.x_bf16 ? 2 : 4;
  add_input(*g, a.f, a.d * es, &g->f);
  add_input(*g, a.dn ? a.xo : nullptr, a.d * xs, &g->x);
  add_input(*g, a.dxo, a.d * (a.dx_bf16 ? 2 : 4), &g->dxo);
  add_input(*g, a.dn, a.d * es, &g->dn);
  add_input(*g, a.gate && a.gate_rows == 1 ? a.gate : nullptr, a.d * (a.g_bf16 ? 2 : 4), &g->gate);
  // The teams' sums go through the rings' space: 4 bytes a feature and team.
  return finish_geom(*g, a.d, kSmem) && g->nst * g->stage_bytes >= 4 * a.d;
}

template <typename K, typename... Args>
cudaError_t launch_teams(K kernel, const TeamGeom& g, int64_t T, int d, cudaStream_t s, Args... args) {
  cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(kernel), g.total);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, ctas_of(T, d), static_cast<unsigned>(g.teams * g.warps * 32), g.total, s, args...);
}

template <int VPT>
cudaError_t launch_fwd(const ResidualArgs& a, const TeamGeom& g, cudaStream_t s) {
  if (!a.gate) return launch_teams(residual_fast_kernel<VPT, kNoGate>, g, a.T, a.d, s, a, g);
  if (a.gate_rows == 1) return launch_teams(residual_fast_kernel<VPT, kTokenGate>, g, a.T, a.d, s, a, g);
  return launch_teams(residual_fast_kernel<VPT, kSharedGate>, g, a.T, a.d, s, a, g);
}

template <int VPT>
cudaError_t launch_bwd(const ResidualBwdArgs& a, const TeamGeom& g, float* sums, float* shared, cudaStream_t s) {
  if (!a.f) return launch_teams(residual_bwd_fast_kernel<VPT, kNoGate, false>, g, a.T, a.d, s, a, g, sums, shared);
  if (!a.gate) return launch_teams(residual_bwd_fast_kernel<VPT, kNoGate, true>, g, a.T, a.d, s, a, g, sums, shared);
  if (a.gate_rows == 1)
    return launch_teams(residual_bwd_fast_kernel<VPT, kTokenGate, true>, g, a.T, a.d, s, a, g, sums, shared);
  return launch_teams(residual_bwd_fast_kernel<VPT, kSharedGate, true>, g, a.T, a.d, s, a, g, sums, shared);
}

}  // namespace

bool residual_fast_ok(const ResidualArgs& a) {
  TeamGeom g;
  return a.d % 8 == 0 && a.d <= kMaxD && aligned16(a.f) && aligned16(a.x) && aligned16(a.gate) && aligned16(a.gpost) &&
         aligned16(a.gpre) && aligned16(a.x_out) && aligned16(a.normed) && fwd_geom(a, &g);
}

bool residual_bwd_fast_ok(const ResidualBwdArgs& a) {
  TeamGeom g;
  return a.T > 0 && a.d % 8 == 0 && a.d <= kMaxD && aligned16(a.f) && aligned16(a.gate) && aligned16(a.gpost) &&
         aligned16(a.xo) && aligned16(a.gpre) && aligned16(a.dxo) && aligned16(a.dn) && aligned16(a.df) &&
         aligned16(a.dx) && aligned16(a.dgate) && bwd_geom(a, &g);
}

int64_t residual_bwd_fast_scratch(int64_t T, int d, int64_t gate_rows) {
  if (T == 0 || d % 8 != 0 || d > kMaxD) return 0;
  const int64_t want = (T - 1) / teams_of(d) + 1;
  const int64_t ctas = want < kMaxCtas ? want : kMaxCtas;
  return 3 * ctas * d + (gate_rows > 1 && gate_rows < T ? ctas * teams_of(d) * 2 * d : 0);
}

cudaError_t launch_residual_fast(const ResidualArgs& a, cudaStream_t s) {
  TeamGeom g;
  if (!fwd_geom(a, &g)) return cudaErrorInvalidValue;
  return vectors_of(a.d) == 1 ? launch_fwd<1>(a, g, s) : launch_fwd<2>(a, g, s);
}

int residual_bwd_parts(const ResidualBwdArgs& a) { return static_cast<int>(ctas_of(a.T, a.d)); }

cudaError_t launch_residual_bwd_fast(const ResidualBwdArgs& a, cudaStream_t s) {
  TeamGeom g;
  if (!bwd_geom(a, &g)) return cudaErrorInvalidValue;
  float* sums = a.scratch;
  float* shared = residual_bwd_shares_gates(a) ? sums + 3ll * residual_bwd_parts(a) * a.d : nullptr;
  return vectors_of(a.d) == 1 ? launch_bwd<1>(a, g, sums, shared, s) : launch_bwd<2>(a, g, sums, shared, s);
}

cudaError_t launch_residual_bwd_join_gate(const ResidualBwdArgs& a, cudaStream_t s) {
  const int64_t teams = static_cast<int64_t>(residual_bwd_parts(a)) * teams_of(a.d);
  const float* shared = a.scratch + 3ll * residual_bwd_parts(a) * a.d;
  if (teams < 2) return cudaSuccess;
  return launch_pdl_grid(residual_bwd_join_gate_kernel, dim3(static_cast<unsigned>(teams - 1), (a.d - 1) / 256 + 1), 256, 0,
                         s, a, shared, teams);
}

cudaError_t take_timeout_residual(unsigned int* flag) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(flag, g_residual_timeout, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_residual_timeout, &zero, sizeof(unsigned int));
}

}  // namespace attnres
