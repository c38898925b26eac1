// Teams of warps that stream rows: what the fast kernels of the gated residual
// and its backward share.
//
// A CTA holds several teams; each takes a run of consecutive rows, one at a
// time. The team's first thread keeps a ring of rows in flight with bulk copies
// (one per input array and row), so the next rows' loads pass under this row's
// sums over the team and no thread holds registers for loads on their way.
#pragma once

#include "common.cuh"
#include "internal.h"
#include "residual.cuh"

namespace attnres {

constexpr int kMaxCtas = 152;          // one per SM of a GB300; bounds the scratch
constexpr int kMaxTeamD = 8192;
constexpr int kMaxStages = 8;
constexpr int kRedOff = 2048;          // after the barriers (at most 32 teams x 8 stages)
constexpr int kRedFloats = 32;         // of a team, for every 4 warps: 2 x 4 values x 4
constexpr int kTeamSmem = 227 * 1024;

struct TeamGeom {
  int warps, teams, nst, stage_bytes, total;
  int n;                      // input arrays of a stage
  const unsigned char* src[5];
  int bytes[5], off[5];       // of one row
  int f, x, dxo, dn, gate;    // offsets in a stage of what is there
  int gain, stages;           // where gains kept in shared memory and the rings begin
  int far_gain;               // gamma_pre is not kept
  int64_t withhold;
};

// How a CTA of up to max_warps warps is cut into teams whose threads take
// 8 * vectors features of a row.
struct TeamShape {
  int vectors, warps, teams;
};
inline TeamShape team_shape(int64_t T, int d, int vectors, int max_warps) {
  TeamShape s;
  s.vectors = vectors;
  s.warps = (d - 1) / (256 * vectors) + 1;
  s.teams = max_warps / s.warps;
  // Teams of several warps meet at named barriers, of which there are 15.
  if (s.warps > 1 && s.teams > 15) s.teams = 15;
  // With few rows every SM gets a CTA before any gets a second team.
  const int64_t each = T > 0 ? (T - 1) / kMaxCtas + 1 : 1;
  if (s.teams > each) s.teams = static_cast<int>(each);
  return s;
}
// 16 features a thread halve the cost of the sums over the team (65536 x 1024 bf16
// at 96 % of the copy bandwidth, with 8 at 85), where not too many lanes idle.
inline bool sixteen_pay(int d) {
  const int w1 = (d - 1) / 256 + 1, w2 = (d - 1) / 512 + 1;
  return 10 * w1 > 15 * w2;  // fill(16) * 1.33 > fill(8), fills being d / (256 w1) and d / (512 w2)
}
inline int64_t team_ctas(int64_t T, const TeamShape& s, int64_t cap) {
  const int64_t want = (T - 1) / s.teams + 1;
  return want < cap ? want : cap;
}
inline int64_t cta_cap() {
  const int n = sm_count();
  return n < kMaxCtas ? n : kMaxCtas;
}

inline void add_input(TeamGeom& g, const void* p, int bytes, int* at) {
  *at = g.stage_bytes;
  if (!p) return;
  g.src[g.n] = static_cast<const unsigned char*>(p);
  g.bytes[g.n] = bytes;
  g.off[g.n++] = g.stage_bytes;
  g.stage_bytes += bytes;
}
// What lies before the rings and the gains: the barriers, and the sums of teams of several warps.
inline int rows_offset(const TeamShape& s) {
  return kRedOff + (s.warps > 1 ? s.teams * ((s.warps + 3) / 4) * kRedFloats * 4 : 0);
}
// Cuts the teams' rings out of `budget` bytes of shared memory, or of all of it
// where the budget does not hold two rows; false if that does not hold `least`. A
// third row of every team may take up to `third` bytes.
inline bool finish_geom(TeamGeom& g, const TeamShape& s, int gain_bytes, int least, int budget, int third) {
  g.warps = s.warps;
  g.teams = s.teams;
  g.gain = rows_offset(s);
  g.stages = g.gain + gain_bytes;
  const int most = (kTeamSmem - g.stages) / (g.teams * g.stage_bytes);
  g.nst = budget / (g.teams * g.stage_bytes);
  if (g.nst < 3 && most >= 3 && 3 * g.teams * g.stage_bytes <= third) g.nst = 3;
  if (g.nst < 2) g.nst = 2;
  if (g.nst > most) g.nst = most;
  if (g.nst > kMaxStages) g.nst = kMaxStages;
  g.total = g.stages + g.nst * g.teams * g.stage_bytes;
  g.withhold = withhold_for(kWithholdResidual);
  return g.nst >= least;
}

#ifdef __CUDACC__

// ------------------------------------------------------- 8 features at a time --

struct V8 {
  float2 p[4];
};
__device__ __forceinline__ V8 fill8(float c) {
  V8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = make_float2(c, c);
  return r;
}
__device__ __forceinline__ V8 ld8(const bf16* p) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  V8 r;
  r.p[0] = make_float2(bf16_lo(v.x), bf16_hi(v.x));
  r.p[1] = make_float2(bf16_lo(v.y), bf16_hi(v.y));
  r.p[2] = make_float2(bf16_lo(v.z), bf16_hi(v.z));
  r.p[3] = make_float2(bf16_lo(v.w), bf16_hi(v.w));
  return r;
}
__device__ __forceinline__ V8 ld8(const float* p) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  V8 r;
  r.p[0] = make_float2(a.x, a.y);
  r.p[1] = make_float2(a.z, a.w);
  r.p[2] = make_float2(b.x, b.y);
  r.p[3] = make_float2(b.z, b.w);
  return r;
}
__device__ __forceinline__ V8 ld8(const void* p, int64_t i, int is_bf16) {
  return is_bf16 ? ld8(static_cast<const bf16*>(p) + i) : ld8(static_cast<const float*>(p) + i);
}
__device__ __forceinline__ void st8(bf16* p, const V8& x) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x.p[0].x, x.p[0].y), pack_bf16x2(x.p[1].x, x.p[1].y),
                                            pack_bf16x2(x.p[2].x, x.p[2].y), pack_bf16x2(x.p[3].x, x.p[3].y));
}
__device__ __forceinline__ void st8(float* p, const V8& x) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x.p[0].x, x.p[0].y, x.p[1].x, x.p[1].y);
  reinterpret_cast<float4*>(p)[1] = make_float4(x.p[2].x, x.p[2].y, x.p[3].x, x.p[3].y);
}
// Results, in global memory: written once, so marked to leave the L2 first, as
// the rows read are. Either mark alone did nothing; with both, 131072 x 2048
// forward took 7 % less (calls that the L2 holds keep their results in it all the
// same). Measured alone: not with the kernel that reads the results after it.
__device__ __forceinline__ void out8(bf16* p, const V8& x) {
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack_bf16x2(x.p[0].x, x.p[0].y), pack_bf16x2(x.p[1].x, x.p[1].y),
                                                 pack_bf16x2(x.p[2].x, x.p[2].y), pack_bf16x2(x.p[3].x, x.p[3].y)));
}
__device__ __forceinline__ void out8(float* p, const V8& x) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(x.p[0].x, x.p[0].y, x.p[1].x, x.p[1].y));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x.p[2].x, x.p[2].y, x.p[3].x, x.p[3].y));
}
__device__ __forceinline__ void out8(void* p, int64_t i, int is_bf16, const V8& x) {
  if (is_bf16)
    out8(static_cast<bf16*>(p) + i, x);
  else
    out8(static_cast<float*>(p) + i, x);
}
__device__ __forceinline__ V8 mul8(const V8& a, const V8& b) {
  V8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = fmul2(a.p[i], b.p[i]);
  return r;
}
__device__ __forceinline__ V8 add8(const V8& a, const V8& b) {
  V8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = make_float2(a.p[i].x + b.p[i].x, a.p[i].y + b.p[i].y);
  return r;
}
__device__ __forceinline__ V8 mul8(const V8& a, float b) { return mul8(a, fill8(b)); }
__device__ __forceinline__ V8 fma8(const V8& a, const V8& b, const V8& c) {
  V8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = ffma2(a.p[i], b.p[i], c.p[i]);
  return r;
}
__device__ __forceinline__ V8 fma8(const V8& a, float b, const V8& c) { return fma8(a, fill8(b), c); }
// sum_k a_k b_k of the thread's 8 features.
__device__ __forceinline__ float dot8(const V8& a, const V8& b) {
  float2 s = fmul2(a.p[0], b.p[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = ffma2(a.p[i], b.p[i], s);
  return s.x + s.y;
}
// The gate's values, and with SLOPE their derivatives.
template <bool SLOPE>
__device__ __forceinline__ void activate8(V8& g, V8& slope, int is_sigmoid) {
  if (is_sigmoid) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 s;
      g.p[i] = sigmoid2(g.p[i], &s);
      if (SLOPE) slope.p[i] = s;
    }
  } else if (SLOPE) {
    slope = fill8(1.f);
  }
}
enum GateKind { kNoGate = 0, kTokenGate = 1, kSharedGate = 2 };

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
  float* red;                  // [2][4][warps, a multiple of 4]
  uint32_t bars;
  unsigned char* ring;
  int64_t r0;                  // first row
  int rows, stride;            // how many, and how far apart
  int issued, next;            // rows whose copies were started; the next one's stage (first thread only)
};

// The team's rows: a run of consecutive ones, or every so manyth one, with all
// teams of the grid walking through the same stretch of memory.
template <bool INTERLEAVED>
__device__ __forceinline__ Team make_team(const TeamGeom& g, int64_t T, unsigned char* smem) {
  Team m;
  m.warps = g.warps;
  m.team = static_cast<int>(threadIdx.x) / (g.warps * 32);
  m.tid = static_cast<int>(threadIdx.x) % (g.warps * 32);
  m.nst = g.nst;
  m.red = reinterpret_cast<float*>(smem + kRedOff) + m.team * kRedFloats * ((g.warps + 3) / 4);
  m.bars = smem_u32(smem) + m.team * g.nst * 8;
  m.ring = smem + g.stages + static_cast<size_t>(m.team) * g.nst * g.stage_bytes;
  const int64_t all = static_cast<int64_t>(gridDim.x) * g.teams;
  if (INTERLEAVED) {
    // By turns over the CTAs first: the last rows then spread over all SMs.
    const int64_t id = static_cast<int64_t>(m.team) * gridDim.x + blockIdx.x;
    m.r0 = id;
    m.rows = T > id ? static_cast<int>((T - id - 1) / all + 1) : 0;
    m.stride = static_cast<int>(all);
  } else {
    const int64_t id = static_cast<int64_t>(blockIdx.x) * g.teams + m.team;
    m.r0 = T * id / all;
    m.rows = static_cast<int>(T * (id + 1) / all - m.r0);
    m.stride = 1;
  }
  m.issued = m.next = 0;
  return m;
}

__device__ __forceinline__ void init_bars(const TeamGeom& g, unsigned char* smem) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < g.teams * g.nst; ++i) mbar_init(smem_u32(smem) + i * 8, 1);
    mbar_fence_init();
  }
  float* red = reinterpret_cast<float*>(smem + kRedOff);
  for (int i = threadIdx.x; i < (g.gain - kRedOff) / 4; i += blockDim.x) red[i] = 0.f;
  __syncthreads();
}

// A bulk copy of bytes that are read once: they leave the L2 first.
__device__ __forceinline__ void bulk_g2s_once(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  uint64_t policy;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar), "l"(policy)
      : "memory");
}

// Starts the copies of the next row of the team's run (its first thread only).
__device__ __forceinline__ void issue_row(Team& m, const TeamGeom& g) {
  const int s = m.next;
  m.next = s + 1 == m.nst ? 0 : s + 1;
  if (m.issued != g.withhold) {  // the test hook leaves this row out
    const uint32_t bar = m.bars + s * 8, dst = smem_u32(m.ring) + s * g.stage_bytes;
    mbar_arrive_expect_tx(bar, g.stage_bytes);
    const int64_t row = m.r0 + static_cast<int64_t>(m.issued) * m.stride;
    for (int i = 0; i < g.n; ++i) bulk_g2s_once(dst + g.off[i], g.src[i] + row * g.bytes[i], g.bytes[i], bar);
  }
  ++m.issued;
}
__device__ __forceinline__ void fill_ring(Team& m, const TeamGeom& g) {
  if (m.tid == 0)
    while (m.issued < m.rows && m.issued < m.nst) issue_row(m, g);
}

// After a wait for row r that ran out: records it and lets the copies in flight land.
__device__ __forceinline__ void give_up(const Team& m, const TeamGeom& g, int r, unsigned int* flag) {
  if (m.tid != 0) return;
  atomicOr(flag, 1u);
  for (; r < m.issued; ++r)
    if (r != g.withhold) (void)mbar_wait(m.bars + r % m.nst * 8, static_cast<uint32_t>(r / m.nst & 1));
}

// Sums of N (2 or 4) values over the team; every thread gets them. Also a
// barrier of the team, which agrees on `ok`. Consecutive calls take the two
// `buf`s in turn. In a warp the lanes' halves (and then quarters) each take one
// of the values that are left, so 4 values cost 6 shuffles and not 20; lanes
// 0, 16, 8 and 24 end with them.
template <int N>
__device__ __forceinline__ bool team_sum(const Team& m, float (&v)[N], int buf, bool ok) {
  static_assert(N == 2 || N == 4, "two or four values");
  const int lane = m.tid & 31;
  const bool upper = lane & 16, odd = lane & 8;
  float c = (upper ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, upper ? v[0] : v[1], 16);
  if constexpr (N == 4) {
    const float b = (upper ? v[3] : v[2]) + __shfl_xor_sync(0xffffffffu, upper ? v[2] : v[3], 16);
    c = (odd ? b : c) + __shfl_xor_sync(0xffffffffu, odd ? c : b, 8);
  } else {
    c += __shfl_xor_sync(0xffffffffu, c, 8);
  }
  c += __shfl_xor_sync(0xffffffffu, c, 4);
  c += __shfl_xor_sync(0xffffffffu, c, 2);
  c += __shfl_xor_sync(0xffffffffu, c, 1);
  if (m.warps == 1) {
    v[0] = __shfl_sync(0xffffffffu, c, 0);
    v[1] = __shfl_sync(0xffffffffu, c, 16);
    if constexpr (N > 2) {
      v[2] = __shfl_sync(0xffffffffu, c, 8);
      v[3] = __shfl_sync(0xffffffffu, c, 24);
    }
    ok = __all_sync(0xffffffffu, ok);
    __syncwarp();  // orders the warp's reads of the stage before its refill
    return ok;
  }
  // [value][warp], the warps padded with zeros to a multiple of 4.
  const int quads = (m.warps + 3) >> 2;
  float* red = m.red + buf * 16 * quads;
  if ((lane & (32 / N - 1)) == 0) red[((lane >> 4) + (lane >> 2 & 2)) * 4 * quads + (m.tid >> 5)] = c;
  ok = named_all(m.team + 1, m.warps * 32, ok);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
  for (int w = 0; w < quads; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float4 o = reinterpret_cast<const float4*>(red)[i * quads + w];
      v[i] += (o.x + o.y) + (o.z + o.w);
    }
  return ok;
}
__device__ __forceinline__ void team_sync(const Team& m) {
  if (m.warps == 1)
    __syncwarp();
  else
    named_sync(m.team + 1, m.warps * 32);
}

#endif  // __CUDACC__

template <typename K, typename... Args>
cudaError_t launch_teams(K kernel, const TeamGeom& g, int64_t ctas, cudaStream_t s, const Args&... args) {
  cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(kernel), g.total);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, static_cast<unsigned>(ctas), static_cast<unsigned>(g.teams * g.warps * 32), g.total, s,
                    args...);
}

}  // namespace attnres
