// The gated residual, its backward, and the backward of RMSNorm.
//
// Forward, per token: y = gamma_post * f * r_f (r_f = 1 / sqrt(mean f^2 +
// eps_post)), x_out = x + scale * act(gate) * y, normed = gamma_pre * x_out *
// r_x. Two means per row, the second over the result of the first.
// Backward, per token, with u = r_x x_out, q = r_f f and h = gamma_pre dn:
//   D  = dx_out + r_x (h - u mean(h u)),        dy = scale act(gate) D
//   df = r_f (gamma_post dy - q mean(gamma_post dy q))
// and per feature, summed over tokens: dgamma_post += dy q, dgamma_pre += dn u,
// dgate += scale act'(gate) gamma_post q D.
//
// The general kernels take any width and any alignment and go through memory
// once per mean; the sums over tokens go through partial rows in the scratch
// that one more kernel adds in a fixed order.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "residual.cuh"

namespace attnres {
namespace {

constexpr int kThreads = 256;      // general kernels: one row per CTA
constexpr int kColumns = 32;       // column kernels: features of a CTA
constexpr int kLanes = 8;          // and tokens in flight per feature
constexpr int kChunks = 64;        // partial rows of the general column sums

__device__ __forceinline__ float ld(const void* p, int64_t i, int is_bf16) {
  return is_bf16 ? to_f32(static_cast<const bf16*>(p)[i]) : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void st(void* p, int64_t i, int is_bf16, float v) {
  if (is_bf16)
    static_cast<bf16*>(p)[i] = from_f32<bf16>(v);
  else
    static_cast<float*>(p)[i] = v;
}

// Sums of a CTA of kThreads threads; every thread gets them.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  __syncthreads();
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) red[warp * N + i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) v[i] += red[w * N + i];
  }
}

// x + scale * act(gate) * y at one element, given r_f (1 without a post-norm).
__device__ __forceinline__ float residual_at(const ResidualArgs& a, int64_t off, int64_t goff, int k, float rf) {
  float y = ld(a.f, off, a.f_bf16) * rf;
  if (a.gpost) y *= a.gpost[k];
  float c = a.scale;
  if (a.gate) {
    const float g = ld(a.gate, goff, a.g_bf16);
    float slope;
    c *= a.sigmoid ? sigmoid(g, &slope) : g;
  }
  return fmaf(c, y, a.x ? ld(a.x, off, a.x_bf16) : 0.f);
}

__global__ void __launch_bounds__(kThreads) residual_generic_kernel(ResidualArgs a) {
  __shared__ float red[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  const float inv_d = 1.0f / static_cast<float>(a.d);
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t row = t * a.d, grow = t / a.gate_rows * a.d;
    float rf = 1.f;
    if (a.gpost) {
      float s[1] = {0.f};
      for (int k = threadIdx.x; k < a.d; k += kThreads) {
        const float f = ld(a.f, row + k, a.f_bf16);
        s[0] = fmaf(f, f, s[0]);
      }
      block_sum(s, red);
      rf = rsqrtf(s[0] * inv_d + a.eps_post);
    }
    float rx = 0.f;
    if (a.normed) {
      float s[1] = {0.f};
      for (int k = threadIdx.x; k < a.d; k += kThreads) {
        const float x = residual_at(a, row + k, grow + k, k, rf);
        s[0] = fmaf(x, x, s[0]);
      }
      block_sum(s, red);
      rx = rsqrtf(s[0] * inv_d + a.eps_pre);
    }
    // Each thread rewrites only elements that no other one reads: x_out may be x.
    for (int k = threadIdx.x; k < a.d; k += kThreads) {
      const float x = residual_at(a, row + k, grow + k, k, rf);
      st(a.x_out, row + k, a.x_bf16, x);
      if (a.normed) st(a.normed, row + k, a.f_bf16, a.gpre[k] * (x * rx));
    }
  }
}

// ------------------------------------------------------------- backward ----

// A row's means, kept for the column sums: r_x, mean(h u), r_f, mean(gamma_post dy q).
struct RowStats {
  float rx, mx, rf, mf;
};

// The gradients at one element.
struct Grad {
  float D, dy, q, u, dn;  // dgate = scale act' gamma_post q D
};
__device__ __forceinline__ Grad grad_at(const ResidualBwdArgs& a, const RowStats& r, int64_t off, int k, float act) {
  Grad g{0.f, 0.f, 0.f, 0.f, 0.f};
  g.D = a.dxo ? ld(a.dxo, off, a.dx_bf16) : 0.f;
  if (a.dn) {
    g.dn = ld(a.dn, off, a.f_bf16);
    g.u = ld(a.xo, off, a.x_bf16) * r.rx;
    g.D = fmaf(r.rx, a.gpre[k] * g.dn - g.u * r.mx, g.D);
  }
  if (a.f) {
    g.q = ld(a.f, off, a.f_bf16) * r.rf;
    g.dy = a.scale * act * g.D;
  }
  return g;
}
__device__ __forceinline__ float act_at(const ResidualBwdArgs& a, int64_t goff, float* slope) {
  if (!a.gate) {
    *slope = 0.f;
    return 1.f;
  }
  const float g = ld(a.gate, goff, a.g_bf16);
  if (!a.sigmoid) {
    *slope = 1.f;
    return g;
  }
  return sigmoid(g, slope);
}
__device__ __forceinline__ float post_gain(const ResidualBwdArgs& a, int k) { return a.gpost ? a.gpost[k] : 1.f; }

__global__ void __launch_bounds__(kThreads) residual_bwd_stats_kernel(ResidualBwdArgs a, RowStats* stats) {
  __shared__ float red[3 * kThreads / 32];
  pdl_trigger();
  pdl_wait();
  const float inv_d = 1.0f / static_cast<float>(a.d);
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t row = t * a.d, grow = t / a.gate_rows * a.d;
    float s[3] = {0.f, 0.f, 0.f};
    for (int k = threadIdx.x; k < a.d; k += kThreads) {
      if (a.dn) {
        const float x = ld(a.xo, row + k, a.x_bf16), h = a.gpre[k] * ld(a.dn, row + k, a.f_bf16);
        s[0] = fmaf(x, x, s[0]);
        s[1] = fmaf(h, x, s[1]);
      }
      if (a.f && a.gpost) {
        const float f = ld(a.f, row + k, a.f_bf16);
        s[2] = fmaf(f, f, s[2]);
      }
    }
    block_sum(s, red);
    RowStats r{0.f, 0.f, 1.f, 0.f};
    if (a.dn) {
      r.rx = rsqrtf(s[0] * inv_d + a.eps_pre);
      r.mx = r.rx * (s[1] * inv_d);
    }
    if (a.f && a.gpost) {
      r.rf = rsqrtf(s[2] * inv_d + a.eps_post);
      float m[1] = {0.f};
      for (int k = threadIdx.x; k < a.d; k += kThreads) {
        float slope;
        const Grad g = grad_at(a, r, row + k, k, act_at(a, grow + k, &slope));
        m[0] = fmaf(a.gpost[k] * g.dy, g.q, m[0]);
      }
      block_sum(m, red);
      r.mf = m[0] * inv_d;
    }
    if (threadIdx.x == 0) stats[t] = r;
  }
}

// Partial sums over a chunk of tokens: rows of `part` are [which][chunk][d],
// which = 0 dgamma_post, 1 dgamma_pre, 2 the gate's only row.
__global__ void __launch_bounds__(kColumns* kLanes)
    residual_bwd_columns_kernel(ResidualBwdArgs a, const RowStats* stats, float* part, int gate_too) {
  __shared__ float red[3][kLanes][kColumns];
  pdl_trigger();
  pdl_wait();
  const int col = threadIdx.x % kColumns, lane = threadIdx.x / kColumns;
  const int64_t k = static_cast<int64_t>(blockIdx.x) * kColumns + col;
  const int64_t t0 = a.T * blockIdx.y / gridDim.y, t1 = a.T * (blockIdx.y + 1) / gridDim.y;
  float s[3] = {0.f, 0.f, 0.f};
  if (k < a.d) {
    const int kk = static_cast<int>(k);
    const float gp = post_gain(a, kk);
    for (int64_t t = t0 + lane; t < t1; t += kLanes) {
      float slope;
      const float act = act_at(a, t / a.gate_rows * a.d + k, &slope);
      const Grad g = grad_at(a, stats[t], t * a.d + k, kk, act);
      s[0] = fmaf(g.dy, g.q, s[0]);
      s[1] = fmaf(g.dn, g.u, s[1]);
      if (gate_too) s[2] = fmaf(a.scale * slope * gp * g.q, g.D, s[2]);
    }
  }
  for (int i = 0; i < 3; ++i) red[i][lane][col] = s[i];
  __syncthreads();
  if (lane < 3 && k < a.d) {
    float sum = 0.f;
    for (int j = 0; j < kLanes; ++j) sum += red[lane][j][col];
    part[(static_cast<int64_t>(lane) * gridDim.y + blockIdx.y) * a.d + k] = sum;
  }
}

// The gate's gradient where some, but not all, tokens share a row: one CTA
// sums a row's tokens for kColumns features.
__global__ void __launch_bounds__(kColumns* kLanes)
    residual_bwd_gate_kernel(ResidualBwdArgs a, const RowStats* stats, int64_t groups, int column_blocks) {
  __shared__ float red[kLanes][kColumns];
  pdl_trigger();
  pdl_wait();
  const int col = threadIdx.x % kColumns, lane = threadIdx.x / kColumns;
  for (int64_t item = blockIdx.x; item < groups * column_blocks; item += gridDim.x) {
    const int64_t group = item / column_blocks, k = item % column_blocks * kColumns + col;
    const int64_t t0 = group * a.gate_rows;
    const int64_t t1 = a.gate_rows < a.T - t0 ? t0 + a.gate_rows : a.T;
    float s = 0.f;
    if (k < a.d) {
      float slope;
      const float act = act_at(a, group * a.d + k, &slope);
      const float c = a.scale * slope * post_gain(a, static_cast<int>(k));
      for (int64_t t = t0 + lane; t < t1; t += kLanes) {
        const Grad g = grad_at(a, stats[t], t * a.d + k, static_cast<int>(k), act);
        s = fmaf(c * g.q, g.D, s);
      }
    }
    red[lane][col] = s;
    __syncthreads();
    if (lane == 0 && k < a.d) {
      for (int j = 1; j < kLanes; ++j) s += red[j][col];
      st(a.dgate, group * a.d + k, a.g_bf16, s);
    }
    __syncthreads();
  }
}

// The gradients of single elements, from the rows' means (after every kernel
// that reads dx_out: dx may be it).
__global__ void __launch_bounds__(kThreads) residual_bwd_rows_kernel(ResidualBwdArgs a, const RowStats* stats) {
  pdl_trigger();
  pdl_wait();
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t row = t * a.d, grow = t / a.gate_rows * a.d;
    const RowStats r = stats[t];
    for (int k = threadIdx.x; k < a.d; k += kThreads) {
      float slope;
      const Grad g = grad_at(a, r, row + k, k, act_at(a, grow + k, &slope));
      if (a.dx) st(a.dx, row + k, a.dx_bf16, g.D);
      if (!a.f) continue;
      const float gp = post_gain(a, k);
      if (a.df) st(a.df, row + k, a.f_bf16, a.gpost ? r.rf * (gp * g.dy - g.q * r.mf) : g.dy);
      if (a.dgate && a.gate_rows == 1) st(a.dgate, row + k, a.g_bf16, a.scale * slope * gp * g.q * g.D);
    }
  }
}

// The last step of the sums over tokens. The first blocks: the partial rows of
// each kind wanted added in a fixed order, 32 runs of them at once (every 32nd)
// for 32 features. Then, where runs of tokens share gate rows, the rows that
// several teams had tokens of: the last part of the first such team and the
// first parts of the others, in order (residual_bwd_join in residual.cuh says
// which way the blocks are cut).
__global__ void __launch_bounds__(1024)
    residual_bwd_reduce_kernel(ResidualBwdArgs a, const float* part, int parts, int kinds, int blocks, ResidualJoin j) {
  __shared__ float red[32][33];
  pdl_trigger();
  pdl_wait();
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int column_blocks = (a.d - 1) / 32 + 1;
  if (static_cast<int>(blockIdx.x) < blocks) {
    // The nth of the kinds: 0 dgamma_post, 1 dgamma_pre, 2 the gate.
    const int nth = blockIdx.x / column_blocks;
    const int which = nth == 0 ? __ffs(kinds) - 1 : (nth == 1 && kinds == 7 ? 1 : 31 - __clz(kinds));
    float* const gain = which == 0 ? a.dgpost : a.dgpre;
    const int64_t first = static_cast<int64_t>(blockIdx.x % column_blocks) * 32;
    float s = 0.f;
    // Without the norm its gain has no part in anything.
    if (first + x < a.d && (which != 0 || a.gpost) && (which != 1 || a.dn)) {
      const float* p = part + static_cast<int64_t>(which) * parts * a.d + first + x;
      // Five loads at once, cut by predicates: a loop with a rest would run the
      // rest's loads one after the other.
      for (int i = y; i < parts; i += 160) {
        float v[5];
#pragma unroll
        for (int u = 0; u < 5; ++u) v[u] = i + 32 * u < parts ? p[static_cast<int64_t>(i + 32 * u) * a.d] : 0.f;
#pragma unroll
        for (int u = 0; u < 5; ++u) s += v[u];
      }
    }
    red[y][x] = s;
    __syncthreads();
    s = warp_sum(red[x][y]);  // warp y: feature first + y
    const int64_t k = first + y;
    if (x != 0 || k >= a.d) return;
    if (which == 2)
      st(a.dgate, k, a.g_bf16, s);
    else
      gain[k] = a.accumulate ? gain[k] + s : s;
    return;
  }
  const int64_t item = blockIdx.x - blocks;
  const int64_t T = a.T, n = j.teams;
  if (j.by_group) {
    // A gate row and 32 features of it, 32 teams' parts at once.
    const int64_t group = item / column_blocks, k = item % column_blocks * 32 + x;
    const int64_t start = group * a.gate_rows, end = a.gate_rows < T - start ? start + a.gate_rows : T;
    const int64_t first = ((start + 1) * n - 1) / T, last = (end * n - 1) / T;  // teams of its first and last token
    if (first == last) return;
    float s = 0.f;
    if (k < a.d)
      for (int64_t i = first + y; i <= last; i += 128) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t u = i + 32 * e;  // (a team without rows has written nothing)
          v[e] = u <= last && (T >= n || T * u / n < T * (u + 1) / n) ? j.part[(u * 2 + (u == first ? 1 : 0)) * a.d + k] : 0.f;
        }
        s += (v[0] + v[1]) + (v[2] + v[3]);
      }
    red[y][x] = s;
    __syncthreads();
    s = warp_sum(red[x][y]);
    const int64_t kk = item % column_blocks * 32 + y;
    if (x == 0 && kk < a.d) st(a.dgate, group * a.d + kk, a.g_bf16, s);
    return;
  }
  // A team and 1024 features, where that team's first row is the first token of
  // its gate row outside the run of the team before.
  const int wide_blocks = (a.d - 1) / 1024 + 1;
  const int64_t t = item / wide_blocks + 1, k = item % wide_blocks * 1024 + threadIdx.x;
  const int64_t row = T * t / n, group = row / a.gate_rows, start = group * a.gate_rows;
  if (row == T * (t + 1) / n || start == row || k >= a.d) return;
  const int64_t first = ((start + 1) * n - 1) / T;
  if (T * (first + 1) / n != row) return;
  const int64_t end = a.gate_rows < T - start ? start + a.gate_rows : T;
  const int64_t last = (end * n - 1) / T;
  float s = j.part[(first * 2 + 1) * a.d + k];
  if (T >= n) {
#pragma unroll 4
    for (int64_t u = t; u <= last; ++u) s += j.part[u * 2 * a.d + k];
  } else {  // a team without rows has written nothing
    for (int64_t u = t; u <= last; ++u)
      if (T * u / n < T * (u + 1) / n) s += j.part[u * 2 * a.d + k];
  }
  st(a.dgate, group * a.d + k, a.g_bf16, s);
}

unsigned row_grid(int64_t T) {
  const int64_t cap = static_cast<int64_t>(sm_count()) * 8;
  return static_cast<unsigned>(T < cap ? T : cap);
}

int run_reduce(const ResidualBwdArgs& a, const float* part, int parts, const ResidualJoin& join, cudaStream_t s) {
  const int kinds = (a.dgpost ? 1 : 0) | (a.dgpre ? 2 : 0) | (residual_bwd_sums_gate(a) && parts > 0 ? 4 : 0);
  const int blocks = ((kinds & 1) + (kinds >> 1 & 1) + (kinds >> 2)) * ((a.d - 1) / 32 + 1);
  const int64_t all = blocks + join.blocks;
  if (!all) return ATTNRES_OK;
  return launch_step([&] {
    return launch_pdl(residual_bwd_reduce_kernel, static_cast<unsigned>(all), 1024, 0, s, a, part, parts, kinds, blocks,
                      join);
  });
}

int run_bwd_generic(const ResidualBwdArgs& a, cudaStream_t s) {
  RowStats* stats = reinterpret_cast<RowStats*>(a.scratch);
  float* part = a.scratch + 4 * a.T;
  const bool gate_sum = residual_bwd_sums_gate(a);
  const int chunks = static_cast<int>(a.T < kChunks ? a.T : kChunks);
  const int column_blocks = (a.d - 1) / kColumns + 1;
  int e = 0;
  if (a.T > 0) {
    e = launch_step([&] { return launch_pdl(residual_bwd_stats_kernel, row_grid(a.T), kThreads, 0, s, a, stats); });
    if (!e && (a.dgpost || a.dgpre || gate_sum))
      e = launch_step([&] {
        return launch_pdl_grid(residual_bwd_columns_kernel, dim3(column_blocks, chunks), kColumns * kLanes, 0, s, a,
                               stats, part, static_cast<int>(gate_sum));
      });
    if (!e && a.dgate && !gate_sum && a.gate_rows > 1) {
      const int64_t groups = (a.T - 1) / a.gate_rows + 1;
      const int64_t items = groups * column_blocks, cap = static_cast<int64_t>(sm_count()) * 32;
      e = launch_step([&] {
        return launch_pdl(residual_bwd_gate_kernel, static_cast<unsigned>(items < cap ? items : cap),
                          kColumns * kLanes, 0, s, a, stats, groups, column_blocks);
      });
    }
    if (!e && (a.dx || a.df || (a.dgate && a.gate_rows == 1)))
      e = launch_step([&] { return launch_pdl(residual_bwd_rows_kernel, row_grid(a.T), kThreads, 0, s, a, stats); });
  }
  if (!e && (a.T > 0 || !a.accumulate)) e = run_reduce(a, part, chunks, ResidualJoin{}, s);
  return e;
}

int run_bwd_fast(const ResidualBwdArgs& a, cudaStream_t s) {
  const int e = launch_step([&] { return launch_residual_bwd_fast(a, s); });
  return e ? e : run_reduce(a, a.scratch, residual_bwd_parts(a), residual_bwd_join(a), s);
}

}  // namespace

int run_residual(const ResidualArgs& a, cudaStream_t s) {
  if (residual_fast_ok(a)) return launch_step([&] { return launch_residual_fast(a, s); });
  return launch_step([&] { return launch_pdl(residual_generic_kernel, row_grid(a.T), kThreads, 0, s, a); });
}

int run_residual_bwd(const ResidualBwdArgs& a, cudaStream_t s) {
  return residual_bwd_fast_ok(a) ? run_bwd_fast(a, s) : run_bwd_generic(a, s);
}

int64_t residual_bwd_scratch(int64_t T, int d, int64_t gate_rows) {
  const int64_t generic = 4 * T + 3 * (T < kChunks ? T : int64_t{kChunks}) * d;
  const int64_t fast = residual_bwd_fast_scratch(T, d, gate_rows);
  return generic > fast ? generic : fast;
}

}  // namespace attnres
