// The Full read over 8-bit rows (attnres.h: e_i = (u . v_i) / rms(v_i), u = w * gamma,
// z = sum_i softmax_i(e) v_i) in one pass over the rows, with a running maximum and sum.
//
// Streaming kernel (rows of up to 2048 features). A row is held by L lanes, 16
// features in each of C steps, so a warp works on 32 / L tokens at once; the
// 8 lanes of a group share its scale. A producer warp brings the rows of the CTA's
// tokens into a ring of shared-memory stages, K sources a stage (one bulk copy of codes
// and one of tails for each source). Per source a lane decodes its 16 C codes once and
// keeps the values, multiplies them with u (in registers; from shared memory it took
// half as long again), adds over the L lanes, and adds the weighted values onto
// its accumulators. rms needs no sum: the mean square comes with the row.
//
// It is bound by instructions, not bytes: a code takes half a conversion to fp16,
// one to fp32 and two half multiply-adds (pairs), and u, values and accumulators
// take most of the registers, so an SM has 7 to 15 warps, which issue in 44 % of the
// cycles. (So half the bytes of bf16 rows are not half the time: 64 x 8192 x 896 takes 117 us,
// the read of bf16 rows 155; 141 x 32768 x 640 798 and 854.) What helped was less around a
// source: several sources a stage (64 x 8192 x 896 with the pre-norm: 178 us with one source
// a stage, 123 with six, 119 now), a rescaling only when the maximum
// has grown by 8, and gains from shared memory (8192 x 896, 33 sources, a query for
// each token: 105 us with scalar loads of gamma and query, 82 now). Scores by the tensor cores, with
// the values weighted here, took 161 us and more; their operands have to be decoded
// and laid out anew.
//
// When there are fewer groups of tokens than warps, `split` warps of a CTA
// share one (each takes every split-th K sources) and, for few tokens, `cluster` CTAs;
// the maxima, sums and accumulators are joined through shared memory (one token, 141
// sources of 640: 8.2 us, 17.7 with the warps of one CTA).
//
// General kernel (wider rows): a CTA a token, the rows read twice.
#include <math.h>

#include "q8.cuh"
#include "tcgen05.cuh"

namespace attnres {
namespace {

__device__ unsigned int g_q8_read_timeout = 0;

constexpr int kMaxStages = 8;
constexpr int kSmemMax = 226 * 1024;
// A query is multiplied with values of up to 2^128 and the products are added up, so it is taken
// 2^-32 times as large and the score 2^32: no sum over a row overflows as long as the query's
// magnitudes (times gamma) add up to less than 2^32. (Below, a product of an ordinary query
// and of a row whose squares are still normal numbers, 2^-63 in size, is far from the smallest.)
constexpr float kQueryDown = 0x1p-32f, kScoreUp = 0x1p32f;

// 16 values into features [k0, k0 + 16) of a row of d features; `vec`: whole
// 16-byte vectors. The values may be strided pairs of registers.
__device__ __forceinline__ void put16(void* out, int out_bf16, int64_t row, int k0, int d, bool vec, const float2 (&v)[8]) {
  if (out_bf16) {
    bf16* o = static_cast<bf16*>(out) + row * d + k0;
    if (vec) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (k0 + 8 * h < d)
          __stcs(reinterpret_cast<uint4*>(o) + h,
                 make_uint4(pack_bf16x2(v[4 * h].x, v[4 * h].y), pack_bf16x2(v[4 * h + 1].x, v[4 * h + 1].y),
                            pack_bf16x2(v[4 * h + 2].x, v[4 * h + 2].y), pack_bf16x2(v[4 * h + 3].x, v[4 * h + 3].y)));
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (k0 + i < d) o[i] = __float2bfloat16_rn(i & 1 ? v[i >> 1].y : v[i >> 1].x);
    }
  } else {
    float* o = static_cast<float*>(out) + row * d + k0;
    if (vec) {
#pragma unroll
      for (int h = 0; h < 4; ++h)
        if (k0 + 4 * h < d)
          __stcs(reinterpret_cast<float4*>(o) + h, make_float4(v[2 * h].x, v[2 * h].y, v[2 * h + 1].x, v[2 * h + 1].y));
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (k0 + i < d) o[i] = i & 1 ? v[i >> 1].y : v[i >> 1].x;
    }
  }
}

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

template <int K, int S, int C, int L, int NW>
struct Q8Read {
  static constexpr int kRows = 32 / L;  // tokens a warp works on
  static constexpr int kWarps = NW;     // consumer warps; one CTA an SM, whose registers they share with the producer
  static constexpr int kThreads = (kWarps + 1) * 32;
  static constexpr int kTile = kWarps * kRows;
  static constexpr int kBox = (16 * C + 2) * 32;  // floats of a warp's share in a join
  static constexpr int kGains = 16 * C * L;       // floats of a row of gains
};

template <int K, int S, int C, int L, int NW, bool kCluster>
__global__ void __launch_bounds__(Q8Read<K, S, C, L, NW>::kThreads, 1)
    q8_read_kernel(Q8ReadArgs a, float log_n, int nstage, int split, int cluster, int vec, int qvec) {
  using R = Q8Read<K, S, C, L, NW>;
  constexpr int kRows = R::kRows, kWarps = R::kWarps;
  const int cl = kCluster ? cluster : 1;
  extern __shared__ __align__(128) unsigned char smem[];
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem);
  uint64_t* empty_bar = full_bar + kMaxStages;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane % L, sub = lane / L;
  const int G = (a.d + 127) / 128, d = a.d, n = a.n_src, Dp = 128 * G;
  const int tail_bytes = q8_tail_bytes(G), stage_bytes = K * R::kTile * (Dp + tail_bytes);
  // Gains by feature, a lane's 16 of a step as four vectors that are L vectors
  // apart: w gamma (or gamma, for Q's rows), then gamma_pre. Zero from d on.
  float* gains = reinterpret_cast<float*>(smem + 2 * kMaxStages * 8);
  unsigned char* ring = reinterpret_cast<unsigned char*>(gains + (a.pre.gamma ? 2 : 1) * R::kGains);
  // Tiles of `teams` groups of kRows tokens; a team of `split` warps has a group.
  const int teams = kWarps / split, steps = (n + K * split * cl - 1) / (K * split * cl);
  const int64_t T = a.T, groups = (T + kRows - 1) / kRows;
  // Contiguous groups [g0, g1) of this CTA (of this cluster of cl CTAs, which
  // share their sources), in tiles whose sizes differ by one at most.
  const int rank = cl > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int64_t unit = blockIdx.x / cl, units = gridDim.x / cl;
  const int64_t g0 = unit * groups / units, g1 = (unit + 1) * groups / units;
  const int64_t ntiles = (g1 - g0 + teams - 1) / teams;
  auto tile_first = [&](int64_t t) { return g0 + t * (g1 - g0) / ntiles; };

  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < nstage; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 1);
      mbar_init(smem_u32(&empty_bar[s]), kWarps);
    }
    mbar_fence_init();
  }
  pdl_wait();
  for (int k = threadIdx.x; k < R::kGains; k += R::kThreads) {
    const int chunk = k >> 4, at = ((chunk / L * 4 + (k >> 2 & 3)) * L + chunk % L) * 4 + (k & 3);
    const float g = k < d ? a.gamma[k] : 0.f;
    gains[at] = (a.w && k < d ? a.w[k] * kQueryDown : kQueryDown) * g;
    if (a.pre.gamma) gains[R::kGains + at] = k < d ? a.pre.gamma[k] : 0.f;
  }
  __syncthreads();

  if (warp == kWarps) {
    // ------------------------------------------------------------ producer
    // A stage holds the codes of K sources, then their tails: for split == 1 the
    // tile's rows of each (a lane copies a source); otherwise K sources for each
    // warp, its team's rows (a lane copies for a warp).
    const int64_t source = q8_source_bytes(a.cap, d);
    const char* rows = static_cast<const char*>(a.rows);
    const char* tails = rows + a.cap * Dp;
    int s = 0;
    uint32_t phase = 0;
    int64_t it = 0;
    bool ok = true;
    for (int64_t t = 0; t < ntiles && ok; ++t) {
      const int64_t r0 = tile_first(t) * kRows, r1 = tile_first(t + 1) * kRows < T ? tile_first(t + 1) * kRows : T;
      const int64_t nr = r1 - r0;
      for (int step = 0; step < steps; ++step) {
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&empty_bar[s]), phase ^ 1u));
        if (!ok) break;
        const uint32_t fb = smem_u32(&full_bar[s]), dst = smem_u32(ring + s * stage_bytes);
        if (it != a.withhold) {  // the test hook leaves this stage unfilled
          const int i0 = (step * cl + rank) * K * split;  // sources of this step, if any
          const int here = n - i0 < K * split ? (n > i0 ? n - i0 : 0) : K * split;
          if (lane == 0) mbar_arrive_expect_tx(fb, static_cast<uint32_t>(nr * here) * static_cast<uint32_t>(Dp + tail_bytes));
          __syncwarp();
          const uint32_t tdst = dst + K * R::kTile * Dp;
          if (split == 1) {
            if (lane < here) {
              const int64_t src = static_cast<int64_t>(i0 + lane) * source;
              bulk_g2s(dst + lane * R::kTile * Dp, rows + src + r0 * Dp, static_cast<uint32_t>(nr) * static_cast<uint32_t>(Dp), fb);
              bulk_g2s(tdst + lane * R::kTile * tail_bytes, tails + src + r0 * tail_bytes,
                       static_cast<uint32_t>(nr) * static_cast<uint32_t>(tail_bytes), fb);
            }
          } else {
            const int team = lane / split, part = lane - team * split;
            const int64_t left = nr - team * kRows;
            if (team < teams && left > 0) {
              const uint32_t few = left < kRows ? static_cast<uint32_t>(left) : static_cast<uint32_t>(kRows);
              for (int q = 0; q < K; ++q) {
                if (part * K + q >= here) break;
                const int64_t src = static_cast<int64_t>(i0 + part * K + q) * source, row = r0 + team * kRows;
                bulk_g2s(dst + (q * R::kTile + lane * kRows) * Dp, rows + src + row * Dp, few * static_cast<uint32_t>(Dp), fb);
                bulk_g2s(tdst + (q * R::kTile + lane * kRows) * tail_bytes, tails + src + row * tail_bytes,
                         few * static_cast<uint32_t>(tail_bytes), fb);
              }
            }
          }
        }
        ++it;
        if (++s == nstage) {
          s = 0;
          phase ^= 1u;
        }
      }
    }
    // Every copy has landed before this CTA's memory goes (a withheld one was
    // never issued); without a timeout the consumers have seen to that.
    if (lane == 0) {
      for (int64_t k = it > nstage ? it - nstage : 0; k < it; ++k)
        if (k != a.withhold) ok &= mbar_wait(smem_u32(&full_bar[k % nstage]), static_cast<uint32_t>((k / nstage) & 1));
      if (!ok) atomicOr(&g_q8_read_timeout, 1u);
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int team = warp / split, part = warp - team * split;
  const bool last_in = (C - 1) * L + j < 8 * G;  // whether the lane's last step holds codes
  const int lane_at = j * 16, tail_at = K * R::kTile * Dp + (warp * kRows + sub) * tail_bytes, ms_at = q8_mean_offset(G);
  const int codes_at = (warp * kRows + sub) * Dp;

  auto gain = [&](int which, int c, int i) {
    return *reinterpret_cast<const float4*>(gains + which * R::kGains + ((c * 4 + i) * L + j) * 4);
  };
  float2 u[8 * C];
  if (a.w) {
#pragma unroll
    for (int i = 0; i < 4 * C; ++i) {
      const float4 g = gain(0, i >> 2, i & 3);
      u[2 * i] = make_float2(g.x, g.y);
      u[2 * i + 1] = make_float2(g.z, g.w);
    }
  }
  auto load_query = [&](const float* q) {
#pragma unroll
    for (int i = 0; i < 4 * C; ++i) {
      const int k = ((i >> 2) * L + j) * 16 + (i & 3) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (qvec) {
        if (k < d) x = *reinterpret_cast<const float4*>(q + k);
      } else {
        if (k < d) x.x = q[k];
        if (k + 1 < d) x.y = q[k + 1];
        if (k + 2 < d) x.z = q[k + 2];
        if (k + 3 < d) x.w = q[k + 3];
      }
      u[2 * i] = make_float2(x.x, x.y);
      u[2 * i + 1] = make_float2(x.z, x.w);
    }
#pragma unroll
    for (int i = 0; i < 4 * C; ++i) {
      const float4 g = gain(0, i >> 2, i & 3);
      u[2 * i] = fmul2(u[2 * i], make_float2(g.x, g.y));
      u[2 * i + 1] = fmul2(u[2 * i + 1], make_float2(g.z, g.w));
    }
  };

  int s = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (int64_t t = 0; t < ntiles; ++t) {
    const int64_t group = tile_first(t) + team, row = group * kRows + sub;
    const bool busy = team < teams && group < tile_first(t + 1), valid = busy && row < T;
    if (!a.w) load_query(a.Q + (valid ? row : 0) * d);
    float2 acc[8 * C];
#pragma unroll
    for (int i = 0; i < 8 * C; ++i) acc[i] = make_float2(0.f, 0.f);
    // A finite start, so that a score of -inf has weight 0 whatever came before.
    float m = -3.402823466e38f, l = 0.f;
    for (int step = 0; step < steps; ++step) {
      // After a wait that ran out the warp goes on without waiting (barriers
      // stay matched, the warp stores nothing) and the failure is on record.
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&full_bar[s]), phase));
      const int first = ((step * cl + rank) * split + part) * K;
      const unsigned char* r = ring + s * stage_bytes + codes_at + lane_at;
      const unsigned char* tail = ring + s * stage_bytes + tail_at;
      const int todo = !busy ? 0 : (n - first < K ? n - first : K);
#pragma unroll 1
      for (int q0 = 0; q0 < todo; q0 += S, r += S * R::kTile * Dp, tail += S * R::kTile * tail_bytes) {
        float2 v[S][8 * C];
        float sc[S][C], x[S], ms[S];
#pragma unroll
        for (int q = 0; q < S; ++q) {
          const bool there = q == 0 || q0 + q < todo;  // the same for the whole warp
          float2 dot = make_float2(0.f, 0.f);
          ms[q] = there ? *reinterpret_cast<const float*>(tail + q * R::kTile * tail_bytes + ms_at) : 0.f;
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const bool in = there && (c + 1 < C || last_in);
            const uint4 code =
                in ? *reinterpret_cast<const uint4*>(r + q * R::kTile * Dp + c * L * 16) : make_uint4(0, 0, 0, 0);
            sc[q][c] = q8_scale(in ? tail[q * R::kTile * tail_bytes + ((c * L + j) >> 3)] : 1u);
            float2 w[8], p = make_float2(0.f, 0.f);
            decode16(code, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              v[q][c * 8 + k] = w[k];
              p = ffma2(w[k], u[c * 8 + k], p);
            }
            dot = ffma2(p, make_float2(sc[q][c], sc[q][c]), dot);
          }
          x[q] = dot.x + dot.y;
        }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1)
#pragma unroll
          for (int q = 0; q < S; ++q) x[q] += __shfl_xor_sync(0xffffffffu, x[q], o);
        float top = -INFINITY;
#pragma unroll
        for (int q = 0; q < S; ++q) {
          x[q] = q == 0 || q0 + q < todo ? x[q] * (rsqrtf(ms[q] + a.eps) * kScoreUp) : -INFINITY;
          top = fmaxf(top, x[q]);
        }
        float most = ms[0];
#pragma unroll
        for (int q = 1; q < S; ++q) most = fmaxf(most, ms[q]);
        // The accumulators are rescaled only when a score passes what they are scaled
        // by by more than 8, which makes weights of up to e^8. A row with a finite mean
        // square has values below 2^64 and leaves room for those. One whose squares pass fp32's
        // range (its score is 0) may have any, up to 240 * 2^120: its weight is held at
        // 1 / n, so that n of them add up within the range.
        const bool up = top > m + 8.f;
        // (Two votes: 141 x 8192 x 640 in 205 us, 216 with one on both conditions, 211 without the second.)
        if (__any_sync(0xffffffffu, up) | __any_sync(0xffffffffu, most == INFINITY)) {
          const float to = most == INFINITY ? fmaxf(fmaxf(top, log_n), m) : (up ? top : m);
          const float f = __expf(m - to);
          l *= f;
          const float2 f2 = make_float2(f, f);
#pragma unroll
          for (int k = 0; k < 8 * C; ++k) acc[k] = fmul2(acc[k], f2);
          m = to;
        }
#pragma unroll
        for (int q = 0; q < S; ++q) {
          const float p = __expf(x[q] - m);
          l += p;
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const float ps = p * sc[q][c];
            const float2 p2 = make_float2(ps, ps);
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[c * 8 + k] = ffma2(p2, v[q][c * 8 + k], acc[c * 8 + k]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&empty_bar[s]));
      if (++s == nstage) {
        s = 0;
        phase ^= 1u;
      }
    }
    if (split > 1) {
      // Join the teams' shares. All warps are through with the ring, whose
      // copies have all been used (with split > 1 a CTA has one tile).
      named_sync(1, kWarps * 32);
      float* box = reinterpret_cast<float*>(ring) + warp * R::kBox;
      if (part > 0 && team < teams) {
#pragma unroll
        for (int k = 0; k < 8 * C; ++k) *reinterpret_cast<float2*>(box + k * 64 + lane * 2) = acc[k];
        box[64 * 8 * C + lane] = m;
        box[64 * 8 * C + 32 + lane] = l;
      }
      named_sync(1, kWarps * 32);
      if (part == 0 && team < teams) {
        for (int q = 1; q < split; ++q) {
          const float* other = box + q * R::kBox;
          const float mo = other[64 * 8 * C + lane], lo = other[64 * 8 * C + 32 + lane];
          const float top = fmaxf(m, mo);  // a NaN score is in l and the accumulators
          const float ca = __expf(m - top), cb = __expf(mo - top);
          l = l * ca + lo * cb;
#pragma unroll
          for (int k = 0; k < 8 * C; ++k)
            acc[k] = ffma2(*reinterpret_cast<const float2*>(other + k * 64 + lane * 2), make_float2(cb, cb),
                           fmul2(acc[k], make_float2(ca, ca)));
          m = top;
        }
      }
    }
    if (kCluster && cl > 1) {
      // The same over the cluster, whose CTAs have one tile too: each leaves
      // its share in its own memory, the first reads them.
      float* box = reinterpret_cast<float*>(ring) + warp * R::kBox;
      if (split == 1) named_sync(1, kWarps * 32);  // all warps are through with the ring
      if (part == 0 && team < teams && rank > 0) {
#pragma unroll
        for (int k = 0; k < 8 * C; ++k) *reinterpret_cast<float2*>(box + k * 64 + lane * 2) = acc[k];
        box[64 * 8 * C + lane] = m;
        box[64 * 8 * C + 32 + lane] = l;
      }
      cluster_sync();
      if (part == 0 && team < teams && rank == 0) {
        for (int q = 1; q < cl; ++q) {
          const uint32_t other = cluster_addr(smem_u32(box), static_cast<uint32_t>(q));
          const float mo = ld_cluster(other + (64 * 8 * C + lane) * 4), lo = ld_cluster(other + (64 * 8 * C + 32 + lane) * 4);
          const float top = fmaxf(m, mo);
          const float ca = __expf(m - top), cb = __expf(mo - top);
          l = l * ca + lo * cb;
#pragma unroll
          for (int k = 0; k < 8 * C; ++k)
            acc[k] = ffma2(ld_cluster2(other + (k * 64 + lane * 2) * 4), make_float2(cb, cb), fmul2(acc[k], make_float2(ca, ca)));
          m = top;
        }
      }
      cluster_sync();  // the shares have been read: their owners may leave
    }
    if (part != 0 || rank != 0 || !ok || !busy) continue;
    const float inv = 1.0f / l;
#pragma unroll
    for (int k = 0; k < 8 * C; ++k) acc[k] = fmul2(acc[k], make_float2(inv, inv));
    auto put = [&](void* out, int c) {
      if (!valid || (c + 1 == C && !last_in)) return;
      float2 o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = acc[c * 8 + k];
      put16(out, a.out_bf16, row, (c * L + j) * 16, d, vec != 0, o);
    };
    if (a.out)
#pragma unroll
      for (int c = 0; c < C; ++c) put(a.out, c);
    if (a.pre.gamma) {
      float2 q2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 8 * C; ++k) q2 = ffma2(acc[k], acc[k], q2);
      float q = q2.x + q2.y;
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
      const float rr = rsqrtf(q / static_cast<float>(d) + a.pre.eps);
#pragma unroll
      for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 g = gain(1, c, i);
          acc[c * 8 + 2 * i] = fmul2(acc[c * 8 + 2 * i], make_float2(rr * g.x, rr * g.y));
          acc[c * 8 + 2 * i + 1] = fmul2(acc[c * 8 + 2 * i + 1], make_float2(rr * g.z, rr * g.w));
        }
        put(a.pre.out, c);
      }
    }
  }
  if (!ok && lane == 0) atomicOr(&g_q8_read_timeout, 1u);
}

// ---------------------------------------------------------------- general --
// Rows of any width, a CTA a token. A warp takes every eighth source's score, with
// u = (w or Q) gamma in shared memory; after the softmax a thread sums 16 features at a
// time over all sources, which it reads again (from the L1 or L2, as a rule). Four loads of 16
// codes a thread are in flight in both. 16384 x 4096, nine sources:
// 276 us, 0.40 of the copy rate (753 with a word a lane and u from global memory); two decodings
// of every code, and the latency of their loads, bound it.
constexpr int kGenThreads = 256, kGenWarps = kGenThreads / 32, kGenBatch = 4;

constexpr int64_t q8_general_smem(int n, int G) { return (n + 512ll * ((G + 3) / 4)) * 4; }

__global__ void __launch_bounds__(kGenThreads, 4) q8_read_general_kernel(Q8ReadArgs a, int vec) {
  extern __shared__ __align__(16) float sm[];
  __shared__ float part[2][kGenWarps];
  const int G = (a.d + 127) / 128, Dp = 128 * G, n = a.n_src, d = a.d, chunks = 8 * G, rounds = (chunks + 31) / 32;
  const int64_t source = q8_source_bytes(a.cap, d);
  // u: 16 features of a chunk as four vectors, 32 vectors apart, so that a warp's lanes read in a row.
  float* u = sm;
  float* z = sm;  // with a pre-norm, once u has been used: features as they come
  float* p = sm + rounds * 512;  // scores, then weights
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();
  // Two sums or maxima in a row use different words, so one barrier each is enough.
  auto block_join = [&](float x, int which, bool largest) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float y = __shfl_xor_sync(0xffffffffu, x, o);
      x = largest ? fmaxf(x, y) : x + y;
    }
    if (lane == 0) part[which][warp] = x;
    __syncthreads();
    x = part[which][0];
#pragma unroll
    for (int i = 1; i < kGenWarps; ++i) x = largest ? fmaxf(x, part[which][i]) : x + part[which][i];
    return x;
  };
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const unsigned char* rows = static_cast<const unsigned char*>(a.rows) + t * Dp;
    const unsigned char* tails = static_cast<const unsigned char*>(a.rows) + a.cap * Dp + t * q8_tail_bytes(G);
    if (a.Q || a.pre.gamma || t == blockIdx.x) {
      const float* q = a.w ? a.w : a.Q + t * d;
      for (int k = threadIdx.x; k < rounds * 512; k += kGenThreads) {
        const int c = k >> 4;
        u[((c >> 5) * 4 + (k >> 2 & 3)) * 128 + (c & 31) * 4 + (k & 3)] = k < d ? q[k] * kQueryDown * a.gamma[k] : 0.f;
      }
    }
    __syncthreads();
    for (int i = warp; i < n; i += kGenWarps) {
      const unsigned char *r = rows + i * source, *tail = tails + i * source;
      float2 dot = make_float2(0.f, 0.f);
      for (int c0 = 0; c0 < rounds; c0 += kGenBatch) {
        uint4 code[kGenBatch];
        uint32_t e[kGenBatch];
#pragma unroll
        for (int b = 0; b < kGenBatch; ++b) {
          const int c = (c0 + b) * 32 + lane;
          code[b] = c < chunks ? *reinterpret_cast<const uint4*>(r + c * 16) : make_uint4(0, 0, 0, 0);
          e[b] = c < chunks ? tail[c >> 3] : 1u;
        }
#pragma unroll
        for (int b = 0; b < kGenBatch; ++b) {
          if (c0 + b >= rounds) break;
          float2 v[8], x = make_float2(0.f, 0.f);
          decode16(code[b], v);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 w = *reinterpret_cast<const float4*>(u + ((c0 + b) * 4 + k) * 128 + lane * 4);
            x = ffma2(v[2 * k], make_float2(w.x, w.y), x);
            x = ffma2(v[2 * k + 1], make_float2(w.z, w.w), x);
          }
          const float s = q8_scale(e[b]);
          dot = ffma2(x, make_float2(s, s), dot);
        }
      }
      const float x = warp_sum(dot.x + dot.y);
      if (lane == 0) p[i] = x * (rsqrtf(*reinterpret_cast<const float*>(tail + q8_mean_offset(G)) + a.eps) * kScoreUp);
    }
    __syncthreads();
    float m = -3.402823466e38f;  // finite, so that a score of -inf has weight 0
    for (int i = threadIdx.x; i < n; i += kGenThreads) m = fmaxf(m, p[i]);
    m = block_join(m, 0, true);
    float l = 0.f;
    for (int i = threadIdx.x; i < n; i += kGenThreads) l += p[i] = __expf(p[i] - m);
    const float inv = 1.0f / block_join(l, 1, false);  // its barrier also orders p
    float q2 = 0.f;
    for (int c = threadIdx.x; c < chunks; c += kGenThreads) {
      float2 acc[8];
      // Weights of at most 1, and what they add up to at the end: where that sum of values passes
      // fp32's range (or a value is NaN) once more, with the weights divided first.
      float first = 1.f, last = inv;
#pragma unroll 1
      for (int pass = 0; pass < 2; ++pass) {
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = make_float2(0.f, 0.f);
        for (int i0 = 0; i0 < n; i0 += kGenBatch) {
          uint4 code[kGenBatch];
          uint32_t e[kGenBatch];
#pragma unroll
          for (int b = 0; b < kGenBatch; ++b) {
            const bool in = i0 + b < n;
            code[b] = in ? *reinterpret_cast<const uint4*>(rows + (i0 + b) * source + c * 16) : make_uint4(0, 0, 0, 0);
            e[b] = in ? tails[(i0 + b) * source + (c >> 3)] : 1u;
          }
#pragma unroll
          for (int b = 0; b < kGenBatch; ++b) {
            if (i0 + b >= n) break;
            const float ps = p[i0 + b] * first * q8_scale(e[b]);
            float2 v[8];
            decode16(code[b], v);
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[k] = ffma2(v[k], make_float2(ps, ps), acc[k]);
          }
        }
        float most = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) most += fabsf(acc[k].x) * 0x1p-5f + fabsf(acc[k].y) * 0x1p-5f;  // finite where they are
        if (most < INFINITY) break;
        first = inv;
        last = 1.f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        acc[k] = fmul2(acc[k], make_float2(last, last));
        q2 = fmaf(acc[k].x, acc[k].x, q2);
        q2 = fmaf(acc[k].y, acc[k].y, q2);
      }
      if (a.out) put16(a.out, a.out_bf16, t, c * 16, d, vec != 0, acc);
      if (a.pre.gamma)
#pragma unroll
        for (int k = 0; k < 8; ++k) *reinterpret_cast<float2*>(z + c * 16 + 2 * k) = acc[k];
    }
    if (a.pre.gamma) {
      const float rr = rsqrtf(block_join(q2, 0, false) / static_cast<float>(d) + a.pre.eps);
      for (int k = threadIdx.x; k < d; k += kGenThreads) {
        const float o = a.pre.gamma[k] * (z[k] * rr);
        if (a.out_bf16)
          static_cast<bf16*>(a.pre.out)[t * d + k] = __float2bfloat16_rn(o);
        else
          static_cast<float*>(a.pre.out)[t * d + k] = o;
      }
    }
    __syncthreads();  // p, z and the joins' words are free again
  }
}

template <int K, int S, int C, int L, int NW, bool kCluster = false>
cudaError_t launch_cl(const Q8ReadArgs& a, cudaStream_t s) {
  using R = Q8Read<K, S, C, L, NW>;
  const int G = q8_groups(a.d), stage_bytes = K * R::kTile * (128 * G + q8_tail_bytes(G));
  const int fixed = 2 * kMaxStages * 8 + (a.pre.gamma ? 2 : 1) * R::kGains * 4;
  int nstage = (kSmemMax - fixed) / stage_bytes;
  nstage = nstage > kMaxStages ? kMaxStages : nstage;
  const int64_t groups = (a.T + R::kRows - 1) / R::kRows;
  const int sms = sm_count();
  // As many warps to a group of tokens as there are to spare, so that each CTA still has one tile.
  int split = 1;
  while (2 * split <= R::kWarps && 2 * split * K <= a.n_src + K - 1 && groups <= static_cast<int64_t>(sms) * (R::kWarps / (2 * split)))
    split *= 2;
  // And as many CTAs (a cluster), as long as every warp of them still has sources.
  const int teams = R::kWarps / split;
  const int64_t tiles = (groups + teams - 1) / teams;
  int cl = 1;
  while (kCluster && 2 * cl <= 8 && tiles * 2 * cl <= sms && 2 * cl * split * K <= a.n_src + K - 1) cl *= 2;
  int ring = nstage * stage_bytes;
  const int boxes = R::kWarps * R::kBox * 4;
  if (split * cl > 1 && ring < boxes) ring = boxes;
  const int smem = fixed + ring;
  const void* fn = reinterpret_cast<const void*>(&q8_read_kernel<K, S, C, L, NW, kCluster>);
  cudaError_t e = allow_dynamic_smem(fn, kSmemMax);
  if (e != cudaSuccess) return e;
  // Rows of both outputs that start on 16-byte boundaries and hold whole 16-byte vectors.
  const int vec = a.d % (a.out_bf16 ? 8 : 4) == 0 && aligned16(a.out) && aligned16(a.pre.out);
  const int qvec = a.Q && a.d % 4 == 0 && aligned16(a.Q);
  const int64_t grid = tiles < sms ? tiles * cl : sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(R::kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cl);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cl > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, q8_read_kernel<K, S, C, L, NW, kCluster>, a, logf(static_cast<float>(a.n_src)), nstage, split,
                            cl, vec, qvec);
}

cudaError_t launch_general(const Q8ReadArgs& a, cudaStream_t s) {
  const int64_t smem = q8_general_smem(a.n_src, q8_groups(a.d));
  if (smem > 200 * 1024) return cudaErrorInvalidValue;
  const void* fn = reinterpret_cast<const void*>(&q8_read_general_kernel);
  cudaError_t e = allow_dynamic_smem(fn, 200 * 1024);
  if (e != cudaSuccess) return e;
  const int vec = a.d % (a.out_bf16 ? 8 : 4) == 0 && aligned16(a.out);
  const int64_t cap = static_cast<int64_t>(sm_count()) * 4;
  return launch_pdl(q8_read_general_kernel, static_cast<unsigned>(a.T < cap ? a.T : cap), kGenThreads, static_cast<int>(smem), s,
                    a, vec);
}

}  // namespace

cudaError_t launch_q8_read(const Q8ReadArgs& a, cudaStream_t s) {
  const int G = q8_groups(a.d);
  // In each line the last C step holds codes: 8 G > (C - 1) L. Few tokens: a
  // token's sources spread over many warps and CTAs, so few to a stage (9 sources:
  // 228 x 640 in 6.0 us, 7.8 by the kernels below; 33: 228 x 2048 in 12.7 and 14.4, 228 x 640
  // in 10.0 and 8.0, 300 x 640 in 10.1 and 8.1).
  const int sms = sm_count();
  if (a.T <= 3 * sms / 2) {
    if (G <= 4) return launch_cl<2, 2, 1, 32, 15, true>(a, s);
    if (G <= 8) return launch_cl<2, 2, 2, 32, 11, true>(a, s);
    if (G <= 12) return launch_cl<1, 1, 3, 32, 7, true>(a, s);
    if (G <= 16) return launch_cl<1, 1, 4, 32, 7, true>(a, s);
  }
  // Warps: 11 where a lane's state fits their 168 registers (C = 3 spills up to 80 bytes, C = 2 with
  // two sources at a time 56), 7 of up to 255 registers otherwise. With C = 3 and L = 16 7 are sooner done
  // (141 x 8192 x 640: 205 us, 208 with 11 and five sources a stage), with L = 32 11 (33 x 8192 x 1216: 100, 114 with 7).
  auto rounds = [&](int tile) { return (a.T + static_cast<int64_t>(sms) * tile - 1) / (static_cast<int64_t>(sms) * tile) * tile; };
  switch (G) {
    case 1: return launch_cl<6, 1, 2, 4, 11>(a, s);
    case 2: return launch_cl<6, 1, 4, 4, 7>(a, s);
    case 3: return launch_cl<5, 1, 3, 8, 11>(a, s);
    case 4: return launch_cl<4, 1, 4, 8, 7>(a, s);
    case 5: case 6: return launch_cl<8, 1, 3, 16, 7>(a, s);
    case 7:
    case 8:
      // Tiles of 14 tokens, or of 11 where their last round leaves fewer SMs
      // idle and no tokens are shared by warps of the first (64 sources of 896: 1200 tokens
      // 30.8 us and 27.1, 2000 tokens 34.7 and 45.8, 850 tokens 20.9 and 26.9).
      return a.T <= 6 * sms || rounds(14) * 20 <= rounds(11) * 21 ? launch_cl<6, 1, 4, 16, 7>(a, s)
                                                                  : launch_cl<4, 2, 2, 32, 11>(a, s);
    case 9: case 10: case 11: case 12: return launch_cl<5, 1, 3, 32, 11>(a, s);
    case 13: case 14: case 15: case 16: return launch_cl<6, 1, 4, 32, 7>(a, s);
    default: return launch_general(a, s);
  }
}

cudaError_t take_timeout_q8_read(unsigned int* flag) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(flag, g_q8_read_timeout, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_q8_read_timeout, &zero, sizeof(unsigned int));
}

}  // namespace attnres
