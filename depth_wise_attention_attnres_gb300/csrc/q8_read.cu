// The Full read over 8-bit rows (attnres.h: e_i = (u . v_i) / rms(v_i), u = w * gamma,
// z = sum_i softmax_i(e) v_i) in one pass over the rows, with a running maximum and sum.
//
// Streaming kernel (rows of up to 2048 features). A row is held by L lanes, 16
// features in each of C steps, so a warp works on 32 / L tokens at once; a
// token's 8 lanes of a group share its scale. Each warp streams its own rows:
// per source, the records of its tokens are consecutive, and one bulk copy
// brings them into a ring of the warp's own in shared memory. No warp waits
// for another, and lane 0 refills a stage as soon as its codes are in
// registers. Per source a lane decodes its 16 C codes once and keeps the values,
// multiplies them with u (in registers for as long as the token lasts), adds over the
// L lanes, and adds the weighted values onto its accumulators. rms needs no
// sum: the mean square comes with the row.
//
// When there are fewer groups of tokens than warps, `split` warps of a CTA
// share one: each takes every split-th source, and the maxima, sums and
// accumulators are joined through shared memory.
//
// General kernel (wider rows): a CTA a token; the scores of all sources, their
// softmax, then the weighted sum, reading the rows twice.
#include <math.h>

#include "q8.cuh"

namespace attnres {
namespace {

__device__ unsigned int g_q8_read_timeout = 0;

constexpr int kMaxStages = 8;
constexpr int kSmemMax = 200 * 1024;
// A query is multiplied with codes of up to 448 before their scale, so it is taken
// 2^-16 times as large and the score 2^16: no finite product of a value and a
// query overflows.
constexpr float kQueryDown = 1.0f / 65536.0f, kScoreUp = 65536.0f;

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

template <int C, int L>
struct Q8Read {
  static constexpr int kRows = 32 / L;               // tokens a warp works on
  static constexpr int kWarps = C <= 2 ? 16 : 8;     // warps of a CTA, one CTA an SM
};

template <int C, int L>
__global__ void __launch_bounds__(Q8Read<C, L>::kWarps * 32, 1) q8_read_kernel(Q8ReadArgs a, int rec, int nstage, int split,
                                                                              int vec) {
  constexpr int kRows = Q8Read<C, L>::kRows, kWarps = Q8Read<C, L>::kWarps;
  extern __shared__ __align__(128) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane % L, sub = lane / L;
  const int G = (a.d + 127) / 128, d = a.d;
  const int stage_bytes = kRows * rec;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem) + warp * kMaxStages;
  unsigned char* ring = smem + kWarps * kMaxStages * 8 + static_cast<size_t>(warp) * nstage * stage_bytes;
  const int teams = kWarps / split, team = warp / split, part = warp - team * split;
  const int64_t T = a.T, groups = (T + kRows - 1) / kRows;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * teams + team, step = static_cast<int64_t>(gridDim.x) * teams;
  const int64_t mine = first < groups ? (groups - 1 - first) / step + 1 : 0;
  const int ni = (a.n_src - part + split - 1) / split;  // sources part, part + split, ..: at least one (split <= n_src)
  const int64_t total = mine * ni;
  const bool last_in = (C - 1) * L + j < 8 * G;  // whether the lane's last step holds codes

  pdl_trigger();
  if (lane == 0) {
    for (int s = 0; s < nstage; ++s) mbar_init(smem_u32(&bars[s]), 1);
    mbar_fence_init();
  }
  __syncwarp();
  pdl_wait();

  // Lane 0's position among the warp's copies: token group pg, source pi.
  int64_t issued = 0, pg = first;
  int pi = part, pstage = 0;
  const char* rows = static_cast<const char*>(a.rows);
  auto issue = [&] {
    const int64_t left = T - pg * kRows;
    const uint32_t bytes = static_cast<uint32_t>(left < kRows ? static_cast<int>(left) : kRows) * static_cast<uint32_t>(rec);
    if (issued != a.withhold) {  // the test hook leaves this stage unfilled
      const uint32_t bar = smem_u32(&bars[pstage]);
      mbar_arrive_expect_tx(bar, bytes);
      bulk_g2s(smem_u32(ring + pstage * stage_bytes), rows + static_cast<int64_t>(pi) * a.row_stride + pg * kRows * rec, bytes,
               bar);
    }
    ++issued;
    if (++pstage == nstage) pstage = 0;
    pi += split;
    if (pi >= a.n_src) {
      pi = part;
      pg += step;
    }
  };
  if (lane == 0)
    for (int s = 0; s < nstage && issued < total; ++s) issue();

  const float inv_d = 1.0f / static_cast<float>(d);
  float2 u[8 * C];
  auto load_u = [&](const float* q) {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = (c * L + j) * 16 + 2 * i;
        u[c * 8 + i] = make_float2(k < d ? q[k] * kQueryDown * a.gamma[k] : 0.f,
                                   k + 1 < d ? q[k + 1] * kQueryDown * a.gamma[k + 1] : 0.f);
      }
  };
  if (a.w) load_u(a.w);

  int stage = 0;
  uint32_t phase = 0;
  bool ok = true;
  int64_t it = 0;
  for (int64_t g = first; g < groups && ok; g += step) {
    const int64_t row = g * kRows + sub;
    const bool valid = row < T;
    if (!a.w) load_u(a.Q + (valid ? row : T - 1) * d);
    float2 acc[8 * C];
#pragma unroll
    for (int i = 0; i < 8 * C; ++i) acc[i] = make_float2(0.f, 0.f);
    // A finite start, so that a score of -inf has weight 0 whatever came before.
    float m = -3.402823466e38f, l = 0.f;
    for (int i = 0; i < ni; ++i, ++it) {
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&bars[stage]), phase))) {
        ok = false;
        break;
      }
      const unsigned char* r = ring + stage * stage_bytes + sub * rec;
      float2 v[8 * C];
      float sc[C];
      float2 dot = make_float2(0.f, 0.f);
      const float ms = *reinterpret_cast<const float*>(r + q8_mean_offset(G));
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const bool in = c + 1 < C || last_in;
        const uint4 code = in ? *reinterpret_cast<const uint4*>(r + (c * L + j) * 16) : make_uint4(0, 0, 0, 0);
        sc[c] = q8_scale(in ? r[128 * G + ((c * L + j) >> 3)] : 1u);
        float2 w[8], p = make_float2(0.f, 0.f);
        decode16(code, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          v[c * 8 + k] = w[k];
          p = ffma2(w[k], u[c * 8 + k], p);
        }
        dot = ffma2(p, make_float2(sc[c], sc[c]), dot);
      }
      __syncwarp();  // the stage's codes are in registers
      if (lane == 0 && issued < total) issue();
      if (++stage == nstage) {
        stage = 0;
        phase ^= 1u;
      }
      float s = dot.x + dot.y;
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      s *= rsqrtf(ms + a.eps) * kScoreUp;
      // The accumulators are rescaled only when a score passes the maximum they
      // are scaled by by more than 8: weights up to e^8 lose nothing in fp32.
      const bool up = s > m + 8.f;
      if (__any_sync(0xffffffffu, up)) {
        const float c = up ? __expf(m - s) : 1.f;
        l *= c;
        const float2 c2 = make_float2(c, c);
#pragma unroll
        for (int k = 0; k < 8 * C; ++k) acc[k] = fmul2(acc[k], c2);
        if (up) m = s;
      }
      const float p = __expf(s - m);
      l += p;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float ps = p * sc[c];
        const float2 p2 = make_float2(ps, ps);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[c * 8 + k] = ffma2(p2, v[c * 8 + k], acc[c * 8 + k]);
      }
    }
    if (split > 1) {
      // Join the team's shares. Each warp's ring is idle: its copies have all
      // been used (a team with split > 1 has one token group).
      float* box = reinterpret_cast<float*>(ring);
#pragma unroll
      for (int k = 0; k < 8 * C; ++k) *reinterpret_cast<float2*>(box + k * 64 + lane * 2) = acc[k];
      box[64 * 8 * C + lane] = m;
      box[64 * 8 * C + 32 + lane] = l;
      named_sync(1 + team, split * 32);
      if (part == 0) {
        const size_t next = static_cast<size_t>(nstage) * stage_bytes / 4;
        for (int q = 1; q < split; ++q) {
          const float* other = box + q * next;
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
    if (part != 0 || !ok) continue;
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
      const float rr = rsqrtf(q * inv_d + a.pre.eps);
#pragma unroll
      for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int k = (c * L + j) * 16 + 2 * i;
          acc[c * 8 + i].x *= rr * (k < d ? a.pre.gamma[k] : 0.f);
          acc[c * 8 + i].y *= rr * (k + 1 < d ? a.pre.gamma[k + 1] : 0.f);
        }
        put(a.pre.out, c);
      }
    }
  }
  if (!ok) {
    if (lane == 0) {
      atomicOr(&g_q8_read_timeout, 1u);
      // Copies still in flight land before this CTA's memory goes (a withheld one was never issued).
      for (int64_t k = issued > nstage ? issued - nstage : 0; k < issued; ++k)
        if (k != a.withhold && k >= it)
          (void)mbar_wait(smem_u32(&bars[k % nstage]), static_cast<uint32_t>((k / nstage) & 1));
    }
    __syncwarp();
  }
}

constexpr int kGenThreads = 256;

__global__ void __launch_bounds__(kGenThreads) q8_read_general_kernel(Q8ReadArgs a, int rec) {
  extern __shared__ __align__(16) float sm[];
  const int G = (a.d + 127) / 128, Dp = 128 * G, n = a.n_src, d = a.d;
  float* z = sm;          // [Dp]
  float* p = sm + Dp;     // [n] scores, then weights
  __shared__ float part[kGenThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();
  auto block_sum = [&](float x) {
    x = warp_sum(x);
    __syncthreads();
    if (lane == 0) part[warp] = x;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < kGenThreads / 32; ++i) t += part[i];
    return t;
  };
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const unsigned char* rows = static_cast<const unsigned char*>(a.rows) + t * rec;
    const float* q = a.w ? a.w : a.Q + t * d;
    for (int i = warp; i < n; i += kGenThreads / 32) {
      const unsigned char* r = rows + i * a.row_stride;
      float dot = 0.f;
      for (int w = lane; w < Dp / 4; w += 32) {
        float2 v0, v1;
        decode4(*reinterpret_cast<const uint32_t*>(r + 4 * w), v0, v1);
        const float s = q8_scale(r[Dp + (w >> 5)]);
        float x = 0.f;
        if (4 * w < d) x += v0.x * (q[4 * w] * kQueryDown * a.gamma[4 * w]);
        if (4 * w + 1 < d) x += v0.y * (q[4 * w + 1] * kQueryDown * a.gamma[4 * w + 1]);
        if (4 * w + 2 < d) x += v1.x * (q[4 * w + 2] * kQueryDown * a.gamma[4 * w + 2]);
        if (4 * w + 3 < d) x += v1.y * (q[4 * w + 3] * kQueryDown * a.gamma[4 * w + 3]);
        dot = fmaf(x, s, dot);
      }
      dot = warp_sum(dot);
      if (lane == 0) p[i] = dot * (rsqrtf(*reinterpret_cast<const float*>(r + q8_mean_offset(G)) + a.eps) * kScoreUp);
    }
    __syncthreads();
    float m = -3.402823466e38f;
    for (int i = 0; i < n; ++i) m = fmaxf(m, p[i]);
    __syncthreads();
    float l = 0.f;
    for (int i = threadIdx.x; i < n; i += kGenThreads) l += p[i] = __expf(p[i] - m);
    const float inv = 1.0f / block_sum(l);  // its barriers also order p
    float q2 = 0.f;
    for (int w = threadIdx.x; w < Dp / 4; w += kGenThreads) {
      float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
      for (int i = 0; i < n; ++i) {
        const unsigned char* r = rows + i * a.row_stride;
        float2 v0, v1;
        decode4(*reinterpret_cast<const uint32_t*>(r + 4 * w), v0, v1);
        const float ps = p[i] * q8_scale(r[Dp + (w >> 5)]);
        acc0 = ffma2(v0, make_float2(ps, ps), acc0);
        acc1 = ffma2(v1, make_float2(ps, ps), acc1);
      }
      const float o[4] = {acc0.x * inv, acc0.y * inv, acc1.x * inv, acc1.y * inv};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = 4 * w + e;
        q2 = fmaf(o[e], o[e], q2);
        z[k] = o[e];
        if (a.out && k < d) {
          if (a.out_bf16)
            static_cast<bf16*>(a.out)[t * d + k] = __float2bfloat16_rn(o[e]);
          else
            static_cast<float*>(a.out)[t * d + k] = o[e];
        }
      }
    }
    if (a.pre.gamma) {
      const float rr = rsqrtf(block_sum(q2) / static_cast<float>(d) + a.pre.eps);
      for (int k = threadIdx.x; k < d; k += kGenThreads) {
        const float o = a.pre.gamma[k] * (z[k] * rr);
        if (a.out_bf16)
          static_cast<bf16*>(a.pre.out)[t * d + k] = __float2bfloat16_rn(o);
        else
          static_cast<float*>(a.pre.out)[t * d + k] = o;
      }
    }
    __syncthreads();
  }
}

template <int C, int L>
cudaError_t launch_cl(const Q8ReadArgs& a, int rec, cudaStream_t s) {
  using R = Q8Read<C, L>;
  const int stage_bytes = R::kRows * rec, fixed = R::kWarps * kMaxStages * 8;
  // The join's boxes take (16 C + 2) * 128 bytes of each ring.
  int nstage = (kSmemMax - fixed) / (R::kWarps * stage_bytes);
  nstage = nstage > kMaxStages ? kMaxStages : nstage;
  const int64_t groups = (a.T + R::kRows - 1) / R::kRows;
  const int sms = sm_count();
  int split = 1;
  while (split < R::kWarps && 2 * split <= a.n_src && groups * 2 * split <= static_cast<int64_t>(sms) * R::kWarps) split *= 2;
  int ring = nstage * stage_bytes;
  const int box = (16 * C + 2) * 128;
  if (split > 1 && ring < box) return cudaErrorInvalidValue;
  const int smem = fixed + R::kWarps * ring;
  const void* fn = reinterpret_cast<const void*>(&q8_read_kernel<C, L>);
  cudaError_t e = allow_dynamic_smem(fn, smem);
  if (e != cudaSuccess) return e;
  // Rows of both outputs that start on 16-byte boundaries and hold whole 16-byte vectors.
  const int vec = a.d % (a.out_bf16 ? 8 : 4) == 0 && aligned16(a.out) && aligned16(a.pre.out);
  const int teams = R::kWarps / split;
  int64_t grid = (groups + teams - 1) / teams;
  if (grid > sms) grid = sms;
  return launch_pdl(q8_read_kernel<C, L>, static_cast<unsigned>(grid), R::kWarps * 32, smem, s, a, rec, nstage, split,
                    vec);
}

cudaError_t launch_general(const Q8ReadArgs& a, int rec, cudaStream_t s) {
  const int64_t smem = (static_cast<int64_t>(a.n_src) + 128 * q8_groups(a.d)) * 4;
  if (smem > 200 * 1024) return cudaErrorInvalidValue;
  const void* fn = reinterpret_cast<const void*>(&q8_read_general_kernel);
  cudaError_t e = allow_dynamic_smem(fn, 200 * 1024);
  if (e != cudaSuccess) return e;
  const int64_t cap = static_cast<int64_t>(sm_count()) * 8;
  return launch_pdl(q8_read_general_kernel, static_cast<unsigned>(a.T < cap ? a.T : cap), kGenThreads, static_cast<int>(smem), s,
                    a, rec);
}

}  // namespace

cudaError_t launch_q8_read(const Q8ReadArgs& a, cudaStream_t s) {
  const int G = q8_groups(a.d), rec = static_cast<int>(q8_row_bytes(a.d));
  switch (G) {
    case 1: return launch_cl<1, 8>(a, rec, s);
    case 2: return launch_cl<2, 8>(a, rec, s);
    case 3: return launch_cl<3, 8>(a, rec, s);
    case 4: return launch_cl<4, 8>(a, rec, s);
    case 5: case 6: return launch_cl<3, 16>(a, rec, s);
    case 7: case 8: return launch_cl<4, 16>(a, rec, s);
    case 9: case 10: case 11: case 12: return launch_cl<3, 32>(a, rec, s);
    case 13: case 14: case 15: case 16: return launch_cl<4, 32>(a, rec, s);
    default: return launch_general(a, rec, s);
  }
}

cudaError_t take_timeout_q8_read(unsigned int* flag) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(flag, g_q8_read_timeout, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_q8_read_timeout, &zero, sizeof(unsigned int));
}

}  // namespace attnres
