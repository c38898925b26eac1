// The global norm of a list of gradients, and the list scaled to a norm.
//
// norm = sqrt(sum g^2) over every element of every tensor; clipping multiplies
// by max_norm / norm where norm exceeds max_norm. Two launches either way: the
// first leaves one partial sum per CTA, the second adds them (in a fixed
// order, every CTA for itself) and writes the norm, or the norm and the
// scaled tensors. Bound by memory: the norm reads every gradient once, the
// scaling reads them again and writes them (a list larger than the L2 has to be
// read twice: no scaling before the norm is known). Measured: 400M bf16 elements'
// norm in 117 us (6.8 TB/s), 800M fp32 clipped to bf16 in 1.16 to 1.19 ms (6.7 to
// 6.9 TB/s over both readings and the writing), in place in 1.45.
//
// Squares are summed in three scales at once, of g, g 2^80 and g 2^-80: fp32
// holds g^2 only for 2^-63 < |g| < 2^63, and bf16 and fp32 gradients go far
// beyond both ends. The sum of g^2 serves unless it overflowed (then the
// scaled-down sum does: what it loses, |g| < 2^17, is below 2^-53 of a sum
// over 2^127) or is under 2^-60 (then the scaled-up one, which is below 2^100).
//
// The tensors' addresses travel as kernel arguments, so a call needs no table
// in device memory; the tensors are cut into units of kUnit elements and every
// CTA takes one run of consecutive units, wherever tensors begin and end.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace attnres {
namespace {

constexpr int kThreads = 512;
constexpr int kUnit = 2048;        // elements
constexpr int kMaxCtas = 456;      // partial sums of one launch
// Resident CTAs of an SM that the two kernels are launched for.
constexpr int kSumsPerSm = 3, kScalePerSm = 2;
constexpr int kMaxTensors = 1024;  // of one launch: 29 KB of the 32,764 bytes of arguments

template <int N>
struct Table {
  const void* src[N];
  void* dst[N];
  int64_t count[N];
  uint32_t first[N + 1];  // first unit of each tensor; first[n]: all units
  uint8_t kind[N];        // 1: src is bf16, 2: dst is bf16
  int n;
};

// Sums of squares of g, g 2^-80 and g 2^80. A batch of loads is summed from
// zero and then added to the thread's total, whose rounding is kept and added at
// the end (total >= batch but for the first ones): small gradients are not lost
// behind large ones, and a total that overflowed stays infinite.
struct Sums {
  float2 mid, big, small;
};
struct Total {
  float s[3] = {0.f, 0.f, 0.f}, rest[3] = {0.f, 0.f, 0.f};
  __device__ __forceinline__ void add(const Sums& b) {
    const float v[3] = {b.mid.x + b.mid.y, b.big.x + b.big.y, b.small.x + b.small.y};
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const float t = s[i] + v[i];
      rest[i] += (s[i] - t) + v[i];
      s[i] = t;
    }
  }
  // After an overflow the rest is not a number.
  __device__ __forceinline__ float value(int i) const { return isfinite(s[i]) ? s[i] + rest[i] : s[i]; }
};

__device__ __forceinline__ void add2(Sums& s, float2 x) {
  const float2 down = make_float2(0x1p-80f, 0x1p-80f), up = make_float2(0x1p80f, 0x1p80f);
  s.mid = ffma2(x, x, s.mid);
  const float2 b = fmul2(x, down), t = fmul2(x, up);
  s.big = ffma2(b, b, s.big);
  s.small = ffma2(t, t, s.small);
}
__device__ __forceinline__ void add_vec(Sums& s, const bf16*, uint4 v) {
  add2(s, make_float2(bf16_lo(v.x), bf16_hi(v.x)));
  add2(s, make_float2(bf16_lo(v.y), bf16_hi(v.y)));
  add2(s, make_float2(bf16_lo(v.z), bf16_hi(v.z)));
  add2(s, make_float2(bf16_lo(v.w), bf16_hi(v.w)));
}
__device__ __forceinline__ void add_vec(Sums& s, const float*, uint4 v) {
  add2(s, make_float2(__uint_as_float(v.x), __uint_as_float(v.y)));
  add2(s, make_float2(__uint_as_float(v.z), __uint_as_float(v.w)));
}

// Elements before the first 16-byte boundary at or after p.
template <typename T>
__device__ __forceinline__ int64_t head_of(const T* p, int64_t n) {
  const int64_t h = static_cast<int64_t>((0 - reinterpret_cast<uintptr_t>(p)) & 15) / static_cast<int64_t>(sizeof(T));
  return h < n ? h : n;
}

template <typename T>
__device__ __forceinline__ void sum_segment(Total& total, const T* p, int64_t n) {
  // Four loads in flight a thread on three CTAs an SM: with eight 400M bf16
  // elements took 120 us (117), with two or four CTAs 123 and 146.
  constexpr int kV = 16 / sizeof(T), kU = 4;
  const int64_t head = head_of(p, n);
  const uint4* v = reinterpret_cast<const uint4*>(p + head);
  const int64_t nv = (n - head) / kV;
  int64_t i = threadIdx.x;
  for (; i + (kU - 1) * kThreads < nv; i += kU * kThreads) {
    uint4 x[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) x[u] = v[i + u * kThreads];
    Sums s{};
#pragma unroll
    for (int u = 0; u < kU; ++u) add_vec(s, p, x[u]);
    total.add(s);
  }
  // The last batch is cut by predicates: its loads too are all in flight at once.
  if (i < nv) {
    uint4 x[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) x[u] = i + u * kThreads < nv ? v[i + u * kThreads] : make_uint4(0, 0, 0, 0);
    Sums s{};
#pragma unroll
    for (int u = 0; u < kU; ++u) add_vec(s, p, x[u]);
    total.add(s);
  }
  Sums s{};
  if (threadIdx.x < head) add2(s, make_float2(to_f32(p[threadIdx.x]), 0.f));
  for (int64_t k = head + nv * kV + threadIdx.x; k < n; k += kThreads) add2(s, make_float2(to_f32(p[k]), 0.f));
  total.add(s);
}

// Runs fn(tensor, first element, elements) over the CTA's share of the units.
template <int N, typename F>
__device__ __forceinline__ void for_segments(const Table<N>& t, F&& fn) {
  const uint32_t units = t.first[t.n];
  uint32_t u = static_cast<uint32_t>(static_cast<uint64_t>(units) * blockIdx.x / gridDim.x);
  const uint32_t end = static_cast<uint32_t>(static_cast<uint64_t>(units) * (blockIdx.x + 1) / gridDim.x);
  if (u >= end) return;
  int lo = 0, hi = t.n - 1;  // the last tensor whose first unit is at or before u
  while (lo < hi) {
    const int m = (lo + hi + 1) / 2;
    if (t.first[m] <= u) lo = m; else hi = m - 1;
  }
  for (int i = lo; u < end; ++i) {
    const uint32_t stop = min(end, t.first[i + 1]);
    const int64_t a = static_cast<int64_t>(u - t.first[i]) * kUnit;
    const int64_t b = min(static_cast<int64_t>(stop - t.first[i]) * kUnit, t.count[i]);
    fn(i, a, b - a);
    u = stop;
  }
}

// Sums over the CTA; every thread gets them. (All in fp32: a tree of positive
// terms is within its depth x 2^-24, and the fp64 units of this GPU are few.)
__device__ __forceinline__ void block_sum3(float (&v)[3], float (*red)[3]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    v[i] = warp_sum(v[i]);
    if (lane == 0) red[warp][i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 3; ++i) v[i] = warp_sum(lane < kThreads / 32 ? red[lane][i] : 0.f);
}

template <int N>
__global__ void __launch_bounds__(kThreads) grad_sums_kernel(const __grid_constant__ Table<N> t, float* part) {
  __shared__ float red[kThreads / 32][3];
  pdl_trigger();
  pdl_wait();
  Total s;
  for_segments(t, [&](int i, int64_t a, int64_t n) {
    if (t.kind[i] & 1)
      sum_segment(s, static_cast<const bf16*>(t.src[i]) + a, n);
    else
      sum_segment(s, static_cast<const float*>(t.src[i]) + a, n);
  });
  float v[3] = {s.value(0), s.value(1), s.value(2)};
  block_sum3(v, red);
  if (threadIdx.x < 3) part[3 * blockIdx.x + threadIdx.x] = threadIdx.x == 0 ? v[0] : (threadIdx.x == 1 ? v[1] : v[2]);
}

// The norm from the partial sums (the same bits in every CTA).
__device__ __forceinline__ float norm_of(const float* part, int parts, float (*red)[3]) {
  float v[3] = {0.f, 0.f, 0.f};
  for (int p = threadIdx.x; p < parts; p += kThreads)
#pragma unroll
    for (int i = 0; i < 3; ++i) v[i] += part[3 * p + i];
  block_sum3(v, red);
  if (isinf(v[0])) return sqrtf(v[1]) * 0x1p80f;
  if (v[0] < 0x1p-60f) return sqrtf(v[2]) * 0x1p-80f;
  return sqrtf(v[0]);
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const float* part, int parts, float* norm) {
  __shared__ float red[kThreads / 32][3];
  pdl_trigger();
  pdl_wait();
  const float r = norm_of(part, parts, red);
  if (threadIdx.x == 0) norm[0] = r;
}

// c times the elements of 16 bytes of source, stored in the destination's type.
__device__ __forceinline__ void scale_vec(const float*, float* dst, uint4 v, float c) {
  *reinterpret_cast<float4*>(dst) = make_float4(c * __uint_as_float(v.x), c * __uint_as_float(v.y),
                                                c * __uint_as_float(v.z), c * __uint_as_float(v.w));
}
__device__ __forceinline__ void scale_vec(const float*, bf16* dst, uint4 v, float c) {
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(c * __uint_as_float(v.x), c * __uint_as_float(v.y)),
                                              pack_bf16x2(c * __uint_as_float(v.z), c * __uint_as_float(v.w)));
}
__device__ __forceinline__ void scale_vec(const bf16*, bf16* dst, uint4 v, float c) {
  *reinterpret_cast<uint4*>(dst) =
      make_uint4(pack_bf16x2(c * bf16_lo(v.x), c * bf16_hi(v.x)), pack_bf16x2(c * bf16_lo(v.y), c * bf16_hi(v.y)),
                 pack_bf16x2(c * bf16_lo(v.z), c * bf16_hi(v.z)), pack_bf16x2(c * bf16_lo(v.w), c * bf16_hi(v.w)));
}
__device__ __forceinline__ void scale_vec(const bf16*, float* dst, uint4 v, float c) {
  float4* to = reinterpret_cast<float4*>(dst);
  to[0] = make_float4(c * bf16_lo(v.x), c * bf16_hi(v.x), c * bf16_lo(v.y), c * bf16_hi(v.y));
  to[1] = make_float4(c * bf16_lo(v.z), c * bf16_hi(v.z), c * bf16_lo(v.w), c * bf16_hi(v.w));
}

// Each thread reads and writes its own elements only: dst may be src.
template <typename TI, typename TO>
__device__ __forceinline__ void scale_segment(const TI* src, TO* dst, int64_t n, float c) {
  constexpr int kV = 16 / sizeof(TI), kU = 8, kStep = kU * kThreads;
  constexpr int kAlign = kV * sizeof(TO) < 16 ? kV * sizeof(TO) : 16;
  int64_t head = head_of(src, n);
  if (reinterpret_cast<uintptr_t>(dst + head) % kAlign) head = n;  // no common boundary: element by element
  const uint4* v = reinterpret_cast<const uint4*>(src + head);
  TO* const out = dst + head;
  const int64_t nv = (n - head) / kV;
  for (int64_t k = threadIdx.x; k < head; k += kThreads) dst[k] = from_f32<TO>(c * to_f32(src[k]));
  for (int64_t k = head + nv * kV + threadIdx.x; k < n; k += kThreads) dst[k] = from_f32<TO>(c * to_f32(src[k]));
  int64_t i = threadIdx.x;
  uint4 x[kU];
  for (; i + (kU - 1) * kThreads < nv; i += kStep) {
#pragma unroll
    for (int u = 0; u < kU; ++u) x[u] = v[i + u * kThreads];
#pragma unroll
    for (int u = 0; u < kU; ++u) scale_vec(src, out + (i + u * kThreads) * kV, x[u], c);
  }
  if (i < nv) {  // the last batch
#pragma unroll
    for (int u = 0; u < kU; ++u) x[u] = i + u * kThreads < nv ? v[i + u * kThreads] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (i + u * kThreads < nv) scale_vec(src, out + (i + u * kThreads) * kV, x[u], c);
  }
}

// The same where max_norm / norm is below fp32's normal range, and so off by up to all of itself, while the scaled
// elements need not be: (g 2^-80) (1 / (norm 2^-80)) max_norm. Here norm > 2^126 max_norm, so max_norm < 4 and the
// reciprocal is normal; a subnormal product is off by half a step of 2^-149, which max_norm makes at most 2^-148.
// Element by element: norms that large are rare.
__device__ __forceinline__ void scale_segment_far(const void* src, void* dst, int kind, int64_t first, int64_t n,
                                                  float inv, float max_norm) {
  for (int64_t k = first + threadIdx.x; k < first + n; k += kThreads) {
    const float g = kind & 1 ? to_f32(static_cast<const bf16*>(src)[k]) : static_cast<const float*>(src)[k];
    const float r = g * 0x1p-80f * inv * max_norm;
    if (kind & 2)
      static_cast<bf16*>(dst)[k] = from_f32<bf16>(r);
    else
      static_cast<float*>(dst)[k] = r;
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads)
    grad_scale_kernel(const __grid_constant__ Table<N> t, const float* part, int parts, float max_norm, float* norm) {
  __shared__ float red[kThreads / 32][3];
  pdl_trigger();
  pdl_wait();
  const float r = norm_of(part, parts, red);
  if (blockIdx.x == 0 && threadIdx.x == 0) norm[0] = r;
  const float c = (r > max_norm && r < INFINITY) ? max_norm / r : 1.0f;
  if (c < 0x1p-126f && max_norm > 0.f) {
    const float inv = 1.0f / (r * 0x1p-80f);
    for_segments(t, [&](int i, int64_t a, int64_t n) {
      scale_segment_far(t.src[i], t.dst[i], t.kind[i], a, n, inv, max_norm);
    });
    return;
  }
  for_segments(t, [&](int i, int64_t a, int64_t n) {
    if (c == 1.0f && t.src[i] == t.dst[i]) return;
    switch (t.kind[i]) {
      case 0: return scale_segment(static_cast<const float*>(t.src[i]) + a, static_cast<float*>(t.dst[i]) + a, n, c);
      case 1: return scale_segment(static_cast<const bf16*>(t.src[i]) + a, static_cast<float*>(t.dst[i]) + a, n, c);
      case 2: return scale_segment(static_cast<const float*>(t.src[i]) + a, static_cast<bf16*>(t.dst[i]) + a, n, c);
      default: return scale_segment(static_cast<const bf16*>(t.src[i]) + a, static_cast<bf16*>(t.dst[i]) + a, n, c);
    }
  });
}

// Tensors [*next, ...) into the table, empty ones left out, until it is full;
// returns the units taken.
template <int N>
uint32_t fill(Table<N>& t, const GradArgs& a, int* next) {
  t.n = 0;
  uint32_t units = 0;
  for (; *next < a.n && t.n < N; ++*next) {
    const int i = *next;
    if (a.counts[i] == 0) continue;
    t.src[t.n] = a.grads[i];
    t.dst[t.n] = a.outs ? a.outs[i] : nullptr;
    t.count[t.n] = a.counts[i];
    t.kind[t.n] = (a.dtypes[i] == ATTNRES_BF16 ? 1 : 0) | (a.outs && a.out_dtypes[i] == ATTNRES_BF16 ? 2 : 0);
    t.first[t.n] = units;
    units += static_cast<uint32_t>((a.counts[i] - 1) / kUnit + 1);
    ++t.n;
  }
  t.first[t.n] = units;
  return units;
}

unsigned ctas_for(uint32_t units, int per_sm) {
  const unsigned cap = std::min<unsigned>(kMaxCtas, static_cast<unsigned>(per_sm * sm_count()));
  return std::min<unsigned>(units, cap);
}

template <int N>
int run_table(const GradArgs& a, cudaStream_t s) {
  Table<N> t;
  int parts = 0;
  for (int next = 0; next < a.n;) {
    const uint32_t units = fill(t, a, &next);
    if (!units) break;
    const unsigned grid = ctas_for(units, kSumsPerSm);
    const int e = launch_step(
        [&] { return launch_pdl(grad_sums_kernel<N>, grid, kThreads, 0, s, t, a.scratch + 3 * parts); });
    if (e) return e;
    parts += static_cast<int>(grid);
  }
  if (!a.outs || parts == 0)
    return launch_step([&] { return launch_pdl(grad_norm_kernel, 1, kThreads, 0, s, a.scratch, parts, a.norm); });
  for (int next = 0; next < a.n;) {
    const uint32_t units = fill(t, a, &next);
    if (!units) break;
    const unsigned grid = ctas_for(units, kScalePerSm);
    const int e = launch_step([&] {
      return launch_pdl(grad_scale_kernel<N>, grid, kThreads, 0, s, t, a.scratch, parts, a.max_norm, a.norm);
    });
    if (e) return e;
  }
  return ATTNRES_OK;
}

}  // namespace

int64_t grads_scratch(int n) {
  const int64_t launches = n < 1 ? 1 : (static_cast<int64_t>(n) - 1) / kMaxTensors + 1;
  return 3 * kMaxCtas * launches;
}

int run_grads(const GradArgs& a, cudaStream_t s) {
  if (a.n <= 32) return run_table<32>(a, s);
  if (a.n <= 256) return run_table<256>(a, s);
  return run_table<kMaxTensors>(a, s);
}

}  // namespace attnres
