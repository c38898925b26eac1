// 8-bit rows: writing them, reading them back, and laying out a weight matrix
// (the format and its rounding are described in attnres.h).
//
// Writing takes one pass: L lanes hold 16 consecutive features of a row each,
// so 8 lanes share a group of 128; its largest magnitude is three shuffles
// away, the scale follows from its bits, and the codes, the exponents and the
// row's mean square (of the values the codes stand for) leave together. Both
// kernels are bound by the bytes they stream; several 16-byte loads a thread
// are issued before the first is used.
#include "q8.cuh"

namespace attnres {
namespace {

constexpr int kThreads = 256;

// Raw storage of 16 features.
template <typename T> struct Raw16 {
  static constexpr int kVecs = sizeof(T);  // 16-byte vectors: 2 of bf16, 4 of fp32
  uint4 v[kVecs];
};

// Features [k0, k0 + 16) of a row, zero from d on. `vec`: rows start on
// 16-byte boundaries and d is a whole number of 16-byte vectors.
template <typename T>
__device__ __forceinline__ void load_raw(const T* row, int k0, int d, bool vec, Raw16<T>& r) {
  constexpr int kPer = 16 / sizeof(T);
  if (vec) {
#pragma unroll
    for (int i = 0; i < Raw16<T>::kVecs; ++i)
      r.v[i] = k0 + i * kPer < d ? __ldcs(reinterpret_cast<const uint4*>(row + k0) + i) : make_uint4(0, 0, 0, 0);
  } else {
    T* e = reinterpret_cast<T*>(r.v);
#pragma unroll
    for (int i = 0; i < 16; ++i) e[i] = k0 + i < d ? row[k0 + i] : from_f32<T>(0.f);
  }
}

__device__ __forceinline__ void widen(const Raw16<bf16>& r, float (&x)[16]) {
  const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ void widen(const Raw16<float>& r, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[4 * i] = __uint_as_float(r.v[i].x);
    x[4 * i + 1] = __uint_as_float(r.v[i].y);
    x[4 * i + 2] = __uint_as_float(r.v[i].z);
    x[4 * i + 3] = __uint_as_float(r.v[i].w);
  }
}

// The largest of a value over the 8 lanes of a group.
__device__ __forceinline__ float max8(float a) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}

// The group's exponent from its 16 features on each of 8 lanes. fmaxf passes
// over a NaN; a group with an infinity is looked at again without it, and its
// infinities become NaN. Every lane of the warp takes part.
__device__ __forceinline__ uint32_t group_exponent(float (&x)[16]) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(x[i]));
  a = max8(a);
  if (__any_sync(0xffffffffu, __float_as_uint(a) >= kInfBits)) {
    a = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if ((__float_as_uint(x[i]) & 0x7fffffffu) >= kInfBits) x[i] = __uint_as_float(0x7fffffffu);
      a = fmaxf(a, fabsf(x[i]));
    }
    a = max8(a);
  }
  return q8_exponent(__float_as_uint(a));
}

__device__ __forceinline__ uint4 encode16(const float (&x)[16], uint32_t e) {
  const float inv = q8_inverse(e), top = q8_top(e);
  float y[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = x[i] * inv;
  if (e == 247u) {  // elsewhere no magnitude passes 448; a NaN stays one
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = fabsf(y[i]) > top ? copysignf(top, y[i]) : y[i];
  }
  return make_uint4(encode4(y[0], y[1], y[2], y[3]), encode4(y[4], y[5], y[6], y[7]),
                    encode4(y[8], y[9], y[10], y[11]), encode4(y[12], y[13], y[14], y[15]));
}

// L lanes a row (8: 4 rows a warp, each lane a chunk of every group; 32: a row
// a warp, 4 groups at a time). kBatch chunks a lane are loaded at once.
template <typename T, int L>
__global__ void __launch_bounds__(kThreads) q8_write_kernel(Q8Rows a, int G, int vec) {
  constexpr int kRows = 32 / L;
  constexpr int kBatch = sizeof(T) == 2 ? 4 : 2;
  const int lane = threadIdx.x & 31, j = lane % L, sub = lane / L;
  const int chunks = 8 * G, steps = (chunks + L - 1) / L;
  const int mean_at = q8_mean_offset(G), tail_bytes = q8_tail_bytes(G);
  const int64_t source = q8_source_bytes(a.cap, a.d);
  const int64_t total = static_cast<int64_t>(a.n) * a.T;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  pdl_trigger();
  pdl_wait();
  for (int64_t r0 = (static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * kRows; r0 < total;
       r0 += warps * kRows) {
    const int64_t r = r0 + sub;
    const bool valid = r < total;
    const int64_t i = valid ? r / a.T : 0, t = valid ? r - i * a.T : 0;
    const T* x = static_cast<const T*>(a.x) + i * a.x_stride + t * a.d;
    unsigned char* out = static_cast<unsigned char*>(a.rows) + i * source + t * (128 * G);
    unsigned char* tail = static_cast<unsigned char*>(a.rows) + i * source + a.cap * (128 * G) + t * tail_bytes;
    const int d = valid ? a.d : 0;  // lanes behind the last row read nothing
    float ms = 0.f;
    for (int c0 = 0; c0 < steps; c0 += kBatch) {
      Raw16<T> raw[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) load_raw(x, ((c0 + b) * L + j) * 16, d, vec, raw[b]);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (c0 + b >= steps) break;  // the same for every lane
        const int chunk = (c0 + b) * L + j;
        float v[16];
        widen(raw[b], v);
        const uint32_t e = group_exponent(v);
        const uint4 code = encode16(v, e);
        float2 w[8], q = make_float2(0.f, 0.f);
        decode16(code, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) q = ffma2(w[k], w[k], q);
        const float s = q8_scale(e);
        ms += (q.x + q.y) * s * s;
        if (valid && chunk < chunks) {
          *reinterpret_cast<uint4*>(out + chunk * 16) = code;
          if ((j & 7) == 0) tail[chunk >> 3] = static_cast<unsigned char>(e);
        }
      }
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) ms += __shfl_xor_sync(0xffffffffu, ms, o);
    if (valid && j == 0) {
      for (int k = G; k < mean_at; ++k) tail[k] = 0;
      *reinterpret_cast<float*>(tail + mean_at) = ms / static_cast<float>(a.d);
      for (int k = mean_at + 4; k < tail_bytes; k += 4) *reinterpret_cast<uint32_t*>(tail + k) = 0;
    }
  }
}

// 16 values into features [k0, k0 + 16) of a row; none from d on.
__device__ __forceinline__ void store_row16(bf16* row, int k0, int d, bool vec, const float2 (&v)[8]) {
  if (vec) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (k0 + 8 * h < d)
        __stcs(reinterpret_cast<uint4*>(row + k0) + h,
               make_uint4(pack_bf16x2(v[4 * h].x, v[4 * h].y), pack_bf16x2(v[4 * h + 1].x, v[4 * h + 1].y),
                          pack_bf16x2(v[4 * h + 2].x, v[4 * h + 2].y), pack_bf16x2(v[4 * h + 3].x, v[4 * h + 3].y)));
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (k0 + i < d) row[k0 + i] = __float2bfloat16_rn(i & 1 ? v[i >> 1].y : v[i >> 1].x);
  }
}
__device__ __forceinline__ void store_row16(float* row, int k0, int d, bool vec, const float2 (&v)[8]) {
  if (vec) {
#pragma unroll
    for (int h = 0; h < 4; ++h)
      if (k0 + 4 * h < d)
        __stcs(reinterpret_cast<float4*>(row + k0) + h, make_float4(v[2 * h].x, v[2 * h].y, v[2 * h + 1].x, v[2 * h + 1].y));
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (k0 + i < d) row[k0 + i] = i & 1 ? v[i >> 1].y : v[i >> 1].x;
  }
}

template <typename T, int L>
__global__ void __launch_bounds__(kThreads) q8_back_kernel(Q8Rows a, int G, int vec) {
  constexpr int kRows = 32 / L, kBatch = 4;
  const int lane = threadIdx.x & 31, j = lane % L, sub = lane / L;
  const int chunks = 8 * G, steps = (chunks + L - 1) / L;
  const int64_t source = q8_source_bytes(a.cap, a.d);
  const int64_t total = static_cast<int64_t>(a.n) * a.T;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  pdl_trigger();
  pdl_wait();
  for (int64_t r = (static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * kRows + sub; r < total;
       r += warps * kRows) {
    const int64_t i = r / a.T, t = r - i * a.T;
    T* out = static_cast<T*>(const_cast<void*>(a.x)) + i * a.x_stride + t * a.d;
    const unsigned char* row = static_cast<const unsigned char*>(a.rows) + i * source + t * (128 * G);
    const unsigned char* tail =
        static_cast<const unsigned char*>(a.rows) + i * source + a.cap * (128 * G) + t * q8_tail_bytes(G);
    for (int c0 = 0; c0 < steps; c0 += kBatch) {
      uint4 code[kBatch];
      uint32_t e[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int chunk = (c0 + b) * L + j;
        const bool in = chunk < chunks;
        code[b] = in ? __ldcs(reinterpret_cast<const uint4*>(row) + chunk) : make_uint4(0, 0, 0, 0);
        e[b] = in ? tail[chunk >> 3] : 1u;
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int chunk = (c0 + b) * L + j;
        if (chunk >= chunks) break;
        float2 v[8];
        decode16(code[b], v);
        const float s = q8_scale(e[b]);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = fmul2(v[k], make_float2(s, s));
        store_row16(out, chunk * 16, a.d, vec, v);
      }
    }
  }
}

// One CTA per block of 128 x 128 weights, 64 of them a thread, held in
// registers between the search for the largest and the rounding.
template <typename T>
__global__ void __launch_bounds__(kThreads) q8_weight_kernel(const T* W, int m, int d, int G, unsigned char* W8) {
  __shared__ float part[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  const int bm = blockIdx.x / G, bk = blockIdx.x - bm * G;
  const int col = bk * 128 + (threadIdx.x & 127), row0 = bm * 128 + (threadIdx.x >> 7);
  float x[64];
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    const int row = row0 + 2 * i;
    x[i] = row < m && col < d ? to_f32(W[static_cast<int64_t>(row) * d + col]) : 0.f;
    // only finite magnitudes count; what is not finite becomes NaN
    if ((__float_as_uint(x[i]) & 0x7fffffffu) >= kInfBits)
      x[i] = __uint_as_float(0x7fffffffu);
    else
      a = fmaxf(a, fabsf(x[i]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
  __syncthreads();
  a = 0.f;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) a = fmaxf(a, part[i]);
  const uint32_t e = q8_exponent(__float_as_uint(a));
  const float inv = q8_inverse(e), top = q8_top(e);
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    const int row = row0 + 2 * i;
    float y = x[i] * inv;
    if (fabsf(y) > top) y = copysignf(top, y);
    if (row < m) W8[static_cast<int64_t>(row) * (128 * G) + col] = static_cast<unsigned char>(encode4(y, 0.f, 0.f, 0.f));
  }
  // The exponents, and with the row's last block the zeros behind them.
  const int stride = q8_block_row(G);
  unsigned char* ex = W8 + static_cast<int64_t>(m) * (128 * G) + static_cast<int64_t>(bm) * stride;
  if (threadIdx.x == 0) ex[bk] = static_cast<unsigned char>(e);
  if (bk == G - 1)
    for (int k = G + threadIdx.x; k < stride; k += kThreads) ex[k] = 0;
}

// Rows of the other side that start on 16-byte boundaries and hold whole vectors.
bool rows_vec(const Q8Rows& a) {
  const int64_t es = a.bf16 ? 2 : 4;
  return aligned16(a.x) && a.d * es % 16 == 0 && (a.n == 1 || a.x_stride * es % 16 == 0);
}

unsigned row_grid(int64_t rows, int per_warp) {
  const int64_t blocks = (rows + per_warp * (kThreads / 32) - 1) / (per_warp * (kThreads / 32));
  const int64_t cap = static_cast<int64_t>(sm_count()) * 8;
  return static_cast<unsigned>(blocks < cap ? blocks : cap);
}

template <typename T>
cudaError_t write_as(const Q8Rows& a, cudaStream_t s) {
  const int G = q8_groups(a.d), vec = rows_vec(a);
  const int64_t rows = a.n * a.T;
  if (G <= 8) return launch_pdl(q8_write_kernel<T, 8>, row_grid(rows, 4), kThreads, 0, s, a, G, vec);
  return launch_pdl(q8_write_kernel<T, 32>, row_grid(rows, 1), kThreads, 0, s, a, G, vec);
}

template <typename T>
cudaError_t back_as(const Q8Rows& a, cudaStream_t s) {
  const int G = q8_groups(a.d), vec = rows_vec(a);
  const int64_t rows = a.n * a.T;
  if (G <= 8) return launch_pdl(q8_back_kernel<T, 8>, row_grid(rows, 4), kThreads, 0, s, a, G, vec);
  return launch_pdl(q8_back_kernel<T, 32>, row_grid(rows, 1), kThreads, 0, s, a, G, vec);
}

}  // namespace

cudaError_t launch_q8_write(const Q8Rows& a, cudaStream_t s) {
  return a.bf16 ? write_as<bf16>(a, s) : write_as<float>(a, s);
}

cudaError_t launch_q8_back(const Q8Rows& a, cudaStream_t s) { return a.bf16 ? back_as<bf16>(a, s) : back_as<float>(a, s); }

cudaError_t launch_q8_weight(const void* W, int m, int d, int is_bf16, void* W8, cudaStream_t s) {
  const int G = q8_groups(d);
  const int64_t blocks = static_cast<int64_t>(q8_groups(m)) * G;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  unsigned char* out = static_cast<unsigned char*>(W8);
  if (is_bf16)
    return launch_pdl(q8_weight_kernel<bf16>, static_cast<unsigned>(blocks), kThreads, 0, s, static_cast<const bf16*>(W), m,
                      d, G, out);
  return launch_pdl(q8_weight_kernel<float>, static_cast<unsigned>(blocks), kThreads, 0, s, static_cast<const float*>(W), m,
                    d, G, out);
}

}  // namespace attnres
