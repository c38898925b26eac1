// 8-bit rows: writing them, reading them back, and laying out a weight matrix
// (the format and its rounding are described in attnres.h).
//
// Writing takes one pass: 8 lanes hold a group of 128 features, 16 each, so its
// largest magnitude is three shuffles away; the scale follows from its bits,
// and the codes, the exponents and the row's mean square (of the values the
// codes stand for) leave together. Both directions are bound by the bytes they
// stream: every load and store of a warp covers whole 128-byte lines (a lane's 16
// features are two or four pieces, 8 lanes apart), and several loads a thread
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

// A lane's 16 features of group g: piece i holds the 16 bytes from feature
// 128 g + (8 i + j) kPer on (lane j of 8), zero from d on. `vec`: rows start on
// 16-byte boundaries and d is a whole number of 16-byte vectors.
template <typename T>
__device__ __forceinline__ void load_raw(const T* row, int g, int j, int d, bool vec, Raw16<T>& r) {
  constexpr int kPer = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < Raw16<T>::kVecs; ++i) {
    const int k = g * 128 + (i * 8 + j) * kPer;
    if (vec) {
      r.v[i] = k < d ? __ldcs(reinterpret_cast<const uint4*>(row + k)) : make_uint4(0, 0, 0, 0);
    } else {
      T* e = reinterpret_cast<T*>(&r.v[i]);
#pragma unroll
      for (int q = 0; q < kPer; ++q) e[q] = k + q < d ? row[k + q] : from_f32<T>(0.f);
    }
  }
}

// The codes of such features, in the same places.
__device__ __forceinline__ void store_codes(unsigned char* group, int j, const uint4& c, bf16) {
  reinterpret_cast<uint2*>(group)[j] = make_uint2(c.x, c.y);
  reinterpret_cast<uint2*>(group)[8 + j] = make_uint2(c.z, c.w);
}
__device__ __forceinline__ void store_codes(unsigned char* group, int j, const uint4& c, float) {
  uint32_t* at = reinterpret_cast<uint32_t*>(group) + j;
  at[0] = c.x;
  at[8] = c.y;
  at[16] = c.z;
  at[24] = c.w;
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

// L lanes a row (8: 4 rows a warp, one group of each at a time; 32: a row a
// warp, 4 groups at a time). kBatch groups a lane are loaded at once.
template <typename T, int L>
__global__ void __launch_bounds__(kThreads) q8_write_kernel(Q8Rows a, int G, int vec) {
  constexpr int kRows = 32 / L;
  constexpr int kBatch = sizeof(T) == 2 ? 4 : 2;
  const int lane = threadIdx.x & 31, j = lane % L, sub = lane / L;
  const int steps = (8 * G + L - 1) / L, gj = j >> 3, j8 = j & 7;
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
      for (int b = 0; b < kBatch; ++b) load_raw(x, (c0 + b) * (L / 8) + gj, j8, d, vec, raw[b]);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (c0 + b >= steps) break;  // the same for every lane
        const int g = (c0 + b) * (L / 8) + gj;
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
        if (valid && g < G) {
          store_codes(out + g * 128, j8, code, T());
          if (j8 == 0) tail[g] = static_cast<unsigned char>(e);
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

// Reading back: a lane's piece is the codes of 16 bytes of output (8 of bf16, 4
// of fp32), so L lanes (16 or 32, all of a warp where the row is long enough)
// read and write whole lines. kBatch pieces a lane are loaded at once.
template <typename T, int L>
__global__ void __launch_bounds__(kThreads) q8_back_kernel(Q8Rows a, int G) {
  constexpr int kPer = 16 / sizeof(T), kRows = 32 / L, kBatch = 8;
  const int lane = threadIdx.x & 31, j = lane % L;
  const int64_t source = q8_source_bytes(a.cap, a.d);
  const int64_t total = static_cast<int64_t>(a.n) * a.T;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  const int pieces = (a.d + kPer - 1) / kPer;
  pdl_trigger();
  pdl_wait();
  for (int64_t r = (static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * kRows + lane / L; r < total;
       r += warps * kRows) {
    const int64_t i = r / a.T, t = r - i * a.T;
    T* out = static_cast<T*>(const_cast<void*>(a.x)) + i * a.x_stride + t * a.d;
    const unsigned char* row = static_cast<const unsigned char*>(a.rows) + i * source + t * (128 * G);
    const unsigned char* tail =
        static_cast<const unsigned char*>(a.rows) + i * source + a.cap * (128 * G) + t * q8_tail_bytes(G);
    for (int p0 = j; p0 < pieces; p0 += kBatch * L) {
      uint2 code[kBatch];
      uint32_t e[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int k = (p0 + b * L) * kPer;
        code[b] = make_uint2(0, 0);
        e[b] = 1;
        if (k < a.d) {
          if (kPer == 8)
            code[b] = __ldcs(reinterpret_cast<const uint2*>(row + k));
          else
            code[b].x = __ldcs(reinterpret_cast<const uint32_t*>(row + k));
          e[b] = tail[k >> 7];
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int k = (p0 + b * L) * kPer;
        if (k >= a.d) break;
        const float s = q8_scale(e[b]);
        const float2 s2 = make_float2(s, s);
        float2 v[4];
        decode4(code[b].x, v[0], v[1]);
        v[0] = fmul2(v[0], s2);
        v[1] = fmul2(v[1], s2);
        if constexpr (kPer == 8) {
          decode4(code[b].y, v[2], v[3]);
          v[2] = fmul2(v[2], s2);
          v[3] = fmul2(v[3], s2);
          __stcs(reinterpret_cast<uint4*>(out + k), make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y),
                                                               pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y)));
        } else {
          __stcs(reinterpret_cast<float4*>(out + k), make_float4(v[0].x, v[0].y, v[1].x, v[1].y));
        }
      }
    }
  }
}

// The same into rows that do not start on 16-byte boundaries: an element a lane,
// so that a warp still writes consecutive elements (16384 rows of 1001 to bf16, four
// sources: TIME us; with 16 elements a lane 348).
template <typename T>
__global__ void __launch_bounds__(kThreads) q8_back_element_kernel(Q8Rows a, int G) {
  constexpr int kBatch = 8;
  const int lane = threadIdx.x & 31;
  const int64_t source = q8_source_bytes(a.cap, a.d);
  const int64_t total = static_cast<int64_t>(a.n) * a.T;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  pdl_trigger();
  pdl_wait();
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); r < total; r += warps) {
    const int64_t i = r / a.T, t = r - i * a.T;
    T* out = static_cast<T*>(const_cast<void*>(a.x)) + i * a.x_stride + t * a.d;
    const unsigned char* row = static_cast<const unsigned char*>(a.rows) + i * source + t * (128 * G);
    const unsigned char* tail =
        static_cast<const unsigned char*>(a.rows) + i * source + a.cap * (128 * G) + t * q8_tail_bytes(G);
    for (int k0 = lane; k0 < a.d; k0 += kBatch * 32) {
      uint32_t code[kBatch], e[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int k = k0 + b * 32;
        code[b] = k < a.d ? row[k] : 0u;
        e[b] = k < a.d ? tail[k >> 7] : 1u;
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int k = k0 + b * 32;
        if (k < a.d) out[k] = from_f32<T>(f16x2_f32(e4m3x2_f16x2(static_cast<uint16_t>(code[b]))).x * q8_scale(e[b]));
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
  const int G = q8_groups(a.d);
  const int64_t rows = a.n * a.T;
  if (!rows_vec(a)) return launch_pdl(q8_back_element_kernel<T>, row_grid(rows, 1), kThreads, 0, s, a, G);
  if (a.d * static_cast<int>(sizeof(T)) <= 256) return launch_pdl(q8_back_kernel<T, 16>, row_grid(rows, 2), kThreads, 0, s, a, G);
  return launch_pdl(q8_back_kernel<T, 32>, row_grid(rows, 1), kThreads, 0, s, a, G);
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
