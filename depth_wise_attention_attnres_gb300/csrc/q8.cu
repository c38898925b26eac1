// 8-bit rows: writing them, reading them back, and laying out a weight matrix
// (the format and its rounding are described in attnres.h).
//
// Writing takes one pass: 8 lanes hold a group of 128 features, 16 each, so its
// largest magnitude is three shuffles away; the scale follows from its bits,
// and the codes, the exponents and the row's mean square (of the values the
// codes stand for) leave together. Both directions are bound by the bytes they
// stream, and several loads a thread are issued before the first is used.
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

// a / b of values that are not negative: 32-bit where both fit (the 64-bit division is a long subroutine).
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  return ((a | b) >> 32) ? a / b : static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
}

// Row number r of n sources of T rows: its source and token, and the row `step` further on.
struct RowAt {
  int64_t i, t;
  __device__ __forceinline__ RowAt(int64_t r, int64_t T) : i(r < T ? 0 : divide(r, T)), t(r < T ? r : r - i * T) {}
  __device__ __forceinline__ void advance(int64_t step, int64_t T) {
    t += step;
    if (t >= T) {
      const int64_t q = t < 2 * T ? 1 : divide(t, T);
      i += q;
      t -= q * T;
    }
  }
};

// L lanes a row: 8 up to 8 groups (4 rows a warp, each lane 16 features of every
// group), 32 beyond (a row a warp, 4 groups at a time). A warp writes a row's
// tail with one 16-byte store (L = 8) or a word a step: with a byte a group,
// narrow rows took 51 us where they now take 32 (262144 rows of 128, bf16).
template <typename T, int L>
__global__ void __launch_bounds__(kThreads) q8_write_kernel(Q8Rows a, int G, int vec) {
  constexpr int kRows = 32 / L;
  constexpr int kBatch = sizeof(T) == 2 ? 4 : 2;  // steps of a row loaded at once
  const int lane = threadIdx.x & 31, j = lane % L;
  const int chunks = 8 * G, steps = (chunks + L - 1) / L;
  const int mean_at = q8_mean_offset(G), tail_bytes = q8_tail_bytes(G);
  const int64_t source = q8_source_bytes(a.cap, a.d);
  const int64_t total = static_cast<int64_t>(a.n) * a.T;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32) * kRows;  // rows between a warp's
  pdl_trigger();
  pdl_wait();
  int64_t r = (static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * kRows + lane / L;
  RowAt at(r, a.T);
  for (; r - lane / L < total; r += step, at.advance(step, a.T)) {  // the same for every lane of the warp
    const bool valid = r < total;
    const int64_t i = valid ? at.i : 0, t = valid ? at.t : 0;
    const T* x = static_cast<const T*>(a.x) + i * a.x_stride + t * a.d;
    unsigned char* out = static_cast<unsigned char*>(a.rows) + i * source + t * (128 * G);
    unsigned char* tail = static_cast<unsigned char*>(a.rows) + i * source + a.cap * (128 * G) + t * tail_bytes;
    const int d = valid ? a.d : 0;  // lanes behind the last row read and write nothing
    float ms = 0.f;
    uint32_t words[2] = {0, 0};  // L = 8: the row's exponents, two words at most
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
        float2 w[8], m2 = make_float2(0.f, 0.f);
        decode16(code, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) m2 = ffma2(w[k], w[k], m2);
        const float s = q8_scale(e);
        ms += (m2.x + m2.y) * s * s;
        if (valid && chunk < chunks) *reinterpret_cast<uint4*>(out + chunk * 16) = code;
        if constexpr (L == 8) {
          words[0] |= c0 + b < 4 ? e << (8 * (c0 + b)) : 0;
          words[1] |= c0 + b < 4 ? 0 : e << (8 * (c0 + b - 4));
        } else {  // four groups' exponents a step: one word of the tail
          uint32_t word = chunk < chunks ? e << (8 * (j >> 3)) : 0;
          word |= __shfl_xor_sync(0xffffffffu, word, 8);
          word |= __shfl_xor_sync(0xffffffffu, word, 16);
          if (valid && j == 0) reinterpret_cast<uint32_t*>(tail)[c0 + b] = word;
        }
      }
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) ms += __shfl_xor_sync(0xffffffffu, ms, o);
    if (valid && j == 0) {
      const float mean = ms / static_cast<float>(a.d);
      if constexpr (L == 8) {
        const uint32_t m = __float_as_uint(mean);
        *reinterpret_cast<uint4*>(tail) = make_uint4(words[0], G <= 4 ? m : words[1], G <= 4 ? 0 : m, 0);
      } else {
        *reinterpret_cast<float*>(tail + mean_at) = mean;
        for (int k = mean_at + 4; k < tail_bytes; k += 4) *reinterpret_cast<uint32_t*>(tail + k) = 0;
      }
    }
  }
}

// Walks the rows of n sources of T rows, `step` rows at a time: where row r lies
// in the [T, d] slices, the codes and the tails. A step adds a constant to each
// place and, past a source's last row, one more. For reading back, whose lanes go from row
// to row by themselves (64 x 8192 x 896: 230 us, 255 with RowAt); the kernels
// whose warps work on a row together are faster with RowAt (65536 x 896 written in 32 us, 38).
template <typename T_>
struct RowWalk {
  T_* x;
  unsigned char *code, *tail;
  int64_t t, T, step_t;                  // row in the source
  int64_t step_x, step_code, step_tail;  // a step without leaving the source
  int64_t wrap_x, wrap_code, wrap_tail;  // past the last row, in addition
  __device__ __forceinline__ RowWalk(const Q8Rows& a, int G, int64_t r, int64_t step) : T(a.T) {
    const int64_t source = q8_source_bytes(a.cap, a.d), width = 128 * G, tail_bytes = q8_tail_bytes(G);
    const int64_t i = divide(r, T), step_i = divide(step, T);
    t = r - i * T;
    step_t = step - step_i * T;
    x = static_cast<T_*>(const_cast<void*>(a.x)) + i * a.x_stride + t * a.d;
    code = static_cast<unsigned char*>(a.rows) + i * source + t * width;
    tail = static_cast<unsigned char*>(a.rows) + i * source + a.cap * width + t * tail_bytes;
    step_x = step_i * a.x_stride + step_t * a.d;
    step_code = step_i * source + step_t * width;
    step_tail = step_i * source + step_t * tail_bytes;
    wrap_x = a.x_stride - T * a.d;
    wrap_code = source - T * width;
    wrap_tail = source - T * tail_bytes;
  }
  __device__ __forceinline__ void advance() {
    t += step_t;
    x += step_x;
    code += step_code;
    tail += step_tail;
    if (t >= T) {
      t -= T;
      x += wrap_x;
      code += wrap_code;
      tail += wrap_tail;
    }
  }
};

// Reading back: a lane's piece is the codes of 16 bytes of output (8 of bf16, 4
// of fp32), so L lanes (16 or 32, all of a warp where the row is long enough)
// read and write whole lines. kBatch pieces a lane are loaded at once, of one row or of several.
template <typename T, int L>
__global__ void __launch_bounds__(kThreads) q8_back_kernel(Q8Rows a, int G) {
  constexpr int kPer = 16 / sizeof(T), kRows = 32 / L, kBatch = 8;
  const int lane = threadIdx.x & 31, j = lane % L;
  const int64_t total = static_cast<int64_t>(a.n) * a.T;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32) * kRows;
  pdl_trigger();
  pdl_wait();
  int64_t r = (static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * kRows + lane / L;
  RowWalk<T> at(a, G, r, step);
  int k = j * kPer;  // the lane's next piece, in row r
  if (k >= a.d) return;
  while (r < total) {
    uint2 code[kBatch];
    uint32_t e[kBatch];
    T* to[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      to[b] = nullptr;
      e[b] = 1;
      code[b] = make_uint2(0, 0);
      if (r < total) {
        if (kPer == 8)
          code[b] = __ldcs(reinterpret_cast<const uint2*>(at.code + k));
        else
          code[b].x = __ldcs(reinterpret_cast<const uint32_t*>(at.code + k));
        e[b] = at.tail[k >> 7];
        to[b] = at.x + k;
        k += L * kPer;
        if (k >= a.d) {
          k = j * kPer;
          r += step;
          at.advance();
        }
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (!to[b]) continue;
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
        __stcs(reinterpret_cast<uint4*>(to[b]), make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y),
                                                          pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y)));
      } else {
        __stcs(reinterpret_cast<float4*>(to[b]), make_float4(v[0].x, v[0].y, v[1].x, v[1].y));
      }
    }
  }
}

// The same into rows that do not start on 16-byte boundaries: an element a lane,
// so that a warp still writes consecutive elements (16384 rows of 1001 to bf16, four
// sources: 53 us; with 16 elements a lane 348).
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
    const int64_t i = divide(r, a.T), t = r - i * a.T;
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

// Weights: a CTA a block of 128 x 128, 64 of them a thread as pieces of 16 bytes, so that a
// warp reads and writes whole lines; with `vec` rows start on 16-byte boundaries and
// hold whole pieces. They stay in registers between the search for the largest magnitude
// and the rounding (2048 x 2048 bf16: 5.2 us, 17.9 with an element a lane; 16384 x 16384 fp32: 242 us,
// 0.82 of the copy rate).
template <typename T>
__global__ void __launch_bounds__(kThreads) q8_weight_kernel(const T* W, int m, int d, int G, int vec, unsigned char* W8) {
  constexpr int kPer = 16 / sizeof(T), kAcross = 128 / kPer, kDown = kThreads / kAcross, kPieces = 128 / kDown;
  __shared__ float part[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  const int bm = blockIdx.x / G, bk = blockIdx.x - bm * G;
  const int col = bk * 128 + threadIdx.x % kAcross * kPer, row0 = bm * 128 + threadIdx.x / kAcross;
  float x[kPieces][kPer];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int row = row0 + i * kDown;
    const T* w = W + static_cast<int64_t>(row) * d + col;
    uint4 piece = make_uint4(0, 0, 0, 0);
    T* e = reinterpret_cast<T*>(&piece);
    if (row < m) {
      if (vec) {
        if (col < d) piece = __ldcs(reinterpret_cast<const uint4*>(w));
      } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k)
          if (col + k < d) e[k] = w[k];
      }
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) x[i][k] = to_f32(e[k]);
  }
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      // only finite magnitudes count; what is not finite becomes NaN
      if ((__float_as_uint(x[i][k]) & 0x7fffffffu) >= kInfBits)
        x[i][k] = __uint_as_float(0x7fffffffu);
      else
        a = fmaxf(a, fabsf(x[i][k]));
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
  for (int i = 0; i < kPieces; ++i) {
    const int row = row0 + i * kDown;
    if (row >= m) break;
    uint32_t code[kPer / 4];
#pragma unroll
    for (int q = 0; q < kPer / 4; ++q) {
      float y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        y[k] = x[i][4 * q + k] * inv;
        if (fabsf(y[k]) > top) y[k] = copysignf(top, y[k]);
      }
      code[q] = encode4(y[0], y[1], y[2], y[3]);
    }
    unsigned char* to = W8 + static_cast<int64_t>(row) * (128 * G) + col;
    if constexpr (kPer == 8)
      *reinterpret_cast<uint2*>(to) = make_uint2(code[0], code[1]);
    else
      *reinterpret_cast<uint32_t*>(to) = code[0];
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
  const int64_t cap = static_cast<int64_t>(sm_count()) * 16;
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
  const int vec = aligned16(W) && d % (is_bf16 ? 8 : 4) == 0;
  if (is_bf16)
    return launch_pdl(q8_weight_kernel<bf16>, static_cast<unsigned>(blocks), kThreads, 0, s, static_cast<const bf16*>(W), m,
                      d, G, vec, out);
  return launch_pdl(q8_weight_kernel<float>, static_cast<unsigned>(blocks), kThreads, 0, s, static_cast<const float*>(W), m,
                    d, G, vec, out);
}

}  // namespace attnres
