// Projection of 8-bit rows by an 8-bit weight matrix (attnres.h): Q = V W^T with
// V [T, d] in e4m3 and one power-of-two scale for each row and group of 128
// features, W [m, d] in e4m3 and one for each 128 x 128 block, Q fp32.
//
// q8_proj_tc_kernel: the tensor cores, tcgen05.mma kind::f8f6f4 (M = 128, N =
// BN, K = 32). The scales change every 128 features, so each such block is
// summed on its own in tensor memory and the epilogue warps add it, scaled,
// onto fp32 sums in registers: sum[t, j] += 2^(ea[t] + eb[j]) * block[t, j], one
// multiply-add an output and block, where the tensor cores do 128. Blocks take
// turns in 512 / BN accumulators, so the MMAs of the next blocks run
// meanwhile. Operands arrive as in the bf16 projection: TMA copies of 128-byte
// rows (128 codes, one block) in the 128-byte swizzle, straight from the rows'
// records, whose exponents a thread of the epilogue reads 16 blocks at a time.
//
// q8_proj_rows_kernel: few tokens. Bound by the weights' bytes and by latency,
// so the work is spread over the SMs by output features and by d: a warp takes
// 4 output features, 8 tokens and up to 512 features of d at a time, with fp32
// multiply-adds, and the KS warps that share an output add up through shared memory.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "q8.cuh"
#include "tcgen05.cuh"

namespace attnres {
namespace {

__device__ unsigned int g_q8_proj_timeout = 0;

// ------------------------------------------------------------- few tokens --
constexpr int kRowCols = 4, kRowTokens = 8, kRowThreads = 128;

template <int KS>
__global__ void __launch_bounds__(kRowThreads) q8_proj_rows_kernel(const unsigned char* rows, int64_t T, int d, int rec,
                                                                    const unsigned char* W8, int m, float* Q, int64_t tgroups) {
  constexpr int kColGroups = 4 / KS;
  __shared__ float part[4][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ks = warp % KS;
  const int G = q8_groups(d), chunks = 8 * G;
  const int64_t cg = blockIdx.x / tgroups;
  const int64_t t0 = (blockIdx.x - cg * tgroups) * kRowTokens;
  const int64_t j0 = (cg * kColGroups + warp / KS) * kRowCols;
  const unsigned char* ex = W8 + static_cast<int64_t>(m) * (128 * G);
  const int exrow = q8_block_row(G);
  pdl_trigger();
  pdl_wait();
  const int nt = T - t0 < kRowTokens ? static_cast<int>(T - t0) : kRowTokens;
  float acc[kRowTokens * kRowCols];
#pragma unroll
  for (int i = 0; i < kRowTokens * kRowCols; ++i) acc[i] = 0.f;
  if (j0 < m) {
    for (int ch = ks * 32 + lane; ch < chunks; ch += KS * 32) {
      uint4 wc[kRowCols], xc[kRowTokens];
#pragma unroll
      for (int c = 0; c < kRowCols; ++c) {
        const int64_t j = j0 + c < m ? j0 + c : m - 1;
        wc[c] = __ldg(reinterpret_cast<const uint4*>(W8 + j * (128 * G)) + ch);
      }
#pragma unroll
      for (int t = 0; t < kRowTokens; ++t)
        xc[t] = t < nt ? __ldg(reinterpret_cast<const uint4*>(rows + (t0 + t) * rec) + ch) : make_uint4(0, 0, 0, 0);
      const uint32_t eb = ex[(j0 >> 7) * exrow + (ch >> 3)];  // 4 columns lie in one block
      float2 w[kRowCols][8];
#pragma unroll
      for (int c = 0; c < kRowCols; ++c) decode16(wc[c], w[c]);
#pragma unroll
      for (int t = 0; t < kRowTokens; ++t) {
        if (t < nt) {
          const uint32_t ea = rows[(t0 + t) * rec + 128 * G + (ch >> 3)];
          float2 x[8];
          decode16(xc[t], x);
          // 2^e, e from -252 to 240, in two factors that are normal fp32 numbers.
          const int e = static_cast<int>(ea + eb) - 254, e1 = e >> 1;
          const float fa = q8_scale(static_cast<uint32_t>(e1 + 127)), fb = q8_scale(static_cast<uint32_t>(e - e1 + 127));
#pragma unroll
          for (int c = 0; c < kRowCols; ++c) {
            float2 p = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 8; ++k) p = ffma2(x[k], w[c][k], p);
            acc[t * kRowCols + c] += (p.x + p.y) * fa * fb;
          }
        }
      }
    }
  }
  // Sum over the lanes: after the step with offset o, lanes with that bit set
  // hold the upper half of the values; lane i ends with value i.
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float keep = up ? acc[i + o] : acc[i], give = up ? acc[i] : acc[i + o];
      acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  part[warp][lane] = acc[0];
  __syncthreads();
  if (ks == 0) {
    float q = part[warp][lane];
#pragma unroll
    for (int k = 1; k < KS; ++k) q += part[warp + k][lane];
    const int t = lane / kRowCols, c = lane % kRowCols;
    if (t < nt && j0 + c < m) Q[(t0 + t) * m + j0 + c] = q;
  }
}

// ------------------------------------------------------------ tensor cores --
constexpr int kBM = 128, kBK = 128;  // rows of a tile; features of a block
constexpr int kATile = kBM * kBK;    // bytes
constexpr int kEpi = 8;              // epilogue warps: two per lane quarter of tensor memory
constexpr int kThreads = (2 + kEpi) * 32;
constexpr int kLd = 36, kStageFloats = 32 * kLd;  // a warp's 32 x 32 staging block, rows of 36 floats
constexpr int kSmemMax = 227 * 1024;

template <int BN> struct Tile {
  static constexpr int kStageBytes = kATile + BN * kBK;
  static constexpr int kFixed = 1024 + 256 + kEpi * kStageFloats * 4;  // alignment slack, barriers, staging
  static constexpr int kFit = (kSmemMax - kFixed) / kStageBytes;
  static constexpr int kStages = kFit < 8 ? kFit : 8;
  static constexpr int kSmem = kFixed + kStages * kStageBytes;
  static constexpr int kAccs = 512 / BN < 4 ? 512 / BN : 4;  // accumulators in tensor memory
  // Instruction descriptor of kind::f8f6f4: fp32 accumulator (bits 4-5 = 1), A
  // and B e4m3 (bits 7-9 and 10-12 = 0), both K-major, N / 8 (17-22), M / 16 (24-28).
  static constexpr uint32_t kIdesc =
      (1u << 4) | (static_cast<uint32_t>(BN >> 3) << 17) | (static_cast<uint32_t>(kBM >> 4) << 24);
};

__device__ __forceinline__ void umma_e4m3(uint32_t tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Byte k (0 to 15) of a vector.
__device__ __forceinline__ uint32_t byte_of(const uint4& v, int k) {
  const uint32_t w = k < 8 ? (k < 4 ? v.x : v.y) : (k < 12 ? v.z : v.w);
  return (w >> ((k & 3) * 8)) & 0xffu;
}

// Persistent, one CTA an SM. Roles as in the bf16 projection: warp 0 lane 0
// streams operand stages, warp 1 holds the tensor memory and its lane 0 issues
// the MMAs, warps 2-9 drain: warp w reads lane quarter w % 4 (one row of the
// tile a lane), the first four warps the lower half of the columns, the others the upper half.
template <int BN>
__global__ void __launch_bounds__(kThreads, 1)
    q8_proj_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const unsigned char* rows, int64_t T, int d, int rec, const unsigned char* W8, int m, float* Q,
                      int vec) {
  using G_ = Tile<BN>;
  constexpr int kS = G_::kStages, kAccs = G_::kAccs, kCols = BN / 2;
  constexpr uint32_t kTmemCols = kAccs * BN;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + kS * G_::kStageBytes);
  uint64_t* empty_bar = full_bar + kS;
  uint64_t* tfull = empty_bar + kS;        // [kAccs] a block's sums are ready
  uint64_t* tempty = tfull + kAccs;        // [kAccs] they have been read
  uint64_t* done_bar = tempty + kAccs;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done_bar + 1);
  float* epi_stage = reinterpret_cast<float*>(smem + kS * G_::kStageBytes + 256);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = q8_groups(d);
  const int ntn = (m + BN - 1) / BN;
  const int64_t ntiles = ((T + kBM - 1) / kBM) * ntn;
  const int64_t mine = blockIdx.x < ntiles ? (ntiles - 1 - blockIdx.x) / gridDim.x + 1 : 0;

  pdl_trigger();
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < kS; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 1);
      mbar_init(smem_u32(&empty_bar[s]), 1);
    }
    for (int k = 0; k < kAccs; ++k) {
      mbar_init(smem_u32(&tfull[k]), 1);
      mbar_init(smem_u32(&tempty[k]), kEpi);
    }
    mbar_init(smem_u32(done_bar), 1);
    mbar_fence_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *tmem_holder;
  pdl_wait();

  bool ok = true;
  if (warp == 0) {
    if (lane == 0) {
      int s = 0;
      uint32_t phase = 0;
      int64_t issued = 0;
      for (int64_t i = 0; i < mine && ok; ++i) {
        const int64_t tile = blockIdx.x + i * gridDim.x;
        const int m0 = static_cast<int>(tile / ntn) * kBM, n0 = static_cast<int>(tile % ntn) * BN;
        for (int kt = 0; kt < G; ++kt) {
          if (!mbar_wait(smem_u32(&empty_bar[s]), phase ^ 1u)) {
            ok = false;
            break;
          }
          const uint32_t fb = smem_u32(&full_bar[s]);
          mbar_arrive_expect_tx(fb, G_::kStageBytes);
          const uint32_t st = smem_u32(smem + s * G_::kStageBytes);
          tma_load_2d(st, &tmA, kt * kBK, m0, fb);
          tma_load_2d(st + kATile, &tmB, kt * kBK, n0, fb);
          ++issued;
          if (++s == kS) {
            s = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        atomicOr(&g_q8_proj_timeout, 1u);
        for (int64_t it = issued > kS ? issued - kS : 0; it < issued; ++it)
          (void)mbar_wait(smem_u32(&full_bar[it % kS]), static_cast<uint32_t>((it / kS) & 1));
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      int s = 0, acc = 0;
      uint32_t phase = 0, aphase = 0;
      for (int64_t i = 0; i < mine && ok; ++i) {
        for (int kt = 0; kt < G; ++kt) {
          if (!mbar_wait(smem_u32(&tempty[acc]), aphase ^ 1u) || !mbar_wait(smem_u32(&full_bar[s]), phase)) {
            ok = false;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t st = smem_u32(smem + s * G_::kStageBytes);
          const uint64_t da = sw128_desc(st), db = sw128_desc(st + kATile);
          const uint32_t tacc = tmem + static_cast<uint32_t>(acc * BN);
#pragma unroll
          for (int k = 0; k < kBK / 32; ++k)
            umma_e4m3(tacc, da + static_cast<uint64_t>(k * 2), db + static_cast<uint64_t>(k * 2), G_::kIdesc, k != 0);
          umma_commit(smem_u32(&empty_bar[s]));
          umma_commit(smem_u32(&tfull[acc]));
          if (++s == kS) {
            s = 0;
            phase ^= 1u;
          }
          if (++acc == kAccs) {
            acc = 0;
            aphase ^= 1u;
          }
        }
      }
      if (!ok) atomicOr(&g_q8_proj_timeout, 1u);
      // Signals once every MMA issued above is done (also after a timeout).
      umma_commit(smem_u32(done_bar));
    }
    __syncwarp();
  } else {
    const int q4 = warp & 3, half = (warp - 2) >> 2;
    float* stg = epi_stage + (warp - 2) * kStageFloats;
    const unsigned char* ex = W8 + static_cast<int64_t>(m) * (128 * G);
    const int exrow = q8_block_row(G);
    int acc = 0;
    uint32_t aphase = 0;
    for (int64_t i = 0; i < mine && ok; ++i) {
      const int64_t tile = blockIdx.x + i * gridDim.x;
      const int64_t rbase = (tile / ntn) * kBM + q4 * 32;
      const int c0 = static_cast<int>(tile % ntn) * BN + half * kCols;  // the warp's first output feature
      const int64_t row = rbase + lane < T ? rbase + lane : T - 1;
      const uint4* ea16 = reinterpret_cast<const uint4*>(rows + row * rec + 128 * G);
      const uint4* eb16 = reinterpret_cast<const uint4*>(ex + static_cast<int64_t>((c0 < m ? c0 : m - 1) >> 7) * exrow);
      float2 sum[kCols / 2];
#pragma unroll
      for (int k = 0; k < kCols / 2; ++k) sum[k] = make_float2(0.f, 0.f);
      uint4 ea = make_uint4(0, 0, 0, 0), eb = ea;
      for (int kt = 0; kt < G; ++kt) {
        if ((kt & 15) == 0) {
          ea = __ldg(ea16 + (kt >> 4));
          eb = __ldg(eb16 + (kt >> 4));
        }
        const int e = static_cast<int>(byte_of(ea, kt & 15)) + static_cast<int>(byte_of(eb, kt & 15)) - 254;
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&tfull[acc]), aphase))) {
          ok = false;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t taddr =
            tmem + (static_cast<uint32_t>(q4 * 32) << 16) + static_cast<uint32_t>(acc * BN + half * kCols);
        // 2^e in two factors when it is no normal fp32 number itself.
        const bool far = __any_sync(0xffffffffu, e < -126 || e > 127);
        const int e1 = far ? e >> 1 : e;
        const float f1 = q8_scale(static_cast<uint32_t>(e1 + 127)), f2 = q8_scale(static_cast<uint32_t>(e - e1 + 127));
        const float2 s2 = make_float2(f1, f1), t2 = make_float2(f2, f2);
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c) {
          float v[32];
          tmem_ld32(taddr + static_cast<uint32_t>(c * 32), v);
          if (c == kCols / 32 - 1) {  // the accumulator has been read
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&tempty[acc]));
          }
          if (far) {
#pragma unroll
            for (int k = 0; k < 16; ++k)
              sum[c * 16 + k] = ffma2(fmul2(make_float2(v[2 * k], v[2 * k + 1]), s2), t2, sum[c * 16 + k]);
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) sum[c * 16 + k] = ffma2(make_float2(v[2 * k], v[2 * k + 1]), s2, sum[c * 16 + k]);
          }
        }
        if (++acc == kAccs) {
          acc = 0;
          aphase ^= 1u;
        }
      }
      if (!ok) break;
      // Each 32 x 32 block is turned around in shared memory, so one store
      // instruction writes four whole 128-byte row segments.
#pragma unroll
      for (int c = 0; c < kCols / 32; ++c) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          *reinterpret_cast<float4*>(stg + lane * kLd + 4 * e) =
              make_float4(sum[c * 16 + 2 * e].x, sum[c * 16 + 2 * e].y, sum[c * 16 + 2 * e + 1].x, sum[c * 16 + 2 * e + 1].y);
        __syncwarp();
        const int col = c0 + c * 32 + 4 * (lane & 7);
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          const int r = h * 4 + (lane >> 3);
          const float4 x = *reinterpret_cast<const float4*>(stg + r * kLd + 4 * (lane & 7));
          if (rbase + r < T) {
            float* q = Q + (rbase + r) * m + col;
            if (vec) {
              if (col < m) *reinterpret_cast<float4*>(q) = x;
            } else {
              if (col < m) q[0] = x.x;
              if (col + 1 < m) q[1] = x.y;
              if (col + 2 < m) q[2] = x.z;
              if (col + 3 < m) q[3] = x.w;
            }
          }
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) atomicOr(&g_q8_proj_timeout, 1u);
  }
  // Teardown: every issued MMA has finished before the tensor memory goes.
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 1) {
    if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(done_bar), 0)) && lane == 0) atomicOr(&g_q8_proj_timeout, 1u);
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// `rows` rows of `width` codes, `stride` bytes apart, as a 2-d tensor: box
// {128, box_rows}, 128-byte swizzle; rows behind the last read as zero.
bool encode_codes(const void* base, int64_t rows, int width, int64_t stride, int box_rows, CUtensorMap* map) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride)};
  const cuuint32_t box[2] = {kBK, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t es[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN>
cudaError_t launch_tc(const void* rows, int64_t T, int d, const void* W8, int m, float* Q, cudaStream_t s) {
  alignas(64) CUtensorMap ma, mb;
  const int G = q8_groups(d), rec = static_cast<int>(q8_row_bytes(d));
  if (!encode_codes(rows, T, 128 * G, rec, kBM, &ma) || !encode_codes(W8, m, 128 * G, 128 * G, BN, &mb))
    return cudaErrorInvalidValue;
  cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(&q8_proj_tc_kernel<BN>), Tile<BN>::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ((T + kBM - 1) / kBM) * ((m + BN - 1) / BN);
  int64_t grid = sm_count();
  if (grid > tiles) grid = tiles;
  return launch_pdl(q8_proj_tc_kernel<BN>, static_cast<unsigned>(grid), kThreads, Tile<BN>::kSmem, s, ma, mb,
                    static_cast<const unsigned char*>(rows), T, d, rec, static_cast<const unsigned char*>(W8), m, Q,
                    m % 4 == 0 && aligned16(Q) ? 1 : 0);
}

template <int KS>
cudaError_t launch_rows(const void* rows, int64_t T, int d, const void* W8, int m, float* Q, cudaStream_t s) {
  const int64_t tgroups = (T + kRowTokens - 1) / kRowTokens;
  const int64_t cols = (4 / KS) * kRowCols, blocks = tgroups * ((m + cols - 1) / cols);
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_pdl(q8_proj_rows_kernel<KS>, static_cast<unsigned>(blocks), kRowThreads, 0, s,
                    static_cast<const unsigned char*>(rows), T, d, static_cast<int>(q8_row_bytes(d)),
                    static_cast<const unsigned char*>(W8), m, Q, tgroups);
}

constexpr int kFewTokens = 16;

}  // namespace

cudaError_t launch_q8_proj(const void* rows, int64_t T, int d, const void* W8, int m, float* Q, cudaStream_t s) {
  if (T > kFewTokens && T < (int64_t{1} << 31) - kBM && tensor_map_encode_fn()) return launch_tc<128>(rows, T, d, W8, m, Q, s);
  const int G = q8_groups(d);
  if (G <= 4) return launch_rows<1>(rows, T, d, W8, m, Q, s);
  if (G <= 8) return launch_rows<2>(rows, T, d, W8, m, Q, s);
  return launch_rows<4>(rows, T, d, W8, m, Q, s);
}

cudaError_t take_timeout_q8_proj(unsigned int* flag) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(flag, g_q8_proj_timeout, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_q8_proj_timeout, &zero, sizeof(unsigned int));
}

}  // namespace attnres
