// Projection of 8-bit rows by an 8-bit weight matrix (attnres.h): Q = V W^T with
// V [T, d] in e4m3 and one power-of-two scale for each row and group of 128
// features, W [m, d] in e4m3 and one for each 128 x 128 block, Q fp32.
//
// q8_proj_tc_kernel: the tensor cores, with the scales applied by them
// (tcgen05.mma kind::mxf8f6f4 with a power-of-two scale for each row and 32 features of
// either operand, K = 32): the rows' and blocks' exponents are such scales as they
// are. Sums stay in fp32 in tensor memory over all of d. Operands arrive by TMA
// copies of 128-byte rows (128 codes, one block) in the 128-byte swizzle.
// 32749 x 2048 x 2048: 105 to 107 us alone (2.6 PFLOP/s, 0.67 of twice the measured bf16
// rate), 121 to 123 in a row of calls (2.3). The MMAs alone, with no copies, waits, scales or
// stores, take 66, with their commits 74. Which of the rest bounds it has not been told apart:
// with one block a stage (116 us), bringing back the operands' copies and the waits for them was the
// largest step, to 102, and the scales took it to 110; the copies are 1.26 GB through
// the L2, 14 TB/s together with the results. Two blocks a stage, with half the waits
// and commits, took it to 107. (Summing each block unscaled and adding it, scaled, in registers
// was measured first: 205 us, bound by the warps that read tensor memory.)
//
// q8_proj_rows_kernel: few tokens. Bound by the weights' bytes and by latency,
// so the work is spread over the SMs by output features and by d: a warp takes
// 4 output features, 8 tokens and up to 512 features of d at a time, with fp32
// multiply-adds, and the KS warps that share an output add up through shared memory.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>
#include <utility>
#include <vector>

#include "q8.cuh"
#include "tcgen05.cuh"

namespace attnres {
namespace {

// ------------------------------------------------------------- few tokens --
constexpr int kRowCols = 4, kRowTokens = 8, kRowThreads = 128;

template <int KS>
__global__ void __launch_bounds__(kRowThreads) q8_proj_rows_kernel(const unsigned char* rows, int64_t cap, int64_t T, int d,
                                                                    const unsigned char* W8, int m, float* Q, int64_t tgroups) {
  constexpr int kColGroups = 4 / KS;
  __shared__ float part[4][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ks = warp % KS;
  const int G = q8_groups(d), chunks = 8 * G;
  const int64_t cg = blockIdx.x / tgroups;
  const int64_t t0 = (blockIdx.x - cg * tgroups) * kRowTokens;
  const int64_t j0 = (cg * kColGroups + warp / KS) * kRowCols;
  const unsigned char* ex = W8 + static_cast<int64_t>(m) * (128 * G);
  const unsigned char* tails = rows + cap * (128 * G);
  const int exrow = q8_block_row(G), tail_bytes = q8_tail_bytes(G);
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
        wc[c] = reinterpret_cast<const uint4*>(W8 + j * (128 * G))[ch];
      }
#pragma unroll
      for (int t = 0; t < kRowTokens; ++t)
        xc[t] = t < nt ? reinterpret_cast<const uint4*>(rows + (t0 + t) * (128 * G))[ch] : make_uint4(0, 0, 0, 0);
      const uint32_t eb = ex[(j0 >> 7) * exrow + (ch >> 3)];  // 4 columns lie in one block
      float2 w[kRowCols][8];
#pragma unroll
      for (int c = 0; c < kRowCols; ++c) decode16(wc[c], w[c]);
#pragma unroll
      for (int t = 0; t < kRowTokens; ++t) {
        if (t < nt) {
          const uint32_t ea = tails[(t0 + t) * tail_bytes + (ch >> 3)];
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
// One kernel for single CTAs (CG = 1: tiles of 128 x BN outputs) and for clusters of
// two CTAs on two SMs that share 256 x BN tiles through cta_group::2 (CG = 2;
// each CTA holds 128 of the tile's rows and BN / 2 of its weight rows, so an SM takes in
// fewer operand bytes per product).
//
// Tensor memory: two fp32 accumulators of BN columns that take turns by tiles,
// then three slots of 12 columns of scales: a word for each of 4 x 32 rows of A
// and of up to 8 x 32 rows of B (lane = row % 32, column = row / 32, the same
// in each lane quarter). An MMA's descriptor says which byte of the words it
// scales by (the format has one for each 32 features; here all MMAs of a block of 128
// use the same), so a word holds the exponents of four blocks as they
// lie in the rows' tails, and is written once for 16 MMAs. (One for each block,
// spread over the bytes, kept the writing warps busy for longer than the MMAs.)
//
// Warps of a CTA: 0-3 write the scales, each its lane quarter; 4, lane 0,
// streams the operands by TMA; 5 holds the tensor memory and, in the even CTA, its
// lane 0 issues the MMAs; 6-13 drain the accumulators, two to a lane quarter.
// Barriers (every wait bounded; for CG = 2 as in the bf16 projection's pairs):
//  * full[s], even CTA: the bytes of both CTAs' operand copies;
//  * empty[s], each CTA: the MMAs that read stage s have finished;
//  * scaled[j], even CTA: the warps that wrote slot j; used[j], each CTA: the
//    MMAs that read it have finished;
//  * tfull[a], each CTA: a tile's sums are ready; tempty[a], even CTA: read;
//  * done, each CTA: every MMA has finished.
__device__ unsigned int g_q8_proj_timeout = 0;

constexpr int kBM = 128, kBK = 128;  // rows of a CTA's tile; features of a block
constexpr int kATile = kBM * kBK;    // bytes
constexpr uint32_t kNextScale = (1u << 4) | (1u << 29);  // the next scale byte of A and of B, in the instruction descriptor
constexpr int kScaleWarps = 4, kProducer = 4, kIssuer = 5, kEpi = 8;
constexpr int kThreads = (kScaleWarps + 2 + kEpi) * 32;
constexpr int kScaleCols = 12, kSlots = 3;
constexpr int kLd = 36, kStageFloats = 32 * kLd;  // a warp's 32 x 32 staging block, rows of 36 floats
constexpr int kSmemMax = 227 * 1024;

template <int BN, int CG> struct Tile {
  static constexpr int kBRows = BN / CG;                               // weight rows a CTA holds
  static constexpr int kBlockBytes = kATile + kBRows * kBK;            // a block's operands
  static constexpr int kFixed = 1024 + 256 + kEpi * kStageFloats * 4;  // alignment slack, barriers, staging
  static constexpr int kFit = (kSmemMax - kFixed) / kBlockBytes;       // blocks
  static constexpr int kBlocks = kFit >= 6 ? 2 : 1;                    // of a stage
  static constexpr int kStageBytes = kBlocks * kBlockBytes;
  static constexpr int kStages = kFit / kBlocks;
  static constexpr int kSmem = kFixed + kStages * kStageBytes;
  static constexpr int kUsed = 2 * BN + kSlots * kScaleCols;
  static constexpr uint32_t kTmemCols = kUsed <= 128 ? 128u : (kUsed <= 256 ? 256u : 512u);
  // Instruction descriptor of kind::mxf8f6f4: A and B e4m3 (bits 7-9 and 10-12 = 0), both K-major, N / 8 (17-22),
  // scales of powers of two (23 = 1), M / 16 (24-28); which scale byte of B (4-5) and A (29-30) is added to it.
  static constexpr uint32_t kIdesc =
      (static_cast<uint32_t>(BN >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(CG * kBM >> 4) << 24);
  static_assert(kStages >= 3 && (2 * kStages + 2 * kSlots + 5) * 8 + 4 <= 256 && kUsed <= 512, "stages and barriers fit");
  static_assert(kBRows % 8 == 0 && BN <= 256, "weight rows come in 8-row swizzle atoms");
};

// The four MMAs of one block (K = 32 each; their operands lie 32 bytes apart).
// The descriptors' low words are the operands' addresses, `hi` is the same for both.
// `accumulate` 0: the first one starts the sums anew.
template <int CG>
__device__ __forceinline__ void umma_block(uint32_t tmem, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, uint32_t sa,
                                           uint32_t accumulate) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n .reg .pred p, t;\n .reg .b32 l;\n .reg .b64 a0, a1, a2, a3, b0, b1, b2, b3;\n"
        " setp.ne.b32 p, %7, 0;\n setp.eq.b32 t, 0, 0;\n mov.b64 a0, {%1, %3};\n mov.b64 b0, {%2, %3};\n"
        " add.u32 l, %1, 2;\n mov.b64 a1, {l, %3};\n add.u32 l, %2, 2;\n mov.b64 b1, {l, %3};\n"
        " add.u32 l, %1, 4;\n mov.b64 a2, {l, %3};\n add.u32 l, %2, 4;\n mov.b64 b2, {l, %3};\n"
        " add.u32 l, %1, 6;\n mov.b64 a3, {l, %3};\n add.u32 l, %2, 6;\n mov.b64 b3, {l, %3};\n"
        " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a0, b0, %4, [%5], [%6], p;\n"
        " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a1, b1, %4, [%5], [%6], t;\n"
        " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a2, b2, %4, [%5], [%6], t;\n"
        " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a3, b3, %4, [%5], [%6], t;\n"
        "}"
        ::"r"(tmem), "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(sa), "r"(sa + 4), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p, t;\n .reg .b32 l;\n .reg .b64 a0, a1, a2, a3, b0, b1, b2, b3;\n"
        " setp.ne.b32 p, %7, 0;\n setp.eq.b32 t, 0, 0;\n mov.b64 a0, {%1, %3};\n mov.b64 b0, {%2, %3};\n"
        " add.u32 l, %1, 2;\n mov.b64 a1, {l, %3};\n add.u32 l, %2, 2;\n mov.b64 b1, {l, %3};\n"
        " add.u32 l, %1, 4;\n mov.b64 a2, {l, %3};\n add.u32 l, %2, 4;\n mov.b64 b2, {l, %3};\n"
        " add.u32 l, %1, 6;\n mov.b64 a3, {l, %3};\n add.u32 l, %2, 6;\n mov.b64 b3, {l, %3};\n"
        " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a0, b0, %4, [%5], [%6], p;\n"
        " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a1, b1, %4, [%5], [%6], t;\n"
        " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a2, b2, %4, [%5], [%6], t;\n"
        " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a3, b3, %4, [%5], [%6], t;\n"
        "}"
        ::"r"(tmem), "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(sa), "r"(sa + 4), "r"(accumulate)
        : "memory");
}

// An arrival on the other CTA's barrier that releases no memory: what it
// announces is in tensor memory, ordered by tcgen05.fence. (A release would
// first wait for every earlier store of the thread: 1 us.)
__device__ __forceinline__ void mbar_arrive_remote_relaxed(uint32_t caddr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(caddr) : "memory");
}

template <int CG>
__device__ __forceinline__ void commit_mmas(uint32_t bar) {
  if constexpr (CG == 1)
    umma_commit(bar);
  else
    umma_commit_pair(bar);
}

// Waits for a barrier that, with CG = 2, the other CTA may signal.
template <int CG>
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity) {
  return CG == 1 ? mbar_wait(bar, parity) : mbar_wait_cluster(bar, parity);
}

template <int BN, int CG>
__global__ void __launch_bounds__(kThreads, 1)
    q8_proj_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const unsigned char* tails, int64_t T, int d, const unsigned char* W8, int m, float* Q, int vec,
                      int64_t withhold) {
  using G_ = Tile<BN, CG>;
  constexpr int kS = G_::kStages, kStageBytes = G_::kStageBytes;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + kS * kStageBytes);
  uint64_t* empty_bar = full_bar + kS;
  uint64_t* scaled_bar = empty_bar + kS;      // [kSlots]
  uint64_t* used_bar = scaled_bar + kSlots;   // [kSlots]
  uint64_t* tfull = used_bar + kSlots;        // [2]
  uint64_t* tempty = tfull + 2;        // [2]
  uint64_t* done_bar = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done_bar + 1);
  float* epi_stage = reinterpret_cast<float*>(smem + kS * kStageBytes + 256);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 1 ? 0u : cluster_rank();
  const int64_t unit = blockIdx.x / CG, units = gridDim.x / CG;  // CTAs or pairs
  const int G = q8_groups(d);
  const int ntn = (m + BN - 1) / BN;
  const int64_t ntiles = ((T + CG * kBM - 1) / (CG * kBM)) * ntn;
  const int64_t mine = unit < ntiles ? (ntiles - 1 - unit) / units + 1 : 0;

  pdl_trigger();
  if (warp == kProducer && lane == 0) {
    for (int s = 0; s < kS; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 1);
      mbar_init(smem_u32(&empty_bar[s]), 1);
    }
    for (int k = 0; k < kSlots; ++k) {
      mbar_init(smem_u32(&scaled_bar[k]), CG * kScaleWarps);
      mbar_init(smem_u32(&used_bar[k]), 1);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(smem_u32(&tfull[k]), 1);
      mbar_init(smem_u32(&tempty[k]), CG * kEpi);
    }
    mbar_init(smem_u32(done_bar), 1);
    mbar_fence_init();
  }
  if (warp == kIssuer) {
    if constexpr (CG == 1) {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                   "r"(G_::kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                   "r"(G_::kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  if constexpr (CG == 1)
    __syncthreads();
  else
    cluster_sync();  // both CTAs' barriers are initialised before any remote use
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *tmem_holder;
  pdl_wait();

  bool ok = true;
  if (warp < kScaleWarps) {
    // Scales: lane l of each quarter holds rows l, 32 + l, .. of A and of B.
    const unsigned char* ex = W8 + static_cast<int64_t>(m) * (128 * G);
    const int exrow = q8_block_row(G), tail_bytes = q8_tail_bytes(G);
    const uint32_t quarter = tmem + (static_cast<uint32_t>(warp * 32) << 16) + 2 * BN;
    const int blocks = (m + 127) >> 7;
    // A word for each of the lane's four rows of A, and of the (at most three)
    // rows of weight blocks under the BN columns, which start at a multiple of 32;
    // the next four blocks' are on their way while these are written.
    const uint32_t* at7[7];
    auto point = [&](int64_t i) {
      const int64_t tile = unit + i * units;
      const int64_t m0 = (tile / ntn) * (CG * kBM) + static_cast<int64_t>(rank) * kBM;
      const int b0 = static_cast<int>(tile % ntn) * BN >> 7;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int64_t row = m0 + c * 32 + lane < T ? m0 + c * 32 + lane : T - 1;
        at7[c] = reinterpret_cast<const uint32_t*>(tails + row * tail_bytes);
      }
#pragma unroll
      for (int c = 0; c < 3; ++c)
        at7[4 + c] = reinterpret_cast<const uint32_t*>(ex + static_cast<int64_t>(b0 + c < blocks ? b0 + c : blocks - 1) * exrow);
    };
    uint32_t next[7];
    auto fetch = [&] {
#pragma unroll
      for (int c = 0; c < 7; ++c) next[c] = *at7[c]++;
    };
    if (mine > 0) {
      point(0);
      fetch();
    }
    int slot = 0;
    uint32_t phase = 0;
    const int quads = (G + 3) / 4;
    for (int64_t i = 0; i < mine && ok; ++i) {
      const int off = static_cast<int>((unit + i * units) % ntn) * BN & 127;
      for (int k4 = 0; k4 < quads; ++k4) {
        uint32_t now[7], bw[8];
#pragma unroll
        for (int c = 0; c < 7; ++c) now[c] = next[c];
        if (k4 + 1 < quads) {
          fetch();
        } else if (i + 1 < mine) {
          point(i + 1);
          fetch();
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const int b = (off + c * 32) >> 7;
          bw[c] = b == 0 ? now[4] : (b == 1 ? now[5] : now[6]);
        }
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&used_bar[slot]), phase ^ 1u))) {
          ok = false;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t at = quarter + static_cast<uint32_t>(slot * kScaleCols);
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(now[0]), "r"(now[1]),
                     "r"(now[2]), "r"(now[3])
                     : "memory");
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(at + 4),
                     "r"(bw[0]), "r"(bw[1]), "r"(bw[2]), "r"(bw[3]), "r"(bw[4]), "r"(bw[5]), "r"(bw[6]), "r"(bw[7])
                     : "memory");
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 1)
            mbar_arrive(smem_u32(&scaled_bar[slot]));
          else
            mbar_arrive_remote_relaxed(cluster_addr(smem_u32(&scaled_bar[slot]), 0));
        }
        if (++slot == kSlots) {
          slot = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) atomicOr(&g_q8_proj_timeout, 1u);
  } else if (warp == kProducer) {
    if (lane == 0) {
      int s = 0;
      uint32_t phase = 0;
      int64_t issued = 0;
      for (int64_t i = 0; i < mine && ok; ++i) {
        const int64_t tile = unit + i * units;
        const int m0 = static_cast<int>(tile / ntn) * (CG * kBM) + static_cast<int>(rank) * kBM;
        const int n0 = static_cast<int>(tile % ntn) * BN + static_cast<int>(rank) * G_::kBRows;
        for (int kt = 0; kt < G; kt += G_::kBlocks) {
          if (!mbar_wait(smem_u32(&empty_bar[s]), phase ^ 1u)) {
            ok = false;
            break;
          }
          const uint32_t fb = smem_u32(&full_bar[s]);
          const uint32_t st = smem_u32(smem + s * kStageBytes);
          // The test hook leaves a stage unfilled, in both CTAs of a pair.
          const int nb = issued == withhold ? 0 : (G - kt < G_::kBlocks ? G - kt : G_::kBlocks);
          if (rank == 0 && nb > 0) mbar_arrive_expect_tx(fb, static_cast<uint32_t>(nb * CG * G_::kBlockBytes));
          for (int b = 0; b < nb; ++b) {
            const uint32_t at = st + static_cast<uint32_t>(b * G_::kBlockBytes);
            if constexpr (CG == 1) {
              tma_load_2d(at, &tmA, (kt + b) * kBK, m0, fb);
              tma_load_2d(at + kATile, &tmB, (kt + b) * kBK, n0, fb);
            } else {
              const uint32_t fbc = cluster_addr(fb, 0);
              tma_load_2d_pair(at, &tmA, (kt + b) * kBK, m0, fbc);
              tma_load_2d_pair(at + kATile, &tmB, (kt + b) * kBK, n0, fbc);
            }
          }
          ++issued;
          if (++s == kS) {
            s = 0;
            phase ^= 1u;
          }
        }
      }
      // The even CTA's full barriers count both CTAs' copies; once the phases
      // it armed complete, no copy of either CTA is in flight. Waited for on every path: this
      // warp may have issued all its stages when another one's wait runs out.
      if (rank == 0)
        for (int64_t it = issued > kS ? issued - kS : 0; it < issued; ++it)
          if (it != withhold) ok &= wait_bar<CG>(smem_u32(&full_bar[it % kS]), static_cast<uint32_t>((it / kS) & 1));
      if (!ok) atomicOr(&g_q8_proj_timeout, 1u);
    }
    __syncwarp();
  } else if (warp == kIssuer) {
    // The warp walks together and one lane issues, so that what the MMAs take
    // (addresses, descriptors) is in uniform registers when they do.
    if (rank == 0) {
      const bool leader = lane == 0;
      int s = 0, slot = 0;
      uint32_t phase = 0, sphase = 0;
      // Stages stay below 2^18 bytes, so adding to the low word carries into nothing.
      const uint64_t desc = sw128_desc(smem_u32(smem));
      const uint32_t desc_lo = static_cast<uint32_t>(desc), desc_hi = static_cast<uint32_t>(desc >> 32);
      for (int64_t i = 0; i < mine && ok; ++i) {
        const int acc = static_cast<int>(i & 1);
        ok = __all_sync(0xffffffffu, wait_bar<CG>(smem_u32(&tempty[acc]), static_cast<uint32_t>(((i >> 1) & 1) ^ 1)));
        if (!ok) break;
        const uint32_t tacc = tmem + static_cast<uint32_t>(acc * BN);
        for (int kt = 0; kt < G; kt += G_::kBlocks) {
          bool got = (kt & 3) != 0 || wait_bar<CG>(smem_u32(&scaled_bar[slot]), sphase);
          got = got && wait_bar<CG>(smem_u32(&full_bar[s]), phase);
          ok = __all_sync(0xffffffffu, got);
          if (!ok) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t st = desc_lo + static_cast<uint32_t>(s * (kStageBytes / 16));
          const uint32_t sa = tmem + static_cast<uint32_t>(2 * BN + slot * kScaleCols);
          const uint32_t idesc = G_::kIdesc + static_cast<uint32_t>(kt & 3) * kNextScale;
          const bool slot_done = ((kt + G_::kBlocks) & 3) == 0 || kt + G_::kBlocks >= G;
          if (leader) {
            umma_block<CG>(tacc, st, st + kATile / 16, desc_hi, idesc, sa, kt != 0);
            if (G_::kBlocks == 2 && kt + 1 < G)
              umma_block<CG>(tacc, st + G_::kBlockBytes / 16, st + (G_::kBlockBytes + kATile) / 16, desc_hi, idesc + kNextScale,
                             sa, 1);
            commit_mmas<CG>(smem_u32(&empty_bar[s]));
            if (slot_done) commit_mmas<CG>(smem_u32(&used_bar[slot]));
          }
          __syncwarp();
          if (++s == kS) {
            s = 0;
            phase ^= 1u;
          }
          if (slot_done && ++slot == kSlots) {
            slot = 0;
            sphase ^= 1u;
          }
        }
        if (ok && leader) commit_mmas<CG>(smem_u32(&tfull[acc]));
        __syncwarp();
      }
      if (leader) {
        if (!ok) atomicOr(&g_q8_proj_timeout, 1u);
        commit_mmas<CG>(smem_u32(done_bar));  // also after a timeout
      }
    }
    __syncwarp();
  } else {
    // Epilogue: each 32 x 32 block is turned around in shared memory, so one
    // store instruction writes four whole 128-byte row segments.
    const int ew = warp - kScaleWarps - 2, q4 = warp & 3, half = ew >> 2;
    float* stg = epi_stage + ew * kStageFloats;
    for (int64_t i = 0; i < mine; ++i) {
      const int acc = static_cast<int>(i & 1);
      if (!__all_sync(0xffffffffu, wait_bar<CG>(smem_u32(&tfull[acc]), static_cast<uint32_t>((i >> 1) & 1)))) {
        ok = false;
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const int64_t tile = unit + i * units;
      const int64_t rbase = (tile / ntn) * (CG * kBM) + static_cast<int64_t>(rank) * kBM + q4 * 32;
      const int n0 = static_cast<int>(tile % ntn) * BN;
      const uint32_t taddr = tmem + (static_cast<uint32_t>(q4 * 32) << 16) + static_cast<uint32_t>(acc * BN);
#pragma unroll 1
      for (int c = half; c < BN / 32; c += 2) {
        if (n0 + c * 32 >= m) break;
        float v[32];
        tmem_ld32(taddr + static_cast<uint32_t>(c * 32), v);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          *reinterpret_cast<float4*>(stg + lane * kLd + 4 * e) =
              make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        __syncwarp();
        const int col = n0 + c * 32 + 4 * (lane & 7);
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
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 1)
          mbar_arrive(smem_u32(&tempty[acc]));
        else
          mbar_arrive_remote_relaxed(cluster_addr(smem_u32(&tempty[acc]), 0));
      }
    }
    if (!ok && lane == 0) atomicOr(&g_q8_proj_timeout, 1u);
  }
  // Teardown: every issued MMA has finished (done) before tensor memory goes
  // and, with CG = 2, before either CTA leaves the other.
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == kIssuer && !__all_sync(0xffffffffu, wait_bar<CG>(smem_u32(done_bar), 0)) && lane == 0)
    atomicOr(&g_q8_proj_timeout, 1u);
  if constexpr (CG == 2) cluster_sync();
  if (warp == kIssuer) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if constexpr (CG == 1)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(G_::kTmemCols) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(G_::kTmemCols) : "memory");
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

template <int BN, int CG>
void tc_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attr)[2], int64_t units, cudaStream_t s) {
  cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(CG * units));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Tile<BN, CG>::kSmem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 1 ? 1 : 2;
}

// How many CTAs (CG = 1) or pairs of them (CG = 2; 0 when clusters cannot be
// launched) the device holds at once; for pairs asked once per device.
template <int BN, int CG>
int tc_units() {
  if (CG == 1) return sm_count();
  static std::mutex mu;
  static std::vector<std::pair<int, int>> known;  // (device, pairs)
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lk(mu);
  for (const auto& k : known)
    if (k.first == dev) return k.second;
  int n = 0;
  const auto kernel = q8_proj_tc_kernel<BN, CG>;
  if (allow_dynamic_smem(reinterpret_cast<const void*>(kernel), Tile<BN, CG>::kSmem) == cudaSuccess) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    tc_config<BN, CG>(cfg, attr, sm_count() / CG, nullptr);
    std::swap(attr[0], attr[1]);
    cfg.numAttrs = 1;  // the occupancy query takes the cluster shape only
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) n = 0;
  }
  (void)cudaGetLastError();
  known.emplace_back(dev, n);
  return n;
}

template <int BN, int CG>
cudaError_t launch_tc(const void* rows, int64_t cap, int64_t T, int d, const void* W8, int m, float* Q, int64_t withhold,
                      cudaStream_t s) {
  using G_ = Tile<BN, CG>;
  alignas(64) CUtensorMap ma, mb;
  const int G = q8_groups(d);
  if (!encode_codes(rows, T, 128 * G, 128 * G, kBM, &ma) || !encode_codes(W8, m, 128 * G, 128 * G, G_::kBRows, &mb))
    return cudaErrorInvalidValue;
  const auto kernel = q8_proj_tc_kernel<BN, CG>;
  cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(kernel), G_::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ((T + CG * kBM - 1) / (CG * kBM)) * ((m + BN - 1) / BN);
  int64_t units = tc_units<BN, CG>();
  if (units > tiles) units = tiles;
  if (units < 1) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  tc_config<BN, CG>(cfg, attr, units, s);
  return cudaLaunchKernelEx(&cfg, kernel, ma, mb, static_cast<const unsigned char*>(rows) + cap * (128 * G), T, d,
                            static_cast<const unsigned char*>(W8), m, Q, m % 4 == 0 && aligned16(Q) ? 1 : 0, withhold);
}

template <int KS>
cudaError_t launch_rows(const void* rows, int64_t cap, int64_t T, int d, const void* W8, int m, float* Q, cudaStream_t s) {
  const int64_t tgroups = (T + kRowTokens - 1) / kRowTokens;
  const int64_t cols = (4 / KS) * kRowCols, blocks = tgroups * ((m + cols - 1) / cols);
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_pdl(q8_proj_rows_kernel<KS>, static_cast<unsigned>(blocks), kRowThreads, 0, s,
                    static_cast<const unsigned char*>(rows), cap, T, d, static_cast<const unsigned char*>(W8), m, Q, tgroups);
}

constexpr int kFewTokens = 16;

// Few tokens: which of the two kernels is sooner done, by their times in us as
// measured for 640 to 4096 features, 640 to 8192 outputs and 1 to 16 tokens (16 x 896 x
// 896: 3.2 by rows, 4.6; 8 x 2048 x 2048: 6.3 and 6.9; 16 x 2048 x 2048: 10.9 and 6.9;
// 4 x 640 x 5120: 5.7 and 4.9; 1 x 4096 x 4096: 9.4 and 13.1). The rows' grows
// with the products and the conversions of the weights, the tensor cores' with the
// blocks that follow each other.
bool rows_are_sooner(int64_t T, int G, int m) {
  return T <= kFewTokens && 2.0 + 1.1e-5 * static_cast<double>(T + 5) * G * m <= 2.65 + 0.265 * G;
}

}  // namespace

cudaError_t launch_q8_proj(const void* rows, int64_t cap, int64_t T, int d, const void* W8, int m, float* Q, int64_t withhold,
                           cudaStream_t s) {
  if (!rows_are_sooner(T, q8_groups(d), m) && T < (int64_t{1} << 31) - 2 * kBM && tensor_map_encode_fn()) {
    // Wide tiles shared by pairs when every pair gets one (8192 x 896: 12.0 us,
    // 13.1 with 128 columns a CTA; 32749 x 2048: 105, 167). A block of a tile takes a CTA
    // about the same time whatever its columns, so fewer are taken only as
    // long as that puts more SMs to work and no SM gets two tiles
    // (512 x 1024: 5.0 us with 64, 6.3 with 128). 224 is the widest that leaves tensor memory for
    // two accumulators and the scales; the last column tile takes as long however few columns
    // are left (1024 and 2048 outputs: 9 % more than they need, 512: 31 %, 256: 75 %).
    const int64_t rt = (T + kBM - 1) / kBM, rp = (T + 2 * kBM - 1) / (2 * kBM);
    const int pairs = tc_units<224, 2>();
    if (pairs > 0 && rp * ((m + 223) / 224) >= pairs) return launch_tc<224, 2>(rows, cap, T, d, W8, m, Q, withhold, s);
    if (rt * ((m + 63) / 64) <= sm_count()) return launch_tc<64, 1>(rows, cap, T, d, W8, m, Q, withhold, s);
    return launch_tc<128, 1>(rows, cap, T, d, W8, m, Q, withhold, s);
  }
  const int G = q8_groups(d);
  if (G <= 4) return launch_rows<1>(rows, cap, T, d, W8, m, Q, s);
  if (G <= 8) return launch_rows<2>(rows, cap, T, d, W8, m, Q, s);
  return launch_rows<4>(rows, cap, T, d, W8, m, Q, s);
}

cudaError_t take_timeout_q8_proj(unsigned int* flag) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(flag, g_q8_proj_timeout, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_q8_proj_timeout, &zero, sizeof(unsigned int));
}

}  // namespace attnres
