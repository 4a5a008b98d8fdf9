// matmul_mx.cuh -- products of microscaled rows on the block-scaled tensor
// cores: Y[m, n] = (sum over blocks of sa sb sum of a b) ra[m] rb[n] + bias[n],
// accumulated in binary32 in tensor memory and rounded once.
//
//   mxfp8  tcgen05.mma kind::mxf8f6f4, K = 32 per MMA, one scale per row
//   mxfp4  kind::mxf4,     K = 64, two scales per row
//   nvfp4  kind::mxf4nvf4, K = 64, four scales per row
//
// A stage of the pipeline is 128 bytes of codes per row (four MMAs) plus the
// words of four scales that cover them: the tiles of 128 rows x 4 scales lie
// in global memory as tensor memory wants them, so a stage's scales are one
// bulk copy per 128 rows and tcgen05.cp spreads each tile over four columns
// (column j holds rows 32 j .. 32 j + 31 of the tile, in all lane quarters).
// Each stage has its own columns: they are written again only once the
// stage's MMAs have completed, which its empty barrier already says.
// Codes past K are zeros (padded rows, zero-filled boxes), rows past the
// operand's end are zero-filled, and a row's scales touch only that row's
// results, so the scale tiles' rows past the end need no value.
#pragma once

#include <cooperative_groups.h>

#include "attention.cuh"
#include "device.cuh"
#include "microscale.cuh"

namespace fqa {

template <int FMT>
struct MxMma {
  static constexpr int kWords = FMT == kMxFp8 ? 1 : (FMT == kMxFp4 ? 2 : 4);   // scale words per row and stage
  // instruction descriptor: element types (E4M3 0, E2M1 1), scale type (UE4M3
  // 0, UE8M0 1), sizes; the scale ids are added per MMA
  static constexpr uint32_t idesc(uint32_t M, uint32_t N) {
    return (FMT == kMxFp8 ? 0u : (1u << 7) | (1u << 10)) | ((N >> 3) << 17) | (FMT == kNvFp4 ? 0u : 1u << 23) |
           ((M >> 7) << 27);
  }
  // word and scale id of MMA kk of a stage
  static constexpr uint32_t word(int kk) { return FMT == kMxFp8 ? 0u : (FMT == kMxFp4 ? kk / 2 : kk); }
  static constexpr uint32_t sf_id(int kk) { return FMT == kMxFp8 ? kk : (FMT == kMxFp4 ? 2 * (kk % 2) : 0u); }
};

template <int FMT, int CTAS>
__device__ __forceinline__ void mma_mx(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
#define FQA_MX_MMA(CG, KIND)                                                                                    \
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::" CG ".kind::" KIND       \
               " [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d_tmem),                                          \
               "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)                        \
               : "memory")
  if constexpr (CTAS == 1) {
    if constexpr (FMT == kMxFp8) FQA_MX_MMA("1", "mxf8f6f4.block_scale.block32");
    if constexpr (FMT == kMxFp4) FQA_MX_MMA("1", "mxf4.block_scale.block32");
    if constexpr (FMT == kNvFp4) FQA_MX_MMA("1", "mxf4nvf4.block_scale.block16");
  } else {
    if constexpr (FMT == kMxFp8) FQA_MX_MMA("2", "mxf8f6f4.block_scale.block32");
    if constexpr (FMT == kMxFp4) FQA_MX_MMA("2", "mxf4.block_scale.block32");
    if constexpr (FMT == kNvFp4) FQA_MX_MMA("2", "mxf4nvf4.block_scale.block16");
  }
#undef FQA_MX_MMA
}

// 32 rows x 16 bytes of shared memory -> four columns of tensor memory, the
// same in every lane quarter.
template <int CTAS>
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint64_t sdesc) {
  if constexpr (CTAS == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

// Shared-memory descriptor without swizzle: 8-row groups of 16-byte rows, 128
// bytes apart (a scale tile).
__device__ __forceinline__ uint64_t make_sdesc_plain(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr >> 4) & 0x3FFFu);
  d |= (uint64_t)(128u >> 4) << 16;
  d |= (uint64_t)(128u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  return d;
}

struct MxMatmulParams {
  const uint8_t* sa;      // scale tiles of A [M] and B [N]
  const uint8_t* sb;
  const float* ra;        // row scales (nvfp4) or null
  const float* rb;
  const float* bias;      // [N] or null
  void* out;              // [M, N]
  int M, N;
  int mmas;               // MMAs of a row: 32-byte steps over its codes
  int KT;                 // scale words of a row
  int out_type;           // 0 BF16, 1 binary32, 2 FP16
  uint32_t* status;
};

__device__ __forceinline__ void store_out(void* out, int type, size_t at, float v) {
  if (type == 0)
    static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
  else if (type == 1)
    static_cast<float*>(out)[at] = v;
  else
    static_cast<__half*>(out)[at] = __float2half_rn(v);
}

// ------------------------------------------------------- few rows of A
//
// One 128 x NT tile per cluster of 1, 2, 4 or 8 CTAs.  B's rows (the weights)
// take the MMA's 128-row side and A's rows (the tokens) its N side, so a
// handful of tokens costs an MMA of N = 16, not one of 128 padded rows, and
// the kernel is bound by the weights' bytes.  The CTAs of a cluster split K:
// at 4096 features there are 32 tiles of weights for 148 SMs, so the stages
// are dealt out to `ranks` CTAs and their binary32 partial tiles are added in
// rank order over distributed shared memory (the same sum every time).
//   warp 0  TMA producer    warp 1  TMEM owner and MMA issuer
//   warps 2-5  epilogue, one lane quarter each
constexpr int kMxSmallThreads = 192;

template <int FMT, int NT>
struct MxSmall {
  using Mma = MxMma<FMT>;
  static constexpr int kPBytes = 128 * 128, kQBytes = NT * 128, kSfBytes = 512 * Mma::kWords;
  static constexpr int kStageBytes = kPBytes + (kQBytes < 1024 ? 1024 : kQBytes) + 2 * kSfBytes;
  static constexpr int kStages = 4;
  static constexpr int kOffBar = kStages * kStageBytes;
  static constexpr int kSmemBytes = kOffBar + (2 * kStages + 1) * 8 + 16 + 1024;
  static constexpr int kSfCols = 8 * Mma::kWords;            // per stage: four for P and four for Q, per word
  static constexpr int kColSf = NT < 32 ? 32 : NT;
  static constexpr int kColsUsed = kColSf + kStages * kSfCols;
  static constexpr int kCols = kColsUsed <= 64 ? 64 : (kColsUsed <= 128 ? 128 : 256);
  static_assert(kColsUsed <= 256 && kStageBytes % 1024 == 0, "tile layout");
  static_assert(NT * 128 * 4 <= kStages * kStageBytes, "a partial tile fits the stages");
};

template <int FMT, int NT>
__global__ void __launch_bounds__(kMxSmallThreads)
    mx_matmul_small_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                           const MxMatmulParams p, int ranks) {
  using T = MxSmall<FMT, NT>;
  using Mma = MxMma<FMT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + T::kOffBar);
  uint64_t* empty = full + T::kStages;
  uint64_t* done = empty + T::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const int rank = blockIdx.x % ranks, tile = blockIdx.x / ranks;
  const int ptiles = (p.N + 127) / 128;
  const int p0 = (tile % ptiles) * 128, q0 = (tile / ptiles) * NT;
  const int stages = (p.mmas + 3) / 4;
  // this rank's stages: [s0, s1), an even share
  const int s0 = (int)((int64_t)stages * rank / ranks), s1 = (int)((int64_t)stages * (rank + 1) / ranks);

  if (threadIdx.x == 0) {
    for (int s = 0; s < T::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, T::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      int issued = 0;
      for (int s = s0; s < s1; ++s) {
        const int i = s - s0, slot = i % T::kStages;
        if (!mbar_wait(&empty[slot], ((i / T::kStages) & 1) ^ 1, abort_flag, p.status)) break;
        uint8_t* st = smem + slot * T::kStageBytes;
        const uint32_t words = min(Mma::kWords, p.KT - s * Mma::kWords);
        mbar_arrive_expect_tx(&full[slot], T::kPBytes + T::kQBytes + 2 * 512 * words);
        tma_load_2d(st, &tmP, &full[slot], s * 128, p0);
        tma_load_2d(st + T::kPBytes, &tmQ, &full[slot], s * 128, q0);
        uint8_t* sf = st + T::kStageBytes - 2 * T::kSfBytes;
        const size_t w0 = (size_t)s * Mma::kWords * 512;
        bulk_load_plain(sf, p.sb + (size_t)(p0 / 128) * p.KT * 512 + w0, 512 * words, &full[slot]);
        bulk_load_plain(sf + T::kSfBytes, p.sa + (size_t)(q0 / 128) * p.KT * 512 + w0, 512 * words, &full[slot]);
        issued = i + 1;
      }
      if (*abort_flag)      // no copy may be in flight when the CTA ends
        for (int i = issued > T::kStages ? issued - T::kStages : 0; i < issued; ++i)
          mbar_wait_drain(&full[i % T::kStages], (i / T::kStages) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t kI = Mma::idesc(128, NT);
      bool any = false;
      // the Q tile's place in its block of 128 rows: 32 rows per column (a tile of
      // 16 rows is only taken where it is the only one, at row 0)
      const uint32_t qcol = (uint32_t)(q0 % 128) / 32;
      for (int s = s0; s < s1; ++s) {
        const int i = s - s0, slot = i % T::kStages;
        if (!mbar_wait(&full[slot], (i / T::kStages) & 1, abort_flag, p.status)) break;
        tc_fence_after();
        const uint32_t st = smem_u32(smem + slot * T::kStageBytes);
        const uint32_t sf = st + T::kStageBytes - 2 * T::kSfBytes;
        const uint32_t tsp = tmem + T::kColSf + slot * T::kSfCols, tsq = tsp + 4 * Mma::kWords;
        const int words = min(Mma::kWords, p.KT - s * Mma::kWords);
        for (int w = 0; w < words; ++w) {
          tmem_cp_scales<1>(tsp + 4 * w, make_sdesc_plain(sf + 512 * w));
          tmem_cp_scales<1>(tsq + 4 * w, make_sdesc_plain(sf + T::kSfBytes + 512 * w));
        }
        const uint64_t dP = make_sdesc_sw128(st, 16, 1024), dQ = make_sdesc_sw128(st + T::kPBytes, 16, 1024);
        const int left = p.mmas - 4 * s;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if (kk >= left) break;
          const uint32_t ids = (Mma::sf_id(kk) << 4) | (Mma::sf_id(kk) << 29);
          mma_mx<FMT, 1>(tmem, dP + 2 * kk, dQ + 2 * kk, kI | ids, tsp + 4 * Mma::word(kk),
                         tsq + 4 * Mma::word(kk) + qcol, any);
          any = true;
        }
        tc_commit(&empty[slot]);
      }
      tc_commit(done);      // also after a timeout: nothing is in flight when the tile ends
      mbar_wait_drain(done, 0);
    }
    __syncwarp();
  }
  // ------------------------------------------------ epilogue
  const int row = 32 * (warp & 3) + lane;                   // of P: an output feature
  const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
  const int pr = p0 + row;
  const int nq = min(NT, p.M - q0);                          // rows of A in the tile
  const float rb = (p.rb != nullptr && pr < p.N) ? p.rb[pr] : 1.0f;
  const float bias = (p.bias != nullptr && pr < p.N) ? p.bias[pr] : 0.0f;
  auto finish = [&](float acc, int qi) {
    if (pr >= p.N) return;
    const float ra = p.ra != nullptr ? __ldg(p.ra + q0 + qi) : 1.0f;
    store_out(p.out, p.out_type, (size_t)(q0 + qi) * p.N + pr, p.ra != nullptr ? fmaf(acc * ra, rb, bias) : acc + bias);
  };
  float* part = reinterpret_cast<float*>(smem);              // [NT][128], over the drained stages
  if (warp >= 2) {
    const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(done, 0, abort_flag, p.status));
    tc_fence_after();
    if (ok) {
#pragma unroll 1
      for (int c = 0; c < NT; c += 16) {
        uint32_t u[16];
        tmem_ld16(tmem + lane_off + (uint32_t)c, u);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float acc = s1 > s0 ? __uint_as_float(u[e]) : 0.0f;
          if (ranks > 1)
            part[(c + e) * 128 + row] = acc;
          else if (c + e < nq)
            finish(acc, c + e);
        }
      }
    }
    tc_fence_before();
  }
  if (ranks > 1) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    if (warp >= 2)
      for (int qi = rank; qi < nq; qi += ranks) {
        float acc = 0.0f;
        for (int r = 0; r < ranks; ++r) acc += cluster.map_shared_rank(part, r)[qi * 128 + row];
        finish(acc, qi);
      }
    cluster.sync();          // nobody leaves while its partial tile may be read
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, T::kCols);
  }
}

}  // namespace fqa
