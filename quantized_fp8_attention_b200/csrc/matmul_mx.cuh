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

#include <climits>
#include <type_traits>

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

// One lane of a whole warp, the same for every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}

// bulk_load() without a cache policy.
__device__ __forceinline__ void bulk_load_plain(void* smem_dst, const void* gsrc, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(gsrc)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// 32 lanes x 32 bit, 16 consecutive columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// mbar_wait_limit() by a whole warp: one answer for all lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint32_t* status,
                                          uint64_t limit_ns) {
  return __all_sync(0xFFFFFFFFu, mbar_wait_limit(bar, parity, abort_flag, status, limit_ns));
}

// Shared address of the same offset in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t mapa_u32(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_cluster_v4(uint32_t cluster_addr, const uint32_t* v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}
__device__ __forceinline__ void ld_shared_v4(uint32_t addr, uint32_t* v) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Barrier of all threads of the cluster, in two halves (whole warps).
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// A result is sum * ra * rb + bias, formed as fma(sum * ra, rb, bias).  Sums that are
// not 0 lie between 2^-20 (two smallest codes under two smallest scales) and 2^43
// (2688^2 2^20), so with ra far from 1 the first product could leave binary32
// although rb brings the result back.  Such an ra is split into first = 2^62 or
// 2^-62 and the rest: sum * first stays between 2^-82 and 2^105, and times rb it
// leaves binary32 only where the rest, which is on first's side of 1, takes the
// result further out.  fma(sum * first * rb, rest, bias) costs one more rounding.
__device__ __forceinline__ bool far_scale(float a) {
  const float m = fabsf(a);
  return (m > 0.0f && m < 0x1p-80f) || (m > 0x1p80f && m <= 0x1.fffffep127f);
}
__device__ __forceinline__ void split_scale(float a, float& first, float& rest) {
  const bool large = fabsf(a) > 1.0f;
  first = large ? 0x1p62f : 0x1p-62f;
  rest = a * (large ? 0x1p-62f : 0x1p62f);       // exact
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
  uint32_t stop;          // kMxNoStop, or a check of the waits: 16 * stage + rank + 1
  uint32_t* status;
};
// (one word for the check, where the struct had padding: 16 more bytes of
// parameters cost each launch 0.35 us on the host)
constexpr uint32_t kMxNoStop = 0xFFFFFFFFu;
static_assert(sizeof(MxMatmulParams) == 80, "no larger");

// In a check of the waits (fqa_debug_mx_matmul_timeout()) CTA `rank` of a cluster
// (-1: each) loads nothing from its stage `stage` on, so that what waits for it
// runs into its limit, a short one.
__device__ __forceinline__ int loads_until(const MxMatmulParams& p, int rank) {
  const uint32_t who = p.stop & 15u;
  return who == 0 || who == (uint32_t)rank + 1 ? (int)(p.stop >> 4) : INT_MAX;
}
__device__ __forceinline__ uint64_t wait_limit(const MxMatmulParams& p) {
  return p.stop == kMxNoStop ? kWaitLimitNs : kWaitLimitNs / 1000;
}

// ------------------------------------------------------- few rows of A
//
// One 128 x NT tile per cluster of 1, 2, 4 or 8 CTAs.  B's rows (the weights)
// take the MMA's 128-row side and A's rows (the tokens) its N side, so a
// handful of tokens costs an MMA of N = 16, not one of 128 padded rows, and
// the kernel is bound by the weights' bytes.  The CTAs of a cluster split K:
// at 4096 features there are 32 tiles of weights for 148 SMs, so the stages
// are dealt out to `ranks` CTAs.  Group g of four tokens belongs to rank
// g % ranks; every CTA writes its binary32 partial sums into the owner's shared
// memory, 16 bytes a thread, and after one cluster barrier the owner adds them
// in rank order (the same sum every time).
//   warp 0  TMA producer    warp 1  TMEM owner and MMA issuer
//   warps 2-9  epilogue: lane quarter warp % 4, every other group of tokens
// (One warp per scheduler runs the epilogue, so its time is its instruction
// count: token by token it took 100 cycles to push and 400 to add up each.)
// One token against 4096 x 4096 nvfp4 (9.4 MB): 5.5 us, of which the first
// stage's way from memory takes 2.4, two stages of MMAs 0.7, the exchange 1;
// 128 tokens 8.4 us; one token against 16384 x 16384: 27 us, 5.3 TB/s.
constexpr int kMxSmallThreads = 320;

template <int FMT, int NT>
struct MxSmall {
  using Mma = MxMma<FMT>;
  static constexpr int kMaxRanks = 8;
  static constexpr int kPBytes = 128 * 128, kQBytes = NT * 128, kSfBytes = 512 * Mma::kWords;
  static constexpr int kStageBytes = kPBytes + (kQBytes < 1024 ? 1024 : kQBytes) + 2 * kSfBytes;
  static constexpr int kStages = NT == 32 ? 3 : 4;           // (32: two CTAs still fit an SM)
  static constexpr int kOffPart = kStages * kStageBytes;     // partial sums of this rank's groups: [group / ranks][source][128] x 4
  // slots of 128 threads x 16 bytes: one per group, and at least one per rank
  static constexpr int kPartBytes = (NT / 4 < kMaxRanks ? kMaxRanks : NT / 4) * 2048;
  static constexpr int kOffRa = kOffPart + kPartBytes;       // row scales of the tile's tokens
  static constexpr int kOffBar = kOffRa + NT * 4;
  static constexpr int kSmemBytes = kOffBar + (2 * kStages + 1) * 8 + 16 + 1024;
  static constexpr int kSfCols = 8 * Mma::kWords;            // per stage: four for P and four for Q, per word
  static constexpr int kColSf = NT < 32 ? 32 : NT;
  static constexpr int kColsUsed = kColSf + kStages * kSfCols;
  static constexpr int kCols = kColsUsed <= 64 ? 64 : (kColsUsed <= 128 ? 128 : 256);
  static constexpr int kPerSm = 2 * (kSmemBytes + 1024) <= 228 * 1024 ? 2 : 1;
  static_assert(kColsUsed <= 256 && kStageBytes % 1024 == 0 && kSmemBytes <= 232448, "tile layout");
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
  volatile int* far_flag = abort_flag + 1;         // a token's row scale is far_scale()
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const int rank = blockIdx.x % ranks, tile = blockIdx.x / ranks;
  const int ptiles = (p.N + 127) / 128;
  const int p0 = (tile % ptiles) * 128, q0 = (tile / ptiles) * NT;
  const int stages = (p.mmas + 3) / 4;
  // this rank's stages: [s0, s1), an even share
  const int s0 = (int)((int64_t)stages * rank / ranks), s1 = (int)((int64_t)stages * (rank + 1) / ranks);
  const int loads = min(s1 - s0, loads_until(p, rank));   // stages it loads

  auto load_stage = [&](int s, int slot) {         // one thread
    uint8_t* st = smem + slot * T::kStageBytes;
    const uint32_t words = min((int)Mma::kWords, p.KT - s * (int)Mma::kWords);
    mbar_arrive_expect_tx(&full[slot], T::kPBytes + T::kQBytes + 2 * 512 * words);
    tma_load_2d(st, &tmP, &full[slot], s * 128, p0);
    tma_load_2d(st + T::kPBytes, &tmQ, &full[slot], s * 128, q0);
    uint8_t* sf = st + T::kStageBytes - 2 * T::kSfBytes;
    const size_t w0 = (size_t)s * Mma::kWords * 512;
    bulk_load_plain(sf, p.sb + (size_t)(p0 / 128) * p.KT * 512 + w0, 512 * words, &full[slot]);
    bulk_load_plain(sf + T::kSfBytes, p.sa + (size_t)(q0 / 128) * p.KT * 512 + w0, 512 * words, &full[slot]);
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < T::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    *far_flag = 0;
    mbar_fence_init();
    grid_wait();
    // the ring's first fill needs nothing else of the CTA
    for (int i = 0; i < min(loads, T::kStages); ++i) load_stage(s0 + i, i);
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc(tmem_slot, T::kCols);
    tmem_relinquish();
  }
  grid_wait();
  tc_fence_before();
  __syncthreads();
  grid_release();                    // (tensor memory is taken)
  if (ranks > 1) cluster_arrive();   // waited for before the first access to a peer
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // (both issuing warps stay whole and elect a lane per step: see the issuer of
  // the large kernel)
  int issued = 0;                    // warp 0: stages loaded
  if (warp == 0) {
    issued = min(loads, T::kStages);
    for (int i = issued; i < loads; ++i) {
      const int slot = i % T::kStages;
      if (!warp_wait(&empty[slot], ((i / T::kStages) & 1) ^ 1, abort_flag, p.status, wait_limit(p))) break;
      if (elect_one()) load_stage(s0 + i, slot);
      __syncwarp();
      issued = i + 1;
    }
  } else if (warp == 1) {
    constexpr uint32_t kI = Mma::idesc(128, NT);
    // (a tile starts a block of 128 rows of scales: those of fewer tokens are only
    // taken where they are the only one)
    for (int s = s0; s < s1; ++s) {
      const int i = s - s0, slot = i % T::kStages;
      if (!warp_wait(&full[slot], (i / T::kStages) & 1, abort_flag, p.status, wait_limit(p))) break;
      tc_fence_after();
      const uint32_t st = smem_u32(smem + slot * T::kStageBytes);
      const uint32_t sf = st + T::kStageBytes - 2 * T::kSfBytes;
      const uint32_t tsp = tmem + T::kColSf + slot * T::kSfCols, tsq = tsp + 4 * Mma::kWords;
      const int words = min((int)Mma::kWords, p.KT - s * (int)Mma::kWords), left = p.mmas - 4 * s;
      const uint64_t dP = make_sdesc_sw128(st, 16, 1024), dQ = make_sdesc_sw128(st + T::kPBytes, 16, 1024);
      const uint64_t dSp = make_sdesc_plain(sf), dSq = make_sdesc_plain(sf + T::kSfBytes);
      if (elect_one()) {
#pragma unroll
        for (int w = 0; w < (int)Mma::kWords; ++w) {
          if (w >= words) break;
          tmem_cp_scales<1>(tsp + 4 * w, dSp + 32 * w);
          tmem_cp_scales<1>(tsq + 4 * w, dSq + 32 * w);
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if (kk >= left) break;
          const uint32_t ids = (Mma::sf_id(kk) << 4) | (Mma::sf_id(kk) << 29);
          mma_mx<FMT, 1>(tmem, dP + 2 * kk, dQ + 2 * kk, kI | ids, tsp + 4 * Mma::word(kk),
                         tsq + 4 * Mma::word(kk), s > s0 || kk > 0);
        }
        tc_commit(&empty[slot]);
      }
      __syncwarp();
    }
    if (elect_one()) tc_commit(done);   // also after a timeout: nothing is in flight when the tile ends
    __syncwarp();
    mbar_wait_drain(done, 0);
    __syncwarp();
  }
  // ------------------------------------------------ epilogue
  const int row = 32 * (warp & 3) + lane;                   // of P: an output feature
  const int half = (warp - 2) >> 2;
  const int pr = p0 + row;
  const int nq = min(NT, p.M - q0);                          // rows of A in the tile
  const bool scaled = p.ra != nullptr;
  float rb = 1.0f, bias = 0.0f;
  bool far = false;
  float* ra = reinterpret_cast<float*>(smem + T::kOffRa);
  if (warp >= 2) {
    // fetched while the products run
    const int q = threadIdx.x - 64;
    if (q < NT) {
      ra[q] = scaled && q < nq ? p.ra[q0 + q] : 1.0f;
      if (far_scale(ra[q])) *far_flag = 1;
    }
    if (pr < p.N) {
      if (p.rb != nullptr) rb = p.rb[pr];
      if (p.bias != nullptr) bias = p.bias[pr];
    }
    bar_sync(1, kMxSmallThreads - 64);
    far = *far_flag != 0;
  }
  // tokens q .. q + 3 of this thread's feature
  auto finish = [&](const float (&acc)[4], int q) {
    if (pr >= p.N) return;
    const float4 r = *reinterpret_cast<const float4*>(ra + q);
    float v[4] = {scaled ? fmaf(acc[0] * r.x, rb, bias) : acc[0] + bias,
                  scaled ? fmaf(acc[1] * r.y, rb, bias) : acc[1] + bias,
                  scaled ? fmaf(acc[2] * r.z, rb, bias) : acc[2] + bias,
                  scaled ? fmaf(acc[3] * r.w, rb, bias) : acc[3] + bias};
    if (FMT == kNvFp4 && far) {      // (512 x 4096 x 4096 10.3 -> 10.5 us, fewer rows unchanged; in a pass or
                                     // loops of its own it cost those more)
      const float a[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (far_scale(a[e])) {
          float first, rest;
          split_scale(a[e], first, rest);
          v[e] = fmaf(acc[e] * first * rb, rest, bias);
        }
    }
    const size_t at = (size_t)(q0 + q) * p.N + pr;
    auto store = [&](auto* out) {
      using O = std::remove_pointer_t<decltype(out)>;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (q + e < nq) out[at + (size_t)e * p.N] = from_f32<O>(v[e]);
    };
    if (p.out_type == 0)
      store(static_cast<__nv_bfloat16*>(p.out));
    else if (p.out_type == 1)
      store(static_cast<float*>(p.out));
    else
      store(static_cast<__half*>(p.out));
  };
  bool ok = true;
  if (warp >= 2) {
    ok = warp_wait(done, 0, abort_flag, p.status, wait_limit(p));
    tc_fence_after();
  }
  if (ranks > 1) cluster_wait();
  const int lg = 31 - __clz(ranks);                          // ranks: a power of two
  const uint32_t part = smem_u32(smem + T::kOffPart) + 16u * (uint32_t)row;
  if (warp >= 2 && ok) {
    const uint32_t acc = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
#pragma unroll 1
    for (int c = 16 * half; c < nq; c += 32) {
      uint32_t u[16];
      tmem_ld16(acc + (uint32_t)c, u);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        if (c + e >= nq) break;
        if (ranks == 1) {
          finish({__uint_as_float(u[e]), __uint_as_float(u[e + 1]), __uint_as_float(u[e + 2]), __uint_as_float(u[e + 3])},
                 c + e);
        } else {
          const int g = (c + e) >> 2;
          st_cluster_v4(mapa_u32(part + 2048u * (uint32_t)(((g >> lg) << lg) + rank), (uint32_t)(g & (ranks - 1))),
                        &u[e]);
        }
      }
    }
    tc_fence_before();
  }
  if (ranks > 1) {
    cluster_arrive();
    cluster_wait();
    if (warp >= 2)
      for (int i = half; 4 * ((i << lg) + rank) < nq; i += 2) {
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        uint32_t v[T::kMaxRanks][4];
#pragma unroll
        for (int r = 0; r < T::kMaxRanks; ++r)
          if (r < ranks) ld_shared_v4(part + 2048u * (uint32_t)((i << lg) + r), v[r]);
#pragma unroll
        for (int r = 0; r < T::kMaxRanks; ++r)
          if (r < ranks)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] += __uint_as_float(v[r][e]);
        finish(acc, 4 * ((i << lg) + rank));
      }
  }
  __syncthreads();
  // after a wait that gave up, in whichever warp: no copy may be in flight when
  // the CTA ends
  if (warp == 0 && *abort_flag)
    for (int i = max(0, issued - T::kStages); i < issued; ++i)
      mbar_wait_drain(&full[i % T::kStages], (i / T::kStages) & 1);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, T::kCols);
  }
}

// ------------------------------------------------------ many rows of A
//
// 256 x 256 tiles by pairs of CTAs (cta_group::2): each CTA holds 128 rows of
// A and 128 of B per stage, the pair's tensor cores share both, so a stage of
// 256 4-bit channels costs each SM 32 KB of codes for 512 cycles of MMAs: the
// largest tile tensor memory allows and the one with the least traffic per
// product.  Persistent: a pair walks over its tiles, and the producer runs
// ahead into the next tile while the epilogue drains the last.
//   warp 0     TMA producer (both CTAs; completion on the leader's barriers)
//   warp 1     TMEM owner; in the leader CTA also the MMA issuer
//   warps 4-11 epilogue: lane quarter warp % 4, columns 128 (warp / 4 - 1) ..
// Tensor memory: the tile's 256 columns of sums, then per stage 4 columns per
// word for A's scales and 8 for B's (both CTAs need all of B's).  There is no
// room for a second tile of sums, so the epilogue first moves its 128 columns
// into registers and gives the columns back before it scales, rounds and
// stores.  Stores go through shared memory, 32 rows x 128 bytes a warp and
// step, as TMA stores (or, where the output's rows are not on 16-byte
// boundaries, as coalesced element stores).
//
// Measured: mxfp8 4608 x 4096 x 4096 57 us (2.7 PFLOP/s), a stage in 553 cycles
// of the 512 its MMAs take; nvfp4 8704 x 12288 x 4096 183 us (4.8 PFLOP/s), 644
// cycles a stage.  What bounds it: power (the clock falls from 1.97 to 1.5-1.6
// GHz; looped without a pause the two take 68 and 207 us) and, for the 4-bit
// formats, the operands' way from L2 (without loads the second takes 144 us).
constexpr int kMxLargeThreads = 384;

// Words by which a pair parts (part_after_giving_up()): kept by each CTA for
// itself, then what both know.
enum : int { kLoaded, kStagesOut, kTilesOut, kGaveUp, kLoaded0, kLoaded1, kStagesBoth, kTilesBoth, kNotes };

template <int FMT>
struct MxLarge {
  using Mma = MxMma<FMT>;
  static constexpr int kOpBytes = 128 * 128;
  static constexpr int kSfaBytes = 512 * Mma::kWords, kSfbBytes = 1024 * Mma::kWords;
  static constexpr int kStageBytes = (2 * kOpBytes + kSfaBytes + kSfbBytes + 1023) / 1024 * 1024;
  static constexpr int kTxBytes = 2 * (2 * kOpBytes + kSfaBytes + kSfbBytes);   // both CTAs
  static constexpr int kStages = 5;
  static constexpr int kOffStage = 0;
  static constexpr int kOffOut = kStages * kStageBytes;      // 8 warps x 4 KB
  static constexpr int kOffCol = kOffOut + 8 * 4096;         // row scales and bias of the tile's columns
  static constexpr int kOffBar = kOffCol + 2 * 256 * 4;
  static constexpr int kOffNote = kOffBar + (2 * kStages + 2) * 8 + 16;   // kNotes words
  static constexpr int kSmemBytes = kOffNote + kNotes * 4 + 1024;
  static constexpr int kColSf = 256, kSfCols = 12 * Mma::kWords;
  static_assert(kColSf + kStages * kSfCols <= 512, "tensor memory");
  static_assert(kSmemBytes <= 232448, "shared memory");
};

// Arrival on a barrier of the cluster.  Only tensor memory is handed over with
// it (ordered by the tcgen05 fences around), so the order of ordinary memory
// stays within the CTA: a release to the cluster waits for every outstanding
// store, 1300 cycles in each tile's critical path.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// Tiled loads of a CTA pair: the destination is this CTA's, the barrier may
// be the peer's (both given as shared addresses of the cluster).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* m, uint32_t bar, int32_t x,
                                                 int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* m, uint32_t bar, int32_t x,
                                                 int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// 2-D tiled store; x on a 16-byte boundary and not negative.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, uint32_t src, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(src), "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// tc_commit() of a pair: arrives on the barrier at this offset in both CTAs.
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// A note in both CTAs of the pair.
__device__ __forceinline__ void note_pair(int* note, int v) {
  for (uint32_t r = 0; r < 2; ++r)
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_u32(smem_u32(note), r)), "r"(v) : "memory");
}
// Takes bytes off what the barrier's phase still expects.
__device__ __forceinline__ void mbar_complete_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// The pair's end after a wait that gave up, in either CTA.  Nothing may reach a CTA
// after it ends, nor an MMA run on, so both wait here (again with a limit) for
//  - the commits that were issued: each stage's MMAs end with one to both CTAs, so
//    these are the MMAs too.  The last on each barrier is enough: the one before
//    was seen here before the issuer could get as far;
//  - the copies in flight, whose bytes complete on the leader's barriers.  A stage
//    that only one CTA loaded would never complete: the leader takes the other's
//    bytes off what it expected, or makes the arrival that it owes with the
//    other's bytes alone.
// (Not inlined: what follows it in the kernel stays next to what comes before.)
template <typename T>
__device__ __noinline__ void part_after_giving_up(volatile int* note, uint32_t rank, uint64_t* full, uint64_t* empty,
                                                  uint64_t* acc_full) {
  constexpr int S = T::kStages;
  if (threadIdx.x == 0) {
    note_pair((int*)note + kLoaded0 + rank, note[kLoaded]);
    if (rank == 0) {
      note_pair((int*)note + kStagesBoth, note[kStagesOut]);
      note_pair((int*)note + kTilesBoth, note[kTilesOut]);
    }
  }
  cluster_arrive();
  cluster_wait();
  if (threadIdx.x == 0) {
    const int n0 = note[kLoaded0], n1 = note[kLoaded1], n = max(n0, n1);
    const int stages = note[kStagesBoth], tiles = note[kTilesBoth];
    for (int j = max(0, stages - S); j < stages; ++j) mbar_wait_drain(&empty[j % S], (j / S) & 1);
    if (tiles > 0) mbar_wait_drain(acc_full, (tiles - 1) & 1);
    if (rank == 0) {
      for (int j = min(n0, n1); j < n; ++j) {
        if (n0 > n1)
          mbar_complete_tx(&full[j % S], T::kTxBytes / 2);
        else
          mbar_arrive_expect_tx(&full[j % S], T::kTxBytes / 2);
      }
      for (int j = max(0, n - S); j < n; ++j) mbar_wait_drain(&full[j % S], (j / S) & 1);
    }
  }
  __syncthreads();
  cluster_arrive();
  cluster_wait();
}

// Tile t of mt x nt: bands of eight row tiles, column by column within a
// band, so that the pairs at work share A's and B's tiles in L2.
__device__ __forceinline__ void large_tile(int64_t t, int mt, int nt, int& m, int& n) {
  const int64_t band = t / (8LL * nt);
  const int rows = min(8, mt - (int)band * 8);
  const int in = (int)(t - band * 8LL * nt);
  n = in / rows;
  m = (int)band * 8 + in % rows;
}

template <int FMT>
__global__ void __launch_bounds__(kMxLargeThreads, 1)
    mx_matmul_large_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                           const __grid_constant__ CUtensorMap tmSa, const __grid_constant__ CUtensorMap tmSb,
                           const __grid_constant__ CUtensorMap tmOut, const MxMatmulParams p, int tma_out) {
  using T = MxLarge<FMT>;
  using Mma = MxMma<FMT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + T::kOffBar);
  uint64_t* empty = full + T::kStages;
  uint64_t* acc_full = empty + T::kStages;
  uint64_t* acc_free = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_free + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* note = reinterpret_cast<volatile int*>(smem + T::kOffNote);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = blockIdx.x & 1;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int mt = (p.M + 255) / 256, nt = (p.N + 255) / 256;
  const int64_t tiles = (int64_t)mt * nt;
  const int stages = (p.mmas + 3) / 4;

  if (threadIdx.x == 0) {
    for (int s = 0; s < T::kStages; ++s) {
      mbar_init(&full[s], 1);        // the leader's expectation; bytes from both CTAs
      mbar_init(&empty[s], 1);       // the pair's commit
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_free, 16);         // the epilogue warps of both CTAs
    *abort_flag = 0;
    note[kGaveUp] = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  grid_wait();
  tc_fence_before();
  __syncthreads();
  grid_release();                    // (tensor memory is taken)
  cluster_arrive();
  cluster_wait();                // the peer's barriers are ready too
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  bool ok = true;                    // no wait of this warp has given up
  if (warp == 0) {
    // ------------------------------------------------ producer
    int i = 0;                       // stages issued so far
    const int until = loads_until(p, (int)rank);
    for (int64_t t = pair; ok && t < tiles; t += pairs) {
      int mi, ni;
      large_tile(t, mt, nt, mi, ni);
      const int arow = mi * 256 + 128 * (int)rank, brow = ni * 256 + 128 * (int)rank;
      for (int s = 0; s < stages; ++s, ++i) {
        const int slot = i % T::kStages;
        if (!(ok = i < until && warp_wait(&empty[slot], ((i / T::kStages) & 1) ^ 1, abort_flag, p.status, wait_limit(p)))) break;
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&full[slot], T::kTxBytes);
          const uint32_t bar = mapa_u32(smem_u32(&full[slot]), 0);
          const uint32_t st = mapa_u32(smem_u32(smem + slot * T::kStageBytes), rank);
          tma_load_2d_pair(st, &tmA, bar, s * 128, arow);
          tma_load_2d_pair(st + T::kOpBytes, &tmB, bar, s * 128, brow);
          tma_load_3d_pair(st + 2 * T::kOpBytes, &tmSa, bar, 0, s * Mma::kWords, arow / 128);
          tma_load_3d_pair(st + 2 * T::kOpBytes + T::kSfaBytes, &tmSb, bar, 0, s * Mma::kWords, ni * 2);
        }
        __syncwarp();
      }
    }
    // nothing may reach this CTA after it ends: the slots' last releases (after a
    // wait that gave up, part_after_giving_up() sees to it)
    if (ok)
      for (int j = max(0, i - T::kStages); j < i; ++j)
        if (!(ok = warp_wait(&empty[j % T::kStages], (j / T::kStages) & 1, abort_flag, p.status, wait_limit(p)))) break;
    if (lane == 0) note[kLoaded] = i;
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    // ------------------------------------------------ MMA issuer
    // The whole warp walks through the loop and one elected lane issues: the
    // descriptors then stay in uniform registers.  From a branch of a single
    // lane each tcgen05 instruction took about 70 cycles to issue (16 of them
    // per stage: 1086 cycles for 512 cycles of MMAs), so the copies alone
    // halved the rate.
    constexpr uint32_t kI = Mma::idesc(256, 256);
    int i = 0, done = 0;             // commits of stages and of tiles
    for (int64_t t = pair; ok && t < tiles; t += pairs) {
      // the last tile's sums have left tensor memory
      if (!(ok = warp_wait(acc_free, (done & 1) ^ 1, abort_flag, p.status, wait_limit(p)))) break;
      for (int s = 0; s < stages; ++s, ++i) {
        const int slot = i % T::kStages;
        if (!(ok = warp_wait(&full[slot], (i / T::kStages) & 1, abort_flag, p.status, wait_limit(p)))) break;
        tc_fence_after();
        const uint32_t st = smem_u32(smem + slot * T::kStageBytes);
        const uint32_t tsa = tmem + T::kColSf + slot * T::kSfCols, tsb = tsa + 4 * Mma::kWords;
        const uint64_t dA = make_sdesc_sw128(st, 16, 1024), dB = make_sdesc_sw128(st + T::kOpBytes, 16, 1024);
        const uint64_t dSa = make_sdesc_plain(st + 2 * T::kOpBytes);
        const uint64_t dSb = make_sdesc_plain(st + 2 * T::kOpBytes + T::kSfaBytes);
        const int left = p.mmas - 4 * s;
        if (elect_one()) {
          // B's two blocks of 128 rows land word by word side by side: eight
          // columns per word
#pragma unroll
          for (int w = 0; w < (int)Mma::kWords; ++w) {
            tmem_cp_scales<2>(tsa + 4 * w, dSa + 32 * w);
            tmem_cp_scales<2>(tsb + 8 * w, dSb + 32 * w);
            tmem_cp_scales<2>(tsb + 8 * w + 4, dSb + 32 * (Mma::kWords + w));
          }
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if (kk >= left) break;
            const uint32_t ids = (Mma::sf_id(kk) << 4) | (Mma::sf_id(kk) << 29);
            mma_mx<FMT, 2>(tmem, dA + 2 * kk, dB + 2 * kk, kI | ids, tsa + 4 * Mma::word(kk),
                           tsb + 8 * Mma::word(kk), s > 0 || kk > 0);
          }
          tc_commit_pair(&empty[slot]);
          if (s == stages - 1) tc_commit_pair(acc_full);
        }
        __syncwarp();
      }
      done += ok;
    }
    if (lane == 0) {
      note[kStagesOut] = i;
      note[kTilesOut] = done;
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------ epilogue
    const int q = warp & 3, half = (warp >> 2) - 1;
    const int et = threadIdx.x - 128;                         // 0..255
    const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + 128u * (uint32_t)half;
    const uint32_t stage = smem_u32(smem + T::kOffOut + (warp - 4) * 4096);
    const uint32_t free_leader = mapa_u32(smem_u32(acc_free), 0);
    const bool cols = p.rb != nullptr || p.bias != nullptr;
    int done = 0;                    // (after a timeout the warps still meet at the barriers below)
    for (int64_t t = pair; t < tiles; t += pairs, ++done) {
      int mi, ni;
      large_tile(t, mt, nt, mi, ni);
      const int row0 = mi * 256 + 128 * (int)rank + 32 * q, n0 = ni * 256 + 128 * half;
      float* sc = reinterpret_cast<float*>(smem + T::kOffCol);
      if (cols) {
        bar_sync(1, 256);            // everyone is through with the last tile's
        const int n = ni * 256 + et;
        sc[et] = (p.rb != nullptr && n < p.N) ? p.rb[n] : 1.0f;
        sc[256 + et] = (p.bias != nullptr && n < p.N) ? p.bias[n] : 0.0f;
        bar_sync(1, 256);
      }
      const float ra = (p.ra != nullptr && row0 + lane < p.M) ? p.ra[row0 + lane] : 1.0f;
      ok = ok && warp_wait(acc_full, done & 1, abort_flag, p.status, wait_limit(p));
      if (!ok) continue;
      tc_fence_after();
      uint32_t u[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(acc + 32u * c, u[c]);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(free_leader);
      const float* rb = sc + 128 * half;
      const float* bias = rb + 256;
      if (FMT == kNvFp4 && far_scale(ra)) {
        // (through local memory, 32 sums at a time: unrolled it cost the loop around
        // it spills)
        float first, rest;
        split_scale(ra, first, rest);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) w[e] = u[c][e];
#pragma unroll 1
          for (int e = 0; e < 32; ++e)
            w[e] = __float_as_uint(fmaf(__uint_as_float(w[e]) * first * rb[32 * c + e], rest, bias[32 * c + e]));
#pragma unroll
          for (int e = 0; e < 32; ++e) u[c][e] = w[e];
        }
      } else if (cols) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 f = *reinterpret_cast<const float4*>(rb + 32 * c + e);
            const float4 g = *reinterpret_cast<const float4*>(bias + 32 * c + e);
            const float2 r2 = make_float2(ra, ra);
            const float2 lo = f2_fma(f2_mul(make_float2(__uint_as_float(u[c][e]), __uint_as_float(u[c][e + 1])), r2),
                                     make_float2(f.x, f.y), make_float2(g.x, g.y));
            const float2 hi = f2_fma(f2_mul(make_float2(__uint_as_float(u[c][e + 2]), __uint_as_float(u[c][e + 3])), r2),
                                     make_float2(f.z, f.w), make_float2(g.z, g.w));
            u[c][e] = __float_as_uint(lo.x);
            u[c][e + 1] = __float_as_uint(lo.y);
            u[c][e + 2] = __float_as_uint(hi.x);
            u[c][e + 3] = __float_as_uint(hi.y);
          }
        }
      }
      if (row0 >= p.M) continue;
      // one step: 32 rows x 128 bytes (64 16-bit or 32 binary32 columns)
      const uint32_t line = stage + (uint32_t)lane * 128u, sw = (uint32_t)(lane & 7);
      auto flush = [&](int col0, int width) {
        if (tma_out) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && n0 + col0 < p.N) {
            tma_store_2d(&tmOut, stage, n0 + col0, row0);
            bulk_commit();
          }
        } else {
          __syncwarp();
          // lanes side by side along the row; eight rows' values before their stores
          const uint32_t per = 128u / (uint32_t)width;       // bytes per value
          for (int j = lane; j < width; j += 32) {
            const int n = n0 + col0 + j;
            const uint32_t byte = (uint32_t)j * per;
#pragma unroll 1
            for (int r0 = 0; r0 < 32; r0 += 8) {
              uint32_t v[8];
#pragma unroll
              for (int r = 0; r < 8; ++r) {                  // (row r0 + r of the stage: its chunks are swizzled by r)
                const uint32_t at = stage + (uint32_t)(r0 + r) * 128u + (((byte >> 4) ^ (uint32_t)r) << 4) + (byte & 12u);
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v[r]) : "r"(at));
              }
#pragma unroll
              for (int r = 0; r < 8; ++r) {
                if (n >= p.N || row0 + r0 + r >= p.M) continue;
                const size_t at = (size_t)(row0 + r0 + r) * p.N + n;
                if (width == 32)
                  static_cast<uint32_t*>(p.out)[at] = v[r];
                else
                  static_cast<uint16_t*>(p.out)[at] = (uint16_t)(v[r] >> (8u * (byte & 2u)));
              }
            }
          }
          __syncwarp();
        }
      };
      auto ready = [&]() {           // the last step's store has read the buffer
        if (tma_out && lane == 0) bulk_wait_read();
        __syncwarp();
      };
      if (p.out_type == 1) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          ready();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            st_shared_v4(line + (((uint32_t)j ^ sw) << 4), u[c][4 * j], u[c][4 * j + 1], u[c][4 * j + 2],
                         u[c][4 * j + 3]);
          flush(32 * c, 32);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          ready();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float lo = __uint_as_float(u[2 * c + j / 4][8 * (j % 4) + 2 * e]);
              const float hi = __uint_as_float(u[2 * c + j / 4][8 * (j % 4) + 2 * e + 1]);
              w[e] = p.out_type == 0 ? pack2<__nv_bfloat16>(lo, hi) : pack2<__half>(lo, hi);
            }
            st_shared_v4(line + (((uint32_t)j ^ sw) << 4), w[0], w[1], w[2], w[3]);
          }
          flush(64 * c, 64);
        }
      }
    }
    if (tma_out && lane == 0) bulk_wait_read();
    __syncwarp();
  }
  tc_fence_before();
  if (__syncthreads_or(!ok) && threadIdx.x == 0) note_pair((int*)note + kGaveUp, 1);
  cluster_arrive();
  cluster_wait();
  // (where all went well the last releases have been waited for)
  if (note[kGaveUp]) part_after_giving_up<T>(note, rank, full, empty, acc_full);
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

}  // namespace fqa
