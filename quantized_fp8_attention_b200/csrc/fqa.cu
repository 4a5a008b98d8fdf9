// fqa.cu -- the library's C ABI (include/fqa.h): host-side argument checks,
// TMA tensor-map encoding and kernel launches.  One translation unit holds
// every kernel, so the device status word needs no relocatable device code.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <utility>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/fqa.h"
#include "attention.cuh"
#include "attention_fp8.cuh"
#include "attention_nvfp4.cuh"
#include "attention_ws.cuh"
#include "correct.cuh"
#include "device.cuh"
#include "matmul_mx.cuh"
#include "microscale.cuh"
#include "quantize.cuh"
#include "quantize_nvfp4.cuh"
#include "rotary.cuh"

namespace fqa {

__device__ uint32_t g_status_word;

constexpr int kMaxDevices = 64;
constexpr int64_t kMxMaxRows = 1 << 24;    // rows and columns of a microscaled operand
constexpr int kMxMaxCols = 1 << 20;

// Per-device lookups, cached only once they succeed: a failed first call
// (e.g. one made while a stream is being captured) is retried by the next.
struct DeviceCache {
  std::mutex mu;
  uint32_t* status = nullptr;
  int num_sms = 0;
};
DeviceCache g_dev[kMaxDevices];

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
std::once_flag g_encode_once;
EncodeTiledFn g_encode = nullptr;

// The answer to a failed runtime call, which keeps its error for whoever asks
// next: taken here, so that a later launch's status is its own.
static fqa_status cuda_failed() {
  cudaGetLastError();
  return FQA_ERR_CUDA;
}

static fqa_status launch_status() {
  return cudaGetLastError() == cudaSuccess ? FQA_OK : FQA_ERR_CUDA;
}

static uint32_t* status_ptr(fqa_status* st) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    *st = cuda_failed();
    return nullptr;
  }
  DeviceCache& c = g_dev[dev];
  std::lock_guard<std::mutex> lock(c.mu);
  if (c.status == nullptr) {
    void* p = nullptr;
    int sms = 0;
    if (cudaGetSymbolAddress(&p, g_status_word) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        p == nullptr || sms <= 0) {
      *st = cuda_failed();
      return nullptr;
    }
    c.num_sms = sms;
    c.status = static_cast<uint32_t*>(p);
  }
  return c.status;
}

static EncodeTiledFn encoder() {
  std::call_once(g_encode_once, []() {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<EncodeTiledFn>(fn);
  });
  return g_encode;
}

// 3-D view (channel, row within the head, head) of a [B,H,N,128] tensor; box
// = 128 B of channels x 128 rows x 1 head, 128-byte swizzle.  Rows past N
// (the short last tile of a sequence) are filled with zeros, never read from
// the next head.
static bool make_tmap(CUtensorMap* m, const void* base, bool fp8, int N, int heads) {
  EncodeTiledFn enc = encoder();
  if (!enc) return false;
  const uint32_t elt = fp8 ? 1 : 2;
  cuuint64_t dims[3] = {128, (cuuint64_t)N, (cuuint64_t)heads};
  cuuint64_t strides[2] = {128ull * elt, 128ull * elt * (cuuint64_t)N};
  cuuint32_t box[3] = {128u / elt, 128u, 1u};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                   const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// 3-D view (byte, row within the head, head) of packed E2M1 codes
// [B,H,N,64 B]; box = 64 B x 128 rows x 1 head, 64-byte swizzle (the layout
// the block-scaled MMA reads through a SWIZZLE_64B descriptor).
static bool make_tmap_fp4(CUtensorMap* m, const void* base, int N, int heads) {
  EncodeTiledFn enc = encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {64, (cuuint64_t)N, (cuuint64_t)heads};
  cuuint64_t strides[2] = {64ull, 64ull * (cuuint64_t)N};
  cuuint32_t box[3] = {64u, 128u, 1u};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// 2-D view (byte, row) of rows of codes, row_bytes a multiple of 16; box = 128
// bytes x box_rows rows, 128-byte swizzle.  Bytes and rows past the end read
// as zeros.
static bool make_tmap_rows(CUtensorMap* m, const void* base, int row_bytes, int rows, int box_rows) {
  EncodeTiledFn enc = encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)row_bytes, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
  cuuint32_t box[2] = {128u, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// 3-D view (word, word column, block of 128 rows) of scale tiles as 32-bit
// words: a tile is 128 words; box = `words` tiles of `blocks` row blocks.  Tiles
// past the end read as zeros.
static bool make_tmap_scales(CUtensorMap* m, const void* base, int KT, int rows, int words, int blocks) {
  EncodeTiledFn enc = encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {128, (cuuint64_t)KT, (cuuint64_t)(rows + 127) / 128};
  cuuint64_t strides[2] = {512ull, 512ull * (cuuint64_t)KT};
  cuuint32_t box[3] = {128u, (cuuint32_t)words, (cuuint32_t)blocks};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// 2-D view of a product [M, N] for stores of 32 rows x 128 bytes, 128-byte
// swizzle; rows on 16-byte boundaries.
static bool make_tmap_out(CUtensorMap* m, const void* base, int type, int M, int N) {
  EncodeTiledFn enc = encoder();
  if (!enc) return false;
  const uint32_t elt = type == FQA_DTYPE_F32 ? 4 : 2;
  cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)M};
  cuuint64_t strides[1] = {(cuuint64_t)N * elt};
  cuuint32_t box[2] = {128u / elt, 32u};
  cuuint32_t estr[2] = {1, 1};
  const CUtensorMapDataType t = type == FQA_DTYPE_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                : type == FQA_DTYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUresult r = enc(m, t, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

static bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Shape checks shared by every call: any N >= 1 (the last 64-token block and
// the last 128-key tile of a head may be short).
static fqa_status check_shape(int B, int H, int N, int d) {
  if (B < 1 || H < 1 || N < 1 || d < 1) return FQA_ERR_INVALID_ARG;
  if (d != 128) return FQA_ERR_UNSUPPORTED;
  if (N > 65536) return FQA_ERR_UNSUPPORTED;
  if ((int64_t)B * H > 65535) return FQA_ERR_UNSUPPORTED;
  if ((int64_t)B * H * N >= (int64_t(1) << 31)) return FQA_ERR_UNSUPPORTED;
  return FQA_OK;
}


// SM count of the current device (valid once status_ptr() succeeded on it).
static int num_sms() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  std::lock_guard<std::mutex> lock(g_dev[dev].mu);
  return g_dev[dev].num_sms;
}

// BF16: persistent launch, one CTA per SM (or per work item, if fewer).
static fqa_status launch_attention_bf16(const void* q, const void* k, const void* v,
                                        const AttnParams& prm, cudaStream_t stream) {
  const int heads = prm.B * prm.H;
  CUtensorMap tq, tk, tv;
  if (!make_tmap(&tq, q, false, prm.N, heads) || !make_tmap(&tk, k, false, prm.N, heads) ||
      !make_tmap(&tv, v, false, prm.N, heads))
    return cuda_failed();
  if (cudaFuncSetAttribute(attn_bf16_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           BfTraits::kSmemBytes) != cudaSuccess)
    return cuda_failed();
  const int items = prm.B * prm.H * ((prm.N + kPairRows - 1) / kPairRows);
  const int sms = num_sms();
  if (sms <= 0) return cuda_failed();
  const int grid = items < sms ? items : sms;
  attn_bf16_kernel<<<grid, kWsThreads, BfTraits::kSmemBytes, stream>>>(tq, tk, tv, prm);
  return launch_status();
}

// FP8: persistent launch of the shared-memory-P kernel, one CTA per SM (or
// per work item, if fewer).
static fqa_status launch_attention_fp8(const void* q, const void* k, const void* v,
                                       const AttnParams& prm, cudaStream_t stream) {
  const int heads = prm.B * prm.H;
  CUtensorMap tq, tk, tv;
  if (!make_tmap(&tq, q, true, prm.N, heads) || !make_tmap(&tk, k, true, prm.N, heads) ||
      !make_tmap(&tv, v, true, prm.N, heads))
    return cuda_failed();
  // the instance that carries only what the call needs: the short-tail patch
  // when N is not a multiple of 128, the key mask and row statistics when
  // given
  const bool tail = prm.N % kBlockN != 0;
  const bool masked = prm.kmask != nullptr || prm.row_stats != nullptr;
  using KernelFn = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const AttnParams);
  KernelFn fn = tail ? (masked ? attn_fp8_kernel<true, true> : attn_fp8_kernel<true, false>)
                     : (masked ? attn_fp8_kernel<false, true> : attn_fp8_kernel<false, false>);
  // a key mask that leaves a key in every 64-key block of an aligned N:
  // patched tiles instead of masking (the caller checks the condition)
  if (prm.patch && !tail && prm.kmask != nullptr) fn = attn_fp8_kernel<false, false, true>;
  if (cudaFuncSetAttribute((const void*)fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           F8Traits::kSmemBytes) != cudaSuccess)
    return cuda_failed();
  const int items = prm.B * prm.H * ((prm.N + 2 * kBlockM - 1) / (2 * kBlockM));
  const int sms = num_sms();
  if (sms <= 0) return cuda_failed();
  const int grid = items < sms ? items : sms;
  fn<<<grid, kF8Threads, F8Traits::kSmemBytes, stream>>>(tq, tk, tv, prm);
  return launch_status();
}

static size_t dtype_bytes(int t) { return t == FQA_DTYPE_F32 ? 4 : 2; }

// -------------------------------------------- launches of microscaled rows

// Launches a kernel that waits for its predecessor itself (grid_wait()), so that
// its CTAs are scheduled and set up while that one ends; in clusters of
// `cluster` CTAs.
template <typename... P, typename... A>
static fqa_status launch_overlapped(void (*fn)(P...), dim3 grid, dim3 block, int smem, cudaStream_t s, int cluster,
                                    A&&... args) {
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, fn, std::forward<A>(args)...) == cudaSuccess ? FQA_OK : cuda_failed();
}

// One launch of the row kernel that fits the row: 16 elements a thread and
// chunk, two chunks in registers (one of binary32: 103 registers a thread left
// two CTAs per SM, 23 us for 1023 x 5100).  A warp takes a row that fits it (no
// CTA-wide sums); else a CTA of just the warps it needs (1023 x 5100 in 512
// threads instead of 320: 19 us); rows beyond 512 threads are read again for
// each step.  Rows off the 16-byte boundaries go through shared memory while
// they fit there.
template <typename T, int FMT, bool kNorm>
static fqa_status launch_mx_rows(const MxRowParams& p, bool vec, bool pairs, cudaStream_t s) {
  constexpr int NCH = sizeof(T) == 4 ? 1 : 2;
  const int chunks = p.KT * MxTraits<FMT>::kWordChunks;
  const int threads = (chunks + NCH - 1) / NCH;  // that hold the row's words, whole
  if (!vec && chunks * kMxChunk <= kMxAnyCols) {
    const int smem = chunks * kMxChunk * 4;
    const auto fn = pairs ? mx_row_any_kernel<T, FMT, kNorm, 2> : mx_row_any_kernel<T, FMT, kNorm, 1>;
    // the default limit of 48 KB holds the row and the kernel's own arrays (a row
    // padded to 12288 values fills it alone)
    if (smem + kMxAnyStatic > 48 * 1024 && cudaFuncSetAttribute((const void*)fn,
                                                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                                kMxAnyCols * 4) != cudaSuccess)
      return cuda_failed();
    return launch_overlapped(fn, p.M, kMxAnyThreads, smem, s, 1, p);
  }
  if (!vec) return launch_overlapped(mx_row_kernel<T, FMT, kNorm, true, 1, true, false>, p.M, 512, 0, s, 1, p);
  if (threads <= 32)
    return launch_overlapped(mx_row_kernel<T, FMT, kNorm, false, NCH, false, true>, (p.M + 3) / 4, 128, 0, s, 1, p);
  if (threads <= 512)
    return launch_overlapped(mx_row_kernel<T, FMT, kNorm, true, NCH, false, true>, p.M, (threads + 31) / 32 * 32, 0, s,
                             1, p);
  return launch_overlapped(mx_row_kernel<T, FMT, kNorm, true, 1, true, true>, p.M, 512, 0, s, 1, p);
}

template <typename T, bool kNorm>
static fqa_status launch_mx_format(const MxRowParams& p, int fmt, bool vec, bool pairs, cudaStream_t s) {
  if (fmt == FQA_MXFP8) return launch_mx_rows<T, kMxFp8, kNorm>(p, vec, pairs, s);
  if (fmt == FQA_MXFP4) return launch_mx_rows<T, kMxFp4, kNorm>(p, vec, pairs, s);
  return launch_mx_rows<T, kNvFp4, kNorm>(p, vec, pairs, s);
}

// align: the widest access that every row of every tensor allows, of 32, 16, 2
// values or 1 (see rows_vectorize()).
template <bool kNorm>
static fqa_status launch_mx(const MxRowParams& p, int dtype, int fmt, int align, cudaStream_t s) {
  const bool vec = align >= 16, pairs = align >= 2;
  if (dtype == FQA_DTYPE_BF16) return launch_mx_format<__nv_bfloat16, kNorm>(p, fmt, vec, pairs, s);
  if (dtype == FQA_DTYPE_F16) return launch_mx_format<__half, kNorm>(p, fmt, vec, pairs, s);
  return launch_mx_format<float, kNorm>(p, fmt, vec, pairs, s);
}

template <typename T, int FMT>
static fqa_status launch_mx_dequantize(const MxDequantParams& p, bool vec, cudaStream_t s) {
  const bool four = !vec && sizeof(T) == 2 && p.K % 4 == 0 && aligned(p.out, 8);
  const int width = vec ? kMxChunk : four ? 4 : 2, items = (p.K + width - 1) / width;
  int tx = 4;                            // items side by side: a power of two, up to a whole CTA
  while (tx < items && tx < 256) tx *= 2;
  // off the 16-byte boundaries a thread has four items in flight: where the rows
  // fill the SMs (8 CTAs each) more than once, narrow ones take only the threads
  // that keep them busy (from mxfp8 to BF16, 5000 x 333 5.6 -> 3.0 us, 40000 x 333
  // 42 -> 18 us; 1200 x 333 alone on its CTAs 1.9 us, so 2.3)
  if (!vec && p.M > 2048)
    while (tx > 64 && 2 * tx >= items) tx /= 2;
  const dim3 block(tx, 256 / tx), grid((p.M + block.y - 1) / block.y);
  if (vec) return launch_overlapped(mx_dequantize_kernel<T, FMT>, grid, block, 0, s, 1, p);
  if constexpr (sizeof(T) == 2)
    if (four) return launch_overlapped(mx_dequantize_any_kernel<T, FMT, 4>, grid, block, 0, s, 1, p);
  return launch_overlapped(mx_dequantize_any_kernel<T, FMT, 2>, grid, block, 0, s, 1, p);
}

template <typename T>
static fqa_status launch_mx_dequantize_format(const MxDequantParams& p, int fmt, bool vec, cudaStream_t s) {
  if (fmt == FQA_MXFP8) return launch_mx_dequantize<T, kMxFp8>(p, vec, s);
  if (fmt == FQA_MXFP4) return launch_mx_dequantize<T, kMxFp4>(p, vec, s);
  return launch_mx_dequantize<T, kNvFp4>(p, vec, s);
}

template <int FMT, int NT>
static fqa_status launch_mx_small(const uint8_t* a, const uint8_t* b, const MxMatmulParams& p, int row_bytes,
                                  cudaStream_t s) {
  using T = MxSmall<FMT, NT>;
  CUtensorMap tp, tq;
  if (!make_tmap_rows(&tp, b, row_bytes, p.N, 128) || !make_tmap_rows(&tq, a, row_bytes, p.M, NT)) return cuda_failed();
  const int64_t tiles = (int64_t)((p.N + 127) / 128) * ((p.M + NT - 1) / NT);
  // split K while all CTAs are resident at once and each keeps two stages; a
  // cluster of eight wants that many free SMs in one GPC, so only up to three
  // quarters of the places (32 tiles: 5.5 us in fours, 6.7 in eights; 8 tiles:
  // 5.7 and 4.9; 16 tiles with one CTA per SM: 8.2 and 12.0)
  const int stages = (p.mmas + 3) / 4, places = T::kPerSm * num_sms();
  int ranks = 1;
  while (ranks < T::kMaxRanks && tiles * ranks * 2 <= (ranks == 4 ? places * 3 / 4 : places) && stages >= 4 * ranks)
    ranks *= 2;
  if (tiles * ranks > INT32_MAX) return FQA_ERR_UNSUPPORTED;
  const auto fn = mx_matmul_small_kernel<FMT, NT>;
  if (cudaFuncSetAttribute((const void*)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmemBytes) != cudaSuccess)
    return cuda_failed();
  return launch_overlapped(fn, dim3((unsigned)(tiles * ranks)), kMxSmallThreads, T::kSmemBytes, s, ranks, tp, tq, p,
                           ranks);
}

template <int FMT>
static fqa_status launch_mx_large(const uint8_t* a, const uint8_t* b, const MxMatmulParams& p, int row_bytes,
                                  cudaStream_t s) {
  using T = MxLarge<FMT>;
  CUtensorMap ta, tb, tsa, tsb, to{};
  const int64_t tiles = (int64_t)((p.M + 255) / 256) * ((p.N + 255) / 256);
  // rows on 16-byte boundaries leave as TMA stores
  const size_t elt = dtype_bytes(p.out_type);
  const bool tma_out = aligned(p.out, 16) && (size_t)p.N * elt % 16 == 0;
  if (!make_tmap_rows(&ta, a, row_bytes, p.M, 128) || !make_tmap_rows(&tb, b, row_bytes, p.N, 128) ||
      !make_tmap_scales(&tsa, p.sa, p.KT, p.M, MxMma<FMT>::kWords, 1) ||
      !make_tmap_scales(&tsb, p.sb, p.KT, p.N, MxMma<FMT>::kWords, 2) ||
      (tma_out && !make_tmap_out(&to, p.out, p.out_type, p.M, p.N)))
    return cuda_failed();
  const auto fn = mx_matmul_large_kernel<FMT>;
  if (cudaFuncSetAttribute((const void*)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmemBytes) != cudaSuccess)
    return cuda_failed();
  return launch_overlapped(fn, dim3(2 * (unsigned)std::min<int64_t>(tiles, num_sms() / 2)), kMxLargeThreads,
                           T::kSmemBytes, s, 2, ta, tb, tsa, tsb, to, p, (int)tma_out);
}

// The kernel by the product's size: the narrowest tile of tokens that holds
// them all, up to 128 x 128 tiles while one round of SMs holds those; beyond,
// pairs on 256 x 256 tiles.  At K = 4096, N = 4096 (nvfp4): 512 rows, 128
// tiles, 11.4 us against 12.1; 768 rows, 192 tiles, 21.4 against 12.6.
template <int FMT>
static fqa_status launch_mx_matmul(const uint8_t* a, const uint8_t* b, const MxMatmulParams& p, int row_bytes,
                                   cudaStream_t s) {
  if (p.M <= 16) return launch_mx_small<FMT, 16>(a, b, p, row_bytes, s);
  if (p.M <= 32) return launch_mx_small<FMT, 32>(a, b, p, row_bytes, s);
  if (p.M <= 64) return launch_mx_small<FMT, 64>(a, b, p, row_bytes, s);
  const int64_t tiles = (int64_t)((p.M + 127) / 128) * ((p.N + 127) / 128);
  if (tiles <= num_sms()) return launch_mx_small<FMT, 128>(a, b, p, row_bytes, s);
  return launch_mx_large<FMT>(a, b, p, row_bytes, s);
}

template <typename T>
static fqa_status launch_rotary(const RotaryParams& p, bool split, bool norm, dim3 grid, cudaStream_t s) {
  using Fn = void (*)(const RotaryParams);
  const bool all = p.pairs == kHeadDim / 2;
  const Fn fns[2][2][2] = {{{rotary_kernel<T, false, false, false>, rotary_kernel<T, false, false, true>},
                            {rotary_kernel<T, false, true, false>, rotary_kernel<T, false, true, true>}},
                           {{rotary_kernel<T, true, false, false>, rotary_kernel<T, true, false, true>},
                            {rotary_kernel<T, true, true, false>, rotary_kernel<T, true, true, true>}}};
  return launch_overlapped(fns[split][norm][all], grid, 256, 0, s, 1, p);
}

}  // namespace fqa

using namespace fqa;

extern "C" {

int fqa_version(void) { return (1 << 16) | 0; }

const char* fqa_status_string(fqa_status s) {
  switch (s) {
    case FQA_OK: return "FQA_OK";
    case FQA_ERR_INVALID_ARG: return "FQA_ERR_INVALID_ARG";
    case FQA_ERR_UNSUPPORTED: return "FQA_ERR_UNSUPPORTED";
    case FQA_ERR_MISALIGNED: return "FQA_ERR_MISALIGNED";
    case FQA_ERR_CUDA: return "FQA_ERR_CUDA";
    case FQA_ERR_TIMEOUT: return "FQA_ERR_TIMEOUT";
  }
  return "FQA_UNKNOWN_STATUS";
}

// Workspace: the K-mean partial sums [B,H,ceil(N/64),128] FP32, then
// (256-byte aligned) the grid-barrier and work-queue counters of the fused
// quantize launch.
static size_t partial_bytes(int B, int H, int N, int d) {
  return (size_t)B * H * ((N + kQBlock - 1) / kQBlock) * d * sizeof(float);
}

size_t fqa_quantize_workspace_bytes(int B, int H, int N, int d) {
  if (check_shape(B, H, N, d) != FQA_OK) return 0;
  return ((partial_bytes(B, H, N, d) + 255) & ~size_t(255)) + 256;
}

static fqa_status quantize_impl(const void* q, const void* k, const void* v, int B, int H, int N, int d,
                                void* q8, void* k8, void* v8, float* sq, float* sk, float* sv,
                                float* sv_max, float* k_mean, float* k_err, void* workspace,
                                size_t workspace_bytes, void* cuda_stream, int in_P = 1) {
  fqa_status st = check_shape(B, H, N, d);
  if (st != FQA_OK) return st;
  const void* ptrs[] = {q, k, v, q8, k8, v8, sq, sk, sv, sv_max, k_mean, workspace};
  for (const void* p : ptrs)
    if (p == nullptr) return FQA_ERR_INVALID_ARG;
  if (workspace_bytes < fqa_quantize_workspace_bytes(B, H, N, d)) return FQA_ERR_INVALID_ARG;
  const void* a16[] = {q, k, v, q8, k8, v8, k_mean, workspace};   // k_mean: read by bulk copies
  for (const void* p : a16)
    if (!aligned(p, 16)) return FQA_ERR_MISALIGNED;
  const void* a4[] = {sq, sk, sv, sv_max, k_err};
  for (const void* p : a4)
    if (!aligned(p, 4)) return FQA_ERR_MISALIGNED;
  uint32_t* status = status_ptr(&st);
  if (!status) return st;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  float* partial = static_cast<float*>(workspace);
  unsigned int* ctr = reinterpret_cast<unsigned int*>(static_cast<uint8_t*>(workspace) +
                                                      ((partial_bytes(B, H, N, d) + 255) & ~size_t(255)));
  const int nunits = B * H * ((N + kQBlock - 1) / kQBlock);
  if (cudaFuncSetAttribute(quantize_fused_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kQuantSmem) != cudaSuccess)
    return cuda_failed();
  int per_sm = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, quantize_fused_kernel, kQuantThreads,
                                                    kQuantSmem) != cudaSuccess ||
      per_sm < 1)
    return cuda_failed();
  int grid = per_sm * num_sms();
  if (grid > nunits) grid = nunits;
  static_assert(kNumCtr * sizeof(unsigned int) <= 256, "counters fit the reserved 256 bytes");
  if (cudaMemsetAsync(ctr, 0, kNumCtr * sizeof(unsigned int), s) != cudaSuccess) return cuda_failed();
  const __nv_bfloat16* qb = static_cast<const __nv_bfloat16*>(q);
  const __nv_bfloat16* kb = static_cast<const __nv_bfloat16*>(k);
  const __nv_bfloat16* vb = static_cast<const __nv_bfloat16*>(v);
  uint8_t* q8b = static_cast<uint8_t*>(q8);
  uint8_t* k8b = static_cast<uint8_t*>(k8);
  uint8_t* v8b = static_cast<uint8_t*>(v8);
  void* args[] = {(void*)&qb, (void*)&kb, (void*)&vb, (void*)&q8b, (void*)&k8b, (void*)&v8b,
                  (void*)&sq, (void*)&sk, (void*)&sv, (void*)&sv_max, (void*)&k_mean,
                  (void*)&partial, (void*)&ctr, (void*)&B, (void*)&H, (void*)&N, (void*)&status,
                  (void*)&k_err, (void*)&in_P};
  // cooperative: every CTA is resident, so the grid barriers cannot wait on
  // a CTA that never starts
  if (cudaLaunchCooperativeKernel((const void*)quantize_fused_kernel, dim3(grid), dim3(kQuantThreads),
                                  args, kQuantSmem, s) != cudaSuccess)
    return cuda_failed();
  return launch_status();
}

fqa_status fqa_quantize(const void* q, const void* k, const void* v, int B, int H, int N, int d,
                        void* q8, void* k8, void* v8, float* sq, float* sk, float* sv,
                        float* sv_max, float* k_mean, void* workspace, size_t workspace_bytes,
                        void* cuda_stream) {
  return quantize_impl(q, k, v, B, H, N, d, q8, k8, v8, sq, sk, sv, sv_max, k_mean, nullptr, workspace,
                       workspace_bytes, cuda_stream);
}

fqa_status fqa_quantize_keyerr(const void* q, const void* k, const void* v, int B, int H, int N, int d,
                               void* q8, void* k8, void* v8, float* sq, float* sk, float* sv,
                               float* sv_max, float* k_mean, float* k_err, void* workspace,
                               size_t workspace_bytes, void* cuda_stream) {
  if (k_err == nullptr) return FQA_ERR_INVALID_ARG;
  return quantize_impl(q, k, v, B, H, N, d, q8, k8, v8, sq, sk, sv, sv_max, k_mean, k_err, workspace,
                       workspace_bytes, cuda_stream);
}

static fqa_status check_attention_common(int B, int H, int N, int d, float softmax_scale,
                                         void* out, fqa_out_dtype out_dtype) {
  fqa_status st = check_shape(B, H, N, d);
  if (st != FQA_OK) return st;
  if (!(std::isfinite(softmax_scale) && softmax_scale > 0.0f)) return FQA_ERR_INVALID_ARG;
  if (out == nullptr) return FQA_ERR_INVALID_ARG;
  if (out_dtype != FQA_OUT_BF16 && out_dtype != FQA_OUT_F32) return FQA_ERR_INVALID_ARG;
  if (!aligned(out, 16)) return FQA_ERR_MISALIGNED;
  return FQA_OK;
}

fqa_status fqa_attention_fp8(const void* q8, const void* k8, const void* v8, const float* sq,
                             const float* sk, const float* sv, const float* sv_max, int B, int H,
                             int N, int d, float softmax_scale, void* out,
                             fqa_out_dtype out_dtype, void* cuda_stream) {
  fqa_status st = check_attention_common(B, H, N, d, softmax_scale, out, out_dtype);
  if (st != FQA_OK) return st;
  const void* ptrs[] = {q8, k8, v8, sq, sk, sv, sv_max};
  for (const void* p : ptrs)
    if (p == nullptr) return FQA_ERR_INVALID_ARG;
  const void* a16[] = {q8, k8, v8};
  for (const void* p : a16)
    if (!aligned(p, 16)) return FQA_ERR_MISALIGNED;
  const void* a4[] = {sq, sk, sv, sv_max};
  for (const void* p : a4)
    if (!aligned(p, 4)) return FQA_ERR_MISALIGNED;
  uint32_t* status = status_ptr(&st);
  if (!status) return st;
  AttnParams prm{B, H, N, softmax_scale, sq, sk, sv, sv_max, out, out_dtype == FQA_OUT_F32, status};
  prm.q8 = static_cast<const uint8_t*>(q8);
  prm.k8 = static_cast<const uint8_t*>(k8);
  prm.kmask = nullptr;
  prm.row_stats = nullptr;
  return launch_attention_fp8(q8, k8, v8, prm, static_cast<cudaStream_t>(cuda_stream));
}

fqa_status fqa_attention_bf16(const void* q, const void* k, const void* v, int B, int H, int N,
                              int d, float softmax_scale, void* out, fqa_out_dtype out_dtype,
                              void* cuda_stream) {
  fqa_status st = check_attention_common(B, H, N, d, softmax_scale, out, out_dtype);
  if (st != FQA_OK) return st;
  const void* ptrs[] = {q, k, v};
  for (const void* p : ptrs) {
    if (p == nullptr) return FQA_ERR_INVALID_ARG;
    if (!aligned(p, 16)) return FQA_ERR_MISALIGNED;
  }
  uint32_t* status = status_ptr(&st);
  if (!status) return st;
  AttnParams prm{B, H, N, softmax_scale, nullptr, nullptr, nullptr, nullptr, out,
                 out_dtype == FQA_OUT_F32, status};
  return launch_attention_bf16(q, k, v, prm, static_cast<cudaStream_t>(cuda_stream));
}

// ------------------------------------------- sequence all-to-all layouts

// Shapes of the all-to-all calls: B, Hl heads, P chunks of Nl tokens
// (N = P * Nl), Nl a multiple of 64 so that no quantization block straddles
// two chunks.
static fqa_status check_a2a(int B, int Hl, int P, int Nl, int d) {
  if (P < 1 || Nl < 1) return FQA_ERR_INVALID_ARG;
  if (Nl % kQBlock != 0) return FQA_ERR_UNSUPPORTED;
  if ((int64_t)P * Nl > 65536) return FQA_ERR_UNSUPPORTED;
  return check_shape(B, Hl, P * Nl, d);
}

fqa_status fqa_quantize_a2a(const void* q, const void* k, const void* v, int B, int Hl, int P, int Nl, int d,
                            void* q8, void* k8, void* v8, float* sq, float* sk, float* sv, float* sv_max,
                            float* k_mean, void* workspace, size_t workspace_bytes, void* cuda_stream) {
  fqa_status st = check_a2a(B, Hl, P, Nl, d);
  if (st != FQA_OK) return st;
  return quantize_impl(q, k, v, B, Hl, P * Nl, d, q8, k8, v8, sq, sk, sv, sv_max, k_mean, nullptr, workspace,
                       workspace_bytes, cuda_stream, P);
}

fqa_status fqa_attention_fp8_a2a(const void* q8, const void* k8, const void* v8, const float* sq,
                                 const float* sk, const float* sv, const float* sv_max, int B, int Hl, int P,
                                 int Nl, int d, float softmax_scale, void* out, fqa_out_dtype out_dtype,
                                 void* cuda_stream) {
  fqa_status st = check_a2a(B, Hl, P, Nl, d);
  if (st != FQA_OK) return st;
  const int N = P * Nl;
  if ((st = check_attention_common(B, Hl, N, d, softmax_scale, out, out_dtype)) != FQA_OK) return st;
  const void* ptrs[] = {q8, k8, v8, sq, sk, sv, sv_max};
  for (const void* p : ptrs)
    if (p == nullptr) return FQA_ERR_INVALID_ARG;
  const void* a16[] = {q8, k8, v8};
  for (const void* p : a16)
    if (!aligned(p, 16)) return FQA_ERR_MISALIGNED;
  const void* a4[] = {sq, sk, sv, sv_max};
  for (const void* p : a4)
    if (!aligned(p, 4)) return FQA_ERR_MISALIGNED;
  uint32_t* status = status_ptr(&st);
  if (!status) return st;
  AttnParams prm{B, Hl, N, softmax_scale, sq, sk, sv, sv_max, out, out_dtype == FQA_OUT_F32, status};
  prm.q8 = static_cast<const uint8_t*>(q8);
  prm.k8 = static_cast<const uint8_t*>(k8);
  prm.out_P = P;
  return launch_attention_fp8(q8, k8, v8, prm, static_cast<cudaStream_t>(cuda_stream));
}

// ---------------------------------------------------- error-corrected path

// ceil(rho * N - 0.01): rho arrives in binary32, whose rounding moves rho * N
// by at most 0.004 for N <= 65536, so a product meant to be an integer (0.05
// of 1280 keys) stays that integer instead of rounding up.
int fqa_corrected_keys(int N, float rho) {
  if (N < 1 || !(rho >= 0.0f) || !(rho <= 1.0f)) return -1;
  const double kc = std::ceil((double)rho * (double)N - 0.01);
  return kc < 0.0 ? 0 : (kc > (double)N ? N : (int)kc);
}

static size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

fqa_status fqa_select_keys(const float* k_err, int B, int H, int N, int kc, uint32_t* kmask, int* idx,
                           void* cuda_stream) {
  fqa_status st = check_shape(B, H, N, 128);
  if (st != FQA_OK) return st;
  if (k_err == nullptr || kmask == nullptr || kc < 1 || kc > N || (idx == nullptr)) return FQA_ERR_INVALID_ARG;
  const void* a4[] = {k_err, kmask, idx};
  for (const void* p : a4)
    if (!aligned(p, 4)) return FQA_ERR_MISALIGNED;
  if (!status_ptr(&st)) return st;
  const int staged = N <= kSelStageMax ? 1 : 0;
  const int smem = staged ? N * 4 : 0;
  if (staged && cudaFuncSetAttribute(select_keys_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kSelStageMax * 4) != cudaSuccess)
    return cuda_failed();
  select_keys_kernel<<<B * H, kSelThreads, smem, static_cast<cudaStream_t>(cuda_stream)>>>(k_err, N, kc, kmask,
                                                                                         idx, staged);
  return launch_status();
}

size_t fqa_attention_fp8_corrected_workspace_bytes(int B, int H, int N, int d, float rho) {
  if (check_shape(B, H, N, d) != FQA_OK) return 0;
  const int kc = fqa_corrected_keys(N, rho);
  if (kc < 0) return 0;
  const size_t rows = (size_t)B * H * N;
  return align256((size_t)B * H * ((N + 31) / 32) * 4)      // key mask
         + align256((size_t)B * H * (size_t)(kc > 0 ? kc : 1) * 4)   // corrected indices
         + align256(rows * 8)                                // (m, l) per row
         + align256(rows * 128 * 4);                         // FP8 part, FP32
}

fqa_status fqa_attention_fp8_corrected(const void* q, const void* k, const void* v, const void* q8,
                                       const void* k8, const void* v8, const float* sq, const float* sk,
                                       const float* sv, const float* sv_max, const float* k_mean,
                                       const float* k_err, int B, int H, int N, int d, float softmax_scale,
                                       float rho, void* out, fqa_out_dtype out_dtype, void* workspace,
                                       size_t workspace_bytes, void* cuda_stream) {
  fqa_status st = check_attention_common(B, H, N, d, softmax_scale, out, out_dtype);
  if (st != FQA_OK) return st;
  const int kc = fqa_corrected_keys(N, rho);
  if (kc < 0) return FQA_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, v, q8, k8, v8, sq, sk, sv, sv_max, k_mean, k_err, workspace};
  for (const void* p : ptrs)
    if (p == nullptr) return FQA_ERR_INVALID_ARG;
  if (workspace_bytes < fqa_attention_fp8_corrected_workspace_bytes(B, H, N, d, rho))
    return FQA_ERR_INVALID_ARG;
  const void* a16[] = {q, k, v, q8, k8, v8, workspace};
  for (const void* p : a16)
    if (!aligned(p, 16)) return FQA_ERR_MISALIGNED;
  const void* a4[] = {sq, sk, sv, sv_max, k_mean, k_err};
  for (const void* p : a4)
    if (!aligned(p, 4)) return FQA_ERR_MISALIGNED;
  uint32_t* status = status_ptr(&st);
  if (!status) return st;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (kc == 0)   // nothing to correct: the plain FP8 path
    return fqa_attention_fp8(q8, k8, v8, sq, sk, sv, sv_max, B, H, N, d, softmax_scale, out, out_dtype,
                             cuda_stream);
  // workspace: key mask | corrected indices | (m, l) | FP8 part (FP32)
  uint8_t* w = static_cast<uint8_t*>(workspace);
  uint32_t* kmask = reinterpret_cast<uint32_t*>(w);
  w += align256((size_t)B * H * ((N + 31) / 32) * 4);
  int* idx = reinterpret_cast<int*>(w);
  w += align256((size_t)B * H * (size_t)kc * 4);
  float2* stats = reinterpret_cast<float2*>(w);
  w += align256((size_t)B * H * N * 8);
  float* o1 = reinterpret_cast<float*>(w);
  if ((st = fqa_select_keys(k_err, B, H, N, kc, kmask, idx, cuda_stream)) != FQA_OK) return st;
  AttnParams prm{B, H, N, softmax_scale, sq, sk, sv, sv_max, o1, 1, status};
  prm.q8 = static_cast<const uint8_t*>(q8);
  prm.k8 = static_cast<const uint8_t*>(k8);
  prm.kmask = kmask;
  prm.row_stats = stats;
  // fewer than 64 corrected keys per head leave a kept key in every 64-key
  // block: the key mask can be applied by patching tiles
  prm.patch = (kc < 64 && N % kBlockN == 0) ? 1 : 0;
  if ((st = launch_attention_fp8(q8, k8, v8, prm, s)) != FQA_OK) return st;
  if (prm.patch) {
    // take the copied keys' terms out of the patched FP8 part's row sums
    CUtensorMap tq8;
    if (!make_tmap(&tq8, q8, true, N, B * H)) return cuda_failed();
    if (cudaFuncSetAttribute(dup_sum_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kDupSmem) !=
        cudaSuccess)
      return cuda_failed();
    DupParams dp{static_cast<const uint8_t*>(k8), sq, sk, kmask, stats, N, softmax_scale, status};
    dup_sum_kernel<<<dim3(N / kBlockM, B * H), kDupThreads, kDupSmem, s>>>(tq8, dp);
    if ((st = launch_status()) != FQA_OK) return st;
  }
  // exact part over the corrected keys, merged into the output: one chunk of
  // 64 (two CTAs per SM; three of its rows carry the K mean) when they fit
  CUtensorMap tq;
  if (!make_tmap(&tq, q, false, N, B * H)) return cuda_failed();
  CorrParams cp{static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k),
                static_cast<const __nv_bfloat16*>(v), k_mean, idx, o1, stats, prm.patch, out,
                out_dtype == FQA_OUT_F32, B, H, N, kc, softmax_scale, status};
  const bool small = kc <= 61;
  const void* fn = small ? (const void*)correct_kernel<64> : (const void*)correct_kernel<128>;
  const int smem = small ? CorrTraits<64>::kSmemBytes : CorrTraits<128>::kSmemBytes;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return cuda_failed();
  const int sms = num_sms() * (small ? CorrTraits<64>::kCtasPerSm : CorrTraits<128>::kCtasPerSm);
  const int ntq = (N + 127) / 128;
  int split = (sms + B * H - 1) / (B * H);       // about one wave of CTAs
  if (split > ntq) split = ntq;
  if (split < 1) split = 1;
  if (small)
    correct_kernel<64><<<dim3(split, B * H), kCorrThreads, smem, s>>>(tq, cp);
  else
    correct_kernel<128><<<dim3(split, B * H), kCorrThreads, smem, s>>>(tq, cp);
  return launch_status();
}

// ------------------------------------------------------- NVFP4 Q.K variant

fqa_status fqa_quantize_nvfp4_qk(const void* q, const void* k, const float* k_mean, int B, int H, int N, int d,
                                 uint8_t* q4, uint8_t* k4, uint8_t* sfq, uint8_t* sfk, float* sq1, float* sk1,
                                 void* cuda_stream) {
  fqa_status st = check_shape(B, H, N, d);
  if (st != FQA_OK) return st;
  const void* ptrs[] = {q, k, k_mean, q4, k4, sfq, sfk, sq1, sk1};
  for (const void* p : ptrs)
    if (p == nullptr) return FQA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16)) return FQA_ERR_MISALIGNED;
  const void* a4[] = {k_mean, q4, k4, sq1, sk1};
  for (const void* p : a4)
    if (!aligned(p, 4)) return FQA_ERR_MISALIGNED;
  const int units = B * H * ((N + 63) / 64);
  quantize_nvfp4_kernel<<<2 * units, kNv4Threads, 0, static_cast<cudaStream_t>(cuda_stream)>>>(
      static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k), k_mean, q4, k4, sfq, sfk,
      sq1, sk1, B, H, N);
  return launch_status();
}

fqa_status fqa_attention_nvfp4(const uint8_t* q4, const uint8_t* k4, const uint8_t* sfq, const uint8_t* sfk,
                               const float* sq1, const float* sk1, const void* v8, const float* sv,
                               const float* sv_max, int B, int H, int N, int d, float softmax_scale, void* out,
                               fqa_out_dtype out_dtype, void* cuda_stream) {
  fqa_status st = check_attention_common(B, H, N, d, softmax_scale, out, out_dtype);
  if (st != FQA_OK) return st;
  const void* ptrs[] = {q4, k4, sfq, sfk, sq1, sk1, v8, sv, sv_max};
  for (const void* p : ptrs)
    if (p == nullptr) return FQA_ERR_INVALID_ARG;
  const void* a16[] = {q4, k4, v8};
  for (const void* p : a16)
    if (!aligned(p, 16)) return FQA_ERR_MISALIGNED;
  if (!aligned(sfq, 8) || !aligned(sfk, 8)) return FQA_ERR_MISALIGNED;
  const void* a4[] = {sq1, sk1, sv, sv_max};
  for (const void* p : a4)
    if (!aligned(p, 4)) return FQA_ERR_MISALIGNED;
  uint32_t* status = status_ptr(&st);
  if (!status) return st;
  const int heads = B * H;
  CUtensorMap tq, tk, tv;
  if (!make_tmap_fp4(&tq, q4, N, heads) || !make_tmap_fp4(&tk, k4, N, heads) ||
      !make_tmap(&tv, v8, true, N, heads))
    return cuda_failed();
  // the short-tail instance only when N is not a multiple of 128
  const bool tail = N % kBlockN != 0;
  using NvKernel = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const NvParams);
  const NvKernel fn = tail ? attn_nvfp4_kernel<true> : attn_nvfp4_kernel<false>;
  if (cudaFuncSetAttribute((const void*)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, NvTraits::kSmemBytes) !=
      cudaSuccess)
    return cuda_failed();
  NvParams prm{B, H, N, softmax_scale, sfq, sfk, sq1, sk1, sv, sv_max, out, out_dtype == FQA_OUT_F32, status};
  const int items = heads * ((N + kBlockM - 1) / kBlockM);
  const int sms = num_sms();
  if (sms <= 0) return cuda_failed();
  const int grid = items < sms ? items : sms;
  fn<<<grid, kNvThreads, NvTraits::kSmemBytes, static_cast<cudaStream_t>(cuda_stream)>>>(tq, tk, tv, prm);
  return launch_status();
}

// ------------------------------------------------- microscaled rows

static bool mx_shape_ok(int64_t rows, int K) { return rows >= 0 && rows <= kMxMaxRows && K >= 1 && K <= kMxMaxCols; }
static bool mx_format_ok(int fmt) { return fmt == FQA_MXFP8 || fmt == FQA_MXFP4 || fmt == FQA_NVFP4; }
static bool dtype_ok(int t) { return t == FQA_DTYPE_BF16 || t == FQA_DTYPE_F32 || t == FQA_DTYPE_F16; }
static int mx_padded(int K) { return (K + 31) / 32 * 32; }
static int mx_words(int K, int fmt) { return (mx_padded(K) + 4 * mx_block(fmt) - 1) / (4 * mx_block(fmt)); }

size_t fqa_mx_code_bytes(int M, int K, fqa_mx_format fmt) {
  if (!mx_format_ok(fmt) || !mx_shape_ok(M, K)) return 0;
  return (size_t)M * (mx_padded(K) / mx_per_byte(fmt));
}

size_t fqa_mx_scale_bytes(int M, int K, fqa_mx_format fmt) {
  if (!mx_format_ok(fmt) || !mx_shape_ok(M, K)) return 0;
  return (size_t)((M + 127) / 128) * mx_words(K, fmt) * 512;
}

// The widest access that every row's start and length are multiples of: 32 or
// 16 bytes, or two elements (2), or one (1).
static int rows_vectorize(const void* base, int64_t ld, int K, size_t elt) {
  for (size_t w : {(size_t)32, (size_t)16, 2 * elt})
    if (K * elt % w == 0 && aligned(base, w) && (ld * (int64_t)elt) % (int64_t)w == 0) return w == 2 * elt ? 2 : (int)w;
  return 1;
}

// The checks and fields common to both row calls.
static fqa_status mx_row_params(MxRowParams* p, const void* x, int dtype, int M, int K, int64_t ldx, int fmt,
                                uint8_t* codes, uint8_t* scales, float* row_scale) {
  if (!dtype_ok(dtype) || !mx_format_ok(fmt) || M < 0 || K < 1) return FQA_ERR_INVALID_ARG;
  if (!mx_shape_ok(M, K)) return FQA_ERR_UNSUPPORTED;
  if (M == 0) return FQA_OK;
  if (x == nullptr || codes == nullptr || scales == nullptr || ldx < 0) return FQA_ERR_INVALID_ARG;
  if (fmt == FQA_NVFP4 && row_scale == nullptr) return FQA_ERR_INVALID_ARG;
  const size_t elt = dtype_bytes(dtype);
  if (!aligned(x, elt) || !aligned(codes, 16) || !aligned(scales, 16) || !aligned(row_scale, 4))
    return FQA_ERR_MISALIGNED;
  *p = MxRowParams{};
  p->x = x;
  p->ldx = ldx;
  p->M = M;
  p->K = K;
  p->Kp = mx_padded(K);
  p->KT = mx_words(K, fmt);
  p->codes = codes;
  p->scales = reinterpret_cast<uint32_t*>(scales);
  p->row_scale = row_scale;
  return FQA_OK;
}

fqa_status fqa_mx_quantize(const void* x, fqa_dtype dtype, int M, int K, int64_t ldx, fqa_mx_format fmt,
                           uint8_t* codes, uint8_t* scales, float* row_scale, void* cuda_stream) {
  MxRowParams p;
  const fqa_status st = mx_row_params(&p, x, dtype, M, K, ldx, fmt, codes, scales, row_scale);
  if (st != FQA_OK || M == 0) return st;
  const int vec = rows_vectorize(x, ldx, K, dtype_bytes(dtype));
  p.wide = vec == 32;
  return launch_mx<false>(p, dtype, fmt, vec, static_cast<cudaStream_t>(cuda_stream));
}

fqa_status fqa_mx_rms_norm(const void* x, fqa_dtype dtype, int M, int K, int64_t ldx, const void* weight,
                           fqa_dtype weight_dtype, float eps, const void* residual, fqa_dtype residual_dtype,
                           int64_t ldr, fqa_mx_format fmt, uint8_t* codes, uint8_t* scales, float* row_scale,
                           void* residual_out, void* cuda_stream) {
  MxRowParams p;
  const fqa_status st = mx_row_params(&p, x, dtype, M, K, ldx, fmt, codes, scales, row_scale);
  if (st != FQA_OK) return st;
  if (!(std::isfinite(eps) && eps >= 0.0f)) return FQA_ERR_INVALID_ARG;
  if (weight_dtype != dtype && weight_dtype != FQA_DTYPE_F32) return FQA_ERR_INVALID_ARG;
  const bool res = residual != nullptr;
  if (res && residual_dtype != dtype && residual_dtype != FQA_DTYPE_F32) return FQA_ERR_INVALID_ARG;
  if (M == 0) return FQA_OK;
  if (weight == nullptr || res != (residual_out != nullptr) || (res && ldr < 0)) return FQA_ERR_INVALID_ARG;
  const size_t welt = dtype_bytes(weight_dtype), relt = dtype_bytes(residual_dtype);
  if (!aligned(weight, welt) || (res && (!aligned(residual, relt) || !aligned(residual_out, relt))))
    return FQA_ERR_MISALIGNED;
  p.weight = weight;
  p.w_f32 = weight_dtype != dtype;
  int vec = std::min(rows_vectorize(x, ldx, K, dtype_bytes(dtype)), rows_vectorize(weight, 0, K, welt));
  p.eps = eps;
  p.residual = residual;
  p.residual_out = residual_out;
  if (res) {
    p.ldr = ldr;
    p.res_f32 = residual_dtype != dtype;
    vec = std::min({vec, rows_vectorize(residual, ldr, K, relt), rows_vectorize(residual_out, K, K, relt)});
  }
  p.wide = vec == 32;
  return launch_mx<true>(p, dtype, fmt, vec, static_cast<cudaStream_t>(cuda_stream));
}

fqa_status fqa_mx_dequantize(const uint8_t* codes, const uint8_t* scales, const float* row_scale, int M, int K,
                             fqa_mx_format fmt, void* out, fqa_dtype out_dtype, void* cuda_stream) {
  if (!mx_format_ok(fmt) || !dtype_ok(out_dtype) || M < 0 || K < 1) return FQA_ERR_INVALID_ARG;
  if (!mx_shape_ok(M, K)) return FQA_ERR_UNSUPPORTED;
  if (M == 0) return FQA_OK;
  if (codes == nullptr || scales == nullptr || out == nullptr) return FQA_ERR_INVALID_ARG;
  if (fmt == FQA_NVFP4 && row_scale == nullptr) return FQA_ERR_INVALID_ARG;
  if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(row_scale, 4) || !aligned(out, dtype_bytes(out_dtype)))
    return FQA_ERR_MISALIGNED;
  const int vec = rows_vectorize(out, K, K, dtype_bytes(out_dtype));
  const MxDequantParams p{codes, scales, row_scale, out, M, K, mx_padded(K), mx_words(K, fmt), vec == 32 || vec == 2};
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (out_dtype == FQA_DTYPE_BF16) return launch_mx_dequantize_format<__nv_bfloat16>(p, fmt, vec >= 16, s);
  if (out_dtype == FQA_DTYPE_F16) return launch_mx_dequantize_format<__half>(p, fmt, vec >= 16, s);
  return launch_mx_dequantize_format<float>(p, fmt, vec >= 16, s);
}

// fqa_mx_matmul(), and its check (stop: see loads_until()).
static fqa_status mx_matmul_checked(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_row_scale,
                                    const uint8_t* b_codes, const uint8_t* b_scales, const float* b_row_scale,
                                    const float* bias, int M, int N, int K, int fmt, void* out, int out_dtype,
                                    void* cuda_stream, uint32_t stop) {
  if (!mx_format_ok(fmt) || !dtype_ok(out_dtype) || M < 0 || N < 0 || K < 1) return FQA_ERR_INVALID_ARG;
  if (!mx_shape_ok(M, K) || !mx_shape_ok(N, K)) return FQA_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return FQA_OK;
  const void* ptrs[] = {a_codes, a_scales, b_codes, b_scales, out};
  for (const void* q : ptrs)
    if (q == nullptr) return FQA_ERR_INVALID_ARG;
  if (fmt == FQA_NVFP4 && (a_row_scale == nullptr || b_row_scale == nullptr)) return FQA_ERR_INVALID_ARG;
  const void* a16[] = {a_codes, a_scales, b_codes, b_scales};
  for (const void* q : a16)
    if (!aligned(q, 16)) return FQA_ERR_MISALIGNED;
  const void* a4[] = {a_row_scale, b_row_scale, bias};
  for (const void* q : a4)
    if (!aligned(q, 4)) return FQA_ERR_MISALIGNED;
  if (!aligned(out, dtype_bytes(out_dtype))) return FQA_ERR_MISALIGNED;
  fqa_status st = FQA_OK;
  uint32_t* status = status_ptr(&st);
  if (!status) return st;
  const int row_bytes = mx_padded(K) / mx_per_byte(fmt);
  const bool nv = fmt == FQA_NVFP4;
  const MxMatmulParams p{a_scales, b_scales, nv ? a_row_scale : nullptr, nv ? b_row_scale : nullptr, bias, out, M, N,
                         (row_bytes + 31) / 32, mx_words(K, fmt), out_dtype, stop, status};
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (fmt == FQA_MXFP8) return launch_mx_matmul<kMxFp8>(a_codes, b_codes, p, row_bytes, s);
  if (fmt == FQA_MXFP4) return launch_mx_matmul<kMxFp4>(a_codes, b_codes, p, row_bytes, s);
  return launch_mx_matmul<kNvFp4>(a_codes, b_codes, p, row_bytes, s);
}

fqa_status fqa_mx_matmul(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_row_scale,
                         const uint8_t* b_codes, const uint8_t* b_scales, const float* b_row_scale,
                         const float* bias, int M, int N, int K, fqa_mx_format fmt, void* out, fqa_dtype out_dtype,
                         void* cuda_stream) {
  return mx_matmul_checked(a_codes, a_scales, a_row_scale, b_codes, b_scales, b_row_scale, bias, M, N, K, fmt, out,
                           out_dtype, cuda_stream, kMxNoStop);
}

// ------------------------------------------------------------- rotary

fqa_status fqa_rotary(const void* q, const void* k, fqa_dtype dtype, int B, int Hq, int Hk, int N, int d,
                      int64_t q_sb, int64_t q_sh, int64_t q_sn, int64_t k_sb, int64_t k_sh, int64_t k_sn,
                      const void* positions, fqa_dtype positions_dtype, int64_t positions_sb, int n_axes,
                      const int* axes, double theta, int flags, const void* q_weight, const void* k_weight, float eps,
                      void* q_out, void* k_out, void* cuda_stream) {
  if (!dtype_ok(dtype) || B < 0 || N < 0 || Hq < 0 || Hk < 0) return FQA_ERR_INVALID_ARG;
  if (d != kHeadDim) return FQA_ERR_UNSUPPORTED;
  if (positions_dtype != FQA_DTYPE_I32 && positions_dtype != FQA_DTYPE_F32) return FQA_ERR_INVALID_ARG;
  if (n_axes < 1 || axes == nullptr || (flags & ~(FQA_ROTARY_SPLIT | FQA_ROTARY_SHARED | FQA_ROTARY_INVERSE)) != 0)
    return FQA_ERR_INVALID_ARG;
  if (n_axes > kRotMaxAxes) return FQA_ERR_UNSUPPORTED;
  if (!(std::isfinite(theta) && theta > 0.0) || !(std::isfinite(eps) && eps >= 0.0f)) return FQA_ERR_INVALID_ARG;
  int width = 0;
  for (int a = 0; a < n_axes; ++a) {
    if (axes[a] < 2 || axes[a] % 2 != 0 || axes[a] > kHeadDim) return FQA_ERR_INVALID_ARG;
    width += axes[a];
  }
  const bool split = flags & FQA_ROTARY_SPLIT;
  if (width > kHeadDim) return FQA_ERR_INVALID_ARG;
  if (split && width % 16 != 0) return FQA_ERR_UNSUPPORTED;
  if ((int64_t)B * N >= (int64_t(1) << 31) || (int64_t)Hq + Hk > 65535) return FQA_ERR_UNSUPPORTED;
  const int total = Hq + Hk;
  if (B == 0 || N == 0 || total == 0) return FQA_OK;
  if (positions == nullptr || positions_sb < 0) return FQA_ERR_INVALID_ARG;
  if ((Hq > 0 && (q == nullptr || q_out == nullptr)) || (Hk > 0 && (k == nullptr || k_out == nullptr)))
    return FQA_ERR_INVALID_ARG;
  const size_t elt = dtype_bytes(dtype);
  if (!aligned(positions, 4) || !aligned(q_out, 16) || !aligned(k_out, 16)) return FQA_ERR_MISALIGNED;
  const void* ae[] = {q, k, q_weight, k_weight};
  for (const void* ptr : ae)
    if (!aligned(ptr, elt)) return FQA_ERR_MISALIGNED;
  RotaryParams p{};
  const int64_t strides[2][3] = {{q_sb, q_sh, q_sn}, {k_sb, k_sh, k_sn}};
  const void* in[2] = {q, k};
  for (int i = 0; i < 2; ++i) {
    p.in[i] = in[i];
    p.sb[i] = strides[i][0];
    p.sh[i] = strides[i][1];
    p.sn[i] = strides[i][2];
    p.vec[i] = aligned(in[i], 16);
    for (int64_t s : strides[i]) p.vec[i] = p.vec[i] && (s * (int64_t)elt) % 16 == 0;
  }
  p.out[0] = q_out;
  p.out[1] = k_out;
  p.weight[0] = q_weight;
  p.weight[1] = k_weight;
  p.heads[0] = Hq;
  p.heads[1] = Hk;
  p.pos = positions;
  p.pos_sb = positions_sb;
  p.pos_f32 = positions_dtype == FQA_DTYPE_F32;
  p.n_axes = n_axes;
  p.B = B;
  p.N = N;
  p.pairs = width / 2;
  p.eps = eps;
  p.sign = (flags & FQA_ROTARY_INVERSE) ? -1.0f : 1.0f;
  for (int a = 0, j = 0; a < n_axes; ++a)
    for (int i = 0; i < axes[a] / 2; ++i, ++j) {
      const double e = (flags & FQA_ROTARY_SHARED) ? 2.0 * j / width : 2.0 * i / axes[a];
      p.f[j] = std::pow(theta, -e) / 6.283185307179586476925;
      p.axis[j] = (uint8_t)a;
    }
  // groups of 16 lanes per token; with few tokens the heads are shared out
  // to more groups, in batches of four, while all CTAs stay resident (three per
  // SM).  Each group forms its token's angles again, so no further: 4608
  // tokens x 48 heads take 30 us in one group, 48 us in twelve
  fqa_status st = FQA_OK;
  if (!status_ptr(&st)) return st;
  const int64_t blocks = ((int64_t)B * N + 15) / 16;
  int64_t chunks = std::min<int64_t>(total, std::max<int64_t>(1, 3LL * num_sms() / blocks));
  p.heads_per_group = (int)((total + chunks - 1) / chunks + 3) / 4 * 4;
  const dim3 grid((unsigned)blocks, (unsigned)((total + p.heads_per_group - 1) / p.heads_per_group));
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  const bool norm = q_weight != nullptr || k_weight != nullptr;
  if (dtype == FQA_DTYPE_BF16) return launch_rotary<__nv_bfloat16>(p, split, norm, grid, s);
  if (dtype == FQA_DTYPE_F16) return launch_rotary<__half>(p, split, norm, grid, s);
  return launch_rotary<float>(p, split, norm, grid, s);
}

fqa_status fqa_e2m1_encode(const float* x, uint8_t* out, size_t npairs, void* cuda_stream) {
  if (x == nullptr || out == nullptr) return FQA_ERR_INVALID_ARG;
  if (npairs == 0) return FQA_OK;
  if (!aligned(x, 8)) return FQA_ERR_MISALIGNED;
  e2m1_encode_kernel<<<148 * 8, 256, 0, static_cast<cudaStream_t>(cuda_stream)>>>(x, out, npairs);
  return launch_status();
}

fqa_status fqa_exp2_error(float lo, float hi, uint32_t* max_rel_bits, void* cuda_stream) {
  if (max_rel_bits == nullptr) return FQA_ERR_INVALID_ARG;
  if (!(lo <= hi) || !(hi <= 0.0f) || !(lo >= -126.0f)) return FQA_ERR_INVALID_ARG;
  if (!aligned(max_rel_bits, 4)) return FQA_ERR_MISALIGNED;
  // negative binary32 values from hi down to lo are consecutive bit patterns
  uint32_t hb, lb;
  const float h = hi == 0.0f ? -0.0f : hi;
  std::memcpy(&hb, &h, 4);
  std::memcpy(&lb, &lo, 4);
  const uint32_t n = lb - hb + 1;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  if (cudaMemsetAsync(max_rel_bits, 0, 4, s) != cudaSuccess) return cuda_failed();
  exp2_error_kernel<<<148 * 16, 256, 0, s>>>(lb, n, reinterpret_cast<unsigned int*>(max_rel_bits));
  return launch_status();
}

fqa_status fqa_e4m3_encode(const float* x, uint8_t* out, size_t n, void* cuda_stream) {
  if (x == nullptr || out == nullptr) return FQA_ERR_INVALID_ARG;
  if (n == 0) return FQA_OK;
  if (!aligned(x, 4)) return FQA_ERR_MISALIGNED;
  e4m3_encode_kernel<<<148 * 8, 256, 0, static_cast<cudaStream_t>(cuda_stream)>>>(x, out, n);
  return launch_status();
}

fqa_status fqa_debug_wait_timeout(uint32_t limit_us, void* cuda_stream) {
  if (limit_us == 0 || limit_us > 2000000u) return FQA_ERR_INVALID_ARG;
  fqa_status st = FQA_OK;
  uint32_t* status = status_ptr(&st);
  if (!status) return st;
  wait_timeout_kernel<<<1, 1, 0, static_cast<cudaStream_t>(cuda_stream)>>>(
      status, (uint64_t)limit_us * 1000ull);
  return launch_status();
}

fqa_status fqa_debug_mx_matmul_timeout(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_row_scale,
                                       const uint8_t* b_codes, const uint8_t* b_scales, const float* b_row_scale,
                                       const float* bias, int M, int N, int K, fqa_mx_format fmt, void* out,
                                       fqa_dtype out_dtype, int rank, int stage, void* cuda_stream) {
  if (rank < -1 || rank > 7 || stage < 0 || stage > 1 << 24) return FQA_ERR_INVALID_ARG;
  return mx_matmul_checked(a_codes, a_scales, a_row_scale, b_codes, b_scales, b_row_scale, bias, M, N, K, fmt, out,
                           out_dtype, cuda_stream, 16u * (uint32_t)stage + (uint32_t)(rank + 1));
}

fqa_status fqa_debug_status(void* cuda_stream, uint32_t* flags_out) {
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(cuda_stream)) != cudaSuccess)
    return cuda_failed();
  uint32_t v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_status_word, sizeof(v)) != cudaSuccess) return cuda_failed();
  if (cudaMemcpyToSymbol(g_status_word, &zero, sizeof(zero)) != cudaSuccess) return cuda_failed();
  if (flags_out) *flags_out = v;
  return (v & kStatusTimeout) ? FQA_ERR_TIMEOUT : FQA_OK;
}

}  // extern "C"

// ---------------------------------------------------------------------------
// fqa_quantize_noalloc: fqa_quantize for callers that cannot allocate device
// memory when they call.  The K-mean partial sums live in a fixed array inside
// the library instead of a caller-provided workspace.
namespace fqa {

// The scratch fqa_quantize needs is the K-mean partial sums,
// B*H*ceil(N/64)*128*4 bytes rounded up to 256, plus 256 bytes of counters.
// 8 MiB of partial sums covers B*H*ceil(N/64) <= 16384 blocks (B=2, H=24,
// N=16896 needs 6.2 MiB); the array holds that plus the counters.
constexpr size_t kNoAllocScratchBytes = (size_t(8) << 20) + 256;

// One copy per GPU that loads the library, held until the process exits.
// In host code this name is only a stand-in: the device address comes from
// cudaGetSymbolAddress below.
static __device__ __align__(256) float g_noalloc_scratch[kNoAllocScratchBytes / sizeof(float)];

struct NoAllocCache {
  std::mutex mu;
  float* ptr = nullptr;
};
NoAllocCache g_noalloc[kMaxDevices];

// Device address of this device's scratch array, looked up with that device
// current; cached once the lookup succeeds (a failed lookup, e.g. during a
// stream capture, is retried by the next call).
static float* noalloc_scratch(fqa_status* st) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    *st = cuda_failed();
    return nullptr;
  }
  NoAllocCache& c = g_noalloc[dev];
  std::lock_guard<std::mutex> lock(c.mu);
  if (c.ptr == nullptr) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || p == nullptr) {
      *st = cuda_failed();
      return nullptr;
    }
    c.ptr = static_cast<float*>(p);
  }
  return c.ptr;
}

}  // namespace fqa

extern "C" size_t fqa_quantize_noalloc_max_workspace_bytes(void) { return kNoAllocScratchBytes; }

extern "C" fqa_status fqa_quantize_noalloc(const void* q, const void* k, const void* v, int B, int H,
                                           int N, int d, void* q8, void* k8, void* v8, float* sq,
                                           float* sk, float* sv, float* sv_max, float* k_mean,
                                           void* cuda_stream) {
  fqa_status st = check_shape(B, H, N, d);
  if (st != FQA_OK) return st;
  if (fqa_quantize_workspace_bytes(B, H, N, d) > kNoAllocScratchBytes) return FQA_ERR_UNSUPPORTED;
  float* scratch = noalloc_scratch(&st);
  if (scratch == nullptr) return st;
  return fqa_quantize(q, k, v, B, H, N, d, q8, k8, v8, sq, sk, sv, sv_max, k_mean, scratch,
                      kNoAllocScratchBytes, cuda_stream);
}
