// microscale.cuh -- microscaled 8- and 4-bit rows: quantization, the RMS norm
// that quantizes its output, and the way back.
//
// A row of K values is padded with zeros to Kp = 32 ceil(K / 32) and held as
//   mxfp8  E4M3 elements, one E8M0 scale (a power of two) per 32
//   mxfp4  E2M1 elements, one E8M0 scale per 32
//   nvfp4  E2M1 elements, one E4M3 scale per 16, one binary32 scale per row
// Rules (amax over the block, everything round to nearest even, saturating):
//   mx:    2^e the smallest power of two (e >= -127) with amax <= L 2^e,
//          L = 448 (E4M3) or 6 (E2M1): no element saturates;
//          code = RN(x 2^-e), an exact product but for subnormal results
//   nvfp4: the row's 2^e the smallest power of two (e >= -126) with
//          amax_row <= 2688 2^e (2688 = 6 * 448, so no block scale
//          saturates); s = E4M3(fl32(amax 2^-e / 6)); code = E2M1(x 2^-e / s),
//          0 where s is 0.  A power of two keeps x 2^-e and every tie of 16-bit
//          inputs exact, so the codes are those of exact arithmetic.
// The quotient by s is x hi + x lo with hi just below 1 / s and lo the rest of
// 1 / s: one multiply and one FMA instead of a division per element, right on
// every tie (a tie is a product of s with a multiple of 1/4).
// Non-finite values: an mx block that holds one gets the scale 0xFF (NaN) and
// zero codes, an nvfp4 row gets a NaN row scale, zero scales and codes.
//
// Scales are kept in the order the block-scaled MMA wants them in tensor
// memory: tiles of 128 rows x 4 blocks, 512 bytes, [row / 128][block / 4]
// [row % 32][row / 32 % 4][block % 4].  A row's four scales of a tile are one
// aligned word; the words of a row are written whole, blocks past Kp as 0.
#pragma once

#include <type_traits>

#include "device.cuh"
#include "launch.cuh"

namespace fqa {

enum MxFormat : int { kMxFp8 = 0, kMxFp4 = 1, kNvFp4 = 2 };

template <int FMT>
struct MxTraits {
  static constexpr int kBlock = FMT == kNvFp4 ? 16 : 32;     // elements per scale
  static constexpr int kBlockChunks = kBlock / 16;           // threads (16 elements each) per scale
  static constexpr int kWordChunks = 4 * kBlockChunks;       // threads per word of four scales
};

__host__ __device__ constexpr int mx_block(int fmt) { return fmt == kNvFp4 ? 16 : 32; }
__host__ __device__ constexpr int mx_per_byte(int fmt) { return fmt == kMxFp8 ? 1 : 2; }

// ------------------------------------------------------- element access

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Two binary32 values -> one word of two 16-bit values, `lo` first in memory.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Four neighbours of a 16-bit type on an 8-byte boundary.
template <typename T>
__device__ __forceinline__ void store_four(T* p, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
}

// 32 bytes per thread in one access (sm_100; address on a 32-byte boundary):
// a whole sector, where two 16-byte stores of a thread would each write half
// of one.
__device__ __forceinline__ void load_32b(const void* p, uint4& a, uint4& b) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
               : "l"(p));
}
__device__ __forceinline__ void store_32b(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// A thread's chunk of a row: 16 elements, as they lie in memory.  kVec: the row
// starts on a 16-byte boundary and K fills whole 16-byte groups, so each group
// is there or not (`wide`: the same in 32 bytes).  Nothing here uses what it
// loads, so that the loads of several chunks and tensors are all in flight
// before the first is needed.
constexpr int kMxChunk = 16;

template <typename T, bool kVec>
struct MxRaw {
  static constexpr int kGroup = 16 / sizeof(T);              // elements per 16 bytes
  uint4 g[kMxChunk / kGroup];
  __device__ __forceinline__ void load(const T* row, int c0, int K, bool wide) {
#pragma unroll
    for (int i = 0; i < kMxChunk / kGroup; ++i) g[i] = make_uint4(0u, 0u, 0u, 0u);
    if (wide) {
#pragma unroll
      for (int i = 0; i < kMxChunk / kGroup; i += 2)
        if (c0 + i * kGroup < K) load_32b(row + c0 + i * kGroup, g[i], g[i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < kMxChunk / kGroup; ++i)
        if (c0 + i * kGroup < K) g[i] = *reinterpret_cast<const uint4*>(row + c0 + i * kGroup);
    }
  }
  __device__ __forceinline__ void get(float (&v)[kMxChunk]) const {
#pragma unroll
    for (int i = 0; i < kMxChunk / kGroup; ++i) {
      const uint32_t w[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 4) {
          v[4 * i + e] = __uint_as_float(w[e]);
        } else {
          const float2 f = unpack2<T>(w[e]);
          v[8 * i + 2 * e] = f.x;
          v[8 * i + 2 * e + 1] = f.y;
        }
      }
    }
  }
};
template <typename T>
struct MxRaw<T, false> {
  T g[kMxChunk];
  __device__ __forceinline__ void load(const T* row, int c0, int K, bool) {
#pragma unroll
    for (int e = 0; e < kMxChunk; ++e) g[e] = c0 + e < K ? row[c0 + e] : from_f32<T>(0.0f);
  }
  __device__ __forceinline__ void get(float (&v)[kMxChunk]) const {
#pragma unroll
    for (int e = 0; e < kMxChunk; ++e) v[e] = to_f32<T>(g[e]);
  }
};

// N values of T as words.
template <typename T, int N>
__device__ __forceinline__ void pack_words(const float* v, uint32_t (&w)[N * sizeof(T) / 4]) {
#pragma unroll
  for (int i = 0; i < (int)(N * sizeof(T) / 4); ++i) {
    if constexpr (sizeof(T) == 4)
      w[i] = __float_as_uint(v[i]);
    else
      w[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
  }
}

template <typename T, bool kVec>
__device__ __forceinline__ void store_chunk(T* row, int c0, int K, bool wide, const float (&v)[kMxChunk]) {
  if constexpr (kVec) {
    constexpr int G = 16 / sizeof(T);
    if (wide) {
#pragma unroll
      for (int i = 0; i < kMxChunk / G; i += 2)
        if (c0 + i * G < K) {
          uint32_t w[8];
          pack_words<T, 2 * G>(&v[i * G], w);
          store_32b(row + c0 + i * G, w);
        }
    } else {
#pragma unroll
      for (int i = 0; i < kMxChunk / G; ++i)
        if (c0 + i * G < K) {
          uint32_t w[4];
          pack_words<T, G>(&v[i * G], w);
          *reinterpret_cast<uint4*>(row + c0 + i * G) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
  } else {
#pragma unroll
    for (int e = 0; e < kMxChunk; ++e)
      if (c0 + e < K) row[c0 + e] = from_f32<T>(v[e]);
  }
}

// ----------------------------------------------------------- the codes

// Largest magnitude of three values, NaN if one is.
__device__ __forceinline__ float amax3(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Largest |v| of a chunk as its bit pattern: ordered like the magnitude, and at
// or above 0x7F800000 exactly when one of them is not finite.
__device__ __forceinline__ uint32_t chunk_amax(const float (&v)[kMxChunk]) {
  float m = amax3(v[0], v[1], v[2]), n = amax3(v[3], v[4], v[5]);
#pragma unroll
  for (int e = 6; e < 14; e += 4) {
    m = amax3(m, v[e], v[e + 1]);
    n = amax3(n, v[e + 2], v[e + 3]);
  }
  return __float_as_uint(amax3(amax3(m, v[14], v[15]), n, n)) & 0x7FFFFFFFu;
}

// Exponent byte of the smallest power of two whose `largest` multiple
// reaches the magnitude, largest = 2^top (1 + part / 2^23); not below `low`.
__device__ __forceinline__ int power_byte(uint32_t amax, int top, uint32_t part, int low) {
  const int b = (int)(amax >> 23) - top + ((amax & 0x7FFFFFu) > part ? 1 : 0);
  return b < low ? low : b;
}

// 2^(127 - byte) for 0 <= byte <= 253.
__device__ __forceinline__ float inverse_power(int byte) { return __uint_as_float((uint32_t)(254 - byte) << 23); }

// Eight binary32 values -> eight E2M1 codes in one word, v[0] in bits [0,4).
__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// v * s and fma(v, a, v * b) for a chunk, two values an instruction.
__device__ __forceinline__ void chunk_mul(float (&v)[kMxChunk], float s) {
#pragma unroll
  for (int e = 0; e < kMxChunk; e += 2) {
    const float2 r = f2_mul(make_float2(v[e], v[e + 1]), make_float2(s, s));
    v[e] = r.x;
    v[e + 1] = r.y;
  }
}
__device__ __forceinline__ void chunk_mul2(float (&v)[kMxChunk], float a, float b) {
#pragma unroll
  for (int e = 0; e < kMxChunk; e += 2) {
    const float2 x = make_float2(v[e], v[e + 1]);
    const float2 r = f2_fma(x, make_float2(a, a), f2_mul(x, make_float2(b, b)));
    v[e] = r.x;
    v[e + 1] = r.y;
  }
}

// x / 6 rounded to nearest, as x h + x l with h + l = 1/6 to 48 bits: off from
// the quotient by 2^-47 of it, while a quotient by 6 that is not a binary32
// value lies at least a sixth of a unit from the midpoint of two.
__device__ __forceinline__ float sixth(float x) {
  constexpr float h = 0x1.555556p-3f, l = -0x1.555556p-28f;
  return __fmaf_rn(x, h, __fmul_rn(x, l));
}

// A value one to three units below 1 / s (inf for 0).
__device__ __forceinline__ float below_reciprocal(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));   // off by at most one unit
  return __uint_as_float(__float_as_uint(r) - 2u);
}

struct MxRowParams {
  const void* x;          // [M] rows of K, row stride ldx (elements)
  const void* residual;   // the same shape, row stride ldr; binary32 if res_f32, else x's type
  void* residual_out;     // contiguous [M,K], residual's type
  const void* weight;     // [K], binary32 if w_f32, else x's type (so w_f32 and res_f32 are 0 for binary32 x)
  int64_t ldx, ldr;
  float eps;
  int M, K, Kp, KT;       // KT words of four scales per row
  int res_f32, w_f32;
  int wide;               // every row on 32-byte boundaries, in whole groups of 32 bytes
  uint8_t* codes;         // [M, Kp] or [M, Kp / 2]
  uint32_t* scales;       // tiles, as words
  float* row_scale;       // [M] (nvfp4)
};

// Writes chunk c (elements [16c, 16c + 16)) of a row whose codes and scale
// words start at `codes` and `words`; amax: the chunk's largest magnitude,
// row_amax: the row's (nvfp4).  Called by whole warps with consecutive c, so the
// threads of a scale and of a word are neighbours.
template <int FMT>
__device__ __forceinline__ void emit_chunk(const MxRowParams& p, uint8_t* codes, uint32_t* words, int c,
                                           float (&v)[kMxChunk], uint32_t amax, uint32_t row_amax) {
  using F = MxTraits<FMT>;
#pragma unroll
  for (int o = 1; o < F::kBlockChunks; o <<= 1) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  uint32_t byte = 0;
  bool zero = false;
  if constexpr (FMT == kNvFp4) {
    if (row_amax < 0x7F800000u) {
      const int e = power_byte(row_amax, 11, 0x280000u, 1);
      const float inv = inverse_power(e);
      byte = e4m3x2(sixth(__uint_as_float(amax) * inv), 0.0f) & 0xFFu;
      const float s = e4m3x2_to_f2(byte).x;
      float hi = below_reciprocal(s);
      float lo = __fmul_rn(__fmaf_rn(-s, hi, 1.0f), hi);   // >= 0, so a zero keeps its sign below
      if (e >= 27 && e <= 207) {       // the row's power goes into both parts, exactly
        hi *= inv;
        lo *= inv;
      } else {                         // where they would leave binary32, into the values
        chunk_mul(v, inv);
      }
      if (byte != 0) chunk_mul2(v, hi, lo);
    }
    zero = byte == 0;
  } else {
    zero = amax >= 0x7F800000u;
    byte = zero ? 0xFFu
                : (uint32_t)(FMT == kMxFp8 ? power_byte(amax, 8, 0x600000u, 0) : power_byte(amax, 2, 0x400000u, 0));
    if (!zero) chunk_mul(v, inverse_power((int)byte));
  }
  if (zero) {
#pragma unroll
    for (int e = 0; e < kMxChunk; ++e) v[e] = 0.0f;
  }
  if (kMxChunk * c < p.Kp) {
    if constexpr (FMT == kMxFp8)
      *reinterpret_cast<uint4*>(codes + kMxChunk * (size_t)c) =
          make_uint4(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]), e4m3x4(v[8], v[9], v[10], v[11]),
                     e4m3x4(v[12], v[13], v[14], v[15]));
    else
      *reinterpret_cast<uint2*>(codes + kMxChunk / 2 * (size_t)c) = make_uint2(e2m1x8(&v[0]), e2m1x8(&v[8]));
  }
  // the word of four scales: each scale's threads shift theirs into place
  uint32_t w = byte << (8 * ((c / F::kBlockChunks) & 3));
  w |= __shfl_xor_sync(0xFFFFFFFFu, w, F::kBlockChunks);
  w |= __shfl_xor_sync(0xFFFFFFFFu, w, 2 * F::kBlockChunks);
  const int word = c / F::kWordChunks;
  if (c % F::kWordChunks == 0 && word < p.KT) words[(size_t)word * 128] = w;
}

// Reductions over the threads of a row: one warp, or the whole CTA (kCta, up to
// 16 warps).
template <bool kCta>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if constexpr (kCta) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = lane < (int)(blockDim.x >> 5) ? red[lane] : 0.0f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    v = __shfl_sync(0xFFFFFFFFu, v, 0);
  }
  return v;
}
template <bool kCta>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* red) {
  v = __reduce_max_sync(0xFFFFFFFFu, v);
  if constexpr (kCta) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = __reduce_max_sync(0xFFFFFFFFu, lane < (int)(blockDim.x >> 5) ? red[lane] : 0u);
  }
  return v;
}

// One row per warp (four a CTA) or per CTA (kCta) of as many warps as its chunks
// of 16 elements need, NCH a thread, held in registers; kLoop: a CTA's row too
// long for that is read again for each step instead.  Normed: h = x + residual in binary32,
// residual_out = h rounded, y = h / sqrt(mean h^2 + eps) * weight, and y is
// quantized (never h's rounding: the norm sees the sum itself).
//
// Bound by memory: every input is read once, all loads of a row are in flight
// before its first sum, in 32-byte accesses.  8704 x 4096 BF16 with residual to
// mxfp8 moves 251 MB in 39 us (6.4 TB/s, 98% of a copy's rate), 12288 x 4096 BF16
// to nvfp4 129 MB in 24 us (two roundings of scales and two products per element;
// mxfp8 153 MB in 24 us).
template <typename T, int FMT, bool kNorm, bool kCta, int NCH, bool kLoop, bool kVec>
__global__ void __launch_bounds__(kCta ? 512 : 128) mx_row_kernel(const MxRowParams p) {
  __shared__ float red_sum[16];
  __shared__ uint32_t red_max[16];
  grid_release();
  grid_wait();
  const int TPR = kCta ? blockDim.x : 32;        // threads per row
  const int t = kCta ? threadIdx.x : threadIdx.x & 31;
  const int row = kCta ? blockIdx.x : blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= p.M) return;                       // whole warps (and no CTA of a row's own)
  const T* x = static_cast<const T*>(p.x) + (int64_t)row * p.ldx;
  const bool res = kNorm && p.residual != nullptr;
  uint8_t* codes = p.codes + (size_t)row * (p.Kp / mx_per_byte(FMT));
  uint32_t* words = p.scales + (size_t)(row >> 7) * p.KT * 128 + (row & 31) * 4 + ((row >> 5) & 3);

  auto add_residual = [&](const auto& raw, float (&v)[kMxChunk]) {
    float r[kMxChunk];
    raw.get(r);
#pragma unroll
    for (int e = 0; e < kMxChunk; e += 2) {
      const float2 h = f2_add(make_float2(v[e], v[e + 1]), make_float2(r[e], r[e + 1]));
      v[e] = h.x;
      v[e + 1] = h.y;
    }
  };
  auto store_h = [&](int c, const float (&v)[kMxChunk]) {
    if (p.res_f32)
      store_chunk<float, kVec>(static_cast<float*>(p.residual_out) + (int64_t)row * p.K, kMxChunk * c, p.K, p.wide, v);
    else
      store_chunk<T, kVec>(static_cast<T*>(p.residual_out) + (int64_t)row * p.K, kMxChunk * c, p.K, p.wide, v);
  };
  // h of NCH chunks, loads first
  auto load_h = [&](int c0, float (&v)[NCH][kMxChunk]) {
    MxRaw<T, kVec> a[NCH];
#pragma unroll
    for (int j = 0; j < NCH; ++j) a[j].load(x, kMxChunk * (c0 + j * TPR), p.K, p.wide);
    if (!res) {
#pragma unroll
      for (int j = 0; j < NCH; ++j) a[j].get(v[j]);
    } else if (p.res_f32) {
      const float* r = static_cast<const float*>(p.residual) + (int64_t)row * p.ldr;
      MxRaw<float, kVec> b[NCH];
#pragma unroll
      for (int j = 0; j < NCH; ++j) b[j].load(r, kMxChunk * (c0 + j * TPR), p.K, p.wide);
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        a[j].get(v[j]);
        add_residual(b[j], v[j]);
      }
    } else {
      const T* r = static_cast<const T*>(p.residual) + (int64_t)row * p.ldr;
      MxRaw<T, kVec> b[NCH];
#pragma unroll
      for (int j = 0; j < NCH; ++j) b[j].load(r, kMxChunk * (c0 + j * TPR), p.K, p.wide);
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        a[j].get(v[j]);
        add_residual(b[j], v[j]);
      }
    }
  };
  auto squares = [&](const float (&v)[kMxChunk]) {
    // four sums of four: short chains keep the rounding small
    float2 s[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
    for (int e = 0; e < kMxChunk; e += 2) {
      const float2 x = make_float2(v[e], v[e + 1]);
      s[(e >> 1) & 1] = f2_fma(x, x, s[(e >> 1) & 1]);
    }
    return (s[0].x + s[0].y) + (s[1].x + s[1].y);
  };
  auto scaled = [&](int c, float rstd, const float (&w)[kMxChunk], float (&v)[kMxChunk]) {
#pragma unroll
    for (int e = 0; e < kMxChunk; e += 2) {
      const float2 r =
          f2_mul(f2_mul(make_float2(v[e], v[e + 1]), make_float2(rstd, rstd)), make_float2(w[e], w[e + 1]));
      v[e] = r.x;
      v[e + 1] = r.y;
    }
    if (kMxChunk * c + kMxChunk > p.K) {         // past K: not 0 * infinity
#pragma unroll
      for (int e = 0; e < kMxChunk; ++e)
        if (kMxChunk * c + e >= p.K) v[e] = 0.0f;
    }
  };
  auto inverse_root = [&](float ss) { return __frsqrt_rn(__fdiv_rn(row_sum<kCta>(ss, red_sum), (float)p.K) + p.eps); };
  auto store_row_scale = [&](uint32_t amax) {
    if (FMT == kNvFp4 && t == 0)
      p.row_scale[row] = __uint_as_float(
          amax < 0x7F800000u ? (uint32_t)power_byte(amax, 11, 0x280000u, 1) << 23 : 0x7FC00000u);
  };

  if constexpr (!kLoop) {
    float v[NCH][kMxChunk];
    MxRaw<T, kVec> w[NCH];                       // the weights ride along with the row's loads
    if (kNorm && !p.w_f32) {
#pragma unroll
      for (int j = 0; j < NCH; ++j) w[j].load(static_cast<const T*>(p.weight), kMxChunk * (t + j * TPR), p.K, p.wide);
    }
    load_h(t, v);
    if constexpr (kNorm) {
      float ss = 0.0f;
#pragma unroll
      for (int j = 0; j < NCH; ++j) ss += squares(v[j]);
      if (res) {
#pragma unroll
        for (int j = 0; j < NCH; ++j) store_h(t + j * TPR, v[j]);
      }
      const float rstd = inverse_root(ss);
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        float f[kMxChunk];
        if (p.w_f32) {
          MxRaw<float, kVec> g;
          g.load(static_cast<const float*>(p.weight), kMxChunk * (t + j * TPR), p.K, p.wide);
          g.get(f);
        } else {
          w[j].get(f);
        }
        scaled(t + j * TPR, rstd, f, v[j]);
      }
    }
    uint32_t amax[NCH], top = 0;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      amax[j] = chunk_amax(v[j]);
      top = max(top, amax[j]);
    }
    if constexpr (FMT == kNvFp4) top = row_max<kCta>(top, red_max);
#pragma unroll
    for (int j = 0; j < NCH; ++j) emit_chunk<FMT>(p, codes, words, t + j * TPR, v[j], amax[j], top);
    store_row_scale(top);
  } else {
    static_assert(NCH == 1, "one chunk per pass");
    // a whole number of passes for every thread: the shuffles need full warps
    const int passes = (p.KT * MxTraits<FMT>::kWordChunks + TPR - 1) / TPR;
    auto normed = [&](int c, float rstd, float (&v)[kMxChunk]) {
      float f[kMxChunk];
      if (p.w_f32) {
        MxRaw<float, kVec> g;
        g.load(static_cast<const float*>(p.weight), kMxChunk * c, p.K, p.wide);
        g.get(f);
      } else {
        MxRaw<T, kVec> g;
        g.load(static_cast<const T*>(p.weight), kMxChunk * c, p.K, p.wide);
        g.get(f);
      }
      scaled(c, rstd, f, v);
    };
    float v[1][kMxChunk];
    float rstd = 1.0f;
    if constexpr (kNorm) {
      float ss = 0.0f;
      for (int i = 0; i < passes; ++i) {
        load_h(t + i * TPR, v);
        ss += squares(v[0]);
      }
      rstd = inverse_root(ss);
    }
    uint32_t amax = 0;
    if constexpr (FMT == kNvFp4) {
      for (int i = 0; i < passes; ++i) {
        load_h(t + i * TPR, v);
        if constexpr (kNorm) normed(t + i * TPR, rstd, v[0]);
        amax = max(amax, chunk_amax(v[0]));
      }
      amax = row_max<kCta>(amax, red_max);
    }
    // residual_out may be residual itself: each thread writes an element only
    // here, after its own last read of it
    for (int i = 0; i < passes; ++i) {
      load_h(t + i * TPR, v);
      if (res) store_h(t + i * TPR, v[0]);
      if constexpr (kNorm) normed(t + i * TPR, rstd, v[0]);
      emit_chunk<FMT>(p, codes, words, t + i * TPR, v[0], chunk_amax(v[0]), amax);
    }
    store_row_scale(amax);
  }
}

// The same for rows off the 16-byte boundaries (an odd K, a shifted view): one
// row per CTA, read element by element along the row, so that a warp's loads and
// stores are one segment, into shared memory as binary32; the chunks are taken
// from there.  (Chunks of 16 straight from memory, element by element, touch a
// sector per lane and load, and needed the row again for every step: 156 us for
// the norm of 8704 x 4097 BF16.)  Now 76 us there, 3.3 TB/s, bound by its 2-byte
// accesses, and 60 us at 8704 x 4098 in pairs.
constexpr int kMxAnyThreads = 256;
constexpr int kMxAnyCols = 49152;            // longest row held
constexpr int kMxAnyWarps = kMxAnyThreads / 32;
constexpr int kMxAnyStatic = 2 * kMxAnyWarps * 4;   // shared memory beside the row: a word per warp for each reduction

// E neighbours (E * sizeof(T) bytes aligned) as binary32, and back.
template <typename T, int E>
struct MxFew {
  std::conditional_t<E == 1, T, std::conditional_t<sizeof(T) == 4, uint2, uint32_t>> raw;
  __device__ __forceinline__ void load(const T* p) { raw = *reinterpret_cast<const decltype(raw)*>(p); }
  __device__ __forceinline__ void get(float (&v)[E]) const {
    if constexpr (E == 1) {
      v[0] = to_f32<T>(raw);
    } else if constexpr (sizeof(T) == 4) {
      v[0] = __uint_as_float(raw.x);
      v[1] = __uint_as_float(raw.y);
    } else {
      const float2 f = unpack2<T>(raw);
      v[0] = f.x;
      v[1] = f.y;
    }
  }
  static __device__ __forceinline__ void store(T* p, const float (&v)[E]) {
    if constexpr (E == 1)
      *p = from_f32<T>(v[0]);
    else if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    else
      *reinterpret_cast<uint32_t*>(p) = pack2<T>(v[0], v[1]);
  }
};

// Place of value e in shared memory: a chunk's four groups of four change places
// with the chunk's number, so that neither the passes along the row nor the
// chunks' 16-byte reads meet in a bank.
__device__ __forceinline__ int mx_any_place(int e) { return e ^ (((e >> 5) & 3) << 2); }

// CTAs per SM that the registers have to allow.  16-bit pairs with a norm: five
// (four by themselves; 8704 x 4098 BF16 to mxfp8 67 -> 60 us; FP32 pairs would
// spill, 1023 x 5102: 17 -> 21 us, and single values lose 6% for nvfp4).  Without
// a norm: six (12288 x 4097 BF16 to mxfp4 56 -> 53 us, although mxfp8 and mxfp4
// spill 36 bytes for it, single values of every type and 16-bit pairs; FP32 pairs
// 48 -> 51 us).
template <typename T, bool kNorm, int E>
constexpr int mx_any_ctas() {
  if (E == 2 && sizeof(T) == 4) return 0;      // as the compiler likes
  return kNorm ? (E == 2 ? 5 : 0) : 6;
}

// E: values per access, two where all rows allow it.
template <typename T, int FMT, bool kNorm, int E>
__global__ void __launch_bounds__(kMxAnyThreads, mx_any_ctas<T, kNorm, E>()) mx_row_any_kernel(const MxRowParams p) {
  extern __shared__ __align__(16) float h[];   // the row's values, zeros past K
  __shared__ float red_sum[kMxAnyWarps];
  __shared__ uint32_t red_max[kMxAnyWarps];
  grid_release();
  grid_wait();
  const int t = threadIdx.x, row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + (int64_t)row * p.ldx;
  const int chunks = p.KT * MxTraits<FMT>::kWordChunks, width = chunks * kMxChunk;
  const bool res = kNorm && p.residual != nullptr;
  float ss = 0.0f;
  constexpr int B = 8, S = E * kMxAnyThreads;    // accesses a thread has in flight, and the step between them
  // residual types: its row's pointers are formed where its type is known
  auto pass = [&](auto type) {
    using R = decltype(type);
    const R* r = static_cast<const R*>(p.residual) + (int64_t)row * p.ldr;
    R* ro = static_cast<R*>(p.residual_out) + (int64_t)row * p.K;
    for (int e0 = E * t; e0 < p.K; e0 += B * S) {
      MxFew<T, E> a[B];
      MxFew<R, E> q[B];
#pragma unroll
      for (int i = 0; i < B; ++i)
        if (e0 + i * S < p.K) a[i].load(x + e0 + i * S);
      if (res) {
#pragma unroll
        for (int i = 0; i < B; ++i)
          if (e0 + i * S < p.K) q[i].load(r + e0 + i * S);
      }
#pragma unroll
      for (int i = 0; i < B; ++i) {
        const int e = e0 + i * S;
        if (e >= p.K) break;
        float v[E];
        a[i].get(v);
        if (res) {
          float w[E];
          q[i].get(w);
#pragma unroll
          for (int k = 0; k < E; ++k) v[k] += w[k];
          MxFew<R, E>::store(ro + e, v);
        }
        MxFew<float, E>::store(h + mx_any_place(e), v);
        if constexpr (kNorm) {
#pragma unroll
          for (int k = 0; k < E; ++k) ss = fmaf(v[k], v[k], ss);
        }
      }
    }
  };
  if (kNorm && p.res_f32)
    pass(float{});
  else
    pass(T{});
  for (int e = p.K + t; e < width; e += kMxAnyThreads) h[mx_any_place(e)] = 0.0f;
  uint32_t top = 0;
  if constexpr (kNorm) {
    const float rstd = __frsqrt_rn(__fdiv_rn(row_sum<true>(ss, red_sum), (float)p.K) + p.eps);
    auto scale = [&](auto type) {
      using W = decltype(type);
      const W* wp = static_cast<const W*>(p.weight);
      for (int e0 = E * t; e0 < p.K; e0 += B * S) {
        MxFew<W, E> w[B];
#pragma unroll
        for (int i = 0; i < B; ++i)
          if (e0 + i * S < p.K) w[i].load(wp + e0 + i * S);
#pragma unroll
        for (int i = 0; i < B; ++i) {
          const int e = e0 + i * S;
          if (e >= p.K) break;
          float f[E], y[E];
          w[i].get(f);
          MxFew<float, E> held;
          held.load(h + mx_any_place(e));
          held.get(y);
#pragma unroll
          for (int k = 0; k < E; ++k) {
            y[k] = __fmul_rn(__fmul_rn(y[k], rstd), f[k]);
            if constexpr (FMT == kNvFp4) top = max(top, __float_as_uint(y[k]) & 0x7FFFFFFFu);
          }
          MxFew<float, E>::store(h + mx_any_place(e), y);
        }
      }
    };
    if (p.w_f32)
      scale(float{});
    else
      scale(T{});
  } else if constexpr (FMT == kNvFp4) {
    for (int e0 = E * t; e0 < p.K; e0 += S)      // this thread's own
#pragma unroll
      for (int k = 0; k < E; ++k) top = max(top, __float_as_uint(h[mx_any_place(e0) + k]) & 0x7FFFFFFFu);
  }
  if constexpr (FMT == kNvFp4) top = row_max<true>(top, red_max);
  __syncthreads();
  uint8_t* codes = p.codes + (size_t)row * (p.Kp / mx_per_byte(FMT));
  uint32_t* words = p.scales + (size_t)(row >> 7) * p.KT * 128 + (row & 31) * 4 + ((row >> 5) & 3);
  for (int c0 = 0; c0 < chunks; c0 += kMxAnyThreads) {      // whole warps: the scales are shared by shuffles
    const int c = c0 + t;
    float v[kMxChunk];
#pragma unroll
    for (int i = 0; i < kMxChunk; i += 4) {
      const float4 f = c < chunks ? *reinterpret_cast<const float4*>(h + mx_any_place(kMxChunk * c + i))
                                  : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      v[i] = f.x; v[i + 1] = f.y; v[i + 2] = f.z; v[i + 3] = f.w;
    }
    emit_chunk<FMT>(p, codes, words, c, v, chunk_amax(v), top);
  }
  if (FMT == kNvFp4 && t == 0)
    p.row_scale[row] = __uint_as_float(
        top < 0x7F800000u ? (uint32_t)power_byte(top, 11, 0x280000u, 1) << 23 : 0x7FC00000u);
}

// ------------------------------------------------------------ and back

// Two E2M1 codes (bits [0,4) and [4,8)) -> their values.
__device__ __forceinline__ float2 e2m1x2_to_f2(uint32_t codes) {
  uint32_t h2;
  asm("{\n\t.reg .b8 c;\n\tcvt.u8.u32 c, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(h2) : "r"(codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&h2));
}

// E8M0 byte -> 2^(byte - 127); 0 -> 2^-127 (subnormal), 255 -> NaN.
__device__ __forceinline__ float e8m0_to_f32(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x7FC00000u : (b == 0u ? 0x00400000u : b << 23));
}

struct MxDequantParams {
  const uint8_t* codes;
  const uint8_t* scales;
  const float* row_scale;
  void* out;              // contiguous [M, K]
  int M, K, Kp, KT;
  int wide;               // as MxRowParams (or, off 16-byte boundaries, rows on boundaries of two values)
};

// value = element * scale (exact in binary32) * row scale, rounded once more to
// the output's type.  A thread takes chunks of 16 elements, blockDim.x of them
// side by side in a row and blockDim.y rows per CTA (a 64-bit division per chunk
// cost 35 instead of 23 us at 12288 x 4096, nvfp4 to BF16: 128 MB, 5.6 TB/s).
template <typename T, int FMT>
__global__ void __launch_bounds__(256) mx_dequantize_kernel(const MxDequantParams p) {
  grid_release();
  grid_wait();
  constexpr int kBlock = MxTraits<FMT>::kBlock;
  const int row = blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= p.M) return;
  const uint8_t* sf = p.scales + (size_t)(row >> 7) * p.KT * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4;
  const uint8_t* codes = p.codes + (size_t)row * (p.Kp / mx_per_byte(FMT));
  const float rs = FMT == kNvFp4 ? p.row_scale[row] : 1.0f;
  T* out = static_cast<T*>(p.out) + (int64_t)row * p.K;
  for (int c = threadIdx.x; kMxChunk * c < p.K; c += blockDim.x) {
    const int blk = kMxChunk * c / kBlock;
    const uint32_t sb = sf[(size_t)(blk >> 2) * 512 + (blk & 3)];
    float v[kMxChunk];
    if constexpr (FMT == kMxFp8) {
      const uint4 g = *reinterpret_cast<const uint4*>(codes + kMxChunk * (size_t)c);
      const uint32_t w[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 f = e4m3x2_to_f2((w[e / 2] >> (16 * (e & 1))) & 0xFFFFu);
        v[2 * e] = f.x;
        v[2 * e + 1] = f.y;
      }
    } else {
      const uint2 g = *reinterpret_cast<const uint2*>(codes + kMxChunk / 2 * (size_t)c);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 f = e2m1x2_to_f2(((e < 4 ? g.x : g.y) >> (8 * (e & 3))) & 0xFFu);
        v[2 * e] = f.x;
        v[2 * e + 1] = f.y;
      }
    }
    const float s = FMT == kNvFp4 ? e4m3x2_to_f2(sb).x : e8m0_to_f32(sb);
#pragma unroll
    for (int e = 0; e < kMxChunk; ++e) v[e] = FMT == kNvFp4 ? v[e] * s * rs : v[e] * s;
    store_chunk<T, true>(out, kMxChunk * c, p.K, p.wide, v);
  }
}

// The same for rows off the 16-byte boundaries: a thread takes W neighbours, so
// that a warp's stores are one segment: four (16-bit rows on 8-byte boundaries),
// or two, stored together where rows start on their boundaries (wide).
template <typename T, int FMT, int W>
__global__ void __launch_bounds__(256) mx_dequantize_any_kernel(const MxDequantParams p) {
  grid_release();
  grid_wait();
  constexpr int kBlock = MxTraits<FMT>::kBlock;
  const int row = blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= p.M) return;
  const uint8_t* sf = p.scales + (size_t)(row >> 7) * p.KT * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4;
  const uint8_t* codes = p.codes + (size_t)row * (p.Kp / mx_per_byte(FMT));
  const float rs = FMT == kNvFp4 ? p.row_scale[row] : 1.0f;
  T* out = static_cast<T*>(p.out) + (int64_t)row * p.K;
  constexpr int B = 4;                           // groups a thread has in flight
  for (int c0 = threadIdx.x; W * c0 < p.K; c0 += B * blockDim.x) {
    uint32_t sb[B];
    uint16_t code[B][W / 2];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int c = c0 + i * (int)blockDim.x;
      if (W * c >= p.K) break;
      const int blk = W * c / kBlock;
      sb[i] = sf[(size_t)(blk >> 2) * 512 + (blk & 3)];
#pragma unroll
      for (int e = 0; e < W / 2; ++e)
        code[i][e] = FMT == kMxFp8 ? *reinterpret_cast<const uint16_t*>(codes + W * (size_t)c + 2 * e)
                                   : codes[W / 2 * (size_t)c + e];
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int c = c0 + i * (int)blockDim.x;
      if (W * c >= p.K) break;
      const float s = FMT == kNvFp4 ? e4m3x2_to_f2(sb[i]).x : e8m0_to_f32(sb[i]);
      float v[W];
#pragma unroll
      for (int e = 0; e < W / 2; ++e) {
        const float2 f = FMT == kMxFp8 ? e4m3x2_to_f2(code[i][e]) : e2m1x2_to_f2(code[i][e]);
        v[2 * e] = FMT == kNvFp4 ? f.x * s * rs : f.x * s;
        v[2 * e + 1] = FMT == kNvFp4 ? f.y * s * rs : f.y * s;
      }
      if constexpr (W == 4) {
        store_four(out + 4 * c, v);
      } else if (p.wide) {
        MxFew<T, 2>::store(out + 2 * c, v);
      } else {
        out[2 * c] = from_f32<T>(v[0]);
        if (2 * c + 1 < p.K) out[2 * c + 1] = from_f32<T>(v[1]);
      }
    }
  }
}

}  // namespace fqa
