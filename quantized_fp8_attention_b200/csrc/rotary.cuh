// rotary.cuh -- rotary positions over one to four axes (time, height, width),
// with the per-head RMS norm of Q and K that precedes them where weights are
// given, from any strided [B, H, N, 128] view to the contiguous layout the
// quantizer takes.
//
//   pair j of a token: turns = position[axis_j] * f_j, f_j = theta^(-2 i / D) / 2 pi
//   (x0, x1) -> (x0 cos - x1 sin, x0 sin + x1 cos), cos and sin of 2 pi turns
// The turns are formed in binary64 and reduced to [-1/2, 1/2] there: at
// position 65536 a binary32 angle is off by up to 2^-8, the reduced one by
// 2^-25 turns.  The rotation runs in binary32 and is rounded once.
//
// Memory-bound: every element read once and written once.  16 lanes hold one
// token's row of 128 channels and walk over its heads, so the 64 angles of a
// token are formed once for all of them (48 rows share them at 24 heads); a
// row is one 256-byte segment on both sides whatever the layout.  2 x 16896
// tokens x 48 heads BF16: 830 MB in 136 us (6.1 TB/s); 4608 tokens x 48 heads
// with norm: 113 MB in 23 us, of which the angles and the launch take about 5.
#pragma once

#include <type_traits>

#include "device.cuh"
#include "microscale.cuh"

namespace fqa {

constexpr int kRotMaxAxes = 4;

struct RotaryParams {
  const void* in[2];            // Q and K
  void* out[2];                 // contiguous [B, H, N, 128]
  const void* weight[2];        // [128] or null
  int64_t sb[2], sh[2], sn[2];  // input strides in elements
  int heads[2];
  int vec[2];                   // rows aligned for vector loads
  const void* pos;              // [B or 1, N, n_axes], int32 or binary32
  int64_t pos_sb;               // 0 when every batch element has the same
  int pos_f32, n_axes;
  int B, N;
  int pairs;                    // rotated pairs: channels [0, 2 pairs); the rest pass through
  int heads_per_group;          // heads of [Q | K] that one group of lanes walks over
  float eps, sign;              // sign -1: the inverse rotation
  double f[64];                 // turns per position, per pair
  uint8_t axis[64];
};

// Asynchronous copy of 16 bytes, global to shared (both on 16-byte boundaries).
__device__ __forceinline__ void cp_async_16(uint32_t smem, const void* g) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(g) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// kSplit: pair j is channels (j, pairs + j); otherwise (2j, 2j + 1).  Pairs
// never cross lanes: interleaved a lane of 16 holds eight neighbours (four
// pairs); split a lane of 8 holds eight channels and their eight partners, and
// the 16 lanes take two heads at a time.  Every access is 16 bytes a lane (16
// lanes with 4 + 4 channels, 8 bytes an access, ran at 3.9 instead of 5.8
// TB/s).  Rows are fetched ahead by asynchronous copies into a ring of shared
// memory in which every thread reads only what it copied itself, so there is no
// barrier: two batches of 64 bytes a thread are in flight whatever the register
// count (one batch ahead in registers: 4608 tokens x 48 heads took 29 us, half
// the memory's rate).
// kNorm: a weight is given for Q or K.  The weight goes into the coefficients
// of the rotation, so a row costs its sum of squares, one factor and the
// rotation; two pairs share each packed instruction.  (Unpacked, with weights
// applied per row, the kernel was bound by its 193 instructions per row and
// warp.)  kAll: all 64 pairs rotate.
template <typename T, bool kSplit, bool kNorm, bool kAll>
__global__ void __launch_bounds__(256, kSplit ? (kNorm ? 2 : 3) : (kNorm ? 3 : 4)) rotary_kernel(const __grid_constant__ RotaryParams p) {
  constexpr int LPR = kSplit ? 8 : 16;                 // lanes per row
  constexpr int P = kSplit ? 8 : 4;                    // channels per piece = pairs per lane
  constexpr int HS = 16 / LPR;                         // heads at a time
  constexpr int U = (kSplit ? 2 : 4) / (sizeof(T) == 4 ? 2 : 1);   // batch: U * HS heads, 64 bytes a thread
  constexpr int V = P * sizeof(T) / 8;                 // 16-byte groups of a lane per row
  constexpr int D = 3;                                 // batches in the ring
  static_assert(U * V == 4, "64 bytes");
  __shared__ uint4 ring[D][4][256];
  grid_wait();                         // (released by its end: CTAs of the next launch between
                                       // these, waiting, left 4608 tokens 31 instead of 25 us)
  const int l = threadIdx.x & (LPR - 1), sub = (threadIdx.x & 15) / LPR;
  const int64_t token = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  const bool here = token < (int64_t)p.B * p.N;
  const int b = here ? (int)(token / p.N) : 0, n = here ? (int)(token - (int64_t)b * p.N) : 0;
  // channels of the lane's two pieces; past the rotated ones, split lanes take
  // neighbours
  const bool rotates = !kSplit || P * l < p.pairs;
  const int c0 = kSplit && rotates ? P * l : 2 * P * l;
  const int c1 = kSplit && rotates ? p.pairs + P * l : 2 * P * l + P;

  const int total = p.heads[0] + p.heads[1];
  const int h0 = blockIdx.y * p.heads_per_group, h1 = min(total, h0 + p.heads_per_group);
  // this group's batches: first those of Q, then those of K
  const int first0 = min(h0, p.heads[0]), last0 = min(h1, p.heads[0]);
  const int first1 = max(h0, p.heads[0]), last1 = max(h1, p.heads[0]);
  const int nb0 = (last0 - first0 + U * HS - 1) / (U * HS), nb = nb0 + (last1 - first1 + U * HS - 1) / (U * HS);
  auto fetch = [&](int t) {
    if (t < nb && here) {
      const int part = t < nb0 ? 0 : 1;
      const int h = part ? first1 + (t - nb0) * U * HS : first0 + t * U * HS, last = part ? last1 : last0;
      const T* in = static_cast<const T*>(p.in[part]) + (int64_t)b * p.sb[part] + (int64_t)n * p.sn[part];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int hh = h + u * HS + sub;
        if (hh >= last) break;
        const T* row = in + (int64_t)(hh - (part ? p.heads[0] : 0)) * p.sh[part];
        uint4* to = &ring[t % D][u * V][threadIdx.x];
        if (p.vec[part]) {
#pragma unroll
          for (int i = 0; i < V; ++i) {                // group i: channels of the first piece, then the second
            constexpr int G = 16 / sizeof(T);
            const int c = i * G < P ? c0 + i * G : c1 + i * G - P;
            cp_async_16(smem_u32(to + i * 256), row + c);
          }
        } else {
          alignas(16) T e[2 * P];
#pragma unroll
          for (int i = 0; i < 2 * P; ++i) e[i] = row[i < P ? c0 + i : c1 + i - P];
#pragma unroll
          for (int i = 0; i < V; ++i) to[i * 256] = reinterpret_cast<const uint4*>(e)[i];
        }
      }
    }
    cp_async_commit();
  };
  fetch(0);
  fetch(1);

  float cs[P], sn[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int j = P * l + i;
    cs[i] = 1.0f;
    sn[i] = 0.0f;
    if (here && j < p.pairs) {
      const int64_t at = (int64_t)b * p.pos_sb + (int64_t)n * p.n_axes + p.axis[j];
      const double x = p.pos_f32 ? (double)static_cast<const float*>(p.pos)[at] : (double)static_cast<const int*>(p.pos)[at];
      const double turns = x * p.f[j];
      sincospif(2.0f * (float)(turns - rint(turns)), &sn[i], &cs[i]);
      sn[i] *= p.sign;
    }
  }

  float2 ca[P / 2], cb[P / 2], cc[P / 2], cd[P / 2];
  bool norm = false;
  auto coefficients = [&](int part) {
    // y0 = x0 a - x1 b, y1 = x0 c + x1 d for pairs 2i, 2i + 1 of the lane
    norm = kNorm && p.weight[part] != nullptr;
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      ca[i] = cd[i] = make_float2(cs[2 * i], cs[2 * i + 1]);
      cc[i] = make_float2(sn[2 * i], sn[2 * i + 1]);
      cb[i] = make_float2(-sn[2 * i], -sn[2 * i + 1]);
    }
    if (norm) {
      const T* wp = static_cast<const T*>(p.weight[part]);
#pragma unroll
      for (int i = 0; i < P / 2; ++i) {
        float2 w0, w1;                 // of the first and second channels of the two pairs
        if constexpr (kSplit) {
          w0 = make_float2(to_f32<T>(wp[c0 + 2 * i]), to_f32<T>(wp[c0 + 2 * i + 1]));
          w1 = make_float2(to_f32<T>(wp[c1 + 2 * i]), to_f32<T>(wp[c1 + 2 * i + 1]));
        } else {
          w0 = make_float2(to_f32<T>(wp[c0 + 4 * i]), to_f32<T>(wp[c0 + 4 * i + 2]));
          w1 = make_float2(to_f32<T>(wp[c0 + 4 * i + 1]), to_f32<T>(wp[c0 + 4 * i + 3]));
        }
        ca[i] = f2_mul(ca[i], w0);
        cc[i] = f2_mul(cc[i], w0);
        cb[i] = f2_mul(cb[i], w1);
        cd[i] = f2_mul(cd[i], w1);
      }
    }
  };

  for (int t = 0; t < nb; ++t) {
    fetch(t + 2);
    const int part = t < nb0 ? 0 : 1;
    if (t == 0 || t == nb0) coefficients(part);
    const int h = part ? first1 + (t - nb0) * U * HS : first0 + t * U * HS, last = part ? last1 : last0;
    T* out = static_cast<T*>(p.out[part]) +
             (((int64_t)b * p.heads[part] + h + sub - (part ? p.heads[0] : 0)) * p.N + n) * kHeadDim;
    cp_async_wait<2>();                // all but the two batches fetched last
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v[2 * P];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint4 g = ring[t % D][u * V + i][threadIdx.x];
        const uint32_t w[4] = {g.x, g.y, g.z, g.w};
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
      // x0 and x1 of pairs 2i, 2i + 1
      float2 x0[P / 2], x1[P / 2];
#pragma unroll
      for (int i = 0; i < P / 2; ++i) {
        x0[i] = kSplit ? make_float2(v[2 * i], v[2 * i + 1]) : make_float2(v[4 * i], v[4 * i + 2]);
        x1[i] = kSplit ? make_float2(v[P + 2 * i], v[P + 2 * i + 1]) : make_float2(v[4 * i + 1], v[4 * i + 3]);
      }
      if (norm) {
        float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < P / 2; ++i) s2 = f2_fma(x1[i], x1[i], f2_fma(x0[i], x0[i], s2));
        float ss = s2.x + s2.y;
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        const float r = rsqrtf(fmaf(ss, 1.0f / kHeadDim, p.eps));
#pragma unroll
        for (int i = 0; i < P / 2; ++i) {
          x0[i] = f2_mul(x0[i], make_float2(r, r));
          x1[i] = f2_mul(x1[i], make_float2(r, r));
        }
      }
      float y[2 * P];
#pragma unroll
      for (int i = 0; i < P / 2; ++i) {
        float2 y0 = f2_fma(x0[i], ca[i], f2_mul(x1[i], cb[i])), y1 = f2_fma(x0[i], cc[i], f2_mul(x1[i], cd[i]));
        if constexpr (!kAll) {       // a channel that does not rotate takes nothing from its neighbour
          const bool on0 = kSplit ? rotates : P * l + 2 * i < p.pairs;
          const bool on1 = kSplit ? rotates : P * l + 2 * i + 1 < p.pairs;
          y0.x = on0 ? y0.x : x0[i].x * (norm ? ca[i].x : 1.0f);
          y1.x = on0 ? y1.x : x1[i].x * (norm ? cd[i].x : 1.0f);
          y0.y = on1 ? y0.y : x0[i].y * (norm ? ca[i].y : 1.0f);
          y1.y = on1 ? y1.y : x1[i].y * (norm ? cd[i].y : 1.0f);
        }
        y[kSplit ? 2 * i : 4 * i] = y0.x;
        y[kSplit ? 2 * i + 1 : 4 * i + 2] = y0.y;
        y[kSplit ? P + 2 * i : 4 * i + 1] = y1.x;
        y[kSplit ? P + 2 * i + 1 : 4 * i + 3] = y1.y;
      }
      if (here && h + u * HS + sub < last) {
        T* dst = out + (int64_t)u * HS * p.N * kHeadDim;
        uint32_t q[4 * V];
        pack_words<T, 2 * P>(y, q);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          constexpr int G = 16 / sizeof(T);
          T* at = dst + (i * G < P ? c0 + i * G : c1 + i * G - P);
          *reinterpret_cast<uint4*>(at) = make_uint4(q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]);
        }
      }
    }
  }
}

}  // namespace fqa
