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
// row is one 256-byte segment on both sides whatever the layout.
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

// A lane's two pieces of four channels of a row, as they lie in memory.
template <typename T>
struct RotRaw {
  uint32_t w[2 * sizeof(T)];
  template <bool kSplit>
  __device__ __forceinline__ void load(const T* row, int c0, int c1, bool here) {
#pragma unroll
    for (int i = 0; i < 2 * (int)sizeof(T); ++i) w[i] = 0u;
    if (!here) return;
    if constexpr (sizeof(T) == 4) {
      const uint4 a = *reinterpret_cast<const uint4*>(row + c0), b = *reinterpret_cast<const uint4*>(row + c1);
      w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
      w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    } else if constexpr (kSplit) {
      const uint2 a = *reinterpret_cast<const uint2*>(row + c0), b = *reinterpret_cast<const uint2*>(row + c1);
      w[0] = a.x; w[1] = a.y; w[2] = b.x; w[3] = b.y;
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(row + c0);
      w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    }
  }
  __device__ __forceinline__ void load_elements(const T* row, int c0, int c1, bool here) {
    T e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = here ? row[(i < 4 ? c0 : c1 - 4) + i] : from_f32<T>(0.0f);
#pragma unroll
    for (int i = 0; i < 2 * (int)sizeof(T); ++i) w[i] = reinterpret_cast<const uint32_t*>(e)[i];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<T>(w[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
};

// kSplit: pair j is channels (j, pairs + j); otherwise (2j, 2j + 1).  Lane l
// holds two pieces of four channels: interleaved the neighbours [8l, 8l + 8),
// split [4l, 4l + 4) and the four partners at pairs + 4l, so that a pair
// never crosses lanes and each lane forms four angles.
template <typename T, bool kSplit>
__global__ void __launch_bounds__(256, 4) rotary_kernel(const __grid_constant__ RotaryParams p) {
  const int l = threadIdx.x & 15;
  const int64_t token = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  const bool here = token < (int64_t)p.B * p.N;
  const int b = here ? (int)(token / p.N) : 0, n = here ? (int)(token - (int64_t)b * p.N) : 0;
  // channels of the lane's two pieces; past the rotated ones, split lanes take
  // eight plain channels
  const bool rotates = !kSplit || 4 * l < p.pairs;
  const int c0 = kSplit && rotates ? 4 * l : 8 * l;
  const int c1 = kSplit && rotates ? p.pairs + 4 * l : 8 * l + 4;

  float cs[4], sn[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = 4 * l + i;
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

  const int total = p.heads[0] + p.heads[1];
  const int h0 = blockIdx.y * p.heads_per_group, h1 = min(total, h0 + p.heads_per_group);
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const int base = part ? p.heads[0] : 0;
    const int first = max(h0, base), last = min(h1, base + p.heads[part]);
    if (first >= last) continue;
    float w[8];
    const bool norm = p.weight[part] != nullptr;
    if (norm) {
      const T* wp = static_cast<const T*>(p.weight[part]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[e] = to_f32<T>(wp[c0 + e]);
        w[4 + e] = to_f32<T>(wp[c1 + e]);
      }
    }
    const T* in = static_cast<const T*>(p.in[part]) + (int64_t)b * p.sb[part] + (int64_t)n * p.sn[part];
    T* out = static_cast<T*>(p.out[part]) + ((int64_t)b * p.heads[part] * p.N + n) * kHeadDim;
    const bool vec = p.vec[part];
    auto rows = [&](auto count, int h) {
      constexpr int U = decltype(count)::value;
      // all loads first, kept as they lie in memory until used
      RotRaw<T> raw[U];
      if (vec) {
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u].template load<kSplit>(in + (int64_t)(h + u - base) * p.sh[part], c0, c1, here);
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u].load_elements(in + (int64_t)(h + u - base) * p.sh[part], c0, c1, here);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float v[8];
        raw[u].get(v);
        if (norm) {
          float ss = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss += v[e] * v[e];
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
          const float r = rsqrtf(ss * (1.0f / kHeadDim) + p.eps);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = v[e] * r * w[e];
        }
        float y[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int a = kSplit ? i : 2 * i, d = kSplit ? 4 + i : 2 * i + 1;
          const bool on = kSplit ? rotates : 4 * l + i < p.pairs;
          y[a] = on ? v[a] * cs[i] - v[d] * sn[i] : v[a];
          y[d] = on ? v[a] * sn[i] + v[d] * cs[i] : v[d];
        }
        if (here) {
          T* dst = out + (int64_t)(h + u - base) * p.N * kHeadDim;
          if constexpr (!kSplit) {
            store_vec<T, 8>(dst + c0, y);
          } else {
            store_vec<T, 4>(dst + c0, {y[0], y[1], y[2], y[3]});
            store_vec<T, 4>(dst + c1, {y[4], y[5], y[6], y[7]});
          }
        }
      }
    };
    int h = first;
    for (; h + 4 <= last; h += 4) rows(std::integral_constant<int, 4>{}, h);
    for (; h < last; ++h) rows(std::integral_constant<int, 1>{}, h);
  }
}

}  // namespace fqa
