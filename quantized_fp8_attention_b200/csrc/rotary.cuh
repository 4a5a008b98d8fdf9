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

// A lane's channels of a row, two pieces of P, as they lie in memory.
template <typename T, int P>
struct RotRaw {
  static constexpr int kWords = P * sizeof(T) / 4;      // of a piece
  uint32_t w[2 * kWords];
  __device__ __forceinline__ void piece(const T* p, int at) {
    if constexpr (kWords % 4 == 0) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 a = *reinterpret_cast<const uint4*>(p + i * 4 / sizeof(T));
        w[at + i] = a.x; w[at + i + 1] = a.y; w[at + i + 2] = a.z; w[at + i + 3] = a.w;
      }
    } else {
      static_assert(kWords == 2, "8 or 16 bytes");
      const uint2 a = *reinterpret_cast<const uint2*>(p);
      w[at] = a.x; w[at + 1] = a.y;
    }
  }
  // kJoined: the pieces are neighbours
  template <bool kJoined>
  __device__ __forceinline__ void load(const T* row, int c0, int c1, bool vec) {
    if (vec) {
      if constexpr (kJoined && kWords == 2) {
        const uint4 a = *reinterpret_cast<const uint4*>(row + c0);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
      } else {
        piece(row + c0, 0);
        piece(row + c1, kWords);
      }
    } else {
      T e[2 * P];
#pragma unroll
      for (int i = 0; i < 2 * P; ++i) e[i] = row[i < P ? c0 + i : c1 + i - P];
#pragma unroll
      for (int i = 0; i < 2 * kWords; ++i) w[i] = reinterpret_cast<const uint32_t*>(e)[i];
    }
  }
  __device__ __forceinline__ void get(float (&v)[2 * P]) const {
#pragma unroll
    for (int i = 0; i < 2 * kWords; ++i) {
      if constexpr (sizeof(T) == 4) {
        v[i] = __uint_as_float(w[i]);
      } else {
        const float2 f = unpack2<T>(w[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
};

// kSplit: pair j is channels (j, pairs + j); otherwise (2j, 2j + 1).  Pairs
// never cross lanes: interleaved a lane of 16 holds eight neighbours (four
// pairs); split a lane of 8 holds eight channels and their eight partners, and
// the 16 lanes take two heads at a time.  Every access is 16 bytes a lane (16
// lanes with 4 + 4 channels, 8 bytes an access, ran at 3.9 instead of 5.8
// TB/s).  Rows are fetched one batch ahead: the first while the angles are
// formed, the next while one is rotated.
// kNorm: a weight is given for Q or K.  The weight goes into the coefficients
// of the rotation, so a row costs its sum of squares, one factor and the
// rotation; two pairs share each packed instruction.  (Unpacked, with weights
// applied per row, the kernel was bound by its 193 instructions per row and
// warp.)  kAll: all 64 pairs rotate.
template <typename T, bool kSplit, bool kNorm, bool kAll>
__global__ void __launch_bounds__(256, sizeof(T) == 4 || (kSplit && kNorm) ? 2 : 3) rotary_kernel(const __grid_constant__ RotaryParams p) {
  constexpr int LPR = kSplit ? 8 : 16;                 // lanes per row
  constexpr int P = kSplit ? 8 : 4;                    // channels per piece = pairs per lane
  constexpr int HS = 16 / LPR;                         // heads at a time
  constexpr int U = (kSplit ? 2 : 4) / (sizeof(T) == 4 ? 2 : 1);   // batch: U * HS heads
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
  RotRaw<T, P> cur[U];
  // rows h + sub, h + HS + sub, .. (below `last`) of Q or K
  auto fetch = [&](int part, int h, int last, RotRaw<T, P> (&raw)[U]) {
    const T* in = static_cast<const T*>(p.in[part]) + (int64_t)b * p.sb[part] + (int64_t)n * p.sn[part];
    const int base = part ? p.heads[0] : 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int hh = h + u * HS + sub;
      if (here && hh < last)
        raw[u].template load<!kSplit>(in + (int64_t)(hh - base) * p.sh[part], c0, c1, p.vec[part]);
    }
  };
  const int part0 = h0 < p.heads[0] ? 0 : 1;
  const int last0 = part0 ? h1 : min(h1, p.heads[0]);
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < RotRaw<T, P>::kWords * 2; ++i) cur[u].w[i] = 0u;
  fetch(part0, h0, last0, cur);

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

  for (int part = part0; part < 2; ++part) {
    const int base = part ? p.heads[0] : 0;
    const int first = max(h0, base), last = min(h1, base + p.heads[part]);
    if (first >= last) continue;
    if (part != part0) fetch(part, first, last, cur);
    // y0 = x0 a - x1 b, y1 = x0 c + x1 d for pairs 2i, 2i + 1 of the lane
    float2 ca[P / 2], cb[P / 2], cc[P / 2], cd[P / 2];
    const bool norm = kNorm && p.weight[part] != nullptr;
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
    T* out = static_cast<T*>(p.out[part]) + ((int64_t)b * p.heads[part] * p.N + n) * kHeadDim;
    for (int h = first; h < last; h += U * HS) {
      RotRaw<T, P> next[U];
#pragma unroll
      for (int u = 0; u < U; ++u) next[u] = cur[u];
      if (h + U * HS < last) fetch(part, h + U * HS, last, next);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int hh = h + u * HS + sub;
        float v[2 * P];
        cur[u].get(v);
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
        if (here && hh < last) {
          T* dst = out + (int64_t)(hh - base) * p.N * kHeadDim;
          uint32_t q[RotRaw<T, P>::kWords * 2];
          pack_words<T, 2 * P>(y, q);
          constexpr int W = RotRaw<T, P>::kWords;
#pragma unroll
          for (int i = 0; i < 2 * W; i += 4) {         // (a 16-byte store may span two neighbouring pieces)
            T* at = dst + (i < W ? c0 : c1 - P) + i * 4 / (int)sizeof(T);
            *reinterpret_cast<uint4*>(at) = make_uint4(q[i], q[i + 1], q[i + 2], q[i + 3]);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) cur[u] = next[u];
    }
  }
}

}  // namespace fqa
