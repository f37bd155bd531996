// One head's row in registers: norm, rotation and their gradients.
//
// A row of D <= 8 T elements belongs to T neighbouring lanes of a warp (T = 8
// for D <= 64, 16 for D <= 128); lane t holds elements 8 t .. 8 t + 7, one
// 16-byte access in bf16.  The rotation is written as
//   y_i = x_i c_i + p_i s_i,
// p_i the element paired with i and the sign of the sine folded into s_i, so
// that both pairings, their inverses (s -> -s) and pass-through elements
// (c = 1, s = 0) are one formula; only the fetch of p differs.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "common.cuh"
#include "launch.h"

namespace fa {

// How the paired element is fetched.
enum class Pair {
  kHalf,     // (i, i + h) with h = rot / 2 a multiple of 8: whole lanes trade
  kHalfAny,  // (i, i + h) with any h: lanes and places differ
  kNext      // (2 i, 2 i + 1): within the lane
};

// 8 elements of a row at element e0 (kVec: 16-byte accesses, 8 | D; else one
// element at a time).  Elements past D are 0 and not stored.
template <bool kVec>
__device__ __forceinline__ void load8(const void* row, int f32, int e0, int D, float (&x)[8]) {
  if constexpr (kVec) {
    if (e0 < D) {
      if (f32) {
        const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(row) + e0);
        const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(row) + e0 + 4);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
      } else {
        const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(row) + e0);
        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[2 * i] = __uint_as_float(u[i] << 16);
          x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.0f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = e0 + i >= D ? 0.0f
             : f32       ? static_cast<const float*>(row)[e0 + i]
                         : __bfloat162float(static_cast<const __nv_bfloat16*>(row)[e0 + i]);
  }
}

template <bool kVec>
__device__ __forceinline__ void store8(void* row, int f32, int e0, int D, const float (&x)[8]) {
  if constexpr (kVec) {
    if (e0 < D) {
      if (f32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(row) + e0);
        o[0] = make_float4(x[0], x[1], x[2], x[3]);
        o[1] = make_float4(x[4], x[5], x[6], x[7]);
      } else {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(row) + e0) =
            make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                       pack_bf16x2(x[6], x[7]));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e0 + i < D) {
        if (f32)
          static_cast<float*>(row)[e0 + i] = x[i];
        else
          static_cast<__nv_bfloat16*>(row)[e0 + i] = __float2bfloat16_rn(x[i]);
      }
  }
}

__device__ __forceinline__ const void* row_ptr(const void* base, int f32, int64_t off) {
  return static_cast<const char*>(base) + off * (f32 ? 4 : 2);
}
__device__ __forceinline__ void* row_ptr(void* base, int f32, int64_t off) {
  return static_cast<char*>(base) + off * (f32 ? 4 : 2);
}

// Sum over the T lanes of a row; every lane of the row gets it.
template <int T>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = T / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// cos and sin of pos * inv_freq.  The angle is taken in turns and reduced in
// fp64 (pos is up to 2^31 and inv_freq a full fp32 value: in fp32 the angle of
// a position past 10^5 would be off by a hundredth of a radian), so only the
// remaining fraction of a turn is rounded to fp32, by 2^-25 turns at most.
__device__ __forceinline__ void angle(int pos, float inv_freq, float* c, float* s) {
  constexpr double kTurnsPerRadian = 0.15915494309189533577;
  const double turns = static_cast<double>(pos) * (static_cast<double>(inv_freq) * kTurnsPerRadian);
  const float f = static_cast<float>(turns - rint(turns));
  sincospif(2.0f * f, s, c);
}

// This lane's (c_i, s_i) of one token from its table of rot / 2 cosines and
// sines (shared memory).
template <Pair kPair>
__device__ __forceinline__ void lane_angles(const float* cos_t, const float* sin_t, int e0, int rot, float (&c)[8],
                                            float (&s)[8]) {
  const int h = rot >> 1;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = e0 + i;
    c[i] = 1.0f;
    s[i] = 0.0f;
    if (e < rot) {
      const int f = kPair == Pair::kNext ? e >> 1 : (e < h ? e : e - h);
      const bool first = kPair == Pair::kNext ? (i & 1) == 0 : e < h;
      c[i] = cos_t[f];
      s[i] = first ? -sin_t[f] : sin_t[f];
    }
  }
}

// x[(i + k) & 7] for a k that all lanes share.
__device__ __forceinline__ void turn8(float (&x)[8], int k) {
#pragma unroll
  for (int b = 1; b < 8; b <<= 1) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = (k & b) ? x[(i + b) & 7] : x[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = y[i];
  }
}

// y_i = x_i c_i + sgn * p_i s_i (sgn -1 turns back).  Called by all lanes of
// a warp; t is the lane's place in its row of T lanes.
template <int T, Pair kPair>
__device__ __forceinline__ void rotate8(const float (&x)[8], const float (&c)[8], const float (&s)[8], float sgn, int t,
                                        int rot, float (&y)[8]) {
  float p[8];
  const int h = rot >> 1;
  if constexpr (kPair == Pair::kNext) {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = x[i ^ 1];
  } else if constexpr (kPair == Pair::kHalf) {
    const int e0 = 8 * t;
    const int src = e0 < h ? t + (h >> 3) : (e0 < rot ? t - (h >> 3) : t);
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = __shfl_sync(0xffffffffu, x[i], src, T);
  } else {
    // element i of the lane is paired with element 8 t + i +- h of the row:
    // place (i +- h) & 7, the same for all lanes, of a lane of its own
    float up[8], dn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) up[i] = dn[i] = x[i];
    turn8(up, h & 7);
    turn8(dn, (8 - (h & 7)) & 7);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = 8 * t + i;
      const float a = __shfl_sync(0xffffffffu, up[i], min((e + h) >> 3, T - 1), T);
      const float b = __shfl_sync(0xffffffffu, dn[i], max(e - h, 0) >> 3, T);
      p[i] = e < h ? a : b;
    }
  }
  // elements past rot pass through as they are (0 * p would turn an infinity into NaN)
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = 8 * t + i < rot ? fmaf(p[i], sgn * s[i], x[i] * c[i]) : x[i];
}

// A norm's weights of this lane (1 without weights, 0 past D).
__device__ __forceinline__ void load_weight8(const NormArgs& n, int e0, int D, float (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = e0 + i;
    w[i] = e >= D                ? 0.0f
           : n.weight == nullptr ? 1.0f
           : n.weight_f32        ? __ldg(static_cast<const float*>(n.weight) + e)
                                 : __bfloat162float(static_cast<const __nv_bfloat16*>(n.weight)[e]);
  }
}

// x <- x r w, r = (mean(x^2) + eps)^(-1/2).
template <int T>
__device__ __forceinline__ void norm8(float (&x)[8], const float (&w)[8], float eps, float inv_d) {
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
  const float r = rsqrtf(row_sum<T>(ss) * inv_d + eps);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
}

}  // namespace fa
