// One head's row in registers: norm, rotation and their gradients.
//
// A row belongs to T neighbouring lanes of a warp, and a lane holds two pieces
// of four elements, a and b, chosen so that no rotated pair crosses lanes:
//   pairs (i, i + h), h = rot / 2: lane t < ceil(h / 4) holds a = 4 t .. and
//       b = h + 4 t .., the two halves of four pairs; the lanes after them
//       hold 8 elements past rot each;
//   pairs (2 i, 2 i + 1): lane t holds 8 t .. 8 t + 7.
// Either way lane t turns by the angles 4 t .. 4 t + 3.  With 8 | D, 8 | rot
// and aligned rows (kVec) a piece is one access of 8 bytes in bf16 and 16 in
// fp32, and T is 8 for D <= 64 and 16 for D <= 128; other rows are read one
// element at a time by a whole warp (T = 32).
// Shuffles are left to the norm's sum.  (With 8 neighbouring elements a lane
// and the partner fetched by shuffles, a row took 2.5 times the instructions:
// 255 us against 165 us for 32 + 8 heads of 128 over 32768 tokens.)
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "common.cuh"
#include "fastmath.cuh"
#include "launch.h"

namespace fa {

// Where a lane's pieces lie.
struct Place {
  int a, b;    // first elements
  int na, nb;  // elements held, 0..4 (0 or 4 with 16-byte rows)
  int pairs;   // kHalf: pairs that turn; 0: both pieces pass through
};
template <bool kNext>
__device__ __forceinline__ Place place_of(int t, int rot, int D) {
  Place p;
  const int h = rot >> 1, turning = (h + 3) >> 2;
  if (kNext || t >= turning) {
    const int first = kNext ? 8 * t : rot + 8 * (t - turning);
    p.a = first;
    p.b = first + 4;
    p.na = min(max(D - p.a, 0), 4);
    p.nb = min(max(D - p.b, 0), 4);
    p.pairs = 0;
  } else {
    p.a = 4 * t;
    p.b = h + 4 * t;
    p.na = p.nb = p.pairs = min(h - 4 * t, 4);
  }
  return p;
}

// Two pieces as loaded.  Loading and unpacking are apart so that a lane can
// have the loads of several rows in flight.
template <bool kVec, bool kF32>
struct Raw {
  uint32_t u[(kVec && !kF32) ? 4 : 8];
};
template <bool kVec, bool kF32>
__device__ __forceinline__ void clear_raw(Raw<kVec, kF32>& r) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(r.u) / 4); ++i) r.u[i] = 0u;
}
template <bool kVec, bool kF32>
__device__ __forceinline__ void load_raw(const void* row, const Place& p, Raw<kVec, kF32>& r) {
  clear_raw(r);
  if constexpr (!kVec) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = i < 4 ? p.a + i : p.b + i - 4;
      if ((i & 3) < (i < 4 ? p.na : p.nb))
        r.u[i] = kF32 ? __float_as_uint(static_cast<const float*>(row)[e])
                      : static_cast<uint32_t>(static_cast<const uint16_t*>(row)[e]) << 16;
    }
  } else if constexpr (kF32) {
    if (p.na) {
      const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const float*>(row) + p.a);
      const uint4 b = *reinterpret_cast<const uint4*>(static_cast<const float*>(row) + p.b);
      r.u[0] = a.x; r.u[1] = a.y; r.u[2] = a.z; r.u[3] = a.w;
      r.u[4] = b.x; r.u[5] = b.y; r.u[6] = b.z; r.u[7] = b.w;
    }
  } else {
    if (p.na) {
      const uint2 a = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(row) + p.a);
      const uint2 b = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(row) + p.b);
      r.u[0] = a.x; r.u[1] = a.y; r.u[2] = b.x; r.u[3] = b.y;
    }
  }
}

// The same through shared memory: a lane copies its own two pieces into its own
// slot (16 bytes of bf16 or 32 of fp32) and reads them back itself, so the
// only wait is for its own copies, and rows in flight cost no registers.
template <bool kF32>
__device__ __forceinline__ void copy_raw(uint32_t slot, const void* row, const Place& p, bool valid) {
  constexpr int kPiece = kF32 ? 16 : 8;
  const int bytes = valid && p.na ? kPiece : 0;  // 0: the slot is filled with zeros
  const char* src = static_cast<const char*>(row);
  const char *a = bytes ? src + p.a * (kPiece / 4) : src, *b = bytes ? src + p.b * (kPiece / 4) : src;
  if constexpr (kF32) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(slot), "l"(a), "r"(bytes) : "memory");
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(slot + 16), "l"(b), "r"(bytes) : "memory");
  } else {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(slot), "l"(a), "r"(bytes) : "memory");
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(slot + 8), "l"(b), "r"(bytes) : "memory");
  }
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}
template <bool kF32>
__device__ __forceinline__ void read_raw(uint32_t slot, Raw<true, kF32>& r) {
#pragma unroll
  for (int w = 0; w < (kF32 ? 2 : 1); ++w)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.u[4 * w]), "=r"(r.u[4 * w + 1]), "=r"(r.u[4 * w + 2]), "=r"(r.u[4 * w + 3])
                 : "r"(slot + 16 * w)
                 : "memory");
}

// The pieces as pairs of fp32: a = v[0], v[1], b = v[2], v[3].
struct Row {
  float2 v[4];
};
template <bool kVec, bool kF32>
__device__ __forceinline__ Row unpack(const Raw<kVec, kF32>& r) {
  Row x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kVec && !kF32)
      x.v[i] = make_float2(__uint_as_float(r.u[i] << 16), __uint_as_float(r.u[i] & 0xffff0000u));
    else
      x.v[i] = make_float2(__uint_as_float(r.u[2 * i]), __uint_as_float(r.u[2 * i + 1]));
  }
  return x;
}

template <bool kVec>
__device__ __forceinline__ void store_row(void* row, int f32, const Place& p, const Row& x) {
  if constexpr (kVec) {
    if (p.na == 0) return;
    if (f32) {
      *reinterpret_cast<float4*>(static_cast<float*>(row) + p.a) = make_float4(x.v[0].x, x.v[0].y, x.v[1].x, x.v[1].y);
      *reinterpret_cast<float4*>(static_cast<float*>(row) + p.b) = make_float4(x.v[2].x, x.v[2].y, x.v[3].x, x.v[3].y);
    } else {
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(row) + p.a) =
          make_uint2(pack_bf16x2(x.v[0].x, x.v[0].y), pack_bf16x2(x.v[1].x, x.v[1].y));
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(row) + p.b) =
          make_uint2(pack_bf16x2(x.v[2].x, x.v[2].y), pack_bf16x2(x.v[3].x, x.v[3].y));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = i < 4 ? p.a + i : p.b + i - 4;
      const float v = (i & 1) ? x.v[i >> 1].y : x.v[i >> 1].x;
      if ((i & 3) < (i < 4 ? p.na : p.nb)) {
        if (f32)
          static_cast<float*>(row)[e] = v;
        else
          static_cast<__nv_bfloat16*>(row)[e] = __float2bfloat16_rn(v);
      }
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
__device__ __forceinline__ float dot8(const Row& x, const Row& y) {
  float2 s = mul2(x.v[0], y.v[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = fma2(x.v[i], y.v[i], s);
  return s.x + s.y;
}
// r = (mean(x^2) + eps)^(-1/2) of a row.
template <int T>
__device__ __forceinline__ float norm_factor(const Row& x, float eps, float inv_d) {
  return rsqrtf(row_sum<T>(dot8(x, x)) * inv_d + eps);
}
__device__ __forceinline__ Row scaled(const Row& x, float f) {
  Row y;
#pragma unroll
  for (int i = 0; i < 4; ++i) y.v[i] = mul2(x.v[i], splat2(f));
  return y;
}
__device__ __forceinline__ Row product(const Row& x, const Row& y) {
  Row z;
#pragma unroll
  for (int i = 0; i < 4; ++i) z.v[i] = mul2(x.v[i], y.v[i]);
  return z;
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

// A linear map of a lane's pieces:
//   kHalf: a' = a c_0,1 + b s_0,1,   b' = b c_2,3 + a s_2,3
//   kNext: v' = v c + swapped(v) s for each pair
// which a rotation, its inverse and either with the norm's weights folded in
// all are.
struct Turn {
  float2 c[4], s[4];
};
template <bool kNext>
__device__ __forceinline__ Row apply(const Row& x, const Turn& f, const Place& p, int rot, int D) {
  Row y;
  if constexpr (kNext) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y.v[i] = fma2(make_float2(x.v[i].y, x.v[i].x), f.s[i], mul2(x.v[i], f.c[i]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) y.v[i] = fma2(x.v[i ^ 2], f.s[i], mul2(x.v[i], f.c[i]));
  }
  // What passes through does so alone: 0 times its partner would turn an
  // infinity there into NaN.
  if (rot < D) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool turns = kNext ? p.a + i < rot : (i & 3) < p.pairs;
      if (turns) continue;
      if (i & 1)
        y.v[i >> 1].y = x.v[i >> 1].y * f.c[i >> 1].y;
      else
        y.v[i >> 1].x = x.v[i >> 1].x * f.c[i >> 1].x;
    }
  }
  return y;
}

// The rotation by a token's angles (tables of rot / 2 cosines and sines in
// shared memory, 16-byte aligned where 8 | rot); sign -1 turns back.
template <bool kNext>
__device__ __forceinline__ Turn rotation(const float* cos_t, const float* sin_t, int t, const Place& p, int rot,
                                         float sign) {
  float c[4], s[4];
  const int h = rot >> 1;
  if ((rot & 7) == 0) {
    float4 cv = make_float4(1.0f, 1.0f, 1.0f, 1.0f), sv = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (4 * t < h) {
      cv = *reinterpret_cast<const float4*>(cos_t + 4 * t);
      sv = *reinterpret_cast<const float4*>(sin_t + 4 * t);
    }
    c[0] = cv.x; c[1] = cv.y; c[2] = cv.z; c[3] = cv.w;
    s[0] = sv.x; s[1] = sv.y; s[2] = sv.z; s[3] = sv.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = 4 * t + i < h;
      c[i] = in ? cos_t[4 * t + i] : 1.0f;
      s[i] = in ? sin_t[4 * t + i] : 0.0f;
    }
  }
  Turn f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kNext) {
      f.c[i] = make_float2(c[i], c[i]);
      f.s[i] = make_float2(-sign * s[i], sign * s[i]);
    } else {
      const int k = 2 * (i & 1);
      f.c[i] = make_float2(c[k], c[k + 1]);
      const float sg = i < 2 ? -sign : sign;
      f.s[i] = make_float2(sg * s[k], sg * s[k + 1]);
    }
  }
  return f;
}
__device__ __forceinline__ Turn identity() {
  Turn f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f.c[i] = make_float2(1.0f, 1.0f);
    f.s[i] = make_float2(0.0f, 0.0f);
  }
  return f;
}
// The map that weighs by w first.
template <bool kNext>
__device__ __forceinline__ void fold(Turn& f, const Row& w) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f.c[i] = mul2(f.c[i], w.v[i]);
    f.s[i] = mul2(f.s[i], kNext ? make_float2(w.v[i].y, w.v[i].x) : w.v[i ^ 2]);
  }
}

// A norm's weights as fp32 in shared memory (1 without weights; `pad` floats,
// 0 past D), and a lane's share of them.
__device__ __forceinline__ void stage_weight(const NormArgs& n, int D, int pad, float* w) {
  for (int e = threadIdx.x; e < pad; e += blockDim.x)
    w[e] = e >= D                ? 0.0f
           : n.weight == nullptr ? 1.0f
           : n.weight_f32        ? __ldg(static_cast<const float*>(n.weight) + e)
                                 : __bfloat162float(static_cast<const __nv_bfloat16*>(n.weight)[e]);
}
template <bool kVec>
__device__ __forceinline__ Row lane_weight(const float* w, const Place& p) {
  Row r;
  if constexpr (kVec) {  // pieces are whole and start on multiples of 4
    const float4 a = p.na ? *reinterpret_cast<const float4*>(w + p.a) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float4 b = p.nb ? *reinterpret_cast<const float4*>(w + p.b) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    r.v[0] = make_float2(a.x, a.y);
    r.v[1] = make_float2(a.z, a.w);
    r.v[2] = make_float2(b.x, b.y);
    r.v[3] = make_float2(b.z, b.w);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = (i & 3) < (i < 4 ? p.na : p.nb) ? w[i < 4 ? p.a + i : p.b + i - 4] : 0.0f;
      if (i & 1)
        r.v[i >> 1].y = v;
      else
        r.v[i >> 1].x = v;
    }
  }
  return r;
}

}  // namespace fa
