// One head's row in registers: norm, rotation and their gradients.
//
// A row belongs to T neighbouring lanes of a warp, and a lane holds two pieces
// of P elements, a and b, chosen so that no rotated pair crosses lanes:
//   pairs (i, i + h), h = rot / 2: lane t < ceil(h / P) holds a = P t .. and
//       b = h + P t .., the two halves of P pairs; the lanes after them hold
//       2 P elements past rot each;
//   pairs (2 i, 2 i + 1): lane t holds 2 P t .. 2 P t + 2 P - 1.
// Either way lane t turns by the angles P t .. P t + P - 1.  Rows on 16-byte
// boundaries with 8 | D take whole pieces (kVec; halves need 2 P | rot): for
// D <= 64, P = 4 and T = 8; above, P = 4 and T = 16, or P = 8 and T = 8 (the
// cache append, which holds rows in registers anyway and gains from fewer
// lanes a row: 61 -> 49 us for 8 prompts of 2048 tokens; the preparation does
// not: 122 -> 124 us forward, 203 -> 197 us backward, and 10 -> 15 us for a
// short batch).  Other rows are read one element at a time by a whole warp
// (P = 4, T = 32).
// What a row costs beside its arithmetic decides, so shuffles are left to the
// norm's sum: with 8 neighbouring elements a lane and the partner fetched by
// shuffles, the forward pass of 32768 tokens took 255 us against 165 us.
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
  int na, nb;  // elements held, 0..P (0 or P with whole pieces)
  int pairs;   // halves: pairs that turn; 0: both pieces pass through
};
template <int P, bool kNext>
__device__ __forceinline__ Place place_of(int t, int rot, int D) {
  Place p;
  const int h = rot >> 1, turning = (h + P - 1) / P;
  if (kNext || t >= turning) {
    const int first = kNext ? 2 * P * t : rot + 2 * P * (t - turning);
    p.a = first;
    p.b = first + P;
    p.na = min(max(D - p.a, 0), P);
    p.nb = min(max(D - p.b, 0), P);
    p.pairs = 0;
  } else {
    p.a = P * t;
    p.b = h + P * t;
    p.na = p.nb = p.pairs = min(h - P * t, P);
  }
  return p;
}
// Element i of the lane's 2 P: its place in the row, and whether the lane has it.
template <int P>
__device__ __forceinline__ int element(const Place& p, int i) {
  return i < P ? p.a + i : p.b + i - P;
}
template <int P>
__device__ __forceinline__ bool has(const Place& p, int i) {
  return i < P ? i < p.na : i - P < p.nb;
}

// Two pieces as loaded.  Loading and unpacking are apart so that a lane can
// have the loads of several rows in flight.
template <int P, bool kVec, bool kF32>
struct Raw {
  static constexpr int kWords = (kVec && !kF32) ? P : 2 * P;
  uint32_t u[kWords];
};
template <int P, bool kVec, bool kF32>
__device__ __forceinline__ void clear_raw(Raw<P, kVec, kF32>& r) {
#pragma unroll
  for (int i = 0; i < r.kWords; ++i) r.u[i] = 0u;
}
template <int P, bool kVec, bool kF32>
__device__ __forceinline__ void load_raw(const void* row, const Place& p, Raw<P, kVec, kF32>& r) {
  clear_raw(r);
  if constexpr (!kVec) {
#pragma unroll
    for (int i = 0; i < 2 * P; ++i) {
      const int e = element<P>(p, i);
      if (has<P>(p, i))
        r.u[i] = kF32 ? __float_as_uint(static_cast<const float*>(row)[e])
                      : static_cast<uint32_t>(static_cast<const uint16_t*>(row)[e]) << 16;
    }
  } else {
    constexpr int kEl = kF32 ? 4 : 2, kHalf = r.kWords / 2;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const char* src = static_cast<const char*>(row) + (q ? p.b : p.a) * kEl;
      if (!(q ? p.nb : p.na)) continue;
      if constexpr (kHalf == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(src);
        r.u[2 * q] = v.x;
        r.u[2 * q + 1] = v.y;
      } else {
#pragma unroll
        for (int w = 0; w < kHalf / 4; ++w) {
          const uint4 v = reinterpret_cast<const uint4*>(src)[w];
          uint32_t* d = r.u + q * kHalf + 4 * w;
          d[0] = v.x; d[1] = v.y; d[2] = v.z; d[3] = v.w;
        }
      }
    }
  }
}

// The same through shared memory: a lane copies its own two pieces into its own
// slots, 16-byte words `kThreads` slots apart, and reads them back itself, so
// the only wait is for its own copies, and rows in flight cost no registers.
template <int P, bool kF32, int kThreads>
__device__ __forceinline__ void copy_raw(uint32_t slot, const char* a, const char* b, const Place& p, bool valid) {
  constexpr int kPiece = P * (kF32 ? 4 : 2);
  // size 0: nothing is read and the slot is filled with zeros
  const int na = valid && p.na ? (kPiece < 16 ? 8 : 16) : 0, nb = valid && p.nb ? (kPiece < 16 ? 8 : 16) : 0;
  if constexpr (kPiece == 8) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(slot), "l"(a), "r"(na) : "memory");
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(slot + 8), "l"(b), "r"(nb) : "memory");
  } else {
#pragma unroll
    for (int w = 0; w < kPiece / 16; ++w) {
      const uint32_t da = slot + w * kThreads * 16, db = slot + (kPiece / 16 + w) * kThreads * 16;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(da), "l"(a + 16 * w), "r"(na) : "memory");
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(db), "l"(b + 16 * w), "r"(nb) : "memory");
    }
  }
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}
template <int P, bool kF32, int kThreads>
__device__ __forceinline__ void read_raw(uint32_t slot, Raw<P, true, kF32>& r) {
#pragma unroll
  for (int w = 0; w < r.kWords / 4; ++w)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.u[4 * w]), "=r"(r.u[4 * w + 1]), "=r"(r.u[4 * w + 2]), "=r"(r.u[4 * w + 3])
                 : "r"(slot + w * kThreads * 16)
                 : "memory");
}

// The pieces as pairs of fp32: a, then b.
template <int P>
struct Row {
  float2 v[P];
};
template <int P, bool kVec, bool kF32>
__device__ __forceinline__ Row<P> unpack(const Raw<P, kVec, kF32>& r) {
  Row<P> x;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if constexpr (kVec && !kF32)
      x.v[i] = make_float2(__uint_as_float(r.u[i] << 16), __uint_as_float(r.u[i] & 0xffff0000u));
    else
      x.v[i] = make_float2(__uint_as_float(r.u[2 * i]), __uint_as_float(r.u[2 * i + 1]));
  }
  return x;
}
template <int P>
__device__ __forceinline__ float at(const Row<P>& x, int i) {
  return (i & 1) ? x.v[i >> 1].y : x.v[i >> 1].x;
}
template <int P>
__device__ __forceinline__ void put(Row<P>& x, int i, float v) {
  if (i & 1)
    x.v[i >> 1].y = v;
  else
    x.v[i >> 1].x = v;
}

template <bool kVec, int P>
__device__ __forceinline__ void store_row(void* row, int f32, const Place& p, const Row<P>& x) {
  if constexpr (kVec) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (!(q ? p.nb : p.na)) continue;
      const float2* v = x.v + q * (P / 2);
      const int e = q ? p.b : p.a;
      if (f32) {
#pragma unroll
        for (int w = 0; w < P / 4; ++w)
          *reinterpret_cast<float4*>(static_cast<float*>(row) + e + 4 * w) =
              make_float4(v[2 * w].x, v[2 * w].y, v[2 * w + 1].x, v[2 * w + 1].y);
      } else if constexpr (P == 8) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(row) + e) =
            make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y), pack_bf16x2(v[2].x, v[2].y),
                       pack_bf16x2(v[3].x, v[3].y));
      } else {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(row) + e) =
            make_uint2(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2 * P; ++i)
      if (has<P>(p, i)) {
        if (f32)
          static_cast<float*>(row)[element<P>(p, i)] = at(x, i);
        else
          static_cast<__nv_bfloat16*>(row)[element<P>(p, i)] = __float2bfloat16_rn(at(x, i));
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
template <int P>
__device__ __forceinline__ float dot(const Row<P>& x, const Row<P>& y) {
  float2 s = mul2(x.v[0], y.v[0]), u = mul2(x.v[1], y.v[1]);
#pragma unroll
  for (int i = 2; i < P; i += 2) {
    s = fma2(x.v[i], y.v[i], s);
    u = fma2(x.v[i + 1], y.v[i + 1], u);
  }
  s = add2(s, u);
  return s.x + s.y;
}
// r = (mean(x^2) + eps)^(-1/2) of a row.
template <int T, int P>
__device__ __forceinline__ float norm_factor(const Row<P>& x, float eps, float inv_d) {
  return rsqrtf(row_sum<T>(dot(x, x)) * inv_d + eps);
}
template <int P>
__device__ __forceinline__ Row<P> scaled(const Row<P>& x, float f) {
  Row<P> y;
#pragma unroll
  for (int i = 0; i < P; ++i) y.v[i] = mul2(x.v[i], splat2(f));
  return y;
}
template <int P>
__device__ __forceinline__ Row<P> product(const Row<P>& x, const Row<P>& y) {
  Row<P> z;
#pragma unroll
  for (int i = 0; i < P; ++i) z.v[i] = mul2(x.v[i], y.v[i]);
  return z;
}

// cos and sin of pos * inv_freq.  The angle is taken in turns and reduced in
// fp64 (pos is up to 2^31 and inv_freq a full fp32 value: in fp32 the angle of
// a position past 10^5 would be off by a hundredth of a radian).  The fraction
// left is rounded to fp32 for sincospif, and what that rounding drops (2^-25
// turns at most) turns the result by its own small angle, which leaves the error
// of sincospif and of one fp32 operation: keys that are rounded to e4m3
// afterwards land on another code than the exact ones where the fp32 error
// crosses a tie.
// Not inlined: short calls wait for instructions to arrive more than for
// anything else.
static __device__ __noinline__ float2 angle(int pos, float inv_freq) {
  constexpr double kTurnsPerRadian = 0.15915494309189533577;
  constexpr float kTwoPi = 6.2831853f;
  const double turns = static_cast<double>(pos) * (static_cast<double>(inv_freq) * kTurnsPerRadian);
  const double frac = turns - rint(turns);
  const float f = static_cast<float>(frac);
  const float rest = kTwoPi * static_cast<float>(frac - static_cast<double>(f));
  float c, s;
  sincospif(2.0f * f, &s, &c);
  return make_float2(fmaf(-s, rest, c), fmaf(c, rest, s));
}

// A linear map of a lane's pieces:
//   halves:     a' = a c_a + b s_a,   b' = b c_b + a s_b
//   neighbours: v' = v c + swapped(v) s for each pair
// which a rotation, its inverse and either with the norm's weights folded in
// all are.
template <int P>
struct Turn {
  float2 c[P], s[P];
};
template <bool kNext, int P>
__device__ __forceinline__ Row<P> apply(const Row<P>& x, const Turn<P>& f, const Place& p, int rot, int D) {
  Row<P> y;
#pragma unroll
  for (int i = 0; i < P; ++i)
    y.v[i] = fma2(kNext ? make_float2(x.v[i].y, x.v[i].x) : x.v[i ^ (P / 2)], f.s[i], mul2(x.v[i], f.c[i]));
  // What passes through does so alone: 0 times its partner would turn an
  // infinity there into NaN.
  if (rot < D) {
#pragma unroll
    for (int i = 0; i < 2 * P; ++i) {
      const bool turns = kNext ? p.a + i < rot : (i & (P - 1)) < p.pairs;
      if (!turns) put(y, i, at(x, i) * ((i & 1) ? f.c[i >> 1].y : f.c[i >> 1].x));
    }
  }
  return y;
}

// The rotation by a token's angles (tables of rot / 2 cosines and sines in
// shared memory, 16-byte aligned where 8 | rot); sign -1 turns back.
template <bool kNext, int P>
__device__ __forceinline__ Turn<P> rotation(const float* cos_t, const float* sin_t, int t, int rot, float sign) {
  float c[P], s[P];
  const int h = rot >> 1;
  if ((rot & 7) == 0) {
#pragma unroll
    for (int w = 0; w < P; w += 4) {
      float4 cv = make_float4(1.0f, 1.0f, 1.0f, 1.0f), sv = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (P * t + w < h) {
        cv = *reinterpret_cast<const float4*>(cos_t + P * t + w);
        sv = *reinterpret_cast<const float4*>(sin_t + P * t + w);
      }
      c[w] = cv.x; c[w + 1] = cv.y; c[w + 2] = cv.z; c[w + 3] = cv.w;
      s[w] = sv.x; s[w + 1] = sv.y; s[w + 2] = sv.z; s[w + 3] = sv.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const bool in = P * t + i < h;
      c[i] = in ? cos_t[P * t + i] : 1.0f;
      s[i] = in ? sin_t[P * t + i] : 0.0f;
    }
  }
  Turn<P> f;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if constexpr (kNext) {
      f.c[i] = make_float2(c[i], c[i]);
      f.s[i] = make_float2(-sign * s[i], sign * s[i]);
    } else {
      const int k = 2 * (i & (P / 2 - 1));
      f.c[i] = make_float2(c[k], c[k + 1]);
      const float sg = i < P / 2 ? -sign : sign;
      f.s[i] = make_float2(sg * s[k], sg * s[k + 1]);
    }
  }
  return f;
}
template <int P>
__device__ __forceinline__ Turn<P> identity() {
  Turn<P> f;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    f.c[i] = make_float2(1.0f, 1.0f);
    f.s[i] = make_float2(0.0f, 0.0f);
  }
  return f;
}
// The map that weighs by w first.
template <bool kNext, int P>
__device__ __forceinline__ void fold(Turn<P>& f, const Row<P>& w) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    f.c[i] = mul2(f.c[i], w.v[i]);
    f.s[i] = mul2(f.s[i], kNext ? make_float2(w.v[i].y, w.v[i].x) : w.v[i ^ (P / 2)]);
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
template <bool kVec, int P>
__device__ __forceinline__ Row<P> lane_weight(const float* w, const Place& p) {
  Row<P> r;
  if constexpr (kVec) {  // pieces are whole and start on multiples of 4
#pragma unroll
    for (int i = 0; i < P; i += 2) {
      const bool in = i < P / 2 ? p.na : p.nb;
      const int e = i < P / 2 ? p.a + 2 * i : p.b + 2 * i - P;
      const float4 v = in ? *reinterpret_cast<const float4*>(w + e) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      r.v[i] = make_float2(v.x, v.y);
      r.v[i + 1] = make_float2(v.z, v.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2 * P; ++i) put(r, i, has<P>(p, i) ? w[element<P>(p, i)] : 0.0f);
  }
  return r;
}

// The row layout of a call (see above): lanes and elements a piece, `wide`
// (4 or 8) for head dims above 64.
struct Layout {
  bool vec;
  int P, T;
};
inline Layout layout_of(int D, int rot, bool next, bool aligned, int wide) {
  const int P = D > 64 ? wide : 4;
  if (aligned && (next || rot % (2 * P) == 0)) return {true, P, D > 64 ? 64 / P : 8};
  return {false, 4, 32};
}

}  // namespace fa
