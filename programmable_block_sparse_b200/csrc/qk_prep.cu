// Norm of queries and keys per head with the position rotation in the same
// pass, and its gradients (formulas: include/flexattn.h).
//
// Both kernels are bound by HBM: a row is read once and written once (the
// backward reads the row and its output gradient).  T lanes hold a row
// (headprep.cuh), so a warp takes 2 (D <= 128) or 4 (D <= 64) rows and every
// access is 16 bytes a lane.  A CTA takes a few tokens and all (or a run of)
// their heads: a token's angles are the same for every head, so their fp64
// reduction and sincos are paid once a token, into shared memory, and each
// group of T lanes keeps its token's cosines and sines in registers while it
// walks the heads, several rows in flight.
#include "headprep.cuh"

namespace fa {
namespace {

constexpr int kPrepThreads = 256;
constexpr int kTableFloats = 16 * 64;  // tokens of a CTA x rot / 2, at most: 16 x 64 or 32 x 32

// cos / sin tables of tokens n0 .. n0 + count - 1 (the caller synchronises).
__device__ __forceinline__ void fill_tables(const RopeArgs& r, int b, int n0, int count, int N, float* cos_t,
                                            float* sin_t) {
  const int h = r.rot >> 1;
  for (int i = threadIdx.x; i < count * h; i += blockDim.x) {
    const int tk = i / h, n = n0 + tk;
    if (n < N) {
      const int pos = r.pos ? __ldg(r.pos + static_cast<int64_t>(r.pos_batch > 1 ? b : 0) * N + n) : n;
      angle(pos, __ldg(r.inv_freq + (i - tk * h)), cos_t + i, sin_t + i);
    }
  }
}

template <int T, Pair kPair, bool kVec>
__global__ void __launch_bounds__(kPrepThreads) prep_kernel(const __grid_constant__ PrepArgs a) {
  constexpr int kGroups = kPrepThreads / T;
  constexpr int U = 4;  // rows in flight per group
  __shared__ float cos_t[kTableFloats], sin_t[kTableFloats];
  const int b = blockIdx.z, n0 = blockIdx.x * a.tokens;
  const int t = threadIdx.x % T, grp = threadIdx.x / T;
  const int tk = grp % a.tokens, sub = grp / a.tokens, per = kGroups / a.tokens;
  const int n = n0 + tk, e0 = 8 * t, rot = a.rope.rot;
  float c[8], s[8];
  if (rot) {
    fill_tables(a.rope, b, n0, a.tokens, a.N, cos_t, sin_t);
    __syncthreads();
    lane_angles<kPair>(cos_t + tk * (rot >> 1), sin_t + tk * (rot >> 1), e0, rot, c, s);
  }
  const float inv_d = 1.0f / static_cast<float>(a.D);
  const int first = blockIdx.y * a.heads, last = first + a.heads;  // of the heads of q, then of k
  int before = 0;
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const RowsIn& in = a.x[side];
    if (in.p == nullptr) continue;
    const RowsOut& out = a.y[side];
    const int h0 = max(first - before, 0), h1 = min(last - before, in.H);
    before += in.H;
    if (h0 >= h1) continue;
    const int norm = a.norm[side].on;
    float w[8];
    if (norm) load_weight8(a.norm[side], e0, a.D, w);
    const int64_t ib = b * in.stride[0] + n * in.stride[2], ob = b * out.stride[0] + n * out.stride[2];
    // every lane of a warp takes the same number of turns (shuffles)
    for (int hb = h0; hb < h1; hb += per * U) {
      float x[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = hb + sub + u * per;
        if (n < a.N && h < h1)
          load8<kVec>(row_ptr(in.p, in.f32, ib + h * in.stride[1]), in.f32, e0, a.D, x[u]);
        else
#pragma unroll
          for (int i = 0; i < 8; ++i) x[u][i] = 0.0f;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (hb + u * per >= h1) break;  // the same for the whole CTA
        const int h = hb + sub + u * per;
        float y[8];
        if (norm) norm8<T>(x[u], w, a.norm[side].eps, inv_d);
        if (rot) {
          rotate8<T, kPair>(x[u], c, s, 1.0f, t, rot, y);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = x[u][i];
        }
        if (n < a.N && h < h1) store8<kVec>(row_ptr(out.p, out.f32, ob + h * out.stride[1]), out.f32, e0, a.D, y);
      }
    }
  }
}

// Gradients.  A CTA walks work items (a token block of one sequence) with a
// stride of the grid, keeps this lane's share of the weight gradients in
// registers over all of them, and writes one partial row per side; the sums
// over CTAs follow in a second kernel in a fixed order.
template <int T, Pair kPair, bool kVec>
__global__ void __launch_bounds__(kPrepThreads) prep_bwd_kernel(const __grid_constant__ PrepBwdArgs a) {
  constexpr int kGroups = kPrepThreads / T;
  constexpr int U = 2;
  __shared__ float cos_t[kTableFloats], sin_t[kTableFloats];
  __shared__ float red[kGroups][T * 8 + 1];
  const int t = threadIdx.x % T, grp = threadIdx.x / T;
  const int tk = grp % a.tokens, sub = grp / a.tokens, per = kGroups / a.tokens;
  const int e0 = 8 * t, rot = a.rope.rot;
  const float inv_d = 1.0f / static_cast<float>(a.D);
  const int blocks = (a.N + a.tokens - 1) / a.tokens;
  float dw[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[0][i] = dw[1][i] = 0.0f;
  for (int64_t item = blockIdx.x; item < static_cast<int64_t>(blocks) * a.B; item += gridDim.x) {
    const int b = static_cast<int>(item / blocks), n0 = static_cast<int>(item % blocks) * a.tokens, n = n0 + tk;
    float c[8], s[8];
    if (rot) {
      __syncthreads();  // the tables of the previous item have been read
      fill_tables(a.rope, b, n0, a.tokens, a.N, cos_t, sin_t);
      __syncthreads();
      lane_angles<kPair>(cos_t + tk * (rot >> 1), sin_t + tk * (rot >> 1), e0, rot, c, s);
    }
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const RowsIn& dy = a.dy[side];
      if (dy.p == nullptr) continue;
      const RowsIn& in = a.x[side];
      const RowsOut& dx = a.dx[side];
      const int norm = a.norm[side].on;
      const float eps = a.norm[side].eps;
      float w[8];
      if (norm) load_weight8(a.norm[side], e0, a.D, w);
      const int64_t gb = b * dy.stride[0] + n * dy.stride[2], xb = b * in.stride[0] + n * in.stride[2];
      const int64_t ob = b * dx.stride[0] + n * dx.stride[2];
      for (int hb = 0; hb < dy.H; hb += per * U) {
        float g[U][8], x[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int h = hb + sub + u * per;
          const bool ok = n < a.N && h < dy.H;
          if (ok) load8<kVec>(row_ptr(dy.p, dy.f32, gb + h * dy.stride[1]), dy.f32, e0, a.D, g[u]);
          if (ok && norm) load8<kVec>(row_ptr(in.p, in.f32, xb + h * in.stride[1]), in.f32, e0, a.D, x[u]);
          if (!ok)
#pragma unroll
            for (int i = 0; i < 8; ++i) g[u][i] = x[u][i] = 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (hb + u * per >= dy.H) break;  // the same for the whole CTA
          const int h = hb + sub + u * per;
          float y[8];
          if (rot) {
            rotate8<T, kPair>(g[u], c, s, -1.0f, t, rot, y);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = g[u][i];
          }
          if (norm) {
            float ss = 0.0f, dot = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              ss = fmaf(x[u][i], x[u][i], ss);
              dot = fmaf(y[i] * w[i], x[u][i], dot);
            }
            const float r = rsqrtf(row_sum<T>(ss) * inv_d + eps);
            const float k = row_sum<T>(dot) * inv_d * r * r;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              dw[side][i] = fmaf(y[i] * r, x[u][i], dw[side][i]);
              y[i] = r * fmaf(-k, x[u][i], y[i] * w[i]);
            }
          }
          if (n < a.N && h < dy.H) store8<kVec>(row_ptr(dx.p, dx.f32, ob + h * dx.stride[1]), dx.f32, e0, a.D, y);
        }
      }
    }
  }
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    if (a.dw[side] == nullptr) continue;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) red[grp][e0 + i] = dw[side][i];
    __syncthreads();
    if (threadIdx.x < a.D) {
      float v = 0.0f;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) v += red[g][threadIdx.x];
      a.partial[(static_cast<int64_t>(blockIdx.x) * 2 + side) * a.D + threadIdx.x] = v;
    }
  }
}

// dw[side][e] = sum over CTAs of partial[cta][side][e]: 32 columns a block, 32
// threads a column, each over every 32nd CTA, joined in a fixed order.
__global__ void __launch_bounds__(1024) prep_dw_kernel(const float* partial, int ctas, int D, float* dq, float* dk) {
  __shared__ float red[32][33];
  const int side = blockIdx.y, e = blockIdx.x * 32 + (threadIdx.x & 31), sl = threadIdx.x >> 5;
  float* out = side ? dk : dq;
  if (out == nullptr) return;
  float v = 0.0f;
  if (e < D) {
#pragma unroll 4
    for (int cta = sl; cta < ctas; cta += 32) v += partial[(static_cast<int64_t>(cta) * 2 + side) * D + e];
  }
  red[sl][threadIdx.x & 31] = v;
  __syncthreads();
  if (sl == 0 && e < D) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += red[i][threadIdx.x];
    out[e] = sum;
  }
}

Pair pair_of(const RopeArgs& r) {
  if (r.rot == 0 || r.interleaved) return Pair::kNext;
  return (r.rot / 2) % 8 == 0 ? Pair::kHalf : Pair::kHalfAny;
}

// The kernel of a call; rows without 16-byte accesses share the any-place
// pairing.
template <int T>
cudaError_t launch_prep_t(const PrepArgs& a, dim3 grid, cudaStream_t st) {
  const Pair pair = pair_of(a.rope);
  auto kern = pair == Pair::kNext ? (a.vec ? prep_kernel<T, Pair::kNext, true> : prep_kernel<T, Pair::kNext, false>)
              : !a.vec            ? prep_kernel<T, Pair::kHalfAny, false>
              : pair == Pair::kHalf ? prep_kernel<T, Pair::kHalf, true>
                                    : prep_kernel<T, Pair::kHalfAny, true>;
  kern<<<grid, kPrepThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <int T>
cudaError_t launch_prep_bwd_t(const PrepBwdArgs& a, int ctas, cudaStream_t st) {
  const Pair pair = pair_of(a.rope);
  auto kern = pair == Pair::kNext
                  ? (a.vec ? prep_bwd_kernel<T, Pair::kNext, true> : prep_bwd_kernel<T, Pair::kNext, false>)
              : !a.vec              ? prep_bwd_kernel<T, Pair::kHalfAny, false>
              : pair == Pair::kHalf ? prep_bwd_kernel<T, Pair::kHalf, true>
                                    : prep_bwd_kernel<T, Pair::kHalfAny, true>;
  kern<<<ctas, kPrepThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prep(PrepArgs a, int num_sms, cudaStream_t st) {
  const int heads = (a.x[0].p ? a.x[0].H : 0) + (a.x[1].p ? a.x[1].H : 0);
  const int groups = kPrepThreads / (a.D <= 64 ? 8 : 16);
  // Four tokens a CTA with all their heads where that fills the GPU; one token
  // a CTA, and its heads cut into runs of one turn of the groups, where it
  // does not (a decode step).
  a.tokens = 4;
  a.heads = heads;
  if (static_cast<int64_t>(a.B) * ((a.N + 3) / 4) < 4 * num_sms) {
    a.tokens = 1;
    a.heads = groups;
  }
  const dim3 grid((a.N + a.tokens - 1) / a.tokens, (heads + a.heads - 1) / a.heads, a.B);
  return a.D <= 64 ? launch_prep_t<8>(a, grid, st) : launch_prep_t<16>(a, grid, st);
}

cudaError_t launch_prep_bwd(PrepBwdArgs a, cudaStream_t st) {
  a.tokens = static_cast<int64_t>(a.B) * ((a.N + 3) / 4) < kPrepBwdMaxCtas ? 1 : 4;
  const int64_t items = static_cast<int64_t>(a.B) * ((a.N + a.tokens - 1) / a.tokens);
  const int ctas = static_cast<int>(items < kPrepBwdMaxCtas ? items : kPrepBwdMaxCtas);
  const cudaError_t e = a.D <= 64 ? launch_prep_bwd_t<8>(a, ctas, st) : launch_prep_bwd_t<16>(a, ctas, st);
  if (e != cudaSuccess || (a.dw[0] == nullptr && a.dw[1] == nullptr)) return e;
  prep_dw_kernel<<<dim3((a.D + 31) / 32, 2), 1024, 0, st>>>(a.partial, ctas, a.D, a.dw[0], a.dw[1]);
  return cudaGetLastError();
}

}  // namespace fa
