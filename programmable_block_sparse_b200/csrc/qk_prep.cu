// Norm of queries and keys per head with the position rotation in the same
// pass, and its gradients (formulas: include/flexattn.h).
//
// Both kernels are bound by HBM: a row is read once and written once (the
// backward reads the row and its output gradient).  T lanes hold a row
// (headprep.cuh).  A CTA takes a few tokens and all (or a run of) their heads:
// a token's angles are the same for every head, so their fp64 reduction and
// sincos are paid once a token, into shared memory, and each group of T lanes
// keeps its token's factors in registers while it walks the heads, several
// rows in flight.
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

// The heads h0 .. h1 - 1 of one side for this group's token.  Every lane of a
// warp takes the same number of turns (shuffles).
template <int T, bool kNext, bool kVec, bool kF32>
__device__ __forceinline__ void prep_rows(const PrepArgs& a, const RowsIn& in, const RowsOut& out, int b, int n, int h0,
                                          int h1, int sub, int per, int norm, float eps, const Place& p,
                                          const Turn& f) {
  constexpr int U = kVec && !kF32 ? 4 : 2;  // rows in flight per group
  const float inv_d = 1.0f / static_cast<float>(a.D);
  const bool here = n < a.N;
  const char* ip = static_cast<const char*>(in.p) +
                   (b * in.stride[0] + n * in.stride[2] + (h0 + sub) * in.stride[1]) * (kF32 ? 4 : 2);
  const int64_t istep = in.stride[1] * per * (kF32 ? 4 : 2);
  char* op = static_cast<char*>(out.p) +
             (b * out.stride[0] + n * out.stride[2] + (h0 + sub) * out.stride[1]) * (out.f32 ? 4 : 2);
  const int64_t ostep = out.stride[1] * per * (out.f32 ? 4 : 2);
  for (int hb = h0; hb < h1; hb += per * U) {
    Raw<kVec, kF32> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (here && hb + sub + u * per < h1)
        load_raw(ip + u * istep, p, raw[u]);
      else
        clear_raw(raw[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (hb + u * per >= h1) break;  // the same for the whole CTA
      const Row x = unpack(raw[u]);
      Row y = apply<kNext>(x, f, p, a.rope.rot, a.D);
      if (norm) y = scaled(y, norm_factor<T>(x, eps, inv_d));
      if (here && hb + sub + u * per < h1) store_row<kVec>(op + u * ostep, out.f32, p, y);
    }
    ip += U * istep;
    op += U * ostep;
  }
}

template <int T, bool kNext, bool kVec>
__global__ void __launch_bounds__(kPrepThreads, kVec ? 4 : 2) prep_kernel(const __grid_constant__ PrepArgs a) {
  constexpr int kGroups = kPrepThreads / T;
  __shared__ __align__(16) float cos_t[kTableFloats], sin_t[kTableFloats], s_w[2][128];
  const int b = blockIdx.z, n0 = blockIdx.x * a.tokens;
  const int t = threadIdx.x % T, grp = threadIdx.x / T;
  const int tk = grp % a.tokens, sub = grp / a.tokens, per = kGroups / a.tokens;
  const int n = n0 + tk, rot = a.rope.rot;
  const Place p = place_of<kNext>(t, rot, a.D);
  for (int side = 0; side < 2; ++side)
    if (a.norm[side].on) stage_weight(a.norm[side], a.D, 128, s_w[side]);
  if (rot) fill_tables(a.rope, b, n0, a.tokens, a.N, cos_t, sin_t);
  __syncthreads();
  const int first = blockIdx.y * a.heads, last = first + a.heads;  // of the heads of q, then of k
  int before = 0;
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const RowsIn& in = a.x[side];
    if (in.p == nullptr) continue;
    const int h0 = max(first - before, 0), h1 = min(last - before, in.H);
    before += in.H;
    if (h0 >= h1) continue;
    Turn f = rot ? rotation<kNext>(cos_t + tk * (rot >> 1), sin_t + tk * (rot >> 1), t, p, rot, 1.0f) : identity();
    const NormArgs& norm = a.norm[side];
    if (norm.on) fold<kNext>(f, lane_weight<kVec>(s_w[side], p));
    if (in.f32)
      prep_rows<T, kNext, kVec, true>(a, in, a.y[side], b, n, h0, h1, sub, per, norm.on, norm.eps, p, f);
    else
      prep_rows<T, kNext, kVec, false>(a, in, a.y[side], b, n, h0, h1, sub, per, norm.on, norm.eps, p, f);
  }
}

// One row's gradient: y, the output gradient turned back, becomes the input
// gradient, and dw takes its share of the weight gradient.
template <int T>
__device__ __forceinline__ void norm_gradient(Row& y, const Row& x, const Row& w, float eps, float inv_d, Row& dw) {
  const Row yw = product(y, w);
  float ss = dot8(x, x), sd = dot8(yw, x);
#pragma unroll
  for (int o = T / 2; o > 0; o >>= 1) {
    ss += __shfl_xor_sync(0xffffffffu, ss, o);
    sd += __shfl_xor_sync(0xffffffffu, sd, o);
  }
  const float r = rsqrtf(ss * inv_d + eps), k = sd * inv_d * r * r;
  const Row xr = scaled(x, r);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    dw.v[i] = fma2(y.v[i], xr.v[i], dw.v[i]);
    y.v[i] = fma2(splat2(-k), xr.v[i], mul2(yw.v[i], splat2(r)));
  }
}

// What one thread walks in a work item: its token's heads of one side, every
// `per`-th from `sub` on.
struct HeadWalk {
  const char *g, *x;  // first head's rows
  int64_t gstep, xstep;
  int heads, turns;
};
__device__ __forceinline__ HeadWalk walk_of(const PrepBwdArgs& a, int side, int b, int n, int sub, int per) {
  const RowsIn &dy = a.dy[side], &in = a.x[side];
  const int ge = dy.f32 ? 4 : 2, xe = in.f32 ? 4 : 2;
  HeadWalk w;
  w.heads = dy.p ? dy.H : 0;
  w.turns = (w.heads + per - 1) / per;
  w.g = static_cast<const char*>(dy.p) + (b * dy.stride[0] + n * dy.stride[2] + sub * dy.stride[1]) * ge;
  w.x = static_cast<const char*>(in.p) + (b * in.stride[0] + n * in.stride[2] + sub * in.stride[1]) * xe;
  w.gstep = dy.stride[1] * per * ge;
  w.xstep = in.stride[1] * per * xe;
  return w;
}

// Gradients.  A CTA walks work items (a token block of one sequence) with a
// stride of the grid and adds up this lane's share of the weight gradients
// over its heads, over its items in shared memory; it writes one partial row
// per side, and the sums over CTAs follow in a second kernel in a fixed order.
// A row takes two reads, so the walk over q's heads and then k's keeps
// kStages - 1 rows a lane in flight through shared memory (copy_raw).  Rows
// that are read one element at a time go without.
template <int T, bool kNext, bool kVec, bool kXF32, bool kGF32>
__global__ void __launch_bounds__(kPrepThreads, kVec ? 3 : 1) prep_bwd_kernel(const __grid_constant__ PrepBwdArgs a) {
  constexpr int kGroups = kPrepThreads / T;
  constexpr int kStages = 5;
  constexpr int kXSlot = kXF32 ? 32 : 16, kGSlot = kGF32 ? 32 : 16;
  constexpr int kStageBytes = kPrepThreads * (kXSlot + kGSlot);
  extern __shared__ __align__(16) uint8_t ring[];  // kVec: kStages x (g slots, x slots)
  __shared__ __align__(16) float cos_t[kTableFloats], sin_t[kTableFloats], s_w[2][128];
  __shared__ float red[2][kGroups][129];
  const int t = threadIdx.x % T, grp = threadIdx.x / T;
  const int tk = grp % a.tokens, sub = grp / a.tokens, per = kGroups / a.tokens;
  const int rot = a.rope.rot;
  const Place p = place_of<kNext>(t, rot, a.D);
  const float inv_d = 1.0f / static_cast<float>(a.D);
  const int blocks = (a.N + a.tokens - 1) / a.tokens;
  for (int side = 0; side < 2; ++side) stage_weight(a.norm[side], a.D, 128, s_w[side]);
#pragma unroll
  for (int i = 0; i < 8; ++i)  // each lane clears, and later adds to, its own places
    if ((i & 3) < (i < 4 ? p.na : p.nb)) red[0][grp][i < 4 ? p.a + i : p.b + i - 4] = red[1][grp][i < 4 ? p.a + i : p.b + i - 4] = 0.0f;
  const uint32_t my_g = kVec ? smem_u32(ring) + threadIdx.x * kGSlot : 0;
  const uint32_t my_x = kVec ? smem_u32(ring) + kPrepThreads * kGSlot + threadIdx.x * kXSlot : 0;
  __syncthreads();
  for (int64_t item = blockIdx.x; item < static_cast<int64_t>(blocks) * a.B; item += gridDim.x) {
    const int b = static_cast<int>(item / blocks), n0 = static_cast<int>(item % blocks) * a.tokens, n = n0 + tk;
    const bool here = n < a.N;
    const HeadWalk w0 = walk_of(a, 0, b, n, sub, per), w1 = walk_of(a, 1, b, n, sub, per);
    const int turns = w0.turns + w1.turns;  // the same for the whole CTA
    auto issue = [&](int i, int stage) {
      if (i < turns) {
        const bool second = i >= w0.turns;
        const HeadWalk& w = second ? w1 : w0;
        const int k = second ? i - w0.turns : i;
        const bool ok = here && sub + k * per < w.heads;
        copy_raw<kGF32>(my_g + stage * kStageBytes, w.g + k * w.gstep, p, ok);
        copy_raw<kXF32>(my_x + stage * kStageBytes, w.x + k * w.xstep, p, ok && a.norm[second].on);
      }
      copy_commit();
    };
    if constexpr (kVec) {
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) issue(i, i);
    }
    Turn f = identity();
    if (rot) {
      __syncthreads();  // the tables of the previous item have been read
      fill_tables(a.rope, b, n0, a.tokens, a.N, cos_t, sin_t);
      __syncthreads();
      f = rotation<kNext>(cos_t + tk * (rot >> 1), sin_t + tk * (rot >> 1), t, p, rot, -1.0f);
    }
    int stage = 0;
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
      const HeadWalk& wk = side ? w1 : w0;
      if (wk.turns == 0) continue;
      const int norm = a.norm[side].on, before = side ? w0.turns : 0;
      const float eps = a.norm[side].eps;
      const Row w = lane_weight<kVec>(s_w[side], p);
      const RowsOut& dx = a.dx[side];
      char* op = static_cast<char*>(dx.p) +
                 (b * dx.stride[0] + n * dx.stride[2] + sub * dx.stride[1]) * (dx.f32 ? 4 : 2);
      const int64_t ostep = dx.stride[1] * per * (dx.f32 ? 4 : 2);
      Row dw;
#pragma unroll
      for (int i = 0; i < 4; ++i) dw.v[i] = make_float2(0.0f, 0.0f);
      for (int k = 0; k < wk.turns; ++k) {
        const bool ok = here && sub + k * per < wk.heads;
        Raw<kVec, kGF32> graw;
        Raw<kVec, kXF32> xraw;
        if constexpr (kVec) {
          issue(before + k + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
          copy_wait<kStages - 1>();
          read_raw<kGF32>(my_g + stage * kStageBytes, graw);
          read_raw<kXF32>(my_x + stage * kStageBytes, xraw);
          stage = stage == kStages - 1 ? 0 : stage + 1;
        } else {
          clear_raw(graw);
          clear_raw(xraw);
          if (ok) load_raw(wk.g + k * wk.gstep, p, graw);
          if (ok && norm) load_raw(wk.x + k * wk.xstep, p, xraw);
        }
        Row y = apply<kNext>(unpack(graw), f, p, rot, a.D);
        if (norm) norm_gradient<T>(y, unpack(xraw), w, eps, inv_d, dw);
        if (ok) store_row<kVec>(op + k * ostep, dx.f32, p, y);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if ((i & 3) < (i < 4 ? p.na : p.nb))
          red[side][grp][i < 4 ? p.a + i : p.b + i - 4] += (i & 1) ? dw.v[i >> 1].y : dw.v[i >> 1].x;
    }
    if constexpr (kVec) copy_wait<0>();
  }
  __syncthreads();
  const int side = threadIdx.x >> 7, e = threadIdx.x & 127;
  if (a.dw[side] != nullptr && e < a.D) {
    float v = 0.0f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) v += red[side][g][e];
    a.partial[(static_cast<int64_t>(blockIdx.x) * 2 + side) * a.D + e] = v;
  }
}

template <int T, bool kNext, bool kVec>
cudaError_t launch_bwd_t(const PrepBwdArgs& a, int ctas, bool xf32, bool gf32, cudaStream_t st) {
  auto kern = xf32 ? (gf32 ? prep_bwd_kernel<T, kNext, kVec, true, true> : prep_bwd_kernel<T, kNext, kVec, true, false>)
                   : (gf32 ? prep_bwd_kernel<T, kNext, kVec, false, true> : prep_bwd_kernel<T, kNext, kVec, false, false>);
  const int ring = kVec ? 5 * kPrepThreads * ((xf32 ? 32 : 16) + (gf32 ? 32 : 16)) : 0;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, ring);
  if (e != cudaSuccess) return e;
  kern<<<ctas, kPrepThreads, ring, st>>>(a);
  return cudaGetLastError();
}

// dw[side][e] = sum over CTAs of partial[cta][side][e]: 8 columns a block, 128
// threads a column, each over every 128th CTA, joined in a fixed order.
__global__ void __launch_bounds__(1024) prep_dw_kernel(const float* partial, int ctas, int D, float* dq, float* dk) {
  __shared__ float red[128][9];
  const int side = blockIdx.y, col = threadIdx.x & 7, e = blockIdx.x * 8 + col, sl = threadIdx.x >> 3;
  float* out = side ? dk : dq;
  if (out == nullptr) return;
  float v = 0.0f;
  if (e < D) {
#pragma unroll 16
    for (int cta = sl; cta < ctas; cta += 128) v += partial[(static_cast<int64_t>(cta) * 2 + side) * D + e];
  }
  red[sl][col] = v;
  __syncthreads();
  if (threadIdx.x < 256) {  // one warp a column: four values a lane, then a tree
    const int c = threadIdx.x >> 5, l = threadIdx.x & 31;
    float sum = (red[l][c] + red[l + 32][c]) + (red[l + 64][c] + red[l + 96][c]);
    sum = row_sum<32>(sum);
    if (l == 0 && blockIdx.x * 8 + c < D) out[blockIdx.x * 8 + c] = sum;
  }
}

// Lanes a row, for rows that take vector accesses and others.
int lanes_of(int D, bool vec) { return !vec ? 32 : (D <= 64 ? 8 : 16); }

// Tokens a CTA: one for each of its groups, fewer (and more groups a token)
// until there are `ctas` CTAs.
int tokens_of(int lanes, int B, int N, int ctas) {
  int tokens = kPrepThreads / lanes;
  while (tokens > 1 && static_cast<int64_t>(B) * ((N + tokens - 1) / tokens) < ctas) tokens /= 2;
  return tokens;
}

}  // namespace

cudaError_t launch_prep(PrepArgs a, int num_sms, cudaStream_t st) {
  const int heads = (a.x[0].p ? a.x[0].H : 0) + (a.x[1].p ? a.x[1].H : 0);
  const bool next = a.rope.rot == 0 || a.rope.interleaved, vec = a.vec && (next || a.rope.rot % 8 == 0);
  const int lanes = lanes_of(a.D, vec);
  // As many tokens a CTA as leave eight CTAs an SM (a group's factors serve all
  // heads of its token); one token a CTA, and its heads cut into runs of one
  // turn of the groups, where even that does not (a decode step).
  a.tokens = tokens_of(lanes, a.B, a.N, 8 * num_sms);
  a.heads = heads;
  if (static_cast<int64_t>(a.B) * ((a.N + a.tokens - 1) / a.tokens) < 4 * num_sms) a.heads = kPrepThreads / lanes;
  auto kern = !vec          ? (next ? prep_kernel<32, true, false> : prep_kernel<32, false, false>)
              : lanes == 8 ? (next ? prep_kernel<8, true, true> : prep_kernel<8, false, true>)
                            : (next ? prep_kernel<16, true, true> : prep_kernel<16, false, true>);
  const dim3 grid((a.N + a.tokens - 1) / a.tokens, (heads + a.heads - 1) / a.heads, a.B);
  kern<<<grid, kPrepThreads, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_prep_bwd(PrepBwdArgs a, cudaStream_t st) {
  // One kernel takes inputs of one type and output gradients of one type; q
  // and k that differ go in turn.
  const bool two = a.dy[0].p && a.dy[1].p &&
                   (a.dy[0].f32 != a.dy[1].f32 || (a.x[0].p && a.x[1].p && a.x[0].f32 != a.x[1].f32));
  if (two) {
    for (int side = 0; side < 2; ++side) {
      PrepBwdArgs one = a;
      one.dy[1 - side] = RowsIn{};
      one.dw[1 - side] = nullptr;
      const cudaError_t e = launch_prep_bwd(one, st);
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }
  const bool next = a.rope.rot == 0 || a.rope.interleaved, vec = a.vec && (next || a.rope.rot % 8 == 0);
  const int lanes = lanes_of(a.D, vec);
  a.tokens = tokens_of(lanes, a.B, a.N, kPrepBwdMaxCtas / 2);
  const int64_t items = static_cast<int64_t>(a.B) * ((a.N + a.tokens - 1) / a.tokens);
  const int ctas = static_cast<int>(items < kPrepBwdMaxCtas ? items : kPrepBwdMaxCtas);
  const bool gf32 = a.dy[a.dy[0].p ? 0 : 1].f32;
  const bool xf32 = a.x[0].p && a.dy[0].p ? a.x[0].f32 : a.x[1].f32;
  cudaError_t e;
  if (!vec)
    e = next ? launch_bwd_t<32, true, false>(a, ctas, xf32, gf32, st) : launch_bwd_t<32, false, false>(a, ctas, xf32, gf32, st);
  else if (lanes == 8)
    e = next ? launch_bwd_t<8, true, true>(a, ctas, xf32, gf32, st) : launch_bwd_t<8, false, true>(a, ctas, xf32, gf32, st);
  else
    e = next ? launch_bwd_t<16, true, true>(a, ctas, xf32, gf32, st) : launch_bwd_t<16, false, true>(a, ctas, xf32, gf32, st);
  if (e != cudaSuccess || (a.dw[0] == nullptr && a.dw[1] == nullptr)) return e;
  prep_dw_kernel<<<dim3((a.D + 7) / 8, 2), 1024, 0, st>>>(a.partial, ctas, a.D, a.dw[0], a.dw[1]);
  return cudaGetLastError();
}

}  // namespace fa
