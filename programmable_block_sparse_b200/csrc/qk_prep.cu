// Norm of queries and keys per head with the position rotation in the same
// pass, and its gradients (formulas: include/flexattn.h).
//
// Both kernels are bound by HBM: a row is read once and written once (the
// backward reads the row and its output gradient).  T lanes hold a row
// (headprep.cuh).  A CTA takes a few tokens and all (or a run of) their heads:
// a token's angles are the same for every head, so their fp64 reduction and
// sincos are paid once a token, into shared memory, and each group of T lanes
// keeps its token's factors in registers while it walks the heads, several
// rows in flight.  Measured at 32 + 8 heads of 128 over 32768 tokens in bf16:
// forward 122 us for 671 MB (5.5 TB/s), 146 instructions for two rows of a
// warp and 68% of the issue slots; backward 184 us for 1007 MB (5.5 TB/s), 74%
// of the issue slots.
#include "headprep.cuh"
#include "smem_limit.h"

namespace fa {
namespace {

constexpr int kPrepThreads = 256;

// cos / sin tables of tokens n0 .. n0 + count - 1 (the caller synchronises).
__device__ __forceinline__ void fill_tables(const RopeArgs& r, int b, int n0, int count, int N, float* cos_t,
                                            float* sin_t) {
  const int h = r.rot >> 1;
  for (int i = threadIdx.x; i < count * h; i += blockDim.x) {
    const int tk = i / h, n = n0 + tk;
    if (n < N) {
      const int pos = r.pos ? __ldg(r.pos + static_cast<int64_t>(r.pos_batch > 1 ? b : 0) * N + n) : n;
      const float2 z = angle(pos, __ldg(r.inv_freq + (i - tk * h)));
      cos_t[i] = z.x;
      sin_t[i] = z.y;
    }
  }
}

// The heads h0 .. h1 - 1 of one side for this group's token.  Every lane of a
// warp takes the same number of turns (shuffles).
template <int T, int P, bool kNext, bool kVec, bool kF32>
__device__ __forceinline__ void prep_rows(const PrepArgs& a, const RowsIn& in, const RowsOut& out, int b, int n, int h0,
                                          int h1, int sub, int per, int norm, float eps, const Place& p,
                                          const Turn<P>& f) {
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
    Raw<P, kVec, kF32> raw[U];
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
      const Row<P> x = unpack(raw[u]);
      Row<P> y = apply<kNext>(x, f, p, a.rope.rot, a.D);
      if (norm) y = scaled(y, norm_factor<T>(x, eps, inv_d));
      if (here && hb + sub + u * per < h1) store_row<kVec>(op + u * ostep, out.f32, p, y);
    }
    ip += U * istep;
    op += U * ostep;
  }
}

// A CTA takes a block of tokens (one for each group of T lanes, or several
// groups a token) and a run of the heads of q and then k.
template <int T, int P, bool kNext, bool kVec>
__global__ void __launch_bounds__(kPrepThreads, kVec ? 4 : 2) prep_kernel(const __grid_constant__ PrepArgs a) {
  constexpr int kGroups = kPrepThreads / T;
  extern __shared__ __align__(16) float tables[];  // cosines, then sines, of the CTA's tokens
  __shared__ __align__(16) float s_w[2][128];
  const int b = blockIdx.z, n0 = blockIdx.x * a.tokens;
  const int t = threadIdx.x % T, grp = threadIdx.x / T;
  const int tk = grp % a.tokens, sub = grp / a.tokens, per = kGroups / a.tokens;
  const int n = n0 + tk, rot = a.rope.rot;
  float *cos_t = tables, *sin_t = tables + a.tokens * (rot >> 1);
  const Place p = place_of<P, kNext>(t, rot, a.D);
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
    Turn<P> f = rot ? rotation<kNext, P>(cos_t + tk * (rot >> 1), sin_t + tk * (rot >> 1), t, rot, 1.0f) : identity<P>();
    const NormArgs& norm = a.norm[side];
    if (norm.on) fold<kNext>(f, lane_weight<kVec, P>(s_w[side], p));
    if (in.f32)
      prep_rows<T, P, kNext, kVec, true>(a, in, a.y[side], b, n, h0, h1, sub, per, norm.on, norm.eps, p, f);
    else
      prep_rows<T, P, kNext, kVec, false>(a, in, a.y[side], b, n, h0, h1, sub, per, norm.on, norm.eps, p, f);
  }
}

// A thread's walk over its token's heads of one tensor, every `per`-th from
// sub on: the two pieces of its next row.
struct Walk {
  const char *a, *b;
  int64_t step;
  int head, end, left;  // next head; turns left (the same for the whole CTA)
};
__device__ __forceinline__ Walk walk_of(const RowsIn& in, const Place& p, int b, int n, int N, int sub, int per) {
  const int el = in.f32 ? 4 : 2;
  Walk w;
  w.end = in.p ? in.H : 0;
  w.left = (w.end + per - 1) / per;
  w.head = n < N ? sub : w.end;  // a token past the end has no heads
  const char* row = static_cast<const char*>(in.p) + (b * in.stride[0] + n * in.stride[2] + sub * in.stride[1]) * el;
  w.a = row + p.a * el;
  w.b = row + p.b * el;
  w.step = in.stride[1] * per * el;
  return w;
}
// Bytes of one row's slots over a CTA's threads.
constexpr int slot_bytes(int P, bool f32) { return kPrepThreads * 2 * P * (f32 ? 4 : 2); }

// One row's gradient: y, the output gradient turned back, becomes the input
// gradient, and dw takes its share of the weight gradient.  Single fp32
// operations: the factors r and k would have to be copied into register pairs
// for packed ones (203 us with those, 184 without; the forward pass is the
// other way round, 122 and 132).
template <int T, int P>
__device__ __forceinline__ void norm_gradient(Row<P>& y, const Row<P>& x, const Row<P>& w, float eps, float inv_d,
                                              bool ok, Row<P>& dw) {
  Row<P> yw;
  float ss = 0.0f, sd = 0.0f;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    yw.v[i] = make_float2(y.v[i].x * w.v[i].x, y.v[i].y * w.v[i].y);
    ss = fmaf(x.v[i].y, x.v[i].y, fmaf(x.v[i].x, x.v[i].x, ss));
    sd = fmaf(yw.v[i].y, x.v[i].y, fmaf(yw.v[i].x, x.v[i].x, sd));
  }
#pragma unroll
  for (int o = T / 2; o > 0; o >>= 1) {
    ss += __shfl_xor_sync(0xffffffffu, ss, o);
    sd += __shfl_xor_sync(0xffffffffu, sd, o);
  }
  // rows that are not there count for nothing, with eps = 0 too
  const float r = ok ? rsqrtf(ss * inv_d + eps) : 0.0f, k = sd * inv_d * r * r;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const float2 xr = make_float2(x.v[i].x * r, x.v[i].y * r);
    dw.v[i].x = fmaf(y.v[i].x, xr.x, dw.v[i].x);
    dw.v[i].y = fmaf(y.v[i].y, xr.y, dw.v[i].y);
    y.v[i].x = fmaf(-k, xr.x, yw.v[i].x * r);
    y.v[i].y = fmaf(-k, xr.y, yw.v[i].y * r);
  }
}

// Gradients.  A CTA walks work items (a token block of one sequence) with a
// stride of the grid and adds up this lane's share of the weight gradients
// over its heads, over its items in shared memory; it writes one partial row
// per side, and the sums over CTAs follow in a second kernel in a fixed order.
// A row takes two reads, so the walk over q's heads and then k's keeps
// kStages - 1 rows a lane in flight through shared memory (copy_raw).  Rows
// that are read one element at a time go without.
constexpr int kBwdStages = 3;  // 182 us; 4: 183, 5 (two CTAs an SM): 206

template <int T, int P, bool kNext, bool kVec, bool kXF32, bool kGF32>
__global__ void __launch_bounds__(kPrepThreads, kVec ? 3 : 1)
    prep_bwd_kernel(const __grid_constant__ PrepBwdArgs a) {
  constexpr int kGroups = kPrepThreads / T;
  constexpr int kStages = kBwdStages;
  constexpr int kXOffset = slot_bytes(P, kGF32), kStageBytes = kXOffset + slot_bytes(P, kXF32);  // g's slots, x's
  // kVec: kStages stages; then cosines and sines of the CTA's tokens
  extern __shared__ __align__(16) uint8_t dynamic[];
  __shared__ __align__(16) float s_w[2][128];
  __shared__ float red[2][kGroups][129];
  const int t = threadIdx.x % T, grp = threadIdx.x / T;
  const int tk = grp % a.tokens, sub = grp / a.tokens, per = kGroups / a.tokens;
  const int rot = a.rope.rot;
  float* cos_t = reinterpret_cast<float*>(dynamic + (kVec ? kStages * kStageBytes : 0));
  float* sin_t = cos_t + a.tokens * (rot >> 1);
  const Place p = place_of<P, kNext>(t, rot, a.D);
  const float inv_d = 1.0f / static_cast<float>(a.D);
  const int blocks = (a.N + a.tokens - 1) / a.tokens;
  for (int side = 0; side < 2; ++side) stage_weight(a.norm[side], a.D, 128, s_w[side]);
#pragma unroll
  for (int i = 0; i < 2 * P; ++i)  // each lane clears, and later adds to, its own places
    if (has<P>(p, i)) red[0][grp][element<P>(p, i)] = red[1][grp][element<P>(p, i)] = 0.0f;
  const uint32_t mine = kVec ? smem_u32(dynamic) + threadIdx.x * 16 : 0;
  __syncthreads();
  for (int64_t item = blockIdx.x; item < static_cast<int64_t>(blocks) * a.B; item += gridDim.x) {
    const int b = static_cast<int>(item / blocks), n0 = static_cast<int>(item % blocks) * a.tokens, n = n0 + tk;
    // the copies run ahead of the arithmetic, from one side into the next
    Walk ag = walk_of(a.dy[0], p, b, n, a.N, sub, per);
    Walk ax = walk_of(a.x[0], p, b, n, a.N, sub, per);  // no rows without a norm
    bool second = false;
    uint32_t fill = mine;
    auto issue = [&]() {
      if (ag.left <= 0 && !second) {
        ag = walk_of(a.dy[1], p, b, n, a.N, sub, per);
        ax = walk_of(a.x[1], p, b, n, a.N, sub, per);
        second = true;
      }
      if (ag.left > 0) {
        copy_raw<P, kGF32, kPrepThreads>(fill, ag.a, ag.b, p, ag.head < ag.end);
        copy_raw<P, kXF32, kPrepThreads>(fill + kXOffset, ax.a, ax.b, p, ag.head < ax.end);
        ag.a += ag.step;
        ag.b += ag.step;
        ax.a += ax.step;
        ax.b += ax.step;
        ag.head += per;
        --ag.left;
      }
      copy_commit();
      fill = fill == mine + (kStages - 1) * kStageBytes ? mine : fill + kStageBytes;
    };
    if constexpr (kVec) {
#pragma unroll 1
      for (int i = 0; i < kStages - 1; ++i) issue();
    }
    Turn<P> f = identity<P>();
    if (rot) {
      __syncthreads();  // the tables of the previous item have been read
      fill_tables(a.rope, b, n0, a.tokens, a.N, cos_t, sin_t);
      __syncthreads();
      f = rotation<kNext, P>(cos_t + tk * (rot >> 1), sin_t + tk * (rot >> 1), t, rot, -1.0f);
    }
    uint32_t take = mine;
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
      if (a.dy[side].p == nullptr) continue;
      const int norm = a.norm[side].on, heads = a.dy[side].H, turns = (heads + per - 1) / per;
      const float eps = a.norm[side].eps;
      const Row<P> w = lane_weight<kVec, P>(s_w[side], p);
      const RowsOut& dx = a.dx[side];
      char* op = static_cast<char*>(dx.p) +
                 (b * dx.stride[0] + n * dx.stride[2] + sub * dx.stride[1]) * (dx.f32 ? 4 : 2);
      const int64_t ostep = dx.stride[1] * per * (dx.f32 ? 4 : 2);
      Row<P> dw;
#pragma unroll
      for (int i = 0; i < P; ++i) dw.v[i] = make_float2(0.0f, 0.0f);
      int head = n < a.N ? sub : heads;
      for (int k = 0; k < turns; ++k) {
        Raw<P, kVec, kGF32> graw;
        Raw<P, kVec, kXF32> xraw;
        if constexpr (kVec) {
          issue();
          copy_wait<kStages - 1>();
          read_raw<P, kGF32, kPrepThreads>(take, graw);
          read_raw<P, kXF32, kPrepThreads>(take + kXOffset, xraw);
          take = take == mine + (kStages - 1) * kStageBytes ? mine : take + kStageBytes;
        } else {
          clear_raw(graw);
          clear_raw(xraw);
          if (head < heads) {
            const RowsIn &dy = a.dy[side], &in = a.x[side];
            load_raw(row_ptr(dy.p, kGF32, b * dy.stride[0] + n * dy.stride[2] + head * dy.stride[1]), p, graw);
            if (norm) load_raw(row_ptr(in.p, kXF32, b * in.stride[0] + n * in.stride[2] + head * in.stride[1]), p, xraw);
          }
        }
        Row<P> y = apply<kNext>(unpack(graw), f, p, rot, a.D);
        if (norm) norm_gradient<T>(y, unpack(xraw), w, eps, inv_d, head < heads, dw);
        if (head < heads) store_row<kVec>(op, dx.f32, p, y);
        op += ostep;
        head += per;
      }
#pragma unroll
      for (int i = 0; i < 2 * P; ++i)
        if (has<P>(p, i)) red[side][grp][element<P>(p, i)] += at(dw, i);
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

template <int T, int P, bool kNext, bool kVec, bool kXF32, bool kGF32>
cudaError_t launch_bwd_one(const PrepBwdArgs& a, int ctas, cudaStream_t st) {
  auto kern = prep_bwd_kernel<T, P, kNext, kVec, kXF32, kGF32>;
  constexpr int kRing = kVec ? kBwdStages * (slot_bytes(P, kXF32) + slot_bytes(P, kGF32)) : 0;
  const int bytes = kRing + a.tokens * a.rope.rot * 4;
  static SmemLimit limit;  // the largest tables: a token of 128 elements for each group
  const cudaError_t e = limit.raise(kern, kRing + kPrepThreads / T * 128 * 4);
  if (e != cudaSuccess) return e;
  kern<<<ctas, kPrepThreads, bytes, st>>>(a);
  return cudaGetLastError();
}
template <int T, int P, bool kNext, bool kVec>
cudaError_t launch_bwd_t(const PrepBwdArgs& a, int ctas, bool xf32, bool gf32, cudaStream_t st) {
  if (xf32)
    return gf32 ? launch_bwd_one<T, P, kNext, kVec, true, true>(a, ctas, st)
                : launch_bwd_one<T, P, kNext, kVec, true, false>(a, ctas, st);
  return gf32 ? launch_bwd_one<T, P, kNext, kVec, false, true>(a, ctas, st)
              : launch_bwd_one<T, P, kNext, kVec, false, false>(a, ctas, st);
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
  const bool next = a.rope.rot == 0 || a.rope.interleaved;
  const Layout l = layout_of(a.D, a.rope.rot, next, a.vec, 4);
  // As many tokens a CTA as leave eight CTAs an SM (a group's factors serve all
  // heads of its token); one token a CTA, and its heads cut into runs of one
  // turn of the groups, where even that does not (a decode step).
  a.tokens = tokens_of(l.T, a.B, a.N, 8 * num_sms);
  a.heads = heads;
  if (static_cast<int64_t>(a.B) * ((a.N + a.tokens - 1) / a.tokens) < 4 * num_sms) a.heads = kPrepThreads / l.T;
  auto kern = !l.vec     ? (next ? prep_kernel<32, 4, true, false> : prep_kernel<32, 4, false, false>)
              : l.T == 8 ? (next ? prep_kernel<8, 4, true, true> : prep_kernel<8, 4, false, true>)
                         : (next ? prep_kernel<16, 4, true, true> : prep_kernel<16, 4, false, true>);
  const dim3 grid((a.N + a.tokens - 1) / a.tokens, (heads + a.heads - 1) / a.heads, a.B);
  kern<<<grid, kPrepThreads, a.tokens * a.rope.rot * 4, st>>>(a);
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
      one.dy[1 - side] = one.x[1 - side] = RowsIn{};
      one.dw[1 - side] = nullptr;
      const cudaError_t e = launch_prep_bwd(one, st);
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }
  const bool next = a.rope.rot == 0 || a.rope.interleaved;
  const Layout l = layout_of(a.D, a.rope.rot, next, a.vec, 4);
  a.tokens = tokens_of(l.T, a.B, a.N, kPrepBwdMaxCtas / 2);
  const int64_t items = static_cast<int64_t>(a.B) * ((a.N + a.tokens - 1) / a.tokens);
  const int ctas = static_cast<int>(items < kPrepBwdMaxCtas ? items : kPrepBwdMaxCtas);
  const bool gf32 = a.dy[a.dy[0].p ? 0 : 1].f32, xf32 = a.x[a.x[0].p ? 0 : 1].f32;
  cudaError_t e;
  if (!l.vec)
    e = next ? launch_bwd_t<32, 4, true, false>(a, ctas, xf32, gf32, st)
             : launch_bwd_t<32, 4, false, false>(a, ctas, xf32, gf32, st);
  else if (l.T == 16)
    e = next ? launch_bwd_t<16, 4, true, true>(a, ctas, xf32, gf32, st)
             : launch_bwd_t<16, 4, false, true>(a, ctas, xf32, gf32, st);
  else
    e = next ? launch_bwd_t<8, 4, true, true>(a, ctas, xf32, gf32, st)
             : launch_bwd_t<8, 4, false, true>(a, ctas, xf32, gf32, st);
  if (e != cudaSuccess || (a.dw[0] == nullptr && a.dw[1] == nullptr)) return e;
  prep_dw_kernel<<<dim3((a.D + 7) / 8, 2), 1024, 0, st>>>(a.partial, ctas, a.D, a.dw[0], a.dw[1]);
  return cudaGetLastError();
}

}  // namespace fa
