// Appending new keys and values to a dense or paged KV cache in bf16, fp32 or
// e4m3 with a scale per block of tokens and head; keys (and the queries of the
// same tokens) are normed and rotated on the way.  Contract and the rule for
// the scales: include/flexattn.h.
//
// A CTA owns an aligned chunk of one sequence's slots (32, or one scale block
// where that is longer) and a run of heads of k, of v or of q.  A scale block
// never spans two chunks, so its largest magnitude is found inside the CTA: the
// rows stay in registers between the pass that finds it and the pass that
// rounds, and each new value is read once.  The maximum goes through shared
// memory atomics on the bits of non-negative floats, which gives the same
// result in every order.  Angles are computed once per token of the chunk and
// shared by the CTA's heads.
#include "headprep.cuh"
#include "smem_limit.h"

namespace fa {
namespace {

// A CTA has 32 groups: of 8 lanes, or whole warps for rows read one element at
// a time.
constexpr int kGroups = 32;
constexpr int threads_of(int T) { return kGroups * T; }
constexpr int kMaxChunk = 128;

// 2^ceil(log2(amax / 448)) from the bits of a finite amax >= 0; 0 for 0.
// 448 = 1.75 * 2^8: the exponent of amax less 8, and one more past 1.75.
__device__ __forceinline__ float pow2_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  if (u == 0u) return 0.0f;
  int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(e, -126);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Four floats as e4m3 codes (round to nearest even, +-448 at most, NaN kept).
__device__ __forceinline__ uint32_t e4m3x4(float2 x, float2 y) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code & 0xffu), __NV_E4M3);
  return __half2float(__half(h));
}

// Where one sequence's new tokens go.
struct Span {
  int start, count;  // first slot, tokens
  bool bad;          // something was refused
};
__device__ __forceinline__ Span append_span(const AppendArgs& a, int b) {
  Span s;
  s.start = __ldg(a.cache_len + b);
  s.count = a.new_len ? __ldg(a.new_len + b) : a.N;
  s.bad = s.count < 0 || s.count > a.N;
  s.count = min(max(s.count, 0), a.N);
  const int cap = a.page_table ? a.page_size * a.pages_per_seq : a.page_size;
  if (s.start < 0 || s.start > cap) {
    s.bad = s.bad || s.start < 0 || s.count > 0;
    s.count = 0;
    s.start = 0;
  } else if (s.count > cap - s.start) {
    s.bad = true;
    s.count = cap - s.start;
  }
  return s;
}

// Queries of ntok tokens from n0 on and nh heads from hq0 on.
template <int T, int P, bool kNext, bool kVec, bool kF32>
__device__ __forceinline__ void append_queries(const AppendArgs& a, int b, int n0, int ntok, int hq0, int nh,
                                               const float* cos_t, const float* sin_t, const float* s_w) {
  constexpr int U = 2;
  const int t = threadIdx.x % T, grp = threadIdx.x / T, rot = a.rope.rot;
  const Place p = place_of<P, kNext>(t, rot, a.E);
  const int rows = ntok * nh;
  for (int r0 = 0; r0 < rows; r0 += U * kGroups) {
    Raw<P, kVec, kF32> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = min(r0 + u * kGroups + grp, rows - 1), n = n0 + r % ntok, h = hq0 + r / ntok;
      load_raw(row_ptr(a.q.p, kF32, b * a.q.stride[0] + h * a.q.stride[1] + n * a.q.stride[2]), p, raw[u]);
    }
    if (r0 == 0) __syncthreads();  // the angles and weights: the first loads go ahead of them
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (r0 + u * kGroups >= rows) break;  // the same for the whole CTA
      const int r = min(r0 + u * kGroups + grp, rows - 1), tk = r % ntok, n = n0 + tk, h = hq0 + r / ntok;
      Row<P> x = unpack(raw[u]);
      if (a.q_norm.on)
        x = product(scaled(x, norm_factor<T>(x, a.q_norm.eps, 1.0f / static_cast<float>(a.E))),
                    lane_weight<kVec, P>(s_w, p));
      if (rot)
        x = apply<kNext>(x, rotation<kNext, P>(cos_t + tk * (rot >> 1), sin_t + tk * (rot >> 1), t, rot, 1.0f), p, rot,
                         a.E);
      if (r0 + u * kGroups + grp < rows)
        store_row<kVec>(row_ptr(a.q_out.p, a.q_out.f32,
                                b * a.q_out.stride[0] + h * a.q_out.stride[1] + n * a.q_out.stride[2]),
                        a.q_out.f32, p, x);
    }
  }
}

// The new rows of heads h0 .. h1 - 1 of one chunk (keys or values): normed,
// turned, and written; the next head's rows are loaded while this one's are
// rounded.
template <int T, int P, bool kNext, bool kVec, int kIters, bool kF32, bool kE4m3>
__device__ __forceinline__ void append_rows(const AppendArgs& a, const RowsIn& in, int b, int h0, int h1, int slot0,
                                            const Span& sp, int end, const Place& p, int D, bool turn, bool norm,
                                            bool is_k, const float* cos_t, const float* sin_t, const float* s_w,
                                            const int* s_outer, const int64_t* s_row, uint32_t (&s_amax)[2][32],
                                            float (&s_inv)[2][32], float (&s_old)[2][32]) {
  const int t = threadIdx.x % T, grp = threadIdx.x / T;
  const int rot = a.rope.rot, h2 = rot >> 1;
  const int sb_log = kE4m3 ? __ffs(a.scale_block) - 1 : 5;
  float* scales = is_k ? a.k_scale : a.v_scale;
  char* cache = static_cast<char*>(is_k ? a.kc : a.vc);
  const int64_t hstep = is_k ? a.kc_stride[1] : a.vc_stride[1];
  const bool cvec = is_k ? a.kc_vec : a.vc_vec;
  const float inv_d = 1.0f / static_cast<float>(D);
  Raw<P, kVec, kF32> raw[kIters];
  auto load = [&](int h) {
    const int64_t off = b * in.stride[0] + h * in.stride[1];
#pragma unroll
    for (int it = 0; it < kIters; ++it) {
      const int n = slot0 - sp.start + grp + it * kGroups;
      if (n >= 0 && n < sp.count)
        load_raw(row_ptr(in.p, kF32, off + n * in.stride[2]), p, raw[it]);
      else
        clear_raw(raw[it]);
    }
  };
  load(h0);
  __syncthreads();  // tables, weights, pages and cleared maxima
  Row<P> w;
  if (norm) w = lane_weight<kVec, P>(s_w, p);
  for (int h = h0; h < h1; ++h) {
    const int par = (h - h0) & 1;
    Row<P> x[kIters];
#pragma unroll
    for (int it = 0; it < kIters; ++it) x[it] = unpack(raw[it]);
#pragma unroll
    for (int it = 0; it < kIters; ++it) {
      const int row = it * kGroups + grp;
      if (norm) x[it] = product(scaled(x[it], norm_factor<T>(x[it], a.k_norm.eps, inv_d)), w);
      if (turn)
        x[it] = apply<kNext>(x[it], rotation<kNext, P>(cos_t + row * h2, sin_t + row * h2, t, rot, 1.0f), p, rot, D);
      if constexpr (kE4m3) {
        // this row's largest finite magnitude (rows without a new token: 0);
        // the maximum passes over NaN by itself, infinities are rare
        float m = 0.0f;
        const int n = slot0 + row - sp.start;
        if (n >= 0 && n < sp.count) {
#pragma unroll
          for (int i = 0; i < P; ++i) m = max3f(m, fabsf(x[it].v[i].x), fabsf(x[it].v[i].y));
          if (m == INFINITY) {
            m = 0.0f;
#pragma unroll
            for (int i = 0; i < 2 * P; ++i) m = fmaxf(m, fabsf(at(x[it], i)) < INFINITY ? fabsf(at(x[it], i)) : 0.0f);
          }
        }
#pragma unroll
        for (int o = T / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (t == 0 && m > 0.0f) atomicMax(&s_amax[par][row >> sb_log], __float_as_uint(m));
      }
    }
    if (h + 1 < h1) load(h + 1);
    if constexpr (kE4m3) {
      __syncthreads();
      const int blk = threadIdx.x;
      if (blk < 32) s_amax[1 - par][blk] = 0u;
      if (blk < (a.chunk >> sb_log)) {
        const int bs = slot0 + (blk << sb_log), first = max(bs, sp.start);
        // touched by a new token, and that token's page is in the pool
        if (first < min(bs + a.scale_block, end) && s_outer[first - slot0] >= 0) {
          float* sc = scales + (static_cast<int64_t>(s_outer[first - slot0]) * in.H + h) * a.scales_per_outer +
                      (bs % a.page_size) / a.scale_block;
          const float fresh = pow2_scale(__uint_as_float(s_amax[par][blk]));
          const bool had = bs < sp.start;
          const float old = had ? *sc : 0.0f, now = had ? fmaxf(old, fresh) : fresh;
          // scale 0: nothing but zeros, infinities (+-448, not 0 * inf) and NaN
          s_inv[par][blk] = now > 0.0f ? 1.0f / now : 1.0f;
          s_old[par][blk] = now > old ? old : -1.0f;  // -1: older codes stay as they are
          if (!had || now != old) *sc = now;
        } else {
          s_old[par][blk] = -1.0f;
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int it = 0; it < kIters; ++it) {
      const int row = it * kGroups + grp, slot = slot0 + row;
      if (s_row[row] < 0) continue;
      const int64_t off = s_row[row] + h * hstep;
      if constexpr (!kE4m3) {
        if (slot < sp.start) continue;
        const int f32 = a.dtype == FA_DTYPE_F32;
        if (kVec && cvec)
          store_row<true>(row_ptr(static_cast<void*>(cache), f32, off), f32, p, x[it]);
        else
          store_row<false>(row_ptr(static_cast<void*>(cache), f32, off), f32, p, x[it]);
      } else {
        const float inv = s_inv[par][row >> sb_log];
        uint8_t* dst = reinterpret_cast<uint8_t*>(cache) + off;
        Row<P> y;
        if (slot >= sp.start) {
          y = scaled(x[it], inv);
        } else {
          // an older token of a block: rounded again where its scale grew
          const float old = s_old[par][row >> sb_log];
          if (old < 0.0f) continue;
#pragma unroll
          for (int i = 0; i < 2 * P; ++i)
            put(y, i, has<P>(p, i) ? e4m3_value(dst[element<P>(p, i)]) * (old * inv) : 0.0f);
        }
        uint32_t code[P / 2];
#pragma unroll
        for (int i = 0; i < P / 2; ++i) code[i] = e4m3x4(y.v[2 * i], y.v[2 * i + 1]);
        if (kVec && cvec) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            if (!(q ? p.nb : p.na)) continue;
            uint8_t* d = dst + (q ? p.b : p.a);
            if constexpr (P == 8)
              *reinterpret_cast<uint2*>(d) = make_uint2(code[2 * q], code[2 * q + 1]);
            else
              *reinterpret_cast<uint32_t*>(d) = code[q];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 2 * P; ++i)
            if (has<P>(p, i)) dst[element<P>(p, i)] = static_cast<uint8_t>(code[i >> 2] >> (8 * (i & 3)));
        }
      }
    }
  }
}

template <int T, int P, bool kNext, bool kVec, int kIters, bool kF32, bool kE4m3>
__global__ void __launch_bounds__(threads_of(T), T == 8 ? 2 : 1) append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int kThreads = threads_of(T);
  extern __shared__ __align__(16) float tables[];  // cosines, then sines, of the chunk's tokens
  __shared__ __align__(16) float s_w[128];
  __shared__ int64_t s_row[kMaxChunk];
  __shared__ int s_outer[kMaxChunk];
  __shared__ uint32_t s_amax[2][32];  // by parity of the head: a head's maxima are
  __shared__ float s_inv[2][32], s_old[2][32];  // cleared while the one before is rounded
  const int b = blockIdx.z, t = threadIdx.x % T, grp = threadIdx.x / T;
  const int rot = a.rope.rot, h2 = rot >> 1;
  float* cos_t = tables;
  float* sin_t = tables + a.chunk * h2;
  const int kv_runs = (a.k.H + a.k_heads - 1) / a.k_heads;
  const Span sp = append_span(a, b);
  if (sp.bad && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) record_error(a.status, FA_ERR_PARAM);
  const int* pos_row =
      a.rope.pos ? a.rope.pos + static_cast<int64_t>(a.rope.pos_batch > 1 ? b : 0) * a.N : nullptr;
  const int pos0 = __ldg(a.cache_len + b);
  // Angles of `count` tokens from n0 on into the tables from row `to` on.
  auto fill = [&](int n0, int count, int to) {
    // (Every eighth angle and products of complex numbers between them saved
    // 4 of 39 us on the prompt below, but moved 2.5 times as many codes across
    // a tie.)
    float *ct = cos_t + to * h2, *st = sin_t + to * h2;
    int k = threadIdx.x / h2, f = threadIdx.x - k * h2;  // stepped without divisions
    const int dk = kThreads / h2, df = kThreads - dk * h2;
    while (k < count) {
      const int n = n0 + k;
      const int pos =
          pos_row ? __ldg(pos_row + n) : static_cast<int>(static_cast<uint32_t>(pos0) + static_cast<uint32_t>(n));
      const float2 z = angle(pos, __ldg(a.rope.inv_freq + f));
      ct[k * h2 + f] = z.x;
      st[k * h2 + f] = z.y;
      k += dk;
      f += df;
      if (f >= h2) {
        f -= h2;
        ++k;
      }
    }
  };

  if (static_cast<int>(blockIdx.y) >= 2 * kv_runs) {
    // ------------------------------------------------------------- queries
    const int n0 = blockIdx.x * a.chunk, ntok = min(a.chunk, a.N - n0);
    if (ntok <= 0) return;
    const int hq0 = (blockIdx.y - 2 * kv_runs) * a.q_heads, nh = min(a.q_heads, a.q.H - hq0);
    if (rot) fill(n0, ntok, 0);
    if (a.q_norm.on) stage_weight(a.q_norm, a.E, 128, s_w);
    append_queries<T, P, kNext, kVec, kF32>(a, b, n0, ntok, hq0, nh, cos_t, sin_t, s_w);
    return;
  }

  // ------------------------------------------------------- keys or values
  const bool is_k = static_cast<int>(blockIdx.y) < kv_runs;
  const int h0 = (is_k ? blockIdx.y : blockIdx.y - kv_runs) * a.k_heads;
  const int end = sp.start + sp.count;  // past the last new slot
  const int64_t first_slot = (static_cast<int64_t>(sp.start / a.chunk) + blockIdx.x) * a.chunk;
  if (sp.count == 0 || first_slot >= end) return;
  const int slot0 = static_cast<int>(first_slot);
  const int D = is_k ? a.E : a.Ev;
  const RowsIn& in = is_k ? a.k : a.v;
  const bool turn = is_k && rot, norm = is_k && a.k_norm.on;
  const Place p = place_of<P, kNext>(t, is_k ? rot : 0, D);
  // page (or sequence) of each slot of the chunk that the call touches, and the
  // slot's offset in the cache; -1: none
  const int64_t* cs = is_k ? a.kc_stride : a.vc_stride;
  for (int i = threadIdx.x; i < a.chunk; i += kThreads) {
    const int slot = slot0 + i;
    int outer = -1;
    if (slot < end) {
      if (!a.page_table) {
        outer = b;
      } else {
        outer = __ldg(a.page_table + static_cast<int64_t>(b) * a.pages_per_seq + slot / a.page_size);
        if (outer < 0 || outer >= a.num_outer) {
          // an id outside the pool is an error only where a new token needs it
          if (slot >= sp.start) record_error(a.status, FA_ERR_PARAM);
          outer = -1;
        }
      }
    }
    s_outer[i] = outer;
    s_row[i] = outer < 0 ? -1 : outer * cs[0] + static_cast<int64_t>(slot % a.page_size) * cs[2];
  }
  if (turn) {
    const int from = max(slot0, sp.start);
    fill(from - sp.start, min(end, slot0 + a.chunk) - from, from - slot0);
  }
  if (norm) stage_weight(a.k_norm, D, 128, s_w);
  if (threadIdx.x < 64) s_amax[threadIdx.x >> 5][threadIdx.x & 31] = 0u;
  const int h1 = min(h0 + a.k_heads, in.H);
  append_rows<T, P, kNext, kVec, kIters, kF32, kE4m3>(a, in, b, h0, h1, slot0, sp, end, p, D, turn, norm, is_k, cos_t,
                                                      sin_t, s_w, s_outer, s_row, s_amax, s_inv, s_old);
}

template <int T, int P, bool kNext, bool kVec, int kIters, bool kF32, bool kE4m3>
cudaError_t launch_append_one(const AppendArgs& a, dim3 grid, size_t smem, cudaStream_t st) {
  auto kern = append_kernel<T, P, kNext, kVec, kIters, kF32, kE4m3>;
  if (smem > 40 * 1024) {
    static SmemLimit limit;  // only chunks of 128 slots come here
    const cudaError_t e = limit.raise(kern, kMaxChunk * 64 * 2 * 4);
    if (e != cudaSuccess) return e;
  }
  kern<<<grid, threads_of(T), smem, st>>>(a);
  return cudaGetLastError();
}
// The kernel for a row layout, a chunk and the types.
template <int T, int P, bool kNext, bool kVec, bool kF32>
cudaError_t launch_append_t(const AppendArgs& a, dim3 grid, size_t smem, cudaStream_t st) {
  if (a.dtype != FA_DTYPE_E4M3) return launch_append_one<T, P, kNext, kVec, 1, kF32, false>(a, grid, smem, st);
  if (a.chunk == 32) return launch_append_one<T, P, kNext, kVec, 1, kF32, true>(a, grid, smem, st);
  if (a.chunk == 64) return launch_append_one<T, P, kNext, kVec, 2, kF32, true>(a, grid, smem, st);
  return launch_append_one<T, P, kNext, kVec, 4, kF32, true>(a, grid, smem, st);
}
template <int T, int P, bool kVec>
cudaError_t launch_append_l(const AppendArgs& a, bool next, dim3 grid, size_t smem, cudaStream_t st) {
  if (a.k.f32)
    return next ? launch_append_t<T, P, true, kVec, true>(a, grid, smem, st)
                : launch_append_t<T, P, false, kVec, true>(a, grid, smem, st);
  return next ? launch_append_t<T, P, true, kVec, false>(a, grid, smem, st)
              : launch_append_t<T, P, false, kVec, false>(a, grid, smem, st);
}

}  // namespace

cudaError_t launch_append(AppendArgs a, int num_sms, cudaStream_t st) {
  const bool next = a.rope.rot == 0 || a.rope.interleaved;
  const Layout l = layout_of(a.E > a.Ev ? a.E : a.Ev, a.rope.rot, next, a.k_vec && a.v_vec && (!a.q.p || a.q_vec), 8);
  a.chunk = a.dtype == FA_DTYPE_E4M3 && a.scale_block > 32 ? a.scale_block : 32;
  // N tokens that start anywhere in a chunk touch this many chunks at most
  const int chunks = static_cast<int>((static_cast<int64_t>(a.N) + a.chunk - 2) / a.chunk) + 1;
  // Heads of k share the chunk's angles, and all heads its start-up (lengths,
  // pages), so a CTA takes several: enough to leave eight CTAs an SM, or two,
  // which run at once, where there is little but the start-up.  Eight prompts
  // of 2048 tokens, 8 heads, inputs not in L2: 72 us with 1 head a CTA, 52 with
  // 2, 43 with 4 and 44 with 8; 8191 tokens into bf16 pages: 30, 20.5, 17.3 and
  // 16.4; one token of 32 sequences (graph replay): 9.9, 8, 11.5, 18.
  const int64_t per_head = static_cast<int64_t>(chunks) * a.B, most = (a.N >= kGroups ? 8 : 2) * num_sms;
  a.k_heads = 1;
  while (a.k_heads < a.k.H && 2 * per_head * ((a.k.H + a.k_heads - 1) / a.k_heads) > most &&
         (a.N >= kGroups || a.k_heads < 2))
    a.k_heads *= 2;
  const int ntok = a.N < a.chunk ? a.N : a.chunk;
  a.q_heads = ntok < kGroups ? (kGroups + ntok - 1) / ntok : 8;
  const int kv_runs = (a.k.H + a.k_heads - 1) / a.k_heads;
  const int q_runs = a.q.p ? (a.q.H + a.q_heads - 1) / a.q_heads : 0;
  const dim3 grid(chunks, 2 * kv_runs + q_runs, a.B);
  const size_t smem = static_cast<size_t>(a.chunk) * (a.rope.rot / 2) * 2 * sizeof(float);
  if (!l.vec) return launch_append_l<32, 4, false>(a, next, grid, smem, st);
  return l.P == 8 ? launch_append_l<8, 8, true>(a, next, grid, smem, st)
                  : launch_append_l<8, 4, true>(a, next, grid, smem, st);
}

}  // namespace fa
