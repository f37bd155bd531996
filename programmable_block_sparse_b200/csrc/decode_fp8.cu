// Split-KV decode over an e4m3 cache: codes under one fp32 scale per block of
// slots and head (definition: include/flexattn.h, flexattn_forward_fp8).
//
// A step streams every code of the visible cache once, so HBM is the bound and
// the codes must reach the tensor cores without a conversion pass over them
// (at this rate an SM has 23 bytes a clock to take; widening every code and
// writing it back to shared memory would cost more issue slots than the whole
// softmax).  So the products run on e4m3 operands (tcgen05 kind::f8f6f4) and
// the other operands are made to fit exactly or nearly so:
//
//   * a bf16 query value has 8 significant bits.  Divided by a power of two s_r
//     that brings its row below 448, it is the sum of two e4m3 terms: hi, its
//     rounding to 4 bits, and lo / 16, what is left, a multiple of its last
//     place of at most 4 bits.  The sum is exact for values down to 2^-14 of
//     the row's largest, and off by 2^-22 of that one at most below.
//   * a softmax weight w needs range as well as precision: beside a key that
//     takes nearly all of the weight (an attention sink) thousands of small
//     ones make up the rest.  Two e4m3 terms end at 2^-20 of the largest.  So w
//     is three e5m2 terms, a + b / 8 + c / 64, which beside e4m3 codes the
//     products take as they are: e5m2 is the upper byte of fp16, so a term is
//     the upper byte of what the terms before it leave, and only the last one
//     is rounded.  2^-8 w at most down to 2^-27 of the row's largest weight
//     (2^-11 w in the mean square), 2^-35 of that largest one below.
//
// The terms are columns of the small N side (Cfg).  With s^k_j, s^v_j the
// scales of key j, c_j the codes, in log2 units:
//   t_rj  = rule(s_r s^k_j scale (hi_r + lo_r / 16) . c^k_j)
//   w_rj  = 2^(t_rj + log2 s^v_j - m_r + 13),  m_r the running maximum of
//           t + log2 s^v, moved when some key passes it by more than 2, so
//           that w <= 2^15 stays inside e5m2 (and fp16)
//   O_r   = sum_j w_rj c^v_j,   l_r = sum_j w_rj / s^v_j,   out = O_r / l_r.
// Carrying the value scale inside the weight keeps it out of the codes and
// bounds the weights' rounding against the largest contribution to the output.
//
// Layout: the 128 keys of a tile are the M side of both products (S^T = K Q^T,
// O^T = V^T W^T with V read MN-major), as in decode.cu: a softmax thread owns
// one key, its TMEM lane, and the 16 rows' scores.  Rows of 128 bytes with a
// 128-byte swizzle; a head dim below 128 is padded with zeros by TMA.
//   warp 0      TMA: one box per page piece, a lane each.
//   warp 1      TMEM allocation; one thread issues the MMAs, whichever product
//               is ready first.
//   warps 2-    softmax (warp % 4 is the TMEM lane quadrant), epilogue.
// Measured: 32 sequences of 4k..32k keys, 32 heads on 8, head dim 128: one query
// 171 us for 1.10 GB of codes and scales (6.42 TB/s, the copy rate), two
// queries (8 rows) 184 us, four 230 us, where the softmax of 16 rows a key is the
// bound; one sequence of 32k keys 18.6 us, of which about 7 are a CTA's start,
// one tile and its end.
#include <cuda_fp8.h>
#include <math.h>

#include "common.cuh"
#include "fastmath.cuh"
#include "launch.h"
#include "mods.cuh"
#include "smem_limit.h"

namespace fa {
namespace {

constexpr int kKeys = 128;        // keys per tile: the M side
constexpr int kMaxRows = 16;      // query rows per CTA
constexpr int kTileBytes = kKeys * 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Start of the running maximum: finite and below any real score.
constexpr float kNoKeyMax = -1.0e30f;
// The maximum moves when a key passes it by more than kSlack; weights carry
// 2^kShift, so they stay at or below 2^(kSlack + kShift) = 32768 < 57344.
constexpr float kSlack = 2.0f;
constexpr float kShift = 13.0f;
// Value scales below this one, 2^-80, count as it.  A weight's exponent carries
// its key's value scale, so the smaller it may be, the sooner the key's share of
// the softmax leaves fp32 beside a large scale; and the share is the weight
// divided by the scale, 2^(15 + 80) at most, of which 2^30 keys still add up.
constexpr float kLeastScale = 8.271806125530277e-25f;

// A CTA of R = 4, 8 or 16 query rows: the softmax works on R scores a key, so
// fewer rows are that much less work (one query of a group of 4 heads on 16
// rows took 330 us where 4 rows take 232).  Sixteen rows go to two sets of four
// softmax warps, 8 rows each, which share the tiles but nothing else.  CTAs of
// up to 8 rows leave registers for three an SM.  Rings of 4 tiles (192 KB in
// flight an SM), or of 5 with 16 rows, whose two CTAs have larger operands.
//
// N side, in groups of 8 rows of 128 bytes (M = 128 takes N in 16s):
//   Q: hi at row 0, lo at row R.
//   weights, R = 4: a at 0, b at 4, c at 8, and 4 rows of zeros;
//            R = 16: a at 0, b at 16, c at 32 (N = 48);
//            R = 8: a, b and c are one group each, and N = 24 is none, so two
//            products, (a, b) and (b, c): the second b's columns are not read.
template <int R>
struct Cfg {
  static constexpr int kSets = R == 16 ? 2 : 1;           // sets of softmax warps
  static constexpr int kOwn = R / kSets;                  // rows of a set
  static constexpr int kThreads = 64 + 128 * kSets;
  static constexpr int kQCols = 2 * R < 16 ? 16 : 2 * R;  // N of K Q^T
  static constexpr int kWCols = R == 16 ? 48 : 16;        // N of V^T W^T
  static constexpr int kWParts = R == 8 ? 2 : 1;          // its products
  static constexpr int kCtas = R <= 8 ? 3 : 2;
  static constexpr int kRing = R <= 8 ? 4 : 5;            // K or V tiles of 16 KB in flight
  static constexpr int kO = 2 * kQCols;                   // TMEM: two S^T buffers, then O^T
  static constexpr int kTmemCols = R <= 8 ? 64 : 128;
  static constexpr int kQBytes = kQCols * 128;
  static constexpr int kWBytes = R == 4 ? 2048 : 3 * R * 128;  // one of two buffers of weights
  static constexpr int kSmemBytes = kRing * kTileBytes + kQBytes + 2 * kWBytes + 1024;
  static_assert(kO + kWParts * kWCols <= kTmemCols, "TMEM columns");
  // 8-column loads that take a set's columns of O^T: where the i-th begins (the
  // set's first row added by the caller).  Four rows lie side by side.
  static constexpr int kOLoads = R == 4 ? 2 : 3;
  static constexpr int o_col(int i) { return R == 4 ? 8 * i : R == 8 && i == 2 ? 24 : i * R; }
  // Where a term's weights go: bytes from the first term's, and the row that
  // the byte's swizzle goes by (4 rows: b shares a's group).
  static constexpr int w_bytes(int term) { return R == 4 ? (term == 2 ? 1024 : 0) : term * R * 128; }
  static constexpr int w_row(int term) { return R == 4 && term == 1 ? 4 : 0; }
};

// kind::f8f6f4 instruction descriptor: e4m3 A, e4m3 or e5m2 B, fp32 accumulator.
constexpr uint32_t idesc_f8(int M, int N, int a_mn_major, int b_e5m2) {
  return (1u << 4) | (static_cast<uint32_t>(b_e5m2) << 10) | (static_cast<uint32_t>(a_mn_major) << 15) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::
          "r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate));
}

__device__ __forceinline__ void put_byte(uint32_t saddr, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(saddr), "r"(v) : "memory");
}
// Two values as (hi, lo) e4m3 pairs: v = hi + lo / 16.
__device__ __forceinline__ void split_e4m3(float v0, float v1, uint32_t& hi, uint32_t& lo) {
  hi = __nv_cvt_float2_to_fp8x2(make_float2(v0, v1), __NV_SATFINITE, __NV_E4M3);
  const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(hi), __NV_E4M3);
  const float2 h = __half22float2(__half2(r));
  lo = __nv_cvt_float2_to_fp8x2(make_float2((v0 - h.x) * 16.0f, (v1 - h.y) * 16.0f), __NV_SATFINITE, __NV_E4M3);
}
// Two weights 0 <= v <= 2^15 as three e5m2 terms, v = a + b / 8 + c / 64: the
// bytes 1 (v0) and 3 (v1) of each word.  The first two are cut off, so that the
// next takes up what they leave, exactly; the last is rounded.  Few bits are left
// by then, so ties are common: `half` sends them up (0x80 in either half) or down
// (0x7f), by the parity of the key.  NaN stays in a.
__device__ __forceinline__ void split_e5m2(float v0, float v1, uint32_t half, uint32_t (&term)[3]) {
  auto bits = [](__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); };
  auto cut = [&](__half2 x) {  // the upper byte of each half
    const uint32_t u = bits(x) & 0xff00ff00u;
    return *reinterpret_cast<const __half2*>(&u);
  };
  const __half2 eight = __float2half2_rn(8.0f);
  const __half2 h = __floats2half2_rn(v0, v1);
  const __half2 r = __hmul2(__hsub2(h, cut(h)), eight);
  const __half2 q = __hmul2(__hsub2(r, cut(r)), eight);
  term[0] = bits(h);
  term[1] = bits(r);
  term[2] = bits(q) + half;
}

template <int kRing>
struct Bars {
  uint64_t full[kRing], empty[kRing];
  uint64_t s_full[2], s_free[2], p_full[2], p_free[2], o_final;
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ int listed_tile(const FwdArgs& a, int64_t brow, int nfull, int j) {
  return j < nfull ? __ldg(a.bm.full_kv_indices + brow * a.bm.Nb + j)
                   : __ldg(a.bm.kv_indices + brow * a.bm.Nb + (j - nfull));
}

// Reduce-scatter of R values per lane over a warp: every lane gets the
// reduction over all lanes of value (lane * R / 32).
template <bool kMax, int R>
__device__ __forceinline__ float reduce_rows(const float (&v)[R], int lane) {
  auto op = [](float x, float y) { return kMax ? fmaxf(x, y) : x + y; };
  float a[R];
#pragma unroll
  for (int i = 0; i < R; ++i) a[i] = v[i];
  int d = 16;
#pragma unroll
  for (int w = R / 2; w >= 1; w >>= 1, d >>= 1) {
    const bool up = lane & d;
#pragma unroll
    for (int i = 0; i < w; ++i) a[i] = op(up ? a[w + i] : a[i], __shfl_xor_sync(0xffffffffu, up ? a[i] : a[w + i], d));
  }
#pragma unroll
  for (; d >= 1; d >>= 1) a[0] = op(a[0], __shfl_xor_sync(0xffffffffu, a[0], d));
  return a[0];
}

// 32 lanes x 32 bit, 8 consecutive columns per thread.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
// The hi columns (from taddr on) and lo columns (from taddr + R on) of N rows
// of a thread's TMEM lane.  Four rows lie side by side: one load of 8.
template <int N, int R>
__device__ __forceinline__ void tmem_rows(uint32_t taddr, uint32_t (&r)[2 * N]) {
#pragma unroll
  for (int c = 0; c < 2 * N; c += 8) tmem_ld8(taddr + (c < N ? c : c - N + R), r + c);
  tmem_wait_ld();
#pragma unroll
  for (int c = 0; c < 2 * N; ++c) asm volatile("" : "+r"(r[c]));  // no use is scheduled before the wait
}
// Likewise 8 columns of O^T.
__device__ __forceinline__ void tmem_out(uint32_t taddr, uint32_t (&o)[8]) {
  tmem_ld8(taddr, o);
  tmem_wait_ld();
#pragma unroll
  for (int c = 0; c < 8; ++c) asm volatile("" : "+r"(o[c]));
}

// The sequence of the given rank by length of its list of tiles, longest first
// (ties by index), for up to 32 sequences with lists of their own; else the
// batch order.  Called by every lane of a warp.
__device__ __forceinline__ int ranked_sequence(const FwdArgs& a, int rank) {
  if (a.B > 32 || a.B == 1 || a.bm.B == 1) return rank;
  const int lane = threadIdx.x & 31;
  int cnt = -1;
  if (lane < a.B) {
    const int64_t row = static_cast<int64_t>(lane) * a.bm.H * a.bm.Mb;
    cnt = __ldg(a.bm.full_kv_num_blocks + row) + __ldg(a.bm.kv_num_blocks + row);
  }
  int r = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const int cj = __shfl_sync(0xffffffffu, cnt, j);
    r += (cj > cnt || (cj == cnt && j < lane)) ? 1 : 0;
  }
  const unsigned hit = __ballot_sync(0xffffffffu, lane < a.B && r == rank);
  return hit ? __ffs(hit) - 1 : rank;
}

// tanh of a score under a cap: the odd series for small arguments, else
// 1 - 2 / (1 + e^(2 |y|)), whose absolute error of about 2^-22 is below 2^-20
// of the result there.
__device__ __forceinline__ float tanh_large(float y) {
  const float e = ex2_approx(2.0f * kLog2e * fabsf(y));
  return copysignf(1.0f - __fdividef(2.0f, 1.0f + e), y);
}

template <int SCORE, int R>
__global__ void __launch_bounds__(Cfg<R>::kThreads, Cfg<R>::kCtas)
    decode_fp8_kernel(const __grid_constant__ FwdArgs a, const __grid_constant__ QuantArgs qa, const Fp8Plan p,
                      const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, int box,
                      float* ws_o, float* ws_lse, float* ws_max) {
  using C = Cfg<R>;
  constexpr int kRing = C::kRing;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars<kRing> bars;
  __shared__ float s_red[2][4][R];
  __shared__ int s_qpos[R], s_head[R], s_pq[R];
  __shared__ float s_slope[R], s_unit[R], s_inv[R];
  __shared__ int64_t s_id[R], s_off[R];  // row of lse; where the row's output begins (-1: no row)
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sKV = smem;
  uint8_t* sQ = smem + kRing * kTileBytes;
  uint8_t* sP = sQ + C::kQBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // grid (KV head x row chunk, split, rank): the longest sequences start first
  const int split = blockIdx.y;
  const int hk = blockIdx.x / p.row_chunks, rc = blockIdx.x % p.row_chunks;
  const int b = ranked_sequence(a, static_cast<int>(blockIdx.z));
  const int S_b = seq_len_b(a.mask, b, a.S);
  // Rows of the chunk: R consecutive ones of the group's G x L (head, position)
  // pairs; with per-head lists, of one head's L positions.
  const int per_head = a.bm.H > 1 ? (a.L + R - 1) / R : 0;
  const int g0 = per_head ? rc / per_head : 0;
  const int rho0 = (per_head ? rc % per_head : rc) * R;
  const int rho_end = per_head ? a.L : a.G * a.L;
  const int bmb = a.bm.B > 1 ? b : 0;
  const int bmh = per_head ? hk * a.G + g0 : 0;
  const int64_t brow = (static_cast<int64_t>(bmb) * a.bm.H + bmh) * a.bm.Mb;
  const int nfull = __ldg(a.bm.full_kv_num_blocks + brow);
  const int ntiles = nfull + __ldg(a.bm.kv_num_blocks + brow);
  const int chunk = (ntiles + p.splits - 1) / p.splits;
  const int t0 = split * chunk;
  const int t1 = min(ntiles, t0 + chunk);
  const int nsub = t1 > t0 ? t1 - t0 : 0;
  volatile int* abort = &bars.abort;
  const bool has_pos = SCORE == FA_SCORE_CAP_THEN_BIAS && a.score.pos != nullptr;

  // Row and outer coordinate (batch, or page) of this lane's box of tile j.
  // Slots at or past the sequence's end are not read: a row past the tensor's
  // end makes TMA fill the box with zeros.
  const int nbox = kKeys / box;
  auto box_addr = [&](int j, int& row, int& outer) {
    const int kv = listed_tile(a, brow, nfull, t0 + j) * kKeys + lane * box;
    row = kv;
    outer = b;
    if (kv >= S_b) {
      row = a.page_table ? a.page_size : a.S;
      outer = 0;
    } else if (a.page_table) {
      outer = cache_page(a.page_table, a.pages_per_seq, a.page_size, a.num_pages, a.status, b, kv);
      row = kv - p.page.quotient(kv) * a.page_size;
    }
  };
  int row_c = 0, outer_c = 0, row_n = 0, outer_n = 0;  // this tile's box, and the next tile's
  // K (u even) or V (u odd) of tile u / 2 into ring entry u % kRing; all lanes of warp 0
  auto issue_load = [&](int u) {
    if (lane < nbox) {
      if (u == 0) {
        box_addr(0, row_c, outer_c);
        if (nsub > 1) box_addr(1, row_n, outer_n);
      } else if ((u & 1) == 0) {
        row_c = row_n;
        outer_c = outer_n;
        if ((u >> 1) + 1 < nsub) box_addr((u >> 1) + 1, row_n, outer_n);
      }
    }
    const int e = u % kRing;
    if (lane == 0) mbar_expect_tx(&bars.full[e], kTileBytes);
    __syncwarp();
    if (lane < nbox)
      tma_load_4d(sKV + e * kTileBytes + lane * box * 128, (u & 1) ? &map_v : &map_k, &bars.full[e], 0, row_c, hk,
                  outer_c);
  };

  // the combine kernel may be set up once every CTA of this grid has started
  asm volatile("griddepcontrol.launch_dependents;");
  const int first_loads = min(kRing, 2 * nsub);
  if (warp == 0) {
    if (lane == 0) {
      for (int s = 0; s < kRing; ++s) {
        mbar_init(&bars.full[s], 1);
        mbar_init(&bars.empty[s], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bars.s_full[i], 1);
        mbar_init(&bars.s_free[i], 4 * C::kSets);
        mbar_init(&bars.p_full[i], 4 * C::kSets);
        mbar_init(&bars.p_free[i], 1);
      }
      mbar_init(&bars.o_final, 1);
      bars.abort = 0;
      mbar_fence_init();
      if (nsub > 0) {
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
      }
    }
    __syncwarp();
    for (int u = 0; u < first_loads; ++u) issue_load(u);
  }
  if (warp == 1) {
    tmem_alloc(&bars.tmem_base, C::kTmemCols);
    if (lane < R) {
      const int rho = rho0 + lane;
      const bool ok = rho < rho_end;
      const int head = hk * a.G + (per_head ? g0 : min(rho / a.L, a.G - 1)), i = per_head ? min(rho, a.L - 1) : rho % a.L;
      const int Hs = a.score.slope_heads > 0 ? a.score.slope_heads : a.Hq;
      s_qpos[lane] = query_pos(i, a.L, S_b);
      s_head[lane] = head;
      const int64_t id = (static_cast<int64_t>(b) * a.Hq + head) * a.L + i;
      s_id[lane] = p.splits == 1 ? id : id * p.splits + split;
      s_off[lane] = !ok             ? -1
                    : p.splits == 1 ? b * a.o_stride[0] + head * a.o_stride[1] + i * a.o_stride[2]
                                    : (id * p.splits + split) * a.Ev;
      s_slope[lane] = distance_slope(head, Hs);
      s_pq[lane] = has_pos ? pos_at(a.score, b, s_qpos[lane], a.S) : 0;
    }
  }
  if (warp >= 2 && warp < 6) {
    // Query rows as hi (rows 0 .. R-1) and lo (R .. 2R-1) terms, 128-byte
    // swizzled; 8 threads a row, 16 values each; rows past 2 R are zero.
    const int r = (threadIdx.x - 64) >> 3, seg = threadIdx.x & 7;
    const int rho = rho0 + r;
    float q[16];
    float amax = 0.0f;
    bool finite = true;
    const bool ok = r < R && rho < rho_end;
    const int head = hk * a.G + (per_head ? g0 : min(rho / a.L, a.G - 1)), i = per_head ? min(rho, a.L - 1) : rho % a.L;
    const __nv_bfloat16* src =
        static_cast<const __nv_bfloat16*>(a.q) + b * a.q_stride[0] + head * a.q_stride[1] + i * a.q_stride[2];
#pragma unroll
    for (int e = 0; e < 16; ++e) q[e] = 0.0f;
    if (ok && seg * 16 < a.E) {  // E is a multiple of 16
      const uint4 v0 = *reinterpret_cast<const uint4*>(src + seg * 16);
      const uint4 v1 = *reinterpret_cast<const uint4*>(src + seg * 16 + 8);
      const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        q[2 * e] = __uint_as_float(w[e] << 16);
        q[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      }
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      finite = finite && fabsf(q[e]) < INFINITY;
      amax = fmaxf(amax, fabsf(q[e]));
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      finite = __shfl_xor_sync(0xffffffffu, static_cast<int>(finite), o) && finite;
    }
    // 2^x with amax / 2^x in (224, 448]
    const uint32_t ab = __float_as_uint(amax);
    int x = static_cast<int>(ab >> 23) - 127 - 8 + ((ab & 0x7fffffu) > 0x600000u ? 1 : 0);
    x = min(max(x, -126), 126);
    if (!finite || amax == 0.0f) x = 0;
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - x) << 23);
    // a row with an infinity or a NaN: every score, and so the output, is NaN
    if (seg == 0 && r < R) s_unit[r] = finite ? __uint_as_float(static_cast<uint32_t>(127 + x) << 23) : NAN;
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t h0, h1, l0, l1;
      split_e4m3(q[4 * c] * inv, q[4 * c + 1] * inv, h0, l0);
      split_e4m3(q[4 * c + 2] * inv, q[4 * c + 3] * inv, h1, l1);
      hi[c] = h0 | (h1 << 16);
      lo[c] = l0 | (l1 << 16);
    }
    auto place = [&](int row) { return (row >> 3) * 1024 + (row & 7) * 128 + ((seg ^ (row & 7)) << 4); };
    if (r < R) {
      *reinterpret_cast<uint4*>(sQ + place(r)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(sQ + place(r + R)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    if (R == 4 && r >= 8)  // rows that Q leaves unused, and the weights (from 12 on) in either buffer
#pragma unroll
      for (int buf = 0; buf < 3; ++buf)
        *reinterpret_cast<uint4*>(sQ + buf * C::kQBytes + place(r)) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = bars.tmem_base;

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA
    if (nsub > 0) {
      int issued = first_loads;
      for (int u = first_loads; u < 2 * nsub; ++u) {
        const bool ok = !*abort && mbar_wait(&bars.empty[u % kRing], ((u / kRing) - 1) & 1, abort, a.status, a.wait_cycles);
        if (!__all_sync(0xffffffffu, ok)) break;
        issue_load(u);
        issued = u + 1;
      }
      // every copy issued lands before this warp leaves (only the last kRing can
      // be pending: earlier entries were waited free before their reuse)
      volatile int never = 0;
      for (int u = (issued > kRing ? issued - kRing : 0); u < issued; ++u)
        mbar_wait(&bars.full[u % kRing], (u / kRing) & 1, &never, nullptr);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_f8(kKeys, C::kQCols, 0, 0);
      constexpr uint32_t idesc_o = idesc_f8(kKeys, C::kWCols, 1, 1);
      const uint64_t dk0 = umma_desc_sw128(smem_u32(sKV), 16, 1024);
      // V^T: M runs along a row of V, one 128-byte block wide; 8 keys a group
      const uint64_t dv0 = umma_desc_sw128(smem_u32(sKV), kTileBytes, 1024);
      const uint64_t dq0 = umma_desc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t dp0 = umma_desc_sw128(smem_u32(sP), 16, 1024);
      const int ksteps = (a.E + 31) / 32;  // Q and K are zero past E
      auto issue_qk = [&](int j) {
        const int e = (2 * j) % kRing, sb = j & 1;
        tc_fence_after();
        for (int kk = 0; kk < ksteps; ++kk)
          umma_f8(tbase + C::kQCols * sb, dk0 + ((e * kTileBytes + kk * 32) >> 4), dq0 + ((kk * 32) >> 4), idesc_s,
                  kk > 0 ? 1u : 0u);
        umma_commit(&bars.s_full[sb]);
        umma_commit(&bars.empty[e]);
      };
      auto issue_pv = [&](int j) {
        const int e = (2 * j + 1) % kRing, pb = j & 1;
        tc_fence_after();
#pragma unroll
        for (int part = 0; part < C::kWParts; ++part)  // from the second, one group of 8 rows further on
#pragma unroll
          for (int kk = 0; kk < kKeys / 32; ++kk)
            umma_f8(tbase + C::kO + part * C::kWCols, dv0 + ((e * kTileBytes + kk * 32 * 128) >> 4),
                    dp0 + ((pb * C::kWBytes + part * 1024 + kk * 32) >> 4), idesc_o, (j > 0 || kk > 0) ? 1u : 0u);
        umma_commit(&bars.p_free[pb]);
        umma_commit(&bars.empty[e]);
      };
      // Whichever product is ready first, but QK of tile j only after PV of
      // tile j - 2: then the commit that hands over S_j (it covers everything
      // issued before) also says that the weights' buffer of tile j - 2 is free.
      // What an entry held before (kRing loads ago: K or V of tile jq - 3 at the
      // latest, or K of tile jp - 2) went into a product that was issued before:
      // a tested barrier is never two phases behind.
      int jq = 0, jp = 0;
      long long idle_from = clock64();
      while (jp < nsub) {
        bool progressed = false;
        if (jq < nsub && jp >= jq - 1 && mbar_test(&bars.full[(2 * jq) % kRing], ((2 * jq) / kRing) & 1) &&
            (jq < 2 || mbar_test(&bars.s_free[jq & 1], ((jq - 2) >> 1) & 1))) {
          issue_qk(jq++);
          progressed = true;
        }
        if (jp < jq && mbar_test(&bars.p_full[jp & 1], (jp >> 1) & 1) &&
            mbar_test(&bars.full[(2 * jp + 1) % kRing], ((2 * jp + 1) / kRing) & 1)) {
          issue_pv(jp++);
          progressed = true;
        }
        if (progressed) {
          idle_from = clock64();
        } else if (*abort) {
          break;
        } else if (clock64() - idle_from > a.wait_cycles) {
          record_error(a.status, FA_ERR_TIMEOUT);
          *abort = 1;
          break;
        }
      }
      // every MMA issued above completes before the epilogue or TMEM release
      umma_commit(&bars.o_final);
      volatile int never = 0;
      mbar_wait(&bars.o_final, 0, &never, nullptr);
    }
  } else {
    // -------------------------------------------------------------- softmax
    constexpr int N = C::kOwn;
    const int qd = warp & 3;
    const int set = (warp - 2) >> 2, row0 = set * N;  // this set's rows: row0 .. row0 + N - 1
    const int bar = 1 + set;
    const int kk = qd * 32 + lane;  // this thread's key of a tile; its TMEM lane
    const uint32_t lane_base = static_cast<uint32_t>(qd * 32) << 16;
    constexpr bool kCapped = SCORE == FA_SCORE_SOFTCAP || SCORE == FA_SCORE_CAP_THEN_BIAS;
    const float c_in = kCapped ? a.scale / a.score.cap : a.scale * kLog2e;
    const float c_out = kCapped ? a.score.cap * kLog2e : 1.0f;
    const bool want_max = a.max_scores != nullptr;
    // nms: kShift less the running maximum of t + log2 s^v, so that the weight
    // of a key is 2^(t + log2 s^v + nms)
    float2 nms[N / 2];
    float tm[N];
    // Distance bias in log2 units: slope times distance.  Positions are counted
    // from the sequence's end, where they are small for the keys that matter:
    // the distance is exact within 2^24 of it, whatever the length.
    float2 l_part[N / 2], unit[N / 2], sl2[N / 2], before[N / 2];  // before: the query's own, negated
#pragma unroll
    for (int r = 0; r < N; ++r) tm[r] = -INFINITY;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const int r = row0 + 2 * i;
      nms[i] = splat2(-kNoKeyMax);
      l_part[i] = make_float2(0.0f, 0.0f);
      unit[i] = make_float2(s_unit[r] * c_in, s_unit[r + 1] * c_in);
      sl2[i] = make_float2(s_slope[r] * kLog2e, s_slope[r + 1] * kLog2e);
      before[i] = make_float2(static_cast<float>(S_b - s_qpos[r]), static_cast<float>(S_b - s_qpos[r + 1]));
    }
    // where the first term of this key's weights goes, by row of an 8-row group
    uint32_t wx[8];
#pragma unroll
    for (int r = 0; r < 8; ++r)
      wx[r] = smem_u32(sP) + (row0 >> 3) * 1024 + r * 128 + (((kk >> 4) ^ r) << 4) + (kk & 15);
    const uint32_t half = (kk & 1) ? 0x00800080u : 0x007f007fu;
    // What the next tiles need comes ahead, a stage an iteration, since each
    // load depends on the one before: tile index, page, scales.  A loaded value
    // is first touched (scaled, clamped) an iteration later: touched at once,
    // it held the warp for 400 of a tile's 1750 cycles.
    auto page_at = [&](int kv) {  // raw: the id may lie outside the pool
      return a.page_table && kv < S_b
                 ? __ldg(a.page_table + static_cast<int64_t>(b) * a.pages_per_seq + p.page.quotient(kv))
                 : b;
    };
    auto scales_at = [&](int kv, int pg, float& ks, float& vs) {  // 1 past the sequence's end
      ks = vs = 1.0f;
      if (kv < S_b) {
        int at = kv;
        if (a.page_table) {
          pg = min(max(pg, 0), a.num_pages - 1);  // warp 0 records an id outside the pool
          at = kv - p.page.quotient(kv) * a.page_size;
        }
        const int64_t i = (static_cast<int64_t>(pg) * a.Hkv + hk) * qa.scales_per_outer + (at >> qa.block_log);
        ks = __ldg(qa.k_scale + i);
        vs = __ldg(qa.v_scale + i);
      }
    };
    const int* list_full = a.bm.full_kv_indices + brow * a.bm.Nb + t0;
    const int* list_part = a.bm.kv_indices + brow * a.bm.Nb + t0 - nfull;
    auto tile_at = [&](int j) { return __ldg((t0 + j < nfull ? list_full : list_part) + j); };
    int kv0 = 0, kv0_1 = 0, n_2 = 0, pg_1 = 0;
    float ks = 1.0f, vs = 1.0f, ks_1 = 1.0f, vs_1 = 1.0f;
    if (nsub > 0) {  // tiles past the last one repeat it
      const int n_0 = tile_at(0), n_1 = tile_at(min(1, nsub - 1));
      n_2 = tile_at(min(2, nsub - 1));
      kv0 = n_0 * kKeys;
      kv0_1 = n_1 * kKeys;
      const int pg_0 = page_at(kv0 + kk);
      pg_1 = page_at(kv0_1 + kk);
      scales_at(kv0 + kk, pg_0, ks, vs);
    }
    bool alive = true;
    for (int j = 0; j < nsub; ++j) {
      const int sb = j & 1;
      const int kv = kv0 + kk;
      const int kv0_2 = n_2 * kKeys;
      scales_at(kv0_1 + kk, pg_1, ks_1, vs_1);
      const int pg_2 = page_at(kv0_2 + kk);
      const int n_3 = tile_at(min(j + 3, nsub - 1));
      vs = fmaxf(vs, kLeastScale);  // a block of zeros has scale 0
      float lv, ivs;  // exact for powers of two; other errors, 2^-21, cancel but between blocks
      asm("lg2.approx.f32 %0, %1;" : "=f"(lv) : "f"(vs));
      asm("rcp.approx.f32 %0, %1;" : "=f"(ivs) : "f"(vs));
      bool ok = alive && __all_sync(0xffffffffu, mbar_wait(&bars.s_full[sb], (j >> 1) & 1, abort, a.status,
                                                           a.wait_cycles));
      float2 t[N / 2];  // score + log2 s^v
      float top = -INFINITY;  // of the weights' exponents
      if (ok) {
        uint32_t sr[2 * N];
        tc_fence_after();
        tmem_rows<N, R>(tbase + lane_base + C::kQCols * sb + row0, sr);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.s_free[sb]);
        const float2 kfac = splat2(ks), lv2 = splat2(lv);
        const float at = static_cast<float>(kv - S_b);
        const int pk = has_pos ? pos_at(a.score, b, kv, a.S) : kv;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          const float2 hi = make_float2(__uint_as_float(sr[2 * i]), __uint_as_float(sr[2 * i + 1]));
          const float2 lo = make_float2(__uint_as_float(sr[N + 2 * i]), __uint_as_float(sr[N + 2 * i + 1]));
          const float2 x = fma2(lo, splat2(0.0625f), hi), f = mul2(unit[i], kfac);
          if constexpr (SCORE == FA_SCORE_NONE)
            t[i] = fma2(x, f, lv2);
          else if constexpr (SCORE == FA_SCORE_ALIBI)
            t[i] = fma2(x, f, fma2(sl2[i], add2(splat2(at), before[i]), lv2));
          else
            t[i] = mul2(x, f);
        }
        if constexpr (kCapped) {
          float2 th[N / 2];
          float big = 0.0f;
          bool nan = false;
#pragma unroll
          for (int i = 0; i < N / 2; ++i) {
            float2 u2;
            th[i] = tanh_poly2(t[i], u2);
            big = max3f(big, u2.x, u2.y);
            nan = nan || !(u2.x + u2.y == u2.x + u2.y);
          }
          if (__any_sync(0xffffffffu, nan || big > kTanhPolyMax * kTanhPolyMax)) {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
              if (!(fabsf(t[i].x) <= kTanhPolyMax)) th[i].x = tanh_large(t[i].x);
              if (!(fabsf(t[i].y) <= kTanhPolyMax)) th[i].y = tanh_large(t[i].y);
            }
          }
#pragma unroll
          for (int i = 0; i < N / 2; ++i) {
            t[i] = fma2(th[i], splat2(c_out), lv2);
            if constexpr (SCORE == FA_SCORE_CAP_THEN_BIAS) {
              const int r = row0 + 2 * i;
              const int d0 = has_pos ? pk - s_pq[r] : kv - s_qpos[r], d1 = has_pos ? pk - s_pq[r + 1] : kv - s_qpos[r + 1];
              t[i] = fma2(sl2[i], make_float2(static_cast<float>(d0), static_cast<float>(d1)), t[i]);
            }
          }
        }
        // Element mask on listed-partial tiles and at the end of the sequence.
        // The rule is chosen once for all rows, so that their tests overlap
        // (rows past the CTA's stand at a valid position, are masked like any
        // other and never written).
        if (t0 + j >= nfull || kv0 + kKeys > S_b) {
          auto mask_rows = [&](auto visible) {
#pragma unroll
            for (int r = 0; r < N; ++r) {
              const bool vis = kv < S_b && visible(r, s_qpos[row0 + r]);
              float& x = (r & 1) ? t[r >> 1].y : t[r >> 1].x;
              x = vis ? x : -INFINITY;
            }
          };
          if (a.mask.kind == FA_MASK_CAUSAL)
            mask_rows([&](int, int q) { return kv <= q; });
          else if (a.mask.kind == FA_MASK_SLIDING_WINDOW)
            mask_rows([&](int, int q) { return kv <= q && (q - kv < a.mask.window || kv < a.mask.n_sink); });
          else
            mask_rows([&](int r, int q) { return mask_visible(a.mask, b, s_head[row0 + r], q, kv, S_b, a.S); });
        }
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          if (want_max) {
            tm[2 * i] = fmaxf(tm[2 * i], t[i].x - lv);
            tm[2 * i + 1] = fmaxf(tm[2 * i + 1], t[i].y - lv);
          }
          const float2 d = add2(t[i], nms[i]);
          top = max3f(top, d.x, d.y);
        }
      }
      // one vote per tile: as usual, or a wait gave up, or a maximum moves
      if (named_bar_or(bar, 128, !ok || top > kSlack + kShift)) {
        if (named_bar_or(bar, 128, !ok)) {
          alive = false;
          break;
        }
        float tv[N];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          tv[2 * i] = t[i].x;
          tv[2 * i + 1] = t[i].y;
        }
        const float v = reduce_rows<true, N>(tv, lane);
        if (lane % (32 / N) == 0) s_red[0][qd][row0 + lane / (32 / N)] = v;
        named_bar_sync(bar, 128);
        float alpha[N];
#pragma unroll
        for (int r = 0; r < N; ++r) {
          const float tmax = fmaxf(fmaxf(s_red[0][0][row0 + r], s_red[0][1][row0 + r]),
                                   fmaxf(s_red[0][2][row0 + r], s_red[0][3][row0 + r]));
          float& mine = (r & 1) ? nms[r >> 1].y : nms[r >> 1].x;
          const float now = fminf(mine, kShift - tmax);
          alpha[r] = ex2_approx(now - mine);
          mine = now;
        }
#pragma unroll
        for (int i = 0; i < N / 2; ++i) l_part[i] = mul2(l_part[i], make_float2(alpha[2 * i], alpha[2 * i + 1]));
        named_bar_sync(bar, 128);  // s_red is read by all before its next use
        if (j > 0) {
          // O^T holds tiles 0 .. j-1: once the last of them is in, rescale
          const int jp = j - 1;
          alive = __all_sync(0xffffffffu, mbar_wait(&bars.p_free[jp & 1], (jp >> 1) & 1, abort, a.status,
                                                    a.wait_cycles));
          if (alive) {
            tc_fence_after();
            const uint32_t ot = tbase + lane_base + C::kO + row0;
#pragma unroll
            for (int i = 0; i < C::kOLoads; ++i) {  // one load at a time: all of them would cost spills
              uint32_t o[8];
              tmem_out(ot + C::o_col(i), o);
#pragma unroll
              for (int c = 0; c < 8; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha[c % N]);
              tmem_st8(ot + C::o_col(i), o);
            }
            tmem_wait_st();
          }
        }
      }
      // Values past the sequence's end may hold anything (0 * NaN is NaN):
      // their rows are cleared before the product reads them.
      if (alive && kv0 + kKeys > S_b) {
        const int u = 2 * j + 1;
        alive = __all_sync(0xffffffffu, mbar_wait(&bars.full[u % kRing], (u / kRing) & 1, abort, a.status, a.wait_cycles));
        if (alive && set == 0 && kv >= S_b) {
          uint4* vrow = reinterpret_cast<uint4*>(sKV + (u % kRing) * kTileBytes + kk * 128);
#pragma unroll
          for (int i = 0; i < 8; ++i) vrow[i] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      if (alive) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          const float2 d = add2(t[i], nms[i]);
          const float2 w = make_float2(ex2_approx(d.x), ex2_approx(d.y));
          l_part[i] = fma2(w, splat2(ivs), l_part[i]);
          uint32_t term[3];
          split_e5m2(w.x, w.y, half, term);
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            put_byte(wx[2 * i + C::w_row(k)] + sb * C::kWBytes + C::w_bytes(k), term[k] >> 8);
            put_byte(wx[2 * i + 1 + C::w_row(k)] + sb * C::kWBytes + C::w_bytes(k), term[k] >> 24);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_full[sb]);
      }
      kv0 = kv0_1;
      kv0_1 = kv0_2;
      n_2 = n_3;
      ks = ks_1;
      vs = vs_1;
      pg_1 = pg_2;
    }
    // every softmax thread arrives here together (the loop is left only
    // through the vote, or at its end)
    bool fin = alive;
    if (fin && nsub > 0) fin = mbar_wait(&bars.o_final, 0, abort, a.status, a.wait_cycles);
    fin = named_bar_and(bar, 128, fin && !*abort);
    if (fin) {
      tc_fence_after();
      uint32_t o[8 * C::kOLoads];  // the terms a, b, c of the set's rows
#pragma unroll
      for (int c = 0; c < 8 * C::kOLoads; ++c) o[c] = 0u;
      if (nsub > 0) {
#pragma unroll
        for (int i = 0; i < C::kOLoads; ++i)
          tmem_out(tbase + lane_base + C::kO + row0 + C::o_col(i), *reinterpret_cast<uint32_t(*)[8]>(o + 8 * i));
      }
      float lp[N];
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        lp[2 * i] = l_part[i].x;
        lp[2 * i + 1] = l_part[i].y;
      }
      const float ls = reduce_rows<false, N>(lp, lane);
      const float lm = reduce_rows<true, N>(tm, lane);
      if (lane % (32 / N) == 0) {
        s_red[0][qd][row0 + lane / (32 / N)] = ls;
        s_red[1][qd][row0 + lane / (32 / N)] = lm;
      }
      named_bar_sync(bar, 128);
      // one thread a row for what the row's 128 columns share
      if (kk < N && s_off[row0 + kk] >= 0) {
        const int rr = row0 + kk;
        const float l = (s_red[0][0][rr] + s_red[0][1][rr]) + (s_red[0][2][rr] + s_red[0][3][rr]);
        const float top = fmaxf(fmaxf(s_red[1][0][rr], s_red[1][1][rr]), fmaxf(s_red[1][2][rr], s_red[1][3][rr]));
        float nm = 0.0f;
#pragma unroll
        for (int r = 0; r < N; ++r)
          if (kk == r) nm = (r & 1) ? nms[r >> 1].y : nms[r >> 1].x;
        // a row without a visible key (in this split) has l = 0: out 0 and lse
        // -inf, unless the caller promised there is none and there is one
        // split; NaN stays NaN
        const bool live = (a.rows_safe && p.splits == 1) || !(l == 0.0f);
        s_inv[rr] = live ? 1.0f / l : 0.0f;
        const float lse = live ? (log2f(l) - nm) * kLn2 : -INFINITY;
        const int64_t id = s_id[rr];
        if (p.splits == 1) {
          if (a.lse) a.lse[id] = lse;
          if (a.max_scores) a.max_scores[id] = top * kLn2;
        } else {
          ws_lse[id] = lse;
          ws_max[id] = top;
        }
      }
      named_bar_sync(bar, 128);
      const int ev = kk;
      const bool half_out = p.splits == 1 && !a.out_f32;
      float* dst = p.splits == 1 ? static_cast<float*>(a.out) : ws_o;
#pragma unroll
      for (int r = 0; r < N; ++r) {
        const int64_t off = s_off[row0 + r];
        const float low = fmaf(__uint_as_float(o[2 * N + r]), 0.125f, __uint_as_float(o[N + r]));
        const float val = fmaf(low, 0.125f, __uint_as_float(o[r])) * s_inv[row0 + r];
        if (off >= 0 && ev < a.Ev) {
          if (half_out)
            static_cast<__nv_bfloat16*>(a.out)[off + ev] = __float2bfloat16_rn(val);
          else
            dst[off + ev] = val;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tbase, C::kTmemCols);
}

// One CTA per query row: merge the splits' (o_s, lse_s, max_s), with
// lse = ln sum e^(lse_s), o = sum e^(lse_s - lse) o_s.  A warp takes every 8th
// split, a lane four columns.
constexpr int kCombineWarps = 8;
__global__ void __launch_bounds__(32 * kCombineWarps)
    combine_fp8_kernel(const __grid_constant__ FwdArgs a, int splits, const float* ws_o, const float* ws_lse,
                       const float* ws_max) {
  __shared__ float s_w[kFp8MaxSplits];
  __shared__ float s_m[kCombineWarps], s_t[kCombineWarps], s_sum[kCombineWarps];
  __shared__ __align__(16) float s_o[kCombineWarps][128];
  const int64_t row_id = blockIdx.x;
  const int i = static_cast<int>(row_id % a.L), h = static_cast<int>((row_id / a.L) % a.Hq);
  const int b = static_cast<int>(row_id / (static_cast<int64_t>(a.L) * a.Hq));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // launched while the decode kernel still runs: wait for its results
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the first splits' outputs come with their weights still unknown
  constexpr int kAhead = 4;
  const float* src = ws_o + row_id * splits * a.Ev + 4 * lane;
  float4 o[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    const int s = warp + u * kCombineWarps;
    if (s < splits && 4 * lane < a.Ev) o[u] = *reinterpret_cast<const float4*>(src + static_cast<int64_t>(s) * a.Ev);
  }
  float m = -INFINITY, top = -INFINITY;
  bool nan = false;
  for (int s = threadIdx.x; s < splits; s += 32 * kCombineWarps) {
    const float v = ws_lse[row_id * splits + s];
    s_w[s] = v;
    nan = nan || v != v;
    m = fmaxf(m, v);
    top = fmaxf(top, ws_max[row_id * splits + s]);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_t[warp] = top;
  }
  nan = __syncthreads_or(nan);
#pragma unroll
  for (int w = 0; w < kCombineWarps; ++w) {
    m = fmaxf(m, s_m[w]);
    top = fmaxf(top, s_t[w]);
  }
  const bool live = a.rows_safe || nan || m != -INFINITY;
  float sum = 0.0f;
  for (int s = threadIdx.x; s < splits; s += 32 * kCombineWarps) {
    const float w = live ? expf(s_w[s] - m) : 0.0f;
    s_w[s] = w;
    sum += w;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  sum = 0.0f;
#pragma unroll
  for (int w = 0; w < kCombineWarps; ++w) sum += s_sum[w];
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add = [&](const float4& v, float w) {
    acc.x = fmaf(w, v.x, acc.x);
    acc.y = fmaf(w, v.y, acc.y);
    acc.z = fmaf(w, v.z, acc.z);
    acc.w = fmaf(w, v.w, acc.w);
  };
  if (4 * lane < a.Ev) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int s = warp + u * kCombineWarps;
      if (s < splits) add(o[u], s_w[s]);
    }
#pragma unroll 4
    for (int s = warp + kAhead * kCombineWarps; s < splits; s += kCombineWarps)
      add(*reinterpret_cast<const float4*>(src + static_cast<int64_t>(s) * a.Ev), s_w[s]);
    *reinterpret_cast<float4*>(&s_o[warp][4 * lane]) = acc;
  }
  __syncthreads();
  const int ev = threadIdx.x;
  if (ev < a.Ev) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kCombineWarps; ++w) v += s_o[w][ev];
    const float val = live ? v / sum : 0.0f;
    const int64_t off = b * a.o_stride[0] + h * a.o_stride[1] + i * a.o_stride[2] + ev;
    if (a.out_f32)
      static_cast<float*>(a.out)[off] = val;
    else
      static_cast<__nv_bfloat16*>(a.out)[off] = __float2bfloat16_rn(val);
  }
  if (threadIdx.x == 0 && a.lse) a.lse[row_id] = live ? m + logf(sum) : -INFINITY;
  if (threadIdx.x == 0 && a.max_scores) a.max_scores[row_id] = top * kLn2;
}

// Codes times scales as bf16 or fp32, 16 codes a thread, for the slots below
// the sequence's end; the slots up to a tile past it become 0 (kernels load
// whole tiles), and so do the values up to the last tile that the lists name
// (lists may be older than the lengths; hidden keys are dropped by selection,
// but their values are multiplied by 0).  The rest is not written.
template <bool kVec>
__global__ void __launch_bounds__(256) restore_kernel(const __grid_constant__ FwdArgs a, const QuantArgs qa,
                                                      const __grid_constant__ RestoreArgs k,
                                                      const __grid_constant__ RestoreArgs v) {
  const bool is_v = blockIdx.y >= static_cast<unsigned>(a.Hkv);
  const RestoreArgs& r = is_v ? v : k;
  const int hk = is_v ? blockIdx.y - a.Hkv : blockIdx.y, b = blockIdx.z;
  const int S_b = seq_len_b(a.mask, b, a.S);
  const int end = min(S_b + 128, a.S);
  const int pieces = (r.D + 15) / 16;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < static_cast<int64_t>(end) * pieces;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int kv = static_cast<int>(i / pieces), e0 = static_cast<int>(i % pieces) * 16;
    float scale = 0.0f;
    const uint8_t* src = nullptr;
    if (kv < S_b) {
      int outer = b, at = kv;
      if (a.page_table) {
        outer = cache_page(a.page_table, a.pages_per_seq, a.page_size, a.num_pages, a.status, b, kv);
        at = kv % a.page_size;
      }
      scale = __ldg(r.scale + (static_cast<int64_t>(outer) * a.Hkv + hk) * qa.scales_per_outer + (at >> qa.block_log));
      src = r.codes + outer * r.stride[0] + hk * r.stride[1] + at * r.stride[2] + e0;
    }
    float x[16];
    if (kVec && src) {
      const uint4 c = *reinterpret_cast<const uint4*>(src);
      const uint32_t u[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
            static_cast<__nv_fp8x2_storage_t>(u[w >> 1] >> (16 * (w & 1))), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        x[2 * w] = f.x * scale;
        x[2 * w + 1] = f.y * scale;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        x[e] = 0.0f;
        if (src && e0 + e < r.D)
          x[e] = __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(src[e]), __NV_E4M3))) * scale;
      }
    }
    const int64_t off = ((static_cast<int64_t>(b) * a.Hkv + hk) * a.S + kv) * r.D + e0;
    if (kVec) {
      if (r.f32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(r.out) + off);
#pragma unroll
        for (int w = 0; w < 4; ++w) o[w] = make_float4(x[4 * w], x[4 * w + 1], x[4 * w + 2], x[4 * w + 3]);
      } else {
        uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(r.out) + off);
#pragma unroll
        for (int w = 0; w < 2; ++w)
          o[w] = make_uint4(pack_bf16x2(x[8 * w], x[8 * w + 1]), pack_bf16x2(x[8 * w + 2], x[8 * w + 3]),
                            pack_bf16x2(x[8 * w + 4], x[8 * w + 5]), pack_bf16x2(x[8 * w + 6], x[8 * w + 7]));
      }
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (e0 + e < r.D) {
          if (r.f32)
            static_cast<float*>(r.out)[off + e] = x[e];
          else
            static_cast<__nv_bfloat16*>(r.out)[off + e] = __float2bfloat16_rn(x[e]);
        }
    }
  }
  // One CTA a head and sequence looks where the lists end.
  if (!is_v || blockIdx.x != 0 || end == a.S) return;
  __shared__ int s_named;
  if (threadIdx.x == 0) s_named = 0;
  __syncthreads();
  const int64_t rows = static_cast<int64_t>(a.bm.H) * a.bm.Mb, row0 = a.bm.B > 1 ? b * rows : 0;
  for (int64_t row = row0 + threadIdx.x; row < row0 + rows; row += 256) {
    const int full = __ldg(a.bm.full_kv_num_blocks + row), part = __ldg(a.bm.kv_num_blocks + row);
    if (full > 0) atomicMax(&s_named, __ldg(a.bm.full_kv_indices + row * a.bm.Nb + full - 1) + 1);
    if (part > 0) atomicMax(&s_named, __ldg(a.bm.kv_indices + row * a.bm.Nb + part - 1) + 1);
  }
  __syncthreads();
  const int64_t last = min(static_cast<int64_t>(s_named) * a.bm.BN, static_cast<int64_t>(a.S));
  const int64_t at = (static_cast<int64_t>(b) * a.Hkv + hk) * a.S;
  for (int64_t i = (at + end) * r.D + threadIdx.x; i < (at + last) * r.D; i += 256) {
    if (r.f32)
      static_cast<float*>(r.out)[i] = 0.0f;
    else
      static_cast<uint16_t*>(r.out)[i] = 0;
  }
}

}  // namespace

FastDiv fast_div(int d) {
  FastDiv f{0u, 0};
  if (d == 1) return f;
  while ((int64_t{1} << f.shift) < d) ++f.shift;
  f.mul = static_cast<uint32_t>(((uint64_t{1} << (31 + f.shift)) + d - 1) / d);
  return f;
}

void plan_decode_fp8(const FwdArgs& a, int split_kv, int num_sms, Fp8Plan* p) {
  const int span = a.bm.H > 1 ? a.L : a.G * a.L;  // rows that share a list of tiles
  p->rows = span <= 4 ? 4 : (span <= 8 ? 8 : kMaxRows);
  p->row_chunks = (a.bm.H > 1 ? a.G : 1) * ((span + p->rows - 1) / p->rows);
  p->page = fast_div(a.page_table ? a.page_size : 1);
  const int64_t units = static_cast<int64_t>(a.B) * a.Hkv * p->row_chunks;
  const int slots = (p->rows <= 8 ? Cfg<8>::kCtas : Cfg<16>::kCtas) * num_sms;
  int64_t splits = split_kv;
  // One round of CTAs where the sequences are few; several, longest first,
  // where many of unequal length are to be balanced.
  if (split_kv == 0) splits = units * 4 <= slots ? slots / units : (2 * slots + units - 1) / units;
  splits = splits < 1 ? 1 : (splits > a.bm.Nb ? a.bm.Nb : splits);
  splits = splits > kFp8MaxSplits ? kFp8MaxSplits : splits;
  const int per = static_cast<int>((a.bm.Nb + splits - 1) / splits);
  p->splits = (a.bm.Nb + per - 1) / per;
  p->workspace_bytes =
      p->splits > 1 ? static_cast<size_t>(a.B) * a.Hq * a.L * p->splits * (a.Ev + 2) * sizeof(float) : 0;
}

namespace {
template <int R>
cudaError_t launch_rows(const FwdArgs& a, const QuantArgs& qa, const Fp8Plan& p, const CUtensorMap& map_k,
                        const CUtensorMap& map_v, int box, float* ws_o, float* ws_lse, float* ws_max,
                        cudaStream_t stream) {
  auto kern = a.score.kind == FA_SCORE_NONE      ? decode_fp8_kernel<FA_SCORE_NONE, R>
              : a.score.kind == FA_SCORE_SOFTCAP ? decode_fp8_kernel<FA_SCORE_SOFTCAP, R>
              : a.score.kind == FA_SCORE_ALIBI   ? decode_fp8_kernel<FA_SCORE_ALIBI, R>
                                                 : decode_fp8_kernel<FA_SCORE_CAP_THEN_BIAS, R>;
  static SmemLimit limit[4];
  const cudaError_t e = limit[a.score.kind].raise(kern, Cfg<R>::kSmemBytes);
  if (e != cudaSuccess) return e;
  kern<<<dim3(a.Hkv * p.row_chunks, p.splits, a.B), Cfg<R>::kThreads, Cfg<R>::kSmemBytes, stream>>>(
      a, qa, p, map_k, map_v, box, ws_o, ws_lse, ws_max);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_decode_fp8(const FwdArgs& a, const QuantArgs& qa, const Fp8Plan& p, const CUtensorMap& map_k,
                              const CUtensorMap& map_v, int box, void* workspace, cudaStream_t stream) {
  float* ws_o = static_cast<float*>(workspace);
  const int64_t rows = static_cast<int64_t>(a.B) * a.Hq * a.L;
  float* ws_lse = ws_o ? ws_o + rows * p.splits * a.Ev : nullptr;
  float* ws_max = ws_o ? ws_lse + rows * p.splits : nullptr;
  cudaError_t e = p.rows == 4   ? launch_rows<4>(a, qa, p, map_k, map_v, box, ws_o, ws_lse, ws_max, stream)
                  : p.rows == 8 ? launch_rows<8>(a, qa, p, map_k, map_v, box, ws_o, ws_lse, ws_max, stream)
                                : launch_rows<16>(a, qa, p, map_k, map_v, box, ws_o, ws_lse, ws_max, stream);
  if (e != cudaSuccess || p.splits == 1) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(rows));
  cfg.blockDim = dim3(32 * kCombineWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, combine_fp8_kernel, a, p.splits, static_cast<const float*>(ws_o),
                            static_cast<const float*>(ws_lse), static_cast<const float*>(ws_max));
}

cudaError_t launch_restore(const FwdArgs& a, const QuantArgs& qa, const RestoreArgs& k, const RestoreArgs& v,
                           cudaStream_t stream) {
  const int64_t pieces = static_cast<int64_t>(a.S) * ((k.D > v.D ? k.D : v.D) + 15) / 16;
  const int64_t blocks = (pieces + 4 * 256 - 1) / (4 * 256);
  const dim3 grid(static_cast<unsigned>(blocks < 4096 ? blocks : 4096), 2 * a.Hkv, a.B);
  if (k.vec && v.vec)
    restore_kernel<true><<<grid, 256, 0, stream>>>(a, qa, k, v);
  else
    restore_kernel<false><<<grid, 256, 0, stream>>>(a, qa, k, v);
  return cudaGetLastError();
}

}  // namespace fa
