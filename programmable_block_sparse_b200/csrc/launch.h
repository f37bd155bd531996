// Host-side launch interfaces between the C ABI layer (api.cu) and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mods.cuh"

namespace fa {

struct ClassifyArgs {
  int* status;  // device status word
  MaskParams mask;
  int B, H, L, S, BM, BN, Mb, Nb;
  int* kv_num_blocks;
  int* kv_indices;
  int* full_kv_num_blocks;
  int* full_kv_indices;
};
cudaError_t launch_classify(const ClassifyArgs& a, cudaStream_t stream);

// Read-only view of a BlockMask; B and H may be 1 (broadcast).
struct BlockMaskView {
  int B, H, Mb, Nb, BM, BN;
  const int* kv_num_blocks;
  const int* kv_indices;
  const int* full_kv_num_blocks;
  const int* full_kv_indices;
};

struct FwdArgs {
  int* status;  // device status word
  const void* q;
  const void* k;
  const void* v;
  void* out;
  float* lse;                 // [B, Hq, L] or null
  float* max_scores;          // [B, Hq, L] or null
  long long wait_cycles;      // budget of each main-path device wait
  int out_f32;                // out is fp32 (else the input dtype)
  int rows_safe;              // every row has a visible key: no empty-row guard
  // paged KV cache (page_table == null: k, v are (B, Hkv, S, D)): logical key
  // j of sequence b is slot j % page_size of page page_table[b * pages_per_seq
  // + j / page_size] of the pools k, v (num_pages, Hkv, page_size, D)
  const int* page_table;
  int page_size, pages_per_seq, num_pages;
  int64_t q_stride[4], k_stride[4], v_stride[4], o_stride[4];
  int B, Hq, Hkv, L, S, E, Ev, G;
  int dtype;                  // FA_DTYPE_*
  float scale;
  MaskParams mask;
  ScoreParams score;
  BlockMaskView bm;
};

// General kernel: any dtype, tiles up to 128 x 128, head dims up to 128.
cudaError_t launch_fwd_simt(const FwdArgs& a, cudaStream_t stream);

// Tensor-core prefill kernel (bf16, BM = BN = 128, E = Ev in {64, 128}).
struct Sm100Maps {
  CUtensorMap q, k, v;
};
// One CTA per pair of query tiles, persistent through cluster launch control.
cudaError_t launch_fwd_sm100(const FwdArgs& a, const Sm100Maps& maps, cudaStream_t stream);

// Split-KV decode for short queries (bf16, E = Ev in {64, 128}, L <= 16) and
// the log-sum-exp combination of its partial results.
struct DecodePlan {
  int rows_per_cta;     // query rows one CTA handles (heads of a group x L), <= 16
  int heads_per_cta;    // query heads per CTA
  int splits;           // KV splits per (b, head group)
  int tiles_per_split;  // listed tiles per split
  size_t workspace_bytes;
};
constexpr int kDecodeMaxRows = 16;
int plan_decode(const FwdArgs& a, int split_kv, int num_sms, DecodePlan* plan);
cudaError_t launch_decode(const FwdArgs& a, const DecodePlan& plan, const Sm100Maps& maps, void* workspace,
                          cudaStream_t stream);

// Backward pass (bf16, E = Ev in {64, 128}, 128 x 128 tiles).
struct BwdArgs {
  int* status;  // device status word
  long long wait_cycles;
  const void *q, *k, *v, *out, *dout;
  const float* lse;  // [B, Hq, L] from the forward pass
  float* dsum;       // workspace: D = rowsum(dout * out), [B, Hq, L]
  void *dq, *dk, *dv;
  int64_t q_stride[4], k_stride[4], v_stride[4], o_stride[4], do_stride[4];
  int64_t dq_stride[4], dk_stride[4], dv_stride[4];
  int dq_f32, dk_f32, dv_f32;  // gradient storage: fp32, else bf16
  int B, Hq, Hkv, L, S, E, G;
  float scale;
  MaskParams mask;
  ScoreParams score;
  BlockMaskView bm;  // key-side lists (the forward's)
  // query-side lists: for key tile n of row (b, h), the query tiles listing it
  int qB, qH;
  const int *q_num_blocks, *q_indices, *full_q_num_blocks, *full_q_indices;
};
struct BwdMaps {
  CUtensorMap q, k, v, dout;
};
cudaError_t launch_bwd(const BwdArgs& a, const BwdMaps& maps, cudaStream_t stream);

// Query-side lists from the key-side lists of a BlockMask.
struct TransposeArgs {
  int B, H, Mb, Nb;
  const int *kv_num_blocks, *kv_indices, *full_kv_num_blocks, *full_kv_indices;
  int *q_num_blocks, *q_indices, *full_q_num_blocks, *full_q_indices;
};
cudaError_t launch_transpose(const TransposeArgs& a, cudaStream_t stream);

// Query / key preparation and cache writes (rows of one head: D <= 128).
struct NormArgs {
  int on;             // 0: no norm
  const void* weight; // [D] or null (1)
  int weight_f32;
  float eps;
};
struct RopeArgs {
  int rot;            // 0: no rotation
  int interleaved;
  const float* inv_freq;
  const int* pos;     // [pos_batch, N] or null
  int pos_batch;
};
struct RowsIn {       // (B, H, N, D) rows; p == null: absent
  const void* p;
  int f32, H;
  int64_t stride[3];
};
struct RowsOut {
  void* p;
  int f32;
  int64_t stride[3];
};
struct PrepArgs {
  RowsIn x[2];        // q, k
  RowsOut y[2];
  NormArgs norm[2];
  RopeArgs rope;
  int B, N, D;
  int vec;            // every row takes 16-byte accesses
  int tokens, heads;  // per CTA (set by the launcher)
};
cudaError_t launch_prep(PrepArgs a, int num_sms, cudaStream_t stream);

struct PrepBwdArgs {
  RowsIn x[2], dy[2];
  RowsOut dx[2];
  float* dw[2];       // fp32 [D] or null
  NormArgs norm[2];
  RopeArgs rope;
  int B, N, D;
  int vec;
  int tokens;         // per work item (set by the launcher)
  float* partial;     // [CTAs][2][D]
};
// CTAs of the backward pass at most: its partial weight gradients are summed
// over them, so the bound fixes the workspace (2 MB) and the order of the sum
// on every device.  Four rounds of three CTAs an SM, so that the last round's
// idle share is small.
constexpr int kPrepBwdMaxCtas = 2048;
cudaError_t launch_prep_bwd(PrepBwdArgs a, cudaStream_t stream);

struct AppendArgs {
  int* status;
  RowsIn k, v, q;     // q.p == null: no queries
  RowsOut q_out;
  NormArgs k_norm, q_norm;
  RopeArgs rope;
  int B, N, E, Ev;
  int k_vec, v_vec, q_vec;  // 16-byte accesses of the inputs (and q_out)
  // the cache: outer index (page, or sequence of a dense cache), head, slot
  void *kc, *vc;
  int64_t kc_stride[3], vc_stride[3];
  int kc_vec, vc_vec;       // rows of the cache take 8-element accesses
  int dtype;                // FA_DTYPE_* of the cache
  float *k_scale, *v_scale;
  int scale_block, scales_per_outer;  // e4m3
  const int* page_table;
  const int *cache_len, *new_len;
  int page_size, pages_per_seq, num_outer;
  int chunk, k_heads, q_heads;  // tokens and heads per CTA (set by the launcher)
};
cudaError_t launch_append(AppendArgs a, int num_sms, cudaStream_t stream);

// Attention over an e4m3 cache (codes under a scale per block of slots and
// head; FwdArgs k, v are the codes).
struct QuantArgs {
  const float *k_scale, *v_scale;  // [outer, Hkv, scales_per_outer]
  int block_log;                   // log2 of the slots per scale
  int scales_per_outer;
};
// Quotients by a fixed divisor of values below 2^31: with s = ceil(log2 d) and
// mul = ceil(2^(31 + s) / d) < 2^32, x / d = (x mul) >> (31 + s) (the error of
// mul is below 2^s / 2^(31 + s) of it, less than 1 / (d x)).
struct FastDiv {
  uint32_t mul;  // 0: d = 1
  int shift;
#ifdef __CUDACC__
  __device__ __forceinline__ int quotient(int x) const {
    return mul == 0 ? x : static_cast<int>(__umulhi(static_cast<uint32_t>(x) << 1, mul) >> shift);
  }
#endif
};
FastDiv fast_div(int d);
struct Fp8Plan {
  int rows;         // query rows of a CTA: 4, 8 or 16
  int row_chunks;   // CTAs that share one KV head's cache
  FastDiv page;     // slots to pages
  int splits;       // KV splits per (sequence, KV head, row chunk)
  size_t workspace_bytes;
};
constexpr int kFp8MaxSplits = 1024;
void plan_decode_fp8(const FwdArgs& a, int split_kv, int num_sms, Fp8Plan* plan);
// k and v maps: bytes, boxes of 128 x `box` slots.
cudaError_t launch_decode_fp8(const FwdArgs& a, const QuantArgs& qa, const Fp8Plan& plan, const CUtensorMap& map_k,
                              const CUtensorMap& map_v, int box, void* workspace, cudaStream_t stream);

// The visible part of an e4m3 cache (dense or paged, FwdArgs) as a dense
// (B, Hkv, S, D) tensor of bf16 or fp32.
struct RestoreArgs {
  const uint8_t* codes;
  int64_t stride[3];
  const float* scale;
  void* out;
  int D, f32, vec;
};
cudaError_t launch_restore(const FwdArgs& a, const QuantArgs& qa, const RestoreArgs& k, const RestoreArgs& v,
                           cudaStream_t stream);

}  // namespace fa
