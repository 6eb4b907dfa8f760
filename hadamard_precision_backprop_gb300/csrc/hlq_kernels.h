// hlq_kernels.h -- host-side launchers of the libhlq kernels (internal).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "hlq.h"

namespace hlq {

// HQ of a [rows, cols] tensor along cols (g_y).  amax_only: per-tensor
// pre-pass into *amax_slot.  Otherwise writes E4M3 codes [rows, cols] and
// scales ([rows] if per_token else [1], from *amax_slot).  The rows may be
// rows row0 .. of a larger tensor (pointers already offset): the random
// words are drawn for their element indices in that tensor.
cudaError_t launch_hq_rows(const void* src, bool bf16, int64_t rows,
                           int64_t cols, bool per_token, bool amax_only,
                           unsigned int* amax_slot, uint8_t* codes,
                           float* scales, int rnd, uint64_t seed,
                           uint32_t stream_id, unsigned int* status,
                           cudaStream_t st, int64_t row0 = 0);

// HQ of a [rows, cols] tensor along rows (w), codes written transposed
// [cols, rows] (E4M3), per-tensor scale from *amax_slot.
// Layer-wise quantizer selection: RNE int4 HQ errors of g_y per tensor
// (scale from *amax_slot) and per token added into sums[0..1] (zeroed by the
// caller), then mse[g] = sums[g] / (rows * cols) and *choice.
cudaError_t launch_hq_mse(const void* src, bool bf16, int64_t rows, int64_t cols,
                          const unsigned int* amax_slot, double* sums, double threshold,
                          double* mse, int32_t* choice, unsigned int* status,
                          cudaStream_t st);

cudaError_t launch_hq_cols(const void* src, bool bf16, int64_t rows,
                           int64_t cols, bool amax_only,
                           unsigned int* amax_slot, uint8_t* codes_t,
                           float* scale, int rnd, uint64_t seed,
                           uint32_t stream_id, unsigned int* status,
                           cudaStream_t st);

// Output formats of launch_hla: int8 codes, their fp16 values, or int4
// codes packed two per byte (even ranks only).
constexpr int kHlaOutI8 = 0, kHlaOutF16 = 1, kHlaOutI4 = 2;

// HLA of src [T, C] along tokens -> codes [C, T*rank/16] in `out_fmt`,
// per-tensor scale RN(amax/qmax) from *amax_slot (qmax 7 for int4, else 127).
// out_ld: row stride of `out` in codes (>= T*rank/16).
// per_col: one amax slot and one scale per column c of src (amax_slot[c],
// scale[c]; the code row of channel c) instead of one for the tensor.
cudaError_t launch_hla(const void* src, bool bf16, int64_t T, int64_t C,
                       int rank, bool amax_only, int out_fmt,
                       unsigned int* amax_slot, void* out, int64_t out_ld,
                       float* scale, unsigned int* status, cudaStream_t st,
                       bool per_col = false);

// HLA along the rows of src [rows, cols]: per 16-block of a row the rank
// lowest-sequency coefficients, per-tensor amax pass (amax_only) or int8 RNE
// codes with s = RN(amax/127) stored as fp16 [rows, out_ld] (column
// rank*b + k), scale[0] = s.
cudaError_t launch_hla_rows(const void* src, bool bf16, int64_t rows, int64_t cols,
                            int rank, bool amax_only, unsigned int* amax_slot, void* out,
                            int64_t out_ld, float* scale, unsigned int* status,
                            cudaStream_t st);

// Fused reader of g_y [T, C] for both paths, one pass per call: amax_only
// gives the HQ maxima (per row into hq_amax[T] when per_token, else one slot)
// and the HLA maximum (hla_amax); otherwise the HQ E4M3 codes qy [T, C] with
// scales sgy ([T] or [1]) and the HLA int8 codes as fp16 qg [C, hla_ld] with
// scale sg[0], exactly as launch_hq_rows and launch_hla produce them.
cudaError_t launch_gy_fused(const void* gy, bool bf16, int64_t T, int64_t C, int rank,
                            bool per_token, bool amax_only, unsigned int* hq_amax,
                            unsigned int* hla_amax, uint8_t* qy, float* sgy, void* qg,
                            int64_t hla_ld, float* sg, int rnd, uint64_t seed,
                            unsigned int* status, cudaStream_t st);

// One CTA waiting on an mbarrier that never completes, for limit_ns: sets
// *result = 0 and raises HLQ_DEV_TIMEOUT in the status word.
// Device address of the library's status word (HLQ_DEV_* flags) on the
// current device; the word lives with the kernels that raise its flags.
cudaError_t status_word_address(unsigned int** out);

cudaError_t launch_wait_timeout_probe(unsigned long long limit_ns, int32_t* result,
                                      unsigned int* status, cudaStream_t st);

// Transform only (fp32 coefficients), for bit-exact checks.
cudaError_t launch_hq_rows_transform(const void* src, bool bf16, int64_t rows,
                                     int64_t cols, float* Y,
                                     unsigned int* status, cudaStream_t st);
cudaError_t launch_hq_cols_transform(const void* src, bool bf16, int64_t rows,
                                     int64_t cols, float* Y,
                                     unsigned int* status, cudaStream_t st);
cudaError_t launch_hla_transform(const void* src, bool bf16, int64_t T,
                                 int64_t C, int rank, float* out,
                                 unsigned int* status, cudaStream_t st);

// in [rows, cols] int8 (row stride cols), or packed int4 -> out [rows, out_ld]
// fp16.
cudaError_t launch_widen_i4_f16(const uint8_t* in, void* out, int64_t rows, int64_t cols,
                                int64_t out_ld, cudaStream_t st);
cudaError_t launch_widen_i8_f16(const int8_t* in, void* out, int64_t rows,
                                int64_t cols, int64_t out_ld, cudaStream_t st);
cudaError_t launch_pack_e4m3_int4(const uint8_t* in, uint8_t* out, int64_t n,
                                  cudaStream_t st);
cudaError_t launch_decode_e4m3(const uint8_t* in, int8_t* out, int64_t n,
                               cudaStream_t st);
cudaError_t launch_decode_f16(const void* in, int8_t* out, int64_t rows,
                              int64_t cols, int64_t ld, cudaStream_t st);

// Operand code formats of the GEMMs.
enum CodeFmt { kFmtE4M3 = 0, kFmtI8 = 1, kFmtF16 = 2 };

// Exact integer GEMM on CUDA cores (dp4a): acc[m, n] = sum_k A[m,k] B[n,k],
// A [M, K], B [N, K] (contraction dim contiguous).  Epilogue:
// out[m, n] = float(acc) * (sa[per_row_a ? m : 0] * sb[0]) * 0.0625f.
// acc_out (nullable) receives the int32 sums.
cudaError_t launch_gemm_simple(const void* A, int fmtA, const void* B,
                               int fmtB, int64_t M, int64_t N, int64_t K,
                               const float* sa, bool per_row_a,
                               const float* sb, float* out, int32_t* acc_out,
                               cudaStream_t st);

// A TMA tensor map over a row-major [rows, cols] bf16 / fp32 matrix with
// boxes of box_rows x box_cols, no swizzle, zero fill outside the matrix.
bool make_tile_map_2d(CUtensorMap* map, const void* ptr, bool bf16, int64_t rows,
                      int64_t cols, int box_cols, int box_rows);

// Tensor-core GEMM (hlq_gemm_tc.cu).  kind 0: E4M3 operands (int4 codes),
// kind 1: fp16 operands (int8 codes).  A [M, K] (row stride lda elements),
// B [N, K] (ldb); out [M, N] fp32 = acc * sa[m or 0] * sb[0] / 16.
// raw (kind 1 only): kRawB / kRawA mark an operand given as int8 codes in
// HBM (row stride in bytes, a multiple of 16, base 16-byte aligned), widened
// to fp16 in shared memory inside the GEMM.
struct GemmPlan {
  int bn = 128;      // tile width (96, 128 or 256)
  int splits = 1;    // K split count (int32 workspace reduction)
  int num_kb = 0;    // k-blocks of 128 bytes
  int chunk_kb = 0;  // k-blocks per exact fp32 accumulation chunk
  int pair = 0;      // 1: a CTA pair per 256-row tile (tcgen05 cta_group::2)
  int stream_k = 0;  // 1: equal k-block runs per SM over all tiles (kind 1,
                     // unsplit, no pairs; partial tiles summed like K splits)
};
GemmPlan plan_gemm_tc(int kind, int64_t M, int64_t N, int64_t K, int num_sms,
                      int max_splits);
size_t gemm_tc_split_ws_bytes(int64_t M, int64_t N);
cudaError_t launch_gemm_tc(int kind, const void* A, int64_t lda, const void* B,
                           int64_t ldb, int64_t M, int64_t N, int64_t K,
                           const GemmPlan& plan, const float* sa, bool per_row_a,
                           const float* sb, float* out, int32_t* acc_out,
                           void* split_ws, unsigned int* status, cudaStream_t st,
                           bool per_col_b = false,  // sb[n] per column (kind 1)
                           int raw = 0);
constexpr int kRawB = 1, kRawA = 2;

// The g_x path with a given workspace (the body of hlq_linear_backward_gx)
// and the workspace it needs.
size_t gx_workspace_bytes(int64_t T, int64_t Cin, int64_t Cout);
hlq_status backward_gx_with_ws(const void* gy, const void* w, int dt, int64_t T,
                               int64_t Cin, int64_t Cout, int block, int gran_gy,
                               int gran_w, int rnd, uint64_t seed, float* gx,
                               void* ws, size_t ws_bytes, void* stream);

// ---------------------------------------------------------------------------
// Operators around the layer in a training step.  Each struct holds one
// call's arguments (row strides in elements) and is a kernel's parameter.
// ---------------------------------------------------------------------------
struct NormFwd {
  const void *x, *residual, *weight, *bias;  // residual, weight, bias may be null
  void *y, *h;                               // h null without residual
  float *mean, *rstd;                        // both or neither
  int64_t ldx, ldr, ldy, ldh, T, C;
  float eps;
  bool x_bf16, w_bf16, y_bf16;  // residual and h have the type of x, bias that of weight
  unsigned int* status;
};
cudaError_t launch_norm_fwd(const NormFwd& p, cudaStream_t st);

struct NormBwd {
  const void *gy, *x, *weight, *gres;  // weight, gres may be null
  const float *mean, *rstd;
  void* gx;
  float *gweight, *gbias;  // either may be null
  float* part;             // [slabs][2][C] partial column sums; null: not wanted
  int64_t ldgy, ldx, ldgr, ldgx, T, C;
  bool gy_bf16, x_bf16, w_bf16, gx_bf16;  // gres has the type of gx
  unsigned int* status;
};
// g_x, and (with part) *slabs slabs of partial column sums, which the join
// adds; 0 slabs: the column sums are written.
int norm_bwd_most_slabs(int64_t T);
cudaError_t launch_norm_bwd(const NormBwd& p, int* slabs, cudaStream_t st);
cudaError_t launch_norm_bwd_join(const NormBwd& p, int slabs, cudaStream_t st);

struct TokenLogprobs {
  const void* logits;
  const int64_t* targets;
  float *logp, *lse;  // lse may be null
  int64_t ld, T, V;
  float scale;
  bool bf16;
  unsigned int* status;
};
int64_t loss_most_rows(int64_t V);  // of one launch
cudaError_t launch_token_logprobs(const TokenLogprobs& p, cudaStream_t st);

struct PolicyLoss {
  const void* logits;
  const int64_t* actions;
  const float *old_logp, *ref_logp, *advantage, *weight;  // ref_logp may be null
  float *stats, *logp;                                    // logp may be null
  void* g;                                                // may be null
  float* part;                                            // [3][T] per-row terms of the sums
  int64_t ld, ldg, T, V;
  float scale, clip_low, clip_high, kl_coef, grad_scale;
  bool bf16;
  unsigned int* status;
};
cudaError_t launch_policy_rows(const PolicyLoss& p, cudaStream_t st);
cudaError_t launch_policy_stats(const PolicyLoss& p, cudaStream_t st);

// Up to kClipTensors tensors of a clipping call, cut into chunks of
// kClipChunk elements; chunk first[i] is the first one of tensor i.
constexpr int kClipTensors = 512;
constexpr int kClipChunk = 8192;
constexpr unsigned char kClipInBf16 = 1, kClipOutBf16 = 2;
struct ClipTable {
  const void* in[kClipTensors];
  void* out[kClipTensors];
  int64_t numel[kClipTensors], first[kClipTensors];
  unsigned char flags[kClipTensors];
  int n;
  int64_t chunks;
};
// The CTAs' norms, and what becomes of them.
struct ClipSums {
  const float* part;  // norms
  int n;
  float max_norm;
  float* norm_coef;
  unsigned int* status;
};
int clip_grid(int64_t chunks, int sms);
cudaError_t launch_clip_norm(const ClipTable& tab, float* part, int grid, cudaStream_t st);
cudaError_t launch_clip_coef(const ClipSums& q, cudaStream_t st);
// `first`: also writes norm and coefficient
cudaError_t launch_clip_scale(const ClipTable& tab, const ClipSums& q, bool first, int grid,
                              cudaStream_t st);

// ---------------------------------------------------------------------------
// Between a block's linear layers.
// ---------------------------------------------------------------------------
// [tokens, heads, D]: strides in elements.
struct Heads {
  void* p;
  int64_t token, head;
};
// Division of 0 <= n < 2^31 by d >= 1: with 2^s >= d, m = ceil(2^(31 + s) / d) is
// below 2^32 and n m / 2^(31 + s) is off by less than n / 2^31 / d < 1 / d.
struct Div {
  uint32_t d, m, s;
};
inline Div div_by(uint32_t d) {
  uint32_t s = 0;
  while (((uint64_t)1 << s) < d) ++s;
  return {d, (uint32_t)((((uint64_t)1 << (31 + s)) + d - 1) / d), 31 + s};
}
// One call of attention or of its backward pass.
struct Attn {
  Heads q, k, v, out;         // out: written forward, read backward
  float* lse;                 // [Tq, Hq], likewise
  Heads gout, gq, gk, gv;     // backward
  float *delta, *lse2;        // backward, workspace: [Hq, Tq] each
  Heads gout16;               // backward, workspace: g_out as bf16; p null where g_out itself is
  const int32_t *seqs_q, *seqs_k;  // both null: sequences of one length
  int batch, Tq, Tk, Hq, Hk, D;
  int Lq, Lk, group;          // of sequences of one length; Hq / Hk
  Div by_batch, by_hq, by_hk, by_group;
  int causal;
  float scale;
  bool bf16, gout_bf16, g_bf16;
  unsigned int* status;
};
bool attn_tc(const Attn& p);  // whether the tensor-core kernels take q, k and v
cudaError_t launch_attn_tc(const Attn& p, cudaStream_t st);
cudaError_t launch_attn_simt(const Attn& p, cudaStream_t st);
// delta, lse2 and g_out as bf16 (where p.gout16 has room for it)
cudaError_t launch_attn_bwd_rows(const Attn& p, cudaStream_t st);
bool attn_bwd_tc(const Attn& p);
cudaError_t launch_attn_bwd_tc(const Attn& p, cudaStream_t st);
cudaError_t launch_attn_bwd_simt(const Attn& p, cudaStream_t st);

struct Dropout {
  const void *x, *residual;  // residual may be null; it has y's type
  void* y;
  const uint64_t* d_seed;    // added to seed; may be null
  int64_t ldx, ldr, ldy, T, C;
  uint64_t seed;
  uint32_t drop;             // of 65536
  float scale;
  bool x_bf16, y_bf16;
};
cudaError_t launch_dropout(const Dropout& p, cudaStream_t st);

}  // namespace hlq
