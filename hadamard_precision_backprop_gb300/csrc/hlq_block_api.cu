// hlq_block_api.cu -- the C ABI of the operators between a block's linear
// layers (declared in include/hlq.h): argument validation and the launch
// sequence of each.
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "hlq.h"
#include "hlq_host.h"
#include "hlq_kernels.h"

namespace hlq {
namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 31;
// of attention: a tile (256 rows at most) may reach past a sequence's end in 32 bits
constexpr int64_t kMaxTokens = kMaxRows - 1024;
constexpr int64_t kMaxStride = (int64_t)1 << 40;
constexpr int kMaxHeadSize = 256;

bool dtype_ok(int dt) { return dt == HLQ_F32 || dt == HLQ_BF16; }
size_t elem_bytes(int dt) { return dt == HLQ_BF16 ? 2 : 4; }
bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// [T, H, D] with these strides: an input's may be anything from 0 on, an
// output's elements are apart from each other.
bool heads_strides_ok(const hlq_heads& x, int64_t T, int64_t H, int64_t D, bool input) {
  const int64_t t = T > 1 ? x.token_stride : 0, h = H > 1 ? x.head_stride : 0;
  if (t < 0 || h < 0 || t > kMaxStride || h > kMaxStride) return false;
  if (input) return true;
  // n - 1 steps of `inner` and one element row fit a step of `outer` (no product: it
  // may leave 64 bits)
  const auto fits = [&](int64_t outer, int64_t n, int64_t inner) {
    return outer >= D && (n <= 1 || n - 1 <= (outer - D) / inner);
  };
  const bool by_token = (H <= 1 || h >= D) && (T <= 1 || fits(t, H, h));
  const bool by_head = (T <= 1 || t >= D) && (H <= 1 || fits(h, T, t));
  return by_token || by_head;
}

Heads heads_of(const hlq_heads& x, int64_t T, int64_t H) {
  return {x.ptr, T > 1 ? x.token_stride : 0, H > 1 ? x.head_stride : 0};
}

hlq_status check_sizes(int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hk, int64_t D, int64_t batch) {
  if (Tq < 0 || Tk < 0 || Hq < 1 || Hk < 1 || Hq % Hk != 0 || D < 1 || batch < 1)
    return HLQ_ERR_SHAPE;
  if (D > kMaxHeadSize || Tq > kMaxTokens || Tk > kMaxTokens || Hq >= kMaxRows ||
      Tq * Hq >= kMaxRows || Tk * Hk >= kMaxRows || batch >= kMaxRows ||
      (batch + 1) * Hq >= kMaxRows / 2)
    return HLQ_ERR_UNSUPPORTED;
  return HLQ_OK;
}

// The checks that both passes share, after check_sizes.
hlq_status check_seqs(int64_t Tq, int64_t Tk, int64_t batch, const int32_t* seqs,
                      const int32_t* seqs_k, float scale) {
  // beyond these its product with log2(e), or the inverse, may leave fp32's range
  if (!(scale >= 0x1p-64f && scale <= 0x1p64f)) return HLQ_ERR_INVALID_ARG;
  if (!seqs && seqs_k) return HLQ_ERR_INVALID_ARG;
  if (!seqs && (Tq % batch != 0 || Tk % batch != 0)) return HLQ_ERR_SHAPE;
  if (seqs && !seqs_k && Tq != Tk) return HLQ_ERR_SHAPE;
  if (!aligned_to(seqs, 4) || !aligned_to(seqs_k, 4)) return HLQ_ERR_ALIGN;
  return HLQ_OK;
}

hlq_status check_heads(const hlq_heads* x, int dt, int64_t T, int64_t H, int64_t D, bool input) {
  if (!x || (T > 0 && !x->ptr)) return HLQ_ERR_INVALID_ARG;
  if (!heads_strides_ok(*x, T, H, D, input)) return HLQ_ERR_SHAPE;
  return aligned_to(x->ptr, elem_bytes(dt)) ? HLQ_OK : HLQ_ERR_ALIGN;
}

#define HLQ_NEED(expr)                \
  do {                                \
    const hlq_status _s = (expr);     \
    if (_s != HLQ_OK) return _s;      \
  } while (0)

Attn attn_of(const hlq_heads& q, const hlq_heads& k, const hlq_heads& v, int dt, int64_t Tq,
             int64_t Tk, int64_t Hq, int64_t Hk, int64_t D, const int32_t* seqs,
             const int32_t* seqs_k, int64_t batch, int causal, float scale) {
  Attn p{};
  p.q = heads_of(q, Tq, Hq), p.k = heads_of(k, Tk, Hk), p.v = heads_of(v, Tk, Hk);
  p.seqs_q = seqs, p.seqs_k = seqs_k ? seqs_k : seqs;
  p.batch = (int)batch, p.Tq = (int)Tq, p.Tk = (int)Tk, p.Hq = (int)Hq, p.Hk = (int)Hk;
  p.D = (int)D;
  p.Lq = (int)(Tq / batch), p.Lk = (int)(Tk / batch), p.group = (int)(Hq / Hk);
  p.by_batch = div_by((uint32_t)batch), p.by_group = div_by((uint32_t)p.group);
  p.by_hq = div_by((uint32_t)Hq), p.by_hk = div_by((uint32_t)Hk);
  p.causal = causal != 0;
  p.scale = scale;
  p.bf16 = dt == HLQ_BF16;
  return p;
}

// Workspace of the backward pass: delta, lse2, and g_out as bf16 (rows of whole
// 16 bytes) where it comes as fp32 beside bf16 queries.
struct BwdWs {
  size_t delta, lse2, gout16, bytes;
  int64_t head16;  // its head stride
};
BwdWs bwd_ws(int64_t Tq, int64_t Hq, int64_t D, int dt, int gout_dt) {
  BwdWs w{};
  const size_t stats = align_up((size_t)Tq * Hq * 4);
  w.lse2 = stats, w.gout16 = 2 * stats;
  w.head16 = (D + 7) / 8 * 8;
  w.bytes = w.gout16;
  if (dt == HLQ_BF16 && gout_dt == HLQ_F32) w.bytes += align_up((size_t)Tq * Hq * w.head16 * 2);
  return w;
}

}  // namespace
}  // namespace hlq

using namespace hlq;

extern "C" {

hlq_status hlq_attention(const hlq_heads* q, const hlq_heads* k, const hlq_heads* v, int dt,
                         int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hk, int64_t D,
                         const int32_t* d_seqs, const int32_t* d_seqs_k, int64_t batch,
                         int causal, float scale, const hlq_heads* out, float* d_lse,
                         void* stream) {
  if (!dtype_ok(dt)) return HLQ_ERR_INVALID_ARG;
  HLQ_NEED(check_sizes(Tq, Tk, Hq, Hk, D, batch));
  HLQ_NEED(check_seqs(Tq, Tk, batch, d_seqs, d_seqs_k, scale));
  HLQ_NEED(check_heads(q, dt, Tq, Hq, D, true));
  HLQ_NEED(check_heads(k, dt, Tk, Hk, D, true));
  HLQ_NEED(check_heads(v, dt, Tk, Hk, D, true));
  HLQ_NEED(check_heads(out, dt, Tq, Hq, D, false));
  if (Tq > 0 && !d_lse) return HLQ_ERR_INVALID_ARG;
  if (!aligned_to(d_lse, 4)) return HLQ_ERR_ALIGN;
  if (Tq == 0) return HLQ_OK;
  Attn p = attn_of(*q, *k, *v, dt, Tq, Tk, Hq, Hk, D, d_seqs, d_seqs_k, batch, causal, scale);
  p.out = heads_of(*out, Tq, Hq), p.lse = d_lse;
  p.status = device_status_ptr();
  if (!p.status) return HLQ_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (attn_tc(p))
    HLQ_LAUNCH("attn_fwd_tc", s, launch_attn_tc(p, s));
  else
    HLQ_LAUNCH("attn_fwd", s, launch_attn_simt(p, s));
  return HLQ_OK;
}

size_t hlq_attention_backward_workspace_bytes(int64_t Tq, int64_t Hq, int64_t D, int dt,
                                              int gout_dt) {
  if (!dtype_ok(dt) || !dtype_ok(gout_dt) || check_sizes(Tq, 0, Hq, 1, D, 1) != HLQ_OK) return 0;
  return bwd_ws(Tq, Hq, D, dt, gout_dt).bytes;
}

hlq_status hlq_attention_backward(const hlq_heads* g_out, int gout_dt, const hlq_heads* q,
                                  const hlq_heads* k, const hlq_heads* v, const hlq_heads* out,
                                  int dt, const float* d_lse, int64_t Tq, int64_t Tk, int64_t Hq,
                                  int64_t Hk, int64_t D, const int32_t* d_seqs,
                                  const int32_t* d_seqs_k, int64_t batch, int causal, float scale,
                                  const hlq_heads* g_q, const hlq_heads* g_k,
                                  const hlq_heads* g_v, int g_dt, void* d_ws, size_t ws_bytes,
                                  void* stream) {
  if (!dtype_ok(dt) || !dtype_ok(gout_dt) || !dtype_ok(g_dt)) return HLQ_ERR_INVALID_ARG;
  HLQ_NEED(check_sizes(Tq, Tk, Hq, Hk, D, batch));
  // the CTAs of both sides are one grid: tiles of 32 rows at least, and one that may
  // stay empty for each sequence, and for the rows outside them
  if ((Tq / 32 + batch + 2) * Hq + (Tk / 32 + batch + 2) * Hk >= kMaxRows)
    return HLQ_ERR_UNSUPPORTED;
  HLQ_NEED(check_seqs(Tq, Tk, batch, d_seqs, d_seqs_k, scale));
  HLQ_NEED(check_heads(g_out, gout_dt, Tq, Hq, D, true));
  HLQ_NEED(check_heads(q, dt, Tq, Hq, D, true));
  HLQ_NEED(check_heads(k, dt, Tk, Hk, D, true));
  HLQ_NEED(check_heads(v, dt, Tk, Hk, D, true));
  HLQ_NEED(check_heads(out, dt, Tq, Hq, D, true));
  HLQ_NEED(check_heads(g_q, g_dt, Tq, Hq, D, false));
  HLQ_NEED(check_heads(g_k, g_dt, Tk, Hk, D, false));
  HLQ_NEED(check_heads(g_v, g_dt, Tk, Hk, D, false));
  if (Tq > 0 && !d_lse) return HLQ_ERR_INVALID_ARG;
  if (!aligned_to(d_lse, 4)) return HLQ_ERR_ALIGN;
  const BwdWs w = bwd_ws(Tq, Hq, D, dt, gout_dt);
  if (w.bytes > 0) {
    if (!d_ws || ws_bytes < w.bytes) return HLQ_ERR_WORKSPACE;
    if (!aligned256(d_ws)) return HLQ_ERR_ALIGN;
  }
  if (Tq == 0 && Tk == 0) return HLQ_OK;
  Attn p = attn_of(*q, *k, *v, dt, Tq, Tk, Hq, Hk, D, d_seqs, d_seqs_k, batch, causal, scale);
  p.out = heads_of(*out, Tq, Hq), p.lse = const_cast<float*>(d_lse);
  p.gout = heads_of(*g_out, Tq, Hq), p.gout_bf16 = gout_dt == HLQ_BF16;
  p.gq = heads_of(*g_q, Tq, Hq), p.gk = heads_of(*g_k, Tk, Hk), p.gv = heads_of(*g_v, Tk, Hk);
  p.g_bf16 = g_dt == HLQ_BF16;
  char* ws = static_cast<char*>(d_ws);
  p.delta = reinterpret_cast<float*>(ws + w.delta), p.lse2 = reinterpret_cast<float*>(ws + w.lse2);
  p.status = device_status_ptr();
  if (!p.status) return HLQ_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool tc = attn_bwd_tc(p);
  if (tc && !p.gout_bf16) p.gout16 = {ws + w.gout16, Hq * w.head16, w.head16};
  if (Tq > 0) HLQ_LAUNCH("attn_bwd_rows", s, launch_attn_bwd_rows(p, s));
  if (tc)
    HLQ_LAUNCH("attn_bwd_tc", s, launch_attn_bwd_tc(p, s));
  else
    HLQ_LAUNCH("attn_bwd", s, launch_attn_bwd_simt(p, s));
  return HLQ_OK;
}

hlq_status hlq_dropout(const void* d_x, int64_t ldx, int x_dt, const void* d_residual,
                       int64_t ldr, int64_t T, int64_t C, double p, uint64_t seed,
                       const uint64_t* d_seed, void* d_y, int64_t ldy, int y_dt, void* stream) {
  if (!dtype_ok(x_dt) || !dtype_ok(y_dt) || !(p >= 0.0 && p <= 1.0)) return HLQ_ERR_INVALID_ARG;
  if (T < 0 || C < 1) return HLQ_ERR_SHAPE;
  if (T >= kMaxRows || C >= kMaxRows) return HLQ_ERR_UNSUPPORTED;
  if (T > 0 && (!d_x || !d_y)) return HLQ_ERR_INVALID_ARG;
  const auto stride_ok = [&](int64_t ld, bool input) {
    return T <= 1 || (ld >= C && ld <= kMaxStride) || (input && ld == 0);
  };
  if (!stride_ok(ldx, true) || !stride_ok(ldy, false) || (d_residual && !stride_ok(ldr, true)))
    return HLQ_ERR_SHAPE;
  if (!aligned_to(d_x, elem_bytes(x_dt)) || !aligned_to(d_y, elem_bytes(y_dt)) ||
      !aligned_to(d_residual, elem_bytes(y_dt)) || !aligned_to(d_seed, 8))
    return HLQ_ERR_ALIGN;
  if (T == 0) return HLQ_OK;
  Dropout a{};
  a.x = d_x, a.residual = d_residual, a.y = d_y, a.d_seed = d_seed;
  a.ldx = ldx, a.ldr = ldr, a.ldy = ldy, a.T = T, a.C = C;
  a.seed = seed;
  a.drop = (uint32_t)std::nearbyint(p * 65536.0);
  a.scale = a.drop < 65536 ? (float)(65536.0 / (65536.0 - a.drop)) : 0.f;
  a.x_bf16 = x_dt == HLQ_BF16, a.y_bf16 = y_dt == HLQ_BF16;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  HLQ_LAUNCH("dropout", s, launch_dropout(a, s));
  return HLQ_OK;
}

}  // extern "C"
