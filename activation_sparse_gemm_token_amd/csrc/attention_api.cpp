// Host side of include/rtlynx_attention.h: argument checks, then the launches.
#include <cmath>

#include "rtl_api.hpp"
#include "rtl_operators.hpp"
#include "rtlynx_attention.h"

namespace {

constexpr int64_t kMaxTokens = (int64_t)1 << 31;
constexpr int64_t kMaxStride = (int64_t)1 << 40, kMaxTokenStride = (int64_t)1 << 23;
constexpr int64_t kMaxRows = (int64_t)1 << 38;
constexpr int64_t kMaxHeads = (int64_t)1 << 20;

bool product_below(int64_t limit, int64_t a, int64_t b, int64_t c) {
  if (a == 0 || b == 0 || c == 0) return true;
  return a < limit && b <= limit / a && c <= (limit - 1) / (a * b);
}

rtl_status check_shape(const rtl_attn_shape* s) {
  if (s == nullptr) return RTL_ERR_NULL_POINTER;
  if (s->sequences < 0 || s->tokens_q < 0 || s->tokens_k < 0 || s->heads_q < 0 || s->heads_k < 0 ||
      s->sequences >= kMaxTokens || s->tokens_q >= kMaxTokens || s->tokens_k >= kMaxTokens || s->heads_q >= kMaxHeads ||
      s->heads_k >= kMaxHeads || s->head_dim < 8 || s->head_dim > RTL_ATTN_MAX_HEAD_DIM || s->head_dim % 8 != 0)
    return RTL_ERR_BAD_SHAPE;
  if (s->heads_k == 0 ? s->heads_q != 0 : s->heads_q % s->heads_k != 0) return RTL_ERR_BAD_SHAPE;
  if (!std::isfinite(s->scale) || s->scale < 0.f) return RTL_ERR_BAD_SHAPE;
  const bool packed = s->q_starts != nullptr;
  if (packed != (s->k_starts != nullptr)) return RTL_ERR_NULL_POINTER;
  if (packed && s->k_lens != nullptr) return RTL_ERR_BAD_SHAPE;
  const int64_t n = packed ? 1 : s->sequences;
  if (!product_below(kMaxRows, n, s->heads_q, s->tokens_q) || !product_below(kMaxRows, n, s->heads_k, s->tokens_k) ||
      !product_below(kMaxRows, s->sequences + 2, s->heads_q, 1))
    return RTL_ERR_BAD_SHAPE;
  if (!rtl::aligned(s->q_starts, 4) || !rtl::aligned(s->k_starts, 4) || !rtl::aligned(s->k_lens, 4)) return RTL_ERR_MISALIGNED;
  return RTL_OK;
}

// `rows`: whether the tensor has any.
rtl_status check_tensor(const rtl_attn_tensor* t, bool rows) {
  if (t == nullptr || (rows && t->data == nullptr)) return RTL_ERR_NULL_POINTER;
  for (int64_t s : {t->batch_stride, t->token_stride, t->head_stride})
    if (s < 0 || s >= kMaxStride || s % 8 != 0) return RTL_ERR_BAD_SHAPE;
  if (t->token_stride >= kMaxTokenStride) return RTL_ERR_BAD_SHAPE;
  return rtl::aligned(t->data, 16) ? RTL_OK : RTL_ERR_MISALIGNED;
}

rtl::AttnTensor tensor(const rtl_attn_tensor* t) {
  return {static_cast<uint16_t*>(t->data), t->batch_stride, t->token_stride, t->head_stride};
}

rtl::AttnPlan plan_of(const rtl_attn_shape* s, bool causal) {
  return rtl::attn_plan(s->sequences, s->tokens_q, s->tokens_k, s->heads_q, s->heads_k, s->head_dim, s->q_starts != nullptr,
                        causal);
}

size_t plan_bytes(const rtl::AttnPlan& p, const rtl_attn_shape* s) {
  return rtl::attn_plan_bytes(p, s->sequences, s->tokens_q, s->heads_q, s->head_dim);
}

int64_t query_rows(const rtl_attn_shape* s) { return (s->q_starts != nullptr ? 1 : s->sequences) * s->heads_q * s->tokens_q; }

int back_splits(const rtl_attn_shape* s) {
  return rtl::attn_back_splits(s->sequences, s->tokens_q, s->tokens_k, s->heads_q, s->heads_k, s->q_starts != nullptr);
}

size_t stats_bytes(const rtl_attn_shape* s) { return ((size_t)query_rows(s) * 8 + 15) / 16 * 16; }

size_t backward_bytes(const rtl_attn_shape* s) {
  const int splits = back_splits(s);
  const size_t rows = (size_t)((s->q_starts != nullptr ? 1 : s->sequences) * s->tokens_k * s->heads_k);
  return stats_bytes(s) + (splits > 1 ? (size_t)splits * 2 * rows * (size_t)s->head_dim * 4 : 0);
}

rtl::AttnArgs arguments(const rtl_attn_shape* s, uint32_t flags) {
  rtl::AttnArgs a{};
  a.q_starts = s->q_starts;
  a.k_starts = s->k_starts;
  a.k_lens = s->k_lens;
  a.sequences = s->sequences;
  a.tq = s->tokens_q;
  a.tk = s->tokens_k;
  a.hq = (int)s->heads_q;
  a.hk = (int)s->heads_k;
  a.group = (int)(s->heads_q / s->heads_k);
  a.d = (int)s->head_dim;
  a.scale = s->scale;
  // A scale of 0 must not meet the -inf of a hidden score.
  a.c = s->scale * 1.4426950408889634f;
  if (a.c < 1.2e-38f) a.c = 1.2e-38f;
  a.causal = (flags & RTL_ATTN_CAUSAL) != 0;
  a.zero_rest = (flags & RTL_ATTN_ZERO_REST) != 0;
  return a;
}

}  // namespace

RTL_API size_t rtl_attention_workspace_bytes(const rtl_attn_shape* shape, uint32_t flags) {
  return check_shape(shape) == RTL_OK ? plan_bytes(plan_of(shape, (flags & RTL_ATTN_CAUSAL) != 0), shape) : 0;
}

RTL_API rtl_status rtl_attention(const rtl_attn_tensor* q, const rtl_attn_tensor* k, const rtl_attn_tensor* v,
                                 const rtl_attn_tensor* o, float* lse, const rtl_attn_shape* shape, void* workspace,
                                 size_t workspace_bytes, uint32_t flags, void* hip_stream) {
  if ((flags & 0xFu) > RTL_ATTN_FP16 || (flags & ~(0xFu | RTL_ATTN_CAUSAL | RTL_ATTN_ZERO_REST)) != 0)
    return RTL_ERR_BAD_FLAGS;
  rtl_status st = check_shape(shape);
  if (st != RTL_OK) return st;
  const bool any = query_rows(shape) > 0 && shape->sequences > 0;
  const rtl_attn_tensor* const all[] = {q, k, v, o};
  for (int i = 0; i < 4; ++i) {
    st = check_tensor(all[i], any && (i == 0 || i == 3 || shape->tokens_k > 0));
    if (st != RTL_OK) return st;
  }
  if (!any) return RTL_OK;
  if (!rtl::aligned(lse, 4) || !rtl::aligned(workspace, 16)) return RTL_ERR_MISALIGNED;
  const rtl::AttnPlan plan = plan_of(shape, (flags & RTL_ATTN_CAUSAL) != 0);
  const size_t need = plan_bytes(plan, shape);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return RTL_ERR_WORKSPACE;
  rtl::AttnArgs a = arguments(shape, flags);
  a.q = tensor(q);
  a.k = tensor(k);
  a.v = tensor(v);
  a.o = tensor(o);
  a.lse = lse;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  st = rtl::check_device(stream);
  if (st != RTL_OK) return st;
  return rtl::from_hip(rtl::launch_attention(a, plan, (flags & 0xFu) == RTL_ATTN_FP16, workspace, stream));
}

RTL_API size_t rtl_attention_backward_workspace_bytes(const rtl_attn_shape* shape) {
  return check_shape(shape) == RTL_OK ? backward_bytes(shape) : 0;
}

RTL_API rtl_status rtl_attention_backward(const rtl_attn_tensor* d_o, const rtl_attn_tensor* q, const rtl_attn_tensor* k,
                                          const rtl_attn_tensor* v, const rtl_attn_tensor* o, const float* lse,
                                          const rtl_attn_tensor* dq, const rtl_attn_tensor* dk, const rtl_attn_tensor* dv,
                                          const rtl_attn_shape* shape, void* workspace, size_t workspace_bytes,
                                          uint32_t flags, void* hip_stream) {
  if ((flags & ~RTL_ATTN_CAUSAL) != 0) return RTL_ERR_BAD_FLAGS;
  rtl_status st = check_shape(shape);
  if (st != RTL_OK) return st;
  const int64_t n = shape->q_starts != nullptr ? (shape->sequences > 0) : shape->sequences;
  const bool any_q = query_rows(shape) > 0 && shape->sequences > 0;
  const bool any_k = n * shape->heads_k * shape->tokens_k > 0;
  for (const rtl_attn_tensor* t : {d_o, q, o, dq})
    if ((st = check_tensor(t, any_q)) != RTL_OK) return st;
  for (const rtl_attn_tensor* t : {k, v, dk, dv})
    if ((st = check_tensor(t, any_k)) != RTL_OK) return st;
  if (!any_q && !any_k) return RTL_OK;
  if (any_q && lse == nullptr) return RTL_ERR_NULL_POINTER;
  if (!rtl::aligned(lse, 4) || !rtl::aligned(workspace, 16)) return RTL_ERR_MISALIGNED;
  const size_t need = backward_bytes(shape);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return RTL_ERR_WORKSPACE;
  rtl::AttnBackArgs a{};
  a.f = arguments(shape, flags);
  a.f.q = tensor(q);
  a.f.k = tensor(k);
  a.f.v = tensor(v);
  a.f.o = tensor(o);
  a.f.lse = const_cast<float*>(lse);
  a.d_o = tensor(d_o);
  a.dq = tensor(dq);
  a.dk = tensor(dk);
  a.dv = tensor(dv);
  a.stats = static_cast<rtl::f32x2*>(workspace);
  a.f.splits = back_splits(shape);
  a.f.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + stats_bytes(shape));
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  st = rtl::check_device(stream);
  if (st != RTL_OK) return st;
  return rtl::from_hip(rtl::launch_attention_backward(a, stream));
}
