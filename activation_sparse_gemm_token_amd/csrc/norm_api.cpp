// Host side of include/rtlynx_norm.h: argument checks, then one launch (two with dweight).
#include "rtl_api.hpp"
#include "rtl_operators.hpp"
#include "rtlynx_norm.h"

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 31;
constexpr int64_t kMaxStride = (int64_t)1 << 40;

bool stride_ok(int64_t s) { return s >= 0 && s < kMaxStride; }

bool sizes_ok(int64_t batch, int64_t tokens, int64_t C) {
  return batch >= 0 && tokens >= 0 && batch < kMaxRows && tokens < kMaxRows && C >= 1 && C <= RTL_NORM_MAX_CHANNELS &&
         (tokens == 0 || batch <= (kMaxRows - 1) / tokens);
}

// The widest access, in elements, that divides every address.
struct Width {
  int bytes = 16;
  void add(const void* p) { add(static_cast<int64_t>(reinterpret_cast<uintptr_t>(p) & 15)); }
  void add(int64_t v) {
    while (v % bytes != 0) bytes /= 2;
  }
  // Weight or bias: beside 16-bit tensors fp32 ones are read 16 bytes at a time whatever the width.
  void affine(const void* p, int64_t stride, int elem, int wsize) {
    if (p == nullptr) return;
    const int64_t at = static_cast<int64_t>(reinterpret_cast<uintptr_t>(p) & 15) | (stride * wsize & 15);
    if (wsize > elem) bytes = at != 0 ? 2 : bytes;
    else add(at);
  }
  int vec(int elem) const { return bytes == 16 ? 16 / elem : bytes == 8 && elem == 2 ? 4 : 1; }
};

size_t partial_bytes(int64_t rows, int64_t C, int64_t groups) {
  const int64_t parts = rtl::norm_parts(rows, groups, C);
  return parts > 1 ? (size_t)(groups * parts) * 2 * (size_t)C * 4 : 0;
}

bool type_flags_ok(uint32_t flags) {
  return (flags & 0xFu) <= RTL_NORM_FP32 && (flags & ~(0xFu | RTL_NORM_AFFINE_FP32)) == 0;
}

}  // namespace

RTL_API rtl_status rtl_layer_norm(const void* x, int64_t batch, int64_t tokens, int64_t C, int64_t x_batch_stride,
                                  int64_t x_token_stride, const void* weight, int64_t weight_batch_stride,
                                  const void* bias, int64_t bias_batch_stride, float offset, float eps, void* y,
                                  int64_t y_batch_stride, int64_t y_token_stride, float* mean, float* rstd,
                                  uint32_t flags, void* hip_stream) {
  if (!type_flags_ok(flags)) return RTL_ERR_BAD_FLAGS;
  if (!sizes_ok(batch, tokens, C)) return RTL_ERR_BAD_SHAPE;
  for (int64_t s : {x_batch_stride, x_token_stride, weight_batch_stride, bias_batch_stride, y_batch_stride,
                    y_token_stride})
    if (!stride_ok(s)) return RTL_ERR_BAD_SHAPE;
  if (batch == 0 || tokens == 0) return RTL_OK;
  if (x == nullptr || y == nullptr || (bias != nullptr && weight == nullptr) || (mean == nullptr) != (rstd == nullptr))
    return RTL_ERR_NULL_POINTER;
  const int type = (int)(flags & 0xFu), elem = type == (int)RTL_NORM_FP32 ? 4 : 2;
  const int wsize = (flags & RTL_NORM_AFFINE_FP32) != 0 ? 4 : elem;
  if (!rtl::aligned(x, elem) || !rtl::aligned(y, elem) || !rtl::aligned(weight, wsize) || !rtl::aligned(bias, wsize) ||
      !rtl::aligned(mean, 4) || !rtl::aligned(rstd, 4))
    return RTL_ERR_MISALIGNED;
  Width w;
  w.add(x);
  w.add(y);
  for (int64_t s : {C, x_batch_stride, x_token_stride, y_batch_stride, y_token_stride}) w.add(s * elem);
  w.affine(weight, weight_batch_stride, elem, wsize);
  w.affine(bias, bias_batch_stride, elem, wsize);
  rtl::NormArgs a{};
  a.x = x;
  a.y = y;
  a.weight = weight;
  a.bias = bias;
  a.mean = mean;
  a.rstd = rstd;
  a.rows = batch * tokens;
  a.tokens = tokens;
  a.xb = x_batch_stride;
  a.xt = x_token_stride;
  a.yb = y_batch_stride;
  a.yt = y_token_stride;
  a.wb = weight_batch_stride;
  a.bb = bias_batch_stride;
  a.offset = offset;
  a.eps = eps;
  a.inv_c = (float)(1.0 / (double)C);
  a.C = (int)C;
  a.affine_fp32 = wsize == 4;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  const rtl_status d = rtl::check_device(stream);
  if (d != RTL_OK) return d;
  return rtl::from_hip(rtl::launch_norm(a, type, w.vec(elem), stream));
}

RTL_API size_t rtl_layer_norm_backward_workspace_bytes(int64_t batch, int64_t tokens, int64_t C, int64_t groups) {
  if (!sizes_ok(batch, tokens, C) || groups < 1 || (groups != 1 && groups != batch)) return 0;
  return partial_bytes(batch * tokens, C, groups);
}

RTL_API rtl_status rtl_layer_norm_backward(const void* dy, int64_t dy_batch_stride, int64_t dy_token_stride,
                                           const void* x, int64_t x_batch_stride, int64_t x_token_stride,
                                           const float* mean, const float* rstd, int64_t batch, int64_t tokens,
                                           int64_t C, const void* weight, int64_t weight_batch_stride, float offset,
                                           int64_t groups, void* dx, int64_t dx_batch_stride, int64_t dx_token_stride,
                                           void* dweight, void* dbias, void* workspace, size_t workspace_bytes,
                                           uint32_t flags, void* hip_stream) {
  if (!type_flags_ok(flags)) return RTL_ERR_BAD_FLAGS;
  if (!sizes_ok(batch, tokens, C) || (groups != 1 && groups != batch)) return RTL_ERR_BAD_SHAPE;
  for (int64_t s : {dy_batch_stride, dy_token_stride, x_batch_stride, x_token_stride, weight_batch_stride,
                    dx_batch_stride, dx_token_stride})
    if (!stride_ok(s)) return RTL_ERR_BAD_SHAPE;
  if (groups == 0) return RTL_OK;                       // no batch, one row of sums per sequence
  if ((dweight == nullptr) != (dbias == nullptr)) return RTL_ERR_NULL_POINTER;
  const int64_t rows = batch * tokens;
  if (rows == 0 && dweight == nullptr) return RTL_OK;
  if (rows > 0 && (dy == nullptr || x == nullptr || mean == nullptr || rstd == nullptr)) return RTL_ERR_NULL_POINTER;
  if (dx == nullptr && dweight == nullptr) return RTL_OK;
  const int type = (int)(flags & 0xFu), elem = type == (int)RTL_NORM_FP32 ? 4 : 2;
  const int wsize = (flags & RTL_NORM_AFFINE_FP32) != 0 ? 4 : elem;
  if (!rtl::aligned(x, elem) || !rtl::aligned(dy, elem) || !rtl::aligned(dx, elem) || !rtl::aligned(weight, wsize) ||
      !rtl::aligned(dweight, wsize) || !rtl::aligned(dbias, wsize) || !rtl::aligned(mean, 4) || !rtl::aligned(rstd, 4) ||
      !rtl::aligned(workspace, 16))
    return RTL_ERR_MISALIGNED;
  const size_t need = dweight != nullptr ? partial_bytes(rows, C, groups) : 0;
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return RTL_ERR_WORKSPACE;
  Width w;
  for (const void* p : {x, dy, (const void*)dx}) w.add(p);
  for (int64_t s : {C, x_batch_stride, x_token_stride, dy_batch_stride, dy_token_stride}) w.add(s * elem);
  if (dx != nullptr) {
    w.add(dx_batch_stride * elem);
    w.add(dx_token_stride * elem);
  }
  w.affine(weight, weight_batch_stride, elem, wsize);
  rtl::NormBackArgs a{};
  a.dy = dy;
  a.x = x;
  a.weight = weight;
  a.mean = mean;
  a.rstd = rstd;
  a.dx = dx;
  a.dweight = dweight;
  a.dbias = dbias;
  a.partials = static_cast<float*>(workspace);
  a.rows = rows;
  a.tokens = tokens > 0 ? tokens : 1;
  a.groups = groups;
  a.parts = rtl::norm_parts(rows, groups, C);
  a.gb = dy_batch_stride;
  a.gt = dy_token_stride;
  a.xb = x_batch_stride;
  a.xt = x_token_stride;
  a.db = dx_batch_stride;
  a.dt = dx_token_stride;
  a.wb = weight_batch_stride;
  a.offset = offset;
  a.inv_c = (float)(1.0 / (double)C);
  a.C = (int)C;
  a.affine_fp32 = wsize == 4;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  const rtl_status d = rtl::check_device(stream);
  if (d != RTL_OK) return d;
  return rtl::from_hip(rtl::launch_norm_backward(a, type, w.vec(elem), stream));
}
