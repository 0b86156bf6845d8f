// Host side of include/rtlynx_rope.h: argument checks, then one launch.
#include "rtl_api.hpp"
#include "rtl_operators.hpp"
#include "rtlynx_rope.h"

namespace {

constexpr int64_t kMaxCount = (int64_t)1 << 31;
constexpr int64_t kMaxStride = (int64_t)1 << 40;

bool stride_ok(int64_t s) { return s > -kMaxStride && s < kMaxStride; }

}  // namespace

RTL_API rtl_status rtl_rope(const rtl_rope_tensor* tensors, int32_t count, int64_t batch, int64_t tokens,
                            int64_t head_dim, int64_t rot_dim, const int64_t* positions,
                            int64_t pos_batch_stride, int64_t pos_token_stride, int32_t axes,
                            const int32_t* axis_pairs, const double* inv_freq, float scale, uint32_t flags,
                            void* hip_stream) {
  const uint32_t type = flags & 0xFu;
  if (type > RTL_ROPE_FP32 || (flags & ~(0xFu | RTL_ROPE_INTERLEAVED | RTL_ROPE_INVERSE)) != 0)
    return RTL_ERR_BAD_FLAGS;
  if (count < 1 || count > 2 || batch < 0 || tokens < 0 || batch >= kMaxCount || tokens >= kMaxCount ||
      (tokens > 0 && batch >= kMaxCount / tokens) || head_dim < 1 || head_dim > RTL_ROPE_MAX_HEAD_DIM || rot_dim < 0 ||
      rot_dim > head_dim || rot_dim % 2 != 0 || axes < 1 || axes > RTL_ROPE_MAX_AXES)
    return RTL_ERR_BAD_SHAPE;
  if (tensors == nullptr || (axis_pairs == nullptr && axes > 1)) return RTL_ERR_NULL_POINTER;
  if (!stride_ok(pos_batch_stride) || !stride_ok(pos_token_stride)) return RTL_ERR_BAD_SHAPE;
  rtl::RopeArgs a{};
  int64_t sum = 0;
  for (int i = 0; i < 3; ++i) a.axis_end[i] = (int)(rot_dim / 2);
  for (int i = 0; axis_pairs != nullptr && i < axes; ++i) {
    if (axis_pairs[i] < 0) return RTL_ERR_BAD_SHAPE;
    sum += axis_pairs[i];
    if (sum > rot_dim / 2) return RTL_ERR_BAD_SHAPE;
    if (i + 1 < axes) a.axis_end[i] = (int)sum;
  }
  if (axis_pairs != nullptr && sum != rot_dim / 2) return RTL_ERR_BAD_SHAPE;
  const int elem = type == RTL_ROPE_FP32 ? 4 : 2;
  int64_t heads = 0;
  int n = 0;
  for (int i = 0; i < count; ++i) {
    const rtl_rope_tensor& t = tensors[i];
    if (t.heads < 0 || t.heads >= (1 << 20)) return RTL_ERR_BAD_SHAPE;
    for (int64_t s : {t.x_batch_stride, t.x_token_stride, t.x_head_stride, t.y_batch_stride, t.y_token_stride,
                      t.y_head_stride})
      if (!stride_ok(s)) return RTL_ERR_BAD_SHAPE;
    if (t.heads == 0 || batch == 0 || tokens == 0) continue;
    if (t.x == nullptr || t.y == nullptr) return RTL_ERR_NULL_POINTER;
    if (!rtl::aligned(t.x, elem) || !rtl::aligned(t.y, elem)) return RTL_ERR_MISALIGNED;
    heads += t.heads;
    a.t[n++] = {t.x, t.y, t.x_batch_stride, t.x_token_stride, t.x_head_stride, t.y_batch_stride, t.y_token_stride,
                t.y_head_stride, (int)t.heads,
                t.x == t.y && t.x_batch_stride == t.y_batch_stride && t.x_token_stride == t.y_token_stride &&
                    t.x_head_stride == t.y_head_stride};
  }
  if (heads == 0) return RTL_OK;
  if (rot_dim > 0) {
    if (positions == nullptr || inv_freq == nullptr) return RTL_ERR_NULL_POINTER;
    if (!rtl::aligned(positions, 8) || !rtl::aligned(inv_freq, 8)) return RTL_ERR_MISALIGNED;
  }
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.total = batch * tokens;
  a.tokens = tokens;
  a.pos_b = pos_batch_stride;
  a.pos_t = pos_token_stride;
  a.dim = (int)head_dim;
  a.rot = (int)rot_dim;
  a.scale = scale;
  a.inverse = (flags & RTL_ROPE_INVERSE) != 0;
  int cus = 0;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  const rtl_status d = rtl::check_device(stream, &cus);
  if (d != RTL_OK) return d;
  return rtl::from_hip(rtl::launch_rope(a, elem, type == RTL_ROPE_FP16, (flags & RTL_ROPE_INTERLEAVED) != 0,
                                        cus > 0 ? cus : 1, stream));
}
