/*
 * rtlynx_rope.h - rotary positions on the queries and keys that a block's
 * projections make, and the gradient of that rotation.
 *
 * Pair i of a head's first rot_dim channels turns by the token's angle
 *
 *   angle(t, i) = position[t, axis(i)] * inv_freq[i]
 *   y0 = scale * (x0 cos - x1 sin),   y1 = scale * (x1 cos + x0 sin)
 *
 * and the channels from rot_dim on are copied unchanged.  Pair i is channels
 * (i, i + rot_dim / 2), or (2i, 2i + 1) with RTL_ROPE_INTERLEAVED.  The
 * rotation is linear, so its gradient is the same call with
 * RTL_ROPE_INVERSE on the output's gradient (the angles negated).
 *
 * The angle is formed in fp64 and reduced to a quarter turn there: at position
 * 10^6 an fp32 product would be off by 0.06 radians.  Sine, cosine and the
 * rotation are fp32, and each result is rounded once to the tensor's type.
 * Long-context scalings live in the caller's inv_freq (stretched positions,
 * a stretched base, or a mix by frequency) and in `scale`.
 *
 * Conventions are those of rtlynx.h, with these differences: tensors are
 * strided (strides in elements, the channel stride is 1), base pointers need
 * only their element's alignment, tensors may pass 2 GiB, and an output may be
 * its own input (y == x with the same strides).  Any other overlap of an output with an
 * input or with another output is the caller's error.
 */
#ifndef RTLYNX_ROPE_H
#define RTLYNX_ROPE_H

#include "rtlynx.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of every x and y of a call (exactly one). */
#define RTL_ROPE_BF16 0x0u
#define RTL_ROPE_FP16 0x1u
#define RTL_ROPE_FP32 0x2u
/* Pairs (2i, 2i + 1) instead of (i, i + rot_dim / 2). */
#define RTL_ROPE_INTERLEAVED 0x10u
/* Turn back: the gradient (or, with scale 1, the inverse) of the rotation. */
#define RTL_ROPE_INVERSE 0x20u

#define RTL_ROPE_MAX_HEAD_DIM 1024
#define RTL_ROPE_MAX_AXES 4

/* One tensor [batch, tokens, heads, head_dim] and where its result goes. */
typedef struct {
  const void* x;
  void* y;
  int64_t heads;
  int64_t x_batch_stride, x_token_stride, x_head_stride; /* elements */
  int64_t y_batch_stride, y_token_stride, y_head_stride;
} rtl_rope_tensor;

/*
 * rtl_rope - rotates `count` (1 or 2, e.g. queries and keys) tensors of the
 * same batch, tokens and head_dim in one launch.
 *
 *   tensors     host array, read during the call only.
 *   head_dim    1 .. RTL_ROPE_MAX_HEAD_DIM; rot_dim even, 0 <= rot_dim <= head_dim.
 *   positions   int64, element (b, t, axis) at b * pos_batch_stride +
 *               t * pos_token_stride + axis (a batch stride of 0 shares one
 *               row of positions); any sign.  |position * inv_freq| up to
 *               2^28 radians keeps the angle exact to fp32.
 *   axes        1 .. RTL_ROPE_MAX_AXES.  axis_pairs: host array of `axes`
 *               counts >= 0 that sum to rot_dim / 2: the first axis_pairs[0] pairs
 *               use axis 0, the next axis_pairs[1] axis 1 and so on.  May be
 *               NULL when axes == 1.
 *   inv_freq    [rot_dim / 2] fp64 device array, radians per position.
 *   scale       multiplies the rotated channels (1 for none).
 *
 * With rot_dim 0 positions and inv_freq may be NULL.  No tokens, batch or heads is a
 * no-op.  Strides may be negative or, for inputs, 0; they must have |stride| < 2^40.
 */
rtl_status rtl_rope(const rtl_rope_tensor* tensors, int32_t count, int64_t batch, int64_t tokens,
                    int64_t head_dim, int64_t rot_dim, const int64_t* positions,
                    int64_t pos_batch_stride, int64_t pos_token_stride, int32_t axes,
                    const int32_t* axis_pairs, const double* inv_freq, float scale,
                    uint32_t flags, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* RTLYNX_ROPE_H */
