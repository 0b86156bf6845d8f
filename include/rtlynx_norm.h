/*
 * rtlynx_norm.h - layer norm of the tokens that a block's projections read,
 * and its gradients.
 *
 *   mean = sum x / C,  rstd = 1 / sqrt(sum (x - mean)^2 / C + eps)
 *   y = (x - mean) * rstd * (offset + weight) + bias
 *
 * weight and bias have one value per channel, or one row per sequence (the
 * modulation that a diffusion transformer forms from its time embedding; offset 1
 * then makes the factor 1 + weight).  Without a weight the factor is 1 and
 * there is no bias.  Sums are fp32, the variance is that of the centred
 * values, and each result is rounded once to the tensor's type.
 *
 * Conventions are those of rtlynx.h, with these differences: x, y, dy and dx
 * are [batch, tokens, C] with strides in elements (the channel stride is 1),
 * base pointers need only their element's alignment (16-byte aligned rows are
 * faster), and tensors may pass 2 GiB.  y may be x (same strides), and dx may
 * be dy or x; any other overlap of an output is the caller's error.
 */
#ifndef RTLYNX_NORM_H
#define RTLYNX_NORM_H

#include "rtlynx.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of x, y, dy and dx (exactly one). */
#define RTL_NORM_BF16 0x0u
#define RTL_NORM_FP16 0x1u
#define RTL_NORM_FP32 0x2u
/* weight, bias and their gradients are fp32 whatever the tensors' type. */
#define RTL_NORM_AFFINE_FP32 0x10u

#define RTL_NORM_MAX_CHANNELS 32768

/*
 * rtl_layer_norm - the forward pass.
 *
 *   C             1 .. RTL_NORM_MAX_CHANNELS.  batch * tokens < 2^31.
 *   weight, bias  [C] or, with a batch stride, one row per sequence (0: one row
 *                 for all); NULL for none, a bias needs a weight.
 *   mean, rstd    fp32 [batch * tokens], what the backward pass reads; both or
 *                 neither NULL.
 *
 * No batch or no tokens is a no-op.  0 <= strides < 2^40.
 */
rtl_status rtl_layer_norm(const void* x, int64_t batch, int64_t tokens, int64_t C,
                          int64_t x_batch_stride, int64_t x_token_stride,
                          const void* weight, int64_t weight_batch_stride,
                          const void* bias, int64_t bias_batch_stride, float offset, float eps,
                          void* y, int64_t y_batch_stride, int64_t y_token_stride,
                          float* mean, float* rstd, uint32_t flags, void* hip_stream);

/*
 * rtl_layer_norm_backward - with g = dy * (offset + weight) and xhat the
 * normalised x:
 *
 *   dx = rstd * (g - mean(g) - xhat * mean(g xhat))
 *   dweight = sum over tokens of dy xhat,  dbias = sum over tokens of dy
 *
 *   groups          rows of weight, dweight and dbias: 1, or batch.
 *   dx              may be NULL.  dweight, dbias: [groups, C], densely
 *                   packed, of the weight's type; both or neither NULL.
 *   workspace       rtl_layer_norm_backward_workspace_bytes(batch, tokens, C,
 *                   groups) bytes (0 for few rows), 16-byte aligned; may be NULL
 *                   without dweight.
 *
 * The sums over tokens are formed in an order that only the sizes fix.  With
 * no tokens dweight and dbias are zeros.
 */
size_t rtl_layer_norm_backward_workspace_bytes(int64_t batch, int64_t tokens, int64_t C, int64_t groups);

rtl_status rtl_layer_norm_backward(const void* dy, int64_t dy_batch_stride, int64_t dy_token_stride,
                                   const void* x, int64_t x_batch_stride, int64_t x_token_stride,
                                   const float* mean, const float* rstd,
                                   int64_t batch, int64_t tokens, int64_t C,
                                   const void* weight, int64_t weight_batch_stride, float offset, int64_t groups,
                                   void* dx, int64_t dx_batch_stride, int64_t dx_token_stride,
                                   void* dweight, void* dbias, void* workspace, size_t workspace_bytes,
                                   uint32_t flags, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* RTLYNX_NORM_H */
