/*
 * rtlynx_dense.h - the dense linear layer with what follows it in its
 * epilogue, and its gradients: the output projection into the residual
 * stream, an MLP's first half, a modulation.  (rtl_layer_linear's dense layers
 * are the plain rtl_dense_linear.)
 *
 *   z = x w^T + bias
 *   y = residual + gate * act(z)
 *
 * Accumulation, bias, activation, gate and residual are fp32 and y is rounded
 * once.  act is none, GELU (z Phi(z)), its tanh form, or SiLU (z / (1 + e^-z)).
 * An infinite z (a sum past fp32, or kept in a type that it passes) has its
 * limits: act inf and 0, slope 1 and 0.
 * The gate has one value per output channel, or one row per sequence (rows of
 * x in equal parts).
 *
 * Conventions are those of rtlynx.h, with these differences: tensors are bf16
 * or fp16 (exactly one flag), K is a multiple of 8, and y may be the residual
 * itself.  N need not be a multiple of anything; bias and gate need only their
 * element's alignment.
 */
#ifndef RTLYNX_DENSE_H
#define RTLYNX_DENSE_H

#include "rtlynx.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of every tensor. */
#define RTL_DENSE_BF16 0x0u
#define RTL_DENSE_FP16 0x1u
/* Activation (one of). */
#define RTL_DENSE_GELU 0x10u
#define RTL_DENSE_GELU_TANH 0x20u
#define RTL_DENSE_SILU 0x30u
/* z is fp32.  A gate's gradient is a sum of dy act(z) and carries z's rounding
 * (0.26 % off in bf16, 0.17 % with fp32); the other gradients hardly do. */
#define RTL_DENSE_Z_FP32 0x200u

/*
 * rtl_linear - the forward pass.
 *
 *   x         [M, K], w [N, K], y [M, N].
 *   bias      [N], or NULL.
 *   gate      [N] for every row (gate_rows 1), or gate_rows (at most 65535) rows of N values,
 *             gate_stride elements apart, each for M / gate_rows rows of x;
 *             NULL for none.
 *   residual  [M, N], or NULL.
 *   z         [M, N], for the backward pass, rounded to the tensors' type or fp32
 *             (RTL_DENSE_Z_FP32); NULL if not wanted.
 *   workspace rtl_linear_workspace_bytes(M, N, K) bytes, 16-byte aligned (0
 *             for most sizes: it serves products split over K).
 *
 * M == 0 or N == 0 is a no-op.  N, K < 2^25, every tensor below 2 GiB, 0 <= gate_stride < 2^40.
 */
size_t rtl_linear_workspace_bytes(int64_t M, int64_t N, int64_t K);

rtl_status rtl_linear(const void* x, const void* w, const void* bias, const void* gate, int64_t gate_rows,
                      int64_t gate_stride, const void* residual, int64_t M, int64_t N, int64_t K, void* y, void* z,
                      void* workspace, size_t workspace_bytes, uint32_t flags, void* hip_stream);

/*
 * rtl_linear_backward - from dy and the forward pass's x, w, gate and z:
 *
 *   dz = gate * dy * act'(z),  dx = dz w,  dw = dz^T x,
 *   dbias = sum over rows of dz,  dgate = sum over a gate row's rows of dy act(z)
 *
 * (The residual's gradient is dy.)  dx [M, K], dw [N, K], dbias [N], dgate
 * [gate_rows, N] densely packed; each may be NULL.  z is needed with an activation
 * or for dgate, x for dw, w for dx.  dz is rounded to the tensors' type before the two
 * products, not before dbias, and its rows are N rounded up to 8 long (below 2 GiB so
 * too).  Sums have an order that only the sizes fix.
 * With M == 0 dw, dbias and dgate are zeros.
 */
size_t rtl_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t gate_rows);

rtl_status rtl_linear_backward(const void* dy, const void* x, const void* w, const void* z, const void* gate,
                               int64_t gate_rows, int64_t gate_stride, int64_t M, int64_t N, int64_t K, void* dx,
                               void* dw, void* dbias, void* dgate, void* workspace, size_t workspace_bytes,
                               uint32_t flags, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* RTLYNX_DENSE_H */
