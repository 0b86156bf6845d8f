/*
 * rtlynx_train.h - training the LoRA branch of the sparse layer: the layer's
 * input kept in 8 bits, and the backward pass that reads it.
 *
 * The forward pass is rtl_sparse_linear (per-token compensation, LoRA on the
 * pruned residual):
 *
 *   Y = s (M * X) W^T + alpha R A^T B^T,   R = X - s (M * X),
 *   s = L1(X) / L1(M * X) per token (1 where that is 0 / 0)
 *
 * with M the 0/1 pattern of the kept channels.  W is frozen; A and B learn.
 * Beside X's checkpoint the backward pass needs nothing from the forward.  It is the
 * default layer's only: the variants of rtl_sparse_linear_prepare_variant and the
 * dense product have no backward here.
 *
 * Conventions are those of rtlynx.h (bf16 tensors as raw words, 16-byte
 * aligned bases, each tensor below 2 GiB counting 256 rows past its end, K a
 * multiple of 4).
 */
#ifndef RTLYNX_TRAIN_H
#define RTLYNX_TRAIN_H

#include "rtlynx.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Channels that share one exponent. */
#define RTL_CKPT_BLOCK 32

/*
 * rtl_checkpoint_pack - the input of a sparse layer in 8 bits.
 *
 *   x      [M, K] bf16, finite, a token's L1 norm within fp32's range (past it s is
 *          NaN, as the layer's is).
 *   codes  [M, K] int8 and exps [M, ceil(K / 32)] uint8: x is stored as
 *          code * 2^(exp - 133), exp the biased exponent of the block's
 *          largest magnitude (so the largest code is 64 .. 127) and code the
 *          nearest integer, ties to even, clamped to +-127.  A power of two as
 *          the step makes every stored value exact in bf16; the error is at most
 *          half a step, 2^-7 of the block's largest magnitude.
 *   idx    [M, ceil(K / 8)] uint8: the kept channels of every group of 4, in
 *          the format of rtl_sparsify_2of4 (bit-exact with it).
 *   stats  [M, 2] fp32: s, and the L1 norm of the kept channels, of x itself.
 *
 * 1.16 bytes per channel instead of 2.  M == 0 is a no-op.
 *
 * One step for a block suits activations of one scale.  Where a few channels are
 * far larger than the rest, the small ones, which are the pruned ones that the
 * LoRA branch learns from, fall below half a step and become code 0: on the
 * diffusion-transformer law of 8 % large channels 56 % of the pruned channels, and
 * the gradients formed from the checkpoint differ from those of X by 17 % (dA, dB)
 * and 9 % (dX; 74 % on its pruned channels, where a zero code has no sign).  With
 * Gaussian and GELU activations dA is off by 1.3 and 2.8 %, dX by 0.6 and 1.3 %.
 * rtl_checkpoint_pack_fine is made for that: 1.9 % and 0.2 % on the same law, 0.7
 * and 1.0 %, 0.03 and 0.06 % on the others.  (All in the 2-norm, 512 x 1024 x 1024,
 * r = 16.)
 */
rtl_status rtl_checkpoint_pack(const uint16_t* x, int64_t M, int64_t K, int8_t* codes, uint8_t* exps,
                               uint8_t* idx, float* stats, void* hip_stream);

/*
 * rtl_checkpoint_pack_fine - the same with a step of their own for a block's pruned
 * channels (1.19 bytes per channel).
 *
 *   exps         [M, ceil(K / 32)]: of the kept channels, as above (the largest
 *                magnitude of a block is always kept), and so are their codes.
 *   pruned_exps  [M, ceil(K / 32)] uint8: the biased exponent of the largest pruned
 *                magnitude.  A pruned channel is code * 2^(pruned_exp - 133); the code
 *                is rounded as above, but is 1 or -1 where a nonzero value would
 *                round to 0, so its sign is kept: dX's last term is sign(X).  The error
 *                is at most half a step, or less than one step there.
 *
 * For rtl_checkpoint_unpack_fine and rtl_sparse_linear_backward_fine, which otherwise
 * are what their namesakes are.
 */
rtl_status rtl_checkpoint_pack_fine(const uint16_t* x, int64_t M, int64_t K, int8_t* codes, uint8_t* exps,
                                    uint8_t* pruned_exps, uint8_t* idx, float* stats, void* hip_stream);

/* rtl_checkpoint_unpack - y [M, K] bf16: the values that codes and exps stand
 * for (exact). */
rtl_status rtl_checkpoint_unpack(const int8_t* codes, const uint8_t* exps, int64_t M, int64_t K,
                                 uint16_t* y, void* hip_stream);
rtl_status rtl_checkpoint_unpack_fine(const int8_t* codes, const uint8_t* exps, const uint8_t* pruned_exps,
                                      const uint8_t* idx, int64_t M, int64_t K, uint16_t* y, void* hip_stream);

/* Device workspace of rtl_sparse_linear_backward; 0 for invalid sizes and for
 * M == 0. */
size_t rtl_sparse_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t r);

/*
 * rtl_sparse_linear_backward_form - which kernels a call of these sizes takes, for
 * tests and for reading profiles (host only; the form depends on the sizes alone):
 *
 *   form[0]  tile columns of G W: 256 or 192, or 64 for the form of few tokens.
 *   form[1]  ranges of its contraction over N.
 *   form[2]  length of G's rows there: N, or N + 4 for padded copies.
 *   form[3], form[4]  channels of a range of G B, and of the checkpoint by A^T.
 *   form[5]  tokens of a range of the products over tokens.
 *
 * RTL_ERR_BAD_SHAPE for the sizes that rtl_sparse_linear_backward refuses.
 */
rtl_status rtl_sparse_linear_backward_form(int64_t M, int64_t N, int64_t K, int64_t r, int64_t form[6]);

/*
 * rtl_sparse_linear_backward - gradients of the layer from G = dL / dY.
 *
 * With X, M, s, Lk = L1 of the kept channels as the checkpoint holds them:
 *
 *   U  = alpha G B                      [M, r]
 *   E  = G W - U A                      gradient at s (M * X)
 *   D  = sum over kept channels of X E  gradient at s
 *   dX = U A + s (M * E) + (D / Lk) sign(X) (1 - s M)     (last term 0 if Lk is 0)
 *   dA = U^T R                          [r, K]
 *   dB = alpha G^T (R A^T)              [N, r]
 *
 *   g        [M, N] bf16, finite: an infinity or NaN makes its token's row of dX, all of
 *            dA and its channel's row of dB not finite, and leaves the rest as it is.
 *   codes, exps, idx, stats: as rtl_checkpoint_pack wrote them.
 *   w_t      [K, N] bf16, the frozen weight transposed (laid out once: it does
 *            not change in training).  Needed for dx only.
 *   lora_a   [r, K], lora_b [N, r] bf16; ignored when r == 0.
 *   dx       [M, K] bf16 or NULL (a first layer's input needs no gradient).
 *   da, db   [r, K], [N, r] bf16, both or neither; required NULL when r == 0.
 *   workspace  rtl_sparse_linear_backward_workspace_bytes(M, N, K, r) bytes,
 *            16-byte aligned, overwritten.
 *
 * N % 4 == 0 (N >= 4), K % 4 == 0, 0 <= r <= RTL_MAX_LORA_RANK.  Products have bf16
 * operands and fp32 sums; U, R A^T, G W and all sums are carried between them
 * in fp32 (U and R A^T enter their second product as three bf16 words, 24 bits);
 * each result is rounded once.  M == 0 writes zeros to da and db.  Deterministic: the order of every
 * sum depends on the sizes only.
 */
rtl_status rtl_sparse_linear_backward(const uint16_t* g, const int8_t* codes, const uint8_t* exps,
                                      const uint8_t* idx, const float* stats, const uint16_t* w_t,
                                      const uint16_t* lora_a, const uint16_t* lora_b, int64_t M,
                                      int64_t N, int64_t K, int64_t r, float lora_scale,
                                      uint16_t* dx, uint16_t* da, uint16_t* db, void* workspace,
                                      size_t workspace_bytes, void* hip_stream);
rtl_status rtl_sparse_linear_backward_fine(const uint16_t* g, const int8_t* codes, const uint8_t* exps,
                                           const uint8_t* pruned_exps, const uint8_t* idx,
                                           const float* stats, const uint16_t* w_t, const uint16_t* lora_a,
                                           const uint16_t* lora_b, int64_t M, int64_t N, int64_t K, int64_t r,
                                           float lora_scale, uint16_t* dx, uint16_t* da, uint16_t* db,
                                           void* workspace, size_t workspace_bytes, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* RTLYNX_TRAIN_H */
