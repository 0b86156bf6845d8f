/*
 * rtlynx_w4.h - linear layers of few rows with 4-bit weights and group scales.
 *
 *   y[m, n] = sum_k x[m, k] * (q[n, k] - z[n, k / group]) * s[n, k / group]
 *
 * The layers of a model that see one row per image or a few rows per prompt
 * (time embedding, modulation, short prompts) are weight traffic and nothing
 * else; beside rtl_sparse_linear, which serves thousands of tokens, these
 * entry points serve 1 to 32 rows at a quarter of the bf16 weights' bytes, and up
 * to 64 where N is above 8192.  More rows are accepted: the weights are read once per
 * 64 of them, or once per 32 where N <= 8192 and tiles of 64 x 64 would be fewer
 * than 256.
 *
 * q is 0..15, z the group's zero point (8 for every group when a weight has
 * none), s a bf16 scale.  Products are formed in fp32 from exact operands:
 * the matrix cores multiply the bf16 activations with 1 + q / 16, which bf16
 * holds exactly, and each group's share of the ones and of its zero point is
 * taken off with the group's sum of x; sums are fp32 and y is rounded once.
 * x must be finite: a row with an infinity or NaN gives NaN.  So does one whose
 * magnitudes, summed over a group, or a scale's sixteenfold pass fp32's range.
 *
 * Conventions are those of rtlynx.h; x, y, codes, scales, zeros and the packed
 * weight may pass 2 GiB.
 */
#ifndef RTLYNX_W4_H
#define RTLYNX_W4_H

#include "rtlynx.h"

#ifdef __cplusplus
extern "C" {
#endif

/* flags: the weight has zero points. */
#define RTL_W4_ZEROS 0x1u

/* Most rows of one call, and channels of a weight. */
#define RTL_W4_MAX_ROWS (1 << 20)
#define RTL_W4_MAX_CHANNELS (1 << 22)

/*
 * rtl_w4_packed_bytes - size of the packed form of a weight [N, K].  Returns 0
 * for invalid sizes (N < 1, K < 1, K > RTL_W4_MAX_CHANNELS, group not 32, 64 or
 * 128, K % group != 0) or unknown flags.
 */
size_t rtl_w4_packed_bytes(int64_t N, int64_t K, int64_t group, uint32_t flags);

/*
 * rtl_w4_pack - lays a weight out for rtl_w4_linear, once when it is loaded.
 *
 *   codes   [N, K / 2] uint8: channel 2i in the low half of byte i, 2i + 1 in
 *           the high half.
 *   scales  [N, K / group] bf16.
 *   zeros   [N, K / group] uint8, 0..15 (the low 4 bits are used); required
 *           with RTL_W4_ZEROS, ignored without.
 *   packed  rtl_w4_packed_bytes(N, K, group, flags) bytes, 16-byte aligned:
 *           16 rows x 128 channels per KiB in the order of the matrix-core operands, then
 *           the scales (and zero points) in the same order.
 */
rtl_status rtl_w4_pack(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros,
                       int64_t N, int64_t K, int64_t group, uint32_t flags,
                       void* packed, size_t packed_bytes, void* hip_stream);

/*
 * rtl_w4_linear - y [M, N] bf16 from x [M, K] bf16 and a packed weight (N, K,
 * group and flags as it was packed with).  M == 0 is a no-op;
 * M <= RTL_W4_MAX_ROWS.  A packed buffer that is too small gives
 * RTL_ERR_WORKSPACE.  The order of the sums depends on the sizes only.
 */
rtl_status rtl_w4_linear(const uint16_t* x, const void* packed, size_t packed_bytes,
                         int64_t M, int64_t N, int64_t K, int64_t group, uint32_t flags,
                         uint16_t* y, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* RTLYNX_W4_H */
