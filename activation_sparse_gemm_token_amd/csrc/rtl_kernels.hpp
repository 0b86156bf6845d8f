// Launch wrappers of librtlynx's kernels (internal; the public interface is
// include/rtlynx.h).  Each returns the status of its own launches (the
// first that failed), never the thread's earlier error.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rtl {

// compute_units: the device's CU count (one or two wavefronts per row).
hipError_t launch_sparsify_2of4(const uint16_t* x, int64_t M, int64_t K, uint16_t* vals,
                                uint8_t* idx, float* scale, bool fold, int compute_units,
                                hipStream_t stream);

// Pre-pass of the fused path: selection, compression into the structured-
// sparse matrix-core operand order, per-token scale, LoRA-down product.
hipError_t launch_prepass(const uint16_t* x, const uint16_t* lora_a, int64_t M, int64_t K,
                          int64_t r, float lora_scale, void* workspace, hipStream_t stream,
                          int comp = 0, int lora = 0);

// Sparse GEMM on the compressed operand plus the scale and LoRA-up epilogue.
// `compute_units`: the device's CU count (the persistent grid's size).
// tile_n: 256 or 192 output columns per tile, 0 to let
// sparse_gemm_tile_n choose (the one that fills the CUs at lower cost).
// prefetch_w: probe W lines into L2 a few steps ahead of their copies (for
// weights not expected in the caches; the ring shapes, r % 8 == 0 and
// K % 8 == 0, only).
hipError_t launch_sparse_gemm(const void* workspace, const uint16_t* w, const uint16_t* lora_b,
                              int64_t M, int64_t N, int64_t K, int64_t r, uint16_t* y,
                              int compute_units, hipStream_t stream, int tile_n = 0,
                              bool prefetch_w = false);
int sparse_gemm_tile_n(int64_t M, int64_t N, int64_t K, int compute_units);

hipError_t launch_dense_gemm(const uint16_t* x, const uint16_t* w, int64_t M, int64_t N,
                             int64_t K, uint16_t* y, hipStream_t stream);

// The same product with an fp32 result.
hipError_t launch_dense_gemm_f32(const uint16_t* x, const uint16_t* w, int64_t M, int64_t N, int64_t K,
                                 float* y, hipStream_t stream);

// Canonical compressed activation (vals, idx, scale or null) into the
// workspace regions of ws_layout(M, K, 0).
hipError_t launch_repack(const uint16_t* vals, const uint8_t* idx, const float* scale, int64_t M,
                         int64_t K, void* workspace, hipStream_t stream);

// Rotary positions.  One tensor [batch, tokens, heads, dim] and its result
// (strides in elements); heads == 0 for an absent second tensor.
struct RopeSide {
  const void* x;
  void* y;
  int64_t xb, xt, xh, yb, yt, yh;
  int heads;
  bool in_place;                         // y is x: copied channels need no copy
};
struct RopeArgs {
  RopeSide t[2];
  const int64_t* positions;
  const double* inv_freq;
  int64_t total, tokens;                 // batch * tokens, tokens
  int64_t pos_b, pos_t;
  int dim, rot;
  int axis_end[3];                       // first pair of axes 1, 2 and 3
  float scale;
  bool inverse;
  int group;                             // tokens per workgroup (set by launch_rope)
};
hipError_t launch_rope(RopeArgs a, int elem_bytes, bool fp16, bool interleaved, int compute_units,
                       hipStream_t stream);

// 4-bit weights: tiles of 16 rows x 128 channels (1 KiB of codes each).
inline int64_t w4_tiles(int64_t N, int64_t K) { return ((N + 15) / 16) * ((K + 127) / 128); }
hipError_t launch_w4_pack(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t N,
                          int64_t K, int group, void* packed, hipStream_t stream);
hipError_t launch_w4_linear(const uint16_t* x, const void* packed, int64_t M, int64_t N, int64_t K,
                            int group, bool zeros, uint16_t* y, hipStream_t stream);

// 8-bit activation checkpoint (include/rtlynx_train.h).
struct Ckpt {
  const int8_t* codes;
  const uint8_t* exps;
  const uint8_t* idx;
  const float* stats;
};
hipError_t launch_checkpoint_pack(const uint16_t* x, int64_t M, int64_t K, int8_t* codes, uint8_t* exps,
                                  uint8_t* idx, float* stats, int compute_units, hipStream_t stream);
hipError_t launch_checkpoint_unpack(const int8_t* codes, const uint8_t* exps, int64_t M, int64_t K,
                                    uint16_t* y, hipStream_t stream);

// Sizes, splits and workspace regions of the layer's backward pass.  Rank is
// padded to 32, 64 or 128, channels and tokens to 64 (zeros).
struct BackwardLayout {
  int64_t M, N, K, r;
  int64_t rp, np, kp, mp;
  int64_t row_chunk, row_splits_g, row_splits_x;   // channel ranges of the token-by-rank products
  int64_t col_chunk, col_splits;                   // token ranges of the products over tokens
  size_t off_ap, off_at, off_bt, off_u_rows, off_u_cols, off_t_cols, off_d, off_part, off_p, total;
};
BackwardLayout backward_layout(int64_t M, int64_t N, int64_t K, int64_t r);
hipError_t launch_backward(const uint16_t* g, const Ckpt& ck, const uint16_t* w_t, const uint16_t* lora_a,
                           const uint16_t* lora_b, const BackwardLayout& L, float alpha, uint16_t* dx,
                           uint16_t* da, uint16_t* db, char* workspace, hipStream_t stream);

}  // namespace rtl
