// Launch wrappers of the operators beside the sparse layer: rotary positions,
// 4-bit linears, the activation checkpoint and the layer's backward pass
// (internal; the public interfaces are include/rtlynx_*.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rtl {

// A launch dimension holds less than 2^32 threads: more workgroups than that of up
// to 512 go to z, in rows of 2^22.  folded_block() is the workgroup's number; those
// past the last one have nothing to do.
inline dim3 folded_grid(int64_t blocks, unsigned y = 1) {
  constexpr int64_t kRow = (int64_t)1 << 22;
  return blocks <= kRow ? dim3((unsigned)blocks, y) : dim3((unsigned)kRow, y, (unsigned)((blocks + kRow - 1) / kRow));
}
__device__ __forceinline__ int64_t folded_block() { return (int64_t)blockIdx.z * gridDim.x + blockIdx.x; }

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
  const uint8_t* exps;                   // of the kept channels
  const uint8_t* pruned_exps;            // exps itself where both share one
  const uint8_t* idx;
  const float* stats;
};
// pruned_exps: NULL for one exponent per block.
hipError_t launch_checkpoint_pack(const uint16_t* x, int64_t M, int64_t K, int8_t* codes, uint8_t* exps,
                                  uint8_t* pruned_exps, uint8_t* idx, float* stats, int compute_units,
                                  hipStream_t stream);
hipError_t launch_checkpoint_unpack(const int8_t* codes, const uint8_t* exps, const uint8_t* pruned_exps,
                                    const uint8_t* idx, int64_t M, int64_t K, uint16_t* y, hipStream_t stream);

// Sizes, splits and workspace regions of the layer's backward pass.  Rank is
// padded to 32, 64 or 128, channels and tokens to 64 (zeros).  Operands of the
// matrix cores are kept in fragments of 1 KiB: [lane][8] bf16, lane l holding
// row l % 16 and contraction indices 8 (l / 16) + [0, 8) of a 16 x 32 block.
struct BackwardLayout {
  int64_t M, N, K, r;
  int64_t rp, np, kp, mp;
  int64_t chunk_g, chunk_x;                        // channels per workgroup of the token-by-rank products
  int64_t splits_g, splits_x;
  int64_t chunk_t, splits_t;                       // tokens per workgroup of the products over tokens
  int64_t p_tile, p_tiles, p_splits;               // G W: tile columns, their number, contraction ranges
  int64_t p_length;                                // and the rows' length there: N, or N + 4 for padded copies
  size_t off_a_down, off_a_up, off_b, off_u, off_uc, off_tc, off_d, off_part, off_p, off_d_part, off_pad, total;
};
BackwardLayout backward_layout(int64_t M, int64_t N, int64_t K, int64_t r);
// The backward pass's P = G W on the dense GEMM's ring (dense_gemm.hip): the
// contraction over N in L.p_splits ranges, each an fp32 result in 16 x 16
// blocks, [range][ceil(M / 16)][kp / 16][lane][4], lane l of block t of every
// four holding token l % 16, channels 16 (l / 16) + 4 t + [0, 4) of the 64; and of
// each tile and range the sums of kept x * P over the tile's channels, d_part
// [range][tile][M].  Rows of g and w_t are L.p_length long, a multiple of 8.
hipError_t launch_grad_gemm(const uint16_t* g, const uint16_t* w_t, const Ckpt& ck, const BackwardLayout& L,
                            float* p, float* d_part, hipStream_t stream);
hipError_t launch_backward(const uint16_t* g, const Ckpt& ck, const uint16_t* w_t, const uint16_t* lora_a,
                           const uint16_t* lora_b, const BackwardLayout& L, float alpha, uint16_t* dx,
                           uint16_t* da, uint16_t* db, char* workspace, hipStream_t stream);

}  // namespace rtl
