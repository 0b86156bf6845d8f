// Host side of include/rtlynx_train.h: argument checks, the backward pass's
// sizes, launches.
#include "rtl_api.hpp"
#include "rtl_common.hpp"
#include "rtl_kernels.hpp"
#include "rtlynx_train.h"

namespace {

constexpr int64_t kMaxBytes = (int64_t)1 << 31;

// A [rows + 256, cols] bf16 tensor below 2 GiB (rows and cols >= 0).
bool size_ok(int64_t rows, int64_t cols) {
  return rows < kMaxBytes && cols < kMaxBytes && (cols == 0 || rows + 256 < kMaxBytes / (2 * cols));
}

bool act_ok(int64_t M, int64_t K) { return M >= 0 && K >= 4 && K % 4 == 0 && size_ok(M, K); }

bool back_ok(int64_t M, int64_t N, int64_t K, int64_t r) {
  return act_ok(M, K) && act_ok(M, N) && size_ok(K, N) && size_ok(N, K) && r >= 0 && r <= RTL_MAX_LORA_RANK;
}

}  // namespace

// Splits: about 768 workgroups for the token-by-rank products and 512 for
// those over tokens (two to three per CU), no finer than two steps each.
rtl::BackwardLayout rtl::backward_layout(int64_t M, int64_t N, int64_t K, int64_t r) {
  BackwardLayout L{};
  L.M = M; L.N = N; L.K = K; L.r = r;
  L.rp = r == 0 ? 0 : r <= 32 ? 32 : r <= 64 ? 64 : 128;
  L.np = round_up(N, 64);
  L.kp = round_up(K, 64);
  L.mp = round_up(M, 64);
  const int64_t row_blocks = (M + 127) / 128;
  int64_t chunk = row_blocks * (L.np + L.kp) / 768;
  L.row_chunk = chunk < 128 ? 128 : round_up(chunk, 64);
  L.row_splits_g = (L.np + L.row_chunk - 1) / L.row_chunk;
  L.row_splits_x = (L.kp + L.row_chunk - 1) / L.row_chunk;
  const int64_t col_blocks = (N + 127) / 128 + (K + 127) / 128;
  chunk = col_blocks * L.mp / 512;
  L.col_chunk = chunk < 128 ? 128 : round_up(chunk, 64);
  L.col_splits = (L.mp + L.col_chunk - 1) / L.col_chunk;
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o += (bytes + 255) / 256 * 256; return at; };
  L.off_ap = take((size_t)(L.rp * L.kp) * 2);
  L.off_at = take((size_t)(L.rp * L.kp) * 2);
  L.off_bt = take((size_t)(L.rp * L.np) * 2);
  L.off_u_rows = take((size_t)(2 * L.rp * M) * 2);
  L.off_u_cols = take((size_t)(4 * L.rp * L.mp) * 2);
  L.off_t_cols = take((size_t)(2 * L.rp * L.mp) * 2);
  L.off_d = take((size_t)M * 4);
  const size_t rows = (size_t)((L.row_splits_g + 2 * L.row_splits_x) * M * L.rp) * 4;
  const size_t cols = (size_t)(L.col_splits * (N + L.kp) * L.rp) * 4;
  L.off_part = take(rows > cols ? rows : cols);
  L.off_p = take((size_t)(M * K) * 4);
  L.total = o;
  return L;
}

RTL_API rtl_status rtl_checkpoint_pack(const uint16_t* x, int64_t M, int64_t K, int8_t* codes, uint8_t* exps,
                                       uint8_t* idx, float* stats, void* hip_stream) {
  if (!act_ok(M, K)) return RTL_ERR_BAD_SHAPE;
  if (M == 0) return RTL_OK;
  if (x == nullptr || codes == nullptr || exps == nullptr || idx == nullptr || stats == nullptr)
    return RTL_ERR_NULL_POINTER;
  if (!rtl::aligned(x, 16) || !rtl::aligned(codes, 16) || !rtl::aligned(exps, 16) || !rtl::aligned(idx, 16) ||
      !rtl::aligned(stats, 16))
    return RTL_ERR_MISALIGNED;
  int cus = 0;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  const rtl_status d = rtl::check_device(stream, &cus);
  if (d != RTL_OK) return d;
  return rtl::from_hip(rtl::launch_checkpoint_pack(x, M, K, codes, exps, idx, stats, cus, stream));
}

RTL_API rtl_status rtl_checkpoint_unpack(const int8_t* codes, const uint8_t* exps, int64_t M, int64_t K, uint16_t* y,
                                         void* hip_stream) {
  if (!act_ok(M, K)) return RTL_ERR_BAD_SHAPE;
  if (M == 0) return RTL_OK;
  if (codes == nullptr || exps == nullptr || y == nullptr) return RTL_ERR_NULL_POINTER;
  if (!rtl::aligned(codes, 16) || !rtl::aligned(exps, 16) || !rtl::aligned(y, 16)) return RTL_ERR_MISALIGNED;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  const rtl_status d = rtl::check_device(stream);
  if (d != RTL_OK) return d;
  return rtl::from_hip(rtl::launch_checkpoint_unpack(codes, exps, M, K, y, stream));
}

RTL_API size_t rtl_sparse_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t r) {
  if (!back_ok(M, N, K, r) || M == 0) return 0;
  return rtl::backward_layout(M, N, K, r).total;
}

RTL_API rtl_status rtl_sparse_linear_backward(const uint16_t* g, const int8_t* codes, const uint8_t* exps,
                                              const uint8_t* idx, const float* stats, const uint16_t* w_t,
                                              const uint16_t* lora_a, const uint16_t* lora_b, int64_t M, int64_t N,
                                              int64_t K, int64_t r, float lora_scale, uint16_t* dx, uint16_t* da,
                                              uint16_t* db, void* workspace, size_t workspace_bytes,
                                              void* hip_stream) {
  if (!back_ok(M, N, K, r)) return RTL_ERR_BAD_SHAPE;
  if ((da == nullptr) != (db == nullptr)) return RTL_ERR_NULL_POINTER;
  if (r == 0 && da != nullptr) return RTL_ERR_BAD_SHAPE;
  if (dx == nullptr && da == nullptr) return RTL_OK;
  if (M == 0 && da == nullptr) return RTL_OK;
  if (!rtl::aligned(dx, 16) || !rtl::aligned(da, 16) || !rtl::aligned(db, 16)) return RTL_ERR_MISALIGNED;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  if (M > 0) {
    if (g == nullptr || codes == nullptr || exps == nullptr || idx == nullptr || stats == nullptr ||
        (dx != nullptr && w_t == nullptr) || (r > 0 && (lora_a == nullptr || lora_b == nullptr)))
      return RTL_ERR_NULL_POINTER;
    if (!rtl::aligned(g, 16) || !rtl::aligned(codes, 16) || !rtl::aligned(exps, 16) || !rtl::aligned(idx, 16) ||
        !rtl::aligned(stats, 16) || (dx != nullptr && !rtl::aligned(w_t, 16)) ||
        (r > 0 && (!rtl::aligned(lora_a, 16) || !rtl::aligned(lora_b, 16))))
      return RTL_ERR_MISALIGNED;
    if (workspace == nullptr || workspace_bytes < rtl::backward_layout(M, N, K, r).total) return RTL_ERR_WORKSPACE;
    if (!rtl::aligned(workspace, 16)) return RTL_ERR_MISALIGNED;
  }
  const rtl_status d = rtl::check_device(stream);
  if (d != RTL_OK) return d;
  const rtl::Ckpt ck{codes, exps, idx, stats};
  return rtl::from_hip(rtl::launch_backward(g, ck, w_t, lora_a, lora_b, rtl::backward_layout(M, N, K, r), lora_scale,
                                            dx, da, db, static_cast<char*>(workspace), stream));
}
