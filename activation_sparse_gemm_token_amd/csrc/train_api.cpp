// Host side of include/rtlynx_train.h: argument checks, the backward pass's
// sizes, launches.
#include "rtl_api.hpp"
#include "rtl_common.hpp"
#include "rtl_operators.hpp"
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

// Splits by sizes alone (a workspace must fit whatever device it is used on).
// Two workgroups of these kernels fit a CU, so the split sizes aim at all of
// them running at once: 256 over G's channels and 256 over the checkpoint's, in
// one launch, and 512 over tokens; a range is a whole number of steps of the
// workgroup's four wavefronts.  (4096 x 3072 x 12288 and 4096 x 12288 x 3072,
// r = 64: 38 and 47 us; 384 and 512 workgroups took 41 and 51, 512 and 512 the
// same, 256 and 192 44 and 73.)
rtl::BackwardLayout rtl::backward_layout(int64_t M, int64_t N, int64_t K, int64_t r) {
  constexpr int64_t kCus = 256;
  BackwardLayout L{};
  L.M = M; L.N = N; L.K = K; L.r = r;
  L.rp = r == 0 ? 0 : r <= 32 ? 32 : r <= 64 ? 64 : 128;
  L.np = round_up(N, 64);
  L.kp = round_up(K, 64);
  L.mp = round_up(M, 64);
  // `length` in as many ranges as `groups` workgroups make of `blocks` blocks.
  auto chunk = [](int64_t length, int64_t groups, int64_t blocks, int64_t step) {
    const int64_t splits = blocks > 0 && groups > blocks ? groups / blocks : 1;
    return length > 0 ? round_up((length + splits - 1) / splits, step) : step;
  };
  const int64_t rows_g = L.rp == 128 ? 32 : 64, rows_x = rows_g / 2;    // tokens per workgroup
  L.chunk_g = chunk(L.np, kCus, (M + rows_g - 1) / rows_g, 256);
  L.splits_g = (L.np + L.chunk_g - 1) / L.chunk_g;
  L.chunk_x = chunk(L.kp, kCus, (M + rows_x - 1) / rows_x, 256);
  L.splits_x = (L.kp + L.chunk_x - 1) / L.chunk_x;
  const int64_t cols_g = L.rp == 128 ? 64 : 128, cols_x = cols_g / 2;   // channels per workgroup
  // Tiles of 64 channels (ranks above 64) are more uneven a load per CU than those
  // of 128, and gain from more and shorter ranges: 864 workgroups instead of 288
  // took 63 us instead of 83 (r = 128); at r = 64 512 were best.
  L.chunk_t = chunk(L.mp, L.rp == 128 ? 7 * kCus / 2 : 2 * kCus, (N + cols_g - 1) / cols_g + (K + cols_x - 1) / cols_x, 128);
  L.splits_t = (L.mp + L.chunk_t - 1) / L.chunk_t;
  // G W: tile columns and contraction ranges by the time they should take, in
  // us.  With 256 and 192 columns a k-step of 64 measured 1.65 and 1.25 with the
  // chip full, plus 8 per tile.  With 64 (few_tokens_kernel) a workgroup's four
  // wavefronts take a step each, 1.7 per workgroup on a CU (2.2 with N % 8 == 4,
  // two loads instead of one), plus 3 once.  Then writing and reading the ranges'
  // results, 0.6 each at the least, and the wide tiles' padded copies of G and W
  // where N % 8 == 4.
  //   77 x 520 x 264:      5.0 us with 64 columns, 12.4 otherwise;
  //   16 x 1024 x 4096:    6.2, 13.3;   2000 x 512 x 512: 8.8, 19.4;
  //   256 x 3072 x 3072:   27.6, 24.4 (with dX 34.0, 33.2);
  //   512 x 3072 x 12288:  144, 48.
  const int64_t tiles_m = (M + 255) / 256, steps = (N + 63) / 64;
  double best = 0;
  for (int64_t tn : {256, 192, 64}) {
    const bool pad = tn != 64 && N % 8 != 0;
    if (pad && !(size_ok(M, N + 4) && size_ok(K, N + 4))) continue;
    const int64_t tiles = (K + tn - 1) / tn, least = tn == 64 ? 4 : 2;
    for (int64_t s = 1; s <= 16 && (s == 1 || steps / s >= least); ++s) {
      const int64_t per = (steps + s - 1) / s;
      if (s > 1 && (s - 1) * per >= steps) continue;                    // the last range would be empty
      const int64_t groups = (tn == 64 ? (M + 63) / 64 : tiles_m) * tiles * s, rounds = (groups + kCus - 1) / kCus;
      const double each = tn == 64 ? (double)((per + 3) / 4) * (N % 8 == 0 ? 1.7 : 2.2)
                                   : (double)per * (tn == 256 ? 1.65 : 1.25) + 8;
      const double t = (double)rounds * each + (tn == 64 ? 3 : 0) + (pad ? 3 + (double)((M + K) * N) * 4 / 5e6 : 0) +
                       0.6 * (double)(s - 1) + (double)s * (double)M * (double)L.kp * 8 / 5e6;
      if (best == 0 || t < best) {
        best = t;
        L.p_tile = tn;
        L.p_tiles = tiles;
        L.p_splits = s;
        L.p_length = pad ? N + 4 : N;
      }
    }
  }
  size_t o = 0;
  auto take = [&](int64_t bytes) { const size_t at = o; o += ((size_t)bytes + 255) / 256 * 256; return at; };
  L.off_a_down = take(L.rp * L.kp * 2);
  L.off_a_up = take(L.rp * L.kp * 2);
  L.off_b = take(L.rp * L.np * 2);
  L.off_u = take(2 * L.rp * L.mp * 2);
  L.off_uc = take(4 * L.rp * L.mp * 2);
  L.off_tc = take(2 * L.rp * L.mp * 2);
  L.off_d = take(L.mp * 4);
  const int64_t rows = (L.splits_g + 2 * L.splits_x) * M * L.rp * 4;
  const int64_t over_t = L.splits_t * (N + L.kp) * L.rp * 4;
  L.off_part = take(rows > over_t ? rows : over_t);
  L.off_p = take(L.p_splits * round_up(M, 16) * L.kp * 4);
  L.off_d_part = take(L.p_splits * L.p_tiles * M * 4);
  if (L.p_length != N) L.off_pad = take((M + K) * L.p_length * 2);
  L.total = o;
  return L;
}

namespace {

// pruned_exps: NULL for one exponent per block (`fine` says which is meant).
rtl_status pack(const uint16_t* x, int64_t M, int64_t K, int8_t* codes, uint8_t* exps, uint8_t* pruned_exps,
                uint8_t* idx, float* stats, bool fine, void* hip_stream) {
  if (!act_ok(M, K)) return RTL_ERR_BAD_SHAPE;
  if (M == 0) return RTL_OK;
  if (x == nullptr || codes == nullptr || exps == nullptr || idx == nullptr || stats == nullptr ||
      (fine && pruned_exps == nullptr))
    return RTL_ERR_NULL_POINTER;
  if (!rtl::aligned(x, 16) || !rtl::aligned(codes, 16) || !rtl::aligned(exps, 16) || !rtl::aligned(idx, 16) ||
      !rtl::aligned(stats, 16) || !rtl::aligned(pruned_exps, 16))
    return RTL_ERR_MISALIGNED;
  int cus = 0;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  const rtl_status d = rtl::check_device(stream, &cus);
  if (d != RTL_OK) return d;
  return rtl::from_hip(rtl::launch_checkpoint_pack(x, M, K, codes, exps, pruned_exps, idx, stats, cus, stream));
}

// pruned_exps and idx: NULL for one exponent per block.
rtl_status unpack(const int8_t* codes, const uint8_t* exps, const uint8_t* pruned_exps, const uint8_t* idx, int64_t M,
                  int64_t K, uint16_t* y, bool fine, void* hip_stream) {
  if (!act_ok(M, K)) return RTL_ERR_BAD_SHAPE;
  if (M == 0) return RTL_OK;
  if (codes == nullptr || exps == nullptr || y == nullptr || (fine && (pruned_exps == nullptr || idx == nullptr)))
    return RTL_ERR_NULL_POINTER;
  if (!rtl::aligned(codes, 16) || !rtl::aligned(exps, 16) || !rtl::aligned(y, 16) || !rtl::aligned(pruned_exps, 16) ||
      !rtl::aligned(idx, 16))
    return RTL_ERR_MISALIGNED;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  const rtl_status d = rtl::check_device(stream);
  if (d != RTL_OK) return d;
  return rtl::from_hip(rtl::launch_checkpoint_unpack(codes, exps, pruned_exps, idx, M, K, y, stream));
}

}  // namespace

RTL_API rtl_status rtl_checkpoint_pack(const uint16_t* x, int64_t M, int64_t K, int8_t* codes, uint8_t* exps,
                                       uint8_t* idx, float* stats, void* hip_stream) {
  return pack(x, M, K, codes, exps, nullptr, idx, stats, false, hip_stream);
}

RTL_API rtl_status rtl_checkpoint_pack_fine(const uint16_t* x, int64_t M, int64_t K, int8_t* codes, uint8_t* exps,
                                            uint8_t* pruned_exps, uint8_t* idx, float* stats, void* hip_stream) {
  return pack(x, M, K, codes, exps, pruned_exps, idx, stats, true, hip_stream);
}

RTL_API rtl_status rtl_checkpoint_unpack(const int8_t* codes, const uint8_t* exps, int64_t M, int64_t K, uint16_t* y,
                                         void* hip_stream) {
  return unpack(codes, exps, nullptr, nullptr, M, K, y, false, hip_stream);
}

RTL_API rtl_status rtl_checkpoint_unpack_fine(const int8_t* codes, const uint8_t* exps, const uint8_t* pruned_exps,
                                              const uint8_t* idx, int64_t M, int64_t K, uint16_t* y, void* hip_stream) {
  return unpack(codes, exps, pruned_exps, idx, M, K, y, true, hip_stream);
}

RTL_API size_t rtl_sparse_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t r) {
  if (!back_ok(M, N, K, r) || M == 0) return 0;
  return rtl::backward_layout(M, N, K, r).total;
}

RTL_API rtl_status rtl_sparse_linear_backward_form(int64_t M, int64_t N, int64_t K, int64_t r, int64_t form[6]) {
  if (form == nullptr) return RTL_ERR_NULL_POINTER;
  if (!back_ok(M, N, K, r)) return RTL_ERR_BAD_SHAPE;
  const rtl::BackwardLayout L = rtl::backward_layout(M, N, K, r);
  const int64_t f[6] = {L.p_tile, L.p_splits, L.p_length, L.chunk_g, L.chunk_x, L.chunk_t};
  for (int i = 0; i < 6; ++i) form[i] = f[i];
  return RTL_OK;
}

namespace {

rtl_status backward(const uint16_t* g, const rtl::Ckpt& ck, const uint16_t* w_t, const uint16_t* lora_a,
                    const uint16_t* lora_b, int64_t M, int64_t N, int64_t K, int64_t r, float lora_scale, uint16_t* dx,
                    uint16_t* da, uint16_t* db, void* workspace, size_t workspace_bytes, void* hip_stream) {
  if (!back_ok(M, N, K, r)) return RTL_ERR_BAD_SHAPE;
  if ((da == nullptr) != (db == nullptr)) return RTL_ERR_NULL_POINTER;
  if (r == 0 && da != nullptr) return RTL_ERR_BAD_SHAPE;
  if (dx == nullptr && da == nullptr) return RTL_OK;
  if (M == 0 && da == nullptr) return RTL_OK;
  if (!rtl::aligned(dx, 16) || !rtl::aligned(da, 16) || !rtl::aligned(db, 16)) return RTL_ERR_MISALIGNED;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  const rtl::BackwardLayout L = rtl::backward_layout(M, N, K, r);
  if (M > 0) {
    if (g == nullptr || ck.codes == nullptr || ck.exps == nullptr || ck.pruned_exps == nullptr || ck.idx == nullptr ||
        ck.stats == nullptr ||
        (dx != nullptr && w_t == nullptr) || (r > 0 && (lora_a == nullptr || lora_b == nullptr)))
      return RTL_ERR_NULL_POINTER;
    if (!rtl::aligned(g, 16) || !rtl::aligned(ck.codes, 16) || !rtl::aligned(ck.exps, 16) ||
        !rtl::aligned(ck.pruned_exps, 16) || !rtl::aligned(ck.idx, 16) || !rtl::aligned(ck.stats, 16) || (dx != nullptr && !rtl::aligned(w_t, 16)) ||
        (r > 0 && (!rtl::aligned(lora_a, 16) || !rtl::aligned(lora_b, 16))))
      return RTL_ERR_MISALIGNED;
    if (workspace == nullptr || workspace_bytes < L.total) return RTL_ERR_WORKSPACE;
    if (!rtl::aligned(workspace, 16)) return RTL_ERR_MISALIGNED;
  }
  const rtl_status d = rtl::check_device(stream);
  if (d != RTL_OK) return d;
  return rtl::from_hip(rtl::launch_backward(g, ck, w_t, lora_a, lora_b, L, lora_scale, dx, da, db,
                                            static_cast<char*>(workspace), stream));
}

}  // namespace

RTL_API rtl_status rtl_sparse_linear_backward(const uint16_t* g, const int8_t* codes, const uint8_t* exps,
                                              const uint8_t* idx, const float* stats, const uint16_t* w_t,
                                              const uint16_t* lora_a, const uint16_t* lora_b, int64_t M, int64_t N,
                                              int64_t K, int64_t r, float lora_scale, uint16_t* dx, uint16_t* da,
                                              uint16_t* db, void* workspace, size_t workspace_bytes,
                                              void* hip_stream) {
  return backward(g, {codes, exps, exps, idx, stats}, w_t, lora_a, lora_b, M, N, K, r, lora_scale, dx, da, db, workspace,
                  workspace_bytes, hip_stream);
}

RTL_API rtl_status rtl_sparse_linear_backward_fine(const uint16_t* g, const int8_t* codes, const uint8_t* exps,
                                                   const uint8_t* pruned_exps, const uint8_t* idx, const float* stats,
                                                   const uint16_t* w_t, const uint16_t* lora_a, const uint16_t* lora_b,
                                                   int64_t M, int64_t N, int64_t K, int64_t r, float lora_scale,
                                                   uint16_t* dx, uint16_t* da, uint16_t* db, void* workspace,
                                                   size_t workspace_bytes, void* hip_stream) {
  return backward(g, {codes, exps, pruned_exps, idx, stats}, w_t, lora_a, lora_b, M, N, K, r, lora_scale, dx, da, db,
                  workspace, workspace_bytes, hip_stream);
}
