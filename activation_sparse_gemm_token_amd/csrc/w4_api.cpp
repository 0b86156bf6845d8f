// Host side of include/rtlynx_w4.h: argument checks, then one launch.
#include "rtl_api.hpp"
#include "rtl_operators.hpp"
#include "rtlynx_w4.h"

namespace {

constexpr int64_t kMaxN = (int64_t)1 << 31;
// 64 rows of x are addressed with 32-bit offsets.
constexpr int64_t kMaxK = RTL_W4_MAX_CHANNELS;

bool weight_ok(int64_t N, int64_t K, int64_t group) {
  return N >= 1 && N < kMaxN && K >= 1 && K <= kMaxK && (group == 32 || group == 64 || group == 128) &&
         K % group == 0;
}

size_t packed_size(int64_t N, int64_t K, int64_t group, bool zeros) {
  return (size_t)rtl::w4_tiles(N, K) * (1024 + 16 * (size_t)(128 / group) * (zeros ? 4 : 2));
}

}  // namespace

RTL_API size_t rtl_w4_packed_bytes(int64_t N, int64_t K, int64_t group, uint32_t flags) {
  if (!weight_ok(N, K, group) || (flags & ~RTL_W4_ZEROS) != 0) return 0;
  return packed_size(N, K, group, (flags & RTL_W4_ZEROS) != 0);
}

RTL_API rtl_status rtl_w4_pack(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t N,
                               int64_t K, int64_t group, uint32_t flags, void* packed, size_t packed_bytes,
                               void* hip_stream) {
  if ((flags & ~RTL_W4_ZEROS) != 0) return RTL_ERR_BAD_FLAGS;
  if (!weight_ok(N, K, group)) return RTL_ERR_BAD_SHAPE;
  const bool z = (flags & RTL_W4_ZEROS) != 0;
  if (codes == nullptr || scales == nullptr || packed == nullptr || (z && zeros == nullptr))
    return RTL_ERR_NULL_POINTER;
  if (!rtl::aligned(codes, 16) || !rtl::aligned(scales, 16) || !rtl::aligned(packed, 16) ||
      (z && !rtl::aligned(zeros, 16)))
    return RTL_ERR_MISALIGNED;
  if (packed_bytes < packed_size(N, K, group, z)) return RTL_ERR_WORKSPACE;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  const rtl_status d = rtl::check_device(stream);
  if (d != RTL_OK) return d;
  return rtl::from_hip(rtl::launch_w4_pack(codes, scales, z ? zeros : nullptr, N, K, (int)group, packed, stream));
}

RTL_API rtl_status rtl_w4_linear(const uint16_t* x, const void* packed, size_t packed_bytes, int64_t M, int64_t N,
                                 int64_t K, int64_t group, uint32_t flags, uint16_t* y, void* hip_stream) {
  if ((flags & ~RTL_W4_ZEROS) != 0) return RTL_ERR_BAD_FLAGS;
  if (!weight_ok(N, K, group) || M < 0 || M > RTL_W4_MAX_ROWS) return RTL_ERR_BAD_SHAPE;
  if (M == 0) return RTL_OK;
  if (x == nullptr || packed == nullptr || y == nullptr) return RTL_ERR_NULL_POINTER;
  if (!rtl::aligned(x, 16) || !rtl::aligned(packed, 16) || !rtl::aligned(y, 16)) return RTL_ERR_MISALIGNED;
  const bool z = (flags & RTL_W4_ZEROS) != 0;
  if (packed_bytes < packed_size(N, K, group, z)) return RTL_ERR_WORKSPACE;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  const rtl_status d = rtl::check_device(stream);
  if (d != RTL_OK) return d;
  return rtl::from_hip(rtl::launch_w4_linear(x, packed, M, N, K, (int)group, z, y, stream));
}
