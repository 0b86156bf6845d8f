// Host side of include/rtlynx_dense.h: argument checks, then the launches.
#include "rtl_api.hpp"
#include "rtl_operators.hpp"
#include "rtlynx_dense.h"

namespace {

constexpr int64_t kMaxBytes = (int64_t)1 << 31;
constexpr int64_t kMaxStride = (int64_t)1 << 40;
constexpr int64_t kMaxGateRows = 65535;
constexpr int64_t kMaxWidth = (int64_t)1 << 25;          // 64 rows, a step of the contraction, stay below 2^32 bytes

int64_t up8(int64_t v) { return (v + 7) / 8 * 8; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

bool bytes_ok(int64_t rows, int64_t cols) {
  return rows == 0 || cols == 0 || (cols < kMaxBytes / 2 && rows <= (kMaxBytes - 1) / (cols * 2));
}

bool sizes_ok(int64_t M, int64_t N, int64_t K) {
  return M >= 0 && N >= 0 && M < kMaxBytes && N < kMaxWidth && K >= 8 && K < kMaxWidth && K % 8 == 0 && bytes_ok(M, K) &&
         bytes_ok(N, K) && bytes_ok(M, N);
}
// dz has rows of np elements.
bool back_sizes_ok(int64_t M, int64_t N, int64_t K) { return sizes_ok(M, N, K) && bytes_ok(M, up8(N)); }

bool gate_ok(int64_t M, int64_t rows, int64_t stride) {
  return rows >= 1 && rows <= kMaxGateRows && stride >= 0 && stride < kMaxStride && M % rows == 0;
}

bool flags_ok(uint32_t flags) { return (flags & 0xFu) <= RTL_DENSE_FP16 && (flags & ~(0x3Fu | RTL_DENSE_Z_FP32)) == 0; }

size_t part_bytes(const rtl::LinearForm& f, int64_t M, int64_t N) {
  return f.splits > 1 ? (size_t)f.splits * (size_t)M * (size_t)N * 4 : 0;
}

struct BackwardBytes {
  size_t dz, bias, gate, part, total;
  int64_t np, parts;
};
BackwardBytes backward_bytes(int64_t M, int64_t N, int64_t K, int64_t groups) {
  BackwardBytes b;
  b.np = up8(N);
  b.parts = rtl::linear_dz_parts(M, N, groups);
  b.dz = up256((size_t)M * (size_t)b.np * 2);
  b.bias = b.gate = up256((size_t)(groups * b.parts) * (size_t)N * 4);
  const size_t dx = part_bytes(rtl::linear_form(M, K, N, false), M, K), dw = part_bytes(rtl::linear_form(N, K, M, false), N, K);
  b.part = up256(dx > dw ? dx : dw);
  b.total = b.dz + b.bias + b.gate + b.part;
  return b;
}

}  // namespace

RTL_API size_t rtl_linear_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (!sizes_ok(M, N, K) || M == 0 || N == 0) return 0;
  return part_bytes(rtl::linear_form(M, N, K, true), M, N);
}

RTL_API rtl_status rtl_linear(const void* x, const void* w, const void* bias, const void* gate, int64_t gate_rows,
                              int64_t gate_stride, const void* residual, int64_t M, int64_t N, int64_t K, void* y, void* z,
                              void* workspace, size_t workspace_bytes, uint32_t flags, void* hip_stream) {
  if (!flags_ok(flags)) return RTL_ERR_BAD_FLAGS;
  if (!sizes_ok(M, N, K) || (gate != nullptr && !gate_ok(M, gate_rows, gate_stride))) return RTL_ERR_BAD_SHAPE;
  if (M == 0 || N == 0) return RTL_OK;
  if (x == nullptr || w == nullptr || y == nullptr) return RTL_ERR_NULL_POINTER;
  for (const void* p : {x, w, residual, (const void*)y, (const void*)z, (const void*)workspace})
    if (!rtl::aligned(p, 16)) return RTL_ERR_MISALIGNED;
  if (!rtl::aligned(bias, 2) || !rtl::aligned(gate, 2)) return RTL_ERR_MISALIGNED;
  const rtl::LinearForm form = rtl::linear_form(M, N, K, true);
  const size_t need = part_bytes(form, M, N);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return RTL_ERR_WORKSPACE;
  rtl::LinearGemm g{};
  g.a = x;
  g.b = w;
  g.lda = g.ldb = K;
  g.a_bytes = M * K * 2;
  g.b_bytes = N * K * 2;
  g.M = M;
  g.N = N;
  g.K = K;
  g.tile_m = form.tile_m;
  g.tile_n = form.tile_n;
  g.splits = form.splits;
  g.part = static_cast<float*>(workspace);
  g.e.bias = static_cast<const uint16_t*>(bias);
  g.e.gate = static_cast<const uint16_t*>(gate);
  g.e.gate_tokens = gate != nullptr ? M / gate_rows : M;
  g.e.gate_stride = gate_rows > 1 ? gate_stride : 0;
  g.e.residual = static_cast<const uint16_t*>(residual);
  g.e.y = static_cast<uint16_t*>(y);
  g.e.z = z;
  g.e.z_fp32 = (flags & RTL_DENSE_Z_FP32) != 0;
  g.e.act = (int)((flags >> 4) & 3u);
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  const rtl_status d = rtl::check_device(stream);
  if (d != RTL_OK) return d;
  return rtl::from_hip(rtl::launch_linear(g, (flags & 0xFu) == RTL_DENSE_FP16, stream));
}

RTL_API size_t rtl_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t gate_rows) {
  if (!back_sizes_ok(M, N, K) || !gate_ok(M, gate_rows, 0) || N == 0) return 0;
  return backward_bytes(M, N, K, gate_rows).total;
}

RTL_API rtl_status rtl_linear_backward(const void* dy, const void* x, const void* w, const void* z, const void* gate,
                                       int64_t gate_rows, int64_t gate_stride, int64_t M, int64_t N, int64_t K, void* dx,
                                       void* dw, void* dbias, void* dgate, void* workspace, size_t workspace_bytes,
                                       uint32_t flags, void* hip_stream) {
  if (!flags_ok(flags)) return RTL_ERR_BAD_FLAGS;
  if (!back_sizes_ok(M, N, K) || !gate_ok(M, gate_rows, gate_stride)) return RTL_ERR_BAD_SHAPE;
  if (N == 0 && (M == 0 || dx == nullptr)) return RTL_OK;
  if (dx == nullptr && dw == nullptr && dbias == nullptr && dgate == nullptr) return RTL_OK;
  const int act = (int)((flags >> 4) & 3u);
  if (M > 0 && N > 0 &&
      (dy == nullptr || (dx != nullptr && w == nullptr) || (dw != nullptr && x == nullptr) ||
       ((act != 0 || dgate != nullptr) && z == nullptr)))
    return RTL_ERR_NULL_POINTER;
  for (const void* p : {dy, x, w, z, (const void*)dx, (const void*)dw, (const void*)workspace})
    if (!rtl::aligned(p, 16)) return RTL_ERR_MISALIGNED;
  for (const void* p : {gate, (const void*)dbias, (const void*)dgate})
    if (!rtl::aligned(p, 2)) return RTL_ERR_MISALIGNED;
  const BackwardBytes b = backward_bytes(M, N, K, gate_rows);
  if (b.total > 0 && (workspace == nullptr || workspace_bytes < b.total)) return RTL_ERR_WORKSPACE;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  const rtl_status st = rtl::check_device(stream);
  if (st != RTL_OK) return st;
  const bool fp16 = (flags & 0xFu) == RTL_DENSE_FP16;
  char* const ws = static_cast<char*>(workspace);
  // dy itself where nothing changes it and its rows are whole 16-byte chunks.
  const bool products = dx != nullptr || dw != nullptr;
  const bool own = products && (act != 0 || gate != nullptr || N % 8 != 0);
  hipError_t e = hipSuccess;
  if ((own || dbias != nullptr || dgate != nullptr) && N > 0) {
    rtl::LinearDz a{};
    a.dy = static_cast<const uint16_t*>(dy);
    a.z = z;
    a.z_fp32 = (flags & RTL_DENSE_Z_FP32) != 0;
    a.gate = static_cast<const uint16_t*>(gate);
    a.gate_stride = gate_rows > 1 ? gate_stride : 0;
    a.M = M;
    a.N = N;
    a.np = b.np;
    a.groups = gate_rows;
    a.parts = b.parts;
    a.act = act;
    a.dz = own ? reinterpret_cast<uint16_t*>(ws) : nullptr;
    a.bias_part = dbias != nullptr ? reinterpret_cast<float*>(ws + b.dz) : nullptr;
    a.gate_part = dgate != nullptr ? reinterpret_cast<float*>(ws + b.dz + b.bias) : nullptr;
    a.dbias = static_cast<uint16_t*>(dbias);
    a.dgate = static_cast<uint16_t*>(dgate);
    e = rtl::launch_linear_dz(a, fp16, stream);
    if (e != hipSuccess) return rtl::from_hip(e);
  }
  const void* const dz = own ? ws : dy;
  rtl::LinearGemm g{};
  g.part = reinterpret_cast<float*>(ws + b.dz + b.bias + b.gate);
  g.e.gate_tokens = 1;
  if (dx != nullptr && M > 0) {                         // [M, K] over N
    const rtl::LinearForm f = rtl::linear_form(M, K, N, false);
    g.a = dz;
    g.b = w;
    g.lda = b.np;
    g.ldb = K;
    g.a_bytes = M * b.np * 2;
    g.b_bytes = N * K * 2;
    g.M = M;
    g.N = K;
    g.K = b.np;
    g.tile_m = f.tile_m;
    g.tile_n = f.tile_n;
    g.splits = f.splits;
    g.e.y = static_cast<uint16_t*>(dx);
    e = rtl::launch_linear_dx(g, fp16, stream);
    if (e != hipSuccess) return rtl::from_hip(e);
  }
  if (dw != nullptr && N > 0) {                         // [N, K] over M
    const rtl::LinearForm f = rtl::linear_form(N, K, M, false);
    g.a = dz;
    g.b = x;
    g.lda = b.np;
    g.ldb = K;
    g.a_bytes = M * b.np * 2;
    g.b_bytes = M * K * 2;
    g.M = N;
    g.N = K;
    g.K = M;
    g.tile_m = f.tile_m;
    g.tile_n = f.tile_n;
    g.splits = f.splits;
    g.e.y = static_cast<uint16_t*>(dw);
    e = rtl::launch_linear_dw(g, fp16, stream);
  }
  return rtl::from_hip(e);
}
