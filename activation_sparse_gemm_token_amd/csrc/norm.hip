// Layer norm and its gradients (include/rtlynx_norm.h).
//
// A row of x stays in the registers of the threads that share it, so x is
// read once: its sum gives the mean, the centred squares the variance, and
// the same registers the result.  4 bytes an element forward and 6 backward in 16
// bits.  9216 rows of 4096 in bf16: 29.0 to 30.1 us, 5.0 TB/s, bound by memory at a
// copy's rate; backward, 8192 rows of 4096: 49 us, 4.1 TB/s with the vector units 76 %
// busy and one workgroup's barrier a row between loads and results, and 6 for the join.
//
// TPR threads share a row (up to 64, a wavefront, without a barrier; 128 to 1024), each
// holds E elements in E / VEC pieces of VEC, piece i at channel
// VEC (TPR i + thread).  VEC is the widest access that divides every row.
#include "rtl_elem.hpp"
#include "rtl_operators.hpp"

namespace rtl {

namespace {

constexpr int kBlock = 256;

// Sum over LANES lanes (16, 32 or a wavefront), the same bits in every one of them: by data-parallel moves within rows of 16 lanes (xor 1
// and 2, mirrored halves, mirrored rows), then by swaps of rows and halves; no trip through LDS.
template <int CTRL>
__device__ __forceinline__ float add_moved(float v) {
  const int w = __builtin_bit_cast(int, v);
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(w, w, CTRL, 0xf, 0xf, false));
}
template <int LANES>
__device__ __forceinline__ float lane_sum(float v) {
  v = add_moved<0xB1>(v);                               // quad_perm 1, 0, 3, 2
  v = add_moved<0x4E>(v);                               // quad_perm 2, 3, 0, 1
  v = add_moved<0x141>(v);                              // row_half_mirror
  v = add_moved<0x140>(v);                              // row_mirror
  if constexpr (LANES == 16) return v;
  const uint32_t a = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  const uint32_t r0 = r[0], r1 = r[1];
  v = __builtin_bit_cast(float, r0) + __builtin_bit_cast(float, r1);
  if constexpr (LANES == 32) return v;
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  const auto h = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  const uint32_t h0 = h[0], h1 = h[1];
  return __builtin_bit_cast(float, h0) + __builtin_bit_cast(float, h1);
}

// Sum over the TPR threads of a row, the same bits in all of them.  `lds` is the
// row's slots [TPR / 64], a fresh set in each call between two barriers.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* lds) {
  v = lane_sum<TPR < 64 ? TPR : 64>(v);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) lds[(threadIdx.x % TPR) >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) v += lds[i];
  }
  return v;
}

// A channel's weight or bias, of the tensors' type or fp32.
template <int TYPE, int VEC>
__device__ __forceinline__ void affine_load(const void* p, int64_t at, bool fp32, float (&v)[VEC]) {
  if (TYPE == kFp32 || fp32) {
    constexpr int kV = VEC == 8 ? 4 : VEC;
    Raw<kFp32, kV> r[VEC / kV];
#pragma unroll
    for (int i = 0; i < VEC / kV; ++i) {
      r[i].load(static_cast<const float*>(p) + at + kV * i);
#pragma unroll
      for (int j = 0; j < kV; ++j) v[kV * i + j] = r[i].get(j);
    }
  } else {
    Raw<TYPE, VEC> r;
    r.load(static_cast<const elem_t<TYPE>*>(p) + at);
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = r.get(j);
  }
}

template <int TYPE, int VEC, int TPR, int E>
__global__ void __launch_bounds__(TPR > kBlock ? TPR : kBlock)
norm_kernel(NormArgs a) {
  constexpr int kThreads = TPR > kBlock ? TPR : kBlock, kRows = kThreads / TPR, kPieces = E / VEC;
  using T = elem_t<TYPE>;
  __shared__ float lds[2][kThreads / 64];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int64_t row = folded_block() * kRows + sub;
  // Rows past the last one: TPR is 64 or less then (no barrier), or there is none.
  if (row >= a.rows) return;
  const int64_t b = row / a.tokens, tok = row - b * a.tokens;
  const T* x = static_cast<const T*>(a.x) + b * a.xb + tok * a.xt;
  Raw<TYPE, VEC> raw[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = VEC * (TPR * i + t);
    if (c < a.C) raw[i].load(x + c);
    else raw[i].zero();
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) sum += raw[i].get(j);
  // Divided by C, not multiplied by its rounded inverse: rows of one value have exactly that mean, and so 0 as their
  // result.  (1000 channels of 1000: the inverse gives a mean half a step too large, and results of -0.019.)
  const float mean = row_sum<TPR>(sum, lds[0]) / (float)a.C;
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = VEC * (TPR * i + t);
    if (c < a.C) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float d = raw[i].get(j) - mean;
        sq += d * d;
      }
    }
  }
  const float rstd = 1.f / __builtin_sqrtf(row_sum<TPR>(sq, lds[1]) * a.inv_c + a.eps);
  if (a.mean != nullptr && t == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(a.y) + b * a.yb + tok * a.yt;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = VEC * (TPR * i + t);
    if (c >= a.C) continue;
    float v[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = (raw[i].get(j) - mean) * rstd;
    if (a.weight != nullptr) {
      float w[VEC];
      affine_load<TYPE, VEC>(a.weight, b * a.wb + c, a.affine_fp32, w);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] *= w[j] + a.offset;
      if (a.bias != nullptr) {
        affine_load<TYPE, VEC>(a.bias, b * a.bb + c, a.affine_fp32, w);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] += w[j];
      }
    }
    store_vec<TYPE, VEC>(y + c, v);
  }
}

// Backward.  A workgroup of 1024 threads (one per CU: 16 wavefronts hide the
// loads; of 512 or 256 threads 91 and 107 us for forward and backward where this
// takes 86) walks its part of a group's rows, 1024 / TPR at a time, and keeps its
// channels' sums over them in registers; it leaves one row of sums: the result
// where the group is one part, else norm_join_kernel adds the parts up in order.
constexpr int kBackBlock = 1024;

template <int TYPE, int VEC, int TPR, int E>
__global__ void __launch_bounds__(kBackBlock)
norm_backward_kernel(NormBackArgs a) {
  constexpr int kRows = kBackBlock / TPR, kPieces = E / VEC, kWaves = TPR < 64 ? 1 : TPR / 64;
  using T = elem_t<TYPE>;
  __shared__ __attribute__((aligned(16))) float sums[kRows > 1 ? 8 * kBackBlock : 1];
  __shared__ float lds[2][kRows][2 * kWaves];           // alternating, so one barrier a row is enough
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int64_t group = folded_block() / a.parts, part = folded_block() - group * a.parts;
  if (group >= a.groups) return;
  const int64_t group_rows = a.rows / a.groups;
  float dw[E], db[E];
#pragma unroll
  for (int i = 0; i < E; ++i) dw[i] = db[i] = 0.f;

  struct Row {
    Raw<TYPE, VEC> x[kPieces], g[kPieces];
    float mean, rstd;
  };
  auto load = [&](Row& r, int64_t at) {                 // row `at` of the group; past the end its last row
    const int64_t row = group * group_rows + (at < group_rows ? at : group_rows - 1);
    const int64_t b = row / a.tokens, tok = row - b * a.tokens;
    const T* x = static_cast<const T*>(a.x) + b * a.xb + tok * a.xt;
    const T* g = static_cast<const T*>(a.dy) + b * a.gb + tok * a.gt;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int c = VEC * (TPR * i + t);
      if (c < a.C) {
        r.x[i].load(x + c);
        r.g[i].load(g + c);
      } else {
        r.x[i].zero();
        r.g[i].zero();
      }
    }
    r.mean = a.mean[row];
    r.rstd = a.rstd[row];
  };
  int flip = 0;
  auto use = [&](const Row& r, int64_t at) {
    const bool live = at < group_rows;
    const int64_t row = group * group_rows + (live ? at : group_rows - 1);
    const int64_t b = row / a.tokens, tok = row - b * a.tokens;
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int c = VEC * (TPR * i + t);
      if (c >= a.C || !live) continue;
      float w[VEC];
      if (a.weight != nullptr) {
        affine_load<TYPE, VEC>(a.weight, b * a.wb + c, a.affine_fp32, w);
#pragma unroll
        for (int j = 0; j < VEC; ++j) w[j] += a.offset;
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) w[j] = 1.f;
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float xhat = (r.x[i].get(j) - r.mean) * r.rstd, dy = r.g[i].get(j), g = dy * w[j];
        dw[VEC * i + j] += dy * xhat;
        db[VEC * i + j] += dy;
        s1 += g * xhat;
        s2 += g;
      }
    }
    if (a.dx == nullptr) return;                        // uniform over the grid
    s1 = lane_sum<TPR < 64 ? TPR : 64>(s1);
    s2 = lane_sum<TPR < 64 ? TPR : 64>(s2);
    if constexpr (TPR > 64) {
      float* const mine = lds[flip][sub];
      if ((threadIdx.x & 63) == 0) {
        mine[2 * (t >> 6)] = s1;
        mine[2 * (t >> 6) + 1] = s2;
      }
      __syncthreads();
      s1 = s2 = 0.f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) {
        s1 += mine[2 * i];
        s2 += mine[2 * i + 1];
      }
      flip ^= 1;
    }
    if (!live) return;
    s1 *= a.inv_c;
    s2 *= a.inv_c;
    T* dx = static_cast<T*>(a.dx) + b * a.db + tok * a.dt;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int c = VEC * (TPR * i + t);
      if (c >= a.C) continue;
      float v[VEC], w[VEC];
      if (a.weight != nullptr) affine_load<TYPE, VEC>(a.weight, b * a.wb + c, a.affine_fp32, w);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float xhat = (r.x[i].get(j) - r.mean) * r.rstd;
        const float g = r.g[i].get(j) * (a.weight != nullptr ? w[j] + a.offset : 1.f);
        v[j] = r.rstd * (g - s2 - xhat * s1);
      }
      store_vec<TYPE, VEC>(dx + c, v);
    }
  };
  // Every thread of the workgroup makes the same number of steps (barriers).
  const int64_t step = a.parts * kRows;
  // The next rows are loaded ahead where 128 registers hold two sets of them beside the sums, counted in the words that
  // they take: one element an access fills a register each.  (2730 rows of 12288 in fp32, ahead with spills: 160 us, 98
  // one row at a time; forward and backward over 8186 rows of 4099 in bf16: 386 and 237.)
  constexpr bool kAhead = kPieces * Raw<TYPE, VEC>::kWords <= 8;
  Row r0, r1;
  int64_t at = part * kRows;
  if constexpr (kAhead) {
    if (at < group_rows) load(r0, at + sub);
    for (; at < group_rows; at += 2 * step) {
      const bool more = at + step < group_rows;
      if (more) load(r1, at + step + sub);
      use(r0, at + sub);
      if (more) {
        if (at + 2 * step < group_rows) load(r0, at + 2 * step + sub);
        use(r1, at + step + sub);
      }
    }
  } else {
    for (; at < group_rows; at += step) {
      load(r0, at + sub);
      use(r0, at + sub);
    }
  }
  if (a.dweight == nullptr) return;
  auto put = [&](int which, int64_t c, float v) {
    void* const out = which == 0 ? a.dweight : a.dbias;
    if (a.parts > 1) a.partials[((group * a.parts + part) * 2 + which) * a.C + c] = v;
    else if (a.affine_fp32) static_cast<float*>(out)[group * a.C + c] = v;
    else static_cast<T*>(out)[group * a.C + c] = from_f32<TYPE>(v);
  };
  // The workgroup's rows were summed in kRows sets: joined through LDS 8 elements of a thread, 8 TPR channels, at a
  // time, in order.  (One set after another, every one between two barriers: 64 rows of 256 14.5 us; this way less
  // than the call's 12 us on the host.)
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const float* const v = which == 0 ? dw : db;
#pragma unroll
    for (int e = 0; e < E; e += 8) {
      if constexpr (kRows > 1) __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = VEC * TPR * (i / VEC) + VEC * t + i % VEC;
        if constexpr (kRows > 1) sums[sub * 8 * TPR + at] = v[e + i];
        else if (TPR * e + at < a.C) put(which, TPR * e + at, v[e + i]);
      }
      if constexpr (kRows > 1) {
        __syncthreads();
        for (int at = threadIdx.x; at < 8 * TPR && TPR * e + at < a.C; at += kBackBlock) {
          float s = sums[at];
#pragma unroll
          for (int k = 1; k < kRows; ++k) s += sums[k * 8 * TPR + at];
          put(which, TPR * e + at, s);
        }
      }
    }
  }
}

// Adds the parts' sums up.  64 columns and 16 threads for each: thread p takes
// parts p, p + 16, ..., the 16 sums are added in order.
template <int TYPE>
__global__ void __launch_bounds__(1024)
norm_join_kernel(const float* __restrict__ partials, int64_t groups, int64_t parts, int64_t C, void* dweight, void* dbias) {
  __shared__ float lds[16][64];
  const int col = threadIdx.x & 63, p = threadIdx.x >> 6;
  const int64_t per = (2 * C + 63) / 64, group = folded_block() / per;
  if (group >= groups) return;
  const int64_t c = (folded_block() - group * per) * 64 + col;            // of 2 C: dweight, then dbias
  float s = 0.f;
  if (c < 2 * C)
    for (int64_t i = p; i < parts; i += 16) s += partials[(group * parts + i) * 2 * C + c];
  lds[p][col] = s;
  __syncthreads();
  if (p != 0 || c >= 2 * C) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) s += lds[i][col];
  void* const out = c < C ? dweight : dbias;
  static_cast<elem_t<TYPE>*>(out)[group * C + (c < C ? c : c - C)] = from_f32<TYPE>(s);
}

// Elements per thread and threads per row by C: up to 2048 channels a wavefront
// a row (or a quarter or half of it, where a whole one would have idle lanes), up to 8192 four, else sixteen.
template <int TYPE, int VEC>
hipError_t run_norm(const NormArgs& a, hipStream_t stream) {
  auto go = [&](auto k, int64_t threads, int64_t rows) {
    const int64_t blocks = (a.rows + rows - 1) / rows;
    return launch(k, threads > 512 ? folded_grid_of_1024(blocks) : folded_grid(blocks), dim3((unsigned)threads), stream, a);
  };
  if (a.C <= 128) return go(&norm_kernel<TYPE, VEC, 16, 8>, 256, 16);
  if (a.C <= 256) return go(&norm_kernel<TYPE, VEC, 32, 8>, 256, 8);
  if (a.C <= 512) return go(&norm_kernel<TYPE, VEC, 64, 8>, 256, 4);
  if (a.C <= 1024) return go(&norm_kernel<TYPE, VEC, 64, 16>, 256, 4);
  if (a.C <= 2048) return go(&norm_kernel<TYPE, VEC, 64, 32>, 256, 4);
  if (a.C <= 4096) return go(&norm_kernel<TYPE, VEC, 256, 16>, 256, 1);
  if (a.C <= 8192) return go(&norm_kernel<TYPE, VEC, 256, 32>, 256, 1);
  return go(&norm_kernel<TYPE, VEC, 1024, 32>, 1024, 1);
}

// As few threads to a row as hold it and its sums in 128 registers: more rows on their way.  (32768 x 1024 in fp32 126
// us with 16 elements a thread, 85 with 8; 13106 x 5120 in bf16 137 us with 1024 threads, 107 with 512.)  They do not
// with 32 elements a thread, past 16384 channels, nor quite with 16 of one access each from 8193 on: 4 to 199 spills.
template <int TYPE, int VEC>
hipError_t run_backward(const NormBackArgs& a, hipStream_t stream) {
  auto go = [&](auto k) { return launch(k, folded_grid_of_1024(a.groups * a.parts), dim3(kBackBlock), stream, a); };
  if (a.C <= 128) return go(&norm_backward_kernel<TYPE, VEC, 16, 8>);
  if (a.C <= 256) return go(&norm_backward_kernel<TYPE, VEC, 32, 8>);
  if (a.C <= 512) return go(&norm_backward_kernel<TYPE, VEC, 64, 8>);
  if constexpr (TYPE == kFp32) {
    if (a.C <= 1024) return go(&norm_backward_kernel<TYPE, VEC, 128, 8>);
    if (a.C <= 2048) return go(&norm_backward_kernel<TYPE, VEC, 256, 8>);
    if (a.C <= 4096) return go(&norm_backward_kernel<TYPE, VEC, 512, 8>);
    if (a.C <= 8192) return go(&norm_backward_kernel<TYPE, VEC, 1024, 8>);
  } else {
    if (a.C <= 1024) return go(&norm_backward_kernel<TYPE, VEC, 64, 16>);
    if (a.C <= 2048) return go(&norm_backward_kernel<TYPE, VEC, 128, 16>);
    if (a.C <= 4096) return go(&norm_backward_kernel<TYPE, VEC, 256, 16>);
    if (a.C <= 8192) return go(&norm_backward_kernel<TYPE, VEC, 512, 16>);
  }
  if (a.C <= 16384) return go(&norm_backward_kernel<TYPE, VEC, 1024, 16>);
  return go(&norm_backward_kernel<TYPE, VEC, 1024, 32>);
}

}  // namespace

// Parts of a group: one workgroup per CU of a 256-CU card over all groups, fewer
// where a part would have no row; one part up to four steps of a workgroup, whose latency is less
// than the second launch's (64 rows of 256: a call of 12 us, 16 in four parts).  A rule on sizes alone, so that the
// sums' order is the same everywhere.
int64_t norm_parts(int64_t rows, int64_t groups, int64_t C) {
  // Rows a workgroup takes at once (half as many in fp32 from 513 channels on).
  const int64_t per = C <= 128 ? 64 : C <= 256 ? 32 : C <= 1024 ? 16 : C <= 2048 ? 8 : C <= 4096 ? 4 : C <= 8192 ? 2 : 1;
  const int64_t group_rows = rows / groups;
  int64_t parts = (256 + groups - 1) / groups;
  const int64_t most = (group_rows + per - 1) / per;
  if (parts > most) parts = most;
  return parts < 1 || most <= 4 ? 1 : parts;
}

hipError_t launch_norm(const NormArgs& a, int type, int vec, hipStream_t stream) {
  if (type == kFp32) return vec == 4 ? run_norm<kFp32, 4>(a, stream) : run_norm<kFp32, 1>(a, stream);
  if (type == kFp16)
    return vec == 8 ? run_norm<kFp16, 8>(a, stream) : vec == 4 ? run_norm<kFp16, 4>(a, stream) : run_norm<kFp16, 1>(a, stream);
  return vec == 8 ? run_norm<kBf16, 8>(a, stream) : vec == 4 ? run_norm<kBf16, 4>(a, stream) : run_norm<kBf16, 1>(a, stream);
}

hipError_t launch_norm_backward(const NormBackArgs& a, int type, int vec, hipStream_t stream) {
  hipError_t e;
  if (type == kFp32) e = vec == 4 ? run_backward<kFp32, 4>(a, stream) : run_backward<kFp32, 1>(a, stream);
  else if (type == kFp16)
    e = vec == 8 ? run_backward<kFp16, 8>(a, stream) : vec == 4 ? run_backward<kFp16, 4>(a, stream) : run_backward<kFp16, 1>(a, stream);
  else
    e = vec == 8 ? run_backward<kBf16, 8>(a, stream) : vec == 4 ? run_backward<kBf16, 4>(a, stream) : run_backward<kBf16, 1>(a, stream);
  if (e != hipSuccess || a.dweight == nullptr || a.parts == 1) return e;
  const dim3 grid = folded_grid_of_1024((2 * a.C + 63) / 64 * a.groups);
  const int out = a.affine_fp32 ? kFp32 : type;
  auto* k = out == kFp32 ? &norm_join_kernel<kFp32> : out == kFp16 ? &norm_join_kernel<kFp16> : &norm_join_kernel<kBf16>;
  return launch(k, grid, dim3(1024), stream, (const float*)a.partials, a.groups, a.parts, (int64_t)a.C, a.dweight, a.dbias);
}

}  // namespace rtl
