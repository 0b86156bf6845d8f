// The 8-bit activation checkpoint (include/rtlynx_train.h): one pass over X
// that writes codes, block exponents, the 2:4 positions and the token's L1
// statistics, and the pass that turns codes back into bf16.
//
// A wavefront owns a part of a token; a lane's unit is 16 bytes (8 channels:
// two groups of 4, a quarter of a block of 32), so the block's largest
// magnitude is two shuffles away and every access is contiguous over the
// wavefront.  The step is the power of two that puts the largest magnitude
// in [64, 128): its biased exponent is bf16's own exponent field of the largest
// magnitude, and the division is an exponent shift, so codes have no rounding
// of their own beyond the one to an integer.  Both kernels are bound by
// HBM: 2 bytes in, 1.16 out per channel, and the other way round.  4096 x 12288:
// 32 us (5.0 TB/s) and 23 us (6.7 TB/s).
#include "rtl_common.hpp"
#include "rtl_operators.hpp"
#include "rtl_checkpoint.hpp"

namespace rtl {

namespace {

constexpr int kWaves = 4;
constexpr int kUnroll = 4;

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

__device__ __forceinline__ uint32_t mag_max(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Two channels of a word as codes in bits 0..7 and 8..15.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int shift) {
  const float a = __builtin_rintf(__builtin_amdgcn_ldexpf(bf16_lo_to_f32(w), shift));
  const float b = __builtin_rintf(__builtin_amdgcn_ldexpf(bf16_hi_to_f32(w), shift));
  const int ia = (int)__builtin_fminf(__builtin_fmaxf(a, -127.f), 127.f);
  const int ib = (int)__builtin_fminf(__builtin_fmaxf(b, -127.f), 127.f);
  return ((uint32_t)ia & 0xffu) | ((uint32_t)ib & 0xffu) << 8;
}

// P wavefronts per token (1, 2 or 4).  WIDE: K % 8 == 0, whole 16-byte units;
// otherwise rows are 8-byte aligned and the last unit is half a one.
template <bool WIDE, int P>
__global__ void __launch_bounds__(64 * kWaves)
checkpoint_pack_kernel(const uint16_t* __restrict__ x, int64_t M, int64_t K, int8_t* __restrict__ codes,
                       uint8_t* __restrict__ exps, uint8_t* __restrict__ idx, float* __restrict__ stats) {
  __shared__ float red[kWaves][2];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, part = wv % P;
  const int64_t row = folded_block() * (kWaves / P) + wv / P;
  const bool live = row < M;
  const int64_t units = (K + 7) / 8;                  // = idx bytes of a row
  const uint16_t* xr = x + row * K;
  int8_t* cr = codes + row * K;
  uint8_t* er = exps + row * ((K + 31) / 32);
  uint8_t* ir = idx + row * units;
  float lk = 0.f, lp = 0.f;
  // Every lane of a live wavefront takes part in the shuffles; lanes past the
  // row hold zeros.
  for (int64_t c0 = 0; live && c0 < units; c0 += 64 * P * kUnroll) {
    u32x4 w[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t c = c0 + (u * P + part) * 64 + lane;
      w[u] = (u32x4){0, 0, 0, 0};
      if (c < units) {
        if constexpr (WIDE) {
          w[u] = *reinterpret_cast<const u32x4*>(xr + 8 * c);
        } else {
          const u32x2 a = *reinterpret_cast<const u32x2*>(xr + 8 * c);
          w[u][0] = a[0];
          w[u][1] = a[1];
          if (8 * c + 8 <= K) {
            const u32x2 b = *reinterpret_cast<const u32x2*>(xr + 8 * c + 4);
            w[u][2] = b[0];
            w[u][3] = b[1];
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t c = c0 + (u * P + part) * 64 + lane;
      // Groups: positions and L1 sums; a group's largest magnitude is its first key.
      const Group4 g0 = rank_group(w[u][0], w[u][1]), g1 = rank_group(w[u][2], w[u][3]);
      const uint32_t code0 = code_from_selector(pair_selector_sorted(g0.first, g0.second));
      const uint32_t code1 = code_from_selector(pair_selector_sorted(g1.first, g1.second));
      lk = add_mag_pair(add_mag_pair(lk, g0.first, g0.second), g1.first, g1.second);
      lp = add_mag_pair(add_mag_pair(lp, g0.third, g0.fourth), g1.third, g1.fourth);
      uint32_t top = mag_max(g0.first, g1.first);
      top = mag_max(top, (uint32_t)__shfl_xor((int)top, 1, 64));
      top = mag_max(top, (uint32_t)__shfl_xor((int)top, 2, 64));
      const int e = (int)(top >> 23);                 // bf16's exponent field
      if (c < units) {
        const int shift = 133 - e;
        const uint32_t lo = code_pair(w[u][0], shift) | code_pair(w[u][1], shift) << 16;
        const uint32_t hi = code_pair(w[u][2], shift) | code_pair(w[u][3], shift) << 16;
        const bool whole = WIDE || 8 * c + 8 <= K;
        if constexpr (WIDE) {
          *reinterpret_cast<u32x2*>(cr + 8 * c) = (u32x2){lo, hi};
        } else {
          *reinterpret_cast<uint32_t*>(cr + 8 * c) = lo;
          if (whole) *reinterpret_cast<uint32_t*>(cr + 8 * c + 4) = hi;
        }
        if ((c & 3) == 0) er[c >> 2] = (uint8_t)e;
        ir[c] = (uint8_t)(code0 | (whole ? code1 << 4 : 0u));
      }
    }
  }
  lk = wave_sum(lk);
  lp = wave_sum(lp);
  if constexpr (P > 1) {
    if (lane == 0) { red[wv][0] = lk; red[wv][1] = lp; }
    __syncthreads();
    lk = lp = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) { lk += red[wv - part + i][0]; lp += red[wv - part + i][1]; }
  }
  if (live && part == 0 && lane == 0) {
    stats[2 * row] = lk > 0.f ? (lk + lp) / lk : 1.0f;
    stats[2 * row + 1] = lk;
  }
}

template <bool WIDE>
__global__ void __launch_bounds__(256)
checkpoint_unpack_kernel(const int8_t* __restrict__ codes, const uint8_t* __restrict__ exps, uint32_t M, uint32_t K,
                         uint16_t* __restrict__ y) {
  const uint32_t units = (K + 7) / 8, blocks = (K + 31) / 32;
  const uint32_t total = M * units;                   // below 2^28: M * K * 2 bytes are below 2 GiB
  for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < total; i += gridDim.x * 256) {
    const uint32_t row = i / units, c = i - row * units;
    const int8_t* src = codes + (size_t)row * K + 8 * c;
    const int e = (int)exps[(size_t)row * blocks + (c >> 2)];
    uint16_t* dst = y + (size_t)row * K + 8 * c;
    if constexpr (WIDE) {
      *reinterpret_cast<u32x4*>(dst) = ckpt_values(*reinterpret_cast<const u32x2*>(src), e);
    } else {
      const bool whole = 8 * c + 8 <= K;
      u32x2 q = {*reinterpret_cast<const uint32_t*>(src), 0};
      if (whole) q[1] = *reinterpret_cast<const uint32_t*>(src + 4);
      const u32x4 v = ckpt_values(q, e);
      *reinterpret_cast<u32x2*>(dst) = (u32x2){v[0], v[1]};
      if (whole) *reinterpret_cast<u32x2*>(dst + 4) = (u32x2){v[2], v[3]};
    }
  }
}

}  // namespace

hipError_t launch_checkpoint_pack(const uint16_t* x, int64_t M, int64_t K, int8_t* codes, uint8_t* exps, uint8_t* idx,
                                  float* stats, int compute_units, hipStream_t stream) {
  // More wavefronts per token while all of them fit the chip at once (8 per
  // SIMD); a wavefront should still have a whole load to make.
  const int64_t fit = 32 * (int64_t)compute_units;
  const int p = 4 * M <= fit && K > 1024 ? 4 : 2 * M <= fit && K > 512 ? 2 : 1;
  const int64_t rows_per = kWaves / p;
  const dim3 grid = folded_grid((M + rows_per - 1) / rows_per), block(64 * kWaves);
  const bool wide = K % 8 == 0;
  auto* k = p == 4   ? (wide ? &checkpoint_pack_kernel<true, 4> : &checkpoint_pack_kernel<false, 4>)
            : p == 2 ? (wide ? &checkpoint_pack_kernel<true, 2> : &checkpoint_pack_kernel<false, 2>)
                     : (wide ? &checkpoint_pack_kernel<true, 1> : &checkpoint_pack_kernel<false, 1>);
  return launch(k, grid, block, stream, x, M, K, codes, exps, idx, stats);
}

hipError_t launch_checkpoint_unpack(const int8_t* codes, const uint8_t* exps, int64_t M, int64_t K, uint16_t* y,
                                    hipStream_t stream) {
  const int64_t blocks = (M * ((K + 7) / 8) + 255) / 256;
  const dim3 grid((unsigned)(blocks < 16384 ? blocks : 16384)), block(256);
  auto* k = K % 8 == 0 ? &checkpoint_unpack_kernel<true> : &checkpoint_unpack_kernel<false>;
  return launch(k, grid, block, stream, codes, exps, (uint32_t)M, (uint32_t)K, y);
}

}  // namespace rtl
