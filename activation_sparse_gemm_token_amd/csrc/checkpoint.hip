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
// memory: 2 bytes in, 1.16 out per channel, and the other way round.  4096 x 12288:
// 37 to 41 us out of the caches (159 MB; 32 with the same input again and again), and
// 23 us for an unpack right after, whose codes are in the last-level cache.
//
// FINE keeps a second exponent per block, the pruned channels' own: two more shuffles
// for its largest magnitude, the third of each group, and one rounding a channel more.
#include <type_traits>

#include "rtl_checkpoint.hpp"
#include "rtl_common.hpp"
#include "rtl_operators.hpp"

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

// Two channels of a word as codes in bits 0..7 and 8..15.  FINE: the pruned ones
// (their bit of `kept` is 0) have a step of their own and no code 0 but of 0.
__device__ __forceinline__ uint32_t code_of(float v, int shift) {
  const float q = __builtin_rintf(__builtin_amdgcn_ldexpf(v, shift));
  return (uint32_t)(int)__builtin_fminf(__builtin_fmaxf(q, -127.f), 127.f) & 0xffu;
}
__device__ __forceinline__ uint32_t pruned_code_of(float v, int shift) {
  const uint32_t q = code_of(v, shift);
  return q == 0 && v != 0.f ? (v < 0.f ? 0xffu : 1u) : q;
}
template <bool FINE>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int shift, int pruned_shift, uint32_t kept) {
  const float a = bf16_lo_to_f32(w), b = bf16_hi_to_f32(w);
  uint32_t ca = code_of(a, shift), cb = code_of(b, shift);
  if constexpr (FINE) {
    if (!(kept & 1u)) ca = pruned_code_of(a, pruned_shift);
    if (!(kept & 2u)) cb = pruned_code_of(b, pruned_shift);
  }
  return ca | cb << 8;
}

// P wavefronts per token (1, 2 or 4).  WIDE: K % 8 == 0, whole 16-byte units;
// otherwise rows are 8-byte aligned and the last unit is half a one.
// FINE: a second exponent per block, of its pruned channels.
template <bool WIDE, int P, bool FINE>
__global__ void __launch_bounds__(64 * kWaves)
checkpoint_pack_kernel(const uint16_t* __restrict__ x, int64_t M, int64_t K, int8_t* __restrict__ codes,
                       uint8_t* __restrict__ exps, uint8_t* __restrict__ pruned_exps, uint8_t* __restrict__ idx,
                       float* __restrict__ stats) {
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
      int p = e;
      if constexpr (FINE) {
        uint32_t next = mag_max(g0.third, g1.third);
        next = mag_max(next, (uint32_t)__shfl_xor((int)next, 1, 64));
        next = mag_max(next, (uint32_t)__shfl_xor((int)next, 2, 64));
        p = (int)(next >> 23);
      }
      if (c < units) {
        const int shift = 133 - e, ps = 133 - p;
        const uint32_t k0 = kept_bits(code0), k1 = kept_bits(code1);
        const uint32_t lo = code_pair<FINE>(w[u][0], shift, ps, k0) | code_pair<FINE>(w[u][1], shift, ps, k0 >> 2) << 16;
        const uint32_t hi = code_pair<FINE>(w[u][2], shift, ps, k1) | code_pair<FINE>(w[u][3], shift, ps, k1 >> 2) << 16;
        const bool whole = WIDE || 8 * c + 8 <= K;
        if constexpr (WIDE) {
          *reinterpret_cast<u32x2*>(cr + 8 * c) = (u32x2){lo, hi};
        } else {
          *reinterpret_cast<uint32_t*>(cr + 8 * c) = lo;
          if (whole) *reinterpret_cast<uint32_t*>(cr + 8 * c + 4) = hi;
        }
        if ((c & 3) == 0) er[c >> 2] = (uint8_t)e;
        if (FINE && (c & 3) == 0) pruned_exps[row * ((K + 31) / 32) + (c >> 2)] = (uint8_t)p;
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

template <bool WIDE, bool FINE>
__global__ void __launch_bounds__(256)
checkpoint_unpack_kernel(const int8_t* __restrict__ codes, const uint8_t* __restrict__ exps,
                         const uint8_t* __restrict__ pruned_exps, const uint8_t* __restrict__ idx, uint32_t M, uint32_t K,
                         uint16_t* __restrict__ y) {
  // 8 channels; FINE: at idx byte i.
  auto values = [&](u32x2 q, int e, size_t block, uint32_t i) {
    if constexpr (FINE) {
      u32x4 pruned, kept;
      ckpt_split8(q, (uint32_t)e, pruned_exps[block], idx[i], pruned, kept);
      return (u32x4)(pruned | kept);
    } else {
      return ckpt_values(q, e);
    }
  };
  const uint32_t units = (K + 7) / 8, blocks = (K + 31) / 32;
  const uint32_t total = M * units;                   // below 2^28: M * K * 2 bytes are below 2 GiB
  for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < total; i += gridDim.x * 256) {
    const uint32_t row = i / units, c = i - row * units;
    const int8_t* src = codes + (size_t)row * K + 8 * c;
    const size_t block = (size_t)row * blocks + (c >> 2);
    const int e = (int)exps[block];
    uint16_t* dst = y + (size_t)row * K + 8 * c;
    if constexpr (WIDE) {
      *reinterpret_cast<u32x4*>(dst) = values(*reinterpret_cast<const u32x2*>(src), e, block, i);
    } else {
      const bool whole = 8 * c + 8 <= K;
      u32x2 q = {*reinterpret_cast<const uint32_t*>(src), 0};
      if (whole) q[1] = *reinterpret_cast<const uint32_t*>(src + 4);
      const u32x4 v = values(q, e, block, i);
      *reinterpret_cast<u32x2*>(dst) = (u32x2){v[0], v[1]};
      if (whole) *reinterpret_cast<u32x2*>(dst + 4) = (u32x2){v[2], v[3]};
    }
  }
}

}  // namespace

hipError_t launch_checkpoint_pack(const uint16_t* x, int64_t M, int64_t K, int8_t* codes, uint8_t* exps,
                                  uint8_t* pruned_exps, uint8_t* idx, float* stats, int compute_units,
                                  hipStream_t stream) {
  // More wavefronts per token while all of them fit the chip at once (8 per
  // SIMD); a wavefront should still have a whole load to make.
  const int64_t fit = 32 * (int64_t)compute_units;
  const int p = 4 * M <= fit && K > 1024 ? 4 : 2 * M <= fit && K > 512 ? 2 : 1;
  const int64_t rows_per = kWaves / p;
  const dim3 grid = folded_grid((M + rows_per - 1) / rows_per), block(64 * kWaves);
  auto pick = [&](auto fine) {
    constexpr bool F = decltype(fine)::value;
    const bool wide = K % 8 == 0;
    return p == 4   ? (wide ? &checkpoint_pack_kernel<true, 4, F> : &checkpoint_pack_kernel<false, 4, F>)
           : p == 2 ? (wide ? &checkpoint_pack_kernel<true, 2, F> : &checkpoint_pack_kernel<false, 2, F>)
                    : (wide ? &checkpoint_pack_kernel<true, 1, F> : &checkpoint_pack_kernel<false, 1, F>);
  };
  auto* k = pruned_exps != nullptr ? pick(std::true_type{}) : pick(std::false_type{});
  return launch(k, grid, block, stream, x, M, K, codes, exps, pruned_exps, idx, stats);
}

hipError_t launch_checkpoint_unpack(const int8_t* codes, const uint8_t* exps, const uint8_t* pruned_exps,
                                    const uint8_t* idx, int64_t M, int64_t K, uint16_t* y, hipStream_t stream) {
  const int64_t blocks = (M * ((K + 7) / 8) + 255) / 256;
  const dim3 grid((unsigned)(blocks < 16384 ? blocks : 16384)), block(256);
  auto* k = pruned_exps != nullptr
                ? (K % 8 == 0 ? &checkpoint_unpack_kernel<true, true> : &checkpoint_unpack_kernel<false, true>)
                : (K % 8 == 0 ? &checkpoint_unpack_kernel<true, false> : &checkpoint_unpack_kernel<false, false>);
  return launch(k, grid, block, stream, codes, exps, pruned_exps, idx, (uint32_t)M, (uint32_t)K, y);
}

}  // namespace rtl
