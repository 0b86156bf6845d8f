// Linear layers of few rows with 4-bit weights and group scales
// (include/rtlynx_w4.h).
//
// At 16 rows or fewer the work is reading the weights: half a byte each, so at
// the card's copy rate some 10^13 weights a second, three or four vector
// operations each.  That leaves no room to widen every code to fp32; the
// matrix cores, idle otherwise, take the products.  A code becomes a bf16
// operand with one shift and one and-or per two codes: q in the upper four
// mantissa bits of 1.0 is 1 + q / 16, exact.  With Sx the group's sum of x
// (one more matrix instruction, against ones),
//
//   sum x (q - z) s = 16 s (sum x (1 + q / 16) - (1 + z / 16) Sx),
//
// whose cancellation costs at most (16 + q) / |q - z| ulps of fp32.
//
// Packed weight: 1 KiB per 16 rows x 128 channels, 16 bytes per lane, so a
// wavefront's load is contiguous and is its own matrix operand: dword j of
// lane l holds channels 32 j + 8 (l / 16) + [0, 8) of row l % 16, channel 2p
// in nibble p and 2p + 1 in nibble p + 4.  Each tile's scales (and zero terms) follow
// in the same tile order, [16 rows][128 / group].
#include "rtl_common.hpp"
#include "rtl_operators.hpp"

namespace rtl {

namespace {

constexpr int kWaves = 8;                 // share a block's channels
constexpr uint32_t kOnes = 0x3f803f80u;   // two bf16 ones

__device__ __forceinline__ bf16x8 widen(uint32_t w) {
  constexpr uint32_t kMask = 0x00780078u;
  u32x4 r;
  r[0] = ((w << 3) & kMask) | kOnes;
  r[1] = ((w >> 1) & kMask) | kOnes;
  r[2] = ((w >> 5) & kMask) | kOnes;
  r[3] = ((w >> 9) & kMask) | kOnes;
  return __builtin_bit_cast(bf16x8, r);
}

// Scale entries of one tile and lane row: GROUPS of 2 bytes (scale) or 4
// (scale, 1 + z / 16).
template <int GROUPS, bool ZEROS>
struct alignas(GROUPS * (ZEROS ? 4 : 2)) Meta {
  typename std::conditional<ZEROS, uint32_t, uint16_t>::type v[GROUPS];
};

// MT tiles of 16 rows of x, NT tiles of 16 rows of the weight.  The block's
// wavefronts take contiguous runs of the channel tiles; their sums are joined
// in LDS, halving the wavefronts each time, in an order the sizes fix.
template <int MT, int NT, int GROUPS, bool ZEROS>
__global__ void __launch_bounds__(64 * kWaves)
w4_linear_kernel(const uint16_t* __restrict__ x, const char* __restrict__ packed, int64_t meta_at, int64_t M,
                 int64_t N, int64_t K, uint16_t* __restrict__ y) {
  constexpr int kDepth = MT == 1 ? (NT == 1 ? 4 : 2) : 1;      // channel tiles requested ahead
  using MetaT = Meta<GROUPS, ZEROS>;
  __shared__ f32x4 red[kWaves / 2][MT * NT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const int64_t tiles_n = (N + 15) / 16, tiles_k = (K + 127) / 128;
  const int64_t nt0 = (int64_t)blockIdx.x * NT, m0 = (int64_t)blockIdx.y * (16 * MT);
  const int64_t k_lo = tiles_k * wave / kWaves, k_hi = tiles_k * (wave + 1) / kWaves;

  const u32x4* wp[NT];
  const MetaT* sp[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t nt = nt0 + t < tiles_n ? nt0 + t : tiles_n - 1;        // past the end: read the last, store nothing
    wp[t] = reinterpret_cast<const u32x4*>(packed) + nt * tiles_k * 64 + lane;
    sp[t] = reinterpret_cast<const MetaT*>(packed + meta_at) + nt * tiles_k * 16 + col;
  }
  const uint16_t* xp[MT];
  bool row_ok[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int64_t row = m0 + 16 * m + col;
    row_ok[m] = row < M;
    xp[m] = x + (row_ok[m] ? row : 0) * K + 8 * quad;
  }

  struct Stage {
    u32x4 w[NT];
    MetaT s[NT];
    u32x4 x[MT][4];
  };
  Stage st[kDepth];
  auto load = [&](Stage& d, int64_t kt) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      d.w[t] = wp[t][kt * 64];
      d.s[t] = sp[t][kt * 16];
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t k = 128 * kt + 32 * j;
        d.x[m][j] = (u32x4){0, 0, 0, 0};
        if (row_ok[m] && k < K) d.x[m][j] = *reinterpret_cast<const u32x4*>(xp[m] + k);
      }
  };

  f32x4 total[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) total[m][t] = (f32x4){0, 0, 0, 0};
  const bf16x8 ones = __builtin_bit_cast(bf16x8, (u32x4){kOnes, kOnes, kOnes, kOnes});

  auto consume = [&](const Stage& d) {
    constexpr int kPer = 4 / GROUPS;                    // matrix instructions per group
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      f32x4 sum[MT], acc[MT][NT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        sum[m] = (f32x4){0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[m][t] = (f32x4){0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int j = g * kPer + i;
#pragma unroll
        for (int m = 0; m < MT; ++m)
          sum[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, d.x[m][j]), ones, sum[m], 0, 0, 0);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const bf16x8 w = widen(d.w[t][j]);
#pragma unroll
          for (int m = 0; m < MT; ++m)
            acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, d.x[m][j]), w, acc[m][t], 0, 0, 0);
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint32_t e = d.s[t].v[g];
        const float scale = 16.0f * bf16_lo_to_f32(e);
        const float zero = ZEROS ? bf16_hi_to_f32(e) : 1.5f;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            total[m][t][i] = __builtin_fmaf(scale, __builtin_fmaf(-zero, sum[m][i], acc[m][t][i]), total[m][t][i]);
      }
    }
  };

#pragma unroll
  for (int i = 0; i < kDepth; ++i)
    if (k_lo + i < k_hi) load(st[i], k_lo + i);
  for (int64_t kt = k_lo; kt < k_hi; kt += kDepth) {
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
      if (kt + i < k_hi) {
        consume(st[i]);
        if (kt + i + kDepth < k_hi) load(st[i], kt + i + kDepth);
      }
    }
  }

#pragma unroll
  for (int half = kWaves / 2; half >= 1; half /= 2) {
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) red[wave - half][m * NT + t][lane] = total[m][t];
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) total[m][t] += red[wave][m * NT + t][lane];
    }
    __syncthreads();
  }
  if (wave != 0) return;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int64_t n = 16 * (nt0 + t) + col;
      const uint32_t p0 = cvt_pk_bf16(total[m][t][0], total[m][t][1]);
      const uint32_t p1 = cvt_pk_bf16(total[m][t][2], total[m][t][3]);
      const int64_t row = m0 + 16 * m + 4 * quad;
      if (n < N) {
        if (row + 0 < M) y[(row + 0) * N + n] = (uint16_t)p0;
        if (row + 1 < M) y[(row + 1) * N + n] = (uint16_t)(p0 >> 16);
        if (row + 2 < M) y[(row + 2) * N + n] = (uint16_t)p1;
        if (row + 3 < M) y[(row + 3) * N + n] = (uint16_t)(p1 >> 16);
      }
    }
}

// One thread per dword of codes, then one per scale entry.  Rows and
// channels past the weight get code 0 and scale 0.
__global__ void __launch_bounds__(256)
w4_pack_kernel(const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scales,
               const uint8_t* __restrict__ zeros, int64_t N, int64_t K, int group, char* __restrict__ packed,
               int64_t meta_at) {
  const int64_t tiles_n = (N + 15) / 16, tiles_k = (K + 127) / 128;
  const int64_t dwords = tiles_n * tiles_k * 256;
  const int groups = 128 / group;
  const int64_t metas = tiles_n * tiles_k * 16 * groups;
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < dwords + metas; i += stride) {
    if (i < dwords) {
      const int j = i & 3, lane = (i >> 2) & 63;
      const int64_t tile = i >> 8, nt = tile / tiles_k, kt = tile - nt * tiles_k;
      const int64_t n = 16 * nt + (lane & 15), k = 128 * kt + 32 * j + 8 * (lane >> 4);
      uint32_t out = 0;
      if (n < N && k < K) {
        const uint32_t in = *reinterpret_cast<const uint32_t*>(codes + n * (K / 2) + k / 2);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint32_t b = (in >> (8 * p)) & 0xffu;
          out |= (b & 15u) << (4 * p) | (b >> 4) << (4 * p + 16);
        }
      }
      reinterpret_cast<uint32_t*>(packed)[i] = out;
    } else {
      const int64_t e = i - dwords;
      const int g = (int)(e % groups);
      const int64_t r = e / groups, tile = r >> 4, nt = tile / tiles_k, kt = tile - nt * tiles_k;
      const int64_t n = 16 * nt + (r & 15), k = 128 * kt + (int64_t)g * group;
      const bool in = n < N && k < K;
      const int64_t at = n * (K / group) + k / group;
      const uint32_t s = in ? scales[at] : 0u;
      if (zeros != nullptr) {
        const uint32_t z = in ? zeros[at] & 15u : 0u;
        // 1 + z / 16 in bf16: z in the upper four mantissa bits of one.
        reinterpret_cast<uint32_t*>(packed + meta_at)[e] = s | (0x3f80u | z << 3) << 16;
      } else {
        reinterpret_cast<uint16_t*>(packed + meta_at)[e] = (uint16_t)s;
      }
    }
  }
}

template <int MT, int NT>
hipError_t launch_tiles(const uint16_t* x, const char* packed, int64_t meta_at, int64_t M, int64_t N, int64_t K,
                        int group, bool zeros, uint16_t* y, hipStream_t stream) {
  const int64_t tiles_n = (N + 15) / 16;
  const dim3 grid((unsigned)((tiles_n + NT - 1) / NT), (unsigned)((M + 16 * MT - 1) / (16 * MT)));
  auto* k = group == 128 ? (zeros ? &w4_linear_kernel<MT, NT, 1, true> : &w4_linear_kernel<MT, NT, 1, false>)
            : group == 64 ? (zeros ? &w4_linear_kernel<MT, NT, 2, true> : &w4_linear_kernel<MT, NT, 2, false>)
                          : (zeros ? &w4_linear_kernel<MT, NT, 4, true> : &w4_linear_kernel<MT, NT, 4, false>);
  return launch(k, grid, dim3(64 * kWaves), stream, x, packed, meta_at, M, N, K, y);
}

}  // namespace

hipError_t launch_w4_linear(const uint16_t* x, const void* packed, int64_t M, int64_t N, int64_t K, int group,
                            bool zeros, uint16_t* y, hipStream_t stream) {
  const int64_t meta_at = w4_tiles(N, K) * 1024;
  const char* p = static_cast<const char*>(packed);
  if (M <= 16) return launch_tiles<1, 1>(x, p, meta_at, M, N, K, group, zeros, y, stream);
  if (M <= 32) return launch_tiles<2, 2>(x, p, meta_at, M, N, K, group, zeros, y, stream);
  return launch_tiles<4, 4>(x, p, meta_at, M, N, K, group, zeros, y, stream);
}

hipError_t launch_w4_pack(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t N, int64_t K,
                          int group, void* packed, hipStream_t stream) {
  const int64_t tiles = w4_tiles(N, K), items = tiles * 256 + tiles * 16 * (128 / group);
  const int64_t blocks = (items + 255) / 256;
  const dim3 grid((unsigned)(blocks < 16384 ? blocks : 16384));
  return launch(&w4_pack_kernel, grid, dim3(256), stream, codes, scales, zeros, N, K, group,
                static_cast<char*>(packed), tiles * 1024);
}

}  // namespace rtl
