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

constexpr uint32_t kOnes = 0x3f803f80u;   // two bf16 ones

// The two constants are kept in registers (the empty asm hides their values):
// as literals they would make the and-or two instructions.
struct WidenConst {
  uint32_t mask, ones;
};
__device__ __forceinline__ WidenConst widen_const() {
  WidenConst c = {0x00780078u, kOnes};
  asm("" : "+s"(c.mask));
  asm("" : "+v"(c.ones));
  return c;
}
__device__ __forceinline__ bf16x8 widen(uint32_t w, const WidenConst& c) {
  u32x4 r;
  r[0] = ((w << 3) & c.mask) | c.ones;
  r[1] = ((w >> 1) & c.mask) | c.ones;
  r[2] = ((w >> 5) & c.mask) | c.ones;
  r[3] = ((w >> 9) & c.mask) | c.ones;
  return __builtin_bit_cast(bf16x8, r);
}

// Scale entries of one tile and lane row: GROUPS of 2 bytes (scale) or 4
// (scale, 1 + z / 16).
template <int GROUPS, bool ZEROS>
struct alignas(GROUPS * (ZEROS ? 4 : 2)) Meta {
  typename std::conditional<ZEROS, uint32_t, uint16_t>::type v[GROUPS];
};

__device__ __forceinline__ f32x4 mfma(u32x4 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), b, c, 0, 0, 0);
}

// One tile of 16 weight rows x 128 channels (w: its 16 bytes, s: its scales)
// times MT tiles of x (x(m, j): operand of step j), added to total.
template <int MT, int NT, int GROUPS, bool ZEROS, typename X>
__device__ __forceinline__ void tile_step(const WidenConst& c, const u32x4 (&w)[NT], const Meta<GROUPS, ZEROS> (&s)[NT], X x,
                                          f32x4 (&total)[MT][NT]) {
  constexpr int kPer = 4 / GROUPS;                      // matrix instructions per group
  const bf16x8 ones = __builtin_bit_cast(bf16x8, (u32x4){kOnes, kOnes, kOnes, kOnes});
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
      u32x4 xv[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        xv[m] = x(m, j);
        sum[m] = mfma(xv[m], ones, sum[m]);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const bf16x8 wv = widen(w[t][j], c);
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m][t] = mfma(xv[m], wv, acc[m][t]);
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint32_t e = s[t].v[g];
      const float scale = 16.0f * bf16_lo_to_f32(e);
      const float zero = ZEROS ? bf16_hi_to_f32(e) : 1.5f;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          total[m][t][i] = __builtin_fmaf(scale, __builtin_fmaf(-zero, sum[m][i], acc[m][t][i]), total[m][t][i]);
    }
  }
}

// Workgroup barrier for data in LDS: waits for this wavefront's LDS operations,
// not (as __syncthreads does) for its loads from memory still in flight.
__device__ __forceinline__ void barrier_lds() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Stores 16 rows (from row0 + 4 (lane / 16)) of column n.
__device__ __forceinline__ void store_column(const f32x4& v, uint16_t* __restrict__ y, int64_t row, int64_t M, int64_t n,
                                             int64_t N) {
  if (n >= N) return;
  const uint32_t p0 = cvt_pk_bf16(v[0], v[1]), p1 = cvt_pk_bf16(v[2], v[3]);
  if (row + 0 < M) y[(row + 0) * N + n] = (uint16_t)p0;
  if (row + 1 < M) y[(row + 1) * N + n] = (uint16_t)(p0 >> 16);
  if (row + 2 < M) y[(row + 2) * N + n] = (uint16_t)p1;
  if (row + 3 < M) y[(row + 3) * N + n] = (uint16_t)(p1 >> 16);
}

// Short channels (K <= 1024, up to 16 rows): one tile of weight rows per
// workgroup, its 4 wavefronts taking two channel tiles at most, all requested at
// once; all of x waits in LDS, [row][channel], rows past M reading 256 zero bytes.
// 1 x 256 x 4096: 2.8 us against 4.4 on the kernel below; 4 x 1024 x 12288: 5.0
// against 5.5.
constexpr int kShortTiles = 8;            // channel tiles
constexpr int kShortWaves = 4;

template <int GROUPS, bool ZEROS>
__global__ void __launch_bounds__(64 * kShortWaves)
w4_short_kernel(const uint16_t* __restrict__ x, const char* __restrict__ packed, int64_t meta_at, int64_t M,
                int64_t N, int64_t K, uint16_t* __restrict__ y) {
  using MetaT = Meta<GROUPS, ZEROS>;
  constexpr int W = kShortWaves, kPer = kShortTiles / W, kX = kShortTiles * 16 * 16 / (64 * W);
  __shared__ u32x4 lds[16 + kShortTiles * 16 * 16];     // zeros, x [M][channel tiles * 16]; then the join
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const int tiles_k = (int)((K + 127) / 128), units = tiles_k * 16, real = (int)(K / 8);   // 16-byte units of a row
  const int64_t nt = folded_block();
  if (nt >= (N + 15) / 16) return;
  const u32x4* wp = reinterpret_cast<const u32x4*>(packed) + nt * tiles_k * 64 + lane;
  const MetaT* sp = reinterpret_cast<const MetaT*>(packed + meta_at) + nt * tiles_k * 16 + col;
  // x is requested first, then the weights, all of them whatever they fetch
  // (past the end: zeros of x, the last weight tile again), so that each wait
  // is for what it needs only.
  const __amdgpu_buffer_rsrc_t xr0 = make_rsrc(x, M * K * 2);
  u32x4 xv[kX];
#pragma unroll
  for (int i = 0; i < kX; ++i) {
    const int at = (int)threadIdx.x + 64 * W * i, m = at / units, u = at - m * units;
    xv[i] = buf_load16(xr0, u < real ? (uint32_t)(m * (int)K + 8 * u) * 2u : kOobOffset);
  }
  u32x4 w[kPer][1];
  MetaT s[kPer][1];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int kt = wave + W * i < tiles_k ? wave + W * i : tiles_k - 1;
    w[i][0] = wp[kt * 64];
    s[i][0] = sp[kt * 16];
  }
  if (threadIdx.x < 16) lds[threadIdx.x] = (u32x4){0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < kX; ++i) {
    const int at = (int)threadIdx.x + 64 * W * i;
    if (at < (int)M * units) lds[16 + at] = xv[i];
  }
  barrier_lds();
  const u32x4* const row = col < (int)M ? lds + 16 + col * units : lds;
  const int step = col < (int)M ? 16 : 0;
  f32x4 total[1][1] = {{{0, 0, 0, 0}}};
  const WidenConst wc = widen_const();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int kt = wave + W * i;
    if (kt < tiles_k) {
      const u32x4* const xr = row + kt * step + quad;
      tile_step<1, 1, GROUPS, ZEROS>(wc, w[i], s[i], [&](int, int j) { return xr[4 * j]; }, total);
    }
  }
  __syncthreads();
  f32x4* const red = reinterpret_cast<f32x4*>(lds);
  if (wave > 0) red[(wave - 1) * 64 + lane] = total[0][0];
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int i = 0; i < W - 1; ++i) total[0][0] += red[i * 64 + lane];
  store_column(total[0][0], y, 4 * quad, M, 16 * nt + col, N);
}

// The rest: 16 NT NW weight rows per workgroup and XR rows of x.  Every step
// brings 128 KW channels of x into LDS, whole rows at a time (an operand load
// straight from memory would read 16 rows one row length apart, i.e. mostly one
// memory channel), and the NW x KW wavefronts take NT weight tiles and 128
// channels each.  Weights are requested four steps before they are used.
//
// What bounds it: at 8 rows a wavefront issues 50 vector instructions for each KiB
// of weights with groups of 128 (32 of them widen the codes, the least this form
// needs) and 61 with groups of 64 and zero points; 1 x 4096 x 24576 takes 11.5 us
// (4.5 TB/s).  From 32 rows on LDS reads and the matrix cores' share grow instead:
// 64 x 4096 x 12288 takes 17.6 us.
template <int XR, int NT, int NW, int KW, int GROUPS, bool ZEROS>
__global__ void __launch_bounds__(64 * NW * KW)
w4_rows_kernel(const uint16_t* __restrict__ x, const char* __restrict__ packed, int64_t meta_at, int64_t M,
               int64_t N, int64_t K, uint16_t* __restrict__ y) {
  using MetaT = Meta<GROUPS, ZEROS>;
  constexpr int MT = XR < 16 ? 1 : XR / 16, kRows = XR; // with 8 rows, operand rows 8 to 15 repeat them, unused
  constexpr int kThreads = 64 * NW * KW, kRowThreads = 16 * KW;           // threads along a row of a step
  constexpr int kLoads = kRows * kRowThreads / kThreads, kRowStep = kThreads / kRowThreads;
  static_assert(kLoads >= 1 && kRows % kRowStep == 0, "whole rows per load");
  constexpr int kJoin = NW * (KW / 2) * MT * NT * 64;
  // x in two buffers, [KW channel tiles][row][16 units, swizzled]: one barrier
  // per step.
  constexpr int kBuf = kRows * kRowThreads;
  __shared__ u32x4 lds[2 * kBuf > kJoin ? 2 * kBuf : kJoin];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const int64_t tiles_n = (N + 15) / 16, tiles_k = (K + 127) / 128;
  const int nw = wave / KW, kg = wave % KW;
  const int64_t nt0 = (folded_block() * NW + nw) * NT, m0 = (int64_t)blockIdx.y * kRows;
  const u32x4* wp[NT];
  const MetaT* sp[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t nt = nt0 + t < tiles_n ? nt0 + t : tiles_n - 1;        // past the end: read the last, store nothing
    wp[t] = reinterpret_cast<const u32x4*>(packed) + nt * tiles_k * 64 + lane;
    sp[t] = reinterpret_cast<const MetaT*>(packed + meta_at) + nt * tiles_k * 16 + col;
  }
  constexpr int kAhead = 4;                             // steps of weights requested ahead,
  // and of x; at 16 rows x 64 weight rows two steps took 9.1 us where one took 9.8
  // (16 x 4096 x 12288, groups of 128).  With groups of 32 two steps spill; at other
  // rows two were slower or spilled.
  constexpr int kAheadX = XR == 8 ? 4 : XR == 16 && NT == 2 && GROUPS < 4 ? 2 : 1;
  u32x4 w[kAhead][NT], xv[kAheadX][kLoads];
  MetaT s[kAhead][NT];
  auto load_w = [&](int b, int64_t tile) {
    const int64_t kt = tile < tiles_k ? tile : tiles_k - 1;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      w[b][t] = wp[t][kt * 64];
      s[b][t] = sp[t][kt * 16];
    }
  };
  // Thread i brings unit i % kRowThreads (8 channels) of rows i / kRowThreads + kRowStep n.
  const int lr = threadIdx.x / kRowThreads, lu = threadIdx.x % kRowThreads;
  // Every load is issued whatever it fetches (rows past M and channels past K
  // read as zeros through the buffer's range, weights past the end fetch the
  // last tile again): a load under a condition would make the compiler wait for
  // all loads in flight where it waits for one.
  const __amdgpu_buffer_rsrc_t xr0 = make_rsrc(x + m0 * K, (M - m0 < kRows ? M - m0 : kRows) * K * 2);
  auto load_x = [&](int b, int64_t step) {
    const int64_t k = 128 * KW * step + 8 * lu;
#pragma unroll
    for (int n = 0; n < kLoads; ++n)
      xv[b][n] = buf_load16(xr0, k < K ? (uint32_t)((lr + kRowStep * n) * K + k) * 2u : kOobOffset);
  };
  auto put_x = [&](int b, int64_t step) {
    u32x4* const to = lds + (step & 1) * kBuf;
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
      const int row = lr + kRowStep * n;
      to[((lu >> 4) * kRows + row) * 16 + ((lu & 15) ^ (row & 15))] = xv[b][n];
    }
  };
  f32x4 total[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) total[m][t] = (f32x4){0, 0, 0, 0};
  const int64_t steps = (tiles_k + KW - 1) / KW;
  const WidenConst wc = widen_const();
#pragma unroll
  for (int b = 0; b < kAheadX; ++b) load_x(b, b);
#pragma unroll
  for (int b = 0; b < kAhead; ++b) load_w(b, KW * b + kg);
  put_x(0, 0);
  load_x(0, kAheadX);
  barrier_lds();
  auto step = [&](int64_t i, auto buf) {
    constexpr int b = decltype(buf)::value;
    put_x((b + 1) % kAheadX, i + 1);
    load_x((b + 1) % kAheadX, i + 1 + kAheadX);
    const u32x4* const xr = lds + (i & 1) * kBuf + (kg * kRows + (col & (kRows - 1) & 15)) * 16;
    // Past the last tile x is zeros and adds nothing.
    tile_step<MT, NT, GROUPS, ZEROS>(wc, w[b], s[b], [&](int m, int j) { return xr[m * 256 + ((4 * j + quad) ^ (col & (kRows - 1) & 15))]; },
                                     total);
    load_w(b, KW * (i + kAhead) + kg);
    barrier_lds();
  };
  for (int64_t i = 0; i < steps; i += kAhead) {
    step(i, std::integral_constant<int, 0>{});
    step(i + 1, std::integral_constant<int, 1>{});
    step(i + 2, std::integral_constant<int, 2>{});
    step(i + 3, std::integral_constant<int, 3>{});
  }
  // Joined over the channel parts, halving them each time.
  f32x4* const red = reinterpret_cast<f32x4*>(lds);
#pragma unroll
  for (int half = KW / 2; half >= 1; half /= 2) {
    __syncthreads();
    if (kg >= half && kg < 2 * half) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) red[(((nw * half + kg - half) * MT + m) * NT + t) * 64 + lane] = total[m][t];
    }
    __syncthreads();
    if (kg < half) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) total[m][t] += red[(((nw * half + kg) * MT + m) * NT + t) * 64 + lane];
    }
  }
  if (kg != 0) return;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t)
      store_column(total[m][t], y, m0 + 16 * m + 4 * quad, m0 + XR < M ? m0 + XR : M, 16 * (nt0 + t) + col, N);
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

template <int XR, int NT, int NW, int KW>
hipError_t launch_rows(const uint16_t* x, const char* packed, int64_t meta_at, int64_t M, int64_t N, int64_t K,
                       int group, bool zeros, uint16_t* y, hipStream_t stream) {
  constexpr int kN = 16 * NT * NW;
  const dim3 grid = folded_grid((N + kN - 1) / kN, (unsigned)((M + XR - 1) / XR));
  auto* k = group == 128  ? (zeros ? &w4_rows_kernel<XR, NT, NW, KW, 1, true> : &w4_rows_kernel<XR, NT, NW, KW, 1, false>)
            : group == 64 ? (zeros ? &w4_rows_kernel<XR, NT, NW, KW, 2, true> : &w4_rows_kernel<XR, NT, NW, KW, 2, false>)
                          : (zeros ? &w4_rows_kernel<XR, NT, NW, KW, 4, true> : &w4_rows_kernel<XR, NT, NW, KW, 4, false>);
  return launch(k, grid, dim3(64 * NW * KW), stream, x, packed, meta_at, M, N, K, y);
}

}  // namespace

hipError_t launch_w4_linear(const uint16_t* x, const void* packed, int64_t M, int64_t N, int64_t K, int group,
                            bool zeros, uint16_t* y, hipStream_t stream) {
  const int64_t meta_at = w4_tiles(N, K) * 1024;
  const char* p = static_cast<const char*>(packed);
  const int64_t tiles_k = (K + 127) / 128, tiles_n = (N + 15) / 16;
  if (M <= 16 && tiles_k <= kShortTiles) {
    auto* k = group == 128  ? (zeros ? &w4_short_kernel<1, true> : &w4_short_kernel<1, false>)
              : group == 64 ? (zeros ? &w4_short_kernel<2, true> : &w4_short_kernel<2, false>)
                            : (zeros ? &w4_short_kernel<4, true> : &w4_short_kernel<4, false>);
    return launch(k, folded_grid(tiles_n), dim3(64 * kShortWaves), stream, x, p, meta_at, M, N, K, y);
  }
  // Weight rows per workgroup: as few as give each CU one workgroup, with all
  // wavefronts along the channels; more once there are enough, which reads x
  // less often, or with few channels, whose steps the loop rounds up to four.
  // Rows of x per workgroup: 64, which reads the weights least often, where that
  // makes a workgroup per CU.  Either way round at the other's sizes (us a call on
  // the GPU in a captured run, groups of 64 without zero points, weights and scales
  // of 600 MB in turn):
  //   1 x 12288 x 4096:  16 rows 10.5, 32 rows 12.8;  1 x 12288 x 4099: 16.7, 12.6;
  //   1 x 4096 x 4096:   16 rows 5.5, 32 rows 6.2;    1 x 4096 x 12288: 13.6, 9.8;
  //   1 x 1536 x 4096:   16 rows 5.1, 32 rows 4.6;
  //   16 x 4096 x 8192:  16 rows 10.9, 64 rows 10.1;  16 x 4096 x 12288: 15.0, 11.0;
  //   16 x 1536 x 4096:  16 rows 6.0, 64 rows 6.1;    16 x 1536 x 4099: 7.6, 6.1;
  //   32 x 4096 x 4096:  32 rows 9.3, 64 rows 11.5;   32 x 4096 x 12288: 16.7, 14.3;
  //   32 weight rows of 32 x rows, 64 of 32, 64 of 64:
  //   64 x 4096 x 4096:  9.6, 11.7, 18.0;    64 x 4096 x 12288:  24.3, 24.6, 21.1;
  //   128 x 4096 x 4096: 15.2, 12.5, 18.5;   128 x 4096 x 8192:  30.1, 26.0, 21.5;
  //   256 x 4096 x 4096: 28.3, 24.7, 20.8;   1024 x 4096 x 4096: 99, 85, 72.
  // (1 x 12288 x 4099 makes 257 workgroups of 16 rows: with groups of 64 they have
  // 145 registers, so a CU holds one, and the last waits for a second round; with
  // groups of 128 there is room for two and they take 12.7.)
  const bool deep = tiles_k > 16;
  if (M <= 8)
    return tiles_n <= 256 && deep ? launch_rows<8, 1, 1, 8>(x, p, meta_at, M, N, K, group, zeros, y, stream)
                                  : launch_rows<8, 1, 2, 4>(x, p, meta_at, M, N, K, group, zeros, y, stream);
  if (M <= 16)
    return tiles_n <= (deep ? 512 : 256) ? launch_rows<16, 1, 1, 8>(x, p, meta_at, M, N, K, group, zeros, y, stream)
                                         : launch_rows<16, 2, 2, 4>(x, p, meta_at, M, N, K, group, zeros, y, stream);
  if (tiles_n <= 512 && (M + 63) / 64 * ((tiles_n + 3) / 4) < 256)
    return launch_rows<32, 1, 2, 4>(x, p, meta_at, M, N, K, group, zeros, y, stream);
  if (M <= 32) return launch_rows<32, 2, 2, 4>(x, p, meta_at, M, N, K, group, zeros, y, stream);
  return launch_rows<64, 2, 2, 4>(x, p, meta_at, M, N, K, group, zeros, y, stream);
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
