// rtl_dense_linear: the dense baseline Y = X W^T on gfx950's dense bf16
// matrix cores (v_mfma_f32_16x16x32_bf16), fp32 accumulation, bf16 output.
// This is the denominator of the speedups the RT-Lynx pages quote against
// dense GEMM (qingkeai article, section 05).  It shares the tiling, the W
// ring in LDS, the step structure and the tile order of the structured-
// sparse kernel, so that the two differ only in the A operand and the
// matrix instruction.
//
// The A tile (256 tokens x 64 channels of X per step) goes through LDS in
// the same swizzled row-major layout as W, copied by the same DMA routine,
// in a 2-stage ring next to the 3-stage W ring (96 + 64 KiB of LDS).
//
// A second form serves the layer's backward pass (G W, launch_grad_gemm):
// an fp32 result in blocks of 16 x 16, 1 KiB each, in the order in which the
// matrix core leaves them with its operands swapped, so the stores, and the
// loads of the kernel that follows, are contiguous.  Every 64 rows of W enter
// LDS in the order that gives a lane 16 consecutive columns over four blocks
// (lane l, block t of 4: row l % 16 of X, columns 16 (l / 16) + 4 t + [0, 4)).
// While the result is in registers its share of D, the sum over a token's kept
// channels of x G W, is taken too.  192-column tiles, and ranges of the
// contraction where the tiles alone leave CUs idle.
#include <type_traits>

#include "gemm_common.hpp"
#include "rtl_checkpoint.hpp"
#include "rtl_kernels.hpp"
#include "rtl_operators.hpp"

namespace rtl {

namespace {

// 8 wavefronts (2 x 4), each 128 x 64 = 8 x 4 blocks of 16 x 16: two per
// SIMD, so that one wave's matrix instructions run while the other waits on
// its LDS reads or at the barrier.  (With 4 wavefronts of 128 x 128 the
// matrix cores idled through every such wait and a step took 30 % longer.)
constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;

// The tiled form's W copy: LDS row R = 16 t + 4 q + e of every 64 holds W's row
// 16 q + 4 t + e.  Instruction I fills LDS rows 8 I + [0, 8), lane l's row being
// 8 I + l / 8, so W's row is a per-lane part, 16 ((l / 8) / 4) + (l / 8) % 4,
// and a uniform part of I.  NI instructions per wavefront (gemm_common.hpp's
// dma_w_tile_asm with these rows; the same hazards and waits).
__device__ __forceinline__ uint32_t w_row_of_instruction(uint32_t I) {
  return 64 * (I >> 3) + 32 * (I & 1) + 4 * ((I >> 1) & 3);
}
__device__ __forceinline__ WTileOffsets w_order_offsets(int64_t K, int64_t n0) {
  const int lane = threadIdx.x & 63, lr = lane >> 3;
  WTileOffsets o;
  o.k_lane = 8 * ((lane & 7) ^ lr);
  o.base = (uint32_t)(((n0 + 16 * (lr >> 2) + (lr & 3)) * K + o.k_lane) * 2);
  o.row8 = 0;
  return o;
}
template <int NI>
__device__ __forceinline__ void dma_w_ordered_asm(__amdgpu_buffer_rsrc_t wr, const WTileOffsets& o, int64_t K,
                                                  int64_t k0, uint32_t lds_stage_addr, bool guard_k) {
  static_assert(NI == 3 || NI == 4, "192 or 256 rows");
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t soff = __builtin_amdgcn_readfirstlane((uint32_t)(k0 * 2));
  const bool chunk_ok = !guard_k || k0 + o.k_lane + 8 <= K;
  uint32_t v[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const uint32_t row = __builtin_amdgcn_readfirstlane(w_row_of_instruction(NI * wave + i) * (uint32_t)(K * 2));
    v[i] = chunk_ok ? o.base + row : kOobOffset - soff;
  }
  const uint32_t l0 = __builtin_amdgcn_readfirstlane(lds_stage_addr + 1024u * NI * wave);
  uint32_t saved;
  if constexpr (NI == 4) {
    asm volatile(
        "s_nop 4\n\t"
        "s_mov_b32 %[sv], m0\n\t"
        "s_mov_b32 m0, %[l0]\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %[v0], %[rs], %[so] offen lds\n\t"
        "s_mov_b32 m0, %[l1]\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %[v1], %[rs], %[so] offen lds\n\t"
        "s_mov_b32 m0, %[l2]\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %[v2], %[rs], %[so] offen lds\n\t"
        "s_mov_b32 m0, %[l3]\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %[v3], %[rs], %[so] offen lds\n\t"
        "s_mov_b32 m0, %[sv]"
        : [sv] "=&s"(saved)
        : [v0] "v"(v[0]), [v1] "v"(v[1]), [v2] "v"(v[2]), [v3] "v"(v[NI - 1]), [rs] "s"(wr), [so] "s"(soff),
          [l0] "s"(l0), [l1] "s"(l0 + 0x400u), [l2] "s"(l0 + 0x800u), [l3] "s"(l0 + 0xc00u)
        : "memory");
  } else {
    asm volatile(
        "s_nop 4\n\t"
        "s_mov_b32 %[sv], m0\n\t"
        "s_mov_b32 m0, %[l0]\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %[v0], %[rs], %[so] offen lds\n\t"
        "s_mov_b32 m0, %[l1]\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %[v1], %[rs], %[so] offen lds\n\t"
        "s_mov_b32 m0, %[l2]\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %[v2], %[rs], %[so] offen lds\n\t"
        "s_mov_b32 m0, %[sv]"
        : [sv] "=&s"(saved)
        : [v0] "v"(v[0]), [v1] "v"(v[1]), [v2] "v"(v[2]), [rs] "s"(wr), [so] "s"(soff), [l0] "s"(l0),
          [l1] "s"(l0 + 0x400u), [l2] "s"(l0 + 0x800u)
        : "memory");
  }
  (void)saved;
}

// The tiled form's result and what it needs to form D.
struct GradOut {
  float* p;
  float* d_part;
  Ckpt ck;
  int64_t blocks_n;                      // 16-column blocks of a row of p
  int64_t splits;                        // ranges of the contraction
};

// KM: how channel tails are handled.  TN: tile columns, 256 or 192.  TILED: fp32
// result in 16 x 16 blocks [M / 16][4 (N / 64)][lane][4] instead of a bf16
// row-major one.  256 columns: 2 x 4 wavefronts of 128 x 64; 192: 4 x 2 of
// 64 x 96 (160 rows of operands read from LDS per step instead of the 176 of
// 2 x 4; measured alike).
template <int KM, int TN, bool TILED>
__global__ void __launch_bounds__(kThreads, 1)
dense_gemm_kernel(const uint16_t* __restrict__ x, const uint16_t* __restrict__ w,
                  int64_t M, int64_t N, int64_t K, std::conditional_t<TILED, GradOut, uint16_t* __restrict__> y) {
  static_assert(TN == 256 || (TN == 192 && TILED), "192 columns: the tiled form only");
  static_assert(!TILED || KM != kAligned8, "the tiled form copies 16 bytes");
  constexpr int kWavesN = TN == 256 ? 4 : 2, kWavesM = kWaves / kWavesN;
  constexpr int kTileN = TN, kWaveM = kTileM / kWavesM, kWaveN = TN / kWavesN;
  constexpr int kRB = kWaveM / 16, kCB = kWaveN / 16;
  constexpr int kWBytes = kTileN * kTileK * 2;
  constexpr int kWStages = 3, kAStages = 2;
  // One LDS block: the W ring, then the A ring; the epilogue reuses all of it.
  constexpr int kLdsBytes = kWStages * kWBytes + kAStages * kTileBytes;
  static_assert(store_lds_bytes<kRB, kCB>(kWaves) <= kLdsBytes, "store staging must fit in the rings");
  __shared__ __attribute__((aligned(16))) char lds[kLdsBytes];
  char* const lds_w = lds;
  char* const lds_a = lds + kWStages * kWBytes;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);   // uniform: scalar addressing
  const int wm = wave / kWavesN, wn = wave % kWavesN;
  const int64_t tiles_m = (M + kTileM - 1) / kTileM, tiles_n = (N + kTileN - 1) / kTileN;
  int64_t tm, tn;
  // Tiled form: [k_lo, k_lo + ksteps) is this workgroup's range of the steps.
  int64_t k_lo = 0, ksteps = (K + kTileK - 1) / kTileK, split = 0;
  if constexpr (TILED) {
    const int64_t tiles = tiles_m * tiles_n, per = (ksteps + y.splits - 1) / y.splits;
    split = blockIdx.x / tiles;
    tile_coords_of(blockIdx.x - split * tiles, tiles_m, tiles_n, tm, tn);
    k_lo = split * per;
    ksteps = ksteps - k_lo < per ? ksteps - k_lo : per;
  } else {
    tile_coords(tiles_m, tiles_n, tm, tn);
  }
  const int64_t n0 = tn * kTileN;
  const int64_t m0 = tm * kTileM;

  f32x4 acc[kRB][kCB];
#pragma unroll
  for (int i = 0; i < kRB; ++i)
#pragma unroll
    for (int j = 0; j < kCB; ++j) acc[i][j] = (f32x4){0, 0, 0, 0};

  // Rows past M / N lie past the end of X / W and read as zeros; channels
  // past K are pointed out of range in the tail modes.
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(x, M * K * 2);
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(w, N * K * 2);
  const WTileOffsets xo = w_tile_offsets<kWaves>(K, m0);
  const WTileOffsets wo = TILED ? w_order_offsets(K, n0) : w_tile_offsets<kWaves>(K, n0);
  const uint32_t f0 = frag_lane_offset(0), f1 = frag_lane_offset(1);
  const char* b_base0 = lds_w + wn * kCB * 2048 + f0;
  const char* b_base1 = lds_w + wn * kCB * 2048 + f1;
  const char* a_base0 = lds_a + wm * kRB * 2048 + f0;
  const char* a_base1 = lds_a + wm * kRB * 2048 + f1;
  constexpr int kTileOps = KM == kAligned8 ? 128 / kWaves : TN / 64;     // of a W tile

  // Both tile copies are issued as inline-asm DMA blocks: no vector-memory
  // operation of the loop is visible to the compiler, so it inserts no
  // vmcnt waits of its own (it cannot always prove that a copy into one
  // stage does not alias the reads of another) and the explicit waits below
  // are exact.  The K % 8 == 4 mode uses the compiler-visible dword copy.
  auto copy_w = [&](int64_t step, char* dst) {
    const int64_t ks = TILED ? k_lo + step : step;
    if constexpr (KM == kAligned8) {
      dma_w_tile_dword<kWaves>(wr, N, K, n0, ks * kTileK, dst);
    } else {
      const uint32_t lds_addr = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)(dst);
      if constexpr (TILED) dma_w_ordered_asm<TN / 64>(wr, wo, K, ks * kTileK, lds_addr, KM == kAligned16);
      else dma_w_tile_asm<kWaves>(wr, wo, K, ks * kTileK, lds_addr, KM == kAligned16);
    }
  };
  auto copy_a = [&](int64_t step, char* dst) {
    const int64_t ks = TILED ? k_lo + step : step;
    if constexpr (KM == kAligned8) {
      dma_w_tile_dword<kWaves>(xr, M, K, m0, ks * kTileK, dst);
    } else {
      const uint32_t lds_addr = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)(dst);
      dma_w_tile_asm<kWaves>(xr, xo, K, ks * kTileK, lds_addr, KM == kAligned16);
    }
  };

  // Step ks: W stage ks % 3, A stage ks % 2.  Each step issues the A copy
  // of step ks + 1, then the W copy of step ks + 2, so at its top only the
  // W copy of step ks + 1 may still be in flight.
  auto step = [&](int64_t ks, auto bw_c, auto ba_c) {
    constexpr int bw = decltype(bw_c)::value;
    constexpr int ba = decltype(ba_c)::value;
    __builtin_amdgcn_sched_barrier(0);
    wait_vm<kTileOps>();
    barrier_no_fence();
    const int64_t ka = ks + 1 < ksteps ? ks + 1 : ksteps - 1;
    const int64_t kw = ks + 2 < ksteps ? ks + 2 : ksteps - 1;
    copy_a(ka, lds_a + (1 - ba) * kTileBytes);
    copy_w(kw, lds_w + (bw + 2) % kWStages * kWBytes);
    __builtin_amdgcn_sched_barrier(0);
    const char* bs0 = b_base0 + bw * kWBytes;
    const char* bs1 = b_base1 + bw * kWBytes;
    const char* as0 = a_base0 + ba * kTileBytes;
    const char* as1 = a_base1 + ba * kTileBytes;
    bf16x8 af[2][kRB];
#pragma unroll
    for (int rb = 0; rb < kRB; ++rb) {
      af[0][rb] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(as0 + rb * 2048));
      af[1][rb] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(as1 + rb * 2048));
    }
    u32x4 q0 = *reinterpret_cast<const u32x4*>(bs0);
    u32x4 q1 = *reinterpret_cast<const u32x4*>(bs1);
#pragma unroll
    for (int cb = 0; cb < kCB; ++cb) {
      const bf16x8 b0 = __builtin_bit_cast(bf16x8, q0), b1 = __builtin_bit_cast(bf16x8, q1);
      if (cb + 1 < kCB) {
        q0 = *reinterpret_cast<const u32x4*>(bs0 + (cb + 1) * 2048);
        q1 = *reinterpret_cast<const u32x4*>(bs1 + (cb + 1) * 2048);
      }
#pragma unroll
      for (int rb = 0; rb < kRB; ++rb)
        acc[rb][cb] = TILED ? __builtin_amdgcn_mfma_f32_16x16x32_bf16(b0, af[0][rb], acc[rb][cb], 0, 0, 0)
                            : __builtin_amdgcn_mfma_f32_16x16x32_bf16(af[0][rb], b0, acc[rb][cb], 0, 0, 0);
#pragma unroll
      for (int rb = 0; rb < kRB; ++rb)
        acc[rb][cb] = TILED ? __builtin_amdgcn_mfma_f32_16x16x32_bf16(b1, af[1][rb], acc[rb][cb], 0, 0, 0)
                            : __builtin_amdgcn_mfma_f32_16x16x32_bf16(af[1][rb], b1, acc[rb][cb], 0, 0, 0);
    }
  };

  copy_w(0, lds_w);
  copy_a(0, lds_a);
  copy_w(ksteps > 1 ? 1 : 0, lds_w + kWBytes);
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  int64_t ks = 0;
  for (; ks + 6 <= ksteps; ks += 6) {
    step(ks + 0, I0{}, I0{});
    step(ks + 1, I1{}, I1{});
    step(ks + 2, I2{}, I0{});
    step(ks + 3, I0{}, I1{});
    step(ks + 4, I1{}, I0{});
    step(ks + 5, I2{}, I1{});
  }
  // 0 to 5 steps left (K need not be a multiple of 384).
  if (ks < ksteps) step(ks + 0, I0{}, I0{});
  if (ks + 1 < ksteps) step(ks + 1, I1{}, I1{});
  if (ks + 2 < ksteps) step(ks + 2, I2{}, I0{});
  if (ks + 3 < ksteps) step(ks + 3, I0{}, I1{});
  if (ks + 4 < ksteps) step(ks + 4, I1{}, I0{});
  __builtin_amdgcn_sched_barrier(0);
  wait_vm<0>();
  barrier_no_fence();                     // every wave is done with the rings

  if constexpr (TILED) {
    const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
    const int64_t mb = (m0 + wm * kWaveM) / 16, nb = (n0 + wn * kWaveN) / 16;
    f32x4* const out = reinterpret_cast<f32x4*>(y.p) + (split * ((M + 15) / 16) + mb) * y.blocks_n * 64 + lane;
    float* const red = reinterpret_cast<float*>(lds);                     // [wavefront column][256 tokens]
    // Blocks of 64 columns that this wavefront's columns lie in (whole or part).
    constexpr int kGroups = kCB / 4 + (kCB % 4 != 0);
    // All of the checkpoint's loads go out first, then P's stores, so the sums
    // wait for neither.
    const CkptRsrc ck = ckpt_rsrc(y.ck, M, N);
    Ckpt16 f[kRB][kGroups];
#pragma unroll
    for (int rb = 0; rb < kRB; ++rb) {
      const CkptRow row = ckpt_row(16 * (mb + rb) + col, N);
#pragma unroll
      for (int q = 0; q < kGroups; ++q)
        f[rb][q] = ckpt_load16(ck, row, (int)(64 * ((nb >> 2) + q) + 16 * quad), (int)N);
    }
#pragma unroll
    for (int rb = 0; rb < kRB; ++rb)
#pragma unroll
      for (int cb = 0; cb < kCB; ++cb)
        if (16 * (mb + rb) < M && nb + cb < y.blocks_n) out[(rb * y.blocks_n + nb + cb) * 64] = acc[rb][cb];
    // nb % 4 is 0, or 2 for the second wavefront column of a 192-column tile.
    const bool whole = kCB % 4 == 0 || (nb & 3) == 0;
#pragma unroll
    for (int rb = 0; rb < kRB; ++rb) {
      float part[kGroups];
#pragma unroll
      for (int q = 0; q < kGroups; ++q) {
        part[q] = 0.f;
        ckpt_clip16(f[rb][q], (int)(64 * ((nb >> 2) + q) + 16 * quad), (int)N);
      }
      if (whole) {
#pragma unroll
        for (int cb = 0; cb < kCB; ++cb) part[cb / 4] += ckpt_kept_dot(f[rb][cb / 4], cb % 4, acc[rb][cb]);
      } else {
#pragma unroll
        for (int cb = 0; cb < kCB; ++cb)
          part[(cb + 2) / 4 % kGroups] += ckpt_kept_dot(f[rb][(cb + 2) / 4 % kGroups], (cb + 2) % 4, acc[rb][cb]);
      }
      float d = 0.f;
#pragma unroll
      for (int q = 0; q < kGroups; ++q) d += __builtin_amdgcn_ldexpf(part[q], (int)f[rb][q].exp - 133);
      d += __shfl_xor(d, 16, 64);
      d += __shfl_xor(d, 32, 64);
      if (quad == 0) red[wn * kTileM + wm * kWaveM + 16 * rb + col] = d;
    }
    __syncthreads();
    const int64_t m = m0 + threadIdx.x;
    if (threadIdx.x < kTileM && m < M) {
      float d = 0.f;
#pragma unroll
      for (int v = 0; v < kWavesN; ++v) d += red[v * kTileM + threadIdx.x];
      y.d_part[(split * tiles_n + tn) * M + m] = d;
    }
  } else if (N % 8 == 0) {
    store_tile_via_lds<kRB, kCB>(acc, lds, y, M, N, m0 + wm * kWaveM, n0 + wn * kWaveN);
  } else {
    store_acc_bf16<kRB, kCB>(acc, y, M, N, m0 + wm * kWaveM, n0 + wn * kWaveN);
  }
}

}  // namespace

hipError_t launch_dense_gemm(const uint16_t* x, const uint16_t* w, int64_t M, int64_t N,
                             int64_t K, uint16_t* y, hipStream_t stream) {
  const int64_t tiles = ((M + kTileM - 1) / kTileM) * ((N + kTileN - 1) / kTileN);
  const dim3 grid((unsigned)tiles), block(kThreads);
  // 16 x 16 blocks: a form of the same loop on v_mfma_f32_32x32x16_bf16
  // (4 x 2 blocks of 32 x 32 per wavefront) measured 8 % slower (253
  // against 235 us at M = 4096, K = 3072, N = 12288).
  auto* k = K % kTileK == 0 ? &dense_gemm_kernel<kFullK, 256, false>
            : K % 8 == 0   ? &dense_gemm_kernel<kAligned16, 256, false>
                           : &dense_gemm_kernel<kAligned8, 256, false>;
  return launch(k, grid, block, stream, x, w, M, N, K, y);
}

hipError_t launch_grad_gemm(const uint16_t* g, const uint16_t* w_t, const Ckpt& ck, const BackwardLayout& L, float* p,
                            float* d_part, hipStream_t stream) {
  const int64_t M = L.M, N = L.K, K = L.p_length;       // result columns N, contraction K
  const GradOut out{p, d_part, ck, L.kp / 16, L.p_splits};
  const dim3 grid((unsigned)((M + kTileM - 1) / kTileM * L.p_tiles * L.p_splits)), block(kThreads);
  auto* k = L.p_tile == 192 ? (K % kTileK == 0 ? &dense_gemm_kernel<kFullK, 192, true>
                                               : &dense_gemm_kernel<kAligned16, 192, true>)
            : K % kTileK == 0 ? &dense_gemm_kernel<kFullK, 256, true>
                              : &dense_gemm_kernel<kAligned16, 256, true>;
  return launch(k, grid, block, stream, g, w_t, M, N, K, out);
}

}  // namespace rtl
