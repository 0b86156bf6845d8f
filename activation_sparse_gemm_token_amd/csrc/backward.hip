// rtl_sparse_linear_backward (include/rtlynx_train.h).
//
// The work is one large product, G W [M, K] over N channels, which runs on the
// dense GEMM's ring (dense_gemm.hip) unless the tokens are few, and the LoRA
// branch, whose products all have one dimension of at most 128 and are bound by
// reading G and the checkpoint:
//
//   1. factors_kernel       A and B as matrix-core fragments, zero-padded.
//   2. rows_kernel          G B, and of the checkpoint (pruned A^T) and (kept
//                           A^T): token-by-rank products over the channels.
//   3. join_rows_kernel     sums the channel ranges in order, forms U = alpha G B,
//                           T = alpha (pruned A^T + (1 - s) kept A^T) and the part
//                           of D that needs no G W, and writes U, (1 - s) U and T in
//                           the lane order of the products that follow, in fp32.
//   4. columns_kernel       G^T T and [pruned; kept]^T [U; (1 - s) U]: products over
//                           the tokens.  Both operands run along tokens, which are
//                           rows in memory: the tile goes through LDS and is read
//                           transposed (ds_read_b64_tr_b16).
//   5. join_columns         sums the token ranges in order into dA and dB (a kernel
//                           of its own where dX is not asked for, else part of 7).
//   6. the dense GEMM       P = G W, in 16 x 16 blocks of fp32, and of each tile
//      or few_tokens_kernel its share of D.
//   7. finish_kernel        D per token, then dX; U A is formed again, a 16-token
//                           strip at a time, on the matrix cores (r is small), so it
//                           never goes to memory.
//
// A kept value's residual (1 - s) x is not a bf16 number; multiplying U (or the
// joined sum) by 1 - s instead keeps the checkpoint's values exact operands.
//
// At 4096 x 3072 x 12288, r = 64 (us, inputs changing from call to call): factors 5,
// rows 43, join 7, columns 49, G W 250 to 275 as the clock drops, dX with the sums of
// dA and dB 29 (27 and, in a launch of their own, 7.6).  Rows and columns read G
// (100 MB) and the checkpoint (14 MB), 22 us at the card's copy rate, and their
// factors' fragments from L2 as often as that.
//
// Fragments instead of transposed matrices: a matrix whose rows are N channels
// apart puts the 16 rows of an operand load on one memory channel; as 1 KiB
// blocks in the order of use every such load is contiguous.
#include "rtl_checkpoint.hpp"
#include "rtl_common.hpp"
#include "rtl_operators.hpp"

namespace rtl {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));

// 8 fp32 values of a lane as three operands of bf16 whose sum they are: each
// word takes the value's next 8 of 24 significant bits (cut off, not rounded, so
// every remainder is exact).  U and T are sums, so they keep fp32's bits between
// the products; held in two words (16 bits) they turned ten times as many last
// bits of the results as fp32's own rounding does.  They travel as fp32, no more
// bytes than two words, and are split where they are used.
struct Words {
  u32x4 w[3];
};
__device__ __forceinline__ Words split24(u32x4 first, u32x4 last) {
  Words r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t a = i < 2 ? first[2 * i] : last[2 * i - 4], b = i < 2 ? first[2 * i + 1] : last[2 * i - 3];
#pragma unroll
    for (int n = 0; n < 3; ++n) {
      r.w[n][i] = __builtin_amdgcn_perm(b, a, 0x07060302u);
      a = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) - __builtin_bit_cast(float, a & 0xffff0000u));
      b = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, b) - __builtin_bit_cast(float, b & 0xffff0000u));
    }
  }
  return r;
}
__device__ __forceinline__ u32x4 raw4(const float* v) {
  return (u32x4){__builtin_bit_cast(uint32_t, v[0]), __builtin_bit_cast(uint32_t, v[1]),
                 __builtin_bit_cast(uint32_t, v[2]), __builtin_bit_cast(uint32_t, v[3])};
}

// 8 channels at channel c of a row of C (C % 4 == 0) of a bf16 tensor, `row` its
// byte offset; zeros past C and past the tensor.  Rows are 16-byte aligned when
// WIDE (C % 8 == 0), else 8-byte, with half a unit at the end.
template <bool WIDE>
__device__ __forceinline__ u32x4 load8(__amdgpu_buffer_rsrc_t t, uint32_t row, int c, int C) {
  if constexpr (WIDE) {
    return buf_load16(t, c < C ? row + 2u * c : kOobOffset);
  } else {
    const u32x2 a = buf_load8(t, c < C ? row + 2u * c : kOobOffset);
    const u32x2 b = buf_load8(t, c + 4 < C ? row + 2u * c + 8u : kOobOffset);
    return (u32x4){a[0], a[1], b[0], b[1]};
  }
}

// 8 channels of the checkpoint at channel c, raw, then pruned and kept values.
struct CkptRaw {
  u32x2 q;
  uint32_t e, p, idx;                                   // p: the pruned channels' exponent
};
template <bool WIDE>
__device__ __forceinline__ CkptRaw ckpt_load8(const CkptRsrc& k, const CkptRow& r, int c, int K) {
  CkptRaw f;
  f.q = buf_load8(k.codes, c < K ? r.codes + c : kOobOffset);
  f.e = __builtin_amdgcn_raw_buffer_load_b8(k.exps, c < K ? r.exps + c / 32 : kOobOffset, 0, 0);
  f.p = __builtin_amdgcn_raw_buffer_load_b8(k.pruned_exps, c < K ? r.exps + c / 32 : kOobOffset, 0, 0);
  f.idx = __builtin_amdgcn_raw_buffer_load_b8(k.idx, c < K ? r.idx + c / 8 : kOobOffset, 0, 0);
  return f;
}
__device__ __forceinline__ void ckpt_split(const CkptRaw& r, u32x4& pruned, u32x4& kept) {
  ckpt_split8(r.q, r.e, r.p, r.idx, pruned, kept);
}
__device__ __forceinline__ void ckpt_split(const Ckpt16& r, int half, u32x4& pruned, u32x4& kept) {
  const u32x2 q = {r.codes[2 * half], r.codes[2 * half + 1]};
  ckpt_split8(q, r.exp, r.pruned_exp, half ? r.idx1 : r.idx0, pruned, kept);
}

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

constexpr f32x4 kZero4 = {0, 0, 0, 0};

// Sums COUNT accumulators over the 4 wavefronts of a workgroup into wavefront
// 0, in the order (0 + 2) + (1 + 3).
template <int COUNT>
__device__ __forceinline__ void join_waves(f32x4* acc, f32x4* lds, int wave, int lane) {
#pragma unroll
  for (int half = 2; half >= 1; half /= 2) {
    __syncthreads();
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int i = 0; i < COUNT; ++i) lds[((wave - half) * COUNT + i) * 64 + lane] = acc[i];
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int i = 0; i < COUNT; ++i) acc[i] += lds[(wave * COUNT + i) * 64 + lane];
    }
  }
}

// --- 1. factors ------------------------------------------------------------
// One thread per lane of a fragment.  a_down [kp / 32][rp / 16]: rows ranks,
// contraction channels (in step h of every two, lanes l / 16 hold channels
// 16 (l / 16) + 8 h + [0, 8) of the 64); a_up [kp / 16][rp / 32]: rows channels in the order of
// P's blocks (row 4 q + e of block t of four: channel 16 q + 4 t + e of the 64),
// contraction ranks; b [np / 32][rp / 16]: rows ranks, contraction output channels.
__global__ void __launch_bounds__(256)
factors_kernel(const uint16_t* __restrict__ a, const uint16_t* __restrict__ b, BackwardLayout L,
               u32x4* __restrict__ a_down, u32x4* __restrict__ a_up, u32x4* __restrict__ b_down) {
  const int64_t na = L.rp * L.kp / 8, nb = L.rp * L.np / 8;
  const int64_t jt = L.rp / 16, rt = L.rp / 32;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < 2 * na + nb; i += (int64_t)gridDim.x * 256) {
    const int lane = (int)(i & 63), row = lane & 15, at = 8 * (lane >> 4);
    uint32_t v[8];
    if (i < na) {
      const int64_t f = i >> 6, j = 16 * (f % jt) + row, step = f / jt;
      const int64_t k = 64 * (step >> 1) + 2 * at + 8 * (step & 1);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = j < L.r && k + e < L.K ? a[j * L.K + k + e] : 0;
    } else if (i < 2 * na) {
      const int64_t f = (i - na) >> 6, t = f / rt, j = 32 * (f % rt) + at;
      const int64_t k = 64 * (t >> 2) + 16 * (row >> 2) + 4 * (t & 3) + (row & 3);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = j + e < L.r && k < L.K ? a[(j + e) * L.K + k] : 0;
    } else {
      const int64_t f = (i - 2 * na) >> 6, j = 16 * (f % jt) + row, n = 32 * (f / jt) + at;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = j < L.r && n + e < L.N ? b[(n + e) * L.r + j] : 0;
    }
    const u32x4 w = {v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16};
    if (i < na) a_down[i] = w;
    else if (i < 2 * na) a_up[i - na] = w;
    else b_down[i - 2 * na] = w;
  }
}

// --- 2. token-by-rank products --------------------------------------------
// A workgroup takes 16 MT tokens and a range of channels, its 4 wavefronts 64
// channels in turn; each keeps the next 64 channels' loads in flight.
template <int MT, int JT, bool WIDE>
__device__ __forceinline__ void g_rows(const uint16_t* __restrict__ g, const u32x4* __restrict__ b,
                                       const BackwardLayout& L, int64_t m0, int64_t lo, int64_t hi, f32x4* lds,
                                       float* __restrict__ out) {
  const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  struct Stage {
    u32x4 x[MT][2], w[2][JT];
  };
  f32x4 acc[MT * JT];
#pragma unroll
  for (int i = 0; i < MT * JT; ++i) acc[i] = kZero4;
  const __amdgpu_buffer_rsrc_t gr = make_rsrc(g, L.M * L.N * 2);
  const int N = (int)L.N;
  uint32_t row[MT];                                     // tokens past M lie past the end: zeros
#pragma unroll
  for (int i = 0; i < MT; ++i) row[i] = (uint32_t)((m0 + 16 * i + col) * L.N * 2);
  auto load = [&](Stage& s, int64_t c) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < MT; ++i) s.x[i][h] = load8<WIDE>(gr, row[i], (int)c + 32 * h + 8 * quad, N);
#pragma unroll
      for (int j = 0; j < JT; ++j) s.w[h][j] = b[((c / 32 + h) * JT + j) * 64 + lane];
    }
  };
  auto use = [&](const Stage& s) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < JT; ++j) acc[i * JT + j] = mfma(s.x[i][h], s.w[h][j], acc[i * JT + j]);
  };
  Stage s0, s1;
  int64_t c = lo + 64 * wave;
  if (c < hi) load(s0, c);
  for (; c + 512 < hi; c += 512) {
    load(s1, c + 256);
    use(s0);
    load(s0, c + 512);
    use(s1);
  }
  if (c + 256 < hi) {
    load(s1, c + 256);
    use(s0);
    use(s1);
  } else if (c < hi) {
    use(s0);
  }
  join_waves<MT * JT>(acc, lds, wave, lane);
  if (wave != 0) return;
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < JT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t m = m0 + 16 * i + 4 * quad + e;
        if (m < L.M) out[m * L.rp + 16 * j + col] = acc[i * JT + j][e];
      }
}

// A lane reads 16 channels of its token: its 8 of both steps of 64 channels
// (a_down has the same order).
template <int MT, int JT>
__device__ __forceinline__ void x_rows(const Ckpt& ck, const u32x4* __restrict__ a, const BackwardLayout& L,
                                       int64_t m0, int64_t lo, int64_t hi, f32x4* lds, float* __restrict__ out) {
  const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  struct Stage {
    Ckpt16 x[MT];
    u32x4 w[2][JT];
  };
  f32x4 acc[2 * MT * JT];                               // pruned, kept
#pragma unroll
  for (int i = 0; i < 2 * MT * JT; ++i) acc[i] = kZero4;
  const CkptRsrc kr = ckpt_rsrc(ck, L.M, L.K);
  const int K = (int)L.K;
  CkptRow row[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) row[i] = ckpt_row(m0 + 16 * i + col, L.K);
  auto load = [&](Stage& s, int64_t c) {
#pragma unroll
    for (int i = 0; i < MT; ++i) s.x[i] = ckpt_load16(kr, row[i], (int)c + 16 * quad, K);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < JT; ++j) s.w[h][j] = a[((c / 32 + h) * JT + j) * 64 + lane];
  };
  auto use = [&](Stage& s, int64_t c) {
#pragma unroll
    for (int i = 0; i < MT; ++i) ckpt_clip16(s.x[i], (int)c + 16 * quad, K);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        u32x4 pruned, kept;
        ckpt_split(s.x[i], h, pruned, kept);
#pragma unroll
        for (int j = 0; j < JT; ++j) {
          acc[i * JT + j] = mfma(pruned, s.w[h][j], acc[i * JT + j]);
          acc[(MT + i) * JT + j] = mfma(kept, s.w[h][j], acc[(MT + i) * JT + j]);
        }
      }
  };
  Stage s0, s1;
  int64_t c = lo + 64 * wave;
  if (c < hi) load(s0, c);
  for (; c + 512 < hi; c += 512) {
    load(s1, c + 256);
    use(s0, c);
    load(s0, c + 512);
    use(s1, c + 256);
  }
  if (c + 256 < hi) {
    load(s1, c + 256);
    use(s0, c);
    use(s1, c + 256);
  } else if (c < hi) {
    use(s0, c);
  }
  join_waves<2 * MT * JT>(acc, lds, wave, lane);
  if (wave != 0) return;
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < JT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t m = m0 + 16 * i + 4 * quad + e;
          if (m < L.M) out[(p * L.M + m) * L.rp + 16 * j + col] = acc[(p * MT + i) * JT + j][e];
        }
}

template <int JT, bool WIDE_G>
__global__ void __launch_bounds__(256, 2)
rows_kernel(const uint16_t* __restrict__ g, const u32x4* __restrict__ b, const u32x4* __restrict__ a, Ckpt ck,
            BackwardLayout L, float* __restrict__ part) {
  constexpr int kG = JT == 8 ? 2 : 4, kX = kG / 2;      // 16-token tiles per workgroup
  __shared__ f32x4 lds[2 * kG * JT * 64];
  const int64_t groups_g = (L.M + 16 * kG - 1) / (16 * kG) * L.splits_g;
  const int64_t slab = L.M * L.rp;
  int64_t id = blockIdx.x;
  if (id < groups_g) {
    const int64_t s = id % L.splits_g, lo = s * L.chunk_g, hi = lo + L.chunk_g < L.np ? lo + L.chunk_g : L.np;
    g_rows<kG, JT, WIDE_G>(g, b, L, id / L.splits_g * (16 * kG), lo, hi, lds, part + s * slab);
  } else {
    id -= groups_g;
    const int64_t s = id % L.splits_x, lo = s * L.chunk_x, hi = lo + L.chunk_x < L.kp ? lo + L.chunk_x : L.kp;
    x_rows<kX, JT>(ck, a, L, id / L.splits_x * (16 * kX), lo, hi, lds, part + (L.splits_g + 2 * s) * slab);
  }
}

// --- 3. U, T and what follows from them -------------------------------------
// 32 tokens per workgroup: one contraction step of the products over tokens.
// Tokens past M are written as zeros.  u [mp / 16][rp / 32][2]: rows tokens,
// contraction ranks; uc [mp / 32][U, (1 - s) U][rp / 16][2] and
// tc [mp / 32][rp / 16][2]: rows ranks, contraction tokens; [2] the halves of a
// lane's 8 fp32 values.
constexpr int kJoinThreads = 512;

template <int RP>
__global__ void __launch_bounds__(kJoinThreads)
join_rows_kernel(const float* __restrict__ part, const float* __restrict__ stats, BackwardLayout L, float alpha,
                 u32x4* __restrict__ u_out, u32x4* __restrict__ uc_out, u32x4* __restrict__ tc_out,
                 float* __restrict__ d_lora) {
  constexpr int kPitch = RP + 4;
  __shared__ __attribute__((aligned(16))) float us[32 * kPitch], ts[32 * kPitch], ds[32 * (RP / 4 + 1)];
  const int64_t m0 = (int64_t)blockIdx.x * 32, slab = L.M * RP;
#pragma unroll
  for (int i = threadIdx.x; i < 32 * RP / 4; i += kJoinThreads) {
    const int r = i / (RP / 4), j = 4 * (i % (RP / 4));
    const int64_t m = m0 + r;
    f32x4 u = kZero4, pr = kZero4, ke = kZero4;
    float keep = 0.f;
    if (m < L.M) {
      const float* p = part + m * RP + j;
      // Few tokens have many ranges: their loads go out 16 at a time.
#pragma unroll 16
      for (int64_t q = 0; q < L.splits_g; ++q) u += *reinterpret_cast<const f32x4*>(p + q * slab);
      p += L.splits_g * slab;
#pragma unroll 8
      for (int64_t q = 0; q < L.splits_x; ++q) {
        pr += *reinterpret_cast<const f32x4*>(p + 2 * q * slab);
        ke += *reinterpret_cast<const f32x4*>(p + (2 * q + 1) * slab);
      }
      keep = 1.f - stats[2 * m];
    }
    f32x4 t;
    float d = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      u[e] *= alpha;
      d += u[e] * ke[e];                                // of D: U (kept A^T), summed over the ranks below
      t[e] = alpha * (pr[e] + keep * ke[e]);
    }
    *reinterpret_cast<f32x4*>(us + r * kPitch + j) = u;
    *reinterpret_cast<f32x4*>(ts + r * kPitch + j) = t;
    ds[r * (RP / 4 + 1) + j / 4] = d;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    float d = 0.f;
#pragma unroll
    for (int j = 0; j < RP / 4; ++j) d += ds[threadIdx.x * (RP / 4 + 1) + j];
    d_lora[m0 + threadIdx.x] = d;
  }
  for (int i = threadIdx.x; i < 2 * (RP / 32) * 64; i += kJoinThreads) {      // u
    const int lane = i & 63, f = i >> 6, tile = f / (RP / 32), step = f % (RP / 32);
    const float* p = us + (16 * tile + (lane & 15)) * kPitch + 32 * step + 8 * (lane >> 4);
    u32x4* o = u_out + (((m0 / 16 + tile) * (RP / 32) + step) * 2) * 64 + lane;
    o[0] = raw4(p);
    o[64] = raw4(p + 4);
  }
  for (int i = threadIdx.x; i < (RP / 16) * 64; i += kJoinThreads) {          // uc, tc
    const int lane = i & 63, jt = i >> 6, j = 16 * jt + (lane & 15), r0 = 8 * (lane >> 4);
    float u[8], k[8], t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t m = m0 + r0 + e;
      u[e] = us[(r0 + e) * kPitch + j];
      k[e] = u[e] * (m < L.M ? 1.f - stats[2 * m] : 0.f);
      t[e] = ts[(r0 + e) * kPitch + j];
    }
    u32x4* o = uc_out + ((int64_t)blockIdx.x * 2 * (RP / 16) + jt) * 128 + lane;
    o[0] = raw4(u);
    o[64] = raw4(u + 4);
    o += (RP / 16) * 128;
    o[0] = raw4(k);
    o[64] = raw4(k + 4);
    o = tc_out + ((int64_t)blockIdx.x * (RP / 16) + jt) * 128 + lane;
    o[0] = raw4(t);
    o[64] = raw4(t + 4);
  }
}

// --- 4. products over tokens ------------------------------------------------
// A workgroup takes 16 CT channels and a range of tokens, its 4 wavefronts 32
// tokens in turn.  Each stages its own 32 tokens in LDS (row pitch: 16 bytes
// past the row, aligned, rows 4 banks apart) and needs no barrier.
template <int CT>
constexpr int col_pitch() { return 16 * CT + 8; }       // bf16 words

// The operand of 16 channels (from c) x 32 tokens of such a tile: lane l gets
// tokens 8 (l / 16) + [0, 8) of channel c + l % 16.  One transposing read
// gives a lane 4 tokens: its 16 lanes name 4 rows of 16 channels.
template <int CT>
__device__ __forceinline__ u32x4 transposed_operand(const uint16_t* tile, int c) {
  const int lane = threadIdx.x & 63;
  const uint16_t* p = tile + (8 * (lane >> 4) + ((lane & 15) >> 2)) * col_pitch<CT>() + c + 4 * (lane & 3);
  using lds_s16x4 = __attribute__((address_space(3))) s16x4;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p));
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * col_pitch<CT>()));
  const u32x2 a2 = __builtin_bit_cast(u32x2, a), b2 = __builtin_bit_cast(u32x2, b);
  return (u32x4){a2[0], a2[1], b2[0], b2[1]};
}

// One 32-token step of one staged tile against its factors.
template <int CT, int JT>
__device__ __forceinline__ void col_step(const uint16_t* tile, const u32x4 (&w)[2 * JT], f32x4* acc) {
  u32x4 x[CT];
#pragma unroll
  for (int i = 0; i < CT; ++i) x[i] = transposed_operand<CT>(tile, 16 * i);
#pragma unroll
  for (int j = 0; j < JT; ++j) {
    const Words s = split24(w[2 * j], w[2 * j + 1]);
#pragma unroll
    for (int n = 0; n < 3; ++n)
#pragma unroll
      for (int i = 0; i < CT; ++i) acc[i * JT + j] = mfma(x[i], s.w[n], acc[i * JT + j]);
    if constexpr (JT == 8) __builtin_amdgcn_sched_barrier(0);   // one split at a time: no registers for more
  }
}

// Where a lane's loads go in a wavefront's tile: 16 bytes of rows lr, lr +
// kRows, ...
template <int CT>
struct ColTile {
  static constexpr int kLanes = 2 * CT, kRows = 64 / kLanes, kLoads = 32 / kRows;
  static constexpr int kWords = 32 * col_pitch<CT>();
  static constexpr int kStage = 4 * kWords * 2;         // bytes, all four wavefronts
};

template <int CT, int JT, bool WIDE>
__device__ __forceinline__ void g_columns(const uint16_t* __restrict__ g, const u32x4* __restrict__ tc,
                                          const BackwardLayout& L, int64_t c0, int64_t lo, int64_t hi, char* lds,
                                          float* __restrict__ out) {
  using T = ColTile<CT>;
  const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint16_t* const tile = reinterpret_cast<uint16_t*>(lds) + wave * T::kWords;
  const int lr = lane / T::kLanes, lc = 8 * (lane % T::kLanes);
  uint16_t* const dst = tile + lr * col_pitch<CT>() + lc;
  f32x4 acc[CT * JT];
#pragma unroll
  for (int i = 0; i < CT * JT; ++i) acc[i] = kZero4;
  u32x4 v[T::kLoads], w[2 * JT];
  const __amdgpu_buffer_rsrc_t gr = make_rsrc(g, L.M * L.N * 2);
  // Past the range: its last tokens again, unused.  Tokens past M: zeros.
  auto load = [&](int64_t at) {
    const int64_t t = at < hi ? at : hi - 32;
#pragma unroll
    for (int i = 0; i < T::kLoads; ++i)
      v[i] = load8<WIDE>(gr, (uint32_t)((t + lr + T::kRows * i) * L.N * 2), (int)c0 + lc, (int)L.N);
  };
  int64_t t = lo + 32 * wave;
  load(t);
  for (; t < hi; t += 128) {
#pragma unroll
    for (int i = 0; i < 2 * JT; ++i) w[i] = tc[(t / 32 * 2 * JT + i) * 64 + lane];
#pragma unroll
    for (int i = 0; i < T::kLoads; ++i) *reinterpret_cast<u32x4*>(dst + T::kRows * i * col_pitch<CT>()) = v[i];
    load(t + 128);
    __builtin_amdgcn_wave_barrier();
    col_step<CT, JT>(tile, w, acc);
    __builtin_amdgcn_wave_barrier();
  }
  join_waves<CT * JT>(acc, reinterpret_cast<f32x4*>(lds), wave, lane);
  if (wave != 0) return;
#pragma unroll
  for (int i = 0; i < CT; ++i)
#pragma unroll
    for (int j = 0; j < JT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t n = c0 + 16 * i + 4 * quad + e;
        if (n < L.N) out[n * L.rp + 16 * j + col] = acc[i * JT + j][e];
      }
}

template <int CT, int JT, bool WIDE>
__device__ __forceinline__ void x_columns(const Ckpt& ck, const u32x4* __restrict__ uc, const BackwardLayout& L,
                                          int64_t c0, int64_t lo, int64_t hi, char* lds, float* __restrict__ out) {
  using T = ColTile<CT>;
  const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint16_t* const tile = reinterpret_cast<uint16_t*>(lds) + wave * T::kWords;
  const int lr = lane / T::kLanes, lc = 8 * (lane % T::kLanes);
  uint16_t* const dst = tile + lr * col_pitch<CT>() + lc;
  f32x4 acc[CT * JT];
#pragma unroll
  for (int i = 0; i < CT * JT; ++i) acc[i] = kZero4;
  CkptRaw v[T::kLoads];
  u32x4 w[2 * JT];
  const CkptRsrc kr = ckpt_rsrc(ck, L.M, L.K);
  auto load = [&](int64_t at) {
    const int64_t t = at < hi ? at : hi - 32;
#pragma unroll
    for (int i = 0; i < T::kLoads; ++i)
      v[i] = ckpt_load8<WIDE>(kr, ckpt_row(t + lr + T::kRows * i, L.K), (int)c0 + lc, (int)L.K);
  };
  int64_t t = lo + 32 * wave;
  load(t);
  for (; t < hi; t += 128) {
    u32x4 kept[T::kLoads];
#pragma unroll
    for (int i = 0; i < 2 * JT; ++i) w[i] = uc[(t / 32 * 4 * JT + i) * 64 + lane];
#pragma unroll
    for (int i = 0; i < T::kLoads; ++i) {
      u32x4 pruned;
      if (!WIDE) v[i].q[1] = c0 + lc + 4 < L.K ? v[i].q[1] : 0u;   // past the row: the next one's
      ckpt_split(v[i], pruned, kept[i]);
      *reinterpret_cast<u32x4*>(dst + T::kRows * i * col_pitch<CT>()) = pruned;
    }
    load(t + 128);
    __builtin_amdgcn_wave_barrier();
    col_step<CT, JT>(tile, w, acc);                     // pruned with U
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < 2 * JT; ++i) w[i] = uc[(t / 32 * 4 * JT + 2 * JT + i) * 64 + lane];
#pragma unroll
    for (int i = 0; i < T::kLoads; ++i) *reinterpret_cast<u32x4*>(dst + T::kRows * i * col_pitch<CT>()) = kept[i];
    __builtin_amdgcn_wave_barrier();
    col_step<CT, JT>(tile, w, acc);                     // kept with (1 - s) U
    __builtin_amdgcn_wave_barrier();
  }
  join_waves<CT * JT>(acc, reinterpret_cast<f32x4*>(lds), wave, lane);
  if (wave != 0) return;
#pragma unroll
  for (int i = 0; i < CT; ++i)
#pragma unroll
    for (int j = 0; j < JT; ++j) {
      const int64_t k = c0 + 16 * i + 4 * quad;
      if (k < L.K) *reinterpret_cast<f32x4*>(out + (int64_t)(16 * j + col) * L.kp + k) = acc[i * JT + j];
    }
}

// CT: 16-channel tiles of G per workgroup; half as many of the checkpoint,
// whose step needs twice the operands.
template <int CT, int JT, bool WIDE_G, bool WIDE_X>
__global__ void __launch_bounds__(256, 2)
columns_kernel(const uint16_t* __restrict__ g, Ckpt ck, const u32x4* __restrict__ uc, const u32x4* __restrict__ tc,
               BackwardLayout L, float* __restrict__ part) {
  constexpr int kJoin = 2 * CT * JT * 64 * 16;
  __shared__ __attribute__((aligned(16))) char lds[kJoin > ColTile<CT>::kStage ? kJoin : ColTile<CT>::kStage];
  const int64_t tiles_g = (L.N + 16 * CT - 1) / (16 * CT), id = blockIdx.x;
  const int64_t lo = (int64_t)blockIdx.y * L.chunk_t, hi = lo + L.chunk_t < L.mp ? lo + L.chunk_t : L.mp;
  if (id < tiles_g)
    g_columns<CT, JT, WIDE_G>(g, tc, L, 16 * CT * id, lo, hi, lds, part + (int64_t)blockIdx.y * L.N * L.rp);
  else
    x_columns<CT / 2, JT, WIDE_X>(ck, uc, L, 8 * CT * (id - tiles_g), lo, hi, lds,
                                  part + (L.splits_t * L.N + (int64_t)blockIdx.y * L.kp) * L.rp);
}

// --- 5. dA and dB -------------------------------------------------------------
// The token ranges' sums, four elements of the padded products at a time, from
// item i on.
struct Factors {
  const float* part;
  uint16_t *da, *db;                                    // null: not asked for
};
__host__ __device__ inline int64_t join_items(const BackwardLayout& L) { return (L.N * L.rp + L.r * L.kp) / 4; }

__device__ __forceinline__ void join_columns(const Factors& f, const BackwardLayout& L, int64_t i, int64_t stride) {
  const int64_t nb = L.N * L.rp, slab_a = L.rp * L.kp, all = join_items(L);
  for (; i < all; i += stride) {
    const bool b = 4 * i < nb;
    const int64_t at = b ? 4 * i : 4 * i - nb, slab = b ? nb : slab_a;
    const float* p = f.part + (b ? 0 : L.splits_t * nb) + at;
    f32x4 v = kZero4;
#pragma unroll 4
    for (int64_t s = 0; s < L.splits_t; ++s) v += *reinterpret_cast<const f32x4*>(p + s * slab);
    const u32x2 o = {cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3])};
    const int64_t row = at / (b ? L.rp : L.kp), c = at - row * (b ? L.rp : L.kp), len = b ? L.r : L.K;
    uint16_t* y = (b ? f.db : f.da) + row * len + c;
    if (len % 4 == 0) {                                 // K always is
      if (c < len) *reinterpret_cast<u32x2*>(y) = o;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < len) y[e] = (uint16_t)(o[e / 2] >> (16 * (e & 1)));
    }
  }
}

__global__ void __launch_bounds__(256) join_columns_kernel(Factors f, BackwardLayout L) {
  join_columns(f, L, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}

// --- 6. G W of few tokens -------------------------------------------------------
// The dense GEMM's tiles of 256 tokens leave most of the chip idle then, and a
// tile's start and end cost more than its products.  Here a workgroup takes 64
// tokens x 64 channels and a range of the contraction, its 4 wavefronts 64 of it
// in turn, operands straight from memory; the wavefronts' sums meet in LDS, where
// each takes 16 tokens.  P and D's shares as in the dense GEMM's form (lane: one
// token, channel 16 quad + 4 t + e of the 64 in block t).
template <bool WIDE>
__global__ void __launch_bounds__(256, 2)
few_tokens_kernel(const uint16_t* __restrict__ g, const uint16_t* __restrict__ w_t, Ckpt ck, BackwardLayout L,
                  float* __restrict__ p, float* __restrict__ d_part) {
  __shared__ f32x4 lds[4 * 16 * 64];
  const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t tiles_m = (L.M + 63) / 64, tiles = tiles_m * L.p_tiles;
  const int64_t split = blockIdx.x / tiles, id = blockIdx.x - split * tiles;
  const int64_t tn = id / tiles_m, m0 = 64 * (id - tn * tiles_m);
  const int64_t steps = (L.N + 63) / 64, per = (steps + L.p_splits - 1) / L.p_splits;
  const int64_t lo = split * per, hi = lo + per < steps ? lo + per : steps;
  const __amdgpu_buffer_rsrc_t gr = make_rsrc(g, L.M * L.N * 2), wr = make_rsrc(w_t, L.K * L.N * 2);
  const int N = (int)L.N;
  uint32_t xrow[4], wrow[4];                            // past the tensors' ends: zeros
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    xrow[i] = (uint32_t)((m0 + 16 * i + col) * L.N * 2);
    wrow[i] = (uint32_t)((64 * tn + 16 * (col >> 2) + 4 * i + (col & 3)) * L.N * 2);
  }
  struct Stage {
    u32x4 x[4][2], w[4][2];
  };
  f32x4 acc[16];                                        // [16 tokens][block]
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = kZero4;
  auto load = [&](Stage& s, int64_t t) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = (int)(64 * t) + 32 * h + 8 * quad;
        s.x[i][h] = load8<WIDE>(gr, xrow[i], c, N);
        s.w[i][h] = load8<WIDE>(wr, wrow[i], c, N);
      }
  };
  auto use = [&](const Stage& s) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[4 * i + j] = mfma(s.w[j][h], s.x[i][h], acc[4 * i + j]);
  };
  Stage s0, s1;
  int64_t t = lo + wave;
  if (t < hi) load(s0, t);
  for (; t + 8 < hi; t += 8) {
    load(s1, t + 4);
    use(s0);
    load(s0, t + 8);
    use(s1);
  }
  if (t + 4 < hi) {
    load(s1, t + 4);
    use(s0);
    use(s1);
  } else if (t < hi) {
    use(s0);
  }
  const int64_t row = m0 + 16 * wave + col;             // this wavefront's tokens from here on
  Ckpt16 f = ckpt_load16(ckpt_rsrc(ck, L.M, L.K), ckpt_row(row, L.K), (int)(64 * tn) + 16 * quad,
                         (int)L.K);
#pragma unroll
  for (int i = 0; i < 16; ++i) lds[(wave * 16 + i) * 64 + lane] = acc[i];
  __syncthreads();
  f32x4 v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = lds[(4 * wave + j) * 64 + lane];
#pragma unroll
    for (int s = 1; s < 4; ++s) v[j] += lds[(16 * s + 4 * wave + j) * 64 + lane];
  }
  const int64_t block = m0 / 16 + wave, rows16 = (L.M + 15) / 16;
  if (block >= rows16) return;
  f32x4* const out = reinterpret_cast<f32x4*>(p) + ((split * rows16 + block) * (L.kp / 16) + 4 * tn) * 64 + lane;
#pragma unroll
  for (int j = 0; j < 4; ++j) out[64 * j] = v[j];
  ckpt_clip16(f, (int)(64 * tn) + 16 * quad, (int)L.K);
  float d = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) d += ckpt_kept_dot(f, j, v[j]);
  d = __builtin_amdgcn_ldexpf(d, (int)f.exp - 133);
  d += __shfl_xor(d, 16, 64);
  d += __shfl_xor(d, 32, 64);
  if (quad == 0 && row < L.M) d_part[(split * L.p_tiles + tn) * L.M + row] = d;
}

// Rows of 8-byte units copied to rows half a unit of 16 bytes longer, the last 8
// bytes zeros: the ring's 16-byte copies then serve N % 8 == 4 too.
__global__ void __launch_bounds__(256)
pad_kernel(const u32x2* __restrict__ g, const u32x2* __restrict__ w_t, int64_t rows_g, int64_t rows_w, int64_t units,
           u32x2* __restrict__ out) {
  const int64_t all = (rows_g + rows_w) * (units + 1);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / (units + 1), u = i - row * (units + 1);
    const u32x2* src = row < rows_g ? g + row * units : w_t + (row - rows_g) * units;
    out[i] = u < units ? src[u] : (u32x2){0, 0};
  }
}

// --- 7. dX -----------------------------------------------------------------------
// 32 tokens (two of P's block rows) and a range of channels per workgroup, its 4
// wavefronts 64 channels (four of P's blocks) in turn: lane l has token l % 16,
// channels 16 (l / 16) + [0, 16), i.e. 16 bytes of codes, one exponent, two
// position bytes and 32 bytes of dX.  Workgroups past `blocks` sum dA and dB, which
// saves a launch where both are asked for.
template <int RT, bool SPLIT>                           // RT: rp / 32, 0 without LoRA; SPLIT: P in ranges
__global__ void __launch_bounds__(256, 2)
finish_kernel(const float* __restrict__ p, const float* __restrict__ d_part, Ckpt ck, const u32x4* __restrict__ u,
              const u32x4* __restrict__ a_up, const float* __restrict__ d_lora, BackwardLayout L, int64_t chunk,
              uint16_t* __restrict__ dx, int64_t blocks, Factors factors) {
  __shared__ float red[256];
  // U's words, the same for the four wavefronts: [rank step][word][16 tokens].  (In
  // registers they left one wavefront per SIMD above rank 64: 4096 x 3072 x 12288,
  // r = 128: 435 us a call instead of 419.)
  __shared__ u32x4 us[RT > 0 ? RT * 3 * 2 * 64 : 1];
  if constexpr (RT > 0) {
    if (blockIdx.x >= blocks) {
      join_columns(factors, L, (blockIdx.x - blocks) * 256 + threadIdx.x, (gridDim.x - blocks) * 256);
      return;
    }
  }
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const int64_t steps = L.kp / 64, rows16 = (L.M + 15) / 16, slab = rows16 * steps * 256;
  const int64_t groups = (rows16 + 1) / 2;
  const int64_t b0 = 2 * (blockIdx.x % groups);
  const int64_t lo = blockIdx.x / groups * chunk, hi = lo + chunk < steps ? lo + chunk : steps;
  float s[2], lk[2];
  const CkptRsrc kr = ckpt_rsrc(ck, L.M, L.K);
  const int K = (int)L.K;
  CkptRow rows[2];
  const f32x4* pr[2];
  bool ok[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t b = b0 + i < rows16 ? b0 + i : rows16 - 1, m = 16 * (b0 + i) + col;
    ok[i] = m < L.M;
    const int64_t row = ok[i] ? m : L.M - 1;
    s[i] = ck.stats[2 * row];
    lk[i] = ck.stats[2 * row + 1];
    rows[i] = ckpt_row(row, L.K);
    pr[i] = reinterpret_cast<const f32x4*>(p) + b * steps * 256 + lane;
  }
  struct Stage {
    f32x4 p[2][4];
    Ckpt16 x[2];
  };
  auto load = [&](Stage& f, int64_t t) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int n = 0; n < 4; ++n) f.p[i][n] = pr[i][(4 * t + n) * 64];
      f.x[i] = ckpt_load16(kr, rows[i], (int)(64 * t + 16 * quad), K);
    }
    if constexpr (SPLIT) {
      // Two ranges' loads at a time, added in the ranges' order.
      int64_t q = 1;
      for (; q + 1 < L.p_splits; q += 2) {
        f32x4 v[2][2][4];
#pragma unroll
        for (int z = 0; z < 2; ++z)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int n = 0; n < 4; ++n) v[z][i][n] = pr[i][(q + z) * slab + (4 * t + n) * 64];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int n = 0; n < 4; ++n) f.p[i][n] = f.p[i][n] + v[0][i][n] + v[1][i][n];
      }
      if (q < L.p_splits)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int n = 0; n < 4; ++n) f.p[i][n] += pr[i][q * slab + (4 * t + n) * 64];
    }
  };
  Stage s0, s1;
  if (lo + wave < hi) load(s0, lo + wave);

  // D: the tiles' and ranges' shares, 8 at a time, then those 8 in order.
  {
    const int64_t m = 16 * b0 + (threadIdx.x & 31), row = m < L.M ? m : L.M - 1;
    float d = 0.f;
#pragma unroll 4
    for (int64_t i = threadIdx.x >> 5; i < L.p_splits * L.p_tiles; i += 8) d += d_part[i * L.M + row];
    red[threadIdx.x] = d;
  }
  for (int z = wave; z < 2 * RT; z += 4) {
    const int i = z & 1, r = z >> 1;
    const u32x4* const f = u + (((b0 + i) * RT + r) * 2) * 64 + lane;
    const Words s3 = split24(f[0], f[64]);
#pragma unroll
    for (int w = 0; w < 3; ++w) us[((r * 3 + w) * 2 + i) * 64 + lane] = s3.w[w];
  }
  __syncthreads();
  float per[2], per_kept[2];                            // D / Lk of a pruned channel; times 1 - s of a kept one
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float d = 0.f;
#pragma unroll
    for (int n = 0; n < 8; ++n) d += red[32 * n + 16 * i + col];
    if constexpr (RT > 0) d -= d_lora[16 * (b0 + i) + col];
    per[i] = lk[i] > 0.f ? d / lk[i] : 0.f;
    per_kept[i] = per[i] * (1.f - s[i]);
  }

  auto finish = [&](Stage& f, int64_t t) {
    uint32_t out[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i) ckpt_clip16(f.x[i], (int)(64 * t + 16 * quad), K);
    f32x4 v[4][2];                                      // U A
#pragma unroll
    for (int n = 0; n < 4; ++n) v[n][0] = v[n][1] = kZero4;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      u32x4 a[4];
#pragma unroll
      for (int n = 0; n < 4; ++n) a[n] = a_up[((4 * t + n) * RT + r) * 64 + lane];
#pragma unroll
      for (int w = 0; w < 3; ++w)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const u32x4 b = us[((r * 3 + w) * 2 + i) * 64 + lane];
#pragma unroll
          for (int n = 0; n < 4; ++n) v[n][i] = mfma(a[n], b, v[n][i]);
        }
      if constexpr (RT == 4) __builtin_amdgcn_sched_barrier(0);   // one rank step's operands at a time
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t b = ckpt_kept16(f.x[i], n), q = f.x[i].codes[n];
        float o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = (int)(q << (24 - 8 * e)) >> 24;
          const float sign = c > 0 ? 1.f : c < 0 ? -1.f : 0.f;
          o[e] = (b >> e) & 1u ? v[n][i][e] + s[i] * (f.p[i][n][e] - v[n][i][e]) + sign * per_kept[i]
                               : v[n][i][e] + sign * per[i];
        }
        out[i][2 * n] = cvt_pk_bf16(o[0], o[1]);
        out[i][2 * n + 1] = cvt_pk_bf16(o[2], o[3]);
      }
    }
    const int64_t k = 64 * t + 16 * quad;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint16_t* y = dx + (16 * (b0 + i) + col) * L.K + k;
      if (ok[i] && k + 16 <= L.K) {
        __builtin_memcpy(__builtin_assume_aligned(y, 8), out[i], 32);
      } else if (ok[i]) {
#pragma unroll
        for (int n = 0; n < 4; ++n)
          if (k + 4 * n < L.K) *reinterpret_cast<u32x2*>(y + 4 * n) = (u32x2){out[i][2 * n], out[i][2 * n + 1]};
      }
    }
  };
  int64_t t = lo + wave;
  for (; t + 8 < hi; t += 8) {
    load(s1, t + 4);
    finish(s0, t);
    load(s0, t + 8);
    finish(s1, t + 4);
  }
  if (t + 4 < hi) {
    load(s1, t + 4);
    finish(s0, t);
    finish(s1, t + 4);
  } else if (t < hi) {
    finish(s0, t);
  }
}

// Workgroups of 256 over this many items, at most 4096 of them.
inline int64_t blocks_of(int64_t items) {
  const int64_t b = (items + 255) / 256;
  return b < 4096 ? b : 4096;
}

template <int JT>
hipError_t launch_lora(const uint16_t* g, const Ckpt& ck, const uint16_t* lora_a, const uint16_t* lora_b,
                       const BackwardLayout& L, float alpha, bool factors, char* ws, hipStream_t stream) {
  constexpr int kCT = JT == 8 ? 4 : 8, kG = JT == 8 ? 2 : 4, kX = kG / 2;
  auto frag = [&](size_t off) { return reinterpret_cast<u32x4*>(ws + off); };
  float* d_lora = reinterpret_cast<float*>(ws + L.off_d);
  float* part = reinterpret_cast<float*>(ws + L.off_part);
  const dim3 factor_blocks((unsigned)blocks_of(L.rp * (2 * L.kp + L.np) / 8));
  hipError_t e = launch(&factors_kernel, factor_blocks, dim3(256), stream, lora_a, lora_b, L,
                        frag(L.off_a_down), frag(L.off_a_up), frag(L.off_b));
  if (e != hipSuccess) return e;
  const bool wg = L.N % 8 == 0, wx = L.K % 8 == 0;
  auto* rk = wg ? &rows_kernel<JT, true> : &rows_kernel<JT, false>;
  const int64_t row_groups = (L.M + 16 * kG - 1) / (16 * kG) * L.splits_g + (L.M + 16 * kX - 1) / (16 * kX) * L.splits_x;
  e = launch(rk, dim3((unsigned)row_groups), dim3(256), stream, g, frag(L.off_b), frag(L.off_a_down), ck, L, part);
  if (e != hipSuccess) return e;
  e = launch(&join_rows_kernel<16 * JT>, dim3((unsigned)(L.mp / 32)), dim3(kJoinThreads), stream, part, ck.stats, L,
             alpha, frag(L.off_u), frag(L.off_uc), frag(L.off_tc), d_lora);
  if (e != hipSuccess || !factors) return e;
  auto* cn = wg ? (wx ? &columns_kernel<kCT, JT, true, true> : &columns_kernel<kCT, JT, true, false>)
                : (wx ? &columns_kernel<kCT, JT, false, true> : &columns_kernel<kCT, JT, false, false>);
  const int64_t col_groups = (L.N + 16 * kCT - 1) / (16 * kCT) + (L.K + 8 * kCT - 1) / (8 * kCT);
  return launch(cn, dim3((unsigned)col_groups, (unsigned)L.splits_t), dim3(256), stream, g, ck, frag(L.off_uc),
                frag(L.off_tc), L, part);
}

}  // namespace

hipError_t launch_backward(const uint16_t* g, const Ckpt& ck, const uint16_t* w_t, const uint16_t* lora_a,
                           const uint16_t* lora_b, const BackwardLayout& L, float alpha, uint16_t* dx, uint16_t* da,
                           uint16_t* db, char* ws, hipStream_t stream) {
  // With no tokens there are no ranges to sum: zeros.
  const Factors factors = {reinterpret_cast<const float*>(ws + L.off_part), da, db};
  const int64_t join_blocks = da != nullptr ? blocks_of(join_items(L)) : 0;
  if (L.M > 0 && L.r > 0) {
    const bool f = da != nullptr;
    const hipError_t e = L.rp == 32   ? launch_lora<2>(g, ck, lora_a, lora_b, L, alpha, f, ws, stream)
                         : L.rp == 64 ? launch_lora<4>(g, ck, lora_a, lora_b, L, alpha, f, ws, stream)
                                      : launch_lora<8>(g, ck, lora_a, lora_b, L, alpha, f, ws, stream);
    if (e != hipSuccess) return e;
  }
  if (L.M == 0 || dx == nullptr)
    return join_blocks == 0 ? hipSuccess
                            : launch(&join_columns_kernel, dim3((unsigned)join_blocks), dim3(256), stream, factors, L);
  float* p = reinterpret_cast<float*>(ws + L.off_p);
  float* d_part = reinterpret_cast<float*>(ws + L.off_d_part);
  if (L.p_length != L.N) {
    uint16_t* const pad = reinterpret_cast<uint16_t*>(ws + L.off_pad);
    const hipError_t e = launch(&pad_kernel, dim3((unsigned)blocks_of((L.M + L.K) * L.p_length / 4)), dim3(256), stream,
                                reinterpret_cast<const u32x2*>(g), reinterpret_cast<const u32x2*>(w_t), L.M, L.K,
                                L.N / 4, reinterpret_cast<u32x2*>(pad));
    if (e != hipSuccess) return e;
    g = pad;
    w_t = pad + L.M * L.p_length;
  }
  const hipError_t e =
      L.p_tile == 64 ? launch(L.N % 8 == 0 ? &few_tokens_kernel<true> : &few_tokens_kernel<false>,
                              dim3((unsigned)((L.M + 63) / 64 * L.p_tiles * L.p_splits)), dim3(256), stream, g, w_t, ck, L,
                              p, d_part)
                     : launch_grad_gemm(g, w_t, ck, L, p, d_part, stream);
  if (e != hipSuccess) return e;
  const bool split = L.p_splits > 1;
  auto* k = L.r == 0     ? (split ? &finish_kernel<0, true> : &finish_kernel<0, false>)
            : L.rp == 32 ? (split ? &finish_kernel<1, true> : &finish_kernel<1, false>)
            : L.rp == 64 ? (split ? &finish_kernel<2, true> : &finish_kernel<2, false>)
                         : (split ? &finish_kernel<4, true> : &finish_kernel<4, false>);
  // About 4096 wavefronts (four per SIMD), each with at least one 64-channel step.
  const int64_t groups = (L.M + 31) / 32, steps = L.kp / 64;
  const int64_t chunk = 4 * ((groups * steps + 4095) / 4096);
  const int64_t blocks = groups * ((steps + chunk - 1) / chunk);
  return launch(k, dim3((unsigned)(blocks + join_blocks)), dim3(256), stream, p, d_part, ck,
                reinterpret_cast<const u32x4*>(ws + L.off_u), reinterpret_cast<const u32x4*>(ws + L.off_a_up),
                reinterpret_cast<const float*>(ws + L.off_d), L, chunk, dx, blocks, factors);
}

}  // namespace rtl
