// rtl_sparse_linear_backward (include/rtlynx_train.h).
//
// The work is one large product, G W [M, K] over N channels, which runs on the
// dense GEMM's ring (dense_gemm.hip, fp32 result), and the LoRA branch, whose
// products all have one dimension of at most 128 and are bound by reading G
// and the checkpoint:
//
//   1. transpose_factors   A as [r][K] and [K][r], B as [r][N], zero-padded, so
//                          every operand is contiguous along its contraction.
//   2. rows_kernel         G B, and of the checkpoint (pruned A^T) and (kept
//                          A^T): token-by-rank products over the channels, split
//                          over channel ranges.
//   3. join_rows           sums the ranges in order, forms U = alpha G B and
//                          T = alpha (pruned A^T + (1 - s) kept A^T), the part of D
//                          that needs no G W, and lays U, (1 - s) U and T out for
//                          the products that follow, each as two bf16 words (hi + lo: 16 bits).
//   4. columns_kernel      G^T T and [pruned; kept]^T [U; (1 - s) U]: products over the
//                          tokens, split over token ranges.  Both operands run along
//                          tokens, which are rows in memory: the tile goes through
//                          LDS and is read transposed (ds_read_b64_tr_b16).
//   5. join_columns        sums the ranges in order into dA and dB.
//   6. the dense GEMM      P = G W.
//   7. finish_kernel       D per token, then dX; U A is formed again, a 16-token
//                          strip at a time, on the matrix cores (r is small), so it
//                          never goes to memory.
//
// A kept value's residual (1 - s) x is not a bf16 number; multiplying U (or the
// joined sum) by 1 - s instead keeps the checkpoint's values exact operands.
#include "rtl_checkpoint.hpp"
#include "rtl_common.hpp"
#include "rtl_kernels.hpp"

namespace rtl {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));

// fp32 as two bf16 words: hi + lo holds 16 significant bits.
__device__ __forceinline__ void split_bf16(float v, uint16_t& hi, uint16_t& lo) {
  const uint32_t h = f32_to_bf16_rne(v);
  hi = (uint16_t)h;
  lo = (uint16_t)f32_to_bf16_rne(v - __builtin_bit_cast(float, h << 16));
}

// 8 channels of a row at channel c of C (C % 4 == 0): rows are 16-byte aligned
// when WIDE (C % 8 == 0), else 8-byte, with half a unit at the end.
template <bool WIDE>
__device__ __forceinline__ u32x4 load8(const uint16_t* row, int64_t c, int64_t C, bool ok) {
  u32x4 v = {0, 0, 0, 0};
  if constexpr (WIDE) {
    if (ok && c < C) v = *reinterpret_cast<const u32x4*>(row + c);
  } else {
    if (ok && c < C) {
      const u32x2 a = *reinterpret_cast<const u32x2*>(row + c);
      v[0] = a[0];
      v[1] = a[1];
      if (c + 8 <= C) {
        const u32x2 b = *reinterpret_cast<const u32x2*>(row + c + 4);
        v[2] = b[0];
        v[3] = b[1];
      }
    }
  }
  return v;
}

// The checkpoint's 8 channels at channel c: pruned and kept values apart.
struct CkptUnit {
  u32x4 pruned, kept;
};
struct CkptRaw {
  u32x2 q;
  uint32_t e, idx;
};
template <bool WIDE>
__device__ __forceinline__ CkptRaw ckpt_load(const Ckpt& k, int64_t row, int64_t c, int64_t K, bool ok) {
  CkptRaw r = {{0, 0}, 0, 0};
  if (ok && c < K) {
    const int8_t* p = k.codes + row * K + c;
    if constexpr (WIDE) {
      r.q = *reinterpret_cast<const u32x2*>(p);
    } else {
      r.q[0] = *reinterpret_cast<const uint32_t*>(p);
      if (c + 8 <= K) r.q[1] = *reinterpret_cast<const uint32_t*>(p + 4);
    }
    r.e = k.exps[row * ((K + 31) / 32) + c / 32];
    r.idx = k.idx[row * ((K + 7) / 8) + c / 8];
  }
  return r;
}
__device__ __forceinline__ CkptUnit ckpt_split(const CkptRaw& r) {
  const u32x4 v = ckpt_values(r.q, (int)r.e), m = kept_masks(r.idx);
  CkptUnit u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    u.kept[i] = v[i] & m[i];
    u.pruned[i] = v[i] & ~m[i];
  }
  return u;
}

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// --- 1. factors ------------------------------------------------------------
// One thread per 8 words of an output row.
__global__ void __launch_bounds__(256)
transpose_factors_kernel(const uint16_t* __restrict__ a, const uint16_t* __restrict__ b, BackwardLayout L,
                         uint16_t* __restrict__ ap, uint16_t* __restrict__ at, uint16_t* __restrict__ bt) {
  const int64_t na = L.rp * L.kp / 8, nb = L.rp * L.np / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < 2 * na + nb; i += (int64_t)gridDim.x * 256) {
    uint16_t v[8];
    if (i < na) {                                   // ap[j][k]: neighbouring threads along k
      const int64_t j = i / (L.kp / 8), k = 8 * (i - j * (L.kp / 8));
      for (int e = 0; e < 8; ++e) v[e] = j < L.r && k + e < L.K ? a[j * L.K + k + e] : 0;
      *reinterpret_cast<u32x4*>(ap + j * L.kp + k) = *reinterpret_cast<u32x4*>(v);
    } else if (i < 2 * na) {                        // at[k][j]: neighbouring threads along k
      const int64_t q = i - na, j = 8 * (q / L.kp), k = q % L.kp;
      for (int e = 0; e < 8; ++e) v[e] = j + e < L.r && k < L.K ? a[(j + e) * L.K + k] : 0;
      *reinterpret_cast<u32x4*>(at + k * L.rp + j) = *reinterpret_cast<u32x4*>(v);
    } else {                                        // bt[j][n]: neighbouring threads along j
      const int64_t q = i - 2 * na, n = 8 * (q / L.rp), j = q % L.rp;
      for (int e = 0; e < 8; ++e) v[e] = j < L.r && n + e < L.N ? b[(n + e) * L.r + j] : 0;
      *reinterpret_cast<u32x4*>(bt + j * L.np + n) = *reinterpret_cast<u32x4*>(v);
    }
  }
}

// --- 2. token-by-rank products --------------------------------------------
// 4 wavefronts of 32 tokens, JT tiles of 16 ranks; channels [lo, hi), a
// multiple of 64 apart from the end.
template <int JT, bool WIDE>
__device__ __forceinline__ void g_rows(const uint16_t* __restrict__ g, const uint16_t* __restrict__ bt,
                                       const BackwardLayout& L, int64_t m0, int64_t lo, int64_t hi,
                                       float* __restrict__ out) {
  const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
  f32x4 acc[2][JT];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < JT; ++j) acc[i][j] = (f32x4){0, 0, 0, 0};
  const int64_t r0 = m0 + col, r1 = r0 + 16;
  const bool ok0 = r0 < L.M, ok1 = r1 < L.M;
  const uint16_t* g0 = g + (ok0 ? r0 : 0) * L.N;
  const uint16_t* g1 = g + (ok1 ? r1 : 0) * L.N;
  const uint16_t* bp = bt + (int64_t)col * L.np;
  for (int64_t c0 = lo; c0 < hi; c0 += 64) {
    u32x4 x0[2], x1[2], w[2][JT];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t c = c0 + 32 * h + 8 * quad;
      x0[h] = load8<WIDE>(g0, c, L.N, ok0);
      x1[h] = load8<WIDE>(g1, c, L.N, ok1);
#pragma unroll
      for (int j = 0; j < JT; ++j) w[h][j] = *reinterpret_cast<const u32x4*>(bp + (int64_t)16 * j * L.np + c);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < JT; ++j) {
        acc[0][j] = mfma(x0[h], w[h][j], acc[0][j]);
        acc[1][j] = mfma(x1[h], w[h][j], acc[1][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < JT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t m = m0 + 16 * i + 4 * quad + e;
        if (m < L.M) out[m * L.rp + 16 * j + col] = acc[i][j][e];
      }
}

template <int JT, bool WIDE>
__device__ __forceinline__ void x_rows(const Ckpt& ck, const uint16_t* __restrict__ ap, const BackwardLayout& L,
                                       int64_t m0, int64_t lo, int64_t hi, float* __restrict__ out_pruned,
                                       float* __restrict__ out_kept) {
  const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
  f32x4 pr[2][JT], ke[2][JT];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < JT; ++j) pr[i][j] = ke[i][j] = (f32x4){0, 0, 0, 0};
  const int64_t r0 = m0 + col, r1 = r0 + 16;
  const bool ok0 = r0 < L.M, ok1 = r1 < L.M;
  const uint16_t* wp = ap + (int64_t)col * L.kp;
  for (int64_t c0 = lo; c0 < hi; c0 += 64) {
    CkptRaw x0[2], x1[2];
    u32x4 w[2][JT];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t c = c0 + 32 * h + 8 * quad;
      x0[h] = ckpt_load<WIDE>(ck, r0, c, L.K, ok0);
      x1[h] = ckpt_load<WIDE>(ck, r1, c, L.K, ok1);
#pragma unroll
      for (int j = 0; j < JT; ++j) w[h][j] = *reinterpret_cast<const u32x4*>(wp + (int64_t)16 * j * L.kp + c);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const CkptUnit u0 = ckpt_split(x0[h]), u1 = ckpt_split(x1[h]);
#pragma unroll
      for (int j = 0; j < JT; ++j) {
        pr[0][j] = mfma(u0.pruned, w[h][j], pr[0][j]);
        ke[0][j] = mfma(u0.kept, w[h][j], ke[0][j]);
        pr[1][j] = mfma(u1.pruned, w[h][j], pr[1][j]);
        ke[1][j] = mfma(u1.kept, w[h][j], ke[1][j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < JT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t m = m0 + 16 * i + 4 * quad + e;
        if (m < L.M) {
          out_pruned[m * L.rp + 16 * j + col] = pr[i][j][e];
          out_kept[m * L.rp + 16 * j + col] = ke[i][j][e];
        }
      }
}

template <int JT, bool WIDE_G, bool WIDE_X>
__global__ void __launch_bounds__(256)
rows_kernel(const uint16_t* __restrict__ g, const uint16_t* __restrict__ bt, const uint16_t* __restrict__ ap, Ckpt ck,
            BackwardLayout L, float* __restrict__ part) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t splits = L.row_splits_g + L.row_splits_x;
  const int64_t s = blockIdx.x % splits;                // channel range: G's first, then the checkpoint's
  const int64_t m0 = blockIdx.x / splits * 128 + 32 * wave;
  if (m0 >= L.M) return;
  const int64_t slab = L.M * L.rp;
  if (s < L.row_splits_g) {
    const int64_t lo = s * L.row_chunk, hi = lo + L.row_chunk < L.np ? lo + L.row_chunk : L.np;
    g_rows<JT, WIDE_G>(g, bt, L, m0, lo, hi, part + s * slab);
  } else {
    const int64_t q = s - L.row_splits_g;
    const int64_t lo = q * L.row_chunk, hi = lo + L.row_chunk < L.kp ? lo + L.row_chunk : L.kp;
    float* p = part + (L.row_splits_g + 2 * q) * slab;
    x_rows<JT, WIDE_X>(ck, ap, L, m0, lo, hi, p, p + slab);
  }
}

// --- 3. U, T and what follows from them -------------------------------------
// 32 tokens per workgroup.  Tokens past M are written as zeros up to mp, so the
// products over tokens need no guard.
__global__ void __launch_bounds__(256)
join_rows_kernel(const float* __restrict__ part, const float* __restrict__ stats, BackwardLayout L, float alpha,
                 uint16_t* __restrict__ u_rows, uint16_t* __restrict__ u_cols, uint16_t* __restrict__ t_cols,
                 float* __restrict__ d_lora) {
  extern __shared__ float lds[];                        // U and U (kept A^T) [32][rp + 1], T [32][rp]
  const int rp = (int)L.rp, pitch = rp + 1;
  float* const us = lds;
  float* const ds = lds + 32 * pitch;
  float* const ts = lds + 2 * 32 * pitch;
  const int64_t m0 = (int64_t)blockIdx.x * 32, slab = L.M * L.rp;
  for (int i = threadIdx.x; i < 32 * rp; i += 256) {
    const int r = i / rp, j = i - r * rp;
    const int64_t m = m0 + r;
    float u = 0.f, pr = 0.f, ke = 0.f, s = 1.f;
    if (m < L.M) {
      const float* p = part + m * L.rp + j;
      for (int64_t q = 0; q < L.row_splits_g; ++q) u += p[q * slab];
      p += L.row_splits_g * slab;
      for (int64_t q = 0; q < L.row_splits_x; ++q) {
        pr += p[2 * q * slab];
        ke += p[(2 * q + 1) * slab];
      }
      s = stats[2 * m];
    }
    u *= alpha;
    us[r * pitch + j] = u;
    ds[r * pitch + j] = u * ke;                         // for D: sum over ranks of U (kept A^T)
    const float t = alpha * (pr + (1.f - s) * ke);
    uint16_t hi, lo;
    if (m < L.M) {
      split_bf16(u, hi, lo);
      u_rows[m * 2 * L.rp + j] = hi;
      u_rows[m * 2 * L.rp + L.rp + j] = lo;
    }
    ts[i] = t;
  }
  __syncthreads();
  if (threadIdx.x < 32 && m0 + threadIdx.x < L.M) {
    float d = 0.f;
    for (int j = 0; j < rp; ++j) d += ds[threadIdx.x * pitch + j];
    d_lora[m0 + threadIdx.x] = d;
  }
  // Transposed: lanes along tokens.
  const int r = threadIdx.x & 31;
  const int64_t m = m0 + r;
  const float keep = m < L.M ? 1.f - stats[2 * m] : 0.f;
  for (int j = threadIdx.x >> 5; j < rp; j += 8) {
    uint16_t hi, lo;
    const float u = us[r * pitch + j];
    split_bf16(u, hi, lo);
    u_cols[(int64_t)j * L.mp + m] = hi;
    u_cols[(int64_t)(L.rp + j) * L.mp + m] = lo;
    split_bf16(u * keep, hi, lo);
    u_cols[(int64_t)(2 * L.rp + j) * L.mp + m] = hi;
    u_cols[(int64_t)(3 * L.rp + j) * L.mp + m] = lo;
    split_bf16(ts[r * rp + j], hi, lo);
    t_cols[(int64_t)j * L.mp + m] = hi;
    t_cols[(int64_t)(L.rp + j) * L.mp + m] = lo;
  }
}

// --- 4. products over tokens ------------------------------------------------
// A workgroup's tile: 64 tokens x 128 channels in LDS, 4 wavefronts of 32
// channels.  Row pitch 272 bytes: 16-byte aligned, rows shifted by 4 banks.
constexpr int kColPitch = 136;                          // bf16 words
constexpr int kColTile = 64 * kColPitch;

// The operand of 16 channels (from c) x 32 tokens (from t) of such a tile:
// lane l gets tokens 8 (l / 16) + [0, 8) of channel l % 16.  One transposing
// read gives a lane 4 tokens: its 16 lanes name 4 rows of 16 channels.
__device__ __forceinline__ u32x4 transposed_operand(const uint16_t* tile, int t, int c) {
  const int lane = threadIdx.x & 63;
  const uint16_t* p = tile + (t + 8 * (lane >> 4) + ((lane & 15) >> 2)) * kColPitch + c + 4 * (lane & 3);
  using lds_s16x4 = __attribute__((address_space(3))) s16x4;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p));
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * kColPitch));
  const u32x2 a2 = __builtin_bit_cast(u32x2, a), b2 = __builtin_bit_cast(u32x2, b);
  return (u32x4){a2[0], a2[1], b2[0], b2[1]};
}

template <int JT, bool WIDE_G, bool WIDE_X>
__global__ void __launch_bounds__(256)
columns_kernel(const uint16_t* __restrict__ g, Ckpt ck, const uint16_t* __restrict__ u_cols,
               const uint16_t* __restrict__ t_cols, BackwardLayout L, float* __restrict__ part) {
  __shared__ __attribute__((aligned(16))) uint16_t tile[2 * kColTile];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const int64_t tiles_g = (L.N + 127) / 128;
  const bool is_g = (int64_t)blockIdx.x < tiles_g;
  const int64_t c0 = 128 * (is_g ? (int64_t)blockIdx.x : (int64_t)blockIdx.x - tiles_g);
  const int64_t t_lo = (int64_t)blockIdx.y * L.col_chunk;
  const int64_t t_hi = t_lo + L.col_chunk < L.mp ? t_lo + L.col_chunk : L.mp;
  const int lr = threadIdx.x >> 4, lc = 8 * (threadIdx.x & 15);   // loader: rows lr + 16 i, channels c0 + lc
  f32x4 acc[2][JT];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < JT; ++j) acc[i][j] = (f32x4){0, 0, 0, 0};

  if (is_g) {
    u32x4 v[4];
    auto load = [&](int64_t t0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t m = t0 + lr + 16 * i;
        v[i] = load8<WIDE_G>(g + (m < L.M ? m : 0) * L.N, c0 + lc, L.N, m < L.M);
      }
    };
    const uint16_t* q = t_cols + (int64_t)col * L.mp + 8 * quad;
    load(t_lo);
    for (int64_t t0 = t_lo; t0 < t_hi; t0 += 64) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<u32x4*>(tile + (lr + 16 * i) * kColPitch + lc) = v[i];
      __syncthreads();
      if (t0 + 64 < t_hi) load(t0 + 64);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x4 x0 = transposed_operand(tile, 32 * h, 32 * wave), x1 = transposed_operand(tile, 32 * h, 32 * wave + 16);
#pragma unroll
        for (int j = 0; j < JT; ++j) {
          const uint16_t* w = q + (int64_t)16 * j * L.mp + t0 + 32 * h;
          const u32x4 hi = *reinterpret_cast<const u32x4*>(w), lo = *reinterpret_cast<const u32x4*>(w + L.rp * L.mp);
          acc[0][j] = mfma(x0, hi, acc[0][j]);
          acc[1][j] = mfma(x1, hi, acc[1][j]);
          acc[0][j] = mfma(x0, lo, acc[0][j]);
          acc[1][j] = mfma(x1, lo, acc[1][j]);
        }
      }
    }
    float* out = part + (int64_t)blockIdx.y * L.N * L.rp;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < JT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t n = c0 + 32 * wave + 16 * i + 4 * quad + e;
          if (n < L.N) out[n * L.rp + 16 * j + col] = acc[i][j][e];
        }
  } else {
    CkptRaw v[4];
    auto load = [&](int64_t t0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t m = t0 + lr + 16 * i;
        v[i] = ckpt_load<WIDE_X>(ck, m, c0 + lc, L.K, m < L.M);
      }
    };
    const uint16_t* q = u_cols + (int64_t)col * L.mp + 8 * quad;
    load(t_lo);
    for (int64_t t0 = t_lo; t0 < t_hi; t0 += 64) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const CkptUnit u = ckpt_split(v[i]);
        *reinterpret_cast<u32x4*>(tile + (lr + 16 * i) * kColPitch + lc) = u.pruned;
        *reinterpret_cast<u32x4*>(tile + kColTile + (lr + 16 * i) * kColPitch + lc) = u.kept;
      }
      __syncthreads();
      if (t0 + 64 < t_hi) load(t0 + 64);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int part_of = 0; part_of < 2; ++part_of) {    // pruned with U, kept with (1 - s) U
          const uint16_t* src = tile + part_of * kColTile;
          const u32x4 x0 = transposed_operand(src, 32 * h, 32 * wave), x1 = transposed_operand(src, 32 * h, 32 * wave + 16);
#pragma unroll
          for (int j = 0; j < JT; ++j) {
            const uint16_t* w = q + (2 * part_of * L.rp + 16 * j) * L.mp + t0 + 32 * h;
            const u32x4 hi = *reinterpret_cast<const u32x4*>(w), lo = *reinterpret_cast<const u32x4*>(w + L.rp * L.mp);
            acc[0][j] = mfma(x0, hi, acc[0][j]);
            acc[1][j] = mfma(x1, hi, acc[1][j]);
            acc[0][j] = mfma(x0, lo, acc[0][j]);
            acc[1][j] = mfma(x1, lo, acc[1][j]);
          }
        }
      }
    }
    float* out = part + (int64_t)L.col_splits * L.N * L.rp + (int64_t)blockIdx.y * L.kp * L.rp;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < JT; ++j) {
        const int64_t k = c0 + 32 * wave + 16 * i + 4 * quad;
        if (k < L.K) *reinterpret_cast<f32x4*>(out + (int64_t)(16 * j + col) * L.kp + k) = acc[i][j];
      }
  }
}

// --- 5. dA and dB -------------------------------------------------------------
__global__ void __launch_bounds__(256)
join_columns_kernel(const float* __restrict__ part, BackwardLayout L, uint16_t* __restrict__ da,
                    uint16_t* __restrict__ db) {
  const int64_t nb = L.N * L.r, na = L.r * L.K;
  const float* pa = part + L.col_splits * L.N * L.rp;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < nb + na; i += (int64_t)gridDim.x * 256) {
    float v = 0.f;
    if (i < nb) {
      const int64_t n = i / L.r, j = i - n * L.r;
      for (int64_t s = 0; s < L.col_splits; ++s) v += part[(s * L.N + n) * L.rp + j];
      db[i] = (uint16_t)f32_to_bf16_rne(v);
    } else {
      const int64_t q = i - nb, j = q / L.K, k = q - j * L.K;
      for (int64_t s = 0; s < L.col_splits; ++s) v += pa[(s * L.rp + j) * L.kp + k];
      da[q] = (uint16_t)f32_to_bf16_rne(v);
    }
  }
}

// --- 7. dX -----------------------------------------------------------------------
// 16 tokens per workgroup, 8 wavefronts along the channels.  A lane's unit is
// the 4 channels (one group) of a token that the matrix core's result layout
// gives it: token l % 16, channels 4 (l / 16) + [0, 4) of 16.
constexpr int kFinWaves = 8;

template <int RT>                                       // rp / 32, 0 without LoRA
__global__ void __launch_bounds__(64 * kFinWaves)
finish_kernel(const float* __restrict__ p, Ckpt ck, const uint16_t* __restrict__ u_rows,
              const uint16_t* __restrict__ at, const float* __restrict__ d_lora, BackwardLayout L,
              uint16_t* __restrict__ dx) {
  __shared__ float red[kFinWaves][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const int64_t m = (int64_t)blockIdx.x * 16 + col;
  const bool ok = m < L.M;
  const int64_t row = ok ? m : L.M - 1;
  const float s = ck.stats[2 * row], lk = ck.stats[2 * row + 1];
  const int8_t* codes = ck.codes + row * L.K;
  const uint8_t* exps = ck.exps + row * ((L.K + 31) / 32);
  const uint8_t* idx = ck.idx + row * ((L.K + 7) / 8);
  const float* pr = p + row * L.K;
  const int64_t tiles = (L.K + 15) / 16;

  float d = 0.f;
  for (int64_t t = wave; t < tiles; t += kFinWaves) {
    const int64_t k = 16 * t + 4 * quad;
    if (k < L.K) {
      const uint32_t q = *reinterpret_cast<const uint32_t*>(codes + k);
      const int e = exps[k / 32];
      const uint32_t b = kept_bits((uint32_t)idx[k / 8] >> (k & 4));
      const f32x4 v = *reinterpret_cast<const f32x4*>(pr + k);
      d += (b & 1u) ? ckpt_value<0>(q, e) * v[0] : 0.f;
      d += (b & 2u) ? ckpt_value<1>(q, e) * v[1] : 0.f;
      d += (b & 4u) ? ckpt_value<2>(q, e) * v[2] : 0.f;
      d += (b & 8u) ? ckpt_value<3>(q, e) * v[3] : 0.f;
    }
  }
  d += __shfl_xor(d, 16, 64);
  d += __shfl_xor(d, 32, 64);
  if (quad == 0) red[wave][col] = d;
  __syncthreads();
  d = 0.f;
#pragma unroll
  for (int w = 0; w < kFinWaves; ++w) d += red[w][col];
  if constexpr (RT > 0) d -= d_lora[row];
  const float per = lk > 0.f ? d / lk : 0.f;            // of a pruned channel; times 1 - s of a kept one
  const float per_kept = per * (1.f - s);

  u32x4 uh[RT > 0 ? RT : 1], ul[RT > 0 ? RT : 1];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const uint16_t* u = u_rows + row * 2 * L.rp + 32 * i + 8 * quad;
    uh[i] = *reinterpret_cast<const u32x4*>(u);
    ul[i] = *reinterpret_cast<const u32x4*>(u + L.rp);
  }
  for (int64_t t = wave; t < tiles; t += kFinWaves) {
    f32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const u32x4 a = *reinterpret_cast<const u32x4*>(at + (16 * t + col) * L.rp + 32 * i + 8 * quad);
      v = mfma(a, uh[i], v);
      v = mfma(a, ul[i], v);
    }
    const int64_t k = 16 * t + 4 * quad;
    if (ok && k < L.K) {
      const uint32_t q = *reinterpret_cast<const uint32_t*>(codes + k);
      const uint32_t b = kept_bits((uint32_t)idx[k / 8] >> (k & 4));
      const f32x4 e = *reinterpret_cast<const f32x4*>(pr + k);
      float o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = (int)(q << (24 - 8 * i)) >> 24;
        const float sign = c > 0 ? 1.f : c < 0 ? -1.f : 0.f;
        o[i] = (b >> i) & 1u ? v[i] + s * (e[i] - v[i]) + sign * per_kept : v[i] + sign * per;
      }
      *reinterpret_cast<u32x2*>(dx + row * L.K + k) = (u32x2){pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
    }
  }
}

template <int JT>
hipError_t launch_lora(const uint16_t* g, const Ckpt& ck, const uint16_t* lora_a, const uint16_t* lora_b,
                       const BackwardLayout& L, float alpha, uint16_t* da, uint16_t* db, char* ws, hipStream_t stream) {
  uint16_t* ap = reinterpret_cast<uint16_t*>(ws + L.off_ap);
  uint16_t* at = reinterpret_cast<uint16_t*>(ws + L.off_at);
  uint16_t* bt = reinterpret_cast<uint16_t*>(ws + L.off_bt);
  uint16_t* u_rows = reinterpret_cast<uint16_t*>(ws + L.off_u_rows);
  uint16_t* u_cols = reinterpret_cast<uint16_t*>(ws + L.off_u_cols);
  uint16_t* t_cols = reinterpret_cast<uint16_t*>(ws + L.off_t_cols);
  float* d_lora = reinterpret_cast<float*>(ws + L.off_d);
  float* part = reinterpret_cast<float*>(ws + L.off_part);
  auto blocks = [](int64_t items) { const int64_t b = (items + 255) / 256; return dim3((unsigned)(b < 4096 ? b : 4096)); };
  hipError_t e = launch(&transpose_factors_kernel, blocks(L.rp * (2 * L.kp + L.np) / 8), dim3(256), stream, lora_a,
                        lora_b, L, ap, at, bt);
  if (e != hipSuccess) return e;
  const bool wg = L.N % 8 == 0, wx = L.K % 8 == 0;
  auto* rk = wg ? (wx ? &rows_kernel<JT, true, true> : &rows_kernel<JT, true, false>)
                : (wx ? &rows_kernel<JT, false, true> : &rows_kernel<JT, false, false>);
  e = launch(rk, dim3((unsigned)((L.row_splits_g + L.row_splits_x) * ((L.M + 127) / 128))), dim3(256), stream,
             g, bt, ap, ck, L, part);
  if (e != hipSuccess) return e;
  {
    BackwardLayout l = L;
    const float* pp = part;
    const float* st = ck.stats;
    void* args[] = {&pp, &st, &l, &alpha, &u_rows, &u_cols, &t_cols, &d_lora};
    const size_t lds = (size_t)(2 * 32 * (L.rp + 1) + 32 * L.rp) * sizeof(float);
    e = hipLaunchKernel(reinterpret_cast<const void*>(&join_rows_kernel), dim3((unsigned)(L.mp / 32)), dim3(256), args,
                        lds, stream);
  }
  if (e != hipSuccess || da == nullptr) return e;
  auto* ckn = wg ? (wx ? &columns_kernel<JT, true, true> : &columns_kernel<JT, true, false>)
                 : (wx ? &columns_kernel<JT, false, true> : &columns_kernel<JT, false, false>);
  e = launch(ckn, dim3((unsigned)((L.N + 127) / 128 + (L.K + 127) / 128), (unsigned)L.col_splits), dim3(256), stream,
             g, ck, u_cols, t_cols, L, part);
  if (e != hipSuccess) return e;
  return launch(&join_columns_kernel, blocks(L.r * (L.N + L.K)), dim3(256), stream, part, L, da, db);
}

}  // namespace

hipError_t launch_backward(const uint16_t* g, const Ckpt& ck, const uint16_t* w_t, const uint16_t* lora_a,
                           const uint16_t* lora_b, const BackwardLayout& L, float alpha, uint16_t* dx, uint16_t* da,
                           uint16_t* db, char* ws, hipStream_t stream) {
  if (L.M == 0) {                                       // no tokens: no ranges to sum, zeros
    const int64_t b = (L.r * (L.N + L.K) + 255) / 256;
    return launch(&join_columns_kernel, dim3((unsigned)(b < 4096 ? b : 4096)), dim3(256), stream,
                  reinterpret_cast<float*>(ws), L, da, db);
  }
  if (L.r > 0) {
    const hipError_t e = L.rp == 32   ? launch_lora<2>(g, ck, lora_a, lora_b, L, alpha, da, db, ws, stream)
                         : L.rp == 64 ? launch_lora<4>(g, ck, lora_a, lora_b, L, alpha, da, db, ws, stream)
                                      : launch_lora<8>(g, ck, lora_a, lora_b, L, alpha, da, db, ws, stream);
    if (e != hipSuccess) return e;
  }
  if (dx == nullptr) return hipSuccess;
  float* p = reinterpret_cast<float*>(ws + L.off_p);
  const hipError_t e = launch_dense_gemm_f32(g, w_t, L.M, L.K, L.N, p, stream);
  if (e != hipSuccess) return e;
  auto* k = L.r == 0     ? &finish_kernel<0>
            : L.rp == 32 ? &finish_kernel<1>
            : L.rp == 64 ? &finish_kernel<2>
                         : &finish_kernel<4>;
  return launch(k, dim3((unsigned)((L.M + 15) / 16)), dim3(64 * kFinWaves), stream, p, ck,
                reinterpret_cast<const uint16_t*>(ws + L.off_u_rows), reinterpret_cast<const uint16_t*>(ws + L.off_at),
                reinterpret_cast<const float*>(ws + L.off_d), L, dx);
}

}  // namespace rtl
