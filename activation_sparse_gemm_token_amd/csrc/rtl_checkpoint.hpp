// Device-side reading of the 8-bit checkpoint (include/rtlynx_train.h).
#pragma once

#include "rtl_common.hpp"
#include "rtl_operators.hpp"

namespace rtl {

// Code in byte b of word q times 2^(e - 133), fp32.
template <int B>
__device__ __forceinline__ float ckpt_value(uint32_t q, int e) {
  return __builtin_amdgcn_ldexpf((float)((int)(q << (24 - 8 * B)) >> 24), e - 133);
}

// 8 codes as 8 bf16: 7 significant bits and a power of two, so the upper half of
// the fp32 value is the value (below 2^-126 too: the smallest step is bf16's).
__device__ __forceinline__ u32x4 ckpt_values(u32x2 q, int e) {
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t a = __builtin_bit_cast(uint32_t, ckpt_value<0>(q[i], e));
    const uint32_t b = __builtin_bit_cast(uint32_t, ckpt_value<1>(q[i], e));
    const uint32_t c = __builtin_bit_cast(uint32_t, ckpt_value<2>(q[i], e));
    const uint32_t d = __builtin_bit_cast(uint32_t, ckpt_value<3>(q[i], e));
    v[2 * i] = __builtin_amdgcn_perm(b, a, 0x07060302u);
    v[2 * i + 1] = __builtin_amdgcn_perm(d, c, 0x07060302u);
  }
  return v;
}

// Kept channels of one group's code (idx0 | idx1 << 2) as bits 0..3.
__device__ __forceinline__ uint32_t kept_bits(uint32_t code) {
  return (1u << (code & 3u)) | (1u << ((code >> 2) & 3u));
}

// 16-bit lane masks of the 8 channels that one idx byte describes.
__device__ __forceinline__ u32x4 kept_masks(uint32_t byte) {
  u32x4 m;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t b = kept_bits(byte >> (4 * i));
    m[2 * i] = (b & 1u) * 0xffffu | ((b >> 1) & 1u) * 0xffff0000u;
    m[2 * i + 1] = ((b >> 2) & 1u) * 0xffffu | ((b >> 3) & 1u) * 0xffff0000u;
  }
  return m;
}

// 8 codes with exponents e (kept channels) and p (pruned), idx byte `byte`, as the
// kept values and the pruned ones, each zero at the other's channels.
__device__ __forceinline__ void ckpt_split8(u32x2 q, uint32_t e, uint32_t p, uint32_t byte, u32x4& pruned, u32x4& kept) {
  const u32x4 m = kept_masks(byte);
  kept = ckpt_values(q, (int)e);
  pruned = ckpt_values(q, (int)p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    kept[i] &= m[i];
    pruned[i] &= ~m[i];
  }
}

// The checkpoint through buffer resources: a load past the tensors or at
// kOobOffset gives zeros and needs no branch, so none is ever under a condition
// (a conditional load makes the compiler wait for every load in flight where it
// waits for one).  All of it is below 2 GiB: 32-bit offsets.
struct CkptRsrc {
  __amdgpu_buffer_rsrc_t codes, exps, pruned_exps, idx;
};
__device__ __forceinline__ CkptRsrc ckpt_rsrc(const Ckpt& c, int64_t M, int64_t K) {
  return {make_rsrc(c.codes, M * K), make_rsrc(c.exps, M * ((K + 31) / 32)),
          make_rsrc(c.pruned_exps, M * ((K + 31) / 32)), make_rsrc(c.idx, M * ((K + 7) / 8))};
}
// A token's offsets in the three; a token past M gives zeros.
struct CkptRow {
  uint32_t codes, exps, idx;
};
__device__ __forceinline__ CkptRow ckpt_row(int64_t row, int64_t K) {
  return {(uint32_t)(row * K), (uint32_t)(row * ((K + 31) / 32)), (uint32_t)(row * ((K + 7) / 8))};
}

// 16 channels of a token at channel k (k % 16 == 0): one lane's share of 64.
// Channels past K have code 0.
struct Ckpt16 {
  u32x4 codes;
  uint32_t exp, pruned_exp, idx0, idx1;   // idx: 4 bits per group, two groups each
};
__device__ __forceinline__ Ckpt16 ckpt_load16(const CkptRsrc& c, const CkptRow& r, int k, int K) {
  Ckpt16 f;
  f.codes = buf_load16(c.codes, k < K ? r.codes + k : kOobOffset);
  f.exp = __builtin_amdgcn_raw_buffer_load_b8(c.exps, k < K ? r.exps + k / 32 : kOobOffset, 0, 0);
  f.pruned_exp = __builtin_amdgcn_raw_buffer_load_b8(c.pruned_exps, k < K ? r.exps + k / 32 : kOobOffset, 0, 0);
  f.idx0 = __builtin_amdgcn_raw_buffer_load_b8(c.idx, k < K ? r.idx + k / 8 : kOobOffset, 0, 0);
  f.idx1 = __builtin_amdgcn_raw_buffer_load_b8(c.idx, k + 8 < K ? r.idx + k / 8 + 1 : kOobOffset, 0, 0);
  return f;
}
// What such a load brings past the end of a row is the next row's: made zeros
// when it is used.
__device__ __forceinline__ void ckpt_clip16(Ckpt16& f, int k, int K) {
#pragma unroll
  for (int i = 1; i < 4; ++i) f.codes[i] = k + 4 * i < K ? f.codes[i] : 0u;
}
// Kept channels of group i (0 to 3) as bits 0..3.
__device__ __forceinline__ uint32_t ckpt_kept16(const Ckpt16& f, int i) {
  return kept_bits((i < 2 ? f.idx0 : f.idx1) >> (4 * (i & 1)));
}

// Sum over the kept ones of group i's 4 channels of code * p.
__device__ __forceinline__ float ckpt_kept_dot(const Ckpt16& f, int i, f32x4 p) {
  const uint32_t b = ckpt_kept16(f, i), q = f.codes[i];
  float d = (b & 1u) ? (float)((int)(q << 24) >> 24) * p[0] : 0.f;
  d += (b & 2u) ? (float)((int)(q << 16) >> 24) * p[1] : 0.f;
  d += (b & 4u) ? (float)((int)(q << 8) >> 24) * p[2] : 0.f;
  d += (b & 8u) ? (float)((int)q >> 24) * p[3] : 0.f;
  return d;
}

}  // namespace rtl
