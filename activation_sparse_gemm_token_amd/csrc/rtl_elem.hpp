// Elements of the three tensor types as fp32 in registers (internal).
#pragma once

#include "rtl_common.hpp"

namespace rtl {

constexpr int kBf16 = 0, kFp16 = 1, kFp32 = 2;

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

template <int TYPE>
using elem_t = std::conditional_t<TYPE == kFp32, float, uint16_t>;

template <int TYPE>
__device__ __forceinline__ float word_to_f32(uint32_t low16) {
  if constexpr (TYPE == kBf16) return __builtin_bit_cast(float, low16 << 16);
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)low16);
}

// Two fp32 values as packed words of a 16-bit type, round to nearest even.
template <int TYPE>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (TYPE == kBf16) return cvt_pk_bf16(a, b);
  else return __builtin_bit_cast(uint32_t, (f16x2){(_Float16)a, (_Float16)b});
}

template <int TYPE>
__device__ __forceinline__ elem_t<TYPE> from_f32(float a) {
  if constexpr (TYPE == kFp32) return a;
  else return (uint16_t)pack2<TYPE>(a, 0.f);
}

// VEC consecutive elements: one access of VEC * size bytes (two of 16 for 32), which the
// caller's alignment allows.
template <int TYPE, int VEC>
struct Raw {
  static constexpr int kBytes = VEC * (TYPE == kFp32 ? 4 : 2);
  static constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const elem_t<TYPE>* p) {
    if constexpr (kBytes == 2) {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else if constexpr (kBytes == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (kBytes == 8) {
      const u32x2 v = *reinterpret_cast<const u32x2*>(p);
      w[0] = v[0], w[1] = v[1];
    } else {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const u32x4 v = reinterpret_cast<const u32x4*>(p)[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * i + j] = v[j];
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (TYPE == kFp32) return __builtin_bit_cast(float, w[i]);
    else return word_to_f32<TYPE>((w[i / 2] >> (16 * (i % 2))) & 0xffffu);
  }
};

template <int TYPE, int VEC>
__device__ __forceinline__ void store_vec(elem_t<TYPE>* p, const float* v) {
  if constexpr (VEC == 1) {
    *p = from_f32<TYPE>(v[0]);
  } else if constexpr (TYPE == kFp32) {
    static_assert(VEC == 4, "16 bytes of fp32");
    *reinterpret_cast<f32x4*>(p) = (f32x4){v[0], v[1], v[2], v[3]};
  } else if constexpr (VEC == 4) {
    *reinterpret_cast<u32x2*>(p) = (u32x2){pack2<TYPE>(v[0], v[1]), pack2<TYPE>(v[2], v[3])};
  } else {
    static_assert(VEC == 8, "16 bytes of 16-bit values");
    *reinterpret_cast<u32x4*>(p) = (u32x4){pack2<TYPE>(v[0], v[1]), pack2<TYPE>(v[2], v[3]),
                                           pack2<TYPE>(v[4], v[5]), pack2<TYPE>(v[6], v[7])};
  }
}

}  // namespace rtl
