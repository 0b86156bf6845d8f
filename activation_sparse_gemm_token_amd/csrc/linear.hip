// The dense linear layer with bias, activation, gate and residual in its
// epilogue, and its gradients (include/rtlynx_dense.h).
//
// linear_gemm_kernel.  256 x 256 tiles (8 wavefronts of 128 x 64), 256 x 128 (8 of
// 64 x 64) or 128 x 128 (4 of 64 x 64) on v_mfma_f32_16x16x32, operands through rings of LDS tiles 64
// channels deep, filled by direct copies.  An operand whose contraction runs along
// memory rows (x and w, forward) is read with 16-byte reads; one whose contraction
// runs across them (w in dx = dz w; dz and x in dw = dz^T x) lies in LDS as it does
// in memory and is read transposed (ds_read_b64_tr_b16), so no matrix is ever
// transposed in memory.
//
// 4096 x 12288 x 4096 with tanh GELU: 335 us, 1230 TFLOP/s, the matrix cores 62 % busy at the 1.9 GHz
// that power leaves them (a plain library product of 8192^3: 1490).  256 x 256 because a step then moves 64 KiB
// for 2048 cycles of products; the smaller ones where there are too few tiles for the card
// (linear_form).
//
// linear_rows_kernel.  Up to 16 or 32 rows of x are bound by reading w: a workgroup takes 16
// channels of w, its wavefronts share out K.  3 x 4099 x 4096: 11.0 us, 3.1 TB/s.
//
// Sizes with too few tiles for the card split the contraction; linear_join_kernel
// adds the parts in order and applies the epilogue.
#include "rtl_elem.hpp"
#include "gemm_common.hpp"
#include "rtl_operators.hpp"

namespace rtl {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));

template <int TYPE>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (TYPE == kBf16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// --- Activations -------------------------------------------------------------
constexpr int kActGelu = 1, kActGeluTanh = 2, kActSilu = 3;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_(float v) { return __builtin_amdgcn_exp2f(v); }
__device__ __forceinline__ float rcp_(float v) { return __builtin_amdgcn_rcpf(v); }

// Phi(-|z|) = erfc(x) / 2 with x = |z| / sqrt 2, as t 2^(p(t) - x^2 log2 e), t = 1 / (1 + 0.45 x).  p is
// a Chebyshev fit of log2(erfc(x) e^(x^2) / (2 t)) over x in [0, 10]: 7e-7 of the value, 1e-5 with
// fp32's rounding of the exponent where the value is 1e-37.
__device__ __forceinline__ float phi_lower(float z) {
  const float t = rcp_(__builtin_fmaf(__builtin_fabsf(z), 0.45f * 0.7071067811865476f, 1.f));
  float p = -0.2632789611816406f;
  p = __builtin_fmaf(p, t, 1.2530169486999512f);
  p = __builtin_fmaf(p, t, -2.137284755706787f);
  p = __builtin_fmaf(p, t, 1.3746801614761353f);
  p = __builtin_fmaf(p, t, -0.38630765676498413f);
  p = __builtin_fmaf(p, t, 0.7103398442268372f);
  p = __builtin_fmaf(p, t, 1.4257042407989502f);
  p = __builtin_fmaf(p, t, -2.976869583129883f);
  return t * exp2_(__builtin_fmaf(z * z, -0.5f * kLog2e, p));
}
// 2^v below fp32's range is 0 here and 1 / (1 + 2^v) loses nothing by it.
__device__ __forceinline__ float sigmoid2(float v) { return rcp_(1.f + exp2_(-v)); }   // of v / log2 e

constexpr float kTanhA = 0.7978845608028654f, kTanhB = 0.044715f;

// z where it multiplies what vanishes at both ends, or at the lower one: the other factor is exactly 0 from `end` on, so no
// finite z's result changes, and an infinite one (a sum past fp32, or past the type that z is kept in) has its limit
// where inf * 0 would not be a number.  NaN stays: the other factor is NaN then.
__device__ __forceinline__ float within(float z, float end) { return __builtin_amdgcn_fmed3f(z, -end, end); }
__device__ __forceinline__ float above(float z, float end) { return __builtin_amdgcn_fmed3f(z, -end, __builtin_inff()); }
constexpr float kGeluEnd = 64.f, kTanhEnd = 16.f, kSiluEnd = 128.f;

__device__ __forceinline__ float act(float z, int kind) {
  switch (kind) {
    case kActGelu: {
      const float low = within(z, kGeluEnd) * phi_lower(z);                            // z Phi(-|z|)
      return z > 0.f ? z - low : low;
    }
    case kActGeluTanh:                                  // (1 + tanh u) / 2 = 1 / (1 + e^-2u)
      return above(z, kTanhEnd) * sigmoid2(2.f * kLog2e * kTanhA * (z + kTanhB * z * z * z));
    case kActSilu:
      return above(z, kSiluEnd) * sigmoid2(kLog2e * z);
    default:
      return z;
  }
}

// act(z) and act'(z).
__device__ __forceinline__ float act_slope(float z, int kind, float& value) {
  switch (kind) {
    case kActGelu: {
      const float low = phi_lower(z), phi = z > 0.f ? 1.f - low : low, c = within(z, kGeluEnd);
      value = z > 0.f ? z - c * low : c * low;
      return phi + c * 0.3989422804014327f * exp2_(-0.5f * kLog2e * z * z);
    }
    case kActGeluTanh: {
      const float s = sigmoid2(2.f * kLog2e * kTanhA * (z + kTanhB * z * z * z));
      value = above(z, kTanhEnd) * s;
      const float c = within(z, kTanhEnd);              // z^3 may be infinite too
      return s + 2.f * c * s * (1.f - s) * kTanhA * (1.f + 3.f * kTanhB * c * c);
    }
    case kActSilu: {
      const float s = sigmoid2(kLog2e * z);
      value = above(z, kSiluEnd) * s;
      return s * (1.f + within(z, kSiluEnd) * (1.f - s));
    }
    default:
      value = z;
      return 1.f;
  }
}

// --- Epilogue ------------------------------------------------------------------
// W consecutive channels n.. of row m: y = residual + gate act(v + bias).  `wide`: N % W == 0, so
// they lie in one access of every tensor of N columns.  `bias`: of these channels.
template <int TYPE, int W>
__device__ __forceinline__ void bias_load(const LinearEpi& e, int64_t n, int64_t N, float (&bias)[W]) {
#pragma unroll
  for (int i = 0; i < W; ++i) bias[i] = e.bias != nullptr && n + i < N ? word_to_f32<TYPE>(e.bias[n + i]) : 0.f;
}

// The gate of these channels in row m (1 without one), and the first row past its rows.
template <int TYPE, int W>
__device__ __forceinline__ int64_t gate_load(const LinearEpi& e, int64_t m, int64_t n, int64_t N, float (&gate)[W]) {
  if (e.gate == nullptr) {
#pragma unroll
    for (int i = 0; i < W; ++i) gate[i] = 1.f;
    return (int64_t)1 << 62;
  }
  const int64_t row = m / e.gate_tokens;
  const uint16_t* const p = e.gate + row * e.gate_stride + n;
#pragma unroll
  for (int i = 0; i < W; ++i) gate[i] = n + i < N ? word_to_f32<TYPE>(p[i]) : 0.f;
  return (row + 1) * e.gate_tokens;
}

// gate act(v + bias) of channels n.. of row m, whose element is `at`.
template <int TYPE, int W>
__device__ __forceinline__ void activate(const LinearEpi& e, int64_t at, int64_t n, int64_t N, bool wide, const float (&bias)[W],
                                         const float (&gate)[W], float (&v)[W]) {
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] += bias[i];
  if (e.z != nullptr) {
    uint16_t* const z = static_cast<uint16_t*>(e.z);
    float* const z32 = static_cast<float*>(e.z);
    if (wide && e.z_fp32) {
#pragma unroll
      for (int i = 0; i < W; i += 4) store_vec<kFp32, 4>(z32 + at + i, v + i);
    } else if (wide) {
      store_vec<TYPE, W>(z + at, v);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (n + i < N) {
          if (e.z_fp32) z32[at + i] = v[i];
          else z[at + i] = from_f32<TYPE>(v[i]);
        }
    }
  }
  switch (e.act) {                                      // one kind per launch
    case kActGelu:
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = act(v[i], kActGelu);
      break;
    case kActGeluTanh:
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = act(v[i], kActGeluTanh);
      break;
    case kActSilu:
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = act(v[i], kActSilu);
      break;
    default:
      break;
  }
  if (e.gate != nullptr) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] *= gate[i];
  }
}

template <int TYPE, int W>
__device__ __forceinline__ void epilogue(const LinearEpi& e, int64_t m, int64_t n, int64_t N, bool wide, const float (&bias)[W],
                                         const float (&gate)[W], float (&v)[W]) {
  const int64_t at = m * N + n;
  activate<TYPE, W>(e, at, n, N, wide, bias, gate, v);
  if (wide) {
    if (e.residual != nullptr) {
      Raw<TYPE, W> r;
      r.load(e.residual + at);
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] += r.get(i);
    }
    store_vec<TYPE, W>(e.y + at, v);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (n + i < N) {
        if (e.residual != nullptr) v[i] += word_to_f32<TYPE>(e.residual[at + i]);
        e.y[at + i] = from_f32<TYPE>(v[i]);
      }
  }
}

// --- The tiled product ------------------------------------------------------------
// Operand tiles of T rows (of x, w, ..: the output's rows or columns) x 64 of the contraction.
// ALONG: the contraction runs along memory rows; LDS rows are 128 bytes, chunk c of 16 bytes
// of row r in slot c ^ (r & 7).  Across: LDS rows are the 64 contraction rows, 2 T bytes each, chunk c of
// row r in slot c ^ swizzle(r): the 4 rows x 2 chunks of a lane group's transposing read, and two groups
// of them, fall on different banks.
template <int T, int WAVES, bool ALONG>
struct Operand {
  static constexpr int kBytes = T * 128, kPitch = ALONG ? 128 : 2 * T;
  static constexpr int kCount = T / (8 * WAVES);        // copy instructions of each wavefront
  static_assert(kCount == 4 || kCount == 2, "copies of a step");
  // The lane's offset in instruction i: first[set(i)] + i / .. * row_bytes; the swizzle makes two sets across.
  uint32_t first[ALONG ? 1 : 2];
  uint32_t row_bytes, step_bytes;                       // uniform
  int chunk;                                            // ALONG: channel within the step

  __device__ static __forceinline__ uint32_t swizzle(uint32_t row) {
    return ALONG ? row & 7 : (row & 3) << 1 | ((row >> 3) & 1) << 3;
  }
  static constexpr int set(int i) { return ALONG ? 0 : T == 256 ? i & 1 : i >> 1; }
  static constexpr bool starts_set(int i) { return i == 0 || (!ALONG && i == (T == 256 ? 1 : 2)); }
  // Rows from r0 on of a tensor with rows of ld elements.
  __device__ __forceinline__ void init(int wave, int64_t r0, int64_t ld) {
    const uint32_t lane = threadIdx.x & 63, slots = kPitch / 16, rows = 1024 / kPitch;
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      const uint32_t row = (kCount * wave + i) * rows + lane / slots, c = (lane % slots) ^ swizzle(row);
      const uint32_t at = ALONG ? (uint32_t)((r0 + row) * ld * 2 + 16 * c) : (uint32_t)(row * ld * 2 + r0 * 2 + 16 * c);
      if (starts_set(i)) first[set(i)] = at - i * (uint32_t)(rows * ld * 2);
      if (i == 0) chunk = ALONG ? 8 * (int)c : 0;
    }
    row_bytes = __builtin_amdgcn_readfirstlane((uint32_t)(rows * ld * 2));
    step_bytes = ALONG ? 128u : __builtin_amdgcn_readfirstlane((uint32_t)(64 * ld * 2));
  }
  // Step s of a contraction of K: what lies past it arrives as zeros (across: it lies past the buffer).
  __device__ __forceinline__ void copy(__amdgpu_buffer_rsrc_t rs, int64_t s, int64_t K, uint32_t lds, int wave) const {
    const uint32_t so = __builtin_amdgcn_readfirstlane((uint32_t)s * step_bytes);
    const bool inside = !ALONG || s * 64 + chunk < K;
    uint32_t v[kCount];
#pragma unroll
    for (int i = 0; i < kCount; ++i) v[i] = inside ? first[set(i)] + i * row_bytes : kOobOffset - so;
    const uint32_t l0 = __builtin_amdgcn_readfirstlane(lds + 1024u * kCount * wave);
    uint32_t saved;
    if constexpr (kCount == 4)
      asm volatile(
          "s_nop 4\n\ts_mov_b32 %[sv], m0\n\t"
          "s_mov_b32 m0, %[l0]\n\ts_nop 0\n\tbuffer_load_dwordx4 %[v0], %[rs], %[so] offen lds\n\t"
          "s_mov_b32 m0, %[l1]\n\ts_nop 0\n\tbuffer_load_dwordx4 %[v1], %[rs], %[so] offen lds\n\t"
          "s_mov_b32 m0, %[l2]\n\ts_nop 0\n\tbuffer_load_dwordx4 %[v2], %[rs], %[so] offen lds\n\t"
          "s_mov_b32 m0, %[l3]\n\ts_nop 0\n\tbuffer_load_dwordx4 %[v3], %[rs], %[so] offen lds\n\t"
          "s_mov_b32 m0, %[sv]"
          : [sv] "=&s"(saved)
          : [v0] "v"(v[0]), [v1] "v"(v[1]), [v2] "v"(v[2]), [v3] "v"(v[3]), [rs] "s"(rs), [so] "s"(so), [l0] "s"(l0),
            [l1] "s"(l0 + 0x400u), [l2] "s"(l0 + 0x800u), [l3] "s"(l0 + 0xc00u)
          : "memory");
    else
      asm volatile(
          "s_nop 4\n\ts_mov_b32 %[sv], m0\n\t"
          "s_mov_b32 m0, %[l0]\n\ts_nop 0\n\tbuffer_load_dwordx4 %[v0], %[rs], %[so] offen lds\n\t"
          "s_mov_b32 m0, %[l1]\n\ts_nop 0\n\tbuffer_load_dwordx4 %[v1], %[rs], %[so] offen lds\n\t"
          "s_mov_b32 m0, %[sv]"
          : [sv] "=&s"(saved)
          : [v0] "v"(v[0]), [v1] "v"(v[1]), [rs] "s"(rs), [so] "s"(so), [l0] "s"(l0), [l1] "s"(l0 + 0x400u)
          : "memory");
    (void)saved;
  }
  // The lane's byte in the blocks of 16 rows from block `first` on (uniform).
  __device__ static __forceinline__ uint32_t read_base(uint32_t first) {
    const uint32_t lane = threadIdx.x & 63, j = lane & 15;
    if constexpr (ALONG) {
      return first * 2048 + j * 128 + (((lane >> 4) ^ (lane & 7)) << 4);
    } else {
      const uint32_t row = 8 * (lane >> 4) + (j >> 2);
      return row * kPitch + ((2 * first + ((j & 3) >> 1)) ^ swizzle(row)) * 16 + 8 * (j & 1);
    }
  }
  // Block b from there (below 8, and `first` a multiple of the blocks read), contraction half h: along,
  // 16 bytes; across, 4 contraction rows, then the 4 below.
  __device__ static __forceinline__ u32x4 read(const char* tile, uint32_t base, int b, int h) {
    if constexpr (ALONG) {
      return *reinterpret_cast<const u32x4*>(tile + (base ^ (64 * h)) + 2048 * b);
    } else {
      using lds_s16x4 = __attribute__((address_space(3))) s16x4;
      const char* const p = tile + (base ^ (32 * b)) + 32 * h * kPitch;
      const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p)));
      const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * kPitch)));
      return (u32x4){x[0], x[1], y[0], y[1]};
    }
  }
};

template <int TYPE, int TM, int TN, int STAGES, bool A_ALONG, bool B_ALONG>
__global__ void __launch_bounds__(2 * TM, TM == 256 || STAGES > 2 ? 1 : 2)
linear_gemm_kernel(LinearGemm g) {
  constexpr int kWaves = TM / 32, kWavesN = TN / 64, kRB = TM * kWavesN / kWaves / 16, kCB = 4;
  using A = Operand<TM, kWaves, A_ALONG>;
  using B = Operand<TN, kWaves, B_ALONG>;
  constexpr int kStage = A::kBytes + B::kBytes, kCopies = A::kCount + B::kCount;
  constexpr int kRowBytes = 64 * 4 + 16, kStaging = kWaves * 64 * kRowBytes;
  static_assert(kRB == 4 || kRB == 8, "wavefronts cover the tile");
  // A, B of the steps; epilogue.
  __shared__ __attribute__((aligned(16))) char lds[kStaging > STAGES * kStage ? kStaging : STAGES * kStage];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / kWavesN, wn = wave % kWavesN;
  const int64_t tiles_m = (g.M + TM - 1) / TM, tiles_n = (g.N + TN - 1) / TN, tiles = tiles_m * tiles_n;
  const int64_t split = blockIdx.x / tiles;
  int64_t tm, tn;
  tile_coords_of(blockIdx.x - split * tiles, tiles_m, tiles_n, tm, tn);
  const int64_t all = (g.K + 63) / 64, per = (all + g.splits - 1) / g.splits, lo = split * per;
  const int64_t steps = all - lo < per ? all - lo : per;               // may be <= 0: nothing of K left
  const int64_t m0 = tm * TM, n0 = tn * TN;

  const __amdgpu_buffer_rsrc_t ar = make_rsrc(g.a, g.a_bytes), br = make_rsrc(g.b, g.b_bytes);
  A oa;
  B ob;
  oa.init(wave, m0, g.lda);
  ob.init(wave, n0, g.ldb);
  const uint32_t at_a = A::read_base(kRB * wm), at_b = B::read_base(kCB * wn);
  f32x4 acc[kRB][kCB];
#pragma unroll
  for (int i = 0; i < kRB; ++i)
#pragma unroll
    for (int j = 0; j < kCB; ++j) acc[i][j] = (f32x4){0, 0, 0, 0};

  // A ring of stages of both operands.  Half of a step's fragments (32 of the contraction) are in registers ahead of
  // their products: the other half is read from LDS during the first half's products, and the next step's first
  // half during the second's.  The barrier between them comes after the last read of a stage, so the copy of
  // step s + STAGES goes out there: with two stages a whole step before it is waited for, which is enough where
  // other wavefronts fill the wait; a 256 x 128 tile has three, which is what LDS holds, a 128 x 128 tile alone on
  // its CU four.  (One stage more for B, the whole step's fragments read at its top: 429 us for a training step of
  // 4096 x 8192 x 2048, 420 this way then; the loop unrolled over the stages is 2 % faster at 4096 x 12288 x 4096
  // forward but spills where operands run across.)
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)(lds);
  auto copy = [&](int64_t s, int stage) {
    oa.copy(ar, lo + s, g.K, lds0 + stage * kStage, wave);
    ob.copy(br, lo + s, g.K, lds0 + stage * kStage + A::kBytes, wave);
  };
  u32x4 fa[2][kRB], fb[2][kCB];
  using First = std::integral_constant<int, 0>;
  using Second = std::integral_constant<int, 1>;
  auto read = [&](int stage, auto half) {
    constexpr int h = decltype(half)::value;
    const char* const ta = lds + stage * kStage;
#pragma unroll
    for (int j = 0; j < kCB; ++j) fb[h][j] = B::read(ta + A::kBytes, at_b, j, h);
#pragma unroll
    for (int i = 0; i < kRB; ++i) fa[h][i] = A::read(ta, at_a, i, h);
  };
  auto multiply = [&](auto half) {
    constexpr int h = decltype(half)::value;
#pragma unroll
    for (int i = 0; i < kRB; ++i)
#pragma unroll
      for (int j = 0; j < kCB; ++j) acc[i][j] = mfma16<TYPE>(fb[h][j], fa[h][i], acc[i][j]);
  };
  if (steps > 0) {
#pragma unroll
    for (int i = 0; i < STAGES; ++i)
      if (i < steps) copy(i, i);
    if (steps >= STAGES) wait_vm<kCopies * (STAGES - 1)>();
    else wait_vm<0>();
    barrier_no_fence();
    read(0, First{});
    int stage = 0;
#pragma unroll 1
    for (int64_t s = 0; s < steps; ++s) {
      const int next = stage + 1 < STAGES ? stage + 1 : 0;
      read(stage, Second{});
      multiply(First{});
      __builtin_amdgcn_sched_barrier(0);
      // This wavefront's reads of the stage are back, and its copies of the next one.
      if (s + STAGES - 1 < steps) wait_vm<kCopies * (STAGES - 2)>();
      else wait_vm<0>();
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      barrier_no_fence();
      // A wavefront waits while its copies go out.  Of the two on a SIMD (8 wavefronts) one copies before its
      // products, the other after, so that the matrix core has the other's meanwhile (4096 x 12288 x 4096 with
      // GELU: 345 us with both before, 329).
      const bool more = s + STAGES < steps;
      if (more && (kWaves == 4 || wave < 4)) copy(s + STAGES, stage);
      __builtin_amdgcn_sched_barrier(0);
      read(next, First{});                              // after the last step: not used
      multiply(Second{});
      __builtin_amdgcn_sched_barrier(0);
      if (kWaves == 8 && more && wave >= 4) copy(s + STAGES, stage);
      stage = next;
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
  barrier_no_fence();                                   // the rings are free
  // Through LDS, 64 rows x 64 channels of the wavefront at a time, so that a lane has 8 consecutive
  // channels of a row (16 bytes of y) and the epilogue is one short loop.
  char* const mine = lds + wave * 64 * kRowBytes;
  const int64_t n = n0 + 64 * wn + 8 * (lane & 7);
  const bool wide = g.N % 8 == 0, whole = wide && g.splits == 1 && g.e.residual != nullptr;
  const bool changed = g.e.bias != nullptr || g.e.gate != nullptr || g.e.z != nullptr || g.e.act != 0;
  float bias[8], gate[8];
  bias_load<TYPE, 8>(g.e, n, g.N, bias);
  int64_t gate_end = 0;
#pragma unroll
  for (int pass = 0; pass < kRB / 4; ++pass) {
    // The residual of the lane's 8 rows is asked for at once: one at a time, each would wait for memory.
    const int64_t m = m0 + 16 * kRB * wm + 64 * pass + (lane >> 3);
    Raw<TYPE, 8> residual[8];
#pragma unroll
    for (int it = 0; it < 8; ++it) {
      residual[it].zero();
      if (whole && m + 8 * it < g.M && n < g.N) residual[it].load(g.e.residual + (m + 8 * it) * g.N + n);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < kCB; ++j)
        *reinterpret_cast<f32x4*>(mine + (16 * i + (lane & 15)) * kRowBytes + (16 * j + 4 * (lane >> 4)) * 4) = acc[4 * pass + i][j];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (whole) {
      if (changed) {
#pragma unroll 1
        for (int it = 0; it < 8; ++it) {
          f32x4* const p = reinterpret_cast<f32x4*>(mine + (8 * it + (lane >> 3)) * kRowBytes + 32 * (lane & 7));
          const f32x4 v0 = p[0], v1 = p[1];
          float v[8] = {v0[0], v0[1], v0[2], v0[3], v1[0], v1[1], v1[2], v1[3]};
          const int64_t r = m + 8 * it;
          if (r >= g.M || n >= g.N) continue;
          if (r >= gate_end) gate_end = gate_load<TYPE, 8>(g.e, r, n, g.N, gate);
          activate<TYPE, 8>(g.e, r * g.N + n, n, g.N, true, bias, gate, v);
          p[0] = (f32x4){v[0], v[1], v[2], v[3]};
          p[1] = (f32x4){v[4], v[5], v[6], v[7]};
        }
      }
#pragma unroll
      for (int it = 0; it < 8; ++it) {
        const f32x4* const p = reinterpret_cast<const f32x4*>(mine + (8 * it + (lane >> 3)) * kRowBytes + 32 * (lane & 7));
        const f32x4 v0 = p[0], v1 = p[1];
        float v[8] = {v0[0], v0[1], v0[2], v0[3], v1[0], v1[1], v1[2], v1[3]};
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += residual[it].get(e);
        if (m + 8 * it < g.M && n < g.N) store_vec<TYPE, 8>(g.e.y + (m + 8 * it) * g.N + n, v);
      }
    } else
#pragma unroll 1
    for (int it = 0; it < 8; ++it) {
      const char* const p = mine + (8 * it + (lane >> 3)) * kRowBytes + 32 * (lane & 7);
      const f32x4 v0 = *reinterpret_cast<const f32x4*>(p), v1 = *reinterpret_cast<const f32x4*>(p + 16);
      float v[8] = {v0[0], v0[1], v0[2], v0[3], v1[0], v1[1], v1[2], v1[3]};
      const int64_t r = m + 8 * it;
      if (r >= g.M || n >= g.N) continue;
      if (g.splits > 1) {
        float* const out = g.part + (split * g.M + r) * g.N + n;
        if (wide) {
          *reinterpret_cast<f32x4*>(out) = v0;
          *reinterpret_cast<f32x4*>(out + 4) = v1;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n + e < g.N) out[e] = v[e];
        }
      } else {
        if (r >= gate_end) gate_end = gate_load<TYPE, 8>(g.e, r, n, g.N, gate);
        epilogue<TYPE, 8>(g.e, r, n, g.N, wide, bias, gate, v);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the next pass writes over what was read
  }
}

template <int TYPE>
__global__ void __launch_bounds__(256)
linear_join_kernel(LinearGemm g) {
  const int64_t per_row = (g.N + 3) / 4, i = folded_block() * 256 + threadIdx.x;
  const int64_t m = i / per_row, n = 4 * (i - m * per_row);
  if (m >= g.M) return;
  const bool wide = g.N % 4 == 0;
  float bias[4], v[4] = {0.f, 0.f, 0.f, 0.f};
  bias_load<TYPE, 4>(g.e, n, g.N, bias);
  for (int s = 0; s < g.splits; ++s) {
    const float* const p = g.part + (s * g.M + m) * g.N + n;
    if (wide) {
      const f32x4 q = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += q[e];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < g.N) v[e] += p[e];
    }
  }
  float gate[4];
  gate_load<TYPE, 4>(g.e, m, n, g.N, gate);
  epilogue<TYPE, 4>(g.e, m, n, g.N, wide, bias, gate, v);
}

// --- Few rows ------------------------------------------------------------------
// w as the matrix core's rows straight from memory (lane l: channel row l % 16, 8 of K at 8 (l / 16)), x
// likewise as its columns; kRowWaves wavefronts take 64 of K in turn.
constexpr int kRowWaves = 8;

template <int TYPE, int MT>
__global__ void __launch_bounds__(64 * kRowWaves)
linear_rows_kernel(LinearGemm g) {
  __shared__ f32x4 lds[kRowWaves / 2][MT][64];
  const int lane = threadIdx.x & 63, row = lane & 15, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int64_t wrow = n0 + row < g.N ? n0 + row : g.N - 1;
  const uint16_t* const w = static_cast<const uint16_t*>(g.b) + wrow * g.K;
  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = (f32x4){0, 0, 0, 0};
  constexpr int kDeep = 4;                              // steps of 64 whose loads go out together
  for (int64_t k0 = 64 * wave; k0 < g.K; k0 += 64 * kRowWaves * kDeep) {
    u32x4 a[kDeep][2], b[kDeep][2][MT];
#pragma unroll
    for (int d = 0; d < kDeep; ++d)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t k = k0 + 64 * kRowWaves * d + 32 * h + 8 * (lane >> 4);
        a[d][h] = (u32x4){0, 0, 0, 0};
        if (k < g.K) a[d][h] = *reinterpret_cast<const u32x4*>(w + k);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          b[d][h][i] = (u32x4){0, 0, 0, 0};
          if (k < g.K && 16 * i + row < g.M)
            b[d][h][i] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(g.a) + (16 * i + row) * g.K + k);
        }
      }
#pragma unroll
    for (int d = 0; d < kDeep; ++d)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[i] = mfma16<TYPE>(a[d][h], b[d][h][i], acc[i]);
  }
#pragma unroll
  for (int half = kRowWaves / 2; half >= 1; half /= 2) {
    __syncthreads();
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int i = 0; i < MT; ++i) lds[wave - half][i][lane] = acc[i];
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[i] += lds[wave][i][lane];
    }
  }
  if (wave != 0) return;
  const int64_t n = n0 + 4 * (lane >> 4);
  float bias[4];
  bias_load<TYPE, 4>(g.e, n, g.N, bias);
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    float v[4] = {acc[i][0], acc[i][1], acc[i][2], acc[i][3]};
    if (16 * i + row < g.M && n < g.N) {
      float gate[4];
      gate_load<TYPE, 4>(g.e, 16 * i + row, n, g.N, gate);
      epilogue<TYPE, 4>(g.e, 16 * i + row, n, g.N, g.N % 4 == 0, bias, gate, v);
    }
  }
}

// --- dz, dbias, dgate -------------------------------------------------------------
// A workgroup takes 32 VEC columns and a part of a gate row's rows, 8 rows at a time; it leaves
// one row of sums for the part.  dz rows are np elements, a multiple of 8, zeros past N.
template <int TYPE, int ZTYPE, int VEC>
__global__ void __launch_bounds__(256)
linear_dz_kernel(LinearDz a) {
  __shared__ float lds[8][32 * VEC];
  const int t = threadIdx.x & 31, sub = threadIdx.x >> 5;
  const int64_t c = ((int64_t)blockIdx.x * 32 + t) * VEC, group = blockIdx.y / a.parts, part = blockIdx.y % a.parts;
  const int64_t rows = a.M / a.groups, per = (rows + a.parts - 1) / a.parts;
  const int64_t lo = part * per, hi = lo + per < rows ? lo + per : rows;
  float gate[VEC], bias_sum[VEC], gate_sum[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    gate[j] = a.gate != nullptr && c + j < a.N ? word_to_f32<TYPE>(a.gate[group * a.gate_stride + c + j]) : 1.f;
    bias_sum[j] = gate_sum[j] = 0.f;
  }
  if (c < a.np) {
    for (int64_t r = lo + sub; r < hi; r += 8) {
      const int64_t at = (group * rows + r) * a.N + c;
      Raw<TYPE, VEC> dy;
      Raw<ZTYPE, VEC> z;
      dy.zero();
      z.zero();
      if (c < a.N) {                                    // VEC divides N, or is 1
        dy.load(a.dy + at);
        if (a.z != nullptr) z.load(static_cast<const elem_t<ZTYPE>*>(a.z) + at);
      }
      float out[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float d = dy.get(j);
        float value, dz = d * gate[j] * act_slope(z.get(j), a.act, value);
        bias_sum[j] += dz;
        gate_sum[j] += d * value;
        out[j] = dz;
      }
      if (a.dz != nullptr) store_vec<TYPE, VEC>(a.dz + (group * rows + r) * a.np + c, out);
    }
  }
  // Sums of the 8 sets of rows, in order.
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* const out = which == 0 ? a.bias_part : a.gate_part;
    if (out == nullptr) continue;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < VEC; ++j) lds[sub][t * VEC + j] = which == 0 ? bias_sum[j] : gate_sum[j];
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * VEC; i += 256) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) s += lds[k][i];
      const int64_t col = (int64_t)blockIdx.x * 32 * VEC + i;
      if (col < a.N) out[(int64_t)blockIdx.y * a.N + col] = s;
    }
  }
}

// dbias, the sum of all parts' rows, and dgate, of each gate row's parts, in order (16 threads a column).
// Workgroups: dbias's columns (where it is wanted), then dgate's by rows.
template <int TYPE>
__global__ void __launch_bounds__(1024)
linear_sums_kernel(LinearDz a) {
  __shared__ float lds[16][64];
  const int col = threadIdx.x & 63, p = threadIdx.x >> 6;
  const int64_t C = a.N, per = (C + 63) / 64, bias = a.dbias != nullptr ? per : 0, id = folded_block();
  const bool is_gate = id >= bias;
  const int64_t row = is_gate ? (id - bias) / per : 0, c = ((is_gate ? id - bias : id) - row * per) * 64 + col;
  if (row >= (a.dgate != nullptr || !is_gate ? a.groups : 0)) return;
  const float* const partials = is_gate ? a.gate_part : a.bias_part;
  const int64_t parts = is_gate ? a.parts : a.groups * a.parts;
  uint16_t* const out = is_gate ? a.dgate : a.dbias;
  float s = 0.f;
  if (c < C)
    for (int64_t i = p; i < parts; i += 16) s += partials[(row * parts + i) * C + c];
  lds[p][col] = s;
  __syncthreads();
  if (p != 0 || c >= C) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) s += lds[i][col];
  out[row * C + c] = from_f32<TYPE>(s);
}

template <int TYPE, bool A_ALONG, bool B_ALONG>
hipError_t run_gemm(const LinearGemm& g, hipStream_t stream) {
  const int64_t tiles = ((g.M + g.tile_m - 1) / g.tile_m) * ((g.N + g.tile_n - 1) / g.tile_n);
  const dim3 grid((unsigned)(tiles * g.splits));
  hipError_t e;
  if (g.tile_n == 256) e = launch(&linear_gemm_kernel<TYPE, 256, 256, 2, A_ALONG, B_ALONG>, grid, dim3(512), stream, g);
  else if (g.tile_m == 256) e = launch(&linear_gemm_kernel<TYPE, 256, 128, 3, A_ALONG, B_ALONG>, grid, dim3(512), stream, g);
  else if (tiles * g.splits > 256) e = launch(&linear_gemm_kernel<TYPE, 128, 128, 2, A_ALONG, B_ALONG>, grid, dim3(256), stream, g);
  else e = launch(&linear_gemm_kernel<TYPE, 128, 128, 4, A_ALONG, B_ALONG>, grid, dim3(256), stream, g);
  if (e != hipSuccess || g.splits == 1) return e;
  return launch(&linear_join_kernel<TYPE>, folded_grid((g.M * ((g.N + 3) / 4) + 255) / 256), dim3(256), stream, g);
}

template <int TYPE>
hipError_t run_linear(const LinearGemm& g, hipStream_t stream) {
  if (g.tile_m == 0) {
    const dim3 grid((unsigned)((g.N + 15) / 16)), block(64 * kRowWaves);
    return g.M <= 16 ? launch(&linear_rows_kernel<TYPE, 1>, grid, block, stream, g)
                     : launch(&linear_rows_kernel<TYPE, 2>, grid, block, stream, g);
  }
  return run_gemm<TYPE, true, true>(g, stream);
}

template <int TYPE>
hipError_t run_dz(const LinearDz& a, hipStream_t stream) {
  const bool wide = a.N % 8 == 0;
  const int64_t cols = 32 * (wide ? 8 : 1);
  const dim3 grid((unsigned)((a.np + cols - 1) / cols), (unsigned)(a.groups * a.parts));
  auto* k = a.z_fp32 ? (wide ? &linear_dz_kernel<TYPE, kFp32, 8> : &linear_dz_kernel<TYPE, kFp32, 1>)
                     : (wide ? &linear_dz_kernel<TYPE, TYPE, 8> : &linear_dz_kernel<TYPE, TYPE, 1>);
  hipError_t e = launch(k, grid, dim3(256), stream, a);
  const int64_t blocks = (a.N + 63) / 64 * ((a.dbias != nullptr ? 1 : 0) + (a.dgate != nullptr ? a.groups : 0));
  if (e != hipSuccess || blocks == 0) return e;
  return launch(&linear_sums_kernel<TYPE>, folded_grid_of_1024(blocks), dim3(1024), stream, a);
}

}  // namespace

// Tile and ranges of the contraction for a product [M, N] over K: the form with the least expected time, in us, from
// measured rates.  A step of 64 takes a 256 x 256 tile 1.48, a 256 x 128 tile 0.85 (one workgroup per CU each) and 128 x
// 128 tiles 0.55 alone on their CU, 0.95 where two share it; a tile takes 9, 7 and 4 more to begin and end.  Ranges of the
// contraction cost a second launch and their fp32 parts, written and read at 4 TB/s.  Measured with the three tiles, bf16:
// 8192 x 2048 x 4096: 107, 122 and 129; 4096 x 2048 x 8192: 163, 116 and 126; 2048 x 2048 x 2048: 48, 31 and 28; 2310 x
// 1160 x 1152: 18 with the smallest, 33 with it and three ranges.
//
// Up to 16 rows go to the kernel for few rows, 17 to 32 where it is expected to take less (its time and the tiles' measured,
// 3 us more than above in these sizes): 32 x 4096 x 4096: 15 us, tiles 18; 32 x 12288 x 4096: 43 and 30.  (Of very wide
// weights tiles would do for 16 rows too: 16 x 24576 x 4096 46 us, 17 rows in tiles 41.)
LinearForm linear_form(int64_t M, int64_t N, int64_t K, bool rows_kernel) {
  if (rows_kernel && M <= 16) return {0, 0, 1};
  const int64_t m256 = (M + 255) / 256, m128 = (M + 127) / 128, n256 = (N + 255) / 256, n128 = (N + 127) / 128;
  const int64_t small = m128 * n128, steps = (K + 63) / 64;
  if (small == 0 || steps == 0) return {128, 128, 1};
  LinearForm best{256, 256, 1};
  double least = (double)((m256 * n256 + 255) / 256) * (1.48 * (double)steps + 9.0);
  const double mixed = (double)((m256 * n128 + 255) / 256) * (0.85 * (double)steps + 7.0);
  if (mixed < least) {
    least = mixed;
    best = {256, 128, 1};
  }
  for (int64_t splits = 1; splits <= 16 && (splits == 1 || steps / splits >= 4); splits *= 2) {
    const int64_t groups = small * splits, each = (steps + splits - 1) / splits;
    double t = groups <= 256 ? 0.55 * (double)each + 4.0 : (double)((groups + 511) / 512) * (0.95 * (double)each + 4.0);
    if (splits > 1) t += 4.0 + (double)splits * (double)M * (double)N * 8.0 / 4e6;
    if (t < least) {
      least = t;
      best = {128, 128, (int)splits};
    }
  }
  if (rows_kernel && M <= 32 && 2.0 + 2e-6 * (double)N * (double)K * (0.21 + 0.0064 * (double)M) < least + 3.0) return {0, 0, 1};
  return best;
}

int64_t linear_dz_parts(int64_t M, int64_t N, int64_t groups) {
  if (N == 0) return 1;
  const int64_t cols = N % 8 == 0 ? 256 : 32, blocks = (N + cols - 1) / cols * groups;
  int64_t parts = (2048 + blocks - 1) / blocks;
  const int64_t most = (M / groups + 31) / 32;
  if (parts > most) parts = most;
  if (parts * groups > 65535) parts = 65535 / groups;
  return parts < 1 ? 1 : parts;
}

hipError_t launch_linear(const LinearGemm& g, bool fp16, hipStream_t stream) {
  return fp16 ? run_linear<kFp16>(g, stream) : run_linear<kBf16>(g, stream);
}
hipError_t launch_linear_dx(const LinearGemm& g, bool fp16, hipStream_t stream) {
  return fp16 ? run_gemm<kFp16, true, false>(g, stream) : run_gemm<kBf16, true, false>(g, stream);
}
hipError_t launch_linear_dw(const LinearGemm& g, bool fp16, hipStream_t stream) {
  return fp16 ? run_gemm<kFp16, false, false>(g, stream) : run_gemm<kBf16, false, false>(g, stream);
}
hipError_t launch_linear_dz(const LinearDz& a, bool fp16, hipStream_t stream) {
  return fp16 ? run_dz<kFp16>(a, stream) : run_dz<kBf16>(a, stream);
}

}  // namespace rtl
