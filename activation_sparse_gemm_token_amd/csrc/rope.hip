// rtl_rope: rotary positions on strided [batch, tokens, heads, head_dim]
// tensors (include/rtlynx_rope.h).
//
// A workgroup takes a few consecutive tokens.  It first forms the sine and
// cosine of each token's angles once, in LDS, and then streams the heads of
// up to two tensors (queries and keys) through them, so the fp64 angle and
// the sine cost one evaluation per (token, pair), not one per head.
//
// A thread's unit is 16 bytes of a head where the layout's alignment allows (in
// the half layout 16 bytes from each half of the rotated part), else the widest
// power of two that does, and the kernel is bound by memory: each element is read
// once and written once.  With inputs and outputs out of the caches 2 x 4608 tokens,
// 24 + 24 heads of 128, bf16 take 46 us (4.9 TB/s; a copy reaches 5.15) and 32768
// tokens, 10 heads of 64, fp32 35 us; with the same ones again and again, partly in
// the last-level cache, 35 and 28.  One token, 40 heads: 3.3 us.
#include "rtl_common.hpp"
#include "rtl_operators.hpp"

namespace rtl {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;              // units in flight per thread

struct Bf16 {
  using raw = uint16_t;
  static __device__ __forceinline__ float up(raw v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }
  static __device__ __forceinline__ raw down(float v) { return (raw)cvt_pk_bf16(v, v); }
};
struct Fp16 {
  using raw = uint16_t;
  static __device__ __forceinline__ float up(raw v) { return (float)__builtin_bit_cast(_Float16, v); }
  static __device__ __forceinline__ raw down(float v) { return __builtin_bit_cast(raw, (_Float16)v); }
};
struct Fp32 {
  using raw = uint32_t;
  static __device__ __forceinline__ float up(raw v) { return __builtin_bit_cast(float, v); }
  static __device__ __forceinline__ raw down(float v) { return __builtin_bit_cast(raw, v); }
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T v[V];
};

// Sine and cosine of position * inv_freq.  The product, its reduction to
// turns and then to the nearest quarter turn are fp64 (exact to fp32 as long
// as the angle is below 2^28 radians); the remaining eighth of a turn either
// side is fp32.
__device__ __forceinline__ void angle(int64_t pos, double inv_freq, float& s, float& c) {
  const double turns = (double)pos * inv_freq * 0.15915494309189533577;   // 1 / (2 pi)
  const double quarters = 4.0 * (turns - __builtin_rint(turns));         // [-2, 2]
  const double q = __builtin_rint(quarters);
  float sr, cr;
  sincospif(0.5f * (float)(quarters - q), &sr, &cr);
  const int n = (int)q & 3;
  const float ss = (n & 1) ? cr : sr, cc = (n & 1) ? sr : cr;
  s = (n & 2) ? -ss : ss;
  c = (n == 1 || n == 2) ? -cc : cc;
}

// V elements per access.  Units of one head: rot / (2 V) pairs of V-element
// pieces in the half layout, rot / V pieces in the interleaved one (rot / 2
// pairs of single elements when V is 1), then the (dim - rot) / V pieces
// that are copied, two to a unit where a rotated one has two (3 x 1155 tokens, 24
// heads of 96 with 40 turned, fp16: 11.2 us against 13.8; interleaved units of one
// and two pieces side by side took 26 us instead of 17).  A row is (token, head); blockIdx.y takes every gridDim.y-th
// block of rows.  A thread keeps its unit and walks rows, kUnroll at a time; the
// first of them are requested before the angles are formed.
template <typename E, int V, bool INTER>
__global__ void __launch_bounds__(kThreads)
rope_kernel(RopeArgs a) {
  using raw = typename E::raw;
  using P = Pack<raw, V>;
  extern __shared__ float table[];                 // [token][cos pairs, sin pairs]
  const int pairs = a.rot / 2;
  const int64_t tok0 = folded_block() * a.group;
  if (tok0 >= a.total) return;
  const int ntok = (int)(a.total - tok0 < a.group ? a.total - tok0 : a.group);
  const int64_t b0 = tok0 / a.tokens, t0 = tok0 - b0 * a.tokens;
  // Batch and position of local token t: the group's tokens are consecutive.
  auto place = [&](int t, int64_t& b, int64_t& tt) {
    b = b0;
    tt = t0 + t;
    while (tt >= a.tokens) { tt -= a.tokens; ++b; }
  };

  constexpr int kPer = INTER ? (V == 1 ? 2 : V) : 2 * V;     // rotated elements per unit
  constexpr bool kTwo = !INTER || V == 1;                    // pieces per unit
  constexpr int kCopy = kTwo ? 2 * V : V;
  const int rot_units = a.rot / kPer;
  const int units = rot_units + (a.dim - a.rot + kCopy - 1) / kCopy;
  const int heads = a.t[0].heads + a.t[1].heads;
  const int lanes = units < kThreads ? units : kThreads;     // threads along a head
  const int rows_at_once = kThreads / lanes;
  const int sub = threadIdx.x / lanes;
  const int step = rows_at_once * (int)gridDim.y;
  const int first = sub * (int)gridDim.y + (int)blockIdx.y;
  const int step_t = step / heads, step_h = step - step_t * heads;
  const int first_t = first / heads, first_h = first - first_t * heads;

  // A batch of rows of unit u: what was read, where it goes, its token's table.
  P x0[kUnroll], x1[kUnroll];
  raw* dst[kUnroll];
  int tk[kUnroll];
  int u = threadIdx.x - sub * lanes, t = first_t, h = first_h;
  bool turn = false, two = false;
  int o0 = 0, o1 = 0;                              // element offsets of the unit's pieces in its head
  auto unit = [&]() {
    turn = u < rot_units;
    if (turn) {
      o0 = INTER ? (V == 1 ? 2 * u : V * u) : V * u;
      o1 = INTER ? o0 + 1 : o0 + pairs;
      two = kTwo;
    } else {
      o0 = a.rot + (u - rot_units) * kCopy;
      o1 = o0 + V;
      two = kTwo && o1 < a.dim;
    }
  };
  auto load = [&]() {
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      dst[j] = nullptr;
      if (t < ntok) {
        const int w = h >= a.t[0].heads;
        const RopeSide& z = a.t[w];
        if (turn || !z.in_place) {
          const int64_t hh = h - (w ? a.t[0].heads : 0);
          int64_t b, tt;
          place(t, b, tt);
          const raw* src = static_cast<const raw*>(z.x) + b * z.xb + tt * z.xt + hh * z.xh;
          dst[j] = static_cast<raw*>(z.y) + b * z.yb + tt * z.yt + hh * z.yh;
          tk[j] = t;
          x0[j] = *reinterpret_cast<const P*>(src + o0);
          if (two) x1[j] = *reinterpret_cast<const P*>(src + o1);
        }
      }
      t += step_t;
      h += step_h;
      if (h >= heads) { h -= heads; ++t; }
    }
  };
  const bool active = sub < rows_at_once && u < units;
  if (active) {
    unit();
    load();
  }

  for (int i = threadIdx.x; i < ntok * pairs; i += kThreads) {
    const int n = i / pairs, p = i - n * pairs;
    int64_t b, tt;
    place(n, b, tt);
    const int axis = (p >= a.axis_end[0]) + (p >= a.axis_end[1]) + (p >= a.axis_end[2]);
    float s, c;
    angle(a.positions[b * a.pos_b + tt * a.pos_t + axis], a.inv_freq[p], s, c);
    table[2 * pairs * n + p] = c * a.scale;
    table[2 * pairs * n + pairs + p] = (a.inverse ? -s : s) * a.scale;
  }
  __syncthreads();
  if (!active) return;

  for (;;) {
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      if (dst[j] == nullptr) continue;
      if (!turn) {
        *reinterpret_cast<P*>(dst[j] + o0) = x0[j];
        if (two) *reinterpret_cast<P*>(dst[j] + o1) = x1[j];
        continue;
      }
      const float* tc = table + 2 * pairs * tk[j];
      if constexpr (INTER && V > 1) {
        const float* c = tc + (V / 2) * u;
        P y;
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          const float p = E::up(x0[j].v[2 * e]), q = E::up(x0[j].v[2 * e + 1]);
          const float cc = c[e], ss = c[pairs + e];
          y.v[2 * e] = E::down(p * cc - q * ss);
          y.v[2 * e + 1] = E::down(q * cc + p * ss);
        }
        *reinterpret_cast<P*>(dst[j] + o0) = y;
      } else {
        const float* c = tc + V * u;
        P y0, y1;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float p = E::up(x0[j].v[e]), q = E::up(x1[j].v[e]);
          const float cc = c[e], ss = c[pairs + e];
          y0.v[e] = E::down(p * cc - q * ss);
          y1.v[e] = E::down(q * cc + p * ss);
        }
        *reinterpret_cast<P*>(dst[j] + o0) = y0;
        *reinterpret_cast<P*>(dst[j] + o1) = y1;
      }
    }
    if (t >= ntok) {                               // this unit's rows are done
      u += lanes;
      if (u >= units) return;
      unit();
      t = first_t;
      h = first_h;
    }
    load();
  }
}

template <typename E, int V>
hipError_t launch_v(const RopeArgs& a, bool inter, dim3 grid, size_t lds, hipStream_t stream) {
  RopeArgs args = a;
  void* ptrs[] = {&args};
  const void* k = inter ? reinterpret_cast<const void*>(&rope_kernel<E, V, true>)
                        : reinterpret_cast<const void*>(&rope_kernel<E, V, false>);
  return hipLaunchKernel(k, grid, dim3(kThreads), ptrs, lds, stream);
}

}  // namespace

hipError_t launch_rope(RopeArgs a, int elem_bytes, bool fp16, bool inter, int compute_units, hipStream_t stream) {
  // Bytes per access: the largest power of two up to 16 that divides every
  // address the call forms (and, in the interleaved layout, holds whole
  // pairs: pieces of single elements otherwise).
  uint64_t bits = 16 | (uint64_t)a.dim * elem_bytes;
  bits |= (uint64_t)(inter ? a.rot : a.rot / 2) * elem_bytes;
  for (const RopeSide& z : a.t) {
    if (z.heads == 0) continue;
    bits |= reinterpret_cast<uintptr_t>(z.x) | reinterpret_cast<uintptr_t>(z.y);
    for (int64_t s : {z.xb, z.xt, z.xh, z.yb, z.yt, z.yh}) bits |= (uint64_t)s * (uint64_t)elem_bytes;
  }
  const int vec = (int)(bits & (~bits + 1)) / elem_bytes;
  const int heads = a.t[0].heads + a.t[1].heads;
  const int pairs = a.rot / 2;
  // Tokens per workgroup: enough rows that a thread has kUnroll units or so,
  // but no fewer than four workgroups per CU where the call has the tokens.
  const int64_t rows_wanted = (int64_t)kThreads * kUnroll * 16 / (elem_bytes * (int64_t)a.dim) + 1;
  int64_t group = (rows_wanted + heads - 1) / heads;
  const int64_t fill = a.total / (4 * (int64_t)compute_units);
  if (group > fill) group = fill;
  const int64_t fit = pairs > 0 ? 2048 / pairs : group;          // 16 KiB of LDS (one token: up to 4 KiB)
  if (group > fit) group = fit;
  if (group < 1) group = 1;
  a.group = (int)group;
  const int64_t blocks = (a.total + group - 1) / group;
  // Few tokens: heads split over workgroups too, each forming the angles anew.
  int64_t split = 1;
  if (blocks < compute_units) {
    const int64_t units = (int64_t)a.dim * elem_bytes / (vec * elem_bytes);
    const int64_t all = group * heads * units;
    split = compute_units / blocks;
    const int64_t most = (all + kThreads - 1) / kThreads;
    if (split > most) split = most;
  }
  const dim3 grid = folded_grid(blocks, (unsigned)split);
  const size_t lds = (size_t)group * 2 * pairs * sizeof(float);
  if (elem_bytes == 4) {
    if (vec >= 4) return launch_v<Fp32, 4>(a, inter, grid, lds, stream);
    if (vec >= 2) return launch_v<Fp32, 2>(a, inter, grid, lds, stream);
    return launch_v<Fp32, 1>(a, inter, grid, lds, stream);
  }
  if (fp16) {
    if (vec >= 8) return launch_v<Fp16, 8>(a, inter, grid, lds, stream);
    if (vec >= 4) return launch_v<Fp16, 4>(a, inter, grid, lds, stream);
    if (vec >= 2) return launch_v<Fp16, 2>(a, inter, grid, lds, stream);
    return launch_v<Fp16, 1>(a, inter, grid, lds, stream);
  }
  if (vec >= 8) return launch_v<Bf16, 8>(a, inter, grid, lds, stream);
  if (vec >= 4) return launch_v<Bf16, 4>(a, inter, grid, lds, stream);
  if (vec >= 2) return launch_v<Bf16, 2>(a, inter, grid, lds, stream);
  return launch_v<Bf16, 1>(a, inter, grid, lds, stream);
}

}  // namespace rtl
