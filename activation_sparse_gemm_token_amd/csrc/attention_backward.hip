// Attention, backward (include/rtlynx_attention.h).
//
//   1. attn_delta_kernel   D = sum of d_o o per query and head, and the log-sum-exp in
//                          log2 units.
//   2. attn_dkv_kernel     dK, dV: a wavefront holds 32 keys, its workgroup walks the
//                          queries of all heads that share the key head.
//   3. attn_dq_kernel      dQ: as the forward pass, 32 queries a wavefront.
//
// S and dP are formed in both (7 products where 5 would do with atomic sums), so
// nothing is added atomically and shared heads sum in registers.  Everything
// between the products stays in registers: a lane's P and dS are operands as they
// stand (attn_common.hpp).  P and dS are rounded to bf16 there; S, dP and all sums
// are fp32.
#include "attn_common.hpp"

namespace rtl {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_(float v) { return __builtin_amdgcn_exp2f(v); }

// 16 lanes a row, 8 channels each.  Rows of a packed batch that lie in no sequence are
// worked on too; nothing reads their values.
__global__ void __launch_bounds__(256)
attn_delta_kernel(AttnBackArgs a) {
  const int lane = threadIdx.x & 15;
  const bool packed = a.f.q_starts != nullptr;
  const int64_t total = a.f.tq * a.f.hq * (packed ? 1 : a.f.sequences);
  const int64_t at = folded_block() * 16 + threadIdx.x / 16;
  if (at >= total) return;
  const int64_t item = at / a.f.tq, row = at - item * a.f.tq, seq = packed ? 0 : item / a.f.hq, head = item - seq * a.f.hq;
  float s = 0.f;
  if (8 * lane < a.f.d) {
    const u32x4 x = *reinterpret_cast<const u32x4*>(a.d_o.p + seq * a.d_o.b + row * a.d_o.t + head * a.d_o.h + 8 * lane);
    const u32x4 y = *reinterpret_cast<const u32x4*>(a.f.o.p + seq * a.f.o.b + row * a.f.o.t + head * a.f.o.h + 8 * lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s += bf16_lo_to_f32(x[i]) * bf16_lo_to_f32(y[i]);
      s += bf16_hi_to_f32(x[i]) * bf16_hi_to_f32(y[i]);
    }
  }
#pragma unroll
  for (int d = 8; d >= 1; d /= 2) s += __shfl_xor(s, d, 16);
  if (lane == 0) {
    a.delta[at] = s;
    const float l = a.f.lse[at];
    a.lse2[at] = l == -__builtin_inff() ? __builtin_inff() : l * kLog2e;
  }
}

// --- dK, dV -------------------------------------------------------------------
constexpr int kKvWaves = 4, kKvKeys = 32 * kKvWaves;

template <int NB>
__global__ void __launch_bounds__(64 * kKvWaves, 1)
attn_dkv_kernel(AttnBackArgs a) {
  using T = Tile<NB>;
  constexpr int kQueries = 64, kTile = kQueries * T::kPitch, kStage = 2 * kTile + 512;
  __shared__ __attribute__((aligned(16))) char lds[2 * kStage];         // Q, dO, lse2, delta of two steps
  const AttnArgs& f = a.f;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (folded_block() >= f.groups) return;
  const int64_t id = xcd_order(folded_block(), f.groups);
  int64_t item = id / f.tiles, t = id - item * f.tiles, seq = 0;
  const bool packed = f.q_starts != nullptr;
  Span qs, ks;
  int64_t kv;
  if (packed) {
    kv = item;
    const int64_t given = t;
    const bool found = find_tile(f.k_starts, f.sequences, f.tk, kKvKeys, t, seq);
    t = uniform64(t);
    seq = uniform64(seq);
    if (!found) {
      const int64_t spare = f.tiles - (given - t);
      rest_rows(f.k_starts, f.sequences, f.tk, t * 64 * kKvWaves + threadIdx.x, spare * 64 * kKvWaves, [&](int64_t row) {
        uint16_t* p = a.dk.p + row * a.dk.t + kv * a.dk.h;
        uint16_t* q = a.dv.p + row * a.dv.t + kv * a.dv.h;
        for (int c = 0; c < f.d; c += 8)
          *reinterpret_cast<u32x4*>(p + c) = *reinterpret_cast<u32x4*>(q + c) = (u32x4){0, 0, 0, 0};
      });
      return;
    }
    qs = packed_span(f.q_starts, seq, f.tq);
    ks = packed_span(f.k_starts, seq, f.tk);
  } else {
    seq = item / f.hk;
    kv = item - seq * f.hk;
    qs = {0, f.tq};
    ks = {0, f.tk};
    if (f.k_lens != nullptr) {
      const int64_t n = f.k_lens[seq];
      ks.len = n < 0 ? 0 : n < f.tk ? n : f.tk;
    }
  }
  const int64_t b = packed ? 0 : seq;
  const int64_t k0 = t * kKvKeys + 32 * wave, key = k0 + (lane & 31);
  const int64_t shift = ks.len - qs.len;
  // Queries that see a key of this workgroup: from `from` on (causal: i + shift >= key).
  int64_t from = 0;
  if (f.causal && t * kKvKeys - shift > 0) from = (t * kKvKeys - shift) / kQueries * kQueries;
  if (t * kKvKeys >= ks.len) from = qs.len;             // behind the filled rows: zeros
  const int64_t per_head = from < qs.len ? (qs.len - from + kQueries - 1) / kQueries : 0;
  const int64_t steps = per_head * f.group;

  TileCopy<NB, kQueries, kKvWaves> cq, cd;
  cq.init(wave, f.q.t, f.d);
  cd.init(wave, a.d_o.t, f.d);
  const uint32_t lds0 = lds_address(lds);
  const int64_t head0 = kv * f.group;
  // Step j: head head0 + j / per_head, queries from + 64 (j % per_head) on.
  int64_t copy_head = 0, copy_at = from;
  auto copy = [&](int buf) {
    const int64_t head = head0 + copy_head, left = qs.len - copy_at;
    const uint32_t to = lds0 + buf * kStage;
    cq.run(f.q.p + b * f.q.b + (qs.start + copy_at) * f.q.t + head * f.q.h, left, to);
    cd.run(a.d_o.p + b * a.d_o.b + (qs.start + copy_at) * a.d_o.t + head * a.d_o.h, left, to + kTile);
    // Wavefront 0 brings lse2, wavefront 1 delta: 64 values, zeros past the sequence (with Q and dO
    // zero there, P = 1 and dS = 0 add nothing).
    if (wave < 2) {
      const int64_t at = (packed ? head * f.tq : (seq * f.hq + head) * f.tq) + qs.start + copy_at;
      const __amdgpu_buffer_rsrc_t rs = make_rsrc((wave == 0 ? a.lse2 : a.delta) + at, 256);
      const uint32_t off = lane < left ? 4 * lane : kOobOffset;
      const uint32_t dst = __builtin_amdgcn_readfirstlane(to + 2 * kTile + 256 * wave);
      uint32_t saved;
      asm volatile(
          "s_nop 4\n\ts_mov_b32 %[sv], m0\n\ts_mov_b32 m0, %[l0]\n\ts_nop 0\n\t"
          "buffer_load_dword %[v0], %[rs], 0 offen lds\n\ts_mov_b32 m0, %[sv]"
          : [sv] "=&s"(saved)
          : [v0] "v"(off), [rs] "s"(rs), [l0] "s"(dst)
          : "memory");
      (void)saved;
    }
    copy_at += kQueries;
    if (copy_at >= qs.len) copy_at = from, ++copy_head;
  };
  if (steps > 0) copy(0);

  u32x4 kf[2 * NB], vf[2 * NB];
  load_rows<NB>(f.k.p + b * f.k.b + (ks.start + k0) * f.k.t + kv * f.k.h, f.k.t, ks.len - k0, f.d, kf);
  load_rows<NB>(f.v.p + b * f.v.b + (ks.start + k0) * f.v.t + kv * f.v.h, f.v.t, ks.len - k0, f.d, vf);
  f32x16 dk[NB], dv[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) dk[nb] = dv[nb] = zero16();
  uint32_t row_off[2 * NB], col_off[NB][2];
#pragma unroll
  for (int c = 0; c < 2 * NB; ++c) row_off[c] = T::row_operand(c);
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    col_off[nb][0] = T::column_operand(nb, 0);
    col_off[nb][1] = T::column_operand(nb, 1);
  }
  const bool dead = key >= ks.len;                      // this lane's key does not exist
  const bool any_dead = k0 + 32 > ks.len;
  int64_t q0 = from;
  for (int64_t j = 0; j < steps; ++j) {
    wait_copies<0>();
    group_barrier();
    if (j + 1 < steps) copy((int)((j + 1) & 1));
    const char* const qt = lds + (j & 1) * kStage;
    const char* const dt = qt + kTile;
    const float* const lt = reinterpret_cast<const float*>(dt + kTile);
    // First query that sees this lane's key; whether all of the step's see all of the wavefront's.
    const int64_t first = f.causal ? key - shift - q0 : 0;
    const bool cut = any_dead || (f.causal && k0 + 31 - shift > q0);
    if (k0 < ks.len && !(f.causal && k0 - shift >= q0 + kQueries)) {
#pragma unroll
      for (int rb = 0; rb < 2; ++rb) {
        const char* const qb = qt + rb * 32 * T::kPitch;
        const char* const db = dt + rb * 32 * T::kPitch;
        f32x16 s = zero16(), dp = zero16();
#pragma unroll
        for (int c = 0; c < 2 * NB; ++c) s = mfma32<kBf16>(lds_read16(qb + row_off[c]), kf[c], s);
#pragma unroll
        for (int c = 0; c < 2 * NB; ++c) dp = mfma32<kBf16>(lds_read16(db + row_off[c]), vf[c], dp);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = 32 * rb + 8 * q + 4 * (lane >> 5);
          const f32x4 l4 = *reinterpret_cast<const f32x4*>(lt + r), d4 = *reinterpret_cast<const f32x4*>(lt + 64 + r);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float p = exp2_(__builtin_fmaf(s[4 * q + i], f.c, -l4[i]));
            if (cut && (dead || r + i < first)) p = 0.f;
            s[4 * q + i] = p;
            dp[4 * q + i] = p * (dp[4 * q + i] - d4[i]);
          }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const u32x4 pw = pack_half<kBf16>(s, half), dw = pack_half<kBf16>(dp, half);
          const char* const qh = qb + 16 * half * T::kPitch;
          const char* const dh = db + 16 * half * T::kPitch;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            dv[nb] = mfma32<kBf16>(column_read(dh, col_off[nb][0], col_off[nb][1]), pw, dv[nb]);
            dk[nb] = mfma32<kBf16>(column_read(qh, col_off[nb][0], col_off[nb][1]), dw, dk[nb]);
          }
        }
      }
    }
    q0 += kQueries;
    if (q0 >= qs.len) q0 = from;
  }
  // A batch's rows behind the filled ones get zeros (their sums are).
  const int64_t left = (packed ? ks.len : f.tk) - k0;
  store_rows<kBf16, NB>(a.dk.p + b * a.dk.b + (ks.start + k0) * a.dk.t + kv * a.dk.h, a.dk.t, left, f.d, dk, f.scale);
  store_rows<kBf16, NB>(a.dv.p + b * a.dv.b + (ks.start + k0) * a.dv.t + kv * a.dv.h, a.dv.t, left, f.d, dv, 1.f);
}

// --- dQ -----------------------------------------------------------------------
constexpr int kDqWaves = 4;

template <int NB>
__global__ void __launch_bounds__(64 * kDqWaves, 2)
attn_dq_kernel(AttnBackArgs a) {
  using T = Tile<NB>;
  constexpr int kKeys = 64, kQueries = 32 * kDqWaves, kTile = kKeys * T::kPitch;
  __shared__ __attribute__((aligned(16))) char lds[4 * kTile];
  const AttnArgs& f = a.f;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (folded_block() >= f.groups) return;
  const int64_t id = xcd_order(folded_block(), f.groups);
  QueryWork w;
  if (!query_work(f, id, kQueries, w)) {
    const int64_t used = (id % f.tiles) - w.tile, spare = f.tiles - used;
    rest_rows(f.q_starts, f.sequences, f.tq, w.tile * 64 * kDqWaves + threadIdx.x, spare * 64 * kDqWaves, [&](int64_t row) {
      uint16_t* p = a.dq.p + row * a.dq.t + w.head * a.dq.h;
      for (int c = 0; c < f.d; c += 8) *reinterpret_cast<u32x4*>(p + c) = (u32x4){0, 0, 0, 0};
    });
    return;
  }
  const int64_t b = f.q_starts != nullptr ? 0 : w.seq;
  const int64_t q0 = w.tile * kQueries + 32 * wave, shift = w.k.len - w.q.len;
  const int64_t row = q0 + (lane & 31);
  const int64_t tile_end = (w.tile + 1) * kQueries < w.q.len ? (w.tile + 1) * kQueries : w.q.len;
  const int64_t wave_end = q0 + 32 < w.q.len ? q0 + 32 : w.q.len;
  int64_t keys = w.k.len, mine = q0 < w.q.len ? w.k.len : 0, all = w.k.len, limit = w.k.len;
  if (f.causal) {
    keys = tile_end + shift < keys ? tile_end + shift : keys;
    mine = wave_end + shift < mine ? wave_end + shift : mine;
    all = q0 + shift + 1 < all ? q0 + shift + 1 : all;
    limit = row + shift + 1 < limit ? row + shift + 1 : limit;
  }
  const int steps = keys > 0 ? (int)((keys + kKeys - 1) / kKeys) : 0;
  TileCopy<NB, kKeys, kDqWaves> ck, cv;
  ck.init(wave, f.k.t, f.d);
  cv.init(wave, f.v.t, f.d);
  const uint32_t lds0 = lds_address(lds);
  auto copy = [&](int j) {
    const int64_t at = (int64_t)j * kKeys;
    const uint32_t buf = lds0 + (j & 1) * 2 * kTile;
    ck.run(w.kp + at * f.k.t, w.k.len - at, buf);
    cv.run(w.vp + at * f.v.t, w.k.len - at, buf + kTile);
  };
  if (steps > 0) copy(0);
  u32x4 qf[2 * NB], df[2 * NB];
  load_rows<NB>(f.q.p + w.q_off + q0 * f.q.t, f.q.t, w.q.len - q0, f.d, qf);
  const int64_t d_off = b * a.d_o.b + w.q.start * a.d_o.t + w.head * a.d_o.h;
  load_rows<NB>(a.d_o.p + d_off + q0 * a.d_o.t, a.d_o.t, w.q.len - q0, f.d, df);
  const bool live = row < w.q.len;
  const float lse2 = live ? a.lse2[w.lse_off + row] : __builtin_inff(), delta = live ? a.delta[w.lse_off + row] : 0.f;
  f32x16 dq[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) dq[nb] = zero16();
  uint32_t row_off[2 * NB], col_off[NB][2];
#pragma unroll
  for (int c = 0; c < 2 * NB; ++c) row_off[c] = T::row_operand(c);
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    col_off[nb][0] = T::column_operand(nb, 0);
    col_off[nb][1] = T::column_operand(nb, 1);
  }
  for (int j = 0; j < steps; ++j) {
    wait_copies<0>();
    group_barrier();
    if (j + 1 < steps) copy(j + 1);
    const int64_t k0 = (int64_t)j * kKeys;
    if (k0 >= mine) continue;
    const char* const kt = lds + (j & 1) * 2 * kTile;
    const char* const vt = kt + kTile;
    const bool cut = k0 + kKeys > all;
    const int left = (int)(limit < k0 ? 0 : limit - k0 < kKeys ? limit - k0 : kKeys);
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      const char* const kk = kt + kb * 32 * T::kPitch;
      const char* const vv = vt + kb * 32 * T::kPitch;
      f32x16 s = zero16(), dp = zero16();
#pragma unroll
      for (int c = 0; c < 2 * NB; ++c) s = mfma32<kBf16>(lds_read16(kk + row_off[c]), qf[c], s);
#pragma unroll
      for (int c = 0; c < 2 * NB; ++c) dp = mfma32<kBf16>(lds_read16(vv + row_off[c]), df[c], dp);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float p = exp2_(__builtin_fmaf(s[i], f.c, -lse2));
        if (cut && 32 * kb + block_row(i) >= left) p = 0.f;
        dp[i] = p * (dp[i] - delta);
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const u32x4 dw = pack_half<kBf16>(dp, half);
        const char* const base = kk + 16 * half * T::kPitch;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) dq[nb] = mfma32<kBf16>(column_read(base, col_off[nb][0], col_off[nb][1]), dw, dq[nb]);
      }
    }
  }
  const int64_t dq_off = b * a.dq.b + w.q.start * a.dq.t + w.head * a.dq.h;
  store_rows<kBf16, NB>(a.dq.p + dq_off + q0 * a.dq.t, a.dq.t, w.q.len - q0, f.d, dq, f.scale);
}

template <int NB>
hipError_t run_backward(AttnBackArgs a, hipStream_t stream) {
  const bool packed = a.f.q_starts != nullptr;
  const int64_t batch = packed ? 1 : a.f.sequences;
  if (a.f.tk > 0 && a.f.hk > 0) {
    a.f.tiles = packed ? a.f.tk / kKvKeys + a.f.sequences + 1 : (a.f.tk + kKvKeys - 1) / kKvKeys;
    a.f.groups = a.f.tiles * a.f.hk * batch;
    const hipError_t e = launch(&attn_dkv_kernel<NB>, folded_grid(a.f.groups), dim3(64 * kKvWaves), stream, a);
    if (e != hipSuccess) return e;
  }
  if (a.f.tq == 0 || a.f.hq == 0) return hipSuccess;
  constexpr int kQueries = 32 * kDqWaves;
  a.f.tiles = packed ? a.f.tq / kQueries + a.f.sequences + 1 : (a.f.tq + kQueries - 1) / kQueries;
  a.f.groups = a.f.tiles * a.f.hq * batch;
  return launch(&attn_dq_kernel<NB>, folded_grid(a.f.groups), dim3(64 * kDqWaves), stream, a);
}

}  // namespace

hipError_t launch_attention_backward(AttnBackArgs a, hipStream_t stream) {
  const int64_t rows = a.f.tq * a.f.hq * (a.f.q_starts != nullptr ? 1 : a.f.sequences);
  if (rows > 0) {
    const hipError_t e = launch(&attn_delta_kernel, folded_grid((rows + 15) / 16), dim3(256), stream, a);
    if (e != hipSuccess) return e;
  }
  if (a.f.d <= 32) return run_backward<1>(a, stream);
  if (a.f.d <= 64) return run_backward<2>(a, stream);
  if (a.f.d <= 96) return run_backward<3>(a, stream);
  return run_backward<4>(a, stream);
}

}  // namespace rtl
