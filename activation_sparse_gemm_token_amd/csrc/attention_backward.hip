// Attention, backward (include/rtlynx_attention.h).
//
//   1. attn_dq_kernel      dQ: as the forward pass, 32 queries a wavefront.  It leaves D = sum of d_o o per
//                          query and head, beside the log-sum-exp in log2 units (+inf where no key is
//                          seen: p is 0 then).
//   2. attn_dkv_kernel     dK, dV: a wavefront holds 32 keys, its workgroup walks the
//                          queries of all heads that share the key head.
//   3. attn_dkv_join_kernel  where few key heads leave few workgroups, 2 splits the queries.
//
// S and dP are formed in both (7 products where 5 would do with atomic sums), so
// nothing is added atomically and shared heads sum in registers.  Everything
// between the products stays in registers: a lane's P and dS are operands as they
// stand (attn_common.hpp).  P and dS are rounded to bf16 there; S, dP and all sums
// are fp32.
//
// 4 packed sequences of 423 to 2955 tokens, 16 heads on 8 of 128: 174 us for dQ, 233 for dK
// and dV and 17 for the join.  The matrix cores are 47 and 44 % busy, the vector units 38 and
// 23, LDS 23 and 33 with the wavefronts' reads: no unit is full.  Two wavefronts share a SIMD,
// whose products and softmax overlap in part, and the longest sequence's tiles run on when the
// others' are done.
#include "attn_common.hpp"

namespace rtl {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_(float v) { return __builtin_amdgcn_exp2f(v); }

// --- dK, dV -------------------------------------------------------------------
// K of a wavefront's 32 keys stays in registers, V in LDS (both in registers, with dK and dV, take more than
// 256: one wavefront per SIMD, 200 moves between register files for every 32 matrix
// instructions, and half the speed); queries come 32 at a time.
constexpr int kKvWaves = 4, kKvKeys = 32 * kKvWaves;

template <int NB>
__global__ void __launch_bounds__(64 * kKvWaves, 2)
attn_dkv_kernel(AttnBackArgs a) {
  using T = Tile<NB>;
  constexpr int kQueries = 32, kTile = kQueries * T::kPitch, kStage = 2 * kTile + 256, kVBytes = kKvKeys * T::kPitch;
  __shared__ __attribute__((aligned(16))) char lds[kVBytes + 2 * kStage];   // V; Q, dO and their statistics of two steps
  const AttnArgs& f = a.f;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (folded_block() >= f.groups) return;
  const bool packed = f.q_starts != nullptr;
  const int64_t block = packed ? xcd_order4(folded_block(), f.groups) : xcd_order(folded_block(), f.groups);
  const int64_t id = block / f.splits;
  int64_t seq, kv, t;
  const int split = (int)(block - id * f.splits);
  Span qs, ks;
  if (packed) {
    const PackedTile p = packed_tile(f.k_starts, f.sequences, f.tk, kKvKeys, f.hk, id);
    if (!p.found) {
      if (p.tile < 0) return;
      const int64_t spare = f.groups / f.splits - (id - p.tile);
      rest_rows(f.k_starts, f.sequences, f.tk, f.hk, p.tile, spare, [&](int64_t row, int64_t head) {
        if (f.splits > 1) {
          float* p = f.part_o + ((split * 2 * f.tk + row) * f.hk + head) * f.d;
          for (int c = 0; c < f.d; c += 4)
            *reinterpret_cast<f32x4*>(p + c) = *reinterpret_cast<f32x4*>(p + f.tk * f.hk * f.d + c) = (f32x4){0, 0, 0, 0};
          return;
        }
        uint16_t* p = a.dk.p + row * a.dk.t + head * a.dk.h;
        uint16_t* q = a.dv.p + row * a.dv.t + head * a.dv.h;
        for (int c = 0; c < f.d; c += 8)
          *reinterpret_cast<u32x4*>(p + c) = *reinterpret_cast<u32x4*>(q + c) = (u32x4){0, 0, 0, 0};
      });
      return;
    }
    t = p.tile;
    seq = p.seq;
    kv = p.head;
    qs = packed_span(f.q_starts, seq, f.tq);
    ks = packed_span(f.k_starts, seq, f.tk);
  } else {
    const int64_t item = id / f.tiles;
    t = id - item * f.tiles;
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
  // Step j: head head0 + j / per_head, queries from + 32 (j % per_head) on; this workgroup's are [lo, steps).
  int64_t steps = per_head * f.group;
  const int64_t per_split = (steps + f.splits - 1) / f.splits, lo = split * per_split;
  steps = lo + per_split < steps ? lo + per_split : steps;

  TileCopy<NB, kQueries, kKvWaves> cq, cd;
  cq.init(wave, f.q.t, f.d);
  cd.init(wave, a.d_o.t, f.d);
  const uint32_t lds0 = lds_address(lds) + kVBytes;
  const int64_t head0 = kv * f.group;
  int64_t copy_head = lo < steps ? lo / per_head : 0, copy_at = lo < steps ? from + (lo - copy_head * per_head) * kQueries : from;
  auto copy = [&](int buf) {
    const int64_t head = head0 + copy_head, left = qs.len - copy_at;
    const uint32_t to = lds0 + buf * kStage;
    cq.run(f.q.p + b * f.q.b + (qs.start + copy_at) * f.q.t + head * f.q.h, clamp_rows(left), to);
    cd.run(a.d_o.p + b * a.d_o.b + (qs.start + copy_at) * a.d_o.t + head * a.d_o.h, clamp_rows(left), to + kTile);
    // Wavefront 0 brings the statistics, zeros past the sequence (with Q and dO zero there, P = 1 and
    // dS = 0 add nothing).
    if (wave == 0) {
      const int64_t at = (packed ? head * f.tq : (seq * f.hq + head) * f.tq) + qs.start + copy_at;
      const __amdgpu_buffer_rsrc_t rs = make_rsrc(a.stats + at, 256);
      const uint32_t off = lane / 2 < left ? 4 * lane : kOobOffset;
      const uint32_t dst = __builtin_amdgcn_readfirstlane(to + 2 * kTile);
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
  int64_t q0 = copy_at;
  if (lo < steps) copy(0);

  {
    TileCopy<NB, kKvKeys, kKvWaves> cv;
    cv.init(wave, f.v.t, f.d);
    cv.run(f.v.p + b * f.v.b + (ks.start + t * kKvKeys) * f.v.t + kv * f.v.h, clamp_rows(ks.len - t * kKvKeys), lds_address(lds));
  }
  u32x4 kf[2 * NB];
  load_rows<NB>(f.k.p + b * f.k.b + (ks.start + k0) * f.k.t + kv * f.k.h, f.k.t, ks.len - k0, f.d, kf);
  settle(kf);
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
  const char* const vt = lds + wave * 32 * T::kPitch;
  auto step = [&](int64_t j, auto stage) __attribute__((always_inline)) {   // its stage a constant, as in the forward pass
    tile_barrier();
    if (j + 1 < steps) copy(1 - stage);
    const char* const qt = lds + kVBytes + decltype(stage)::value * kStage;
    const char* const dt = qt + kTile;
    const float* const st = reinterpret_cast<const float*>(dt + kTile);
    if (k0 < ks.len && !(f.causal && k0 - shift >= q0 + kQueries)) {
      f32x16 s = zero16(), dp = zero16();
#pragma unroll
      for (int c = 0; c < 2 * NB; ++c) s = mfma32<kBf16>(lds_read16(qt + row_off[c]), kf[c], s);
#pragma unroll
      for (int c = 0; c < 2 * NB; ++c) dp = mfma32<kBf16>(lds_read16(dt + row_off[c]), lds_read16(vt + row_off[c]), dp);
      // Hidden scores: keys that do not exist, and queries before the first one that sees the lane's key.
      if (any_dead || (f.causal && k0 + 31 - shift > q0)) {
        const int first = dead ? kQueries : f.causal ? clamp_rows(key - shift - q0) : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = block_row(i) < first ? -__builtin_inff() : s[i];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float* const r = st + 2 * (8 * q + 4 * (lane >> 5));
        const f32x4 s0 = *reinterpret_cast<const f32x4*>(r), s1 = *reinterpret_cast<const f32x4*>(r + 4);
        const float l4[4] = {s0[0], s0[2], s1[0], s1[2]}, d4[4] = {s0[1], s0[3], s1[1], s1[3]};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = exp2_(__builtin_fmaf(s[4 * q + i], f.c, -l4[i]));
          s[4 * q + i] = p;
          dp[4 * q + i] = p * (dp[4 * q + i] - d4[i]);
        }
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const u32x4 pw = pack_half<kBf16>(s, half), dw = pack_half<kBf16>(dp, half);
        const char* const qh = qt + 16 * half * T::kPitch;
        const char* const dh = dt + 16 * half * T::kPitch;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) dv[nb] = mfma32<kBf16>(column_read(dh, col_off[nb][0], col_off[nb][1]), pw, dv[nb]);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) dk[nb] = mfma32<kBf16>(column_read(qh, col_off[nb][0], col_off[nb][1]), dw, dk[nb]);
      }
    }
    q0 += kQueries;
    if (q0 >= qs.len) q0 = from;
  };
  for (int64_t j = lo; j < steps; j += 2) {
    step(j, std::integral_constant<int, 0>{});
    if (j + 1 < steps) step(j + 1, std::integral_constant<int, 1>{});
  }
  if (lo >= steps) wait_copies<0>();                    // V's copy must not outlive the workgroup
  // A batch's rows behind the filled ones get zeros (their sums are).
  const int64_t left = (packed ? ks.len : f.tk) - k0;
  if (f.splits > 1) {
    const int64_t total = packed ? f.tk : f.sequences * f.tk, at = (packed ? ks.start : seq * f.tk) + key;
    if ((lane & 31) >= left) return;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = 32 * nb + 8 * q + 4 * (lane >> 5);
        if (c >= f.d) continue;
        float* const p = f.part_o + ((split * 2 * total + at) * f.hk + kv) * f.d + c;
        *reinterpret_cast<f32x4*>(p) = (f32x4){dk[nb][4 * q], dk[nb][4 * q + 1], dk[nb][4 * q + 2], dk[nb][4 * q + 3]};
        *reinterpret_cast<f32x4*>(p + total * f.hk * f.d) =
            (f32x4){dv[nb][4 * q], dv[nb][4 * q + 1], dv[nb][4 * q + 2], dv[nb][4 * q + 3]};
      }
    return;
  }
  store_rows<kBf16, NB>(a.dk.p + b * a.dk.b + (ks.start + k0) * a.dk.t + kv * a.dk.h, a.dk.t, left, f.d, dk, f.scale);
  store_rows<kBf16, NB>(a.dv.p + b * a.dv.b + (ks.start + k0) * a.dv.t + kv * a.dv.h, a.dv.t, left, f.d, dv, 1.f);
}

// Adds the splits' dK and dV up, in order: 8 channels per thread.
__global__ void __launch_bounds__(256)
attn_dkv_join_kernel(AttnBackArgs a) {
  const AttnArgs& f = a.f;
  const bool packed = f.q_starts != nullptr;
  const int64_t total = packed ? f.tk : f.sequences * f.tk, size = total * f.hk * f.d;
  const int64_t i = (folded_block() * 256 + threadIdx.x) * 8;
  if (i >= 2 * size) return;
  const bool is_v = i >= size;
  const int64_t at = is_v ? i - size : i;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < f.splits; ++s) {
    const f32x4* const p = reinterpret_cast<const f32x4*>(f.part_o + s * 2 * size + i);
    const f32x4 x = p[0], y = p[1];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += x[e], v[4 + e] += y[e];
  }
  const float factor = is_v ? 1.f : f.scale;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] *= factor;
  const int64_t c = at % f.d, kv = at / f.d % f.hk, row = at / f.d / f.hk, seq = packed ? 0 : row / f.tk;
  const AttnTensor& t = is_v ? a.dv : a.dk;
  store_vec<kBf16, 8>(t.p + seq * t.b + (row - seq * f.tk) * t.t + kv * t.h + c, v);
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
  const int64_t id = f.q_starts != nullptr ? xcd_order4(folded_block(), f.groups) : xcd_order(folded_block(), f.groups);
  QueryWork w;
  if (!query_work(f, id, kQueries, w)) {
    if (w.tile < 0) return;
    const int64_t spare = f.groups - (id - w.tile);
    rest_rows(f.q_starts, f.sequences, f.tq, f.hq, w.tile, spare, [&](int64_t row, int64_t head) {
      uint16_t* p = a.dq.p + row * a.dq.t + head * a.dq.h;
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
    ck.run(w.kp + at * f.k.t, clamp_rows(w.k.len - at), buf);
    cv.run(w.vp + at * f.v.t, clamp_rows(w.k.len - at), buf + kTile);
  };
  if (steps > 0) copy(0);
  u32x4 qf[2 * NB], df[2 * NB];
  load_rows<NB>(f.q.p + w.q_off + q0 * f.q.t, f.q.t, w.q.len - q0, f.d, qf);
  const int64_t d_off = b * a.d_o.b + w.q.start * a.d_o.t + w.head * a.d_o.h;
  load_rows<NB>(a.d_o.p + d_off + q0 * a.d_o.t, a.d_o.t, w.q.len - q0, f.d, df);
  // Whether all of the tile's queries, or some of them, see no more keys than the two tiles of LDS hold.
  const bool live = row < w.q.len, few = steps <= 2;
  const bool near = steps > 0 && (few || (f.causal && w.tile * kQueries + shift < 2 * kKeys));
  float lse2 = live ? f.lse[w.lse_off + row] : -__builtin_inff();
  lse2 = lse2 == -__builtin_inff() ? __builtin_inff() : lse2 * kLog2e;
  float delta = 0.f;
  if (!few) {                                           // D, 8 channels of d_o o at a time, then both halves of the wavefront
    u32x4 of[2 * NB];
    load_rows<NB>(f.o.p + w.o_off + q0 * f.o.t, f.o.t, w.q.len - q0, f.d, of);
#pragma unroll
    for (int c = 0; c < 2 * NB; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        delta += bf16_lo_to_f32(df[c][i]) * bf16_lo_to_f32(of[c][i]);
        delta += bf16_hi_to_f32(df[c][i]) * bf16_hi_to_f32(of[c][i]);
      }
    delta = half_sum(delta);
  }
  settle(qf);
  settle(df);
  asm volatile("" : "+v"(lse2), "+v"(delta));
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
  // Few keys: o is near the values, ds a difference of near numbers, and o's rounding in D would show (with two
  // keys dQ and dK were 0.4 % off instead of 0.24 %).  D is the sum of p dP too: formed so for the queries
  // whose keys fit the two tiles of LDS.
  if (near) {
    if (steps >= 2) copy(1);
    tile_barrier();
    float sum = 0.f;
    if (mine > 0 && (few || q0 + shift < 2 * kKeys)) {
      const int left = clamp_rows(limit);
#pragma unroll 1
      for (int kb = 0; kb < (steps >= 2 ? 4 : 2); ++kb) {
        const char* const kk = lds + (kb >> 1) * 2 * kTile + (kb & 1) * 32 * T::kPitch;
        f32x16 s = zero16(), dp = zero16();
#pragma unroll
        for (int c = 0; c < 2 * NB; ++c) s = mfma32<kBf16>(lds_read16(kk + row_off[c]), qf[c], s);
#pragma unroll
        for (int c = 0; c < 2 * NB; ++c) dp = mfma32<kBf16>(lds_read16(kk + kTile + row_off[c]), df[c], dp);
#pragma unroll
        for (int i = 0; i < 16; ++i) sum += 32 * kb + block_row(i) < left ? exp2_(__builtin_fmaf(s[i], f.c, -lse2)) * dp[i] : 0.f;
      }
    }
    sum = half_sum(sum);
    delta = limit <= 2 * kKeys ? sum : delta;
  }
  if (live && lane < 32) a.stats[w.lse_off + row] = (f32x2){lse2, delta};       // for the dK / dV kernel
  auto step = [&](int j, auto stage) __attribute__((always_inline)) {
    tile_barrier();
    if (j + 1 < steps && !(near && j == 0)) copy(j + 1);
    const int64_t k0 = (int64_t)j * kKeys;
    if (k0 >= mine) return;
    const char* const kt = lds + decltype(stage)::value * 2 * kTile;
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
  };
  for (int j = 0; j < steps; j += 2) {
    step(j, std::integral_constant<int, 0>{});
    if (j + 1 < steps) step(j + 1, std::integral_constant<int, 1>{});
  }
  const int64_t dq_off = b * a.dq.b + w.q.start * a.dq.t + w.head * a.dq.h;
  store_rows<kBf16, NB>(a.dq.p + dq_off + q0 * a.dq.t, a.dq.t, w.q.len - q0, f.d, dq, f.scale);
}

template <int NB>
hipError_t run_backward(AttnBackArgs a, hipStream_t stream) {
  const bool packed = a.f.q_starts != nullptr;
  const int64_t batch = packed ? 1 : a.f.sequences;
  if (a.f.tq > 0 && a.f.hq > 0) {
    AttnBackArgs q = a;
    constexpr int kQueries = 32 * kDqWaves;
    q.f.tiles = packed ? a.f.tq / kQueries + a.f.sequences + 1 : (a.f.tq + kQueries - 1) / kQueries;
    q.f.groups = q.f.tiles * a.f.hq * batch;
    const hipError_t e = launch(&attn_dq_kernel<NB>, folded_grid(q.f.groups), dim3(64 * kDqWaves), stream, q);
    if (e != hipSuccess) return e;
  }
  if (a.f.tk == 0 || a.f.hk == 0) return hipSuccess;
  a.f.tiles = packed ? a.f.tk / kKvKeys + a.f.sequences + 1 : (a.f.tk + kKvKeys - 1) / kKvKeys;
  a.f.groups = a.f.tiles * a.f.hk * batch * a.f.splits;
  const hipError_t e = launch(&attn_dkv_kernel<NB>, folded_grid(a.f.groups), dim3(64 * kKvWaves), stream, a);
  if (e != hipSuccess || a.f.splits == 1) return e;
  const int64_t items = batch * a.f.tk * a.f.hk * (a.f.d / 8) * 2;
  return launch(&attn_dkv_join_kernel, folded_grid((items + 255) / 256), dim3(256), stream, a);
}

}  // namespace

// Ranges of the queries that a tile of keys' sums are shared out over: few key heads leave few workgroups
// with long walks.  Up to four workgroups per CU (two run at a time), 256 queries at least for each.  (The
// sequences above: 371 us with one range, 292 with two, and 17 for the join.)
int attn_back_splits(int64_t sequences, int64_t tq, int64_t tk, int64_t hq, int64_t hk, bool packed) {
  if (hk == 0 || tk == 0 || sequences == 0) return 1;
  const int64_t tiles = (packed ? tk / kKvKeys + sequences / 2 + 1 : sequences * ((tk + kKvKeys - 1) / kKvKeys)) * hk;
  int64_t splits = 1024 / tiles;
  const int64_t queries = (packed ? tq / sequences : tq) * (hq / hk);
  if (splits > queries / 256) splits = queries / 256;
  return splits < 1 ? 1 : splits > 16 ? 16 : (int)splits;
}

hipError_t launch_attention_backward(AttnBackArgs a, hipStream_t stream) {
  if (a.f.d <= 32) return run_backward<1>(a, stream);
  if (a.f.d <= 64) return run_backward<2>(a, stream);
  if (a.f.d <= 96) return run_backward<3>(a, stream);
  return run_backward<4>(a, stream);
}

}  // namespace rtl
