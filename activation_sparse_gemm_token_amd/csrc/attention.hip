// Attention, forward (include/rtlynx_attention.h): one pass over the keys with
// the softmax's running maximum and sum.
//
// attn_forward_kernel.  A wavefront holds 32 queries: their operands, O^T in
// fp32 and, per lane, one query's maximum and sum; its workgroup of 128 queries
// shares tiles of keys and values in LDS, copied one tile ahead.  Scores are compared with
// the maximum the accumulators are scaled by; that maximum moves (and O^T is
// rescaled) only when some score passes it by more than 2^8, which changes no
// result (any reference would do) and leaves the rescaling out of most steps.
//
// attn_few_kernel.  Few queries over many keys are bound by reading K and V:
// the queries of all heads that share a key head are one tile of 32 rows, every
// wavefront walks its own tiles of 32 keys (its own copies, no barrier), and the
// keys are split over workgroups until the card is full; attn_join_kernel adds
// the parts up.
#include "attn_common.hpp"

namespace rtl {

namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;
// Weights are formed relative to 2^-kLift of the reference maximum.  fp16 has no steps below 2^-24: with the largest weight
// at 1, 400 000 keys of 2^-26 each beside it would all round to 0.  At 2^7 they keep 2^-32 of it, under half a step of the result
// for a million keys, and with the slack stay below 65504.
template <int TYPE>
constexpr float kLift = TYPE == kFp16 ? 7.f : 0.f;

__device__ __forceinline__ float exp2_(float v) { return __builtin_amdgcn_exp2f(v); }
__device__ __forceinline__ float ninf() { return -__builtin_inff(); }

// A lane's running softmax: reference maximum (log2 units), what the sums are scaled by (kLift below it, 0 where no
// key was seen), this half's share of the sum, and of the last steps' part of it.  In one sum faint weights, added one at a time,
// would vanish beside a strong key's; the part goes into the sum every kPart steps (a sum for each step, formed
// before it is added, cost 4 % of the time).
struct Running {
  float m, mu, l, part;
  __device__ __forceinline__ void init() { m = ninf(), mu = 0.f, l = part = 0.f; }
  __device__ __forceinline__ void join() { l += part, part = 0.f; }
};
constexpr int kPart = 16;

// One block of scores into weights; O^T is rescaled where the maximum moved.  `top`: the largest
// score of the lane's query in this step, in log2 units.
template <int TYPE, int NB>
__device__ __forceinline__ void move_maximum(Running& r, float top, f32x16 (&o)[NB]) {
  if (__any(top > r.m + kSlack)) {
    const float m = __builtin_fmaxf(r.m, top), mu = m == ninf() ? 0.f : m;
    const float f = exp2_(r.m - mu);
    r.mu = mu - kLift<TYPE>;
    r.m = m;
    r.l *= f;
    r.part *= f;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[nb][i] *= f;
  }
}

__device__ __forceinline__ float max16(const f32x16& s) {
  float m = s[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) m = __builtin_fmaxf(m, s[i]);
  return m;
}

// Queries and keys of a tile, wavefronts per SIMD.  One wavefront's softmax hides behind the others' products, so what
// counts is how many share a SIMD: three with 32 keys and 168 registers, four with 64 keys up to head_dim 64.
//
// 2 x 4608 tokens, 24 heads of 128: 489 us with the join of the last tiles, 1070 TFLOP/s.  The matrix cores are 61 % busy
// and the vector units 47 at 1.8 GHz, where a lighter kernel has 2.2 and more, so power takes its part; LDS is 31 % busy with
// the wavefronts' reads, without conflicts, and not what bounds it.  A large product reaches 1490 TFLOP/s.  Measured when
// this took 500 to 508 us, and not kept: two
// wavefronts with tiles of 64 keys 521; 8 wavefronts to a workgroup 533 (of 3 or 4 stages 588, 537); the next step's scores formed
// during a softmax 550; 64 queries a wavefront, which halves the reads of LDS but takes 512 registers of two kinds,
// with moves between them, 612; higher wave priority during the products 512.
constexpr int kForwardWaves = 4, kForwardQueries = 32 * kForwardWaves;
template <int NB>
constexpr int forward_keys() { return NB <= 2 ? 64 : 32; }
template <int NB>
constexpr int forward_occupancy() { return NB <= 2 ? 4 : 3; }

template <int TYPE, int NB>
__global__ void __launch_bounds__(64 * kForwardWaves, forward_occupancy<NB>())
attn_forward_kernel(AttnArgs a) {
  using T = Tile<NB>;
  constexpr int kKeys = forward_keys<NB>(), kKb = kKeys / 32, kTile = kKeys * T::kPitch;
  __shared__ __attribute__((aligned(16))) char lds[4 * kTile];          // K, V of two steps
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t id = folded_block();
  if (id >= a.groups) return;
  // The first workgroups take whole tiles, the others a part of the keys of one (launch_attention).
  int part = -1;
  int64_t part_tile = 0;
  if (id < a.whole) {
    id = a.q_starts != nullptr ? xcd_order4(id, a.whole) : xcd_order(id, a.whole);
  } else {
    part_tile = (id - a.whole) / a.splits;
    part = (int)(id - a.whole - part_tile * a.splits);
    id = a.whole + part_tile;
  }
  QueryWork w;
  if (!query_work(a, id, kForwardQueries, w)) {
    if (w.tile < 0) return;
    // No tile left: some rows may lie in no sequence.
    const int64_t spare = a.groups - (id - w.tile);
    rest_rows(a.q_starts, a.sequences, a.tq, a.hq, w.tile, spare, [&](int64_t row, int64_t head) {
      if (a.lse != nullptr) a.lse[head * a.tq + row] = ninf();
      if (a.zero_rest) {
        uint16_t* p = a.o.p + row * a.o.t + head * a.o.h;
        for (int c = 0; c < a.d; c += 8) *reinterpret_cast<u32x4*>(p + c) = (u32x4){0, 0, 0, 0};
      }
    });
    return;
  }
  const int64_t q0 = w.tile * kForwardQueries + 32 * wave, shift = w.k.len - w.q.len;
  const int64_t row = q0 + (lane & 31);
  // Keys that the tile, and this wavefront, see; keys that all of its queries see; this lane's.
  const int64_t tile_end = (w.tile + 1) * kForwardQueries < w.q.len ? (w.tile + 1) * kForwardQueries : w.q.len;
  const int64_t wave_end = q0 + 32 < w.q.len ? q0 + 32 : w.q.len;
  int64_t keys = w.k.len, mine = q0 < w.q.len ? w.k.len : 0, all = w.k.len, limit = w.k.len;
  if (a.causal) {
    keys = tile_end + shift < keys ? tile_end + shift : keys;
    mine = wave_end + shift < mine ? wave_end + shift : mine;
    all = q0 + shift + 1 < all ? q0 + shift + 1 : all;
    limit = row + shift + 1 < limit ? row + shift + 1 : limit;
  }
  // Steps [from, steps) of the workgroup, below my_steps of the wavefront, hidden keys from cut_step on.
  int from = 0, steps = keys > 0 ? (int)((keys + kKeys - 1) / kKeys) : 0;
  const int my_steps = mine > 0 ? (int)((mine + kKeys - 1) / kKeys) : 0, cut_step = all > 0 ? (int)(all / kKeys) : 0;
  if (part >= 0) {
    const int per = (steps + a.splits - 1) / a.splits;
    from = part * per;
    steps = from + per < steps ? from + per : steps;
  }

  TileCopy<NB, kKeys, kForwardWaves> ck, cv;
  ck.init(wave, a.k.t, a.d);
  cv.init(wave, a.v.t, a.d);
  const uint32_t lds0 = lds_address(lds);
  const uint16_t* kp = w.kp + (int64_t)from * kKeys * a.k.t;
  const uint16_t* vp = w.vp + (int64_t)from * kKeys * a.v.t;
  int64_t left = w.k.len - (int64_t)from * kKeys;       // keys from the next copy's first on
  auto copy = [&](int stage) {
    const uint32_t buf = lds0 + stage * 2 * kTile;
    ck.run(kp, clamp_rows(left), buf);
    cv.run(vp, clamp_rows(left), buf + kTile);
    kp += kKeys * a.k.t;
    vp += kKeys * a.v.t;
    left -= kKeys;
  };
  if (from < steps) copy(0);

  u32x4 qf[2 * NB];
  load_rows<NB>(a.q.p + w.q_off + q0 * a.q.t, a.q.t, w.q.len - q0, a.d, qf);
  settle(qf);
  f32x16 o[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) o[nb] = zero16();
  Running run;
  run.init();
  uint32_t row_off[2 * NB], col_off[NB][2];
#pragma unroll
  for (int c = 0; c < 2 * NB; ++c) row_off[c] = T::row_operand(c);
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    col_off[nb][0] = T::column_operand(nb, 0);
    col_off[nb][1] = T::column_operand(nb, 1);
  }

  // A step's LDS stage is a constant, so that its addresses are the reads' offsets and not additions, 16 of the
  // step's 70 vector instructions (2 x 4608 tokens, 24 heads of 128: 488 us, 508 with a stage from j).
  auto step = [&](int j, auto stage) __attribute__((always_inline)) {
    tile_barrier();                                     // tile j is whole, tile j - 1 is no longer read
    if (j >= my_steps) {
      if (j + 1 < steps) copy(1 - stage);
      return;
    }
    const char* const kt = lds + decltype(stage)::value * 2 * kTile;
    const char* const vt = kt + kTile;
    f32x16 s[kKb];
#pragma unroll
    for (int kb = 0; kb < kKb; ++kb) {
      s[kb] = zero16();
#pragma unroll
      for (int c = 0; c < 2 * NB; ++c) s[kb] = mfma32<TYPE>(lds_read16(kt + kb * 32 * T::kPitch + row_off[c]), qf[c], s[kb]);
    }
    if (j + 1 < steps) copy(1 - stage);                 // the matrix core has the scores to work on meanwhile
    if (j >= cut_step) {
      const int seen = clamp_rows(limit - (int64_t)j * kKeys);
#pragma unroll
      for (int kb = 0; kb < kKb; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[kb][i] = 32 * kb + block_row(i) < seen ? s[kb][i] : ninf();
    }
    float top = max16(s[0]);
    if constexpr (kKb == 2) top = __builtin_fmaxf(top, max16(s[kKb - 1]));
    move_maximum<TYPE, NB>(run, half_max(top) * a.c, o);
#pragma unroll
    for (int kb = 0; kb < kKb; ++kb) {
      f32x16 p;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        p[i] = exp2_(__builtin_fmaf(s[kb][i], a.c, -run.mu));
        run.part += p[i];
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const u32x4 pw = pack_half<TYPE>(p, half);
        const char* const base = vt + (32 * kb + 16 * half) * T::kPitch;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) o[nb] = mfma32<TYPE>(column_read(base, col_off[nb][0], col_off[nb][1]), pw, o[nb]);
      }
    }
  };
  for (int j = from; j < steps; j += 2) {
    step(j, std::integral_constant<int, 0>{});
    if (j + 1 < steps) step(j + 1, std::integral_constant<int, 1>{});
    if ((j - from) % kPart == kPart - 2) run.join();
  }
  run.join();
  const float l = half_sum(run.l);
  const int64_t rows = w.q.len - q0;
  if (part >= 0) {
    const int r = 32 * wave + (lane & 31), h = lane >> 5;
    const int64_t at = (part_tile * a.splits + part) * kForwardQueries + r;
    if ((lane & 31) >= rows) return;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = 32 * nb + 8 * q + 4 * h;
        if (c < a.d)
          *reinterpret_cast<f32x4*>(a.part_o + at * a.d + c) =
              (f32x4){o[nb][4 * q], o[nb][4 * q + 1], o[nb][4 * q + 2], o[nb][4 * q + 3]};
      }
    if (h == 0) {
      a.part_ml[2 * at] = run.m;
      a.part_ml[2 * at + 1] = l;
    }
    return;
  }
  store_rows<TYPE, NB>(a.o.p + w.o_off + q0 * a.o.t, a.o.t, rows, a.d, o, l == 0.f ? 0.f : 1.f / l);
  if (a.lse != nullptr && lane < 32 && lane < rows)
    a.lse[w.lse_off + row] = l == 0.f ? ninf() : (run.mu + __builtin_amdgcn_logf(l)) * kLn2;
}

// --- Few queries ------------------------------------------------------------
// Row r of a key head's queries is token r / group, head group kv + r % group.
constexpr int kFewWaves = 4, kFewKeys = 32;

template <int TYPE, int NB>
__global__ void __launch_bounds__(64 * kFewWaves, 1)
attn_few_kernel(AttnArgs a) {
  using T = Tile<NB>;
  constexpr int kTile = kFewKeys * T::kPitch, kWaveBytes = 4 * kTile;
  constexpr int kJoin = kFewWaves * 64 * (16 * NB + 2) * 4;             // O^T, maximum and sum of every wavefront
  __shared__ __attribute__((aligned(16))) char lds[kFewWaves * kWaveBytes > kJoin ? kFewWaves * kWaveBytes : kJoin];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t rows = a.tq * a.group, tiles = (rows + 31) / 32;
  int64_t id = folded_block();
  if (id >= a.groups) return;
  const int split = (int)(id % a.splits);
  id /= a.splits;
  const int64_t tile = id % tiles;
  id /= tiles;
  const int64_t kv = id % a.hk, seq = id / a.hk;
  int64_t len = a.tk;
  if (a.k_lens != nullptr) {
    const int64_t n = a.k_lens[seq];
    len = n < 0 ? 0 : n < a.tk ? n : a.tk;
  }
  // This workgroup's keys [lo, hi), in whole rounds of the wavefronts' tiles.
  constexpr int64_t kRound = kFewWaves * kFewKeys;
  const int64_t per = (((len + a.splits - 1) / a.splits) + kRound - 1) / kRound * kRound;
  const int64_t lo = split * per, hi = lo + per < len ? lo + per : len;

  const int64_t r = tile * 32 + (lane & 31), tok = r / a.group, head = kv * a.group + r % a.group;
  const bool live = r < rows;
  const int64_t shift = len - a.tq;
  int64_t limit = len;
  if (a.causal && tok + shift + 1 < limit) limit = tok + shift + 1;
  const int64_t first_tok = tile * 32 / a.group;
  const int64_t all = a.causal && first_tok + shift + 1 < len ? first_tok + shift + 1 : len;

  const uint16_t* const kp = a.k.p + seq * a.k.b + kv * a.k.h;
  const uint16_t* const vp = a.v.p + seq * a.v.b + kv * a.v.h;
  TileCopy<NB, kFewKeys, 1> ck, cv;
  ck.init(0, a.k.t, a.d);
  cv.init(0, a.v.t, a.d);
  char* const mine = lds + wave * kWaveBytes;
  const uint32_t lds0 = lds_address(mine);
  auto copy = [&](int64_t at, int buf) {
    ck.run(kp + at * a.k.t, clamp_rows(len - at), lds0 + buf * 2 * kTile);
    cv.run(vp + at * a.v.t, clamp_rows(len - at), lds0 + buf * 2 * kTile + kTile);
  };
  const int64_t first = lo + kFewKeys * wave;
  if (first < hi) copy(first, 0);
  u32x4 qf[2 * NB];
#pragma unroll
  for (int c = 0; c < 2 * NB; ++c) {
    qf[c] = (u32x4){0, 0, 0, 0};
    const int ch = 16 * c + 8 * (lane >> 5);
    if (live && ch < a.d) qf[c] = *reinterpret_cast<const u32x4*>(a.q.p + seq * a.q.b + tok * a.q.t + head * a.q.h + ch);
  }
  settle(qf);
  f32x16 o[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) o[nb] = zero16();
  Running run;
  run.init();
  uint32_t row_off[2 * NB], col_off[NB][2];
#pragma unroll
  for (int c = 0; c < 2 * NB; ++c) row_off[c] = T::row_operand(c);
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    col_off[nb][0] = T::column_operand(nb, 0);
    col_off[nb][1] = T::column_operand(nb, 1);
  }
  int buf = 0;
  for (int64_t k0 = first; k0 < hi; k0 += kRound, buf ^= 1) {
    // The other buffer's last reads were consumed in the step before.
    if (k0 + kRound < hi) {
      copy(k0 + kRound, buf ^ 1);
      wait_copies<2 * TileCopy<NB, kFewKeys, 1>::kCount>();
    } else {
      wait_copies<0>();
    }
    const char* const kt = mine + buf * 2 * kTile;
    const char* const vt = kt + kTile;
    f32x16 s = zero16();
#pragma unroll
    for (int c = 0; c < 2 * NB; ++c) s = mfma32<TYPE>(lds_read16(kt + row_off[c]), qf[c], s);
    if (k0 + kFewKeys > all || k0 + kFewKeys > hi) {
      const int64_t end = limit < hi ? limit : hi;
      const int left = (int)(end < k0 ? 0 : end - k0 < kFewKeys ? end - k0 : kFewKeys);
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = block_row(i) < left ? s[i] : ninf();
    }
    move_maximum<TYPE, NB>(run, half_max(max16(s)) * a.c, o);
    f32x16 p;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      p[i] = exp2_(__builtin_fmaf(s[i], a.c, -run.mu));
      run.part += p[i];
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const u32x4 pw = pack_half<TYPE>(p, half);
      const char* const base = vt + 16 * half * T::kPitch;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) o[nb] = mfma32<TYPE>(column_read(base, col_off[nb][0], col_off[nb][1]), pw, o[nb]);
    }
    if ((k0 - first) % (kPart * kRound) == (kPart - 1) * kRound) run.join();
    // The next step copies over the buffer read here.
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
  run.join();
  // The wavefronts' results joined: every one brings its own, then sums a block of 32 channels.
  __syncthreads();
  float* const jo = reinterpret_cast<float*>(lds);                      // [wave][16 NB][64]
  float* const jm = jo + kFewWaves * 16 * NB * 64;                      // [wave][2][64]
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int i = 0; i < 16; ++i) jo[((wave * NB + nb) * 16 + i) * 64 + lane] = o[nb][i];
  jm[(wave * 2) * 64 + lane] = run.m;
  jm[(wave * 2 + 1) * 64 + lane] = half_sum(run.l);
  __syncthreads();
  float m = ninf(), l = 0.f, f[kFewWaves];
#pragma unroll
  for (int v = 0; v < kFewWaves; ++v) m = __builtin_fmaxf(m, jm[(v * 2) * 64 + lane]);
  const float mu = m == ninf() ? 0.f : m;
#pragma unroll
  for (int v = 0; v < kFewWaves; ++v) {
    f[v] = exp2_(jm[(v * 2) * 64 + lane] - mu);
    l += f[v] * jm[(v * 2 + 1) * 64 + lane];
  }
  if (wave >= NB) return;
  float sum[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    sum[i] = 0.f;
#pragma unroll
    for (int v = 0; v < kFewWaves; ++v) sum[i] += f[v] * jo[((v * NB + wave) * 16 + i) * 64 + lane];
  }
  if (!live) return;
  const int h = lane >> 5;
  const int64_t at = (seq * a.hk + kv) * rows + r;                      // row of the parts
  if (a.splits > 1) {
    float* const out = a.part_o + ((int64_t)split * a.sequences * a.hk * rows + at) * a.d;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = 32 * wave + 8 * q + 4 * h;
      if (c < a.d) *reinterpret_cast<f32x4*>(out + c) = (f32x4){sum[4 * q], sum[4 * q + 1], sum[4 * q + 2], sum[4 * q + 3]};
    }
    if (wave == 0 && h == 0) {
      float* const ml = a.part_ml + ((int64_t)split * a.sequences * a.hk * rows + at) * 2;
      ml[0] = m;
      ml[1] = l;
    }
    return;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint16_t* const out = a.o.p + seq * a.o.b + tok * a.o.t + head * a.o.h;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int c = 32 * wave + 8 * q + 4 * h;
    if (c < a.d)
      *reinterpret_cast<u32x2*>(out + c) = (u32x2){pack2<TYPE>(sum[4 * q] * inv, sum[4 * q + 1] * inv),
                                                   pack2<TYPE>(sum[4 * q + 2] * inv, sum[4 * q + 3] * inv)};
  }
  if (a.lse != nullptr && wave == 0 && h == 0)
    a.lse[(seq * a.hq + head) * a.tq + tok] = l == 0.f ? ninf() : (mu - kLift<TYPE> + __builtin_amdgcn_logf(l)) * kLn2;
}

// Adds up the splits' parts: 4 channels of a row per thread.  TILES: parts [tile][split][row] of the
// last tiles of attn_forward_kernel, else [split][row] of attn_few_kernel.
template <int TYPE, bool TILES>
__global__ void __launch_bounds__(256)
attn_join_kernel(AttnArgs a) {
  const int per_row = a.d / 4;
  const int64_t i = folded_block() * 256 + threadIdx.x, at = i / per_row;
  const int c = 4 * (int)(i - at * per_row);
  int64_t first, step, seq, head, tok;                  // rows of the parts; the query
  if constexpr (TILES) {
    const int64_t tile = at / kForwardQueries, r = at - tile * kForwardQueries;
    if (tile >= (a.groups - a.whole) / a.splits) return;
    first = tile * a.splits * kForwardQueries + r;
    step = kForwardQueries;
    const int64_t id = a.whole + tile, item = id / a.tiles, t = id - item * a.tiles;
    tok = t * kForwardQueries + r;
    if (tok >= a.tq) return;
    seq = item / a.hq;
    head = item - seq * a.hq;
  } else {
    const int64_t rows = a.tq * a.group, total = a.sequences * a.hk * rows;
    if (at >= total) return;
    first = at;
    step = total;
    const int64_t r = at % rows, kv = at / rows % a.hk;
    seq = at / rows / a.hk;
    tok = r / a.group;
    head = kv * a.group + r % a.group;
  }
  float m = ninf();
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s) m = __builtin_fmaxf(m, a.part_ml[(first + s * step) * 2]);
  const float mu = m == ninf() ? 0.f : m;
  float l = 0.f;
  f32x4 sum = {0, 0, 0, 0};
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s) {
    const float* const ml = a.part_ml + (first + s * step) * 2;
    const float f = exp2_(ml[0] - mu);
    l += f * ml[1];
    sum += f * *reinterpret_cast<const f32x4*>(a.part_o + (first + s * step) * a.d + c);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<u32x2*>(a.o.p + seq * a.o.b + tok * a.o.t + head * a.o.h + c) =
      (u32x2){pack2<TYPE>(sum[0] * inv, sum[1] * inv), pack2<TYPE>(sum[2] * inv, sum[3] * inv)};
  if (a.lse != nullptr && c == 0)
    a.lse[(seq * a.hq + head) * a.tq + tok] = l == 0.f ? ninf() : (mu - kLift<TYPE> + __builtin_amdgcn_logf(l)) * kLn2;
}

template <int TYPE, int NB>
hipError_t run_forward(AttnArgs a, const AttnPlan& plan, hipStream_t stream) {
  a.splits = plan.splits;
  if (plan.few) {
    const int64_t rows = a.tq * a.group;
    a.groups = a.sequences * a.hk * ((rows + 31) / 32) * a.splits;
    const hipError_t e = launch(&attn_few_kernel<TYPE, NB>, folded_grid(a.groups), dim3(64 * kFewWaves), stream, a);
    if (e != hipSuccess || a.splits == 1) return e;
    const int64_t items = a.sequences * a.hk * rows * (a.d / 4);
    return launch(&attn_join_kernel<TYPE, false>, folded_grid((items + 255) / 256), dim3(256), stream, a);
  }
  // Packed: as many tiles as the sequences can have, and one for the rows in none.
  const bool packed = a.q_starts != nullptr;
  a.tiles = packed ? a.tq / kForwardQueries + a.sequences + 1 : (a.tq + kForwardQueries - 1) / kForwardQueries;
  const int64_t tiles = a.tiles * a.hq * (packed ? 1 : a.sequences);
  a.whole = tiles - plan.tail;
  a.groups = a.whole + plan.tail * a.splits;
  const hipError_t e = launch(&attn_forward_kernel<TYPE, NB>, folded_grid(a.groups), dim3(64 * kForwardWaves), stream, a);
  if (e != hipSuccess || plan.tail == 0) return e;
  const int64_t items = plan.tail * kForwardQueries * (a.d / 4);
  return launch(&attn_join_kernel<TYPE, true>, folded_grid((items + 255) / 256), dim3(256), stream, a);
}

template <int TYPE>
hipError_t by_blocks(const AttnArgs& a, const AttnPlan& plan, hipStream_t stream) {
  if (a.d <= 32) return run_forward<TYPE, 1>(a, plan, stream);
  if (a.d <= 64) return run_forward<TYPE, 2>(a, plan, stream);
  if (a.d <= 96) return run_forward<TYPE, 3>(a, plan, stream);
  return run_forward<TYPE, 4>(a, plan, stream);
}

}  // namespace

// Up to 32 queries of a sequence go to attn_few_kernel, its keys in ranges of at least 256 until there is one workgroup
// per CU (one token, 65536 keys in 8 heads: 53 us; two 61, three 71: more parts to join).  The kernel for tiles took 490
// us where this one takes 92 (8 sequences of 16384 keys, 8 key heads).
//
// Otherwise tiles of 128 queries; a batch's tiles are alike, so where their number is no multiple of what the card
// holds (256 CUs times the wavefronts per SIMD) the last, partly filled round would leave CUs idle: the keys of its
// tiles are split over workgroups, 256 keys at least for each.  Tiles of causal batches are never split: with about as
// many keys as queries they differ, and the short ones come last.  More than 32 causal queries over many more keys have
// alike tiles all the same and too few of them (64 over 30000 keys of 8 heads: 8 workgroups, 715 us; 32 queries 35, 512
// queries without the mask 78).  Nor are packed ones, whose lengths only the device knows (8 of one query over 16384 keys
// each, 32 heads on 8: 382 us, 91 as a batch).
AttnPlan attn_plan(int64_t sequences, int64_t tq, int64_t tk, int64_t hq, int64_t hk, int64_t d, bool packed, bool causal) {
  AttnPlan p{false, 1, 0};
  if (packed || sequences == 0 || tq == 0 || hk == 0 || hq == 0) return p;
  if (tq <= 32) {
    const int64_t rows = tq * (hq / hk), groups = sequences * hk * ((rows + 31) / 32);
    int64_t splits = (256 + groups - 1) / groups;
    const int64_t most = (tk + 255) / 256;
    if (splits > most) splits = most;
    p.few = true;
    p.splits = splits < 1 ? 1 : (int)splits;
    return p;
  }
  if (causal) return p;
  const int64_t slots = 256 * (d <= 64 ? forward_occupancy<2>() : forward_occupancy<4>());
  const int64_t tiles = sequences * hq * ((tq + kForwardQueries - 1) / kForwardQueries), tail = tiles % slots;
  if (tail == 0) return p;
  int64_t splits = slots / tail;
  if (splits > tk / 256) splits = tk / 256;
  if (splits > 16) splits = 16;
  if (splits >= 2) {
    p.splits = (int)splits;
    p.tail = tail;
  }
  return p;
}

size_t attn_plan_bytes(const AttnPlan& p, int64_t sequences, int64_t tq, int64_t hq, int64_t d) {
  if (p.splits <= 1) return 0;
  return (size_t)p.splits * (size_t)(p.few ? sequences * hq * tq : p.tail * kForwardQueries) * (size_t)(d + 2) * 4;
}

hipError_t launch_attention(AttnArgs a, const AttnPlan& plan, bool fp16, void* workspace, hipStream_t stream) {
  const int64_t rows = plan.few ? a.sequences * a.hq * a.tq : plan.tail * kForwardQueries;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = plan.splits > 1 ? a.part_o + plan.splits * rows * a.d : nullptr;
  return fp16 ? by_blocks<kFp16>(a, plan, stream) : by_blocks<kBf16>(a, plan, stream);
}

}  // namespace rtl
