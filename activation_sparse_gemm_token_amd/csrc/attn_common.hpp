// Pieces shared by the attention kernels (internal).
//
// Every product runs on v_mfma_f32_32x32x16 with the scores transposed: the
// matrix core leaves a lane 16 scores of one column (its query, or in the
// dK / dV kernel its key), so a softmax row's statistics are one register per
// lane, and the scores of a lane are, as they stand, the right-hand operand of
// the next product.  That operand gives lane l rows 8 (l / 32) + [0, 8) of each
// 16; what the lane holds are rows 4 (l / 32) + [0, 4) and 8 + 4 (l / 32) +
// [0, 4).  A contraction may run in any order, so the left-hand operand is read in
// that order too: it is a transposed tile (rows of K, V, Q or dO in memory,
// channels wanted along the operand's rows), which ds_read_b64_tr_b16 delivers
// four rows at a time.
//
// Tiles of 32 or 64 rows go from memory to LDS by direct copies, 16 bytes a lane.  A
// row takes 128 or 256 bytes of LDS (head_dim up to 64, or 128), channels past
// head_dim and rows past the sequence arrive as zeros.  Chunk c of 16 bytes of row r
// lies in slot c ^ swizzle(r): the 16 rows at one chunk that an ordinary
// operand read touches at a time fall on different banks, and so do the 4 rows x 2
// chunks x 2 groups of a transposing read.
#pragma once

#include "rtl_elem.hpp"
#include "rtl_operators.hpp"

namespace rtl {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

template <int TYPE>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (TYPE == kBf16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ f32x16 zero16() {
  f32x16 v;
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.f;
  return v;
}

// 8 scores of a lane (half a 32-row block) as an operand.
template <int TYPE>
__device__ __forceinline__ u32x4 pack_half(const f32x16& p, int half) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack2<TYPE>(p[8 * half + 2 * i], p[8 * half + 2 * i + 1]);
  return w;
}

// Row of a 32-row block that element i of a lane's 16 belongs to.
__device__ __forceinline__ int block_row(int i) { return (i & 3) + 8 * (i >> 2) + 4 * ((threadIdx.x & 63) >> 5); }

// A value of lane l and of lane l ^ 32, the same bits in both: their maximum, their sum.
// (A bit cast takes a copy of a vector's element: of the element itself it reads the first.)
struct Halves {
  float lo, hi;
};
__device__ __forceinline__ Halves both_halves(float v) {
  const uint32_t w = __builtin_bit_cast(uint32_t, v);
  const auto s = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  const uint32_t lo = s[0], hi = s[1];
  return {__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi)};
}
__device__ __forceinline__ float half_max(float v) {
  const Halves h = both_halves(v);
  return __builtin_fmaxf(h.lo, h.hi);
}
__device__ __forceinline__ float half_sum(float v) {
  const Halves h = both_halves(v);
  return h.lo + h.hi;
}

// Where things lie in a tile: NB blocks of 32 channels.
template <int NB>
struct Tile {
  static constexpr int kPitch = NB <= 2 ? 128 : 256;    // bytes of a row
  static constexpr int kRowsPerCopy = 1024 / kPitch;    // rows of one copy instruction of a wavefront

  __device__ static __forceinline__ uint32_t swizzle(uint32_t row) {
    return NB <= 2 ? ((row >> 2) & 1) | (row & 3) << 1
                   : ((row >> 3) & 1) | ((row >> 2) & 1) << 1 | (row & 3) << 2;
  }
  // Byte of an ordinary operand read: row l % 32 of a block, channels 16 c + 8 (l / 32) + [0, 8);
  // blocks are 32 kPitch apart.
  __device__ static __forceinline__ uint32_t row_operand(int c) {
    const uint32_t lane = threadIdx.x & 63, row = lane & 31;
    return row * kPitch + ((2 * c + (lane >> 5)) ^ swizzle(row)) * 16;
  }
  // Byte of a transposing read: rows 4 (l / 32) + [0, 4) + 8 e of 16, channel 32 nb + l % 32; sets of
  // 16 rows are 16 kPitch apart.
  __device__ static __forceinline__ uint32_t column_operand(int nb, int e) {
    const uint32_t lane = threadIdx.x & 63, j = lane & 15;
    const uint32_t row = 4 * (lane >> 5) + (j >> 2) + 8 * e;
    const uint32_t chunk = 4 * nb + 2 * ((lane >> 4) & 1) + ((j & 3) >> 1);
    return row * kPitch + (chunk ^ swizzle(row)) * 16 + 8 * (j & 1);
  }
};

__device__ __forceinline__ u32x4 lds_read16(const char* p) { return *reinterpret_cast<const u32x4*>(p); }

__device__ __forceinline__ u32x2 lds_read_tr(const char* p) {
  using lds_s16x4 = __attribute__((address_space(3))) s16x4;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p)));
}

// One transposed operand: 16 rows of the tile from `base`, channels by the lane's two offsets.
__device__ __forceinline__ u32x4 column_read(const char* base, uint32_t first, uint32_t second) {
  const u32x2 a = lds_read_tr(base + first), b = lds_read_tr(base + second);
  return (u32x4){a[0], a[1], b[0], b[1]};
}

// A wavefront's part of a tile copy: COUNT instructions of 1 KiB to consecutive LDS.
// Inline assembly so that the compiler adds no waits of its own; the caller waits
// (vmcnt) and passes a barrier.  The block has no outputs besides a scalar save of
// M0; one wait state follows each M0 write, and s_nop 4 covers a scalar operand
// written just before.
template <int COUNT>
__device__ __forceinline__ void copy_to_lds(__amdgpu_buffer_rsrc_t rs, const uint32_t (&v)[COUNT], uint32_t lds) {
  static_assert(COUNT == 1 || COUNT == 2 || COUNT == 4 || COUNT == 8, "instructions of a copy");
  uint32_t saved;
  lds = __builtin_amdgcn_readfirstlane(lds);
  if constexpr (COUNT == 1) {
    asm volatile(
        "s_nop 4\n\ts_mov_b32 %[sv], m0\n\t"
        "s_mov_b32 m0, %[l0]\n\ts_nop 0\n\tbuffer_load_dwordx4 %[v0], %[rs], 0 offen lds\n\t"
        "s_mov_b32 m0, %[sv]"
        : [sv] "=&s"(saved)
        : [v0] "v"(v[0]), [rs] "s"(rs), [l0] "s"(lds)
        : "memory");
  } else if constexpr (COUNT == 2) {
    asm volatile(
        "s_nop 4\n\ts_mov_b32 %[sv], m0\n\t"
        "s_mov_b32 m0, %[l0]\n\ts_nop 0\n\tbuffer_load_dwordx4 %[v0], %[rs], 0 offen lds\n\t"
        "s_mov_b32 m0, %[l1]\n\ts_nop 0\n\tbuffer_load_dwordx4 %[v1], %[rs], 0 offen lds\n\t"
        "s_mov_b32 m0, %[sv]"
        : [sv] "=&s"(saved)
        : [v0] "v"(v[0]), [v1] "v"(v[1]), [rs] "s"(rs), [l0] "s"(lds), [l1] "s"(lds + 0x400u)
        : "memory");
  } else if constexpr (COUNT == 4) {
    asm volatile(
        "s_nop 4\n\ts_mov_b32 %[sv], m0\n\t"
        "s_mov_b32 m0, %[l0]\n\ts_nop 0\n\tbuffer_load_dwordx4 %[v0], %[rs], 0 offen lds\n\t"
        "s_mov_b32 m0, %[l1]\n\ts_nop 0\n\tbuffer_load_dwordx4 %[v1], %[rs], 0 offen lds\n\t"
        "s_mov_b32 m0, %[l2]\n\ts_nop 0\n\tbuffer_load_dwordx4 %[v2], %[rs], 0 offen lds\n\t"
        "s_mov_b32 m0, %[l3]\n\ts_nop 0\n\tbuffer_load_dwordx4 %[v3], %[rs], 0 offen lds\n\t"
        "s_mov_b32 m0, %[sv]"
        : [sv] "=&s"(saved)
        : [v0] "v"(v[0]), [v1] "v"(v[1]), [v2] "v"(v[2]), [v3] "v"(v[3]), [rs] "s"(rs), [l0] "s"(lds),
          [l1] "s"(lds + 0x400u), [l2] "s"(lds + 0x800u), [l3] "s"(lds + 0xc00u)
        : "memory");
  } else {
    const uint32_t lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
    copy_to_lds<4>(rs, lo, lds);
    copy_to_lds<4>(rs, hi, lds + 0x1000u);
  }
  (void)saved;
}

// Copies ROWS rows of a strided head into a tile.  The lane's share: byte offset and row of each of
// its instructions, from a base at the tile's first row.  WAVES wavefronts share the copy.
template <int NB, int ROWS, int WAVES>
struct TileCopy {
  using T = Tile<NB>;
  static constexpr int kCount = ROWS / T::kRowsPerCopy / WAVES;
  static_assert(kCount >= 1 && kCount * WAVES * T::kRowsPerCopy == ROWS, "every wavefront copies");
  uint32_t off[kCount];                                 // past head_dim: out of every buffer
  uint32_t lds;                                         // of the wavefront within the tile
  int row0;                                             // of instruction 0; kRowsPerCopy apart

  __device__ __forceinline__ void init(int wave, int64_t token_stride, int d) {
    const uint32_t lane = threadIdx.x & 63, slots = T::kPitch / 16;
    const int first = wave * kCount;
    row0 = first * T::kRowsPerCopy + (int)(lane / slots);
    lds = (uint32_t)first * 1024u;
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      const uint32_t row = row0 + i * T::kRowsPerCopy;
      const uint32_t chunk = (lane % slots) ^ T::swizzle(row);
      off[i] = (int)(8 * chunk) < d ? row * (uint32_t)(token_stride * 2) + chunk * 16 : kOobOffset;
    }
  }
  // Rows from `left` on are zeros.  `base` is the tile's first row (uniform).
  __device__ __forceinline__ void run(const void* base, int left, uint32_t lds_tile) const {
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(base, 0x7fffffff);
    if (left >= ROWS) {
      copy_to_lds<kCount>(rs, off, lds_tile + lds);
    } else {
      uint32_t v[kCount];
#pragma unroll
      for (int i = 0; i < kCount; ++i) v[i] = row0 + i * T::kRowsPerCopy < left ? off[i] : kOobOffset;
      copy_to_lds<kCount>(rs, v, lds_tile + lds);
    }
  }
};

__device__ __forceinline__ uint32_t lds_address(const char* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)(p);
}

// 32 rows of a head as the right-hand operand of 2 NB products of 16 channels: lane l has row
// l % 32, channels 16 c + 8 (l / 32) + [0, 8).  Rows past `left` and channels past d are zeros.
template <int NB>
__device__ __forceinline__ void load_rows(const uint16_t* base, int64_t token_stride, int64_t left, int d, u32x4 (&f)[2 * NB]) {
  const int lane = threadIdx.x & 63, row = lane & 31;
  const uint16_t* p = base + row * token_stride + 8 * (lane >> 5);
#pragma unroll
  for (int c = 0; c < 2 * NB; ++c) {
    f[c] = (u32x4){0, 0, 0, 0};
    if (row < left && 16 * c + 8 * (lane >> 5) < d) f[c] = *reinterpret_cast<const u32x4*>(p + 16 * c);
  }
}

// Waits for loaded operands here.  Left to the first product, the compiler's wait would stand inside
// the loop, and take the copies in flight for the loads.
template <int N>
__device__ __forceinline__ void settle(u32x4 (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+v"(f[i]));
}

// Stores a transposed result (a lane's column is row l % 32 of the tensor): halves of the wavefront
// exchange 4 channels each, so that a lane has 8 consecutive ones, 16 bytes.
template <int TYPE, int NB>
__device__ __forceinline__ void store_rows(uint16_t* base, int64_t token_stride, int64_t left, int d, const f32x16 (&acc)[NB],
                                           float factor) {
  const int lane = threadIdx.x & 63, row = lane & 31, h = lane >> 5;
  uint16_t* p = base + row * token_stride + 8 * h;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      uint32_t x[2], y[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[i] = pack2<TYPE>(acc[nb][8 * a + 2 * i] * factor, acc[nb][8 * a + 2 * i + 1] * factor);
        y[i] = pack2<TYPE>(acc[nb][8 * a + 4 + 2 * i] * factor, acc[nb][8 * a + 4 + 2 * i + 1] * factor);
        const auto s = __builtin_amdgcn_permlane32_swap(x[i], y[i], false, false);
        x[i] = s[0];
        y[i] = s[1];
      }
      const int c = 32 * nb + 16 * a;
      if (row < left && c + 8 * h < d) *reinterpret_cast<u32x4*>(p + c) = (u32x4){x[0], x[1], y[0], y[1]};
    }
}

// ---------------------------------------------------------------------------
// Which rows a workgroup works on.
// ---------------------------------------------------------------------------
struct Span {
  int64_t start;                                        // first row (packed), or 0
  int64_t len;
};

// Rows [start, start + len) of packed sequence s, cut to the tensor.
__device__ __forceinline__ Span packed_span(const int32_t* starts, int64_t s, int64_t total) {
  int64_t lo = starts[s], hi = starts[s + 1];
  lo = lo < 0 ? 0 : lo > total ? total : lo;
  hi = hi < lo ? lo : hi > total ? total : hi;
  return {lo, hi - lo};
}

// Number `id` of the workgroups of a packed batch: tile `tile` of `rows` rows of a sequence in a head; sequences go
// one after another, then heads, then tiles.  Not found: this workgroup has nothing to do (`tile` < 0), or none is left and
// `tile` counts those past the last one.
struct PackedTile {
  bool found;
  int64_t seq, head, tile;
};

// Up to 64 sequences, a lane to each: the longest first (a long one started last would run alone at the end).
__device__ __forceinline__ PackedTile longest_first(const int32_t* starts, int64_t sequences, int64_t total, int rows,
                                                    int64_t heads, int64_t id) {
  const int lane = threadIdx.x & 63, count = (int)sequences;
  int32_t n = 0;
  if (lane < count) n = (int32_t)((packed_span(starts, lane, total).len + rows - 1) / rows);
  int64_t before = 0, all = 0;                          // tiles of the sequences before this lane's, of all
  for (int k = 0; k < count; ++k) {
    const int32_t other = __builtin_amdgcn_readlane(n, k);
    before += ((other > n) | ((other == n) & (k < lane))) ? other : 0;      // no branch: `all` would lose its scalar register
    all += other;
  }
  const uint64_t hit = __ballot(id >= before * heads && id < (before + n) * heads);
  if (hit == 0) return {false, 0, 0, id - all * heads};
  const int at = __builtin_ctzll(hit);
  const int64_t lo = (uint32_t)__builtin_amdgcn_readlane((int)before, at);
  const int64_t hi = __builtin_amdgcn_readlane((int)(before >> 32), at);
  const int64_t in = id - (hi << 32 | lo) * heads, tiles = __builtin_amdgcn_readlane(n, at), head = in / tiles;
  return {true, at, head, in - head * tiles};
}

// More sequences: sequence s has the slots from first(s) = floor((its start - the first's) / rows) + s on, which is as
// many as its tiles or one more, so that it is found by a search and not by a walk over those before it (for 100 000
// sequences of a token in 8 heads the walks would take seconds).  64 places a step: 2 steps up to 4096 sequences, 4 up to
// 16 million.
__device__ __forceinline__ PackedTile by_slot(const int32_t* starts, int64_t sequences, int64_t total, int rows, int64_t heads,
                                              int64_t id) {
  const int lane = threadIdx.x & 63;
  const int64_t begin = packed_span(starts, 0, total).start;
  auto place = [&](int64_t s) {                         // where sequence s starts, and the last one ends
    if (s < sequences) return packed_span(starts, s, total).start;
    const Span last = packed_span(starts, sequences - 1, total);
    return last.start + last.len;
  };
  auto first = [&](int64_t s) { return (place(s) - begin) / rows + s; };
  const int64_t slot = id / heads;
  int64_t seq = 0, width = sequences + 1;               // the last s with first(s) <= slot is one of `width` from seq on
  while (width > 1) {
    const int64_t step = (width + 63) / 64, off = lane * step;
    const uint64_t hit = __ballot(off < width && first(seq + (off < width ? off : 0)) <= slot);
    const int64_t at = hit == 0 ? 0 : (63 - __builtin_clzll(hit)) * step;
    seq += at;
    width = width - at < step ? width - at : step;
  }
  const int64_t here = first(seq), in = id - here * heads;
  if (seq == sequences) return {false, 0, 0, in};
  const int64_t slots = first(seq + 1) - here;
  if (in < 0 || in >= slots * heads) return {false, 0, 0, -1};        // starts that do not rise
  const int64_t head = in / slots, tile = in - head * slots;
  const int64_t t = tile * rows < packed_span(starts, seq, total).len ? tile : -1;
  return {t >= 0, seq, head, t};
}

__device__ __forceinline__ PackedTile packed_tile(const int32_t* starts, int64_t sequences, int64_t total, int rows,
                                                  int64_t heads, int64_t id) {
  return sequences <= 64 ? longest_first(starts, sequences, total, rows, heads, id)
                         : by_slot(starts, sequences, total, rows, heads, id);
}

__device__ __forceinline__ int clamp_rows(int64_t v) { return (int)(v < 0 ? 0 : v < 1 << 20 ? v : 1 << 20); }

// Workgroups go to the 8 XCDs in turn, each with its own L2: number `id` of `total` renumbered so
// that an XCD has consecutive ones (which share keys and values).
__device__ __forceinline__ int64_t xcd_order(int64_t id, int64_t total) {
  const int64_t xcd = id % 8, local = id / 8, per = total / 8, extra = total % 8;
  return xcd * per + (xcd < extra ? xcd : extra) + local;
}

// The same for packed batches, whose work falls from first to last: 4 consecutive ones to an XCD in turn.
__device__ __forceinline__ int64_t xcd_order4(int64_t id, int64_t total) {
  const int64_t in = id % 32, block = id - in;
  return block + 32 <= total ? block + (in % 8) * 4 + in / 8 : id;
}

// Number of copies still in flight that may stay so.
template <int N>
__device__ __forceinline__ void wait_copies() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }
// The workgroup's barrier between two tiles: this wavefront's copies have arrived, and its reads of the tile before, which
// the next copy writes over, are back (in one block: products, and the waits that they bring, may move across an asm).
__device__ __forceinline__ void tile_barrier() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// What a workgroup of query tiles works on: rows [row, row + ..) of one sequence's queries in one head.
struct QueryWork {
  int64_t seq, head, tile;
  Span q, k;
  const uint16_t *kp, *vp;                              // key row 0 of the sequence
  int64_t q_off, o_off, lse_off;                        // query row 0: elements into q, o and lse
};

// Number `id` of the grid.  Causal tiles go from the last, which sees the most keys, to the first.  False: no
// such tile, `tile` then counts the workgroups past the last one, or is negative.
__device__ __forceinline__ bool query_work(const AttnArgs& a, int64_t id, int rows, QueryWork& w) {
  int64_t t;
  if (a.q_starts != nullptr) {
    const PackedTile p = packed_tile(a.q_starts, a.sequences, a.tq, rows, a.hq, id);
    t = w.tile = p.tile;
    if (!p.found) return false;
    w.seq = p.seq;
    w.head = p.head;
    w.q = packed_span(a.q_starts, w.seq, a.tq);
    w.k = packed_span(a.k_starts, w.seq, a.tk);
    w.lse_off = w.head * a.tq + w.q.start;
  } else {
    const int64_t item = id / a.tiles;
    t = id - item * a.tiles;
    w.seq = item / a.hq;
    w.head = item - w.seq * a.hq;
    w.q = {0, a.tq};
    w.k = {0, a.tk};
    if (a.k_lens != nullptr) {
      const int64_t n = a.k_lens[w.seq];
      w.k.len = n < 0 ? 0 : n < a.tk ? n : a.tk;
    }
    w.lse_off = (w.seq * a.hq + w.head) * a.tq;
  }
  const int64_t b = a.q_starts != nullptr ? 0 : w.seq, kv = w.head / a.group;
  w.tile = a.causal ? (w.q.len + rows - 1) / rows - 1 - t : t;
  w.q_off = b * a.q.b + w.q.start * a.q.t + w.head * a.q.h;
  w.o_off = b * a.o.b + w.q.start * a.o.t + w.head * a.o.h;
  w.kp = a.k.p + b * a.k.b + w.k.start * a.k.t + kv * a.k.h;
  w.vp = a.v.p + b * a.v.b + w.k.start * a.v.t + kv * a.v.h;
  return true;
}

// The rows of a packed tensor that lie in no sequence, in every head: f(row, head) for the share of workgroup
// number `part` of those past the last tile, which are at least one; `parts` of 256 threads at most stride over them.
template <typename F>
__device__ __forceinline__ void rest_rows(const int32_t* starts, int64_t sequences, int64_t total, int64_t heads, int64_t part,
                                          int64_t parts, F f) {
  const int64_t first = packed_span(starts, 0, total).start;
  const Span last = packed_span(starts, sequences - 1, total);
  const int64_t end = last.start + last.len, rest = (first + total - end) * heads;
  for (int64_t i = part * blockDim.x + threadIdx.x; i < rest; i += parts * blockDim.x) {
    const int64_t row = i / heads;
    f(row < first ? row : end + row - first, i - row * heads);
  }
}

}  // namespace rtl
