// Attention of many query rows a key-value head over the paged cache: the new
// tokens of a chunk (causal, with windows, prefixes, documents, capped scores and
// a distance bias), and the sequences that share a prefix.
//
//   z = scale q.k;  z = cap tanh(z / cap);  z -= slope |pos - p|
//   out = sum_p e^(z_p - m) v_p / sum_p e^(z_p - m),  lse = m + log sum_p e^(z_p - m)
//
// A workgroup takes a block of 32 kW rows, 32 a wave, through the places that any
// of them sees, 64 at a time:
//  - keys and values go from memory to registers one tile ahead, are converted
//    there, and put into one of two LDS buffers; rows are padded so that no two
//    lanes of a read share a bank;
//  - S^T = K Q^T by v_mfma_f32_32x32x16_bf16: a lane then has 32 scores of one
//    query row, so the running maximum takes one exchange between lanes;
//  - O^T = V^T P^T: the scores' registers are the P^T operand as they stand, with
//    the places in an order that V's transposing LDS reads follow.
//
// Two waves share a SIMD up to heads of 128, one's softmax beside the other's products;
// a larger head's accumulators take the registers of both.  The workgroup stays on its
// CU and goes from piece to piece with the next tiles already under way.  Blocks have
// 256 rows where a tile of them fits the registers: the keys pass through LDS half as
// often (2048 tokens behind 14336 in 8 bits 666 us, with 128 rows 840; four prompts of
// documents 98 us, 125).
//
// Bound by the matrix cores and the vector unit together: of the cycles of 2048 tokens
// behind 14336 the first are busy in 38 %, the second in 42 %, and they overlap little.
// Rates: 816 TFLOP/s there (8192^3 product on this card: 1255); 16-bit prompts of 8192
// tokens 702, of 4 x 2048 669; heads of 256 525, with capped scores 350.
#include <cstddef>

#include "attention_common.hpp"
#include "tile_plan.hpp"

namespace engram {
namespace {

using namespace attn;

constexpr int kTile = kWideTile;
constexpr float kLazy = 8.0f;

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Accumulators that the wave's own instructions scale or add to, rarely.  In large
// heads they are to stay where the matrix core has them: left to itself the compiler
// moves all of them to and fro around each of its products.  A product's result takes
// up to 18 waits to be readable by other instructions, and what is written there some
// before it is read.
template <bool kKeep>
__device__ __forceinline__ void scale(f32x16 &o, float by) {
  if constexpr (!kKeep) {
    o *= by;
  } else {
    asm volatile("s_nop 15\n\ts_nop 7");
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float x = o[i], y;
      asm volatile("v_accvgpr_read_b32 %1, %0\n\tv_mul_f32 %1, %1, %2\n\tv_accvgpr_write_b32 %0, %1\n\ts_nop 3"
                   : "+a"(x), "=&v"(y) : "v"(by));
      o[i] = x;
    }
  }
}
template <bool kKeep>
__device__ __forceinline__ float plus(float o, float more) {
  if constexpr (!kKeep) return o + more;
  float y;
  asm volatile("s_nop 15\n\ts_nop 7\n\tv_accvgpr_read_b32 %1, %0\n\tv_add_f32 %1, %1, %2\n\tv_accvgpr_write_b32 %0, %1\n\ts_nop 3"
               : "+a"(o), "=&v"(y) : "v"(more));
  return o;
}

// Over lanes l and l ^ 32, which hold one query row.
__device__ __forceinline__ float pair_max(float x) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float pair_sum(float x) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// 4 places' values of one dimension a lane: lanes 4 r .. 4 r + 3 of 16 address 4
// dimensions each of place r, and lane i gets dimension i of the four.
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x2 read_transposed(const uint8_t *p) {
  typedef __attribute__((address_space(3))) s16x4 *Lds;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p)));
}

// A tile in LDS: keys in rows of 2 D + 16 bytes (16 places at one piece of 16 bytes
// lie in different banks), values in rows of 64 bytes or 192 past a multiple of 256
// (so do 4 places' 64 bytes, which half a wave's transposing read takes at once).
template <int kDb>
struct Stage {
  static constexpr int kKeyRow = 64 * kDb + 16;
  static constexpr int kValueRow = 64 * kDb + (kDb % 2 ? 0 : 64);
  static constexpr int kValues = kTile * kKeyRow;
  static constexpr int kBytes = kTile * (kKeyRow + kValueRow);
};

// What a workgroup works at next: a block, or a run's piece of one, of a key-value
// head.  Wave 0 writes the tickets to LDS, a piece ahead.
struct Ticket {
  TileBlock w;
  int32_t kvh, t0, count, flags;           // bit 0: there is one; bit 1: its whole block; bit 2: not the run's first
};
constexpr int kBlockWords = sizeof(TileBlock) / 4;

template <int kDb, bool kMx, int kW, bool kRules>
__global__ __launch_bounds__(64 * kW, kDb <= 4 ? 2 : 1) void tile_wide_kernel(TileAttention a, TilePlan plan) {
  constexpr int D = 32 * kDb, kThreads = 64 * kW;
  constexpr int kRowBytes = kMx ? D : 2 * D;
  // Large heads' tiles are staged in two rounds, for want of registers.
  constexpr int kPieces = kRowBytes / 16, kRounds = !kMx && kTile * kPieces > 3 * kThreads ? 2 : 1, kPart = kTile / kRounds;
  constexpr int kLoads = (kPart * kPieces + kThreads - 1) / kThreads;
  constexpr bool kKeep = kDb > 4;
  using S = Stage<kDb>;
  extern __shared__ u32x4 stages_lds[];      // [2] stages
  uint8_t *const lds = reinterpret_cast<uint8_t *>(stages_lds);
  // Of the tiles in flight, by tile % 3: places on pages outside the cache, and
  // places whose values are not all finite.
  __shared__ uint32_t absent_lds[3][2], odd_lds[3][2];
  __shared__ Ticket ticket_lds[4];
  __shared__ int work_lds[2];

  const CacheView &c = a.cache;
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int mask = (1 << c.page_shift) - 1;
  const ScoreUnit su = score_unit(a, kLog2e);
  const TileList &list = plan.list[0];
  const TileHeader head = *list.header;
  Work work;
  if (!first_work(list, head, c.kv_heads, kThreads, work_lds, &work)) return;

  // Wave 0: ticket n's block is requested, and later written down.  Whole blocks are
  // dealt out in their order, every second round backwards (but for the last three
  // bits, which keep a head's blocks on one XCD).
  int next_block = work.block, next_kvh = work.kvh, next_unit = work.unit, left = work.left, word = 0;
  auto place_in_order = [&](int n) {
    const int b = blockIdx.x;
    return n * list.runs + (n % 2 && list.runs % 8 == 0 ? (list.runs - 8 - (b & ~7)) + (b & 7) : b);
  };
  auto ask_ticket = [&](int n) {
    if (head.direct) {
      const int e = place_in_order(n);
      next_kvh = e % c.kv_heads;
      next_block = e < head.blocks * c.kv_heads ? list.order[e / c.kv_heads] : -1;
    } else if (left <= 0) {
      next_block = -1;
    }
    if (next_block >= 0 && lane < kBlockWords) word = reinterpret_cast<const int *>(list.blocks + next_block)[lane];
  };
  auto write_ticket = [&](int n) {
    Ticket &t = ticket_lds[n & 3];
    const bool there = __builtin_amdgcn_readfirstlane(next_block) >= 0;
    const int tiles = __builtin_amdgcn_readlane(word, offsetof(TileBlock, a_n) / 4) +
                      __builtin_amdgcn_readlane(word, offsetof(TileBlock, b_n) / 4);
    const int unit = head.direct ? 0 : next_unit, count = head.direct ? tiles : min(tiles - unit, left);
    if (lane < kBlockWords) reinterpret_cast<int *>(&t.w)[lane] = word;
    if (lane == 0) {
      t.kvh = next_kvh, t.t0 = unit, t.count = count;
      t.flags = (there ? 1 : 0) | (count == tiles ? 2 : 0) | (n > 0 ? 4 : 0);
    }
    if (!head.direct) {
      left -= count;
      next_unit = 0;
      if (++next_block == head.blocks) next_block = 0, ++next_kvh;
    }
  };
  if (wave == 0) {
    ask_ticket(0);
    write_ticket(0);
    ask_ticket(1);
    write_ticket(1);
  }
  if (tid < 6) absent_lds[tid / 2][tid % 2] = odd_lds[tid / 2][tid % 2] = 0;
  __syncthreads();
  auto uniform = [](int x) { return __builtin_amdgcn_readfirstlane(x); };

  // Three tiles are under way: the pages of one are asked for, the keys and values of
  // the one before it, and the one before that is worked at.  A piece's tiles follow
  // those of the piece before it.
  struct Tile {
    int p0, kvh, flags;                      // flags: 1: there is one, 2: some row does not see all of it
    uint64_t used;                           // bit i: some row sees place p0 + i
  };
  int ask_piece = -1, ask_t = 0, ask_t1 = 0;
  TileBlock aw{};                            // what of the piece's block the tiles need
  int ask_kvh = 0;
  const int32_t *table = nullptr;
  bool fetch = false;                        // a ticket has been asked for
  auto range = [](int lo, int hi) {          // bits lo .. hi - 1, as far as there are any
    lo = min(max(lo, 0), 64), hi = min(max(hi, lo), 64);
    return (hi == 64 ? ~uint64_t(0) : (uint64_t(1) << hi) - 1) & (lo == 64 ? uint64_t(0) : ~uint64_t(0) << lo);
  };
  int page[kRounds][kLoads];
  auto ask_tile = [&]() {
    if (ask_t == ask_t1) {
      const Ticket &t = ticket_lds[(ask_piece + 1) & 3];
      if (!(uniform(t.flags) & 1)) return Tile{0, 0, 0, 0};
      ++ask_piece;
      aw.kind = uniform(t.w.kind), aw.seq = uniform(t.w.seq), aw.len = uniform(t.w.len);
      aw.a_lo = uniform(t.w.a_lo), aw.a_hi = uniform(t.w.a_hi), aw.b_lo = uniform(t.w.b_lo), aw.b_hi = uniform(t.w.b_hi);
      aw.a_tile = uniform(t.w.a_tile), aw.a_n = uniform(t.w.a_n), aw.b_tile = uniform(t.w.b_tile);
      aw.all_lo = uniform(t.w.all_lo), aw.all_hi = uniform(t.w.all_hi);
      aw.all_first = uniform(t.w.all_first), aw.all_last = uniform(t.w.all_last);
      ask_kvh = uniform(t.kvh), ask_t = uniform(t.t0), ask_t1 = ask_t + uniform(t.count);
      table = aw.kind == kSharedPrefix ? a.prefix_table + int64_t(aw.seq) * a.prefix_width
                                       : a.table + int64_t(aw.seq) * a.table_width;
      if (aw.len == 0) table = list.queue;   // any memory: there is no place to look up
      if (wave == 0 && ask_piece > 0) ask_ticket(ask_piece + 1);
      fetch = ask_piece > 0;                 // the first two are written
    }
    const int p0 = aw.place(ask_t++, kTile), last = max(0, aw.len - 1);
    const bool plain = (p0 >= aw.all_lo && p0 + kTile <= aw.all_hi) || (p0 >= aw.all_first && p0 + kTile <= aw.all_last);
#pragma unroll
    for (int x = 0; x < kRounds; ++x)
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        page[x][i] = table[min(p0 + kPart * x + (tid + i * kThreads) / kPieces, last) >> c.page_shift];
    return Tile{p0, ask_kvh, plain ? 1 : 3, range(aw.a_lo - p0, aw.a_hi - p0) | range(aw.b_lo - p0, aw.b_hi - p0)};
  };

  // A thread's pieces of a tile: 16 bytes of keys and of values.
  u32x4 key[kLoads], value[kLoads];
  uint32_t scales[kLoads];                   // the key's and the value's byte (8-bit format)
  uint32_t shown = 0;                        // bit i: piece i is of a place that is used, on a page
  uint32_t missing = 0;                      // ... on no page of the cache
  auto load = [&](const Tile &t, int round) {
    shown = missing = 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int id = tid + i * kThreads, at = id % kPieces, in_tile = kPart * round + id / kPieces;
      const bool in = (kPart * kPieces % kThreads == 0 || id < kPart * kPieces) && (t.used >> in_tile & 1);
      const bool there = unsigned(page[round][i]) < unsigned(c.pages);
      shown |= uint32_t(in & there) << i;
      missing |= uint32_t(in & !there) << i;
      // What is not there is read from the cache's first row instead, and not used.
      const int64_t place = (in & there) ? ((int64_t(page[round][i]) * c.kv_heads + t.kvh) << c.page_shift) + ((t.p0 + in_tile) & mask) : 0;
      key[i] = *reinterpret_cast<const u32x4 *>(static_cast<const uint8_t *>(c.k) + place * kRowBytes + 16 * at);
      value[i] = *reinterpret_cast<const u32x4 *>(static_cast<const uint8_t *>(c.v) + place * kRowBytes + 16 * at);
      if constexpr (kMx)
        scales[i] = c.k_scales[place * kDb + at / 2] | uint32_t(c.v_scales[place * kDb + at / 2]) << 8;
    }
  };
  auto put = [&](const Tile &tile, int t, int round) {       // tile number t
    uint8_t *const st = lds + t % 2 * S::kBytes;
    const bool edge = tile.flags & 2;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int id = tid + i * kThreads, in_tile = kPart * round + id / kPieces, at = id % kPieces;
      if (kPart * kPieces % kThreads != 0 && id >= kPart * kPieces) break;
      constexpr int kOut = kMx ? 2 : 1;    // pieces of 8 values
      u32x4 k[kOut], v[kOut];
      if constexpr (kMx) {
        const float ks = e8m0_to_float(scales[i] & 255u);
        const float vs = e8m0_to_float(min(scales[i] >> 8, 254u));
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          k[x / 4][x % 4] = mx_pair(key[i][x / 2], ks, x & 1);
          v[x / 4][x % 4] = mx_pair(value[i][x / 2], vs, x & 1);
        }
      } else {
        k[0] = key[i], v[0] = value[i];
      }
      if (edge || missing) {
        const bool keep = shown >> i & 1;
        bool finite = true;
#pragma unroll
        for (int o = 0; o < kOut; ++o) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            k[o][x] = keep ? k[o][x] : 0u;
            v[o][x] = keep ? v[o][x] : 0u;
            finite = finite & ((v[o][x] & 0x7F80u) != 0x7F80u) & ((v[o][x] & 0x7F800000u) != 0x7F800000u);
          }
        }
        // A weight of 0 times a value that is not finite would reach rows that do
        // not see it: it counts as 0 here, and add_odd() gives it to those that do.
        if (!finite) {
          atomicOr(&odd_lds[t % 3][in_tile / 32], 1u << (in_tile & 31));
#pragma unroll
          for (int o = 0; o < kOut; ++o)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              if ((v[o][x] & 0x7F80u) == 0x7F80u) v[o][x] &= 0xFFFF0000u;
              if ((v[o][x] & 0x7F800000u) == 0x7F800000u) v[o][x] &= 0xFFFFu;
            }
        }
        if (missing >> i & 1) {
          atomicOr(&absent_lds[t % 3][in_tile / 32], 1u << (in_tile & 31));
          if (at == 0 && tile.kvh == 0 && a.bad_pages) atomicAdd(a.bad_pages, 1);
        }
      }
#pragma unroll
      for (int o = 0; o < kOut; ++o) {
        *reinterpret_cast<u32x4 *>(st + in_tile * S::kKeyRow + (kOut * at + o) * 16) = k[o];
        *reinterpret_cast<u32x4 *>(st + S::kValues + in_tile * S::kValueRow + (kOut * at + o) * 16) = v[o];
      }
    }
  };

  Tile now = ask_tile();
#pragma unroll
  for (int x = 0; x < kRounds; ++x) {
    load(now, x);
    put(now, 0, x);
  }
  Tile soon = ask_tile();                    // its pages; keys and values below
  if (wave == 0 && fetch) write_ticket(ask_piece + 1);
  fetch = false;
  __syncthreads();

  int t = 0;                                 // tiles since the start
  for (int piece = 0;; ++piece) {
    const Ticket &ticket = ticket_lds[piece & 3];
    const int flags = uniform(ticket.flags);
    if (!(flags & 1)) return;
    TileBlock w{};
    w.kind = uniform(ticket.w.kind), w.seq = uniform(ticket.w.seq), w.token0 = uniform(ticket.w.token0);
    w.first = uniform(ticket.w.first), w.row0 = uniform(ticket.w.row0), w.rows = uniform(ticket.w.rows);
    w.len = uniform(ticket.w.len);
    const int kvh = uniform(ticket.kvh), count = uniform(ticket.count);
    const bool whole = flags & 2;

    // This lane's query row, and what it sees.
    const int row = wave * kRows + col;
    const bool active = wave * kRows < w.rows;
    const QueryRow qr = query_row(a, w, kvh, min(row, w.rows - 1));
    const int pos = w.first + qr.tok;
    bf16x8 q[2 * kDb];
#pragma unroll
    for (int kk = 0; kk < 2 * kDb; ++kk) {
      u32x4 v = *reinterpret_cast<const u32x4 *>(a.q + qr.at * D + 16 * kk + 8 * half);
#pragma unroll
      for (int x = 0; x < 4; ++x) v[x] = (v[x] ^ su.flip) & su.keep;
      q[kk] = __builtin_bit_cast(bf16x8, v);
    }
    RowSees r{0, w.len, 0, 0};
    if (w.kind == kChunk) r = token_sees(a.rules, w.seq, qr.token, pos, w.len);
    const float slope = kRules && a.rules.slopes ? a.rules.slopes[qr.head] * kLog2e : 0.0f;
    // A tile that all rows of a wave see needs no masks.
    int4 lim = {r.lo, r.lo + r.n, r.first, r.first + r.m};
#pragma unroll
    for (int x = 1; x < 32; x *= 2) {
      lim.x = max(lim.x, __shfl_xor(lim.x, x));
      lim.y = min(lim.y, __shfl_xor(lim.y, x));
      lim.z = max(lim.z, __shfl_xor(lim.z, x));
      lim.w = min(lim.w, __shfl_xor(lim.w, x));
    }
    lim = {uniform(lim.x), uniform(lim.y), uniform(lim.z), uniform(lim.w)};
    auto plain = [&](int p0) { return (p0 >= lim.x && p0 + kTile <= lim.y) || (p0 >= lim.z && p0 + kTile <= lim.w); };

    float m = -INFINITY, l = 0.0f;           // l: of this lane's places
    f32x16 o[kDb];
#pragma unroll
    for (int n = 0; n < kDb; ++n) o[n] = f32x16{};

    for (int end = t + count; t < end; ++t) {
      const int p0 = now.p0;
      const Tile coming = soon;
      if (coming.flags) load(coming, 0);
      if (kRounds == 1 && coming.flags) soon = ask_tile();
      // (tile + 2) % 3 was read before the last barrier, and is written after the next.
      if (tid < 2) absent_lds[(t + 2) % 3][tid] = odd_lds[(t + 2) % 3][tid] = 0;
      const uint8_t *const st = lds + t % 2 * S::kBytes;
      const uint32_t absent[2] = {absent_lds[t % 3][0], absent_lds[t % 3][1]};
      const uint32_t odd[2] = {odd_lds[t % 3][0], odd_lds[t % 3][1]};
      const bool any_absent = __builtin_amdgcn_readfirstlane(absent[0] | absent[1]) != 0;
      const bool any_odd = __builtin_amdgcn_readfirstlane(odd[0] | odd[1]) != 0;

      auto stage_rest = [&] {                // the second round, as a part of the work on the tile before
        if (kRounds == 2 && coming.flags) {
          put(coming, t + 1, 0);
          load(coming, 1);
          soon = ask_tile();
        }
      };
      if (!active) stage_rest();
      if (active) {
        // Operands come 4 at a time, each four requested before the four before it
        // are used: more would not fit the registers.
        bf16x8 kf[2][4];
        auto read_keys = [&](int i, bf16x8(&f)[4]) {
#pragma unroll
          for (int x = 0; x < 4; ++x)
            f[x] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(
                st + (32 * (x % 2) + col) * S::kKeyRow + 32 * (2 * i + x / 2) + 16 * half));
        };
        const uint8_t *const vp = st + S::kValues + (4 * half + lane % 16 / 4) * S::kValueRow +
                                  32 * (lane / 16 % 2) + 8 * (lane % 4);
        bf16x8 vf[2][4];
        auto read_values = [&](int i, bf16x8(&f)[4]) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int j = (4 * i + x) / kDb, n = (4 * i + x) % kDb;
            const u32x2 lo = read_transposed(vp + 16 * j * S::kValueRow + 64 * n);
            const u32x2 hi = read_transposed(vp + (16 * j + 8) * S::kValueRow + 64 * n);
            f[x] = as_frag(lo[0], lo[1], hi[0], hi[1]);
          }
        };
        f32x16 z[2] = {};
        read_keys(0, kf[0]);
#pragma unroll
        for (int i = 0; i < kDb; ++i) {
          if (i + 1 < kDb) read_keys(i + 1, kf[(i + 1) % 2]);
          else read_values(0, vf[0]);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int x = 0; x < 4; ++x) z[x % 2] = mfma32(kf[i % 2][x], q[2 * i + x / 2], z[x % 2]);
          __builtin_amdgcn_sched_barrier(0);
        }
        stage_rest();
        // Register 4 i + j of tile half u: place 32 u + 8 i + 4 half + j.
        const bool masked = !plain(p0) || any_absent;
        if constexpr (kRules) {
#pragma unroll
          for (int x = 0; x < 32; ++x) z[x / 16][x % 16] *= su.unit;
          if (a.rules.cap > 0.0f) {
            float far = 0.0f;
#pragma unroll
            for (int x = 0; x < 32; ++x) far = fmaxf(far, fabsf(z[x / 16][x % 16]));
            if (__any(!(far <= kTanhSplit))) {
#pragma unroll
              for (int x = 0; x < 32; ++x) {
                const float y = z[x / 16][x % 16];
                z[x / 16][x % 16] = su.cap2 * (fabsf(y) <= kTanhSplit ? tanh_small(y) : tanh_large(y));
              }
            } else {
#pragma unroll
              for (int x = 0; x < 32; ++x) z[x / 16][x % 16] = su.cap2 * tanh_small(z[x / 16][x % 16]);
            }
          }
          if (a.rules.slopes) {
            // Distances below 2^24 are whole numbers in fp32, larger ones off by half a step.
            const float ahead = float(pos - p0 - 4 * half);
#pragma unroll
            for (int x = 0; x < 32; ++x) {
              const float back = ahead - float(32 * (x / 16) + 8 * (x % 16 / 4) + x % 4);
              z[x / 16][x % 16] = __builtin_fmaf(-slope, fabsf(back), z[x / 16][x % 16]);
            }
          }
        }
        if (masked) {
          const int from_lo = p0 + 4 * half - r.lo, from_first = p0 + 4 * half - r.first;
          const uint32_t away[2] = {absent[0] >> (4 * half), absent[1] >> (4 * half)};
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            const int at = 8 * (x % 16 / 4) + x % 4, step = 32 * (x / 16) + at;
            const bool ok = ((unsigned(from_lo + step) < unsigned(r.n)) | (unsigned(from_first + step) < unsigned(r.m))) &
                            !(away[x / 16] & 1u << at);
            z[x / 16][x % 16] = ok ? z[x / 16][x % 16] : -INFINITY;
          }
        }
        float top = z[0][0];
#pragma unroll
        for (int x = 1; x < 32; ++x) top = fmaxf(top, z[x / 16][x % 16]);
        top = pair_max(kRules ? top : top * su.unit);
        // The weights' reference follows the largest score only where that is 2^8 above it.
        if (__any(top > m + kLazy)) {
          const float mn = fmaxf(m, top);
          const float keep = mn == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
          m = mn;
          l *= keep;
#pragma unroll
          for (int n = 0; n < kDb; ++n) scale<kKeep>(o[n], keep);
        }
        const float ms = m == -INFINITY ? 0.0f : m;
        float sum[2] = {};
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          const float y = z[x / 16][x % 16];
          z[x / 16][x % 16] = __builtin_amdgcn_exp2f(kRules ? y - ms : __builtin_fmaf(y, su.unit, -ms));
          sum[x / 16] += z[x / 16][x % 16];
        }
        l += sum[0] + sum[1];
        bf16x8 p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x16 &e = z[j / 2];
          const int x = 8 * (j % 2);
          p[j] = as_frag(pack_bf16x2(e[x], e[x + 1]), pack_bf16x2(e[x + 2], e[x + 3]),
                         pack_bf16x2(e[x + 4], e[x + 5]), pack_bf16x2(e[x + 6], e[x + 7]));
        }
#pragma unroll
        for (int i = 0; i < kDb; ++i) {
          __builtin_amdgcn_sched_barrier(0);
          if (i + 1 < kDb) read_values(i + 1, vf[(i + 1) % 2]);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int j = (4 * i + x) / kDb, n = (4 * i + x) % kDb;
            o[n] = mfma32(vf[i % 2][x], p[j], o[n]);
          }
        }
        if (any_odd) {                       // values that are not finite, to the rows that see them
          for (int i = 0; i < kTile; ++i) {
            if (!(__builtin_amdgcn_readfirstlane(odd[i / 32]) >> (i & 31) & 1)) continue;
            float e = 0.0f;                  // the weight, in the half that holds it
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (x == i / 32 * 16 + (i & 31) / 8 * 4 + i % 4) e = z[x / 16][x % 16];
            e = __shfl(e, col + 32 * (i / 4 & 1));
            const int p = p0 + i;
            const int32_t *const mine = w.kind == kSharedPrefix ? a.prefix_table + int64_t(w.seq) * a.prefix_width
                                                                : a.table + int64_t(w.seq) * a.table_width;
            const int pg = mine[p >> c.page_shift];
            const int64_t place = ((int64_t(pg) * c.kv_heads + kvh) << c.page_shift) + (p & mask);
            const bool ok = sees(r, p);
#pragma unroll
            for (int n = 0; n < kDb; ++n) {
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                float v[4];
                values_at<kMx>(c, c.v, c.v_scales, place, 32 * n + 8 * x + 4 * half, v);
#pragma unroll
                for (int y = 0; y < 4; ++y)
                  o[n][4 * x + y] = plus<kKeep>(o[n][4 * x + y], ok && !(fabsf(v[y]) < INFINITY) ? e * v[y] : 0.0f);
              }
              __builtin_amdgcn_sched_barrier(0);      // no more of these loads at a time: registers
            }
          }
        }
      }
      if (coming.flags) put(coming, t + 1, kRounds - 1);
      else soon = Tile{0, 0, 0, 0};
      now = coming;
      if (wave == 0 && fetch) write_ticket(ask_piece + 1);
      fetch = false;
      __syncthreads();
    }

    // Lane: row col, dimensions 32 n + 8 i + 4 half + 0 .. 3.
    if (active) {
      l = pair_sum(l);
      if (whole && plan.whole_rows == 0) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        if (row < w.rows) {
          if (a.lse && half == 0)
            a.lse[qr.at] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
          uint16_t *const dst = a.out + qr.at * D + 4 * half;
#pragma unroll
          for (int n = 0; n < kDb; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<u32x2 *>(dst + 32 * n + 8 * i) =
                  u32x2{pack_bf16x2(o[n][4 * i] * inv, o[n][4 * i + 1] * inv),
                        pack_bf16x2(o[n][4 * i + 2] * inv, o[n][4 * i + 3] * inv)};
        }
      } else if (row < w.rows) {
        // A run's first piece, or a later one; or, whole, the row's own place.
        const int64_t at = whole ? (w.kind == kSharedPrefix ? int64_t(a.T) * a.q_heads : 0) + qr.at
                                 : list.part_row(work.run, flags & 4, row);
        if (half == 0) plan.ml[at] = float2{m, l};
        float *const dst = plan.o + at * D + 4 * half;
#pragma unroll
        for (int n = 0; n < kDb; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<f32x4 *>(dst + 32 * n + 8 * i) =
                f32x4{o[n][4 * i], o[n][4 * i + 1], o[n][4 * i + 2], o[n][4 * i + 3]};
      }
    }
  }
}

template <int kDb, bool kMx, int kW, bool kRules>
hipError_t launch(const TileAttention &a, const TilePlan &plan, hipStream_t stream) {
  const void *kernel = reinterpret_cast<const void *>(&tile_wide_kernel<kDb, kMx, kW, kRules>);
  constexpr int kLds = 2 * Stage<kDb>::kBytes;
  const hipError_t e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((tile_wide_kernel<kDb, kMx, kW, kRules>), dim3(plan.list[0].runs), dim3(64 * kW), kLds, stream,
                     a, plan);
  return hipGetLastError();
}

template <int kDb, bool kMx>
hipError_t by_waves(const TileAttention &a, const TilePlan &plan, hipStream_t stream) {
  const bool rules = a.rules.cap > 0.0f || a.rules.slopes;
  if constexpr (kDb <= 4) {
    if (plan.list[0].block_rows == 8 * kRows)
      return rules ? launch<kDb, kMx, 8, true>(a, plan, stream) : launch<kDb, kMx, 8, false>(a, plan, stream);
  }
  return rules ? launch<kDb, kMx, 4, true>(a, plan, stream) : launch<kDb, kMx, 4, false>(a, plan, stream);
}

template <int kDb>
hipError_t by_format(const TileAttention &a, const TilePlan &plan, hipStream_t stream) {
  return a.cache.k_scales ? by_waves<kDb, true>(a, plan, stream) : by_waves<kDb, false>(a, plan, stream);
}

}  // namespace

int tile_wide_rows(int32_t head_dim, int64_t rows) { return rows > 4 * kRows && head_dim <= 128 ? 8 * kRows : 4 * kRows; }

hipError_t launch_tile_wide(const TileAttention &a, const TilePlan &plan, hipStream_t stream) {
  switch (a.cache.head_dim / 32) {
    case 1: return by_format<1>(a, plan, stream);
    case 2: return by_format<2>(a, plan, stream);
    case 3: return by_format<3>(a, plan, stream);
    case 4: return by_format<4>(a, plan, stream);
    case 5: return by_format<5>(a, plan, stream);
    case 6: return by_format<6>(a, plan, stream);
    case 7: return by_format<7>(a, plan, stream);
    default: return by_format<8>(a, plan, stream);
  }
}

}  // namespace engram
