// Attention of one new token per sequence over the paged cache.
//
//   out = sum_p e^(scale q.k_p - m) v_p / sum_p e^(scale q.k_p - m),
//   m = max_p scale q.k_p,  lse = m + log sum_p e^(scale q.k_p - m)
//
// Bound by reading the seen keys and values once: 64 ragged streams of up to
// 4096 places in 8 bits, 333 MB, take 69 us (4.8 TB/s) and 5 us to join; one of
// 131072 places in bf16, 537 MB, 93 us (5.8 TB/s) and 5.  One of 500 places takes
// 9.3 us, by latency alone.  The query heads of one key-value head share a
// workgroup (up to 32 of them), so that each key and value is read once.  The
// work of all sequences is cut into equal runs, a workgroup each (chunks of the
// longest length instead: 76 to 92 us for the 64 streams); what of a run is not
// a whole sequence's goes to a second kernel, which joins the parts in order.
//
// A wave takes 32 places at a time, straight from memory into registers:
//  - S^T = K Q^T by v_mfma_f32_16x16x32_bf16: the lane l of a 16-place tile
//    holds 16 bytes of place l % 16 per step, in any order of the dimensions
//    as long as q's is the same;
//  - a lane then has 8 scores of query head l % 16, so the running maximum
//    takes two exchanges between lanes and the sums none before the end;
//  - O^T = V^T P^T: those 8 scores are the lane's B operand as they stand
//    (places 4 g .. 4 g + 3 of either tile, g = l / 16), and its A operand
//    are the same 8 places' values of dimension base + w (l % 16) + n, for
//    n = 0 .. w - 1 in turn: a lane reads w neighbouring dimensions of each
//    of its 8 places, and an 8 x w transpose between its own registers (one
//    v_perm for two values) is all that V needs;
//  - a weight goes through the matrix cores as the sum of two bf16 values, 2^-15
//    off at most.  Weights in one bf16 value add 6 to 8 % to the error that the
//    result's own rounding makes (1.66e-3 of its norm) and save little: the 64
//    streams take 70.9 instead of 71.9 us, one of 500 places 8.9 instead of 9.3,
//    64 streams of 32 query heads a key-value head 28.2 instead of 29.4.
// No lane waits for another in the loop: waves run apart, and the next 32
// places are requested as soon as a register is free.  The next sequence's
// first places are requested before this one's results are joined in LDS.
#include <algorithm>

#include "attention_common.hpp"
#include "attention_lds.hpp"

namespace engram {
namespace {

using namespace attn;

constexpr int kTile = 32;                  // places a wave takes at a time
constexpr int kUnit = kTile * kW;          // places the work is dealt out by
constexpr int kMaxChunk = 4096;            // places whose pages are held in LDS at a time
constexpr int kMinPage = 8;

// ---------------------------------------------------------------- the plan

// The host does not know the lengths, so the workgroups deal out the work
// themselves: the units of all (sequence, key-value head) pairs, in that order,
// are cut into as many equal runs as there are workgroups.  A run's pieces of
// pairs that it does not hold whole (two at most: its first and its last) go
// to the workspace, and join_kernel adds a pair's pieces in order.  Pairs of
// few units (direct_units) take one workgroup each, and there is nothing to join.
// 256 workgroups, one a CU: 512 read no faster, and have twice the pieces (one
// stream of 131072 places 98 us, with 512 of them 101, with 768 106).
constexpr int64_t kBlocks = 256;

// Up to 4 units (512 places) the join costs more than it saves (one stream of
// 300 places: 8.4 us against 10.7 us; of 1000: 13.9 against 10.5 us).  Where the
// pairs fill the CUs on their own, up to 16 units and some 540 KB a pair, what a
// workgroup streams in the time that dealing out and joining take (64 streams
// of up to 1000 places in bf16: 36.7 against 43.2 us; 32 of up to 2000 in 8 bits
// 23.6 against 29.4, in bf16, 40 of them, 53.5 against 46.3 us).
inline int64_t direct_units(int64_t pairs, int64_t unit_bytes) {
  return pairs < kBlocks ? 4 : std::max<int64_t>(4, std::min<int64_t>(16, 544 * 1024 / unit_bytes));
}

inline int64_t ceil_div(int64_t x, int64_t by) { return (x + by - 1) / by; }

struct Plan {
  int64_t pairs, units, blocks;            // units: of one pair at most
  int head_blocks;
  bool direct;
};

// span: the places seen at most, from a multiple of kTile on.  row_bytes: of a
// key or a value.
Plan plan_for(int n_seqs, int q_heads, int kv_heads, int64_t span, int64_t row_bytes) {
  Plan p{};
  p.head_blocks = int(ceil_div(q_heads / kv_heads, kHeadBlock));
  p.pairs = int64_t(n_seqs) * kv_heads * p.head_blocks;
  p.units = std::max<int64_t>(1, ceil_div(span, kUnit));
  p.direct = p.units <= direct_units(p.pairs, 2 * kUnit * row_bytes);
  p.blocks = p.direct ? p.pairs : std::min(kBlocks, p.pairs * p.units);
  return p;
}

// The workspace: of each run two pieces [heads of a block][head_dim] and their
// (m, sum), then the units before each sequence and their number in a run.
struct Split {
  float *o;
  float2 *ml;
  int32_t *before;         // [n_seqs + 1], [n_seqs + 1] units of a run
  int32_t blocks, head_blocks, block_heads;
  bool direct;
};

// The places of a sequence that are seen, from its start rounded down to a tile.
struct Seen {
  int start, len, base, units;
};
__device__ __forceinline__ Seen seen_of(const PagedAttention &a, int64_t s) {
  // Constant while the kernel runs: a uniform s is a scalar load, which does not
  // wait for the vector loads in flight.
  typedef const int32_t __attribute__((address_space(4))) *Constant;
  const int64_t room = int64_t(a.table_width) << a.cache.page_shift;
  const int stated = reinterpret_cast<Constant>(reinterpret_cast<uintptr_t>(a.lens))[s];
  const int len = int(min(int64_t(min(max(stated, 0), a.max_len)), room));
  const int start = a.window > 0 ? max(0, len - a.window) : 0;
  const int base = start / kTile * kTile;
  return {start, len, base, int((int64_t(len) - base + kUnit - 1) / kUnit)};
}

// Where a run starts: this workgroup's first unit is unit `local` of the
// sequence s's pairs.  Writes the workspace's `before` too (workgroup 0).
struct Run {
  int s, local, left;
};
__device__ __forceinline__ Run run_of(const PagedAttention &a, const Split &sp, int pairs) {
  __shared__ int wave_lds[kW], run_lds[2];
  const int per_thread = (a.n_seqs + 64 * kW - 1) / (64 * kW);
  const int s0 = threadIdx.x * per_thread, s1 = min(a.n_seqs, s0 + per_thread);
  int mine = 0;
  for (int s = s0; s < s1; ++s) mine += seen_of(a, s).units * pairs;
  int upto = mine;
#pragma unroll
  for (int x = 1; x < 64; x *= 2) {
    const int y = __shfl_up(upto, x);
    if (int(threadIdx.x & 63) >= x) upto += y;
  }
  if ((threadIdx.x & 63) == 63) wave_lds[threadIdx.x >> 6] = upto;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < kW; ++w) {
    if (w == int(threadIdx.x >> 6)) upto += total;
    total += wave_lds[w];
  }
  int before = upto - mine;
  const int per = max(1, (total + sp.blocks - 1) / sp.blocks);
  const int64_t u0 = int64_t(blockIdx.x) * per;
  if (u0 >= before && u0 < upto) {
    int s = s0, local = int(u0) - before;
    for (;; ++s) {
      const int n = seen_of(a, s).units * pairs;
      if (local < n) break;
      local -= n;
    }
    run_lds[0] = s, run_lds[1] = local;
  }
  if (blockIdx.x == 0) {
    for (int s = s0; s < s1; ++s) {
      sp.before[s] = before;
      before += seen_of(a, s).units * pairs;
    }
    if (threadIdx.x == 0) sp.before[a.n_seqs] = total, sp.before[a.n_seqs + 1] = per;
  }
  __syncthreads();
  if (u0 >= total) return {0, 0, 0};
  return {run_lds[0], run_lds[1], int(min(int64_t(per), total - u0))};
}

// What a workgroup works at: places c0 .. c1 - 1, a stretch of a piece (the
// units of a pair that its run holds), whose pages LDS has room for.
struct Work {
  Seen seen;
  int s, pair, kvh, hb, index;             // index: which piece of the run
  int end, c0, c1, tiles, page0, pages;
  bool whole;                              // the piece is its whole pair
};

template <int kDb, bool kMx, int kHt>
__global__ __launch_bounds__(64 * kW, kDb * kHt > 6 ? 1 : 2) void paged_attention_kernel(
    PagedAttention a, Split sp) {
  constexpr int D = 32 * kDb, kRowBytes = kMx ? D : 2 * D, kAcc = D / 16;
  constexpr int kPageRegs = (kMaxChunk / kMinPage + 1 + 64 * kW - 1) / (64 * kW);
  using P = Pieces<kDb>;
  // Two of each: the next stretch's are written while this one's are in use.
  __shared__ int64_t page_lds[2][kMaxChunk / kMinPage + 1];   // a page's first row, or -1
  __shared__ int bad_lds[2][kW];
  __shared__ float2 ml_lds[2][kW][kHt][16];
  extern __shared__ f32x4 o_lds[];           // [1 or 2][kW][kAcc][4][heads of a tile]

  const CacheView &c = a.cache;
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = a.q_heads / c.kv_heads, pairs = c.kv_heads * sp.head_blocks;
  const int mask = (1 << c.page_shift) - 1;
  const float to_log2 = a.scale * kLog2e;

  Run run{int(blockIdx.x / pairs), 0, 1};
  if (!sp.direct) run = run_of(a, sp, pairs);
  run.s = __builtin_amdgcn_readfirstlane(run.s);
  run.local = __builtin_amdgcn_readfirstlane(run.local);
  run.left = __builtin_amdgcn_readfirstlane(run.left);

  auto next_work = [&](Work &w) {
    if (w.c1 < w.end) {
      w.c0 = w.c1;
    } else {
      for (;; ++run.s) {
        if (run.left <= 0) return false;
        w.seen = seen_of(a, run.s);
        if (sp.direct || w.seen.units > 0) break;
      }
      w.s = run.s;
      w.pair = sp.direct ? int(blockIdx.x % pairs) : run.local / w.seen.units;
      const int unit = sp.direct ? 0 : run.local - w.pair * w.seen.units;
      const int count = sp.direct ? w.seen.units : min(w.seen.units - unit, run.left);
      run.left -= sp.direct ? 1 : count;
      run.local += count;
      if (run.local == w.seen.units * pairs) ++run.s, run.local = 0;
      w.whole = count == w.seen.units;
      ++w.index;
      w.kvh = w.pair / sp.head_blocks;
      w.hb = w.pair - w.kvh * sp.head_blocks;
      w.c0 = w.seen.base + unit * kUnit;
      w.end = int(min(int64_t(w.seen.len), int64_t(w.c0) + int64_t(count) * kUnit));
    }
    w.c1 = min(w.end, w.c0 + kMaxChunk);
    w.tiles = (w.c1 - w.c0 + kTile - 1) / kTile;
    w.page0 = w.c0 >> c.page_shift;
    w.pages = ((w.c0 + max(1, w.tiles) * kTile - 1) >> c.page_shift) - w.page0 + 1;
    return true;
  };

  // The pages of a stretch: requested into registers, later put in LDS.
  auto shown_page = [&](const Work &w, int e) {
    const int first = (w.page0 + e) << c.page_shift;
    return e < w.pages && first < w.c1 && first + mask >= w.seen.start;
  };
  auto ask_pages = [&](const Work &w, int(&page)[kPageRegs]) {
#pragma unroll
    for (int k = 0; k < kPageRegs; ++k) {
      const int e = threadIdx.x + k * 64 * kW;
      page[k] = -1;
      if (shown_page(w, e)) page[k] = a.table[int64_t(w.s) * a.table_width + w.page0 + e];
    }
  };
  auto put_pages = [&](const Work &w, const int(&page)[kPageRegs], int buf) {
    bool bad = false;
#pragma unroll
    for (int k = 0; k < kPageRegs; ++k) {
      const int e = threadIdx.x + k * 64 * kW;
      if (e >= w.pages) break;
      const bool in = page[k] >= 0 && page[k] < c.pages;
      bad |= !in && shown_page(w, e);
      page_lds[buf][e] = in ? (int64_t(page[k]) * c.kv_heads + w.kvh) << c.page_shift : -1;
    }
    if (bad && w.pair == 0 && a.bad_pages) atomicAdd(a.bad_pages, 1);
    const bool any = __any(bad);
    if (lane == 0) bad_lds[buf][wave] = any;
  };
  // LDS written by all, read by all; loads stay in flight.
  auto barrier = [&] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);            // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  auto bad_of = [&](int buf) {
    int any = 0;
#pragma unroll
    for (int x = 0; x < kW; ++x) any |= bad_lds[buf][x];
    return __builtin_amdgcn_readfirstlane(any) != 0;
  };

  // Query heads as B operands: lane l holds 8 dimensions of head l % 16 a step.
  // In the 8-bit format a lane's 16 bytes of K are two steps.
  bf16x8 q[kHt][kDb];
  auto heads_of = [&](const Work &w) {             // kHt = 1 only for up to 16
    return min(16 * kHt, group - w.hb * kHeadBlock);
  };
  auto row0_of = [&](const Work &w) {
    return int64_t(w.s) * a.q_heads + w.kvh * group + w.hb * kHeadBlock;
  };
  auto load_q = [&](const Work &w) {
    const int heads = heads_of(w);
    const uint16_t *src = a.q + row0_of(w) * D;
#pragma unroll
    for (int t = 0; t < kHt; ++t)
#pragma unroll
      for (int kk = 0; kk < kDb; ++kk) {
        const int d = kMx && (kk | 1) < kDb ? 64 * (kk / 2) + 16 * g + 8 * (kk & 1) : 32 * kk + 8 * g;
        // Columns past the last head repeat it; nothing reads their results.
        q[t][kk] = __builtin_bit_cast(
            bf16x8, *reinterpret_cast<const u32x4 *>(src + min(16 * t + col, heads - 1) * D + d));
      }
  };

  Held<kDb, kMx> held;
  auto row_of = [&](const Work &w, int buf, int p) {
    const int64_t r = page_lds[buf][(p >> c.page_shift) - w.page0];
    return (r < 0 ? 0 : r) + (p & mask);       // a page that is not seen: rows of page 0 instead
  };
  auto load_k = [&](const Work &w, int buf, int tile) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t row = row_of(w, buf, w.c0 + kTile * tile + 16 * u + col);
      const uint8_t *src = static_cast<const uint8_t *>(c.k) + row * kRowBytes;
      if constexpr (!kMx) {
#pragma unroll
        for (int kk = 0; kk < kDb; ++kk) load_bytes<16>(&held.k[u][4 * kk], src + 64 * kk + 16 * g);
      } else {
        const uint8_t *sc = c.k_scales + row * kDb;
#pragma unroll
        for (int j = 0; j < kDb / 2; ++j) {
          load_bytes<16>(&held.k[u][4 * j], src + 64 * j + 16 * g);
          held.ks[u][j] = sc[2 * j + (g >> 1)];
        }
        if constexpr (kDb % 2) {
          load_bytes<8>(&held.k[u][2 * (kDb - 1)], src + 32 * (kDb - 1) + 8 * g);
          held.ks[u][kDb / 2] = sc[kDb - 1];
        }
      }
    }
  };
  auto load_v = [&](const Work &w, int buf, int tile) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t row = row_of(w, buf, w.c0 + kTile * tile + 16 * u + 4 * g);
      const uint8_t *src = static_cast<const uint8_t *>(c.v) + row * kRowBytes;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        each_piece<P::kN>([&](auto piece) {
          constexpr int wd = P::width(piece.value), first = P::base(piece.value);
          if constexpr (kMx) {
            load_bytes<wd>(&held.v[4 * u + j][first / 64], src + j * kRowBytes + first + wd * col);
            held.vs[4 * u + j][piece.value] = c.v_scales[(row + j) * kDb + (first + wd * col) / 32];
          } else {
            load_bytes<2 * wd>(&held.v[4 * u + j][first / 32],
                              src + j * kRowBytes + 2 * (first + wd * col));
          }
        });
      }
    }
  };

  float m[kHt], l[kHt];
  f32x4 o[kHt][kAcc];
  auto reset = [&] {
#pragma unroll
    for (int t = 0; t < kHt; ++t) {
      m[t] = -INFINITY, l[t] = 0.0f;
#pragma unroll
      for (int n = 0; n < kAcc; ++n) o[t][n] = f32x4{};
    }
  };
  reset();

  // A piece's parts, the waves' results, to LDS; then joined by all threads, two
  // neighbouring dimensions of four places in O^T each, in wave order.
  auto part_lds = [&](const Work &w) {
    return o_lds + attn::part_begin(kAcc, sp.block_heads, w.index);
  };
  auto give = [&](const Work &w, int t, int here) {
    f32x4 *const ob = part_lds(w) + wave * kAcc * 4 * here;
    if (col < here) {
#pragma unroll
      for (int n = 0; n < kAcc; ++n) ob[n * 4 * here + g * here + col] = o[t][n];
    }
  };
  auto join = [&](const Work &w) {
    const int heads = heads_of(w);
    const f32x4 *const ob = part_lds(w);
#pragma unroll
    for (int t = 0; t < kHt; ++t) {
      const int here = min(16, heads - 16 * t);
      if (here <= 0) break;
      if (t > 0) {
        barrier();
        give(w, t, here);
        barrier();
      }
      for (int k = threadIdx.x; k < kAcc / 2 * 4 * here; k += 64 * kW) {
        const int n = k / (4 * here) * 2, lane_of = k - n * 2 * here;      // (g, column) of the parts
        const int gg = lane_of / here, head = lane_of - gg * here;
        float top = -INFINITY, sum = 0.0f;
        float2 ml[kW];
        f32x4 part0[kW], part1[kW];
#pragma unroll
        for (int x = 0; x < kW; ++x) {
          ml[x] = ml_lds[w.index & 1][x][t][head];
          part0[x] = ob[(x * kAcc + n) * 4 * here + lane_of];
          part1[x] = ob[(x * kAcc + n + 1) * 4 * here + lane_of];
          top = fmaxf(top, ml[x].x);
        }
        const float ms = top == -INFINITY ? 0.0f : top;
        f32x4 a0{}, a1{};
#pragma unroll
        for (int x = 0; x < kW; ++x) {
          const float keep = __builtin_amdgcn_exp2f(ml[x].x - ms);
          sum += ml[x].y * keep;
          a0 += part0[x] * keep;
          a1 += part1[x] * keep;
        }
        const int64_t row = row0_of(w) + 16 * t + head;
        // A run's first piece, or a later one (the run's last) that it does not hold whole.
        const int64_t part = (2 * int64_t(blockIdx.x) + (w.index > 0)) * sp.block_heads + 16 * t + head;
        const float inv = !w.whole ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
        if (k < here) {
          if (!w.whole) sp.ml[part] = float2{top, sum};
          else if (a.lse) a.lse[row] = sum == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
        }
        int first = 0, wd = P::width(0);
        each_piece<P::kN>([&](auto piece) {
          if (16 * n >= P::base(piece.value)) first = P::base(piece.value), wd = P::width(piece.value);
        });
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int d = first + wd * (4 * gg + r) + n - first / 16;
          if (w.whole) *reinterpret_cast<uint32_t *>(a.out + row * D + d) = pack_bf16x2(a0[r] * inv, a1[r] * inv);
          else *reinterpret_cast<float2 *>(sp.o + part * D + d) = float2{a0[r], a1[r]};
        }
      }
    }
    reset();
    if (!attn::two_buffers(kAcc, sp.block_heads)) barrier();
  };

  Work w{};
  w.index = -1;
  if (!next_work(w)) return;
  int page[kPageRegs];
  ask_pages(w, page);
  put_pages(w, page, 0);
  barrier();
  // A stretch's first loads; then, while they fly, the join of the piece before
  // it and the pages of the one after it.  Loads are issued without a condition
  // (a stretch's last ones for nothing, from the cache): a wave then waits for
  // no more of them than it needs.
  Work before{};
  bool join_before = false;
  for (int buf = 0;; buf ^= 1) {
    load_q(w);
    __builtin_amdgcn_sched_barrier(0);
    load_k(w, buf, max(0, min(wave, w.tiles - 1)));
    __builtin_amdgcn_sched_barrier(0);
    load_v(w, buf, max(0, min(wave, w.tiles - 1)));
    __builtin_amdgcn_sched_barrier(0);
    if (join_before) join(before);
    const bool any_bad = bad_of(buf);
    Work nw = w;
    const bool more = next_work(nw);
    if (more) ask_pages(nw, page);
    // q waited for here, once, and not in the loop, which would do so each time.
#pragma unroll
    for (int t = 0; t < kHt; ++t)
#pragma unroll
      for (int kk = 0; kk < kDb; ++kk) asm volatile("" : "+v"(q[t][kk]));

    if (wave < w.tiles) {
      int tile = wave;
      do {
        const int next = min(tile + kW, w.tiles - 1);
        const int p0 = w.c0 + kTile * tile;
        f32x4 z[kHt][2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
          for (int t = 0; t < kHt; ++t) z[t][u] = f32x4{};
#pragma unroll
          for (int kk = 0; kk < kDb; ++kk) {
            bf16x8 f;
            if constexpr (kMx) {
              const uint32_t *w = &held.k[u][2 * kk];
              const float sc = __uint_as_float(held.ks[u][kk / 2] << 23);
              f = as_frag(mx_pair(w[0], sc, false), mx_pair(w[0], sc, true), mx_pair(w[1], sc, false),
                          mx_pair(w[1], sc, true));
            } else {
              const uint32_t *w = &held.k[u][4 * kk];
              f = as_frag(w[0], w[1], w[2], w[3]);
            }
#pragma unroll
            for (int t = 0; t < kHt; ++t)
              z[t][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, q[t][kk], z[t][u], 0, 0, 0);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        load_k(w, buf, next);
        __builtin_amdgcn_sched_barrier(0);

        // Bits 4 u + r: place 16 u + 4 g + r of the tile is seen.  The values of
        // others, which may be anything, count as 0 (times a scale that is finite).
        const bool whole = !any_bad && p0 >= w.seen.start && p0 + kTile <= w.seen.len;
        uint32_t shown = 0xFF;
        if (!whole) {
          shown = 0;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int p = p0 + 16 * u + 4 * g;
            const bool page = page_lds[buf][(p >> c.page_shift) - w.page0] >= 0;
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (page && p + r >= w.seen.start && p + r < w.seen.len) shown |= 1u << (4 * u + r);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < int(sizeof(held.v[0]) / 4); ++i)
              held.v[j][i] = shown >> j & 1 ? held.v[j][i] : 0;
        }

        bf16x8 wt[kHt], wt_rest[kHt];               // the weights, as B operands
#pragma unroll
        for (int t = 0; t < kHt; ++t) {
          float e[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) e[j] = z[t][j / 4][j % 4] * to_log2;
          if (!whole) {
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = shown >> j & 1 ? e[j] : -INFINITY;
          }
          float top = e[0];
#pragma unroll
          for (int j = 1; j < 8; ++j) top = fmaxf(top, e[j]);
          top = column_max(top);
          if (__any(top > m[t])) {                 // rarely after the first tiles
            const float mn = fmaxf(m[t], top);
            const float keep = mn == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m[t] - mn);
            m[t] = mn;
            l[t] *= keep;
#pragma unroll
            for (int n = 0; n < kAcc; ++n) o[t][n] *= keep;
          }
          const float ms = m[t] == -INFINITY ? 0.0f : m[t];
          float sum = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            e[j] = __builtin_amdgcn_exp2f(e[j] - ms);
            sum += e[j];
          }
          l[t] += sum;
          // For the matrix cores each is the sum of two bf16 values: its upper 16 bits,
          // and what they leave, below 2^-7 of it, rounded: 2^-15 off.  The sum is of
          // the fp32 ones.
          uint32_t top16[4], rest[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t a = __float_as_uint(e[2 * j]), b = __float_as_uint(e[2 * j + 1]);
            top16[j] = __builtin_amdgcn_perm(b, a, 0x07060302u);
            rest[j] = pack_bf16x2(e[2 * j] - __uint_as_float(a & 0xFFFF0000u),
                                  e[2 * j + 1] - __uint_as_float(b & 0xFFFF0000u));
          }
          wt[t] = as_frag(top16[0], top16[1], top16[2], top16[3]);
          wt_rest[t] = as_frag(rest[0], rest[1], rest[2], rest[3]);
        }

        each_piece<P::kN>([&](auto piece) {
          constexpr int wd = P::width(piece.value), first = P::base(piece.value);
#pragma unroll
          for (int i = 0; i < wd / 2; ++i) {
            uint32_t x[8];                   // dimensions 2 i, 2 i + 1 of the lane's 8 places
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if constexpr (kMx)
                x[j] = mx_pair(held.v[j][first / 64 + i / 2],
                               __uint_as_float(min(held.vs[j][piece.value], 254u) << 23), i & 1);
              else
                x[j] = held.v[j][first / 32 + i];
            }
            const bf16x8 even = as_frag(__builtin_amdgcn_perm(x[1], x[0], 0x05040100u),
                                        __builtin_amdgcn_perm(x[3], x[2], 0x05040100u),
                                        __builtin_amdgcn_perm(x[5], x[4], 0x05040100u),
                                        __builtin_amdgcn_perm(x[7], x[6], 0x05040100u));
            const bf16x8 odd = as_frag(__builtin_amdgcn_perm(x[1], x[0], 0x07060302u),
                                       __builtin_amdgcn_perm(x[3], x[2], 0x07060302u),
                                       __builtin_amdgcn_perm(x[5], x[4], 0x07060302u),
                                       __builtin_amdgcn_perm(x[7], x[6], 0x07060302u));
            const int n = first / 16 + 2 * i;
#pragma unroll
            for (int t = 0; t < kHt; ++t) {
              o[t][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(even, wt[t], o[t][n], 0, 0, 0);
              o[t][n + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(odd, wt[t], o[t][n + 1], 0, 0, 0);
              o[t][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(even, wt_rest[t], o[t][n], 0, 0, 0);
              o[t][n + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(odd, wt_rest[t], o[t][n + 1], 0, 0, 0);
            }
          }
        });
        __builtin_amdgcn_sched_barrier(0);
        load_v(w, buf, next);
        __builtin_amdgcn_sched_barrier(0);
      } while ((tile += kW) < w.tiles);
    }

    if (w.c1 == w.end) {                           // the end of a piece
#pragma unroll
      for (int t = 0; t < kHt; ++t) {
        l[t] = column_sum(l[t]);
        if (g == 0) ml_lds[w.index & 1][wave][t][col] = float2{m[t], l[t]};
      }
      give(w, 0, min(16, heads_of(w)));
    }
    if (more) put_pages(nw, page, buf ^ 1);
    barrier();
    if (!more) break;
    join_before = w.c1 == w.end;
    before = w;
    w = nw;
  }
  join(w);
}

// A pair's pieces to its result, in order: one workgroup per (sequence, query
// head), D / 4 lanes a piece.
constexpr int kJoinThreads = 64;
__global__ __launch_bounds__(kJoinThreads) void join_kernel(PagedAttention a, Split sp) {
  __shared__ f32x4 part_lds[kJoinThreads];
  __shared__ float2 ml_lds[kJoinThreads / 8];
  const int D = a.cache.head_dim, lanes = D / 4;
  const int64_t row = blockIdx.x;
  const int s = int(row / a.q_heads), h = int(row - int64_t(s) * a.q_heads);
  const int group = a.q_heads / a.cache.kv_heads, kvh = h / group, in_group = h - kvh * group;
  const int hb = in_group / kHeadBlock, pair = kvh * sp.head_blocks + hb;
  const int first = sp.before[s], per = sp.before[a.n_seqs + 1];
  const int units = (sp.before[s + 1] - first) / (a.cache.kv_heads * sp.head_blocks);
  const int u0 = first + pair * units, u1 = u0 + units;
  const int r0 = u0 / per;
  const int parts = units == 0 ? 0 : (u1 - 1) / per - r0 + 1;
  if (parts == 1) return;                          // its run has written the result
  // The first run holds the pair's beginning: as its first piece, or its last.
  const int64_t at0 = int64_t(in_group - hb * kHeadBlock);
  // Each group of D / 4 lanes takes every rows-th piece; the groups' results are
  // joined in their order.
  const int rows = kJoinThreads / lanes, mine = threadIdx.x / lanes, at = threadIdx.x % lanes;
  f32x4 o{};
  float m = -INFINITY, l = 0.0f;
  if (mine < rows) {
#pragma unroll 4
    for (int i = mine; i < parts; i += rows) {
      const int64_t part = (2 * int64_t(r0 + i) + (i == 0 && int64_t(r0) * per < u0)) * sp.block_heads + at0;
      const float2 ml = sp.ml[part];
      const f32x4 v = reinterpret_cast<const f32x4 *>(sp.o)[part * lanes + at];
      const float top = fmaxf(m, ml.x), ms = top == -INFINITY ? 0.0f : top;
      const float keep = __builtin_amdgcn_exp2f(m - ms), add = __builtin_amdgcn_exp2f(ml.x - ms);
      o = o * keep + v * add;
      l = l * keep + ml.y * add;
      m = top;
    }
    part_lds[threadIdx.x] = o;
    if (at == 0) ml_lds[mine] = float2{m, l};
  }
  __syncthreads();
  if (mine != 0) return;
  float top = m;
  for (int w = 1; w < rows; ++w) top = fmaxf(top, ml_lds[w].x);
  const float ms = top == -INFINITY ? 0.0f : top;
  float keep = __builtin_amdgcn_exp2f(m - ms), sum = l * keep;
  o *= keep;
  for (int w = 1; w < rows; ++w) {
    const float2 ml = ml_lds[w];
    keep = __builtin_amdgcn_exp2f(ml.x - ms);
    sum += ml.y * keep;
    o += part_lds[w * lanes + at] * keep;
  }
  if (at == 0 && a.lse)
    a.lse[row] = sum == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  reinterpret_cast<u32x2 *>(a.out + row * D)[at] =
      u32x2{pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv)};
}

template <int kDb, bool kMx, int kHt>
hipError_t launch(const PagedAttention &a, const Split &sp, hipStream_t stream) {
  const void *kernel = reinterpret_cast<const void *>(&paged_attention_kernel<kDb, kMx, kHt>);
  const unsigned lds = attn::result_bytes(2 * kDb, sp.block_heads);
  if (lds > attn::kResultLds) {              // more than a launch may have without asking
    const hipError_t e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, int(lds));
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((paged_attention_kernel<kDb, kMx, kHt>), dim3(sp.blocks), dim3(64 * kW),
                     lds, stream, a, sp);
  return hipGetLastError();
}

template <int kDb, bool kMx>
hipError_t by_heads(const PagedAttention &a, const Split &sp, hipStream_t stream) {
  return sp.block_heads > 16 ? launch<kDb, kMx, 2>(a, sp, stream) : launch<kDb, kMx, 1>(a, sp, stream);
}

template <int kDb>
hipError_t by_format(const PagedAttention &a, const Split &sp, hipStream_t stream) {
  return a.cache.k_scales ? by_heads<kDb, true>(a, sp, stream) : by_heads<kDb, false>(a, sp, stream);
}

inline int block_heads(int q_heads, int kv_heads) { return std::min(kHeadBlock, q_heads / kv_heads); }

}  // namespace

int64_t paged_attention_units(int32_t n_seqs, int32_t q_heads, int32_t kv_heads, int32_t max_len) {
  const Plan p = plan_for(n_seqs, q_heads, kv_heads, max_len, 1);
  return p.pairs * p.units;
}

int64_t paged_attention_workspace(int32_t n_seqs, int32_t q_heads, int32_t kv_heads,
                                  int32_t head_dim, int32_t max_len) {
  // As for bf16, without a window: other calls take no more workgroups.
  const Plan p = plan_for(n_seqs, q_heads, kv_heads, max_len, 2 * head_dim);
  if (p.direct) return 0;
  const int64_t parts = 2 * p.blocks * block_heads(q_heads, kv_heads);
  return (parts * (head_dim + 2) + n_seqs + 2) * int64_t(sizeof(float));
}

hipError_t launch_paged_attention(const PagedAttention &a, hipStream_t stream) {
  const int hkv = a.cache.kv_heads, D = a.cache.head_dim;
  const int64_t row_bytes = a.cache.k_scales ? D + D / 32 : 2 * D;
  const int64_t span = a.window > 0 ? std::min<int64_t>(a.max_len, int64_t(a.window) + kTile - 1) : a.max_len;
  const Plan p = plan_for(a.n_seqs, a.q_heads, hkv, span, row_bytes);
  Split sp{};
  sp.blocks = int32_t(p.blocks);
  sp.head_blocks = p.head_blocks;
  sp.block_heads = block_heads(a.q_heads, hkv);
  sp.direct = p.direct;
  if (!p.direct) {
    const int64_t parts = 2 * p.blocks * sp.block_heads;
    sp.o = static_cast<float *>(a.workspace);
    sp.ml = reinterpret_cast<float2 *>(sp.o + parts * D);
    sp.before = reinterpret_cast<int32_t *>(sp.ml + parts);
  }
  hipError_t err;
  switch (D / 32) {
    case 1: err = by_format<1>(a, sp, stream); break;
    case 2: err = by_format<2>(a, sp, stream); break;
    case 3: err = by_format<3>(a, sp, stream); break;
    case 4: err = by_format<4>(a, sp, stream); break;
    case 5: err = by_format<5>(a, sp, stream); break;
    case 6: err = by_format<6>(a, sp, stream); break;
    case 7: err = by_format<7>(a, sp, stream); break;
    default: err = by_format<8>(a, sp, stream);
  }
  if (err != hipSuccess || p.direct) return err;
  hipLaunchKernelGGL(join_kernel, dim3(unsigned(int64_t(a.n_seqs) * a.q_heads)),
                     dim3(kJoinThreads), 0, stream, a, sp);
  return hipGetLastError();
}

}  // namespace engram
