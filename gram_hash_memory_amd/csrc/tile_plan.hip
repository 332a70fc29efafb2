// The plan of attention of several query rows a key-value head, and the join of its
// parts.
//
// The host knows neither the tokens of a sequence nor its length, so a kernel of one
// workgroup a list writes the blocks down.  Where there are enough blocks, the
// workgroups of the lists' kernels take whole ones, those of most tiles first; where
// there are too few to fill the GPU, equal runs of all tiles, and a third kernel adds
// the parts of a block in order.  Which, the plan kernel decides.  It takes 7 us, a
// chain of dependent loads and scans (13 us for 64 blocks with documents, whose starts
// it reads); the join 5 us for a few blocks, 28 us for 256 rows of each of 256 runs
// (134 MB read), 13 us for 64 sequences behind a shared prefix.
#include <algorithm>
#include <cstdint>

#include "attention_common.hpp"
#include "tile_plan.hpp"

namespace engram {
namespace {

using namespace attn;

constexpr int kPlanThreads = 1024;
// Contexts that are never cut, which saves the join's launch: two single tokens over up
// to 500 places 23.5 us (cut: 26.5), over up to 900 29.6 us (cut: 25.5).
constexpr int kWholePlaces = 512;
// What cutting costs, in tiles of the list.  Wide: three ragged prompts of capped scores
// 161 us whole and 241 us cut (which 4 would choose), 2048 tokens behind 14336 632 us
// whole and 690 us cut; from 8 to 40 nothing changes.  Narrow: 64 sequences behind a
// prefix 71 us with 3, 76 us with 1, the same with 12.
constexpr int kWideJoin = 8, kNarrowJoin = 3;

inline int64_t ceil_div(int64_t x, int64_t by) { return (x + by - 1) / by; }

// The sum of x over the threads before this one; *total: over all of them.
__device__ __forceinline__ int scan_before(int x, int *total) {
  __shared__ int wave_lds[kPlanThreads / 64];
  int upto = x;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int y = __shfl_up(upto, d);
    if (int(threadIdx.x & 63) >= d) upto += y;
  }
  __syncthreads();                           // wave_lds may still be read
  if ((threadIdx.x & 63) == 63) wave_lds[threadIdx.x >> 6] = upto;
  __syncthreads();
  int sum = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    if (w == int(threadIdx.x >> 6)) upto += sum;
    sum += wave_lds[w];
  }
  *total = sum;
  return upto - x;
}

__device__ __forceinline__ int max_all(int x) {
  __shared__ int wave_lds[kPlanThreads / 64];
#pragma unroll
  for (int d = 1; d < 64; d *= 2) x = max(x, __shfl_xor(x, d));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) wave_lds[threadIdx.x >> 6] = x;
  __syncthreads();
  x = wave_lds[0];
#pragma unroll
  for (int w = 1; w < kPlanThreads / 64; ++w) x = max(x, wave_lds[w]);
  return x;
}

// The new tokens of problem i: a chunk's sequences, or the groups and then the
// sequences over their own places.
__device__ __forceinline__ int tokens_of(const TileAttention &a, int i, int *token0) {
  if (a.prefix_table && i >= a.n_groups) {
    *token0 = i - a.n_groups;
    return 1;
  }
  const int begin = min(max(a.cu[i], 0), a.T), end = min(max(a.cu[i + 1], begin), a.T);
  *token0 = begin;
  return end - begin;
}

// Which list problem i belongs to.
__device__ __forceinline__ int list_of(const TileAttention &a, const TilePlan &plan, int i, int rows) {
  return (a.prefix_table && i >= a.n_groups) || rows <= plan.narrow_rows ? 1 : 0;
}

__global__ __launch_bounds__(kPlanThreads) void plan_kernel(TileAttention a, TilePlan plan) {
  const TileList list = blockIdx.x == 0 ? plan.list[0] : plan.list[1];
  if (list.max_blocks == 0) return;
  const int group = a.q_heads / a.cache.kv_heads, tid = threadIdx.x;
  const int problems = a.n_groups + a.n_seqs;
  int blocks = 0;
  for (int base = 0; base < problems; base += kPlanThreads) {
    const int i = base + tid;
    int token0, n = 0;
    if (i < problems) {
      const int rows = tokens_of(a, i, &token0) * group;
      if (list_of(a, plan, i, rows) == int(blockIdx.x)) n = (rows + list.block_rows - 1) / list.block_rows;
    }
    int total;
    const int at = blocks + scan_before(n, &total);
    blocks += total;
    if (i < problems) list.first_block[i] = at;
    for (int k = 0; k < n && at + k < list.max_blocks; ++k) {
      list.blocks[at + k].seq = i;
      list.blocks[at + k].row0 = k * list.block_rows;
    }
  }
  blocks = min(blocks, list.max_blocks);     // more only where cu does not rise
  __syncthreads();

  // With documents 8 neighbouring threads look at a block's tokens.
  const int threads = a.rules.doc_starts ? 8 : 1, sub = tid % threads;
  int units = 0, longest = 0;
  for (int base = 0; base < blocks; base += kPlanThreads / threads) {
    const int b = base + tid / threads;
    int mine = 0;
    TileBlock w{};
    if (b < blocks) {
      const int i = list.blocks[b].seq;
      w.row0 = list.blocks[b].row0;
      const int n = tokens_of(a, i, &w.token0);
      w.rows = min(list.block_rows, n * group - w.row0);
      w.group = -1;
      if (!a.prefix_table) {
        w.kind = kChunk, w.seq = i;
        w.len = length_of(a.lens[i], a.max_len, a.table_width, a.cache.page_shift);
        w.first = w.len - n;
        const int t0 = w.row0 / group, t1 = (w.row0 + w.rows - 1) / group;
        int a_lo = 0x7FFFFFFF, a_hi = 0, b_lo = 0x7FFFFFFF, b_hi = 0;
        w.all_hi = w.all_last = 0x7FFFFFFF;
        const int prefix = prefix_of(a.rules, i, w.len);
        auto add = [&](int t, int doc) {
          const RowSees r = row_sees(a.rules, prefix, doc, w.first + t, w.len);
          if (r.n > 0) b_lo = min(b_lo, r.lo), b_hi = max(b_hi, r.lo + r.n);
          if (r.m > 0) a_lo = min(a_lo, r.first), a_hi = max(a_hi, r.first + r.m);
          w.all_lo = max(w.all_lo, r.lo), w.all_hi = min(w.all_hi, r.lo + r.n);
          w.all_first = max(w.all_first, r.first), w.all_last = min(w.all_last, r.first + r.m);
        };
        if (threads > 1) {
          for (int t = t0 + sub; t <= t1; t += 64) {
            int doc[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) doc[x] = a.rules.doc_starts[w.token0 + min(t + 8 * x, t1)];
#pragma unroll
            for (int x = 0; x < 8; ++x) add(min(t + 8 * x, t1), doc[x]);
          }
#pragma unroll
          for (int x = 1; x < 8; x *= 2) {
            a_lo = min(a_lo, __shfl_xor(a_lo, x)), a_hi = max(a_hi, __shfl_xor(a_hi, x));
            b_lo = min(b_lo, __shfl_xor(b_lo, x)), b_hi = max(b_hi, __shfl_xor(b_hi, x));
            w.all_lo = max(w.all_lo, __shfl_xor(w.all_lo, x)), w.all_hi = min(w.all_hi, __shfl_xor(w.all_hi, x));
            w.all_first = max(w.all_first, __shfl_xor(w.all_first, x));
            w.all_last = min(w.all_last, __shfl_xor(w.all_last, x));
          }
        } else {                             // the first token with a place sees the first one, the last one the last
          add(t0, 0);
          add(min(t1, max(t0, -w.first)), 0);
          add(t1, 0);
        }
        if (a_hi > 0) w.a_lo = a_lo, w.a_hi = a_hi;
        if (b_hi > 0) w.b_lo = b_lo, w.b_hi = b_hi;
      } else if (i < a.n_groups) {
        w.kind = kSharedPrefix, w.seq = i;
        w.len = length_of(a.prefix_lens[i], a.max_prefix, a.prefix_width, a.cache.page_shift);
        w.b_hi = w.all_hi = w.len;
      } else {
        w.kind = kOwnPlaces, w.seq = i - a.n_groups;
        w.len = length_of(a.lens[w.seq], a.max_len, a.table_width, a.cache.page_shift);
        w.b_hi = w.all_hi = w.len;
        // The last group that does not begin behind the sequence.
        int lo = 0, hi = a.n_groups;
        while (lo < hi) {
          const int mid = (lo + hi) / 2;
          if (a.cu[mid] <= w.seq) lo = mid + 1;
          else hi = mid;
        }
        if (lo > 0) {
          int begin;
          const int members = tokens_of(a, lo - 1, &begin);
          if (w.seq >= begin && w.seq < begin + members) {
            w.group = lo - 1;
            w.group_row = (w.seq - begin) * group + w.row0;
          }
        }
      }
      w.a_tile = w.a_lo / list.tile;
      w.a_n = w.a_hi > 0 ? (w.a_hi - 1) / list.tile + 1 - w.a_tile : 0;
      w.b_tile = w.b_lo / list.tile;
      if (w.a_n > 0) w.b_tile = max(w.b_tile, w.a_tile + w.a_n);
      w.b_n = w.b_hi > 0 ? max(0, (w.b_hi - 1) / list.tile + 1 - w.b_tile) : 0;
      // Rows that see nothing need their zeros: a tile without places.
      if (w.kind != kOwnPlaces && w.tiles() == 0) w.b_n = 1;
      mine = sub == 0 ? w.tiles() : 0;
      longest = max(longest, mine);
    }
    int total;
    w.before = units + scan_before(mine, &total);
    units += total;
    if (b < blocks && sub == 0) list.blocks[b] = w;
  }
  longest = max_all(longest);
  // Whole blocks, those of most tiles first, take as long as their mean load and half
  // a block, or as the longest one; runs as long as their share, and the join.
  const int64_t pairs = int64_t(blocks) * a.cache.kv_heads;
  const int64_t total = int64_t(units) * a.cache.kv_heads;
  const int per = int(max(int64_t(1), (total + list.runs - 1) / list.runs));
  const int64_t queued = max(int64_t(longest), pairs > list.runs ? per + units / blocks / 2 : int64_t(0));
  const bool direct = !list.can_split || queued <= per + (blockIdx.x == 0 ? kWideJoin : kNarrowJoin);
  if (tid == 0) {
    *list.header = TileHeader{units, blocks, per, direct};
    *list.queue = 0;
  }
  if (!direct) return;
  // The order: a count of each number of tiles, then each block's place.
  __shared__ int bins[kPlanThreads];
  bins[tid] = 0;
  __syncthreads();
  auto bin_of = [&](int b) { return kPlanThreads - 1 - min(kPlanThreads - 1, list.blocks[b].tiles()); };
  for (int b = tid; b < blocks; b += kPlanThreads) atomicAdd(&bins[bin_of(b)], 1);
  __syncthreads();
  int all;
  const int before = scan_before(bins[tid], &all);
  bins[tid] = before;
  __syncthreads();
  for (int b = tid; b < blocks; b += kPlanThreads) list.order[atomicAdd(&bins[bin_of(b)], 1)] = b;
}

// ---------------------------------------------------------------- the join

// A row's parts to its result, in order; D / 4 lanes a row, `chunks` workgroups a
// (block, head).  Without a shared prefix the blocks of `list` that runs cut, one for
// the first boundary in each; with one all blocks of own places (the narrow list),
// whose rows look up their group's.
constexpr int kJoinThreads = 256;
__global__ __launch_bounds__(kJoinThreads) void tile_join_kernel(TileAttention a, TilePlan plan, TileList list, int chunks,
                                                                 bool both) {
  __shared__ int found_lds;
  const TileHeader head = *list.header;
  const int D = a.cache.head_dim, lanes = D / 4, at_once = kJoinThreads / lanes, kv_heads = a.cache.kv_heads;
  const int chunk = blockIdx.x % chunks;
  int b = blockIdx.x / chunks, kvh;
  if (both) {
    kvh = b % kv_heads, b /= kv_heads;
    if (b >= head.blocks) return;
  } else {
    // The block that run b + 1 cuts, unless an earlier run does.
    if (head.direct) return;
    const int64_t total = int64_t(head.units) * kv_heads, u = int64_t(b + 1) * head.per;
    if (u >= total) return;
    kvh = int(u / head.units);
    const int local = int(u - int64_t(kvh) * head.units);
    if (threadIdx.x == 0) found_lds = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < head.blocks; i += kJoinThreads) {
      const int at = local - list.blocks[i].before;
      if (at > 0 && at < list.blocks[i].tiles() && at <= head.per) found_lds = i;
    }
    __syncthreads();
    b = found_lds;
    if (b < 0) return;
  }
  const TileBlock w = list.blocks[b];
  const int slot = threadIdx.x / lanes, at = threadIdx.x % lanes;
  if (slot >= at_once || w.kind == kSharedPrefix) return;

  // Where the parts of a block's row are: n of them from run r0 on, the first one the
  // run's later piece or not; or one, a row of whole pieces (r0 < 0).
  struct Parts {
    int64_t place;                           // of the whole row, or of the first run's part
    int n, stride;
    bool later;
  };
  auto parts_of = [&](const TileHeader &h, const TileBlock &x, int64_t parts, int block_rows, int64_t q_row, int row) {
    Parts p{(x.kind == kSharedPrefix ? int64_t(a.T) * a.q_heads : 0) + q_row, x.tiles() > 0 ? 1 : 0, 0, false};
    if (h.direct || x.tiles() == 0) return p;
    const int64_t u0 = int64_t(kvh) * h.units + x.before;
    const int r0 = int(u0 / h.per), r1 = int((u0 + x.tiles() - 1) / h.per);
    if (r0 != r1) p = Parts{parts + 2 * int64_t(r0) * block_rows + row, r1 - r0 + 1, block_rows, int64_t(r0) * h.per < u0};
    return p;
  };
  auto place_of = [](const Parts &p, int i) { return p.place + (2 * int64_t(i) + (i == 0 && p.later)) * p.stride; };

  for (int row = chunk * at_once + slot; row < w.rows; row += chunks * at_once) {
    const int64_t q_row = query_row(a, w, kvh, row).at;
    const Parts mine = parts_of(head, w, list.parts, list.block_rows, q_row, row);
    Parts prefix{0, 0, 0, false};
    if (both && w.group >= 0) {
      int begin;
      const int rows = tokens_of(a, w.group, &begin) * (a.q_heads / kv_heads);
      const bool narrow = list_of(a, plan, w.group, rows) == 1;
      const int64_t parts = narrow ? plan.list[1].parts : plan.list[0].parts;
      const int block_rows = narrow ? plan.list[1].block_rows : plan.list[0].block_rows;
      const TileBlock *blocks = narrow ? plan.list[1].blocks : plan.list[0].blocks;
      const int32_t *first = narrow ? plan.list[1].first_block : plan.list[0].first_block;
      const TileHeader h = narrow ? *plan.list[1].header : *plan.list[0].header;
      const int in_group = w.group_row + row;
      prefix = parts_of(h, blocks[first[w.group] + in_group / block_rows], parts, block_rows, q_row, in_group % block_rows);
    }
    const int n = prefix.n + mine.n;
    auto place = [&](int i) { return i < prefix.n ? place_of(prefix, i) : place_of(mine, i - prefix.n); };
    float top = -INFINITY;
#pragma unroll 8
    for (int i = 0; i < n; ++i) top = fmaxf(top, plan.ml[place(i)].x);
    const float ms = top == -INFINITY ? 0.0f : top;
    f32x4 o{};
    float l = 0.0f;
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const int64_t p = place(i);
      const float2 ml = plan.ml[p];
      const f32x4 v = reinterpret_cast<const f32x4 *>(plan.o)[p * lanes + at];
      const float keep = __builtin_amdgcn_exp2f(ml.x - ms);
      o += v * keep;
      l += ml.y * keep;
    }
    if (at == 0 && a.lse) a.lse[q_row] = l == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(l)) * kLn2;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    reinterpret_cast<u32x2 *>(a.out + q_row * D)[at] =
        u32x2{pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv)};
  }
}

// ---------------------------------------------------------------- the sizes

struct Sizes {
  TileList list[2];
  int64_t whole_rows, rows;                  // rows: of parts, all together
  int32_t narrow_rows;
};

Sizes sizes_of(int32_t T, int32_t n_seqs, int32_t n_groups, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
               int32_t max_len, int32_t max_prefix) {
  Sizes s{};
  const int64_t group = q_heads / kv_heads, rows = T * group;
  const int64_t problems = n_groups > 0 ? n_groups : n_seqs;
  TileList &wide = s.list[0], &narrow = s.list[1];
  // Few rows a problem on the average: all of them in narrow blocks (64 sequences of
  // 64 rows over up to 4095 places 294 us, in wide blocks 357; of 96 rows 416 against
  // 368; one of 64 rows over 14336 places 66 against 60).  Else narrow blocks for the
  // problems that have no more than one, where there may be several whose places take
  // long to read: 2048 tokens and 63 single ones over up to 4095 places 270 us (all wide:
  // 370), over up to 1000 174 us (146); 512 tokens and 3 single ones 71 us either way,
  // 7 single ones over up to 900 62 us (59).  Two more launches are some 5 us.
  const bool all_narrow = rows <= 2 * kRows * problems;
  const bool some_narrow = all_narrow || n_groups > 0 || (n_seqs >= 8 && max_len > 2 * kWholePlaces);
  narrow.block_rows = tile_narrow_rows(head_dim, n_groups > 0 && !all_narrow ? group : ceil_div(rows, problems));
  narrow.tile = kNarrowTile;
  narrow.runs = tile_narrow_groups(head_dim, narrow.block_rows);
  s.narrow_rows = all_narrow ? 0x7FFFFFFF : some_narrow ? narrow.block_rows : 0;
  wide.block_rows = tile_wide_rows(head_dim, ceil_div(rows, problems));
  wide.tile = kWideTile;
  wide.runs = 256;                           // one a CU
  if (!all_narrow) wide.max_blocks = int32_t(std::min<int64_t>(0x7FFFFFFF, rows / wide.block_rows + problems));
  if (some_narrow) {
    const int64_t most = all_narrow ? rows / narrow.block_rows + problems : problems;
    const int64_t own = n_groups > 0 ? n_seqs * ceil_div(group, narrow.block_rows) : 0;
    narrow.max_blocks = int32_t(std::min<int64_t>(0x7FFFFFFF, most + own));
  }
  s.whole_rows = n_groups > 0 ? 2 * int64_t(T) * q_heads : 0;
  s.rows = s.whole_rows;
  for (TileList &l : s.list) {
    l.can_split = std::max(max_len, max_prefix) > kWholePlaces;
    l.parts = s.rows;
    if (l.can_split && l.max_blocks > 0) s.rows += 2 * int64_t(l.runs) * l.block_rows;
  }
  return s;
}

inline int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }

// Lays the plan out from `workspace` on; returns its bytes.
int64_t lay_out(const Sizes &s, int64_t problems, int64_t head_dim, void *workspace, TilePlan *plan) {
  const uintptr_t base = reinterpret_cast<uintptr_t>(workspace);      // null for the bytes alone
  int64_t at = 256;
  for (int i = 0; i < 2; ++i) {
    TileList l = s.list[i];
    l.header = reinterpret_cast<TileHeader *>(base + 128 * i);
    l.queue = reinterpret_cast<int32_t *>(base + 128 * i + 64);
    l.blocks = reinterpret_cast<TileBlock *>(base + at);
    at += align256(l.max_blocks * int64_t(sizeof(TileBlock)));
    l.order = reinterpret_cast<int32_t *>(base + at);
    at += align256(int64_t(l.max_blocks) * 4);
    l.first_block = reinterpret_cast<int32_t *>(base + at);
    if (l.max_blocks > 0) at += align256(problems * 4);
    plan->list[i] = l;
  }
  plan->ml = reinterpret_cast<float2 *>(base + at);
  at += align256(s.rows * int64_t(sizeof(float2)));
  plan->o = reinterpret_cast<float *>(base + at);
  plan->whole_rows = s.whole_rows;
  plan->narrow_rows = s.narrow_rows;
  return at + s.rows * head_dim * int64_t(sizeof(float));
}

// Workgroups of a (block, head) in the join: each takes kJoinRows rows.
constexpr int kJoinRows = 32;
inline int join_chunks(int block_rows) { return int(ceil_div(block_rows, kJoinRows)); }

constexpr int64_t kMostGroups = (int64_t(1) << 32) / kJoinThreads - 1;

}  // namespace

int64_t tile_attention_workspace(int32_t T, int32_t n_seqs, int32_t n_groups, int32_t q_heads, int32_t kv_heads,
                                 int32_t head_dim, int32_t max_len, int32_t max_prefix) {
  const Sizes s = sizes_of(T, n_seqs, n_groups, q_heads, kv_heads, head_dim, max_len, max_prefix);
  const int64_t tiles = ceil_div(std::max(max_len, max_prefix), kWideTile) + 2;
  const int64_t rows = int64_t(T) * (q_heads / kv_heads);
  if (rows > 1 << 30 || s.whole_rows > 0x7FFFFFFF) return -1;
  for (const TileList &l : s.list) {
    // Tiles are counted in 31 bits, a head's and a run's; the join's workgroups in 24.
    if (l.max_blocks > 0x7FFFFFFF / tiles / kv_heads) return -1;
    if (s.whole_rows > 0 && int64_t(l.max_blocks) * kv_heads * join_chunks(l.block_rows) > kMostGroups) return -1;
  }
  TilePlan plan;
  return lay_out(s, n_groups + int64_t(n_seqs), head_dim, nullptr, &plan);
}

hipError_t launch_tile_attention(const TileAttention &a, hipStream_t stream) {
  const int D = a.cache.head_dim, hkv = a.cache.kv_heads;
  const Sizes s = sizes_of(a.T, a.n_seqs, a.n_groups, a.q_heads, hkv, D, a.max_len, a.max_prefix);
  TilePlan plan{};
  lay_out(s, a.n_groups + int64_t(a.n_seqs), D, a.workspace, &plan);
  hipLaunchKernelGGL(plan_kernel, dim3(2), dim3(kPlanThreads), 0, stream, a, plan);
  hipError_t err = hipGetLastError();
  if (err == hipSuccess && plan.list[0].max_blocks > 0) err = launch_tile_wide(a, plan, stream);
  if (err == hipSuccess && plan.list[1].max_blocks > 0) err = launch_tile_narrow(a, plan, stream);
  const bool both = plan.whole_rows > 0;
  for (int i = 0; i < 2 && err == hipSuccess; ++i) {
    const TileList &l = plan.list[i];
    if (l.max_blocks == 0 || !(l.can_split || both) || (both && i == 0)) continue;
    const int chunks = join_chunks(l.block_rows);
    const int64_t blocks = both ? int64_t(l.max_blocks) * hkv : l.runs - 1;
    hipLaunchKernelGGL(tile_join_kernel, dim3(unsigned(blocks * chunks)), dim3(kJoinThreads), 0, stream, a, plan, l, chunks,
                       both);
    err = hipGetLastError();
  }
  return err;
}

}  // namespace engram
