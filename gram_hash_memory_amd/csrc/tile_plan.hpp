// How attention of several query rows a key-value head is cut up (tile_plan.hip),
// for the kernels that compute it (tile_wide.hip, tile_narrow.hip).
//
// A problem is a sequence's new tokens over its places, a group of sequences over
// their prefix, or a sequence's one token over its own places.  Its query rows of
// one key-value head (token-major, the heads of its group inside) are cut into
// blocks, and the places that a block's rows see into tiles.  Problems of many rows
// go to the wide list, whose blocks have 128 or 256 rows, 32 a wave: bound by the
// matrix cores.  Problems of few go to the narrow list, whose blocks have 16 or 32
// rows and whose waves share the places: bound by reading them.
#pragma once

#include "common.hpp"

namespace engram {
namespace attn {

constexpr int kRows = 32;                  // query rows of a wave
constexpr int kWideTile = 64;              // places of a tile
constexpr int kNarrowWaves = 4, kNarrowTile = 32 * kNarrowWaves;

enum TileKind : int32_t { kChunk = 0, kSharedPrefix = 1, kOwnPlaces = 2 };

// A block of query rows, for every key-value head: rows row0 .. row0 + rows - 1 of
// its problem, row = token * group + head of the group.  Its rows see places of
// [a_lo, a_hi) and [b_lo, b_hi); its tiles are a_n from a_tile on, then b_n from
// b_tile on, none of them twice.
struct TileBlock {
  int32_t kind, seq;                       // seq: the row of the page table
  int32_t token0, first;                   // the problem's first token, and its place
  int32_t row0, rows, len;
  int32_t a_lo, a_hi, b_lo, b_hi;
  int32_t a_tile, a_n, b_tile, b_n;
  int32_t before;                          // tiles of a head in the blocks before this one
  int32_t all_lo, all_hi, all_first, all_last;     // all rows see [all_lo, all_hi) and [all_first, all_last)
  int32_t group, group_row;                // own places: the group (-1: none), the first row in it

  __device__ __forceinline__ int tiles() const { return a_n + b_n; }
  // The first place of tile t of `size` places.
  __device__ __forceinline__ int place(int t, int size) const {
    return (t < a_n ? a_tile + t : b_tile + t - a_n) * size;
  }
  // Whether any row sees place p.
  __device__ __forceinline__ bool used(int p) const {
    return (unsigned(p - b_lo) < unsigned(b_hi - b_lo)) | (unsigned(p - a_lo) < unsigned(a_hi - a_lo));
  }
};

struct TileHeader {
  int32_t units;                           // tiles of all blocks, of a head
  int32_t blocks;
  int32_t per;                             // tiles of a run
  int32_t direct;                          // whole blocks, those of most tiles first, instead of runs
};

// One list of blocks, in the workspace.
struct TileList {
  TileHeader *header;
  int32_t *queue;
  TileBlock *blocks;
  int32_t *order;                          // the blocks by falling tiles (direct)
  int32_t *first_block;                    // of each problem of the list
  int32_t max_blocks, runs;                // workgroups
  int32_t block_rows, tile;
  int32_t can_split;
  int64_t parts;                           // where its runs' parts begin in o and ml

  // A run's first piece, or a later one (its last), of a block that it does not hold whole.
  __device__ __forceinline__ int64_t part_row(int run, bool later, int row) const {
    return parts + (2 * int64_t(run) + later) * block_rows + row;
  }
};

// o and ml hold rows of results before their division by the sum: with a shared
// prefix first one for each query row of whole pieces over the own places, then one
// of those over the prefix; then two blocks for each run.
struct TilePlan {
  TileList list[2];                        // wide, narrow
  float *o;
  float2 *ml;
  int64_t whole_rows;                      // 0: whole pieces are results
  int32_t narrow_rows;                     // most rows of a narrow problem (own places are always narrow)
};

// What a query row sees: places lo .. lo + n - 1 and first .. first + m - 1.
struct RowSees {
  int lo, n, first, m;
};
__device__ __forceinline__ bool sees(const RowSees &r, int p) {
  return (unsigned(p - r.lo) < unsigned(r.n)) | (unsigned(p - r.first) < unsigned(r.m));
}
// The places of its prefix that sequence `seq` of `len` places has.
__device__ __forceinline__ int prefix_of(const AttentionRules &a, int seq, int len) {
  return a.prefix_lens ? max(0, min(a.prefix_lens[seq], len)) : 0;
}
// The token at place `pos` of a sequence of `len` places, whose document begins at `doc`.
__device__ __forceinline__ RowSees row_sees(const AttentionRules &a, int prefix, int doc, int pos, int len) {
  doc = max(0, doc);
  RowSees r;
  r.lo = max(doc, a.window > 0 ? pos - a.window + 1 : 0);
  r.n = max(0, max(0, min(pos + 1, len)) - r.lo);
  r.first = doc;
  r.m = max(0, prefix - doc);
  return r;
}
__device__ __forceinline__ RowSees token_sees(const AttentionRules &a, int seq, int token, int pos, int len) {
  return row_sees(a, prefix_of(a, seq, len), a.doc_starts ? a.doc_starts[token] : 0, pos, len);
}

// A sequence's length as the kernels take it.
__device__ __forceinline__ int length_of(int stated, int max_len, int width, int page_shift) {
  return int(min(int64_t(min(max(stated, 0), max_len)), int64_t(width) << page_shift));
}

// A query row of a block, of one key-value head.
struct QueryRow {
  int tok, token, head;
  int64_t at;                              // in q, out and lse, in rows
};
__device__ __forceinline__ QueryRow query_row(const TileAttention &a, const TileBlock &w, int kvh, int row) {
  const int group = a.q_heads / a.cache.kv_heads, in_problem = w.row0 + row;
  QueryRow q;
  q.tok = in_problem / group;
  q.token = w.token0 + q.tok;
  q.head = kvh * group + in_problem - q.tok * group;
  q.at = int64_t(q.token) * a.q_heads + q.head;
  return q;
}

// Scores are kept in units of log 2: z = unit * (q.k), the sign of the scale in q
// (q is zeroed where the scale is 0); with a cap, cap2 * tanh(z).
struct ScoreUnit {
  float unit, cap2;
  uint32_t flip, keep;
};
__device__ __forceinline__ ScoreUnit score_unit(const TileAttention &a, float log2e) {
  const float s = fabsf(a.scale);
  ScoreUnit u;
  u.unit = s == 0.0f ? 1.0f : a.rules.cap > 0.0f ? s / a.rules.cap : s * log2e;
  u.cap2 = a.rules.cap * log2e;
  u.flip = a.scale < 0.0f ? 0x80008000u : 0u;
  u.keep = s == 0.0f ? 0u : 0xFFFFFFFFu;
  return u;
}

// The block and tile that a workgroup begins with, and the tiles of its run.  All
// threads; false: nothing to do.
struct Work {
  int run, left, block, unit, kvh;
};
__device__ __forceinline__ bool first_work(const TileList &list, const TileHeader &head, int kv_heads, int threads,
                                           int *lds, Work *w) {
  *w = Work{int(blockIdx.x), 0, 0, 0, 0};
  if (head.direct) return head.blocks > 0;
  // Neighbouring runs share keys: they go to one XCD.
  if (list.runs % 8 == 0) w->run = w->run % 8 * (list.runs / 8) + w->run / 8;
  const int64_t total = int64_t(head.units) * kv_heads, u0 = int64_t(w->run) * head.per;
  if (u0 >= total) return false;
  w->left = int(min(int64_t(head.per), total - u0));
  w->kvh = int(u0 / head.units);
  const int local = int(u0 - int64_t(w->kvh) * head.units);
  for (int b = threadIdx.x; b < head.blocks; b += threads) {
    const int at = local - list.blocks[b].before;
    if (at >= 0 && at < list.blocks[b].tiles()) lds[0] = b, lds[1] = at;
  }
  __syncthreads();
  w->block = __builtin_amdgcn_readfirstlane(lds[0]);
  w->unit = __builtin_amdgcn_readfirstlane(lds[1]);
  __syncthreads();
  return true;
}
// The next whole block off the queue; false: none is left.
__device__ __forceinline__ bool next_block(const TileList &list, const TileHeader &head, int kv_heads, int *lds,
                                           Work *w) {
  if (threadIdx.x == 0) {
    const int at = atomicAdd(list.queue, 1);
    lds[0] = at < head.blocks * kv_heads ? list.order[at / kv_heads] : -1;
    lds[1] = at % kv_heads;
  }
  __syncthreads();
  w->block = __builtin_amdgcn_readfirstlane(lds[0]);
  w->kvh = __builtin_amdgcn_readfirstlane(lds[1]);
  w->unit = 0;
  __syncthreads();
  return w->block >= 0;
}

}  // namespace attn

// tile_wide.hip, tile_narrow.hip: plan.list[0] and plan.list[1].
hipError_t launch_tile_wide(const TileAttention &a, const attn::TilePlan &plan, hipStream_t stream);
hipError_t launch_tile_narrow(const TileAttention &a, const attn::TilePlan &plan, hipStream_t stream);
// Rows of a block, for problems of so many.
int tile_wide_rows(int32_t head_dim, int64_t rows);
int tile_narrow_rows(int32_t head_dim, int64_t rows);
int tile_narrow_groups(int32_t head_dim, int32_t block_rows);      // workgroups that run at once

}  // namespace engram
