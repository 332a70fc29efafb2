// What the tile kernels of chunk_attention.hip work at: blocks of query rows, the
// tiles of places that each block sees, and where parts of results are kept.
#pragma once

#include "common.hpp"

namespace engram {
namespace attn {

constexpr int kTile = 64;                  // places of a tile

enum TileKind : int32_t { kChunk = 0, kSharedPrefix = 1, kOwnPlaces = 2 };

// A block of query rows of one problem (a sequence's new tokens, a group's
// sequences over their prefix, a sequence over its own places), for every
// key-value head: rows row0 .. row0 + rows - 1 of the problem, row = token * group
// + head of the group.  Its rows see places of [a_lo, a_hi) and [b_lo, b_hi); its
// tiles are a_n from a_tile on, then b_n from b_tile on, none of them twice.
struct TileBlock {
  int32_t kind, seq;                       // seq: the row of the page table
  int32_t token0, first;                   // the problem's first token, and its place
  int32_t row0, rows, len;
  int32_t a_lo, a_hi, b_lo, b_hi;
  int32_t a_tile, a_n, b_tile, b_n;
  int32_t before;                          // tiles of a head in the blocks before this one
  int32_t prefix_block, prefix_row;        // own places: the group's first block, the first row in it (-1: none)
};

struct TileHeader {
  int32_t units;                           // tiles of all blocks, of a head
  int32_t blocks;
  int32_t per;                             // tiles of a run
  int32_t direct;                          // whole blocks off the queue instead of runs
};

// The workspace.  o and ml hold rows of results before their division by the sum:
// first a row for each query row of whole pieces (shared prefix: two, for the
// prefix and the own places), then two blocks for each run.
struct TilePlan {
  TileHeader *header;
  int32_t *queue;
  TileBlock *blocks;
  int32_t *first_block;                    // of each problem
  float *o;
  float2 *ml;
  int32_t max_blocks, runs, whole_rows;
  int32_t can_split;

  __device__ __forceinline__ int64_t part_row(int run, bool later, int block, int row) const {
    return whole_rows + (2 * int64_t(run) + later) * block + row;
  }
};

// What a query row sees: places lo .. lo + n - 1 and first .. first + m - 1.
struct RowSees {
  int lo, n, first, m;
};
__device__ __forceinline__ bool sees(const RowSees &r, int p) {
  return unsigned(p - r.lo) < unsigned(r.n) || unsigned(p - r.first) < unsigned(r.m);
}
// The token at place `pos` of a sequence of `len` places.
__device__ __forceinline__ RowSees row_sees(const AttentionRules &a, int seq, int token, int pos, int len) {
  const int doc = a.doc_starts ? max(0, a.doc_starts[token]) : 0;
  RowSees r;
  r.lo = max(doc, a.window > 0 ? pos - a.window + 1 : 0);
  r.n = max(0, max(0, min(pos + 1, len)) - r.lo);
  r.first = doc;
  r.m = max(0, (a.prefix_lens ? max(0, min(a.prefix_lens[seq], len)) : 0) - doc);
  return r;
}

// A sequence's length as the kernels take it.
__device__ __forceinline__ int length_of(int stated, int max_len, int width, int page_shift) {
  return int(min(int64_t(min(max(stated, 0), max_len)), int64_t(width) << page_shift));
}

}  // namespace attn
}  // namespace engram
