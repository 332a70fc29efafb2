// Where the pieces of a paged-attention workgroup's run lie in LDS.  Plain
// constexpr functions, so that a host program can check them for every shape.
#pragma once

namespace engram {
namespace attn {

constexpr int kW = 4;                      // waves of a workgroup
constexpr int kHeadBlock = 32;             // query heads of a workgroup
constexpr int kTileHeads = 16;             // of a matrix-core tile
constexpr unsigned kResultLds = 49152;     // for the waves' results: 64 KB with the rest

// 16-byte places that the waves' results of a piece of `heads` heads take, `acc`
// accumulator registers each: a tile of heads at a time.
constexpr int part_places(int acc, int heads) {
  return kW * acc * 4 * (heads < kTileHeads ? heads : kTileHeads);
}

// Two buffers, where they fit: a piece is joined while the next one's results are
// written.  block_heads: the heads of the widest piece.
constexpr bool two_buffers(int acc, int block_heads) {
  return 2u * 16 * part_places(acc, block_heads) <= kResultLds;
}
constexpr unsigned result_bytes(int acc, int block_heads) {
  return (two_buffers(acc, block_heads) ? 2u : 1u) * 16 * part_places(acc, block_heads);
}

// The first place of a run's piece number `index`.  It goes by the widest piece:
// the pieces before and after it may have more heads than it has (a key-value
// head's last block may have fewer).
constexpr int part_begin(int acc, int block_heads, int index) {
  return two_buffers(acc, block_heads) ? (index & 1) * part_places(acc, block_heads) : 0;
}

}  // namespace attn
}  // namespace engram
