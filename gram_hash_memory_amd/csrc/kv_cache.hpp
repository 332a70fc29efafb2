// The paged key-value cache: addressing, and the 8-bit format's rounding.
//
// A head's head_dim values of one token are contiguous in the cache.  The
// kernels that move them give a lane 8 consecutive values at a time, 16 bytes
// of bf16, neighbouring lanes neighbouring ones: every load and store of a
// wave is then of whole runs, and a 32-value block of the 8-bit format is four
// neighbouring lanes.
#pragma once

#include "common.hpp"

namespace engram {
namespace kvc {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// The index of a place's row among all rows of the cache.
__device__ __forceinline__ int64_t row_index(const CacheView &c, int64_t slot, int head) {
  const int64_t page = slot >> c.page_shift;
  const int64_t in_page = slot & ((int64_t(1) << c.page_shift) - 1);
  return ((page * c.kv_heads + head) << c.page_shift) + in_page;
}

// 16 bytes past the caches where there is much to move once: the stores
// otherwise push out what is still to be read, and written lines wait in the
// caches for their turn (8192 tokens written and 32768 read back: 55.3 us with
// plain stores, 50.7 us so; norm and rotation of 8192 tokens, its loads too: 37.8
// and 32 us).
template <bool kOnce>
__device__ __forceinline__ u32x4 load16(const void *p) {
  if constexpr (kOnce) return __builtin_nontemporal_load(static_cast<const u32x4 *>(p));
  else return *static_cast<const u32x4 *>(p);
}
template <bool kOnce>
__device__ __forceinline__ void save16(void *p, u32x4 v) {
  if constexpr (kOnce) __builtin_nontemporal_store(v, static_cast<u32x4 *>(p));
  else *static_cast<u32x4 *>(p) = v;
}

__device__ __forceinline__ bool slot_ok(const CacheView &c, int64_t slot) {
  return slot >= 0 && slot < c.slots;
}

// 8 bf16 values of a lane to e4m3 codes with the scale that the four lanes of
// its block share.  The scale is 2^e with e the smallest that brings the
// block's largest finite magnitude m 2^E (1 <= m < 2) to 448 = 1.75 * 2^8 or
// below: E - 8, one more where m > 1.75; at least -95, so that 2^-e is a normal
// fp32 number, and the products with it are exact.  All lanes of the wave run
// this.
__device__ __forceinline__ uint32_t quantize8(const u32x4 w, u32x2 *codes) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
    top = max(top, lo < 0x7F80u ? lo : 0u);
    top = max(top, hi < 0x7F80u ? hi : 0u);
  }
  top = max(top, uint32_t(__shfl_xor(int(top), 1)));
  top = max(top, uint32_t(__shfl_xor(int(top), 2)));
  int e = int(top >> 7) - 127 - 8 + ((top & 0x7Fu) > 0x60u);
  e = top == 0 ? 0 : max(e, -95);
  const float inv = __uint_as_float(uint32_t(127 - e) << 23);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int p = __builtin_amdgcn_cvt_pk_fp8_f32(bf16_lo(w[2 * i]) * inv, bf16_hi(w[2 * i]) * inv, 0,
                                            false);
    p = __builtin_amdgcn_cvt_pk_fp8_f32(bf16_lo(w[2 * i + 1]) * inv,
                                        bf16_hi(w[2 * i + 1]) * inv, p, true);
    (*codes)[i] = uint32_t(p);
  }
  return uint32_t(e + 127);
}

// Values 8 piece .. 8 piece + 7 of the cache's row `row` (ok: this lane has a
// place to write to); a block's four lanes are 4-aligned neighbours.  All lanes
// of the wave run this.
template <bool kMx>
__device__ __forceinline__ void store8(void *data, uint8_t *scales, int head_dim, int64_t row,
                                       int piece, bool ok, const u32x4 w) {
  if constexpr (kMx) {
    u32x2 codes;
    const uint32_t byte = quantize8(w, &codes);
    if (!ok) return;
    *reinterpret_cast<u32x2 *>(static_cast<uint8_t *>(data) + row * head_dim + 8 * piece) = codes;
    if (piece % 4 == 0) scales[row * (head_dim / 32) + piece / 4] = uint8_t(byte);
  } else {
    if (!ok) return;
    *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(data) + row * head_dim + 8 * piece) = w;
  }
}

}  // namespace kvc
}  // namespace engram
