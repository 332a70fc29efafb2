// The paged key-value cache: addressing, and the 8-bit format's rounding.
//
// A head's head_dim values of one token are contiguous in the cache.  The
// kernels that move them give each such row to LP lanes (head_dim / 16
// rounded up to a power of two; lanes past head_dim / 16 idle), 16
// consecutive values a lane: a 32-value block of the 8-bit format is then two
// neighbouring lanes.
#pragma once

#include "common.hpp"

namespace engram {
namespace kvc {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

inline int lanes_per_row(int head_dim) {
  const int n = head_dim / 16;
  return n <= 2 ? 2 : n <= 4 ? 4 : n <= 8 ? 8 : 16;
}

// The index of a place's row among all rows of the cache.
__device__ __forceinline__ int64_t row_index(const CacheView &c, int64_t slot, int head) {
  const int64_t page = slot >> c.page_shift;
  const int64_t in_page = slot & ((int64_t(1) << c.page_shift) - 1);
  return ((page * c.kv_heads + head) << c.page_shift) + in_page;
}

__device__ __forceinline__ bool slot_ok(const CacheView &c, int64_t slot) {
  return slot >= 0 && slot < c.slots;
}

// 16 bf16 values (8 dwords, value 2i in the low half of dword i) of a lane to
// e4m3 codes with the scale that they share with the neighbouring lane's.
// The scale is 2^e with e the smallest that brings the block's largest finite
// magnitude m 2^E (1 <= m < 2) to 448 = 1.75 * 2^8 or below: E - 8, one more
// where m > 1.75; at least -95, so that 2^-e is a normal fp32 number, and the
// products with it are exact.  All lanes of the wave run this.
__device__ __forceinline__ uint32_t quantize16(const uint32_t (&w)[8], uint32_t (&codes)[4]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
    top = max(top, lo < 0x7F80u ? lo : 0u);
    top = max(top, hi < 0x7F80u ? hi : 0u);
  }
  top = max(top, uint32_t(__shfl_xor(int(top), 1)));
  int e = int(top >> 7) - 127 - 8 + ((top & 0x7Fu) > 0x60u);
  e = top == 0 ? 0 : max(e, -95);
  const float inv = __uint_as_float(uint32_t(127 - e) << 23);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int p = __builtin_amdgcn_cvt_pk_fp8_f32(bf16_lo(w[2 * i]) * inv, bf16_hi(w[2 * i]) * inv, 0,
                                            false);
    p = __builtin_amdgcn_cvt_pk_fp8_f32(bf16_lo(w[2 * i + 1]) * inv,
                                        bf16_hi(w[2 * i + 1]) * inv, p, true);
    codes[i] = uint32_t(p);
  }
  return uint32_t(e + 127);
}

// A lane's 16 values into the cache's row `row` (ok: this lane has a place to
// write to).  All lanes of the wave run this.
template <bool kMx>
__device__ __forceinline__ void store16(void *data, uint8_t *scales, int head_dim, int64_t row,
                                        int sub, bool ok, const uint32_t (&w)[8]) {
  if constexpr (kMx) {
    uint32_t codes[4];
    const uint32_t byte = quantize16(w, codes);
    if (!ok) return;
    uint8_t *dst = static_cast<uint8_t *>(data) + row * head_dim + 16 * sub;
    *reinterpret_cast<u32x4 *>(dst) = u32x4{codes[0], codes[1], codes[2], codes[3]};
    if (sub % 2 == 0) scales[row * (head_dim / 32) + sub / 2] = uint8_t(byte);
  } else {
    if (!ok) return;
    u32x4 *dst = reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(data) + row * head_dim + 16 * sub);
    dst[0] = u32x4{w[0], w[1], w[2], w[3]};
    dst[1] = u32x4{w[4], w[5], w[6], w[7]};
  }
}

}  // namespace kvc
}  // namespace engram
