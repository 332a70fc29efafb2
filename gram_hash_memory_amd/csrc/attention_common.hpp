// Pieces that the attention kernels share: conversions of the cache's formats
// to matrix-core operands, and the registers that a wave holds 32 places in.
#pragma once

#include <utility>

#include "kv_cache.hpp"

namespace engram {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Two e4m3fn codes times 2^e as a bf16 pair (exact: 4 bits of significand).
__device__ __forceinline__ uint32_t mx_pair(uint32_t codes, float scale, bool high) {
  return __builtin_bit_cast(
      uint32_t, high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(int(codes), scale, true)
                     : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(int(codes), scale, false));
}

__device__ __forceinline__ bf16x8 as_frag(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(bf16x8, u32x4{a, b, c, d});
}

// How the head_dim = 32 * kDb dimensions fall to 16 lanes: pieces of 16, 8, 4,
// 2 neighbouring dimensions a lane (the binary digits of 2 * kDb).
template <int kDb>
struct Pieces {
  static constexpr int kN = (kDb >> 3) + ((kDb >> 2) & 1) + ((kDb >> 1) & 1) + (kDb & 1);
  static constexpr int width(int c) {
    for (int w = 16; w >= 2; w /= 2)
      if (2 * kDb & w)
        if (c-- == 0) return w;
    return 0;
  }
  static constexpr int base(int c) { return c == 0 ? 0 : base(c - 1) + 16 * width(c - 1); }
};

template <int kN, typename F, int... kI>
__device__ __forceinline__ void each_piece(F &&f, std::integer_sequence<int, kI...>) {
  (f(std::integral_constant<int, kI>{}), ...);
}
template <int kN, typename F>
__device__ __forceinline__ void each_piece(F &&f) {
  each_piece<kN>(f, std::make_integer_sequence<int, kN>{});
}

template <int kBytes>
__device__ __forceinline__ void load_bytes(uint32_t *dst, const uint8_t *src) {
  if constexpr (kBytes >= 16) {
#pragma unroll
    for (int i = 0; i < kBytes / 16; ++i) {
      const u32x4 v = reinterpret_cast<const u32x4 *>(src)[i];
      dst[4 * i] = v[0], dst[4 * i + 1] = v[1], dst[4 * i + 2] = v[2], dst[4 * i + 3] = v[3];
    }
  } else if constexpr (kBytes == 8) {
    const u32x2 v = *reinterpret_cast<const u32x2 *>(src);
    dst[0] = v[0], dst[1] = v[1];
  } else if constexpr (kBytes == 4) {
    dst[0] = *reinterpret_cast<const uint32_t *>(src);
  } else {
    dst[0] = *reinterpret_cast<const uint16_t *>(src);
  }
}

// 32 places' keys and values in a lane's registers, as they lie in the cache.
template <int kDb, bool kMx>
struct Held {
  static constexpr int kN = Pieces<kDb>::kN;
  uint32_t k[2][kMx ? 2 * kDb : 4 * kDb];      // place l % 16 of either tile
  uint32_t ks[2][(kDb + 1) / 2];
  uint32_t v[8][kMx ? (kDb + 1) / 2 : kDb];    // places 4 g .. 4 g + 3 of either tile
  uint32_t vs[8][kN];
};

// Over the 4 lanes of one column (l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ float column_max(float x) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float column_sum(float x) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// The values of dimensions d .. d + 3 of a place's row (d % 4 == 0) of keys or values.
template <bool kMx>
__device__ __forceinline__ void values_at(const CacheView &c, const void *data, const uint8_t *scales, int64_t row, int d,
                                          float *v) {
  if constexpr (kMx) {
    const uint32_t codes = *reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(data) + row * c.head_dim + d);
    const float scale = e8m0_to_float(min(uint32_t(scales[row * (c.head_dim / 32) + d / 32]), 254u));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = e4m3fn_to_float(codes >> (8 * i) & 255u) * scale;
  } else {
    const u32x2 w = *reinterpret_cast<const u32x2 *>(static_cast<const uint16_t *>(data) + row * c.head_dim + d);
    v[0] = bf16_lo(w[0]), v[1] = bf16_hi(w[0]), v[2] = bf16_lo(w[1]), v[3] = bf16_hi(w[1]);
  }
}

// The value of one dimension of a place's row.
template <bool kMx>
__device__ __forceinline__ float value_at(const CacheView &c, int64_t row, int d) {
  if constexpr (!kMx) return bf16_lo(static_cast<const uint16_t *>(c.v)[row * c.head_dim + d]);
  return e4m3fn_to_float(static_cast<const uint8_t *>(c.v)[row * c.head_dim + d]) *
         e8m0_to_float(min(uint32_t(c.v_scales[row * (c.head_dim / 32) + d / 32]), 254u));
}

// tanh of a score to be capped.  Up to kTanhSplit y T(y^2), because the form with
// an exponential would lose the small results' digits: T goes through the values of
// tanh(y) / y at the six Chebyshev points of y^2 in [0, 25/64] and 1 at 0; it is off
// by less than 2^-30 of the result, with its roundings 2^-23.
constexpr float kTanhSplit = 0.625f;
__device__ __forceinline__ float tanh_small(float y) {
  const float x = y * y;
  float t = 0.002292744815349579f;
  t = __builtin_fmaf(t, x, -0.008343945257365704f);
  t = __builtin_fmaf(t, x, 0.02176891826093197f);
  t = __builtin_fmaf(t, x, -0.053959257900714874f);
  t = __builtin_fmaf(t, x, 0.13333304226398468f);
  t = __builtin_fmaf(t, x, -0.3333333432674408f);
  return y * __builtin_fmaf(t, x, 1.0f);
}
__device__ __forceinline__ float tanh_large(float y) {
  return 1.0f - 2.0f * __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(2.0f * kLog2e * y) + 1.0f);
}

}  // namespace attn
}  // namespace engram
