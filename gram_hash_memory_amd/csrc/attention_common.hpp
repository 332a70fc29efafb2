// Pieces that the attention kernels share: conversions of the cache's formats
// to matrix-core operands, and the plan of the kernels that take several query
// rows a sequence (chunk_attention.hip, cache_weights.hip).
#pragma once

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
