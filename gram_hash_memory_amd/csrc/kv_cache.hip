// Keys and values into and out of the paged cache.
//
// Both move bytes and nothing else (the 8-bit format's rounding costs some 60
// vector instructions for 16 values).  A group of LP lanes takes one (token,
// head) row of keys or of values; the rows of a token are neighbours, so a
// wave reads and writes runs of several hundred bytes.
#include "kv_cache.hpp"

namespace engram {
namespace {

using namespace kvc;

template <int LP, bool kMx>
__global__ __launch_bounds__(kThreads) void cache_write_kernel(
    CacheView c, const uint16_t *__restrict__ k, int64_t k_token, int64_t k_head,
    const uint16_t *__restrict__ v, int64_t v_token, int64_t v_head,
    const int64_t *__restrict__ slots, int64_t rows, int32_t *__restrict__ bad_slots) {
  const int64_t at = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  const int sub = int(at % LP);
  const int64_t row = at / LP;                     // token * 2 kv_heads + (keys, then values)
  const int heads = 2 * c.kv_heads;
  const int64_t t = row / heads;
  const int h = int(row - t * heads);
  const bool is_v = h >= c.kv_heads;
  const int head = is_v ? h - c.kv_heads : h;
  bool ok = row < rows;
  int64_t slot = -1;
  if (ok) {
    slot = slots[t];
    ok = slot_ok(c, slot);
    if (!ok && slot != -1 && bad_slots && h == 0 && sub == 0) atomicAdd(bad_slots, 1);
  }
  ok = ok && sub * 16 < c.head_dim;
  uint32_t w[8] = {};
  if (ok) {
    const uint16_t *src = (is_v ? v + t * v_token + head * v_head : k + t * k_token + head * k_head);
    const u32x4 *p = reinterpret_cast<const u32x4 *>(src + 16 * sub);
    const u32x4 a = p[0], b = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = a[i], w[4 + i] = b[i];
  }
  store16<kMx>(is_v ? c.v : c.k, is_v ? c.v_scales : c.k_scales, c.head_dim,
               ok ? row_index(c, slot, head) : 0, sub, ok, w);
}

template <int LP, bool kMx>
__global__ __launch_bounds__(kThreads) void cache_read_kernel(
    CacheView c, const int64_t *__restrict__ slots, int64_t rows, uint16_t *__restrict__ k,
    uint16_t *__restrict__ v, int32_t *__restrict__ bad_slots) {
  const int64_t at = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  const int sub = int(at % LP);
  const int64_t row = at / LP;
  if (row >= rows || sub * 16 >= c.head_dim) return;
  const int heads = 2 * c.kv_heads;
  const int64_t t = row / heads;
  const int h = int(row - t * heads);
  const bool is_v = h >= c.kv_heads;
  const int head = is_v ? h - c.kv_heads : h;
  const int64_t slot = slots[t];
  const bool ok = slot_ok(c, slot);
  if (!ok && slot != -1 && bad_slots && h == 0 && sub == 0) atomicAdd(bad_slots, 1);
  u32x4 a{}, b{};
  if (ok) {
    const int64_t r = row_index(c, slot, head);
    const void *data = is_v ? c.v : c.k;
    if constexpr (kMx) {
      const uint8_t *src = static_cast<const uint8_t *>(data) + r * c.head_dim + 16 * sub;
      const u32x4 q = *reinterpret_cast<const u32x4 *>(src);
      const float scale = e8m0_to_float((is_v ? c.v_scales : c.k_scales)[r * (c.head_dim / 32) + sub / 2]);
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(q[i]), false);
        const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(int(q[i]), true);
        o[2 * i] = pack_bf16x2(lo[0] * scale, lo[1] * scale);
        o[2 * i + 1] = pack_bf16x2(hi[0] * scale, hi[1] * scale);
      }
      a = u32x4{o[0], o[1], o[2], o[3]};
      b = u32x4{o[4], o[5], o[6], o[7]};
    } else {
      const u32x4 *p = reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(data) + r * c.head_dim + 16 * sub);
      a = p[0], b = p[1];
    }
  }
  u32x4 *dst = reinterpret_cast<u32x4 *>((is_v ? v : k) + (t * c.kv_heads + head) * c.head_dim + 16 * sub);
  dst[0] = a;
  dst[1] = b;
}

template <typename F>
hipError_t by_row(const CacheView &c, F &&f) {
  const bool mx = c.k_scales != nullptr;
  switch (lanes_per_row(c.head_dim)) {
#define ENGRAM_ROW(LP)                                                            \
  case LP:                                                                        \
    if (mx) f(std::integral_constant<int, LP>{}, std::true_type{});              \
    else f(std::integral_constant<int, LP>{}, std::false_type{});                \
    break
    ENGRAM_ROW(2);
    ENGRAM_ROW(4);
    ENGRAM_ROW(8);
    ENGRAM_ROW(16);
#undef ENGRAM_ROW
  }
  return hipGetLastError();
}

}  // namespace

int64_t cache_move_blocks(int32_t kv_heads, int32_t head_dim, int64_t T) {
  return (T * 2 * kv_heads * lanes_per_row(head_dim) + kThreads - 1) / kThreads;
}

hipError_t launch_cache_write(const CacheView &c, const uint16_t *k, int64_t k_token,
                              int64_t k_head, const uint16_t *v, int64_t v_token, int64_t v_head,
                              const int64_t *slots, int32_t T, int32_t *bad_slots,
                              hipStream_t stream) {
  const dim3 grid(unsigned(cache_move_blocks(c.kv_heads, c.head_dim, T)));
  return by_row(c, [&](auto lp, auto mx) {
    hipLaunchKernelGGL((cache_write_kernel<lp.value, mx.value>), grid, dim3(kThreads), 0, stream,
                       c, k, k_token, k_head, v, v_token, v_head, slots,
                       int64_t(T) * 2 * c.kv_heads, bad_slots);
  });
}

hipError_t launch_cache_read(const CacheView &c, const int64_t *slots, int32_t T, uint16_t *k,
                             uint16_t *v, int32_t *bad_slots, hipStream_t stream) {
  const dim3 grid(unsigned(cache_move_blocks(c.kv_heads, c.head_dim, T)));
  return by_row(c, [&](auto lp, auto mx) {
    hipLaunchKernelGGL((cache_read_kernel<lp.value, mx.value>), grid, dim3(kThreads), 0, stream,
                       c, slots, int64_t(T) * 2 * c.kv_heads, k, v, bad_slots);
  });
}

}  // namespace engram
