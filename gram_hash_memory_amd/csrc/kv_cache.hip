// Keys and values into and out of the paged cache.
//
// Both move bytes and nothing else: 8192 tokens of 8 heads of 128 written in 8
// bits take 13 us (3.9 TB/s), 32768 read back 38 us (5.3 TB/s).  A group of LP
// lanes takes one (token, head) row of keys or of values, 8 values a lane; the
// rows of a token are neighbours, so every load and store of a wave covers
// whole runs (16 values a lane, two stores 32 bytes apart: 15 and 44 us).
#include "kv_cache.hpp"

namespace engram {
namespace {

using namespace kvc;

// Lanes of a row: head_dim / 8 rounded up to a power of two; those past
// head_dim / 8 idle.
inline int row_lanes(int head_dim) {
  const int n = head_dim / 8;
  return n <= 4 ? 4 : n <= 8 ? 8 : n <= 16 ? 16 : 32;
}

// n / d for the uniform d: recip = floor((2^32 - 1) / d) makes the estimate at
// most one short.
__device__ __forceinline__ uint32_t quotient(uint32_t n, uint32_t d, uint32_t recip) {
  const uint32_t q = __umulhi(n, recip);
  return q + (n - q * d >= d);
}

// Piece i of a thread: its row, token, head and side.
struct Row {
  uint32_t t;
  int head;
  bool is_v, first, in;
};
__device__ __forceinline__ Row row_of(uint32_t row, uint32_t rows, const CacheView &c,
                                      uint32_t recip) {
  const uint32_t heads = 2 * c.kv_heads;           // of a token: the keys', then the values'
  const uint32_t t = quotient(row, heads, recip), h = row - t * heads;
  const bool is_v = h >= uint32_t(c.kv_heads);
  return {t, int(is_v ? h - c.kv_heads : h), is_v, h == 0, row < rows};
}

template <int LP, bool kMx, int kPer>
__global__ __launch_bounds__(kThreads) void cache_write_kernel(
    CacheView c, const uint16_t *__restrict__ k, int64_t k_token, int64_t k_head,
    const uint16_t *__restrict__ v, int64_t v_token, int64_t v_head,
    const int64_t *__restrict__ slots, uint32_t rows, uint32_t recip,
    int32_t *__restrict__ bad_slots) {
  constexpr uint32_t kRows = kThreads / LP;
  const int sub = threadIdx.x % LP;
  const uint32_t first = blockIdx.x * (kRows * kPer) + threadIdx.x / LP;
  Row r[kPer];
  int64_t slot[kPer];
  u32x4 w[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    r[i] = row_of(first + i * kRows, rows, c, recip);
    slot[i] = -1;
    w[i] = u32x4{};
    if (!r[i].in || 8 * sub >= c.head_dim) continue;
    slot[i] = slots[r[i].t];
    w[i] = *reinterpret_cast<const u32x4 *>(
        (r[i].is_v ? v + r[i].t * v_token + r[i].head * v_head
                   : k + r[i].t * k_token + r[i].head * k_head) + 8 * sub);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const bool ok = slot_ok(c, slot[i]);
    if (!ok && slot[i] != -1 && bad_slots && r[i].first && sub == 0) atomicAdd(bad_slots, 1);
    store8<kMx>(r[i].is_v ? c.v : c.k, r[i].is_v ? c.v_scales : c.k_scales, c.head_dim,
                ok ? row_index(c, slot[i], r[i].head) : 0, sub, ok, w[i]);
  }
}

template <int LP, bool kMx, int kPer>
__global__ __launch_bounds__(kThreads) void cache_read_kernel(
    CacheView c, const int64_t *__restrict__ slots, uint32_t rows, uint32_t recip,
    uint16_t *__restrict__ k, uint16_t *__restrict__ v, int32_t *__restrict__ bad_slots) {
  constexpr uint32_t kRows = kThreads / LP;
  const int sub = threadIdx.x % LP;
  if (8 * sub >= c.head_dim) return;
  const uint32_t first = blockIdx.x * (kRows * kPer) + threadIdx.x / LP;
  Row r[kPer];
  int64_t slot[kPer];
  u32x4 w[kPer];                                   // 8 bf16 values, or 8 codes in [0], [1]
  uint32_t scale[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    r[i] = row_of(first + i * kRows, rows, c, recip);
    slot[i] = r[i].in ? slots[r[i].t] : -1;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    w[i] = u32x4{};
    scale[i] = 127;
    if (!slot_ok(c, slot[i])) continue;
    const int64_t at = row_index(c, slot[i], r[i].head) * c.head_dim + 8 * sub;
    const void *data = r[i].is_v ? c.v : c.k;
    if constexpr (kMx) {
      const u32x2 q = *reinterpret_cast<const u32x2 *>(static_cast<const uint8_t *>(data) + at);
      w[i][0] = q[0], w[i][1] = q[1];
      scale[i] = (r[i].is_v ? c.v_scales : c.k_scales)[at / 32];
    } else {
      w[i] = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(data) + at);
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (!r[i].in) continue;
    if (slot[i] != -1 && !slot_ok(c, slot[i]) && bad_slots && r[i].first && sub == 0)
      atomicAdd(bad_slots, 1);
    if constexpr (kMx) {
      const float f = e8m0_to_float(scale[i]);
      const uint32_t q[2] = {w[i][0], w[i][1]};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(q[e]), false);
        const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(int(q[e]), true);
        w[i][2 * e] = pack_bf16x2(lo[0] * f, lo[1] * f);
        w[i][2 * e + 1] = pack_bf16x2(hi[0] * f, hi[1] * f);
      }
    }
    save16<(kPer > 1)>((r[i].is_v ? v : k) +
                           (int64_t(r[i].t) * c.kv_heads + r[i].head) * c.head_dim + 8 * sub,
                       w[i]);
  }
}

// Pieces a thread takes: 2 where that still leaves every CU several workgroups
// (1: 58 us for the two moves above, 2: 50, 4: 58).
constexpr int kManyPieces = 2;
constexpr int64_t kManyBlocks = 2048;

template <typename F>
hipError_t by_row(const CacheView &c, F &&f) {
  const bool mx = c.k_scales != nullptr;
  switch (row_lanes(c.head_dim)) {
#define ENGRAM_ROW(LP)                                                            \
  case LP:                                                                        \
    if (mx) f(std::integral_constant<int, LP>{}, std::true_type{});              \
    else f(std::integral_constant<int, LP>{}, std::false_type{});                \
    break
    ENGRAM_ROW(4);
    ENGRAM_ROW(8);
    ENGRAM_ROW(16);
    ENGRAM_ROW(32);
#undef ENGRAM_ROW
  }
  return hipGetLastError();
}

}  // namespace

int64_t cache_move_blocks(int32_t kv_heads, int32_t head_dim, int64_t T) {
  return (T * 2 * kv_heads * row_lanes(head_dim) + kThreads - 1) / kThreads;
}

namespace {

// f(lanes per row, format, pieces a thread, grid).
template <typename F>
hipError_t by_size(const CacheView &c, int64_t T, F &&f) {
  const int64_t blocks = cache_move_blocks(c.kv_heads, c.head_dim, T);
  return by_row(c, [&](auto lp, auto mx) {
    if (blocks >= kManyBlocks)
      f(lp, mx, std::integral_constant<int, kManyPieces>{},
        dim3(unsigned((blocks + kManyPieces - 1) / kManyPieces)));
    else
      f(lp, mx, std::integral_constant<int, 1>{}, dim3(unsigned(blocks)));
  });
}

uint32_t recip_of(const CacheView &c) { return 0xFFFFFFFFu / uint32_t(2 * c.kv_heads); }

}  // namespace

hipError_t launch_cache_write(const CacheView &c, const uint16_t *k, int64_t k_token,
                              int64_t k_head, const uint16_t *v, int64_t v_token, int64_t v_head,
                              const int64_t *slots, int32_t T, int32_t *bad_slots,
                              hipStream_t stream) {
  return by_size(c, T, [&](auto lp, auto mx, auto per, dim3 grid) {
    hipLaunchKernelGGL((cache_write_kernel<lp.value, mx.value, per.value>), grid, dim3(kThreads),
                       0, stream, c, k, k_token, k_head, v, v_token, v_head, slots,
                       uint32_t(T) * 2 * c.kv_heads, recip_of(c), bad_slots);
  });
}

hipError_t launch_cache_read(const CacheView &c, const int64_t *slots, int32_t T, uint16_t *k,
                             uint16_t *v, int32_t *bad_slots, hipStream_t stream) {
  return by_size(c, T, [&](auto lp, auto mx, auto per, dim3 grid) {
    hipLaunchKernelGGL((cache_read_kernel<lp.value, mx.value, per.value>), grid, dim3(kThreads), 0,
                       stream, c, slots, uint32_t(T) * 2 * c.kv_heads, recip_of(c), k, v,
                       bad_slots);
  });
}

}  // namespace engram
