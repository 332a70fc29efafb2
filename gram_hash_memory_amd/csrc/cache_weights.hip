// The attention weight that each place of the cache gets from new tokens,
//
//   w_p += sum over the tokens and heads that see p of e^(z_p - lse),
//
// with z as in tile_wide.hip.  A wave owns 32 places of one key-value head:
// their keys stay in its registers as matrix-core operands, the query rows of the
// sequence go by 32 at a time, and a lane adds up the weights of 8 places from
// every 16th row, in row order; lanes are joined once, at the end.  One wave writes
// a place, so the sums do not depend on timing.
#include "attention_common.hpp"
#include "tile_plan.hpp"

namespace engram {
namespace {

using namespace attn;

constexpr int kWaves = 4, kPlaces = 32;      // of a wave

template <int kDb, bool kMx>
__global__ __launch_bounds__(64 * kWaves, kDb <= 4 ? 4 : 2) void cache_weights_kernel(CacheWeights a, int chunks) {
  constexpr int D = 32 * kDb, kRowBytes = kMx ? D : 2 * D;
  const CacheView &c = a.cache;
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const int64_t pair = blockIdx.x / chunks;
  const int s = int(pair / c.kv_heads), kvh = int(pair - int64_t(s) * c.kv_heads);
  const int p0 = __builtin_amdgcn_readfirstlane(
      (int(blockIdx.x - pair * chunks) * kWaves + int(threadIdx.x >> 6)) * kPlaces);
  const int len = length_of(a.lens[s], a.max_len, a.table_width, c.page_shift);
  if (p0 >= len) return;
  const int begin = min(max(a.cu[s], 0), a.T), end = min(max(a.cu[s + 1], begin), a.T);
  const int group = a.q_heads / c.kv_heads, mask = (1 << c.page_shift) - 1;
  const int first = len - (end - begin);     // the first new token's place

  // The tokens that may see one of these places.
  int t0 = 0, t1 = end - begin;
  if (!(a.rules.prefix_lens && p0 < a.rules.prefix_lens[s])) {
    t0 = max(t0, p0 - first);
    if (a.rules.window > 0) t1 = int(min(int64_t(t1), int64_t(p0) + kPlaces - 1 + a.rules.window - first));
  }
  if (t0 >= t1) return;

  // 16 query rows as B operands, with what they see: requested before the keys, and
  // the next 16 before these are used.
  struct Rows {
    bf16x8 q[kDb];
    RowSees sees;
    float lse, slope;
    int pos;
    bool live;
  };
  const int r1 = t1 * group;
  auto load_rows = [&](int r0, Rows &x) {
    const int row = min(r0 + col, r1 - 1), tok = row / group, token = begin + tok;
    const int head = kvh * group + row - tok * group;
    const int64_t q_row = int64_t(token) * a.q_heads + head;
#pragma unroll
    for (int kk = 0; kk < kDb; ++kk) {
      const int d = kMx && (kk | 1) < kDb ? 64 * (kk / 2) + 16 * g + 8 * (kk & 1) : 32 * kk + 8 * g;
      x.q[kk] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(a.q + q_row * D + d));
    }
    x.pos = first + tok;
    x.sees = row_sees(a.rules, s, token, x.pos, len);
    x.lse = a.lse[q_row];
    x.slope = a.rules.slopes ? a.rules.slopes[head] * kLog2e : 0.0f;
    x.live = r0 + col < r1;
  };
  Rows rows[2];
  load_rows(t0 * group, rows[0]);
  // What is to be added to: lanes col < 8 write a place each.
  const int out_p = p0 + 16 * (col / 4) + 4 * g + col % 4;
  float *const out = a.weights + pair * a.weights_stride + out_p;
  const bool writes = col < 8 && out_p < len;
  const float old = writes ? *out : 0.0f;

  // Keys: place 16 u + col, as A operands.  In the 8-bit format 16 bytes are two steps.
  bf16x8 k[2][kDb];
  uint32_t absent = 0;                       // bit 16 u + x: place 16 u + x is on no page of the cache
  int64_t place[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int p = p0 + 16 * u + col;
    const int page = p < len ? a.table[int64_t(s) * a.table_width + (p >> c.page_shift)] : -1;
    const bool there = unsigned(page) < unsigned(c.pages);
    absent |= uint32_t(__ballot(!there) & 0xFFFFu) << (16 * u);
    place[u] = there ? ((int64_t(page) * c.kv_heads + kvh) << c.page_shift) + (p & mask) : 0;
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint8_t *const src = static_cast<const uint8_t *>(c.k) + place[u] * kRowBytes;
    if constexpr (!kMx) {
#pragma unroll
      for (int kk = 0; kk < kDb; ++kk)
        k[u][kk] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(src + 64 * kk + 16 * g));
    } else {
      const uint8_t *const sc = c.k_scales + place[u] * kDb;
      u32x4 code[(kDb + 1) / 2];
      float scale[(kDb + 1) / 2];
#pragma unroll
      for (int j = 0; j < kDb / 2; ++j) {
        code[j] = *reinterpret_cast<const u32x4 *>(src + 64 * j + 16 * g);
        scale[j] = e8m0_to_float(sc[2 * j + (g >> 1)]);
      }
      if constexpr (kDb % 2) {
        const u32x2 x = *reinterpret_cast<const u32x2 *>(src + 32 * (kDb - 1) + 8 * g);
        code[kDb / 2] = u32x4{x[0], x[1], 0, 0};
        scale[kDb / 2] = e8m0_to_float(sc[kDb - 1]);
      }
#pragma unroll
      for (int kk = 0; kk < kDb; ++kk) {
        const uint32_t x = code[kk / 2][2 * (kk % 2)], y = code[kk / 2][2 * (kk % 2) + 1];
        const float f = scale[kk / 2];
        k[u][kk] = as_frag(mx_pair(x, f, false), mx_pair(x, f, true), mx_pair(y, f, false), mx_pair(y, f, true));
      }
    }
  }

  const float unit = a.rules.cap > 0.0f ? a.scale / a.rules.cap : a.scale * kLog2e;
  const float cap2 = a.rules.cap * kLog2e;
  f32x4 sum[2] = {};
  bool bad = false;
  auto add_rows = [&](const Rows &x) {
    f32x4 z[2] = {};
#pragma unroll
    for (int kk = 0; kk < kDb; ++kk)
#pragma unroll
      for (int u = 0; u < 2; ++u) z[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k[u][kk], x.q[kk], z[u], 0, 0, 0);
    const bool weighs = x.lse != -INFINITY;
    const float lse = weighs ? x.lse * kLog2e : 0.0f;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = 16 * u + 4 * g + j, p = p0 + at;
        float y = z[u][j] * unit;
        if (a.rules.cap > 0.0f) {
          const float small = tanh_small(y), large = tanh_large(y);
          y = cap2 * (fabsf(y) <= kTanhSplit ? small : large);
        }
        if (a.rules.slopes) y = __builtin_fmaf(-x.slope, float(abs(x.pos - p)), y);
        const bool seen = x.live & sees(x.sees, p), gone = absent >> at & 1;
        bad |= seen & gone;
        const float e = __builtin_amdgcn_exp2f(y - lse);
        sum[u][j] += (seen & weighs & !gone) ? e : 0.0f;
      }
  };
  for (int r0 = t0 * group; r0 < r1; r0 += 32) {
    if (r0 + 16 < r1) load_rows(r0 + 16, rows[1]);
    add_rows(rows[0]);
    if (r0 + 32 < r1) load_rows(r0 + 32, rows[0]);
    if (r0 + 16 < r1) add_rows(rows[1]);
  }
  if (bad && kvh == 0 && a.bad_pages) atomicAdd(a.bad_pages, 1);

  // The 16 lanes of a column: each sum in all of them, then one written a lane.
  float mine = 0.0f;
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x = sum[u][j];
#pragma unroll
      for (int d = 1; d < 16; d *= 2) x += __shfl_xor(x, d);
      if (col == 4 * u + j) mine = x;
    }
  if (writes) *out = old + mine;
}

template <int kDb>
hipError_t launch(const CacheWeights &a, int64_t blocks, int chunks, hipStream_t stream) {
  if (a.cache.k_scales)
    hipLaunchKernelGGL((cache_weights_kernel<kDb, true>), dim3(unsigned(blocks)), dim3(64 * kWaves), 0, stream, a, chunks);
  else
    hipLaunchKernelGGL((cache_weights_kernel<kDb, false>), dim3(unsigned(blocks)), dim3(64 * kWaves), 0, stream, a, chunks);
  return hipGetLastError();
}

inline int64_t chunks_of(int32_t max_len) { return (int64_t(max_len) + kWaves * kPlaces - 1) / (kWaves * kPlaces); }

}  // namespace

int64_t cache_weights_blocks(int32_t n_seqs, int32_t kv_heads, int32_t max_len) {
  return int64_t(n_seqs) * kv_heads * chunks_of(max_len);
}

hipError_t launch_cache_weights(const CacheWeights &a, hipStream_t stream) {
  const int64_t blocks = cache_weights_blocks(a.n_seqs, a.cache.kv_heads, a.max_len);
  const int chunks = int(chunks_of(a.max_len));
  switch (a.cache.head_dim / 32) {
    case 1: return launch<1>(a, blocks, chunks, stream);
    case 2: return launch<2>(a, blocks, chunks, stream);
    case 3: return launch<3>(a, blocks, chunks, stream);
    case 4: return launch<4>(a, blocks, chunks, stream);
    case 5: return launch<5>(a, blocks, chunks, stream);
    case 6: return launch<6>(a, blocks, chunks, stream);
    case 7: return launch<7>(a, blocks, chunks, stream);
    default: return launch<8>(a, blocks, chunks, stream);
  }
}

}  // namespace engram
