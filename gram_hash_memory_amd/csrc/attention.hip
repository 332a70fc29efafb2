// Attention of one new token per sequence over the paged cache.
//
//   out = sum_p e^(scale q.k_p - m) v_p / sum_p e^(scale q.k_p - m),
//   m = max_p scale q.k_p,  lse = m + log sum_p e^(scale q.k_p - m)
//
// Bound by reading the seen keys and values once.  The query heads of one
// key-value head share a workgroup (up to 32 of them), so that each key and
// value is read once; a sequence's places are cut into chunks, a workgroup
// each, whose partial results a second kernel joins in the chunks' order.
//
// A wave takes 32 places at a time, straight from memory into registers:
//  - S^T = K Q^T by v_mfma_f32_16x16x32_bf16: the lane l of a 16-place tile
//    holds 16 bytes of place l % 16 per step, in any order of the dimensions
//    as long as q's is the same;
//  - a lane then has 8 scores of query head l % 16, so the running maximum
//    takes two exchanges between lanes and the sums none before the end;
//  - O^T = V^T P^T: those 8 scores are the lane's B operand as they stand
//    (places 4 g .. 4 g + 3 of either tile, g = l / 16), and its A operand
//    are the same 8 places' values of dimension base + w (l % 16) + n, for
//    n = 0 .. w - 1 in turn: a lane reads w neighbouring dimensions of each
//    of its 8 places, and an 8 x w transpose between its own registers (one
//    v_perm for two values) is all that V needs.
// No lane waits for another in the loop: waves run apart, and the next 32
// places are requested as soon as a register is free.
#include <algorithm>

#include "kv_cache.hpp"

namespace engram {
namespace {

using kvc::row_index;

constexpr int kTile = 32;                  // places a wave takes at a time
constexpr int kMaxChunk = 4096;            // places of a workgroup: their pages are held in LDS
constexpr int kMinPage = 8;
constexpr int kHeadBlock = 32;             // query heads of a workgroup
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// ---------------------------------------------------------------- the plan

// The grid is laid out for sequences of max_len places (the host does not know
// their lengths); workgroups past a sequence's end leave at once.
constexpr int64_t kWantedBlocks = 2048;
constexpr int64_t kMinChunk = 256;
constexpr int64_t kMaxSplits = 256;
constexpr int kSingleSpan = 512;

struct Plan {
  int head_blocks, chunk, splits, waves;   // chunk: a multiple of kTile * waves
};

inline int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

Plan plan_for(int n_seqs, int q_heads, int kv_heads, int head_dim, int span) {
  Plan p{};
  const int group = q_heads / kv_heads;
  p.head_blocks = (group + kHeadBlock - 1) / kHeadBlock;
  const int64_t pairs = int64_t(n_seqs) * kv_heads * p.head_blocks;
  if (span <= kSingleSpan) {
    // 8 waves where their results fit 56 KB of LDS for the join (and a wave 256 registers).
    p.waves = head_dim / 32 * std::min(16, group) <= 64 ? 8 : 4;
    p.chunk = int(round_up(std::max(span, 1), kTile * p.waves));
    p.splits = 1;
    return p;
  }
  p.waves = 4;
  const int64_t even = (int64_t(span) * pairs + kWantedBlocks - 1) / kWantedBlocks;
  const int64_t most = (int64_t(span) + kMaxSplits - 1) / kMaxSplits;
  p.chunk = int(std::min<int64_t>(
      kMaxChunk, round_up(std::max({even, most, kMinChunk}), kTile * p.waves)));
  p.splits = int((int64_t(span) + p.chunk - 1) / p.chunk);
  return p;
}

// The plan of a call: that of its window's places, in no more parts than the
// workspace (sized without the window) has room for.
Plan plan_for(const PagedAttention &a) {
  const int hkv = a.cache.kv_heads;
  const Plan whole = plan_for(a.n_seqs, a.q_heads, hkv, a.cache.head_dim, a.max_len);
  if (a.window <= 0 || int64_t(a.window) + kTile - 1 >= a.max_len) return whole;
  const int span = a.window + kTile - 1;   // the first place is rounded down to a tile
  Plan p = plan_for(a.n_seqs, a.q_heads, hkv, a.cache.head_dim, span);
  if (p.splits > whole.splits) {
    p.chunk = int(round_up((int64_t(span) + whole.splits - 1) / whole.splits, kTile * p.waves));
    p.splits = int((int64_t(span) + p.chunk - 1) / p.chunk);
  }
  return p;
}

// ---------------------------------------------------------------- the kernel

struct Split {
  float *o;                // [n_seqs * q_heads][splits][head_dim], relative to 2^m
  float2 *ml;              // [n_seqs * q_heads][splits]: m (of base 2), the sum
  int chunk, splits, head_blocks;
};

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

// Two e4m3fn codes times 2^e as a bf16 pair (exact: 4 bits of significand).
__device__ __forceinline__ uint32_t mx_pair(uint32_t codes, float scale, bool high) {
  return __builtin_bit_cast(
      uint32_t, high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(int(codes), scale, true)
                     : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(int(codes), scale, false));
}

__device__ __forceinline__ bf16x8 as_frag(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(bf16x8, u32x4{a, b, c, d});
}

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

// The places of a sequence that are seen.
struct Seen {
  int start, len;
};
__device__ __forceinline__ Seen seen_of(const PagedAttention &a, int64_t s) {
  const int64_t room = int64_t(a.table_width) << a.cache.page_shift;
  const int len = int(min(int64_t(min(max(a.lens[s], 0), a.max_len)), room));
  return {a.window > 0 ? max(0, len - a.window) : 0, len};
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

template <int kDb, bool kMx, int kHt, int kW>
__global__ __launch_bounds__(64 * kW, kDb * kHt > 8 ? 1 : 2) void paged_attention_kernel(
    PagedAttention a, Split sp) {
  constexpr int D = 32 * kDb, kRowBytes = kMx ? D : 2 * D, kAcc = D / 16;
  using P = Pieces<kDb>;
  __shared__ int64_t page_lds[kMaxChunk / kMinPage + 1];   // a page's first row, or -1
  __shared__ float2 ml_lds[kW][kHt][16];
  extern __shared__ f32x4 o_lds[];                         // [kW - 1][kAcc][4][heads of a tile]

  const CacheView &c = a.cache;
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t id = blockIdx.x;
  const int split = int(id % sp.splits);
  id /= sp.splits;
  const int hb = int(id % sp.head_blocks);
  id /= sp.head_blocks;
  const int kvh = int(id % c.kv_heads);
  const int64_t s = id / c.kv_heads;
  const int group = a.q_heads / c.kv_heads;
  const int heads = min(16 * kHt, group - hb * kHeadBlock);   // here; kHt = 1 only for up to 16
  const int64_t row0 = s * a.q_heads + kvh * group + hb * kHeadBlock;

  const Seen seen = seen_of(a, s);
  const int base = seen.start / kTile * kTile;
  const int64_t c0_wide = int64_t(base) + int64_t(split) * sp.chunk;
  if (c0_wide >= seen.len && sp.splits > 1) return;
  const int c0 = int(min(c0_wide, int64_t(seen.len)));
  const int c1 = int(min(int64_t(seen.len), int64_t(c0) + sp.chunk));
  const int tiles = (c1 - c0 + kTile - 1) / kTile;

  // The pages of these places.
  const int mask = (1 << c.page_shift) - 1;
  const int page0 = c0 >> c.page_shift;
  const int pages = tiles == 0 ? 0 : int((int64_t(c0) + tiles * kTile - 1) >> c.page_shift) - page0 + 1;
  bool bad = false;
  for (int e = threadIdx.x; e < pages; e += 64 * kW) {
    const int64_t first = int64_t(page0 + e) << c.page_shift;
    int64_t row = -1;
    if (first < c1 && first + mask >= seen.start) {
      const int page = a.table[s * a.table_width + page0 + e];
      if (page >= 0 && page < c.pages) row = (int64_t(page) * c.kv_heads + kvh) << c.page_shift;
      else bad = true;
    }
    page_lds[e] = row;
  }
  if (bad && kvh == 0 && hb == 0 && a.bad_pages) atomicAdd(a.bad_pages, 1);
  const bool any_bad = __syncthreads_or(bad);

  // Query heads as B operands: lane l holds 8 dimensions of head l % 16 a step.
  // In the 8-bit format a lane's 16 bytes of K are two steps.
  bf16x8 q[kHt][kDb];
#pragma unroll
  for (int t = 0; t < kHt; ++t)
#pragma unroll
    for (int kk = 0; kk < kDb; ++kk) {
      const int d = kMx && (kk | 1) < kDb ? 64 * (kk / 2) + 16 * g + 8 * (kk & 1) : 32 * kk + 8 * g;
      u32x4 v{};
      if (16 * t + col < heads)
        v = *reinterpret_cast<const u32x4 *>(a.q + (row0 + 16 * t + col) * D + d);
      q[t][kk] = __builtin_bit_cast(bf16x8, v);
    }

  Held<kDb, kMx> held;
  auto row_of = [&](int p) {
    const int64_t r = page_lds[(p >> c.page_shift) - page0];
    return (r < 0 ? 0 : r) + (p & mask);       // a page that is not seen: rows of page 0 instead
  };
  auto load_k = [&](int tile) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t row = row_of(c0 + kTile * tile + 16 * u + col);
      const uint8_t *src = static_cast<const uint8_t *>(c.k) + row * kRowBytes;
      if constexpr (!kMx) {
#pragma unroll
        for (int kk = 0; kk < kDb; ++kk) load_bytes<16>(&held.k[u][4 * kk], src + 64 * kk + 16 * g);
      } else {
        const uint8_t *sc = c.k_scales + row * kDb;
#pragma unroll
        for (int j = 0; j < kDb / 2; ++j) {
          load_bytes<16>(&held.k[u][4 * j], src + 64 * j + 16 * g);
          held.ks[u][j] = sc[2 * j + (g >> 1)];
        }
        if constexpr (kDb % 2) {
          load_bytes<8>(&held.k[u][2 * (kDb - 1)], src + 32 * (kDb - 1) + 8 * g);
          held.ks[u][kDb / 2] = sc[kDb - 1];
        }
      }
    }
  };
  auto load_v = [&](int tile) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t row = row_of(c0 + kTile * tile + 16 * u + 4 * g);
      const uint8_t *src = static_cast<const uint8_t *>(c.v) + row * kRowBytes;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        each_piece<P::kN>([&](auto piece) {
          constexpr int w = P::width(piece.value), first = P::base(piece.value);
          if constexpr (kMx) {
            load_bytes<w>(&held.v[4 * u + j][first / 64], src + j * kRowBytes + first + w * col);
            held.vs[4 * u + j][piece.value] = c.v_scales[(row + j) * kDb + (first + w * col) / 32];
          } else {
            load_bytes<2 * w>(&held.v[4 * u + j][first / 32],
                              src + j * kRowBytes + 2 * (first + w * col));
          }
        });
      }
    }
  };

  const float to_log2 = a.scale * kLog2e;
  float m[kHt], l[kHt];
  f32x4 o[kHt][kAcc];
#pragma unroll
  for (int t = 0; t < kHt; ++t) {
    m[t] = -INFINITY, l[t] = 0.0f;
#pragma unroll
    for (int n = 0; n < kAcc; ++n) o[t][n] = f32x4{};
  }

  int tile = wave;
  if (tile < tiles) {
    load_k(tile);
    load_v(tile);
  }
  while (tile < tiles) {
    const int p0 = c0 + kTile * tile;
    f32x4 z[kHt][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int t = 0; t < kHt; ++t) z[t][u] = f32x4{};
#pragma unroll
      for (int kk = 0; kk < kDb; ++kk) {
        bf16x8 f;
        if constexpr (kMx) {
          const uint32_t *w = &held.k[u][2 * kk];
          const float sc = __uint_as_float(held.ks[u][kk / 2] << 23);
          f = as_frag(mx_pair(w[0], sc, false), mx_pair(w[0], sc, true), mx_pair(w[1], sc, false),
                      mx_pair(w[1], sc, true));
        } else {
          const uint32_t *w = &held.k[u][4 * kk];
          f = as_frag(w[0], w[1], w[2], w[3]);
        }
#pragma unroll
        for (int t = 0; t < kHt; ++t)
          z[t][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, q[t][kk], z[t][u], 0, 0, 0);
      }
    }
    const int next = tile + kW;
    load_k(min(next, tiles - 1));              // the last time for nothing, from the cache

    // Bits 4 u + r: place 16 u + 4 g + r of the tile is seen.
    const bool whole = !any_bad && p0 >= seen.start && p0 + kTile <= seen.len;
    uint32_t shown = 0xFF;
    if (!whole) {
      shown = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int p = p0 + 16 * u + 4 * g;
        const bool page = page_lds[(p >> c.page_shift) - page0] >= 0;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (page && p + r >= seen.start && p + r < seen.len) shown |= 1u << (4 * u + r);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!(shown >> j & 1)) {
#pragma unroll
          for (int i = 0; i < int(sizeof(held.v[0]) / 4); ++i) held.v[j][i] = 0;
#pragma unroll
          for (int i = 0; i < P::kN; ++i) held.vs[j][i] = 127;
        }
    }

    bf16x8 w[kHt];                             // the weights, as B operands
#pragma unroll
    for (int t = 0; t < kHt; ++t) {
      float e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = z[t][j / 4][j % 4] * to_log2;
      if (!whole) {
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = shown >> j & 1 ? e[j] : -INFINITY;
      }
      float top = e[0];
#pragma unroll
      for (int j = 1; j < 8; ++j) top = fmaxf(top, e[j]);
      top = column_max(top);
      if (__any(top > m[t])) {                 // rarely after the first tiles
        const float mn = fmaxf(m[t], top);
        const float keep = mn == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m[t] - mn);
        m[t] = mn;
        l[t] *= keep;
#pragma unroll
        for (int n = 0; n < kAcc; ++n) o[t][n] *= keep;
      }
      const float ms = m[t] == -INFINITY ? 0.0f : m[t];
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        e[j] = __builtin_amdgcn_exp2f(e[j] - ms);
        sum += e[j];
      }
      l[t] += sum;
      // Rounded to bf16 for the matrix cores; the sum is of the fp32 ones.
      w[t] = as_frag(pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]), pack_bf16x2(e[4], e[5]),
                     pack_bf16x2(e[6], e[7]));
    }

    each_piece<P::kN>([&](auto piece) {
      constexpr int wd = P::width(piece.value), first = P::base(piece.value);
#pragma unroll
      for (int i = 0; i < wd / 2; ++i) {
        uint32_t x[8];                   // dimensions 2 i, 2 i + 1 of the lane's 8 places
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if constexpr (kMx)
            x[j] = mx_pair(held.v[j][first / 64 + i / 2],
                           __uint_as_float(held.vs[j][piece.value] << 23), i & 1);
          else
            x[j] = held.v[j][first / 32 + i];
        }
        const bf16x8 even = as_frag(__builtin_amdgcn_perm(x[1], x[0], 0x05040100u),
                                    __builtin_amdgcn_perm(x[3], x[2], 0x05040100u),
                                    __builtin_amdgcn_perm(x[5], x[4], 0x05040100u),
                                    __builtin_amdgcn_perm(x[7], x[6], 0x05040100u));
        const bf16x8 odd = as_frag(__builtin_amdgcn_perm(x[1], x[0], 0x07060302u),
                                   __builtin_amdgcn_perm(x[3], x[2], 0x07060302u),
                                   __builtin_amdgcn_perm(x[5], x[4], 0x07060302u),
                                   __builtin_amdgcn_perm(x[7], x[6], 0x07060302u));
        const int n = first / 16 + 2 * i;
#pragma unroll
        for (int t = 0; t < kHt; ++t) {
          o[t][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(even, w[t], o[t][n], 0, 0, 0);
          o[t][n + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(odd, w[t], o[t][n + 1], 0, 0, 0);
        }
      }
    });
    tile = next;
    if (tile < tiles) load_v(tile);
  }

  // The waves' results joined by wave 0, in wave order.
#pragma unroll
  for (int t = 0; t < kHt; ++t) {
    l[t] = column_sum(l[t]);
    if (g == 0) ml_lds[wave][t][col] = float2{m[t], l[t]};
  }
#pragma unroll
  for (int t = 0; t < kHt; ++t) {
    const int here = min(16, heads - 16 * t);
    if (here <= 0) break;
    const bool on = col < here;
    if (t > 0) __syncthreads();
    if (wave > 0 && on) {
#pragma unroll
      for (int n = 0; n < kAcc; ++n)
        o_lds[((wave - 1) * kAcc + n) * 4 * here + g * here + col] = o[t][n];
    }
    __syncthreads();
    if (wave > 0 || !on) continue;
    float top = m[t];
#pragma unroll
    for (int x = 1; x < kW; ++x) top = fmaxf(top, ml_lds[x][t][col].x);
    const float ms = top == -INFINITY ? 0.0f : top;
    float keep = __builtin_amdgcn_exp2f(m[t] - ms), sum = l[t] * keep;
#pragma unroll
    for (int n = 0; n < kAcc; ++n) o[t][n] *= keep;
#pragma unroll 1
    for (int x = 1; x < kW; ++x) {
      const float2 ml = ml_lds[x][t][col];
      keep = __builtin_amdgcn_exp2f(ml.x - ms);
      sum += ml.y * keep;
#pragma unroll
      for (int n = 0; n < kAcc; ++n)
        o[t][n] += o_lds[((x - 1) * kAcc + n) * 4 * here + g * here + col] * keep;
    }
    const int64_t row = row0 + 16 * t + col;
    const bool last = sp.splits == 1;
    const float inv = !last ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
    if (g == 0) {
      if (!last) sp.ml[row * sp.splits + split] = float2{top, sum};
      else if (a.lse) a.lse[row] = sum == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
    }
    each_piece<P::kN>([&](auto piece) {
      constexpr int wd = P::width(piece.value), first = P::base(piece.value);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = first + wd * (4 * g + r);
        if (last) {
          uint16_t *dst = a.out + row * D + d;
#pragma unroll
          for (int i = 0; i < wd / 2; ++i)
            reinterpret_cast<uint32_t *>(dst)[i] = pack_bf16x2(
                o[t][first / 16 + 2 * i][r] * inv, o[t][first / 16 + 2 * i + 1][r] * inv);
        } else {
          float *dst = sp.o + (row * sp.splits + split) * D + d;
#pragma unroll
          for (int i = 0; i < wd; ++i) dst[i] = o[t][first / 16 + i][r];
        }
      }
    });
  }
}

// The parts of a sequence's chunks to its result, in the chunks' order: one
// workgroup per (sequence, query head), D / 4 lanes a part.
constexpr int kJoinThreads = 256;
__global__ __launch_bounds__(kJoinThreads) void join_kernel(PagedAttention a, Split sp) {
  __shared__ f32x4 part_lds[kJoinThreads];
  __shared__ float top_lds[kJoinThreads / 64], sum_lds[kJoinThreads / 64];
  const int D = a.cache.head_dim, lanes = D / 4;
  const int64_t row = blockIdx.x;
  const Seen seen = seen_of(a, row / a.q_heads);
  const int base = seen.start / kTile * kTile;
  const int parts = int((int64_t(seen.len) - base + sp.chunk - 1) / sp.chunk);
  const float2 *ml = sp.ml + row * sp.splits;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float top = -INFINITY;
  for (int i = threadIdx.x; i < parts; i += kJoinThreads) top = fmaxf(top, ml[i].x);
  for (int x = 1; x < 64; x *= 2) top = fmaxf(top, __shfl_xor(top, x));
  if (lane == 0) top_lds[wave] = top;
  __syncthreads();
  for (int w = 0; w < kJoinThreads / 64; ++w) top = fmaxf(top, top_lds[w]);
  const float ms = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f;
  for (int i = threadIdx.x; i < parts; i += kJoinThreads)
    sum += ml[i].y * __builtin_amdgcn_exp2f(ml[i].x - ms);
  for (int x = 1; x < 64; x *= 2) sum += __shfl_xor(sum, x);
  if (lane == 0) sum_lds[wave] = sum;

  const int rows = kJoinThreads / lanes, mine = threadIdx.x / lanes, at = threadIdx.x % lanes;
  f32x4 o{};
  if (mine < rows) {
    const f32x4 *src = reinterpret_cast<const f32x4 *>(sp.o + row * sp.splits * D) + at;
    for (int i = mine; i < parts; i += rows) o += src[int64_t(i) * lanes] * __builtin_amdgcn_exp2f(ml[i].x - ms);
    part_lds[threadIdx.x] = o;
  }
  __syncthreads();
  sum = 0.0f;
  for (int w = 0; w < kJoinThreads / 64; ++w) sum += sum_lds[w];
  if (threadIdx.x == 0 && a.lse)
    a.lse[row] = sum == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
  if (mine != 0) return;
  for (int w = 1; w < rows; ++w) o += part_lds[w * lanes + at];
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  reinterpret_cast<u32x2 *>(a.out + row * D)[at] =
      u32x2{pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv)};
}

template <int kDb, bool kMx, int kHt, int kW>
hipError_t launch(const PagedAttention &a, const Plan &p, const Split &sp, hipStream_t stream) {
  const int group = a.q_heads / a.cache.kv_heads;
  const unsigned lds = unsigned((kW - 1) * (2 * kDb) * 4 * std::min(16, group) * sizeof(f32x4));
  const int64_t blocks = int64_t(a.n_seqs) * a.cache.kv_heads * p.head_blocks * p.splits;
  hipLaunchKernelGGL((paged_attention_kernel<kDb, kMx, kHt, kW>), dim3(unsigned(blocks)),
                     dim3(64 * kW), lds, stream, a, sp);
  return hipGetLastError();
}

template <int kDb, bool kMx>
hipError_t by_heads(const PagedAttention &a, const Plan &p, const Split &sp, hipStream_t stream) {
  const bool two = a.q_heads / a.cache.kv_heads > 16;
  if (p.waves == 8) {
    if constexpr (kDb <= 4)
      if (two) return launch<kDb, kMx, 2, 8>(a, p, sp, stream);
    return launch<kDb, kMx, 1, 8>(a, p, sp, stream);
  }
  return two ? launch<kDb, kMx, 2, 4>(a, p, sp, stream) : launch<kDb, kMx, 1, 4>(a, p, sp, stream);
}

template <int kDb>
hipError_t by_format(const PagedAttention &a, const Plan &p, const Split &sp, hipStream_t stream) {
  return a.cache.k_scales ? by_heads<kDb, true>(a, p, sp, stream)
                          : by_heads<kDb, false>(a, p, sp, stream);
}

}  // namespace

int64_t paged_attention_workspace(int32_t n_seqs, int32_t q_heads, int32_t kv_heads,
                                  int32_t head_dim, int32_t max_len) {
  const Plan p = plan_for(n_seqs, q_heads, kv_heads, head_dim, max_len);
  if (p.splits == 1) return 0;
  return int64_t(n_seqs) * q_heads * p.splits * (head_dim + 2) * int64_t(sizeof(float));
}

int64_t paged_attention_blocks(const PagedAttention &a) {
  const Plan p = plan_for(a);
  return std::max(int64_t(a.n_seqs) * a.cache.kv_heads * p.head_blocks * p.splits,
                  int64_t(a.n_seqs) * a.q_heads);
}

hipError_t launch_paged_attention(const PagedAttention &a, hipStream_t stream) {
  const Plan p = plan_for(a);
  const int64_t parts = int64_t(a.n_seqs) * a.q_heads * p.splits;
  float *ws = static_cast<float *>(a.workspace);
  const Split sp{ws, reinterpret_cast<float2 *>(ws + parts * a.cache.head_dim), p.chunk, p.splits,
                 p.head_blocks};
  hipError_t err;
  switch (a.cache.head_dim / 32) {
    case 1: err = by_format<1>(a, p, sp, stream); break;
    case 2: err = by_format<2>(a, p, sp, stream); break;
    case 3: err = by_format<3>(a, p, sp, stream); break;
    case 4: err = by_format<4>(a, p, sp, stream); break;
    case 5: err = by_format<5>(a, p, sp, stream); break;
    case 6: err = by_format<6>(a, p, sp, stream); break;
    case 7: err = by_format<7>(a, p, sp, stream); break;
    default: err = by_format<8>(a, p, sp, stream);
  }
  if (err != hipSuccess || p.splits == 1) return err;
  hipLaunchKernelGGL(join_kernel, dim3(unsigned(int64_t(a.n_seqs) * a.q_heads)),
                     dim3(kJoinThreads), 0, stream, a, sp);
  return hipGetLastError();
}

}  // namespace engram
