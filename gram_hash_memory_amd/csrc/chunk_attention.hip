// Attention of several query rows a key-value head over the paged cache: the new
// tokens of a chunk (causal, with windows, prefixes, documents, capped scores and
// a distance bias), and the sequences that share a prefix.
//
//   z = scale q.k;  z = cap tanh(z / cap);  z -= slope |pos - p|
//   out = sum_p e^(z_p - m) v_p / sum_p e^(z_p - m),  lse = m + log sum_p e^(z_p - m)
//
// The rows of one key-value head (token-major, the heads of its group inside) are
// cut into blocks of 32 kW, a wave taking 32 of them; a workgroup takes a block
// through the places that any of its rows sees, 64 at a time:
//  - keys and values go from memory to registers one tile ahead, are converted
//    there, and put into one of two LDS buffers; rows are padded so that no two
//    lanes of a read share a bank;
//  - S^T = K Q^T by v_mfma_f32_32x32x16_bf16: a lane then has 32 scores of one
//    query row, so the running maximum takes one exchange between lanes;
//  - O^T = V^T P^T: the scores' registers are the P^T operand as they stand, with
//    the places in an order that V's transposing LDS reads follow.
// plan_kernel lists the blocks first; the workgroups take whole blocks off a queue
// or, where those are too few to fill the GPU, equal runs of all tiles, whose parts
// join_kernel adds in order.
#include <algorithm>

#include "attention_common.hpp"
#include "tile_plan.hpp"

namespace engram {
namespace {

using namespace attn;

constexpr int kRows = 32;                  // query rows of a wave
constexpr int kWholeTiles = 8;             // contexts that are never cut
constexpr int kJoinTiles = 4;              // what a join takes, in tiles

inline int64_t ceil_div(int64_t x, int64_t by) { return (x + by - 1) / by; }

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Over lanes l and l ^ 32, which hold one query row.
__device__ __forceinline__ float pair_max(float x) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float pair_sum(float x) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// 4 places' values of one dimension a lane: lanes 4 r .. 4 r + 3 of 16 address 4
// dimensions each of place r, and lane i gets dimension i of the four.
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x2 read_transposed(const uint8_t *p) {
  typedef __attribute__((address_space(3))) s16x4 *Lds;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p)));
}

// A tile in LDS: keys in rows of 2 D + 16 bytes (16 places at one piece of 16 bytes
// lie in different banks), values in rows of 64 bytes or 192 past a multiple of 256
// (so do 4 places' 64 bytes, which half a wave's transposing read takes at once).
template <int kDb>
struct Stage {
  static constexpr int kKeyRow = 64 * kDb + 16;
  static constexpr int kValueRow = 64 * kDb + (kDb % 2 ? 0 : 64);
  static constexpr int kValues = kTile * kKeyRow;
  static constexpr int kBytes = kTile * (kKeyRow + kValueRow);
};

template <bool kMx>
__device__ __forceinline__ float cache_value(const CacheView &c, const void *data, const uint8_t *scales,
                                             int64_t place, int d) {
  if constexpr (!kMx) return bf16_lo(static_cast<const uint16_t *>(data)[place * c.head_dim + d]);
  return e4m3fn_to_float(static_cast<const uint8_t *>(data)[place * c.head_dim + d]) *
         e8m0_to_float(min(uint32_t(scales[place * (c.head_dim / 32) + d / 32]), 254u));
}

template <int kDb, bool kMx, int kW>
__global__ __launch_bounds__(64 * kW, kDb <= 4 ? 2 : 1) void tile_attention_kernel(
    TileAttention a, TilePlan plan) {
  constexpr int D = 32 * kDb, kThreads = 64 * kW, kBlock = kRows * kW;
  constexpr int kRowBytes = kMx ? D : 2 * D;
  constexpr int kPieces = kRowBytes / 16, kLoads = (kTile * kPieces + kThreads - 1) / kThreads;
  using S = Stage<kDb>;
  extern __shared__ u32x4 stages_lds[];      // [2] stages
  uint8_t *const lds = reinterpret_cast<uint8_t *>(stages_lds);
  // Of the tiles in flight, by tile % 3: places on pages outside the cache, and
  // places whose values are not all finite.
  __shared__ uint32_t absent_lds[3][2], odd_lds[3][2];
  __shared__ int4 limits_lds[kW];
  __shared__ int work_lds[2];

  const CacheView &c = a.cache;
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int group = a.q_heads / c.kv_heads;
  const int mask = (1 << c.page_shift) - 1;
  // Scores in units of log 2.  A negative scale goes into the queries' signs.
  const float unit = (a.rules.cap > 0.0f ? fabsf(a.scale) / a.rules.cap : fabsf(a.scale) * kLog2e);
  const float cap2 = a.rules.cap * kLog2e;
  const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;

  const TileHeader head = *plan.header;
  const int runs = gridDim.x;
  int run = blockIdx.x, left = 0, block = 0, unit_at = 0, kvh = 0, piece = -1;
  if (!head.direct) {
    const int per_xcd = runs / 8;            // neighbouring runs share keys: one XCD
    if (runs % 8 == 0) run = run % 8 * per_xcd + run / 8;
    const int64_t total = int64_t(head.units) * c.kv_heads;
    const int64_t u0 = int64_t(run) * head.per;
    if (u0 >= total) return;
    left = int(min(int64_t(head.per), total - u0));
    kvh = int(u0 / head.units);
    const int local = int(u0 - int64_t(kvh) * head.units);
    for (int b = tid; b < head.blocks; b += kThreads) {
      const int at = local - plan.blocks[b].before;
      if (at >= 0 && at < plan.blocks[b].a_n + plan.blocks[b].b_n) work_lds[0] = b, work_lds[1] = at;
    }
    __syncthreads();
    block = __builtin_amdgcn_readfirstlane(work_lds[0]);
    unit_at = __builtin_amdgcn_readfirstlane(work_lds[1]);
    __syncthreads();
  }

  for (;;) {
    int count;                               // tiles of this piece
    bool whole = true;
    if (head.direct) {
      if (tid == 0) work_lds[0] = atomicAdd(plan.queue, 1);
      __syncthreads();
      const int at = __builtin_amdgcn_readfirstlane(work_lds[0]);
      if (at >= head.blocks * c.kv_heads) break;
      block = head.blocks - 1 - at / c.kv_heads;
      kvh = at % c.kv_heads;
      unit_at = 0;
    }
    const TileBlock w = plan.blocks[block];
    const int units = w.a_n + w.b_n;
    count = units;
    if (units == 0) {                        // no places of its own
      if (!head.direct && ++block == head.blocks) block = 0, ++kvh;
      __syncthreads();
      continue;
    }
    if (!head.direct) {
      count = min(units - unit_at, left);
      whole = count == units;
    }
    ++piece;
    const bool shared = w.kind == kSharedPrefix;
    const int32_t *table = shared ? a.prefix_table + int64_t(w.seq) * a.prefix_width
                                  : a.table + int64_t(w.seq) * a.table_width;

    // This lane's query row, and what it sees.
    const int row = wave * kRows + col;
    const bool live = row < w.rows;
    const int in_problem = w.row0 + min(row, w.rows - 1);
    const int tok = in_problem / group, token = w.token0 + tok;
    const int q_head = kvh * group + in_problem - tok * group;
    const int64_t q_row = int64_t(token) * a.q_heads + q_head;
    RowSees r{0, w.len, 0, 0};
    const int pos = w.first + tok;
    if (w.kind == kChunk) r = row_sees(a.rules, w.seq, token, pos, w.len);
    const float slope = w.kind == kChunk && a.rules.slopes ? a.rules.slopes[q_head] * kLog2e : 0.0f;
    // A tile that all rows of a wave, or of the block, see needs no masks.
    int4 lim = {r.lo, r.lo + r.n, r.first, r.first + r.m};
#pragma unroll
    for (int x = 1; x < 32; x *= 2) {
      lim.x = max(lim.x, __shfl_xor(lim.x, x));
      lim.y = min(lim.y, __shfl_xor(lim.y, x));
      lim.z = max(lim.z, __shfl_xor(lim.z, x));
      lim.w = min(lim.w, __shfl_xor(lim.w, x));
    }
    if (lane == 0) limits_lds[wave] = lim;
    if (tid < 6) absent_lds[tid / 2][tid % 2] = odd_lds[tid / 2][tid % 2] = 0;

    bf16x8 q[2 * kDb];
#pragma unroll
    for (int kk = 0; kk < 2 * kDb; ++kk) {
      u32x4 v = *reinterpret_cast<const u32x4 *>(a.q + q_row * D + 16 * kk + 8 * half);
      v ^= u32x4{flip, flip, flip, flip};
      q[kk] = __builtin_bit_cast(bf16x8, v);
    }
    const bool active = wave * kRows < w.rows;
    __syncthreads();
    int4 all = limits_lds[0];
#pragma unroll
    for (int x = 1; x < kW; ++x) {
      const int4 y = limits_lds[x];
      all = {max(all.x, y.x), min(all.y, y.y), max(all.z, y.z), min(all.w, y.w)};
    }

    auto place_of = [&](int t) {             // the first place of the block's tile t
      return (t < w.a_n ? w.a_tile + t : w.b_tile + t - w.a_n) * kTile;
    };
    auto plain = [&](const int4 &l, int p0) {
      return (p0 >= l.x && p0 + kTile <= l.y) || (p0 >= l.z && p0 + kTile <= l.w);
    };

    auto used = [&](int p) {                 // by any row of the block
      return unsigned(p - w.b_lo) < unsigned(w.b_hi - w.b_lo) ||
             unsigned(p - w.a_lo) < unsigned(w.a_hi - w.a_lo);
    };

    // A thread's pieces of a tile: their pages, requested two tiles ahead, and
    // their 16 bytes of keys and of values, one tile ahead.
    int page[kLoads];
    u32x4 key[kLoads], value[kLoads];
    uint32_t scales[kLoads];                 // the key's and the value's byte (8-bit format)
    uint32_t shown = 0;                      // bit i: piece i is of a place that is used, on a page
    uint32_t missing = 0;                    // ... on no page of the cache
    auto ask_pages = [&](int t) {
      const int p0 = place_of(t);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int p = p0 + (tid + i * kThreads) / kPieces;
        page[i] = w.len > 0 ? table[min(p, w.len - 1) >> c.page_shift] : -1;
      }
    };
    auto load = [&](int t) {
      const int p0 = place_of(t);
      shown = missing = 0;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int id = tid + i * kThreads, p = p0 + id / kPieces, at = id % kPieces;
        const bool in_tile = kTile * kPieces % kThreads == 0 || id < kTile * kPieces;
        const bool in = in_tile && used(p), there = unsigned(page[i]) < unsigned(c.pages);
        shown |= (in && there ? 1u : 0u) << i;
        missing |= (in && !there ? 1u : 0u) << i;
        // What is not there is read from the cache's first row instead, and not used.
        const int64_t place = in && there
            ? ((int64_t(page[i]) * c.kv_heads + kvh) << c.page_shift) + (p & mask) : 0;
        key[i] = *reinterpret_cast<const u32x4 *>(static_cast<const uint8_t *>(c.k) + place * kRowBytes + 16 * at);
        value[i] = *reinterpret_cast<const u32x4 *>(static_cast<const uint8_t *>(c.v) + place * kRowBytes + 16 * at);
        if constexpr (kMx)
          scales[i] = c.k_scales[place * kDb + at / 2] | uint32_t(c.v_scales[place * kDb + at / 2]) << 8;
      }
    };
    auto put = [&](int t, int buf, bool edge) {
      uint8_t *const st = lds + buf * S::kBytes;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int id = tid + i * kThreads, in_tile = id / kPieces, at = id % kPieces;
        if (kTile * kPieces % kThreads != 0 && id >= kTile * kPieces) break;
        constexpr int kOut = kMx ? 2 : 1;    // pieces of 8 values
        u32x4 k[kOut], v[kOut];
        if constexpr (kMx) {
          const float ks = e8m0_to_float(scales[i] & 255u);
          const float vs = e8m0_to_float(min(scales[i] >> 8, 254u));
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            k[x / 4][x % 4] = mx_pair(key[i][x / 2], ks, x & 1);
            v[x / 4][x % 4] = mx_pair(value[i][x / 2], vs, x & 1);
          }
        } else {
          k[0] = key[i], v[0] = value[i];
        }
        if (edge || missing) {
          const bool keep = shown >> i & 1;
          bool finite = true;
#pragma unroll
          for (int o = 0; o < kOut; ++o) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              k[o][x] = keep ? k[o][x] : 0u;
              v[o][x] = keep ? v[o][x] : 0u;
              finite = finite && (v[o][x] & 0x7F80u) != 0x7F80u &&
                       (v[o][x] & 0x7F800000u) != 0x7F800000u;
            }
          }
          // A weight of 0 times a value that is not finite would reach rows that do
          // not see it: it counts as 0 here, and add_odd() gives it to those that do.
          if (!finite) {
            atomicOr(&odd_lds[t % 3][in_tile / 32], 1u << (in_tile & 31));
#pragma unroll
            for (int o = 0; o < kOut; ++o)
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                if ((v[o][x] & 0x7F80u) == 0x7F80u) v[o][x] &= 0xFFFF0000u;
                if ((v[o][x] & 0x7F800000u) == 0x7F800000u) v[o][x] &= 0xFFFFu;
              }
          }
          if (missing >> i & 1) {
            atomicOr(&absent_lds[t % 3][in_tile / 32], 1u << (in_tile & 31));
            if (at == 0 && kvh == 0 && a.bad_pages) atomicAdd(a.bad_pages, 1);
          }
        }
#pragma unroll
        for (int o = 0; o < kOut; ++o) {
          *reinterpret_cast<u32x4 *>(st + in_tile * S::kKeyRow + (kOut * at + o) * 16) = k[o];
          *reinterpret_cast<u32x4 *>(st + S::kValues + in_tile * S::kValueRow + (kOut * at + o) * 16) = v[o];
        }
      }
    };

    float m = -INFINITY, l = 0.0f;           // l: of this lane's places
    f32x16 o[kDb];
#pragma unroll
    for (int n = 0; n < kDb; ++n) o[n] = f32x16{};

    const int t1 = unit_at + count;
    ask_pages(unit_at);
    load(unit_at);
    ask_pages(min(unit_at + 1, t1 - 1));
    put(unit_at, 0, !plain(all, place_of(unit_at)));
    __syncthreads();

    for (int t = unit_at, buf = 0; t < t1; ++t, buf ^= 1) {
      const int p0 = place_of(t);
      if (t + 1 < t1) {
        load(t + 1);
        ask_pages(min(t + 2, t1 - 1));
      }
      // (tile + 2) % 3 was read before the last barrier, and is written after the next.
      if (tid < 2) absent_lds[(t + 2) % 3][tid] = odd_lds[(t + 2) % 3][tid] = 0;
      const uint8_t *const st = lds + buf * S::kBytes;
      const uint32_t absent[2] = {absent_lds[t % 3][0], absent_lds[t % 3][1]};
      const uint32_t odd[2] = {odd_lds[t % 3][0], odd_lds[t % 3][1]};
      const bool any_absent = __builtin_amdgcn_readfirstlane(absent[0] | absent[1]) != 0;
      const bool any_odd = __builtin_amdgcn_readfirstlane(odd[0] | odd[1]) != 0;

      if (active) {
        f32x16 z[2] = {};
#pragma unroll
        for (int kk = 0; kk < 2 * kDb; ++kk)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const u32x4 f = *reinterpret_cast<const u32x4 *>(st + (32 * u + col) * S::kKeyRow + 32 * kk + 16 * half);
            z[u] = mfma32(__builtin_bit_cast(bf16x8, f), q[kk], z[u]);
          }
        // Register 4 i + j of tile half u: place 32 u + 8 i + 4 half + j.
        const bool masked = !plain(lim, p0) || any_absent;
        if (a.rules.cap > 0.0f) {
          float far = 0.0f;
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            z[x / 16][x % 16] *= unit;
            far = fmaxf(far, fabsf(z[x / 16][x % 16]));
          }
          if (__any(!(far <= kTanhSplit))) {
#pragma unroll
            for (int x = 0; x < 32; ++x) {
              const float y = z[x / 16][x % 16];
              z[x / 16][x % 16] = cap2 * (fabsf(y) <= kTanhSplit ? tanh_small(y) : tanh_large(y));
            }
          } else {
#pragma unroll
            for (int x = 0; x < 32; ++x) z[x / 16][x % 16] = cap2 * tanh_small(z[x / 16][x % 16]);
          }
        } else {
#pragma unroll
          for (int x = 0; x < 32; ++x) z[x / 16][x % 16] *= unit;
        }
        if (w.kind == kChunk && a.rules.slopes) {
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            const int p = p0 + 32 * (x / 16) + 8 * (x % 16 / 4) + 4 * half + x % 4;
            z[x / 16][x % 16] = __builtin_fmaf(-slope, float(abs(pos - p)), z[x / 16][x % 16]);
          }
        }
        if (masked) {
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            const int in_half = 8 * (x % 16 / 4) + 4 * half + x % 4;
            const bool ok = sees(r, p0 + 32 * (x / 16) + in_half) && !(absent[x / 16] >> in_half & 1);
            z[x / 16][x % 16] = ok ? z[x / 16][x % 16] : -INFINITY;
          }
        }
        float top = z[0][0];
#pragma unroll
        for (int x = 1; x < 32; ++x) top = fmaxf(top, z[x / 16][x % 16]);
        top = pair_max(top);
        if (__any(top > m)) {
          const float mn = fmaxf(m, top);
          const float keep = mn == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
          m = mn;
          l *= keep;
#pragma unroll
          for (int n = 0; n < kDb; ++n) o[n] *= keep;
        }
        const float ms = m == -INFINITY ? 0.0f : m;
        float sum[2] = {};
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          z[x / 16][x % 16] = __builtin_amdgcn_exp2f(z[x / 16][x % 16] - ms);
          sum[x / 16] += z[x / 16][x % 16];
        }
        l += sum[0] + sum[1];
        const uint8_t *const vp = st + S::kValues + (4 * half + lane % 16 / 4) * S::kValueRow +
                                  32 * (lane / 16 % 2) + 8 * (lane % 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x16 &e = z[j / 2];
          const int x = 8 * (j % 2);
          const bf16x8 p = as_frag(pack_bf16x2(e[x], e[x + 1]), pack_bf16x2(e[x + 2], e[x + 3]),
                                   pack_bf16x2(e[x + 4], e[x + 5]), pack_bf16x2(e[x + 6], e[x + 7]));
#pragma unroll
          for (int n = 0; n < kDb; ++n) {
            const u32x2 lo = read_transposed(vp + 16 * j * S::kValueRow + 64 * n);
            const u32x2 hi = read_transposed(vp + (16 * j + 8) * S::kValueRow + 64 * n);
            o[n] = mfma32(as_frag(lo[0], lo[1], hi[0], hi[1]), p, o[n]);
          }
        }
        if (any_odd) {                       // values that are not finite, to the rows that see them
          for (int i = 0; i < kTile; ++i) {
            if (!(__builtin_amdgcn_readfirstlane(odd[i / 32]) >> (i & 31) & 1)) continue;
            float e = 0.0f;                  // the weight, in the half that holds it
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (x == i / 32 * 16 + (i & 31) / 8 * 4 + i % 4) e = z[x / 16][x % 16];
            e = __shfl(e, col + 32 * (i / 4 & 1));
            const int p = p0 + i;
            const int pg = table[p >> c.page_shift];
            const int64_t place = ((int64_t(pg) * c.kv_heads + kvh) << c.page_shift) + (p & mask);
            const bool ok = sees(r, p);
#pragma unroll
            for (int n = 0; n < kDb; ++n)
#pragma unroll
              for (int x = 0; x < 16; ++x) {
                const float v = cache_value<kMx>(c, c.v, c.v_scales, place, 32 * n + 8 * (x / 4) + 4 * half + x % 4);
                if (ok && !(fabsf(v) < INFINITY)) o[n][x] += e * v;
              }
          }
        }
      }
      if (t + 1 < t1) put(t + 1, buf ^ 1, !plain(all, place_of(t + 1)));
      __syncthreads();
    }

    // Lane: row col, dimensions 32 n + 8 i + 4 half + 0 .. 3.
    if (active) {
      l = pair_sum(l);
      if (whole && plan.whole_rows == 0) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        if (live) {
          if (a.lse && half == 0)
            a.lse[q_row] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
          uint16_t *const dst = a.out + q_row * D + 4 * half;
#pragma unroll
          for (int n = 0; n < kDb; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<u32x2 *>(dst + 32 * n + 8 * i) =
                  u32x2{pack_bf16x2(o[n][4 * i] * inv, o[n][4 * i + 1] * inv),
                        pack_bf16x2(o[n][4 * i + 2] * inv, o[n][4 * i + 3] * inv)};
        }
      } else if (live) {
        // A run's first piece, or a later one; or, whole, the row's own place.
        const int64_t at = whole ? (shared ? int64_t(a.T) * a.q_heads : 0) + q_row
                                 : plan.part_row(run, piece > 0, kBlock, row);
        if (half == 0) plan.ml[at] = float2{m, l};
        float *const dst = plan.o + at * D + 4 * half;
#pragma unroll
        for (int n = 0; n < kDb; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<f32x4 *>(dst + 32 * n + 8 * i) =
                f32x4{o[n][4 * i], o[n][4 * i + 1], o[n][4 * i + 2], o[n][4 * i + 3]};
      }
    }
    if (!head.direct) {
      left -= count;
      if (left == 0) break;
      unit_at = 0;
      if (++block == head.blocks) block = 0, ++kvh;
    }
  }
}

// ---------------------------------------------------------------- the plan

constexpr int kPlanThreads = 1024;

// The sum of x over the threads before this one; *total: over all of them.
__device__ __forceinline__ int scan_before(int x, int *total) {
  __shared__ int wave_lds[kPlanThreads / 64];
  int upto = x;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int y = __shfl_up(upto, d);
    if (int(threadIdx.x & 63) >= d) upto += y;
  }
  __syncthreads();                           // wave_lds may still be read
  if ((threadIdx.x & 63) == 63) wave_lds[threadIdx.x >> 6] = upto;
  __syncthreads();
  int sum = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    if (w == int(threadIdx.x >> 6)) upto += sum;
    sum += wave_lds[w];
  }
  *total = sum;
  return upto - x;
}

__device__ __forceinline__ int64_t max_all(int x) {
  __shared__ int wave_lds[kPlanThreads / 64];
#pragma unroll
  for (int d = 1; d < 64; d *= 2) x = max(x, __shfl_xor(x, d));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) wave_lds[threadIdx.x >> 6] = x;
  __syncthreads();
  x = wave_lds[0];
#pragma unroll
  for (int w = 1; w < kPlanThreads / 64; ++w) x = max(x, wave_lds[w]);
  return x;
}

// One workgroup lists the blocks of all problems: a chunk's sequences, or the
// groups over their prefixes and then the sequences over their own places.
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(TileAttention a, TilePlan plan, int block_rows) {
  const int group = a.q_heads / a.cache.kv_heads, tid = threadIdx.x;
  const int problems = a.n_groups + a.n_seqs;
  auto tokens_of = [&](int i, int *token0) {
    if (a.prefix_table && i >= a.n_groups) {
      *token0 = i - a.n_groups;
      return 1;
    }
    const int begin = min(max(a.cu[i], 0), a.T), end = min(max(a.cu[i + 1], begin), a.T);
    *token0 = begin;
    return end - begin;
  };
  int blocks = 0;
  for (int base = 0; base < problems; base += kPlanThreads) {
    const int i = base + tid;
    int token0, n = 0;
    if (i < problems) n = (tokens_of(i, &token0) * group + block_rows - 1) / block_rows;
    int total;
    const int at = blocks + scan_before(n, &total);
    blocks += total;
    if (i < problems) plan.first_block[i] = at;
    for (int k = 0; k < n && at + k < plan.max_blocks; ++k) {
      plan.blocks[at + k].seq = i;
      plan.blocks[at + k].row0 = k * block_rows;
    }
  }
  blocks = min(blocks, plan.max_blocks);     // more only where cu does not rise
  __syncthreads();

  int units = 0, longest = 0;
  for (int base = 0; base < blocks; base += kPlanThreads) {
    const int b = base + tid;
    int mine = 0;
    TileBlock w{};
    if (b < blocks) {
      const int i = plan.blocks[b].seq;
      w.row0 = plan.blocks[b].row0;
      const int n = tokens_of(i, &w.token0);
      w.rows = min(block_rows, n * group - w.row0);
      w.prefix_block = -1;
      if (!a.prefix_table) {
        w.kind = kChunk, w.seq = i;
        w.len = length_of(a.lens[i], a.max_len, a.table_width, a.cache.page_shift);
        w.first = w.len - n;
        const int t0 = w.row0 / group, t1 = (w.row0 + w.rows - 1) / group;
        int a_lo = 0x7FFFFFFF, a_hi = 0, b_lo = 0x7FFFFFFF, b_hi = 0;
        auto add = [&](int t) {
          const RowSees r = row_sees(a.rules, i, w.token0 + t, w.first + t, w.len);
          if (r.n > 0) b_lo = min(b_lo, r.lo), b_hi = max(b_hi, r.lo + r.n);
          if (r.m > 0) a_lo = min(a_lo, r.first), a_hi = max(a_hi, r.first + r.m);
        };
        if (a.rules.doc_starts) {
#pragma unroll 8
          for (int t = t0; t <= t1; ++t) add(t);
        } else {                             // the first token sees the first place, the last one the last
          add(t0);
          add(t1);
        }
        if (a_hi > 0) w.a_lo = a_lo, w.a_hi = a_hi;
        if (b_hi > 0) w.b_lo = b_lo, w.b_hi = b_hi;
      } else if (i < a.n_groups) {
        w.kind = kSharedPrefix, w.seq = i;
        w.len = length_of(a.prefix_lens[i], a.max_prefix, a.prefix_width, a.cache.page_shift);
        w.b_hi = w.len;
      } else {
        w.kind = kOwnPlaces, w.seq = i - a.n_groups;
        w.len = length_of(a.lens[w.seq], a.max_len, a.table_width, a.cache.page_shift);
        w.b_hi = w.len;
        // The last group that does not begin behind the sequence.
        int lo = 0, hi = a.n_groups;
        while (lo < hi) {
          const int mid = (lo + hi) / 2;
          if (a.cu[mid] <= w.seq) lo = mid + 1;
          else hi = mid;
        }
        if (lo > 0) {
          int g0;
          const int members = tokens_of(lo - 1, &g0);
          if (w.seq >= g0 && w.seq < g0 + members) {
            w.prefix_block = plan.first_block[lo - 1];
            w.prefix_row = (w.seq - g0) * group + w.row0;
          }
        }
      }
      w.a_tile = w.a_lo / kTile;
      w.a_n = w.a_hi > 0 ? (w.a_hi + kTile - 1) / kTile - w.a_tile : 0;
      w.b_tile = w.b_lo / kTile;
      if (w.a_n > 0) w.b_tile = max(w.b_tile, w.a_tile + w.a_n);
      w.b_n = w.b_hi > 0 ? max(0, (w.b_hi + kTile - 1) / kTile - w.b_tile) : 0;
      // A chunk's rows that see nothing need their zeros: a tile without places.
      if (w.kind == kChunk && w.a_n + w.b_n == 0) w.b_n = 1;
      mine = w.a_n + w.b_n;
      longest = max(longest, mine);
    }
    int total;
    w.before = units + scan_before(mine, &total);
    units += total;
    if (b < blocks) plan.blocks[b] = w;
  }
  longest = max_all(longest);
  if (tid == 0) {
    // Whole blocks off a queue take as long as their mean load and half a block, or
    // as the longest one; runs as long as their share, and the join of its parts.
    const int64_t pairs = int64_t(blocks) * a.cache.kv_heads;
    const int64_t total = int64_t(units) * a.cache.kv_heads;
    const int per = int(max(int64_t(1), (total + plan.runs - 1) / plan.runs));
    const int64_t queued = max(int64_t(longest), pairs > plan.runs ? per + longest / 2 : 0);
    *plan.header = TileHeader{units, blocks, per, !plan.can_split || queued <= per + kJoinTiles};
    *plan.queue = 0;
  }
}

// ---------------------------------------------------------------- the join

// A query row's parts to its result, in order.  D / 4 lanes a row.
constexpr int kJoinThreads = 256;
__global__ __launch_bounds__(kJoinThreads) void tile_join_kernel(TileAttention a, TilePlan plan, int block_rows,
                                                                 int chunks) {
  const TileHeader head = *plan.header;
  const int D = a.cache.head_dim, lanes = D / 4, at_once = kJoinThreads / lanes;
  const int b = blockIdx.x / (a.cache.kv_heads * chunks);
  const int rest = blockIdx.x % (a.cache.kv_heads * chunks), kvh = rest / chunks;
  if (b >= head.blocks) return;
  const bool both = plan.whole_rows > 0;
  if (!both && head.direct) return;
  const TileBlock w = plan.blocks[b];
  if (w.kind == kSharedPrefix) return;       // joined with the own places
  const int slot = threadIdx.x / lanes, at = threadIdx.x % lanes;
  if (slot >= at_once) return;
  const int group = a.q_heads / a.cache.kv_heads;

  for (int row = rest % chunks * at_once + slot; row < w.rows; row += chunks * at_once) {
    const int in_problem = w.row0 + row, tok = in_problem / group;
    const int64_t q_row = int64_t(w.token0 + tok) * a.q_heads + kvh * group + in_problem - tok * group;
    f32x4 o{};
    float m = -INFINITY, l = 0.0f;
    auto add = [&](int64_t place) {
      const float2 ml = plan.ml[place];
      const f32x4 v = reinterpret_cast<const f32x4 *>(plan.o)[place * lanes + at];
      const float top = fmaxf(m, ml.x), ms = top == -INFINITY ? 0.0f : top;
      const float keep = __builtin_amdgcn_exp2f(m - ms), more = __builtin_amdgcn_exp2f(ml.x - ms);
      o = o * keep + v * more;
      l = l * keep + ml.y * more;
      m = top;
    };
    // The parts of a block's row; false: its result is written already.
    auto add_block = [&](const TileBlock &x, int in_block) {
      const int units = x.a_n + x.b_n;
      if (units == 0) return true;
      const int64_t u0 = int64_t(kvh) * head.units + x.before, u1 = u0 + units;
      const int r0 = head.direct ? 0 : int(u0 / head.per), r1 = head.direct ? 0 : int((u1 - 1) / head.per);
      if (r0 == r1) {
        if (both) add((x.kind == kSharedPrefix ? int64_t(a.T) * a.q_heads : 0) + q_row);
        return both;
      }
      for (int r = r0; r <= r1; ++r)
        add(plan.part_row(r, r == r0 && int64_t(r) * head.per < u0, block_rows, in_block));
      return true;
    };
    if (both && w.prefix_block >= 0)
      add_block(plan.blocks[w.prefix_block + (w.prefix_row + row) / block_rows], (w.prefix_row + row) % block_rows);
    if (!add_block(w, row)) return;
    if (at == 0 && a.lse) a.lse[q_row] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    reinterpret_cast<u32x2 *>(a.out + q_row * D)[at] =
        u32x2{pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv)};
  }
}

// ---------------------------------------------------------------- the launches

// The host knows neither the tokens of a sequence nor its length.
struct Sizes {
  int waves, runs;
  int64_t max_blocks, whole_rows, rows;      // rows: of partial results
  bool can_split;
};
Sizes sizes_of(int32_t T, int32_t n_seqs, int32_t n_groups, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
               int32_t max_len, int32_t max_prefix) {
  Sizes s{};
  const int64_t group = q_heads / kv_heads;
  const int64_t problems = n_groups > 0 ? n_groups : n_seqs;
  // 8 waves where a problem has the rows for them and the registers suffice.
  s.waves = head_dim <= 128 && T * group > 128 * problems ? 8 : 4;
  s.runs = s.waves == 8 || head_dim > 128 ? 256 : 512;
  const int64_t block = kRows * s.waves;
  s.max_blocks = T * group / block + problems;
  if (n_groups > 0) s.max_blocks += n_seqs * ceil_div(group, block);
  const int64_t tiles = ceil_div(std::max(max_len, max_prefix), kTile);
  s.can_split = tiles > kWholeTiles;
  s.whole_rows = n_groups > 0 ? 2 * int64_t(T) * q_heads : 0;
  s.rows = s.whole_rows + (s.can_split ? 2 * s.runs * block : 0);
  return s;
}

inline int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }

template <int kDb, bool kMx, int kW>
hipError_t launch(const TileAttention &a, const TilePlan &plan, hipStream_t stream) {
  const void *kernel = reinterpret_cast<const void *>(&tile_attention_kernel<kDb, kMx, kW>);
  constexpr int kLds = 2 * Stage<kDb>::kBytes;
  const hipError_t e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((tile_attention_kernel<kDb, kMx, kW>), dim3(plan.runs), dim3(64 * kW), kLds, stream, a, plan);
  return hipGetLastError();
}

template <int kDb, bool kMx>
hipError_t by_waves(const TileAttention &a, const TilePlan &plan, int waves, hipStream_t stream) {
  if constexpr (kDb <= 4) {
    if (waves == 8) return launch<kDb, kMx, 8>(a, plan, stream);
  }
  return launch<kDb, kMx, 4>(a, plan, stream);
}

template <int kDb>
hipError_t by_format(const TileAttention &a, const TilePlan &plan, int waves, hipStream_t stream) {
  return a.cache.k_scales ? by_waves<kDb, true>(a, plan, waves, stream) : by_waves<kDb, false>(a, plan, waves, stream);
}

}  // namespace

int64_t tile_attention_workspace(int32_t T, int32_t n_seqs, int32_t n_groups, int32_t q_heads, int32_t kv_heads,
                                 int32_t head_dim, int32_t max_len, int32_t max_prefix) {
  const Sizes s = sizes_of(T, n_seqs, n_groups, q_heads, kv_heads, head_dim, max_len, max_prefix);
  const int64_t tiles = std::max<int64_t>(1, ceil_div(std::max(max_len, max_prefix), kTile)) + 1;
  if (s.max_blocks > 0x7FFFFFFF / (8 * tiles) / kv_heads || s.whole_rows > 0x7FFFFFFF) return -1;
  return 256 + align256(s.max_blocks * int64_t(sizeof(TileBlock))) + align256((n_groups + int64_t(n_seqs)) * 4) +
         align256(s.rows * 8) + s.rows * head_dim * 4;
}

hipError_t launch_tile_attention(const TileAttention &a, hipStream_t stream) {
  const int D = a.cache.head_dim, hkv = a.cache.kv_heads;
  const Sizes s = sizes_of(a.T, a.n_seqs, a.n_groups, a.q_heads, hkv, D, a.max_len, a.max_prefix);
  TilePlan plan{};
  uint8_t *at = static_cast<uint8_t *>(a.workspace);
  plan.header = reinterpret_cast<TileHeader *>(at);
  plan.queue = reinterpret_cast<int32_t *>(at + 64);
  plan.blocks = reinterpret_cast<TileBlock *>(at += 256);
  plan.first_block = reinterpret_cast<int32_t *>(at += align256(s.max_blocks * int64_t(sizeof(TileBlock))));
  plan.ml = reinterpret_cast<float2 *>(at += align256((a.n_groups + int64_t(a.n_seqs)) * 4));
  plan.o = reinterpret_cast<float *>(at + align256(s.rows * 8));
  plan.max_blocks = int32_t(s.max_blocks);
  plan.runs = s.runs;
  plan.whole_rows = int32_t(s.whole_rows);
  plan.can_split = s.can_split;
  const int block = kRows * s.waves;
  hipLaunchKernelGGL(plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a, plan, block);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  switch (D / 32) {
    case 1: err = by_format<1>(a, plan, s.waves, stream); break;
    case 2: err = by_format<2>(a, plan, s.waves, stream); break;
    case 3: err = by_format<3>(a, plan, s.waves, stream); break;
    case 4: err = by_format<4>(a, plan, s.waves, stream); break;
    case 5: err = by_format<5>(a, plan, s.waves, stream); break;
    case 6: err = by_format<6>(a, plan, s.waves, stream); break;
    case 7: err = by_format<7>(a, plan, s.waves, stream); break;
    default: err = by_format<8>(a, plan, s.waves, stream);
  }
  if (err != hipSuccess || (!s.can_split && s.whole_rows == 0)) return err;
  // Workgroups of a (block, head): one for each run of rows that it takes at once.
  const int at_once = kJoinThreads / (D / 4);
  const int rows = int(std::min<int64_t>(block, int64_t(a.T) * (a.q_heads / hkv)));
  const int chunks = std::max(1, (rows + at_once - 1) / at_once);
  hipLaunchKernelGGL(tile_join_kernel, dim3(unsigned(s.max_blocks * hkv * chunks)), dim3(kJoinThreads), 0, stream, a,
                     plan, block, chunks);
  return hipGetLastError();
}

}  // namespace engram
