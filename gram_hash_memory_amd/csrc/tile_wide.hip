// Attention of many query rows a key-value head over the paged cache: the new
// tokens of a chunk (causal, with windows, prefixes, documents, capped scores and
// a distance bias), and the sequences that share a prefix.
//
//   z = scale q.k;  z = cap tanh(z / cap);  z -= slope |pos - p|
//   out = sum_p e^(z_p - m) v_p / sum_p e^(z_p - m),  lse = m + log sum_p e^(z_p - m)
//
// A workgroup takes a block of 32 kW rows, 32 a wave, through the places that any
// of them sees, 64 at a time:
//  - keys and values go from memory to registers one tile ahead, are converted
//    there, and put into one of two LDS buffers; rows are padded so that no two
//    lanes of a read share a bank;
//  - S^T = K Q^T by v_mfma_f32_32x32x16_bf16: a lane then has 32 scores of one
//    query row, so the running maximum takes one exchange between lanes;
//  - O^T = V^T P^T: the scores' registers are the P^T operand as they stand, with
//    the places in an order that V's transposing LDS reads follow.
// Two workgroups' waves, or one's 8, share a SIMD: one's softmax fills the other's
// waits for the matrix core.
#include "attention_common.hpp"
#include "tile_plan.hpp"

namespace engram {
namespace {

using namespace attn;

constexpr int kTile = kWideTile;
constexpr float kLazy = 8.0f;

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

template <int kDb, bool kMx, int kW, bool kRules>
__global__ __launch_bounds__(64 * kW, kDb <= 4 ? 2 : 1) void tile_wide_kernel(
    TileAttention a, TilePlan plan) {
  constexpr int D = 32 * kDb, kThreads = 64 * kW;
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
  const int mask = (1 << c.page_shift) - 1;
  const ScoreUnit su = score_unit(a, kLog2e);
  const TileList &list = plan.list[0];
  const TileHeader head = *list.header;
  Work work;
  if (!first_work(list, head, c.kv_heads, kThreads, work_lds, &work)) return;

  for (int piece = 0;; ++piece) {
    if (head.direct && !next_block(list, head, c.kv_heads, work_lds, &work)) return;
    const TileBlock w = list.blocks[work.block];
    const int count = head.direct ? w.tiles() : min(w.tiles() - work.unit, work.left);
    const bool whole = count == w.tiles();
    const int kvh = work.kvh;
    const bool shared = w.kind == kSharedPrefix;
    const int32_t *table = shared ? a.prefix_table + int64_t(w.seq) * a.prefix_width
                                  : a.table + int64_t(w.seq) * a.table_width;

    // This lane's query row, and what it sees.
    const int row = wave * kRows + col;
    const bool live = row < w.rows;
    const QueryRow qr = query_row(a, w, kvh, min(row, w.rows - 1));
    const int pos = w.first + qr.tok;
    RowSees r{0, w.len, 0, 0};
    if (w.kind == kChunk) r = row_sees(a.rules, w.seq, qr.token, pos, w.len);
    const float slope = kRules && a.rules.slopes ? a.rules.slopes[qr.head] * kLog2e : 0.0f;
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
      u32x4 v = *reinterpret_cast<const u32x4 *>(a.q + qr.at * D + 16 * kk + 8 * half);
#pragma unroll
      for (int x = 0; x < 4; ++x) v[x] = (v[x] ^ su.flip) & su.keep;
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

    auto place_of = [&](int t) { return w.place(t, kTile); };
    auto plain = [&](const int4 &l, int p0) {
      return (p0 >= l.x && p0 + kTile <= l.y) || (p0 >= l.z && p0 + kTile <= l.w);
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
        const bool in = in_tile && w.used(p), there = unsigned(page[i]) < unsigned(c.pages);
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

    const int t0 = work.unit, t1 = t0 + count;
    ask_pages(t0);
    load(t0);
    ask_pages(min(t0 + 1, t1 - 1));
    put(t0, 0, !plain(all, place_of(t0)));
    __syncthreads();

    for (int t = t0, buf = 0; t < t1; ++t, buf ^= 1) {
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
        // Operands come 4 at a time, each four requested before the four before it
        // are used: more would not fit the registers.
        bf16x8 kf[2][4];
        auto read_keys = [&](int i, bf16x8(&f)[4]) {
#pragma unroll
          for (int x = 0; x < 4; ++x)
            f[x] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(
                st + (32 * (x % 2) + col) * S::kKeyRow + 32 * (2 * i + x / 2) + 16 * half));
        };
        const uint8_t *const vp = st + S::kValues + (4 * half + lane % 16 / 4) * S::kValueRow +
                                  32 * (lane / 16 % 2) + 8 * (lane % 4);
        bf16x8 vf[2][4];
        auto read_values = [&](int i, bf16x8(&f)[4]) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int j = (4 * i + x) / kDb, n = (4 * i + x) % kDb;
            const u32x2 lo = read_transposed(vp + 16 * j * S::kValueRow + 64 * n);
            const u32x2 hi = read_transposed(vp + (16 * j + 8) * S::kValueRow + 64 * n);
            f[x] = as_frag(lo[0], lo[1], hi[0], hi[1]);
          }
        };
        f32x16 z[2] = {};
        read_keys(0, kf[0]);
#pragma unroll
        for (int i = 0; i < kDb; ++i) {
          if (i + 1 < kDb) read_keys(i + 1, kf[(i + 1) % 2]);
          else read_values(0, vf[0]);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int x = 0; x < 4; ++x) z[x % 2] = mfma32(kf[i % 2][x], q[2 * i + x / 2], z[x % 2]);
          __builtin_amdgcn_sched_barrier(0);
        }
        // Register 4 i + j of tile half u: place 32 u + 8 i + 4 half + j.
        const bool masked = !plain(lim, p0) || any_absent;
        if constexpr (kRules) {
#pragma unroll
          for (int x = 0; x < 32; ++x) z[x / 16][x % 16] *= su.unit;
          if (a.rules.cap > 0.0f) {
            float far = 0.0f;
#pragma unroll
            for (int x = 0; x < 32; ++x) far = fmaxf(far, fabsf(z[x / 16][x % 16]));
            if (__any(!(far <= kTanhSplit))) {
#pragma unroll
              for (int x = 0; x < 32; ++x) {
                const float y = z[x / 16][x % 16];
                z[x / 16][x % 16] = su.cap2 * (fabsf(y) <= kTanhSplit ? tanh_small(y) : tanh_large(y));
              }
            } else {
#pragma unroll
              for (int x = 0; x < 32; ++x) z[x / 16][x % 16] = su.cap2 * tanh_small(z[x / 16][x % 16]);
            }
          }
          if (a.rules.slopes) {
            // Distances below 2^24 are whole numbers in fp32, larger ones off by half a step.
            const float ahead = float(pos - p0 - 4 * half);
#pragma unroll
            for (int x = 0; x < 32; ++x) {
              const float back = ahead - float(32 * (x / 16) + 8 * (x % 16 / 4) + x % 4);
              z[x / 16][x % 16] = __builtin_fmaf(-slope, fabsf(back), z[x / 16][x % 16]);
            }
          }
        }
        if (masked) {
          const int from_lo = p0 + 4 * half - r.lo, from_first = p0 + 4 * half - r.first;
          const uint32_t away[2] = {absent[0] >> (4 * half), absent[1] >> (4 * half)};
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            const int at = 8 * (x % 16 / 4) + x % 4, step = 32 * (x / 16) + at;
            const bool ok = ((unsigned(from_lo + step) < unsigned(r.n)) | (unsigned(from_first + step) < unsigned(r.m))) &
                            !(away[x / 16] & 1u << at);
            z[x / 16][x % 16] = ok ? z[x / 16][x % 16] : -INFINITY;
          }
        }
        float top = z[0][0];
#pragma unroll
        for (int x = 1; x < 32; ++x) top = fmaxf(top, z[x / 16][x % 16]);
        top = pair_max(kRules ? top : top * su.unit);
        // The weights' reference follows the largest score only where that is 2^8 above it.
        if (__any(top > m + kLazy)) {
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
          const float y = z[x / 16][x % 16];
          z[x / 16][x % 16] = __builtin_amdgcn_exp2f(kRules ? y - ms : __builtin_fmaf(y, su.unit, -ms));
          sum[x / 16] += z[x / 16][x % 16];
        }
        l += sum[0] + sum[1];
        bf16x8 p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x16 &e = z[j / 2];
          const int x = 8 * (j % 2);
          p[j] = as_frag(pack_bf16x2(e[x], e[x + 1]), pack_bf16x2(e[x + 2], e[x + 3]),
                         pack_bf16x2(e[x + 4], e[x + 5]), pack_bf16x2(e[x + 6], e[x + 7]));
        }
#pragma unroll
        for (int i = 0; i < kDb; ++i) {
          __builtin_amdgcn_sched_barrier(0);
          if (i + 1 < kDb) read_values(i + 1, vf[(i + 1) % 2]);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int j = (4 * i + x) / kDb, n = (4 * i + x) % kDb;
            o[n] = mfma32(vf[i % 2][x], p[j], o[n]);
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
            for (int n = 0; n < kDb; ++n) {
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                float v[4];
                values_at<kMx>(c, place, 32 * n + 8 * x + 4 * half, v);
#pragma unroll
                for (int y = 0; y < 4; ++y)
                  if (ok && !(fabsf(v[y]) < INFINITY)) o[n][4 * x + y] += e * v[y];
              }
              __builtin_amdgcn_sched_barrier(0);      // no more of these loads at a time: registers
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
            a.lse[qr.at] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
          uint16_t *const dst = a.out + qr.at * D + 4 * half;
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
        const int64_t at = whole ? (shared ? int64_t(a.T) * a.q_heads : 0) + qr.at
                                 : list.part_row(work.run, piece > 0, row);
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
      work.left -= count;
      if (work.left == 0) return;
      work.unit = 0;
      if (++work.block == head.blocks) work.block = 0, ++work.kvh;
    }
  }
}

template <int kDb, bool kMx, int kW, bool kRules>
hipError_t launch(const TileAttention &a, const TilePlan &plan, hipStream_t stream) {
  const void *kernel = reinterpret_cast<const void *>(&tile_wide_kernel<kDb, kMx, kW, kRules>);
  constexpr int kLds = 2 * Stage<kDb>::kBytes;
  const hipError_t e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((tile_wide_kernel<kDb, kMx, kW, kRules>), dim3(plan.list[0].runs), dim3(64 * kW), kLds, stream,
                     a, plan);
  return hipGetLastError();
}

template <int kDb, bool kMx>
hipError_t by_waves(const TileAttention &a, const TilePlan &plan, hipStream_t stream) {
  const bool rules = a.rules.cap > 0.0f || a.rules.slopes;
  if constexpr (kDb <= 4) {
    if (plan.list[0].block_rows == 8 * kRows)
      return rules ? launch<kDb, kMx, 8, true>(a, plan, stream) : launch<kDb, kMx, 8, false>(a, plan, stream);
  }
  return rules ? launch<kDb, kMx, 4, true>(a, plan, stream) : launch<kDb, kMx, 4, false>(a, plan, stream);
}

template <int kDb>
hipError_t by_format(const TileAttention &a, const TilePlan &plan, hipStream_t stream) {
  return a.cache.k_scales ? by_waves<kDb, true>(a, plan, stream) : by_waves<kDb, false>(a, plan, stream);
}

}  // namespace

hipError_t launch_tile_wide(const TileAttention &a, const TilePlan &plan, hipStream_t stream) {
  switch (a.cache.head_dim / 32) {
    case 1: return by_format<1>(a, plan, stream);
    case 2: return by_format<2>(a, plan, stream);
    case 3: return by_format<3>(a, plan, stream);
    case 4: return by_format<4>(a, plan, stream);
    case 5: return by_format<5>(a, plan, stream);
    case 6: return by_format<6>(a, plan, stream);
    case 7: return by_format<7>(a, plan, stream);
    default: return by_format<8>(a, plan, stream);
  }
}

}  // namespace engram
