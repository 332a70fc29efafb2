// Attention of up to 32 query rows a key-value head over the paged cache, with the
// rules of tile_wide.hip: single tokens, drafts, the places that a sequence has
// behind a shared prefix.
//
// Bound by reading the keys and values once.  The four waves of a workgroup share
// the places, 32 each of a tile of 128, and run apart: keys and values go from
// memory to registers and into the matrix cores as in attention.hip, without LDS,
// the next tile requested as soon as a register is free, its pages a tile earlier.
// At the end of a block, or of a run's piece of one, the waves' results are joined
// in LDS.
//
// 64 single tokens over up to 4095 places in 8 bits with capped scores and a distance
// bias (338 MB): 78 us, 4.4 TB/s; the cap's and the bias's arithmetic is what keeps it
// from the copy's rate.  Pages are asked for two tiles ahead because a wait for them
// was one for the next tile's keys as well (251 us).
#include "attention_common.hpp"
#include "tile_plan.hpp"

namespace engram {
namespace {

using namespace attn;

constexpr int kWaves = kNarrowWaves, kThreads = 64 * kWaves;

// What a workgroup works at: `count` tiles of a block, for one key-value head.
struct Piece {
  int kvh, t0, count, run;
  bool whole, later;
};

// kHt: tiles of 16 query rows.
template <int kDb, bool kMx, int kHt>
__device__ __forceinline__ void work_piece(const TileAttention &a, const TilePlan &plan, const TileBlock &w,
                                           const Piece &piece, f32x4 *o_lds, float2 (*ml_lds)[kHt][16]) {
  constexpr int D = 32 * kDb, kRowBytes = kMx ? D : 2 * D, kAcc = D / 16;
  using P = Pieces<kDb>;
  const CacheView &c = a.cache;
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int mask = (1 << c.page_shift) - 1, kvh = piece.kvh;
  const ScoreUnit su = score_unit(a, kLog2e);
  const bool shared = w.kind == kSharedPrefix;
  const int32_t *table = shared ? a.prefix_table + int64_t(w.seq) * a.prefix_width
                                : a.table + int64_t(w.seq) * a.table_width;
  if (w.len == 0) table = plan.list[1].queue;          // any memory: there is no place to look up

  // This lane's query rows, 16 t + col, and what they see.
  bf16x8 q[kHt][kDb];
  RowSees r[kHt];
  int pos[kHt];
  float slope[kHt];
  int4 lim = {-0x7FFFFFFF, 0x7FFFFFFF, -0x7FFFFFFF, 0x7FFFFFFF};
#pragma unroll
  for (int t = 0; t < kHt; ++t) {
    const QueryRow qr = query_row(a, w, kvh, min(16 * t + col, w.rows - 1));
    pos[t] = w.first + qr.tok;
    r[t] = RowSees{0, w.len, 0, 0};
    if (w.kind == kChunk) r[t] = token_sees(a.rules, w.seq, qr.token, pos[t], w.len);
    slope[t] = a.rules.slopes ? a.rules.slopes[qr.head] * kLog2e : 0.0f;
    lim = {max(lim.x, r[t].lo), min(lim.y, r[t].lo + r[t].n), max(lim.z, r[t].first), min(lim.w, r[t].first + r[t].m)};
#pragma unroll
    for (int kk = 0; kk < kDb; ++kk) {
      const int d = kMx && (kk | 1) < kDb ? 64 * (kk / 2) + 16 * g + 8 * (kk & 1) : 32 * kk + 8 * g;
      u32x4 v = *reinterpret_cast<const u32x4 *>(a.q + qr.at * D + d);
#pragma unroll
      for (int x = 0; x < 4; ++x) v[x] = (v[x] ^ su.flip) & su.keep;
      q[t][kk] = __builtin_bit_cast(bf16x8, v);
    }
  }
#pragma unroll
  for (int x = 1; x < 16; x *= 2) {
    lim.x = max(lim.x, __shfl_xor(lim.x, x));
    lim.y = min(lim.y, __shfl_xor(lim.y, x));
    lim.z = max(lim.z, __shfl_xor(lim.z, x));
    lim.w = min(lim.w, __shfl_xor(lim.w, x));
  }
  lim = {__builtin_amdgcn_readfirstlane(lim.x), __builtin_amdgcn_readfirstlane(lim.y),
         __builtin_amdgcn_readfirstlane(lim.z), __builtin_amdgcn_readfirstlane(lim.w)};

  const int t1 = piece.t0 + piece.count;
  auto place_of = [&](int t) { return w.place(min(t, t1 - 1), kNarrowTile) + 32 * wave; };

  // The pages of a tile's places 16 u + col, and 16 u + 4 g .. + 3 (a page holds 4
  // places from a multiple of 4 on together): asked for two tiles ahead, before the
  // next tile's keys, so that no wait for them is a wait for anything else.
  struct Pages {
    int key[2], value[2];
  };
  auto ask_pages = [&](int t, Pages &pg) {
    const int p0 = place_of(t), last = max(0, w.len - 1);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      pg.key[u] = table[min(p0 + 16 * u + col, last) >> c.page_shift];
      pg.value[u] = table[min(p0 + 16 * u + 4 * g, last) >> c.page_shift];
    }
  };
  // Rows of pages that are not there are those of the cache's beginning.
  auto row_of = [&](int page, int p) {
    return unsigned(page) < unsigned(c.pages) ? ((int64_t(page) * c.kv_heads + kvh) << c.page_shift) + (p & mask) : int64_t(0);
  };
  Held<kDb, kMx> held;
  auto load_k = [&](int t, const Pages &pg) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t row = row_of(pg.key[u], place_of(t) + 16 * u + col);
      const uint8_t *const src = static_cast<const uint8_t *>(c.k) + row * kRowBytes;
      if constexpr (!kMx) {
#pragma unroll
        for (int kk = 0; kk < kDb; ++kk) load_bytes<16>(&held.k[u][4 * kk], src + 64 * kk + 16 * g);
      } else {
        const uint8_t *const sc = c.k_scales + row * kDb;
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
  auto load_v = [&](int t, const Pages &pg) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t row = row_of(pg.value[u], place_of(t) + 16 * u + 4 * g);
      const uint8_t *const src = static_cast<const uint8_t *>(c.v) + row * kRowBytes;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        each_piece<P::kN>([&](auto at) {
          constexpr int wd = P::width(at.value), first = P::base(at.value);
          if constexpr (kMx) {
            load_bytes<wd>(&held.v[4 * u + j][first / 64], src + j * kRowBytes + first + wd * col);
            held.vs[4 * u + j][at.value] = c.v_scales[(row + j) * kDb + (first + wd * col) / 32];
          } else {
            load_bytes<2 * wd>(&held.v[4 * u + j][first / 32], src + j * kRowBytes + 2 * (first + wd * col));
          }
        });
      }
    }
  };

  float m[kHt], l[kHt];
  f32x4 o[kHt][kAcc];
#pragma unroll
  for (int t = 0; t < kHt; ++t) {
    m[t] = -INFINITY, l[t] = 0.0f;
#pragma unroll
    for (int n = 0; n < kAcc; ++n) o[t][n] = f32x4{};
  }
  bool bad = false;

  // Tile t, whose pages are `here`; those of t + 1 are `next`, and `here` then takes
  // those of t + 2.
  auto step = [&](int t, Pages &here, Pages &next) {
    const int p0 = place_of(t);
    f32x4 z[kHt][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int y = 0; y < kHt; ++y) z[y][u] = f32x4{};
#pragma unroll
      for (int kk = 0; kk < kDb; ++kk) {
        bf16x8 f;
        if constexpr (kMx) {
          const uint32_t *k = &held.k[u][2 * kk];
          const float sc = __uint_as_float(held.ks[u][kk / 2] << 23);
          f = as_frag(mx_pair(k[0], sc, false), mx_pair(k[0], sc, true), mx_pair(k[1], sc, false), mx_pair(k[1], sc, true));
        } else {
          const uint32_t *k = &held.k[u][4 * kk];
          f = as_frag(k[0], k[1], k[2], k[3]);
        }
#pragma unroll
        for (int y = 0; y < kHt; ++y) z[y][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, q[y][kk], z[y][u], 0, 0, 0);
      }
    }
    // Bits 4 u + r: place 16 u + 4 g + r is on a page of the cache, and used.
    uint32_t there = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const bool page = unsigned(here.value[u]) < unsigned(c.pages);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const bool used = w.used(p0 + 16 * u + 4 * g + x);
        there |= uint32_t(used & page) << (4 * u + x);
        bad |= used & !page;
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    ask_pages(t + 2, here);
    load_k(t + 1, next);
    __builtin_amdgcn_sched_barrier(0);

    const bool plain = ((p0 >= lim.x && p0 + 32 <= lim.y) || (p0 >= lim.z && p0 + 32 <= lim.w)) && !__any(there != 0xFF);
    bf16x8 wt[kHt];                          // the weights, as B operands
    float e[kHt][8];
#pragma unroll
    for (int y = 0; y < kHt; ++y) {
      float(&x)[8] = e[y];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = z[y][j / 4][j % 4] * su.unit;
      if (a.rules.cap > 0.0f) {
        float far = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) far = fmaxf(far, fabsf(x[j]));
        if (__any(!(far <= kTanhSplit))) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float small = tanh_small(x[j]), large = tanh_large(x[j]);
            x[j] = su.cap2 * (fabsf(x[j]) <= kTanhSplit ? small : large);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = su.cap2 * tanh_small(x[j]);
        }
      }
      if (a.rules.slopes) {
        const float ahead = float(pos[y] - p0 - 4 * g);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          x[j] = __builtin_fmaf(-slope[y], fabsf(ahead - float(16 * (j / 4) + j % 4)), x[j]);
      }
      if (!plain) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bool ok = ((there >> j & 1) != 0) & sees(r[y], p0 + 16 * (j / 4) + 4 * g + j % 4);
          x[j] = ok ? x[j] : -INFINITY;
        }
      }
      float top = x[0];
#pragma unroll
      for (int j = 1; j < 8; ++j) top = fmaxf(top, x[j]);
      top = column_max(top);
      if (__any(top > m[y])) {               // rarely after the first tiles
        const float mn = fmaxf(m[y], top);
        const float keep = mn == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m[y] - mn);
        m[y] = mn;
        l[y] *= keep;
#pragma unroll
        for (int n = 0; n < kAcc; ++n) o[y][n] *= keep;
      }
      const float ms = m[y] == -INFINITY ? 0.0f : m[y];
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = __builtin_amdgcn_exp2f(x[j] - ms);
        sum += x[j];
      }
      l[y] += sum;
      wt[y] = as_frag(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }

    uint32_t odd = 0;                        // bit 4 u + r, in the lanes that hold one
    each_piece<P::kN>([&](auto at) {
      constexpr int wd = P::width(at.value), first = P::base(at.value);
#pragma unroll
      for (int i = 0; i < wd / 2; ++i) {
        uint32_t x[8];                       // dimensions 2 i, 2 i + 1 of the lane's 8 places
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if constexpr (kMx)
            x[j] = mx_pair(held.v[j][first / 64 + i / 2],
                           __uint_as_float(min(held.vs[j][at.value], 254u) << 23), i & 1);
          else
            x[j] = held.v[j][first / 32 + i];
        }
        // Values that no row sees count as 0.  Where some rows see a place and others
        // do not, so do values that are not finite, which a weight of 0 would spread;
        // the rows that see them get them below.
        if (!plain) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x[j] = there >> j & 1 ? x[j] : 0u;
            const bool lo = (x[j] & 0x7F80u) == 0x7F80u, hi = (x[j] & 0x7F800000u) == 0x7F800000u;
            odd |= uint32_t(lo | hi) << j;
            x[j] &= (lo ? 0u : 0xFFFFu) | (hi ? 0u : 0xFFFF0000u);
          }
        }
        const bf16x8 even = as_frag(__builtin_amdgcn_perm(x[1], x[0], 0x05040100u), __builtin_amdgcn_perm(x[3], x[2], 0x05040100u),
                                    __builtin_amdgcn_perm(x[5], x[4], 0x05040100u), __builtin_amdgcn_perm(x[7], x[6], 0x05040100u));
        const bf16x8 uneven = as_frag(__builtin_amdgcn_perm(x[1], x[0], 0x07060302u), __builtin_amdgcn_perm(x[3], x[2], 0x07060302u),
                                      __builtin_amdgcn_perm(x[5], x[4], 0x07060302u), __builtin_amdgcn_perm(x[7], x[6], 0x07060302u));
        const int n = first / 16 + 2 * i;
#pragma unroll
        for (int y = 0; y < kHt; ++y) {
          o[y][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(even, wt[y], o[y][n], 0, 0, 0);
          o[y][n + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(uneven, wt[y], o[y][n + 1], 0, 0, 0);
        }
      }
    });
    __builtin_amdgcn_sched_barrier(0);
    load_v(t + 1, next);
    __builtin_amdgcn_sched_barrier(0);

    if (__any(odd != 0)) {
      for (int j = 0; j < 8; ++j) {
        const uint64_t holders = __ballot(odd >> j & 1);
        for (int gg = 0; gg < 4; ++gg) {     // place 16 (j / 4) + 4 gg + j % 4
          if (!(holders >> (16 * gg) & 0xFFFFu)) continue;
          const int p = p0 + 16 * (j / 4) + 4 * gg + j % 4;
          const int64_t row = row_of(table[p >> c.page_shift], p);
#pragma unroll
          for (int y = 0; y < kHt; ++y) {
            float x = 0.0f;                  // the weight of this lane's row
#pragma unroll
            for (int k = 0; k < 8; ++k) x = k == j ? e[y][k] : x;
            x = __shfl(x, 16 * gg + col);
            const bool ok = sees(r[y], p);
            // Accumulator n's register k: dimension first + wd (4 g + k) + n - first / 16.
            each_piece<P::kN>([&](auto at) {
              constexpr int wd = P::width(at.value), first = P::base(at.value);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
#pragma unroll
                for (int n = 0; n < wd; ++n) {
                  const float v = value_at<kMx>(c, row, first + wd * (4 * g + k) + n);
                  if (ok && !(fabsf(v) < INFINITY)) o[y][first / 16 + n][k] += x * v;
                }
                __builtin_amdgcn_sched_barrier(0);      // no more of these loads at a time: registers
              }
            });
          }
        }
      }
    }
  };

  if (piece.count > 0) {
    Pages even, uneven;
    ask_pages(piece.t0, even);
    ask_pages(piece.t0 + 1, uneven);
    load_k(piece.t0, even);
    load_v(piece.t0, even);
    for (int t = piece.t0; t < t1; t += 2) {
      step(t, even, uneven);
      if (t + 1 < t1) step(t + 1, uneven, even);
    }
  }
  if (__any(bad) && lane == 0 && kvh == 0 && a.bad_pages) atomicAdd(a.bad_pages, 1);

  // The waves' results, 16 rows at a time, joined in wave order by all threads: two
  // neighbouring dimensions of four places in O^T each.
#pragma unroll
  for (int t = 0; t < kHt; ++t) {
    l[t] = column_sum(l[t]);
    if (g == 0) ml_lds[wave][t][col] = float2{m[t], l[t]};
  }
#pragma unroll
  for (int t = 0; t < kHt; ++t) {
#pragma unroll
    for (int n = 0; n < kAcc; ++n) o_lds[(wave * kAcc + n) * 64 + lane] = o[t][n];
    __syncthreads();
    for (int k = threadIdx.x; k < kAcc / 2 * 64; k += kThreads) {
      const int n = k / 64 * 2, from = k % 64, row = 16 * t + from % 16, gg = from / 16;
      if (row >= w.rows) continue;
      float top = -INFINITY, sum = 0.0f;
      float2 ml[kWaves];
#pragma unroll
      for (int x = 0; x < kWaves; ++x) {
        ml[x] = ml_lds[x][t][from % 16];
        top = fmaxf(top, ml[x].x);
      }
      const float ms = top == -INFINITY ? 0.0f : top;
      f32x4 a0{}, a1{};
#pragma unroll
      for (int x = 0; x < kWaves; ++x) {
        const float keep = __builtin_amdgcn_exp2f(ml[x].x - ms);
        sum += ml[x].y * keep;
        a0 += o_lds[(x * kAcc + n) * 64 + from] * keep;
        a1 += o_lds[(x * kAcc + n + 1) * 64 + from] * keep;
      }
      const int64_t q_row = query_row(a, w, kvh, row).at;
      const bool result = piece.whole && plan.whole_rows == 0;
      const int64_t at = result ? q_row : piece.whole ? (shared ? int64_t(a.T) * a.q_heads : 0) + q_row
                                                      : plan.list[1].part_row(piece.run, piece.later, row);
      const float inv = !result ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
      if (n == 0 && gg == 0) {
        if (!result) plan.ml[at] = float2{top, sum};
        else if (a.lse) a.lse[q_row] = sum == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
      }
      int first = 0, wd = P::width(0);
      each_piece<P::kN>([&](auto at_piece) {
        if (16 * n >= P::base(at_piece.value)) first = P::base(at_piece.value), wd = P::width(at_piece.value);
      });
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int d = first + wd * (4 * gg + y) + n - first / 16;
        if (result) *reinterpret_cast<uint32_t *>(a.out + q_row * D + d) = pack_bf16x2(a0[y] * inv, a1[y] * inv);
        else *reinterpret_cast<float2 *>(plan.o + at * D + d) = float2{a0[y], a1[y]};
      }
    }
    __syncthreads();
  }
}

// 32 rows of larger heads than this do not fit the registers; of smaller ones they save
// reading the places twice, which costs 16 rows nothing to leave out.
constexpr int kMostTwo = 160;
// Registers for two workgroups a CU where they suffice.
constexpr int groups_per_cu(int db, int ht) { return db * ht <= 4 ? 2 : 1; }

template <int kDb, bool kMx, int kHt>
__global__ __launch_bounds__(kThreads, groups_per_cu(kDb, kHt)) void tile_narrow_kernel(TileAttention a, TilePlan plan) {
  extern __shared__ f32x4 o_lds[];           // [kWaves][D / 16][64]: 16 rows of the waves' results
  __shared__ float2 ml_lds[kWaves][kHt][16];
  __shared__ int work_lds[2];
  const int kv_heads = a.cache.kv_heads;
  const TileList &list = plan.list[1];
  const TileHeader head = *list.header;
  Work work;
  if (!first_work(list, head, kv_heads, kThreads, work_lds, &work)) return;
  for (int piece = 0;; ++piece) {
    if (head.direct && !next_block(list, head, kv_heads, work_lds, &work)) return;
    const TileBlock w = list.blocks[work.block];
    const int count = head.direct ? w.tiles() : min(w.tiles() - work.unit, work.left);
    work_piece<kDb, kMx, kHt>(a, plan, w, Piece{work.kvh, work.unit, count, work.run, count == w.tiles(), piece > 0}, o_lds,
                              ml_lds);
    if (!head.direct) {
      work.left -= count;
      if (work.left == 0) return;
      work.unit = 0;
      if (++work.block == head.blocks) work.block = 0, ++work.kvh;
    }
  }
}

template <int kDb, bool kMx, int kHt>
hipError_t launch(const TileAttention &a, const TilePlan &plan, hipStream_t stream) {
  const void *kernel = reinterpret_cast<const void *>(&tile_narrow_kernel<kDb, kMx, kHt>);
  constexpr int kLds = kWaves * 2 * kDb * 64 * int(sizeof(f32x4));
  if (kLds + 2048 > 65536) {                 // more than a launch may have without asking
    const hipError_t e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((tile_narrow_kernel<kDb, kMx, kHt>), dim3(plan.list[1].runs), dim3(kThreads), kLds, stream, a, plan);
  return hipGetLastError();
}

template <int kDb, bool kMx>
hipError_t by_rows(const TileAttention &a, const TilePlan &plan, hipStream_t stream) {
  if constexpr (kDb <= kMostTwo / 32) {
    if (plan.list[1].block_rows > 16) return launch<kDb, kMx, 2>(a, plan, stream);
  }
  return launch<kDb, kMx, 1>(a, plan, stream);
}

template <int kDb>
hipError_t by_format(const TileAttention &a, const TilePlan &plan, hipStream_t stream) {
  return a.cache.k_scales ? by_rows<kDb, true>(a, plan, stream) : by_rows<kDb, false>(a, plan, stream);
}

}  // namespace

int tile_narrow_rows(int32_t head_dim, int64_t rows) { return rows > 16 && head_dim <= kMostTwo ? 32 : 16; }

int tile_narrow_groups(int32_t head_dim, int32_t block_rows) {
  return 256 * groups_per_cu(head_dim / 32, block_rows / 16);
}

hipError_t launch_tile_narrow(const TileAttention &a, const TilePlan &plan, hipStream_t stream) {
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
