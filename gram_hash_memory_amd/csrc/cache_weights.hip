// The attention weight that each place of the cache gets from new tokens,
//
//   w_p += sum over the tokens and heads that see p of e^(z_p - lse),
//
// with z as in tile_wide.hip.  A wave owns 64 or 32 places of one key-value head: their keys
// stay in its registers as matrix-core operands, the query rows of the sequence go by 16 at a
// time, the next 16 requested before these are used, and a lane adds up the weights of its
// places from every 16th row, in row order; lanes are joined once, at the end.  One wave
// writes a place, so the sums do not depend on timing.  No tile passes through shared memory:
// keys are read once, and the query rows, which all of a head's waves read, come from the L2.
// Where few rows see a place the reading of the keys bounds it (64 streams of up to 4095
// places in 8 bits, 180 MB with the weights: 49 us), where many do, the exponential and its
// bookkeeping, some ten operations a place and row (64 tokens after 16320 places: 32 us).
#include "attention_common.hpp"
#include "tile_plan.hpp"

namespace engram {
namespace {

using namespace attn;

// One wave a workgroup: its places are free for the next wave's as soon as it is done (64
// streams of up to 4095 places: 49 us, with 2, 4, 8 and 16 waves 54, 66, 79 and 89).
constexpr int kThreads = 64;

// kU: tiles of 16 places that a wave takes; a query row's part of the work, what it sees
// and its sum, is shared by them.
template <int kDb, bool kMx, int kU>
__global__ __launch_bounds__(kThreads, kU == 2 && kDb <= 4 ? 4 : 2) void cache_weights_kernel(CacheWeights a, int chunks) {
  constexpr int D = 32 * kDb, kRowBytes = kMx ? D : 2 * D, kPlaces = 16 * kU;
  constexpr int kWords = kMx ? (kDb + 1) / 2 : kDb;          // of 16 bytes a lane and key
  const CacheView &c = a.cache;
  const int lane = threadIdx.x, col = lane & 15, g = lane >> 4;
  const int64_t pair = blockIdx.x / chunks;
  const int s = int(pair / c.kv_heads), kvh = int(pair - int64_t(s) * c.kv_heads);
  const int p0 = int(blockIdx.x - pair * chunks) * kPlaces;
  const int len = length_of(a.lens[s], a.max_len, a.table_width, c.page_shift);
  if (p0 >= len) return;
  const int begin = min(max(a.cu[s], 0), a.T), end = min(max(a.cu[s + 1], begin), a.T);
  const int group = a.q_heads / c.kv_heads, mask = (1 << c.page_shift) - 1;
  const int first = len - (end - begin);     // the first new token's place

  // The tokens that may see one of these places.
  int t0 = 0, t1 = end - begin;
  const int prefix = prefix_of(a.rules, s, len);
  if (p0 >= prefix) {
    t0 = max(t0, p0 - first);
    if (a.rules.window > 0) t1 = int(min(int64_t(t1), int64_t(p0) + kPlaces - 1 + a.rules.window - first));
  }
  if (t0 >= t1) return;

  int page[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u)
    page[u] = a.table[int64_t(s) * a.table_width + (min(p0 + 16 * u + col, len - 1) >> c.page_shift)];

  // 16 query rows as B operands, with what they see; the next 16 are requested before
  // these are used.
  struct Rows {
    bf16x8 q[kDb];
    float lse, slope;
    int pos, doc;
    bool live;
  };
  const int r1 = t1 * group;
  const int skip_tokens = 16 / group, skip_rows = 16 % group;
  int tok = t0 + col / group, in_token = col % group;          // this lane's row of the next 16
  auto load_rows = [&](int r0, Rows &x) {
    x.live = r0 + col < r1;
    const int mine_tok = x.live ? tok : t1 - 1, head = kvh * group + (x.live ? in_token : group - 1);
    const int token = begin + mine_tok;
    const int64_t q_row = int64_t(token) * a.q_heads + head;
#pragma unroll
    for (int kk = 0; kk < kDb; ++kk) {
      const int d = kMx && (kk | 1) < kDb ? 64 * (kk / 2) + 16 * g + 8 * (kk & 1) : 32 * kk + 8 * g;
      x.q[kk] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(a.q + q_row * D + d));
    }
    x.pos = first + mine_tok;
    x.doc = a.rules.doc_starts ? a.rules.doc_starts[token] : 0;
    x.lse = a.lse[q_row];
    x.slope = a.rules.slopes ? a.rules.slopes[head] * kLog2e : 0.0f;
    tok += skip_tokens, in_token += skip_rows;
    if (in_token >= group) ++tok, in_token -= group;
  };

  Rows rows[2];
  load_rows(t0 * group, rows[0]);

  // Keys as they lie in the cache: place 16 u + col.
  u32x4 word[kU][kWords];
  uint32_t key_scale[kU][kWords];
  uint64_t absent = 0;                       // bit 16 u + x: place 16 u + x is on no page of the cache
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int p = p0 + 16 * u + col;
    const bool there = p < len && unsigned(page[u]) < unsigned(c.pages);
    absent |= (__ballot(!there) & 0xFFFFu) << (16 * u);
    const int64_t place = there ? ((int64_t(page[u]) * c.kv_heads + kvh) << c.page_shift) + (p & mask) : 0;
    const uint8_t *const src = static_cast<const uint8_t *>(c.k) + place * kRowBytes;
    const uint8_t *const sc = c.k_scales + place * kDb;
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      if constexpr (!kMx) {
        word[u][j] = *reinterpret_cast<const u32x4 *>(src + 64 * j + 16 * g);
      } else if (2 * j + 1 < kDb) {          // 16 bytes are two of the matrix core's steps
        word[u][j] = *reinterpret_cast<const u32x4 *>(src + 64 * j + 16 * g);
        key_scale[u][j] = sc[2 * j + (g >> 1)];
      } else {
        const u32x2 x = *reinterpret_cast<const u32x2 *>(src + 64 * j + 8 * g);
        word[u][j] = u32x4{x[0], x[1], 0, 0};
        key_scale[u][j] = sc[2 * j];
      }
    }
  }
  // Lane col of a row of 4 kU lanes writes place 16 (col / 4) + 4 g + col % 4.
  const int out_p = p0 + 16 * (col / 4) + 4 * g + col % 4;
  float *const out = a.weights + pair * a.weights_stride + out_p;
  const bool writes = col < 4 * kU && out_p < len;
  const float old = writes ? *out : 0.0f;

  bf16x8 k[kU][kDb];                         // A operands
#pragma unroll
  for (int u = 0; u < kU; ++u)
#pragma unroll
    for (int kk = 0; kk < kDb; ++kk) {
      if constexpr (kMx) {
        const uint32_t x = word[u][kk / 2][2 * (kk % 2)], y = word[u][kk / 2][2 * (kk % 2) + 1];
        const float f = e8m0_to_float(key_scale[u][kk / 2]);
        k[u][kk] = as_frag(mx_pair(x, f, false), mx_pair(x, f, true), mx_pair(y, f, false), mx_pair(y, f, true));
      } else {
        k[u][kk] = __builtin_bit_cast(bf16x8, word[u][kk]);
      }
    }

  const float unit = a.rules.cap > 0.0f ? a.scale / a.rules.cap : a.scale * kLog2e;
  const float cap2 = a.rules.cap * kLog2e;
  bool bad = false;
  f32x4 sum[kU] = {};
  auto add_rows = [&](const Rows &x) {
    f32x4 z[kU] = {};
#pragma unroll
    for (int kk = 0; kk < kDb; ++kk)
#pragma unroll
      for (int u = 0; u < kU; ++u) z[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k[u][kk], x.q[kk], z[u], 0, 0, 0);
    const RowSees r = row_sees(a.rules, prefix, x.doc, x.pos, len);
    const bool weighs = x.live & (x.lse != -INFINITY);
    const float lse = weighs ? x.lse * kLog2e : INFINITY;        // a row without weights: 2^-infinity
    const bool all = ((p0 >= r.lo) & (p0 + kPlaces <= r.lo + r.n)) | ((p0 >= r.first) & (p0 + kPlaces <= r.first + r.m));
    float times = unit;
    if (a.rules.cap > 0.0f) {
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float y = z[u][j] * unit, small = tanh_small(y), large = tanh_large(y);
          z[u][j] = cap2 * (fabsf(y) <= kTanhSplit ? small : large);
        }
      times = 1.0f;
    }
    if (a.rules.slopes) {
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          z[u][j] = __builtin_fmaf(-x.slope, float(abs(x.pos - p0 - (16 * u + 4 * g + j))), z[u][j] * times);
      times = 1.0f;
    }
    if (absent == 0 && __all(all)) {         // every row sees every place
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(z[u][j], times, -lse));
          sum[u][j] += weighs ? e : 0.0f;
        }
    } else {
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int at = 16 * u + 4 * g + j;
          const bool seen = x.live & sees(r, p0 + at), gone = absent >> at & 1;
          bad |= seen & gone;
          const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(z[u][j], times, -lse));
          sum[u][j] += (seen & weighs & !gone) ? e : 0.0f;
        }
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
  float total = 0.0f;
#pragma unroll
  for (int u = 0; u < kU; ++u)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x = sum[u][j];
#pragma unroll
      for (int d = 1; d < 16; d *= 2) x += __shfl_xor(x, d);
      total = col == 4 * u + j ? x : total;
    }
  if (writes) *out = old + total;
}

// Few rows a sequence: what counts is how many waves have keys on their way, and 32 places
// leave registers for 16 of them on a compute unit (64 streams of up to 4095 places in 8 bits,
// 4 rows a key-value head, in workgroups of 4 waves: 66 us, with 64 places 91).  Many rows: that a row's part is shared
// (64 tokens after 16320 places, 256 rows a head: 31 us, with 32 places 41, in workgroups of 4).
constexpr int tiles_of(int db, bool few) { return few || db > 4 ? 2 : 4; }
bool few_rows(int32_t T, int32_t n_seqs, int32_t group) { return int64_t(T) * group <= 32 * int64_t(n_seqs); }
int64_t chunks_of(int32_t max_len, int tiles) {
  return (max_len + int64_t(16) * tiles - 1) / (16 * tiles);
}

template <int kDb, bool kFew>
hipError_t launch(const CacheWeights &a, hipStream_t stream) {
  constexpr int kU = tiles_of(kDb, kFew);
  const int64_t chunks = chunks_of(a.max_len, kU), blocks = int64_t(a.n_seqs) * a.cache.kv_heads * chunks;
  if (a.cache.k_scales)
    hipLaunchKernelGGL((cache_weights_kernel<kDb, true, kU>), dim3(unsigned(blocks)), dim3(kThreads), 0, stream, a,
                       int(chunks));
  else
    hipLaunchKernelGGL((cache_weights_kernel<kDb, false, kU>), dim3(unsigned(blocks)), dim3(kThreads), 0, stream, a,
                       int(chunks));
  return hipGetLastError();
}

template <int kDb>
hipError_t by_rows(const CacheWeights &a, hipStream_t stream) {
  return few_rows(a.T, a.n_seqs, a.q_heads / a.cache.kv_heads) ? launch<kDb, true>(a, stream) : launch<kDb, false>(a, stream);
}

}  // namespace

int64_t cache_weights_blocks(int32_t n_seqs, int32_t kv_heads, int32_t max_len) {
  return (int64_t(n_seqs) * kv_heads * chunks_of(max_len, 2) + 3) / 4;
}

hipError_t launch_cache_weights(const CacheWeights &a, hipStream_t stream) {
  switch (a.cache.head_dim / 32) {
    case 1: return by_rows<1>(a, stream);
    case 2: return by_rows<2>(a, stream);
    case 3: return by_rows<3>(a, stream);
    case 4: return by_rows<4>(a, stream);
    case 5: return by_rows<5>(a, stream);
    case 6: return by_rows<6>(a, stream);
    case 7: return by_rows<7>(a, stream);
    default: return by_rows<8>(a, stream);
  }
}

}  // namespace engram
