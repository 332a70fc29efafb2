// The places of largest weight of each sequence and key-value head, in their order,
// copied to other pages: select_kernel finds them, move_kernel copies.
//
// A workgroup selects for one head: the weights as whole numbers of the same order,
// then the keep-th largest by its digits (11, 11 and 10 bits, a histogram each), then
// one pass in the places' order that numbers the places above it, and as many of
// those equal to it as there is room for, the first ones.  Up to 32768 weights stay
// in the threads' registers, so they are read once; what takes the time is the
// histograms' atomics and the chain of scans (one head of 32768 places 36 us, 128 of up
// to 4608 18 us).  The copy is bound by memory: 16 bytes a thread and tensor,
// neighbours on neighbouring ones (258 MB in 47 us, 5.5 TB/s).
#include <algorithm>

#include "attention_common.hpp"
#include "tile_plan.hpp"

namespace engram {
namespace {

using namespace attn;

constexpr int kThreads = 1024, kBins = 2048, kSlab = 4 * kThreads, kHeld = 8;

// Four weights at any address of a weight.
typedef float Unaligned4 __attribute__((ext_vector_type(4), aligned(4)));

// Whole numbers in the order of the weights: NaN lowest, -0 equal to 0.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (!(x == x)) return 0;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The sum of x over the threads before this one; *total: over all of them.
__device__ __forceinline__ uint32_t scan_before(uint32_t x, uint32_t *lds, uint32_t *total) {
  uint32_t upto = x;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t y = __shfl_up(upto, d);
    if (int(threadIdx.x & 63) >= d) upto += y;
  }
  if ((threadIdx.x & 63) == 63) lds[threadIdx.x >> 6] = upto;
  __syncthreads();
  uint32_t sum = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) {
    if (w == int(threadIdx.x >> 6)) upto += sum;
    sum += lds[w];
  }
  *total = sum;
  __syncthreads();
  return upto - x;
}

__global__ __launch_bounds__(kThreads) void select_kernel(CacheEvict a) {
  __shared__ uint32_t bins[kBins];
  __shared__ uint32_t scan_lds[kThreads / 64];
  __shared__ uint32_t found_lds[2];
  const int tid = threadIdx.x, kv_heads = a.cache.kv_heads;
  const int64_t pair = blockIdx.x;
  const int s = int(pair / kv_heads);
  const int len = length_of(a.lens[s], a.max_len, a.table_width, a.cache.page_shift);
  const int count = min(len, a.keep);
  const float *const weights = a.weights + pair * a.weights_stride;
  float *const new_weights = a.new_weights + pair * a.new_weights_stride;
  int32_t *const kept = a.kept + pair * a.keep;
  if (tid == 0 && pair == int64_t(s) * kv_heads) a.new_lens[s] = count;
  for (int i = count + tid; i < a.keep; i += kThreads) kept[i] = -1;
  for (int64_t i = count + tid; i < a.new_weights_stride; i += kThreads) new_weights[i] = 0.0f;
  if (len <= a.keep || count == 0) {         // all or nothing: there is no count-th largest to look for
    for (int i = tid; i < count; i += kThreads) kept[i] = i, new_weights[i] = weights[i];
    return;
  }

  // The first and the last places are above all weights.  A thread has 4 neighbouring
  // places of every 4096; the first kHeld times 4096 stay in its registers.
  const int sinks = a.sinks, recent = len - a.recent;
  auto keys_of = [&](const f32x4 &w, int p) {
    u32x4 key;
#pragma unroll
    for (int j = 0; j < 4; ++j) key[j] = p + j < sinks || p + j >= recent ? 0xFFFFFFFFu : key_of(w[j]);
    return key;
  };
  auto weights_at = [&](int p) {
    f32x4 w{};
    if (p + 4 <= len) {
      w = *reinterpret_cast<const Unaligned4 *>(weights + p);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (p + j < len) w[j] = weights[p + j];
    }
    return w;
  };
  const int slabs = (len + kSlab - 1) / kSlab;
  f32x4 held[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (i < slabs) held[i] = weights_at(i * kSlab + 4 * tid);
  auto each_slab = [&](auto &&f) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (i < slabs) f(i * kSlab + 4 * tid, held[i]);
    for (int i = kHeld; i < slabs; ++i) f(i * kSlab + 4 * tid, weights_at(i * kSlab + 4 * tid));
  };

  uint32_t want = uint32_t(count), limit = 0, known = 0;      // the want-th largest of those that begin as `limit`
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digit = pass == 2 ? 0x3FFu : 0x7FFu;
    for (int i = tid; i < kBins; i += kThreads) bins[i] = 0;
    __syncthreads();
    each_slab([&](int p, const f32x4 &w) {
      const u32x4 key = keys_of(w, p);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool mine = p + j < len && (key[j] & known) == limit;
        const uint32_t bin = key[j] >> shift & digit;
        // Equal weights are common (none at all): one addition for a wave's most likely bin.
        const uint64_t live = __ballot(mine);
        if (live == 0) continue;
        const uint32_t likely = __builtin_amdgcn_readlane(bin, __builtin_ctzll(live));
        const uint64_t same = __ballot(mine && bin == likely);
        if (mine && bin != likely) atomicAdd(&bins[bin], 1u);
        if ((tid & 63) == 0) atomicAdd(&bins[likely], uint32_t(__popcll(same)));
      }
    });
    __syncthreads();
    // Bins from the highest on: thread i has 2047 - 2 i and 2046 - 2 i.
    const uint32_t hi = bins[kBins - 1 - 2 * tid], lo = bins[kBins - 2 - 2 * tid];
    uint32_t total;
    const uint32_t above = scan_before(hi + lo, scan_lds, &total);
    if (want > above && want <= above + hi) found_lds[0] = kBins - 1 - 2 * tid, found_lds[1] = want - above;
    if (want > above + hi && want <= above + hi + lo)
      found_lds[0] = kBins - 2 - 2 * tid, found_lds[1] = want - above - hi;
    __syncthreads();
    limit |= found_lds[0] << shift;
    known |= digit << shift;
    want = found_lds[1];
    __syncthreads();
  }

  // Those above the limit, and the first `want` of those equal to it.
  uint32_t above = 0, equal = 0;
  each_slab([&](int p, const f32x4 &w) {
    const u32x4 key = keys_of(w, p);
    uint32_t mine = 0;                       // equal ones in the upper half, above it in the lower
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (p + j < len) mine += key[j] > limit ? 1u : key[j] == limit ? 0x10000u : 0u;
    uint32_t total;
    const uint32_t before = scan_before(mine, scan_lds, &total);
    uint32_t up = above + (before & 0xFFFFu), eq = equal + (before >> 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (p + j >= len) break;
      const bool is_above = key[j] > limit, is_equal = key[j] == limit;
      if (is_above || (is_equal && eq < want)) {
        const uint32_t at = up + min(eq, want);
        kept[at] = p + j;
        new_weights[at] = w[j];
      }
      up += is_above, eq += is_equal;
    }
    above += total & 0xFFFFu, equal += total >> 16;
  });
}

constexpr int kMoveThreads = 256;

template <bool kMx>
__global__ __launch_bounds__(kMoveThreads) void move_kernel(CacheEvict a, int pieces, int64_t blocks_of_head) {
  const CacheView &c = a.cache;
  const int64_t pair = blockIdx.x / blocks_of_head;
  const int s = int(pair / c.kv_heads), kvh = int(pair - int64_t(s) * c.kv_heads);
  const int64_t id = (blockIdx.x - pair * blocks_of_head) * kMoveThreads + threadIdx.x;
  const int i = int(id / pieces), at = int(id - int64_t(i) * pieces);
  if (i >= a.keep) return;
  const int p = a.kept[pair * a.keep + i];
  if (p < 0) return;
  const int mask = (1 << c.page_shift) - 1;
  const int page = a.table[int64_t(s) * a.table_width + (p >> c.page_shift)];
  const int to = a.to_table[int64_t(s) * a.to_width + (i >> c.page_shift)];
  const bool there = unsigned(page) < unsigned(c.pages), room = unsigned(to) < unsigned(c.pages);
  if (!(there && room) && at == 0 && kvh == 0 && a.bad_pages) atomicAdd(a.bad_pages, 1);
  if (!room) return;
  const int64_t src = there ? ((int64_t(page) * c.kv_heads + kvh) << c.page_shift) + (p & mask) : 0;
  const int64_t dst = ((int64_t(to) * c.kv_heads + kvh) << c.page_shift) + (i & mask);
  u32x4 k = static_cast<const u32x4 *>(c.k)[src * pieces + at];
  u32x4 v = static_cast<const u32x4 *>(c.v)[src * pieces + at];
  if (!there) k = v = u32x4{};
  static_cast<u32x4 *>(c.k)[dst * pieces + at] = k;
  static_cast<u32x4 *>(c.v)[dst * pieces + at] = v;
  if (kMx && at % 2 == 0) {
    const int blocks = pieces / 2;
    c.k_scales[dst * blocks + at / 2] = there ? c.k_scales[src * blocks + at / 2] : 127;
    c.v_scales[dst * blocks + at / 2] = there ? c.v_scales[src * blocks + at / 2] : 127;
  }
}

inline int pieces_of(const CacheView &c) { return c.head_dim / (c.k_scales ? 16 : 8); }
inline int64_t head_blocks(int64_t keep, int pieces) { return (keep * pieces + kMoveThreads - 1) / kMoveThreads; }

}  // namespace

int64_t cache_evict_blocks(const CacheView &c, int32_t n_seqs, int32_t keep) {
  return int64_t(n_seqs) * c.kv_heads * std::max<int64_t>(1, head_blocks(keep, pieces_of(c)));
}

hipError_t launch_cache_evict(const CacheEvict &a, hipStream_t stream) {
  const int64_t pairs = int64_t(a.n_seqs) * a.cache.kv_heads;
  hipLaunchKernelGGL(select_kernel, dim3(unsigned(pairs)), dim3(kThreads), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.keep == 0) return e;
  const int pieces = pieces_of(a.cache);
  const int64_t blocks = head_blocks(a.keep, pieces);
  if (a.cache.k_scales)
    hipLaunchKernelGGL(move_kernel<true>, dim3(unsigned(pairs * blocks)), dim3(kMoveThreads), 0, stream, a, pieces, blocks);
  else
    hipLaunchKernelGGL(move_kernel<false>, dim3(unsigned(pairs * blocks)), dim3(kMoveThreads), 0, stream, a, pieces, blocks);
  return hipGetLastError();
}

}  // namespace engram
