// Attention of one new token per sequence over the paged cache.
//
//   out = sum_p e^(scale q.k_p - m) v_p / sum_p e^(scale q.k_p - m),
//   m = max_p scale q.k_p,  lse = m + log sum_p e^(scale q.k_p - m)
//
// The plain kernel: one workgroup per (sequence, query head); its 4 waves take
// 64 places at a time each, a lane a place for the scores and head_dim / 64
// dimensions for the sums, and keep a running maximum and sum of their own;
// they are joined in LDS, in wave order.
#include "kv_cache.hpp"

namespace engram {
namespace {

using namespace kvc;

constexpr int kMaxD = ENGRAM_MAX_ATTN_HEAD_DIM;

template <bool kMx>
__device__ __forceinline__ float cache_value(const void *data, const uint8_t *scales, int D,
                                             int64_t row, int d) {
  if constexpr (kMx)
    return e4m3fn_to_float(static_cast<const uint8_t *>(data)[row * D + d]) *
           e8m0_to_float(scales[row * (D / 32) + d / 32]);
  else
    return __uint_as_float(uint32_t(static_cast<const uint16_t *>(data)[row * D + d]) << 16);
}

template <bool kMx>
__global__ __launch_bounds__(kThreads) void paged_attention_kernel(PagedAttention a) {
  __shared__ float q_lds[kMaxD];
  __shared__ float p_lds[kWaves][64];
  __shared__ int64_t row_lds[kWaves][64];
  __shared__ float o_lds[kWaves][kMaxD], m_lds[kWaves], l_lds[kWaves];
  const CacheView &c = a.cache;
  const int D = c.head_dim, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t pair = blockIdx.x;
  const int64_t s = pair / a.q_heads;
  const int h = int(pair - s * a.q_heads), kvh = h / (a.q_heads / c.kv_heads);
  for (int d = threadIdx.x; d < D; d += kThreads)
    q_lds[d] = __uint_as_float(uint32_t(a.q[pair * D + d]) << 16);
  __syncthreads();
  const int32_t *table = a.table + s * a.table_width;
  const int64_t room = int64_t(a.table_width) << c.page_shift;
  const int len = int(min(int64_t(min(max(a.lens[s], 0), a.max_len)), room));
  const int start = a.window > 0 ? max(0, len - a.window) : 0;
  float m = -INFINITY, l = 0.0f, o[kMaxD / 64] = {};
  bool bad = false;
  for (int p0 = start + 64 * wave; p0 < len; p0 += 64 * kWaves) {
    const int p = p0 + lane;
    float z = -INFINITY;
    int64_t row = -1;
    if (p < len) {
      const int page = table[p >> c.page_shift];
      if (page >= 0 && page < c.pages) {
        row = row_index(c, (int64_t(page) << c.page_shift) + (p & ((1 << c.page_shift) - 1)), kvh);
        float dot = 0.0f;
        for (int d = 0; d < D; ++d)
          dot = fmaf(q_lds[d], cache_value<kMx>(c.k, c.k_scales, D, row, d), dot);
        z = dot * a.scale;
      } else {
        bad = true;
      }
    }
    float top = z;
    for (int x = 1; x < 64; x *= 2) top = fmaxf(top, __shfl_xor(top, x));
    const float mn = fmaxf(m, top);
    const float keep = mn == -INFINITY ? 0.0f : expf(m - mn);
    const float w = row < 0 ? 0.0f : expf(z - mn);
    float sum = w;
    for (int x = 1; x < 64; x *= 2) sum += __shfl_xor(sum, x);
    l = l * keep + sum;
    m = mn;
    p_lds[wave][lane] = w;
    row_lds[wave][lane] = row;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int i = 0; i < kMaxD / 64; ++i) o[i] *= keep;
    for (int j = 0; j < 64; ++j) {
      const int64_t r = row_lds[wave][j];
      if (r < 0) continue;
      const float w2 = p_lds[wave][j];
#pragma unroll
      for (int i = 0; i < kMaxD / 64; ++i)
        if (64 * i + lane < D)
          o[i] = fmaf(w2, cache_value<kMx>(c.v, c.v_scales, D, r, 64 * i + lane), o[i]);
    }
    __builtin_amdgcn_wave_barrier();
  }
  if (bad && a.bad_pages) atomicAdd(a.bad_pages, 1);
  if (lane == 0) m_lds[wave] = m, l_lds[wave] = l;
#pragma unroll
  for (int i = 0; i < kMaxD / 64; ++i)
    if (64 * i + lane < D) o_lds[wave][64 * i + lane] = o[i];
  __syncthreads();
  float mt = -INFINITY, lt = 0.0f;
  for (int w = 0; w < kWaves; ++w) mt = fmaxf(mt, m_lds[w]);
  const float mf = mt == -INFINITY ? 0.0f : mt;
  for (int w = 0; w < kWaves; ++w) lt += l_lds[w] * expf(m_lds[w] - mf);
  for (int d = threadIdx.x; d < D; d += kThreads) {
    float sum = 0.0f;
    for (int w = 0; w < kWaves; ++w) sum += o_lds[w][d] * expf(m_lds[w] - mf);
    a.out[pair * D + d] = f32_to_bf16(lt > 0.0f ? sum / lt : 0.0f);
  }
  if (threadIdx.x == 0 && a.lse) a.lse[pair] = lt > 0.0f ? mt + logf(lt) : -INFINITY;
}

}  // namespace

int64_t paged_attention_workspace(int32_t, int32_t, int32_t, int32_t, int32_t) { return 0; }

hipError_t launch_paged_attention(const PagedAttention &a, hipStream_t stream) {
  const dim3 grid(unsigned(int64_t(a.n_seqs) * a.q_heads));
  if (a.cache.k_scales)
    hipLaunchKernelGGL(paged_attention_kernel<true>, grid, dim3(kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL(paged_attention_kernel<false>, grid, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace engram
