// Per-head RMS norm of queries and keys and their rotation, out of one row of
// the QKV projection, the keys (and values) into the paged cache where asked.
//
//   y = x / sqrt(mean(x^2) + eps) * w;  (a, b) -> (a cos - b sin, b cos + a sin)
//
// Bound by the bytes of qkv, q and k.  A wave takes a token's heads, LP lanes
// a head (kv_cache.hpp), so a token's angles are formed once a wave, one a
// lane: position * inv_freq in fp64, in turns, less the nearest whole number
// (an angle at position 10^6 in fp32 would be off by 0.06), then sine and
// cosine of the remaining half turn in fp32.  A lane holds two pieces of 8
// values such that both members of a pair are its own: with halves, the
// pieces sub and sub + rotary_dim/16; interleaved or past rotary_dim, the
// pieces 2 sub and 2 sub + 1.  In either layout its 8 pairs are the pairs
// 8 sub .. 8 sub + 7, so its 8 angles serve every head.
#include "kv_cache.hpp"

namespace engram {
namespace {

using namespace kvc;

constexpr int kMaxPairs = ENGRAM_MAX_ATTN_HEAD_DIM / 2;
constexpr int kRowShorts = 1024;          // 64 / LP rows of 16 LP values

__device__ __forceinline__ void wave_sync() {
  // LDS written by one lane of a wave, read by another: the hardware keeps a
  // wave's LDS accesses in order, the compiler has to as well.
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ void unpack8(const u32x4 q, float *x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[2 * i] = bf16_lo(q[i]), x[2 * i + 1] = bf16_hi(q[i]);
}

enum CacheMode { kNoCache, kBf16, kMxfp8 };

template <int LP, bool kInter, CacheMode kMode>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_kernel(QkRope a) {
  constexpr int kRows = 64 / LP;
  __shared__ __attribute__((aligned(16))) float2 cs_lds[kWaves][kMaxPairs];
  __shared__ __attribute__((aligned(16))) uint16_t row_lds[kMode == kNoCache ? 1 : kWaves][kRowShorts];

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int sub = lane % LP, in_wave = lane / LP;
  const int64_t id = int64_t(blockIdx.x) * kWaves + wave;
  const int64_t t = id / a.waves_per_token;
  if (t >= a.T) return;                              // the whole wave; no barrier below
  const int first = int(id - t * a.waves_per_token) * a.heads_per_wave;
  const int last = min(a.heads, first + a.heads_per_wave);
  const int D = a.head_dim, half = a.rotary_dim / 2;

  // The wave's angles, and this lane's 8 of them.
  float2 *cs = cs_lds[wave];
  const double pos = double(a.positions[t]);
  for (int i = lane; i < half; i += 64) {
    const double turns = pos * a.inv_freq[i] * 0.15915494309189535;      // 1 / (2 pi)
    float s, c;
    sincospif(2.0f * float(turns - rint(turns)), &s, &c);
    cs[i] = float2{c, s};
  }
  wave_sync();
  const bool lane_on = 16 * sub < D;
  const int nrot = a.rotary_dim / 16;
  const bool rotated = sub < nrot;
  const int pa = 8 * (rotated && !kInter ? sub : 2 * sub);
  const int pb = rotated && !kInter ? pa + 8 * nrot : pa + 8;
  float cosv[8], sinv[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 v = cs[rotated ? 8 * sub + j : 0];
    cosv[j] = v.x, sinv[j] = v.y;
  }

  const uint16_t *row = a.qkv + t * a.token_stride;
  int64_t slot = -1;
  bool slot_in = false;
  if constexpr (kMode != kNoCache) {
    slot = a.slots[t];
    slot_in = slot_ok(a.cache, slot);
    if (!slot_in && slot != -1 && a.bad_slots && first == 0 && lane == 0) atomicAdd(a.bad_slots, 1);
  }

  for (int h0 = first; h0 < last; h0 += kRows) {
    const int h = h0 + in_wave;
    const bool on = h < last && lane_on;
    const bool is_v = h >= a.q_heads + a.kv_heads;
    const bool is_k = !is_v && h >= a.q_heads;
    const int oa = is_v ? 16 * sub : pa, ob = is_v ? 16 * sub + 8 : pb;
    u32x4 ra{}, rb{};
    if (on) {
      ra = *reinterpret_cast<const u32x4 *>(row + h * D + oa);
      rb = *reinterpret_cast<const u32x4 *>(row + h * D + ob);
    }
    float x[16];
    unpack8(ra, x);
    unpack8(rb, x + 8);
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int m = 1; m < LP; m *= 2) ss += __shfl_xor(ss, m);
    const float r = 1.0f / sqrtf(ss / float(D) + a.eps);
    float w[16] = {};
    if (on) {
      const uint16_t *wt = is_k ? a.k_weight : a.q_weight;
      unpack8(*reinterpret_cast<const u32x4 *>(wt + pa), w);
      unpack8(*reinterpret_cast<const u32x4 *>(wt + pb), w + 8);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = x[i] * r * w[i];
    if (rotated) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int ia = kInter ? 2 * j : j, ib = kInter ? 2 * j + 1 : 8 + j;
        const float u = x[ia], v = x[ib];
        x[ia] = u * cosv[j] - v * sinv[j];
        x[ib] = v * cosv[j] + u * sinv[j];
      }
    }
    if (!is_v) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ra[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
        rb[i] = pack_bf16x2(x[8 + 2 * i], x[9 + 2 * i]);
      }
    }
    if (on && !is_v) {
      uint16_t *dst = !is_k ? a.q + (t * a.q_heads + h) * D
                            : a.k ? a.k + (t * a.kv_heads + h - a.q_heads) * D : nullptr;
      if (dst) {
        *reinterpret_cast<u32x4 *>(dst + oa) = ra;
        *reinterpret_cast<u32x4 *>(dst + ob) = rb;
      }
    }
    if constexpr (kMode != kNoCache) {
      if (h0 + kRows <= a.q_heads) continue;         // only queries in this pass
      // Keys and values to 16 consecutive values a lane, by way of LDS.
      uint16_t *mine = row_lds[wave] + in_wave * 16 * LP;
      if (lane_on) {
        *reinterpret_cast<u32x4 *>(mine + oa) = ra;
        *reinterpret_cast<u32x4 *>(mine + ob) = rb;
      }
      wave_sync();
      const u32x4 lo = *reinterpret_cast<const u32x4 *>(mine + 16 * sub);
      const u32x4 hi = *reinterpret_cast<const u32x4 *>(mine + 16 * sub + 8);
      wave_sync();
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = lo[i], o[4 + i] = hi[i];
      const bool put = on && slot_in && (is_k || is_v);
      const int head = is_v ? h - a.q_heads - a.kv_heads : h - a.q_heads;
      store16<kMode == kMxfp8>(is_v ? a.cache.v : a.cache.k,
                               is_v ? a.cache.v_scales : a.cache.k_scales, D,
                               put ? row_index(a.cache, slot, head) : 0, sub, put, o);
    }
  }
}

template <int LP, bool kInter, CacheMode kMode>
void launch(const QkRope &a, unsigned blocks, hipStream_t stream) {
  hipLaunchKernelGGL((qk_norm_rope_kernel<LP, kInter, kMode>), dim3(blocks), dim3(kThreads), 0,
                     stream, a);
}

template <int LP, bool kInter>
void by_cache(const QkRope &a, unsigned blocks, hipStream_t stream) {
  if (!a.cache.k) launch<LP, kInter, kNoCache>(a, blocks, stream);
  else if (!a.cache.k_scales) launch<LP, kInter, kBf16>(a, blocks, stream);
  else launch<LP, kInter, kMxfp8>(a, blocks, stream);
}

template <int LP>
void by_pairs(const QkRope &a, bool inter, unsigned blocks, hipStream_t stream) {
  if (inter) by_cache<LP, true>(a, blocks, stream);
  else by_cache<LP, false>(a, blocks, stream);
}

}  // namespace

int64_t qk_rope_plan(QkRope *a) {
  a->heads = a->q_heads + (a->cache.k ? 2 : 1) * a->kv_heads;
  a->heads_per_wave = a->heads;
  a->waves_per_token = (a->heads + a->heads_per_wave - 1) / a->heads_per_wave;
  return (int64_t(a->T) * a->waves_per_token + kWaves - 1) / kWaves;
}

hipError_t launch_qk_norm_rope(const QkRope &a, bool interleaved, int64_t blocks,
                               hipStream_t stream) {
  const unsigned n = unsigned(blocks);
  switch (lanes_per_row(a.head_dim)) {
    case 2: by_pairs<2>(a, interleaved, n, stream); break;
    case 4: by_pairs<4>(a, interleaved, n, stream); break;
    case 8: by_pairs<8>(a, interleaved, n, stream); break;
    default: by_pairs<16>(a, interleaved, n, stream);
  }
  return hipGetLastError();
}

}  // namespace engram
