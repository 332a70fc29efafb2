// Per-head RMS norm of queries and keys and their rotation, out of one row of
// the QKV projection, the keys (and values) into the paged cache where asked.
//
//   y = x / sqrt(mean(x^2) + eps) * w;  (a, b) -> (a cos - b sin, b cos + a sin)
//
// Bound by the bytes of qkv, q and k: 8192 tokens of 32 + 8 heads of 128 take
// 32 us, 5.2 TB/s.  A wave takes some of a token's heads, LP lanes a head; all
// of its rows are requested before its angles are formed, one a lane: position *
// inv_freq in fp64, in turns, less the nearest whole number (an angle at
// position 10^6 in fp32 would be off by 0.06).  A lane holds two pieces of 8
// values such that both members of a pair are its own: with halves, the pieces
// sub and sub + rotary_dim/16; interleaved or past rotary_dim, the pieces 2 sub
// and 2 sub + 1.  In either layout its 8 pairs are the pairs 8 sub .. 8 sub + 7,
// so its 8 angles serve every head.
//
// Waves have queries only, in fp32, or keys too (and the queries that share a
// pass with them), in fp64: a cache in 8 bits rounds the keys again, and fp32
// leaves 3 values of 2048 x 8 x 128 on the wrong side of both borders at once, a
// whole step of 8 bits off (fp64 none).  At 8192 tokens that costs 1.7 us.  An
// fp64 result is rounded to fp32 and that to bf16, as a conversion of a double
// does: 1 in 2^17 is then half-way between two bf16 values and goes to the even
// one.
//
// Two passes a wave and 5 waves a SIMD: one register more for each value in
// flight costs more than it brings (4 passes, 117 registers: 36.4 us).
#include "kv_cache.hpp"

namespace engram {
namespace {

using namespace kvc;

constexpr int kMaxPairs = ENGRAM_MAX_ATTN_HEAD_DIM / 2;
constexpr int kMaxPasses = 2;             // of a wave
constexpr int64_t kFewWaves = 4096;
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

// cos(pi t), sin(pi t) for |t| <= 1: the quarter turn it is in, and the series
// of the rest, at most pi/4 away (the first terms left out are below 2^-41).
__device__ __forceinline__ double2 cos_sin(double t) {
  const double quarter = rint(2.0 * t), x = (t - 0.5 * quarter) * 3.14159265358979323846;
  const double y = x * x;
  double c = -1.0 / 3628800 + y * (1.0 / 479001600);
  c = fma(y, c, 1.0 / 40320);
  c = fma(y, c, -1.0 / 720);
  c = fma(y, c, 1.0 / 24);
  c = fma(y, c, -0.5);
  c = fma(y, c, 1.0);
  double s = -1.0 / 39916800 + y * (1.0 / 6227020800);
  s = fma(y, s, 1.0 / 362880);
  s = fma(y, s, -1.0 / 5040);
  s = fma(y, s, 1.0 / 120);
  s = fma(y, s, -1.0 / 6);
  s = fma(x * y, s, x);
  const int q = int(quarter) & 3;
  const double a = q & 1 ? s : c, b = q & 1 ? c : s;
  return double2{q == 1 || q == 2 ? -a : a, q >= 2 ? -b : b};
}

// Lanes of a head, 16 values each: head_dim / 16 rounded up to a power of two,
// at least 4 (a block of the cache's 8-bit format); those past head_dim / 16 idle.
inline int lanes_per_row(int head_dim) {
  const int n = head_dim / 16;
  return n <= 4 ? 4 : n <= 8 ? 8 : 16;
}

// 8 values times r to bf16.
__device__ __forceinline__ u32x4 pack8(const float *x, float r) {
  return u32x4{pack_bf16x2(x[0] * r, x[1] * r), pack_bf16x2(x[2] * r, x[3] * r),
               pack_bf16x2(x[4] * r, x[5] * r), pack_bf16x2(x[6] * r, x[7] * r)};
}

enum CacheMode { kNoCache, kBf16, kMxfp8 };

template <int LP, bool kInter, CacheMode kMode, int kPass>
__global__ __launch_bounds__(kThreads, 5) void qk_norm_rope_kernel(QkRope a) {
  constexpr int kRows = 64 / LP;
  __shared__ __attribute__((aligned(16))) double2 cs_lds[kWaves][kMaxPairs];
  __shared__ __attribute__((aligned(16))) uint16_t row_lds[kMode == kNoCache ? 1 : kWaves][kRowShorts];

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int sub = lane % LP, in_wave = lane / LP;
  const int64_t id = int64_t(blockIdx.x) * kWaves + wave;
  const int64_t t = id / a.waves_per_token;
  if (t >= a.T) return;                              // the whole wave; no barrier below
  const int part = int(id - t * a.waves_per_token);
  // Passes of queries only, and the others: waves of their own.
  const int q_passes = a.q_heads / kRows, kv_passes = (a.heads + kRows - 1) / kRows - q_passes;
  const int kv_part = part - a.q_waves;
  const bool keys = kv_part >= 0;
  const int pass0 = keys ? q_passes + kPass * kv_part : kPass * part;
  const int pass1 = min(pass0 + kPass, keys ? q_passes + kv_passes : q_passes);
  const int D = a.head_dim, half = a.rotary_dim / 2;

  // All of the wave's rows are requested before anything is waited for.
  const bool lane_on = 16 * sub < D;
  const int nrot = a.rotary_dim / 16;
  const bool rotated = sub < nrot;
  const int pa = 8 * (rotated && !kInter ? sub : 2 * sub);
  const int pb = rotated && !kInter ? pa + 8 * nrot : pa + 8;
  const uint16_t *row = a.qkv + t * a.token_stride;
  u32x4 ra[kPass], rb[kPass];
#pragma unroll
  for (int i = 0; i < kPass; ++i) {
    const int h = (pass0 + i) * kRows + in_wave;
    const bool is_v = h >= a.q_heads + a.kv_heads;
    ra[i] = rb[i] = u32x4{};
    if (pass0 + i < pass1 && h < a.heads && lane_on) {
      ra[i] = load16<kPass != 1>(row + h * D + (is_v ? 16 * sub : pa));
      rb[i] = load16<kPass != 1>(row + h * D + (is_v ? 16 * sub + 8 : pb));
    }
  }
  u32x4 wa{}, wb{};
  if (lane_on) {
    wa = *reinterpret_cast<const u32x4 *>(a.q_weight + pa);
    wb = *reinterpret_cast<const u32x4 *>(a.q_weight + pb);
  }
  int64_t slot = -1;
  bool slot_in = false;
  if constexpr (kMode != kNoCache) {
    slot = a.slots[t];
    slot_in = slot_ok(a.cache, slot);
    if (!slot_in && slot != -1 && a.bad_slots && part == 0 && lane == 0) atomicAdd(a.bad_slots, 1);
  }

  // The wave's angles, and this lane's 8 of them.
  double2 *cs = cs_lds[wave];
  const double pos = double(a.positions[t]);
  for (int i = lane; i < half; i += 64) {
    const double turns = pos * a.inv_freq[i] * 0.15915494309189535;      // 1 / (2 pi)
    const double halves = 2.0 * (turns - rint(turns));
    if (keys) {
      cs[i] = cos_sin(halves);
    } else {
      const float f = float(halves), rest = 3.14159265f * float(halves - double(f));
      float s, c;
      sincospif(f, &s, &c);
      reinterpret_cast<float2 *>(cs)[i] = float2{fmaf(-s, rest, c), fmaf(c, rest, s)};
    }
  }
  wave_sync();
  const int my_cs = rotated ? 8 * sub : 0;

  if (!keys) {
    // In fp32; x * weight is exact (two times 8 bits), and the norm, common to the
    // head, comes last.
    float cosv[8], sinv[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 v = reinterpret_cast<const float2 *>(cs)[my_cs + j];
      cosv[j] = v.x, sinv[j] = v.y;
    }
    float w[16];
    unpack8(wa, w);
    unpack8(wb, w + 8);
#pragma unroll
    for (int i = 0; i < kPass; ++i) {
      if (pass0 + i >= pass1) break;
      const int h = (pass0 + i) * kRows + in_wave;
      float x[16];
      unpack8(ra[i], x);
      unpack8(rb[i], x + 8);
      float ss = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int m = 1; m < LP; m *= 2) ss += __shfl_xor(ss, m);
      const float r = 1.0f / sqrtf(fmaf(ss, a.inv_dim, a.eps));
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] *= w[e];
      if (rotated) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int ia = kInter ? 2 * j : j, ib = kInter ? 2 * j + 1 : 8 + j;
          const float u = x[ia], v = x[ib];
          x[ia] = fmaf(u, cosv[j], -(v * sinv[j]));
          x[ib] = fmaf(v, cosv[j], u * sinv[j]);
        }
      }
      if (!lane_on) continue;
      uint16_t *dst = a.q + (t * a.q_heads + h) * D;
      save16<kPass != 1>(dst + pa, pack8(x, r));
      save16<kPass != 1>(dst + pb, pack8(x + 8, r));
    }
    return;
  }

  // With keys: in fp64 up to the results, so that what an 8-bit cache rounds again
  // lies on the right side of its borders.
#pragma unroll
  for (int i = 0; i < kPass; ++i) {
    if (pass0 + i >= pass1) break;
    const int h = (pass0 + i) * kRows + in_wave;
    const bool on = h < a.heads && lane_on;
    const bool is_v = h >= a.q_heads + a.kv_heads;
    const bool is_k = !is_v && h >= a.q_heads;
    const int oa = is_v ? 16 * sub : pa, ob = is_v ? 16 * sub + 8 : pb;
    if ((pass0 + i) * kRows < a.q_heads + a.kv_heads) {
      float x[16], w[16];
      unpack8(ra[i], x);
      unpack8(rb[i], x + 8);
      u32x4 w0{}, w1{};
      if (lane_on) {
        const uint16_t *wt = is_k ? a.k_weight : a.q_weight;
        w0 = *reinterpret_cast<const u32x4 *>(wt + pa);
        w1 = *reinterpret_cast<const u32x4 *>(wt + pb);
      }
      unpack8(w0, w);
      unpack8(w1, w + 8);
      double ss = 0.0;
#pragma unroll
      for (int e = 0; e < 16; ++e) ss = fma(double(x[e]), double(x[e]), ss);
#pragma unroll
      for (int m = 1; m < LP; m *= 2) ss += __shfl_xor(ss, m);
      const double r = rsqrt(fma(ss, 1.0 / D, double(a.eps)));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int ia = kInter ? 2 * j : j, ib = kInter ? 2 * j + 1 : 8 + j;
        const double2 v = cs[my_cs + j];
        const double p = double(x[ia] * w[ia]), q = double(x[ib] * w[ib]);
        // Past rotary_dim p and q alone: the terms of 0 are of 0 times 0, as an
        // infinity times 0 is NaN.  (Selecting the results instead: 1.2 us of 31 more
        // for 2048 tokens into an 8-bit cache.)
        const double c = rotated ? v.x : 1.0, sn = rotated ? v.y : 0.0;
        const double ps = rotated ? p : 0.0, qs = rotated ? q : 0.0;
        x[ia] = float(fma(p, c, -(qs * sn)) * r);
        x[ib] = float(fma(q, c, ps * sn) * r);
      }
      if (!is_v) ra[i] = pack8(x, 1.0f), rb[i] = pack8(x + 8, 1.0f);
    }
    if (on && !is_v) {
      uint16_t *dst = !is_k ? a.q + (t * a.q_heads + h) * D
                            : a.k ? a.k + (t * a.kv_heads + h - a.q_heads) * D : nullptr;
      if (dst) {
        save16<kPass != 1>(dst + oa, ra[i]);
        save16<kPass != 1>(dst + ob, rb[i]);
      }
    }
    if constexpr (kMode != kNoCache) {
      // Keys and values to 8 consecutive ones a lane and step, by way of LDS.
      uint16_t *mine = row_lds[wave] + in_wave * 16 * LP;
      if (lane_on) {
        *reinterpret_cast<u32x4 *>(mine + oa) = ra[i];
        *reinterpret_cast<u32x4 *>(mine + ob) = rb[i];
      }
      wave_sync();
      const u32x4 o[2] = {*reinterpret_cast<const u32x4 *>(mine + 8 * sub),
                          *reinterpret_cast<const u32x4 *>(mine + 8 * (LP + sub))};
      wave_sync();
      const bool put = h < a.heads && slot_in && (is_k || is_v);
      const int head = is_v ? h - a.q_heads - a.kv_heads : h - a.q_heads;
      const int64_t to = put ? row_index(a.cache, slot, head) : 0;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int piece = e * LP + sub;
        store8<kMode == kMxfp8>(is_v ? a.cache.v : a.cache.k,
                                is_v ? a.cache.v_scales : a.cache.k_scales, D, to, piece,
                                put && 8 * piece < D, o[e]);
      }
    }
  }
}

template <int LP, bool kInter, CacheMode kMode>
void launch(const QkRope &a, unsigned blocks, hipStream_t stream) {
  if (a.passes_per_wave == 1)
    hipLaunchKernelGGL((qk_norm_rope_kernel<LP, kInter, kMode, 1>), dim3(blocks), dim3(kThreads), 0,
                       stream, a);
  else
    hipLaunchKernelGGL((qk_norm_rope_kernel<LP, kInter, kMode, kMaxPasses>), dim3(blocks),
                       dim3(kThreads), 0, stream, a);
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

// A wave forms its token's angles, so it takes two passes of 64 / LP heads where
// there are waves enough.
int64_t qk_rope_plan(QkRope *a) {
  a->heads = a->q_heads + (a->cache.k ? 2 : 1) * a->kv_heads;
  a->inv_dim = 1.0f / float(a->head_dim);
  const int rows = 64 / lanes_per_row(a->head_dim), passes = (a->heads + rows - 1) / rows;
  a->passes_per_wave = int64_t(a->T) * passes <= kFewWaves ? 1 : kMaxPasses;
  const int per = a->passes_per_wave, q_passes = a->q_heads / rows;
  a->q_waves = (q_passes + per - 1) / per;
  a->waves_per_token = a->q_waves + (passes - q_passes + per - 1) / per;
  return (int64_t(a->T) * a->waves_per_token + kWaves - 1) / kWaves;
}

hipError_t launch_qk_norm_rope(const QkRope &a, bool interleaved, int64_t blocks,
                               hipStream_t stream) {
  const unsigned n = unsigned(blocks);
  switch (lanes_per_row(a.head_dim)) {
    case 4: by_pairs<4>(a, interleaved, n, stream); break;
    case 8: by_pairs<8>(a, interleaved, n, stream); break;
    default: by_pairs<16>(a, interleaved, n, stream);
  }
  return hipGetLastError();
}

}  // namespace engram
