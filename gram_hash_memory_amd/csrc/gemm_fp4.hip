// The MXFP4 copy of a bf16 weight, and the product of few tokens with it.
//
//   out[t][n] = bf16(sum_k x[t][k] * e2m1(code[n][k]) * 2^(scale[n][k/32] - 127))
//
// v_mfma_f32_16x16x32_bf16 with the weight as A and x as B; one
// v_cvt_scalef32_pk_bf16_fp4 makes two scaled bf16 values (exact).  Workgroups
// take 16 * kN columns and 16 * kM tokens, their 8 waves the steps of 128 k in
// turn, so that a row's next 512 bytes are under way at any time.
//
// Bound by reading the weight once where tokens are few (one token of 6144 x
// 20480, weights that the last cache does not hold: 16.9 us, 4.0 TB/s; of 4096 x
// 6144: 6.5 us, of which some 4 are launch and two memory latencies).  64 tokens
// of 6144 x 20480 take 28.3 us (2.5 TB/s, 0.57 PFLOP/s; 24.8 us where the weight
// is still in the last cache).  Of those cycles the matrix cores are busy 27 %,
// the VALU 30 %, LDS 21 %, the vector cache's addressing 61 % and its return path
// 73 % (every CU pulls all of x), and waves spend 35 % of theirs waiting for data.
//
// What the vector cache takes goes by the runs of addresses in 16 neighbouring
// lanes, a clock each, so neighbouring lanes read neighbouring bytes and LDS
// puts them in the matrix cores' order: weights by way of 1 KB a wave, x by
// LDS-DMA straight into the wave's own LDS.  (Both from memory into the matrix
// cores' order in registers, 16 rows in 16 lanes: 53 us instead of 28.)  The
// scales of all columns come first, in one batch: a byte a lane beside the
// weights would pull a line each (+6 us at one token).
#include <algorithm>

#include "gemm_common.hpp"

namespace engram {
namespace {

constexpr int kThreads = 256;

// e2m1 code of x (already divided by the scale), to the nearest value, ties to
// the even code, saturated: the comparisons' borders are the midpoints.
__device__ __forceinline__ uint32_t e2m1_rne(float x) {
  const float a = fabsf(x);
  const uint32_t code = uint32_t(a > 0.25f) + uint32_t(a >= 0.75f) + uint32_t(a > 1.25f) +
                        uint32_t(a >= 1.75f) + uint32_t(a > 2.5f) + uint32_t(a >= 3.5f) +
                        uint32_t(a > 5.0f);
  return code | ((__float_as_uint(x) >> 28) & 8u);
}

// One thread per block of 32 k: 64 bytes of bf16 in, 16 bytes of codes out.  A
// weight's bytes, once when it is loaded: 20480 x 6144 takes 74 us, 4.3 TB/s of
// the copy's 5.1; 4096 x 4096 13 us.
__global__ __launch_bounds__(kThreads) void quantize_fp4_kernel(const uint16_t *__restrict__ w,
                                                                int64_t blocks,
                                                                uint8_t *__restrict__ codes,
                                                                uint8_t *__restrict__ scales) {
  const int64_t b = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (b >= blocks) return;
  const u32x4 *src = reinterpret_cast<const u32x4 *>(w + b * 32);
  uint32_t v[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const u32x4 q = src[i];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[4 * i + e] = q[e];
  }
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(v[i])), fabsf(bf16_hi(v[i]))));
  int byte = 127;
  if (amax > 0.0f) {
    int e;
    frexpf(amax, &e);                       // amax = m * 2^e, 0.5 <= m < 1
    byte = min(max(e - 1 - 2 + 127, 0), 254);
  }
  const int shift = 127 - byte;             // x = w * 2^shift, exact
  u32x4 out{};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t c = e2m1_rne(ldexpf(bf16_lo(v[i]), shift)) |
                       e2m1_rne(ldexpf(bf16_hi(v[i]), shift)) << 4;
    out[i / 4] |= c << (8 * (i % 4));
  }
  *reinterpret_cast<u32x4 *>(codes + b * 16) = out;
  scales[b] = uint8_t(byte);
}

// ---------------------------------------------------------------- the product

typedef float f32x4v __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8;
constexpr int kCus = 256;
constexpr uint32_t kOutside = 0x7FFFFFF0u;      // an offset past every buffer: loads give 0

// The codes of byte kByte times the scale, as a bf16 pair (exact).
template <int kByte>
__device__ __forceinline__ uint32_t e2m1_pair(uint32_t codes, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, kByte));
}

// Blocks whose scales a workgroup holds in LDS at a time, and the pitch of a
// column's (an odd number of dwords, for the banks).
constexpr int kSegBlocks = 256;
inline __host__ __device__ int scale_pitch(int blocks) {
  const int n = blocks < kSegBlocks ? blocks : kSegBlocks;
  return ((n + 3) / 4 | 1) * 4;
}

// Dwords of scales a thread brings in.
template <int kN>
constexpr int scale_batch() {
  return (16 * kN * (kSegBlocks / 4 + 1) + kWaves * 64 - 1) / (kWaves * 64);
}

// LDS: the scales, each wave's 1 KB for its weights' order, each wave's two
// halves of a step of x; afterwards the partial sums [waves][16 or 32][kPitch].
template <int kM>
constexpr int x_half_bytes() { return 16 * kM * 128; }
template <int kM, int kN>
size_t project_lds() {
  const size_t loop = scale_batch<kN>() * kWaves * 64 * sizeof(uint32_t) + kWaves * (1024 + 2 * x_half_bytes<kM>());
  return std::max(loop, sizeof(float) * std::min(kM, 2) * kWaves * 16 * (16 * kN + 4));
}

// Columns 16 * kN and tokens 16 * kM of a workgroup; its waves take the steps
// of 4 blocks in turn.
template <int kM, int kN>
__global__ __launch_bounds__(kWaves * 64, 1) void project_fp4_kernel(
    const uint16_t *__restrict__ x, const uint8_t *__restrict__ codes,
    const uint8_t *__restrict__ scales, uint16_t *__restrict__ out, int T, int K, int N,
    int tiles_m) {
  constexpr int kTm = 16 * kM, kTn = 16 * kN, kPitch = kTn + 4;
  constexpr int kHalf = x_half_bytes<kM>();
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];

  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Token tiles of one column tile are 8 workgroups apart: on one XCD, at one time.
  const int tm = int(blockIdx.x / 8) % tiles_m, tn = int(blockIdx.x / 8) / tiles_m * 8 + int(blockIdx.x % 8);
  const int64_t n0 = int64_t(tn) * kTn;
  if (n0 >= N) return;                           // the whole workgroup
  const int64_t m0 = int64_t(tm) * kTm;
  const int blocks = K / 32, steps = (blocks + 3) / 4;
  const __amdgpu_buffer_rsrc_t rx = gemm::make_rsrc(x + m0 * K, (T - m0) * K * 2);
  const __amdgpu_buffer_rsrc_t rc = gemm::make_rsrc(codes + n0 * (K / 2), (N - n0) * (K / 2));
  const __amdgpu_buffer_rsrc_t rs = gemm::make_rsrc(scales + n0 * blocks, (N - n0) * blocks);

  // The scales of a segment to LDS: the first one's requested in one batch ahead
  // of all else, later ones' (K above 8192) in a loop.
  const int pitch = scale_pitch(blocks), words = pitch / 4;
  const bool by_word = blocks % 4 == 0 && reinterpret_cast<uintptr_t>(scales) % 4 == 0;
  uint32_t *const sc_lds = reinterpret_cast<uint32_t *>(smem);
  auto scale_offset = [&](int i, int b0) {
    const int row = i / words, at = b0 + 4 * (i - row * words);
    return row < kTn && at < blocks ? uint32_t(row) * blocks + at : kOutside;
  };
  auto load_scale = [&](uint32_t off) {
    if (by_word) return uint32_t(__builtin_amdgcn_raw_buffer_load_b32(rs, off, 0, 0));
    uint32_t v = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      v |= uint32_t(__builtin_amdgcn_raw_buffer_load_b8(rs, off + e, 0, 0)) << (8 * e);
    return v;
  };
  constexpr int kBatch = scale_batch<kN>();
  uint32_t sreg[kBatch];
  if (by_word) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      sreg[k] = __builtin_amdgcn_raw_buffer_load_b32(rs, scale_offset(tid + k * kWaves * 64, 0), 0, 0);
  } else {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) sreg[k] = load_scale(scale_offset(tid + k * kWaves * 64, 0));
  }
  __builtin_amdgcn_sched_barrier(0);

  // Weights: 4 neighbouring lanes request a step's 4 blocks of a column, 64 bytes
  // (the vector cache takes a clock per run of addresses in 16 lanes: 16 columns
  // in 16 lanes cost 4 times as many).
  constexpr int kSlots = 2;
  u32x4 fc[kSlots][kN];
  const uint32_t c_row = uint32_t(lane / 4) * (K / 2) + 16 * (lane % 4);
  uint8_t *const ws = smem + kBatch * kWaves * 64 * 4 + wave * 1024;
  uint8_t *const w_put = ws + 64 * (lane / 4) + 16 * ((lane % 4) ^ (lane / 16));
  const uint8_t *const w_get = ws + 64 * r + 4 * g;
  auto load_w = [&](const int slot, int step) {
    const bool in = 4 * step + lane % 4 < blocks;
#pragma unroll
    for (int j = 0; j < kN; ++j)
      fc[slot][j] = __builtin_bit_cast(
          u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                     rc, in ? c_row + uint32_t(16 * j) * (K / 2) + 64 * step : kOutside, 0, 0));
  };

  // x: half a step (64 k, 128 bytes of each token) at a time into the wave's own
  // LDS, 8 tokens an instruction.  16-byte piece p of token t lies at p ^ (t / 2 % 8),
  // so that the 16 tokens of a fragment read different banks.
  uint8_t *const xs = smem + (kBatch * kWaves * 64 * 4 + kWaves * 1024) + wave * 2 * kHalf;
  uint32_t x_off[2];
#pragma unroll
  for (int u = 0; u < 2; ++u)
    x_off[u] = uint32_t(8 * u + lane / 8) * K * 2 + 16 * ((lane % 8) ^ (4 * u + lane / 16));
  auto load_x = [&](const int h, int step) {
    const bool in = step < steps;
#pragma unroll
    for (int u = 0; u < 2 * kM; ++u)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rx, xs + h * kHalf + u * 1024, 16,
          in ? x_off[u % 2] + uint32_t(u / 2 * 16) * K * 2 + 256 * step + 128 * h : kOutside, 0, 0, 0);
  };

  f32x4v acc[kN][kM];
#pragma unroll
  for (int j = 0; j < kN; ++j)
#pragma unroll
    for (int t = 0; t < kM; ++t) acc[j][t] = f32x4v{};
  // (A scale's byte goes to the exponent field, all that the conversion reads: byte 0 is 2^-127.)
  auto convert = [&](uint32_t codes, uint32_t scales4, const int b) {
    const float f = __uint_as_float((scales4 >> (8 * b) & 0xFFu) << 23);
    return u32x4{e2m1_pair<0>(codes, f), e2m1_pair<1>(codes, f), e2m1_pair<2>(codes, f),
                 e2m1_pair<3>(codes, f)};
  };
  auto multiply = [&](const int slot, int step) {
    // From the order of the request to that of the matrix cores: lane group g's
    // dword g of each of the 4 blocks, by way of 1 KB of the wave's own LDS (whose
    // accesses keep their order).
    uint32_t w[kN][4], sc[kN];
    const int at = 4 * (step % (kSegBlocks / 4));
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      *reinterpret_cast<u32x4 *>(w_put) = fc[slot][j];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[j][i] = *reinterpret_cast<const uint32_t *>(w_get + 16 * (i ^ (r / 4)));
      sc[j] = *reinterpret_cast<const uint32_t *>(smem + (16 * j + r) * pitch + at);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // This half landed: what was requested after it is the other half and
      // one step's weights.
      __builtin_amdgcn_s_waitcnt(gemm::waitcnt(2 * kM + kN, 15));
      asm volatile("" ::: "memory");
      u32x4 fx[2][kM];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int t = 0; t < kM; ++t)
          fx[i][t] = *reinterpret_cast<const u32x4 *>(
              xs + h * kHalf + (16 * t + r) * 128 + 16 * ((4 * i + g) ^ (r / 2)));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int b = 2 * h + i;
        if (4 * step + b < blocks) {               // uniform: past K there is no x
#pragma unroll
          for (int j = 0; j < kN; ++j) {
            const u32x4 v = convert(w[j][b], sc[j], b);
#pragma unroll
            for (int t = 0; t < kM; ++t)
              acc[j][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(bf16x8, v), __builtin_bit_cast(bf16x8, fx[i][t]), acc[j][t], 0, 0, 0);
          }
        }
      }
      // The half is in registers: the next step's may overwrite it.
      __builtin_amdgcn_s_waitcnt(gemm::waitcnt(63, 0));
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      load_x(h, step + kWaves);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  load_w(0, wave);
  __builtin_amdgcn_sched_barrier(0);
  load_x(0, wave);
  load_x(1, wave);
  __builtin_amdgcn_sched_barrier(0);
  load_w(1, wave + kWaves);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int k = 0; k < kBatch; ++k) sc_lds[tid + k * kWaves * 64] = sreg[k];
  // A segment's steps are a multiple of kSlots * kWaves (but the last one's).
  for (int seg = 0; seg < steps; seg += kSegBlocks / 4) {
    if (seg > 0) {
      __syncthreads();
      for (int i = tid; i < kTn * words; i += kWaves * 64)
        sc_lds[i] = load_scale(scale_offset(i, 4 * seg));
    }
    __syncthreads();
    const int end = min(steps, seg + kSegBlocks / 4);
    for (int s = seg + wave; s < end; s += kSlots * kWaves) {
#pragma unroll
      for (int p = 0; p < kSlots; ++p) {
        if (p > 0 && s + kWaves * p >= end) break;
        multiply(p, s + kWaves * p);
        load_w(p, s + kWaves * (p + kSlots));
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }

  // The waves' sums added in wave order, up to 32 tokens at a time.  D of a 16 x
  // 16 block: lane l holds token l % 16, columns 4 (l / 16) .. + 3.
  constexpr int kTiles = kM < 2 ? 1 : 2;
  using Part = float[kTiles * 16][kPitch];
  Part *red = reinterpret_cast<Part *>(smem);
  __builtin_amdgcn_s_waitcnt(gemm::waitcnt(0, 0));       // the last, unread x
  const bool whole = N % 4 == 0;                         // 4 columns a store
#pragma unroll
  for (int t0 = 0; t0 < kM; t0 += kTiles) {
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int j = 0; j < kN; ++j)
        *reinterpret_cast<f32x4v *>(&red[wave][16 * t + r][16 * j + 4 * g]) = acc[j][t0 + t];
    __syncthreads();
    for (int i = tid; i < kTiles * 16 * (kTn / 4); i += kWaves * 64) {
      const int m = i / (kTn / 4), n = 4 * (i % (kTn / 4));
      f32x4v sum = *reinterpret_cast<const f32x4v *>(&red[0][m][n]);
#pragma unroll
      for (int w = 1; w < kWaves; ++w) sum += *reinterpret_cast<const f32x4v *>(&red[w][m][n]);
      const int64_t row = m0 + 16 * t0 + m;
      if (row >= T) continue;
      uint16_t *dst = out + row * N + n0 + n;
      if (whole) {
        if (n0 + n < N)
          *reinterpret_cast<u32x2 *>(dst) = u32x2{pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3])};
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n0 + n + e < N) dst[e] = f32_to_bf16(sum[e]);
      }
    }
  }
}

template <int kM, int kN>
hipError_t launch_tile(const uint16_t *x, const uint8_t *codes, const uint8_t *scales,
                       uint16_t *out, int32_t T, int32_t K, int32_t N, hipStream_t stream) {
  const int64_t tiles_m = (T + 16 * kM - 1) / (16 * kM);
  const int64_t tiles_n = (int64_t(N) + 16 * kN - 1) / (16 * kN);
  const size_t lds = project_lds<kM, kN>();
  if (lds > 65536) {                             // what a launch may have without asking
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(&project_fp4_kernel<kM, kN>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, int(lds));
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((project_fp4_kernel<kM, kN>), dim3(unsigned((tiles_n + 7) / 8 * 8 * tiles_m)),
                     dim3(kWaves * 64), lds, stream, x, codes, scales, out, T, K, N, int(tiles_m));
  return hipGetLastError();
}

template <int kM>
hipError_t by_columns(int n, const uint16_t *x, const uint8_t *codes, const uint8_t *scales,
                      uint16_t *out, int32_t T, int32_t K, int32_t N, hipStream_t stream) {
  switch (n) {
    case 1: return launch_tile<kM, 1>(x, codes, scales, out, T, K, N, stream);
    case 2: return launch_tile<kM, 2>(x, codes, scales, out, T, K, N, stream);
    case 3: return launch_tile<kM, 3>(x, codes, scales, out, T, K, N, stream);
    case 4: return launch_tile<kM, 4>(x, codes, scales, out, T, K, N, stream);
    default: return launch_tile<kM, 5>(x, codes, scales, out, T, K, N, stream);
  }
}

}  // namespace

hipError_t launch_quantize_fp4(const uint16_t *w, int32_t N, int32_t K, uint8_t *codes,
                               uint8_t *scales, hipStream_t stream) {
  const int64_t blocks = int64_t(N) * (K / 32);
  hipLaunchKernelGGL(quantize_fp4_kernel, dim3(unsigned((blocks + kThreads - 1) / kThreads)),
                     dim3(kThreads), 0, stream, w, blocks, codes, scales);
  return hipGetLastError();
}

namespace {

struct Tile {
  int m, n;
};

// The tile with the least to pull through a CU's vector cache: per 32 k a tile
// takes 64 bytes a token and 17 a column, and the CUs take ceil(tiles / 256)
// tiles each.  (64 tokens of 6144 x 20480 in tiles of 32 tokens: 36.6 us instead
// of 28.9.)  At most 5 x 16 columns, as LDS is full with 64 tokens then: past 256
// tiles of them some CUs take a second (64 tokens, K 6144: 20480 columns 28.9 us,
// 20496 41.3, 40960 55.9; 32 tokens: 22.3, 27.8, 40.9).
Tile pick_tile(int32_t T, int32_t N) {
  Tile best{1, 1};
  int64_t least = INT64_MAX;
  for (const int m : {1, 2, 4})
    for (int n = 1; n <= 5; ++n) {
      const int64_t tiles = ((int64_t(T) + 16 * m - 1) / (16 * m)) * ((int64_t(N) + 16 * n - 1) / (16 * n));
      const int64_t cost = (tiles + kCus - 1) / kCus * (64 * 16 * std::min<int64_t>(m, (T + 15) / 16) + 17 * 16 * n);
      if (cost < least) least = cost, best = {m, n};
    }
  return best;
}

}  // namespace

int64_t project_fp4_blocks(int32_t T, int32_t N) {
  const Tile t = pick_tile(T, N);
  const int64_t tiles_m = (int64_t(T) + 16 * t.m - 1) / (16 * t.m);
  return ((int64_t(N) + 16 * t.n - 1) / (16 * t.n) + 7) / 8 * 8 * tiles_m;
}

hipError_t launch_project_fp4(const uint16_t *x, const uint8_t *codes, const uint8_t *scales,
                              uint16_t *out, int32_t T, int32_t K, int32_t N,
                              hipStream_t stream) {
  const Tile t = pick_tile(T, N);
  switch (t.m) {
    case 1: return by_columns<1>(t.n, x, codes, scales, out, T, K, N, stream);
    case 2: return by_columns<2>(t.n, x, codes, scales, out, T, K, N, stream);
    default: return by_columns<4>(t.n, x, codes, scales, out, T, K, N, stream);
  }
}

}  // namespace engram
