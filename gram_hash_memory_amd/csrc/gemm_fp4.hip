// The MXFP4 copy of a bf16 weight, and the product of few tokens with it.
//
//   out[t][n] = bf16(sum_k x[t][k] * e2m1(code[n][k]) * 2^(scale[n][k/32] - 127))
//
// The plain kernel: one wave per output column, a lane a block of 32 k at a
// time, the lanes' sums added at the end.
#include "common.hpp"

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

// One thread per block of 32 k: 64 bytes of bf16 in, 16 bytes of codes out.
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

__device__ __forceinline__ float e2m1_to_float(uint32_t c) {
  const uint32_t e = (c >> 1) & 3u, m = c & 1u;
  const float a = e ? __uint_as_float((e + 126u) << 23 | m << 22) : 0.5f * float(m);
  return c & 8u ? -a : a;
}

__global__ __launch_bounds__(kThreads) void project_fp4_kernel(
    const uint16_t *__restrict__ x, const uint8_t *__restrict__ codes,
    const uint8_t *__restrict__ scales, uint16_t *__restrict__ out, int T, int K, int N) {
  const int lane = threadIdx.x & 63;
  const int64_t n = int64_t(blockIdx.x) * (kThreads / 64) + (threadIdx.x >> 6);
  if (n >= N) return;
  const int blocks = K / 32;
  for (int t = 0; t < T; ++t) {
    float sum = 0.0f;
    for (int b = lane; b < blocks; b += 64) {
      const u32x4 q = *reinterpret_cast<const u32x4 *>(codes + (n * blocks + b) * 16);
      const uint16_t *xt = x + int64_t(t) * K + 32 * b;
      float part = 0.0f;
      for (int i = 0; i < 32; ++i) {
        const uint32_t c = (q[i / 8] >> (4 * (i % 8))) & 15u;
        part = fmaf(__uint_as_float(uint32_t(xt[i]) << 16), e2m1_to_float(c), part);
      }
      sum += ldexpf(part, int(scales[n * blocks + b]) - 127);
    }
    for (int m = 1; m < 64; m *= 2) sum += __shfl_xor(sum, m);
    if (lane == 0) out[int64_t(t) * N + n] = f32_to_bf16(sum);
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

hipError_t launch_project_fp4(const uint16_t *x, const uint8_t *codes, const uint8_t *scales,
                              uint16_t *out, int32_t T, int32_t K, int32_t N,
                              hipStream_t stream) {
  const int per = kThreads / 64;
  hipLaunchKernelGGL(project_fp4_kernel, dim3(unsigned((int64_t(N) + per - 1) / per)),
                     dim3(kThreads), 0, stream, x, codes, scales, out, T, K, N);
  return hipGetLastError();
}

}  // namespace engram
