// Linear layer of a few 16-bit activation rows with 4-bit weights and group
// scales, and the offline quantiser of its weights.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "half16.cuh"
#include "ptx.cuh"
#include "w4a4.h"
#include "w4a4_internal.h"

namespace w4a4 {
namespace {

constexpr int kW16Threads = 256;
constexpr int kW16MaxM = 64;

// ------------------------------------------------------------ quantiser
// One thread per group: two passes over its `group` fp32 weights (the second
// from L1).  Runs once, offline.
template <class T, bool OFFSET>
__global__ void __launch_bounds__(256)
    quantize_w4a16_kernel(const float* __restrict__ W, int64_t N, int64_t K, int64_t ldw, int group,
                          int8_t* __restrict__ Wq, uint16_t* __restrict__ scale, uint16_t* __restrict__ offset) {
  const int64_t groups = K / group;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= N * groups) return;
  const int64_t n = i / groups, g = i - n * groups;
  const float* w = W + n * ldw + g * group;
  float lo = w[0], hi = w[0];
  for (int j = 1; j < group; ++j) {
    lo = fminf(lo, w[j]);
    hi = fmaxf(hi, w[j]);
  }
  uint16_t sb, ob = 0;
  float o = 0.f;
  if (OFFSET) {
    sb = T::from_f32((hi - lo) / 15.f);
    ob = T::from_f32(fmaf(8.f, T::to_f32(sb), lo));
    o = T::to_f32(ob);
  } else {
    sb = T::from_f32(fmaxf(fabsf(lo), fabsf(hi)) / 7.f);
  }
  const float s = T::to_f32(sb);
  int8_t* dst = Wq + n * (K / 2) + g * (group / 2);
  for (int j = 0; j < group; j += 2) {
    int q[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float v = s != 0.f ? rintf((w[j + e] - o) / s) : 0.f;
      q[e] = static_cast<int>(fminf(fmaxf(v, OFFSET ? -8.f : -7.f), 7.f));
    }
    dst[j / 2] = static_cast<int8_t>((q[0] & 15) | ((q[1] & 15) << 4));
  }
  scale[i] = sb;
  if (OFFSET) offset[i] = ob;
}

// ------------------------------------------------------------ product
// One warp per weight row and chunk of eight activation rows; a lane takes
// eight columns (one packed word) at a time and sums in fp32.
template <class T>
__global__ void __launch_bounds__(kW16Threads)
    linear_w4a16_kernel(const uint16_t* __restrict__ x, int64_t ldx, const int8_t* __restrict__ Wq,
                        const uint16_t* __restrict__ scale, const uint16_t* __restrict__ offset, int group,
                        const uint16_t* __restrict__ bias, uint16_t* __restrict__ y, int64_t ldy, int64_t M,
                        int64_t N, int64_t K) {
  const int lane = threadIdx.x & 31;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * (kW16Threads / 32) + (threadIdx.x >> 5);
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * 8;
  if (n >= N) return;
  const int64_t groups = K / group;
  float acc[8] = {};
  for (int64_t k = lane * 8; k < K; k += 256) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(Wq + n * (K / 2) + k / 2);
    const float s = T::to_f32(scale[n * groups + k / group]);
    const float o = offset != nullptr ? T::to_f32(offset[n * groups + k / group]) : 0.f;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = fmaf(s, static_cast<float>(static_cast<int>(w << (28 - 4 * j)) >> 28), o);
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      if (m0 + m >= M) break;
      const uint4 xv = *reinterpret_cast<const uint4*>(x + (m0 + m) * ldx + k);
      const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = T::to_f32x2(xw[j]);
        acc[m] = fmaf(f.x, v[2 * j], acc[m]);
        acc[m] = fmaf(f.y, v[2 * j + 1], acc[m]);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < 8; ++m) {
    for (int d = 16; d > 0; d >>= 1) acc[m] += __shfl_xor_sync(0xFFFFFFFFu, acc[m], d);
    if (lane == 0 && m0 + m < M) {
      const float b = bias != nullptr ? T::to_f32(bias[n]) : 0.f;
      y[(m0 + m) * ldy + n] = T::from_f32(acc[m] + b);
    }
  }
}

int check_w4a16(int64_t N, int64_t K, int group, int dtype) {
  if (group != 32 && group != 64 && group != 128) return W4A4_ERR_GROUP;
  if (dtype != W4A4_BF16 && dtype != W4A4_FP16) return W4A4_ERR_ARG;
  if (N < 1 || N > (int64_t(1) << 24)) return W4A4_ERR_SHAPE;
  if (K < 32 || K % 32 != 0 || K > (int64_t(1) << 17)) return W4A4_ERR_SHAPE;
  if (K % group != 0) return W4A4_ERR_GROUP;
  return W4A4_OK;
}

}  // namespace
}  // namespace w4a4

using namespace w4a4;

extern "C" {

int w4a4_quantize_weight_w4a16(const float* W, int64_t N, int64_t K, int64_t ldw, int group, int dtype, int8_t* Wq,
                               void* scale, void* offset, void* stream) {
  if (W == nullptr || Wq == nullptr || scale == nullptr) return W4A4_ERR_NULL;
  int st = check_w4a16(N, K, group, dtype);
  if (st != W4A4_OK) return st;
  if (ldw < K) return W4A4_ERR_SHAPE;
  if (ldw % 4 != 0 || !aligned_to(W, 16) || !aligned_to(Wq, 16) || !aligned_to(scale, 2) || !aligned_to(offset, 2))
    return W4A4_ERR_ALIGN;
  DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != W4A4_OK) return st;
  const int64_t blocks = (N * (K / group) + 255) / 256;
  auto kernel = dtype == W4A4_BF16 ? (offset ? quantize_w4a16_kernel<Bf16, true> : quantize_w4a16_kernel<Bf16, false>)
                                   : (offset ? quantize_w4a16_kernel<Fp16, true> : quantize_w4a16_kernel<Fp16, false>);
  kernel<<<static_cast<unsigned>(blocks), 256, 0, static_cast<cudaStream_t>(stream)>>>(
      W, N, K, ldw, group, Wq, static_cast<uint16_t*>(scale), static_cast<uint16_t*>(offset));
  return cudaGetLastError() == cudaSuccess ? W4A4_OK : W4A4_ERR_CUDA;
}

int w4a4_linear_w4a16(const void* x, int64_t ldx, const int8_t* Wq, const void* scale, const void* offset, int group,
                      const void* bias, void* y, int64_t ldy, int64_t M, int64_t N, int64_t K, int dtype,
                      void* stream) {
  if (Wq == nullptr || scale == nullptr) return W4A4_ERR_NULL;
  // an empty batch (M == 0) may pass NULL for its zero-size tensors
  if (M != 0 && (x == nullptr || y == nullptr)) return W4A4_ERR_NULL;
  int st = check_w4a16(N, K, group, dtype);
  if (st != W4A4_OK) return st;
  if (M < 0 || M > kW16MaxM || ldx < K || ldy < N) return W4A4_ERR_SHAPE;
  if (ldx % 8 != 0 || !aligned_to(x, 16) || !aligned_to(Wq, 16)) return W4A4_ERR_ALIGN;
  if (!aligned_to(scale, 2) || !aligned_to(offset, 2) || !aligned_to(bias, 2) || !aligned_to(y, 2))
    return W4A4_ERR_ALIGN;
  DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != W4A4_OK) return st;
  if (M == 0) return W4A4_OK;
  const dim3 grid(static_cast<unsigned>((N + kW16Threads / 32 - 1) / (kW16Threads / 32)),
                  static_cast<unsigned>((M + 7) / 8), 1);
  auto kernel = dtype == W4A4_BF16 ? linear_w4a16_kernel<Bf16> : linear_w4a16_kernel<Fp16>;
  kernel<<<grid, kW16Threads, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint16_t*>(x), ldx, Wq, static_cast<const uint16_t*>(scale),
      static_cast<const uint16_t*>(offset), group, static_cast<const uint16_t*>(bias), static_cast<uint16_t*>(y), ldy,
      M, N, K);
  return cudaGetLastError() == cudaSuccess ? W4A4_OK : W4A4_ERR_CUDA;
}

}  // extern "C"
