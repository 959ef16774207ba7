// RMS norm of every query and key head with the rotary rotation of both over
// several position axes, in one pass.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "half16.cuh"
#include "ptx.cuh"
#include "w4a4.h"
#include "w4a4_internal.h"

namespace w4a4 {
namespace {

constexpr int kRopeMaxD = 256;
constexpr int kRopeMaxAxes = 8;

struct RopeSide {
  const uint16_t* in;
  uint16_t* out;
  int64_t in_t, in_h, out_t, out_h;   // token and head strides in elements
  const uint16_t* weight;             // [D] or nullptr: no norm
};

struct RopeArgs {
  RopeSide q, k;
  int Hq, H;                 // query heads, all heads
  int64_t T;
  int D, R;                  // R == 0: no rotation
  float eps;
  const void* positions;
  int pos64;
  int64_t pos_stride;
  int axes;
  const double* freq;
  const int32_t* axis;
  int interleaved;
};

// One block per token, one thread per element of a head; the angles are
// formed once per token.
template <class T>
__global__ void __launch_bounds__(kRopeMaxD) qk_norm_rope_kernel(const RopeArgs a) {
  __shared__ float cs[kRopeMaxD / 2], sn[kRopeMaxD / 2];
  __shared__ float u[kRopeMaxD];
  __shared__ float sums[kRopeMaxD / 32];
  const int64_t t = blockIdx.x;
  const int d = threadIdx.x;
  if (2 * d < a.R) {
    const int ax = min(max(a.axis[d], 0), a.axes - 1);
    const int64_t at = t * a.pos_stride + ax;
    const double pos = a.pos64 ? static_cast<double>(static_cast<const int64_t*>(a.positions)[at])
                               : static_cast<double>(static_cast<const int32_t*>(a.positions)[at]);
    double turns = pos * (a.freq[d] * 0.15915494309189533577);   // 1 / (2 pi)
    turns -= rint(turns);
    float s, c;
    sincospif(2.f * static_cast<float>(turns), &s, &c);
    cs[d] = c;
    sn[d] = s;
  }
  for (int h = 0; h < a.H; ++h) {
    const RopeSide& side = h < a.Hq ? a.q : a.k;
    const int hh = h < a.Hq ? h : h - a.Hq;
    float v = d < a.D ? T::to_f32(side.in[t * side.in_t + hh * side.in_h + d]) : 0.f;
    if (side.weight != nullptr) {
      float ss = v * v;
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
      if ((d & 31) == 0) sums[d >> 5] = ss;
      __syncthreads();
      float total = 0.f;
      for (int w = 0; w < kRopeMaxD / 32; ++w) total += sums[w];
      const float r = rsqrtf(total / static_cast<float>(a.D) + a.eps);
      if (d < a.D) v = v * r * T::to_f32(side.weight[d]);
    }
    u[d] = v;
    __syncthreads();
    if (d < a.D) {
      if (d < a.R) {
        const int half = a.R / 2;
        const int i = a.interleaved ? d >> 1 : (d < half ? d : d - half);
        const bool first = a.interleaved ? (d & 1) == 0 : d < half;
        const float p = u[a.interleaved ? d ^ 1 : (first ? d + half : d - half)];
        v = first ? v * cs[i] - p * sn[i] : v * cs[i] + p * sn[i];
      }
      side.out[t * side.out_t + hh * side.out_h + d] = T::from_f32(v);
    }
    __syncthreads();
  }
}

int check_side(const void* in, int64_t in_t, int64_t in_h, const void* out, int64_t out_t, int64_t out_h,
               const void* weight, int64_t T, int64_t H, int64_t D) {
  const int64_t lim = int64_t(1) << 40;
  if (in_t > lim || in_h > lim || out_t > lim || out_h > lim) return W4A4_ERR_SHAPE;
  if (T > 1 && (in_t < D || out_t < D)) return W4A4_ERR_SHAPE;
  if (H > 1 && (in_h < D || out_h < D)) return W4A4_ERR_SHAPE;
  if (in_t % 8 != 0 || in_h % 8 != 0 || out_t % 8 != 0 || out_h % 8 != 0) return W4A4_ERR_ALIGN;
  if (!aligned_to(in, 16) || !aligned_to(out, 16) || !aligned_to(weight, 16)) return W4A4_ERR_ALIGN;
  return W4A4_OK;
}

}  // namespace
}  // namespace w4a4

using namespace w4a4;

extern "C" int w4a4_qk_norm_rope(const void* q, int64_t q_token_stride, int64_t q_head_stride, int64_t Hq,
                                 const void* k, int64_t k_token_stride, int64_t k_head_stride, int64_t Hk,
                                 const void* q_weight, const void* k_weight, float eps, const void* positions,
                                 int position_bits, int64_t pos_stride, int axes, const double* freq,
                                 const int32_t* axis, int64_t R, int interleaved, void* q_out,
                                 int64_t q_out_token_stride, int64_t q_out_head_stride, void* k_out,
                                 int64_t k_out_token_stride, int64_t k_out_head_stride, int64_t T, int64_t D,
                                 int dtype, void* stream) {
  if (T < 0 || T > (int64_t(1) << 30)) return W4A4_ERR_SHAPE;
  if (T != 0 && (q == nullptr || q_out == nullptr || (Hk != 0 && (k == nullptr || k_out == nullptr))))
    return W4A4_ERR_NULL;
  if (T != 0 && positions != nullptr && (freq == nullptr || axis == nullptr)) return W4A4_ERR_NULL;
  if (dtype != W4A4_BF16 && dtype != W4A4_FP16) return W4A4_ERR_ARG;
  if (D < 8 || D > kRopeMaxD || D % 8 != 0) return W4A4_ERR_SHAPE;
  if (Hq < 1 || Hk < 0 || Hq > 4096 || Hk > 4096 || Hq + Hk > 4096) return W4A4_ERR_SHAPE;
  if (!(eps >= 0.f) || eps > 3.0e38f) return W4A4_ERR_ARG;
  if (positions != nullptr) {
    if (R < 2 || R > D || R % 2 != 0 || (!interleaved && R % 16 != 0)) return W4A4_ERR_SHAPE;
    if (axes < 1 || axes > kRopeMaxAxes || (T > 1 && pos_stride < axes)) return W4A4_ERR_SHAPE;
    if (position_bits != 32 && position_bits != 64) return W4A4_ERR_ARG;
    if (!aligned_to(positions, position_bits / 8) || !aligned_to(freq, 8) || !aligned_to(axis, 4))
      return W4A4_ERR_ALIGN;
  }
  int st = check_side(q, q_token_stride, q_head_stride, q_out, q_out_token_stride, q_out_head_stride, q_weight, T, Hq, D);
  if (st != W4A4_OK) return st;
  if (Hk != 0) {
    st = check_side(k, k_token_stride, k_head_stride, k_out, k_out_token_stride, k_out_head_stride, k_weight, T, Hk, D);
    if (st != W4A4_OK) return st;
  }
  DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != W4A4_OK) return st;
  if (T == 0) return W4A4_OK;
  RopeArgs a{};
  a.q = RopeSide{static_cast<const uint16_t*>(q), static_cast<uint16_t*>(q_out), q_token_stride, q_head_stride,
                 q_out_token_stride, q_out_head_stride, static_cast<const uint16_t*>(q_weight)};
  a.k = RopeSide{static_cast<const uint16_t*>(k), static_cast<uint16_t*>(k_out), k_token_stride, k_head_stride,
                 k_out_token_stride, k_out_head_stride, static_cast<const uint16_t*>(k_weight)};
  a.Hq = static_cast<int>(Hq);
  a.H = static_cast<int>(Hq + Hk);
  a.T = T;
  a.D = static_cast<int>(D);
  a.R = positions != nullptr ? static_cast<int>(R) : 0;
  a.eps = eps;
  a.positions = positions;
  a.pos64 = position_bits == 64;
  a.pos_stride = pos_stride;
  a.axes = axes;
  a.freq = freq;
  a.axis = axis;
  a.interleaved = interleaved != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto kernel = dtype == W4A4_BF16 ? qk_norm_rope_kernel<Bf16> : qk_norm_rope_kernel<Fp16>;
  kernel<<<static_cast<unsigned>(T), kRopeMaxD, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? W4A4_OK : W4A4_ERR_CUDA;
}
