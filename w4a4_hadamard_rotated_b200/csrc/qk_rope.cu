// RMS norm of every query and key head with the rotary rotation of both over
// several position axes, in one pass.
//
//   u = h / sqrt(mean(h^2) + eps) * weight,  angle_i = position[axis_i] freq_i,
//   (a, b) -> (a cos - b sin, a sin + b cos) over the pairs (2i, 2i + 1) or (i, i + R/2)
// Every element is read once and written once (4 T (Hq + Hk) D bytes) for
// about ten operations: bound by HBM on many tokens, by latency on few.
//
// Design
//   * LPH lanes share a head, eight elements (16 bytes) each, so a warp moves
//     32 / LPH heads at a time and the norm's sum is log2(LPH) shuffles.  In
//     halves order the partner of element i is R/16 lanes away (R % 16 == 0),
//     eight shuffles; interleaved pairs lie inside a lane.
//   * The angles depend on the token only.  A block takes a few whole tokens:
//     its threads form each token's R/2 sines and cosines once into shared
//     memory, every warp then keeps those of its elements in registers for
//     all heads of its token, the norm's weights too.
//   * The angle is reduced in turns: position * freq / 2 pi in fp64, less its
//     nearest whole number, then sincospi in fp32.  In fp32 a position of
//     2^17 would leave 7 bits of the fraction of a turn.
//   * Four loads of a warp are in flight before the first is used, the first
//     four while the angles are formed.
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

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kRopeBatch = 4;          // heads (times 32 / LPH) a warp has in flight

__device__ __forceinline__ uint4 ldg128(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// warps_per_token: 1, 2, 4 or 8; a block takes 8 / warps_per_token tokens.
template <class T, int LPH, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 3) qk_norm_rope_kernel(const RopeArgs a, const int warps_per_token) {
  constexpr int kHeads = 32 / LPH;     // heads per warp and step
  constexpr int kAngles = INTER ? 4 : 8;
  __shared__ __align__(16) float cs[kRopeWarps][kRopeMaxD / 2], sn[kRopeWarps][kRopeMaxD / 2];
  // q, k, the weights and the positions may be the previous kernel's output
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tokens = kRopeWarps / warps_per_token;
  const int slot = warp / warps_per_token;           // which token of the block
  const int part = warp - slot * warps_per_token;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens;
  const int64_t t = t0 + slot;
  const int e = lane & (LPH - 1);                    // elements 8 e .. 8 e + 7 of the head
  const bool active = t < a.T && 8 * e < a.D;
  const int step = warps_per_token * kHeads;
  const int first = part * kHeads + lane / LPH;

  const uint16_t* qi = a.q.in + t * a.q.in_t + 8 * e;
  const uint16_t* ki = a.k.in + t * a.k.in_t + 8 * e;
  uint16_t* qo = a.q.out + t * a.q.out_t + 8 * e;
  uint16_t* ko = a.k.out + t * a.k.out_t + 8 * e;
  uint4 next[kRopeBatch];
  auto load = [&](int h0) {
#pragma unroll
    for (int b = 0; b < kRopeBatch; ++b) {
      const int h = h0 + b * step;
      if (active && h < a.H)
        next[b] = ldg128(h < a.Hq ? qi + h * a.q.in_h : ki + (h - a.Hq) * a.k.in_h);
      else
        next[b] = make_uint4(0u, 0u, 0u, 0u);
    }
  };
  load(first);

  const int half = a.R >> 1;
  for (int i = threadIdx.x; i < tokens * half; i += kRopeThreads) {
    const int s = i / half, j = i - s * half;
    if (t0 + s >= a.T) break;
    const int ax = min(max(a.axis[j], 0), a.axes - 1);
    const int64_t at = (t0 + s) * a.pos_stride + ax;
    const double pos = a.pos64 ? static_cast<double>(static_cast<const int64_t*>(a.positions)[at])
                               : static_cast<double>(static_cast<const int32_t*>(a.positions)[at]);
    double turns = pos * (a.freq[j] * 0.15915494309189533577);   // 1 / (2 pi)
    turns -= rint(turns);
    float sv, cv;
    sincospif(2.f * static_cast<float>(turns), &sv, &cv);
    cs[s][j] = cv;
    sn[s][j] = sv;
  }
  __syncthreads();

  // this lane's angles (0 turns where nothing rotates) and weights
  float c[kAngles], s[kAngles];
  int from = lane;                                   // halves: the partner's lane
  {
    int at = -1;
    float sign = 1.f;
    if (INTER) {
      if (8 * e < a.R) at = 4 * e;
    } else if (8 * e < a.R) {
      const bool low = 8 * e < half;
      at = low ? 8 * e : 8 * e - half;
      from = low ? lane + half / 8 : lane - half / 8;
      sign = low ? -1.f : 1.f;                       // a cos - b sin, b cos + a sin
    }
#pragma unroll
    for (int i = 0; i < kAngles; ++i) {
      const bool turned = at >= 0 && at + i < half;
      c[i] = turned ? cs[slot][at + i] : 1.f;
      s[i] = turned ? (INTER ? sn[slot][at + i] : sign * sn[slot][at + i]) : 0.f;
    }
  }
  const uint32_t one = T::from_f32x2(1.f, 1.f);
  uint4 wq = make_uint4(one, one, one, one), wk = wq;
  const bool norm_q = a.q.weight != nullptr, norm_k = a.k.weight != nullptr;
  if (norm_q && 8 * e < a.D) wq = *reinterpret_cast<const uint4*>(a.q.weight + 8 * e);
  if (norm_k && 8 * e < a.D) wk = *reinterpret_cast<const uint4*>(a.k.weight + 8 * e);
  const float inv_d = 1.f / static_cast<float>(a.D);

  for (int h0 = part * kHeads; h0 < a.H; h0 += kRopeBatch * step) {   // the same for the warp
    const int mine = h0 + lane / LPH;
#pragma unroll
    for (int b = 0; b < kRopeBatch; ++b) {
      const int h = mine + b * step;
      const bool is_q = h < a.Hq;
      const uint32_t w[4] = {is_q ? wq.x : wk.x, is_q ? wq.y : wk.y, is_q ? wq.z : wk.z, is_q ? wq.w : wk.w};
      const uint32_t in[4] = {next[b].x, next[b].y, next[b].z, next[b].w};
      float u[8];
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = T::to_f32x2(in[i]);
        u[2 * i] = f.x;
        u[2 * i + 1] = f.y;
        sum = fmaf(f.x, f.x, fmaf(f.y, f.y, sum));
      }
#pragma unroll
      for (int d = LPH / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
      const bool norm = is_q ? norm_q : norm_k;
      const float r = norm ? rsqrtf(fmaf(sum, inv_d, a.eps)) : 1.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 g = T::to_f32x2(w[i]);
        u[2 * i] *= r * g.x;
        u[2 * i + 1] *= r * g.y;
      }
      uint32_t out[4];
      if (INTER) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool turned = 8 * e + 2 * i < a.R;
          const float x = u[2 * i] * c[i % kAngles] - u[2 * i + 1] * s[i % kAngles];
          const float y = u[2 * i] * s[i % kAngles] + u[2 * i + 1] * c[i % kAngles];
          out[i] = T::from_f32x2(turned ? x : u[2 * i], turned ? y : u[2 * i + 1]);
          if (!turned && !norm) out[i] = in[i];       // copied bit for bit, NaN included
        }
      } else {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float other = __shfl_sync(0xFFFFFFFFu, u[i], from);
          v[i] = from == lane ? u[i] : fmaf(u[i], c[i % kAngles], other * s[i % kAngles]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          out[i] = T::from_f32x2(v[2 * i], v[2 * i + 1]);
          if (from == lane && !norm) out[i] = in[i];  // copied bit for bit, NaN included
        }
      }
      if (active && h < a.H)
        *reinterpret_cast<uint4*>(is_q ? qo + h * a.q.out_h : ko + (h - a.Hq) * a.k.out_h) =
            make_uint4(out[0], out[1], out[2], out[3]);
    }
    if (h0 + kRopeBatch * step < a.H) load(mine + kRopeBatch * step);
  }
}

template <class T>
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream) {
  const int lph = a.D <= 64 ? 8 : (a.D <= 128 ? 16 : 32);
  // warps per token: all eight for few tokens (latency), else as many as leave
  // each warp a batch of loads
  int wpt = 8;
  if (a.T > 1184)
    while (wpt > 1 && a.H * lph < wpt * 32 * kRopeBatch) wpt /= 2;
  const int tokens = kRopeWarps / wpt;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.T + tokens - 1) / tokens), 1, 1);
  cfg.blockDim = dim3(kRopeThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.interleaved) {
    if (lph == 8) return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<T, 8, true>, a, wpt);
    if (lph == 16) return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<T, 16, true>, a, wpt);
    return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<T, 32, true>, a, wpt);
  }
  if (lph == 8) return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<T, 8, false>, a, wpt);
  if (lph == 16) return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<T, 16, false>, a, wpt);
  return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<T, 32, false>, a, wpt);
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
  const cudaError_t e = dtype == W4A4_BF16 ? launch_rope<Bf16>(a, s) : launch_rope<Fp16>(a, s);
  return e == cudaSuccess ? W4A4_OK : W4A4_ERR_CUDA;
}
