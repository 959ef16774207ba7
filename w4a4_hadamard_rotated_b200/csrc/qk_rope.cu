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
//     all heads of its token, multiplied with the norm's weights: an element
//     is r (own u_i + other u_pair), r the reciprocal root of its head.
//   * The angle is reduced in turns: position * freq / 2 pi in fp64, less its
//     nearest whole number, then sincospi in fp32.  In fp32 a position of
//     2^17 leaves 10 bits of the fraction of a turn.
//   * Four to eight loads of a lane are in flight before the first is used, the
//     first of a token while its angles are formed.  The blocks stay: each walks
//     over tokens, so a token's latency hides behind the other warps' streams
//     (blocks of one token each took 427 us where these take 219).
// Measured: 32760 tokens, 40 + 40 heads of 128: 219 us, 6.1 TB/s; 4608 tokens,
// 24 + 24 heads: 25 us; one token of 32 + 8 heads 4.4 us, all of it latency.
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
// Blocks per SM and 16-byte loads a lane has in flight: three of 80 registers
// and four loads where that fits without spilling, else two and eight.
// Measured at 32760 tokens of 40 + 40 heads of 128 (1.34 GB): interleaved 219 us
// against 223, halves (which need the pair's angles and weights too) 247 against
// 246 with spills; at 1001 tokens of 32 + 8 heads of 64, halves 6.2 against 7.8 us.
constexpr int rope_blocks(bool inter, bool copy) { return inter && !copy ? 3 : 2; }
constexpr int rope_batch(bool inter, bool copy) { return inter && !copy ? 4 : 8; }

__device__ __forceinline__ uint4 ldg128(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// One side (queries or keys) of one token: this lane's elements of the heads
// first, first + step, ...
// COPY: some elements do not turn (R < D).
template <class T, int LPH, bool INTER, bool COPY>
struct RopeWalk {
  static constexpr int kBatch = rope_batch(INTER, COPY);
  const uint16_t* in;
  uint16_t* out;
  int64_t in_step, out_step;
  int left;                                          // heads from this lane's first one on
  int step;
  bool active;                                       // the lane holds elements of its token's heads
  uint4 x[kBatch];

  __device__ __forceinline__ void init(const RopeSide& side, int H, int64_t t, int e, int head, int step_, bool active_) {
    in = side.in + t * side.in_t + head * side.in_h + 8 * e;
    out = side.out + t * side.out_t + head * side.out_h + 8 * e;
    in_step = step_ * side.in_h;
    out_step = step_ * side.out_h;
    left = H - head;
    step = step_;
    active = active_;
  }
  __device__ __forceinline__ void load() {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      x[b] = make_uint4(0u, 0u, 0u, 0u);
      if (active && b * step < left) x[b] = ldg128(in + b * in_step);
    }
    in += kBatch * in_step;
  }
  // own[i], other[i]: what this element and its pair's other one contribute
  // to element i, the weights of the norm included.  `from`: halves: the lane
  // of the pair's other element.  `copy`: bit i: word i is copied.
  __device__ __forceinline__ void run(bool norm, float inv_d, float eps, const float (&own)[8], const float (&other)[8],
                                      int from, uint32_t copy, int steps) {
    for (; steps > 0; steps -= kBatch) {         // the same for the warp
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (b >= steps) break;
        const uint32_t w[4] = {x[b].x, x[b].y, x[b].z, x[b].w};
        float u[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = T::to_f32x2(w[i]);
          u[2 * i] = f.x;
          u[2 * i + 1] = f.y;
        }
        float r = 1.f;
        if (norm) {
          float sum = u[0] * u[0];
#pragma unroll
          for (int i = 1; i < 8; ++i) sum = fmaf(u[i], u[i], sum);
#pragma unroll
          for (int d = LPH / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
          r = rsqrtf(fmaf(sum, inv_d, eps));
        }
        float v[8];
        if (INTER) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = fmaf(u[i ^ 1], other[i], u[i] * own[i]) * r;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = T::to_f32x2(__shfl_sync(0xFFFFFFFFu, w[i], from));
            v[2 * i] = fmaf(f.x, other[2 * i], u[2 * i] * own[2 * i]) * r;
            v[2 * i + 1] = fmaf(f.y, other[2 * i + 1], u[2 * i + 1] * own[2 * i + 1]) * r;
          }
        }
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = T::from_f32x2(v[2 * i], v[2 * i + 1]);
        if (COPY) {
          // what does not turn: the element times its weight, or its bits where
          // there is no norm (NaN and infinities next to it included)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (copy >> i & 1)
              o[i] = norm ? T::from_f32x2(u[2 * i] * own[2 * i] * r, u[2 * i + 1] * own[2 * i + 1] * r) : w[i];
        }
        if (active && b * step < left) *reinterpret_cast<uint4*>(out + b * out_step) = make_uint4(o[0], o[1], o[2], o[3]);
      }
      out += kBatch * out_step;
      left -= kBatch * step;
      if (steps > kBatch) load();
    }
  }
};

// 16 bytes of shared memory as floats.
__device__ __forceinline__ void lds4(const float* p, float* v) {
  const float4 f = *reinterpret_cast<const float4*>(p);
  v[0] = f.x;
  v[1] = f.y;
  v[2] = f.z;
  v[3] = f.w;
}

// `parts` warps (1, 2, 4 or 8, of one block) share a token.
template <class T, int LPH, bool INTER, bool COPY>
__global__ void __launch_bounds__(kRopeThreads, rope_blocks(INTER, COPY)) qk_norm_rope_kernel(const RopeArgs a, const int parts) {
  constexpr int kHeads = 32 / LPH;                   // heads per warp and step
  __shared__ double freq[kRopeMaxD / 2];
  __shared__ int axis[kRopeMaxD / 2];
  __shared__ __align__(16) float weights[2][kRopeMaxD];   // of the norms of q and k; 1 without
  // per token: cosines and sines, from the angle's half = R / 2 on those of no turn
  __shared__ __align__(16) float cs[kRopeWarps][kRopeMaxD / 2 + 8], sn[kRopeWarps][kRopeMaxD / 2 + 8];
  // q, k, the weights and the positions may be the previous kernel's output
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tokens = kRopeWarps / parts;
  const int slot = warp / parts, part = warp - slot * parts;
  const int e = lane & (LPH - 1);                    // elements 8 e .. 8 e + 7 of the head
  const bool active = 8 * e < a.D;
  const int step = parts * kHeads;
  const int half = a.R >> 1;
  const int head = part * kHeads + lane / LPH;

  RopeWalk<T, LPH, INTER, COPY> walk;
  int64_t t = static_cast<int64_t>(blockIdx.x) * tokens + slot;
  double pos = 0.;                                   // lane i: the position on axis i
  auto begin = [&] {
    walk.init(a.q, a.Hq, t, e, head, step, active);
    walk.load();
    if (lane < a.axes && half != 0) {
      const int64_t at = t * a.pos_stride + lane;
      pos = a.pos64 ? static_cast<double>(static_cast<const int64_t*>(a.positions)[at])
                    : static_cast<double>(static_cast<const int32_t*>(a.positions)[at]);
    }
  };
  if (t < a.T) begin();
  for (int j = threadIdx.x; j < half; j += kRopeThreads) {
    freq[j] = a.freq[j] * 0.15915494309189533577;    // in turns: 1 / (2 pi)
    axis[j] = min(max(a.axis[j], 0), a.axes - 1);
  }
  for (int j = threadIdx.x; j < 2 * kRopeMaxD; j += kRopeThreads) {
    const uint16_t* w = j < kRopeMaxD ? a.q.weight : a.k.weight;
    const int d = j & (kRopeMaxD - 1);
    weights[j / kRopeMaxD][d] = w != nullptr && d < a.D ? T::to_f32(w[d]) : 1.f;
  }
  for (int j = half + lane; j < kRopeMaxD / 2 + 8; j += 32) {
    cs[warp][j] = 1.f;
    sn[warp][j] = 0.f;
  }
  __syncthreads();

  int from = lane;                                   // halves: the lane of the pair's other element
  int angle = 4 * e;                                 // the lane's first angle
  int pair = 8 * e;                                  // halves: the pair's other element of the lane's first one
  float sign = 1.f;
  if (!INTER) {
    angle = kRopeMaxD / 2;                           // no turn
    if (8 * e < a.R) {
      const bool low = 8 * e < half;
      angle = low ? 8 * e : 8 * e - half;
      pair = low ? 8 * e + half : 8 * e - half;
      from = low ? lane + half / 8 : lane - half / 8;
      sign = low ? -1.f : 1.f;
    }
  }
  uint32_t copy = 0;                                 // words that do not turn
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (8 * e + 2 * i >= a.R) copy |= 1u << i;
  const float inv_d = 1.f / static_cast<float>(a.D);

  while (t < a.T) {                                  // the same for the warps of a token
    for (int j0 = part * 32; j0 < half; j0 += parts * 32) {
      const int j = min(j0 + lane, half - 1);
      double turns = __shfl_sync(0xFFFFFFFFu, pos, axis[j]) * freq[j];
      turns -= rint(turns);
      float sv, cv;
      sincospif(2.f * static_cast<float>(turns), &sv, &cv);
      if (j0 + lane < half) {
        cs[slot][j] = cv;
        sn[slot][j] = sv;
      }
    }
    bar_sync(1 + slot, parts * 32);
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
      const bool norm = (side == 0 ? a.q.weight : a.k.weight) != nullptr;
      const int H = side == 0 ? a.Hq : a.H - a.Hq;
      if (side == 1) {
        if (H == 0) break;
        walk.init(a.k, H, t, e, head, step, active);
        walk.load();
      }
      // element i turns into own * u_i + other * u_pair
      float own[8], other[8], w[8];
      lds4(&weights[side][8 * e], w);
      lds4(&weights[side][8 * e + 4], w + 4);
      if (INTER) {
        float c[4], s[4];
        lds4(&cs[slot][angle], c);
        lds4(&sn[slot][angle], s);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          own[i] = c[i / 2] * w[i];
          other[i] = (i & 1 ? s[i / 2] : -s[i / 2]) * w[i ^ 1];
        }
      } else {
        float c[8], s[8], wp[8];
        lds4(&cs[slot][angle], c);
        lds4(&cs[slot][angle + 4], c + 4);
        lds4(&sn[slot][angle], s);
        lds4(&sn[slot][angle + 4], s + 4);
        lds4(&weights[side][pair], wp);
        lds4(&weights[side][pair + 4], wp + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          own[i] = c[i] * w[i];
          other[i] = sign * s[i] * wp[i];
        }
      }
      const int steps = H > part * kHeads ? (H - part * kHeads + step - 1) / step : 0;
      walk.run(norm, inv_d, a.eps, own, other, from, copy, steps);
    }
    bar_sync(1 + slot, parts * 32);                  // the angles have been read
    t += static_cast<int64_t>(gridDim.x) * tokens;
    if (t < a.T) begin();                            // in flight while the next angles are formed
  }
}

template <class T>
cudaError_t launch_rope(const RopeArgs& a, int num_sms, cudaStream_t stream) {
  const int lph = a.D <= 64 ? 8 : (a.D <= 128 ? 16 : 32);
  // Warps per token.  A warp's time is about that of its head steps plus four
  // more for the angles and the rest of a token, and the tokens run in rounds
  // of what the GPU holds: take the number that costs least (one or two for
  // many tokens, as many as have heads to take for few).
  const int heads = 32 / lph, Hk = a.H - a.Hq;
  const int64_t most = static_cast<int64_t>(num_sms) * rope_blocks(a.interleaved != 0, a.R < a.D);
  int parts = 1;
  int64_t best = INT64_MAX;
  for (int p = 1; p <= kRopeWarps; p *= 2) {
    const int64_t at_once = most * (kRopeWarps / p);
    const int64_t rounds = (a.T + at_once - 1) / at_once;
    const int64_t cost = rounds * (4 + (a.Hq + p * heads - 1) / (p * heads) + (Hk + p * heads - 1) / (p * heads));
    if (cost < best) best = cost, parts = p;
  }
  const int tokens = kRopeWarps / parts;
  const int64_t blocks = (a.T + tokens - 1) / tokens;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks < most ? blocks : most), 1, 1);
  cfg.blockDim = dim3(kRopeThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int which = (lph == 8 ? 0 : lph == 16 ? 4 : 8) + (a.interleaved ? 2 : 0) + (a.R < a.D ? 1 : 0);
  switch (which) {
    case 0: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<T, 8, false, false>, a, parts);
    case 1: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<T, 8, false, true>, a, parts);
    case 2: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<T, 8, true, false>, a, parts);
    case 3: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<T, 8, true, true>, a, parts);
    case 4: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<T, 16, false, false>, a, parts);
    case 5: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<T, 16, false, true>, a, parts);
    case 6: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<T, 16, true, false>, a, parts);
    case 7: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<T, 16, true, true>, a, parts);
    case 8: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<T, 32, false, false>, a, parts);
    case 9: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<T, 32, false, true>, a, parts);
    case 10: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<T, 32, true, false>, a, parts);
    default: return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<T, 32, true, true>, a, parts);
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
  const cudaError_t e = dtype == W4A4_BF16 ? launch_rope<Bf16>(a, dev->num_sms, s) : launch_rope<Fp16>(a, dev->num_sms, s);
  return e == cudaSuccess ? W4A4_OK : W4A4_ERR_CUDA;
}
