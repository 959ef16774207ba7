// Softmax attention over packed sequences: full or causal, grouped heads.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "half16.cuh"
#include "ptx.cuh"
#include "w4a4.h"
#include "w4a4_internal.h"

namespace w4a4 {
namespace {

struct AttnArgs {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  float* lse;
  int64_t q_t, q_h, k_t, k_h, v_t, v_h, o_t, o_h;   // token and head strides in elements
  const int32_t *cu_q, *cu_k;
  int B, Tq, Tk, Hq, Hk;
  int causal;
  float scale;
};

__device__ __forceinline__ int cu_at(const int32_t* cu, int b, int total) {
  return cu == nullptr ? (b == 0 ? 0 : total) : min(max(cu[b], 0), total);
}

// One warp per query row and head; the running maximum and sum of the
// softmax, one key at a time.
template <class T, int D>
__global__ void __launch_bounds__(256) attention_rows_kernel(const AttnArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t row = w / a.Hq;
  const int h = static_cast<int>(w - row * a.Hq);
  if (row >= a.Tq) return;
  // the sequence of this row: the last b with cu_q[b] <= row, if row < cu_q[b + 1]
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (cu_at(a.cu_q, mid, a.Tq) <= row) lo = mid; else hi = mid;
  }
  const int q0 = cu_at(a.cu_q, lo, a.Tq), q1 = cu_at(a.cu_q, lo + 1, a.Tq);
  if (row < q0 || row >= q1) return;
  const int k0 = cu_at(a.cu_k, lo, a.Tk), k1 = cu_at(a.cu_k, lo + 1, a.Tk);
  const int Lk = max(k1 - k0, 0);
  int64_t seen = Lk;
  if (a.causal) seen = min(static_cast<int64_t>(Lk), row - q0 + Lk - (q1 - q0) + 1);
  const int hk = h / (a.Hq / a.Hk);
  float qv[E], acc[E] = {};
  for (int e = 0; e < E; ++e) qv[e] = T::to_f32(a.q[row * a.q_t + h * a.q_h + lane * E + e]);
  float m = -INFINITY, l = 0.f;
  for (int64_t j = 0; j < seen; ++j) {
    float s = 0.f;
    for (int e = 0; e < E; ++e) s = fmaf(qv[e], T::to_f32(a.k[(k0 + j) * a.k_t + hk * a.k_h + lane * E + e]), s);
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    s *= a.scale;
    const float mn = fmaxf(m, s);
    const float f = m == -INFINITY ? 0.f : expf(m - mn);
    const float p = s == -INFINITY ? 0.f : expf(s - mn);
    l = l * f + p;
    for (int e = 0; e < E; ++e) acc[e] = fmaf(p, T::to_f32(a.v[(k0 + j) * a.v_t + hk * a.v_h + lane * E + e]), acc[e] * f);
    m = mn;
  }
  const float r = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  for (int e = 0; e < E; ++e) a.out[row * a.o_t + h * a.o_h + lane * E + e] = T::from_f32(acc[e] * r);
  if (a.lse != nullptr && lane == 0) a.lse[row * a.Hq + h] = l == 0.f ? -INFINITY : m + logf(l);
}

int check_heads(const void* p, int64_t t, int64_t h, int64_t T, int64_t H, int64_t D) {
  const int64_t lim = int64_t(1) << 38;   // bytes of a stride stay below 2^40
  if (t > lim || h > lim) return W4A4_ERR_SHAPE;
  if ((T > 1 && t < D) || (H > 1 && h < D)) return W4A4_ERR_SHAPE;
  if (t % 8 != 0 || h % 8 != 0 || !aligned_to(p, 16)) return W4A4_ERR_ALIGN;
  return W4A4_OK;
}

}  // namespace
}  // namespace w4a4

using namespace w4a4;

extern "C" {

size_t w4a4_attention_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

int w4a4_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k,
                   int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
                   int64_t v_head_stride, void* out, int64_t out_token_stride, int64_t out_head_stride, float* lse,
                   const int32_t* cu_q, const int32_t* cu_k, int64_t B, int64_t Tq, int64_t Tk, int64_t Hq,
                   int64_t Hk, int64_t D, int causal, float scale, int dtype, void* workspace,
                   size_t workspace_bytes, void* stream) {
  if (Tq < 0 || Tk < 0 || Tq > (int64_t(1) << 30) || Tk > (int64_t(1) << 30)) return W4A4_ERR_SHAPE;
  if (Tq != 0 && (q == nullptr || out == nullptr)) return W4A4_ERR_NULL;
  if (Tk != 0 && (k == nullptr || v == nullptr)) return W4A4_ERR_NULL;
  if (B < 1 || B > (int64_t(1) << 24)) return W4A4_ERR_SHAPE;
  if ((cu_q == nullptr) != (cu_k == nullptr) || (cu_q == nullptr && B != 1)) return W4A4_ERR_NULL;
  if (D != 64 && D != 128) return W4A4_ERR_SHAPE;
  if (Hq < 1 || Hq > 65535 || Hk < 1 || Hq % Hk != 0) return W4A4_ERR_SHAPE;
  if (dtype != W4A4_BF16 && dtype != W4A4_FP16) return W4A4_ERR_ARG;
  if (!(scale > 0.f) || scale > 3.0e38f) return W4A4_ERR_ARG;
  int st;
  if ((st = check_heads(q, q_token_stride, q_head_stride, Tq, Hq, D)) != W4A4_OK) return st;
  if ((st = check_heads(out, out_token_stride, out_head_stride, Tq, Hq, D)) != W4A4_OK) return st;
  if ((st = check_heads(k, k_token_stride, k_head_stride, Tk, Hk, D)) != W4A4_OK) return st;
  if ((st = check_heads(v, v_token_stride, v_head_stride, Tk, Hk, D)) != W4A4_OK) return st;
  if (!aligned_to(lse, 4) || !aligned_to(cu_q, 4) || !aligned_to(cu_k, 4)) return W4A4_ERR_ALIGN;
  DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != W4A4_OK) return st;
  if (Tq == 0) return W4A4_OK;
  const size_t need = w4a4_attention_workspace_bytes(Tq, Tk, B, Hq, Hk, D);
  if (need != 0 && (workspace == nullptr || workspace_bytes < need || !aligned_to(workspace, 256)))
    return W4A4_ERR_WORKSPACE;
  AttnArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.q_t = q_token_stride, a.q_h = q_head_stride;
  a.k_t = k_token_stride, a.k_h = k_head_stride;
  a.v_t = v_token_stride, a.v_h = v_head_stride;
  a.o_t = out_token_stride, a.o_h = out_head_stride;
  a.cu_q = cu_q, a.cu_k = cu_k;
  a.B = static_cast<int>(B), a.Tq = static_cast<int>(Tq), a.Tk = static_cast<int>(Tk);
  a.Hq = static_cast<int>(Hq), a.Hk = static_cast<int>(Hk);
  a.causal = causal != 0;
  a.scale = scale;
  const int64_t blocks = (Tq * Hq + 7) / 8;
  auto kernel = dtype == W4A4_BF16 ? (D == 64 ? attention_rows_kernel<Bf16, 64> : attention_rows_kernel<Bf16, 128>)
                                   : (D == 64 ? attention_rows_kernel<Fp16, 64> : attention_rows_kernel<Fp16, 128>);
  if (blocks > 0x7FFFFFFF) return W4A4_ERR_SHAPE;
  kernel<<<static_cast<unsigned>(blocks), 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? W4A4_OK : W4A4_ERR_CUDA;
}

}  // extern "C"
