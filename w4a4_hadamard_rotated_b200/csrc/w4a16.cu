// Linear layer of a few 16-bit activation rows with 4-bit weights and group
// scales, and the offline quantiser of its weights.
//
//   y[m, n] = sum_g ( s[n, g] sum_{k in g} q[n, k] x[m, k] + o[n, g] sum_{k in g} x[m, k] ) + b[n]
// Every weight is used once per row of x: N K / 2 bytes of codes and 2 N K / group
// of scales against 2 M N K flops, bound by the weight stream up to the largest M.
//
// Design (linear_w4a16_kernel<T, RT, NT, GROUP, OFFSET>)
//   * Warp-level mma.m16n8k16 with fp32 sums: the weights are the 16-row A
//     operand, x the 8-column B operand.  One instruction per 256 weights
//     leaves the issue slots to the widening, the dearest part (11 per 8 codes);
//     tcgen05 would want the widened weights in shared or tensor memory first,
//     four times the bytes of the stream, for a product this small.
//   * Codes become exact 16-bit integers: (code ^ 8) in the mantissa of 128
//     (bf16) or 1024 (fp16), less 136 or 1032.  Products and sums of a group
//     are then those of integers and x; the scale multiplies a group's sum in fp32
//     once, nothing is rounded before y.
//   * The order of k inside a group is free as long as both operands share
//     it: a lane reads 8 bytes of a weight row, so four lanes hold 64 columns, and
//     nibbles 0 and 4, 1 and 5, ... of a word become the pairs of an operand
//     register; x is read where it lies and paired the same way.  For groups of 32 lanes
//     0, 1 and 2, 3 swap a word, so that an instruction stays inside a group.
//   * Sums of x per group (offsets) come from one more product per step with
//     an A operand of ones, shared by the RT row tiles.
//   * A warp takes RT tiles of 16 weight rows and a slice of k; the 8 warps
//     of a CTA and the CTAs of a cluster split k, so that a few thousand rows
//     fill the GPU too, and their partial sums meet in shared memory in a
//     fixed order (no atomics).  More activation rows want more weight rows
//     per warp, since x is read once per warp.
//   * Each warp feeds itself: a ring of stages of 128 columns that TMA boxes
//     fill (weights 64 bytes a row, x 64 columns a row, both swizzled so that
//     the operand reads are free of bank conflicts; what is out of range
//     arrives as zeros), one lane issuing, no barrier between warps.
//   Every wait is bounded; an expired one records W4A4_ERR_TIMEOUT, ends the
//   warp's sums early and lets its copies land.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "half16.cuh"
#include "ptx.cuh"
#include "w4a4.h"
#include "w4a4_internal.h"

namespace w4a4 {
namespace {

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
constexpr int kW16Warps = 8;

template <class T>
struct Widen;
template <>
struct Widen<Bf16> {
  // the codes at bits 0..3 and 16..19 of w, as bf16 integers
  static __device__ __forceinline__ uint32_t pair(uint32_t w) {
    uint32_t v, r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(v) : "r"(w), "r"(0x000F000Fu), "r"(0x43084308u));   // (w & mask) ^ magic
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                     __floats2bfloat162_rn(136.f, 136.f));
    r = *reinterpret_cast<const uint32_t*>(&d);
    return r;
  }
  static constexpr uint32_t kOnes = 0x3F803F80u;
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
template <>
struct Widen<Fp16> {
  static __device__ __forceinline__ uint32_t pair(uint32_t w) {
    uint32_t v;
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(v) : "r"(w), "r"(0x000F000Fu), "r"(0x64086408u));
    const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&v), __floats2half2_rn(1032.f, 1032.f));
    return *reinterpret_cast<const uint32_t*>(&d);
  }
  static constexpr uint32_t kOnes = 0x3C003C00u;
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

constexpr int kW16Cols = 128;        // columns of a stage

struct W16Args {
  const uint16_t *scale, *offset, *bias;
  uint16_t* y;
  int64_t ldy;
  int M, N, K;
  int split;           // CTAs of a cluster, each with a slice of k
  unsigned int* status;
  unsigned long long wait_ns;
};

template <int RT, int NT>
struct W16Shape {
  static constexpr int kRows = RT * 16, kCols = NT * 8;
  static constexpr uint32_t kW = kRows * 64;                 // codes of a stage
  // x of a stage: two boxes of 64 columns, 128-byte swizzle; for one or two
  // rows (RT == 1) one unswizzled box of 128 columns
  static constexpr uint32_t kXBox = RT == 1 ? 512 : NT * 1024;
  static constexpr uint32_t kX = RT == 1 ? 512 : 2 * kXBox;
  static constexpr uint32_t kStage = kW + kX;               // a multiple of the swizzle pattern: 512 bytes (RT == 1), 1024
  static constexpr int kStages = RT == 1 ? 5 : (NT == 1 ? 3 : 2);
  static constexpr uint32_t kRing = kW16Warps * kStages * kStage;
  static constexpr uint32_t kParts = (kW16Warps + 1) * kRows * kCols * sizeof(float);
  static constexpr uint32_t kSmem = (kRing > kParts ? kRing : kParts) + 1024;
};

// The scales (or offsets) of a row's groups in a stage: kW16Cols / GROUP
// 16-bit numbers from `at` on, those past the row's last group are that group's.
template <int GROUP>
struct Scales {
  static constexpr int kCount = kW16Cols / GROUP;
  uint32_t w[kCount == 4 ? 2 : 1];
  __device__ __forceinline__ void load(const uint16_t* row, int at, int groups, bool wide) {
    if (kCount == 1) {
      w[0] = row[min(at, groups - 1)];
    } else if (wide) {                                 // rows of an even number of 4 or 8 bytes
      if (kCount == 2) {
        w[0] = *reinterpret_cast<const uint32_t*>(row + min(at, groups - 2));
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(row + min(at, groups - 4));
        w[0] = v.x;
        w[kCount == 4 ? 1 : 0] = v.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kCount; i += 2)
        w[i / 2] = row[min(at + i, groups - 1)] | static_cast<uint32_t>(row[min(at + i + 1, groups - 1)]) << 16;
    }
  }
  template <class T>
  __device__ __forceinline__ float get(int i) const {
    return T::to_f32(static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1))));
  }
};

// grid.x = row tile sets * split; 8 warps.
template <class T, int RT, int NT, int GROUP, bool OFFSET>
__global__ void __launch_bounds__(kW16Warps * 32, 2)
    linear_w4a16_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                        const W16Args a) {
  using Shape = W16Shape<RT, NT>;
  constexpr int kRows = Shape::kRows, kCols = Shape::kCols, kStages = Shape::kStages;
  constexpr int kGroups = kW16Cols / GROUP;
  extern __shared__ uint8_t smem_dyn[];
  __shared__ uint64_t full[kW16Warps][kStages];
  uint8_t* smem = align1024_shared(smem_dyn);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int rank = static_cast<int>(blockIdx.x) % a.split;
  const int row0 = static_cast<int>(blockIdx.x) / a.split * kRows;
  const int groups = a.K / GROUP;
  // this warp's stages of k
  const int units = (a.K + kW16Cols - 1) / kW16Cols, shares = a.split * kW16Warps, share = rank * kW16Warps + warp;
  const int u0 = static_cast<int>(static_cast<int64_t>(units) * share / shares);
  const int n = static_cast<int>(static_cast<int64_t>(units) * (share + 1) / shares) - u0;
  uint8_t* ring = smem + warp * kStages * Shape::kStage;

  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&full[warp][s], 1);
    fence_mbar_init();
    fence_async_shared();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  __syncwarp();
  griddep_wait();
  griddep_launch_dependents();

  auto issue = [&](int i) {                            // lane 0
    const int s = i % kStages, col = (u0 + i) * kW16Cols;
    uint8_t* at = ring + s * Shape::kStage;
    mbar_arrive_expect_tx(&full[warp][s], Shape::kW + static_cast<uint32_t>(a.M) * 256u);
    tma_load_2d(at, &tmW, &full[warp][s], col / 2, row0);
    tma_load_2d(at + Shape::kW, &tmX, &full[warp][s], col, 0);
    if (RT > 1) tma_load_2d(at + Shape::kW + Shape::kXBox, &tmX, &full[warp][s], col + 64, 0);
  };
  if (lane == 0)
    for (int i = 0; i < kStages && i < n; ++i) issue(i);

  // rows past N take the last row's scales; their codes are zeros and their results dropped
  const uint16_t *srow[RT][2], *orow[RT][2];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t row = min(row0 + 16 * i + 8 * h + g, a.N - 1);
      srow[i][h] = a.scale + row * groups;
      if (OFFSET) orow[i][h] = a.offset + row * groups;
    }
  const bool wide = groups % kGroups == 0 &&
                    ((reinterpret_cast<uintptr_t>(a.scale) | reinterpret_cast<uintptr_t>(a.offset)) & (2 * kGroups - 1)) == 0;
  Scales<GROUP> sc[RT][2], of[RT][2];
  auto load_scales = [&](int i) {
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        sc[r][h].load(srow[r][h], (u0 + i) * kGroups, groups, wide);
        if (OFFSET) of[r][h].load(orow[r][h], (u0 + i) * kGroups, groups, wide);
      }
  };
  float acc[RT][NT][4] = {};
  if (n > 0) load_scales(0);
  bool ok = true;

  for (int i = 0; i < n; ++i) {
    const int s = i % kStages;
    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&full[warp][s], (i / kStages) & 1, nullptr, a.status, a.wait_ns));
    if (!ok) break;
    const uint32_t wbase = smem_u32(ring + s * Shape::kStage), xbase = wbase + Shape::kW;
    const Scales<GROUP>(&s0)[RT][2] = sc;
    float sf[RT][2][kGroups], of32[RT][2][kGroups];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < kGroups; ++e) {
          sf[r][h][e] = s0[r][h].template get<T>(e);
          of32[r][h][e] = OFFSET ? of[r][h].template get<T>(e) : 0.f;
        }
    if (i + 1 < n) load_scales(i + 1);
    float sum[RT][NT][4] = {}, xs[NT][4] = {};
#pragma unroll
    for (int k = 0; k < 2; ++k) {                      // 64 columns each
      // x as the B operand: this lane's 16 elements of row 8 j + g, as pairs (0, 4), (1, 5), (2, 6), (3, 7)
      uint32_t xb[NT][2][4];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          // which eight columns: with groups of 32 the order after the swap below
          const int c = GROUP < 64 ? (4 * v | (t & 1) << 1 | t >> 1) : 2 * t + v;
          uint4 q = make_uint4(0u, 0u, 0u, 0u);
          if (8 * j + g < a.M) {
            if (RT == 1) q = lds128(xbase + g * 256 + k * 128 + c * 16);
            else q = lds128(xbase + k * Shape::kXBox + (8 * j + g) * 128 + ((c ^ g) << 4));
          }
          xb[j][v][0] = __byte_perm(q.x, q.z, 0x5410);
          xb[j][v][1] = __byte_perm(q.x, q.z, 0x7632);
          xb[j][v][2] = __byte_perm(q.y, q.w, 0x5410);
          xb[j][v][3] = __byte_perm(q.y, q.w, 0x7632);
        }
      uint2 w[RT][2];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = 16 * r + 8 * h + g, chunk = 2 * k + (t >> 1);
          w[r][h] = lds64(wbase + row * 64 + ((chunk ^ (row >> 1 & 3)) << 4) + 8 * (t & 1));
          if (GROUP < 64) {                            // lanes 0, 1 give their second word for the first of lanes 2, 3
            const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, t < 2 ? w[r][h].y : w[r][h].x, 2);
            if (t < 2) w[r][h].y = got; else w[r][h].x = got;
          }
        }
#pragma unroll
      for (int v = 0; v < 2; ++v) {                    // 32 columns each
#pragma unroll
        for (int p = 0; p < 2; ++p) {
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const uint32_t lo = v == 0 ? w[r][0].x : w[r][0].y, hi = v == 0 ? w[r][1].x : w[r][1].y;
            const uint32_t A[4] = {Widen<T>::pair(lo >> (8 * p)), Widen<T>::pair(hi >> (8 * p)),
                                   Widen<T>::pair(lo >> (8 * p + 4)), Widen<T>::pair(hi >> (8 * p + 4))};
#pragma unroll
            for (int j = 0; j < NT; ++j) Widen<T>::mma(sum[r][j], A, xb[j][v][2 * p], xb[j][v][2 * p + 1]);
          }
          if (OFFSET) {
            const uint32_t ones[4] = {Widen<T>::kOnes, Widen<T>::kOnes, Widen<T>::kOnes, Widen<T>::kOnes};
#pragma unroll
            for (int j = 0; j < NT; ++j) Widen<T>::mma(xs[j], ones, xb[j][v][2 * p], xb[j][v][2 * p + 1]);
          }
        }
        const int col = 64 * k + 32 * v + 32;          // columns done
        if (col % GROUP == 0) {
          const int e = col / GROUP - 1;
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                acc[r][j][q] = fmaf(sf[r][q >> 1][e], sum[r][j][q], acc[r][j][q]);
                if (OFFSET) acc[r][j][q] = fmaf(of32[r][q >> 1][e], xs[j][q], acc[r][j][q]);
                sum[r][j][q] = 0.f;
              }
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) xs[j][q] = 0.f;
        }
      }
    }
    __syncwarp();                                      // every lane has read the stage
    if (lane == 0 && i + kStages < n) issue(i + kStages);
  }
  if (!ok && lane == 0)                                // what is in flight lands before the memory is used again
    for (int s = 0; s < kStages && s < n; ++s) {
      (void)mbar_wait(&full[warp][s], 0, nullptr, nullptr, 100000000ull);
      (void)mbar_wait(&full[warp][s], 1, nullptr, nullptr, 100000000ull);
    }

  // partial sums of the warps, joined in order; then those of the cluster
  __syncthreads();                                     // the rings are free
  float* part = reinterpret_cast<float*>(smem);        // [warps][kRows][kCols], then the CTA's [kRows][kCols]
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2*>(&part[(warp * kRows + 16 * r + 8 * h + g) * kCols + 8 * j + 2 * t]) =
            make_float2(acc[r][j][2 * h], acc[r][j][2 * h + 1]);
  __syncthreads();
  float* mine = part + kW16Warps * kRows * kCols;
  for (int i = threadIdx.x; i < kRows * kCols; i += kW16Warps * 32) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kW16Warps; ++w) v += part[w * kRows * kCols + i];
    mine[i] = v;
  }
  if (a.split > 1) cluster_sync();
  else __syncthreads();
  // output i: row i % kRows, activation row i / kRows; the CTAs of a cluster share them out
  for (int i = rank * kW16Warps * 32 + threadIdx.x; i < kRows * a.M; i += a.split * kW16Warps * 32) {
    const int r = i % kRows, m = i / kRows, row = row0 + r;
    float v = 0.f;
    if (a.split > 1) {
      for (int c = 0; c < a.split; ++c) v += ld_cluster(&mine[r * kCols + m], c);
    } else {
      v = mine[r * kCols + m];
    }
    if (row < a.N) {
      if (a.bias != nullptr) v += T::to_f32(a.bias[row]);
      a.y[m * a.ldy + row] = T::from_f32(v);
    }
  }
  if (a.split > 1) cluster_sync();                     // nobody leaves while its sums are read
}

// The call's operands as the launcher takes them.
struct W16Call {
  const uint16_t* x;
  int64_t ldx;
  const int8_t* wq;
  bool bf16;
  int num_sms;
  cudaStream_t stream;
};

template <class T, int RT, int NT, int GROUP, bool OFFSET>
cudaError_t launch_w16(const W16Call& c, W16Args a) {
  using Shape = W16Shape<RT, NT>;
  CUtensorMap tmW, tmX;
  if (tensor_map_2d(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.wq, a.N, a.K / 2, a.K / 2, 64, Shape::kRows,
                    CU_TENSOR_MAP_SWIZZLE_64B) != W4A4_OK ||
      tensor_map_2d(&tmX, c.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, c.x, a.M, a.K,
                    c.ldx * 2, RT == 1 ? 128 : 64, a.M,
                    RT == 1 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B) != W4A4_OK)
    return cudaErrorInvalidValue;
  auto kernel = linear_w4a16_kernel<T, RT, NT, GROUP, OFFSET>;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape::kSmem);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  const int64_t tiles = (a.N + Shape::kRows - 1) / Shape::kRows;
  // slices of k: until there are two CTAs per SM, as long as a warp keeps a stage
  const int64_t units = a.K / kW16Cols;
  int split = 1;
  while (split < 8 && tiles * split < 2 * c.num_sms && units >= 2 * split * kW16Warps) split *= 2;
  a.split = split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * split), 1, 1);
  cfg.blockDim = dim3(kW16Warps * 32, 1, 1);
  cfg.dynamicSmemBytes = Shape::kSmem;
  cfg.stream = c.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, tmW, tmX, a);
}

template <class T, int GROUP, bool OFFSET>
cudaError_t launch_w16_rows(const W16Call& c, const W16Args& a) {
  if (a.M <= 2) return launch_w16<T, 1, 1, GROUP, OFFSET>(c, a);
  if (a.M <= 8) return launch_w16<T, 2, 1, GROUP, OFFSET>(c, a);
  return launch_w16<T, 2, 2, GROUP, OFFSET>(c, a);
}

template <class T>
cudaError_t launch_w16_all(const W16Call& c, const W16Args& a, int group) {
  const bool o = a.offset != nullptr;
  if (group == 32) return o ? launch_w16_rows<T, 32, true>(c, a) : launch_w16_rows<T, 32, false>(c, a);
  if (group == 64) return o ? launch_w16_rows<T, 64, true>(c, a) : launch_w16_rows<T, 64, false>(c, a);
  return o ? launch_w16_rows<T, 128, true>(c, a) : launch_w16_rows<T, 128, false>(c, a);
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
  W16Args a{};
  a.scale = static_cast<const uint16_t*>(scale);
  a.offset = static_cast<const uint16_t*>(offset);
  a.bias = static_cast<const uint16_t*>(bias);
  a.ldy = ldy;
  a.N = static_cast<int>(N);
  a.K = static_cast<int>(K);
  a.status = dev->status;
  a.wait_ns = wait_limit_ns();
  W16Call c{nullptr, ldx, Wq, dtype == W4A4_BF16, dev->num_sms, static_cast<cudaStream_t>(stream)};
  // sixteen rows at a time: more read the weights again, from L2 where they fit it
  for (int64_t m = 0; m < M; m += 16) {
    c.x = static_cast<const uint16_t*>(x) + m * ldx;
    a.y = static_cast<uint16_t*>(y) + m * ldy;
    a.M = static_cast<int>(M - m < 16 ? M - m : 16);
    const cudaError_t e = c.bf16 ? launch_w16_all<Bf16>(c, a, group) : launch_w16_all<Fp16>(c, a, group);
    if (e != cudaSuccess) return W4A4_ERR_CUDA;
  }
  return W4A4_OK;
}

}  // extern "C"
