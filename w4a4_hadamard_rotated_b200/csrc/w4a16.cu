// Linear layer of a few 16-bit activation rows with 4-bit weights and group
// scales, and the offline quantiser of its weights.
//
//   y[m, n] = sum_g ( s[n, g] sum_{k in g} q[n, k] x[m, k] + o[n, g] sum_{k in g} x[m, k] ) + b[n]
// Every weight is used once per row of x: N K / 2 bytes of codes and 2 N K / group
// of scales against 2 M N K flops, bound by the weight stream up to the largest M.
//
// Design (linear_w4a16_kernel<T, RT, NT, FEW, WARPS, GROUP, OFFSET>)
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
//   * A warp takes RT tiles of 16 weight rows and a slice of k; the 8, 12 or
//     16 warps of a CTA split k, and their partial sums meet in shared memory
//     in a fixed order (no atomics).  More activation rows want more weight
//     rows per warp, since x is read once per warp.
//   * Each warp feeds itself: a ring of stages of 128 columns that TMA boxes
//     fill (weights 64 bytes a row, x 64 columns a row, both swizzled so that
//     the operand reads are free of bank conflicts; what is out of range
//     arrives as zeros), one lane issuing, no barrier between warps.
// Measured (graph replays): 1 x 3072 -> 3072 4.4 us, 1 x 5120 -> 30720 26 us
// (3.2 TB/s; issue slots 55% and ALU 53% busy: each warp's chain of wait, read,
// widen and multiply, and four rounds for 3.24), 8 x 12288 -> 3072 with offsets 11.3 us,
// 16 x 5120 -> 13824 of groups of 32 25.6 us.
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
// (w & mask) ^ magic
__device__ __forceinline__ uint32_t and_xor(uint32_t w, uint32_t mask, uint32_t magic) {
  uint32_t v;
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(v) : "r"(w), "r"(mask), "r"(magic));
  return v;
}

template <class T>
struct Widen;
template <>
struct Widen<Bf16> {
  static __device__ __forceinline__ uint32_t pair(uint32_t w) {
    const uint32_t v = and_xor(w, 0x000F000Fu, 0x43084308u);          // 136 + q
    const __nv_bfloat162 d =
        __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), __floats2bfloat162_rn(136.f, 136.f));
    return *reinterpret_cast<const uint32_t*>(&d);
  }
  // codes 0 and 4, 1 and 5, 2 and 6, 3 and 7 of a word as pairs of integers
  static __device__ __forceinline__ void word(uint32_t w, uint32_t (&p)[4]) {
    p[0] = pair(w);
    p[1] = pair(w >> 4);
    p[2] = pair(w >> 8);
    p[3] = pair(w >> 12);
  }
  static constexpr uint32_t kOnes = 0x3F803F80u;
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  }
};
template <>
struct Widen<Fp16> {
  // the low nibbles of the bytes: 1032 + q;  the high ones where they lie, 16
  // times as large: 1024 + 16 (q + 8) = 1152 + 16 q, one multiply-add (exact)
  static __device__ __forceinline__ uint32_t low(uint32_t w) {
    const uint32_t v = and_xor(w, 0x000F000Fu, 0x64086408u);
    const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&v), __floats2half2_rn(1032.f, 1032.f));
    return *reinterpret_cast<const uint32_t*>(&d);
  }
  static __device__ __forceinline__ uint32_t high(uint32_t w) {
    const uint32_t v = and_xor(w, 0x00F000F0u, 0x64806480u);
    const __half2 d = __hfma2(*reinterpret_cast<const __half2*>(&v), __floats2half2_rn(0.0625f, 0.0625f),
                              __floats2half2_rn(-72.f, -72.f));
    return *reinterpret_cast<const uint32_t*>(&d);
  }
  static __device__ __forceinline__ void word(uint32_t w, uint32_t (&p)[4]) {
    p[0] = low(w);
    p[1] = high(w);
    p[2] = low(w >> 8);
    p[3] = high(w >> 8);
  }
  static constexpr uint32_t kOnes = 0x3C003C00u;
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  }
};

constexpr int kW16Cols = 128;        // columns of a stage

struct W16Args {
  const uint16_t *scale, *offset, *bias;
  uint16_t* y;
  int64_t ldy;
  int M, N, K;
  int tiles;           // sets of RT * 16 rows
  unsigned int* status;
  unsigned long long wait_ns;
};

// FEW: one or two activation rows.  WARPS: of a CTA, which share k.
template <int RT, int NT, bool FEW, int WARPS, bool OFFSET>
struct W16Shape {
  static_assert(RT == 1 || RT == 2, "rows of a warp: whole lanes' worth of scales");
  static constexpr int kRows = RT * 16;
  static constexpr int kCols = FEW ? 2 : NT * 8;             // columns of a partial sum
  static constexpr uint32_t kW = kRows * 64;                 // codes of a stage
  // x of a stage: two boxes of 64 columns, 128-byte swizzle; for one or two
  // rows one unswizzled box of 128 columns
  static constexpr uint32_t kXBox = FEW ? 512 : NT * 1024;
  static constexpr uint32_t kX = FEW ? 512 : 2 * kXBox;
  static constexpr uint32_t kStage = kW + kX;          // a multiple of the swizzles' period: 512 bytes, with x swizzled 1024
  static constexpr int kStages = FEW && WARPS <= 8 ? 3 : 2;
  // groups of a row whose scales a warp holds at a time (with offsets, which
  // take as much room again, half as many), and the row pitch that holds them
  // from any beginning, rounded down to 8 groups
  static constexpr int kHeld = OFFSET ? 8 : 16;
  static constexpr int kPitch = kHeld + 8;
  static constexpr uint32_t kScale = kRows * kPitch * 2;     // of one such chunk
  static constexpr uint32_t kWarp = (OFFSET ? 4 : 2) * kScale;
  static constexpr uint32_t kPart = WARPS * kRows * kCols * sizeof(float);
  static constexpr uint32_t kRing = WARPS * kStages * kStage;
  static constexpr uint32_t kSmem = kRing + kPart + WARPS * kWarp + 1024;
  static_assert(kSmem <= 226 * 1024, "does not fit an SM's shared memory");
  static constexpr int kBlocks = kSmem <= 113 * 1024 && WARPS <= 8 ? 2 : 1;
};

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
}

// Scales (or offsets) first .. first + count - 1 of a warp's rows into shared
// memory, [row][PITCH], beginning at first rounded down to `unit` groups:
// where rows are whole units of 16 (unit 8) or 4 bytes (unit 2) as asynchronous
// copies, to be waited for by cp_async_wait(), else loaded and stored here.
// Rows past N take the last one's.
template <int ROWS, int PITCH>
__device__ __forceinline__ void fetch_scales(uint16_t* to, const uint16_t* from, int row0, int N, int groups, int first,
                                             int count, int unit) {
  const int lane = threadIdx.x & 31;
  constexpr int kLanes = 32 / (ROWS < 32 ? ROWS : 32);       // lanes of a row
  const int last = min(first + count, groups) - 1;
#pragma unroll
  for (int r = 0; r < ROWS; r += 32 / kLanes) {
    const int row = r + lane / kLanes;
    const uint16_t* src = from + static_cast<int64_t>(min(row0 + row, N - 1)) * groups;
    uint16_t* dst = to + row * PITCH;
    const int g0 = first & -unit;
    if (unit == 8) {
      for (int g = g0 + 8 * (lane % kLanes); g <= last; g += 8 * kLanes) cp_async<16>(smem_u32(dst + (g - g0)), src + g);
    } else if (unit == 2) {
      for (int g = g0 + 2 * (lane % kLanes); g <= last; g += 2 * kLanes) cp_async<4>(smem_u32(dst + (g - g0)), src + g);
    } else {
      for (int g = g0 + lane % kLanes; g <= last; g += kLanes) dst[g - g0] = src[g];
    }
  }
}

// A persistent grid over sets of RT * 16 weight rows; each warp with its slice of k.
template <class T, int RT, int NT, bool FEW, int WARPS, int GROUP, bool OFFSET>
__global__ void __launch_bounds__(WARPS * 32, W16Shape<RT, NT, FEW, WARPS, OFFSET>::kBlocks)
    linear_w4a16_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                        const W16Args a) {
  using Shape = W16Shape<RT, NT, FEW, WARPS, OFFSET>;
  constexpr int kRows = Shape::kRows, kCols = Shape::kCols, kStages = Shape::kStages;
  constexpr int kGroups = kW16Cols / GROUP;            // groups of a stage
  constexpr int kPitch = Shape::kPitch;
  constexpr int kEvery = Shape::kHeld / kGroups;         // stages whose scales are held at a time
  extern __shared__ uint8_t smem_dyn[];
  __shared__ uint64_t full[WARPS][kStages];
  uint8_t* smem = align1024_shared(smem_dyn);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int groups = a.K / GROUP;
  // this warp's stages of k
  const int units = (a.K + kW16Cols - 1) / kW16Cols;
  const int u0 = units * warp / WARPS, n = units * (warp + 1) / WARPS - u0;
  uint8_t* ring = smem + warp * kStages * Shape::kStage;
  float* part = reinterpret_cast<float*>(smem + Shape::kRing);            // [warps][kRows][kCols]
  uint16_t* scales = reinterpret_cast<uint16_t*>(smem + Shape::kRing + Shape::kPart + warp * Shape::kWarp);
  const uintptr_t bits = reinterpret_cast<uintptr_t>(a.scale) | reinterpret_cast<uintptr_t>(a.offset);
  const int unit = groups % 8 == 0 && (bits & 15) == 0 ? 8 : (groups % 2 == 0 && (bits & 3) == 0 ? 2 : 1);

  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&full[warp][s], 1);
    fence_mbar_init();
    fence_async_shared();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  // the first stages' codes on their way into L2 while the previous kernel of the
  // stream ends (a prefetch reads nothing into this kernel)
  if (lane < kStages && lane < n)
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(&tmW)),
                 "r"((u0 + lane) * (kW16Cols / 2)), "r"(static_cast<int>(blockIdx.x) * kRows) : "memory");
  __syncwarp();
  griddep_wait();
  griddep_launch_dependents();

  // ---- the two streams ahead of the sums: stages (lane 0, by TMA) and chunks of scales
  int in_tile = blockIdx.x, in_i = 0, in_s = 0;
  auto issue = [&] {                                   // lane 0
    if (in_tile >= a.tiles || n == 0) return;
    const int col = (u0 + in_i) * kW16Cols;
    uint8_t* at = ring + in_s * Shape::kStage;
    uint64_t* bar = &full[warp][in_s];
    mbar_arrive_expect_tx(bar, Shape::kW + static_cast<uint32_t>(a.M) * 256u);
    tma_load_2d(at, &tmW, bar, col / 2, in_tile * kRows);
    tma_load_2d(at + Shape::kW, &tmX, bar, col, 0);
    if (!FEW) tma_load_2d(at + Shape::kW + Shape::kXBox, &tmX, bar, col + 64, 0);
    if (++in_s == kStages) in_s = 0;
    if (++in_i == n) in_i = 0, in_tile += gridDim.x;
  };
  int sc_tile = blockIdx.x, sc_i = 0, sc_b = 0;        // the next chunk to fetch, and its buffer
  auto fetch = [&] {
    if (sc_tile >= a.tiles || n == 0) return;
    const int first = (u0 + sc_i) * kGroups, count = min(kEvery, n - sc_i) * kGroups;
    uint16_t* to = scales + sc_b * (Shape::kScale / 2);
    fetch_scales<kRows, kPitch>(to, a.scale, sc_tile * kRows, a.N, groups, first, count, unit);
    if (OFFSET) fetch_scales<kRows, kPitch>(to + Shape::kScale, a.offset, sc_tile * kRows, a.N, groups, first, count, unit);
    sc_b ^= 1;
    sc_i += kEvery;
    if (sc_i >= n) sc_i = 0, sc_tile += gridDim.x;
  };
  if (lane == 0)
    for (int i = 0; i < kStages; ++i) issue();
  fetch();

  int s = 0, sb = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (int tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
    const int row0 = tile * kRows;
    // the row this thread writes in the end (the threads are whole multiples of kRows)
    const int r_out = threadIdx.x % kRows, row = row0 + r_out;
    const float bias = a.bias != nullptr && row < a.N ? T::to_f32(a.bias[row]) : 0.f;
    float acc[RT][NT][4] = {};
    const uint16_t *sc = scales, *of = scales;
    for (int i = 0; i < n && ok; ++i) {
      if (i % kEvery == 0) {                           // this chunk has arrived, the next one sets off
        cp_async_wait();
        __syncwarp();
        const int skip = ((u0 + i) * kGroups) & (unit - 1);
        sc = scales + sb * (Shape::kScale / 2) + skip;
        of = sc + Shape::kScale;
        sb ^= 1;
        fetch();
      }
      ok = warp_wait_converged<true>(&full[warp][s], phase, nullptr, a.status, a.wait_ns);
      if (!ok) break;
      const uint32_t wbase = smem_u32(ring + s * Shape::kStage), xbase = wbase + Shape::kW;
      float sum[RT][NT][4], xs[NT][4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {                    // 64 columns each
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
              if (FEW) q = lds128(xbase + g * 256 + k * 128 + c * 16);
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
            if (GROUP < 64) {                          // lanes 0, 1 give their second word for the first of lanes 2, 3
              const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, t < 2 ? w[r][h].y : w[r][h].x, 2);
              if (t < 2) w[r][h].y = got; else w[r][h].x = got;
            }
          }
#pragma unroll
        for (int v = 0; v < 2; ++v) {                  // 32 columns each
          const int col = 64 * k + 32 * v;             // of the stage
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            uint32_t lo[4], hi[4];
            Widen<T>::word(v == 0 ? w[r][0].x : w[r][0].y, lo);
            Widen<T>::word(v == 0 ? w[r][1].x : w[r][1].y, hi);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const uint32_t A[4] = {lo[2 * p], hi[2 * p], lo[2 * p + 1], hi[2 * p + 1]};
#pragma unroll
              for (int j = 0; j < NT; ++j) {
                if (col % GROUP == 0 && p == 0) Widen<T>::mma_first(sum[r][j], A, xb[j][v][0], xb[j][v][1]);
                else Widen<T>::mma(sum[r][j], A, xb[j][v][2 * p], xb[j][v][2 * p + 1]);
              }
            }
          }
          if (OFFSET) {
            const uint32_t ones[4] = {Widen<T>::kOnes, Widen<T>::kOnes, Widen<T>::kOnes, Widen<T>::kOnes};
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
              for (int j = 0; j < NT; ++j) {
                if (col % GROUP == 0 && p == 0) Widen<T>::mma_first(xs[j], ones, xb[j][v][0], xb[j][v][1]);
                else Widen<T>::mma(xs[j], ones, xb[j][v][2 * p], xb[j][v][2 * p + 1]);
              }
          }
          if ((col + 32) % GROUP == 0) {               // a group is done
            const int e = min(i % kEvery * kGroups + col / GROUP, groups - 1 - (u0 + i - i % kEvery) * kGroups);
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int at = (16 * r + 8 * h + g) * kPitch + e;
                const float sf = T::to_f32(sc[at]), o = OFFSET ? T::to_f32(of[at]) : 0.f;
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                  for (int q = 2 * h; q < 2 * h + 2; ++q) {
                    acc[r][j][q] = fmaf(sf, sum[r][j][q], acc[r][j][q]);
                    if (OFFSET) acc[r][j][q] = fmaf(o, xs[j][q], acc[r][j][q]);
                  }
              }
          }
        }
      }
      __syncwarp();                                    // every lane has read the stage
      if (lane == 0) issue();
      if (++s == kStages) s = 0, phase ^= 1;
    }

    // partial sums of the warps, joined in order
    float* mine = part + warp * kRows * kCols;
    if (tile != static_cast<int>(blockIdx.x)) __syncthreads();   // the last tile's sums have been read
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (!FEW || t == 0)
            *reinterpret_cast<float2*>(&mine[(16 * r + 8 * h + g) * kCols + 8 * j + 2 * t]) =
                make_float2(acc[r][j][2 * h], acc[r][j][2 * h + 1]);
    __syncthreads();
    for (int m = threadIdx.x / kRows; m < a.M; m += WARPS * 32 / kRows) {
      const float* p = part + r_out * kCols + m;
      if (row < a.N) {
        float v = bias;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) v += p[w * kRows * kCols];
        a.y[m * a.ldy + row] = T::from_f32(v);
      }
    }
  }
  cp_async_wait();
  if (!ok && lane == 0)                                // an expired wait: what is in flight lands before the CTA ends
    for (int i = 0; i < kStages; ++i) {
      (void)mbar_wait(&full[warp][i], 0, nullptr, nullptr, 100000000ull);
      (void)mbar_wait(&full[warp][i], 1, nullptr, nullptr, 100000000ull);
    }
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

template <class T, int RT, int NT, bool FEW, int WARPS, int GROUP, bool OFFSET>
cudaError_t launch_w16(const W16Call& c, W16Args a) {
  using Shape = W16Shape<RT, NT, FEW, WARPS, OFFSET>;
  CUtensorMap tmW, tmX;
  if (tensor_map_2d(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.wq, a.N, a.K / 2, a.K / 2, 64, Shape::kRows,
                    CU_TENSOR_MAP_SWIZZLE_64B) != W4A4_OK ||
      tensor_map_2d(&tmX, c.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, c.x, a.M, a.K,
                    c.ldx * 2, FEW ? 128 : 64, a.M,
                    FEW ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B) != W4A4_OK)
    return cudaErrorInvalidValue;
  auto kernel = linear_w4a16_kernel<T, RT, NT, FEW, WARPS, GROUP, OFFSET>;
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
  a.tiles = (a.N + Shape::kRows - 1) / Shape::kRows;
  const int most = c.num_sms * Shape::kBlocks;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.tiles < most ? a.tiles : most), 1, 1);
  cfg.blockDim = dim3(WARPS * 32, 1, 1);
  cfg.dynamicSmemBytes = Shape::kSmem;
  cfg.stream = c.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, tmW, tmX, a);
}

// Rows and warps of a CTA.  16 warps share an SM either way: two CTAs of 8, or
// one of 16, which halves the slices of k.  A warp's stage of 32 rows takes 1.6
// times as long as one of 16, a tile about 1.5 of the former besides its
// stages, and the tiles run in rounds of what the GPU holds: take the least.
// Measured against one another: 1x4096->4096 32 rows x 16 warps 4.3, 16 x 8 5.0 us;
// 1x4096->1024 16 x 16 3.6, 16 x 8 4.1; 8x12288->3072 32 x 16 11.2, 16 x 8 12.8, 32 x 8 12.9;
// 4x5120->5120 32 x 8 9.2, 32 x 16 10.7; 1x5120->30720 32 x 8 27, 16 x 8 32, 32 x 16 31.
template <class T, int NT, bool FEW, int GROUP, bool OFFSET>
cudaError_t launch_w16_tiles(const W16Call& c, const W16Args& a) {
  const int units = (a.K + kW16Cols - 1) / kW16Cols;
  int best = 0;
  float least = 0.f;
  for (int i = 0; i < 4; ++i) {
    const int rows = i & 1 ? 32 : 16, warps = i & 2 ? 16 : 8, at_once = c.num_sms * 16 / warps;
    const int rounds = ((a.N + rows - 1) / rows + at_once - 1) / at_once;
    const float cost = rounds * ((units + warps - 1) / warps * (i & 1 ? 1.f : 0.62f) + 1.5f);
    if (i == 0 || cost < least) least = cost, best = i;
  }
  switch (best) {
    case 0: return launch_w16<T, 1, NT, FEW, 8, GROUP, OFFSET>(c, a);
    case 1: return launch_w16<T, 2, NT, FEW, 8, GROUP, OFFSET>(c, a);
    case 2: return launch_w16<T, 1, NT, FEW, 16, GROUP, OFFSET>(c, a);
    default: return launch_w16<T, 2, NT, FEW, 16, GROUP, OFFSET>(c, a);
  }
}

template <class T, int GROUP, bool OFFSET>
cudaError_t launch_w16_rows(const W16Call& c, const W16Args& a) {
  if (a.M <= 2) return launch_w16_tiles<T, 1, true, GROUP, OFFSET>(c, a);
  if (a.M <= 8) return launch_w16_tiles<T, 1, false, GROUP, OFFSET>(c, a);
  // More rows of x than weights per stage: two CTAs of 32 rows do not fit an
  // SM.  One of 32 rows and 12 warps, or two of 16 rows and 8 warps, which read
  // x twice as often, split k less and share an SM (a last round of one CTA per
  // SM takes about half): microseconds of groups of 32, by their rounds.  Measured
  // at 16 rows, groups of 128, 32 x 12 against 16 x 8: 4096->1024 7.4 and 4.8,
  // 5120->5120 14.4 and 11.5, 2048->30000 30 and 24, 12288->3072 14.3 and 15.4;
  // groups of 32: 5120->13824 25.3 and 27.0.
  const int units = (a.K + kW16Cols - 1) / kW16Cols;
  const int wide = (a.N + 31) / 32, narrow = (a.N + 15) / 16, pair = 2 * c.num_sms, rest = narrow % pair;
  const float rounds = narrow / pair + (rest == 0 ? 0.f : rest <= c.num_sms ? 0.55f : 1.f);
  if (0.5f + rounds * (0.9f + 1.55f * ((units + 7) / 8)) <
      2.f + (wide + c.num_sms - 1) / c.num_sms * (0.7f + 1.8f * ((units + 11) / 12)))
    return launch_w16<T, 1, 2, false, 8, GROUP, OFFSET>(c, a);
  return launch_w16<T, 2, 2, false, 12, GROUP, OFFSET>(c, a);
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
