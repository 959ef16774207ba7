// Softmax attention over packed sequences: full or causal, grouped heads, long
// prompts and single tokens.
//
//   s_j = scale q . k_j,  m = max_j s_j,  l = sum_j e^(s_j - m),
//   out = sum_j e^(s_j - m) v_j / l,  lse = m + log l
// in one pass over the keys: a running maximum and sum per row, the output
// rescaled when the maximum moves.  4 D flops per (head, visible pair); on long
// prompts the tensor cores and the exponentials bound it, over a cache for
// few queries the bytes of k and v.
//
// Design (attention_tc_kernel<T, D, NQ, SPLIT, FEW>)
//   * A CTA owns NQ tiles of 128 query rows of one key head and walks 128-key
//     tiles.  The rows of a tile are (token, head) pairs: G heads that read
//     the same key head times 128 / G tokens (one 3-D TMA box), so grouped
//     heads share every key tile and a single token fills G rows of it.
//   * Warp roles: one TMA producer warp (k and v tiles through one ring), one
//     thread that issues the MMAs, and four softmax warps per query tile.
//       S = Q K^T   tcgen05.mma kind::f16, 128 x 128 x D, both from shared memory
//       O += P V    P from tensor memory, v as it lies (MN-major B operand)
//     S (128 columns) and O (D columns) stay in tensor memory in fp32.
//   * A softmax thread owns one row: it reads its 128 scores, so maximum and
//     sum need no shuffles, and writes the weights, rounded to 16 bits (the
//     MMA's operand type: half a step relative to each weight, in the sums of
//     v only; the softmax's own sum takes them unrounded), over the scores.
//   * With NQ = 2 the two tiles alternate: while the softmax of one runs, the
//     tensor cores do O += P V and the next S of the other.  MMAs execute in
//     issue order, so S(j + 1) may overwrite the P(j) that the MMA before it
//     read, and a commit of S(j + 1) tells that O(j) is complete: the softmax
//     warps rescale O themselves, no further role and no further barrier.
//   * The maximum in use follows the running one only when it falls behind
//     by more than 8 (fp16: 4, in log2 units), so that the rescaling of O, a
//     round trip through tensor memory, becomes rare.  The result is the same
//     quotient.
//   * In fp16 all weights and sums are 2^11 times as large (at most 2^15 with
//     what the maximum may be behind; fp16 holds 2^16), or keys 2^-14 below the
//     largest would already be subnormal and those 2^-25 below it nothing, while
//     the sum counts them in full: 4095 of them behind one whose value is 0 came
//     out 86% too small.  Now that begins at 2^-25 and 2^-36.
//   * Masks select (-inf) rather than add, on the tiles they cut only.  Value
//     rows behind a sequence's end inside its last tile are zeroed in
//     shared memory, so whatever lies there reaches nothing.
//   * Few tiles (SPLIT): the keys of a sequence are cut into chunks, one CTA
//     each (NQ = 1, two CTAs per SM); they write O and lse in fp32 to the
//     workspace and attention_join_kernel weighs them by e^(lse_c - lse).  A
//     sequence of one chunk is written at once.
//   * Few rows (FEW), a token or some over caches: the tile keeps 32 rows of q
//     in shared memory and one softmax warp, and the ring holds a third k or v
//     tile instead of the other 96 rows; the MMAs still run over 128 rows, those
//     behind the 32 of whatever lies there and read by nobody (8 tokens over 66796
//     keys: 51 us; with 128 rows, four warps and two tiles 58).
// Measured (D 128, calls back to back for seconds, where the board's power limit
// of 1000 W holds the clock at 1.6 to 1.75 GHz; in parentheses the first 10 ms of a
// rested GPU): bf16, 4608 x 24 heads 249 us, 1.05 PF/s (215 us, 1.21); 32760 x 10
// heads 4.73 ms, 1.16 PF/s (4.09, 1.35); fp16, eight causal prompts, 11168 tokens x
// 40/8 heads 438 us, 0.78 PF/s (384, 0.89); bf16, 8 tokens x 32/8 heads over 66796
// keys 57 us, 4.8 TB/s (52, 5.2).
//   Every wait is bounded; an expired wait records W4A4_ERR_TIMEOUT, every
//   role stops, copies and MMAs drain and tensor memory is freed.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "half16.cuh"
#include "ptx.cuh"
#include "w4a4.h"
#include "w4a4_internal.h"

namespace w4a4 {
namespace {

constexpr int kTile = 128;             // query rows per MMA tile and keys per key tile
constexpr int kFewRows = 32;           // query rows of a tile of few
// Every block looks for its place among the sequences, so their search grows
// with their square: 16384 single tokens x 8/8 heads take 25 ms, a million would
// take minutes.
constexpr int64_t kMaxSequences = 65536;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// log2: how far the maximum in use may fall behind, and how far below it the
// weights' unit lies
template <class T>
constexpr float kBehind = std::is_same<T, Bf16>::value ? 8.f : 4.f;
template <class T>
constexpr float kUnit = std::is_same<T, Bf16>::value ? 0.f : 11.f;

struct AttnArgs {
  uint16_t* out;
  float* lse;
  int64_t o_t, o_h;                    // token and head strides in elements
  const int32_t *cu_q, *cu_k;
  int B, Tq, Tk, Hq;
  int G;                               // heads of one key head packed into a tile
  int groups;                          // packed head sets per key head
  int tokens;                          // tokens per 128-row tile: 128 / G
  int causal;
  float scale_log2;                    // scale * log2 e
  int chunk;                           // SPLIT: key tiles per chunk
  int blocks;                          // SPLIT: upper bound of a head set's places
  float* part_o;                       // SPLIT: [chunks][Tq][Hq][D]
  float* part_lse;                     // SPLIT: [chunks][Tq][Hq], log2 units
  unsigned int* status;
  unsigned long long wait_ns;
};

__device__ __forceinline__ int cu_at(const int32_t* cu, int b, int total) {
  return cu == nullptr ? (b == 0 ? 0 : total) : min(max(cu[b], 0), total);
}

// Where a block works.
struct Place {
  int q0, nq;        // the sequence's first query row, their number
  int k0, nk;        // the same of its keys
  int tile;          // its number among the sequence's query tiles (NQ * tokens each)
  int chunk;         // SPLIT: which chunk of the keys
};

// The place of block `index`: sequences in order, each with its query tiles
// times its key chunks.  A warp walks the sequences 32 kEach at a time.
template <int kEach>
__device__ __forceinline__ bool find_place(const AttnArgs& a, int index, int tokens, int chunk_tiles, Place& p) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32 * kEach) {
    const int b = b0 + lane * kEach;
    int cq[kEach + 1], ck[kEach + 1];
#pragma unroll
    for (int i = 0; i <= kEach; ++i) {
      cq[i] = b + i <= a.B ? cu_at(a.cu_q, b + i, a.Tq) : 0;
      ck[i] = b + i <= a.B ? cu_at(a.cu_k, b + i, a.Tk) : 0;
    }
    int n[kEach], chunks[kEach], sum = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int nq = max(cq[i + 1] - cq[i], 0), nk = max(ck[i + 1] - ck[i], 0);
      chunks[i] = 1;
      if (chunk_tiles != 0) chunks[i] = max(1, ((nk + kTile - 1) / kTile + chunk_tiles - 1) / chunk_tiles);
      n[i] = b + i < a.B ? (nq + tokens - 1) / tokens * chunks[i] : 0;
      sum += n[i];
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if (lane >= d) incl += o;
    }
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, before + incl > index);
    if (hit != 0) {
      // the block's sequence among the four of this lane, if it is this lane
      int at = index - (before + incl - sum), i = 0;
      for (; i < kEach - 1 && at >= n[i]; ++i) at -= n[i];
      int q0 = cq[0], q1 = cq[1], k0 = ck[0], k1 = ck[1], ch = chunks[0], most = n[0];
#pragma unroll
      for (int j = 1; j < kEach; ++j)
        if (i == j) q0 = cq[j], q1 = cq[j + 1], k0 = ck[j], k1 = ck[j + 1], ch = chunks[j], most = n[j];
      const int src = __ffs(hit) - 1;
      at = __shfl_sync(0xFFFFFFFFu, at, src);
      most = __shfl_sync(0xFFFFFFFFu, most, src);
      ch = __shfl_sync(0xFFFFFFFFu, ch, src);
      p.q0 = __shfl_sync(0xFFFFFFFFu, q0, src);
      p.nq = max(__shfl_sync(0xFFFFFFFFu, q1, src) - p.q0, 0);
      p.k0 = __shfl_sync(0xFFFFFFFFu, k0, src);
      p.nk = max(__shfl_sync(0xFFFFFFFFu, k1, src) - p.k0, 0);
      if (at < 0 || at >= most) return false;        // lengths whose sums do not fit an int
      p.tile = at / ch;
      p.chunk = at - p.tile * ch;
      return true;
    }
    before += __shfl_sync(0xFFFFFFFFu, incl, 31);
  }
  return false;
}

// The sequence that holds query row `row`: the last that begins at or before
// it, by a warp that looks at 32 at a time.
__device__ __forceinline__ bool find_token(const AttnArgs& a, int row, Place& p) {
  const int lane = threadIdx.x & 31;
  int lo = 0, among = a.B;
  while (among > 1) {
    const int step = (among + 31) / 32;
    const bool in = lane * step < among && cu_at(a.cu_q, lo + lane * step, a.Tq) <= row;
    const int last = 31 - __clz(__ballot_sync(0xFFFFFFFFu, in) | 1u);
    lo += last * step;
    among = min(step, among - last * step);
  }
  p.q0 = cu_at(a.cu_q, lo, a.Tq);
  p.nq = cu_at(a.cu_q, lo + 1, a.Tq) - p.q0;
  p.k0 = cu_at(a.cu_k, lo, a.Tk);
  p.nk = max(cu_at(a.cu_k, lo + 1, a.Tk) - p.k0, 0);
  return row >= p.q0 && row < p.q0 + p.nq;
}

template <int D, int NQ, bool FEW>
struct AttnShape {
  static constexpr int kChunks = D / 64;                        // 64-column boxes of a row
  static constexpr uint32_t kBox = kTile * 128;                 // 16 KB: 128 rows of 64 columns
  static constexpr uint32_t kQBox = FEW ? kFewRows * 128 : kBox;
  static constexpr uint32_t kQBytes = NQ * kChunks * kQBox;
  static constexpr uint32_t kSlot = kChunks * kBox;             // one k or v tile
  static constexpr int kSlots = FEW ? (D == 128 ? 3 : 6) : NQ == 1 ? (D == 128 ? 2 : 4) : (D == 128 ? 5 : 8);
  static constexpr uint32_t kSmem = kQBytes + kSlots * kSlot + 1024;
  static constexpr uint32_t kTmemCols = NQ == 1 ? 256 : 512;
  static constexpr int kSoftmaxWarps = FEW ? 1 : 4;             // per query tile
  static constexpr int kThreads = (NQ * kSoftmaxWarps + 2) * 32;
  // FEW: an MMA reads 128 rows of q all the same, those behind the box out of the ring
  static_assert((kChunks - 1) * kQBox + kBox <= kQBytes + kSlots * kSlot, "");
  static __device__ constexpr uint32_t s_col(int t) { return t * kTile; }
  static __device__ constexpr uint32_t o_col(int t) { return NQ * kTile + t * D; }
};

template <int NQ, int SLOTS>
struct AttnBars {
  uint64_t q_full;
  uint64_t full[SLOTS];
  uint64_t empty[SLOTS];
  uint64_t tail;           // the tile whose rows behind the sequence are zeroed
  uint64_t s_full[NQ];     // scores of the next tile are in tensor memory
  uint64_t p_half[NQ];     // the first 64 keys' weights are in tensor memory (and O is rescaled)
  uint64_t p_full[NQ];     // the other 64 keys' too
  uint64_t o_full[NQ];     // the last O += P V is done
  uint64_t drain;
  Place place;
  int found;
  uint32_t tmem_base;
  int abort_flag;
};

// MMA issue by a whole warp, `elected` in one lane: the operands' addresses
// stay in uniform registers, which code under a lane's branch cannot use (a
// measured 75 cycles an instruction there, against the 64 it runs).  The
// descriptors' upper halves are constants.
__device__ __forceinline__ uint64_t desc64(uint32_t lo, uint32_t hi) {
  return static_cast<uint64_t>(hi) << 32 | lo;
}
template <bool ACC>
__device__ __forceinline__ void mma_ss(uint32_t elected, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "n"(ACC ? 1 : 0), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t elected, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t elected, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(elected)
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The largest of three, NaN if one is.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The weights 2^(c s + shift) of 32 scores, in place and as 16 pairs of 16 bits.
// (A polynomial on the FMA pipe for an eighth or a quarter of them, to relieve
// the exponential unit, measured slower: 5.29 and 5.42 against 5.15 ms at
// 32760 keys x 10 heads, where the power cap binds.)
template <class T>
__device__ __forceinline__ void weigh32(uint32_t (&s)[32], uint64_t cc, uint64_t ss, uint32_t (&p)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 x = unpack2(fma2(pack2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), cc, ss));
    const float w0 = ex2(x.x), w1 = ex2(x.y);
    s[2 * i] = __float_as_uint(w0);
    s[2 * i + 1] = __float_as_uint(w1);
    p[i] = T::from_f32x2(w0, w1);
  }
}

template <class T, int D, int NQ, bool SPLIT, bool FEW>
__global__ void __launch_bounds__(AttnShape<D, NQ, FEW>::kThreads, NQ == 1 ? 2 : 1)
    attention_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const AttnArgs a) {
  using Shape = AttnShape<D, NQ, FEW>;
  constexpr int kSlots = Shape::kSlots;
  constexpr bool kBf16 = std::is_same<T, Bf16>::value;
  extern __shared__ uint8_t smem_dyn[];
  __shared__ AttnBars<NQ, kSlots> bars;
  uint8_t* smem = align1024_shared(smem_dyn);
  uint8_t* ring = smem + Shape::kQBytes;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  constexpr int kMmaWarp = NQ * Shape::kSoftmaxWarps;
  constexpr int kLoadWarp = kMmaWarp + 1;

  // q, k, v and the lengths may be the previous kernel's output (launched
  // with programmatic stream serialization)
  if (warp == kLoadWarp) {
    if (lane == 0) {
      mbar_init(&bars.q_full, 1);
      for (int s = 0; s < kSlots; ++s) {
        mbar_init(&bars.full[s], 1);
        mbar_init(&bars.empty[s], 1);
      }
      mbar_init(&bars.tail, 1);
      for (int t = 0; t < NQ; ++t) {
        mbar_init(&bars.s_full[t], 1);
        mbar_init(&bars.p_half[t], Shape::kSoftmaxWarps);
        mbar_init(&bars.p_full[t], Shape::kSoftmaxWarps);
        mbar_init(&bars.o_full[t], 1);
      }
      mbar_init(&bars.drain, 1);
      bars.abort_flag = 0;
      fence_mbar_init();
      fence_async_shared();
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    tmem_alloc(&bars.tmem_base, Shape::kTmemCols);
    tmem_relinquish();
  }
  griddep_wait();
  // Long causal tiles first: the block order runs backwards.  FEW and SPLIT:
  // the host knows an upper bound of the places only, far above their number
  // when it is not one sequence that has all queries and keys; so a block walks
  // over places, the grid's size apart (64 tokens over 64 caches of 2000:
  // 22 us, a block for each possible place 40).  The barriers go on from place to place.
  int index = static_cast<int>(blockIdx.x);
  if (!SPLIT && a.causal) index = static_cast<int>(gridDim.x) - 1 - index;
  uint32_t tiles_done = 0, places_done = 0;          // key tiles, places with keys
  uint32_t loads = 0, tails = 0;                     // producer: ring loads, cut tiles
  int slot = 0;                                      // MMA: of the k tile last used
  uint32_t phase = 0;
  while (true) {
    if (warp == 0) {
      Place p{};
      const bool found = a.B <= 32 ? find_place<1>(a, index, NQ * a.tokens, SPLIT ? a.chunk : 0, p)
                                   : find_place<4>(a, index, NQ * a.tokens, SPLIT ? a.chunk : 0, p);
      if (lane == 0) {
        bars.place = p;
        bars.found = found;
      }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_launch_dependents();
    if (!bars.found) break;
    const uint32_t tmem_base = bars.tmem_base;
    const Place pl = bars.place;
    volatile int* abort_flag = &bars.abort_flag;
    // key head, its first query head, and the tokens of the block
    const int kh = static_cast<int>(blockIdx.y) / a.groups;
    const int h0 = static_cast<int>(blockIdx.y) * a.G;
    const int tok0 = pl.tile * NQ * a.tokens;
    // key tiles [j0, n_t) of query tile t: up to the last key its last token sees
    const int j0 = SPLIT ? pl.chunk * a.chunk : 0;
    int n[NQ], n_all = 0;
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
      const int first = tok0 + t * a.tokens;
      const int last = min(first + a.tokens, pl.nq) - 1;
      int seen = pl.nk;
      if (a.causal) seen = min(seen, last + pl.nk - pl.nq + 1);
      if (first >= pl.nq) seen = 0;
      int end = (max(seen, 0) + kTile - 1) / kTile;
      if (SPLIT) end = min(end, j0 + a.chunk);
      n[t] = max(end - j0, 0);
      n_all = max(n_all, n[t]);
    }

    if (warp == kLoadWarp) {
      // ---------------------------------------------------------------- producer
      if (n_all > 0) {
        if (lane == 0) {
          uint32_t boxes = 0;
          for (int t = 0; t < NQ; ++t) boxes += n[t] > 0 ? 1 : 0;
          const uint32_t rows = static_cast<uint32_t>(a.tokens * a.G);
          mbar_arrive_expect_tx(&bars.q_full, boxes * Shape::kChunks * rows * 128);
          for (int t = 0; t < NQ; ++t) {
            if (n[t] == 0) continue;
            for (int c = 0; c < Shape::kChunks; ++c)
              tma_load_3d(smem + (t * Shape::kChunks + c) * Shape::kQBox, &tmQ, &bars.q_full, 64 * c, h0,
                          pl.q0 + tok0 + t * a.tokens);
          }
        }
        bool tail_pending = false;
        for (int i = 0; i < 2 * n_all; ++i) {
          const int s = static_cast<int>(loads % kSlots);
          if (!warp_wait_converged(&bars.empty[s], ((loads / kSlots) & 1) ^ 1, abort_flag, a.status, a.wait_ns)) break;
          const int row = (j0 + i / 2) * kTile;                 // first key of the tile, within the sequence
          const bool is_v = (i & 1) != 0;
          // value rows behind the sequence that are rows of the tensor (the
          // copy itself zero-fills behind the tensor's end)
          const bool cut = is_v && row + kTile > pl.nk && pl.k0 + pl.nk < a.Tk;
          uint64_t* bar = cut ? &bars.tail : &bars.full[s];
          if (lane == 0) {
            mbar_arrive_expect_tx(bar, Shape::kSlot);
            for (int c = 0; c < Shape::kChunks; ++c)
              tma_load_3d(ring + s * Shape::kSlot + c * Shape::kBox, is_v ? &tmV : &tmK, bar, 64 * c, kh, pl.k0 + row);
          }
          __syncwarp();
          ++loads;
          if (cut) {   // at most once a place: the sequence's last tile
            // the wait ignores the abort flag: the copy always lands
            tail_pending = !warp_wait_converged(&bars.tail, tails++ & 1, nullptr, a.status, a.wait_ns);
            if (tail_pending) {
              *abort_flag = 1;
              break;
            }
            for (int c = 0; c < Shape::kChunks; ++c) {
              const uint32_t base = smem_u32(ring + s * Shape::kSlot + c * Shape::kBox);
              for (int e = (pl.nk - row) * 8 + lane; e < kTile * 8; e += 32) sts128(base + e * 16, make_uint4(0, 0, 0, 0));
            }
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.full[s]);
          }
        }
        // every issued copy lands before the CTA exits or goes on
        if (lane == 0) {
          bool landed = mbar_wait(&bars.q_full, places_done & 1, nullptr, nullptr, 100000000ull);
          if (tail_pending) landed &= mbar_wait(&bars.tail, (tails - 1) & 1, nullptr, nullptr, 100000000ull);
          for (uint32_t s = 0; s < kSlots && s < loads; ++s) {
            const uint32_t n_s = loads / kSlots + (s < loads % kSlots ? 1 : 0);
            if (tail_pending && s == (loads - 1) % kSlots) continue;
            landed &= mbar_wait(&bars.full[s], (n_s - 1) & 1, nullptr, nullptr, 100000000ull);
          }
          if (!landed) *abort_flag = 1;
        }
        __syncwarp();
      }
    } else if (warp == kMmaWarp) {
      // ---------------------------------------------------------------- MMA issuer
      if (n_all > 0) {
        constexpr uint32_t idesc_s = idesc_f16(kTile, kTile, kBf16, false);
        constexpr uint32_t idesc_o = idesc_f16(kTile, D, kBf16, true);
        const uint32_t el = lane == 0 ? 1u : 0u;
        const uint64_t qd = sw128_kmajor_desc(smem_u32(smem));
        const uint64_t kd = sw128_kmajor_desc(smem_u32(ring));
        const uint64_t vd = sw128_mnmajor_desc(smem_u32(ring), Shape::kBox);
        const uint32_t q_lo = static_cast<uint32_t>(qd), k_lo = static_cast<uint32_t>(kd), v_lo = static_cast<uint32_t>(vd);
        const uint32_t k_hi = static_cast<uint32_t>(kd >> 32), v_hi = static_cast<uint32_t>(vd >> 32);
        auto score = [&](int t, uint32_t kt) {         // kt: the k tile's descriptor, lower half
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint64_t qa = desc64(q_lo + (t * Shape::kChunks + k / 4) * (Shape::kQBox >> 4) + (k % 4) * 2, k_hi);
            const uint64_t ka = desc64(kt + (k / 4) * (Shape::kBox >> 4) + (k % 4) * 2, k_hi);
            if (k == 0) mma_ss<false>(el, tmem_base + Shape::s_col(t), qa, ka, idesc_s);
            else mma_ss<true>(el, tmem_base + Shape::s_col(t), qa, ka, idesc_s);
          }
          commit(el, &bars.s_full[t]);
        };
        bool ok = warp_wait_converged<true>(&bars.q_full, places_done & 1, abort_flag, a.status, a.wait_ns) &&
                  warp_wait_converged(&bars.full[slot], phase, abort_flag, a.status, a.wait_ns);
        if (ok) {
          tc_fence_after();
#pragma unroll
          for (int t = 0; t < NQ; ++t)
            if (n[t] > 0) score(t, k_lo + slot * (Shape::kSlot >> 4));
          commit(el, &bars.empty[slot]);
        }
        auto next = [&] {
          if (++slot == kSlots) slot = 0, phase ^= 1;
        };
        for (int j = 0; ok && j < n_all; ++j) {
          next();
          const int sv = slot;
          ok = warp_wait_converged(&bars.full[sv], phase, abort_flag, a.status, a.wait_ns);
          next();
          const int sk = slot;
          const uint32_t vt = v_lo + sv * (Shape::kSlot >> 4), kt = k_lo + sk * (Shape::kSlot >> 4);
          bool k_ready = false;
#pragma unroll
          for (int t = 0; t < NQ; ++t) {
            if (!ok || j >= n[t]) continue;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              ok = ok && warp_wait_converged(half == 0 ? &bars.p_half[t] : &bars.p_full[t], (tiles_done + j) & 1, abort_flag, a.status, a.wait_ns);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int k = half * (kTile / 32); k < (half + 1) * (kTile / 32); ++k)
                mma_ts(el, tmem_base + Shape::o_col(t), tmem_base + Shape::s_col(t) + k * 8,
                       desc64(vt + k * (16 * 128 >> 4), v_hi), idesc_o, k != 0 ? 1u : (j != 0 ? 1u : 0u));
            }
            if (!ok) continue;
            if (j + 1 == n[t]) commit(el, &bars.o_full[t]);
            if (j + 1 < n[t]) {
              if (!k_ready) {
                ok = warp_wait_converged(&bars.full[sk], phase, abort_flag, a.status, a.wait_ns);
                if (!ok) continue;
                tc_fence_after();
                k_ready = true;
              }
              score(t, kt);
            }
          }
          // the tiles' last readers free the slots
          if (ok) {
            commit(el, &bars.empty[sv]);
            if (j + 1 < n_all) commit(el, &bars.empty[sk]);
          }
        }
        commit(el, &bars.drain);
        if (lane == 0 && !mbar_wait(&bars.drain, places_done & 1, nullptr, nullptr, 100000000ull)) *abort_flag = 1;
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------------- softmax
      const int t = warp >> 2;                       // query tile
      const int r = (warp & 3) * 32 + lane;          // row of the tile = tensor-memory lane
      const uint32_t lanes = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      const uint32_t s_at = lanes + Shape::s_col(t), o_at = lanes + Shape::o_col(t);
      const int r_tok = r / a.G;
      const int tok = tok0 + t * a.tokens + r_tok;   // within the sequence
      const int head = h0 + r - r_tok * a.G;
      const bool valid = r_tok < a.tokens && tok < pl.nq;
      // keys this row sees, and the fewest any row of the tile sees, both counted from tile j0
      int seen = pl.nk, fewest = pl.nk;
      if (a.causal) {
        seen = min(seen, tok + pl.nk - pl.nq + 1);
        fewest = min(fewest, tok0 + t * a.tokens + pl.nk - pl.nq + 1);
      }
      seen -= j0 * kTile;
      fewest -= j0 * kTile;
      const int nt = n[t];
      float m = -INFINITY;                           // the score of weight 1, times scale_log2: the maximum in use less kUnit
      uint64_t l2[2] = {0, 0};                       // partial sums (four fp32)
      const float c = a.scale_log2;
      bool ok = true;
      for (int j = 0; j < nt; ++j) {
        ok = warp_wait_converged(&bars.s_full[t], (tiles_done + j) & 1, abort_flag, a.status, a.wait_ns);
        if (!ok) break;
        tc_fence_after();
        uint32_t sv[4][32];
#pragma unroll
        for (int g = 0; g < 4; ++g) tmem_ld_32x32b_x32(s_at + 32 * g, sv[g]);
        tmem_wait_ld();
        if (fewest < (j + 1) * kTile) {              // a tile that a mask cuts (the same for the warp)
          const int lim = seen - j * kTile;
#pragma unroll
          for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int i = 0; i < 32; ++i) sv[g][i] = 32 * g + i < lim ? sv[g][i] : 0xFF800000u;
        }
        float mx[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          mx[g] = __uint_as_float(sv[g][0]);
#pragma unroll
          for (int i = 1; i < 31; i += 2) mx[g] = max3(mx[g], __uint_as_float(sv[g][i]), __uint_as_float(sv[g][i + 1]));
        }
        const float top = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], __uint_as_float(sv[0][31]), __uint_as_float(sv[1][31])),
                               max3(__uint_as_float(sv[2][31]), __uint_as_float(sv[3][31]), -INFINITY)) * c;
        const bool behind = top - m > kBehind<T> + kUnit<T>;     // false for -inf - -inf
        if (j == 0) {
          if (behind) m = top - kUnit<T>;
        } else if (__any_sync(0xFFFFFFFFu, behind)) {
          const float f = behind ? ex2(m - (top - kUnit<T>)) : 1.f;
          if (behind) m = top - kUnit<T>;
          const uint64_t ff = pack2(f, f);
          const uint64_t zero = 0;
          l2[0] = fma2(l2[0], ff, zero);
          l2[1] = fma2(l2[1], ff, zero);
#pragma unroll 1
          for (int g = 0; g < D / 16; ++g) {
            uint32_t o[16];
            tmem_ld_32x32b_x16(o_at + 16 * g, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st_32x32b_x16(o_at + 16 * g, o);
          }
        }
        const float shift = m == -INFINITY ? 0.f : -m;
        const uint64_t cc = pack2(c, c), ss = pack2(shift, shift);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t p[16];
          weigh32<T>(sv[g], cc, ss, p);
          tmem_st_32x32b_x16(s_at + 16 * g, p);
          if (g & 1) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(g == 1 ? &bars.p_half[t] : &bars.p_full[t]);
          }
        }
        // the sum, off the path of the MMA
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          const uint32_t* e = &sv[i / 16][(2 * i) % 32];
          l2[0] = add2(l2[0], pack2(__uint_as_float(e[0]), __uint_as_float(e[1])));
          l2[1] = add2(l2[1], pack2(__uint_as_float(e[2]), __uint_as_float(e[3])));
        }
      }
      if (ok && nt > 0) {
        ok = warp_wait_converged(&bars.o_full[t], places_done & 1, abort_flag, a.status, a.wait_ns);
        tc_fence_after();
      }
      if (ok) {
        // ---- out = O / l, lse = m + log l (log2 units until the end)
        const float2 la = unpack2(add2(l2[0], l2[1]));
        const float l = la.x + la.y;
        const float inv = l == 0.f ? 0.f : 1.f / l;            // no key seen: 0 (l is NaN for NaN scores)
        const float lse2 = l == 0.f ? -INFINITY : m + lg2(l);
        const int64_t row = static_cast<int64_t>(pl.q0) + tok;
        const bool part = SPLIT && pl.nk > static_cast<int64_t>(a.chunk) * kTile;    // one of several chunks
        float* po = nullptr;
        uint16_t* out = nullptr;
        if (valid) {
          const int64_t at = row * a.Hq + head;
          if (part) {
            const int64_t pat = static_cast<int64_t>(pl.chunk) * a.Tq * a.Hq + at;
            a.part_lse[pat] = lse2;
            po = a.part_o + pat * D;
          } else {
            if (a.lse != nullptr) a.lse[at] = lse2 * kLn2;
            out = a.out + row * a.o_t + head * a.o_h;
          }
        }
#pragma unroll
        for (int g = 0; g < D / 32; ++g) {
          uint32_t o[32];
          if (nt > 0) {                              // the same for the warp
            tmem_ld_32x32b_x32(o_at + 32 * g, o);
            tmem_wait_ld();
          }
          if (valid) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(nt > 0 && l != 0.f ? __uint_as_float(o[i]) * inv : 0.f);
            if (part) {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<uint4*>(po + 32 * g + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            } else {
#pragma unroll
              for (int i = 0; i < 32; i += 8) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  w[e] = T::from_f32x2(__uint_as_float(o[i + 2 * e]), __uint_as_float(o[i + 2 * e + 1]));
                *reinterpret_cast<uint4*>(out + 32 * g + i) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
          __syncwarp();                              // the loads are collective
        }
      }
    }
    if (!FEW || !SPLIT) break;
    index += static_cast<int>(gridDim.x);
    if (index >= a.blocks) break;
    // copies have landed, MMAs are done and read: the next place may begin
    if (n_all > 0) ++places_done, tiles_done += n_all;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*abort_flag) break;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(bars.tmem_base, Shape::kTmemCols);
  }
}

// out = sum_c e^(lse_c - lse) O_c over the chunks of a row's keys, lse = log
// sum_c e^(lse_c).  WARPS (1 or 4) warps share a (token, head) row, every
// WARPS-th chunk each, and meet in shared memory in order.
template <class T, int D, int WARPS>
__global__ void __launch_bounds__(128) attention_join_kernel(const AttnArgs a) {
  constexpr int E = D / 32;
  __shared__ float met[4][D + 1];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (4 / WARPS) + warp / WARPS;
  const int64_t rows = static_cast<int64_t>(a.Tq) * a.Hq;
  if (w >= rows) return;                             // WARPS == 4: the whole block
  const int tok = static_cast<int>(w / a.Hq);
  const int head = static_cast<int>(w - static_cast<int64_t>(tok) * a.Hq);
  Place p{};
  if (!find_token(a, tok, p)) return;
  const int tiles = (p.nk + kTile - 1) / kTile;
  const int chunks = (tiles + a.chunk - 1) / a.chunk;
  if (chunks <= 1) return;                           // written already
  float top = -INFINITY;
  for (int c = lane; c < chunks; c += 32) top = fmaxf(top, a.part_lse[c * rows + w]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
  const float base = top == -INFINITY ? 0.f : top;
  float sum = 0.f, acc[E] = {};
#pragma unroll 4
  for (int c = warp % WARPS; c < chunks; c += WARPS) {
    const float z = a.part_lse[c * rows + w];
    if (z == -INFINITY) continue;                    // a chunk of which nothing is seen
    const float f = ex2(z - base);
    sum += f;
    const float* o = a.part_o + (c * rows + w) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(f, o[e], acc[e]);
  }
  if (WARPS > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) met[warp][lane * E + e] = acc[e];
    if (lane == 0) met[warp][D] = sum;
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int v = 1; v < WARPS; ++v) {
      sum += met[v][D];
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += met[v][lane * E + e];
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint32_t* out = reinterpret_cast<uint32_t*>(a.out + tok * a.o_t + head * a.o_h + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2) out[e / 2] = T::from_f32x2(acc[e] * inv, acc[e + 1] * inv);
  if (a.lse != nullptr && lane == 0) a.lse[w] = sum == 0.f ? -INFINITY : (base + lg2(sum)) * kLn2;
}

// ------------------------------------------------------------ host side
// How a call is cut into blocks.  A function of the sizes alone, so that the
// workspace size is one too (148 SMs: a B200).
struct Plan {
  int G, tokens, nq;
  bool few;             // tiles of kFewRows rows
  int chunk;            // key tiles per chunk, 0: not split
  int64_t blocks;       // upper bound of (query tile, chunk) pairs over the sequences
  int64_t chunks;       // upper bound of chunks of one sequence
};

Plan make_plan(int64_t Tq, int64_t Tk, int64_t B, int64_t Hq, int64_t Hk) {
  Plan p{};
  const int64_t share = Hq / Hk;
  // heads per tile: the largest divisor of the group that leaves at most 8 of
  // the tile's 128 rows empty
  p.G = 1;
  for (int d = 1; d <= kTile && d <= share; ++d)
    if (share % d == 0 && kTile / d * d >= 120) p.G = d;
  p.tokens = kTile / p.G;
  p.few = p.G <= kFewRows && Tq <= B * (kFewRows / p.G);
  if (p.few) p.tokens = kFewRows / p.G;
  const int64_t sets = Hq / p.G;
  // query tiles over the sequences at most: a sum of ceil(n / rows) over B
  // parts of Tq, each part with one row at least
  auto tiles_of = [&](int64_t rows) {
    const int64_t t = (Tq + B * (rows - 1)) / rows;
    return t < Tq ? t : Tq;
  };
  const int64_t two = tiles_of(2 * p.tokens) * sets;
  const int64_t one = tiles_of(p.tokens) * sets;
  p.nq = Tq <= B * p.tokens || two < 148 ? 1 : 2;
  p.blocks = tiles_of(p.nq * p.tokens);
  p.chunks = 1;
  const int64_t base = p.few ? B * sets : one;       // blocks of a call that is not split
  if (p.nq == 1 && (p.few || base < 296)) {
    const int64_t tiles = (Tk + kTile - 1) / kTile, each = (tiles + B - 1) / B;
    // Into how many chunks the keys of a sequence of `each` tiles go.
    // Microseconds: a tile while each block has an SM, and else; to begin and
    // end a block; for the join, and each chunk's part of it.  Few rows are
    // bound by the keys' bytes (1 token x 32 / 8 heads over 131072 keys: 32
    // tiles a chunk 88, 24 122, 8 107 us; 8 over 8192: 16 49, 8 53, 32 73; 4
    // over 1000: 1 11.0, 4 13.9); tiles of many rows share the keys through L2
    // (16384 queries x 1 head in two pieces 130 us, in one 210; 2048 x 8 heads
    // in chunks of four tiles 44, in one piece 29).
    const float alone = p.few ? 1.2f : 1.6f, beside = p.few ? 1.8f : 2.2f, ends = p.few ? 8.f : 5.f;
    // Tiles of 128 rows get a block for each place there can be, and where the
    // sequences are alike most of a batch's are none (64 x 39 queries x 8/1 heads
    // over 8192 keys in chunks of 16 tiles: 768 of 49920): 6 ns each.
    const float join = p.few ? 2.f : 4.f, piece = p.few ? 0.02f : Tq * Hq * 1.6e-4f, none = 0.006f;
    // Upper bound of the (query tile, chunk) pairs of the sequences
    auto places = [&](int64_t c) {
      const int64_t most = (Tq + p.tokens - 1) / p.tokens;      // query tiles of one sequence
      if (B == 1) return most * ((tiles + c - 1) / c);
      return std::min(most * (tiles / c + B), tiles_of(p.tokens) * (tiles / c + 1));
    };
    // The workspace holds a line (516 bytes at 128 columns) for each row and each
    // chunk of the longest sequence there can be, one with all the keys: at most
    // 128 MB (128 x 16 queries x 8/1 heads over 32768 keys would take 7.5 GB
    // beside 2.1 GB of keys and values)
    const int64_t lines = Tq * Hq * 516, room = (int64_t(1) << 27) / lines;
    const int64_t shortest = p.few ? 1 : room == 0 ? tiles : (tiles + room - 1) / room;
    int64_t chunk = 0;
    float least = 0.f;
    for (int64_t n = 1; n <= 256 && n <= (each > 1 ? each : 1); n += n < 8 ? 1 : n / 4) {
      int64_t c = (each + n - 1) / n, pieces = n;
      if (n > 1 && c < shortest) {
        if (B == 1 || shortest >= each) break;      // one sequence: fewer pieces were looked at
        c = shortest, pieces = (each + c - 1) / c;
      }
      const int64_t blocks = base * pieces;
      float cost = ((blocks + 295) / 296) * (c * (blocks <= 148 ? alone : beside) + ends) +
                   (n > 1 ? join + pieces * piece : 0.f);
      if (!p.few && n > 1) cost += std::max<int64_t>(places(c) * sets - blocks, 0) * none;
      if (n == 1 || cost < least) least = cost, chunk = n == 1 ? 0 : c;
    }
    if (p.few) {
      // Caches differ in length and the longest one ends last: where a join
      // costs little beside the rest, what is twice the average is cut too (a
      // cache of 32769 and 39 of 500, a query each, 8/8 heads: 70 us, whole 410;
      // 64 of 2001: 96 and 88).  The estimate is that of alike sequences: below
      // 30 us a long one stays whole (the same caches, 32/4 heads: 388 us), as it
      // does in batches of more rows (five queries each: 411 us)
      if (chunk == 0 && least > 30.f) chunk = 2 * each < 16 ? 16 : 2 * each;
      if (chunk != 0 && chunk * room < tiles) chunk = room == 0 ? tiles : (tiles + room - 1) / room;
    }
    if (chunk != 0 && chunk < tiles && (p.few || chunk * B < tiles)) {
      p.chunk = static_cast<int>(chunk);
      p.blocks = places(chunk);
      p.chunks = (tiles + chunk - 1) / chunk;
    }
  }
  return p;
}

int check_heads(const void* p, int64_t t, int64_t h, int64_t T, int64_t H, int64_t D) {
  const int64_t lim = int64_t(1) << 38;   // bytes of a stride stay below 2^40
  if (t > lim || h > lim) return W4A4_ERR_SHAPE;
  if ((T > 1 && t < D) || (H > 1 && h < D)) return W4A4_ERR_SHAPE;
  if (t % 8 != 0 || h % 8 != 0 || !aligned_to(p, 16)) return W4A4_ERR_ALIGN;
  return W4A4_OK;
}


// 3-D map over a [tokens, heads, D] tensor of 16-bit elements (strides in
// elements): box {64, box_heads, box_tokens}, 128-byte swizzle; rows out of
// range read as zero.
int heads_map(CUtensorMap* map, const void* base, bool bf16, int64_t T, int64_t H, int64_t D, int64_t t_stride,
              int64_t h_stride, int box_heads, int box_tokens) {
  return tensor_map_3d(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, base, D, H, T,
                       2 * (H > 1 ? h_stride : D), 2 * (T > 1 ? t_stride : H * D), 64, box_heads, box_tokens,
                       CU_TENSOR_MAP_SWIZZLE_128B);
}

template <class T, int D, int NQ, bool SPLIT, bool FEW>
cudaError_t launch_tc(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV, const AttnArgs& a,
                      int64_t blocks, int64_t sets, int64_t chunks, cudaStream_t stream) {
  using Shape = AttnShape<D, NQ, FEW>;
  auto kernel = attention_tc_kernel<T, D, NQ, SPLIT, FEW>;
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
  cudaLaunchConfig_t cfg = {};
  // FEW and SPLIT, see the kernel: as many places as there are if a sequence's
  // queries are one tile, two rounds of what the GPU holds at least
  int64_t most = blocks;
  if (FEW && SPLIT) most = std::max((592 + sets - 1) / sets, (static_cast<int64_t>(a.Tk) / kTile + 1) / a.chunk + a.B);
  cfg.gridDim = dim3(static_cast<unsigned>(blocks < most ? blocks : most), static_cast<unsigned>(sets), 1);
  cfg.blockDim = dim3(Shape::kThreads, 1, 1);
  cfg.dynamicSmemBytes = Shape::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, tmQ, tmK, tmV, a);
  if (e != cudaSuccess || !SPLIT) return e;
  const int64_t rows = static_cast<int64_t>(a.Tq) * a.Hq;
  cfg.blockDim = dim3(128, 1, 1);
  cfg.dynamicSmemBytes = 0;
  // Four warps a row when a sequence may have many chunks and the rows fit the
  // GPU at once: 128 chunks of one token 14.4 us with the attention, by a warp
  // 34.5; two chunks of 16384 tokens 155 us and 139
  if (chunks > 8 && rows <= 148 * 16) {
    cfg.gridDim = dim3(static_cast<unsigned>(rows), 1, 1);
    return cudaLaunchKernelEx(&cfg, attention_join_kernel<T, D, 4>, a);
  }
  cfg.gridDim = dim3(static_cast<unsigned>((rows + 3) / 4), 1, 1);
  return cudaLaunchKernelEx(&cfg, attention_join_kernel<T, D, 1>, a);
}

template <class T, int D>
cudaError_t launch_plan(const Plan& p, const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                        const AttnArgs& a, cudaStream_t stream) {
  const int64_t sets = a.Hq / p.G;
  auto launch = [&](auto split, auto few) {
    return launch_tc<T, D, 1, decltype(split)::value, decltype(few)::value>(tmQ, tmK, tmV, a, p.blocks, sets, p.chunks, stream);
  };
  using Yes = std::true_type;
  using No = std::false_type;
  if (p.few) return p.chunk != 0 ? launch(Yes{}, Yes{}) : launch(No{}, Yes{});
  if (p.nq == 1) return p.chunk != 0 ? launch(Yes{}, No{}) : launch(No{}, No{});
  return launch_tc<T, D, 2, false, false>(tmQ, tmK, tmV, a, p.blocks, sets, p.chunks, stream);
}

}  // namespace
}  // namespace w4a4

using namespace w4a4;

extern "C" {

// SPLIT: [chunks][Tq][Hq][D] fp32 partial outputs, [chunks][Tq][Hq] fp32 lse
size_t w4a4_attention_workspace_bytes(int64_t Tq, int64_t Tk, int64_t B, int64_t Hq, int64_t Hk, int64_t D) {
  if (Tq <= 0 || Tk < 0 || B < 1 || Hq < 1 || Hk < 1 || Hq % Hk != 0 || D < 1) return 0;
  if (Tq > (int64_t(1) << 30) || Tk > (int64_t(1) << 30) || B > kMaxSequences || Hq > 65535 || D > 128) return 0;
  const Plan p = make_plan(Tq, Tk, B, Hq, Hk);
  if (p.chunk == 0) return 0;
  return static_cast<size_t>(p.chunks) * static_cast<size_t>(Tq) * static_cast<size_t>(Hq) * (D + 1) * 4;
}

int w4a4_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k,
                   int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
                   int64_t v_head_stride, void* out, int64_t out_token_stride, int64_t out_head_stride, float* lse,
                   const int32_t* cu_q, const int32_t* cu_k, int64_t B, int64_t Tq, int64_t Tk, int64_t Hq,
                   int64_t Hk, int64_t D, int causal, float scale, int dtype, void* workspace,
                   size_t workspace_bytes, void* stream) {
  if (Tq < 0 || Tk < 0 || Tq > (int64_t(1) << 30) || Tk > (int64_t(1) << 30)) return W4A4_ERR_SHAPE;
  if (Tq != 0 && (q == nullptr || out == nullptr)) return W4A4_ERR_NULL;
  if (Tk != 0 && (k == nullptr || v == nullptr)) return W4A4_ERR_NULL;
  if (B < 1 || B > kMaxSequences) return W4A4_ERR_SHAPE;
  if ((cu_q == nullptr) != (cu_k == nullptr) || (cu_q == nullptr && B != 1)) return W4A4_ERR_NULL;
  if (D != 64 && D != 128) return W4A4_ERR_SHAPE;
  if (Hq < 1 || Hq > 65535 || Hk < 1 || Hq % Hk != 0) return W4A4_ERR_SHAPE;
  if (dtype != W4A4_BF16 && dtype != W4A4_FP16) return W4A4_ERR_ARG;
  if (!(scale > 0.f) || scale > 1.0e38f) return W4A4_ERR_ARG;
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
  const Plan p = make_plan(Tq, Tk, B, Hq, Hk);
  if (p.blocks > 0x7FFFFFFF) return W4A4_ERR_SHAPE;
  AttnArgs a{};
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.o_t = out_token_stride, a.o_h = out_head_stride;
  a.cu_q = cu_q, a.cu_k = cu_k;
  a.B = static_cast<int>(B), a.Tq = static_cast<int>(Tq), a.Tk = static_cast<int>(Tk), a.Hq = static_cast<int>(Hq);
  a.G = p.G;
  a.groups = static_cast<int>(Hq / Hk) / p.G;
  a.tokens = p.tokens;
  a.causal = causal != 0;
  a.scale_log2 = scale * kLog2e;
  a.chunk = p.chunk;
  a.blocks = static_cast<int>(p.blocks);
  a.part_o = static_cast<float*>(workspace);
  a.part_lse = a.part_o + (p.chunk != 0 ? p.chunks * Tq * Hq * D : 0);
  a.status = dev->status;
  a.wait_ns = wait_limit_ns();
  const bool bf16 = dtype == W4A4_BF16;
  CUtensorMap tmQ, tmK, tmV;
  if ((st = heads_map(&tmQ, q, bf16, Tq, Hq, D, q_token_stride, q_head_stride, p.G, p.tokens)) != W4A4_OK) return st;
  if (Tk == 0) {
    tmK = tmV = tmQ;     // never read: no key tile
  } else {
    if ((st = heads_map(&tmK, k, bf16, Tk, Hk, D, k_token_stride, k_head_stride, 1, kTile)) != W4A4_OK) return st;
    if ((st = heads_map(&tmV, v, bf16, Tk, Hk, D, v_token_stride, v_head_stride, 1, kTile)) != W4A4_OK) return st;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (bf16) e = D == 64 ? launch_plan<Bf16, 64>(p, tmQ, tmK, tmV, a, s) : launch_plan<Bf16, 128>(p, tmQ, tmK, tmV, a, s);
  else e = D == 64 ? launch_plan<Fp16, 64>(p, tmQ, tmK, tmV, a, s) : launch_plan<Fp16, 128>(p, tmQ, tmK, tmV, a, s);
  return e == cudaSuccess ? W4A4_OK : W4A4_ERR_CUDA;
}

}  // extern "C"
