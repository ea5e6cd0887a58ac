// Causal attention over packed prompts with grouped heads: the gradients.
//
//   P = e^(S - lse), S = Q K^T / sqrt(d);  D_i = sum dO_i o_i;  dP = dO V^T;  dS = P (dP - D);
//   dV = P^T dO,  dK = dS^T Q / sqrt(d), both summed over the query heads of the group;  dQ = dS K / sqrt(d).
//
// Three launches (fp16: four), deterministic, without atomics:
//   stats   (-lse, -D) of every row, one pass over o and dO (bound by memory); fp16: magnitudes of dO's and v's rows
//   tops    fp16: the largest magnitudes of each sequence and head
//   q       one item per 128-row query tile and query head: Q and dO stay, K and V stream past
//   kv      one item per 128-key tile and kv head: K and V stay, the group's Q and dO stream past
// S and dP are computed in both, seven products in place of five: the price of writing every gradient
// once, in a fixed order. (Adding dQ up with atomics would need 64 KB of fp32 traffic per tile and
// would change the result from run to run; grouped heads' dK and dV add up in TMEM.) Where few kv heads make few
// kv items, the group's heads are split into parts, whose fp32 sums a last kernel adds up in order.
//
// Both are one kernel. X1, X2 are the tiles that stay, Y1, Y2 the ones that stream (128 rows each,
// used as halves of 64 rows):
//            X1  X2   Y1  Y2    scores (rows = X)   acc1 +=     acc2 +=
//   kv       K   V    Q   dO    S^T, dP^T           P^T Y2      dS^T Y1
//   q        Q   dO   K   V     S,   dP                         dS Y1
// Per half: S = X1 Y1^T and dP = X2 Y2^T into one of two or three TMEM buffers; a warpgroup turns them into
// P and dS, rounded to the element type over the scores (two values a column); the accumulating
// products read them from TMEM. One half's products run while the other half's warpgroup computes.
//   warps 0-3 / 4-7  half 0 / 1: a thread owns one row of X and 64 columns
//   warp 8 TMA, warp 9 products (one thread), warp 10 items, warp 11 the streamed rows' statistics (kv)
// The streamed tiles go through a ring of halves (64 rows of Y1 and of Y2), each released by its own
// accumulating products: whole pairs left the loads half a step's time only.
//
// Statistics of streamed rows (kv) would be needed per column of S^T, by every thread for every column: read from
// shared memory, against the products' operands, they took 800 of 2000 cycles a half. They ride along in the
// products instead: one more step of 16 along the reduced axis, X = constants, Y = -lse sqrt(d) and -D as
// three parts each of 16-bit type, whose products with the constants add up to the fp32 value (24 bits
// and more). P = 2^(S' log2 e / sqrt(d)) and dS = P dP' then need no other input. (What the parts cannot hold, lse of a
// million and more in fp16, is added to their columns by the softmax warpgroups.)
//
// P and dS are rounded to the element type; sums, statistics and accumulators are fp32. In bf16 that is half a step of each, 2^-8
// at most. fp16's steps are absolute below 2^-14, where P (about 1 / keys) and dS = P (dP - D) of small gradients lie, and its
// range ends at 2^16. So fp16 holds P times 2^14 (P <= 1), and dS times a power of two from the bound
//   |dS_ij| <= |dP_ij| + |D_i| <= 2 d max|dO_i| max|v|   (the row's largest magnitude; that of v in the sequence and kv head)
// that brings the bound to 2^13 ... 2^14: one per row in the q kernel, one per sequence and part of a group (with the largest |dO_i| of
// its heads) in kv. Both are taken out again from the fp32 accumulators. dS of any fp16 input is then in range, and half a
// step is 2^-11 of each down to 2^-27 of its bound, an absolute 2^-38 of the bound below. The rows' magnitudes ride along in the
// statistics' pass; a small kernel finds the sequences'.
//
// D from the given o carries o's rounding, which dS = P (dP - D) shares along the whole row: against the
// rounding of dS itself that is about one part in sqrt(keys), so it shows only in a sequence's first
// rows. The q kernel takes D = sum P dP / sum P there instead: the first query tile has one key tile, so a
// row's sums are at hand (the two halves exchange theirs). sum P is 1 but for what lse's own rounding leaves: of scores of a
// million, whose lse has steps of 1/16, it may be 0.9, and D must follow. It leaves that D for the kv kernel.
// Error of dq at 2000 rows of d = 64 in fp16, relative to the result's own rounding: 1.55 before, 1.44 after.
//
// Bound by the tensor cores: a 128 x 128 pair of tiles costs 4 (kv) or 3 (q) products of 512 cycles at
// d = 128, next to 1024 cycles of exponentials.
//
// Streamed rows behind the sequence's end are cleared in shared memory before use, and their
// columns of P and dS set to zero: what they hold, NaN included, does not count.
#pragma once
#include "clear_seq_prompt.cuh"

namespace clear {

struct SeqBwdParams {
  SeqView out1, out2;    // kv: dv, dk; q: -, dq
  // kv with parts > 1: each item takes one part of the group's heads and writes fp32 sums [parts][kv_heads][n_tok][d].
  int parts;
  float *part1, *part2;
  float2* stats;         // [q_heads, n_tok]: (-lse, -D)
  // fp16: largest magnitudes: of each row of dO [q_heads, n_tok] and of v [kv_heads, n_tok], and of a whole sequence in each head, the
  // same, at the sequence's first token.
  float *mag_g, *mag_v, *top_g, *top_v;
  const int* seq_start;
  int n_seq, n_tok, q_heads, kv_heads, group;
  float scale, scale_log2;
};

// The power of two that brings 2 d a b, the bound of |dS| of rows with magnitudes a and b, to [2^13, 2^14). Zero, infinite and NaN
// bounds stay: such rows hold nothing that could be kept.
template <int D>
__device__ __forceinline__ int lift_of(float a, float b) {
  const float bound = (2.f * D) * a * b;
  return bound > 0.f && bound < INFINITY ? 13 - ilogbf(bound) : 0;
}
constexpr float kBwdLift = 14.f;  // fp16: P is held times 2^14
__device__ __forceinline__ float pow2(int e) { return __int_as_float((127 + e) << 23); }  // -126 <= e <= 127

struct SeqStatsParams {
  SeqView o, g, v;
  const float* lse;
  float2* stats;
  float *mag_g, *mag_v;
  const int* seq_start;
  int n_seq, n_tok, q_heads, group;
};

constexpr int kStatsThreads = 256;

// The larger magnitude of each half of two pairs of fp16 (NaN gives way).
__device__ __forceinline__ uint32_t max_abs(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a & 0x7fff7fffu), "r"(b & 0x7fff7fffu));
  return r;
}

// D / 8 lanes take one row of o and dO, in fp16 those of a group's first head also one of v.
template <typename E, int D>
__global__ void __launch_bounds__(kStatsThreads) clear_seq_bwd_stats_kernel(const __grid_constant__ SeqStatsParams p) {
  using T = typename E::type;
  constexpr int kLanes = D / 8;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x % kLanes;
  constexpr bool kMags = !std::is_same<E, Bf16>::value;
  const long long row = ((long long)blockIdx.x * kStatsThreads + threadIdx.x) / kLanes;  // token-major: heads are next to each other
  const long long t = row / p.q_heads;
  const int h = (int)(row - t * p.q_heads);
  // Rows behind the last sequence are left out. Where the offsets do not ascend, the last one need not be the largest: warps that
  // reach behind it look for the sequence that ends last.
  int end = __ldg(p.seq_start + p.n_seq);
  end = end >= 0 && end < p.n_tok ? end : p.n_tok;
  if (__any_sync(0xffffffffu, t >= end && t < p.n_tok)) {
    int top = end;
    for (int s = threadIdx.x & 31; s < p.n_seq; s += 32) {
      int first, len;
      seq_range(p.seq_start, p.n_tok, s, &first, &len);
      top = first + len > top ? first + len : top;
    }
    end = __reduce_max_sync(0xffffffffu, top);
  }
  const bool in = t < end;
  const int hk = kMags ? h / p.group : 0;
  const bool first = kMags && h == hk * p.group;
  float sum = 0.f;
  uint32_t mag = 0;  // largest magnitudes of dO (low) and v
  if (in) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.o.ptr) + h * p.o.sh + t * p.o.st) + lane);
    const uint4 b = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.g.ptr) + h * p.g.sh + t * p.g.st) + lane);
    uint4 c = make_uint4(0, 0, 0, 0);
    if (first) c = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.v.ptr) + hk * p.v.sh + t * p.v.st) + lane);
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
    #pragma unroll
    for (int e = 0; e < 4; ++e) sum = fmaf(E::hi(x[e]), E::hi(y[e]), fmaf(E::lo(x[e]), E::lo(y[e]), sum));
    if (kMags) {
      const uint32_t g = max_abs(max_abs(b.x, b.y), max_abs(b.z, b.w)), v = max_abs(max_abs(c.x, c.y), max_abs(c.z, c.w));
      mag = max_abs(__byte_perm(g, v, 0x5410), __byte_perm(g, v, 0x7632));
    }
  }
  #pragma unroll
  for (int d = kLanes / 2; d > 0; d >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (kMags) mag = max_abs(mag, __shfl_xor_sync(0xffffffffu, mag, d));
  }
  if (in && lane == 0) {
    const float l = __ldg(p.lse + (long long)h * p.n_tok + t);
    // A row without a finite score (lse -inf) has P = 0: 2^(-inf) instead of 2^(-inf + inf).
    p.stats[(long long)h * p.n_tok + t] = make_float2(l == -INFINITY ? -INFINITY : -l, -sum);
    if (kMags) p.mag_g[(long long)h * p.n_tok + t] = Fp16::lo(mag);
    if (first) p.mag_v[(long long)hk * p.n_tok + t] = Fp16::hi(mag);
  }
}

// The largest magnitudes of each sequence's rows in head blockIdx.y of dO, and of v with the first head of its group: a block takes
// every gridDim.x-th sequence, up to 128 rows by one warp, more by all. Whether a NaN takes part does not matter. It and the q
// kernel behind it are programmatic dependents: their launches hide behind the kernel before.
constexpr int kTopsThreads = 512, kTopsWarps = kTopsThreads / 32;
constexpr int kTopsAlone = 128;
__global__ void __launch_bounds__(kTopsThreads) clear_seq_bwd_tops_kernel(const __grid_constant__ SeqBwdParams p) {
  __shared__ float2 best[kTopsWarps];
  const int h = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hk = h / p.group;
  const bool with_v = h == hk * p.group;
  const float* const mag_g = p.mag_g + (long long)h * p.n_tok;
  const float* const mag_v = p.mag_v + (long long)hk * p.n_tok;
  float* const top_g = p.top_g + (long long)h * p.n_tok;
  float* const top_v = p.top_v + (long long)hk * p.n_tok;
  asm volatile("griddepcontrol.wait;\ngriddepcontrol.launch_dependents;" ::: "memory");
  // Over the rows from, from + step, ...: the largest in the warp.
  const auto largest = [&](int first, int len, int from, int step) {
    float g = 0.f, v = 0.f;
    #pragma unroll 4
    for (int i = from; i < len; i += step) {
      g = fmaxf(g, mag_g[first + i]);
      if (with_v) v = fmaxf(v, mag_v[first + i]);
    }
    #pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, d));
      v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    }
    return make_float2(g, v);
  };
  const auto store = [&](int first, float2 x) {
    top_g[first] = x.x;
    if (with_v) top_v[first] = x.y;
  };
  for (long long s0 = blockIdx.x; s0 < p.n_seq; s0 += (long long)kTopsWarps * gridDim.x) {
    int first, len;
    const long long mine = s0 + (long long)warp * gridDim.x;
    if (mine < p.n_seq) {
      seq_range(p.seq_start, p.n_tok, (int)mine, &first, &len);
      if (len > 0 && len <= kTopsAlone) {
        const float2 x = largest(first, len, lane, 32);
        if (lane == 0) store(first, x);
      }
    }
    for (long long s = s0; s < p.n_seq && s < s0 + (long long)kTopsWarps * gridDim.x; s += gridDim.x) {
      seq_range(p.seq_start, p.n_tok, (int)s, &first, &len);
      if (len <= kTopsAlone) continue;
      const float2 x = largest(first, len, tid, kTopsThreads);
      if (lane == 0) best[warp] = x;
      __syncthreads();
      if (warp == 0) {
        float2 y = best[lane % kTopsWarps];
        #pragma unroll
        for (int d = kTopsWarps / 2; d > 0; d >>= 1) {
          y.x = fmaxf(y.x, __shfl_xor_sync(0xffffffffu, y.x, d));
          y.y = fmaxf(y.y, __shfl_xor_sync(0xffffffffu, y.y, d));
        }
        if (lane == 0) store(first, y);
      }
      __syncthreads();
    }
  }
}

template <int D, bool kKv>
struct PromptBwdLayout {
  // TMEM: half buffers of S (64 columns) and dP (64), then the accumulators. At d = 64 the products are short and a third
  // buffer has the next half's scores there before its warpgroup has finished the last one's (dQ 45 to 39 us on 4096
  // packed tokens of 16 heads); at d = 128 kv has no room for one, and q ran no faster with it.
  static constexpr int kBufs = D == 128 ? 2 : 3;
  static constexpr int kAcc1 = kBufs * 128, kAcc2 = kAcc1 + (kKv ? D : 0);
  static_assert(kAcc2 + D <= 512, "tensor memory");
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kBlock = 128 * 128;                // X: 128 rows x 64 elements
  static constexpr int kHalfTile = 64 * D * 2;
  static constexpr int kYBlock = 64 * 128;                // Y: 64 rows x 64 elements
  static constexpr int kStages = D == 128 ? 4 : 8;        // halves of (Y1, Y2)
  static constexpr int kStageBytes = 2 * kHalfTile;
  // Statistics as operands, in 8-row x 16-byte blocks without swizzle: per stage 64 rows of 8 values; then 128 rows
  // of constants for S, 128 for dP and 128 rows of zeros (the second half of each 16-step).
  static constexpr int kAug = 0;
  static constexpr int kOnes = kAug + kStages * 1024;
  static constexpr int kZeros = kOnes + 4096;
  static constexpr int kX = kOnes + 6144;
  static constexpr int kY = kX + 2 * kTileBytes;
  static constexpr int kBars = kY + kStages * kStageBytes;
  static_assert(kX % 1024 == 0 && kBars % 16 == 0, "alignment");
  static constexpr int bXFull = 0, bXEmpty = 1;
  static constexpr int bYFull = 2, bYEmpty = bYFull + kStages;
  static constexpr int bS = bYEmpty + kStages;            // + buffer: S and dP written
  static constexpr int bP = bS + kBufs;                   // + buffer: P and dS written
  static constexpr int bAcc = bP + kBufs;                     // the item's last accumulating product done
  static constexpr int bAccFree = bAcc + 1;               // the accumulators have been read
  static constexpr int bItemFull = bAccFree + 1, bItemEmpty = bItemFull + kPrItems;
  static constexpr int bDrain = bItemEmpty + kPrItems;
  static constexpr int bD = bDrain + 1;                   // both halves' sums of a first tile (q: in the statistics' place)
  static constexpr int kNumBars = bD + 1;
  static constexpr int kItems = (kBars + kNumBars * 8 + 15) & ~15;
  static constexpr int kMisc = kItems + kPrItems * 16;
  static constexpr int kInfo = kMisc + 16;                 // int[kStages]; fp16: see below
  static constexpr int kAlloc = kInfo + kStages * 4 + 1024;
  static_assert(kAlloc <= 232448, "shared memory");
};

// A matrix descriptor without swizzle: 8-row x 16-byte blocks, k_step bytes apart along the reduced axis and 128 along the rows.
__device__ __forceinline__ uint64_t smem_desc_plain(uint32_t saddr, uint32_t k_step) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((k_step >> 4) & 0x3FFFu) << 16) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1u << 46);
}

// Statistics that do not fit their three parts in fp16: such a row's are added to its column by the threads that use it. -inf, the
// statistics of a row without a finite score, does: P is 0.
constexpr float kFarLimit = 8e6f;
__device__ __forceinline__ bool is_far(float x, float d) { return (fabsf(x) > kFarLimit && x != -INFINITY) || fabsf(d) > kFarLimit; }

// v as three 16-bit parts: v = c0 a + c1 b + c2 c with the constants below. bf16 has fp32's range: the constants
// are 1, each part takes 8 bits. fp16 takes 11 bits each; its constants (2^7, 2^-3, 2^-13) reach from 8e6 down to steps of
// 2^-37. -inf is cut to the limit.
template <typename E>
__device__ __forceinline__ void split3(float v, uint32_t* ab, uint32_t* c) {
  constexpr bool kB = std::is_same<E, Bf16>::value;
  constexpr float kLimit = kB ? 3e38f : kFarLimit;
  constexpr float c0 = kB ? 1.f : 128.f, c1 = kB ? 1.f : 0.125f, c2 = kB ? 1.f : 1.f / 8192.f;
  v = v > kLimit ? kLimit : v < -kLimit ? -kLimit : v;
  const uint32_t w0 = E::pack(v / c0, 0.f);
  v = fmaf(-c0, E::lo(w0), v);
  const uint32_t w1 = E::pack(v / c1, 0.f);
  v = fmaf(-c1, E::lo(w1), v);
  *ab = (w0 & 0xffffu) | (w1 << 16);
  *c = E::pack(v / c2, 0.f) & 0xffffu;
}

// A streamed row's -lse as it is added to its column of S: times sqrt(d), and in fp16 with P's power of two.
template <typename E>
__device__ __forceinline__ float shift_of(float neg_lse, float root) {
  return std::is_same<E, Bf16>::value ? neg_lse * root : fmaf(neg_lse, root, kBwdLift * 0.69314718055994530942f * root);
}

// fp16: adds to a half's 64 columns of S and dP, in this warp's lanes, the statistics of the rows that are far, `left` of the rows
// being the sequence's. Whole warp; rare, and not inlined: it would cost the loop around it registers.
__device__ __noinline__ void add_far(uint32_t s_tm, const float2* stats, int left, float root) {
  #pragma unroll 1
  for (int c = 0; c < 64; c += 32) {
    uint32_t s[32], g[32];
    tmem_ld32(s_tm + c, s);
    tmem_ld32(s_tm + 64 + c, g);
    tmem_wait_ld(s);
    tmem_wait_ld(g);
    #pragma unroll
    for (int e = 0; e < 32; ++e) {
      const float2 w = c + e < left ? stats[c + e] : make_float2(0.f, 0.f);
      const float x = shift_of<Fp16>(w.x, root);
      if (is_far(x, w.y)) {
        s[e] = __float_as_uint(__uint_as_float(s[e]) + x);
        g[e] = __float_as_uint(__uint_as_float(g[e]) + w.y);
      }
    }
    tmem_st32(s_tm + c, s);
    tmem_st32(s_tm + 64 + c, g);
  }
  tmem_wait_st();
}

// An item as the ring carries it: {the sequence's first token, its length (0: end of the list), X tile, head}.
// fp16, kv: with a half's statistics comes a word, 2 * (the power of two in dS) + (whether a row is far).
template <typename E, int D, bool kKv>
__global__ void __launch_bounds__(kPrThreads, 1)
clear_seq_prompt_bwd_kernel(const __grid_constant__ CUtensorMap tm_x1, const __grid_constant__ CUtensorMap tm_x2,
                            const __grid_constant__ CUtensorMap tm_y1, const __grid_constant__ CUtensorMap tm_y2,
                            const __grid_constant__ SeqBwdParams p) {
  using L = PromptBwdLayout<D, kKv>;
  using T = typename E::type;
  constexpr bool kF16 = !std::is_same<E, Bf16>::value;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  int4* items = reinterpret_cast<int4*>(smem + L::kItems);
  int* info = reinterpret_cast<int*>(smem + L::kInfo);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&bars[L::bXFull], 1);
    mbar_init(&bars[L::bXEmpty], 1);
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&bars[L::bYFull + s], kKv ? 2 : 1);  // the copies, and the statistics' warp
      mbar_init(&bars[L::bYEmpty + s], 1);
    }
    for (int i = 0; i < L::kBufs; ++i) {
      mbar_init(&bars[L::bS + i], 1);
      mbar_init(&bars[L::bP + i], 4);
    }
    mbar_init(&bars[L::bAcc], 1);
    mbar_init(&bars[L::bAccFree], 8);
    mbar_init(&bars[L::bD], 256);
    for (int i = 0; i < kPrItems; ++i) {
      mbar_init(&bars[L::bItemFull + i], 1);
      mbar_init(&bars[L::bItemEmpty + i], 10 + (kKv ? 1 : 0));  // loader, issuer, eight softmax warps, statistics
    }
    mbar_init(&bars[L::bDrain], 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (kKv) {  // the constants that the statistics' parts are multiplied with: columns 0-2 for S, 3-5 for dP
    const int which = threadIdx.x >> 7, r = threadIdx.x & 127;
    constexpr bool kB = std::is_same<E, Bf16>::value;
    const uint32_t ab = E::pack(kB ? 1.f : 128.f, kB ? 1.f : 0.125f), c = E::pack(kB ? 1.f : 1.f / 8192.f, 0.f) & 0xffffu;
    const uint4 w = which == 0   ? make_uint4(ab, c, 0, 0)
                    : which == 1 ? make_uint4(0, ab << 16, (ab >> 16) | (c << 16), 0)
                                 : make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(smem + L::kOnes + which * 2048 + r * 16) = w;
    fence_proxy_async_smem();
  }
  if (kF16 && !kKv) asm volatile("griddepcontrol.wait;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  uint32_t n_item = 0;
  const auto next_item = [&](int4* it, int site) -> bool {
    const uint32_t s = n_item % kPrItems;
    if (!warp_wait(&bars[L::bItemFull + s], (n_item / kPrItems) & 1, abort_flag, kDevTimeoutOther, site, (int)n_item)) return false;
    *it = items[s];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[L::bItemEmpty + s]);
    ++n_item;
    return it->y > 0;
  };
  // Streamed tiles of an item: kv: for each head of the group the query tiles from the key tile on;
  // q: the key tiles up to the query tile.
  const auto n_tiles = [](const int4& it) { return (it.y + 127) >> 7; };
  // An item's head: q: the query head; kv: kv head * parts + part, with the group's heads [h_first, h_first + h_count).
  const auto h_first = [&](const int4& it) {
    const int hk = it.w / p.parts, part = it.w - hk * p.parts;
    return hk * p.group + part * p.group / p.parts;
  };
  const auto h_count = [&](const int4& it) {
    const int part = it.w % p.parts;
    return (part + 1) * p.group / p.parts - part * p.group / p.parts;
  };
  const float root = 1.f / p.scale;  // sqrt(d)
  const auto steps_of = [&](const int4& it) { return kKv ? h_count(it) * (n_tiles(it) - it.z) : it.z + 1; };

  if (warp == 8) {
    // ------------------------------------------------------------------ loader
    regs_dec<kPrRegsLow>();
    int4 it;
    uint32_t n = 0, slot = 0, x_loads = 0;
    bool ok = true;
    while (ok && next_item(&it, 50)) {
      if (lane == 0) {
        const int steps = steps_of(it), per = kKv ? n_tiles(it) - it.z : steps, head0 = kKv ? h_first(it) : it.w / p.group;
        ok = seq_wait(&bars[L::bXEmpty], (n & 1) ^ 1, abort_flag, kDevTimeoutTmaEmpty, 1, (int)n);
        if (ok) {
          mbar_arrive_expect_tx(&bars[L::bXFull], 2 * L::kTileBytes);
          const int head = kKv ? it.w / p.parts : it.w;
          load_seq_tile<D>(smem + L::kX, &tm_x1, &bars[L::bXFull], it.x + it.z * 128, head);
          load_seq_tile<D>(smem + L::kX + L::kTileBytes, &tm_x2, &bars[L::bXFull], it.x + it.z * 128, head);
          ++x_loads;
        }
        for (int i = 0; i < 2 * steps && ok; ++i) {  // halves
          const uint32_t s = slot % L::kStages;
          ok = seq_wait(&bars[L::bYEmpty + s], ((slot / L::kStages) & 1) ^ 1, abort_flag, kDevTimeoutTmaEmpty, 2, (int)n, i);
          if (!ok) break;
          const int tile = kKv ? it.z + (i >> 1) % per : i >> 1;
          const int head = kKv ? head0 + (i >> 1) / per : head0;
          const int tok = it.x + tile * 128 + (i & 1) * 64;
          uint8_t* dst = smem + L::kY + s * L::kStageBytes;
          mbar_arrive_expect_tx(&bars[L::bYFull + s], L::kStageBytes);
          #pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            tma_load_3d(dst + c * L::kYBlock, &tm_y1, &bars[L::bYFull + s], c * 64, tok, head);
            tma_load_3d(dst + L::kHalfTile + c * L::kYBlock, &tm_y2, &bars[L::bYFull + s], c * 64, tok, head);
          }
          ++slot;
        }
      }
      ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
      ++n;
    }
    if (lane == 0 && *abort_flag) {  // let the copies in flight land
      if (x_loads > 0) drain_wait(&bars[L::bXFull], (x_loads - 1) & 1);
      for (uint32_t s = slot > L::kStages ? slot - L::kStages : 0; s < slot; ++s)
        drain_wait(&bars[L::bYFull + s % L::kStages], (s / L::kStages) & 1);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------------ issuer
    regs_dec<kPrRegsLow>();
    constexpr uint32_t idesc_s = idesc_seq<E>(128, 64, 0, 0);
    constexpr uint32_t idesc_a = idesc_seq<E>(128, D, 0, 1);
    const uint64_t xdesc = smem_desc_sw128(smem_u32(smem + L::kX), 16, 1024);
    const uint64_t ykdesc = smem_desc_sw128(smem_u32(smem + L::kY), 16, 1024);         // as K-major B operand
    const uint64_t ymdesc = smem_desc_sw128(smem_u32(smem + L::kY), L::kYBlock, 1024);  // as MN-major B operand
    int4 it;
    uint32_t n = 0;                 // items
    uint32_t np = 0;                // bit b: the phase of buffer b's next P and dS
    uint32_t stage = 0, phase = 0;  // of the next pair in the ring
    bool ok = true;
    while (ok && next_item(&it, 51)) {
      if (elect_one()) {
        const int steps = steps_of(it);
        // S and dP of the streamed half in stage s, into buffer b
        const auto scores = [&](uint32_t b, uint32_t s) {
          const uint64_t yd = ykdesc + (uint64_t)((s * L::kStageBytes) >> 4);
          #pragma unroll
          for (int x = 0; x < 2; ++x) {
            #pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              umma_ss(tmem + b * 128 + x * 64, xdesc + ((x * L::kTileBytes + (kk >> 2) * L::kBlock + (kk & 3) * 32) >> 4),
                      yd + ((x * L::kHalfTile + (kk >> 2) * L::kYBlock + (kk & 3) * 32) >> 4), idesc_s, kk > 0);
            if (kKv) {
              const uint32_t aug = L::kAug + s * 1024, ones = L::kOnes + x * 2048;
              umma_ss(tmem + b * 128 + x * 64, smem_desc_plain(smem_u32(smem + ones), L::kZeros - ones),
                      smem_desc_plain(smem_u32(smem + aug), L::kZeros - aug), idesc_s, 1);
            }
          }
          umma_commit(&bars[L::bS + b]);
        };
        const auto accumulate = [&](uint32_t buf, uint32_t s, bool first) {
          ok = ok && seq_wait(&bars[L::bP + buf], (np >> buf) & 1, abort_flag, kDevTimeoutMma, 12, (int)n, (int)s);
          if (!ok) return;
          np ^= 1u << buf;
          tc_fence_after();
          const uint64_t yd = ymdesc + (uint64_t)((s * L::kStageBytes) >> 4);
          if (kKv) {
            #pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_ts(tmem + L::kAcc1, tmem + buf * 128 + kk * 8, yd + ((L::kHalfTile + kk * 2048) >> 4), idesc_a, (!first || kk > 0) ? 1u : 0u);
          }
          #pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_ts(tmem + L::kAcc2, tmem + buf * 128 + 64 + kk * 8, yd + ((kk * 2048) >> 4), idesc_a, (!first || kk > 0) ? 1u : 0u);
          umma_commit(&bars[L::bYEmpty + s]);
        };
        // The next half in the ring: waits for it and moves on.
        const auto next_half = [&](int i) {
          const uint32_t s = stage;
          ok = ok && seq_wait(&bars[L::bYFull + s], phase, abort_flag, kDevTimeoutMma, 11, (int)n, i);
          if (++stage == L::kStages) {
            stage = 0;
            phase ^= 1;
          }
          return s;
        };
        ok = seq_wait(&bars[L::bXFull], n & 1, abort_flag, kDevTimeoutMma, 10, (int)n);
        const int halves = 2 * steps;
        int ahead = 0;           // halves whose scores have been issued
        uint32_t st[L::kBufs];   // the stage of each buffer's half
        const auto issue_scores = [&](uint32_t b) {
          const uint32_t x = next_half(ahead);
          if (ok) scores(b, x);
          if (ok && ++ahead == halves) umma_commit(&bars[L::bXEmpty]);
          return x;
        };
        #pragma unroll
        for (int u = 0; u < L::kBufs; ++u) {
          st[u] = 0;
          if (u < halves && ok) st[u] = issue_scores(u);
        }
        // The accumulators are free once the previous item's have been written out.
        ok = ok && seq_wait(&bars[L::bAccFree], (n & 1) ^ 1, abort_flag, kDevTimeoutMma, 14, (int)n);
        for (int i = 0; i < halves && ok; i += L::kBufs) {
          #pragma unroll
          for (int u = 0; u < L::kBufs; ++u) {
            if (i + u < halves && ok) {
              accumulate(u, st[u], i + u == 0);
              if (ok && ahead < halves) st[u] = issue_scores(u);
            }
          }
        }
        if (ok) umma_commit(&bars[L::bAcc]);
      }
      __syncwarp();
      ok = __all_sync(0xffffffffu, ok);
      ++n;
    }
    if (__any_sync(0xffffffffu, *abort_flag)) {  // let the products in flight end
      if (elect_one()) {
        umma_commit(&bars[L::bDrain]);
        drain_wait(&bars[L::bDrain], 0);
      }
      __syncwarp();
    }
  } else if (warp == 10) {
    // ------------------------------------------------------------------ item finder
    regs_dec<kPrRegsLow>();
    TileList list;
    const int heads = kKv ? p.kv_heads * p.parts : p.q_heads;
    const long long total = list.init(p.seq_start, p.n_seq, p.n_tok, 128) * heads;
    if (kKv && blockIdx.x == 0) {
      for (int s = lane; s < p.n_seq; s += 32) {
        const int a = __ldg(p.seq_start + s), b = __ldg(p.seq_start + s + 1);
        if (a < 0 || b < a || b > p.n_tok) record_bad_index(kSiteSeqStart, s, a, b);
      }
    }
    uint32_t n = 0;
    for (int r = 0;; ++r) {
      const long long x = deal(r, blockIdx.x, gridDim.x);
      int4 it = make_int4(0, 0, 0, 0);
      const bool more = x < total;
      if (more) {
        int lv;  // steps: level + 1 query tiles (kv: those from the key tile on) or key tiles (q)
        const int s = list.find(x / heads, &lv);
        int first, len;
        seq_range(p.seq_start, p.n_tok, s, &first, &len);
        it = make_int4(first, len, kKv ? ((len + 127) >> 7) - 1 - lv : lv, (int)(x % heads));
      } else if ((long long)r * gridDim.x < total) {
        continue;
      }
      const uint32_t s = n % kPrItems;
      if (!warp_wait(&bars[L::bItemEmpty + s], ((n / kPrItems) & 1) ^ 1, abort_flag, kDevTimeoutOther, 3, (int)n)) break;
      if (lane == 0) {
        items[s] = it;
        mbar_arrive(&bars[L::bItemFull + s]);
      }
      __syncwarp();
      ++n;
      if (!more) break;
    }
  } else if (warp == 11) {
    // ------------------------------------------------------------------ statistics of streamed rows
    regs_dec<kPrRegsLow>();
    if constexpr (kKv) {
      int4 it;
      uint32_t slot = 0;
      bool ok = true;
      while (ok && next_item(&it, 52)) {
        const int steps = steps_of(it), per = n_tiles(it) - it.z, head0 = h_first(it);
        // The item's power of two: its loads are under way with those of the first half's statistics.
        int lift = 0;
        float top_g = 0.f, top_v = 0.f;
        if (kF16) {
          for (int h = lane; h < h_count(it); h += 32) top_g = fmaxf(top_g, p.top_g[(long long)(head0 + h) * p.n_tok + it.x]);
          top_v = p.top_v[(long long)(it.w / p.parts) * p.n_tok + it.x];
        }
        for (int i = 0; i < 2 * steps; ++i, ++slot) {
          const int t0 = (it.z + (i >> 1) % per) * 128 + (i & 1) * 64;
          const float2* src = p.stats + (long long)(head0 + (i >> 1) / per) * p.n_tok + it.x + t0;
          float2 v[2];
          #pragma unroll
          for (int e = 0; e < 2; ++e) v[e] = t0 + e * 32 + lane < it.y ? src[e * 32 + lane] : make_float2(0.f, 0.f);
          const uint32_t s = slot % L::kStages;
          ok = warp_wait(&bars[L::bYEmpty + s], ((slot / L::kStages) & 1) ^ 1, abort_flag, kDevTimeoutOther, 4, (int)slot);
          if (!ok) break;
          if (kF16 && i == 0) {
            #pragma unroll
            for (int d = 16; d > 0; d >>= 1) top_g = fmaxf(top_g, __shfl_xor_sync(0xffffffffu, top_g, d));
            lift = lift_of<D>(top_g, top_v);
          }
          bool any = false;
          #pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t l01, l2, d01, d2;
            float x = shift_of<E>(v[e].x, root), d = v[e].y;
            if (kF16 && is_far(x, d)) {
              any = true;
              x = d = 0.f;
            }
            split3<E>(x, &l01, &l2);
            split3<E>(d, &d01, &d2);
            *reinterpret_cast<uint4*>(smem + L::kAug + s * 1024 + (e * 32 + lane) * 16) =
                make_uint4(l01, l2 | (d01 << 16), (d01 >> 16) | (d2 << 16), 0);
          }
          if (kF16) {
            any = __any_sync(0xffffffffu, any);
            if (lane == 0) info[s] = 2 * lift + (int)any;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[L::bYFull + s]);
        }
      }
    }
  } else {
    // ------------------------------------------------------------------ P, dS and the epilogue
    regs_inc<kPrRegsHigh>();
    const int half = warp >> 2;
    const int row = threadIdx.x & 127;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint64_t sc2 = f32x2_pack(p.scale_log2, p.scale_log2);
    uint32_t n = 0, slot = 0, nd_phase = 0;
    // Bit b: the phase of buffer b's next scores; both halves' uses of it change it. Waiting by parity is sound: the buffer's last
    // use is three halves back (within an item) or before the accumulators' last product (earlier items), and this
    // warpgroup has seen something later than that: its own last half, or the item's end.
    uint32_t ns = 0;
    int4 it;
    while (next_item(&it, 53 + half)) {
      const int steps = steps_of(it), per = kKv ? n_tiles(it) - it.z : steps;
      const bool valid = it.z * 128 + row < it.y;
      const long long tok = (long long)it.x + it.z * 128 + row;
      float2 mine = make_float2(0.f, 0.f);
      int lift = 0;  // fp16: the power of two in dS
      if (!kKv && valid) {
        mine = p.stats[(long long)it.w * p.n_tok + tok];
        const float a = kF16 ? p.mag_g[(long long)it.w * p.n_tok + tok] : 0.f;
        const float b = kF16 ? p.top_v[(long long)(it.w / p.group) * p.n_tok + it.x] : 0.f;
        mine.x *= 1.4426950408889634f;
        if (kF16) lift = lift_of<D>(a, b);
      }
      for (int i = 0; i < steps; ++i, ++slot) {
        const uint32_t buf = (2 * i + half) % L::kBufs;
        const int yt = kKv ? it.z + i % per : i;
        const uint32_t st = (2 * slot + half) % L::kStages;
        const uint32_t phase = (ns >> buf) & 1;
        ns ^= 1u << buf;
        if constexpr (L::kBufs == 3) ns ^= 1u << ((2 * i + 1 - half) % 3);  // the other half's use
        if (!warp_wait(&bars[L::bS + buf], phase, abort_flag, kDevTimeoutSoftmax, 20 + half, (int)slot, i)) goto done;
        tc_fence_after();
        const uint32_t s_tm = tmem + lane_base + buf * 128, d_tm = s_tm + 64;
        // Columns kept: kv: query c >= key row on the diagonal, inside the sequence; q: key c <= query row.
        int lo = 0, hi = 128;
        if (kKv) {
          if (yt == it.z) lo = row;
          hi = it.y - yt * 128;
        } else if (yt == it.z) {
          hi = row + 1;
        }
        lo -= half * 64;
        hi -= half * 64;
        // Streamed rows of this half behind the sequence's end: clear them (a zero of P or dS times NaN is NaN).
        const int left = it.y - yt * 128;
        if (left < 128) {
          const int r = half * 64 + (row & 63);
          if (r >= left) {
            uint8_t* y = smem + L::kY + st * L::kStageBytes + (row >> 6) * L::kHalfTile + (row & 63) * 128;
            #pragma unroll
            for (int c = 0; c < D / 8; ++c) *reinterpret_cast<uint4*>(y + (c >> 3) * L::kYBlock + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        uint64_t more2 = 0;  // fp16, kv: from P's power of two to dS's
        if (kF16 && kKv) {
          const int word = info[st];
          lift = word >> 1;
          const float more = pow2(lift - (int)kBwdLift);
          more2 = f32x2_pack(more, more);
          if (word & 1) {
            const int t0 = yt * 128 + half * 64;
            add_far(s_tm, p.stats + (long long)(h_first(it) + i / per) * p.n_tok + it.x + t0, it.y - t0, root);
          }
        }
        const bool all = lo <= 0 && hi >= 64;
        const bool warp_all = __all_sync(0xffffffffu, all);
        if (!kKv && it.z == 0) {  // a sequence's first rows: D = sum P dP / sum P over the only key tile
          float sum = 0.f, all_p = 0.f;
          #pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t s[32], g[32];
            tmem_ld32(s_tm + c * 32, s);
            tmem_ld32(d_tm + c * 32, g);
            tmem_wait_ld(s);
            tmem_wait_ld(g);
            #pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c * 32 + e < hi) {
                const float pe = ex2_approx(fmaf(__uint_as_float(s[e]), p.scale_log2, mine.x));
                all_p += pe;
                sum = fmaf(pe, __uint_as_float(g[e]), sum);
              }
          }
          float2* sums = reinterpret_cast<float2*>(smem + L::kAug);
          sums[half * 128 + row] = make_float2(sum, all_p);
          mbar_arrive(&bars[L::bD]);
          if (!warp_wait(&bars[L::bD], nd_phase & 1, abort_flag, kDevTimeoutSoftmax, 26 + half, (int)nd_phase)) goto done;
          ++nd_phase;
          const float2 u = sums[row], w = sums[128 + row];
          all_p = u.y + w.y;
          mine.y = all_p == 0.f ? 0.f : -(u.x + w.x) / all_p;
          if (half == 0 && valid) p.stats[(long long)it.w * p.n_tok + tok].y = mine.y;
        }
        if (!kKv && kF16 && i == 0) mine.x += (float)lift;  // from here on P, which only dS needs, has its factor
        const auto tile = [&](auto cut) {
          #pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t s[32], g[32], wp[16], wd[16];
            tmem_ld32(s_tm + c * 32, s);
            tmem_ld32(d_tm + c * 32, g);
            tmem_wait_ld(s);
            tmem_wait_ld(g);
            #pragma unroll
            for (int e = 0; e < 16; ++e) {
              const uint64_t s2 = f32x2_pack(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
              const uint64_t g2 = f32x2_pack(__uint_as_float(g[2 * e]), __uint_as_float(g[2 * e + 1]));
              const uint64_t x = kKv ? f32x2_mul(s2, sc2) : f32x2_fma(s2, sc2, f32x2_pack(mine.x, mine.x));
              float p0 = ex2_approx(f32x2_lo(x)), p1 = ex2_approx(f32x2_hi(x));
              uint64_t pp = f32x2_pack(p0, p1);
              if (kF16 && kKv) pp = f32x2_mul(pp, more2);
              const uint64_t ds = f32x2_mul(pp, kKv ? g2 : f32x2_add(g2, f32x2_pack(mine.y, mine.y)));
              float d0 = f32x2_lo(ds), d1 = f32x2_hi(ds);
              if constexpr (decltype(cut)::value) {
                const int col = c * 32 + 2 * e;
                const bool k0 = col >= lo && col < hi, k1 = col + 1 >= lo && col + 1 < hi;
                p0 = k0 ? p0 : 0.f;
                d0 = k0 ? d0 : 0.f;
                p1 = k1 ? p1 : 0.f;
                d1 = k1 ? d1 : 0.f;
              }
              if (kKv) wp[e] = E::pack(p0, p1);
              wd[e] = E::pack(d0, d1);
            }
            if (kKv) tmem_st16(s_tm + c * 16, wp);
            tmem_st16(d_tm + c * 16, wd);
          }
        };
        if (warp_all) tile(std::false_type{});
        else tile(std::true_type{});
        tmem_wait_st();
        warp_arrive_tc(&bars[L::bP + buf]);
      }
      // ---- epilogue: kv: this half writes dv (0) or dk (1); q: its half of dq's columns
      if (!warp_wait(&bars[L::bAcc], n & 1, abort_flag, kDevTimeoutSoftmax, 24 + half, (int)n)) goto done;
      ++n;
      tc_fence_after();
      {
        constexpr int kCols = kKv ? D : D / 2;
        const bool one = kKv && half == 0;
        const SeqView& out = one ? p.out1 : p.out2;
        const int c0 = kKv ? 0 : half * (D / 2);
        const uint32_t acc = tmem + lane_base + (one ? L::kAcc1 : L::kAcc2) + c0;
        const float drop = !kF16 ? 1.f : pow2(-(one ? (int)kBwdLift : lift));
        const float f = one ? drop : p.scale * drop;
        const bool sums = kKv && p.parts > 1;
        const int hk = kKv ? it.w / p.parts : it.w;
        T* dst = static_cast<T*>(out.ptr) + hk * out.sh + tok * out.st + c0;
        float* part = sums ? (one ? p.part1 : p.part2) + (((long long)(it.w % p.parts) * p.kv_heads + hk) * p.n_tok + tok) * D : nullptr;
        #pragma unroll
        for (int c = 0; c < kCols / 32; ++c) {
          uint32_t ov[32];
          tmem_ld32(acc + c * 32, ov);
          tmem_wait_ld(ov);
          if (valid && sums) {
            if (kF16) {
              #pragma unroll
              for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * drop);
            }
            #pragma unroll
            for (int e = 0; e < 8; ++e)
              reinterpret_cast<uint4*>(part)[c * 8 + e] = make_uint4(ov[4 * e], ov[4 * e + 1], ov[4 * e + 2], ov[4 * e + 3]);
          } else if (valid) {
            #pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w[4];
              #pragma unroll
              for (int u = 0; u < 4; ++u)
                w[u] = E::pack(__uint_as_float(ov[8 * e + 2 * u]) * f, __uint_as_float(ov[8 * e + 2 * u + 1]) * f);
              reinterpret_cast<uint4*>(dst)[c * 4 + e] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
      }
      warp_arrive_tc(&bars[L::bAccFree]);
    }
  done:;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// Adds up the parts of dV and dK in their order: a thread takes 8 elements of one row of one of the two.
template <typename E, int D>
__global__ void __launch_bounds__(kStatsThreads) clear_seq_bwd_join_kernel(const __grid_constant__ SeqBwdParams p) {
  using T = typename E::type;
  constexpr int kLanes = D / 8;
  const long long rows = (long long)p.kv_heads * p.n_tok;
  const long long i = (long long)blockIdx.x * kStatsThreads + threadIdx.x;
  const int c = (int)(i % kLanes);
  const long long r = i / kLanes;
  const bool one = r < rows;
  const long long row = one ? r : r - rows;
  const int h = (int)(row / p.n_tok);
  const int t = r < 2 * rows ? (int)(row - (long long)h * p.n_tok) : -1;
  // Only rows that belong to a sequence have been summed. The search finds a row's sequence where the offsets ascend; the warp
  // looks through the whole list for a row (of its 32 / kLanes) that the search has not placed: padding, or offsets out of order.
  int lo = 0, n = p.n_seq;
  while (n > 1) {
    const int m = n / 2;
    if (__ldg(p.seq_start + lo + m) <= t) {
      lo += m;
      n -= m;
    } else {
      n = m;
    }
  }
  int first, len;
  seq_range(p.seq_start, p.n_tok, lo, &first, &len);
  bool in = t >= first && t < first + len;
  const int lane = threadIdx.x & 31;
  for (unsigned lost = __ballot_sync(0xffffffffu, !in && t >= 0 && c == 0); lost; lost &= lost - 1) {
    const int x = __shfl_sync(0xffffffffu, t, __ffs(lost) - 1);
    bool found = false;
    for (int s = lane; s < p.n_seq; s += 32) {
      seq_range(p.seq_start, p.n_tok, s, &first, &len);
      found = found || (x >= first && x < first + len);
    }
    if (__any_sync(0xffffffffu, found) && x == t) in = true;
  }
  if (!in) return;
  const float* src = (one ? p.part1 : p.part2) + (row * D + c * 8);
  float y[8] = {};
  for (int k = 0; k < p.parts; ++k) {
    const float4 a = *reinterpret_cast<const float4*>(src + k * rows * D), b = *reinterpret_cast<const float4*>(src + k * rows * D + 4);
    y[0] += a.x; y[1] += a.y; y[2] += a.z; y[3] += a.w;
    y[4] += b.x; y[5] += b.y; y[6] += b.z; y[7] += b.w;
  }
  const float f = one ? 1.f : p.scale;
  const SeqView& out = one ? p.out1 : p.out2;
  T* dst = static_cast<T*>(out.ptr) + h * out.sh + t * out.st;
  reinterpret_cast<uint4*>(dst)[c] =
      make_uint4(E::pack(y[0] * f, y[1] * f), E::pack(y[2] * f, y[3] * f), E::pack(y[4] * f, y[5] * f), E::pack(y[6] * f, y[7] * f));
}

}  // namespace clear
