// Causal attention over packed prompts with grouped heads: the forward pass.
//
// Row i of a sequence keeps the keys j <= i of its own sequence:
//   S = Q K^T / sqrt(d), P = e^(S - m), O = P V / sum P, lse = m + log sum P.
//
// Bound by the tensor cores and, next to them, by the exponentials: a 128 x 128 tile of S costs two products of 128 * 128 * d
// multiply-adds (512 cycles each at d = 128) and 16384 exponentials (1024 cycles of the special-function unit), so both
// are kept busy at once by two query tiles per block. Measured, neither is full (48 and 50 % at six prompts of 130 to 4608
// tokens, 32 and 8 heads: 256 us, 0.87 PFLOP/s; one of 16896, 24 and 8 heads: 1590 us, 1.10 PFLOP/s under the power cap): a step is
// the chain from S over the softmax and P V to the next S of the buffer.
//
// One block per SM walks a list of items, an item being 256 query rows (tiles A and B of 128) of one
// head of one sequence; each key/value tile of 128 is loaded once for both.
//   warps 0-3 / 4-7  softmax and epilogue of tile A / B; a thread owns one row (= one TMEM lane)
//   warp 8           TMA: Q tiles, then K and V tiles through one ring (K0 K1 V0 K2 V1 ...)
//   warp 9           one thread issues the products: S = Q K^T into TMEM, then O += P V with P from TMEM
//   warp 11          finds the block's items, ahead of the others, through a small ring
// TMEM: two buffers of S (three at d = 64) of 128 columns, then O of A and of B. P overwrites S, 16-bit, two values a
// column: the 32 keys of each 32 columns go into the first 16. The tiles of S take the buffers in turn, in the order A0, B0,
// A1, B1, ... (A0, A1, ... for an item without tile B); the next one's product is issued behind the P V that
// frees its buffer (clear_seq_order.h, with the waits that follow from it).
// While one tile's softmax runs, the other tile's products do: the issuer alternates A, B. (An issuer for each
// tile mixes the two tiles' products in the tensor pipe: 1782 us in place of 1416 at 16896 tokens and 24 heads.)
//
// Short batches (kSplit). With two query tiles an item, a few heads of a few thousand tokens are too few items for 148 SMs,
// and the last tiles' items bound the whole. There an item is one query tile: "tile A" takes its even key tiles and
// "tile B" the odd ones, and the two halves' (m, l, O) are joined at the end, O_A and O_B lying in the same lanes of TMEM.
// Every key tile then serves 128 rows instead of 256.
//
// Items are ordered by their number of key tiles, the longest first, over all sequences, and dealt to
// the blocks back and forth, so that every block gets about the same work. Heads of one group follow
// one another: they read the same keys and values, from L2.
//
// The running maximum is followed lazily: O and the sum are rescaled only when a row's maximum has
// grown by more than 2^8, which changes nothing but rounding. P is rounded to the element type for
// the second product (half a step of each probability; fp16 holds them times 2^7, see Fp16::kLift); sums are of the unrounded values.
//
// Value rows behind the sequence's end belong to the next sequence or to nothing. Their
// probabilities are zero, but 0 * NaN is not: the threads of the tile that uses them (the diagonal's)
// clear those rows in shared memory before they hand over P.
#pragma once
#include <type_traits>

#include "clear_common.cuh"
#include "clear_seq_common.cuh"
#include "clear_seq_order.h"

namespace clear {

constexpr int kPrThreads = 384;
constexpr uint32_t kPrRegsLow = 88, kPrRegsHigh = 208;
static_assert(2 * 128 * kPrRegsHigh + 128 * kPrRegsLow <= 384 * 168, "register split exceeds the launch allocation");
constexpr int kPrItems = 4;  // item ring
constexpr float kPrRescale = 8.0f;
constexpr int kPrParts = 2;  // P is handed to its product in halves of 64 keys

struct SeqPromptParams {
  SeqView o;
  float* lse;            // [q_heads, n_tok]
  const int* seq_start;  // [n_seq + 1]
  int n_seq, n_tok, q_heads, group;
  float scale_log2;      // log2(e) / sqrt(d)
};

// A sequence's tokens [first, first + len), cut to the packed tensors; a decreasing or outlying
// offset leaves it empty.
__device__ __forceinline__ void seq_range(const int* __restrict__ seq_start, int n_tok, int s, int* first, int* len) {
  const int a = __ldg(seq_start + s), b = __ldg(seq_start + s + 1);
  const bool ok = a >= 0 && b >= a && b <= n_tok;
  *first = ok ? a : 0;
  *len = ok ? b - a : 0;
}

// The list of items over all sequences, held by one warp (every lane calls every function). Tile y
// of the list, in descending order of its level (index among its sequence's tiles).
struct TileList {
  const int* seq_start;
  int n_seq, n_tok, rows;  // rows: query rows of a tile
  int level;               // the level of the last tile asked for
  int here;                // tiles of that level
  long long above;         // tiles of higher levels
  int s0, passed;          // sequences before s0 have `passed` tiles of that level, all before the last one asked for
  __device__ __forceinline__ int tiles_of(int s) const {
    int a, n;
    seq_range(seq_start, n_tok, s, &a, &n);
    return (n + rows - 1) / rows;
  }
  // Number of sequences with a tile of this level.
  __device__ __forceinline__ int at_level(int lv) const {
    int c = 0;
    for (int s = threadIdx.x & 31; s < n_seq; s += 32) c += tiles_of(s) > lv;
    return __reduce_add_sync(0xffffffffu, c);
  }
  // Sets up the list; returns its number of tiles.
  __device__ __forceinline__ long long init(const int* ss, int ns, int nt, int r) {
    seq_start = ss; n_seq = ns; n_tok = nt; rows = r;
    long long sum = 0;
    int top = 0;
    for (int s = threadIdx.x & 31; s < n_seq; s += 32) {
      const int n = tiles_of(s);
      sum += n;
      top = n > top ? n : top;
    }
    #pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    level = __reduce_max_sync(0xffffffffu, top) - 1;
    above = 0;
    here = at_level(level);
    s0 = passed = 0;
    return sum;
  }
  // Tile y (not before the last one asked for): its sequence and level. Each level's sequences are gone through once.
  __device__ __forceinline__ int find(long long y, int* lv) {
    while (y >= above + here && level > 0) {
      above += here;
      --level;
      here = at_level(level);
      s0 = passed = 0;
    }
    *lv = level;
    for (; s0 < n_seq; s0 += 32) {
      const int s = s0 + (threadIdx.x & 31);
      unsigned has = __ballot_sync(0xffffffffu, s < n_seq && tiles_of(s) > level);
      const int c = __popc(has);
      int rank = (int)(y - above) - passed;
      if (rank < c) {
        while (rank-- > 0) has &= has - 1;
        return s0 + __ffs(has) - 1;
      }
      passed += c;
    }
    return 0;
  }
};

// Item number of round r for a block: rounds run back and forth over the blocks.
__device__ __forceinline__ long long deal(int r, int block, int blocks) {
  return (long long)r * blocks + ((r & 1) ? blocks - 1 - block : block);
}

// Waits for this thread's loads from tensor memory; x is not used before it.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&x)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]), "+r"(x[6]), "+r"(x[7]), "+r"(x[8]),
                 "+r"(x[9]), "+r"(x[10]), "+r"(x[11]), "+r"(x[12]), "+r"(x[13]), "+r"(x[14]), "+r"(x[15]), "+r"(x[16]),
                 "+r"(x[17]), "+r"(x[18]), "+r"(x[19]), "+r"(x[20]), "+r"(x[21]), "+r"(x[22]), "+r"(x[23]), "+r"(x[24]),
                 "+r"(x[25]), "+r"(x[26]), "+r"(x[27]), "+r"(x[28]), "+r"(x[29]), "+r"(x[30]), "+r"(x[31])
               :
               : "memory");
}

template <int D>
struct PromptLayout {
  static constexpr int kBufs = D == 128 ? 2 : 3;
  static constexpr int kO = kBufs * 128;                 // O of tile A; tile B's follows
  static_assert(kO + 2 * D <= 512, "tensor memory");
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kBlock = 128 * 128;               // 128 rows x 64 elements, 128-byte swizzle
  static constexpr int kStages = D == 128 ? 5 : 8;       // ring of K and V tiles
  static constexpr int kQ = 0;
  static constexpr int kRing = kQ + 2 * kTileBytes;
  static constexpr int kBars = kRing + kStages * kTileBytes;
  static constexpr int bQFull = 0, bQEmpty = 1;
  static constexpr int bFull = 2, bEmpty = bFull + kStages;
  // A barrier for each buffer and query tile: a warpgroup sees only the phases that are its own, and so is never more than one
  // behind, which is what waiting by parity needs.
  static constexpr int bS = bEmpty + kStages;            // + 2 * buffer + tile: S written
  static constexpr int bP = bS + 2 * kBufs;              // + buffer * kPrParts + part: P's part written (and O rescaled)
  static constexpr int bO = bP + kBufs * kPrParts;       // + tile: a P V done
  static constexpr int bItemFull = bO + 2, bItemEmpty = bItemFull + kPrItems;
  static constexpr int bDrain = bItemEmpty + kPrItems;
  static constexpr int bJoin = bDrain + 1, bJoined = bDrain + 2;    // kSplit: (m, l) of both halves written; O of both read
  static constexpr int kNumBars = bDrain + 3;
  static constexpr int kItems = (kBars + kNumBars * 8 + 15) & ~15;  // int4[kPrItems]
  static constexpr int kMisc = kItems + kPrItems * 16;
  static constexpr int kAlloc = kMisc + 16 + 1024;
  static_assert(kAlloc <= 232448, "shared memory");
};

template <typename E>
__host__ __device__ constexpr uint32_t idesc_seq(int M, int N, int a_mn, int b_mn) {
  return std::is_same<E, Bf16>::value ? idesc_bf16_f32(M, N, a_mn, b_mn)
                                      : (idesc_bf16_f32(M, N, a_mn, b_mn) & ~((1u << 7) | (1u << 10)));  // fp16: format 0
}

// One 128-row tile of d columns: tokens from tok of head h.
template <int D>
__device__ __forceinline__ void load_seq_tile(uint8_t* dst, const CUtensorMap* m, uint64_t* bar, int tok, int h) {
  #pragma unroll
  for (int c = 0; c < D / 64; ++c) tma_load_3d(dst + c * kHalfBytes, m, bar, c * 64, tok, h);
}

// An item as the ring carries it: {first token of tile A, query rows left from there, tile A's number, head}.
template <typename E, int D, bool kSplit>
__global__ void __launch_bounds__(kPrThreads, 1)
clear_seq_prompt_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ SeqPromptParams p) {
  using L = PromptLayout<D>;
  using T = typename E::type;
  constexpr int kRows = kSplit ? 128 : 256;  // query rows of an item
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  int4* items = reinterpret_cast<int4*>(smem + L::kItems);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&bars[L::bQFull], 1);
    mbar_init(&bars[L::bQEmpty], 1);
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&bars[L::bFull + s], 1);
      mbar_init(&bars[L::bEmpty + s], 1);
    }
    for (int b = 0; b < L::kBufs; ++b) {
      mbar_init(&bars[L::bS + 2 * b], 1);
      mbar_init(&bars[L::bS + 2 * b + 1], 1);
      for (int i = 0; i < kPrParts; ++i) mbar_init(&bars[L::bP + b * kPrParts + i], 4);
    }
    mbar_init(&bars[L::bO], 1);
    mbar_init(&bars[L::bO + 1], 1);
    for (int i = 0; i < kPrItems; ++i) {
      mbar_init(&bars[L::bItemFull + i], 1);
      mbar_init(&bars[L::bItemEmpty + i], 10);  // the loader, the issuer, eight softmax warps
    }
    mbar_init(&bars[L::bDrain], 1);
    mbar_init(&bars[L::bJoin], 8);
    mbar_init(&bars[L::bJoined], 8);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const auto order_of = [](const int4& it) {
    const int tiles = it.z + 1;  // of tile A
    return kSplit ? PromptOrder<L::kBufs, kSplit>{(tiles + 1) / 2, tiles / 2}
                  : PromptOrder<L::kBufs, kSplit>{tiles, it.y > 128 ? tiles + 1 : 0};
  };

  // The next item; false at the end of the list (or on an expired wait). Whole warp.
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

  if (warp == 8) {
    // ------------------------------------------------------------------ loader
    regs_dec<kPrRegsLow>();
    int4 it;
    uint32_t n = 0, slot = 0, q_loads = 0;
    bool ok = true;
    while (ok && next_item(&it, 40)) {
      if (lane == 0) {
        const int hk = it.w / p.group;
        const bool two = !kSplit && it.y > 128;
        const int tiles = it.z + (two ? 2 : 1);  // key tiles of the item
        const int seq0 = it.x - it.z * 128;      // the sequence's first token
        ok = seq_wait(&bars[L::bQEmpty], (n & 1) ^ 1, abort_flag, kDevTimeoutTmaEmpty, 1, (int)n);
        if (ok) {
          mbar_arrive_expect_tx(&bars[L::bQFull], (two ? 2 : 1) * L::kTileBytes);
          load_seq_tile<D>(smem + L::kQ, &tm_q, &bars[L::bQFull], it.x, it.w);
          if (two) load_seq_tile<D>(smem + L::kQ + L::kTileBytes, &tm_q, &bars[L::bQFull], it.x + 128, it.w);
          ++q_loads;
        }
        const auto load = [&](const CUtensorMap* m, int tok) {
          const uint32_t s = slot % L::kStages;
          ok = ok && seq_wait(&bars[L::bEmpty + s], ((slot / L::kStages) & 1) ^ 1, abort_flag, kDevTimeoutTmaEmpty, 2, (int)n, tok);
          if (!ok) return;
          mbar_arrive_expect_tx(&bars[L::bFull + s], L::kTileBytes);
          load_seq_tile<D>(smem + L::kRing + s * L::kTileBytes, m, &bars[L::bFull + s], tok, hk);
          ++slot;
        };
        for (int j = 0; j <= tiles && ok; ++j) {
          if (j < tiles) load(&tm_k, seq0 + j * 128);
          if (j > 0) load(&tm_v, seq0 + (j - 1) * 128);
        }
      }
      ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
      ++n;
    }
    if (lane == 0 && *abort_flag) {  // let the copies in flight land
      if (q_loads > 0) drain_wait(&bars[L::bQFull], (q_loads - 1) & 1);
      for (uint32_t s = slot > L::kStages ? slot - L::kStages : 0; s < slot; ++s)
        drain_wait(&bars[L::bFull + s % L::kStages], (s / L::kStages) & 1);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------------ issuer
    regs_dec<kPrRegsLow>();
    constexpr uint32_t idesc_qk = idesc_seq<E>(128, 128, 0, 0);
    constexpr uint32_t idesc_pv = idesc_seq<E>(128, D, 0, 1);
    const uint64_t qdesc = smem_desc_sw128(smem_u32(smem + L::kQ), 16, 1024);
    const uint64_t kdesc = smem_desc_sw128(smem_u32(smem + L::kRing), 16, 1024);
    const uint64_t vdesc = smem_desc_sw128(smem_u32(smem + L::kRing), L::kBlock, 1024);
    int4 it;
    uint32_t n = 0;
    uint32_t uses = 0;           // bit b: whether buffer b has had an odd number of uses in earlier items
    uint32_t base = 0, wrap = 0; // stage and phase of the item's first tile in the ring
    bool ok = true;
    // A place in the ring.
    struct Place {
      uint32_t stage, phase;
      __device__ __forceinline__ void advance(uint32_t k) {
        stage += k;
        if (stage >= L::kStages) {
          stage -= L::kStages;
          phase ^= 1;
        }
      }
    };
    while (ok && next_item(&it, 41)) {
      const bool two = !kSplit && it.y > 128;
      const int nA = it.z + 1, nB = two ? it.z + 2 : 0;
      const int tiles = two ? nB : nA, total = nA + nB;
      const PromptOrder<L::kBufs, kSplit> order = order_of(it);
      if (elect_one()) {
        // The next tile of S to be computed (key tile jq of query tile hq), and of P to be used. Ring order:
        // K0, K1, V0, K2, V1, ..., V(tiles-1).
        int jq = 0, hq = 0, gq = 0, jp = 0, hp = 0;
        Place kp{base, wrap}, vp{base, wrap};
        vp.advance(tiles == 1 ? 1 : 2);
        const auto next = [&](int& j, int& h) {  // returns whether key tile j is done with
          if (kSplit) {
            ++j;
            h ^= 1;
            return true;
          }
          if (two && h == 0) {
            h = 1;
            return false;
          }
          ++j;
          h = two && j >= nA ? 1 : 0;
          return true;
        };
        const auto full = [&](const Place& x) {
          ok = ok && seq_wait(&bars[L::bFull + x.stage], x.phase, abort_flag, kDevTimeoutMma, 11, (int)n, (int)x.stage);
        };
        const auto qk = [&](int b) {
          full(kp);
          if (!ok) return;
          const uint64_t kd = kdesc + (uint64_t)((kp.stage * L::kTileBytes) >> 4);
          const uint64_t qd = qdesc + (uint64_t)((kSplit ? 0 : hq * L::kTileBytes) >> 4);
          #pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * L::kBlock + (kk & 3) * 32) >> 4;
            umma_ss(tmem + b * 128, qd + off, kd + off, idesc_qk, kk > 0);
          }
          umma_commit(&bars[L::bS + 2 * b + hq]);
          const uint32_t st = kp.stage;
          const int j = jq;
          if (next(jq, hq)) {
            umma_commit(&bars[L::bEmpty + st]);
            kp.advance(j == 0 ? 1 : 2);
          }
          if (++gq == total) umma_commit(&bars[L::bQEmpty]);
        };
        const auto pv = [&](int b, uint32_t phase) {
          full(vp);
          const uint64_t vd = vdesc + (uint64_t)((vp.stage * L::kTileBytes) >> 4);
          const uint32_t o_tm = tmem + L::kO + hp * D;
          #pragma unroll
          for (int i = 0; i < kPrParts; ++i) {
            ok = ok && seq_wait(&bars[L::bP + b * kPrParts + i], phase, abort_flag, kDevTimeoutMma, 13, (int)n, jp);
            if (!ok) return;
            tc_fence_after();
            #pragma unroll
            for (int kk = i * (8 / kPrParts); kk < (i + 1) * (8 / kPrParts); ++kk)
              umma_ts(o_tm, tmem + b * 128 + (kk >> 1) * 32 + (kk & 1) * 8, vd + (uint64_t)((kk * 2048) >> 4), idesc_pv,
                      (jp > (kSplit ? hp : 0) || kk > 0) ? 1u : 0u);
          }
          umma_commit(&bars[L::bO + hp]);
          const uint32_t st = vp.stage;
          if (next(jp, hp)) {
            umma_commit(&bars[L::bEmpty + st]);
            vp.advance(jp == tiles - 1 ? 1 : 2);
          }
        };
        ok = seq_wait(&bars[L::bQFull], n & 1, abort_flag, kDevTimeoutMma, 10, (int)n);
        const bool alone = order.alone();
        #pragma unroll
        for (int b = 0; b < L::kBufs; ++b)
          if (b < total && ok && order.first(b)) qk(b);
        // Both halves' O have been read before either is written anew.
        if (kSplit) ok = ok && seq_wait(&bars[L::bJoined], (n & 1) ^ 1, abort_flag, kDevTimeoutMma, 15, (int)n);
        uint32_t flip = 0;
        for (int g = 0; g < total && ok; g += L::kBufs) {
          #pragma unroll
          for (int b = 0; b < L::kBufs; ++b) {
            if (g + b < total && ok) {
              pv(b, ((uses >> b) & 1) ^ flip);
              if (ok && gq < total) qk(alone ? b ^ 1 : b);
            }
          }
          flip ^= 1;
        }
      }
      #pragma unroll
      for (int b = 0; b < L::kBufs; ++b) uses ^= (((total - b + L::kBufs - 1) / L::kBufs) & 1) << b;
      base += 2 * tiles;
      wrap ^= (base / L::kStages) & 1;
      base %= L::kStages;
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
    regs_dec<kPrRegsLow>();
  } else if (warp == 11) {
    // ------------------------------------------------------------------ item finder
    regs_dec<kPrRegsLow>();
    TileList list;
    const long long total = list.init(p.seq_start, p.n_seq, p.n_tok, kRows) * p.q_heads;
    if (blockIdx.x == 0) {  // offsets that decrease or reach outside leave their sequence out: say so
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
        int lv;
        const int s = list.find(x / p.q_heads, &lv);
        int first, len;
        seq_range(p.seq_start, p.n_tok, s, &first, &len);
        it = make_int4(first + lv * kRows, len - lv * kRows, lv * (kRows / 128), (int)(x % p.q_heads));
      } else if ((long long)r * gridDim.x < total) {
        continue;  // a round that is not full: none for this block
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
  } else {
    // ------------------------------------------------------------------ softmax + epilogue
    regs_inc<kPrRegsHigh>();
    const int half = warp >> 2;
    const int row = threadIdx.x & 127;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t o_tm = tmem + lane_base + L::kO + half * D;
    uint32_t joins = 0;
    uint32_t no = 0, tiles_before = 0;  // P V products of this query tile and key tiles of earlier items
    uint32_t ns = 0;                    // bit b: the phase of buffer b's next S for this query tile
    int4 it;
    while (next_item(&it, 42 + half)) {
      const uint32_t ring0 = 2 * tiles_before;  // the item's first place in the ring
      const bool two = !kSplit && it.y > 128;
      const int all_tiles = it.z + (two ? 2 : 1);
      tiles_before += all_tiles;
      const PromptOrder<L::kBufs, kSplit> order = order_of(it);
      if (!kSplit && half == 1 && !two) continue;  // no tile B
      const int row0 = kSplit ? 0 : half * 128;                                    // of the item's rows
      const int tiles = kSplit ? (all_tiles - half + 1) / 2 : it.z + 1 + half;     // key tiles that this half takes
      const bool valid = row0 + row < it.y;
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < tiles; ++i) {
        const int j = kSplit ? 2 * i + half : i;  // the key tile
        const int g = order.place(half, i);
        const uint32_t buf = g % L::kBufs;
        const uint32_t s_tm = tmem + lane_base + buf * 128;
        if (!warp_wait(&bars[L::bS + 2 * buf + half], (ns >> buf) & 1, abort_flag, kDevTimeoutSoftmax, 20 + half, g, j)) goto done;
        ns ^= 1u << buf;
        tc_fence_after();
        // The exponentials of the first 64 keys are taken with the maximum in use while the true maximum of all 128 is
        // still being found: the comparisons run in the special-function unit's shadow. Only where the
        // maximum has to move are they taken again.
        const bool diagonal = kSplit ? j == all_tiles - 1 : j == tiles - 1;  // key c is kept by row r iff c <= r
        uint32_t a0[32], a1[32], a2[32], a3[32], w0[16], w1[16];
        tmem_ld32(s_tm, a0);
        tmem_ld32(s_tm + 32, a1);
        tmem_ld32(s_tm + 64, a2);
        tmem_ld32(s_tm + 96, a3);
        tmem_wait_ld(a0);
        tmem_wait_ld(a1);
        tmem_wait_ld(a2);
        tmem_wait_ld(a3);
        const auto cut = [&](uint32_t (&x)[32], int c0) {
          if (diagonal) {
            #pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c0 + e > row) x[e] = 0xff800000u;
          }
        };
        cut(a0, 0);
        cut(a1, 32);
        cut(a2, 64);
        cut(a3, 96);
        const uint64_t sc2 = f32x2_pack(p.scale_log2, p.scale_log2);
        uint64_t sum[2] = {0, 0};
        const auto probabilities = [&](const uint32_t (&x)[32], float base, uint32_t (&w)[16]) {
          const uint64_t nb2 = f32x2_pack(-base, -base);
          #pragma unroll
          for (int e = 0; e < 16; ++e) {
            const uint64_t y = f32x2_fma(f32x2_pack(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), sc2, nb2);
            const float p0 = ex2_approx(f32x2_lo(y)), p1 = ex2_approx(f32x2_hi(y));
            sum[e & 1] = f32x2_add(sum[e & 1], f32x2_pack(p0, p1));
            w[e] = E::pack(p0, p1);
          }
        };
        float base = (m == -INFINITY ? 0.f : m) - E::kLift;
        probabilities(a0, base, w0);
        probabilities(a1, base, w1);
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        const auto largest = [&](const uint32_t (&x)[32]) {
          #pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float& y = mx[(e >> 1) & 3];
            y = fmax3(y, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
          }
        };
        largest(a0);
        largest(a1);
        largest(a2);
        largest(a3);
        const float top = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * p.scale_log2;
        const bool grow = top > m + kPrRescale || (m == -INFINITY && top > m);
        if (__any_sync(0xffffffffu, grow)) {
          // A row that does not ask for it keeps its maximum: its result has no part in its neighbours'.
          const float m_new = grow ? top : m;
          const float a = m == -INFINITY ? 0.f : ex2_approx(m - m_new);
          m = m_new;
          l *= a;
          if (i > 0) {  // once the last P V is done
            if (!warp_wait(&bars[L::bO + half], (no + i - 1) & 1, abort_flag, kDevTimeoutSoftmax, 22 + half, (int)no, j)) goto done;
            tc_fence_after();
            #pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              tmem_ld32(o_tm + c * 32, a0);
              tmem_wait_ld(a0);
              #pragma unroll
              for (int e = 0; e < 32; ++e) a0[e] = __float_as_uint(__uint_as_float(a0[e]) * a);
              tmem_st32(o_tm + c * 32, a0);
            }
          }
          tmem_ld32(s_tm, a0);
          tmem_ld32(s_tm + 32, a1);
          tmem_wait_ld(a0);
          tmem_wait_ld(a1);
          cut(a0, 0);
          cut(a1, 32);
          sum[0] = sum[1] = 0;
          base = (m == -INFINITY ? 0.f : m) - E::kLift;
          probabilities(a0, base, w0);
          probabilities(a1, base, w1);
        }
        const auto hand_over = [&](int part) {
          tmem_wait_st();
          warp_arrive_tc(&bars[L::bP + buf * kPrParts + part]);
        };
        if (diagonal && it.y < row0 + 128) {  // the tile reaches behind the sequence's end: clear its value rows there
          const uint32_t v = ring0 + (j == all_tiles - 1 ? 2 * all_tiles - 1 : 2 * j + 2), st = v % L::kStages;
          if (!warp_wait(&bars[L::bFull + st], (v / L::kStages) & 1, abort_flag, kDevTimeoutSoftmax, 26 + half, (int)v, j)) goto done;
          if (row0 + row >= it.y) {
            uint8_t* r = smem + L::kRing + st * L::kTileBytes + row * 128;
            #pragma unroll
            for (int c = 0; c < D / 8; ++c) *reinterpret_cast<uint4*>(r + (c >> 3) * L::kBlock + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        tmem_st16(s_tm, w0);
        tmem_st16(s_tm + 32, w1);
        hand_over(0);
        probabilities(a2, base, w0);
        tmem_st16(s_tm + 64, w0);
        probabilities(a3, base, w1);
        tmem_st16(s_tm + 96, w1);
        if (order.looks_back(half, i) &&
            !warp_wait(&bars[L::bO + half], (no + i - 1) & 1, abort_flag, kDevTimeoutSoftmax, 30 + half, (int)no, j))
          goto done;
        hand_over(1);
        sum[0] = f32x2_add(sum[0], sum[1]);
        l += f32x2_lo(sum[0]) + f32x2_hi(sum[0]);
      }
      // ---- epilogue
      no += tiles;
      if (tiles > 0 && !warp_wait(&bars[L::bO + half], (no - 1) & 1, abort_flag, kDevTimeoutSoftmax, 24 + half, (int)no)) goto done;
      tc_fence_after();
      const long long tok = (long long)it.x + row0 + row;
      T* dst = static_cast<T*>(p.o.ptr) + it.w * p.o.sh + tok * p.o.st;
      const auto store32 = [&](const uint32_t (&ov)[32], float f, int c) {
        #pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t w[4];
          #pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = E::pack(__uint_as_float(ov[8 * e + 2 * i]) * f, __uint_as_float(ov[8 * e + 2 * i + 1]) * f);
          reinterpret_cast<uint4*>(dst)[c * 4 + e] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      };
      if constexpr (!kSplit) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        #pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ov[32];
          tmem_ld32(o_tm + c * 32, ov);
          tmem_wait_ld(ov);
          if (valid) store32(ov, inv, c);
        }
        if (valid && p.lse) p.lse[(long long)it.w * p.n_tok + tok] = (m - E::kLift + log2f(l)) * 0.69314718055994530942f;
      } else {
        static_assert(2 * 256 * sizeof(float2) <= L::kTileBytes, "the copies of (m, l) lie where the second Q tile would be");
        float2* ml = reinterpret_cast<float2*>(smem + L::kQ + L::kTileBytes) + order.sums(joins) * 256;
        ml[half * 128 + row] = make_float2(m, l);
        warp_arrive_tc(&bars[L::bJoin]);
        if (!warp_wait(&bars[L::bJoin], joins & 1, abort_flag, kDevTimeoutSoftmax, 28 + half, (int)joins)) goto done;
        ++joins;
        tc_fence_after();
        const float2 other = ml[(half ^ 1) * 128 + row];
        const float2 a = half == 0 ? make_float2(m, l) : other, b = half == 0 ? other : make_float2(m, l);
        const float top = fmaxf(a.x, b.x);
        float wa = a.x == -INFINITY ? 0.f : ex2_approx(a.x - top), wb = b.x == -INFINITY ? 0.f : ex2_approx(b.x - top);
        const float sum = fmaf(wa, a.y, wb * b.y);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        wa *= inv;
        wb *= inv;
        const bool both = all_tiles > 1;  // else O_B has not been written
        #pragma unroll
        for (int c = half * (D / 64); c < (half + 1) * (D / 64); ++c) {  // this half's share of the columns
          uint32_t ov[32], ob[32];
          tmem_ld32(tmem + lane_base + L::kO + c * 32, ov);
          tmem_ld32(tmem + lane_base + L::kO + D + c * 32, ob);
          tmem_wait_ld(ov);
          tmem_wait_ld(ob);
          #pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float x = __uint_as_float(ov[e]) * wa;
            ov[e] = __float_as_uint(both ? fmaf(__uint_as_float(ob[e]), wb, x) : x);
          }
          if (valid) store32(ov, 1.f, c);
        }
        if (valid && half == 0 && p.lse) p.lse[(long long)it.w * p.n_tok + tok] = (top - E::kLift + log2f(sum)) * 0.69314718055994530942f;
        warp_arrive_tc(&bars[L::bJoined]);
      }
      tc_fence_before();  // before the next item's first P: its P V overwrites O
    }
  done:;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

}  // namespace clear
