// Attention of one new token per sequence over a paged key/value cache.
//
// For query head h of sequence s, over the keys j < seq_len[s] of kv head h / group:
//   x_j = q . k_j / sqrt(d),  m = max x_j,  l = sum e^(x_j - m),  o = sum e^(x_j - m) v_j / l,
//   lse = m + log l;  a sequence of length 0 has o = 0, lse = -inf.
//
// Bound by memory: every cached byte is read once and serves 2 * group operations, far below what even
// the warp-level matrix instruction sustains; tcgen05 needs 64 rows at least and a block-wide hand-over
// of its operands, which would only add latency. So: mma.sync m16n8k16 with 16 keys (for the scores) or 16
// elements of d (for the output) as its rows and 8 query heads of the group as its columns:
//   S^T = K Q^T,  O^T += V^T P^T,
// operands by ldmatrix; P goes from the first product's result to the second's operand by movmatrix. A kv
// head's query heads (16 at most at a time) share one reading of the cache.
//
// Work split. The unit is a (sequence, kv head, 16 heads of its group); its keys are cut into
// tiles of 64. All units' tiles form one line, and each of the grid's blocks takes an equal piece of it, so
// ragged batches and single long sequences load every SM alike. A unit's start counts as some tiles more: finishing a
// piece costs about a microsecond, so a block with many short units has fewer tiles (kUnitCost). A piece that is not a whole unit
// leaves (m, l, O) in the workspace, and a second small kernel joins the pieces of a unit in
// their order along the keys: no atomics, the same bits on every run. It is launched as a
// programmatic dependent, so its launch hides behind the first kernel.
//
// Inside a block each of 4 warps takes every fourth 16-key slice and runs alone: its own ring of
// copies, its own running (m, l, O); the four are joined once per piece. The copies run on into the block's next
// piece while this one is finished: a batch of many short sequences streams like one long one. Where pages hold a multiple of 16
// rows, a slice lies in one page and TMA brings it: two instructions by one lane, one box of 16 whole rows each for the keys and the
// values. (A bulk copy per row by every lane cost some 250 instructions a slice: they take uniform operands, so 32 addresses
// are a loop.) Other page sizes take 16-byte asynchronous copies from wherever each row lies.
// Both leave the 128-byte (64-byte) swizzle that keeps ldmatrix free of bank conflicts. Value rows past
// the sequence's end are cleared before use, so what a page holds behind the last token
// (NaN included) does not count. Softmax statistics and sums are fp32; probabilities are rounded
// to the matrix instruction's 16-bit type (bf16, or fp16 for fp16 and E4M3 caches: half a step, 2^-8 or 2^-11 of each at
// most; fp16 holds them times 2^7, see Fp16::kLift).
//
// E4M3 caches: codes are widened exactly to fp16 after ldmatrix; the keys' scale goes into the score
// scale, the values' into the output. The codes of one 32-bit register belong to four neighbouring elements of d
// (k) or two (v), so q is loaded and o written in that order. bf16 queries are brought
// into fp16's range by a power of two per head, found from the head's largest magnitude; smaller elements keep
// at least 24 bits below the largest one.
#pragma once
#include <type_traits>

#include "clear_common.cuh"
#include "clear_seq_common.cuh"

namespace clear {

constexpr int kDecWarps = 4;
constexpr int kDecThreads = kDecWarps * 32;
constexpr int kDecSlice = 16;                        // keys a warp takes at a time
constexpr int kDecTile = kDecWarps * kDecSlice;      // keys of the work split's unit
constexpr int kDecRows = 16;                         // query heads of one unit
constexpr int kDecMaxStages = 8;
constexpr int kDecMaxBlocks = 3 * 160;               // blocks of the grid: as many as are resident at once
constexpr float kDecRescale = 8.0f;                  // log2 units a head's maximum may grow before O is rescaled

struct SeqDecodeParams {
  SeqView q, o;      // [q_heads, n_seq, d]
  float* lse;        // [q_heads, n_seq] or null
  SeqCache c;
  const int* seq_len;
  int n_seq, q_heads, kv_heads, group, m_tiles;
  int max_len;       // rows that the page table has entries for: longer sequences are cut (and reported)
  float scale_log2;  // log2(e) / sqrt(d)
  int tma;           // pages hold a multiple of 16 rows: slices come by TMA
  // Workspace: per block two pieces (its first and its last): (m, l) and O of 16 rows; and, per
  // block, the split unit that begins in it.
  float* part_o;   // [2 * blocks][16][d]
  float2* part_ml; // [2 * blocks][16]
  int4* split;     // [blocks]: {unit's sequence or -1, kv head * m_tiles + tile, last block, first piece's slot}
};

// First place of block b of n (of w places), and the block that holds place x.
__device__ __forceinline__ long long dec_first(long long w, int b, int n) { return w * b / n; }
__device__ __forceinline__ int dec_block_of(long long w, long long x, int n) { return (int)(((x + 1) * n - 1) / w); }

// Blocks that get work: every one of them at least one place.
__device__ __forceinline__ int dec_blocks(long long w, int grid) { return w < grid ? (w > 0 ? (int)w : 1) : grid; }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <bool kHalf>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kHalf)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transposes an 8 x 8 matrix of 16-bit values held as a fragment (row lane / 4, columns 2 (lane % 4) and the next).
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// Two E4M3 codes (the low 16 bits) as two fp16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
  return r;
}

template <bool kF8, int D, int kN>
struct DecLayout {
  static constexpr int kRowBytes = D * (kF8 ? 1 : 2);
  // Resident blocks per SM. E4M3 slices bring half the bytes for the same instructions and want more warps: 96 sequences of 94 to
  // 6000 tokens, d = 128, take 71 us with two and 62 us with three. (bf16 at d = 64: 200000 tokens 72 and 79 us.)
  static constexpr int kPerSm = kF8 && kN == 1 ? 3 : 2;
  static constexpr int kRing = kPerSm == 3 ? 12288 : kN == 1 ? 24576 : 20480;  // bytes of a warp's ring of copies, at most
  static constexpr int kBox = kRowBytes < 128 ? kRowBytes : 128;     // bytes of row in one box: one swizzled block of 16 rows
  static constexpr int kBoxes = kRowBytes / kBox;
  static constexpr int kSide = kDecSlice * kRowBytes;                // the slice's keys; its values follow
  static constexpr int kSliceBytes = 2 * kSide;
  // Tiles' time that finishing a unit takes: about a microsecond, and a tile of 256-byte rows takes half of one. Measured with 0, 1,
  // 2, 4 and 8 on 256 sequences of 23 to 1500 tokens: 256-byte rows (bf16, d = 128) 99, 89, 88, 89 and 94 us; 128 bytes (bf16, d = 64) 72,
  // 65, 58, 56 and 62, (E4M3, d = 128) 90, 73, 67, 58 and 64; 64 bytes 72, 58, 53, 47 and 51.
  static constexpr int kUnitCost = kRowBytes >= 256 ? 2 : 4;
  static constexpr int kStages = kRing / kSliceBytes < kDecMaxStages ? kRing / kSliceBytes : kDecMaxStages;
  static constexpr int kRows = 8 * kN;
  static constexpr int kJoin = kDecWarps * kStages * kSliceBytes;    // O of the four warps, then their (m, l)
  static constexpr int kJoinMl = kJoin + kDecWarps * kRows * D * 4;
  static constexpr int kBars = kJoinMl + kDecWarps * kRows * 8;      // a barrier per warp and stage
  static constexpr int kLoc = kBars + kDecWarps * kDecMaxStages * 8; // dec_locate's scratch, then the flag of an expired wait
  static constexpr int kSmem = kLoc + 96;
  static_assert(kPerSm * (kSmem + 1024) <= 233472, "resident blocks (1 KB of each is the system's)");
  // Byte offset of 16-byte chunk c of row r within a side.
  static __device__ __forceinline__ int at(int r, int c) {
    if constexpr (kBox == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    else return (c >> 3) * (kDecSlice * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
  }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
// This thread's arrival on the barrier follows its copies so far.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Where a block's piece of the line of tiles begins: its sequence, and the sum of the tiles before it.
struct DecStart {
  long long total, before;  // places of all units; places of the sequences before seq
  int seq;
};

__device__ __forceinline__ int dec_len(const SeqDecodeParams& p, int s) {
  const int n = __ldg(p.seq_len + s);
  return n < p.max_len ? n : p.max_len;
}
__device__ __forceinline__ int dec_tiles(const SeqDecodeParams& p, int s) {
  const int n = dec_len(p, s);
  return n > 0 ? (n - 1) / kDecTile + 1 : 0;
}

// Places on the line of one unit of sequence s: kCost, then one per tile.
template <int kCost>
__device__ __forceinline__ int dec_places(const SeqDecodeParams& p, int s) {
  const int n = dec_tiles(p, s);
  return n > 0 ? n + kCost : 0;
}

// Every thread sums a contiguous share of the sequences; a scan over the block finds the share, and
// its owner walks it. All threads return the same.
template <int kCost>
__device__ __forceinline__ DecStart dec_locate(const SeqDecodeParams& p, long long* sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per_seq = p.kv_heads * p.m_tiles;
  const int share = (p.n_seq + kDecThreads - 1) / kDecThreads;
  const int s0 = tid * share, s1 = s0 + share < p.n_seq ? s0 + share : p.n_seq;
  long long mine = 0;
  for (int s = s0; s < s1; ++s) mine += (long long)dec_places<kCost>(p, s) * per_seq;
  long long incl = mine;
  #pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) sm[warp] = incl;
  if (tid == 0) { sm[8] = 0; sm[9] = 0; }
  __syncthreads();
  long long base = 0, total = 0;
  #pragma unroll
  for (int w = 0; w < kDecWarps; ++w) {
    if (w < warp) base += sm[w];
    total += sm[w];
  }
  const long long x = dec_first(total, blockIdx.x, dec_blocks(total, gridDim.x));
  long long before = base + incl - mine;
  if (x >= before && x < before + mine) {
    int s = s0;
    while (true) {
      const long long n = (long long)dec_places<kCost>(p, s) * per_seq;
      if (x < before + n || s + 1 >= s1) break;
      before += n;
      ++s;
    }
    sm[8] = before;
    sm[9] = s;
  }
  __syncthreads();
  DecStart r{total, sm[8], (int)sm[9]};
  __syncthreads();
  return r;
}

// kN: tiles of 8 query heads (1 or 2).
template <typename E, bool kF8, int D, int kN>
__global__ void __launch_bounds__(kDecThreads, DecLayout<kF8, D, kN>::kPerSm) clear_seq_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ SeqDecodeParams p) {
  using T = typename E::type;
  using L = DecLayout<kF8, D, kN>;
  constexpr bool kHalf = kF8 || !std::is_same<E, Bf16>::value;  // the matrix instruction's 16-bit type
  constexpr float kLift = kHalf ? Fp16::kLift : Bf16::kLift;
  constexpr int kSteps = D / 16;
  extern __shared__ __align__(1024) uint8_t dsm[];
  // All shared memory is dynamic: static arrays would sit before it, padded to its alignment.
  long long* const loc = reinterpret_cast<long long*>(dsm + L::kLoc);
  uint64_t* const bars = reinterpret_cast<uint64_t*>(dsm + L::kBars) + (threadIdx.x >> 5) * kDecMaxStages;  // the warp's
  volatile int* const give_up = reinterpret_cast<volatile int*>(dsm + L::kLoc + 88);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  if (lane < L::kStages) mbar_init(&bars[lane], p.tma ? 1 : 32);
  if (tid == 0) *give_up = 0;
  fence_barrier_init();

  // Sequences without a key.
  for (int s = blockIdx.x; s < p.n_seq; s += gridDim.x) {
    const int n = __ldg(p.seq_len + s);
    if (n > p.max_len && tid == 0) record_bad_index(kSiteSeqLen, s, n, p.max_len);
    if (n > 0) continue;
    for (int i = tid; i < p.q_heads * (D / 8); i += kDecThreads) {
      const int h = i / (D / 8), c = i % (D / 8);
      reinterpret_cast<uint4*>(static_cast<T*>(p.o.ptr) + h * p.o.sh + s * p.o.st)[c] = make_uint4(0, 0, 0, 0);
    }
    if (p.lse)
      for (int h = tid; h < p.q_heads; h += kDecThreads) p.lse[(long long)h * p.n_seq + s] = -INFINITY;
  }

  constexpr int kCost = L::kUnitCost;
  const DecStart st = dec_locate<kCost>(p, loc);
  const long long total = st.total;
  const int blocks = dec_blocks(total, gridDim.x);
  const bool busy = (int)blockIdx.x < blocks;
  long long x = busy ? dec_first(total, blockIdx.x, blocks) : 0;  // where the current piece begins
  const long long x_end = busy ? dec_first(total, blockIdx.x + 1, blocks) : 0;
  int split_seq = -1, split_unit = 0, split_last = 0, split_slot = 0;
  bool first_piece = true;
  uint8_t* const ring = dsm + warp * (L::kStages * L::kSliceBytes);
  const uint32_t ring_u = smem_u32(ring);
  uint32_t loads = 0, reads = 0;  // slices asked for and used, over all pieces
  bool ok = true;                 // no wait has expired
  constexpr int kE = kF8 ? 1 : 2; // bytes of an element

  // A piece: tiles [tile0, tile1) of the nt tiles of unit (seq, hk, mt), and the warp's slices of it:
  // first, first + 4, ..., mine of them.
  struct Piece {
    int seq, len, unit, hk, mt, tile0, tile1, nt, first, mine;
    long long unit0;  // the unit's first place on the line
    long long end;    // where the piece ends on the line
  };
  int walk_seq = st.seq;
  long long walk_before = st.before;
  const auto piece_at = [&](long long x) {  // x does not go back
    Piece c;
    const int per_seq = p.kv_heads * p.m_tiles;
    int n = dec_places<kCost>(p, walk_seq);
    while ((long long)n * per_seq <= x - walk_before) {
      walk_before += (long long)n * per_seq;
      ++walk_seq;
      n = dec_places<kCost>(p, walk_seq);
    }
    c.seq = walk_seq;
    c.nt = n - kCost;
    c.len = dec_len(p, c.seq);
    c.unit = (int)((x - walk_before) / n);
    c.hk = c.unit / p.m_tiles;
    c.mt = c.unit - c.hk * p.m_tiles;
    c.unit0 = walk_before + (long long)c.unit * n;
    c.end = x_end - c.unit0 < n ? x_end : c.unit0 + n;
    const int y0 = (int)(x - c.unit0) - kCost, y1 = (int)(c.end - c.unit0) - kCost;
    c.tile0 = y0 > 0 ? y0 : 0;
    c.tile1 = y1 > 0 ? y1 : 0;  // a piece of the unit's start alone has no tile
    const int slices = (c.len - 1) / kDecSlice + 1;
    const int end = (long long)c.tile1 * kDecWarps < slices ? c.tile1 * kDecWarps : slices;
    c.first = c.tile0 * kDecWarps + warp;
    c.mine = c.first < end ? (end - 1 - c.first) / kDecWarps + 1 : 0;
    return c;
  };

  // ---- the stream of copies: slice li of piece ld, which is the current piece or (ahead) the one after it
  Piece ld{};
  int li = 0;
  bool ahead = false;
  // Page numbers, by TMA: lane j holds that of slice group + j (32 slices at a time); otherwise: lane r
  // holds that of row r of the slice.
  int id = -1, row = 0, group = -32;
  const auto load_next = [&]() {
    if (!ok) return;
    if (li >= ld.mine) {
      const long long e = ld.end;
      if (ahead || e >= x_end) return;
      ld = piece_at(e);
      li = 0;
      group = -32;
      ahead = true;
      if (ld.mine == 0) return;
    }
    if (!p.tma || li >= group + 32) {
      group = li;
      const int i = p.tma ? li + lane : li;
      const int key = (ld.first + i * kDecWarps) * kDecSlice + (p.tma ? 0 : lane & 15);
      id = -1;
      if (i < ld.mine && key < ld.len) {
        const int pg = p.c.page_div.div(key);
        row = key - pg * p.c.page_size;
        id = pg < p.c.max_pages ? __ldg(p.c.table + ld.seq * p.c.table_stride + pg) : -1;
        if ((unsigned)id >= (unsigned)p.c.n_pages) {  // no such page: it reads as zeros
          record_bad_index(kSiteDecodePage, ld.seq, key, id);
          id = -1;
        }
      }
    }
    const uint32_t s = loads % L::kStages;
    if (p.tma) {
      const int page = __shfl_sync(0xffffffffu, id, li - group), r = __shfl_sync(0xffffffffu, row, li - group);
      if (lane == 0) {
        uint8_t* dst = ring + s * L::kSliceBytes;
        mbar_arrive_expect_tx(&bars[s], L::kSliceBytes);
        tma_load_5d(dst, &tm_k, &bars[s], 0, ld.hk, r, 0, page);
        tma_load_5d(dst + L::kSide, &tm_v, &bars[s], 0, ld.hk, r, 0, page);
      }
      __syncwarp();
    } else {
      constexpr int kChunks = L::kRowBytes / 16, kPer = 32 / kChunks;  // chunks of a row, rows of one copy instruction
      const bool take = id >= 0;
      const long long ko = take ? (id * p.c.ks[0] + row * p.c.ks[1] + ld.hk * p.c.ks[2]) * kE : 0;
      const long long vo = take ? (id * p.c.vs[0] + row * p.c.vs[1] + ld.hk * p.c.vs[2]) * kE : 0;
      const int c = lane % kChunks;
      const uint32_t dst = ring_u + s * L::kSliceBytes;
      #pragma unroll
      for (int r0 = 0; r0 < kDecSlice; r0 += kPer) {
        const int r = r0 + lane / kChunks;
        const long long a = __shfl_sync(0xffffffffu, ko, r), b = __shfl_sync(0xffffffffu, vo, r);
        const bool in = __shfl_sync(0xffffffffu, (int)take, r);
        cp_async16(dst + L::at(r, c), static_cast<const uint8_t*>(p.c.k) + a + c * 16, in);
        cp_async16(dst + L::kSide + L::at(r, c), static_cast<const uint8_t*>(p.c.v) + b + c * 16, in);
      }
      cp_async_arrive(&bars[s]);
    }
    ++loads;
    ++li;
  };

  // ---- queries of a piece: column g of each tile, in the order that the keys' registers have
  uint32_t qb[kN][kSteps][2];
  const auto load_queries = [&](const Piece& c) {
    #pragma unroll
    for (int n = 0; n < kN; ++n) {
      const int h = c.mt * kDecRows + n * 8 + g;
      const bool in = h < p.group;
      const T* src = static_cast<const T*>(p.q.ptr) + (long long)(c.hk * p.group + (in ? h : 0)) * p.q.sh + c.seq * p.q.st;
      #pragma unroll
      for (int kk = 0; kk < kSteps; ++kk) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(src + kk * 16);
        qb[n][kk][0] = in ? __ldg(w + (kF8 ? 2 * t : t)) : 0u;
        qb[n][kk][1] = in ? __ldg(w + (kF8 ? 2 * t + 1 : t + 4)) : 0u;
      }
    }
  };

  Piece cur{};
  if (x < x_end) {
    cur = ld = piece_at(x);
    load_next();
    load_queries(cur);
  }
  while (x < x_end) {
    while (loads - reads < (uint32_t)L::kStages) {
      const uint32_t was = loads;
      load_next();
      if (loads == was) break;
    }
    const int len = cur.len, hk = cur.hk, nt = cur.nt, tile0 = cur.tile0, tile1 = cur.tile1, seq = cur.seq, mine = cur.mine, first = cur.first;
    const long long unit0 = cur.unit0;
    const bool some = tile1 > tile0;
    const int rows = p.group - cur.mt * kDecRows < kDecRows ? p.group - cur.mt * kDecRows : kDecRows;
    const int h0 = hk * p.group + cur.mt * kDecRows;  // query head of column 0
    float sl[kN][2];  // score scale of columns 2t and 2t + 1
    #pragma unroll
    for (int n = 0; n < kN; ++n) {
      sl[n][0] = sl[n][1] = p.scale_log2;
      if constexpr (kF8) {
        int e = 0;
        if constexpr (std::is_same<E, Bf16>::value) {
          float top = 0.f;
          #pragma unroll
          for (int kk = 0; kk < kSteps; ++kk)
            #pragma unroll
            for (int u = 0; u < 2; ++u) top = fmaxf(top, fmaxf(fabsf(E::lo(qb[n][kk][u])), fabsf(E::hi(qb[n][kk][u]))));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          if (top > 0.f && top < INFINITY) e = ilogbf(top);
          // 2^-e in two factors: e may be as low as -133, and 2^133 is no fp32 number.
          const float down0 = exp2f((float)(-e / 2)), down1 = exp2f((float)(-e - (-e / 2)));
          #pragma unroll
          for (int kk = 0; kk < kSteps; ++kk)
            #pragma unroll
            for (int u = 0; u < 2; ++u)
              qb[n][kk][u] = Fp16::pack(E::lo(qb[n][kk][u]) * down0 * down1, E::hi(qb[n][kk][u]) * down0 * down1);
        }
        const float mul = p.scale_log2 * __ldg(p.c.k_scale + hk);
        #pragma unroll
        for (int u = 0; u < 2; ++u) sl[n][u] = ldexpf(mul, __shfl_sync(0xffffffffu, e, (2 * t + u) * 4));
      }
    }

    float m[kN][2], l[kN][2], o[kN][kSteps][4];
    #pragma unroll
    for (int n = 0; n < kN; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
      #pragma unroll
      for (int j = 0; j < kSteps; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.f;
    }

    for (int i = 0; i < mine; ++i) {
      const uint32_t s = reads % L::kStages;
      ok = ok && warp_wait(&bars[s], (reads / L::kStages) & 1, give_up, kDevTimeoutTmaFull, 36, seq, i);
      if (!ok) break;
      const uint32_t ks = ring_u + s * L::kSliceBytes;
      const uint32_t vs = ks + L::kSide;
      const int left = len - (first + i * kDecWarps) * kDecSlice;  // keys of the slice inside the sequence
      if (left < kDecSlice && p.tma) {  // values behind the end (asynchronous copies have left zeros there)
        for (int e = lane; e < (kDecSlice - left) * (L::kRowBytes / 16); e += 32) {
          const int r = left + e / (L::kRowBytes / 16), c = e % (L::kRowBytes / 16);
          *reinterpret_cast<uint4*>(ring + s * L::kSliceBytes + L::kSide + L::at(r, c)) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();  // a later copy will overwrite them
        __syncwarp();
      }
      // S^T = K Q^T: rows g and g + 8 are keys, columns 2t and 2t + 1 query heads
      float c[kN][4] = {};
      if constexpr (!kF8) {
        #pragma unroll
        for (int kk = 0; kk < kSteps; ++kk) {
          uint32_t a[4];  // keys 0-7 and 8-15 of the first 8 elements, then of the next
          ldsm4(a, ks + L::at(lane & 15, kk * 2 + (lane >> 4)));
          #pragma unroll
          for (int n = 0; n < kN; ++n) mma16816<kHalf>(c[n], a, qb[n][kk][0], qb[n][kk][1]);
        }
      } else {
        #pragma unroll
        for (int kk = 0; kk < kSteps; kk += 2) {
          uint32_t b[4];  // keys 0-7 and 8-15 of 16 elements, then of the next 16
          ldsm4(b, ks + L::at(lane & 15, kk + (lane >> 4)));
          #pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t a[4] = {e4m3x2_to_f16x2(b[2 * u]), e4m3x2_to_f16x2(b[2 * u + 1]), e4m3x2_to_f16x2(b[2 * u] >> 16),
                                   e4m3x2_to_f16x2(b[2 * u + 1] >> 16)};
            #pragma unroll
            for (int n = 0; n < kN; ++n) mma16816<kHalf>(c[n], a, qb[n][kk + u][0], qb[n][kk + u][1]);
          }
        }
      }
      #pragma unroll
      for (int n = 0; n < kN; ++n)
        #pragma unroll
        for (int u = 0; u < 4; ++u) c[n][u] = left >= kDecSlice || g + 8 * (u >> 1) < left ? c[n][u] * sl[n][u & 1] : -INFINITY;
      // Online softmax. The maximum in use follows the true one only when that has grown by 2^8: the result is the
      // same up to rounding, since numerator and denominator share it, and O is rarely rescaled. A lane looks at its own two
      // keys first; only if some lane's score asks for it are the true maxima found.
      bool grow = false;
      #pragma unroll
      for (int n = 0; n < kN; ++n)
        #pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float top = fmaxf(c[n][u], c[n][2 + u]);
          grow = grow || top > m[n][u] + kDecRescale || (m[n][u] == -INFINITY && top > m[n][u]);
        }
      if (__any_sync(0xffffffffu, grow)) {
        #pragma unroll
        for (int n = 0; n < kN; ++n)
          #pragma unroll
          for (int u = 0; u < 2; ++u) {
            float top = fmaxf(c[n][u], c[n][2 + u]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            // A head that does not ask for it keeps its maximum: its result has no part in its neighbours'.
            const float m_new = top > m[n][u] + kDecRescale || (m[n][u] == -INFINITY && top > m[n][u]) ? top : m[n][u];
            const float a = m[n][u] == -INFINITY ? 0.f : ex2_approx(m[n][u] - m_new);
            m[n][u] = m_new;
            l[n][u] *= a;
            #pragma unroll
            for (int j = 0; j < kSteps; ++j) {
              o[n][j][u] *= a;
              o[n][j][2 + u] *= a;
            }
          }
      }
      uint32_t pb[kN][2];  // P^T: keys 2t, 2t + 1 (and 8 further) of column g
      #pragma unroll
      for (int n = 0; n < kN; ++n)
        #pragma unroll
        for (int r = 0; r < 2; ++r) {
          float e[2];
          #pragma unroll
          for (int u = 0; u < 2; ++u) {
            e[u] = ex2_approx(c[n][2 * r + u] - ((m[n][u] == -INFINITY ? 0.f : m[n][u]) - kLift));
            l[n][u] += e[u];
          }
          pb[n][r] = movmatrix(kHalf ? Fp16::pack(e[0], e[1]) : Bf16::pack(e[0], e[1]));
        }
      // O^T += V^T P^T: rows are elements of d
      if constexpr (!kF8) {
        #pragma unroll
        for (int j = 0; j < kSteps; ++j) {
          uint32_t a[4];  // elements 0-7 and 8-15 of keys 0-7, then of keys 8-15
          ldsm4t(a, vs + L::at((lane & 7) + ((lane >> 4) << 3), j * 2 + ((lane >> 3) & 1)));
          #pragma unroll
          for (int n = 0; n < kN; ++n) mma16816<kHalf>(o[n][j], a, pb[n][0], pb[n][1]);
        }
      } else {
        #pragma unroll
        for (int j = 0; j < kSteps; j += 2) {
          uint32_t b[4];  // keys 0-7 and 8-15 of 16 elements, then of the next 16
          ldsm4t(b, vs + L::at(lane & 15, j + (lane >> 4)));
          #pragma unroll
          for (int u = 0; u < 2; ++u) {
            // A register holds keys 2t and 2t + 1 of elements 2g and 2g + 1: bring each element's keys together. Rows g
            // and g + 8 of the product are elements 2g and 2g + 1.
            const uint32_t w0 = __byte_perm(b[2 * u], 0, 0x3120), w1 = __byte_perm(b[2 * u + 1], 0, 0x3120);
            const uint32_t a[4] = {e4m3x2_to_f16x2(w0), e4m3x2_to_f16x2(w0 >> 16), e4m3x2_to_f16x2(w1), e4m3x2_to_f16x2(w1 >> 16)};
            #pragma unroll
            for (int n = 0; n < kN; ++n) mma16816<kHalf>(o[n][j + u], a, pb[n][0], pb[n][1]);
          }
        }
      }
      __syncwarp();  // the slice has been read: its place may be filled again
      ++reads;
      load_next();
    }
    #pragma unroll
    for (int n = 0; n < kN; ++n)
      #pragma unroll
      for (int u = 0; u < 2; ++u) {
        l[n][u] += __shfl_xor_sync(0xffffffffu, l[n][u], 4);
        l[n][u] += __shfl_xor_sync(0xffffffffu, l[n][u], 8);
        l[n][u] += __shfl_xor_sync(0xffffffffu, l[n][u], 16);
      }
    __syncthreads();  // the last piece's results have been read
    float* jo = reinterpret_cast<float*>(dsm + L::kJoin);
    float2* jml = reinterpret_cast<float2*>(dsm + L::kJoinMl);
    #pragma unroll
    for (int n = 0; n < kN; ++n)
      #pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int row = warp * L::kRows + n * 8 + 2 * t + u;
        if (g == 0) jml[row] = make_float2(m[n][u] - kLift, l[n][u]);  // l and O have the factor 2^kLift
        #pragma unroll
        for (int j = 0; j < kSteps; ++j) {
          float* d = jo + row * D + j * 16;
          if constexpr (!kF8) {
            d[g] = o[n][j][u];
            d[g + 8] = o[n][j][2 + u];
          } else {
            *reinterpret_cast<float2*>(d + 2 * g) = make_float2(o[n][j][u], o[n][j][2 + u]);
          }
        }
      }
    // The next piece: its copies are under way; its queries are asked for before the others are waited for.
    x = cur.end;
    if (x < x_end) {
      if (!ahead) {
        ld = piece_at(x);
        li = 0;
        group = -32;
      }
      cur = ld;
      ahead = false;
      load_queries(cur);
    }
    __syncthreads();
    const bool whole = tile0 == 0 && tile1 == nt;
    const int slot = 2 * blockIdx.x + (first_piece ? 0 : 1);
    const float vscale = kF8 ? __ldg(p.c.v_scale + hk) : 1.f;
    constexpr int kPerRow = kDecThreads / (8 * kN);  // threads a row
    {
      const int row = tid / kPerRow, part = tid % kPerRow;
      float mm = -INFINITY, w[kDecWarps], ll = 0.f;
      #pragma unroll
      for (int i = 0; i < kDecWarps; ++i) mm = fmaxf(mm, jml[i * L::kRows + row].x);
      #pragma unroll
      for (int i = 0; i < kDecWarps; ++i) {
        const float2 ml = jml[i * L::kRows + row];
        w[i] = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - mm);
        ll += w[i] * ml.y;
      }
      // A row whose scores are all -inf keeps nothing: o = 0, lse = -inf, as for a sequence of length 0.
      const float inv = whole ? (ll == 0.f ? 0.f : vscale / ll) : vscale;
      if (row < rows && some) {
        #pragma unroll
        for (int c = part; c < D / 8; c += kPerRow) {
          float y[8];
          #pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = 0.f;
          #pragma unroll
          for (int i = 0; i < kDecWarps; ++i) {
            const float4 a = *reinterpret_cast<const float4*>(jo + (i * L::kRows + row) * D + c * 8);
            const float4 b = *reinterpret_cast<const float4*>(jo + (i * L::kRows + row) * D + c * 8 + 4);
            y[0] = fmaf(w[i], a.x, y[0]); y[1] = fmaf(w[i], a.y, y[1]); y[2] = fmaf(w[i], a.z, y[2]); y[3] = fmaf(w[i], a.w, y[3]);
            y[4] = fmaf(w[i], b.x, y[4]); y[5] = fmaf(w[i], b.y, y[5]); y[6] = fmaf(w[i], b.z, y[6]); y[7] = fmaf(w[i], b.w, y[7]);
          }
          #pragma unroll
          for (int e = 0; e < 8; ++e) y[e] *= inv;
          if (whole) {
            T* dst = static_cast<T*>(p.o.ptr) + (long long)(h0 + row) * p.o.sh + seq * p.o.st;
            reinterpret_cast<uint4*>(dst)[c] =
                make_uint4(E::pack(y[0], y[1]), E::pack(y[2], y[3]), E::pack(y[4], y[5]), E::pack(y[6], y[7]));
          } else {
            float* dst = p.part_o + ((long long)slot * kDecRows + row) * D + c * 8;
            *reinterpret_cast<float4*>(dst) = make_float4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<float4*>(dst + 4) = make_float4(y[4], y[5], y[6], y[7]);
          }
        }
        if (part == 0) {
          if (!whole) p.part_ml[slot * kDecRows + row] = make_float2(mm, ll);
          else if (p.lse) p.lse[(long long)(h0 + row) * p.n_seq + seq] = (mm + log2f(ll)) * 0.69314718055994530942f;
        }
      }
    }
    if (tile0 == 0 && some && !whole) {  // a split unit begins here (it is this block's last piece)
      split_seq = seq;
      split_unit = hk * p.m_tiles + (h0 - hk * p.group) / kDecRows;
      split_last = dec_block_of(total, unit0 + kCost + nt - 1, blocks);
      split_slot = slot;
    }
    if (some) first_piece = false;
  }
  if (!ok && lane < L::kStages && loads > (uint32_t)lane) {  // an expired wait: let this warp's copies land
    const uint32_t last = loads - 1 - (loads - 1 - lane) % L::kStages;
    drain_wait(&bars[lane], (last / L::kStages) & 1);
  }
  __syncthreads();
  if (tid == 0) p.split[blockIdx.x] = make_int4(split_seq, split_unit, split_last, split_slot);
}

// Joins the pieces of the split unit that begins in block blockIdx.x of the first kernel, for head
// blockIdx.y of the unit: kJoinParts groups of D threads (one per element of d) take every kJoinParts-th piece.
constexpr int kJoinParts = 4;

template <typename E, int D>
__global__ void __launch_bounds__(kJoinParts * D) clear_seq_decode_join_kernel(const __grid_constant__ SeqDecodeParams p) {
  using T = typename E::type;
  __shared__ float2 ml[kDecMaxBlocks];  // (weight, -) of each piece
  __shared__ float red[kJoinParts][D];
  __shared__ float2 wsum[kJoinParts * D / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 u = p.split[blockIdx.x];
  if (u.x < 0) return;
  const int hk = u.y / p.m_tiles, mt = u.y - hk * p.m_tiles;
  const int row = blockIdx.y;
  if (mt * kDecRows + row >= p.group) return;
  const int h = hk * p.group + mt * kDecRows + row;
  const int n = u.z - (int)blockIdx.x + 1;  // pieces: this block's last, then the first of each block up to u.z
  const int tid = threadIdx.x, part = tid / D, e = tid % D;
  const auto slot = [&](int i) { return i == 0 ? u.w : 2 * ((int)blockIdx.x + i); };
  float m = -INFINITY;
  for (int i = tid; i < n; i += kJoinParts * D) {
    const float2 x = p.part_ml[slot(i) * kDecRows + row];
    ml[i] = x;
    m = fmaxf(m, x.x);
  }
  #pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if ((tid & 31) == 0) wsum[tid >> 5].x = m;
  __syncthreads();
  #pragma unroll
  for (int i = 0; i < kJoinParts * D / 32; ++i) m = fmaxf(m, wsum[i].x);
  float l = 0.f, o = 0.f;
  #pragma unroll 8
  for (int i = part; i < n; i += kJoinParts) {
    const float2 x = ml[i];
    const float w = x.x == -INFINITY ? 0.f : ex2_approx(x.x - m);
    l = fmaf(w, x.y, l);
    o = fmaf(w, p.part_o[((long long)slot(i) * kDecRows + row) * D + e], o);
  }
  red[part][e] = o;
  if (e == 0) wsum[part].y = l;
  __syncthreads();
  if (part != 0) return;
  l = 0.f;
  o = 0.f;
  #pragma unroll
  for (int i = 0; i < kJoinParts; ++i) {
    l += wsum[i].y;
    o += red[i][e];
  }
  o = l == 0.f ? 0.f : o / l;
  T* dst = static_cast<T*>(p.o.ptr) + h * p.o.sh + u.x * p.o.st;
  if constexpr (std::is_same<E, Bf16>::value) dst[e] = __float2bfloat16_rn(o);
  else dst[e] = __float2half_rn(o);
  if (p.lse && e == 0) p.lse[(long long)h * p.n_seq + u.x] = (m + log2f(l)) * 0.69314718055994530942f;
}

}  // namespace clear
