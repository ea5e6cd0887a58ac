// Attention of one new token per sequence over a paged key/value cache.
//
// For query head h of sequence s, over the keys j < seq_len[s] of kv head h / group:
//   x_j = q . k_j / sqrt(d),  m = max x_j,  l = sum e^(x_j - m),  o = sum e^(x_j - m) v_j / l,
//   lse = m + log l;  a sequence of length 0 has o = 0, lse = -inf.
//
// Bound by memory: every cached byte is read once and serves 2 * group operations (group <= 16 rows
// fill one 16-row matrix tile), far below what even the warp-level matrix instruction sustains;
// tcgen05 needs 64 rows at least and its operands through shared-memory descriptors, which would
// only add latency. So: mma.sync m16n8k16 with the group's query heads as the 16 rows (one matrix
// tile per kv head reads the cache once for all its query heads), operands by ldmatrix.
//
// Work split. The unit is a (sequence, kv head, 16-row tile of its group); its keys are cut into
// tiles of 64. All units' tiles form one line, and each of the grid's blocks takes an equal piece of it, so
// ragged batches and single long sequences load every SM alike. A piece that is not a whole unit
// leaves (m, l, O) in the workspace, and a second small kernel joins the pieces of a unit in
// their order along the keys: no atomics, the same bits on every run. It is launched as a
// programmatic dependent, so its launch hides behind the first kernel.
//
// Inside a block each of 4 warps takes every fourth 16-key slice and runs alone: its own ring of
// asynchronous copies, its own running (m, l, O); the four are joined once per piece. Rows past the
// sequence's end are not read but filled with zeros, so what a page holds behind the last token
// (NaN included) does not count. Softmax statistics and sums are fp32; probabilities are rounded
// to the matrix instruction's 16-bit type (bf16, or fp16 for fp16 and E4M3 caches: half a step,
// 2^-9 or 2^-12 of each, of random sign).
//
// E4M3 caches: codes are widened exactly to fp16 after ldmatrix; the keys' scale goes into the score
// scale, the values' into the output. The codes of one 32-bit register belong to four neighbouring elements of d
// (k) or two (v), so q is loaded and o written in that order. bf16 queries are brought
// into fp16's range by a power of two per row, found from the row's largest magnitude; smaller elements keep
// at least 24 bits below the largest one.
#pragma once
#include <type_traits>

#include "clear_seq_common.cuh"

namespace clear {

constexpr int kDecWarps = 4;
constexpr int kDecThreads = kDecWarps * 32;
constexpr int kDecSlice = 16;                        // keys a warp takes at a time
constexpr int kDecTile = kDecWarps * kDecSlice;      // keys of the work split's unit
constexpr int kDecRows = 16;                         // query heads of one matrix tile
constexpr int kDecRing = 24576;                      // bytes of a warp's ring of copies
constexpr int kDecMaxStages = 8;
constexpr float kDecRescale = 8.0f;                  // log2 units a row's maximum may grow before O is rescaled

struct SeqDecodeParams {
  SeqView q, o;      // [q_heads, n_seq, d]
  float* lse;        // [q_heads, n_seq] or null
  SeqCache c;
  const int* seq_len;
  int n_seq, q_heads, kv_heads, group, m_tiles;
  float scale_log2;  // log2(e) / sqrt(d)
  // Workspace: per block two pieces (its first and its last): (m, l) and O of 16 rows; and, per
  // block, the split unit that begins in it.
  float* part_o;   // [2 * blocks][16][d]
  float2* part_ml; // [2 * blocks][16]
  int4* split;     // [blocks]: {unit's sequence or -1, kv head * m_tiles + tile, last block, first piece's slot}
};

// First tile of block b of n (of w tiles), and the block that holds tile x.
__device__ __forceinline__ long long dec_first(long long w, int b, int n) { return w * b / n; }
__device__ __forceinline__ int dec_block_of(long long w, long long x, int n) { return (int)(((x + 1) * n - 1) / w); }

// Blocks that get work: every one of them at least one tile, so no piece is empty.
__device__ __forceinline__ int dec_blocks(long long w, int grid) { return w < grid ? (w > 0 ? (int)w : 1) : grid; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

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
// Two E4M3 codes (the low 16 bits) as two fp16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
  return r;
}

template <bool kF8, int D>
struct DecLayout {
  static constexpr int kRowBytes = D * (kF8 ? 1 : 2);
  static constexpr int kChunks = kRowBytes / 16;                  // 16-byte chunks of a row
  static constexpr int kSliceBytes = 2 * kDecSlice * kRowBytes;   // keys, then values
  static constexpr int kStages = kDecRing / kSliceBytes < kDecMaxStages ? kDecRing / kSliceBytes : kDecMaxStages;
  static constexpr int kWarpBytes = kStages * kSliceBytes;
  static constexpr int kJoinBytes = kDecWarps * kDecRows * (D + 2) * 4;  // reuses the rings
  static constexpr int kRings = kDecWarps * kWarpBytes;
  static constexpr int kSmem = kRings > kJoinBytes ? kRings : kJoinBytes;
  // Byte offset of chunk c of row r: chunks are exchanged within a row so that the eight rows that ldmatrix
  // reads at a time lie in eight different 16-byte bank groups.
  static __device__ __forceinline__ int at(int r, int c) {
    return kRowBytes == 64 ? r * 64 + ((c ^ ((r >> 1) & 3)) << 4) : r * kRowBytes + ((c ^ (r & 7)) << 4);
  }
};

// Where a block's piece of the line of tiles begins: its sequence, and the sum of the tiles before it.
struct DecStart {
  long long total, before;  // tiles of all units; tiles of the sequences before seq
  int seq;
};

__device__ __forceinline__ int dec_tiles(const SeqDecodeParams& p, int s) {
  const int n = __ldg(p.seq_len + s);
  return n > 0 ? (n - 1) / kDecTile + 1 : 0;
}

// Every thread sums a contiguous share of the sequences; a scan over the block finds the share, and
// its owner walks it. All threads return the same.
__device__ __forceinline__ DecStart dec_locate(const SeqDecodeParams& p, long long* sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per_seq = p.kv_heads * p.m_tiles;
  const int share = (p.n_seq + kDecThreads - 1) / kDecThreads;
  const int s0 = tid * share, s1 = s0 + share < p.n_seq ? s0 + share : p.n_seq;
  long long mine = 0;
  for (int s = s0; s < s1; ++s) mine += (long long)dec_tiles(p, s) * per_seq;
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
      const long long n = (long long)dec_tiles(p, s) * per_seq;
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

template <typename E, bool kF8, int D>
__global__ void __launch_bounds__(kDecThreads, 2) clear_seq_decode_kernel(const __grid_constant__ SeqDecodeParams p) {
  using T = typename E::type;
  using L = DecLayout<kF8, D>;
  constexpr bool kHalf = kF8 || !std::is_same<E, Bf16>::value;  // the matrix instruction's 16-bit type
  constexpr int kKSteps = D / 16;
  extern __shared__ __align__(128) uint8_t dsm[];
  __shared__ long long loc[10];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;

  // Sequences without a key.
  for (int s = blockIdx.x; s < p.n_seq; s += gridDim.x) {
    if (__ldg(p.seq_len + s) > 0) continue;
    for (int i = tid; i < p.q_heads * (D / 8); i += kDecThreads) {
      const int h = i / (D / 8), c = i % (D / 8);
      reinterpret_cast<uint4*>(static_cast<T*>(p.o.ptr) + h * p.o.sh + s * p.o.st)[c] = make_uint4(0, 0, 0, 0);
    }
    if (p.lse)
      for (int h = tid; h < p.q_heads; h += kDecThreads) p.lse[(long long)h * p.n_seq + s] = -INFINITY;
  }

  const DecStart st = dec_locate(p, loc);
  const long long total = st.total;
  const int blocks = dec_blocks(total, gridDim.x);
  const bool busy = (int)blockIdx.x < blocks;
  long long x = busy ? dec_first(total, blockIdx.x, blocks) : 0;
  const long long x_end = busy ? dec_first(total, blockIdx.x + 1, blocks) : 0;
  int seq = st.seq;
  long long before = st.before;
  int split_seq = -1, split_unit = 0, split_last = 0, split_slot = 0;
  bool first_piece = true;
  const uint32_t ring = smem_u32(dsm) + warp * L::kWarpBytes;

  while (x < x_end) {
    // ---- the piece [tile0, tile1) of unit (seq, hk, mt)
    int nt = dec_tiles(p, seq);
    while ((long long)nt * p.kv_heads * p.m_tiles <= x - before) {
      before += (long long)nt * p.kv_heads * p.m_tiles;
      ++seq;
      nt = dec_tiles(p, seq);
    }
    const int len = __ldg(p.seq_len + seq);
    const int unit = (int)((x - before) / nt);
    const int hk = unit / p.m_tiles, mt = unit - hk * p.m_tiles;
    const long long unit0 = before + (long long)unit * nt;
    const int tile0 = (int)(x - unit0);
    const int tile1 = (int)((x_end - unit0 < nt) ? x_end - unit0 : nt);
    const int rows = p.group - mt * kDecRows < kDecRows ? p.group - mt * kDecRows : kDecRows;
    const int h0 = hk * p.group + mt * kDecRows;  // query head of row 0

    // ---- the warp's slices: first, first + 4, ... below n_slices
    const int n_slices = tile1 * kDecWarps < (len + kDecSlice - 1) / kDecSlice ? tile1 * kDecWarps : (len + kDecSlice - 1) / kDecSlice;
    const int first = tile0 * kDecWarps + warp;
    const int mine = first < n_slices ? (n_slices - 1 - first) / kDecWarps + 1 : 0;
    const int* table = p.c.table + seq * p.c.table_stride;

    auto load_slice = [&](int i) {
      if (i < mine) {
        const int key0 = (first + i * kDecWarps) * kDecSlice;
        // Lane r (and r + 16) finds row r's place; the copies then fetch it by shuffles.
        const int key = key0 + (lane & 15);
        const bool in = key < len;
        long long ko = 0, vo = 0;
        bool ok = in;
        if (in) {
          const int pg = p.c.page_div.div(key);
          const int row = key - pg * p.c.page_size;
          const int id = pg < p.c.max_pages ? __ldg(table + pg) : -1;
          ok = (unsigned)id < (unsigned)p.c.n_pages;
          if (ok) {
            ko = id * p.c.ks[0] + row * p.c.ks[1];
            vo = id * p.c.vs[0] + row * p.c.vs[1];
          } else {
            record_bad_index(kSiteDecodePage, seq, key, id);
          }
        }
        ko += hk * p.c.ks[2];
        vo += hk * p.c.vs[2];
        const uint32_t dst = ring + (i % L::kStages) * L::kSliceBytes;
        constexpr int kPer = 32 / L::kChunks;  // rows of one copy instruction
        const int c = lane % L::kChunks;
        #pragma unroll
        for (int r0 = 0; r0 < kDecSlice; r0 += kPer) {
          const int r = r0 + lane / L::kChunks;
          const long long a = __shfl_sync(0xffffffffu, ko, r);
          const long long b = __shfl_sync(0xffffffffu, vo, r);
          const bool take = __shfl_sync(0xffffffffu, (int)ok, r);
          cp_async16(dst + L::at(r, c), static_cast<const uint8_t*>(p.c.k) + a * (kF8 ? 1 : 2) + c * 16, take);
          cp_async16(dst + kDecSlice * L::kRowBytes + L::at(r, c), static_cast<const uint8_t*>(p.c.v) + b * (kF8 ? 1 : 2) + c * 16, take);
        }
      }
      cp_async_commit();
    };
    #pragma unroll
    for (int i = 0; i < L::kStages - 1; ++i) load_slice(i);

    // ---- queries: rows g and g + 8 of the matrix tile, in the order the keys' registers have
    uint32_t qa[kKSteps][4];
    float sl[2] = {p.scale_log2, p.scale_log2};
    {
      #pragma unroll
      for (int r = 0; r < 2; ++r) {
        const bool in = g + 8 * r < rows;
        const T* src = static_cast<const T*>(p.q.ptr) + (long long)(h0 + (in ? g + 8 * r : 0)) * p.q.sh + seq * p.q.st;
        #pragma unroll
        for (int kk = 0; kk < kKSteps; ++kk) {
          const uint32_t* w = reinterpret_cast<const uint32_t*>(src + kk * 16);
          qa[kk][r] = in ? __ldg(w + (kF8 ? 2 * t : t)) : 0u;
          qa[kk][2 + r] = in ? __ldg(w + (kF8 ? 2 * t + 1 : t + 4)) : 0u;
        }
      }
      if constexpr (kF8) {
        const float ks = __ldg(p.c.k_scale + hk);
        #pragma unroll
        for (int r = 0; r < 2; ++r) {
          int e = 0;
          if constexpr (std::is_same<E, Bf16>::value) {
            float top = 0.f;
            #pragma unroll
            for (int kk = 0; kk < kKSteps; ++kk)
              #pragma unroll
              for (int u = r; u < 4; u += 2) top = fmaxf(top, fmaxf(fabsf(E::lo(qa[kk][u])), fabsf(E::hi(qa[kk][u]))));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            if (top > 0.f && top < INFINITY) e = ilogbf(top);
            // 2^-e in two factors: e may be as low as -133, and 2^133 is no fp32 number.
            const float down0 = exp2f((float)(-e / 2)), down1 = exp2f((float)(-e - (-e / 2)));
            #pragma unroll
            for (int kk = 0; kk < kKSteps; ++kk)
              #pragma unroll
              for (int u = r; u < 4; u += 2)
                qa[kk][u] = Fp16::pack(E::lo(qa[kk][u]) * down0 * down1, E::hi(qa[kk][u]) * down0 * down1);
          }
          sl[r] *= ks;
          sl[r] = ldexpf(sl[r], e);
        }
      }
    }

    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[D / 8][4];
    #pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    for (int i = 0; i < mine; ++i) {
      load_slice(i + L::kStages - 1);
      cp_async_wait<L::kStages - 1>();
      __syncwarp();
      const uint32_t ks = ring + (i % L::kStages) * L::kSliceBytes;
      const uint32_t vs = ks + kDecSlice * L::kRowBytes;
      // S = Q K^T: two 8-key tiles
      float s[2][4] = {};
      if constexpr (!kF8) {
        #pragma unroll
        for (int kk = 0; kk < kKSteps; ++kk) {
          uint32_t b[4];
          ldsm4(b, ks + L::at((lane & 7) + ((lane >> 4) << 3), kk * 2 + ((lane >> 3) & 1)));
          mma16816<kHalf>(s[0], qa[kk], b[0], b[1]);
          mma16816<kHalf>(s[1], qa[kk], b[2], b[3]);
        }
      } else {
        #pragma unroll
        for (int kk = 0; kk < kKSteps; kk += 2) {
          uint32_t b[4];  // keys 0-7 and 8-15 of chunk kk, then of chunk kk + 1
          ldsm4(b, ks + L::at((lane & 7) + (((lane >> 3) & 1) << 3), kk + (lane >> 4)));
          #pragma unroll
          for (int u = 0; u < 4; ++u)
            mma16816<kHalf>(s[u & 1], qa[kk + (u >> 1)], e4m3x2_to_f16x2(b[u]), e4m3x2_to_f16x2(b[u] >> 16));
        }
      }
      // Online softmax of rows g (elements 0, 1 of each tile) and g + 8 (elements 2, 3)
      const int key0 = (first + i * kDecWarps) * kDecSlice;
      float top[2];
      #pragma unroll
      for (int r = 0; r < 2; ++r) {
        #pragma unroll
        for (int n = 0; n < 2; ++n)
          #pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& v = s[n][2 * r + e];
            v = key0 + n * 8 + 2 * t + e < len ? v * sl[r] : -INFINITY;
          }
        float x4 = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
        x4 = fmaxf(x4, __shfl_xor_sync(0xffffffffu, x4, 1));
        top[r] = fmaxf(x4, __shfl_xor_sync(0xffffffffu, x4, 2));
      }
      // The maximum in use follows the true one only when that has grown by 2^8: the result is the
      // same up to rounding, since numerator and denominator share it, and O is rarely rescaled.
      const bool grow = top[0] > m[0] + kDecRescale || top[1] > m[1] + kDecRescale || (m[0] == -INFINITY && top[0] > m[0]) ||
                        (m[1] == -INFINITY && top[1] > m[1]);
      if (__any_sync(0xffffffffu, grow)) {
        #pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float m_new = fmaxf(m[r], top[r]);
          const float a = m[r] == -INFINITY ? 0.f : ex2_approx(m[r] - m_new);
          m[r] = m_new;
          l[r] *= a;
          #pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            o[n][2 * r] *= a;
            o[n][2 * r + 1] *= a;
          }
        }
      }
      uint32_t pa[4];
      #pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float base = m[r] == -INFINITY ? 0.f : m[r];
        #pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float p0 = ex2_approx(s[n][2 * r] - base), p1 = ex2_approx(s[n][2 * r + 1] - base);
          l[r] += p0 + p1;
          pa[2 * n + r] = kHalf ? Fp16::pack(p0, p1) : Bf16::pack(p0, p1);
        }
      }
      // O += P V
      if constexpr (!kF8) {
        #pragma unroll
        for (int n = 0; n < D / 8; n += 2) {
          uint32_t b[4];
          ldsm4t(b, vs + L::at((lane & 7) + (((lane >> 3) & 1) << 3), n + (lane >> 4)));
          mma16816<kHalf>(o[n], pa, b[0], b[1]);
          mma16816<kHalf>(o[n + 1], pa, b[2], b[3]);
        }
      } else {
        #pragma unroll
        for (int c = 0; c < D / 16; c += 2) {
          uint32_t b[4];  // keys 0-7 and 8-15 of chunk c, then of chunk c + 1
          ldsm4t(b, vs + L::at((lane & 7) + (((lane >> 3) & 1) << 3), c + (lane >> 4)));
          #pragma unroll
          for (int u = 0; u < 2; ++u) {
            // A register holds keys 2t and 2t + 1 of elements 2g and 2g + 1: bring each element's keys together.
            const uint32_t w0 = __byte_perm(b[2 * u], 0, 0x3120), w1 = __byte_perm(b[2 * u + 1], 0, 0x3120);
            mma16816<kHalf>(o[2 * (c + u)], pa, e4m3x2_to_f16x2(w0), e4m3x2_to_f16x2(w1));
            mma16816<kHalf>(o[2 * (c + u) + 1], pa, e4m3x2_to_f16x2(w0 >> 16), e4m3x2_to_f16x2(w1 >> 16));
          }
        }
      }
      __syncwarp();  // the slice has been read: its place may be filled again
    }
    cp_async_wait<0>();
    #pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
    __syncthreads();  // every warp is done with its ring: it now holds the four warps' results
    float* jo = reinterpret_cast<float*>(dsm);
    float2* jml = reinterpret_cast<float2*>(jo + kDecWarps * kDecRows * D);
    #pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = warp * kDecRows + g + 8 * r;
      if (t == 0) jml[row] = make_float2(m[r], l[r]);
      #pragma unroll
      for (int n = 0; n < D / 8; n += 2) {
        float* d = jo + row * D;
        if constexpr (!kF8) {
          *reinterpret_cast<float2*>(d + n * 8 + 2 * t) = make_float2(o[n][2 * r], o[n][2 * r + 1]);
          *reinterpret_cast<float2*>(d + n * 8 + 8 + 2 * t) = make_float2(o[n + 1][2 * r], o[n + 1][2 * r + 1]);
        } else {
          *reinterpret_cast<float4*>(d + n * 8 + 4 * t) =
              make_float4(o[n][2 * r], o[n + 1][2 * r], o[n][2 * r + 1], o[n + 1][2 * r + 1]);
        }
      }
    }
    __syncthreads();
    const bool whole = tile0 == 0 && tile1 == nt;
    const int slot = 2 * blockIdx.x + (first_piece ? 0 : 1);
    const float vscale = kF8 ? __ldg(p.c.v_scale + hk) : 1.f;
    constexpr int kPerRow = kDecThreads / kDecRows;  // 8 threads a row
    {
      const int row = tid / kPerRow, part = tid % kPerRow;
      float mm = -INFINITY, w[kDecWarps], ll = 0.f;
      #pragma unroll
      for (int i = 0; i < kDecWarps; ++i) mm = fmaxf(mm, jml[i * kDecRows + row].x);
      #pragma unroll
      for (int i = 0; i < kDecWarps; ++i) {
        const float2 ml = jml[i * kDecRows + row];
        w[i] = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - mm);
        ll += w[i] * ml.y;
      }
      // A row whose scores are all -inf keeps nothing: o = 0, lse = -inf, as for a sequence of length 0.
      const float inv = whole ? (ll == 0.f ? 0.f : vscale / ll) : vscale;
      if (row < rows) {
        #pragma unroll
        for (int c = part; c < D / 8; c += kPerRow) {
          float y[8];
          #pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = 0.f;
          #pragma unroll
          for (int i = 0; i < kDecWarps; ++i) {
            const float4 a = *reinterpret_cast<const float4*>(jo + (i * kDecRows + row) * D + c * 8);
            const float4 b = *reinterpret_cast<const float4*>(jo + (i * kDecRows + row) * D + c * 8 + 4);
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
    if (tile0 == 0 && !whole) {  // a split unit begins here (it is this block's last piece)
      split_seq = seq;
      split_unit = unit;
      split_last = dec_block_of(total, unit0 + nt - 1, blocks);
      split_slot = slot;
    }
    first_piece = false;
    x = unit0 + tile1;
    __syncthreads();  // the results have been read: the rings may be filled again
  }
  if (tid == 0) p.split[blockIdx.x] = make_int4(split_seq, split_unit, split_last, split_slot);
}

// Joins the pieces of the split unit that begins in block blockIdx.x of the first kernel, for row
// blockIdx.y of its matrix tile; one thread per element of d.
template <typename E, int D>
__global__ void __launch_bounds__(D) clear_seq_decode_join_kernel(const __grid_constant__ SeqDecodeParams p) {
  using T = typename E::type;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 u = p.split[blockIdx.x];
  if (u.x < 0) return;
  const int hk = u.y / p.m_tiles, mt = u.y - hk * p.m_tiles;
  const int row = blockIdx.y;
  if (mt * kDecRows + row >= p.group) return;
  const int h = hk * p.group + mt * kDecRows + row;
  const int n = u.z - (int)blockIdx.x + 1;  // pieces: this block's last, then the first of each block up to u.z
  const auto slot = [&](int i) { return i == 0 ? u.w : 2 * ((int)blockIdx.x + i); };
  float m = -INFINITY;
  for (int i = 0; i < n; ++i) m = fmaxf(m, p.part_ml[slot(i) * kDecRows + row].x);
  float l = 0.f, o = 0.f;
  #pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float2 ml = p.part_ml[slot(i) * kDecRows + row];
    const float w = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - m);
    l = fmaf(w, ml.y, l);
    o = fmaf(w, p.part_o[((long long)slot(i) * kDecRows + row) * D + threadIdx.x], o);
  }
  o = l == 0.f ? 0.f : o / l;
  T* dst = static_cast<T*>(p.o.ptr) + h * p.o.sh + u.x * p.o.st;
  if constexpr (std::is_same<E, Bf16>::value) dst[threadIdx.x] = __float2bfloat16_rn(o);
  else dst[threadIdx.x] = __float2half_rn(o);
  if (p.lse && threadIdx.x == 0) p.lse[(long long)h * p.n_seq + u.x] = (m + log2f(l)) * 0.69314718055994530942f;
}

}  // namespace clear
