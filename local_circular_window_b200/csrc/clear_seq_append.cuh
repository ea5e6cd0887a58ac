// Appending to a paged key/value cache, with the rotary embedding applied on the way.
//
// Token t of sequence s has the position p = seq_len[s] - (seq_start[s + 1] - t): seq_len counts the
// sequence's tokens in the cache after this call, its new tokens being the last of them. Of each
// query and key head the first `rot` elements are turned as rot / 2 pairs, pair i by the angle
// p * base^(-2i / rot): (a, b) -> (a cos - b sin, a sin + b cos). A pair is either two neighbours,
// (2i, 2i + 1), or element i of each half, (i, i + rot / 2). Rotated queries and keys go to packed
// outputs; rotated keys and plain values go to the cache's rows of position p.
//
// Angles. p * rate is taken in double as whole and fractional turns; only the fraction, in
// [-1/2, 1/2], is rounded to fp32 (an angle error of at most pi 2^-25), so far positions lose nothing.
// One (token, pair) angle serves every head, so the double work is a few percent of the pass.
//
// An E4M3 cache stores e4m3(x / scale) from the fp32 rotated value: rounding to the input type first
// would round twice. The quotient is taken as x * (1 / scale), 1.5 units in the last place of fp32 off at most.
//
// Bound by memory: every 16-byte chunk is read once and written once or twice (keys: packed output
// and cache). A thread moves 32 bytes of a head: chunks 2i and 2i + 1, or, for paired halves, chunk i
// of each half, so both elements of each pair are in one thread.
//
// A token's place (sequence, position and page) is a chain of three loads, its angles some hundred instructions. The
// inputs depend on neither: each thread asks for its first 32 bytes before them. A block takes one token. With few tokens it has a
// thread for each 32 bytes where the heads allow it (16 tokens of 24 and 8 heads: 3.6 us). With many it has 128, so that many
// blocks of an SM are copying while others wait for their angles: 9177 tokens of 32 and 8 heads take 43 us, 5.6 TB/s; 61 us
// with 384 threads a token, 45 with two tokens in 128.
#pragma once
#include "clear_seq_common.cuh"

namespace clear {

constexpr int kAppendMaxThreads = 512;
constexpr int kAppendMaxPairs = 64;

struct SeqAppendParams {
  SeqView q, k, v, q_out, k_out;  // q.ptr, q_out.ptr, k_out.ptr may be null
  SeqCache c;
  const int *seq_start, *seq_len;
  int n_seq, n_tok, q_heads, kv_heads;
  int rot;
  double turns[kAppendMaxPairs];  // rate of pair i in turns per position: base^(-2i / rot) / (2 pi)
};

// The sequence that holds token t, or -1. Where the offsets ascend it is the last s with seq_start[s] <= t, found by a search in which
// the 32 lanes of a warp probe at once (one round for 32 sequences, two for 1024). A token that the search has not placed
// (padding, or offsets out of order) is looked for in the whole list. A sequence whose offsets decrease or leave [0, n_tok] holds no
// token. Terminates whatever seq_start holds.
__device__ __forceinline__ int seq_of_token(const int* __restrict__ seq_start, int n_seq, int n_tok, int t, int lane, int* end) {
  int lo = 0, n = n_seq;  // candidates [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lane * step;
    const bool le = at < n && __ldg(seq_start + lo + at) <= t;
    const int hits = __popc(__ballot_sync(0xffffffffu, le));
    const int first = hits > 0 ? (hits - 1) * step : 0;
    lo += first;
    n = n - first < step ? n - first : step;
  }
  const int a = __ldg(seq_start + lo), b = __ldg(seq_start + lo + 1);
  *end = b;
  if (a >= 0 && a <= t && t < b && b <= n_tok) return lo;
  int s = -1;
  for (int i = lane; i < n_seq && s < 0; i += 32) {
    const int c = __ldg(seq_start + i), e = __ldg(seq_start + i + 1);
    if (c >= 0 && c <= t && t < e && e <= n_tok) s = i;
  }
  s = __reduce_max_sync(0xffffffffu, s);
  if (s >= 0) *end = __ldg(seq_start + s + 1);
  return s;
}

// Offsets that decrease or reach outside leave their sequence out: says so. One block's warps beside the first call it, while that one
// follows its chain of loads. Not inlined: as a loop of the kernel's own it took 5 % of a long prompt's time (16384 tokens: 79.7 and
// 76 us).
__device__ __noinline__ void report_bad_offsets(const int* __restrict__ seq_start, int n_seq, int n_tok, int first, int step) {
  for (int s = first; s < n_seq; s += step) {
    const int a = __ldg(seq_start + s), b = __ldg(seq_start + s + 1);
    if (a < 0 || b < a || b > n_tok) record_bad_index(kSiteSeqStart, s, a, b);
  }
}

// E: element type; kF8: E4M3 cache; D: head dim; kHalves: pairs of halves.
template <typename E, bool kF8, int D, bool kHalves>
__global__ void __launch_bounds__(kAppendMaxThreads) clear_seq_append_kernel(const __grid_constant__ SeqAppendParams p) {
  using T = typename E::type;
  constexpr int kItems = D / 16;  // 32-byte items per head
  __shared__ float2 cs[kAppendMaxPairs];  // pair 8 i + e at 8 e + i: threads of neighbouring items read neighbours
  __shared__ long long row_at[2];         // element offset of the cache row of k and of v, or -1: not stored
  __shared__ int pos_at;                  // position, or -1: nothing to do
  const int tid = threadIdx.x, lane = tid & 31;
  const int t = blockIdx.x;
  const int items = (p.q_heads + 2 * p.kv_heads) * kItems;
  const int rot_items = p.rot >> 4;

  // Item i: 32 bytes of a query, key or value head.
  const auto load = [&](int i, uint4* w0, uint4* w1) {
    int h = i / kItems;
    const int it = i % kItems;
    const SeqView& in = h < p.q_heads ? p.q : h < p.q_heads + p.kv_heads ? p.k : p.v;
    const bool is_v = h >= p.q_heads + p.kv_heads;
    h -= h < p.q_heads ? 0 : is_v ? p.q_heads + p.kv_heads : p.q_heads;
    const bool apart = kHalves && !is_v && it < rot_items;
    const T* src = static_cast<const T*>(in.ptr) + h * in.sh + t * in.st;
    *w0 = reinterpret_cast<const uint4*>(src)[apart ? it : 2 * it];  // plain loads: outputs may be the inputs
    *w1 = reinterpret_cast<const uint4*>(src)[apart ? it + rot_items : 2 * it + 1];
  };
  uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
  if (tid < items) load(tid, &w0, &w1);

  if (tid < 32) {
    int pos = -1;
    long long kr = -1, vr = -1;
    int end;
    const int s = seq_of_token(p.seq_start, p.n_seq, p.n_tok, t, lane, &end);
    if (s >= 0) {
      const long long x = (long long)__ldg(p.seq_len + s) - (end - t);
      if (x >= 0) {  // a negative position is padding
        pos = (int)x;
        const int pg = p.c.page_div.div(pos);
        const int row = pos - pg * p.c.page_size;
        const int id = pg < p.c.max_pages ? __ldg(p.c.table + s * p.c.table_stride + pg) : -1;
        if ((unsigned)id < (unsigned)p.c.n_pages) {
          kr = id * p.c.ks[0] + row * p.c.ks[1];
          vr = id * p.c.vs[0] + row * p.c.vs[1];
        } else if (lane == 0) {
          record_bad_index(kSiteAppendPage, s, pos, id);
        }
      }
    }
    if (lane == 0) {
      pos_at = pos;
      row_at[0] = kr;
      row_at[1] = vr;
    }
  } else if (blockIdx.x == 0) {
    report_bad_offsets(p.seq_start, p.n_seq, p.n_tok, tid - 32, blockDim.x - 32);
  }
  __syncthreads();
  const int pos = pos_at;
  if (pos < 0) return;
  for (int i = tid; i < (p.rot >> 1); i += blockDim.x) {
    const double turn = (double)pos * p.turns[i];
    float s, c;
    sincospif((float)(2.0 * (turn - rint(turn))), &s, &c);
    cs[(i & 7) * 8 + (i >> 3)] = make_float2(c, s);
  }
  __syncthreads();

  for (int i = tid; i < items; i += blockDim.x) {
    if (i != tid) load(i, &w0, &w1);
    int h = i / kItems;
    const int it = i % kItems;
    const bool is_q = h < p.q_heads;
    if (!is_q) h -= p.q_heads;
    const bool is_v = !is_q && h >= p.kv_heads;
    if (is_v) h -= p.kv_heads;
    const bool turned = !is_v && it < rot_items;
    const int c0 = (kHalves && turned) ? it : 2 * it;
    const int c1 = (kHalves && turned) ? it + rot_items : 2 * it + 1;
    uint32_t x[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
    float f[16];
    #pragma unroll
    for (int e = 0; e < 8; ++e) {
      f[2 * e] = E::lo(x[e]);
      f[2 * e + 1] = E::hi(x[e]);
    }
    if (turned) {
      if (kHalves) {
        #pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 w = cs[e * 8 + it];
          const float lo = f[e], hi = f[8 + e];
          f[e] = fmaf(lo, w.x, -hi * w.y);
          f[8 + e] = fmaf(lo, w.y, hi * w.x);
        }
      } else {
        #pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 w = cs[e * 8 + it];
          const float lo = f[2 * e], hi = f[2 * e + 1];
          f[2 * e] = fmaf(lo, w.x, -hi * w.y);
          f[2 * e + 1] = fmaf(lo, w.y, hi * w.x);
        }
      }
      #pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = E::pack(f[2 * e], f[2 * e + 1]);
    }
    const uint4 y0 = make_uint4(x[0], x[1], x[2], x[3]), y1 = make_uint4(x[4], x[5], x[6], x[7]);
    if (!is_v) {
      const SeqView& out = is_q ? p.q_out : p.k_out;
      if (out.ptr) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(out.ptr) + h * out.sh + t * out.st);
        dst[c0] = y0;
        dst[c1] = y1;
      }
    }
    if (!is_q) {
      const long long row = row_at[is_v];
      if (row >= 0) {
        const long long at = row + h * (is_v ? p.c.vs[2] : p.c.ks[2]);
        void* base = is_v ? p.c.v : p.c.k;
        if constexpr (kF8) {
          const float inv = 1.f / __ldg((is_v ? p.c.v_scale : p.c.k_scale) + h);
          uint32_t y[4];
          #pragma unroll
          for (int e = 0; e < 4; ++e)
            y[e] = pack_e4m3x2(f[4 * e] * inv, f[4 * e + 1] * inv) | (pack_e4m3x2(f[4 * e + 2] * inv, f[4 * e + 3] * inv) << 16);
          uint2* dst = reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + at);
          dst[c0] = make_uint2(y[0], y[1]);
          dst[c1] = make_uint2(y[2], y[3]);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(base) + at);
          dst[c0] = y0;
          dst[c1] = y1;
        }
      }
    }
  }
}

}  // namespace clear
