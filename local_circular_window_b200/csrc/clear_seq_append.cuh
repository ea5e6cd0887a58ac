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
// would round twice.
//
// Bound by memory: every 16-byte chunk is read once and written once or twice (keys: packed output
// and cache). A thread moves 32 bytes of a head: chunks 2i and 2i + 1, or, for paired halves, chunk i
// of each half, so both elements of each pair are in one thread.
#pragma once
#include "clear_seq_common.cuh"

namespace clear {

constexpr int kAppendThreads = 256;
constexpr int kAppendMaxPairs = 64;

struct SeqAppendParams {
  SeqView q, k, v, q_out, k_out;  // q.ptr, q_out.ptr, k_out.ptr may be null
  SeqCache c;
  const int *seq_start, *seq_len;
  int n_seq, n_tok, q_heads, kv_heads;
  int rot;
  double turns[kAppendMaxPairs];  // rate of pair i in turns per position: base^(-2i / rot) / (2 pi)
};

// The sequence that holds token t: the last s with seq_start[s] <= t, by a search in which the 32
// lanes of a warp probe at once (one round for 32 sequences, two for 1024). -1 if t lies outside
// of [seq_start[s], seq_start[s + 1]). Terminates whatever seq_start holds.
__device__ __forceinline__ int seq_of_token(const int* __restrict__ seq_start, int n_seq, int t, int lane) {
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
  return (__ldg(seq_start + lo) <= t && t < __ldg(seq_start + lo + 1)) ? lo : -1;
}

// E: element type; kF8: E4M3 cache; D: head dim; kHalves: pairs of halves; kTok: tokens per block.
template <typename E, bool kF8, int D, bool kHalves, int kTok>
__global__ void __launch_bounds__(kAppendThreads) clear_seq_append_kernel(const __grid_constant__ SeqAppendParams p) {
  using T = typename E::type;
  constexpr int kItems = D / 16;  // 32-byte items per head
  __shared__ float2 cs[kTok][kAppendMaxPairs];
  __shared__ int tok_pos[kTok];            // position, or -1: nothing to do
  __shared__ long long k_row[kTok], v_row[kTok];  // element offset of the cache row, or -1: not stored
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * kTok;

  if (warp < kTok) {
    const int t = t0 + warp;
    int pos = -1;
    long long kr = -1, vr = -1;
    if (t < p.n_tok) {
      const int s = seq_of_token(p.seq_start, p.n_seq, t, lane);
      if (s >= 0) {
        const long long x = (long long)__ldg(p.seq_len + s) - ((long long)__ldg(p.seq_start + s + 1) - t);
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
    }
    if (lane == 0) {
      tok_pos[warp] = pos;
      k_row[warp] = kr;
      v_row[warp] = vr;
    }
  }
  __syncthreads();
  const int pairs = p.rot >> 1;
  for (int i = threadIdx.x; i < kTok * pairs; i += kAppendThreads) {
    const int j = i / pairs, pr = i - j * pairs;
    if (tok_pos[j] >= 0) {
      const double turn = (double)tok_pos[j] * p.turns[pr];
      float s, c;
      sincospif((float)(2.0 * (turn - rint(turn))), &s, &c);
      cs[j][pr] = make_float2(c, s);
    }
  }
  __syncthreads();

  const int heads = p.q_heads + 2 * p.kv_heads;
  const int per_tok = heads * kItems;
  const int rot_items = p.rot >> 4;
  for (int i = threadIdx.x; i < kTok * per_tok; i += kAppendThreads) {
    const int j = kTok == 1 ? 0 : i / per_tok;
    const int r = i - j * per_tok;
    if (tok_pos[j] < 0) continue;
    int h = r / kItems;
    const int it = r % kItems;
    const long long t = t0 + j;
    const bool is_q = h < p.q_heads;
    if (is_q && !p.q.ptr) continue;
    if (!is_q) h -= p.q_heads;
    const bool is_v = !is_q && h >= p.kv_heads;
    if (is_v) h -= p.kv_heads;
    const SeqView& in = is_q ? p.q : is_v ? p.v : p.k;
    const bool turned = !is_v && it < rot_items;
    const int c0 = (kHalves && it < rot_items) ? it : 2 * it;
    const int c1 = (kHalves && it < rot_items) ? it + rot_items : 2 * it + 1;
    const T* src = static_cast<const T*>(in.ptr) + h * in.sh + t * in.st;
    const uint4 w0 = reinterpret_cast<const uint4*>(src)[c0];  // plain loads: outputs may be the inputs
    const uint4 w1 = reinterpret_cast<const uint4*>(src)[c1];
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
          const float2 a = cs[j][it * 8 + e];
          const float lo = f[e], hi = f[8 + e];
          f[e] = fmaf(lo, a.x, -hi * a.y);
          f[8 + e] = fmaf(lo, a.y, hi * a.x);
        }
      } else {
        #pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 a = cs[j][it * 8 + e];
          const float lo = f[2 * e], hi = f[2 * e + 1];
          f[2 * e] = fmaf(lo, a.x, -hi * a.y);
          f[2 * e + 1] = fmaf(lo, a.y, hi * a.x);
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
      const long long row = is_v ? v_row[j] : k_row[j];
      if (row >= 0) {
        const long long at = row + h * (is_v ? p.c.vs[2] : p.c.ks[2]);
        void* base = is_v ? p.c.v : p.c.k;
        if constexpr (kF8) {
          const float scale = __ldg((is_v ? p.c.v_scale : p.c.k_scale) + h);
          uint32_t y[4];
          #pragma unroll
          for (int e = 0; e < 4; ++e)
            y[e] = pack_e4m3x2(f[4 * e] / scale, f[4 * e + 1] / scale) |
                   (pack_e4m3x2(f[4 * e + 2] / scale, f[4 * e + 3] / scale) << 16);
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
