// What the token-sequence operators share: element types, the description of a packed batch and of
// a paged key/value cache, and the checks that kernels make of indexes held in device memory.
//
// A packed batch holds the tokens of all its sequences one after another along the token axis;
// sequence s has the tokens [seq_start[s], seq_start[s + 1]). Offsets, lengths and page numbers live
// in device memory, so a captured graph can be replayed with others; the host cannot check them.
// Every kernel therefore checks each one before it is used as an address: a bad one is skipped and
// recorded in a device error word of its own (kDevBadIndex, reported by clear_attn_check()).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sm100_ptx.cuh"

namespace clear {

// Sites of recorded bad indexes (second word of the diagnosis record).
enum SeqSite : int { kSiteAppendPage = 32, kSiteDecodePage = 33, kSiteSeqStart = 34, kSiteSeqLen = 35 };

// Records a length, offset or page number out of range: the first one wins.
__device__ __noinline__ void record_bad_index(int site, int c0, int c1, int c2) {
  if (atomicCAS(&g_clear_device_error[kDevIndex], 0, (int)kDevBadIndex) == 0) {
    int* const diag = g_clear_device_diag[kDevIndex];
    diag[0] = kDevBadIndex;
    diag[1] = site;
    diag[2] = blockIdx.x;
    diag[3] = threadIdx.x;
    diag[4] = 0;
    diag[5] = c0;
    diag[6] = c1;
    diag[7] = c2;
    __threadfence();
  }
}

// A bounded wait like mbar_wait, for waits that are short and many: the timer, a slow read, is first looked at
// after some polls.
__device__ __forceinline__ bool seq_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int err_code, int site,
                                         int c0 = 0, int c1 = 0) {
  const uint32_t a = smem_u32(bar);
  uint64_t t0 = 0;
  for (uint32_t spins = 1;; ++spins) {
    if (mbar_try_wait(a, parity)) return true;
    if ((spins & 63u) == 0) {
      if (*abort_flag) return false;
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > kWaitLimitNs) {
        record_timeout(abort_flag, err_code, site, (int)parity, c0, c1, (int)(a & 0xffff));
        return false;
      }
    }
  }
}

// The same for a whole warp: every lane returns the same, so that a warp leaves its loop together.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int err_code, int site,
                                          int c0 = 0, int c1 = 0) {
  return __all_sync(0xffffffffu, seq_wait(bar, parity, abort_flag, err_code, site, c0, c1));
}

// One arrival for the whole warp, behind its tensor-memory accesses so far (which the caller has waited for).
__device__ __forceinline__ void warp_arrive_tc(uint64_t* bar) {
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// After an expired wait: waits, again with a limit, for a copy or product still in flight, whatever
// the abort flag says, so that nothing writes shared or tensor memory after the block has left.
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_test(bar, parity) && globaltimer_ns() - t0 < kWaitLimitNs) __nanosleep(100);
}

// 16-bit element types: one pair per 32-bit register, the lower half first.
//
// kLift: probabilities relative to the maximum in use, which may be 2^8 below the true one, are held times 2^kLift.
// bf16 has fp32's exponents: each is rounded by half a step, 2^-8 of itself at most, however small. fp16's steps are absolute below
// 2^-14: plain probabilities would be off by up to 2^-25 of the largest key's weight each, all with one sign where many keys are
// alike. Times 2^7 they stay below 2^15, half a step is 2^-11 of each down to 2^-21 of the largest weight, and an
// absolute 2^-32 of it below: 2^-15 in all from 131072 keys.
struct Bf16 {
  using type = __nv_bfloat16;
  static constexpr float kLift = 0.f;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_bf16x2(lo, hi); }
  static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
};
struct Fp16 {
  using type = __half;
  static constexpr float kLift = 7.f;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ float lo(uint32_t w) {
    return __half2float(__ushort_as_half((unsigned short)(w & 0xffffu)));
  }
  static __device__ __forceinline__ float hi(uint32_t w) {
    return __half2float(__ushort_as_half((unsigned short)(w >> 16)));
  }
};

// Two fp32 values as two E4M3 codes (round to nearest even, magnitudes above 448 saturate, NaN stays).
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Division of a non-negative int by a fixed positive int without a divide: for d not a power of
// two, with shift = ceil(log2 d) and mul = floor(2^(31 + shift) / d) + 1, n / d = (n * mul) >>
// (31 + shift) for every 0 <= n < 2^31: mul exceeds 2^(31 + shift) / d by e <= 1, so the quotient
// is off by at most n * e / 2^(31 + shift) < 2^-shift <= 1 / d, too little to reach the next
// integer. mul < 2^32, since d > 2^(shift - 1). A power of two is a plain shift.
struct FastDiv {
  uint32_t d, mul, shift;
  __device__ __forceinline__ int div(int n) const {
    if (mul == 0) return n >> shift;
    return (int)(((uint64_t)(uint32_t)n * mul) >> (31 + shift));
  }
};
inline FastDiv make_fast_div(int d) {
  FastDiv f{(uint32_t)d, 0, 0};
  while ((1ull << f.shift) < (unsigned)d) ++f.shift;
  if ((1ull << f.shift) != (unsigned)d) f.mul = (uint32_t)((1ull << (31 + f.shift)) / (unsigned)d + 1);
  return f;
}

// Base address and element strides of a [heads, tokens, d] view (d contiguous).
struct SeqView {
  void* ptr;
  long long sh, st;
};

// A paged cache: token p of a sequence lies in row p % page_size of page table[seq][p / page_size].
struct SeqCache {
  void *k, *v;
  long long ks[3], vs[3];  // element strides {page, token, head}; d contiguous
  const int* table;        // [n_seq][table_stride]
  long long table_stride;
  int max_pages, n_pages, page_size;
  FastDiv page_div;
  const float *k_scale, *v_scale;  // E4M3 caches: one dequantisation scale per kv head
};

}  // namespace clear
