// The order of one item's products in the causal prompt forward, and the waits that this order asks of the softmax
// warpgroups. Plain C++: the kernel and the host-side check of its barriers use the same functions.
//
// An item has nA key tiles for query tile A (or, with split keys, its even ones) and nB for query tile B (its odd ones).
// Their tiles of S are numbered g = 0, 1, ... in the order A0, B0, A1, B1, ..., and use the buffers of S in turn. The
// products run in the order in which they are issued: S of the tiles with first(g), then, for each g, P V of g and one
// further S.
#pragma once

#if defined(__CUDACC__)
#define CLEAR_ORDER_HD __host__ __device__ __forceinline__
#else
#define CLEAR_ORDER_HD inline
#endif

namespace clear {

template <int kBufs, bool kSplit>
struct PromptOrder {
  int nA, nB;  // tiles of each; nB = 0: no tile B

  // Place in the order of key tile i of query tile `half` (split keys: of the half's i-th key tile).
  CLEAR_ORDER_HD int place(int half, int i) const {
    if (kSplit) return 2 * i + half;
    return nB == 0 ? i : i < nA ? 2 * i + half : 2 * nA;  // tile B has one key tile more
  }
  // With two buffers, a query tile that is alone has S of tile g + 1 issued behind P V of g and not of g - 1.
  CLEAR_ORDER_HD bool alone() const { return kBufs == 2 && !kSplit && nB == 0; }
  // Whether S of tile g is issued before any P V.
  CLEAR_ORDER_HD bool first(int g) const { return g < kBufs && !(alone() && g > 0); }
  // A wait by parity must be neither two phases ahead of its barrier nor one behind it. S of a tile that is issued behind
  // the last P V of its own query tile tells that this P V is done. Where it does not, the warpgroup looks at that P V's
  // barrier before it hands over the second half of P, while the next one cannot be done: with three buffers
  // always; with two, where S of tile g is behind P V of g - 2 (of g - 1 if it is alone), only tile B's last key tile, whose place
  // follows tile B's last but one directly.
  CLEAR_ORDER_HD bool looks_back(int half, int i) const {
    return kBufs == 3 ? i > 0 : !kSplit && nB > 0 && half == 1 && i == nA;
  }
  // Which copy of the halves' exchanged (m, l) an item uses, `joins` items with an exchange lying before it. A half without a key
  // tile waits for nothing between two items, so it may write while the other half still reads the last item's
  // sums. It is held at the next exchange's barrier, though: with two copies the one it writes has been read.
  CLEAR_ORDER_HD int sums(unsigned joins) const { return (int)(joins & 1u); }
};

}  // namespace clear
