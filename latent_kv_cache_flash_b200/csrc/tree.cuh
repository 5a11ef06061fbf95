// Device helpers of the tree calls: a sequence's drafted tokens and who sees them.
#pragma once

#include "common.cuh"

namespace gqla {

// The drafted tree of a tree call (gqla_tree).  on == 0: the sequence has s_q
// new tokens, which see each other causally.
struct TreeView {
  int32_t on;
  const uint64_t* masks;   // [batch, s_q] (decode calls)
  const int32_t* sizes;    // [batch] or nullptr: s_q each
};

__host__ __device__ __forceinline__ uint64_t low_bits(int n) { return n >= 64 ? ~0ull : (1ull << n) - 1; }

// A sequence's new tokens: n of them, the newest of its L tokens, after
// `base` tokens of context that every new token sees.  L = -1 (flagged): the
// sequence's rows must be skipped.
struct NewTokens {
  int L, n, base;
};

__device__ __forceinline__ NewTokens new_tokens(const KvLayout& ly, const TreeView& tr, int b, int s_q, int32_t* st) {
  NewTokens nt;
  if (!tr.on) {
    nt.L = seq_len_checked(ly, b, s_q, st);
    nt.n = s_q;
  } else {
    nt.L = ly.seq_lens[b];
    nt.n = tr.sizes ? tr.sizes[b] : s_q;
    int bits = 0;
    if (nt.n < 0 || nt.n > s_q) bits = GQLA_DEV_BAD_TREE;
    else if (nt.L < nt.n) bits = GQLA_DEV_SHORT_SEQ;
    else if (nt.L > ly.max_seq_len ||
             (ly.page_size == 0 ? nt.L > ly.capacity : nt.L > 0 && (nt.L - 1) / ly.page_size >= ly.mbps))
      bits = GQLA_DEV_OVERFLOW;
    if (bits) {
      flag_status(st, bits);
      nt.L = -1;
      nt.n = 0;
    }
  }
  nt.base = nt.L - nt.n;
  return nt;
}

// New tokens that new token i of sequence b sees (bit j: the j-th), i < nt.n.
__device__ __forceinline__ uint64_t new_mask(const TreeView& tr, const NewTokens& nt, int b, int s_q, int i) {
  return tr.masks[(long long)b * s_q + i] & low_bits(nt.n);
}

// New tokens that at least one of the sequence's new tokens sees.  All 32
// lanes of a warp call it.
__device__ __forceinline__ uint64_t new_union(const TreeView& tr, const NewTokens& nt, int b, int s_q) {
  uint64_t u = 0;
  for (int i = threadIdx.x & 31; i < nt.n; i += 32) u |= tr.masks[(long long)b * s_q + i];
  const uint32_t lo = __reduce_or_sync(0xffffffffu, (uint32_t)u), hi = __reduce_or_sync(0xffffffffu, (uint32_t)(u >> 32));
  return (((uint64_t)hi << 32) | lo) & low_bits(nt.n);
}

// Tokens t0 .. t0 + 63 seen by a row (bit t - t0) that sees the context and
// the new tokens of `mask`.
__device__ __forceinline__ uint64_t seen_word(uint64_t mask, int base, int t0) {
  const int d = base - t0;
  if (d >= 64) return ~0ull;
  if (d >= 0) return (mask << d) | low_bits(d);
  return d > -64 ? mask >> -d : 0ull;
}

}  // namespace gqla
