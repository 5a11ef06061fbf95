// How the tensor-core tree kernels share a batch's work.
//
// A unit is one block of `row_block` (drafted token, head) rows of one
// sequence (and group); it costs one step per tile of `tile` tokens of that
// sequence.  Laid end to end (sequence, group, row block, tile) the steps form
// one list, whose equal contiguous shares go to the workers (a CTA or a pair
// of CTAs): lengths and tree sizes are known on the device only, and a share
// of the list is the same work whatever they are.  A split of the longest
// length instead leaves the workers of short sequences idle (16 sequences of
// 1000..8000 tokens, 32 heads in 8 groups: 146 us so, 82 shared out).  A worker
// whose share starts or ends inside a unit writes a partial result (at most
// two), which the merge pass joins.
#pragma once

#include "tree.cuh"

namespace gqla {

struct TreeWork {
  int groups;      // units of a row block: groups (expanded cache), 1 (latent cache)
  int m;           // rows of a drafted token in a unit's group
  int row_block;
  int tile;
  int unit_tiles;  // what one more unit costs a worker in starts and results, in tiles
  int workers;
  int s_q;
};

struct SeqWork {
  NewTokens nt;
  int rblocks, tiles;
  long long items;
  __device__ __forceinline__ int units(const TreeWork& w) const { return tiles > 0 ? w.groups * rblocks : 0; }
};

__device__ __forceinline__ SeqWork seq_work(const TreeWork& w, const KvLayout& ly, const TreeView& tr, int b,
                                            int32_t* st) {
  SeqWork s;
  s.nt = new_tokens(ly, tr, b, w.s_q, st);
  s.rblocks = (s.nt.n * w.m + w.row_block - 1) / w.row_block;
  s.tiles = s.nt.L > 0 ? (s.nt.L + w.tile - 1) / w.tile : 0;
  s.items = (long long)w.groups * s.rblocks * s.tiles;
  return s;
}

// How many shares a list of `total` tiles in `units` units, the longest of
// `longest` tiles, is cut into: a tile each where there are workers enough; else
// one for each worker.  Or, where all units are of one length, as many to each
// unit, so that a worker has a part of one of them, if the tiles that this adds
// to a share cost less than a second unit does (9 sequences of 146 tokens, 72
// units of 3 tiles over 148 SMs, expanded: 19.9 us a call with 148 shares, 17.1
// with 144).
__device__ __forceinline__ long long shares_used(const TreeWork& w, long long total, int units, int longest) {
  if (total <= w.workers) return total < 1 ? 1 : total;
  if (units > w.workers || (long long)units * longest != total) return w.workers;
  const int k = w.workers / units;
  const long long even = (long long)units * (k < longest ? k : longest);
  return total * (w.workers - even) <= (long long)w.unit_tiles * even * w.workers ? even : w.workers;
}
__device__ __forceinline__ long long share_begin(long long i, long long total, long long shares) {
  return (i * total) >> 32 ? i * total / shares : (uint32_t)(i * total) / (uint32_t)shares;
}
// The share that holds item x: the last one that begins at or before it.
__device__ __forceinline__ long long share_of(long long x, long long total, long long shares) {
  const long long n = (x + 1) * shares + total - 1;
  return (n >> 32 ? n / total : (uint32_t)n / (uint32_t)total) - 1;
}

// One unit's part of a share: tiles tile0 .. tile0 + n - 1.
struct TreeSegment {
  int b, g, rb;
  NewTokens nt;
  int tile0, n, tiles;
};

// Walks the segments of one share: `s` is the work of sequence b, whose first
// item has list position `first`, at or before `at`.
struct SegmentWalk {
  int b;
  long long first, at, hi;
  SeqWork s;
  __device__ __forceinline__ bool next(const TreeWork& w, const KvLayout& ly, const TreeView& tr, TreeSegment* o) {
    if (at >= hi) return false;
    while (at >= first + s.items) {      // ends: at < hi <= the list's length
      first += s.items;
      s = seq_work(w, ly, tr, ++b, nullptr);
    }
    const long long local = at - first;
    int unit;
    if (local >> 32) {
      unit = (int)(local / s.tiles);
      o->tile0 = (int)(local % s.tiles);
    } else {
      unit = (int)((uint32_t)local / (uint32_t)s.tiles);
      o->tile0 = (int)((uint32_t)local % (uint32_t)s.tiles);
    }
    o->b = b;
    o->g = unit / s.rblocks;
    o->rb = unit % s.rblocks;
    o->nt = s.nt;
    o->tiles = s.tiles;
    const long long left = hi - at;
    o->n = left < s.tiles - o->tile0 ? (int)left : s.tiles - o->tile0;
    at += o->n;
    return true;
  }
};

// The next segment, for all lanes of a warp; `walk` and `out` are in shared memory.
struct SharedSegment {
  TreeSegment seg;
  int has;
};
__device__ __forceinline__ bool warp_next(SegmentWalk& walk, SharedSegment& out, const TreeWork& w, const KvLayout& ly,
                                          const TreeView& tr, TreeSegment* o) {
  if ((threadIdx.x & 31) == 0) out.has = walk.next(w, ly, tr, &out.seg);
  __syncwarp();
  *o = out.seg;
  const bool has = out.has;
  __syncwarp();
  return has;
}

// Block-wide: kWalks walkers of worker `id`'s share, readable after the next
// block barrier.  Worker 0 (`writes`) also writes the list position of every
// sequence's first item (prefix[batch]: the list's length, then the shares) and
// the sequences' status bits.  One warp does it, 32 sequences at a time: for a small batch
// that is one round of loads, and a kernel's first pass through its code is
// bound by fetching it (block-wide scans took 2500 cycles more).
template <int kWalks>
__device__ __forceinline__ void share_start(const TreeWork& w, const KvLayout& ly, const TreeView& tr, int id,
                                            bool writes, long long* prefix, int32_t* st, SegmentWalk* walks) {
  const int lane = threadIdx.x & 31;
  SeqWork mine;
  mine.items = 0;
  if (lane < ly.batch) mine = seq_work(w, ly, tr, lane, writes ? st : nullptr);
  long long total = mine.items;
  int units = lane < ly.batch ? mine.units(w) : 0, longest = units ? mine.tiles : 0;
#pragma unroll 4
  for (int b = lane + 32; b < ly.batch; b += 32) {
    const SeqWork s = seq_work(w, ly, tr, b, writes ? st : nullptr);
    total += s.items;
    units += s.units(w);
    if (s.units(w)) longest = max(longest, s.tiles);
  }
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const long long shares = shares_used(w, total, __reduce_add_sync(0xffffffffu, units), __reduce_max_sync(0xffffffffu, longest));
  const long long lo = id < shares ? share_begin(id, total, shares) : total;
  const long long hi = id < shares ? share_begin(id + 1, total, shares) : total;
  if (lane < kWalks) walks[lane].at = walks[lane].hi = 0;
  __syncwarp();
  long long base = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < ly.batch; b0 += 32) {
    const int b = b0 + lane;
    if (b0 > 0) {
      mine.items = 0;
      if (b < ly.batch) mine = seq_work(w, ly, tr, b, nullptr);
    }
    long long inc = mine.items;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    const long long first = base + inc - mine.items;
    if (lo < hi && first <= lo && lo < first + mine.items) {
#pragma unroll 1
      for (int i = 0; i < kWalks; ++i) walks[i] = SegmentWalk{b, first, lo, hi, mine};
    }
    if (writes && b < ly.batch) prefix[b] = first;
    base += __shfl_sync(0xffffffffu, inc, 31);
    if (!writes && base > lo) break;
  }
  if (writes && lane == 0) {
    prefix[ly.batch] = total;
    prefix[ly.batch + 1] = shares;
  }
  __syncwarp();
}

// A worker's two partial results: slot 0 of a unit begun by an earlier worker,
// slot 1 of one it begins and leaves to the next.  So the parts of a unit of
// items u0 .. u0 + tiles - 1 are slot 1 of share_of(u0) and slot 0 of every
// worker after it up to share_of(u0 + tiles - 1); with both the same worker
// the unit is whole and was written to the output.
__device__ __forceinline__ long long part_slot(long long worker, bool begins) { return 2 * worker + (begins ? 1 : 0); }

// The log-sum-exp of a part that met a bad page, whose row is zeros.  A NaN of
// its own: arithmetic gives the one with all bits set, which stands for rows
// with a score of NaN or +inf.
__device__ __forceinline__ float bad_part() { return __uint_as_float(0x7fc00bad); }
__device__ __forceinline__ bool is_bad_part(float lse) { return __float_as_uint(lse) == 0x7fc00bad; }

// The batch's list as the merge needs it, in a warp's lanes: lane b has sequence
// b's.  With up to 32 sequences it needs the lengths only, which the attention
// kernel does not write: the merge then makes it, and fetches its code, while
// that kernel still runs.
struct TreeList {
  long long first, total, shares;
  int n, rblocks, tiles;
};

__device__ __forceinline__ bool parts_known_early(const KvLayout& ly) { return ly.batch <= 32; }

__device__ __forceinline__ TreeList tree_list(const TreeWork& w, const KvLayout& ly, const TreeView& tr) {
  const int lane = threadIdx.x & 31;
  SeqWork s{};
  if (lane < ly.batch) s = seq_work(w, ly, tr, lane, nullptr);
  long long inc = s.items;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  const long long total = __shfl_sync(0xffffffffu, inc, 31);
  const int units = lane < ly.batch ? s.units(w) : 0;
  const long long shares = shares_used(w, total, __reduce_add_sync(0xffffffffu, units),
                                       __reduce_max_sync(0xffffffffu, units ? s.tiles : 0));
  return TreeList{inc - s.items, total, shares, s.nt.n, s.rblocks, s.tiles};
}

// Where a row of sequence b stands for the merge: its row block, and the workers
// that hold its unit's parts.  For a warp.
struct RowParts {
  int rb;              // row block
  long long first;     // the workers first .. first + n - 1; n = 0: a row without a unit
  int n;
};

__device__ __forceinline__ RowParts row_parts(const TreeWork& w, const KvLayout& ly, const TreeView& tr,
                                              const TreeList& list, int b, int group, int row, const long long* prefix) {
  TreeList s;
  if (parts_known_early(ly)) {
    s.total = list.total;
    s.shares = list.shares;
    s.first = __shfl_sync(0xffffffffu, list.first, b);
    s.n = __shfl_sync(0xffffffffu, list.n, b);
    s.rblocks = __shfl_sync(0xffffffffu, list.rblocks, b);
    s.tiles = __shfl_sync(0xffffffffu, list.tiles, b);
  } else {
    const SeqWork q = seq_work(w, ly, tr, b, nullptr);
    s = TreeList{prefix[b], prefix[ly.batch], prefix[ly.batch + 1], q.nt.n, q.rblocks, q.tiles};
  }
  RowParts r;
  r.rb = row / w.row_block;
  r.first = 0;
  r.n = 0;
  if (row < s.n * w.m && s.tiles > 0) {
    const long long u0 = s.first + (long long)(group * s.rblocks + r.rb) * s.tiles;
    r.first = share_of(u0, s.total, s.shares);
    r.n = (int)(share_of(u0 + s.tiles - 1, s.total, s.shares) - r.first) + 1;
  }
  return r;
}

}  // namespace gqla
