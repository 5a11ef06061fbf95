// The steps of tree decoding around the attention: masks of a drafted tree,
// verification of its tokens against the target's probabilities, and the move
// of the accepted path's cache rows to their final slots.
#include <cooperative_groups.h>
#include <math.h>

#include "pair.cuh"
#include "tree.h"

namespace gqla {

namespace cg = cooperative_groups;

namespace {

constexpr int kMaxTree = GQLA_MAX_TREE;

// ------------------------------------------------------------------ masks
// One CTA per sequence, one thread per token: a token's mask is the walk to
// its root, at most n_tokens steps through shared memory.
__global__ void __launch_bounds__(kMaxTree) tree_masks_kernel(int n_tokens, const int32_t* __restrict__ parents,
                                                              const int32_t* __restrict__ sizes,
                                                              uint64_t* __restrict__ masks, int32_t* st) {
  ptx::pdl_wait();
  ptx::pdl_trigger();
  __shared__ int up[kMaxTree];
  const int b = blockIdx.x, i = threadIdx.x;
  int n = sizes ? sizes[b] : n_tokens;
  if (n < 0 || n > n_tokens) {
    if (i == 0) flag_status(st, GQLA_DEV_BAD_TREE);
    n = 0;
  }
  if (i < n) {
    int p = parents[(long long)b * n_tokens + i];
    if (p < -1 || p >= i) {
      flag_status(st, GQLA_DEV_BAD_TREE);
      p = -2;
    }
    up[i] = p;
  }
  __syncthreads();
  if (i >= n_tokens) return;
  uint64_t m = 0;
  int a = i < n ? i : -1;
  while (a >= 0) {               // parents come before their children, so this ends
    m |= 1ull << a;
    a = up[a];
  }
  masks[(long long)b * n_tokens + i] = a == -2 ? 0 : m;
}

// ----------------------------------------------------------------- verify
// After k refusals at a token, the weights are
//     w_k(v) = max(p(v) - A_k q(v), 0),   A_k = Z_0 + ... + Z_{k-1},
// since max(max(p - a q, 0) - z q, 0) = max(p - (a + z) q, 0) for q >= 0: one
// scalar stands for the whole residual, and nothing of vocabulary size is
// kept.  Everything a test needs but Z is single elements, which are gathered
// for all drafted tokens up front; the rows are streamed once per refusal
// (Z_k = sum_v w_k(v)) and once for the draw when the path ends in a leaf.
//
// A cluster of C CTAs serves a sequence.  The row is cut into C * kVWarps
// contiguous ranges, one per warp; each pass leaves the ranges' sums in every
// CTA's shared memory, which everyone adds in the same order, so all take the
// same decisions and the result does not depend on timing.  The draw
// finds the range by those sums, and one warp scans that range again.
// Sums are in 64 bits: the rows have up to some 10^5 terms, and a draw next to
// a border must not depend on how they are grouped.
// Bound by the passes' latencies, one after the other (loads, 64-bit sums, the
// exchange: about 2 us each).  64 trees of 24 over 128000 fp32: 49..52 us, of
// which the rows' bytes would take 10; 16 of 16 over 100003 bf16: 19.5..21.6; one
// of 6 over 32000: 6.4..6.8 (several boxes and seeds).  Where rows of target and
// draft lie differently to 16-byte boundaries a residual's sums go element by
// element: 62 for 50 us, 23.9 for 19.8.
constexpr int kVWarps = 16;
constexpr int kVThreads = kVWarps * 32;
constexpr int kMaxCluster = 8;
constexpr int kVUnroll = 3;      // 16-byte loads of each row in flight a lane: 96 KB an SM with two CTAs on it
constexpr int kVKeep = 8;        // 16-byte groups of each row that a lane can hold

struct VerifyParams {
  int n_tokens, vocab;
  const int32_t* parents;
  const int32_t* sizes;
  const int32_t* tokens;
  const void* target;
  const void* draft;
  long long tp, dp;      // pitches in elements
  const float* u_accept;
  const float* u_sample;
  int32_t* accepted;
  int32_t* n_accepted;
  int32_t* next_token;
  int32_t* st;
};

// A probability: negative and NaN count as 0.
__device__ __forceinline__ float prob(float x) { return x > 0.f ? x : 0.f; }

template <typename T>
struct Row {
  static constexpr int kVec = 16 / sizeof(T);
  const T* p;            // element 0
  int off;               // elements between the 16-byte boundary at or below p, and p
  __device__ Row(const T* base) : p(base), off((int)(((uintptr_t)base & 15) / sizeof(T))) {}
  __device__ int groups(int V) const { return (off + V + kVec - 1) / kVec; }
  // 16-byte groups wholly inside the row
  __device__ int inner_begin() const { return off ? 1 : 0; }
  __device__ int inner_end(int V) const { return (off + V) / kVec; }
  __device__ uint4 raw(int g) const { return __ldg(reinterpret_cast<const uint4*>(p - off) + g); }
  // elements of 16-byte group g, out of range ones as 0; first element's index
  __device__ int load(int g, int V, float* x) const {
    const int v0 = g * kVec - off;
    if (v0 >= 0 && v0 + kVec <= V) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(p + v0));
      const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int k = 0; k < kVec; ++k) x[k] = prob(to_f32(e[k]));
    } else {
      scalar(v0, V, x);
    }
    return v0;
  }
  __device__ void scalar(int v0, int V, float* x) const {
#pragma unroll
    for (int k = 0; k < kVec; ++k) x[k] = v0 + k >= 0 && v0 + k < V ? prob(to_f32(p[v0 + k])) : 0.f;
  }
  // the elements from v0 on, where v0 is the start of a group of another row
  __device__ void load_from(int v0, int V, float* x) const {
    if (v0 >= 0 && v0 + kVec <= V && ((v0 + off) & (kVec - 1)) == 0) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(p + v0));
      const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int k = 0; k < kVec; ++k) x[k] = prob(to_f32(e[k]));
    } else {
      scalar(v0, V, x);
    }
  }
};

// The weights at one token of the tree.
template <typename T, bool POINT>
struct Weights {
  Row<T> p, q;
  double A;              // of the rows' residual (POINT: unused)
  const int* out;        // POINT: tokens refused here
  int n_out;
  __device__ Weights(const T* pr, const T* qr) : p(pr), q(qr), A(0.0), out(nullptr), n_out(0) {}
  // weights of group g of p, kVec of them; index of the first
  __device__ int load(int g, int V, double* w) const {
    constexpr int kVec = Row<T>::kVec;
    float x[kVec], y[kVec];
    const int v0 = p.load(g, V, x);
    if constexpr (POINT) {
#pragma unroll
      for (int k = 0; k < kVec; ++k) w[k] = x[k];
      for (int o = 0; o < n_out; ++o)
#pragma unroll
        for (int k = 0; k < kVec; ++k)
          if (out[o] == v0 + k) w[k] = 0.0;
    } else if (A == 0.0) {
#pragma unroll
      for (int k = 0; k < kVec; ++k) w[k] = x[k];
    } else {
      q.load_from(v0, V, y);
#pragma unroll
      for (int k = 0; k < kVec; ++k) {
        const double d = fma(-A, (double)y[k], (double)x[k]);
        w[k] = d > 0.0 ? d : 0.0;
      }
    }
    return v0;
  }
};

// The weights of whole 16-byte groups, summed.  Conversions from 32 to 64 bits
// run at 16 a cycle an SM, a quarter of the rate of 64-bit arithmetic, and with
// two of them a weight a pass of 2 x 128000 fp32 over 8 CTAs took 5.0 us from
// L2.  Done on the bits, and with negative values, NaN and all from 2 on looked
// for in the OR of the words (bits 31 and 30), a weight is about 9 instructions.
// On the bits a zero or a subnormal becomes up to 2^-126, which cannot matter to
// a sum above 1e-25 (A >= 1: without a probability there is no weight either).
// A smaller sum, or one with such a value in it, is taken again with conversions.
template <typename T>
struct FastSum {
  double s;
  uint32_t any;        // OR of the words
  __device__ __forceinline__ FastSum() : s(0.0), any(0) {}
  // element k of a group as a double, for values in [0, 2)
  static __device__ __forceinline__ double widen(const uint4& w, int k) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(&w);
    if (sizeof(T) == 4) return __hiloint2double((int)((u[k] >> 3) | 0x38000000u), (int)(u[k] << 29));
    const uint32_t x = u[k >> 1];
    return __hiloint2double((int)(((k & 1 ? x >> 3 : x << 13) & 0x1fffe000u) | 0x38000000u), 0);
  }
  __device__ __forceinline__ void add(const uint4& pw, const uint4& qw, double minus_a, bool residual) {
    any |= pw.x | pw.y | pw.z | pw.w;
    if (!residual) {
#pragma unroll
      for (int k = 0; k < 16 / (int)sizeof(T); ++k) s += widen(pw, k);
    } else {
      any |= qw.x | qw.y | qw.z | qw.w;
#pragma unroll
      for (int k = 0; k < 16 / (int)sizeof(T); ++k) {
        const double d = fma(minus_a, widen(qw, k), widen(pw, k));
        if (__double2hiint(d) >= 0) s += d;
      }
    }
  }
  __device__ __forceinline__ double value() const { return any ? s : 0.0; }
  __device__ __forceinline__ bool careful() const {
    return (any & (sizeof(T) == 4 ? 0xc0000000u : 0xc000c000u)) || (any && s > 0.0 && s < 1e-25);
  }
};

__device__ __forceinline__ double warp_sum_f64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A value into shared memory of a CTA of the cluster, counted by a barrier there.
// A cluster barrier a pass, whose release waits for all of a thread's writes, in
// its place: 52.4 us for 49.4 (64 x 128000 fp32), 20.7 for 19.5 (16 x 100003 bf16).
__device__ __forceinline__ void send_f64(uint32_t at, double v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(at),
               "l"(__double_as_longlong(v)), "r"(bar)
               : "memory");
}

// KEEP: a lane holds its part of the token's rows in registers from the first
// pass on, up to kVKeep 16-byte groups of each.
template <typename T, bool POINT, bool KEEP>
__global__ void __launch_bounds__(kVThreads, KEEP ? 1 : 2) verify_kernel(const VerifyParams p) {
  ptx::pdl_wait();
  ptx::pdl_trigger();
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int b = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int V = p.vocab;
  __shared__ double s_p[kMaxTree], s_q[kMaxTree];        // each token's probability after its parent
  __shared__ float s_u[kMaxTree];
  __shared__ int s_tok[kMaxTree], s_out[kMaxTree];
  __shared__ unsigned long long s_kids[kMaxTree];
  __shared__ double s_sum[2][kMaxCluster * kVWarps];     // range sums of the last passes
  __shared__ __align__(8) uint64_t s_bar[2];             // all of them have come
  const T* target = (const T*)p.target + (long long)b * p.n_tokens * p.tp;
  const T* draft = (const T*)p.draft + (long long)b * p.n_tokens * p.dp;

  int n = p.sizes ? p.sizes[b] : p.n_tokens;
  if (n < 0 || n > p.n_tokens) {
    if (tid == 0 && rank == 0) flag_status(p.st, GQLA_DEV_BAD_TREE);
    n = 0;
  }
  if (tid < kMaxTree) s_kids[tid] = 0;
  if (tid == 0) {
    ptx::mbar_init(&s_bar[0], 1);
    ptx::mbar_init(&s_bar[1], 1);
    ptx::fence_barrier_init();
  }
  cluster.sync();               // every CTA of the cluster runs: its shared memory may be written
  if (tid >= 1 && tid < n) {
    const long long at = (long long)b * p.n_tokens + tid;
    const int up = p.parents[at], x = p.tokens[at];
    s_tok[tid] = x;
    s_u[tid] = p.u_accept[at];
    if (up < 0 || up >= tid || x < 0 || x >= V) {
      if (rank == 0) flag_status(p.st, GQLA_DEV_BAD_TREE);
    } else {
      s_p[tid] = prob(to_f32(target[up * p.tp + x]));
      if (!POINT) s_q[tid] = prob(to_f32(draft[up * p.dp + x]));
      atomicOr(&s_kids[up], 1ull << tid);
    }
  }
  __syncthreads();
  int32_t* path = p.accepted + (long long)b * p.n_tokens;
  if (n == 0) {                 // the whole cluster takes this way
    if (rank == 0 && tid < p.n_tokens) path[tid] = -1;
    if (rank == 0 && tid == 0) {
      p.n_accepted[b] = 0;
      p.next_token[b] = -1;
    }
    return;
  }

  // One pass over the row: every range's sum into every CTA's s_sum[buf].
  int buf = 0;
  uint32_t passes = 0;
  bool ok = true;
  uint4 held_p[KEEP ? kVKeep : 1], held_q[KEEP && !POINT ? kVKeep : 1];
  const T* held = nullptr;      // the row of p that they are of
  auto pass = [&](const Weights<T, POINT>& w) {
    constexpr int kVec = Row<T>::kVec;
    buf ^= 1;
    if (tid == 0) ptx::mbar_arrive_expect_tx(&s_bar[buf], C * kVWarps * 8);
    const int groups = w.p.groups(V), per = (groups + C * kVWarps - 1) / (C * kVWarps);
    const int range = rank * kVWarps + warp;
    const int g1 = min(groups, (range + 1) * per);
    double acc = 0.0;
    FastSum<T> fast;
    const int g = range * per;
    // groups that need care one by one: the row's ends, rows of p and q that
    // do not share their alignment, a range that holds a refused token
    bool plain = POINT || w.A == 0.0 || w.p.off == w.q.off;
    if constexpr (POINT) {
      const int v0 = g * kVec - w.p.off, v1 = g1 * kVec - w.p.off;
      for (int o = 0; o < w.n_out; ++o) plain &= w.out[o] < v0 || w.out[o] >= v1;
    }
    const int in0 = plain ? max(g, w.p.inner_begin()) : g1, in1 = plain ? min(g1, w.p.inner_end(V)) : g1;
    for (int k = g + lane; k < min(in0, g1); k += 32) {
      double x[kVec];
      w.load(k, V, x);
#pragma unroll
      for (int e = 0; e < kVec; ++e) acc += x[e];
    }
    const bool residual = !POINT && w.A != 0.0;
    if constexpr (KEEP) {
      // the range's whole groups, whether or not this pass takes them one by one
      const int h0 = max(g, w.p.inner_begin()), h1 = min(g1, w.p.inner_end(V));
      const bool both = !POINT && w.p.off == w.q.off;
      if (held != w.p.p) {
        held = w.p.p;
#pragma unroll
        for (int u = 0; u < kVKeep; ++u) {
          const bool in = h0 + 32 * u + lane < h1;       // groups past the range are zeros
          held_p[u] = in ? w.p.raw(h0 + 32 * u + lane) : make_uint4(0, 0, 0, 0);
          if (!POINT) held_q[u] = in && both && residual ? w.q.raw(h0 + 32 * u + lane) : make_uint4(0, 0, 0, 0);
        }
      }
#pragma unroll
      for (int u = 0; u < kVKeep; ++u)
        if (in0 + 32 * u < in1) fast.add(held_p[u], held_q[POINT ? 0 : u], -w.A, residual);
    }
    for (int k = KEEP ? in1 : in0 + lane; k < in1; k += 32 * kVUnroll) {
      uint4 x[kVUnroll], y[kVUnroll];
#pragma unroll
      for (int u = 0; u < kVUnroll; ++u) {
        // groups past the range are zeros
        x[u] = y[u] = make_uint4(0, 0, 0, 0);
        if (k + 32 * u < in1) {
          x[u] = w.p.raw(k + 32 * u);
          if (residual) y[u] = w.q.raw(k + 32 * u);
        }
      }
#pragma unroll
      for (int u = 0; u < kVUnroll; ++u)
        if (k - lane + 32 * u < in1) fast.add(x[u], y[u], -w.A, residual);
    }
    if (fast.careful()) {
      for (int k = in0 + lane; k < in1; k += 32) {
        double x[kVec];
        w.load(k, V, x);
#pragma unroll
        for (int e = 0; e < kVec; ++e) acc += x[e];
      }
    } else {
      acc += fast.value();
    }
    for (int k = max(in1, in0) + lane; k < g1; k += 32) {
      double x[kVec];
      w.load(k, V, x);
#pragma unroll
      for (int e = 0; e < kVec; ++e) acc += x[e];
    }
    const double sum = warp_sum_f64(acc);
    // A CTA's sums of the pass after the next cannot come before all its warps
    // have sent the next one's, and so have read these.
    if (lane < C) send_f64(pairx::at_rank(&s_sum[buf][range], lane), sum, pairx::at_rank(&s_bar[buf], lane));
    if (ok) ok = ptx::mbar_wait(&s_bar[buf], (passes >> 1) & 1);
    ++passes;
  };
  // Sum over all ranges.
  auto total = [&]() {
    double part = 0.0;
    for (int k = lane; k < C * kVWarps; k += 32) part += s_sum[buf][k];
    return warp_sum_f64(part);
  };

  int cur = 0, count = 1, n_out = 0;
  double Z = 1.0;
  bool summed = false;          // s_sum[buf] belongs to w
  unsigned long long kids = s_kids[0];
  Weights<T, POINT> w(target, draft);
  w.out = s_out;
  if (rank == 0 && tid == 0) path[0] = 0;
  while (kids) {
    const int j = __ffsll(kids) - 1;
    kids &= kids - 1;
    double wx;
    if constexpr (POINT) {
      wx = s_p[j];
      for (int o = 0; o < n_out; ++o)
        if (s_out[o] == s_tok[j]) wx = 0.0;
    } else {
      wx = fma(-w.A, s_q[j], s_p[j]);
      wx = wx > 0.0 ? wx : 0.0;
    }
    const double q = POINT ? 1.0 : s_q[j];
    if ((double)s_u[j] * Z * q < wx) {
      if (rank == 0 && tid == 0) path[count] = j;
      ++count;
      cur = j;
      kids = s_kids[j];
      w = Weights<T, POINT>(target + cur * p.tp, draft + cur * p.dp);
      w.out = s_out;
      n_out = 0;
      Z = 1.0;
      summed = false;
      continue;
    }
    Weights<T, POINT> rest = w;
    if constexpr (POINT) {
      __syncthreads();          // the list is still read by the test above
      if (tid == 0) s_out[n_out] = s_tok[j];
      __syncthreads();
      rest.n_out = n_out + 1;
    } else {
      rest.A += Z;
    }
    pass(rest);
    const double z = total();
    summed = z > 0.0;
    if (summed) {
      w = rest;
      n_out = rest.n_out;
      Z = z;
    }
  }

  // ---------------------------------------------------------------- the draw
  if (!summed) pass(w);
  if (warp == 0) {
    constexpr int kVec = Row<T>::kVec;
    double part = 0.0;
    if (lane < C)
      for (int k = 0; k < kVWarps; ++k) part += s_sum[buf][lane * kVWarps + k];
    double z = 0.0;
    for (int c = 0; c < C; ++c) z += __shfl_sync(0xffffffffu, part, c);
    const double aim = (double)p.u_sample[b] * z;
    // the CTA, then its warp, whose range the aim falls into; where rounding
    // leaves none, the last one with any mass
    int own = -1;
    double before = 0.0, sum = 0.0;
    for (int c = 0; c < C; ++c) {
      const double s = __shfl_sync(0xffffffffu, part, c);
      if (s > 0.0) {
        own = c;
        before = sum;
      }
      sum += s;
      if (sum > aim) break;
    }
    const bool some = own >= 0 && z < INFINITY;          // false for NaN and inf, too
    if (!some) {
      if (rank == 0 && lane == 0) {
        flag_status(p.st, GQLA_DEV_BAD_PROBS);
        p.next_token[b] = -1;
      }
    } else if (own == rank) {
      int range = -1;
      sum = before;
      for (int k = 0; k < kVWarps; ++k) {
        const double s = s_sum[buf][own * kVWarps + k];
        if (s > 0.0) {
          range = own * kVWarps + k;
          before = sum;
        }
        sum += s;
        if (sum > aim) break;
      }
      const int groups = w.p.groups(V), per = (groups + C * kVWarps - 1) / (C * kVWarps);
      const int g1 = min(groups, (range + 1) * per);
      // a contiguous part of the range a lane: one scan over the lanes finds the
      // part, which its lane goes through again
      const int g0 = range * per, part_n = (g1 - g0 + 31) / 32;
      const int l0 = min(g1, g0 + lane * part_n), l1 = min(g1, l0 + part_n);
      double mine = 0.0;
      int late = -1;            // the part's last token with any weight
#pragma unroll 4
      for (int g = l0; g < l1; ++g) {
        double x[kVec];
        const int v0 = w.load(g, V, x);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          mine += x[e];
          if (x[e] > 0.0) late = v0 + e;
        }
      }
      double upto = mine;       // inclusive over the lanes
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double t = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += t;
      }
      const unsigned over = __ballot_sync(0xffffffffu, before + upto > aim);
      const int first = over ? __ffs(over) - 1 : 32;
      // rounding may leave none: the last token with weight before it
      int last = __reduce_max_sync(0xffffffffu, lane <= first ? late : -1);
      if (lane == first) {
        double c = before + (upto - mine);
        bool found = false;
        for (int g = l0; g < l1 && !found; ++g) {
          double x[kVec];
          const int v0 = w.load(g, V, x);
#pragma unroll
          for (int e = 0; e < kVec; ++e) {
            c += x[e];
            if (!found && x[e] > 0.0 && c > aim) {
              found = true;
              last = v0 + e;
            }
          }
        }
      }
      if (first < 32) last = __shfl_sync(0xffffffffu, last, first);
      if (lane == 0) p.next_token[b] = last;
    }
  }
  if (rank == 0) {
    if (tid == 0) p.n_accepted[b] = count;
    for (int k = count + tid; k < p.n_tokens; k += kVThreads) path[k] = -1;
  }
  // Every CTA has received what the others send to it in the last pass, so it may
  // end; one that gave up stays for another limit, for what may still come.
  if (!ok) {
    flag_status(p.st, GQLA_DEV_TIMEOUT);
    ptx::mbar_wait(&s_bar[buf], ((passes - 1) >> 1) & 1);
  }
}

// ----------------------------------------------------------------- commit
// One CTA per (pool, sequence), or several, each with a slice of every row, where
// there are few and rows are long (53 sequences, 12 rows of 8448 bytes: 17.9 us
// with one, 6.0 with slices).  The path increases, so accepted[k] >= k: the
// row that position k receives is never one that an earlier position
// overwrote only if all sources of a batch are read before its rows are
// written, and later batches read at or behind their own first position,
// which no earlier batch wrote.  Bound by latency for one pool (4 sequences of
// 576 bf16: 3.0 us) and by HBM for many (64 sequences, 32 pools: 8.3 us, of
// which the moved bytes would take 3.6).
constexpr int kCThreads = 128;
constexpr int kCBatch = 8;       // granules in flight a thread
constexpr int kMaxPools = 240;   // of one launch: 16 bytes each of the kernel's arguments

struct CommitParams {
  KvLayout ly;
  TreeView tree;
  int n_tokens;
  const int32_t* accepted;
  const int32_t* n_accepted;
  int32_t* lens_out;
  int32_t* st;
  gqla_pool pools[kMaxPools];
};

// The block's slice of every row, in granules of U: rows * w below 2^31.
template <typename U>
__device__ __forceinline__ void move_rows(char* base, long long row_bytes, const long long* src, const long long* dst,
                                          int rows) {
  const uint32_t per = (uint32_t)(row_bytes / sizeof(U));
  const uint32_t c0 = (uint32_t)((uint64_t)per * blockIdx.z / gridDim.z);
  const uint32_t w = (uint32_t)((uint64_t)per * (blockIdx.z + 1) / gridDim.z) - c0;
  const uint32_t items = rows * w;
  for (uint32_t i0 = threadIdx.x; i0 < items + threadIdx.x; i0 += kCThreads * kCBatch) {
    U x[kCBatch];
#pragma unroll
    for (int u = 0; u < kCBatch; ++u) {
      const uint32_t i = i0 + u * kCThreads;
      if (i < items) x[u] = reinterpret_cast<const U*>(base + src[i / w] * row_bytes)[c0 + i % w];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kCBatch; ++u) {
      const uint32_t i = i0 + u * kCThreads;
      if (i < items) reinterpret_cast<U*>(base + dst[i / w] * row_bytes)[c0 + i % w] = x[u];
    }
  }
}

__global__ void __launch_bounds__(kCThreads) commit_kernel(const __grid_constant__ CommitParams p) {
  ptx::pdl_wait();
  ptx::pdl_trigger();
  __shared__ long long s_src[kMaxTree], s_dst[kMaxTree];
  const int b = blockIdx.y, tid = threadIdx.x;
  const bool report = blockIdx.x == 0 && blockIdx.z == 0;
  const NewTokens nt = new_tokens(p.ly, p.tree, b, p.n_tokens, report && tid == 0 ? p.st : nullptr);
  const int keep = p.n_accepted[b];
  bool bad = nt.L < 0;
  if (!bad && (keep < 0 || keep > nt.n)) {
    if (report && tid == 0) flag_status(p.st, GQLA_DEV_BAD_TREE);
    bad = true;
  }
  long long from = -1, to = -1;
  bool wrong = false;
  if (!bad && tid < keep) {
    const int32_t* path = p.accepted + (long long)b * p.n_tokens;
    const int a = path[tid];
    if (a < tid || a >= nt.n || (tid > 0 && path[tid - 1] >= a)) {
      if (report) flag_status(p.st, GQLA_DEV_BAD_TREE);
      wrong = true;
    } else if (a != tid) {
      from = token_row(p.ly, b, nt.base + a, report ? p.st : nullptr);
      to = token_row(p.ly, b, nt.base + tid, report ? p.st : nullptr);
      wrong = from < 0 || to < 0;
    }
  }
  bad |= __syncthreads_or(wrong) != 0;
  if (report && tid == 0 && p.lens_out) p.lens_out[b] = bad ? p.ly.seq_lens[b] : nt.base + keep;
  if (bad) return;
  // the rows that move, in path order (once one moves, all behind it do)
  const int first = keep - __syncthreads_count(from >= 0);
  if (from >= 0) {
    s_src[tid - first] = from;
    s_dst[tid - first] = to;
  }
  __syncthreads();
  const int rows = keep - first;
  if (rows == 0) return;
  const gqla_pool pool = p.pools[blockIdx.x];
  const uintptr_t a = (uintptr_t)pool.base | (uintptr_t)pool.row_bytes;
  char* base = (char*)pool.base;
  if ((a & 15) == 0) move_rows<uint4>(base, pool.row_bytes, s_src, s_dst, rows);
  else if ((a & 3) == 0) move_rows<uint32_t>(base, pool.row_bytes, s_src, s_dst, rows);
  else move_rows<uint16_t>(base, pool.row_bytes, s_src, s_dst, rows);
}

}  // namespace

cudaError_t tree_masks(int batch, int n_tokens, const int32_t* parents, const int32_t* sizes, uint64_t* masks,
                       int32_t* st, cudaStream_t s) {
  const cudaError_t e = launch_pdl(tree_masks_kernel, dim3(batch), dim3(kMaxTree), 0, s, n_tokens, parents, sizes,
                                   masks, st);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

namespace {

template <typename T, bool POINT, bool KEEP>
cudaError_t launch_verify(const VerifyParams& p, int batch, int C, cudaStream_t s) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(batch * C));
  cfg.blockDim = dim3(kVThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, verify_kernel<T, POINT, KEEP>, p);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}
template <typename T, bool POINT>
cudaError_t launch_verify(const VerifyParams& p, int batch, int C, bool keep, cudaStream_t s) {
  return keep ? launch_verify<T, POINT, true>(p, batch, C, s) : launch_verify<T, POINT, false>(p, batch, C, s);
}

}  // namespace

cudaError_t verify_tree(int batch, int n_tokens, int vocab, const int32_t* parents, const int32_t* sizes,
                        const int32_t* tokens, const void* target, int64_t target_pitch, const void* draft,
                        int64_t draft_pitch, gqla_dtype dtype, const float* u_accept, const float* u_sample,
                        int32_t* accepted, int32_t* n_accepted, int32_t* next_token, int32_t* st, cudaStream_t s) {
  VerifyParams p{n_tokens, vocab, parents, sizes, tokens, target, draft, target_pitch, draft ? draft_pitch : 0,
                 u_accept, u_sample, accepted, n_accepted, next_token, st};
  // CTAs per sequence, as long as every warp keeps two loads a lane: a
  // sequence's passes follow one another, and the one with the most of them
  // decides the time, so up to four times what the GPU holds at once.  With 8
  // and with 4 at most: 64 sequences over 128000 fp32, 8 of which are two waves,
  // 51.9 and 59.5 us (bf16 45.6 and 50.1); 16 over 100003 bf16 21.6 and 26.0; one
  // over 32000 fp32 6.8 and 7.5
  const int groups = vocab / (dtype == GQLA_F32 ? 4 : 8);
  int C = 1;
  while (C < kMaxCluster && 2 * C * kVThreads * 2 <= groups && (long long)batch * C * 2 <= 8LL * num_sms()) C *= 2;
  // Rows stay in registers where they fit and a CTA an SM holds the batch: held,
  // and streamed again each pass, 8 sequences over 128000 fp32 take 17.1 and 18.9
  // us, one over 32000 6.8 and 7.5, 16 over 100003 bf16, which fill the SMs, 21.6
  // and 21.3.  With more, two CTAs an SM hide each other's latencies.
  const bool keep = (long long)batch * C <= num_sms() && groups + 2 <= (long long)C * kVWarps * 32 * kVKeep;
  if (dtype == GQLA_F32)
    return draft ? launch_verify<float, false>(p, batch, C, keep, s) : launch_verify<float, true>(p, batch, C, keep, s);
  return draft ? launch_verify<__nv_bfloat16, false>(p, batch, C, keep, s)
               : launch_verify<__nv_bfloat16, true>(p, batch, C, keep, s);
}

cudaError_t commit_tree(const KvLayout& ly, const TreeView& tree, int n_tokens, const int32_t* accepted,
                        const int32_t* n_accepted, const gqla_pool* pools, int n_pools, int32_t* lens_out,
                        int32_t* st, cudaStream_t s) {
  CommitParams p;
  p.ly = ly;
  p.tree = tree;
  p.n_tokens = n_tokens;
  p.accepted = accepted;
  p.n_accepted = n_accepted;
  p.st = st;
  for (int at = 0; at < n_pools; at += kMaxPools) {
    const int n = n_pools - at < kMaxPools ? n_pools - at : kMaxPools;
    for (int k = 0; k < n; ++k) p.pools[k] = pools[at + k];
    p.lens_out = at == 0 ? lens_out : nullptr;
    long long widest = 0;
    for (int k = 0; k < n; ++k) widest = pools[at + k].row_bytes > widest ? pools[at + k].row_bytes : widest;
    // at least a load of 16 bytes a thread in a row's slice; and, with up to 64
    // rows of 2^29 granules, below 2^31 granules a block
    long long slices = 4LL * num_sms() / ((long long)n * ly.batch);
    if (slices > widest / (kCThreads * 16)) slices = widest / (kCThreads * 16);
    const long long least = 1 + widest / (1 << 25);
    slices = slices < least ? least : slices > 33 ? 33 : slices;
    cudaError_t e = launch_pdl(commit_kernel, dim3((unsigned)n, (unsigned)ly.batch, (unsigned)slices), dim3(kCThreads), 0, s, p);
    count_launch();
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace gqla
