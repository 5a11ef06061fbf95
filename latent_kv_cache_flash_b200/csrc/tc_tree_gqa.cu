// Tree attention over the expanded per-group cache, bf16, on tcgen05.
//
// Row (i, h) of a sequence's drafted token i: s_t = scale <q, k_t> over the
// tokens it sees, out = sum_t softmax(s)_t v_t.  Context tokens are seen by
// all rows; the drafted ones by a 64-bit word a row.
//
// Two forms, by the rows of a (sequence, group):
//  * up to 128: one CTA, M = 128 rows, tiles of 64 tokens;
//  * more: a pair of CTAs (cta_group::2), M = 256 rows, tiles of 128 tokens.
//    Each CTA stages half of a tile's keys and half of its value columns, so
//    a row's K/V costs half the shared-memory and L2 traffic per SM: at the
//    tensor pipe's pace 128 rows alone would need 64 bytes a cycle an SM.
// Either way a stage is 40 KB a CTA (24 KB keys, 16 KB values), five of them.
//
// Per worker (CTA or pair), a share of the batch's tile list (tree_work.cuh):
//  * warp 0 loads tiles through a ring, across the share's segments;
//  * warp 1 issues S = Q K^T and warp 2 O += P[j % 2] V: from one thread a
//    tile's two commits would hold up the next tile's MMAs.  Q is in tensor
//    memory (from shared memory it would take 64 of the SM's 128 bytes a cycle
//    beside the keys and the loads), and so is P;
//  * two softmax warpgroups take alternate tiles, a thread a row: online softmax
//    in the log2 domain.  A warp takes a row's 64 or 128 scores into registers
//    and hands S back at once, so the next scores come while it works.  P is
//    rounded to bf16, the tensor cores' type beside these values (relative error
//    of the output against 64 bits 0.0021..0.0023, its own rounding 0.0017); its
//    sum is taken in fp32 before the rounding.
// Tensor memory: S 128 columns (two buffers of 64 tokens), P 2 x 64, O 128, Q 96.
//
// Measured: 16 sequences of 1000..8000 tokens, 16 drafted, 32 heads in 8 groups
// (one CTA, half its rows in use): 81 us with the merge, HBM's own time 47; 8 of
// 32000, 32 drafted, 128 heads in 16 groups (pairs): 594 us a call by itself and
// 670..760 in a row, where the power limit holds the clock; the flops take 412
// at the burst rate.  A pair's tile takes about 1865 cycles, 1280 of them the
// tensor pipe's, the rest the exponentials' (XU pipe 52% busy) and their hand-over.
#include <math.h>

#include "pair.cuh"
#include "tc.h"
#include "tree.h"
#include "tree_work.cuh"

namespace gqla {

namespace {

constexpr int kM = 128;                              // rows of a CTA
constexpr int kDqk = 192, kDv = 128;
constexpr int kBox = 64 * 128;                       // 64 rows of 128 bytes
constexpr int kKBytes = 3 * kBox, kVBytes = 2 * kBox;
constexpr int kStageBytes = kKBytes + kVBytes;
constexpr int kStages = 5;
constexpr int kTurn = 32 * 20;                       // floats of a warp's 32 rows x 16 columns, padded
constexpr size_t kSmemBytes = (size_t)kStages * kStageBytes + 8 * kTurn * 4 + 1024;
constexpr int kThreads = 12 * 32;
// registers of a softmax thread and of the others: 256 x 200 + 128 x 104 of
// the 384 x 168 that the block is launched with
constexpr int kRegsSoftmax = 200, kRegsOther = 104;
constexpr uint32_t kSCol = 0, kPCol = 128, kOCol = 256, kQCol = 384, kCols = 512;
constexpr float kRescaleLog2 = 8.f;
constexpr float kLn2 = 0.69314718055994531f;

static_assert(kSmemBytes + 4096 <= 227 * 1024, "the stage ring, the row statistics and the barriers");
static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= kThreads * 168, "register shares within the launch's");

struct TreeGqaParams {
  KvLayout ly;
  TreeView tree;
  TreeWork work;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;          // or nullptr
  float* o_part;       // [worker][2][row_block][128]
  float* lse_part;     // [worker][2][row_block]; bad_part(): the segment met a bad page
  long long* prefix;   // [batch + 2]
  int n_h, G, m;
  KRow kr;
  float scale_log2;    // of |scale|
  uint32_t q_flip;     // sign bits of a bf16 pair where the scale is negative
  int32_t* st;
};

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// Scores of tokens that the row does not see become -inf: their weight
// 2^(s scale - m) is zero.
__device__ __forceinline__ void hide_unseen(uint32_t* v, uint32_t seen) {
#pragma unroll
  for (int t = 0; t < 32; ++t)
    if (!((seen >> t) & 1)) v[t] = __float_as_uint(-INFINITY);
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}

// Barrier 3 of the eight softmax warps: whether `x` holds in any thread.
__device__ __forceinline__ bool any_of_256(bool x) {
  uint32_t r;
  asm volatile(
      "{\n"
      ".reg .pred p, q;\n"
      "setp.ne.u32 p, %1, 0;\n"
      "barrier.cta.red.or.pred q, 3, 256, p;\n"
      "selp.u32 %0, 1, 0, q;\n"
      "}\n"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

template <int kCtas>
struct Ctas {
  static constexpr int kT = 64 * kCtas;              // tokens of a tile
  static constexpr int kRows = kM * kCtas;
  static constexpr int kSBufs = 2 / kCtas;           // S buffers in 128 columns
  static __device__ __forceinline__ uint32_t rank() { return kCtas == 2 ? pairx::cta_rank() : 0; }
  static __device__ __forceinline__ void sync() {
    if (kCtas == 2) pairx::cluster_sync();
    else __syncthreads();
  }
  static __device__ __forceinline__ void alloc(uint32_t* dst) {
    if (kCtas == 2) {
      pairx::tmem_alloc(dst, kCols);
      pairx::tmem_relinquish();
    } else {
      ptx::tmem_alloc(dst, kCols);
      ptx::tmem_relinquish();
    }
  }
  static __device__ __forceinline__ void dealloc(uint32_t t) {
    if (kCtas == 2) pairx::tmem_dealloc(t, kCols);
    else ptx::tmem_dealloc(t, kCols);
  }
  static __device__ __forceinline__ void commit(uint64_t* bar) {
    if (kCtas == 2) pairx::umma_commit_both(bar);
    else ptx::umma_commit(bar);
  }
  static __device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if (kCtas == 2) pairx::umma_bf16_ts(d, a, b, idesc, acc);
    else ptx::umma_bf16_ts(d, a, b, idesc, acc);
  }
  static __device__ __forceinline__ void load(void* dst, const CUtensorMap* map, uint64_t* bar, uint32_t bar0, int c0,
                                              int c1) {
    if (kCtas == 2) pairx::tma_load_2d(dst, map, bar0, c0, c1);
    else ptx::tma_load_2d(dst, map, bar, c0, c1);
  }
  // arrival on CTA 0's barrier; `shared_too`: after writes to shared memory
  static __device__ __forceinline__ void arrive0(uint64_t* bar, uint32_t bar0, bool shared_too) {
    if (kCtas == 1) ptx::mbar_arrive(bar);
    else if (shared_too) pairx::arrive_release(bar0);
    else pairx::arrive(bar0);
  }
};

template <int kCtas>
__global__ void __launch_bounds__(kThreads, 1)
    tree_gqa_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                    const TreeGqaParams p) {
  using C = Ctas<kCtas>;
  constexpr int kT = C::kT;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages], s_full[2], p_full[2], s_free[C::kSBufs], q_full, pv_done[2], o_full,
      m_ready[2][4], drain[2];
  __shared__ float row_max[kM], row_sum[2][kM], row_at[2][kM];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  __shared__ volatile int bad_page[kStages];
  __shared__ SegmentWalk sm_walk[4];    // of the producer, the issuers, the softmax warps: out of their registers
  __shared__ SharedSegment sm_seg[2];   // of the issuers
  __shared__ TreeSegment sm_next;
  __shared__ int sm_more;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = C::rank();
  const int worker = blockIdx.x / kCtas;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&s_full[s], 1);
      ptx::mbar_init(&p_full[s], 4 * kCtas);
      ptx::mbar_init(&pv_done[s], 1);
      ptx::mbar_init(&drain[s], 1);
      for (int w = 0; w < 4; ++w) ptx::mbar_init(&m_ready[s][w], 1);
    }
    ptx::mbar_init(&q_full, 4 * kCtas);
    for (int s = 0; s < C::kSBufs; ++s) ptx::mbar_init(&s_free[s], 4 * kCtas);
    ptx::mbar_init(&o_full, 1);
    abort_flag = 0;
    ptx::fence_barrier_init();
  }
  // launched while the kernel ahead of it may still run: wait for it before
  // any access to global memory (and to tensor memory, which that kernel may
  // still be about to take), then let the next kernel launch
  ptx::pdl_wait();
  ptx::pdl_trigger();
  if (warp == 1) C::alloc(&tmem_base_sh);
  if (warp == 3) {
    share_start<4>(p.work, p.ly, p.tree, worker, worker == 0 && rank == 0, p.prefix, p.st, sm_walk);
    if (lane == 0) sm_more = sm_walk[3].next(p.work, p.ly, p.tree, &sm_next);
  }
  ptx::tc_fence_before();
  C::sync();                                          // barriers and tensor memory are ready
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  TreeSegment sg;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      if (lane == 0) {
        ptx::prefetch_tmap(&kmap);
        ptx::prefetch_tmap(&vmap);
        uint32_t it = 0;
        bool ok = true;
        while (ok && sm_walk[0].next(p.work, p.ly, p.tree, &sg)) {
          for (int j = 0; j < sg.n; ++j, ++it) {
            const int s = (int)(it % kStages);
            const uint32_t k = it / kStages;
            const int t0 = (sg.tile0 + j) * kT;
            // pool rows of the tile's 64-token parts; a part behind the
            // sequence takes the first part's rows, which nobody sees
            int row[kCtas], bad = 0;
  #pragma unroll
            for (int c = 0; c < kCtas; ++c) {
              const int t = t0 + 64 * c < sg.nt.L ? t0 + 64 * c : t0;
              long long r = token_row(p.ly, sg.b, t, p.st);
              if (r < 0) {
                bad = 1;
                r = 0;
              }
              row[c] = (int)r;
            }
            if (k > 0 && !pairx::wait_long(&empty[s], (uint32_t)((k - 1) & 1))) ok = false;
            if (!ok || *(volatile int*)&abort_flag) {
              ok = false;
              break;
            }
            bad_page[s] = bad;
            __threadfence_block();
            uint8_t* dst = smem + s * kStageBytes;
            if (rank == 0) ptx::mbar_arrive_expect_tx(&full[s], kCtas * kStageBytes);
            const uint32_t fb = pairx::at_rank(&full[s], 0);
            const int krow = kCtas == 2 && rank == 1 ? row[kCtas - 1] : row[0];
            C::load(dst, &kmap, &full[s], fb, p.kr.nope_at(sg.g), krow);
            C::load(dst + kBox, &kmap, &full[s], fb, p.kr.nope_at(sg.g) + 64, krow);
            C::load(dst + 2 * kBox, &kmap, &full[s], fb, p.kr.rope_at(sg.g), krow);
            uint8_t* dv = dst + kKBytes;
            if (kCtas == 2) {          // 64 value columns of 128 tokens
              C::load(dv, &vmap, &full[s], fb, sg.g * kDv + 64 * (int)rank, row[0]);
              C::load(dv + kBox, &vmap, &full[s], fb, sg.g * kDv + 64 * (int)rank, row[kCtas - 1]);
            } else {                   // 128 value columns of 64 tokens
              C::load(dv, &vmap, &full[s], fb, sg.g * kDv, row[0]);
              C::load(dv + kBox, &vmap, &full[s], fb, sg.g * kDv + 64, row[0]);
            }
          }
        }
        if (!ok) {
          flag_status(p.st, GQLA_DEV_TIMEOUT);
          atomicExch(&abort_flag, 1);
        }
        // every copy of this CTA has landed and been read
        for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i)
          pairx::wait_long(&empty[i % kStages], (uint32_t)((i / kStages) & 1));
      }
    } else if (warp == 1) {
      // ------------------------------------------- issuer of S = Q K^T
      if (rank == 0) {
        constexpr uint32_t idesc = ptx::idesc_bf16(C::kRows, kT, false, false);
        const uint32_t base = ptx::smem_u32(smem);
        uint32_t it = 0;
        uint32_t segs = 0, uses[C::kSBufs] = {};
        bool ok = true;
        while (ok && warp_next(sm_walk[1], sm_seg[0], p.work, p.ly, p.tree, &sg)) {
          ok = pairx::wait_long(&q_full, segs & 1);
          ++segs;
          for (int j = 0; j < sg.n; ++j, ++it) {
            const int s = __shfl_sync(0xffffffffu, (int)(it % kStages), 0);
            if (ok) ok = pairx::wait_long(&full[s], (uint32_t)((it / kStages) & 1));
            const int sb = j % C::kSBufs;
            if (ok && uses[sb] > 0) ok = pairx::wait_long(&s_free[sb], (uses[sb] - 1) & 1);
            ++uses[sb];
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            ptx::tc_fence_after();
            const uint64_t kd0 = ptx::umma_desc_sw128(base + s * kStageBytes, 16, 1024);
            if (pairx::elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kDqk / 16; ++kk)
                C::mma_ts(tmem + kSCol + 64u * sb, tmem + kQCol + 8u * kk,
                          ptx::umma_desc_add(kd0, (kk >> 2) * kBox + (kk & 3) * 32), idesc, kk > 0);
              C::commit(&s_full[j & 1]);
            }
            __syncwarp();
          }
          ok = __all_sync(0xffffffffu, ok);
        }
        if (!ok && lane == 0) {
          flag_status(p.st, GQLA_DEV_TIMEOUT);
          atomicExch(&abort_flag, 1);
        }
        __syncwarp();
        // every issued MMA has finished before tensor memory is released
        if (pairx::elect_one()) C::commit(&drain[0]);
        __syncwarp();
        pairx::wait_long(&drain[0], 0);
      }
    } else if (warp == 2) {
      // --------------------------------------------- issuer of O += P V
      if (rank == 0) {
        constexpr uint32_t idesc = ptx::idesc_bf16(C::kRows, kDv, false, true);
        const uint32_t base = ptx::smem_u32(smem);
        uint32_t it = 0;
        uint32_t uses[2] = {0, 0};
        bool ok = true;
        while (ok && warp_next(sm_walk[2], sm_seg[1], p.work, p.ly, p.tree, &sg)) {
          for (int j = 0; j < sg.n; ++j, ++it) {
            const int sb = j & 1, s = __shfl_sync(0xffffffffu, (int)(it % kStages), 0);
            ok = pairx::wait_long(&p_full[sb], uses[sb] & 1);
            ++uses[sb];
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            ptx::tc_fence_after();
            const uint64_t vd0 = ptx::umma_desc_sw128(base + s * kStageBytes + kKBytes, kBox, 1024);
            const uint32_t keep = j > 0;
            if (pairx::elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kT / 16; ++kk)
                C::mma_ts(tmem + kOCol, tmem + kPCol + 64u * sb + 8u * kk, ptx::umma_desc_add(vd0, kk * 2048), idesc,
                          kk > 0 ? 1u : keep);
              C::commit(&pv_done[sb]);
              C::commit(&empty[s]);
              if (j == sg.n - 1) C::commit(&o_full);
            }
            __syncwarp();
          }
        }
        if (!ok && lane == 0) {
          flag_status(p.st, GQLA_DEV_TIMEOUT);
          atomicExch(&abort_flag, 1);
        }
        __syncwarp();
        if (pairx::elect_one()) C::commit(&drain[1]);
        __syncwarp();
        pairx::wait_long(&drain[1], 0);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ------------------------------------------- softmax and epilogue warps
    const int gp = warp >= 8 ? 1 : 0;           // this group's tiles: j % 2 == gp
    const int qd = warp & 3;
    const int row = 32 * qd + lane;             // row of the CTA = TMEM lane
    const uint32_t tl = tmem + ((uint32_t)(32 * qd) << 16);
    const uint32_t s_col = tl + kSCol + 64u * (gp % C::kSBufs), p_col = tl + kPCol + 64u * gp;
    const uint32_t p_bar = pairx::at_rank(&p_full[gp], 0), q_bar = pairx::at_rank(&q_full, 0),
                   s_bar = pairx::at_rank(&s_free[gp % C::kSBufs], 0);
    uint32_t uses = 0, others = 0, segs = 0;    // tiles of this group, of the other one, segments
    uint32_t posts = 0;                         // maxima that the other group's warp posted
    uint32_t it0 = 0;   // a share has fewer than 2^32 tiles: the pool's rows are below 2^31
    bool ok = true;
    const float2 scale2 = make_float2(p.scale_log2, p.scale_log2);

    // The even group puts the segment's queries into tensor memory, a row a
    // thread; rows past the drafted tokens are zeros.
    auto load_q = [&]() {
      if (gp != 0) return;
      const int r = sg.rb * C::kRows + kM * (int)rank + row;
      const bool real = r < sg.nt.n * p.m;
      const int tok = real ? r / p.m : 0;
      const uint4* src = reinterpret_cast<const uint4*>(
          p.q + (((long long)sg.b * p.work.s_q + tok) * p.n_h + sg.g * p.m + (real ? r - tok * p.m : 0)) * kDqk);
#pragma unroll
      for (int c = 0; c < kDqk / 32; ++c) {
        uint32_t v[16];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint4 w = real ? src[4 * c + e] : make_uint4(0, 0, 0, 0);
          v[4 * e] = w.x ^ p.q_flip;
          v[4 * e + 1] = w.y ^ p.q_flip;
          v[4 * e + 2] = w.z ^ p.q_flip;
          v[4 * e + 3] = w.w ^ p.q_flip;
        }
        tmem_st16(tl + kQCol + 16u * c, v);
      }
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) C::arrive0(&q_full, q_bar, false);
    };

    // P's place is free once its last PV is complete.  A warp without rows
    // waits too, or it would arrive twice for one tile.
    auto p_place_free = [&]() { return uses < 2 || pairx::wait_long(&pv_done[gp], (uses - 2) & 1); };

    bool more = sm_more;
    sg = sm_next;
    asm volatile("bar.sync 3, 256;" ::: "memory");
    if (more) load_q();
    while (more) {
      if (threadIdx.x == 128) sm_more = sm_walk[3].next(p.work, p.ly, p.tree, &sm_next);
      const int rows_here = sg.nt.n * p.m - sg.rb * C::kRows - kM * (int)rank;   // rows of this CTA in use
      const bool valid = row < rows_here, active = 32 * qd < rows_here;
      const int r = sg.rb * C::kRows + kM * (int)rank + row;
      float m_used = -INFINITY, l_sum = 0.f;
      int bad = 0;
      for (int j = gp; j < sg.n; j += 2) {
        const int t0 = (sg.tile0 + j) * kT;
        const int s = (int)((it0 + j) % kStages);
        if (ok) ok = pairx::wait_long(&s_full[gp], uses & 1);
        ok = __all_sync(0xffffffffu, ok);
        ++uses;
        if (!ok) break;
        ptx::tc_fence_after();
        bad |= bad_page[s];
        const bool tail = t0 + kT > sg.nt.base;       // new tokens in the tile
        uint32_t sv[kT];
        if (active) {
#pragma unroll
          for (int c = 0; c < kT / 32; ++c) ptx::tmem_ld32(s_col + 32u * c, sv + 32 * c);
          ptx::tmem_ld_wait();
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) C::arrive0(&s_free[gp % C::kSBufs], s_bar, false);   // the next tile's scores may come
        if (active) {
          if (tail) {
            const uint64_t mask = valid ? new_mask(p.tree, sg.nt, sg.b, p.work.s_q, r / p.m) : 0;
#pragma unroll
            for (int c = 0; c < kT / 32; ++c)
              hide_unseen(sv + 32 * c, (uint32_t)seen_word(mask, sg.nt.base, t0 + 32 * c));
          }
          float mx = -INFINITY;
          {
            float part[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) part[e] = __uint_as_float(sv[e]);
#pragma unroll
            for (int t = 4; t < kT; ++t) part[t & 3] = fmaxf(part[t & 3], __uint_as_float(sv[t]));
            const float raw = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
            if (valid && raw != -INFINITY) mx = raw * p.scale_log2;
          }
          // The running maximum passes from group to group with the tiles.  It
          // follows a larger score only when that grew by more than 2^8 (P
          // stays below 2^8, exact enough in bf16 as in fp32), so O is hardly
          // ever rescaled.
          float m_prev = -INFINITY;
          if (j > 0) {
            if (ok) ok = pairx::wait_long(&m_ready[gp ^ 1][qd], (posts + ((j - 1) >> 1)) & 1);
            m_prev = row_max[row];
          }
          const float m_new = m_prev == -INFINITY || mx > m_prev + kRescaleLog2 ? mx : m_prev;
          row_max[row] = m_new;
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&m_ready[gp][qd]);
          if (m_used != m_new) {
            // before the first score above -inf the sum is 0, or NaN
            if (m_used != -INFINITY) l_sum *= ptx::fast_exp2(m_used - m_new);
            m_used = m_new;
          }
          const bool grew = m_prev != -INFINITY && m_new != m_prev;
          if (__any_sync(0xffffffffu, grew)) {
            // O holds the tiles up to j - 1 once their PV is complete; the PV
            // of this tile waits for this warp's P
            if (ok) ok = pairx::wait_long(&pv_done[gp ^ 1], (others + ((j - 1) >> 1)) & 1);
            ptx::tc_fence_after();
            const float factor = grew ? ptx::fast_exp2(m_prev - m_new) : 1.f;
            for (int c = 0; c < kDv / 16; ++c) {
              uint32_t ov[16];
              tmem_ld16(tl + kOCol + 16u * c, ov);
              ptx::tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * factor);
              tmem_st16(tl + kOCol + 16u * c, ov);
            }
          }
          // a row that has seen nothing yet: 2^(-inf) = 0 from any finite m
          const float neg_m = m_new == -INFINITY ? 0.f : -m_new;
          const float2 neg2 = make_float2(neg_m, neg_m);
          if (ok) ok = p_place_free();
          ptx::tc_fence_after();
          float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
#pragma unroll
          for (int c = 0; c < kT / 32; ++c) {
            uint32_t* v = sv + 32 * c;
            uint32_t pk[16];
#pragma unroll
            for (int t = 0; t < 32; t += 4) {
              float2 a = fma2(make_float2(__uint_as_float(v[t]), __uint_as_float(v[t + 1])), scale2, neg2);
              float2 d = fma2(make_float2(__uint_as_float(v[t + 2]), __uint_as_float(v[t + 3])), scale2, neg2);
              a = make_float2(ptx::fast_exp2(a.x), ptx::fast_exp2(a.y));
              d = make_float2(ptx::fast_exp2(d.x), ptx::fast_exp2(d.y));
              acc0 = add2(acc0, a);
              acc1 = add2(acc1, d);
              pk[t / 2] = ptx::pack_bf16(a.x, a.y);
              pk[t / 2 + 1] = ptx::pack_bf16(d.x, d.y);
            }
            tmem_st16(p_col + 16u * c, pk);
          }
          l_sum += (acc0.x + acc0.y) + (acc1.x + acc1.y);
          ptx::tmem_st_wait();
        }
        else if (ok) ok = p_place_free();
        if (tail) {
          // value rows that no query sees may hold anything: zero them
          const uint64_t used = new_union(p.tree, sg.nt, sg.b, p.work.s_q);
          uint8_t* sV = smem + s * kStageBytes + kKBytes;
          for (int i = 32 * qd + lane; i < 2 * 64 * 8; i += 128) {
            const int t = (i >> 3) & 63, box = i >> 9;
            const int at = t0 + (kCtas == 2 ? 64 * box : 0);
            if (!((seen_word(used, sg.nt.base, at) >> t) & 1))
              *reinterpret_cast<uint4*>(sV + box * kBox + ptx::swz128(t, i & 7)) = make_uint4(0, 0, 0, 0);
          }
          ptx::fence_proxy_async_smem();
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) C::arrive0(&p_full[gp], p_bar, tail);
      }
      row_sum[gp][row] = bad ? -1.f : l_sum;
      row_at[gp][row] = m_used;
      others += (sg.n + gp) >> 1;
      if (active) posts += (sg.n + gp) >> 1;          // a warp without rows neither posts nor waits
      it0 += sg.n;
      // both groups have seen their last scores: the queries are free, and
      // the other group's sum is readable
      asm volatile("bar.sync 3, 256;" ::: "memory");
      const TreeSegment cur = sg;
      more = sm_more;
      sg = sm_next;
      if (ok && more) load_q();
      if (ok) ok = pairx::wait_long(&o_full, segs & 1);
      ok = __all_sync(0xffffffffu, ok);
      ++segs;
      if (ok && active) {
        ptx::tc_fence_after();
        // a group's sum stands at the last maximum that the group saw
        const float mt = row_max[row];
        float l = 0.f;
        bool broken = false;
#pragma unroll
        for (int g2 = 0; g2 < 2; ++g2) {
          const float lg = row_sum[g2][row], mg = row_at[g2][row];
          broken |= lg < 0.f;
          l += mg == -INFINITY ? lg : lg * ptx::fast_exp2(mg - mt);
        }
        // NaN where a score was NaN or +inf, or so large that its weight overflows
        if (l == INFINITY) l = NAN;
        const bool none = broken || (l == 0.f && mt == -INFINITY);
        const float inv = none ? 0.f : 1.f / l;
        const bool whole = cur.n == cur.tiles;
        const int used = cur.nt.n * p.m - cur.rb * C::kRows - kM * (int)rank;
        const int tok = valid ? r / p.m : 0;
        const long long grow = ((long long)cur.b * p.work.s_q + tok) * p.n_h + cur.g * p.m + (r - tok * p.m);
        const long long prow = part_slot(worker, cur.tile0 == 0) * C::kRows + kM * (int)rank + row;
        for (int c = 0; c < 4; ++c) {
          const int col = 64 * gp + 16 * c;
          uint32_t o[16];
          tmem_ld16(tl + kOCol + col, o);
          ptx::tmem_ld_wait();
          float v[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = none ? 0.f : __uint_as_float(o[e]) * inv;
          if (whole) {
            if (valid) {
            __nv_bfloat16* dst = p.out + grow * kDv + col;
#pragma unroll
            for (int e = 0; e < 16; e += 8)
              *reinterpret_cast<uint4*>(dst + e) =
                  make_uint4(ptx::pack_bf16(v[e], v[e + 1]), ptx::pack_bf16(v[e + 2], v[e + 3]),
                             ptx::pack_bf16(v[e + 4], v[e + 5]), ptx::pack_bf16(v[e + 6], v[e + 7]));
            }
          } else {
            // turned in shared memory: 64 bytes of a row for four lanes
            float* turn = reinterpret_cast<float*>(smem + kStages * kStageBytes) + (warp - 4) * kTurn;
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<float4*>(turn + lane * 20 + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int rr = 8 * k + (lane >> 2);
              const float4 w = *reinterpret_cast<const float4*>(turn + rr * 20 + 4 * (lane & 3));
              if (32 * qd + rr < used)
                *reinterpret_cast<float4*>(p.o_part + (prow - lane + rr) * kDv + col + 4 * (lane & 3)) = w;
            }
            __syncwarp();
          }
        }
        if (valid && gp == 0) {
          const float lse = none ? -INFINITY : (mt + log2f(l)) * kLn2;
          if (!whole) p.lse_part[prow] = broken ? bad_part() : lse;
          else if (p.lse) p.lse[grow] = lse;
        }
      }
      ptx::tc_fence_before();
      // O and the statistics are free for the next segment; one warp that gave
      // up ends the loop for all
      if (any_of_256(!ok)) {
        ok = false;
        break;
      }
    }
    if (!ok && lane == 0) {
      flag_status(p.st, GQLA_DEV_TIMEOUT);
      atomicExch(&abort_flag, 1);
    }
  }
  // ------------------------------------------------------------ teardown
  __syncwarp();
  ptx::tc_fence_before();
  C::sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    C::dealloc(tmem);
  }
}

// Rows that no worker wrote: those of units split over several workers (the
// log-sum-exp merge of their parts), and zeros for slots behind a tree and for
// sequences that were flagged or hold nothing.  A warp a row, one after the
// other: a warp for every row of 30 x 14 tokens, 128 heads, of which none had
// parts, took 38 us, most of it in making the list (the call 64 us, now 47).
__global__ void __launch_bounds__(256) tree_gqa_merge(const TreeGqaParams p) {
  ptx::pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long rows = (long long)p.ly.batch * p.work.s_q * p.n_h;
  TreeList list{};
  if (parts_known_early(p.ly)) list = tree_list(p.work, p.ly, p.tree);
  ptx::pdl_wait();
  for (long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); row < rows; row += (long long)gridDim.x * 8) {
    const int h = (int)(row % p.n_h);
    const long long bi = row / p.n_h;
    const int b = (int)(bi / p.work.s_q), r = (int)(bi % p.work.s_q) * p.m + h % p.m;
    const RowParts u = row_parts(p.work, p.ly, p.tree, list, b, h / p.m, r, p.prefix);
    if (u.n == 1) continue;              // one worker held all its tiles and wrote the output
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float lse = -INFINITY;
    const int rr = r % p.work.row_block;
    // a lane a part: log-sum-exps and weights, then all lanes the values
    float mx = -INFINITY, Z = 0.f, z0 = -INFINITY;
    bool bad = false, nan = false;
    for (int i = lane; i < u.n; i += 32) {
      const float z = p.lse_part[part_slot(u.first + i, i == 0) * p.work.row_block + rr];
      if (i < 32) z0 = z;
      bad |= is_bad_part(z);
      nan |= z != z;
      mx = fmaxf(mx, z);
    }
    mx = warp_max(mx);
    bad = __any_sync(0xffffffffu, bad);
    if (__any_sync(0xffffffffu, nan)) mx = NAN;      // and so will be the row
    for (int i0 = 0; i0 < u.n && !bad && mx != -INFINITY; i0 += 32) {
      const int left = min(32, u.n - i0);
      if (i0 > 0)
        z0 = lane < left ? p.lse_part[part_slot(u.first + i0 + lane, false) * p.work.row_block + rr] : -INFINITY;
      const float e = expf(z0 - mx);
      Z += warp_sum(e);
#pragma unroll 4
      for (int i = 0; i < left; ++i) {
        const float w = __shfl_sync(0xffffffffu, e, i);
        const long long at = part_slot(u.first + i0 + i, i0 + i == 0) * p.work.row_block + rr;
        const float4 v = *reinterpret_cast<const float4*>(p.o_part + at * kDv + 4 * lane);
        acc.x = fmaf(w, v.x, acc.x);
        acc.y = fmaf(w, v.y, acc.y);
        acc.z = fmaf(w, v.z, acc.z);
        acc.w = fmaf(w, v.w, acc.w);
      }
    }
    if (Z != 0.f) {
      const float inv = 1.f / Z;
      acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      lse = mx + logf(Z);
    }
    *reinterpret_cast<uint2*>(p.out + row * kDv + 4 * lane) =
        make_uint2(ptx::pack_bf16(acc.x, acc.y), ptx::pack_bf16(acc.z, acc.w));
    if (lane == 0 && p.lse) p.lse[row] = lse;
  }
}

int ctas_of(const Problem& p) { return p.m * p.d.s_q > kM ? 2 : 1; }

TreeWork work_of(const Problem& p) {
  const int c = ctas_of(p);
  return TreeWork{p.d.G, p.m, kM * c, 64 * c, 3, num_sms() / c, p.d.s_q};
}

}  // namespace

bool tc_tree_gqa_supports(const Problem& p) {
  const auto& d = p.d;
  if (d.dtype != GQLA_BF16 || p.d_qk != kDqk || d.d_rope != 64 || d.d_v != kDv) return false;
  if (p.ly.page_size != 0 && p.ly.page_size % 64 != 0) return false;
  const long long rows = p.ly.page_size == 0 ? (long long)p.ly.batch * p.ly.capacity
                                             : (long long)p.ly.num_pages * p.ly.page_size;
  return rows < (1LL << 31) && p.rows < (1LL << 31);
}

size_t tc_tree_gqa_workspace(const Problem& p) {
  const TreeWork w = work_of(p);
  const size_t parts = (size_t)2 * w.workers * w.row_block;
  return align256((size_t)(p.ly.batch + 2) * 8) + align256(parts * 4) + parts * kDv * 4;
}

cudaError_t tc_tree_gqa(const Problem& p, const TreeView& tree, const void* q, const void* k_pool, const void* v_pool,
                        void* out, float* lse, void* workspace, int32_t* st, cudaStream_t s) {
  CUtensorMap kmap, vmap;
  if (!gqa_pool_maps(p, k_pool, v_pool, &kmap, &vmap)) return cudaErrorInvalidValue;
  TreeGqaParams prm;
  prm.ly = p.ly;
  prm.tree = tree;
  prm.work = work_of(p);
  prm.q = (const __nv_bfloat16*)q;
  prm.out = (__nv_bfloat16*)out;
  prm.lse = lse;
  char* ws = (char*)workspace;
  prm.prefix = (long long*)ws;
  ws += align256((size_t)(p.ly.batch + 2) * 8);
  const size_t parts = (size_t)2 * prm.work.workers * prm.work.row_block;
  prm.lse_part = (float*)ws;
  prm.o_part = (float*)(ws + align256(parts * 4));
  prm.n_h = p.d.n_h;
  prm.G = p.d.G;
  prm.m = p.m;
  prm.kr = p.kr;
  // The sign of the scale goes into the queries, exactly; then the largest
  // score is the largest product.  A scale of 0 is the least one whose scores
  // still round to 0: an unseen score enters as -inf, and 0 x -inf is NaN.
  prm.scale_log2 = p.d.scale == 0.f ? 1e-37f : fabsf(p.d.scale) * 1.4426950408889634f;
  prm.q_flip = p.d.scale < 0.f ? 0x80008000u : 0u;
  prm.st = st;
  const int ctas = ctas_of(p);
  auto kernel = ctas == 2 ? tree_gqa_kernel<2> : tree_gqa_kernel<1>;
  cudaError_t e = ensure_smem_limit((const void*)kernel, (int)kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(prm.work.workers * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = ctas == 2 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kernel, kmap, vmap, prm);
  count_launch();
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const long long blocks = (p.rows + 7) / 8, most = 8LL * num_sms();
  e = launch_pdl(tree_gqa_merge, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, s, prm);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gqla
