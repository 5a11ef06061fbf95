// Tree attention over the latent cache (the absorbed form), bf16, on tcgen05.
//
// Row (i, h) of a sequence's drafted token i has the absorbed query
// q~ = [W_uk^g q_nope ; q_rope] (576 elements), scores s_t = scale <q~, c_t>
// against the latent rows c_t = [c_KV ; k_rope] that it sees, and the latent
// output o~ = sum_t softmax(s)_t c_KV,t (512), lifted by W_uv^g at the end.
// Every head reads the same rows, so a tile of tokens serves 64 (token, head)
// rows of a sequence at once.
//
// A unit is 64 rows, the largest whose O (64 x 512 fp32) leaves tensor memory
// for Q~ and S: with M = 64 an accumulator takes 16 of every 32 lanes, lanes
// 16-31 hold O (2 x 256 columns), lanes 0-15 Q~ (288) and two S (2 x 64).
// M = 64 runs the tensor pipe at half its rate (64 cycles for N = 128, K = 16,
// 4096 of 8192 flop a cycle).  M = 128 over a pair of CTAs has the full rate
// but, loaded as here, would stage a tile's rows twice, for the scores by token
// and for the values by column: 36 + 32 KB of a tile of 64 tokens a CTA for 64
// rows, where this form takes 72 KB, and O (256 columns) with two S (64) leaves
// 192 of 512 columns for Q~, which needs 288.  Counted, not built; halves passed
// between the CTAs of a pair, and a part of Q~ in shared memory, are open.
// A tile of 64 tokens costs the pipe 2176 cycles.
//
// One persistent CTA an SM takes a share of the batch's tile list
// (tree_work.cuh).  Warps 0 and 3 load tiles (72 KB, 3 stages; one thread
// brings about 27 bytes a cycle) and, in a stage of their own, each unit's
// queries, which are as large, warp 1 issues S = Q~ C^T, warp 2 O += P C.
// Two groups of four softmax warps take alternate tiles: one group alone took
// 3650 cycles a tile, most of it latency, and was what the pipe waited for; now
// a tile takes about 2400.
//
// Q~ and P are rounded to bf16, the type of the latent rows that they multiply:
// against 64 bits the output is 0.0024..0.0025 off (relative, norms), 0.0017 of
// it its own rounding.  Q~ as two bf16 values would bring 0.0018..0.0021, for 32
// score steps more a tile (1024 cycles to the 2176) and room that there is not.
// Measured with the lifts and merges: 8 sequences of 1000..8000 tokens, 8
// drafted, 128 heads: 109 us; 8 of 16000, 16 drafted: 860..930 in a row, where the
// power limit holds the clock, the flops taking 352 at the burst rate of M = 128.
#include <math.h>

#include "pair.cuh"
#include "tc.h"
#include "tree.h"
#include "tree_work.cuh"

namespace gqla {

namespace {

constexpr int kR = 512, kDr = 64, kE = kR + kDr;
constexpr int kM = 64;                               // rows of a unit
constexpr int kT = 64;                               // tokens of a tile
constexpr int kStages = 3;
constexpr int kChunks = kE / 64;                     // 128-byte column chunks of a row
constexpr int kChunk = kT * 128;
constexpr int kStageBytes = kChunks * kChunk;
constexpr int kPBytes = kM * 128;
constexpr size_t kSmemBytes = (size_t)kStages * kStageBytes + kPBytes + 1024;
constexpr int kThreads = 12 * 32;
constexpr uint32_t kCols = 512, kQCols = kE / 2, kSCol = kQCols;
constexpr uint32_t kOLane = 16u << 16;               // O in lanes 16-31 of each quarter
constexpr float kRescaleLog2 = 8.f;
constexpr float kLn2 = 0.69314718055994531f;

static_assert(kSCol + 2 * kT <= kCols, "Q~ and the S buffers share the low half-lanes");
static_assert(kSmemBytes + 2048 <= 227 * 1024, "the stage ring, P, and the static variables below");

struct TreeAbsorbParams {
  KvLayout ly;
  TreeView tree;
  TreeWork work;
  int d_nope;
  float* o_lat;                // [batch][units][block]: those that one worker held whole
  float* lse_lat;              // [rows]
  float* o_part;               // [worker][2][block]
  float* lse_part;             // [worker][2][64]; bad_part(): the segment met a bad page
  int units;                   // row blocks of a sequence's slots
  int merged;                  // tree_latent_merge has joined the parts
  long long* prefix;           // [batch + 2]
  int n_h, G, m;
  float scale_log2;            // of |scale|
  uint32_t q_flip;             // sign bits of a bf16 pair where the scale is negative
  int32_t* st;
};

// 16 lanes x 32 columns, the shape of ptx::tmem_st16x64 with 16 repeats.
__device__ __forceinline__ void tmem_st16x32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x64b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Barrier 1 of the softmax warps: whether `x` holds in any thread.
__device__ __forceinline__ bool softmax_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n"
      ".reg .pred p, q;\n"
      "setp.ne.u32 p, %1, 0;\n"
      "barrier.cta.red.or.pred q, 1, 256, p;\n"
      "selp.u32 %0, 1, 0, q;\n"
      "}\n"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

constexpr long long kBlockFloats = (long long)kM * kR;

__global__ void __launch_bounds__(kThreads, 1)
    tree_absorb_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap lifted_map,
                       const __grid_constant__ CUtensorMap rope_map, const TreeAbsorbParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sP = smem + kStages * kStageBytes;
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages], s_full[2], s_free[2], p_full[2], pv_done[2],
      m_ready[2][4], q_full, o_full, drain[2];
  __shared__ float row_max[2][kM];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  __shared__ volatile int bad_page[kStages];
  __shared__ SegmentWalk sm_walk[5];    // of the producers, the issuers, the softmax warps: out of their registers
  __shared__ SharedSegment sm_seg[2];   // of the issuers
  __shared__ TreeSegment sm_next;
  __shared__ int sm_more;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int worker = blockIdx.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&full[s], 2);
      ptx::mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(&s_full[s], 1);
      ptx::mbar_init(&s_free[s], 4);
      ptx::mbar_init(&p_full[s], 4);
      ptx::mbar_init(&pv_done[s], 1);
      ptx::mbar_init(&drain[s], 1);
      for (int w = 0; w < 4; ++w) ptx::mbar_init(&m_ready[s][w], 1);
    }
    ptx::mbar_init(&q_full, 8);
    ptx::mbar_init(&o_full, 1);
    abort_flag = 0;
    ptx::fence_barrier_init();
  }
  // Launched while the query lift ahead of it still runs.  That kernel started
  // after all before it had ended, holds no tensor memory and writes the lifted
  // queries only: the producers wait for it before they load those, and every
  // thread before the block ends (one sequence of 500, 4 drafted: 27 us a call
  // with the wait here, now 24).
  ptx::pdl_trigger();
  if (warp == 1) {
    ptx::tmem_alloc(&tmem_base_sh, kCols);
    ptx::tmem_relinquish();
  }
  if (warp == 3) {
    share_start<5>(p.work, p.ly, p.tree, worker, worker == 0, p.prefix, p.st, sm_walk);
    if (lane == 0) sm_more = sm_walk[4].next(p.work, p.ly, p.tree, &sm_next);
  }
  ptx::tc_fence_before();
  __syncthreads();                                    // barriers and tensor memory are ready
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  TreeSegment sg;

  if (warp == 0 || warp == 3) {
    // ---------------------------------------------------------- producers
    const int c_lo = warp == 0 ? 0 : 5, c_hi = warp == 0 ? 5 : kChunks;
    if (lane == 0) {
      ptx::prefetch_tmap(&lifted_map);
      ptx::prefetch_tmap(&kv_map);
      uint32_t it = 0;
      bool ok = true;
      ptx::pdl_wait();
      while (ok && sm_walk[warp == 0 ? 0 : 1].next(p.work, p.ly, p.tree, &sg)) {
        // a segment takes a stage for its queries, then one a tile
        for (int j = -1; j < sg.n; ++j, ++it) {
          const int s = (int)(it % kStages);
          const uint32_t k = it / kStages;
          long long row = j < 0 ? (long long)sg.b * p.work.s_q * p.n_h + sg.rb * kM
                                : token_row(p.ly, sg.b, (sg.tile0 + j) * kT, p.st);
          const int bad = row < 0;
          if (bad) row = 0;
          if (k > 0 && !pairx::wait_long(&empty[s], (uint32_t)((k - 1) & 1))) ok = false;
          if (!ok || *(volatile int*)&abort_flag) {
            ok = false;
            break;
          }
          if (warp == 0) {
            bad_page[s] = bad;
            __threadfence_block();
          }
          uint8_t* dst = smem + s * kStageBytes;
          ptx::mbar_arrive_expect_tx(&full[s], (c_hi - c_lo) * kChunk);
          const CUtensorMap* map = j < 0 ? &lifted_map : &kv_map;
          for (int c = c_lo; c < c_hi; ++c) {
            if (j < 0 && c == kChunks - 1) ptx::tma_load_2d(dst + c * kChunk, &rope_map, &full[s], p.d_nope, (int)row);
            else ptx::tma_load_2d(dst + c * kChunk, map, &full[s], 64 * c, (int)row);
          }
        }
      }
      if (!ok) {
        flag_status(p.st, GQLA_DEV_TIMEOUT);
        atomicExch(&abort_flag, 1);
      }
      // every copy of this thread has landed
      for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i)
        pairx::wait_long(&full[i % kStages], (uint32_t)((i / kStages) & 1));
    }
  } else if (warp == 1) {
    // ------------------------------------------- issuer of S = Q~ C^T
    constexpr uint32_t idesc = ptx::idesc_bf16(kM, kT, false, false);
    const uint32_t base = ptx::smem_u32(smem);
    uint32_t it = 0;
    uint32_t segs = 0, uses[2] = {0, 0};
    bool ok = true;
    while (ok && warp_next(sm_walk[2], sm_seg[0], p.work, p.ly, p.tree, &sg)) {
      ok = pairx::wait_long(&q_full, segs & 1);
      ++segs;
      if (lane == 0) ptx::mbar_arrive(&empty[it % kStages]);   // the queries' stage has been read
      ++it;
      for (int j = 0; j < sg.n; ++j, ++it) {
        const int s = __shfl_sync(0xffffffffu, (int)(it % kStages), 0), sb = j & 1;
        if (ok) ok = pairx::wait_long(&full[s], (uint32_t)((it / kStages) & 1));
        if (ok && uses[sb] > 0) ok = pairx::wait_long(&s_free[sb], (uses[sb] - 1) & 1);
        ++uses[sb];
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint64_t bd0 = ptx::umma_desc_sw128(base + s * kStageBytes, 16, 1024);
        const uint32_t d = tmem + kSCol + (uint32_t)kT * sb;
        if (pairx::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kE / 16; ++kk)
            ptx::umma_bf16_ts(d, tmem + 8u * kk, ptx::umma_desc_add(bd0, (kk >> 2) * kChunk + (kk & 3) * 32), idesc,
                              kk > 0);
          ptx::umma_commit(&s_full[sb]);
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
    if (pairx::elect_one()) ptx::umma_commit(&drain[0]);
    __syncwarp();
    pairx::wait_long(&drain[0], 0);
  } else if (warp == 2) {
    // --------------------------------------------- issuer of O += P C
    constexpr uint32_t idesc = ptx::idesc_bf16(kM, 256, false, true);
    const uint32_t base = ptx::smem_u32(smem);
    const uint64_t ad0 = ptx::umma_desc_sw128(ptx::smem_u32(sP), 16, 1024);
    uint32_t it = 0;
    uint32_t uses[2] = {0, 0};
    bool ok = true;
    while (ok && warp_next(sm_walk[3], sm_seg[1], p.work, p.ly, p.tree, &sg)) {
      ++it;                                      // the queries' stage
      for (int j = 0; j < sg.n; ++j, ++it) {
        const int s = __shfl_sync(0xffffffffu, (int)(it % kStages), 0), sb = j & 1;
        ok = pairx::wait_long(&p_full[sb], uses[sb] & 1);
        ++uses[sb];
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint64_t bd0 = ptx::umma_desc_sw128(base + s * kStageBytes, kChunk, 1024);
        const uint32_t keep = j > 0;
        if (pairx::elect_one()) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int kk = 0; kk < kT / 16; ++kk)
              ptx::umma_bf16(tmem + kOLane + 256u * h, ptx::umma_desc_add(ad0, kk * 32),
                             ptx::umma_desc_add(bd0, 4 * h * kChunk + kk * 2048), idesc, kk > 0 ? 1u : keep);
          ptx::umma_commit(&pv_done[sb]);
          ptx::umma_commit(&empty[s]);
          if (j == sg.n - 1) ptx::umma_commit(&o_full);
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) {
      flag_status(p.st, GQLA_DEV_TIMEOUT);
      atomicExch(&abort_flag, 1);
    }
    __syncwarp();
    if (pairx::elect_one()) ptx::umma_commit(&drain[1]);
    __syncwarp();
    pairx::wait_long(&drain[1], 0);
  } else {
    // ------------------------------------------- softmax and epilogue warps
    const int gp = (warp - 4) >> 2;             // this group's tiles: j % 2 == gp
    const int qd = warp & 3;
    const uint32_t tl = tmem + ((uint32_t)(32 * qd) << 16);
    // S and O are read through the 16-lane shape: thread t holds row
    // 8 (t % 2) + t / 4 of the quarter and the columns of parity (t / 2) % 2,
    // so threads t and t ^ 2 share a row, 32 tokens each.
    const int half = (lane >> 1) & 1;
    const int row = 16 * qd + 8 * (lane & 1) + (lane >> 2);
    const uint32_t s_col = tl + kSCol + (uint32_t)kT * gp;
    uint32_t uses = 0, others = 0, segs = 0;    // tiles of this group, of the other one, segments
    uint32_t posts = 0;                         // maxima that the other group's warp posted
    uint32_t it0 = 0;   // a share has fewer than 2^32 tiles: the pool's rows are below 2^31
    bool ok = true;

    // The segment's queries from their stage into lanes 0-15, through the same
    // shape as S: a thread has the words of one parity of its row (from global
    // memory, a row a lane, they took 5500 cycles).  The even group takes words
    // 0..127 and the 32 of the RoPE part, the odd one the rest.
    auto load_q = [&]() {
      const int s = (int)(it0 % kStages);
      if (ok) ok = pairx::wait_long(&full[s], (uint32_t)((it0 / kStages) & 1));
      ok = __all_sync(0xffffffffu, ok);
      int at = row;
      asm volatile("" : "+r"(at));   // or the swizzled offsets stay in registers through the tile loop
      auto word = [&](int j) {
        return *reinterpret_cast<const uint32_t*>(smem + s * kStageBytes + (j >> 5) * kChunk +
                                                  ptx::swz128(at, (j >> 2) & 7) + (j & 3) * 4) ^ p.q_flip;
      };
#pragma unroll 1
      for (int c = 2 * gp; c < 2 * gp + 2; ++c) {
        uint32_t out[32];
#pragma unroll
        for (int v = 0; v < 32; ++v) out[v] = word(64 * c + half + 2 * v);
        ptx::tmem_st16x64(tl + 64u * c, out);
      }
      if (gp == 0) {
        uint32_t out[16];
#pragma unroll
        for (int v = 0; v < 16; ++v) out[v] = word(256 + half + 2 * v);
        tmem_st16x32(tl + 256u, out);
      }
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&q_full);
    };

    bool more = sm_more;
    sg = sm_next;
    softmax_any(false);
    if (more) load_q();
    while (more) {
      if (threadIdx.x == 128) sm_more = sm_walk[4].next(p.work, p.ly, p.tree, &sm_next);
      const int rows_here = sg.nt.n * p.n_h - sg.rb * kM;      // rows of the unit in use
      const bool valid = row < rows_here, active = 16 * qd < rows_here;
      const int r = sg.rb * kM + row;
      float m_used = -INFINITY, l_sum = 0.f;                   // l_sum: of this thread's tokens
      int bad = 0;
      for (int j = gp; j < sg.n; j += 2) {
        const int t0 = (sg.tile0 + j) * kT;
        const int s = (int)((it0 + 1u + j) % kStages);
        if (ok) ok = pairx::wait_long(&s_full[gp], uses & 1);
        ok = __all_sync(0xffffffffu, ok);
        ++uses;
        if (!ok) break;
        ptx::tc_fence_after();
        bad |= bad_page[s];
        const bool tail = t0 + kT > sg.nt.base;                // new tokens in the tile
        uint32_t sv[kT / 2];                                   // tokens 2 v + half
        if (active) {
          ptx::tmem_ld16x64(s_col, sv);
          ptx::tmem_ld_wait();
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&s_free[gp]);
        float factor = 1.f;
        if (active) {
          if (tail) {
            const uint64_t mask = valid ? new_mask(p.tree, sg.nt, sg.b, p.work.s_q, r / p.n_h) : 0;
            const uint64_t seen = seen_word(mask, sg.nt.base, t0) >> half;
#pragma unroll
            for (int v = 0; v < kT / 2; ++v)
              if (!((seen >> (2 * v)) & 1)) sv[v] = __float_as_uint(-INFINITY);
          }
          float part[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) part[e] = __uint_as_float(sv[e]);
#pragma unroll
          for (int v = 4; v < kT / 2; ++v) part[v & 3] = fmaxf(part[v & 3], __uint_as_float(sv[v]));
          float raw = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
          raw = fmaxf(raw, __shfl_xor_sync(0xffffffffu, raw, 2));
          const float mx = valid && raw != -INFINITY ? raw * p.scale_log2 : -INFINITY;
          // The running maximum passes from group to group with the tiles.  It
          // follows a larger score only when that grew by more than 2^8, so O
          // is hardly ever rescaled.
          float m_prev = -INFINITY;
          if (j > 0) {
            if (ok) ok = pairx::wait_long(&m_ready[gp ^ 1][qd], (posts + ((j - 1) >> 1)) & 1);
            m_prev = row_max[gp ^ 1][row];
          }
          const float m_new = m_prev == -INFINITY || mx > m_prev + kRescaleLog2 ? mx : m_prev;
          if (half == 0) row_max[gp][row] = m_new;
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&m_ready[gp][qd]);
          if (m_used != m_new) {
            // before the first score above -inf the sum is 0, or NaN
            if (m_used != -INFINITY) l_sum *= ptx::fast_exp2(m_used - m_new);
            m_used = m_new;
          }
          if (m_prev != -INFINITY && m_new != m_prev) factor = ptx::fast_exp2(m_prev - m_new);
          // a row that has seen nothing yet: 2^(-inf) = 0 from any finite m
          const float neg_m = m_new == -INFINITY ? 0.f : -m_new;
          float acc[2] = {0.f, 0.f};
#pragma unroll
          for (int v = 0; v < kT / 2; ++v) {
            const float e = ptx::fast_exp2(fmaf(__uint_as_float(sv[v]), p.scale_log2, neg_m));
            sv[v] = __float_as_uint(e);
            acc[v & 1] += e;
          }
          l_sum += acc[0] + acc[1];
        }
        // The PV of tile j - 1 reads P's place and adds to O: it must be
        // complete before either is written.  A warp without rows waits too,
        // or it would arrive twice for one tile.
        if (ok && j > 0) ok = pairx::wait_long(&pv_done[gp ^ 1], (others + ((j - 1) >> 1)) & 1);
        if (active) {
          ptx::tc_fence_after();
          if (__any_sync(0xffffffffu, factor != 1.f)) {
#pragma unroll 1
            for (int c = 0; c < kR / 64; ++c) {
              uint32_t ov[32];
              ptx::tmem_ld16x64(tl + kOLane + 64u * c, ov);
              ptx::tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * factor);
              ptx::tmem_st16x64(tl + kOLane + 64u * c, ov);
            }
            ptx::tmem_st_wait();
          }
          // P row: the half == 0 thread writes tokens 0..31, its partner
          // 32..63; each trades the 16 values the other one needs
          uint32_t pk[kT / 4];                                 // bf16 pairs of tokens 32 half + 2 i, + 1
#pragma unroll
          for (int i = 0; i < kT / 4; ++i) {
            const uint32_t send = half ? sv[i] : sv[kT / 4 + i];
            const uint32_t recv = __shfl_xor_sync(0xffffffffu, send, 2);
            pk[i] = half ? ptx::pack_bf16(__uint_as_float(recv), __uint_as_float(sv[kT / 4 + i]))
                         : ptx::pack_bf16(__uint_as_float(sv[i]), __uint_as_float(recv));
          }
#pragma unroll
          for (int g = 0; g < kT / 16; ++g)
            *reinterpret_cast<uint4*>(sP + ptx::swz128(row, 4 * half + g)) =
                make_uint4(pk[4 * g], pk[4 * g + 1], pk[4 * g + 2], pk[4 * g + 3]);
        }
        if (tail) {
          // latent rows that no query sees may hold anything: zero their values
          const uint64_t used = seen_word(new_union(p.tree, sg.nt, sg.b, p.work.s_q), sg.nt.base, t0);
          uint8_t* sV = smem + s * kStageBytes;
          for (int i = 32 * qd + lane; i < kT * 8 * 8; i += 128) {
            const int t = i >> 6, rem = i & 63;
            if (!((used >> t) & 1))
              *reinterpret_cast<uint4*>(sV + (rem >> 3) * kChunk + ptx::swz128(t, rem & 7)) = make_uint4(0, 0, 0, 0);
          }
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&p_full[gp]);
      }
      const float l_row = l_sum + __shfl_xor_sync(0xffffffffu, l_sum, 2);
      others += (sg.n + gp) >> 1;
      if (active) posts += (sg.n + gp) >> 1;          // a warp without rows neither posts nor waits
      it0 += 1 + sg.n;
      // both groups have seen their last scores: the queries' place is free, and
      // the next segment's scores come while this one ends
      ok = !softmax_any(!ok);
      const bool whole = sg.n == sg.tiles;
      const int last = (sg.n - 1) & 1;
      const long long grow = (long long)sg.b * p.work.s_q * p.n_h + r;
      const long long slot = part_slot(worker, sg.tile0 == 0);
      float* block = whole ? p.o_lat + ((long long)sg.b * p.units + sg.rb) * kBlockFloats : p.o_part + slot * kBlockFloats;
      more = ok && sm_more;
      sg = sm_next;
      if (more) load_q();
      if (ok) ok = pairx::wait_long(&o_full, segs & 1);
      ++segs;
      // O is complete: the groups' sums, and the maxima they stand at, take P's place
      float* row_sum = reinterpret_cast<float*>(sP);
      float* row_at = row_sum + 2 * kM;
      if (half == 0) {
        row_sum[kM * gp + row] = bad ? -1.f : l_row;
        row_at[kM * gp + row] = m_used;
      }
      ok = !softmax_any(!ok);
      if (ok && active) {
        ptx::tc_fence_after();
        // a group's sum stands at the last maximum that the group saw
        const float mt = row_max[last][row];
        float l = 0.f;
        bool broken = false;
#pragma unroll
        for (int g2 = 0; g2 < 2; ++g2) {
          const float lg = row_sum[kM * g2 + row], mg = row_at[kM * g2 + row];
          broken |= lg < 0.f;
          l += mg == -INFINITY ? lg : lg * ptx::fast_exp2(mg - mt);
        }
        // NaN where a score was NaN or +inf, or so large that its weight overflows
        if (l == INFINITY) l = NAN;
        const bool none = broken || (l == 0.f && mt == -INFINITY);
        const float inv = none ? 0.f : 1.f / l;
        float* dst = block + (long long)row * kR + 4 * half;
#pragma unroll 1
        for (int c = 4 * gp; c < 4 * gp + 4; ++c) {
          uint32_t ov[32];
          ptx::tmem_ld16x64(tl + kOLane + 64u * c, ov);
          ptx::tmem_ld_wait();
          // of each 8 columns a row's threads have the even and the odd ones:
          // traded, each stores four neighbours, 32 bytes a row together
#pragma unroll
          for (int v = 0; v < 8; ++v) {
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = none ? 0.f : __uint_as_float(ov[4 * v + i]) * inv;
            const float g0 = __shfl_xor_sync(0xffffffffu, half ? w[0] : w[2], 2);
            const float g1 = __shfl_xor_sync(0xffffffffu, half ? w[1] : w[3], 2);
            if (valid)
              *reinterpret_cast<float4*>(dst + 64 * c + 8 * v) =
                  half ? make_float4(g0, w[2], g1, w[3]) : make_float4(w[0], g0, w[1], g1);
          }
        }
        if (valid && gp == 0 && half == 0) {
          const float lse = broken ? bad_part() : none ? -INFINITY : (mt + log2f(l)) * kLn2;
          (whole ? p.lse_lat + grow : p.lse_part + slot * kM + row)[0] = lse;
        }
      }
      ptx::tc_fence_before();
      // O and the statistics are free for the next segment; one warp that gave
      // up ends the loop for all
      if (softmax_any(!ok)) {
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
  ptx::pdl_wait();
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kCols);
  }
}

// ------------------------------------------------------------- merge and lift
// out[row] = o~[row] W_uv^g, o~ the merge of a row's parts by their
// log-sum-exps.  CTA: kRows rows of group g (rows of all sequences, in order)
// x kN of the 128 outputs, a warp a row: W_uv^g streams in while the warps merge,
// then row blocks x output quarters x parts of the 512 of
// mma.sync tiles, one warp each.  o~ enters as the sum of two bf16 values (16
// bits of mantissa): rounded to one it would add as much error as q~ or P.
using bf16 = __nv_bfloat16;
constexpr int kUpN = 128;
constexpr int up_threads(int rows) { return rows * 32; }     // a warp a row
constexpr int kUpApitch = (kR + 8) * 2;
constexpr size_t up_smem(int rows, int n) { return (size_t)2 * rows * kUpApitch + (size_t)kR * (n + 8) * 2; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// The parts of a row joined in o_lat, a block a row: for few units over all
// SMs, whose rows come in many parts.  tree_merge_up_kernel reads a row's parts
// once for every block of outputs, on a few SMs (5 tokens, 32 heads, 20000 of
// context, 49 parts a row: 62 us with it alone, 49 with this pass).
__global__ void __launch_bounds__(128) tree_latent_merge(const TreeAbsorbParams p) {
  ptx::pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = blockIdx.x;
  const int bs = (int)(row / ((long long)p.work.s_q * p.n_h));
  const int lr = (int)(row - (long long)bs * p.work.s_q * p.n_h);
  const bool early = parts_known_early(p.ly);
  TreeList list{};
  if (early) list = tree_list(p.work, p.ly, p.tree);
  ptx::pdl_wait();
  const RowParts u = row_parts(p.work, p.ly, p.tree, list, bs, 0, lr, p.prefix);
  if (u.n <= 1) return;
  const int ur = lr % kM;
  const long long at = (long long)ur * kR + 128 * warp + 4 * lane;
  float mx = -INFINITY, Z = 0.f, z0 = -INFINITY;
  bool bad = false, nan = false;
  for (int i = lane; i < u.n; i += 32) {
    const float z = p.lse_part[part_slot(u.first + i, i == 0) * kM + ur];
    if (i < 32) z0 = z;
    bad |= is_bad_part(z);
    nan |= z != z;
    mx = fmaxf(mx, z);
  }
  mx = warp_max(mx);
  bad = __any_sync(0xffffffffu, bad);
  if (__any_sync(0xffffffffu, nan)) mx = NAN;        // and so will be the row
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < u.n && !bad && mx != -INFINITY; i0 += 32) {
    const int left = min(32, u.n - i0);
    if (i0 > 0) z0 = lane < left ? p.lse_part[part_slot(u.first + i0 + lane, false) * kM + ur] : -INFINITY;
    const float e = expf(z0 - mx);
    Z += warp_sum(e);
#pragma unroll 8
    for (int i = 0; i < left; ++i) {
      const float w = __shfl_sync(0xffffffffu, e, i);
      const float4 v = *reinterpret_cast<const float4*>(p.o_part + part_slot(u.first + i0 + i, i0 + i == 0) * kBlockFloats + at);
      acc.x = fmaf(w, v.x, acc.x);
      acc.y = fmaf(w, v.y, acc.y);
      acc.z = fmaf(w, v.z, acc.z);
      acc.w = fmaf(w, v.w, acc.w);
    }
  }
  const float inv = Z != 0.f ? 1.f / Z : 0.f;
  *reinterpret_cast<float4*>(p.o_lat + ((long long)bs * p.units + u.rb) * kBlockFloats + at) =
      make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  if (threadIdx.x == 0) p.lse_lat[row] = bad ? bad_part() : Z != 0.f ? mx + logf(Z) : -INFINITY;
}

template <int kRows, int kN>
__global__ void __launch_bounds__(up_threads(kRows)) tree_merge_up_kernel(const TreeAbsorbParams p, const bf16* __restrict__ W_uv,
                                                                   bf16* __restrict__ out, float* __restrict__ lse_out,
                                                                   long long rows_g) {
  extern __shared__ __align__(16) uint8_t sm[];
  ptx::pdl_trigger();   // the next call's first kernel may launch (it waits for this one)
  constexpr int kUpBpitch = (kN + 8) * 2;
  const int g = blockIdx.y, n0 = blockIdx.z * kN;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t a = ptx::smem_u32(sm), b = a + 2 * kRows * kUpApitch;
  // row lr of the group: head lr % m of slot lr / m
  auto grow_of = [&](int rr) -> long long {
    const long long lr = (long long)blockIdx.x * kRows + rr;
    return lr < rows_g ? (lr / p.m) * p.n_h + g * p.m + lr % p.m : -1;
  };
  const int rr = warp;
  const long long row = grow_of(rr);
  const int bs = row >= 0 ? (int)(row / ((long long)p.work.s_q * p.n_h)) : 0;
  const int lr = row >= 0 ? (int)(row - (long long)bs * p.work.s_q * p.n_h) : 0;   // row of the sequence
  const bool early = parts_known_early(p.ly);
  TreeList list{};
  RowParts u;
  if (early) {
    list = tree_list(p.work, p.ly, p.tree);
    u = row_parts(p.work, p.ly, p.tree, list, bs, 0, lr, p.prefix);
  }
  // rows of slots past their trees only, and known to be: zeros
  if (early && !__syncthreads_or(row >= 0 && u.n > 0)) {
    ptx::pdl_wait();                   // the call ahead may still read what is written here
    if (row >= 0) {
      for (int c = lane; c < kN / 8; c += 32)
        *reinterpret_cast<uint4*>(out + row * kUpN + n0 + 8 * c) = make_uint4(0, 0, 0, 0);
      if (lane == 0 && lse_out && n0 == 0) lse_out[row] = -INFINITY;
    }
    return;
  }
  const bf16* Wg = W_uv + (size_t)g * kR * kUpN + n0;
  for (int i = threadIdx.x; i < kR * (kN / 8); i += blockDim.x)
    cp_async16(b + (i / (kN / 8)) * kUpBpitch + (i % (kN / 8)) * 16, Wg + (size_t)(i / (kN / 8)) * kUpN + (i % (kN / 8)) * 8);
  asm volatile("cp.async.commit_group;" ::: "memory");
  // the attention's results are read from here on (W_uv^g is already on its way)
  ptx::pdl_wait();
  if (!early) u = row_parts(p.work, p.ly, p.tree, list, bs, 0, lr, p.prefix);
  {
    float4 acc[4];
#pragma unroll
    for (int q4 = 0; q4 < 4; ++q4) acc[q4] = make_float4(0.f, 0.f, 0.f, 0.f);
    float lse = -INFINITY;
    if (row >= 0) {
      if (u.n > 0) {
        const int rb = u.rb, ur = lr % kM, n = u.n;
        const long long first = u.first;
        const long long at = (long long)ur * kR + 4 * lane;     // this lane: 4 columns of every 128
        if (n == 1 || p.merged) {
          const float4* src = reinterpret_cast<const float4*>(p.o_lat + ((long long)bs * p.units + rb) * kBlockFloats + at);
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) acc[q4] = src[32 * q4];
          lse = p.lse_lat[row];
        } else {
          // a lane a part: log-sum-exps and weights, then all lanes the values
          float mx = -INFINITY, Z = 0.f, z0 = -INFINITY;
          bool bad = false, nan = false;
          for (int i = lane; i < n; i += 32) {
            const float z = p.lse_part[part_slot(first + i, i == 0) * kM + ur];
            if (i < 32) z0 = z;
            bad |= is_bad_part(z);
            nan |= z != z;
            mx = fmaxf(mx, z);
          }
          mx = warp_max(mx);
          bad = __any_sync(0xffffffffu, bad);
          if (__any_sync(0xffffffffu, nan)) mx = NAN;
          for (int i0 = 0; i0 < n && !bad && mx != -INFINITY; i0 += 32) {
            const int left = min(32, n - i0);
            if (i0 > 0) z0 = lane < left ? p.lse_part[part_slot(first + i0 + lane, false) * kM + ur] : -INFINITY;
            const float e = expf(z0 - mx);
            Z += warp_sum(e);
#pragma unroll 4
            for (int i = 0; i < left; ++i) {
              const float w = __shfl_sync(0xffffffffu, e, i);
              const float4* src =
                  reinterpret_cast<const float4*>(p.o_part + part_slot(first + i0 + i, i0 + i == 0) * kBlockFloats + at);
#pragma unroll
              for (int q4 = 0; q4 < 4; ++q4) {
                const float4 v = src[32 * q4];
                acc[q4].x = fmaf(w, v.x, acc[q4].x);
                acc[q4].y = fmaf(w, v.y, acc[q4].y);
                acc[q4].z = fmaf(w, v.z, acc[q4].z);
                acc[q4].w = fmaf(w, v.w, acc[q4].w);
              }
            }
          }
          if (Z != 0.f) {
            const float inv = 1.f / Z;
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4)
              acc[q4] = make_float4(acc[q4].x * inv, acc[q4].y * inv, acc[q4].z * inv, acc[q4].w * inv);
            lse = mx + logf(Z);
          }
        }
        if (is_bad_part(lse)) lse = -INFINITY; // a bad page: its values are zeros
      }
      if (lane == 0 && lse_out && n0 == 0) lse_out[row] = lse;
    }
#pragma unroll
    for (int q4 = 0; q4 < 4; ++q4) {
      const float x[4] = {acc[q4].x, acc[q4].y, acc[q4].z, acc[q4].w};
      float lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) lo[e] = x[e] - __bfloat162float(__float2bfloat16_rn(x[e]));
      uint8_t* at = sm + rr * kUpApitch + (128 * q4 + 4 * lane) * 2;
      *reinterpret_cast<uint2*>(at) = make_uint2(ptx::pack_bf16(x[0], x[1]), ptx::pack_bf16(x[2], x[3]));
      *reinterpret_cast<uint2*>(at + kRows * kUpApitch) = make_uint2(ptx::pack_bf16(lo[0], lo[1]), ptx::pack_bf16(lo[2], lo[3]));
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();

  // few tiles are split over the 512 as well, so that all warps have a part
  constexpr int kRb = kRows / 16, kNq = kN / 32, kTiles = kRb * kNq, kParts = kTiles <= 4 ? 4 : 1;
  const int tile = warp % kTiles, part = warp / kTiles;
  const int wr = tile % kRb, wn = tile / kRb;
  float acc[4][4];
#pragma unroll
  for (int n = 0; n < 4; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
  const int arow = wr * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, acol = (lane >> 4) * 8;
  const int bk = (lane & 7) + ((lane >> 3) & 1) * 8, bn = wn * 32 + (lane >> 4) * 8;
  if (part < kParts) {
#pragma unroll 4
    for (int k0 = part * (kR / kParts); k0 < (part + 1) * (kR / kParts); k0 += 16) {
      uint32_t hi[4], lo[4];
      const uint32_t at = a + arow * kUpApitch + (k0 + acol) * 2;
      ptx::ldsm_x4(at, hi[0], hi[1], hi[2], hi[3]);
      ptx::ldsm_x4(at + kRows * kUpApitch, lo[0], lo[1], lo[2], lo[3]);
#pragma unroll
      for (int np = 0; np < 2; ++np) {
        uint32_t bf[4];
        ptx::ldsm_x4_t(b + (k0 + bk) * kUpBpitch + (bn + np * 16) * 2, bf[0], bf[1], bf[2], bf[3]);
        ptx::mma_bf16_16816(acc[2 * np], hi, bf[0], bf[1]);
        ptx::mma_bf16_16816(acc[2 * np + 1], hi, bf[2], bf[3]);
        ptx::mma_bf16_16816(acc[2 * np], lo, bf[0], bf[1]);
        ptx::mma_bf16_16816(acc[2 * np + 1], lo, bf[2], bf[3]);
      }
    }
  }
  if (kParts > 1) {
    float4* sums = reinterpret_cast<float4*>(sm);     // over the merged rows
    __syncthreads();
    if (part > 0 && part < kParts)
#pragma unroll
      for (int n = 0; n < 4; ++n)
        sums[((part * kTiles + tile) * 4 + n) * 32 + lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
    __syncthreads();
    if (part == 0)
      for (int o = 1; o < kParts; ++o)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const float4 v = sums[((o * kTiles + tile) * 4 + n) * 32 + lane];
          acc[n][0] += v.x;
          acc[n][1] += v.y;
          acc[n][2] += v.z;
          acc[n][3] += v.w;
        }
  }
  if (part > 0) return;
#pragma unroll
  for (int h2 = 0; h2 < 2; ++h2) {
    const long long grow = grow_of(wr * 16 + (lane >> 2) + 8 * h2);
    if (grow < 0) continue;
#pragma unroll
    for (int n = 0; n < 4; ++n)
      *reinterpret_cast<uint32_t*>(out + grow * kUpN + n0 + wn * 32 + n * 8 + 2 * (lane & 3)) =
          ptx::pack_bf16(acc[n][2 * h2], acc[n][2 * h2 + 1]);
  }
}

template <int kRows, int kN>
cudaError_t launch_merge_up(const TreeAbsorbParams& prm, const Problem& p, const void* W_uv, void* out, float* lse,
                            cudaStream_t s) {
  const long long rows_g = (long long)p.ly.batch * p.d.s_q * p.m;
  auto kernel = tree_merge_up_kernel<kRows, kN>;
  cudaError_t e = ensure_smem_limit((const void*)kernel, (int)up_smem(kRows, kN));
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3((unsigned)((rows_g + kRows - 1) / kRows), p.d.G, kUpN / kN), dim3(up_threads(kRows)),
                    up_smem(kRows, kN), s, prm, (const bf16*)W_uv, (bf16*)out, lse, rows_g);
}

int units_of(const Problem& p) { return (int)(((long long)p.d.s_q * p.d.n_h + kM - 1) / kM); }

TreeWork work_of(const Problem& p) { return TreeWork{1, p.d.n_h, kM, kT, 3, num_sms(), p.d.s_q}; }

}  // namespace

bool tc_tree_absorb_supports(const Problem& p) {
  const auto& d = p.d;
  if (d.dtype != GQLA_BF16 || d.r != kR || d.d_rope != kDr || d.d_v != kUpN) return false;
  if (!gemm_absorb_q_supports(p) || d.d_nope % 8 != 0) return false;
  if (p.ly.page_size != 0 && p.ly.page_size % kT != 0) return false;
  const long long pool = p.ly.page_size == 0 ? (long long)p.ly.batch * p.ly.capacity
                                             : (long long)p.ly.num_pages * p.ly.page_size;
  return pool < (1LL << 31) && p.rows < (1LL << 31) && d.G <= 65535;
}

namespace {
struct AbsorbWs {
  size_t qt, o_lat, lse_lat, o_part, lse_part, prefix, bytes;
};
AbsorbWs ws_of(const Problem& p) {
  const size_t parts = (size_t)2 * work_of(p).workers * kM;
  AbsorbWs w;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at = align256(at + n);
    return here;
  };
  w.qt = take((size_t)p.rows * kR * 2);
  w.o_lat = take((size_t)p.ly.batch * units_of(p) * kBlockFloats * 4);
  w.lse_lat = take((size_t)p.rows * 4);
  w.o_part = take((size_t)2 * work_of(p).workers * kBlockFloats * 4);
  w.lse_part = take(parts * 4);
  w.prefix = take((size_t)(p.ly.batch + 2) * 8);
  w.bytes = at;
  return w;
}
}  // namespace

size_t tc_tree_absorb_workspace(const Problem& p) { return ws_of(p).bytes; }

cudaError_t tc_tree_absorb(const Problem& p, const TreeView& tree, const void* q, const void* latent, const void* W_uk,
                           const void* W_uv, void* out, float* lse, void* workspace, int32_t* st, cudaStream_t s) {
  const AbsorbWs w = ws_of(p);
  char* ws = (char*)workspace;
  bf16* qt = (bf16*)(ws + w.qt);
  cudaError_t e = absorb_q_mma(p, q, W_uk, qt, s);
  if (e != cudaSuccess) return e;
  const long long nrows = p.ly.page_size == 0 ? (long long)p.ly.batch * p.ly.capacity
                                              : (long long)p.ly.num_pages * p.ly.page_size;
  CUtensorMap kv_map, lifted_map, rope_map;
  if (!tmap_bf16_sw128(&kv_map, latent, kE, nrows, kE, kT) || !tmap_bf16_sw128(&lifted_map, qt, kR, p.rows, kR, kM) ||
      !tmap_bf16_sw128(&rope_map, q, p.d_qk, p.rows, p.d_qk, kM))
    return cudaErrorInvalidValue;
  TreeAbsorbParams prm;
  prm.ly = p.ly;
  prm.tree = tree;
  prm.work = work_of(p);
  prm.d_nope = p.d.d_nope;
  prm.o_lat = (float*)(ws + w.o_lat);
  prm.lse_lat = (float*)(ws + w.lse_lat);
  prm.o_part = (float*)(ws + w.o_part);
  prm.lse_part = (float*)(ws + w.lse_part);
  prm.prefix = (long long*)(ws + w.prefix);
  prm.n_h = p.d.n_h;
  prm.G = p.d.G;
  prm.m = p.m;
  prm.units = units_of(p);
  prm.merged = 0;
  // The sign of the scale goes into the queries, exactly; then the largest
  // score is the largest product.  A scale of 0 is the least one whose scores
  // still round to 0: an unseen score enters as -inf, and 0 x -inf is NaN.
  prm.scale_log2 = p.d.scale == 0.f ? 1e-37f : fabsf(p.d.scale) * 1.4426950408889634f;
  prm.q_flip = p.d.scale < 0.f ? 0x80008000u : 0u;
  prm.st = st;
  e = ensure_smem_limit((const void*)tree_absorb_kernel, (int)kSmemBytes);
  if (e != cudaSuccess) return e;
  e = launch_pdl(tree_absorb_kernel, dim3(prm.work.workers), dim3(kThreads), kSmemBytes, s, kv_map, lifted_map, rope_map, prm);
  count_launch();
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // parts of a row, as far as the host can tell: a max_seq_len far above the
  // lengths brings the extra pass to short contexts too
  const long long units = (long long)p.ly.batch * prm.units, tiles = ((long long)p.ly.max_seq_len + kT - 1) / kT;
  const long long parts = prm.work.workers / units < tiles ? prm.work.workers / units : tiles;
  prm.merged = parts > 5;
  if (prm.merged) {
    e = launch_pdl(tree_latent_merge, dim3((unsigned)p.rows), dim3(128), 0, s, prm);
    count_launch();
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  // 32 rows a CTA and all outputs; with too few rows for that on every SM, 16
  // rows and a quarter of them (a CTA's time is then the latency of its loads)
  const long long rows_g = (long long)p.ly.batch * p.d.s_q * p.m;
  if ((rows_g + 31) / 32 * p.d.G >= num_sms() / 2) e = launch_merge_up<32, 128>(prm, p, W_uv, out, lse, s);
  else e = launch_merge_up<16, 32>(prm, p, W_uv, out, lse, s);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gqla
