// Tree attention on CUDA cores: fp32 problems (true fp32 arithmetic, no TF32)
// and bf16 dims that the tensor-core kernels do not take, over the expanded
// cache and over the latent cache.
//
// Block = (split of the tokens, 32 (token, head) rows of a sequence and group),
// tiles of 64 tokens, a thread on 2 rows.  Scores: those rows x 4 tokens, the
// keys through shared memory 32 dims at a time.  Values: the same rows x 4
// columns of every 64, so a row's statistics stay in its threads, P from shared
// memory and the values through it, 64 columns of the tile at a time: all their
// loads are in flight together (read token by token where they are used, a tile
// took 16 latencies), and the next dims' keys and the next columns' values while
// this one's products run (6 x 26 tokens, 16 heads, rank 200, fp32: 66 -> 50 us a
// call, with the queries' and the lifts' loads batched).  The absorbed form takes the heads of all groups as one
// group, so a latent row is read once for 32 rows.  Everything is held in fp32.
// Bound by latency when it is short and by the issue of its shared-memory reads
// when it is long.  The tiny model's heads (3 x 7 tokens, 8 heads, 1000 of
// context, fp32): 17 us; a row at a time a warp, without tiles, 390.  Four rows
// a thread halve those reads a product, and lose by their registers and fewer
// blocks (16 x 16 tokens, 16 heads of 48 and 64, 1000 of context: 80 us, with 2
// rows then 66, now 59; 4 sequences of 300: 21.5, 19 and 18).
#include <math.h>

#include "tree.h"

namespace gqla {

namespace {

constexpr int kRows = 32, kTok = 64, kDimChunk = 32, kThreads = 256;
constexpr int kCols = 64;                  // value columns at a time
constexpr int kPitch = kDimChunk + 4;      // floats; 16-byte rows, no bank conflicts
constexpr int kPPitch = kRows + 4;

struct SimtParams {
  KvLayout ly;
  TreeView tree;
  int s_q, groups, m, n_h, rtiles, splits;
  long long chunk;             // tokens of a split
  int dk, dv, ksplit, kro_base, kro_gs, koff_gs, voff_gs;
  long long krs, vrs;          // elements between token rows
  float scale;
  long long rows;              // batch * s_q * n_h
  int q_pitch, q_split;        // query row: elements j < q_split from qa, the rest from qb
  float* o_part;               // [splits][rows][dv]
  float* lse_part;             // [splits][rows]
  int32_t* st;
};

__host__ __device__ __forceinline__ int q_floats(int dk) { return ((dk + kDimChunk - 1) / kDimChunk) * kDimChunk + 4; }

// qa: fp32 lifted queries [rows, q_split] (latent form) or nullptr; qb: the
// queries [rows, q_pitch], read from element q_skip on.  kU: 64-column parts of
// the values.
template <typename T, int kU>
__global__ void __launch_bounds__(kThreads, kU == 1 ? 3 : kU == 2 ? 2 : 1)
    tree_simt_kernel(const SimtParams p, const float* __restrict__ qa, const T* __restrict__ qb, int q_skip,
                     const T* __restrict__ kpool, const T* __restrict__ vpool) {
  // After the query lift (latent form), only its result has to be waited for:
  // that kernel started when all before it had ended.  Without one, the kernel
  // ahead may be what writes the lengths, sizes or pages.
  if (qa == nullptr) ptx::pdl_wait();
  ptx::pdl_trigger();
  extern __shared__ __align__(16) float sm[];
  const int qw = q_floats(p.dk);
  float* sQ = sm;                            // [kRows][qw]
  float* sK = sQ + kRows * qw;               // [kTok][kPitch]
  float* sP = sK + kTok * kPitch;            // [kTok][kPPitch]
  float* sV = sP + kTok * kPPitch;           // [kTok][kCols]
  __shared__ long long s_row[kTok];
  const int tid = threadIdx.x, lane = tid & 31;
  const int split = blockIdx.x % p.splits;
  const int unit = blockIdx.x / p.splits;
  const int rt = unit % p.rtiles, bg = unit / p.rtiles, g = bg % p.groups, b = bg / p.groups;
  const NewTokens nt = new_tokens(p.ly, p.tree, b, p.s_q, split == 0 && g == 0 && rt == 0 && tid == 0 ? p.st : nullptr);
  const bool pages_ok = seq_pages_ok(p.ly, b, nt.L, p.st);     // includes a __syncthreads
  const int r0 = rt * kRows, rows_used = nt.n * p.m;
  const int t_begin = (int)min(split * p.chunk, (long long)max(nt.L, 0));
  const int t_end = (int)min((split + 1) * p.chunk, (long long)nt.L);
  auto grow_of = [&](int r) { return ((long long)b * p.s_q + r / p.m) * p.n_h + g * p.m + r % p.m; };
  const int ty = tid >> 4, tx = tid & 15;    // rows 2 ty + a; tokens tx + 16 i; columns 4 tx + e of each 64
  if (qa != nullptr) ptx::pdl_wait();
  if (!pages_ok || r0 >= rows_used || t_begin >= t_end) {
    if (tid < kRows && r0 + tid < p.s_q * p.m) p.lse_part[split * p.rows + grow_of(r0 + tid)] = -INFINITY;
    return;
  }
  {
    long long row[kRows / 8];                // a warp's rows
#pragma unroll
    for (int k = 0; k < kRows / 8; ++k) {
      const int rr = (tid >> 5) + 8 * k;
      row[k] = r0 + rr < rows_used ? grow_of(r0 + rr) : -1;
    }
#pragma unroll 2
    for (int j = lane; j < qw - 4; j += 32) {
      float x[kRows / 8];
#pragma unroll
      for (int k = 0; k < kRows / 8; ++k)
        x[k] = row[k] < 0 || j >= p.dk ? 0.f
               : j < p.q_split         ? qa[row[k] * p.q_split + j]
                                       : to_f32(qb[row[k] * p.q_pitch + q_skip + (j - p.q_split)]);
#pragma unroll
      for (int k = 0; k < kRows / 8; ++k) sQ[((tid >> 5) + 8 * k) * qw + j] = x[k];
    }
  }
  uint64_t mask[2];
  float mx[2], l[2];
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    const int r = r0 + 2 * ty + a;
    mask[a] = r < rows_used ? new_mask(p.tree, nt, b, p.s_q, r / p.m) : 0;
    mx[a] = -INFINITY;
    l[a] = 0.f;
  }
  const uint64_t used = new_union(p.tree, nt, b, p.s_q);
  float acc[kU][2][4];
#pragma unroll
  for (int u = 0; u < kU; ++u)
#pragma unroll
    for (int a = 0; a < 2; ++a) acc[u][a][0] = acc[u][a][1] = acc[u][a][2] = acc[u][a][3] = 0.f;
  const int koff = g * p.koff_gs, kro = p.kro_base + g * p.kro_gs, voff = g * p.voff_gs;

  for (int t0 = t_begin; t0 < t_end; t0 += kTok) {
    if (tid < kTok) s_row[tid] = t0 + tid < nt.L ? token_row(p.ly, b, t0 + tid, nullptr) : -1;
    float s[2][4] = {};
    __syncthreads();                         // rows are known
    T kx[kTok * kDimChunk / kThreads];       // the next dims of the keys, a warp a token's 32
    auto load_keys = [&](int d0) {
      const int j = d0 + lane;
      const int at = j < p.ksplit ? koff + j : kro + (j - p.ksplit);
#pragma unroll
      for (int i = 0; i < kTok * kDimChunk / kThreads; ++i) {
        const long long row = s_row[(tid >> 5) + 8 * i];
        kx[i] = row >= 0 && j < p.dk ? kpool[row * p.krs + at] : T(0.f);
      }
    };
    load_keys(0);
    for (int d0 = 0; d0 < p.dk; d0 += kDimChunk) {
      if (d0 > 0) __syncthreads();           // the keys ahead are read
#pragma unroll
      for (int i = 0; i < kTok * kDimChunk / kThreads; ++i) sK[((tid >> 5) + 8 * i) * kPitch + lane] = to_f32(kx[i]);
      __syncthreads();
      if (d0 + kDimChunk < p.dk) load_keys(d0 + kDimChunk);
#pragma unroll
      for (int d = 0; d < kDimChunk; d += 4) {
        float4 q4[2], k4[4];
#pragma unroll
        for (int a = 0; a < 2; ++a) q4[a] = *reinterpret_cast<const float4*>(sQ + (2 * ty + a) * qw + d0 + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) k4[i] = *reinterpret_cast<const float4*>(sK + (tx + 16 * i) * kPitch + d);
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            s[a][i] = fmaf(q4[a].w, k4[i].w, fmaf(q4[a].z, k4[i].z, fmaf(q4[a].y, k4[i].y, fmaf(q4[a].x, k4[i].x, s[a][i]))));
      }
    }
    const uint64_t any = seen_word(used, nt.base, t0);   // value rows that no row sees are not read
    T vx[kTok / 4];                          // the next 64 columns of the values
    auto load_values = [&](int u) {
      const int col = kCols * u + (tid & 63);
#pragma unroll
      for (int k = 0; k < kTok / 4; ++k) {
        const int t = (tid >> 6) + 4 * k;
        const long long row = s_row[t];
        vx[k] = row >= 0 && t0 + t < t_end && ((any >> t) & 1) && col < p.dv ? vpool[row * p.vrs + voff + col] : T(0.f);
      }
    };
    load_values(0);
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const uint64_t seen = seen_word(mask[a], nt.base, t0);
      const bool real = r0 + 2 * ty + a < rows_used;
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // a select: an unseen key may hold anything
        s[a][i] = real && ((seen >> (tx + 16 * i)) & 1) ? s[a][i] * p.scale : -INFINITY;
        top = fmaxf(top, s[a][i]);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float m_new = fmaxf(mx[a], top);
      const float corr = mx[a] == -INFINITY ? 0.f : expf(mx[a] - m_new);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[a][i] = s[a][i] == -INFINITY ? 0.f : expf(s[a][i] - m_new);
        sum += s[a][i];
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      l[a] = l[a] * corr + sum;
      mx[a] = m_new;
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[u][a][e] *= corr;
    }
    // a row's P is written and read by its own 16 threads
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float2*>(sP + (tx + 16 * i) * kPPitch + 2 * ty) = make_float2(s[0][i], s[1][i]);
    __syncwarp();
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (u > 0) __syncthreads();            // the columns before are read
#pragma unroll
      for (int k = 0; k < kTok / 4; ++k) sV[((tid >> 6) + 4 * k) * kCols + (tid & 63)] = to_f32(vx[k]);
      __syncthreads();
      if (u + 1 < kU) load_values(u + 1);
#pragma unroll 4
      for (int t = 0; t < kTok; ++t) {
        const float2 w = *reinterpret_cast<const float2*>(sP + t * kPPitch + 2 * ty);
        const float pr[2] = {w.x, w.y};
        const float4 v = *reinterpret_cast<const float4*>(sV + t * kCols + 4 * tx);
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          acc[u][a][0] = fmaf(pr[a], v.x, acc[u][a][0]);
          acc[u][a][1] = fmaf(pr[a], v.y, acc[u][a][1]);
          acc[u][a][2] = fmaf(pr[a], v.z, acc[u][a][2]);
          acc[u][a][3] = fmaf(pr[a], v.w, acc[u][a][3]);
        }
      }
    }
    __syncthreads();                         // the rows, P and the values are read
  }
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    const int r = r0 + 2 * ty + a;
    if (r >= p.s_q * p.m) continue;
    const long long row = split * p.rows + grow_of(r);
    // a sum of 0: nothing seen; of NaN: a score was NaN or +inf, and so are the outputs
    if (tx == 0) p.lse_part[row] = l[a] != 0.f ? mx[a] + logf(l[a]) : -INFINITY;
    if (r >= rows_used) continue;
    const float inv = l[a] != 0.f ? 1.f / l[a] : 0.f;
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (kCols * u + 4 * tx + e < p.dv) p.o_part[row * p.dv + kCols * u + 4 * tx + e] = acc[u][a][e] * inv;
  }
}

// The log-sum-exp merge of a row's splits, a warp a row: a lane a split for the
// weights, then all lanes the columns.
template <typename T>
__global__ void __launch_bounds__(128) tree_simt_merge(int S, long long rows, int dv, const float* __restrict__ o_part,
                                                       const float* __restrict__ lse_part, T* __restrict__ out,
                                                       float* __restrict__ lse_out) {
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  float mx = -INFINITY, z0 = -INFINITY;
  bool nan = false;
  for (int i = lane; i < S; i += 32) {
    const float z = lse_part[i * rows + row];
    if (i < 32) z0 = z;
    nan |= z != z;
    mx = fmaxf(mx, z);
  }
  mx = warp_max(mx);
  if (__any_sync(0xffffffffu, nan)) mx = NAN;        // and so will be the row
  float Z = 0.f;
  for (int c0 = 0; c0 < dv; c0 += 128) {         // 4 columns a lane at a time
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    Z = 0.f;
    for (int i0 = 0; i0 < S && mx != -INFINITY; i0 += 32) {
      const int left = min(32, S - i0);
      float z = z0;
      if (i0 > 0) z = lane < left ? lse_part[(i0 + lane) * rows + row] : -INFINITY;
      const float e = expf(z - mx);
      Z += warp_sum(e);
#pragma unroll 4
      for (int i = 0; i < left; ++i) {
        const float w = __shfl_sync(0xffffffffu, e, i);
        const float* src = o_part + ((i0 + i) * rows + row) * dv + c0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          // a split without weight wrote no values
          if (w != 0.f && c0 + lane + 32 * k < dv) acc[k] = fmaf(w, src[lane + 32 * k], acc[k]);
      }
    }
    const float inv = Z != 0.f ? 1.f / Z : 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c0 + lane + 32 * k < dv) out[row * dv + c0 + lane + 32 * k] = from_f32<T>(acc[k] * inv);
  }
  if (lane == 0 && lse_out) lse_out[row] = Z != 0.f ? mx + logf(Z) : -INFINITY;
}

// The latent form's two products, q~ = W_uk^g q_nope and out = o~ W_uv^g: 32
// rows of group g x 32 outputs a block, the weights and the rows through shared
// memory up to 256 of the inner dimension at a time, so that a block's loads
// are in flight together (element by element where they are used, 200 of them
// took 18 us).  kLift: the weights are [output][inner], else [inner][output].
constexpr int kLRows = 32, kLCols = 32, kLInner = 256;
constexpr int kLPitch = kLCols + 1, kAPitch = kLRows + 4;

template <typename TA, typename TW, typename TO, bool kLift>
__global__ void __launch_bounds__(256) tree_lift_kernel(const TA* __restrict__ A, int a_pitch, const TW* __restrict__ W,
                                                        TO* __restrict__ out, long long rows_g, int n_h, int m, int inner,
                                                        int outs) {
  if (kLift) ptx::pdl_wait();                // else below
  ptx::pdl_trigger();
  extern __shared__ __align__(16) float sm[];
  float* sA = sm;                            // [inner][kAPitch]
  float* sW = sA + min(inner, kLInner) * kAPitch;        // [inner][kLPitch]
  const int g = blockIdx.y, n0 = blockIdx.z * kLCols;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto grow_of = [&](int i) -> long long {
    const long long lr = (long long)blockIdx.x * kLRows + i;
    return lr < rows_g ? (lr / m) * n_h + g * m + lr % m : -1;
  };
  const TW* Wg = W + (size_t)g * inner * outs;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};       // rows 4 warp + i, output n0 + lane
  long long rows[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) rows[i] = grow_of(4 * warp + i);
  for (int k0 = 0; k0 < inner; k0 += kLInner) {
    const int nk = min(kLInner, inner - k0);
    if (k0 > 0) __syncthreads();
    if (kLift) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = 4 * warp + i;
#pragma unroll 4
        for (int k = lane; k < nk; k += 32)
          sW[k * kLPitch + n] = n0 + n < outs ? to_f32(Wg[(size_t)(n0 + n) * inner + k0 + k]) : 0.f;
      }
    } else {
#pragma unroll 16
      for (int k = warp; k < nk; k += 8)
        sW[k * kLPitch + lane] = n0 + lane < outs ? to_f32(Wg[(size_t)(k0 + k) * outs + n0 + lane]) : 0.f;
      // the kernel ahead makes the rows; the weights were there before it
      if (k0 == 0) ptx::pdl_wait();
    }
#pragma unroll 4
    for (int k = lane; k < nk; k += 32) {
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = rows[i] >= 0 ? to_f32(A[rows[i] * a_pitch + k0 + k]) : 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) sA[k * kAPitch + 4 * warp + i] = x[i];
    }
    __syncthreads();
#pragma unroll 8
    for (int k = 0; k < nk; ++k) {
      const float w = sW[k * kLPitch + lane];
      const float4 a = *reinterpret_cast<const float4*>(sA + k * kAPitch + 4 * warp);
      acc[0] = fmaf(a.x, w, acc[0]);
      acc[1] = fmaf(a.y, w, acc[1]);
      acc[2] = fmaf(a.z, w, acc[2]);
      acc[3] = fmaf(a.w, w, acc[3]);
    }
  }
  if (n0 + lane < outs)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (rows[i] >= 0) out[rows[i] * outs + n0 + lane] = from_f32<TO>(acc[i]);
    }
}

template <typename TA, typename TW, typename TO, bool kLift>
cudaError_t launch_lift(const Problem& p, const TA* A, int a_pitch, const void* W, TO* out, int inner, int outs,
                        cudaStream_t s) {
  const long long rows_g = (long long)p.ly.batch * p.d.s_q * p.m;
  const int nk = inner < kLInner ? inner : kLInner;
  const size_t smem = (size_t)nk * (kAPitch + kLPitch) * 4;
  auto kernel = tree_lift_kernel<TA, TW, TO, kLift>;
  cudaError_t e = ensure_smem_limit((const void*)kernel, (int)smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kernel, dim3((unsigned)((rows_g + kLRows - 1) / kLRows), p.d.G, (outs + kLCols - 1) / kLCols), dim3(256),
                 smem, s, A, a_pitch, (const TW*)W, out, rows_g, p.d.n_h, p.m, inner, outs);
  count_launch();
  return e;
}

struct SimtPlan {
  int groups, m, rtiles, splits, dk, dv;
  long long chunk;
  size_t qt, o_lat, o_part, lse_part, bytes;
};

// Splits of whole tiles of 64 tokens.  The library's choice: blocks for four
// waves of the SMs, 64 splits at most; a requested count is honoured up to the
// number of tiles and to 256.
SimtPlan plan_of(const Problem& p, gqla_path path, int requested) {
  SimtPlan w;
  const bool lat = path == GQLA_PATH_ABSORB;
  w.groups = lat ? 1 : p.d.G;
  w.m = lat ? p.d.n_h : p.m;
  w.dk = lat ? p.E : p.d_qk;
  w.dv = lat ? p.d.r : p.d.d_v;
  w.rtiles = (int)(((long long)p.d.s_q * w.m + kRows - 1) / kRows);
  const long long units = (long long)p.ly.batch * w.groups * w.rtiles;
  // a max_seq_len above a sequence's slots says nothing about its length
  const long long slots = p.ly.page_size == 0 ? p.ly.capacity : (long long)p.ly.mbps * p.ly.page_size;
  const long long tiles = ((p.ly.max_seq_len < slots ? p.ly.max_seq_len : slots) + kTok - 1) / kTok;
  long long S = requested > 0 ? requested : 4LL * num_sms() / units;
  const long long most = requested > 0 ? 256 : 64;
  S = S > most ? most : S;
  S = S > tiles ? tiles : S;
  S = S < 1 ? 1 : S;
  const long long per = (tiles + S - 1) / S;
  w.splits = (int)((tiles + per - 1) / per);
  w.chunk = per * kTok;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at = align256(at + n);
    return here;
  };
  w.qt = take(lat ? (size_t)p.rows * p.d.r * 4 : 0);
  w.o_lat = take(lat ? (size_t)p.rows * p.d.r * 4 : 0);
  w.o_part = take((size_t)w.splits * p.rows * w.dv * 4);
  w.lse_part = take((size_t)w.splits * p.rows * 4);
  w.bytes = at;
  return w;
}

template <typename T, int kU>
cudaError_t launch_attention(const Problem& p, const SimtPlan& w, const SimtParams& prm, const float* qa, const void* q,
                             int q_skip, const void* k, const void* v, cudaStream_t s) {
  const size_t smem = (size_t)(kRows * q_floats(w.dk) + kTok * kPitch + kTok * kPPitch + kTok * kCols) * 4;
  auto kernel = tree_simt_kernel<T, kU>;
  cudaError_t e = ensure_smem_limit((const void*)kernel, (int)smem);
  if (e != cudaSuccess) return e;
  const long long blocks = (long long)p.ly.batch * w.groups * w.rtiles * w.splits;
  if (blocks >= (1LL << 31)) return cudaErrorInvalidValue;
  e = launch_pdl(kernel, dim3((unsigned)blocks), dim3(kThreads), smem, s, prm, qa, (const T*)q, q_skip, (const T*)k,
                 (const T*)v);
  count_launch();
  return e;
}

template <typename T>
cudaError_t run(const Problem& p, const TreeView& tree, gqla_path path, const SimtPlan& w, const void* q, const void* k,
                const void* v, const void* W_uk, const void* W_uv, void* out, float* lse, char* ws, int32_t* st,
                cudaStream_t s) {
  const auto& d = p.d;
  const bool lat = path == GQLA_PATH_ABSORB;
  float* qt = lat ? (float*)(ws + w.qt) : nullptr;      // nullptr: no query lift runs ahead
  cudaError_t e = cudaSuccess;
  if (lat) e = launch_lift<T, T, float, true>(p, (const T*)q, p.d_qk, W_uk, qt, d.d_nope, d.r, s);
  if (e != cudaSuccess) return e;
  SimtParams a;
  a.ly = p.ly;
  a.tree = tree;
  a.s_q = d.s_q;
  a.groups = w.groups;
  a.m = w.m;
  a.n_h = d.n_h;
  a.rtiles = w.rtiles;
  a.splits = w.splits;
  a.chunk = w.chunk;
  a.dk = w.dk;
  a.dv = w.dv;
  a.ksplit = lat ? d.r : d.d_nope;
  a.koff_gs = lat ? 0 : p.kr.gs;
  a.kro_base = lat ? d.r : p.kr.rope;
  a.kro_gs = lat ? 0 : p.kr.rope_gs;
  a.voff_gs = lat ? 0 : d.d_v;
  a.krs = lat ? p.E : p.kr.pitch;
  a.vrs = lat ? p.E : (long long)d.G * d.d_v;
  a.scale = d.scale;
  a.rows = p.rows;
  a.q_pitch = p.d_qk;
  a.q_split = lat ? d.r : 0;
  a.o_part = (float*)(ws + w.o_part);
  a.lse_part = (float*)(ws + w.lse_part);
  a.st = st;
  const int q_skip = lat ? d.d_nope : 0;
  if (w.dv <= 64) e = launch_attention<T, 1>(p, w, a, qt, q, q_skip, k, v, s);
  else if (w.dv <= 128) e = launch_attention<T, 2>(p, w, a, qt, q, q_skip, k, v, s);
  else if (w.dv <= 256) e = launch_attention<T, 4>(p, w, a, qt, q, q_skip, k, v, s);
  else e = launch_attention<T, 8>(p, w, a, qt, q, q_skip, k, v, s);
  if (e != cudaSuccess) return e;
  const dim3 merge_grid((unsigned)((p.rows + 3) / 4));
  count_launch();
  if (!lat)
    return launch_pdl(tree_simt_merge<T>, merge_grid, dim3(128), 0, s, w.splits, p.rows, w.dv, (const float*)a.o_part,
                      (const float*)a.lse_part, (T*)out, lse);
  float* o_lat = (float*)(ws + w.o_lat);
  e = launch_pdl(tree_simt_merge<float>, merge_grid, dim3(128), 0, s, w.splits, p.rows, w.dv, (const float*)a.o_part,
                 (const float*)a.lse_part, o_lat, lse);
  if (e != cudaSuccess) return e;
  return launch_lift<float, T, T, false>(p, o_lat, d.r, W_uv, (T*)out, d.r, d.d_v, s);
}

}  // namespace

int tree_simt_splits(const Problem& p, gqla_path path, int requested) { return plan_of(p, path, requested).splits; }

size_t tree_simt_workspace(const Problem& p, gqla_path path, int requested) { return plan_of(p, path, requested).bytes; }

cudaError_t tree_simt_decode(const Problem& p, const TreeView& tree, gqla_path path, int requested, const void* q,
                             const void* k_pool, const void* v_pool, const void* W_uk, const void* W_uv, void* out,
                             float* lse, void* workspace, int32_t* st, cudaStream_t s) {
  const SimtPlan w = plan_of(p, path, requested);
  char* ws = (char*)workspace;
  return p.d.dtype == GQLA_F32
             ? run<float>(p, tree, path, w, q, k_pool, v_pool, W_uk, W_uv, out, lse, ws, st, s)
             : run<__nv_bfloat16>(p, tree, path, w, q, k_pool, v_pool, W_uk, W_uv, out, lse, ws, st, s);
}

}  // namespace gqla
