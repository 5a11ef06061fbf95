// C-ABI entry points of tree decoding: host-side validation and dispatch.
#include "gqla.h"
#include "launch.h"
#include "tc.h"
#include "tree.h"

using namespace gqla;

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
// Pointers to 4-byte elements; nullptr is aligned.
template <typename... P>
bool aligned4(const P*... p) {
  return ((... | (uintptr_t)p) & 3u) == 0;
}

gqla_status check_layout(const gqla_kv_layout* l) {
  if (!l || !l->seq_lens) return GQLA_ERR_INVALID_ARG;
  if (l->batch < 1 || l->max_seq_len < 1 || l->page_size < 0) return GQLA_ERR_INVALID_ARG;
  if (l->batch > 65535) return GQLA_ERR_UNSUPPORTED;
  if (l->page_size == 0) {
    if (l->capacity < 1) return GQLA_ERR_INVALID_ARG;
  } else {
    if (!l->block_table || l->max_blocks_per_seq < 1 || l->num_pages < 1) return GQLA_ERR_INVALID_ARG;
  }
  return GQLA_OK;
}

// make_problem for s_q up to GQLA_MAX_TREE: the causal calls take 4 at most,
// and what else it derives does not depend on s_q.
gqla_status make_tree_problem(const gqla_dims* dims, const gqla_kv_layout* layout, gqla_path path, Problem* p) {
  if (!dims || dims->s_q < 1 || dims->s_q > GQLA_MAX_TREE) return GQLA_ERR_INVALID_ARG;
  gqla_dims one = *dims;
  one.s_q = 1;
  const gqla_status s = make_problem(&one, layout, 1, path, p);
  if (s != GQLA_OK) return s;
  p->d.s_q = dims->s_q;
  p->rows = (long long)layout->batch * dims->s_q * dims->n_h;
  return GQLA_OK;
}

bool on_tensor_cores(const Problem& p, gqla_path path) {
  return path == GQLA_PATH_ABSORB ? tc_tree_absorb_supports(p) : tc_tree_gqa_supports(p);
}

size_t workspace_of(const Problem& p, gqla_path path, int num_splits) {
  if (!on_tensor_cores(p, path)) return tree_simt_workspace(p, path, num_splits);
  return path == GQLA_PATH_ABSORB ? tc_tree_absorb_workspace(p) : tc_tree_gqa_workspace(p);
}

gqla_status decode_tree(const gqla_dims* dims, const gqla_kv_layout* layout, const gqla_tree* tree, gqla_path path,
                        const void* q, const void* k_pool, const void* v_pool, const void* W_uk, const void* W_uv,
                        void* out, float* lse, int32_t num_splits, void* workspace, size_t workspace_bytes,
                        int32_t* dev_status, void* stream) {
  Problem p;
  if (!tree || !tree->masks) return GQLA_ERR_INVALID_ARG;
  const gqla_status s = make_tree_problem(dims, layout, path, &p);
  if (s != GQLA_OK) return s;
  const bool lat = path == GQLA_PATH_ABSORB;
  if (!q || !k_pool || !v_pool || !out || (lat && (!W_uk || !W_uv))) return GQLA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out)) return GQLA_ERR_ALIGNMENT;
  if (lat && (!aligned16(W_uk) || !aligned16(W_uv))) return GQLA_ERR_ALIGNMENT;
  if (((uintptr_t)tree->masks & 7u) || !aligned4(tree->sizes, lse, dev_status, layout->seq_lens, layout->block_table))
    return GQLA_ERR_ALIGNMENT;
  const bool tc = on_tensor_cores(p, path);
  if (!tc && (!simt_supports(p, path) || p.rows >= (1LL << 31) || p.d.G > 65535)) return GQLA_ERR_UNSUPPORTED;
  const size_t need = workspace_of(p, path, num_splits);
  if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u)) return GQLA_ERR_WORKSPACE;
  const TreeView v{1, tree->masks, tree->sizes};
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  if (!tc) e = tree_simt_decode(p, v, path, num_splits, q, k_pool, v_pool, W_uk, W_uv, out, lse, workspace, dev_status, st);
  else if (lat) e = tc_tree_absorb(p, v, q, k_pool, W_uk, W_uv, out, lse, workspace, dev_status, st);
  else e = tc_tree_gqa(p, v, q, k_pool, v_pool, out, lse, workspace, dev_status, st);
  return e == cudaSuccess ? GQLA_OK : GQLA_ERR_CUDA;
}

}  // namespace

extern "C" {

gqla_status gqla_append_tree(const gqla_dims* dims, const gqla_kv_layout* layout, const int32_t* sizes,
                             const void* new_rows, void* latent, const void* W_uk, const void* W_uv, void* k_pool,
                             void* v_pool, int32_t* dev_status, void* stream) {
  Problem p;
  const gqla_status s = make_tree_problem(dims, layout, GQLA_PATH_GQA, &p);
  if (s != GQLA_OK) return s;
  if (!new_rows) return GQLA_ERR_INVALID_ARG;
  const bool expand = k_pool || v_pool;
  if (!latent && !expand) return GQLA_ERR_INVALID_ARG;
  if (expand && (!k_pool || !v_pool || !W_uk || !W_uv)) return GQLA_ERR_INVALID_ARG;
  if (!aligned16(new_rows) || (latent && !aligned16(latent))) return GQLA_ERR_ALIGNMENT;
  if (expand && (!aligned16(W_uk) || !aligned16(W_uv) || !aligned16(k_pool) || !aligned16(v_pool)))
    return GQLA_ERR_ALIGNMENT;
  if (!aligned4(sizes, dev_status, layout->seq_lens, layout->block_table)) return GQLA_ERR_ALIGNMENT;
  // without a latent pool the expansion must read the dense new rows
  if (!latent && !tc_expand_supports(p)) return GQLA_ERR_UNSUPPORTED;
  const TreeView v{1, nullptr, sizes};
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = latent ? append_rows(p, v, new_rows, latent, dev_status, st) : cudaSuccess;
  if (e == cudaSuccess && expand) {
    // the new rows are dense: the tensor-core form packs many sequences' new
    // tokens into each 128-row tile
    if (tc_expand_supports(p)) e = tc_expand_dense(p, v, new_rows, k_pool, v_pool, W_uk, W_uv, dev_status, st);
    else e = simt_expand(p, v, latent, W_uk, W_uv, k_pool, v_pool, p.d.s_q, dev_status, st);
  }
  return e == cudaSuccess ? GQLA_OK : GQLA_ERR_CUDA;
}

gqla_status gqla_decode_tree_gqa(const gqla_dims* dims, const gqla_kv_layout* layout, const gqla_tree* tree,
                                 const void* q, const void* k_pool, const void* v_pool, void* out, float* lse,
                                 int32_t num_splits, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                 void* stream) {
  return decode_tree(dims, layout, tree, GQLA_PATH_GQA, q, k_pool, v_pool, nullptr, nullptr, out, lse, num_splits,
                     workspace, workspace_bytes, dev_status, stream);
}

gqla_status gqla_decode_tree_absorb(const gqla_dims* dims, const gqla_kv_layout* layout, const gqla_tree* tree,
                                    const void* q, const void* latent, const void* W_uk, const void* W_uv,
                                    void* out, float* lse, int32_t num_splits, void* workspace,
                                    size_t workspace_bytes, int32_t* dev_status, void* stream) {
  return decode_tree(dims, layout, tree, GQLA_PATH_ABSORB, q, latent, latent, W_uk, W_uv, out, lse, num_splits,
                     workspace, workspace_bytes, dev_status, stream);
}

size_t gqla_tree_workspace_bytes(const gqla_dims* dims, const gqla_kv_layout* layout, int32_t num_splits,
                                 gqla_path path) {
  Problem p;
  if (make_tree_problem(dims, layout, path, &p) != GQLA_OK) return 0;
  return workspace_of(p, path, num_splits);
}

int32_t gqla_tree_num_splits(const gqla_dims* dims, const gqla_kv_layout* layout, int32_t num_splits,
                             gqla_path path) {
  Problem p;
  if (make_tree_problem(dims, layout, path, &p) != GQLA_OK) return 0;
  return on_tensor_cores(p, path) ? 1 : tree_simt_splits(p, path, num_splits);
}

gqla_status gqla_tree_masks(int32_t batch, int32_t n_tokens, const int32_t* parents, const int32_t* sizes,
                            uint64_t* masks, int32_t* dev_status, void* stream) {
  if (batch < 1 || n_tokens < 1 || n_tokens > GQLA_MAX_TREE || !parents || !masks) return GQLA_ERR_INVALID_ARG;
  if (((uintptr_t)masks & 7u) || !aligned4(parents, sizes, dev_status)) return GQLA_ERR_ALIGNMENT;
  const cudaError_t e = tree_masks(batch, n_tokens, parents, sizes, masks, dev_status, (cudaStream_t)stream);
  return e == cudaSuccess ? GQLA_OK : GQLA_ERR_CUDA;
}

gqla_status gqla_verify_tree(int32_t batch, int32_t n_tokens, int32_t vocab, const int32_t* parents,
                             const int32_t* sizes, const int32_t* tokens, const void* target, int64_t target_pitch,
                             const void* draft, int64_t draft_pitch, gqla_dtype probs_dtype, const float* u_accept,
                             const float* u_sample, int32_t* accepted, int32_t* n_accepted, int32_t* next_token,
                             int32_t* dev_status, void* stream) {
  if (batch < 1 || n_tokens < 1 || n_tokens > GQLA_MAX_TREE || vocab < 1) return GQLA_ERR_INVALID_ARG;
  if (!parents || !tokens || !target || !u_accept || !u_sample || !accepted || !n_accepted || !next_token)
    return GQLA_ERR_INVALID_ARG;
  if (target_pitch < vocab || (draft && draft_pitch < vocab)) return GQLA_ERR_INVALID_ARG;
  if (probs_dtype != GQLA_F32 && probs_dtype != GQLA_BF16) return GQLA_ERR_INVALID_ARG;
  // rows may start anywhere (an odd vocabulary), elements not
  const uintptr_t el = probs_dtype == GQLA_F32 ? 3 : 1;
  if (((uintptr_t)target & el) || ((uintptr_t)draft & el)) return GQLA_ERR_ALIGNMENT;
  if (!aligned4(parents, sizes, tokens, u_accept, u_sample, accepted, n_accepted, next_token, dev_status))
    return GQLA_ERR_ALIGNMENT;
  if (batch > (1 << 24) || vocab > (1 << 30)) return GQLA_ERR_UNSUPPORTED;
  const cudaError_t e = verify_tree(batch, n_tokens, vocab, parents, sizes, tokens, target, target_pitch, draft,
                                    draft_pitch, probs_dtype, u_accept, u_sample, accepted, n_accepted, next_token,
                                    dev_status, (cudaStream_t)stream);
  return e == cudaSuccess ? GQLA_OK : GQLA_ERR_CUDA;
}

gqla_status gqla_commit_tree(const gqla_kv_layout* layout, int32_t n_tokens, const int32_t* sizes,
                             const int32_t* accepted, const int32_t* n_accepted, const gqla_pool* pools,
                             int32_t n_pools, int32_t* seq_lens_out, int32_t* dev_status, void* stream) {
  const gqla_status s = check_layout(layout);
  if (s != GQLA_OK) return s;
  if (n_tokens < 1 || n_tokens > GQLA_MAX_TREE || !accepted || !n_accepted || !pools || n_pools < 1)
    return GQLA_ERR_INVALID_ARG;
  if (seq_lens_out == layout->seq_lens) return GQLA_ERR_INVALID_ARG;
  for (int i = 0; i < n_pools; ++i) {
    if (!pools[i].base || pools[i].row_bytes < 2) return GQLA_ERR_INVALID_ARG;
    if (((uintptr_t)pools[i].base & 1) || (pools[i].row_bytes & 1)) return GQLA_ERR_ALIGNMENT;
    if (pools[i].row_bytes > (1 << 30)) return GQLA_ERR_UNSUPPORTED;
  }
  if (!aligned4(sizes, accepted, n_accepted, seq_lens_out, dev_status, layout->seq_lens, layout->block_table))
    return GQLA_ERR_ALIGNMENT;
  const KvLayout ly{layout->seq_lens, layout->block_table, layout->batch, layout->max_seq_len, layout->page_size,
                    layout->page_size == 0 ? layout->capacity : layout->max_blocks_per_seq * layout->page_size,
                    layout->max_blocks_per_seq, layout->num_pages};
  const cudaError_t e = commit_tree(ly, TreeView{1, nullptr, sizes}, n_tokens, accepted,
                                    n_accepted, pools, n_pools, seq_lens_out, dev_status, (cudaStream_t)stream);
  return e == cudaSuccess ? GQLA_OK : GQLA_ERR_CUDA;
}

}  // extern "C"
