// moe_tree.cu -- moe_tree_attention: the plan, and the form in which all CTAs share all items.
#include "moe_tree.cuh"

namespace attn {

// More than 32 rows an item are compute on mma.sync tiles, which read K and V once for 64 rows; the
// tiles of 128 rows on tcgen05 keep up with memory.  Drafts of up to 64 tokens over contexts of up to
// 9000 (12 query, 2 key/value heads of 128): 46.0 us here, 34.9 there; 8 tokens behind 131000
// positions (32 query, 8 key/value heads: 32 rows): 263 us here, at the copy rate.
static bool many_rows(const Params &p) { return static_cast<int64_t>(p.max_q) * p.group > 32; }

static int plan_tree(const moe_kv_cache *c, const Params &p, Plan *plan) {
  const int64_t rows = static_cast<int64_t>(p.max_q) * p.group, tile = rows <= 16 ? 16 : 32;
  return make_plan(c, p, p.n_seqs, static_cast<int64_t>(p.n_rows) * p.group / tile + p.n_seqs, rows,
                   static_cast<int64_t>(p.table_width) << p.page_shift, plan);
}

template <typename T, int D>
static cudaError_t launch_rows(const Work &w, const Plan &plan, cudaStream_t stream) {
  if (plan.rows == 16) return launch_line<T, D, 1, kSeqs>(w, plan.grid, stream);
  return launch_line<T, D, 2, kSeqs>(w, plan.grid, stream);
}

}  // namespace attn

extern "C" int moe_tree_attention_workspace(const moe_kv_cache *cache, const moe_attention *a,
                                            int32_t max_q, int64_t *bytes) {
  attn::Params p;
  int rc = attn::check_attention(cache, a, &p);
  if (rc != MOE_OK) return rc;
  if (max_q < 1 || !bytes) return MOE_ERR_INVALID_ARG;
  if (max_q > MOE_TREE_MAX_Q) return MOE_ERR_UNSUPPORTED;
  if (p.n_seqs == 0 || p.n_rows == 0) {
    *bytes = 0;
    return MOE_OK;
  }
  p.max_q = max_q;
  if (attn::many_rows(p)) return attn::tiles_workspace(cache, p, bytes);
  attn::Plan plan;
  rc = attn::plan_tree(cache, p, &plan);
  if (rc == MOE_OK) *bytes = plan.bytes;
  return rc;
}

extern "C" int moe_tree_attention(const moe_kv_cache *cache, const moe_attention *a,
                                  const uint64_t *tree_mask, int32_t max_q, void *workspace,
                                  int64_t workspace_bytes, void *stream) {
  attn::Work w;
  int rc = attn::check_attention(cache, a, &w.p);
  if (rc != MOE_OK) return rc;
  if (max_q < 1 || !attn::aligned(tree_mask, 8) || workspace_bytes < 0 ||
      !attn::aligned(workspace, 16))
    return MOE_ERR_INVALID_ARG;
  if (max_q > MOE_TREE_MAX_Q) return MOE_ERR_UNSUPPORTED;
  if (w.p.n_seqs == 0 || w.p.n_rows == 0) return MOE_OK;
  w.p.mask = tree_mask;
  w.p.max_q = max_q;
  if (attn::many_rows(w.p))
    return attn::run_tiles(cache, w.p, workspace, workspace_bytes,
                           static_cast<cudaStream_t>(stream));
  attn::Plan plan;
  rc = attn::plan_tree(cache, w.p, &plan);
  if (rc != MOE_OK) return rc;
  if (plan.bytes && (!workspace || workspace_bytes < plan.bytes)) return MOE_ERR_INVALID_ARG;
  attn::use_workspace(plan, workspace, &w);
  w.list = nullptr;
  w.n_list = 0;
  w.g = {};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (plan.cluster)
    e = attn::launch_clusters(cache, w, plan.rows, plan.cluster, st);
  else if (cache->dtype == MOE_DTYPE_BF16)
    e = cache->head_dim == 64 ? attn::launch_rows<__nv_bfloat16, 64>(w, plan, st)
                              : attn::launch_rows<__nv_bfloat16, 128>(w, plan, st);
  else
    e = cache->head_dim == 64 ? attn::launch_rows<__half, 64>(w, plan, st)
                              : attn::launch_rows<__half, 128>(w, plan, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
