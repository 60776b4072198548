// moe_sparse.cu -- moe_sparse_attention: attention of each row over the pages that are listed for it.
//
// The kernel is that of moe_tree.cuh with another reading of positions: an item is one row and one key/value
// head, its line of positions the listed pages one after the other.  The row's query heads are the rows of
// the matrix products.  Bound by the bytes of K and V on the listed pages: 32 tokens, 32 pages of 64, 8 heads of 128
// (261 MB) 48.6 us, of which start and join take 7.5; by what a tile costs where they lie in L2: 512 rows, 100 pages of
// 16, 2 heads of 64 (419 MB) 62 us; by latency for one token (9.5 us).  (A third CTA an SM with a stage less, heads of
// 64: 57.6 us on those 512 rows, but 114 us for 87 on 64 tokens with 16 heads.)
#include "moe_sparse.cuh"

namespace attn {

static int plan_sparse(const moe_kv_cache *c, const Params &p, int n_list, Plan *plan) {
  const int64_t pages = std::min<int64_t>(p.table_width, n_list);
  const int rc = make_plan(c, p, p.n_rows, p.n_rows, p.group, pages << p.page_shift, plan);
  if (rc != MOE_OK || !plan->cluster || resident(*plan)) return rc;
  return make_plan(c, p, p.n_rows, p.n_rows, p.group, pages << p.page_shift, plan, false);
}

template <typename T, int D>
static cudaError_t launch_rows(const Work &w, const Plan &plan, cudaStream_t stream) {
  if (plan.cluster)
    return launch_listed_clusters<T, D>(w, plan.rows, plan.cluster, stream);
  return plan.rows == 16 ? launch_line<T, D, 1, kListed>(w, plan.grid, stream)
                         : launch_line<T, D, 2, kListed>(w, plan.grid, stream);
}

static int check_sparse(const moe_kv_cache *cache, const moe_attention *a, int n_select, Params *p) {
  const int rc = check_attention(cache, a, p);
  if (rc != MOE_OK) return rc;
  if (n_select < 1) return MOE_ERR_INVALID_ARG;
  return p->group > 32 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

}  // namespace attn

extern "C" int moe_sparse_attention_workspace(const moe_kv_cache *cache, const moe_attention *a,
                                              int32_t n_select, int64_t *bytes) {
  attn::Params p;
  int rc = attn::check_sparse(cache, a, n_select, &p);
  if (rc != MOE_OK) return rc;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = 0;
  if (p.n_seqs == 0 || p.n_rows == 0) return MOE_OK;
  attn::Plan plan;
  rc = attn::plan_sparse(cache, p, n_select, &plan);
  if (rc == MOE_OK) *bytes = plan.bytes;
  return rc;
}

extern "C" int moe_sparse_attention(const moe_kv_cache *cache, const moe_attention *a,
                                    const int32_t *pages, int32_t n_select, void *workspace,
                                    int64_t workspace_bytes, void *stream) {
  attn::Work w;
  int rc = attn::check_sparse(cache, a, n_select, &w.p);
  if (rc != MOE_OK) return rc;
  if (!attn::aligned(pages, 4) || workspace_bytes < 0 || !attn::aligned(workspace, 16))
    return MOE_ERR_INVALID_ARG;
  if (w.p.n_seqs == 0 || w.p.n_rows == 0) return MOE_OK;
  if (!pages) return MOE_ERR_INVALID_ARG;
  attn::Plan plan;
  rc = attn::plan_sparse(cache, w.p, n_select, &plan);
  if (rc != MOE_OK) return rc;
  if (plan.bytes && (!workspace || workspace_bytes < plan.bytes)) return MOE_ERR_INVALID_ARG;
  attn::use_workspace(plan, workspace, &w);
  w.list = pages;
  w.n_list = n_select;
  w.g = {};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (cache->dtype == MOE_DTYPE_BF16)
    e = cache->head_dim == 64 ? attn::launch_rows<__nv_bfloat16, 64>(w, plan, st)
                              : attn::launch_rows<__nv_bfloat16, 128>(w, plan, st);
  else
    e = cache->head_dim == 64 ? attn::launch_rows<__half, 64>(w, plan, st)
                              : attn::launch_rows<__half, 128>(w, plan, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
