// moe_prefix_tree.cu -- moe_prefix_attention of short sequences, as in moe_tree_attention with the shared pages from the
// group's first sequence.  What K and V of a short prefix cost more than once (they are in L2) is less than the tiles
// of 128 rows take for their items and for joining them.
#include "moe_tree.cuh"

namespace attn {

// Up to which a sequence's positions may go, for clusters of 8.  (us by clusters and by the tiles, with a table
// that could hold more.  32 query, 8 key/value heads of 128, 2 tokens behind 600, 4000, 8000 and 14000 positions,
// clusters of 8: 7.8, 18.0; 14.2, 22.2; 22.1, 26.5; 33.7, 28.7.  Drafts of 8: 11.2, 18.3; 19.1, 22.4; 29.0, 25.0.  2
// key/value heads, clusters of 16: 7.1, 16.9; 10.3, 22.3; 13.3, 26.7; 18.0, 31.4.)
constexpr int64_t kFewRows = 8192, kMoreRows = 4096;

// With more items all CTAs share them, when K and V of all sequences are no more than this: the tiles take 16 us and
// some for each item (a sequence and key/value head), which goes by its rows; the line 9 and the bytes at 8.9 TB/s.
// (us on the tiles and so, one token a sequence, 32 query, 8 key/value heads of 128.  8 sequences behind 1024 + 200
// positions, 40 MB: 18.0, 15.4; 4096 + 200, 141 MB: 22.1, 25.8.  64 sequences, 128 + 50, 47 MB: 30.5, 17.3; 512 + 100,
// 160 MB: 29.3, 30.4.  Drafts of 8, 64 sequences, 1024 + 200, 321 MB: 71.7, 62.9; 2048 + 100, 563 MB: 71.8, 94.0.)
static bool line_is_shorter(double items, double rows, double bytes) {
  return bytes <= 8.9e6 * (7 + items * (0.016 + 0.0018 * rows));
}

static int plan_prefix(const moe_kv_cache *c, const Params &p, bool *takes, Plan *plan) {
  const int64_t positions = static_cast<int64_t>(p.table_width) << p.page_shift;
  const int64_t rows = static_cast<int64_t>(p.max_q) * p.group, items = static_cast<int64_t>(p.n_seqs) * p.hkv;
  *takes = false;
  if (rows > 32) return MOE_OK;
  const int64_t most = static_cast<int64_t>(p.n_rows) * p.group / (rows <= 16 ? 16 : 32) + p.n_seqs;
  int rc = make_plan(c, p, p.n_seqs, most, rows, positions, plan);
  // (38 drafts of 4 behind 4000 positions, one key/value head, 304 CTAs in clusters: 33.7 us, 25.3 on the tiles; 18
  // tokens, 2 heads, 288 CTAs: 15.9, 27.8)
  if (rc == MOE_OK && plan->cluster > 0 && resident(*plan) &&
      (plan->cluster == 16 || positions <= (rows <= 16 ? kFewRows : kMoreRows))) {
    *takes = true;
    return rc;
  }
  if (!line_is_shorter(items, rows, 4. * items * positions * c->head_dim)) return MOE_OK;
  rc = make_plan(c, p, p.n_seqs, most, rows, positions, plan, false);
  *takes = rc == MOE_OK;
  return rc;
}

int prefix_tree_workspace(const moe_kv_cache *c, const Params &p, bool *takes, int64_t *bytes) {
  Plan plan;
  const int rc = plan_prefix(c, p, takes, &plan);
  if (rc == MOE_OK && *takes) *bytes = plan.bytes;
  return rc;
}

template <typename T, int D>
static cudaError_t launch_rows(const Work &w, const Plan &plan, cudaStream_t stream) {
  const int items = w.p.n_seqs * w.p.hkv;
  if (!plan.cluster)
    return plan.rows == 16 ? launch_line<T, D, 1, kGrouped>(w, plan.grid, stream)
                           : launch_line<T, D, 2, kGrouped>(w, plan.grid, stream);
  if (plan.rows == 16)
    return plan.cluster == 8 ? launch_cluster<T, D, 1, 8, kGrouped>(w, items, stream)
                             : launch_cluster<T, D, 1, 16, kGrouped>(w, items, stream);
  return plan.cluster == 8 ? launch_cluster<T, D, 2, 8, kGrouped>(w, items, stream)
                           : launch_cluster<T, D, 2, 16, kGrouped>(w, items, stream);
}

int run_prefix_tree(const moe_kv_cache *c, const Params &p, const Prefixes &g, void *workspace,
                    int64_t workspace_bytes, cudaStream_t stream) {
  Plan plan;
  bool takes;
  const int rc = plan_prefix(c, p, &takes, &plan);
  if (rc != MOE_OK) return rc;
  if (plan.bytes && (!workspace || workspace_bytes < plan.bytes)) return MOE_ERR_INVALID_ARG;
  Work w = {};
  w.p = p;
  w.g = g;
  use_workspace(plan, workspace, &w);
  cudaError_t e;
  if (c->dtype == MOE_DTYPE_BF16)
    e = c->head_dim == 64 ? launch_rows<__nv_bfloat16, 64>(w, plan, stream)
                          : launch_rows<__nv_bfloat16, 128>(w, plan, stream);
  else
    e = c->head_dim == 64 ? launch_rows<__half, 64>(w, plan, stream)
                          : launch_rows<__half, 128>(w, plan, stream);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace attn
