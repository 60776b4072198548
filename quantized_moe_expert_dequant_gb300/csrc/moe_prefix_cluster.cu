// moe_prefix_cluster.cu -- moe_prefix_attention of few and short sequences: a cluster of CTAs takes each, as in
// moe_tree_attention, with the shared pages from the group's first sequence.  What K and V of a short prefix cost
// more than once (they are in L2) is less than the tiles of 128 rows with their joining kernel take.
#include "moe_tree.cuh"

namespace attn {

// Up to which a sequence's positions may go, for clusters of 8.  (us by clusters and by the tiles, with a table
// that could hold more.  32 query, 8 key/value heads of 128, 2 tokens behind 600, 4000, 8000 and 14000 positions,
// clusters of 8: 7.8, 18.0; 14.2, 22.2; 22.1, 26.5; 33.7, 28.7.  Drafts of 8: 11.2, 18.3; 19.1, 22.4; 29.0, 25.0.  2
// key/value heads, clusters of 16: 7.1, 16.9; 10.3, 22.3; 13.3, 26.7; 18.0, 31.4.)
constexpr int64_t kFewRows = 8192, kMoreRows = 4096;

int takes_prefix_clusters(const moe_kv_cache *c, const Params &p, bool *takes) {
  const int64_t positions = static_cast<int64_t>(p.table_width) << p.page_shift;
  const int64_t rows = static_cast<int64_t>(p.max_q) * p.group;
  *takes = false;
  if (rows > 32) return MOE_OK;
  Plan plan;
  const int rc = make_plan(c, p, p.n_seqs, p.n_rows, rows, positions, &plan);
  // (304 CTAs in clusters of 8 are not all resident at once: 38 drafts of 4 behind 4000 positions, one key/value
  // head: 33.7 us, 25.3 on the tiles; 288 are: 18 tokens, 2 heads, 15.9 and 27.8)
  *takes = rc == MOE_OK && plan.cluster > 0 && 10 * static_cast<int64_t>(plan.grid) <= 19 * plan.sms &&
           (plan.cluster == 16 || positions <= (rows <= 16 ? kFewRows : kMoreRows));
  return rc;
}

template <typename T, int D>
static cudaError_t launch_rows(const Work &w, const Plan &plan, cudaStream_t stream) {
  const int items = w.p.n_seqs * w.p.hkv;
  if (plan.rows == 16)
    return plan.cluster == 8 ? launch_cluster<T, D, 1, 8, kGrouped>(w, items, stream)
                             : launch_cluster<T, D, 1, 16, kGrouped>(w, items, stream);
  return plan.cluster == 8 ? launch_cluster<T, D, 2, 8, kGrouped>(w, items, stream)
                           : launch_cluster<T, D, 2, 16, kGrouped>(w, items, stream);
}

int run_prefix_clusters(const moe_kv_cache *c, const Params &p, const Prefixes &g, cudaStream_t stream) {
  Plan plan;
  const int64_t rows = static_cast<int64_t>(p.max_q) * p.group;
  const int rc = make_plan(c, p, p.n_seqs, p.n_rows, rows,
                           static_cast<int64_t>(p.table_width) << p.page_shift, &plan);
  if (rc != MOE_OK) return rc;
  Work w = {};
  w.p = p;
  w.g = g;
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
