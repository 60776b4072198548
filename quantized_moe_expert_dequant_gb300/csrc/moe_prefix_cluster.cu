// moe_prefix_cluster.cu -- moe_prefix_attention of few and short sequences: a cluster of CTAs takes each, as in
// moe_tree_attention, with the shared pages from the group's first sequence.  What K and V of a short prefix cost
// more than once (they are in L2) is less than the tiles of 128 rows with their joining kernel take.
#include "moe_tree.cuh"

namespace attn {

// Up to which a sequence's positions may go.
constexpr int64_t kShortPositions = 4096;

int takes_prefix_clusters(const moe_kv_cache *c, const Params &p, bool *takes) {
  const int64_t positions = static_cast<int64_t>(p.table_width) << p.page_shift;
  const int64_t rows = static_cast<int64_t>(p.max_q) * p.group;
  *takes = false;
  if (rows > 32 || positions > kShortPositions) return MOE_OK;
  Plan plan;
  const int rc = make_plan(c, p, p.n_seqs, p.n_rows, rows, positions, &plan);
  *takes = rc == MOE_OK && plan.cluster > 0;
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
