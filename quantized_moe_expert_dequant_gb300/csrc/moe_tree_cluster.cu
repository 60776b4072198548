// moe_tree_cluster.cu -- the form of moe_tree_attention in which a cluster of CTAs takes an item.
#include "moe_tree.cuh"

namespace attn {

template <typename T, int D>
static cudaError_t launch_rows(const Work &w, int rows, int cs, cudaStream_t stream) {
  const int items = w.p.n_seqs * w.p.hkv;
  if (rows == 16)
    return cs == 8 ? launch_cluster<T, D, 1, 8, kSeqs>(w, items, stream)
                   : launch_cluster<T, D, 1, 16, kSeqs>(w, items, stream);
  return cs == 8 ? launch_cluster<T, D, 2, 8, kSeqs>(w, items, stream)
                 : launch_cluster<T, D, 2, 16, kSeqs>(w, items, stream);
}

cudaError_t launch_clusters(const moe_kv_cache *c, const Work &w, int rows, int cs,
                            cudaStream_t stream) {
  if (c->dtype == MOE_DTYPE_BF16)
    return c->head_dim == 64 ? launch_rows<__nv_bfloat16, 64>(w, rows, cs, stream)
                             : launch_rows<__nv_bfloat16, 128>(w, rows, cs, stream);
  return c->head_dim == 64 ? launch_rows<__half, 64>(w, rows, cs, stream)
                           : launch_rows<__half, 128>(w, rows, cs, stream);
}

}  // namespace attn
