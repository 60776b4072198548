// moe_tree_cluster.cu -- the form of moe_tree_attention in which a cluster of CTAs takes an item.
#include "moe_tree.cuh"

namespace attn {

template <typename T, int D, int WR, int CS>
static cudaError_t launch(const Work &w, cudaStream_t stream) {
  const auto kern = tree_kernel<T, D, WR, CS>;
  static SmemLimit limit;
  cudaError_t e = limit.set(reinterpret_cast<const void *>(kern), Tree<D>::kSmem, CS > 8);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(w.p.n_seqs * w.p.hkv * CS);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Tree<D>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = CS;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, w);
}

template <typename T, int D>
static cudaError_t launch_rows(const Work &w, int rows, int cs, cudaStream_t stream) {
  if (rows == 16)
    return cs == 8 ? launch<T, D, 1, 8>(w, stream) : launch<T, D, 1, 16>(w, stream);
  return cs == 8 ? launch<T, D, 2, 8>(w, stream) : launch<T, D, 2, 16>(w, stream);
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
