// moe_sparse_cluster.cu -- the form of moe_sparse_attention in which a cluster of CTAs takes a row.
#include "moe_sparse.cuh"

namespace attn {

template <typename T, int D>
cudaError_t launch_listed_clusters(const Work &w, int rows, int cs, cudaStream_t stream) {
  const int items = w.p.n_rows * w.p.hkv;
  if (rows == 16)
    return cs == 8 ? launch_cluster<T, D, 1, 8, kListed>(w, items, stream)
                   : launch_cluster<T, D, 1, 16, kListed>(w, items, stream);
  return cs == 8 ? launch_cluster<T, D, 2, 8, kListed>(w, items, stream)
                 : launch_cluster<T, D, 2, 16, kListed>(w, items, stream);
}

template cudaError_t launch_listed_clusters<__nv_bfloat16, 64>(const Work &, int, int, cudaStream_t);
template cudaError_t launch_listed_clusters<__nv_bfloat16, 128>(const Work &, int, int, cudaStream_t);
template cudaError_t launch_listed_clusters<__half, 64>(const Work &, int, int, cudaStream_t);
template cudaError_t launch_listed_clusters<__half, 128>(const Work &, int, int, cudaStream_t);

}  // namespace attn
