// moe_sparse.cuh -- what the two translation units of moe_sparse_attention share.
#pragma once

#include "moe_tree.cuh"

namespace attn {

// Few rows: each and each key/value head by a cluster of cs (8 or 16) CTAs (moe_sparse_cluster.cu).
template <typename T, int D>
cudaError_t launch_listed_clusters(const Work &w, int rows, int cs, cudaStream_t stream);

}  // namespace attn
