// moe_prompt_tree.cu -- the masked form of the tiles of 128 rows, for large trees of drafted tokens
// (moe_tree_attention).
#include "moe_tiles.cuh"

namespace attn {

int run_tree_tiles(const moe_kv_cache *cache, const Params &p, void *workspace,
                   int64_t workspace_bytes, cudaStream_t stream) {
  return run<kTree>(cache, p, workspace, workspace_bytes, stream);
}

}  // namespace attn
