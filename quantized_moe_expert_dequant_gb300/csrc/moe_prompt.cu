// moe_prompt.cu -- causal attention of packed prompts (moe_prompt_attention).
#include "moe_tiles.cuh"

namespace attn {

int tiles_workspace(const moe_kv_cache *cache, const Params &p, int64_t *bytes) {
  PromptPlan plan;
  const int rc = make_plan(cache, p, &plan);
  if (rc == MOE_OK) *bytes = plan.bytes;
  return rc;
}

int run_tiles(const moe_kv_cache *cache, const Params &p, void *workspace, int64_t workspace_bytes,
              cudaStream_t stream) {
  return p.mask ? run_tree_tiles(cache, p, workspace, workspace_bytes, stream)
                : run<false>(cache, p, workspace, workspace_bytes, stream);
}

}  // namespace attn

extern "C" int moe_prompt_attention_workspace(const moe_kv_cache *cache, const moe_attention *a,
                                              int64_t *bytes) {
  attn::Params p;
  const int rc = attn::check_attention(cache, a, &p);
  if (rc != MOE_OK) return rc;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  if (p.n_seqs == 0 || p.n_rows == 0) {
    *bytes = 0;
    return MOE_OK;
  }
  return attn::tiles_workspace(cache, p, bytes);
}

extern "C" int moe_prompt_attention(const moe_kv_cache *cache, const moe_attention *a,
                                    void *workspace, int64_t workspace_bytes, void *stream) {
  attn::Params p;
  const int rc = attn::check_attention(cache, a, &p);
  if (rc != MOE_OK) return rc;
  if (workspace_bytes < 0 || !attn::aligned(workspace, 16)) return MOE_ERR_INVALID_ARG;
  if (p.n_seqs == 0 || p.n_rows == 0) return MOE_OK;
  return attn::run_tiles(cache, p, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" int moe_debug_attention_wait_cycles(int64_t cycles) {
  if (cycles < 0) return MOE_ERR_INVALID_ARG;
  attn::debug_wait_cycles.store(cycles, std::memory_order_relaxed);
  return MOE_OK;
}
