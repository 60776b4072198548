// moe_prompt_shared.cu -- attention of decoded or drafted tokens of sequences that share their first pages
// (moe_prefix_attention), in the tiles of 128 rows.
//
// The rows of all sequences of a group over their shared positions are one item's rows, so that K and V of the
// prefix are read once for up to 256 rows; the positions that a sequence has for itself are items of their own.
// Both lie on one line that the CTAs share evenly, and one kernel joins their parts.  Bound by the products on long
// prefixes (32 sequences of 8 tokens behind 65536 positions, 32 query, 8 key/value heads of 128: 240 us, a step of 256
// rows and 128 positions 1.51 us), by memory and the beginning and end of items otherwise (64 tokens behind 8192 shared
// positions and 500 of their own: 52 us, floor 24).
#include "moe_tiles.cuh"

namespace attn {

static int check_prefix(const moe_kv_cache *cache, const moe_attention *a, int n_groups, int max_q,
                        Params *p) {
  const int rc = check_attention(cache, a, p);
  if (rc != MOE_OK) return rc;
  if (n_groups < 0 || max_q < 1) return MOE_ERR_INVALID_ARG;
  p->max_q = max_q;
  if (max_q > MOE_TREE_MAX_Q) return MOE_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(p->n_seqs) * p->hkv > INT32_MAX ||
      static_cast<int64_t>(p->n_seqs) + n_groups > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace attn

extern "C" int moe_prefix_attention_workspace(const moe_kv_cache *cache, const moe_attention *a,
                                              int32_t n_groups, int32_t max_q, int64_t *bytes) {
  attn::Params p;
  const int rc = attn::check_prefix(cache, a, n_groups, max_q, &p);
  if (rc != MOE_OK) return rc;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = 0;
  if (p.n_seqs == 0 || p.n_rows == 0) return MOE_OK;
  bool tree;
  int err = attn::prefix_tree_workspace(cache, p, &tree, bytes);
  if (err != MOE_OK || tree) return err;
  attn::PromptPlan plan;
  err = attn::make_plan(cache, p, &plan, n_groups);
  if (err == MOE_OK) *bytes = plan.bytes;
  return err;
}

extern "C" int moe_prefix_attention(const moe_kv_cache *cache, const moe_attention *a,
                                    const int32_t *cu_group, const int32_t *prefix_len,
                                    int32_t n_groups, const uint64_t *tree_mask, int32_t max_q,
                                    void *workspace, int64_t workspace_bytes, void *stream) {
  attn::Params p;
  const int rc = attn::check_prefix(cache, a, n_groups, max_q, &p);
  if (rc != MOE_OK) return rc;
  if (!attn::aligned(cu_group, 4) || !attn::aligned(prefix_len, 4) || !attn::aligned(tree_mask, 8) ||
      workspace_bytes < 0 || !attn::aligned(workspace, 16))
    return MOE_ERR_INVALID_ARG;
  if (p.n_seqs == 0 || p.n_rows == 0) return MOE_OK;
  if (n_groups > 0 && (!cu_group || !prefix_len)) return MOE_ERR_INVALID_ARG;
  p.mask = tree_mask;
  const attn::Prefixes g = {cu_group, prefix_len, n_groups};
  bool tree;
  int64_t bytes;
  int err = attn::prefix_tree_workspace(cache, p, &tree, &bytes);
  if (err != MOE_OK) return err;
  if (tree)
    return attn::run_prefix_tree(cache, p, g, workspace, workspace_bytes,
                                 static_cast<cudaStream_t>(stream));
  attn::PromptPlan plan;
  err = attn::make_plan(cache, p, &plan, n_groups);
  if (err != MOE_OK) return err;
  return attn::run_planned<attn::kShared>(cache, p, g, plan, workspace, workspace_bytes,
                                          static_cast<cudaStream_t>(stream));
}
