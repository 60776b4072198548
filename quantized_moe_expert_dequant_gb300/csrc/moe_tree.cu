// moe_tree.cu -- moe_tree_attention: the plan, and the form in which all CTAs share all items.
#include "moe_tree.cuh"

namespace attn {

struct Plan {
  int grid, rows;  // CTAs, rows of a tile
  int cluster;     // CTAs of an item's cluster; 0: all CTAs share all items
  int64_t part, ml, shared, bytes;  // offsets in the workspace
};

// More than 32 rows an item are compute on mma.sync tiles, which read K and V once for 64 rows; the
// tiles of 128 rows on tcgen05 keep up with memory.  Drafts of up to 64 tokens over contexts of up to
// 9000 (12 query, 2 key/value heads of 128): 46.0 us here, 34.9 there; 8 tokens behind 131000
// positions (32 query, 8 key/value heads: 32 rows): 263 us here, at the copy rate.
static bool many_rows(const Params &p) { return static_cast<int64_t>(p.max_q) * p.group > 32; }

constexpr int64_t kClusterPositions = 16384;  // up to which a cluster takes an item

static int make_plan(const moe_kv_cache *c, const Params &p, int max_q, Plan *plan) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MOE_ERR_CUDA;
  const int64_t rows = static_cast<int64_t>(max_q) * p.group;
  plan->rows = rows <= 16 ? 16 : 32;
  // With few items a cluster takes each, when the 16 or 8 CTAs of every one can be resident at once: one
  // kernel instead of two.  (32 query, 8 key/value heads of 128, one token, shared line against clusters
  // of 16: 500 positions 8.5, 6.8 us; 4000 15.1, 10.8; 8000 18.2, 14.8; 16000 21.8, 22.6; 32000 34.7,
  // 39.2.  16 items of 4000: 15.2, clusters of 16 17.2, of 8 12.4; 32 items of 2000: 13.8, of 8 10.1.)
  plan->cluster = 0;
  plan->part = plan->ml = plan->shared = plan->bytes = 0;
  const int64_t clusters = static_cast<int64_t>(p.n_seqs) * p.hkv;
  if ((static_cast<int64_t>(p.table_width) << p.page_shift) <= kClusterPositions)
    plan->cluster = clusters * 16 <= sms ? 16 : clusters * 8 <= sms * kCtasPerSm ? 8 : 0;
  plan->grid = static_cast<int>(clusters) * plan->cluster;
  if (plan->cluster) return MOE_OK;
  // no more CTAs than the largest batch that the arguments allow has work for
  const int64_t len =
      (static_cast<int64_t>(p.table_width) << p.page_shift) / tile_of(c->head_dim) + 1;
  const int64_t items =
      (static_cast<int64_t>(p.n_rows) * p.group / plan->rows + p.n_seqs) * p.hkv;
  const int64_t most = len >= INT32_MAX || items >= INT32_MAX ? INT64_MAX : items * len;
  if (most / (sms * kCtasPerSm) >= INT32_MAX) return MOE_ERR_UNSUPPORTED;
  plan->grid = static_cast<int>(
      std::min<int64_t>(sms * kCtasPerSm, most * tile_of(c->head_dim) / kMinPositions + 1));
  plan->part = 0;
  plan->ml = plan->part + 8ll * plan->grid * plan->rows * c->head_dim;
  plan->shared = plan->ml + 16ll * plan->grid * plan->rows;
  plan->bytes = plan->shared + static_cast<int64_t>(sizeof(Shared)) * plan->grid;
  return MOE_OK;
}

template <typename T, int D, int WR>
static cudaError_t launch(const Work &w, int grid, cudaStream_t stream) {
  const auto kern = tree_kernel<T, D, WR, 0>;
  static SmemLimit limit;
  cudaError_t e = limit.set(reinterpret_cast<const void *>(kern), Tree<D>::kSmem);
  if (e != cudaSuccess) return e;
  kern<<<grid, kThreads, Tree<D>::kSmem, stream>>>(w);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // the joining blocks are set up while the kernel runs and wait for its end
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 16 * WR / (kThreads / 32));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<T, D, 16 * WR>, w);
}

template <typename T, int D>
static cudaError_t launch_rows(const Work &w, const Plan &plan, cudaStream_t stream) {
  if (plan.rows == 16) return launch<T, D, 1>(w, plan.grid, stream);
  return launch<T, D, 2>(w, plan.grid, stream);
}

}  // namespace attn

extern "C" int moe_tree_attention_workspace(const moe_kv_cache *cache, const moe_attention *a,
                                            int32_t max_q, int64_t *bytes) {
  attn::Params p;
  int rc = attn::check_attention(cache, a, &p);
  if (rc != MOE_OK) return rc;
  if (max_q < 1 || !bytes) return MOE_ERR_INVALID_ARG;
  if (max_q > MOE_TREE_MAX_Q) return MOE_ERR_UNSUPPORTED;
  if (p.n_seqs == 0 || p.n_rows == 0) {
    *bytes = 0;
    return MOE_OK;
  }
  p.max_q = max_q;
  if (attn::many_rows(p)) return attn::tiles_workspace(cache, p, bytes);
  attn::Plan plan;
  rc = attn::make_plan(cache, p, max_q, &plan);
  if (rc == MOE_OK) *bytes = plan.bytes;
  return rc;
}

extern "C" int moe_tree_attention(const moe_kv_cache *cache, const moe_attention *a,
                                  const uint64_t *tree_mask, int32_t max_q, void *workspace,
                                  int64_t workspace_bytes, void *stream) {
  attn::Work w;
  int rc = attn::check_attention(cache, a, &w.p);
  if (rc != MOE_OK) return rc;
  if (max_q < 1 || !attn::aligned(tree_mask, 8) || workspace_bytes < 0 ||
      !attn::aligned(workspace, 16))
    return MOE_ERR_INVALID_ARG;
  if (max_q > MOE_TREE_MAX_Q) return MOE_ERR_UNSUPPORTED;
  if (w.p.n_seqs == 0 || w.p.n_rows == 0) return MOE_OK;
  w.p.mask = tree_mask;
  w.p.max_q = max_q;
  if (attn::many_rows(w.p))
    return attn::run_tiles(cache, w.p, workspace, workspace_bytes,
                           static_cast<cudaStream_t>(stream));
  attn::Plan plan;
  rc = attn::make_plan(cache, w.p, max_q, &plan);
  if (rc != MOE_OK) return rc;
  if (plan.bytes && (!workspace || workspace_bytes < plan.bytes)) return MOE_ERR_INVALID_ARG;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  w.part = reinterpret_cast<float *>(ws + plan.part);
  w.part_ml = reinterpret_cast<float2 *>(ws + plan.ml);
  w.shared = reinterpret_cast<attn::Shared *>(ws + plan.shared);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (plan.cluster)
    e = attn::launch_clusters(cache, w, plan.rows, plan.cluster, st);
  else if (cache->dtype == MOE_DTYPE_BF16)
    e = cache->head_dim == 64 ? attn::launch_rows<__nv_bfloat16, 64>(w, plan, st)
                              : attn::launch_rows<__nv_bfloat16, 128>(w, plan, st);
  else
    e = cache->head_dim == 64 ? attn::launch_rows<__half, 64>(w, plan, st)
                              : attn::launch_rows<__half, 128>(w, plan, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
