// moe_attention.cuh -- what the attention kernels share: the launch parameters, the checks of a
// sequence's device-side description, 16-bit types and the mma.sync building blocks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "moe_decode.h"

namespace attn {

constexpr int kDevErrBadId = 1;    // the bits of a device error word (moe_status documents them)
constexpr int kDevErrTimeout = 2;
constexpr float kNegInf = -__builtin_huge_valf();

struct Params {
  const void *q, *k, *v;
  void *out;
  int64_t q_row, q_head, o_row, o_head;         // element strides
  int64_t page_stride, head_stride, tok_stride;  // element strides of K and V alike
  const int32_t *cu, *ctx, *table;
  const uint64_t *mask;                          // tree masks, or null: causal
  int32_t *err;
  int64_t table_stride;
  int n_seqs, n_rows, table_width, n_pages, page_shift, hq, hkv, group, max_q;
  float scale_log2;                              // scale * log2(e)
  float octave;                                  // by how much the score of half a weight is less
};

constexpr int kMaxLen = 1 << 30;  // positions of a sequence: every index of one fits 32 bits

// One sequence's queries and positions, checked against the host's bounds: a description that is
// out of range sets the error bit and counts as a sequence without queries.
struct Seq {
  int row0, nq, ctx, len;  // first row, rows, positions before them, positions in all
};

__device__ __forceinline__ Seq load_seq(const Params &p, int s, bool report) {
  Seq r;
  r.row0 = p.cu[s];
  const int64_t end = p.cu[s + 1];
  r.ctx = p.ctx[s];
  const int64_t nq = end - r.row0;
  const int64_t len = nq + r.ctx;
  const bool ok = r.row0 >= 0 && nq >= 0 && end <= p.n_rows && nq <= p.max_q && r.ctx >= 0 &&
                  len <= (static_cast<int64_t>(p.table_width) << p.page_shift) && len <= kMaxLen;
  if (!ok && report && p.err) atomicOr(p.err, kDevErrBadId);
  r.nq = ok ? static_cast<int>(nq) : 0;
  r.len = ok ? static_cast<int>(len) : 0;
  return r;
}

__device__ __forceinline__ void pdl_launch() {  // the next kernel may be set up
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() {  // the kernel before this one has ended
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ float exp2_approx(float x) {  // 2 ulp; -inf gives 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 bytes global -> shared; reads nothing and writes zeros when !valid.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// The 16-bit type of a cache.
//
// The softmax's weights meet v in it: half a step of rounding relative to each weight, the size of the output's
// own rounding, as long as the type has the range.  bf16 has fp32's.  fp16 ends at 65504 and loses bits
// below 2^-14, while its 2^-25 (half the least step) times 10^5 positions is more than its precision: so
// weights are formed times 2^kRow (moe_tree.cuh) or relative to less than the maximum (reference, in
// moe_tiles.cuh), which divides out.  (One reference over 131072 positions, N(0, 1) scores, a first position
// 17 above with v = 0: relative error of the output 3.7e-2 without.)
template <typename T>
struct Half;

template <>
struct Half<__nv_bfloat16> {
  static constexpr float kRow = 0.f;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  // D[16 x 8] += A[16 x 16] B[16 x 8], fp32 accumulation.
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

template <>
struct Half<__half> {
  static constexpr float kRow = 15.f;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    const __half2 h = *reinterpret_cast<const __half2 *>(&w);
    return __half22float2(h);
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

// ------------------------------------------------------------------ host side
inline bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

inline bool bad_stride(int64_t s) { return s < 0 || s % 8; }

// Checks a cache description; page_size is bounded further by the attention calls.
inline int check_cache(const moe_kv_cache *c) {
  if (!c || !c->k || !c->v || c->n_pages < 1 || c->page_size < 1 || c->n_kv_heads < 1)
    return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_DTYPE_BF16 && c->dtype != MOE_DTYPE_F16) return MOE_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || bad_stride(c->page_stride) ||
      bad_stride(c->head_stride) || bad_stride(c->token_stride))
    return MOE_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return MOE_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(c->n_pages) * c->page_size > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Checks an attention call's arguments and fills the kernels' parameters.
inline int check_attention(const moe_kv_cache *c, const moe_attention *a, Params *p) {
  const int rc = check_cache(c);
  if (rc != MOE_OK) return rc;
  if (!a || a->n_seqs < 0 || a->n_rows < 0 || a->n_q_heads < 1 || a->n_q_heads % c->n_kv_heads)
    return MOE_ERR_INVALID_ARG;
  if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
    return MOE_ERR_UNSUPPORTED;
  if (a->n_q_heads / c->n_kv_heads > 64) return MOE_ERR_UNSUPPORTED;
  if (a->n_rows > 0 && a->n_seqs > 0) {
    if (!a->q || !a->out || !a->cu_q || !a->ctx_len || !a->page_table) return MOE_ERR_INVALID_ARG;
    if (a->table_width < 1 || a->table_stride < a->table_width) return MOE_ERR_INVALID_ARG;
  }
  if (!(a->scale > 0.f) || a->scale > 1e30f) return MOE_ERR_INVALID_ARG;
  if (!aligned(a->q, 16) || !aligned(a->out, 16) || !aligned(a->cu_q, 4) ||
      !aligned(a->ctx_len, 4) || !aligned(a->page_table, 4) || !aligned(a->device_error, 4) ||
      bad_stride(a->q_row_stride) || bad_stride(a->q_head_stride) ||
      bad_stride(a->out_row_stride) || bad_stride(a->out_head_stride))
    return MOE_ERR_INVALID_ARG;
  p->q = a->q;
  p->k = c->k;
  p->v = c->v;
  p->out = a->out;
  p->q_row = a->q_row_stride;
  p->q_head = a->q_head_stride;
  p->o_row = a->out_row_stride;
  p->o_head = a->out_head_stride;
  p->page_stride = c->page_stride;
  p->head_stride = c->head_stride;
  p->tok_stride = c->token_stride;
  p->cu = a->cu_q;
  p->ctx = a->ctx_len;
  p->table = a->page_table;
  p->mask = nullptr;
  p->err = a->device_error;
  p->table_stride = a->table_stride;
  p->n_seqs = a->n_seqs;
  p->n_rows = a->n_rows;
  p->table_width = a->table_width;
  p->n_pages = c->n_pages;
  p->page_shift = 31 - __builtin_clz(static_cast<unsigned>(c->page_size));
  p->hq = a->n_q_heads;
  p->hkv = c->n_kv_heads;
  p->group = a->n_q_heads / c->n_kv_heads;
  p->max_q = a->n_rows;
  p->scale_log2 = a->scale * 1.4426950408889634f;
  p->octave = 1.f / std::max(p->scale_log2, 1e-30f);  // (of scores that small, nine are not seen)
  return MOE_OK;
}

// Raises a kernel's limits of dynamic shared memory and cluster size, once per device (a call of the
// runtime takes about a microsecond).
struct SmemLimit {
  std::atomic<uint64_t> done{0};
  cudaError_t set(const void *kernel, int bytes, bool large_clusters = false) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && large_clusters)  // more than 8 CTAs
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
  }
};

// Limit of the tiles' waits in cycles; 0: the usual one (moe_debug_attention_wait_cycles).
inline std::atomic<int64_t> debug_wait_cycles{0};

// Attention in tiles of 128 rows on the 5th-generation tensor cores: causal, or by p.mask
// (moe_prompt.cu, moe_prompt_tree.cu).
int tiles_workspace(const moe_kv_cache *cache, const Params &p, int64_t *bytes);
int run_tiles(const moe_kv_cache *cache, const Params &p, void *workspace, int64_t workspace_bytes,
              cudaStream_t stream);
int run_tree_tiles(const moe_kv_cache *cache, const Params &p, void *workspace,
                   int64_t workspace_bytes, cudaStream_t stream);

}  // namespace attn
