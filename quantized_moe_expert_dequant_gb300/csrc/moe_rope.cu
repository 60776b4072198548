// moe_rope.cu -- norms of the query and key heads and the position rotation in one pass, with the
// keys and values written to their slots in the pages of a cache (moe_qk_norm_rope).
//
//   y = gamma * x / sqrt(mean(x^2) + eps)                          per query and key head
//   (y_a, y_b) -> (y_a cos t - y_b sin t, y_b cos t + y_a sin t),  t = position * inv_freq[i]
//
// for the pairs (a, b) = (i, i + R/2) or (2i, 2i + 1), i < R/2; elements from R on are not turned,
// values are only rounded.  Everything is fp32 until one rounding at the end.
//
// A head is D / 16 lanes wide: each lane holds two runs of 8 elements, chosen so that both members
// of its rotated pairs are its own, so a head needs log2(D / 16) shuffles (the mean) and no
// shared memory.  The angles of a token are the same for all of its heads: the block forms them
// once.  An angle is reduced to turns in fp64 (a position near 10^6 has an fp32 angle with an
// error of 0.03 rad), its sine and cosine are fp32 (sincospif).
#include "moe_attention.cuh"

namespace rope {

struct Args {
  const void *in[3];              // q, k, v
  int64_t row[3], head[3];        // element strides
  void *q_out, *k, *v;
  int64_t qo_row, qo_head, page_stride, head_stride, tok_stride;
  const void *gamma[2];
  const double *inv_freq;
  const int32_t *positions, *slots;
  int32_t *err;
  int n_tokens, hq, hkv, rot, interleaved, page_size, n_pages, tokens_per_block;
  float eps;
};

constexpr int kMaxThreads = 512;
constexpr int kMaxTokensPerBlock = 16;

template <typename In>
__device__ __forceinline__ void load8(const In *p, float (&x)[8]) {
  if constexpr (sizeof(In) == 4) {
    const float4 a = *reinterpret_cast<const float4 *>(p);
    const float4 b = *reinterpret_cast<const float4 *>(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = attn::Half<In>::unpack(w[i]);
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
}

template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&x)[8]) {
  uint4 a;
  a.x = attn::Half<T>::pack(x[0], x[1]);
  a.y = attn::Half<T>::pack(x[2], x[3]);
  a.z = attn::Half<T>::pack(x[4], x[5]);
  a.w = attn::Half<T>::pack(x[6], x[7]);
  *reinterpret_cast<uint4 *>(p) = a;
}

template <typename In, typename T, int D>
__global__ void __launch_bounds__(kMaxThreads) norm_rope_kernel(const Args p) {
  constexpr int L = D / 16;  // lanes of a head
  __shared__ float2 s_cs[kMaxTokensPerBlock][D / 2];
  const int heads = p.hq + 2 * p.hkv;
  const int t0 = blockIdx.x * p.tokens_per_block;
  const int nt = min(p.tokens_per_block, p.n_tokens - t0);
  const int half = p.rot / 2;
  for (int i = threadIdx.x; i < nt * half; i += blockDim.x) {
    const int t = i / half, f = i - t * half;
    double turn = static_cast<double>(p.positions[t0 + t]) * p.inv_freq[f] * 0.15915494309189535;
    turn -= rint(turn);
    float2 cs;
    sincospif(2.f * static_cast<float>(turn), &cs.y, &cs.x);
    s_cs[t][f] = cs;
  }
  __syncthreads();
  const int items = nt * heads * L;
  for (int base = 0; base < items; base += blockDim.x) {
    const int it = base + threadIdx.x;
    const bool live = it < items;
    const int unit = (live ? it : 0) / L, l = (live ? it : 0) - unit * L;
    const int t = unit / heads, h = unit - t * heads;
    const int64_t tok = t0 + t;
    const int slot = p.slots[tok];
    const int kind = h < p.hq ? 0 : h < p.hq + p.hkv ? 1 : 2;
    const int hh = h - (kind == 0 ? 0 : kind == 1 ? p.hq : p.hq + p.hkv);
    // the two runs of 8 elements of this lane
    int ca = 2 * l, cb = 2 * l + 1;
    if (!p.interleaved && l < p.rot / 16) ca = l, cb = l + p.rot / 16;
    const bool work = live && slot >= 0;
    float a[8] = {}, b[8] = {};
    if (work) {
      const In *src = static_cast<const In *>(p.in[kind]) + tok * p.row[kind] + hh * p.head[kind];
      load8(src + 8 * ca, a);
      load8(src + 8 * cb, b);
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(a[i], a[i], fmaf(b[i], b[i], sum));
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (!work) continue;
    if (kind < 2) {
      if (p.gamma[kind]) {
        const float r = 1.f / sqrtf(sum * (1.f / D) + p.eps);
        float ga[8], gb[8];
        load8(static_cast<const T *>(p.gamma[kind]) + 8 * ca, ga);
        load8(static_cast<const T *>(p.gamma[kind]) + 8 * cb, gb);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] *= r * ga[i], b[i] *= r * gb[i];
      }
      if (l < p.rot / 16) {
        const float2 *cs = &s_cs[t][8 * l];
        if (p.interleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 u = cs[i], w = cs[4 + i];
            const float x = a[2 * i], y = a[2 * i + 1], z = b[2 * i], q = b[2 * i + 1];
            a[2 * i] = x * u.x - y * u.y, a[2 * i + 1] = y * u.x + x * u.y;
            b[2 * i] = z * w.x - q * w.y, b[2 * i + 1] = q * w.x + z * w.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 u = cs[i];
            const float x = a[i], y = b[i];
            a[i] = x * u.x - y * u.y, b[i] = y * u.x + x * u.y;
          }
        }
      }
    }
    T *dst;
    if (kind == 0) {
      dst = static_cast<T *>(p.q_out) + tok * p.qo_row + hh * p.qo_head;
    } else {
      const int page = slot / p.page_size;
      if (page >= p.n_pages) {
        if (p.err) atomicOr(p.err, attn::kDevErrBadId);
        continue;
      }
      dst = static_cast<T *>(kind == 1 ? p.k : p.v) + page * p.page_stride + hh * p.head_stride +
            (slot - page * p.page_size) * p.tok_stride;
    }
    store8(dst + 8 * ca, a);
    store8(dst + 8 * cb, b);
  }
}

template <typename In, typename T>
static cudaError_t launch(Args p, int dim, cudaStream_t stream) {
  const int per_token = (p.hq + 2 * p.hkv) * (dim / 16);
  p.tokens_per_block = per_token >= 256 ? 1 : 256 / per_token;
  if (p.tokens_per_block > kMaxTokensPerBlock) p.tokens_per_block = kMaxTokensPerBlock;
  int threads = (p.tokens_per_block * per_token + 31) / 32 * 32;
  if (threads > kMaxThreads) threads = kMaxThreads;
  const int grid = (p.n_tokens + p.tokens_per_block - 1) / p.tokens_per_block;
  if (dim == 64)
    norm_rope_kernel<In, T, 64><<<grid, threads, 0, stream>>>(p);
  else
    norm_rope_kernel<In, T, 128><<<grid, threads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace rope

extern "C" int moe_qk_norm_rope(const moe_kv_cache *cache, const moe_norm_rope *a, void *stream) {
  const int rc = attn::check_cache(cache);
  if (rc != MOE_OK) return rc;
  if (!a || a->n_tokens < 0 || a->n_q_heads < 1 || a->rot_dim < 0 ||
      a->rot_dim > cache->head_dim || !(a->eps >= 0.f) || !(a->eps <= 1.f))
    return MOE_ERR_INVALID_ARG;
  if (a->rot_dim % 16) return MOE_ERR_UNSUPPORTED;
  if (a->in_dtype != MOE_DTYPE_F32 && a->in_dtype != cache->dtype) return MOE_ERR_UNSUPPORTED;
  if (a->interleaved != 0 && a->interleaved != 1) return MOE_ERR_INVALID_ARG;
  if (static_cast<int64_t>(a->n_q_heads) + 2 * static_cast<int64_t>(cache->n_kv_heads) > 65536)
    return MOE_ERR_UNSUPPORTED;
  const int64_t unit = a->in_dtype == MOE_DTYPE_F32 ? 4 : 8;  // elements of 16 bytes
  const int64_t in_strides[6] = {a->q_row_stride,  a->q_head_stride, a->k_row_stride,
                                 a->k_head_stride, a->v_row_stride,  a->v_head_stride};
  for (const int64_t s : in_strides)
    if (s < 0 || s % unit) return MOE_ERR_INVALID_ARG;
  if (attn::bad_stride(a->q_out_row_stride) || attn::bad_stride(a->q_out_head_stride))
    return MOE_ERR_INVALID_ARG;
  const void *ptrs[6] = {a->q, a->k, a->v, a->q_out, a->q_weight, a->k_weight};
  for (const void *p : ptrs)
    if (!attn::aligned(p, 16)) return MOE_ERR_INVALID_ARG;
  if (!attn::aligned(a->positions, 4) || !attn::aligned(a->slots, 4) ||
      !attn::aligned(a->inv_freq, 8) || !attn::aligned(a->device_error, 4))
    return MOE_ERR_INVALID_ARG;
  if (a->n_tokens == 0) return MOE_OK;
  if (!a->q || !a->k || !a->v || !a->q_out || !a->slots) return MOE_ERR_INVALID_ARG;
  if (a->rot_dim > 0 && (!a->positions || !a->inv_freq)) return MOE_ERR_INVALID_ARG;
  rope::Args p;
  p.in[0] = a->q, p.in[1] = a->k, p.in[2] = a->v;
  p.row[0] = a->q_row_stride, p.row[1] = a->k_row_stride, p.row[2] = a->v_row_stride;
  p.head[0] = a->q_head_stride, p.head[1] = a->k_head_stride, p.head[2] = a->v_head_stride;
  p.q_out = a->q_out, p.k = cache->k, p.v = cache->v;
  p.qo_row = a->q_out_row_stride, p.qo_head = a->q_out_head_stride;
  p.page_stride = cache->page_stride, p.head_stride = cache->head_stride;
  p.tok_stride = cache->token_stride;
  p.gamma[0] = a->q_weight, p.gamma[1] = a->k_weight;
  p.inv_freq = a->inv_freq;
  p.positions = a->positions, p.slots = a->slots, p.err = a->device_error;
  p.n_tokens = a->n_tokens, p.hq = a->n_q_heads, p.hkv = cache->n_kv_heads;
  p.rot = a->rot_dim, p.interleaved = a->interleaved;
  p.page_size = cache->page_size, p.n_pages = cache->n_pages;
  p.eps = a->eps;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf16 = cache->dtype == MOE_DTYPE_BF16, f32 = a->in_dtype == MOE_DTYPE_F32;
  const cudaError_t e =
      bf16 ? (f32 ? rope::launch<float, __nv_bfloat16>(p, cache->head_dim, st)
                  : rope::launch<__nv_bfloat16, __nv_bfloat16>(p, cache->head_dim, st))
           : (f32 ? rope::launch<float, __half>(p, cache->head_dim, st)
                  : rope::launch<__half, __half>(p, cache->head_dim, st));
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
