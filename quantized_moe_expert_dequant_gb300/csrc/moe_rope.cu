// moe_rope.cu -- norms of the query and key heads and the position rotation in one pass, with the
// keys and values written to their slots in the pages of a cache (moe_qk_norm_rope).
//
//   y = gamma * x / sqrt(mean(x^2) + eps)                          per query and key head
//   (y_a, y_b) -> (y_a cos t - y_b sin t, y_b cos t + y_a sin t),  t = position * inv_freq[i]
//
// for the pairs (a, b) = (i, i + R/2) or (2i, 2i + 1), i < R/2; elements from R on are not turned,
// values are only rounded.  Everything is fp32 until one rounding at the end.
//
// Bound by the bytes in and out.  A head is D / 16 lanes wide: each lane holds two runs of 8 elements,
// chosen so that both members of its rotated pairs are its own, so a head needs log2(D / 16)
// shuffles (the mean) and no shared memory.  The angles of a token are the same for all of its heads:
// the block forms them once.  An angle is reduced to turns in fp64 (a position near 10^6 has an fp32
// angle with an error of 0.03 rad), its sine and cosine are fp32 (sincospif).  Resident blocks walk
// the tokens; the next token's elements are on their way, and the angles of the next few tokens are
// formed by all warps at once, while this one is worked on.  8192 tokens of 32 query and 8 key/value
// heads of 128 in bf16 (201 MB): 53.1 us with a block a token that loads after its angles, 44.5 us
// resident with a token's angles at a time (two warps form them, the others wait), 37.5 us so
// (5.4 TB/s); two blocks an SM 42.8, deeper copies through shared memory 46.8.
#include <algorithm>

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
  int n_tokens, hq, hkv, rot, interleaved, page_size, n_pages, tokens_per_block, batch;
  float eps;
};

constexpr int kMaxThreads = 384;
constexpr int kBlocksPerSm = 3;  // 56 registers a thread
constexpr int kMaxTokensPerBlock = 16;

template <typename In>
struct Raw {  // 8 elements as they are in memory
  static constexpr int kWords = sizeof(In) / 2;
  uint4 w[kWords];
  __device__ __forceinline__ void load(const In *p) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint4 *>(p)[i];
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    if constexpr (sizeof(In) == 4) {
      x[0] = __uint_as_float(w[0].x), x[1] = __uint_as_float(w[0].y);
      x[2] = __uint_as_float(w[0].z), x[3] = __uint_as_float(w[0].w);
      x[4] = __uint_as_float(w[1].x), x[5] = __uint_as_float(w[1].y);
      x[6] = __uint_as_float(w[1].z), x[7] = __uint_as_float(w[1].w);
    } else {
      const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = attn::Half<In>::unpack(u[i]);
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
      }
    }
  }
};

template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&x)[8]) {
  Raw<T> r;
  r.load(p);
  r.get(x);
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
__global__ void __launch_bounds__(kMaxThreads, kBlocksPerSm) norm_rope_kernel(const Args p) {
  constexpr int L = D / 16;  // lanes of a head
  __shared__ float2 s_cs[2][kMaxTokensPerBlock][D / 2];
  const int heads = p.hq + 2 * p.hkv, half = p.rot / 2, per = p.tokens_per_block;
  // this lane's place in every group of tokens: token, head, and two runs of 8 elements
  const int it = blockIdx.y * blockDim.x + threadIdx.x;
  const int line = it / L, l = it - line * L;
  const int t = line / heads, h = line - t * heads;
  const bool live = t < per;
  const int kind = h < p.hq ? 0 : h < p.hq + p.hkv ? 1 : 2;  // query, key, value
  const int head = h - (kind == 0 ? 0 : kind == 1 ? p.hq : p.hq + p.hkv);
  const int lanes = p.rot / 16;  // of a head that turn something; lane j has angles 8 j .. 8 j + 7
  const bool turned = kind < 2 && l < lanes;
  int ca = 2 * l, cb = 2 * l + 1;
  if (!p.interleaved && l < lanes) ca = l, cb = l + lanes;
  const In *in = static_cast<const In *>(p.in[kind]) + head * p.head[kind];
  const T *gamma = kind < 2 ? static_cast<const T *>(p.gamma[kind]) : nullptr;

  // The angles of `batch` of the block's groups at a time, so that every warp forms some: with a
  // group at a time two warps did, and the others waited for them half of the time.
  const int step = gridDim.x * per, first = blockIdx.x * per;  // tokens from group to group
  const auto angles = [&](int tok0, int buf) {
    for (int i = threadIdx.x; i < p.batch * per * half; i += blockDim.x) {
      const int tt = i / half, f = i - tt * half;
      const int tok = tok0 + tt / per * step + tt % per;
      if (tok >= p.n_tokens) continue;
      double turn = static_cast<double>(p.positions[tok]) * p.inv_freq[f] * 0.15915494309189535;
      turn -= rint(turn);
      float2 cs;
      sincospif(2.f * static_cast<float>(turn), &cs.y, &cs.x);
      s_cs[buf][tt][f % 8 * lanes + f / 8] = cs;
    }
  };
  Raw<In> ra, rb;
  int slot = -1;
  const auto fetch = [&](int tok) {
    slot = -1;
    if (!live || tok >= p.n_tokens) return;
    slot = p.slots[tok];
    const In *src = in + tok * p.row[kind];
    ra.load(src + 8 * ca);
    rb.load(src + 8 * cb);
  };

  fetch(first + t);
  if (half > 0) angles(first, 0);
  int in_batch = 0, buf = 1;
  for (int tok0 = first; tok0 < p.n_tokens; tok0 += step) {
    if (in_batch == 0) {
      __syncthreads();  // this batch's angles are there, and the last one's are no longer read
      const int then = tok0 + p.batch * step;
      if (half > 0 && then < p.n_tokens) angles(then, buf);
      buf ^= 1;
    }
    const int tok = tok0 + t;
    const int at = slot;
    float a[8] = {}, b[8] = {};
    if (at >= 0) ra.get(a), rb.get(b);
    fetch(tok + step);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(a[i], a[i], fmaf(b[i], b[i], sum));
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (gamma) {
      const float r = rsqrtf(fmaf(sum, 1.f / D, p.eps));
      float w[8];
      load8(gamma + 8 * ca, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] *= r * w[i];
      load8(gamma + 8 * cb, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] *= r * w[i];
    }
    if (turned && at >= 0) {
      const float2 *cs = &s_cs[buf][in_batch * per + t][l];
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = cs[i * lanes], w = cs[(4 + i) * lanes];
          const float x = a[2 * i], y = a[2 * i + 1], z = b[2 * i], q = b[2 * i + 1];
          a[2 * i] = x * v.x - y * v.y, a[2 * i + 1] = y * v.x + x * v.y;
          b[2 * i] = z * w.x - q * w.y, b[2 * i + 1] = q * w.x + z * w.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 v = cs[i * lanes];
          const float x = a[i], y = b[i];
          a[i] = x * v.x - y * v.y, b[i] = y * v.x + x * v.y;
        }
      }
    }
    if (at >= 0) {
      T *dst;
      bool ok = true;
      if (kind == 0) {
        dst = static_cast<T *>(p.q_out) + tok * p.qo_row + head * p.qo_head;
      } else {
        const int page = at / p.page_size;
        ok = page < p.n_pages;
        if (!ok && p.err) atomicOr(p.err, attn::kDevErrBadId);
        dst = static_cast<T *>(kind == 1 ? p.k : p.v) + page * p.page_stride +
              head * p.head_stride + (at - page * p.page_size) * p.tok_stride;
      }
      if (ok) {
        store8(dst + 8 * ca, a);
        store8(dst + 8 * cb, b);
      }
    }
    if (++in_batch == p.batch) in_batch = 0;
  }
}

template <typename In, typename T, int D>
static cudaError_t launch(Args p, cudaStream_t stream) {
  const int per_token = (p.hq + 2 * p.hkv) * (D / 16);
  p.tokens_per_block = per_token >= 256 ? 1 : 256 / per_token;
  if (p.tokens_per_block > kMaxTokensPerBlock) p.tokens_per_block = kMaxTokensPerBlock;
  const int items = p.tokens_per_block * per_token;
  int threads = (items + 31) / 32 * 32;
  if (threads > kMaxThreads) threads = kMaxThreads;
  p.batch = kMaxTokensPerBlock / p.tokens_per_block;
  if (p.rot > 0) p.batch = std::min(p.batch, std::max(1, threads / (p.tokens_per_block * p.rot / 2)));
  const int parts = (items + threads - 1) / threads;  // blocks that share a group of tokens
  const auto kern = norm_rope_kernel<In, T, D>;
  const int groups = (p.n_tokens + p.tokens_per_block - 1) / p.tokens_per_block;
  int grid = groups;
  if (groups > 152) {  // else every block has one group whatever is resident
    int dev = 0, sms = 0, per_sm = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, 0);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) per_sm = 1;
    const int most = sms * per_sm / parts;
    if (grid > most) grid = most < 1 ? 1 : most;
  }
  kern<<<dim3(grid, parts), threads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename In, typename T>
static cudaError_t launch(const Args &p, int dim, cudaStream_t stream) {
  return dim == 64 ? launch<In, T, 64>(p, stream) : launch<In, T, 128>(p, stream);
}

}  // namespace rope

extern "C" int moe_qk_norm_rope(const moe_kv_cache *cache, const moe_norm_rope *a, void *stream) {
  const int rc = attn::check_cache(cache);
  if (rc != MOE_OK) return rc;
  if (!a || a->n_tokens < 0 || a->n_q_heads < 1 || a->rot_dim < 0 ||
      a->rot_dim > cache->head_dim || !(a->eps >= 0.f) || !(a->eps <= 1.f))
    return MOE_ERR_INVALID_ARG;
  if (a->rot_dim % 16 || a->n_tokens > 1 << 29) return MOE_ERR_UNSUPPORTED;
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
