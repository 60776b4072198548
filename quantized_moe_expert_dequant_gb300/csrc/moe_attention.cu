// moe_attention.cu -- attention over the pages of a cache (moe_tree_attention, moe_prompt_attention).
//
//   out_r = sum_j p_rj v_j / sum_j p_rj,   p_rj = exp(scale * q_r . k_j - m_r)  over the positions j
//   that row r sees, m_r their largest score: one pass over K and V with the running maximum and
//   sum; what was summed before a larger maximum is scaled down to it.
//
// The rows of an item are the queries of one sequence for all query heads that share a key/value
// head: row R is query R / group, head R % group.  A CTA of four warps takes ROWS = 16 WR rows of
// them and walks 64 positions at a time; WR warps split the rows, 4 / WR warps the positions, so a
// single decoded token still uses all four.
#include "moe_attention.cuh"

namespace attn {

constexpr int kTile = 64;  // positions of a step
constexpr int kThreads = 128;
constexpr int kStages = 2;

template <int D>
__device__ __forceinline__ uint32_t swizzled(int row, int chunk) {  // byte offset in a [64][D] tile
  return static_cast<uint32_t>(row * D * 2 + ((chunk ^ (row & 7)) << 4));
}

// Copies positions [64 t, 64 t + 64) of K and V into shared memory; rows past the sequence and on
// a page outside the cache are zeros (what stale pages hold, NaN included, is never multiplied).
template <typename T, int D>
__device__ __forceinline__ void load_tile(const Params &p, const Seq &s, const int32_t *pages,
                                          int64_t head_off, int tile, uint32_t k_smem,
                                          uint32_t v_smem) {
  constexpr int kChunks = D / 8, kStep = kThreads / kChunks;
  const int c = threadIdx.x % kChunks, r0 = threadIdx.x / kChunks;
#pragma unroll
  for (int i = 0; i < kTile / kStep; ++i) {
    const int r = r0 + i * kStep, pos = tile * kTile + r;
    bool valid = pos < s.len;
    int64_t off = 0;
    if (valid) {
      const int page = pages[pos >> p.page_shift];
      valid = static_cast<unsigned>(page) < static_cast<unsigned>(p.n_pages);
      if (!valid && p.err) atomicOr(p.err, kDevErrBadId);
      off = valid ? page * p.page_stride + head_off +
                        (pos & ((1 << p.page_shift) - 1)) * p.tok_stride + 8 * c
                  : 0;
    }
    const uint32_t d = swizzled<D>(r, c);
    cp_async16(k_smem + d, static_cast<const T *>(p.k) + off, valid);
    cp_async16(v_smem + d, static_cast<const T *>(p.v) + off, valid);
  }
}

template <typename T, int D, int WR>
__global__ void __launch_bounds__(kThreads) paged_attention_kernel(const Params p) {
  constexpr int ROWS = 16 * WR, WT = 4 / WR, TW = kTile / WT;  // TW positions of a warp per tile
  constexpr int kTileBytes = kTile * D * 2;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[4][16], s_l[4][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q4 = lane & 3;
  const int wr = warp % WR, wt = warp / WR;
  const int kvh = blockIdx.y;
  const Seq s = load_seq(p, blockIdx.z, blockIdx.x == 0 && kvh == 0 && threadIdx.x == 0);
  const int rows = s.nq * p.group, R0 = blockIdx.x * ROWS;
  if (R0 >= rows) return;
  const int32_t *pages = p.table + blockIdx.z * p.table_stride;
  const int64_t head_off = kvh * p.head_stride;
  // positions that any row of this tile sees
  const int last_q = min(rows - 1, R0 + ROWS - 1) / p.group;
  const int seen = p.mask ? s.len : s.ctx + last_q + 1;
  const int tiles = (seen + kTile - 1) / kTile;

  // this lane's two rows: queries, heads, masks
  int row_q[2];
  uint64_t row_mask[2];
  bool row_ok[2];
  const uint32_t *qp[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int R = R0 + wr * 16 + g + 8 * h;
    row_ok[h] = R < rows;
    row_q[h] = row_ok[h] ? R / p.group : 0;
    const int head = kvh * p.group + (row_ok[h] ? R - row_q[h] * p.group : 0);
    qp[h] = reinterpret_cast<const uint32_t *>(static_cast<const T *>(p.q) +
                                               (s.row0 + row_q[h]) * p.q_row + head * p.q_head);
    if (p.mask)
      row_mask[h] = p.mask[s.row0 + row_q[h]];
    else
      row_mask[h] = 0;
  }
  uint32_t qa[D / 16][4];
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    qa[kk][0] = row_ok[0] ? qp[0][8 * kk + q4] : 0u;
    qa[kk][1] = row_ok[1] ? qp[1][8 * kk + q4] : 0u;
    qa[kk][2] = row_ok[0] ? qp[0][8 * kk + 4 + q4] : 0u;
    qa[kk][3] = row_ok[1] ? qp[1][8 * kk + 4 + q4] : 0u;
  }

  float o[D / 8][4], m[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

  const uint32_t base = smem_u32(smem);
  if (tiles > 0) load_tile<T, D>(p, s, pages, head_off, 0, base, base + kTileBytes);
  cp_async_commit();
  for (int t = 0; t < tiles; ++t) {
    const uint32_t ks = base + (t % kStages) * 2 * kTileBytes, vs = ks + kTileBytes;
    if (t + 1 < tiles) {
      const uint32_t n = base + ((t + 1) % kStages) * 2 * kTileBytes;
      load_tile<T, D>(p, s, pages, head_off, t + 1, n, n + kTileBytes);
    }
    cp_async_commit();
    cp_async_wait<1>();
    __syncthreads();

    float sc[TW / 8][4];
#pragma unroll
    for (int j = 0; j < TW / 8; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
      for (int j = 0; j < TW / 16; ++j) {
        uint32_t b[4];
        const int mi = lane >> 3;
        ldmatrix_x4(b, ks + swizzled<D>(wt * TW + 16 * j + (lane & 7) + 8 * (mi >> 1),
                                        2 * kk + (mi & 1)));
        Half<T>::mma(sc[2 * j], qa[kk], b[0], b[1]);
        Half<T>::mma(sc[2 * j + 1], qa[kk], b[2], b[3]);
      }
    // positions that not every row of the tile sees
    const int pos0 = t * kTile + wt * TW + 2 * q4;
    if ((t + 1) * kTile > s.ctx) {
#pragma unroll
      for (int j = 0; j < TW / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int pos = pos0 + 8 * j + (e & 1), d = pos - s.ctx, h = e >> 1;
          const bool vis = d < 0 || (p.mask ? d < s.nq && ((row_mask[h] >> (d & 63)) & 1)
                                            : d <= row_q[h]);
          if (!vis) sc[j][e] = kNegInf;
        }
    }
    float scale[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float top = m[h];
#pragma unroll
      for (int j = 0; j < TW / 8; ++j) top = fmaxf(top, fmaxf(sc[j][2 * h], sc[j][2 * h + 1]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float ref = top == kNegInf ? 0.f : top;  // no position seen so far
      scale[h] = exp2_approx((m[h] - ref) * p.scale_log2);
      m[h] = top;
      const float off = ref * p.scale_log2;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < TW / 8; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float x = exp2_approx(fmaf(sc[j][2 * h + e], p.scale_log2, -off));
          sc[j][2 * h + e] = x;
          sum += x;
        }
      l[h] = l[h] * scale[h] + sum;
    }
#pragma unroll
    for (int j = 0; j < D / 8; ++j) {
      o[j][0] *= scale[0], o[j][1] *= scale[0];
      o[j][2] *= scale[1], o[j][3] *= scale[1];
    }
#pragma unroll
    for (int j = 0; j < TW / 16; ++j) {
      // p enters the product in the cache's type (as v is): half a step of it relative to the row's
      // largest p, the size of the output's own rounding
      const uint32_t a[4] = {Half<T>::pack(sc[2 * j][0], sc[2 * j][1]),
                             Half<T>::pack(sc[2 * j][2], sc[2 * j][3]),
                             Half<T>::pack(sc[2 * j + 1][0], sc[2 * j + 1][1]),
                             Half<T>::pack(sc[2 * j + 1][2], sc[2 * j + 1][3])};
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        uint32_t b[4];
        const int mi = lane >> 3;
        ldmatrix_x4_trans(b, vs + swizzled<D>(wt * TW + 16 * j + (lane & 7) + 8 * (mi & 1),
                                              2 * d + (mi >> 1)));
        Half<T>::mma(o[2 * d], a, b[0], b[1]);
        Half<T>::mma(o[2 * d + 1], a, b[2], b[3]);
      }
    }
    __syncthreads();
  }

  // join the warps that split the positions, and the rows' sums over their four lanes
  float *s_o = reinterpret_cast<float *>(smem);  // [4][16][D]
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    const int r = g + 8 * h;
    if (q4 == 0) s_m[warp][r] = m[h], s_l[warp][r] = l[h];
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
      *reinterpret_cast<float2 *>(s_o + (warp * 16 + r) * D + 8 * j + 2 * q4) =
          make_float2(o[j][2 * h], o[j][2 * h + 1]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < ROWS * D / 8; i += kThreads) {
    const int r = i / (D / 8), c = i % (D / 8), R = R0 + r;
    if (R >= rows) break;
    float top = kNegInf;
#pragma unroll
    for (int w = 0; w < WT; ++w) top = fmaxf(top, s_m[w * WR + r / 16][r % 16]);
    const float ref = top == kNegInf ? 0.f : top;
    float sum = 0.f, x[8] = {};
#pragma unroll
    for (int w = 0; w < WT; ++w) {
      const int ww = w * WR + r / 16;
      const float f = exp2_approx((s_m[ww][r % 16] - ref) * p.scale_log2);
      sum += f * s_l[ww][r % 16];
      const float *src = s_o + (ww * 16 + r % 16) * D + 8 * c;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fmaf(f, src[e], x[e]);
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;  // a row that sees nothing is zeros
    const int tok = R / p.group, head = kvh * p.group + R - tok * p.group;
    uint4 w;
    w.x = Half<T>::pack(x[0] * inv, x[1] * inv);
    w.y = Half<T>::pack(x[2] * inv, x[3] * inv);
    w.z = Half<T>::pack(x[4] * inv, x[5] * inv);
    w.w = Half<T>::pack(x[6] * inv, x[7] * inv);
    *reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + (s.row0 + tok) * p.o_row +
                               head * p.o_head + 8 * c) = w;
  }
}

template <typename T, int D, int WR>
static cudaError_t launch(const Params &p, int max_q, cudaStream_t stream) {
  const auto kern = paged_attention_kernel<T, D, WR>;
  constexpr int bytes = kStages * 2 * kTile * D * 2;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(max_q) * p.group;
  const dim3 grid(static_cast<unsigned>((rows + 16 * WR - 1) / (16 * WR)), p.hkv, p.n_seqs);
  kern<<<grid, kThreads, bytes, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, int D>
static cudaError_t launch_rows(const Params &p, int max_q, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(max_q) * p.group;
  if (rows <= 16) return launch<T, D, 1>(p, max_q, stream);
  if (rows <= 32) return launch<T, D, 2>(p, max_q, stream);
  return launch<T, D, 4>(p, max_q, stream);
}

static cudaError_t launch_any(const moe_kv_cache *c, const Params &p, int max_q,
                              cudaStream_t stream) {
  if (c->dtype == MOE_DTYPE_BF16)
    return c->head_dim == 64 ? launch_rows<__nv_bfloat16, 64>(p, max_q, stream)
                             : launch_rows<__nv_bfloat16, 128>(p, max_q, stream);
  return c->head_dim == 64 ? launch_rows<__half, 64>(p, max_q, stream)
                           : launch_rows<__half, 128>(p, max_q, stream);
}

}  // namespace attn

extern "C" int moe_prompt_attention(const moe_kv_cache *cache, const moe_attention *a,
                                    void *stream) {
  attn::Params p;
  const int rc = attn::check_attention(cache, a, &p);
  if (rc != MOE_OK) return rc;
  if (p.n_seqs > 65535 || p.hkv > 65535) return MOE_ERR_UNSUPPORTED;
  if (p.n_seqs == 0 || p.n_rows == 0) return MOE_OK;
  return attn::launch_any(cache, p, p.n_rows, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}
