// moe_pages.cu -- which pages of a cache a token reads: the bounds of a page's keys (moe_page_bounds) and the
// selection by them (moe_select_pages).
//
//   lo_jd = min, hi_jd = max of k_d over the positions on page j
//   score_j = sum over the query heads of a key/value head of sum_d max(q_d lo_jd, q_d hi_jd)
//           = sum_d Q+_d hi_jd + Q-_d lo_jd,   Q+ (Q-): sum over the heads of the positive (negative) q
// No key of the page has a larger q . k summed over the heads.
//
// Both read their input once and do little with it: bytes and, with few rows, latency bound them.
#include "moe_attention.cuh"

namespace attn {

constexpr int kBlock = 256;
constexpr int kWarps = kBlock / 32;

__device__ __forceinline__ uint4 load16(const void *p) { return *static_cast<const uint4 *>(p); }

template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
  using V = __nv_bfloat162;
  static constexpr uint32_t kMost = 0x7f807f80u, kLeast = 0xff80ff80u;  // +inf, -inf
};
template <>
struct Pair<__half> {
  using V = __half2;
  static constexpr uint32_t kMost = 0x7c007c00u, kLeast = 0xfc00fc00u;
};
// The lesser and the larger of two pairs; a NaN stays (bounds of a page's keys).
template <typename T>
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
  using V = typename Pair<T>::V;
  const V r = __hmin2_nan(*reinterpret_cast<const V *>(&a), *reinterpret_cast<const V *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}
template <typename T>
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  using V = typename Pair<T>::V;
  const V r = __hmax2_nan(*reinterpret_cast<const V *>(&a), *reinterpret_cast<const V *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}
// The larger of two pairs without NaN (sizes: what bounds the error of the scores that are numbers).
template <typename T>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  using V = typename Pair<T>::V;
  const V r = __hmax2(*reinterpret_cast<const V *>(&a), *reinterpret_cast<const V *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}

// ------------------------------------------------------------------ bounds of a page's keys
// Pages of a sequence that hold its new positions.
__device__ __forceinline__ int touched(const Params &p, const Seq &s) {
  return s.nq ? ((s.len - 1) >> p.page_shift) - (s.ctx >> p.page_shift) + 1 : 0;
}

// One block a touched page (blockIdx.x, counted over all sequences) and key/value head: D / 8 threads side
// by side read a position, so that a page of 64 is four loads a thread, all under way at once.  A launch and three
// dependent loads: 32 tokens, 8 heads of 128 (2.3 MB) 3.5 us, prompts of 9230 tokens, 2 heads of 64 (2.7 MB) 4.9 us.
template <typename T, int D>
__global__ void __launch_bounds__(kBlock) bounds_kernel(const Params p, T *bounds) {
  constexpr int kChunks = D / 8, kRows = kBlock / kChunks;
  __shared__ int s_sum[kWarps], s_seq, s_page;
  __shared__ uint4 s_lo[kWarps][kChunks], s_hi[kWarps][kChunks];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_launch();
  // the sequence that the page belongs to
  if (threadIdx.x == 0) s_seq = -1;
  int64_t below = 0;
  for (int b = 0; b < p.n_seqs; b += kBlock) {
    const int i = b + threadIdx.x;
    int mine = 0, first = 0;
    if (i < p.n_seqs) {
      const Seq s = load_seq(p, i, blockIdx.x == 0 && blockIdx.y == 0);
      mine = touched(p, s), first = s.ctx >> p.page_shift;
    }
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = x;
    __syncthreads();
    int64_t before = below + x - mine;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s_sum[w];
      below += s_sum[w];
    }
    if (before <= blockIdx.x && blockIdx.x < before + mine)
      s_seq = i, s_page = first + static_cast<int>(blockIdx.x - before);
    if (below > blockIdx.x && blockIdx.x > 0) break;  // (block 0 checks all sequences)
  }
  __syncthreads();
  if (s_seq < 0) return;
  const int at = s_page;
  const Seq s = load_seq(p, s_seq, false);
  const int page = p.table[s_seq * p.table_stride + at];
  if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.n_pages)) {
    if (threadIdx.x == 0 && p.err) atomicOr(p.err, kDevErrBadId);
    return;
  }
  const int held = min(1 << p.page_shift, s.len - (at << p.page_shift));
  const int c = threadIdx.x % kChunks, r0 = threadIdx.x / kChunks;
  const T *k = static_cast<const T *>(p.k) + page * p.page_stride + blockIdx.y * p.head_stride + 8 * c;
  uint32_t lo[4], hi[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) lo[e] = Pair<T>::kMost, hi[e] = Pair<T>::kLeast;
#pragma unroll 4
  for (int r = r0; r < held; r += kRows) {
    const uint4 x = load16(k + r * p.tok_stride);
    const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) lo[e] = min2_nan<T>(lo[e], y[e]), hi[e] = max2_nan<T>(hi[e], y[e]);
  }
#pragma unroll
  for (int o = kChunks; o < 32; o <<= 1)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      lo[e] = min2_nan<T>(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], o));
      hi[e] = max2_nan<T>(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], o));
    }
  if (lane < kChunks) {
    s_lo[warp][lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    s_hi[warp][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  }
  __syncthreads();
  if (threadIdx.x >= 2 * kChunks) return;
  const bool top = threadIdx.x >= kChunks;
  uint4 v = top ? s_hi[0][c] : s_lo[0][c];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) {
    const uint4 x = top ? s_hi[w][c] : s_lo[w][c];
    v.x = top ? max2_nan<T>(v.x, x.x) : min2_nan<T>(v.x, x.x);
    v.y = top ? max2_nan<T>(v.y, x.y) : min2_nan<T>(v.y, x.y);
    v.z = top ? max2_nan<T>(v.z, x.z) : min2_nan<T>(v.z, x.z);
    v.w = top ? max2_nan<T>(v.w, x.w) : min2_nan<T>(v.w, x.w);
  }
  T *dst = bounds + ((static_cast<int64_t>(page) * p.hkv + blockIdx.y) * 2 + top) * D + 8 * c;
  *reinterpret_cast<uint4 *>(dst) = v;
}

// ------------------------------------------------------------------ selection
// The order of two pages may hang on the last bit of their scores, so it is decided in two steps: fp32 scores
// with a bound on their error tell which pages are certainly among the k best and which are certainly
// not; what lies between is compared by scores in fp64.  A score is the fp32 sum of terms Q b, Q a sum over the heads of
// numbers of one sign.  It is off by less than `error` times the sum of the terms' sizes, and that is at most
// max_d |b_d| times sum_d |Q_d|.
//
// When sums in fp64 are exact: of g heads and D dimensions a score has g D products q b (each meets one of its two
// bounds).  Of a product in [2^s, 2^(s+2)) the last bit is at least 2^(s-20) (two numbers of 11 bits; bf16, 8 bits: 2^(s-14)),
// the sum of all is below g D 2^(S+2), S that of the largest, and fp64 holds 53 bits: so while S - s <= 31 - log2(g D)
// (bf16: 37), that is, while the largest product is not 2^(29 - log2(g D)) (2^(35 - ...)) times the least one that is
// not 0, every partial sum of Q and of the terms is exact, in any order.  4 heads of 128: 2^20 and 2^26; 64: 2^16 and 2^22.
// Beyond that they are sums of g + 2 D / 32 + 5 roundings in an order that is the same for all pages: pages with the
// same bounds still tie, others that are equal but for these roundings may not.
constexpr int kMaxPages = 65536;     // of a sequence: a bit each in shared memory
constexpr int kKeys = 8192;          // scores that are kept in shared memory
constexpr int kBins = 1024;
constexpr int kFew = 64;             // pages compared in fp64 one against the other

struct Select {
  Params p;
  const void *bounds;  // [n_pages][hkv][2][D]
  // [rows of this launch][hkv][2 width]: scores of the pages, then for each 16 the largest bound of the sum of a
  // score's terms' sizes
  float *score;
  int32_t *out;        // [n_rows][hkv][n_select]
  int row0, rows, width, n_select, sink, recent;
  float error;         // of a score, relative to the sizes' sum
};

__device__ __forceinline__ bool better(double a, int i, double b, int j) {
  return a > b || (a == b && i < j);
}

// Q- and Q+ of a row and key/value head, side by side as the bounds are.  Returns this thread's sum of sizes.
template <typename T, int D, typename V>
__device__ __forceinline__ V sum_heads(const Params &p, int row, int kvh, V *s_q) {
  const T *q = static_cast<const T *>(p.q) + row * p.q_row +
               static_cast<int64_t>(kvh) * p.group * p.q_head;
  V size = 0;
  for (int d = threadIdx.x; d < D; d += blockDim.x) {
    V down = 0, up = 0;
#pragma unroll 8
    for (int h = 0; h < p.group; ++h) {
      const V x = static_cast<float>(q[h * p.q_head + d]);
      if (x < 0) down += x; else up += x;  // (a NaN goes up)
    }
    s_q[d] = down, s_q[D + d] = up;
    size += up - down;
  }
  return size;
}

// The bounds of some pages in registers: eight lanes take a page, so that what they read is 128 bytes in a row
// and three exchanges add their parts; a block holds 32 PAGES pages, first + 32 t + (thread / 8).
template <typename T, int D, int PAGES>
struct Block {
  static constexpr int kParts = 2 * D / 64;  // 16-byte parts of a page's bounds that a lane takes
  uint4 x[PAGES][kParts];
  float top[PAGES];  // the largest size of a bound; -1: no page
  int at[PAGES];     // of the pages that are fetched next

  // Looks up pages first .. count - 1 of a sequence.
  __device__ __forceinline__ void look(const Select &w, int seq, int first, int count) {
#pragma unroll
    for (int t = 0; t < PAGES; ++t) {
      const int j = first + (threadIdx.x >> 3) + t * (kBlock / 8);
      at[t] = j < count ? w.p.table[seq * w.p.table_stride + j] : -1;
    }
  }
  // The bounds of those pages; pages outside the cache are reported.
  __device__ __forceinline__ void fetch(const Select &w, int kvh, int first, int count) {
    const Params &p = w.p;
    const int part = threadIdx.x & 7;
#pragma unroll
    for (int t = 0; t < PAGES; ++t) {
      const int j = first + (threadIdx.x >> 3) + t * (kBlock / 8);
      top[t] = static_cast<unsigned>(at[t]) < static_cast<unsigned>(p.n_pages) ? 0.f : -1.f;
      if (top[t] < 0.f && j < count && j >= w.sink && part == 0 && p.err)
        atomicOr(p.err, kDevErrBadId);
    }
#pragma unroll
    for (int t = 0; t < PAGES; ++t) {
      const T *src = static_cast<const T *>(w.bounds) +
                     (static_cast<int64_t>(top[t] < 0.f ? 0 : at[t]) * p.hkv + kvh) * 2 * D + 8 * part;
#pragma unroll
      for (int e = 0; e < kParts; ++e) x[t][e] = load16(src + 64 * e);
    }
  }
  __device__ __forceinline__ void sizes() {
#pragma unroll
    for (int t = 0; t < PAGES; ++t) {
      uint32_t m = 0u;
#pragma unroll
      for (int e = 0; e < kParts; ++e)
        m = max2<T>(max2<T>(m, x[t][e].x & 0x7fff7fffu),
                    max2<T>(max2<T>(x[t][e].y & 0x7fff7fffu, x[t][e].z & 0x7fff7fffu),
                            x[t][e].w & 0x7fff7fffu));
      const float2 f = Half<T>::unpack(m);
      float v = fmaxf(f.x, f.y);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
      if (top[t] >= 0.f) top[t] = v;
    }
  }
  // Scores for the sums q; -infinity without a page.
  __device__ __forceinline__ void score(const float *s_q, float (&s)[PAGES]) const {
    const int part = threadIdx.x & 7;
    const auto both = [](uint32_t v) {
      const float2 f = Half<T>::unpack(v);
      return pair(f.x, f.y);
    };
#pragma unroll
    for (int t = 0; t < PAGES; ++t) {
      uint64_t sum[kParts];
#pragma unroll
      for (int e = 0; e < kParts; ++e) {
        const float4 *q = reinterpret_cast<const float4 *>(s_q + 64 * e + 8 * part);
        const float4 a = q[0], b = q[1];
        sum[e] = mul2(pair(a.x, a.y), both(x[t][e].x));
        sum[e] = fma2(pair(a.z, a.w), both(x[t][e].y), sum[e]);
        sum[e] = fma2(pair(b.x, b.y), both(x[t][e].z), sum[e]);
        sum[e] = fma2(pair(b.z, b.w), both(x[t][e].w), sum[e]);
      }
#pragma unroll
      for (int o = kParts / 2; o > 0; o >>= 1)
#pragma unroll
        for (int e = 0; e < o; ++e) sum[e] = add2(sum[e], sum[e + o]);
      const float2 f = unpair(sum[0]);
      s[t] = f.x + f.y;
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1)
#pragma unroll
      for (int t = 0; t < PAGES; ++t) s[t] += __shfl_xor_sync(0xffffffffu, s[t], o);
#pragma unroll
    for (int t = 0; t < PAGES; ++t)
      if (top[t] < 0.f) s[t] = kNegInf;
  }
};

// The sum of sizes of a block's sum_heads, added to *s_size (0 before; its order does not matter: a bound).
template <int D>
__device__ __forceinline__ void add_size(float size, float *s_size) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) size += __shfl_xor_sync(0xffffffffu, size, o);
  if ((threadIdx.x & 31) == 0 && threadIdx.x < D) atomicAdd(s_size, size);
}

// Pages between which a row's selection chooses: all but the last `recent`; 0 when it takes every page.
__device__ __forceinline__ int scored(const Select &w, const Row &row) {
  const int pages = row.nq ? ((row.ctx - 1) >> w.p.page_shift) + 1 : 0;
  return pages > w.n_select ? pages - w.recent : 0;
}

// For chunks, whose rows share what is read: scores of 16 rows and kTurns * 128 pages a block into w.score, on
// mma.sync.  The sums Q of a row, scaled by a power of two so that the type holds the largest, are split in two
// numbers of 16 bits (error 2^-18 of each Q; bounds are exact), rows are the rows of the products, pages the
// columns; each truncation of an fp32 sum counts 2^-23.  A lane's 16 bytes of a bound are its places of two
// products: the order of the dimensions is the same for both factors.  (In fp32 on the other units, four rows a
// block: 512 rows, 2000 pages, 2 heads of 64: 85 us; 24 so.)
constexpr int kRowTile = 16, kTurns = 2, kPagesATurn = 128;

template <typename T, int D>
__global__ void __launch_bounds__(kBlock) score_kernel(const Select w) {
  constexpr int kStride = 2 * D + 32;  // elements: 64 bytes of padding keep the rows' banks apart
  constexpr int kSteps = 2 * D / 32;   // of 32 dimensions, two products
  __shared__ __align__(16) T s_q[2][kRowTile][kStride];  // larger and smaller part
  __shared__ float s_size[kRowTile], s_scale[kRowTile];
  __shared__ int s_seq[kRowTile], s_count[kRowTile];
  const Params &p = w.p;
  pdl_wait();
  pdl_launch();
  const int first = w.row0 + blockIdx.x * kRowTile, kvh = blockIdx.y;
  const int begin = blockIdx.z * kTurns * kPagesATurn;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x < kRowTile) {
    const int r = threadIdx.x;
    Row row = {};
    if (blockIdx.x * kRowTile + r < w.rows) row = load_row(p, first + r, 1);
    s_seq[r] = row.seq, s_count[r] = scored(w, row);
  }
  __syncthreads();
  int most = 0;
#pragma unroll
  for (int r = 0; r < kRowTile; ++r) most = max(most, s_count[r]);
  if (begin >= most || begin + kTurns * kPagesATurn <= w.sink) return;
  const int g = lane >> 2, q4 = lane & 3;
  uint4 b[2][kSteps];
  bool there[2];
  const auto fetch = [&](int seq, int count, int at) {  // the bounds of two times eight pages
    int page[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int j = at + 8 * t + g;
      page[t] = j < count ? p.table[seq * p.table_stride + j] : -1;
      there[t] = static_cast<unsigned>(page[t]) < static_cast<unsigned>(p.n_pages);
      if (!there[t] && j < count && j >= w.sink && q4 == 0 && p.err) atomicOr(p.err, kDevErrBadId);
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const T *src = static_cast<const T *>(w.bounds) +
                     (static_cast<int64_t>(there[t] ? page[t] : 0) * p.hkv + kvh) * 2 * D + 8 * q4;
#pragma unroll
      for (int k = 0; k < kSteps; ++k) b[t][k] = load16(src + 32 * k);
    }
  };
  const auto end_of = [&](int r0, int *count) {  // of the rows from r0 on that are of one sequence
    int r1 = r0;
    for (*count = 0; r1 < kRowTile && s_seq[r1] == s_seq[r0]; ++r1) *count = max(*count, s_count[r1]);
    return r1;
  };
  int count, r1 = end_of(0, &count);
  fetch(s_seq[0], count, begin + 16 * warp);  // on its way during the sums
  // a warp takes two rows' sums, a lane some neighbouring dimensions
  constexpr int V = D / 32;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = 2 * warp + e;
    float down[V] = {}, up[V] = {}, size = 0.f, top = 0.f;
    if (s_count[r] > 0) {
      const T *q = static_cast<const T *>(p.q) + (first + r) * p.q_row +
                   static_cast<int64_t>(kvh) * p.group * p.q_head + V * lane;
#pragma unroll 4
      for (int h = 0; h < p.group; ++h)
#pragma unroll
        for (int v = 0; v < V; v += 2) {
          const float2 x = Half<T>::unpack(*reinterpret_cast<const uint32_t *>(q + h * p.q_head + v));
          if (x.x < 0.f) down[v] += x.x; else up[v] += x.x;  // (a NaN goes up)
          if (x.y < 0.f) down[v + 1] += x.y; else up[v + 1] += x.y;
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) size += up[v] - down[v], top = fmaxf(top, fmaxf(up[v], -down[v]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      size += __shfl_xor_sync(0xffffffffu, size, o);
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    // fp16: the largest (2^-24 .. 2^22) is brought to 2^14 .. 2^15
    float scale = 1.f, back = 1.f;
    if (Half<T>::kRow > 0.f && top > 0.f && top < 1e30f) {
      const int shift = 127 + 14 - static_cast<int>(__float_as_uint(top) >> 23);
      scale = __uint_as_float((127 + shift) << 23), back = __uint_as_float((127 - shift) << 23);
    }
    if (lane == 0) s_size[r] = size, s_scale[r] = back;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int v = 0; v < V; v += 2) {
        const float x = (s ? up[v] : down[v]) * scale, y = (s ? up[v + 1] : down[v + 1]) * scale;
        const uint32_t large = Half<T>::pack(x, y);
        const float2 f = Half<T>::unpack(large);
        const uint32_t small = Half<T>::pack(x - f.x, y - f.y);
        *reinterpret_cast<uint32_t *>(&s_q[0][r][s * D + V * lane + v]) = large;
        *reinterpret_cast<uint32_t *>(&s_q[1][r][s * D + V * lane + v]) = small;
      }
  }
  __syncthreads();
  for (int r0 = 0; r0 < kRowTile; r0 = r1) {
    const int seq = s_seq[r0];
    r1 = end_of(r0, &count);
    for (int turn = 0; turn < kTurns; ++turn) {
      const int at = begin + turn * kPagesATurn + 16 * warp;
      if (at >= count) break;
      if (r0 + turn > 0) fetch(seq, count, at);
      // of the larger parts 32 products are summed by themselves, so that the error does not grow with the dimensions
      float sum[2][4] = {}, small[2][4] = {};
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        float large[2][4] = {};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const uint4 lo = *reinterpret_cast<const uint4 *>(&s_q[s][g][32 * k + 8 * q4]);
          const uint4 hi = *reinterpret_cast<const uint4 *>(&s_q[s][g + 8][32 * k + 8 * q4]);
          const uint32_t a0[4] = {lo.x, hi.x, lo.y, hi.y}, a1[4] = {lo.z, hi.z, lo.w, hi.w};
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            Half<T>::mma(s ? small[t] : large[t], a0, b[t][k].x, b[t][k].y);
            Half<T>::mma(s ? small[t] : large[t], a1, b[t][k].z, b[t][k].w);
          }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int c = 0; c < 4; ++c) sum[t][c] += large[t][c];
      }
      float most[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        uint32_t m = 0u;
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
          m = max2<T>(max2<T>(m, b[t][k].x & 0x7fff7fffu),
                      max2<T>(max2<T>(b[t][k].y & 0x7fff7fffu, b[t][k].z & 0x7fff7fffu),
                              b[t][k].w & 0x7fff7fffu));
        const float2 f = Half<T>::unpack(m);
        float top = fmaxf(f.x, f.y);  // the largest size of a bound of page g
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const bool none = !there[t];
        most[t] = none ? 0.f : top;
        const bool none0 = __shfl_sync(0xffffffffu, none, 8 * q4), none1 = __shfl_sync(0xffffffffu, none, 8 * q4 + 4);
        const int j = at + 8 * t + 2 * q4;
#pragma unroll
        for (int c = 0; c < 4; c += 2) {  // row g or g + 8, pages j and j + 1
          const int r = g + 4 * c;
          if (r < r0 || r >= r1 || j >= s_count[r]) continue;
          float *dst = w.score + (static_cast<int64_t>(blockIdx.x * kRowTile + r) * p.hkv + kvh) * 2 * w.width + j;
          const float s0 = none0 ? kNegInf : (sum[t][c] + small[t][c]) * s_scale[r];
          const float s1 = none1 ? kNegInf : (sum[t][c + 1] + small[t][c + 1]) * s_scale[r];
          if (j + 1 < s_count[r])
            *reinterpret_cast<float2 *>(dst) = make_float2(s0, s1);
          else
            *dst = s0;
        }
      }
      float size = fmaxf(most[0], most[1]);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) size = fmaxf(size, __shfl_xor_sync(0xffffffffu, size, o));
      if (lane >= r0 && lane < r1 && at < s_count[lane])
        w.score[((static_cast<int64_t>(blockIdx.x * kRowTile + lane) * p.hkv + kvh) * 2 + 1) * w.width +
                at / 16] = size * s_size[lane];
    }
  }
}

// Larger scores have larger keys; NaN has -infinity's.
__device__ __forceinline__ uint32_t key_of(float s) {
  if (!(s == s)) s = kNegInf;
  const uint32_t b = __float_as_uint(s);
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float score_of(uint32_t key) {
  return __uint_as_float(key >> 31 ? key & 0x7fffffffu : ~key);
}
__device__ __forceinline__ uint64_t key_of(double s) {
  if (!(s == s)) s = -__builtin_huge_val();
  const uint64_t b = __double_as_longlong(s);
  return b >> 63 ? ~b : b | 0x8000000000000000ull;
}

// Sum over the block, for every thread.
__device__ __forceinline__ int block_sum(int v, int *s_sum) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = v;
  __syncthreads();
  int all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) all += s_sum[w];
  return all;
}
// Sum over the threads before this one.
__device__ __forceinline__ int block_below(int v, int *s_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s_sum[warp] = x;
  __syncthreads();
  int base = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w)
    if (w < warp) base += s_sum[w];
  return base + x - v;
}

__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Stores to the shared memory of the cluster's first CTA, at this CTA's address.
__device__ __forceinline__ void store_first(uint32_t addr, uint32_t v) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
      "st.shared::cluster.u32 [a], %1;\n\t}" ::"r"(addr),
      "r"(v)
      : "memory");
}

// The pages of a row and key/value head.  CS = 0: one block, the scores are in w.score.  CS > 0: a cluster of
// CS blocks scores the pages, and its first takes all scores in its shared memory and chooses.  The k-th score is
// found by bins between the least and the largest, mostly one pass, and by rank among the few in its bin.  Bound by
// latency: of 9.7 us for one token, 2047 pages and 8 heads, 3 are the loads of the row, its queries and bounds, 1.2 the
// scores, 0.9 the cluster's barrier, 1 each the bins and the masks of those chosen.  (32 tokens, 500 pages: 12.6 us,
// 17.9 with the scores in a kernel of their own.)  CS = 0 is bound by its barriers, so eight blocks an SM, in 32
// registers: 512 rows, 2 heads, 2000 pages, all 1024 blocks at once, 35.2 us with the scores; 38.4 with six in 40, no
// better than without a limit (47, 37.8), although 32 spill some words.  (Apart and cold: 23.4 the scores, 24.2 this.)
// So too where they are more than fit: us with eight, six, no limit, 2048 rows, 2 heads, 2000 pages 109, 116, 114; 2048
// rows, 8 heads of 128, 2048 pages 471, 496, 492; 4096 rows, 4 heads, 2000 pages 402, 443, 437.  One token each of 16
// sequences, 8 heads, 9376 pages 194, 196, 192.
// A least number for CS > 0 too lets the compiler take up to 205 registers: 12.9 us for the one token, 9.7 without.
template <typename T, int D, int CS>
__global__ void __launch_bounds__(kBlock, CS ? 0 : 8) pick_kernel(const Select w) {
  extern __shared__ __align__(16) uint32_t s_dyn[];
  __shared__ int s_sum[kWarps], s_bin, s_above, s_in_bin, s_count, s_in, s_mid_count, s_at[kFew];
  __shared__ uint32_t s_range[3 * (CS ? CS : 1)];  // of each block's part: least and largest key, largest size
  __shared__ double s_q[2 * D], s_exact[kFew];
  __shared__ float s_edge[2];
  const Params &p = w.p;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = CS > 1 ? blockIdx.x % CS : 0;
  const int row_i = w.row0 + blockIdx.x / (CS ? CS : 1), kvh = blockIdx.y;
  // behind score_kernel, which has waited for the batch, only the scores are waited for
  const bool behind = CS == 0 && w.width > w.n_select;
  if (!behind) pdl_wait();
  pdl_launch();
  if (blockIdx.x == 0 && row_i == 0 && kvh == 0)
    for (int i = threadIdx.x; i < p.n_seqs; i += kBlock) load_seq(p, i, true);
  const Row row = load_row(p, row_i, 1);
  const int pages = row.nq ? ((row.ctx - 1) >> p.page_shift) + 1 : 0;
  int32_t *out = w.out + (static_cast<int64_t>(row_i) * p.hkv + kvh) * w.n_select;
  if (pages <= w.n_select) {
    if (behind) pdl_wait();
    if (row.nq && rank == 0)
      for (int i = threadIdx.x; i < w.n_select; i += kBlock) out[i] = i < pages ? i : -1;
    return;
  }
  const int words = (pages + 31) / 32, j0 = w.sink, j1 = pages - w.recent, n = j1 - j0;
  const int want = w.n_select - w.sink - w.recent;
  // keys of 32 bits; where many scores are the same, the exact ones of 64 bits take their place
  uint32_t *s_sel = s_dyn, *s_mid = s_sel + words, *s_bins = s_mid + words, *s_keys = s_bins + kBins;
  float *score = w.score + (static_cast<int64_t>(blockIdx.x) * p.hkv + kvh) * 2 * w.width;
  const bool kept = CS > 0 || n <= kKeys;
  const auto key_at = [&](int i) { return kept ? s_keys[i] : key_of(score[j0 + i]); };
  uint32_t lo = ~0u, hi = 0u;
  uint32_t most = 0u;  // the largest size, which is positive or NaN: the order is that of the bits, and a NaN stays
  if constexpr (CS > 0) {
    constexpr int P = 4, kPages = P * (kBlock / 8);
    __shared__ __align__(16) float s_sums[2 * D];
    __shared__ float s_size;
    if (CS > 1) cluster_arrive();
    float size = 0.f;
    if (threadIdx.x == 0) s_size = 0.f;
    Block<T, D, P> b;
    int at = j0 + rank * kPages;
    const int end = want > 0 ? j1 : 0;
    b.look(w, row.seq, at, end);  // on their way during the sums
    __syncthreads();
    const float sizes = sum_heads<T, D>(p, row_i, kvh, s_sums);
    b.fetch(w, kvh, at, end);
    b.look(w, row.seq, at + CS * kPages, end);
    add_size<D>(sizes, &s_size);
    __syncthreads();
    if (CS > 1) cluster_wait();  // the first block is there
    for (; at < end; at += CS * kPages) {
      b.sizes();
      float s[P];
      b.score(s_sums, s);
#pragma unroll
      for (int t = 0; t < P; ++t) {
        const int i = at - j0 + (threadIdx.x >> 3) + t * (kBlock / 8);
        if ((threadIdx.x & 7) != 0 || i >= n) continue;
        const uint32_t key = key_of(s[t]);
        lo = min(lo, key), hi = max(hi, key);
        size = fmaxf(size, b.top[t]);
        if (CS > 1)
          store_first(smem_u32(s_keys + i), key);
        else
          s_keys[i] = key;
      }
      b.fetch(w, kvh, at + CS * kPages, end);
      b.look(w, row.seq, at + 2 * CS * kPages, end);
    }
    most = __float_as_uint(size * s_size);
  }
  if (rank == 0) {
    for (int i = threadIdx.x; i < words; i += kBlock) {
      // all 32 bits from bit 32 i on that are before j0 or from j1 to the end
      uint32_t m = 0;
      const int from = 32 * i;
      if (from < j0) m |= j0 - from >= 32 ? ~0u : (1u << (j0 - from)) - 1;
      if (from + 32 > j1) m |= from >= j1 ? ~0u : ~0u << (j1 - from);
      if (from + 32 > pages) m &= (1u << (pages - from)) - 1;
      s_sel[i] = m, s_mid[i] = 0u;
    }
    for (int i = threadIdx.x; i < kBins; i += kBlock) s_bins[i] = 0u;
    if (threadIdx.x == 0) s_count = s_in = s_mid_count = 0;
  }
  if (behind) pdl_wait();
  if (CS == 0 && want > 0) {
#pragma unroll 8
    for (int i = threadIdx.x; i < n; i += kBlock) {
      const uint32_t key = key_of(score[j0 + i]);
      if (kept) s_keys[i] = key;
      lo = min(lo, key), hi = max(hi, key);
    }
    for (int i = j0 / 16 + threadIdx.x; i <= (j1 - 1) / 16; i += kBlock)
      most = max(most, __float_as_uint(score[w.width + i]));
  }
  lo = __reduce_min_sync(0xffffffffu, lo), hi = __reduce_max_sync(0xffffffffu, hi);
  most = __reduce_max_sync(0xffffffffu, most);
  __shared__ uint32_t s_part[3][kWarps];
  if (lane == 0) s_part[0][warp] = lo, s_part[1][warp] = hi, s_part[2][warp] = most;
  __syncthreads();
#pragma unroll
  for (int v = 0; v < kWarps; ++v)
    lo = min(lo, s_part[0][v]), hi = max(hi, s_part[1][v]), most = max(most, s_part[2][v]);
  if constexpr (CS > 1) {
    if (threadIdx.x == 0) {
      store_first(smem_u32(s_range + 3 * rank), lo);
      store_first(smem_u32(s_range + 3 * rank + 1), hi);
      store_first(smem_u32(s_range + 3 * rank + 2), most);
    }
    cluster_arrive();
    cluster_wait();
    if (rank > 0) return;
#pragma unroll
    for (int v = 0; v < CS; ++v)
      lo = min(lo, s_range[3 * v]), hi = max(hi, s_range[3 * v + 1]), most = max(most, s_range[3 * v + 2]);
  }
  if (want > 0) {
    float size = __uint_as_float(most);
    if (!(size <= 3e38f)) size = -kNegInf;
    const float error = 2.f * w.error * size + 1e-40f;  // (products below fp32's range)
    // [lo, hi]: keys among which the want-th largest is; `above` keys are larger than those
    int above = 0, inside = n;
    while (lo < hi && inside > kFew / 4) {
      const int shift = max(0, 32 - __clz(hi - lo) - 10);
#pragma unroll 4
      for (int i = threadIdx.x; i < n; i += kBlock) {
        const uint32_t key = key_at(i);
        if (lo <= key && key <= hi) atomicAdd(&s_bins[(key - lo) >> shift], 1u);
      }
      __syncthreads();
      // bins from the largest keys down, some a thread
      constexpr int kEach = kBins / kBlock;
      uint32_t c[kEach];
      int sum = 0;
#pragma unroll
      for (int e = 0; e < kEach; ++e) c[e] = s_bins[kBins - 1 - kEach * threadIdx.x - e], sum += c[e];
      int before = above + block_below(sum, s_sum);
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        if (before < want && want <= before + static_cast<int>(c[e]))
          s_bin = kBins - 1 - kEach * threadIdx.x - e, s_above = before, s_in_bin = c[e];
        before += c[e];
        s_bins[kBins - 1 - kEach * threadIdx.x - e] = 0u;
      }
      __syncthreads();
      const uint32_t from = lo + (static_cast<uint32_t>(s_bin) << shift);
      lo = from;
      hi = min(hi, from + ((1u << shift) - 1));
      above = s_above, inside = s_in_bin;
    }
    // certainly in, and those that only fp64 can tell; a warp takes 32 pages, a word of the masks
    const float t_hi = score_of(hi) + error, t_lo = score_of(lo) - error;
    int in = 0, mid = 0;
#pragma unroll 4
    for (int i = warp; i < words; i += kWarps) {
      const int j = 32 * i + lane;
      bool is_in = false, is_mid = false;
      if (j >= j0 && j < j1) {
        const float s = score_of(key_at(j - j0));
        is_in = s > t_hi;
        is_mid = !is_in && !(s < t_lo);
      }
      const uint32_t m_in = __ballot_sync(0xffffffffu, is_in);
      const uint32_t m_mid = __ballot_sync(0xffffffffu, is_mid);
      in += __popc(m_in), mid += __popc(m_mid);
      if (lane == 0) s_sel[i] |= m_in, s_mid[i] = m_mid;
      if (is_mid) {
        const int at = atomicAdd(&s_count, 1);
        if (at < kFew) s_at[at] = j;
      }
    }
    if (lane == 0) atomicAdd(&s_in, in), atomicAdd(&s_mid_count, mid);
    __syncthreads();
    in = s_in, mid = s_mid_count;
    int need = want - in;  // of the mid ones: 1 .. mid
    // A few: fp32 tells those that are further than the error from the first that is left out, or from the last
    // that is taken.
    const bool told = need >= mid;
    if (told) {
      for (int i = threadIdx.x; i < words; i += kBlock) s_sel[i] |= s_mid[i];
    } else if (mid <= kFew) {
      float s = 0.f;
      int j = 0, ahead = 0;
      if (threadIdx.x < mid) {
        j = s_at[threadIdx.x];
        s = score_of(key_at(j - j0));
        for (int i = 0; i < mid; ++i) {
          const float other = score_of(key_at(s_at[i] - j0));
          ahead += other > s || (other == s && s_at[i] < j);
        }
        if (ahead == need - 1) s_edge[0] = s;
        if (ahead == need) s_edge[1] = s;
      }
      __syncthreads();
      const bool taken = threadIdx.x < mid && s > s_edge[1] + error;
      const bool left = threadIdx.x < mid && !taken && !(s < s_edge[0] - error);
      if (taken) atomicOr(&s_sel[j >> 5], 1u << (j & 31));
      if (threadIdx.x == 0) s_count = 0;
      need -= __syncthreads_count(taken);
      mid = __syncthreads_count(left);
      if (left) s_at[atomicAdd(&s_count, 1)] = j;
      __syncthreads();
    }
    if (!told && need > 0) {
      sum_heads<T, D>(p, row_i, kvh, s_q);
      __syncthreads();
      bool any = !(error <= 3e38f);  // (zeros times bounds that are infinite are NaN, which has the lowest score)
      for (int d = threadIdx.x; d < 2 * D; d += kBlock) any |= s_q[d] != 0.;
      any = __syncthreads_or(any);  // without (a row of padding), fp32 scores are exact: 0, or the lowest
      const auto exact = [&](int j) {  // a whole warp
        const int page = p.table[row.seq * p.table_stride + j];
        if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.n_pages))
          return -__builtin_huge_val();
        const T *src =
            static_cast<const T *>(w.bounds) + (static_cast<int64_t>(page) * p.hkv + kvh) * 2 * D;
        double x = 0.;
        for (int d = lane; d < 2 * D; d += 32)
          x = fma(s_q[d], static_cast<double>(static_cast<float>(src[d])), x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        return x == x ? x : -__builtin_huge_val();
      };
      if (mid <= kFew) {
        for (int i = warp; i < mid; i += kWarps) {
          const double x = any ? exact(s_at[i]) : score_of(key_at(s_at[i] - j0));
          if (lane == 0) s_exact[i] = x;
        }
        __syncthreads();
        if (threadIdx.x < mid) {
          const double x = s_exact[threadIdx.x];
          const int j = s_at[threadIdx.x];
          int ahead = 0;
          for (int i = 0; i < mid; ++i) ahead += better(s_exact[i], s_at[i], x, j);
          if (ahead < need) atomicOr(&s_sel[j >> 5], 1u << (j & 31));
        }
      } else {
        // Many pages with the same score but for rounding.  Their fp64 keys take the scores' place, and
        // the need-th largest is found bit by bit.  (Without `any` they have the same: the bins have told 0 and
        // the lowest apart.)
        uint64_t *key = CS ? reinterpret_cast<uint64_t *>(s_keys) - j0 : reinterpret_cast<uint64_t *>(score);
        for (int i = warp; any && i < words; i += kWarps)
          for (uint32_t m = s_mid[i]; m; m &= m - 1) {
            const int j = 32 * i + __ffs(m) - 1;
            const double x = exact(j);
            if (lane == 0) key[j] = key_of(x);
          }
        __syncthreads();
        const auto count = [&](uint64_t least) {
          int c = 0;
          for (int i = threadIdx.x; i < words; i += kBlock)
            for (uint32_t m = s_mid[i]; m; m &= m - 1) c += key[32 * i + __ffs(m) - 1] >= least;
          return block_sum(c, s_sum);
        };
        uint64_t last = 0;
        for (int b = 63; any && b >= 0; --b)
          if (count(last | 1ull << b) >= need) last |= 1ull << b;
        const int ties = any ? need - count(last + 1) : need;  // the lower pages
        const int each = (words + kBlock - 1) / kBlock;
        const int i0 = min(words, static_cast<int>(threadIdx.x) * each), i1 = min(words, i0 + each);
        int mine = 0;
        for (int i = i0; i < i1; ++i)
          for (uint32_t m = s_mid[i]; m; m &= m - 1)
            mine += !any || key[32 * i + __ffs(m) - 1] == last;
        int before = block_below(mine, s_sum);
        for (int i = i0; i < i1; ++i)
          for (uint32_t m = s_mid[i]; m; m &= m - 1) {
            const uint64_t x = any ? key[32 * i + __ffs(m) - 1] : last;
            if (x > last || (x == last && before++ < ties)) s_sel[i] |= m & -m;
          }
      }
    }
  }
  __syncthreads();
  // the pages in order
  int done = 0;
  for (int b = 0; b < words; b += kBlock) {
    const int i = b + threadIdx.x;
    const uint32_t mine = i < words ? s_sel[i] : 0u;
    int at = done + block_below(__popc(mine), s_sum);
    for (uint32_t m = mine; m; m &= m - 1, ++at)
      if (at < w.n_select) out[at] = 32 * i + __ffs(m) - 1;
    if (b + kBlock < words) done += block_sum(__popc(mine), s_sum);
  }
}

struct SelectPlan {
  int cluster;    // blocks that take a row and head; 0: scores go through the workspace
  int rows;       // of one launch
  int64_t bytes;
};

// Scores of all rows at once, while they take no more than this.
constexpr int64_t kMostScores = 1ll << 28;

static int plan_select(const Params &p, SelectPlan *plan) {
  if (p.table_width > kMaxPages || p.hkv > 65535) return MOE_ERR_UNSUPPORTED;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MOE_ERR_CUDA;
  plan->bytes = 0;
  plan->rows = p.n_rows;
  // Sequences of some rows share what is read; a token by itself is taken by one kernel, with as many blocks as
  // there is room for.
  if (p.n_rows < 4 * static_cast<int64_t>(p.n_seqs) && p.table_width <= kKeys) {
    plan->cluster = 16;
    while (plan->cluster > 1 && static_cast<int64_t>(p.n_rows) * p.hkv * plan->cluster > 2 * sms)
      plan->cluster /= 2;
    return MOE_OK;
  }
  plan->cluster = 0;
  const int64_t row = 8ll * p.hkv * p.table_width;
  plan->rows = static_cast<int>(std::min<int64_t>(p.n_rows, std::max<int64_t>(1, kMostScores / row)));
  plan->bytes = row * plan->rows;
  return MOE_OK;
}

template <typename T, int D, int CS>
static cudaError_t launch_cluster(const Select &w, cudaStream_t stream) {
  const auto pick = pick_kernel<T, D, CS>;
  const auto smem = [](int pages) { return 4 * (2 * ((pages + 31) / 32) + kBins) + 8 * pages; };
  static SmemLimit limit;
  cudaError_t e = limit.set(reinterpret_cast<const void *>(pick), smem(kKeys), CS > 8);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(w.rows * CS, w.p.hkv);
  cfg.blockDim = dim3(kBlock);
  cfg.dynamicSmemBytes = smem(w.width);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CS;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CS > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, pick, w);
}

template <typename T, int D>
static cudaError_t launch_select(Select w, const SelectPlan &plan, cudaStream_t stream) {
  const Params &p = w.p;
  w.row0 = 0;
  w.rows = p.n_rows;
  switch (plan.cluster) {
    case 16: return launch_cluster<T, D, 16>(w, stream);
    case 8: return launch_cluster<T, D, 8>(w, stream);
    case 4: return launch_cluster<T, D, 4>(w, stream);
    case 2: return launch_cluster<T, D, 2>(w, stream);
    case 1: return launch_cluster<T, D, 1>(w, stream);
  }
  const auto pick = pick_kernel<T, D, 0>;
  const auto smem = [](int pages) {
    return 4 * (2 * ((pages + 31) / 32) + kBins + std::min(pages, kKeys));
  };
  static SmemLimit limit;
  cudaError_t e = limit.set(reinterpret_cast<const void *>(pick), smem(kMaxPages));
  if (e != cudaSuccess) return e;
  constexpr int kPages = kTurns * kPagesATurn;
  // truncations of 2^-23: 32 of products, as many for the split in two of bf16, 2 D / 32 + 2 of sums, group of Q's
  w.error = (32 + (Half<T>::kRow > 0.f ? 0 : 32) + 2 * D / 32 + 4 + p.group) * 1.2e-7f;
  for (; w.row0 < p.n_rows; w.row0 += plan.rows) {
    w.rows = std::min(plan.rows, p.n_rows - w.row0);
    if (p.table_width > w.n_select) {  // (otherwise every page of every row is selected)
      const dim3 grid((w.rows + kRowTile - 1) / kRowTile, p.hkv, (p.table_width + kPages - 1) / kPages);
      e = launch_early(score_kernel<T, D>, grid, kBlock, 0, stream, w);
      if (e != cudaSuccess) return e;
    }
    e = launch_early(pick, dim3(w.rows, p.hkv), kBlock, smem(w.width), stream, w);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace attn

extern "C" int moe_page_bounds(const moe_kv_cache *cache, const moe_attention *a, void *bounds,
                               void *stream) {
  attn::Params p;
  const int rc = attn::check_attention(cache, a, &p, 0);
  if (rc != MOE_OK) return rc;
  if (!bounds || !attn::aligned(bounds, 16)) return MOE_ERR_INVALID_ARG;
  if (p.hkv > 65535) return MOE_ERR_UNSUPPORTED;
  if (p.n_seqs == 0 || p.n_rows == 0) return MOE_OK;
  // a sequence of r > 0 rows has new positions on at most min(r, (r - 1) / page + 2) pages
  const int64_t pages = std::min<int64_t>(p.n_rows, (p.n_rows >> p.page_shift) + 2ll * p.n_seqs);
  const dim3 grid(static_cast<unsigned>(pages), p.hkv);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  using B = __nv_bfloat16;
  using H = __half;
  cudaError_t e;
  if (cache->dtype == MOE_DTYPE_BF16)
    e = attn::launch_early(cache->head_dim == 64 ? attn::bounds_kernel<B, 64> : attn::bounds_kernel<B, 128>,
                           grid, attn::kBlock, 0, st, p, static_cast<B *>(bounds));
  else
    e = attn::launch_early(cache->head_dim == 64 ? attn::bounds_kernel<H, 64> : attn::bounds_kernel<H, 128>,
                           grid, attn::kBlock, 0, st, p, static_cast<H *>(bounds));
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" int moe_select_pages_workspace(const moe_kv_cache *cache, const moe_attention *a,
                                          int64_t *bytes) {
  attn::Params p;
  int rc = attn::check_attention(cache, a, &p, attn::kUsesQ);
  if (rc != MOE_OK) return rc;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = 0;
  if (p.n_seqs == 0 || p.n_rows == 0) return MOE_OK;
  attn::SelectPlan plan;
  rc = attn::plan_select(p, &plan);
  if (rc == MOE_OK) *bytes = plan.bytes;
  return rc;
}

extern "C" int moe_select_pages(const moe_kv_cache *cache, const moe_attention *a, const void *bounds,
                                int32_t n_select, int32_t sink, int32_t recent, int32_t *pages,
                                void *workspace, int64_t workspace_bytes, void *stream) {
  attn::Select w;
  int rc = attn::check_attention(cache, a, &w.p, attn::kUsesQ);
  if (rc != MOE_OK) return rc;
  if (sink < 0 || recent < 1 || n_select < static_cast<int64_t>(sink) + recent ||
      !attn::aligned(bounds, 16) || !attn::aligned(pages, 4) || workspace_bytes < 0 ||
      !attn::aligned(workspace, 16))
    return MOE_ERR_INVALID_ARG;
  if (w.p.n_seqs == 0 || w.p.n_rows == 0) return MOE_OK;
  if (!bounds || !pages) return MOE_ERR_INVALID_ARG;
  attn::SelectPlan plan;
  rc = attn::plan_select(w.p, &plan);
  if (rc != MOE_OK) return rc;
  if (plan.bytes && (!workspace || workspace_bytes < plan.bytes)) return MOE_ERR_INVALID_ARG;
  w.bounds = bounds;
  w.score = static_cast<float *>(workspace);
  w.out = pages;
  w.width = w.p.table_width;
  w.n_select = n_select;
  w.sink = sink;
  w.recent = recent;
  w.error = (w.p.group + 12) * 6e-8f;  // group roundings of Q, 10 of a score (Block), one way after the other
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (cache->dtype == MOE_DTYPE_BF16)
    e = cache->head_dim == 64 ? attn::launch_select<__nv_bfloat16, 64>(w, plan, st)
                              : attn::launch_select<__nv_bfloat16, 128>(w, plan, st);
  else
    e = cache->head_dim == 64 ? attn::launch_select<__half, 64>(w, plan, st)
                              : attn::launch_select<__half, 128>(w, plan, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
