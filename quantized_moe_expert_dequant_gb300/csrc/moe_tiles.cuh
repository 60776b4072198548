// moe_tiles.cuh -- attention in tiles of 128 rows over the pages of a cache, on the 5th-generation tensor
// cores: causal for packed prompts (moe_prompt.cu), by masks for large trees of drafted tokens
// (moe_prompt_tree.cu).
//
//   out_r = sum_j p_rj v_j / sum_j p_rj,   p_rj = exp(scale * q_r . k_j - m_r)  over the positions j
//   that row r sees, in one pass over K and V; m_r goes by some of the scores (reference).
//
// Bound by the two products (4 D flops per row and position).  An item is two tiles of up to 128 rows of
// one sequence and one key/value head: row R of a tile is token R / group, query head R % group, so
// all query heads of a key/value head share the K and V that are loaded once, and a short prompt
// still fills the tiles.  Per 128 positions and tile:
//   S = Q K^T    128 x 128 x D, both operands in shared memory, S in TMEM
//   softmax      four warps, one row a thread: S from TMEM to registers, P to TMEM in 16 bits
//   O += P V     128 x D x 128, P from TMEM, V from shared memory, O in TMEM
// The two tiles take turns: while four warps are at one tile's softmax, the tensor cores work on
// the other tile.  One warp issues all products, in an order in which they also complete, one finds
// the items, one copies.  O is only scaled down when a row's weights have outgrown what the type
// holds (kMostWeight).
//
// One persistent CTA an SM.  Measured (32 query, 8 key/value heads of 128, bf16, 8192 tokens, causal):
// 2567 us with 64-row tiles on mma.sync, 496 us with one CTA per two tiles, 374 us when the
// products' loop is uniform in its warp (descriptors in a one-lane branch cost 100 cycles a product),
// 348 us with the work shared evenly, 341 us without a maximum in every step (1.61 PFLOP/s; called again and
// again, at the power limit and 1910 instead of 2070 MHz, 367 us: 1.50 PFLOP/s).  A step of
// 128 positions takes 2620 cycles, the products 2048 of them at the peak rate: with both operands in
// shared memory S runs at 128 bytes a cycle, the limit, and takes about 90 cycles instead of 64 a
// product.  Slower were sixteen softmax warps of half a row a thread (403 us to 374), a ring of four
// tiles (455 to 356), and handing P over in halves once no maximum is in the way (409 to 342).
#pragma once

#include "moe_attention.cuh"
#include "moe_tcgen05.cuh"

#include <type_traits>

namespace attn {

constexpr int kPos = 128;               // positions of a step
constexpr int kSoftmaxWarps = 8;        // four a tile
constexpr int kPromptThreads = 32 * (kSoftmaxWarps + 4);  // and products, copies, items, an idle warp
// 168 registers at launch; 2 x 128 x 216 + 128 x 72 = 384 x 168
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;
constexpr int kItems = 4;               // items between the warp that finds them and the others
// Sum of a row's weights in a step from which O is rescaled: no weight is larger, so none is infinite in fp16.
template <typename T>
constexpr float kMostWeight = std::is_same<T, __half>::value ? 65504.f : 8192.f;

template <int D>
struct Prompt {
  static constexpr int kTileBytes = kPos * D * 2;             // K, V or a tile of Q
  static constexpr int kStages = D == 128 ? 5 : 8;            // ring of K and V tiles, in turn
  static constexpr int kSmem = (2 + kStages) * kTileBytes + 1024;
  static constexpr int kColumns = 512;                        // S0 S1 (128 each) O0 O1 (D each)
  // Heads of 64 leave TMEM room for P beside S: the next S is then computed as soon as the last one
  // has been read, and the softmax bounds the step.  With heads of 128, P lies over S, and S waits
  // for P V.
  static constexpr bool kBeside = D == 64;
};

struct PromptParams {
  Params p;
  CUtensorMap q, k, v;
  int tokens;        // of a tile: 128 / group
  float *part;       // [2 G][2][D / 4][128][4]: parts of outputs, four columns of a tile's rows together
  float2 *part_ml;   // [2 G][2][128] (reference maximum, sum)
  struct Share *share;  // [G], null when no item can be shared
  // of a wait of the copies and the products; the other warps' is fixed and they leave with these (a limit in
  // memory in each wait of the softmax: 124 us for 120 on chunks behind prefixes, heads of 64)
  tc::Limit limit;
};

// ------------------------------------------------------------------ who does what
// An item is one sequence, one key/value head and two tiles of rows; its cost is the positions that
// its last row sees (all, with tree masks), and kItemCost for its beginning and end.  The costs of all
// items, sequence by sequence, head by head, form one line that the CTAs share evenly, whatever the
// lengths are; a boundary inside an item becomes a boundary between two of its steps, or moves to
// the item's edge when fewer than kMinSteps steps would be cut off.  (16 packed prompts of 62 to 1984
// tokens, cost 160, 224, 320: 96.9, 94.7, 96.3 us; least 2, 4 steps: 93.5, 94.7.)
constexpr int kItemCost = 224;
constexpr int kMinSteps = 2;
// Steps of the longest item that the table allows, from which items are shared at all: below, a boundary
// moves to the nearer edge of its item, and no parts are joined.  (32 query, 8 key/value heads of 128,
// us shared and not: one prompt of 700 tokens 21.6, 18.2; of 1000 27.3, 21.1; of 2000 43.7, 46.8; of
// 4000 105, 121; 16 of 1000 147, 143.)
constexpr int kShareSteps = 9;

struct Spot {  // the place before a step of an item
  int seq, head, tile, step;
};

__device__ __forceinline__ bool before(const Spot &a, const Spot &b) {
  if (a.seq != b.seq) return a.seq < b.seq;
  if (a.head != b.head) return a.head < b.head;
  if (a.tile != b.tile) return a.tile < b.tile;
  return a.step < b.step;
}
__device__ __forceinline__ bool same_item(const Spot &a, const Spot &b) {
  return a.seq == b.seq && a.head == b.head && a.tile == b.tile;
}

// What a CTA tells join_kernel: whether an item goes on into the next CTA (its last), which it is, and
// whether its first is the continuation of an earlier CTA's and ends here.
struct Share {
  int tail, head, head_ends;
  int row0, nq, kvh, tok0;
};

// Cost of the first k of a head's `tiles` items; per tokens an item.
__device__ __forceinline__ int64_t head_cost(const Seq &s, bool tree, int per, int tiles, int k) {
  if (tree) return static_cast<int64_t>(k) * (s.len + kItemCost);
  const int64_t full = k < tiles ? k : k - 1;
  return static_cast<int64_t>(k) * (s.ctx + kItemCost) + per * (full * (full + 1) / 2) +
         (k == tiles ? s.nq : 0);
}
__device__ __forceinline__ int item_steps(const Seq &s, bool tree, int per, int tile) {
  const int64_t seen =
      tree ? s.len
           : s.ctx + min(static_cast<int64_t>(tile + 1) * per, static_cast<int64_t>(s.nq));
  return static_cast<int>((seen + kPos - 1) / kPos);
}
__device__ __forceinline__ int item_count(const Seq &s, int per) { return (s.nq + per - 1) / per; }

__device__ __forceinline__ Spot spot_at(const Seq &s, bool tree, bool shared, int seq, int per,
                                        int64_t y) {
  const int tiles = item_count(s, per);
  const int64_t whole = head_cost(s, tree, per, tiles, tiles);
  Spot r;
  r.seq = seq;
  r.head = static_cast<int>(y / whole);
  y -= r.head * whole;
  // k (ctx + kItemCost) + per k (k + 1) / 2 = y, then the exact k next to it
  const float b = s.ctx + kItemCost + 0.5f * per;
  int k = tree ? static_cast<int>(y / (s.len + kItemCost))
               : static_cast<int>((sqrtf(b * b + 2.f * per * static_cast<float>(y)) - b) / per);
  k = max(0, min(k, tiles - 1));
  while (k > 0 && head_cost(s, tree, per, tiles, k) > y) --k;
  while (k + 1 < tiles && head_cost(s, tree, per, tiles, k + 1) <= y) ++k;
  const int64_t at = head_cost(s, tree, per, tiles, k), cost = head_cost(s, tree, per, tiles, k + 1) - at;
  const int n = item_steps(s, tree, per, k);
  int step = static_cast<int>((y - at) * n / cost);
  if (!shared) step = 2 * (y - at) < cost ? 0 : n;  // the nearer edge
  if (step < kMinSteps) step = 0;
  r.tile = k;
  r.step = step;
  if (step > 0 && n - step < kMinSteps) r.tile = k + 1, r.step = 0;
  return r;
}

// Sums v over the block (every thread gets the sum) and gives each thread the sum before it.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *s_warp, int64_t *below) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  int64_t base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kPromptThreads / 32; ++w) {
    if (w < warp) base += s_warp[w];
    all += s_warp[w];
  }
  *below = base + x - v;
  return all;
}

// The CTA's part of the line: from s_spot[0] to s_spot[1].  False when there is nothing at all.
__device__ __forceinline__ bool find_part(const Params &p, bool tree, bool shared, int per,
                                          int64_t *s_warp, Spot *s_spot) {
  const auto cost = [&](const Seq &s) {
    if (s.nq == 0) return static_cast<int64_t>(0);
    const int tiles = item_count(s, per);
    return p.hkv * head_cost(s, tree, per, tiles, tiles);
  };
  int64_t total = 0, below = 0, mine = 0;
  Seq s = {0, 0, 0, 0};
  for (int b = 0; b < p.n_seqs; b += kPromptThreads) {
    const int i = b + threadIdx.x;
    mine = 0;
    if (i < p.n_seqs) s = load_seq(p, i, blockIdx.x == 0), mine = cost(s);
    total += block_scan(mine, s_warp, &below);
  }
  if (total == 0) return false;
  const int64_t edge[2] = {blockIdx.x * total / gridDim.x, (blockIdx.x + 1) * total / gridDim.x};
  if (threadIdx.x == 0 && edge[1] == total) s_spot[1] = {p.n_seqs, 0, 0, 0};
  int64_t sum = 0;
  for (int b = 0; b < p.n_seqs; b += kPromptThreads) {
    const int i = b + threadIdx.x;
    if (p.n_seqs > kPromptThreads) {
      mine = 0;
      if (i < p.n_seqs) s = load_seq(p, i, false), mine = cost(s);
      const int64_t all = block_scan(mine, s_warp, &below);
      below += sum;
      sum += all;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (below <= edge[e] && edge[e] < below + mine)
        s_spot[e] = spot_at(s, tree, shared, i, per, edge[e] - below);
  }
  __syncthreads();
  return true;
}

// An item as the warps work on it: the sequence, its first token here, the steps from `a` on that are
// this CTA's, and how many of them each tile has.  more = 0: the CTA's part of the line is done.
struct alignas(16) Item {
  int more, seq, kvh, row0, ctx, nq, len, tok0, a, count[2], steps, whole, pad[3];
};
static_assert(sizeof(Item) == 64, "read as four 16-byte words");

// Walks a CTA's part of the line, item by item.
struct Walk {
  const Params &p;
  const bool tree;
  const int tokens, per;
  Spot at, end;
  Seq s;
  int tiles;

  __device__ __forceinline__ Walk(const Params &p, bool tree, int tokens, const Spot *spot)
      : p(p), tree(tree), tokens(tokens), per(2 * tokens), at(spot[0]), end(spot[1]) {
    s = load_seq(p, min(at.seq, p.n_seqs - 1), false);
    tiles = item_count(s, per);
  }
  __device__ __forceinline__ Item next() {
    Item r = {};
    for (;;) {
      if (!before(at, end) || at.seq >= p.n_seqs) return r;
      if (at.tile < tiles) break;
      at.tile = 0;
      if (s.nq == 0 || ++at.head >= p.hkv) {
        at.head = 0;
        if (++at.seq >= p.n_seqs) return r;
        s = load_seq(p, at.seq, false);
        tiles = item_count(s, per);
      }
    }
    r.more = 1;
    r.seq = at.seq, r.kvh = at.head;
    r.row0 = s.row0, r.ctx = s.ctx, r.nq = s.nq, r.len = s.len;
    r.tok0 = at.tile * per;
    r.a = at.step;
    const int n = item_steps(s, tree, per, at.tile);
    const int b = same_item(at, end) ? end.step : n;
    r.whole = r.a == 0 && b == n;
    const int n0 = tree ? n : (s.ctx + min(r.tok0 + tokens, s.nq) + kPos - 1) / kPos;
    r.count[0] = max(0, min(b, n0) - r.a);
    r.count[1] = r.tok0 + tokens < s.nq ? b - r.a : 0;
    r.steps = max(r.count[0], r.count[1]);
    at.step = 0;
    ++at.tile;
    return r;
  }
};

__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The largest score of a row, and the lowest of the maxima of its quarters.
struct Top {
  float max, low;
};
__device__ __forceinline__ Top row_max(const uint32_t (&x)[4][32]) {
  float top[4];  // four chains: one of 64 dependent maxima took 500 cycles
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    top[c] = __uint_as_float(x[c][0]);
#pragma unroll
    for (int e = 1; e < 31; e += 2)
      top[c] = max3(top[c], __uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1]));
    top[c] = fmaxf(top[c], __uint_as_float(x[c][31]));
  }
  return {fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])),
          fminf(fminf(top[0], top[1]), fminf(top[2], top[3]))};
}

// What a row's weights are taken relative to from its first step on: the maximum there, in bf16.  fp16
// holds 2^16 down to 2^-14 in full.  Most rows get scores above those of their first step, so the maximum
// is at 2^0; but a score that stands out from the lowest quarter's by more than 2^6 is higher by as much, up to
// 2^8, so that the others keep their bits beside it.  A row that outgrows its reference later has a score that
// stands out, at 2^8 from then on; the 128 weights of a step then stay below 2^16.
// (8192 tokens, heads of 128, scores with a standard deviation of 1.5, 3, 4.5, 6: 383, 383, 383, 446 us; 382, 384,
// 404, 434 us with the maximum and 2^13 as the bound; 375, 453, 490, 489 us with the maximum always at 2^10.)
template <typename T>
__device__ __forceinline__ float reference(const Top &t, const Params &p) {
  if (!std::is_same<T, __half>::value) return t.max;
  const float up = fminf(fmaxf((t.max - t.low) * p.scale_log2 - 6.f, 0.f), 8.f);
  return t.max - up * p.octave;  // -inf: no score is seen
}
template <typename T>
__device__ __forceinline__ float outgrown(float top, const Params &p) {
  return std::is_same<T, __half>::value ? top - 8.f * p.octave : top;
}

// The weights exp2(scale * x - off) of 32 positions: their pairs in 16 bits in y, added to sum.  Eight
// positions at a time, the use of each eight one group behind their exponentials.
template <typename T>
__device__ __forceinline__ void weights(const uint32_t (&x)[32], float off, float scale,
                                        uint64_t (&sum)[2], uint32_t (&y)[16]) {
  const uint64_t sc = pair(scale, scale), shift = pair(-off, -off);
  float w[2][8];
#pragma unroll
  for (int g = 0; g < 5; ++g) {
    if (g < 4) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float2 a = unpair(fma2(
            pair(__uint_as_float(x[8 * g + e]), __uint_as_float(x[8 * g + e + 1])), sc, shift));
        w[g & 1][e] = exp2_approx(a.x);
        w[g & 1][e + 1] = exp2_approx(a.y);
      }
    }
    if (g > 0) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float pa = w[(g - 1) & 1][e], pb = w[(g - 1) & 1][e + 1];
        sum[e / 2 % 2] = add2(sum[e / 2 % 2], pair(pa, pb));
        // the weights meet v in the cache's type
        y[(8 * (g - 1) + e) / 2] = Half<T>::pack(pa, pb);
      }
    }
  }
}

// The weights of a row's 128 positions, stored to TMEM at tp; their sum.
template <typename T>
__device__ __forceinline__ float store_weights(const uint32_t (&x)[4][32], float off, float scale,
                                               uint32_t tp) {
  uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t y[16];
    weights<T>(x[c], off, scale, sum, y);
    tc::tmem_store16(tp + 16 * c, y);
  }
  const float2 total = unpair(add2(sum[0], sum[1]));
  return total.x + total.y;
}

template <typename T, int D, bool tree>
__global__ void __launch_bounds__(kPromptThreads, 1)
    prompt_kernel(const __grid_constant__ PromptParams w) {
  using C = Prompt<D>;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t s_q[2], s_q_free[2], s_full[C::kStages], s_empty[C::kStages],
      s_s[2], s_x[2], s_p[2], s_o[2], s_end, s_item_full[kItems], s_item_free[kItems];
  __shared__ Item s_item[kItems];
  __shared__ int64_t s_warp[kPromptThreads / 32];
  __shared__ Spot s_spot[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_gone;
  const Params &p = w.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  const auto bar = [](uint64_t &b) { return smem_u32(&b); };
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::bar_init(bar(s_q[i]), 1);
      tc::bar_init(bar(s_q_free[i]), 1);
      tc::bar_init(bar(s_s[i]), 1);
      tc::bar_init(bar(s_x[i]), kSoftmaxWarps / 2);
      tc::bar_init(bar(s_p[i]), kSoftmaxWarps / 2);
      tc::bar_init(bar(s_o[i]), 1);
    }
    for (int i = 0; i < C::kStages; ++i) {
      tc::bar_init(bar(s_full[i]), 1);
      tc::bar_init(bar(s_empty[i]), 1);
    }
    for (int i = 0; i < kItems; ++i) {
      tc::bar_init(bar(s_item_full[i]), 1);
      tc::bar_init(bar(s_item_free[i]), kSoftmaxWarps + 2);
    }
    tc::bar_init(bar(s_end), 1);
    s_gone = 0;
    tc::bar_fence_init();
  }
  pdl_launch();
  const bool any = find_part(p, tree, w.share != nullptr, 2 * w.tokens, s_warp, s_spot);
  if (w.share && threadIdx.x == 0) {
    Share sh = {};
    if (any && before(s_spot[0], s_spot[1])) {
      const Spot &a = s_spot[0], &b = s_spot[1];
      const bool one = same_item(a, b);  // nothing but a piece of one item
      sh.head = a.step > 0;
      sh.head_ends = !one;
      sh.tail = b.step > 0 && !(one && a.step > 0);
      if (sh.tail) {
        const Seq q = load_seq(p, b.seq, false);
        sh.row0 = q.row0, sh.nq = q.nq, sh.kvh = b.head, sh.tok0 = b.tile * 2 * w.tokens;
      }
    }
    w.share[blockIdx.x] = sh;
  }
  if (!any || !before(s_spot[0], s_spot[1])) return;
  if (warp == kSoftmaxWarps) tc::tmem_alloc(smem_u32(&s_tmem), C::kColumns);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = s_tmem;
  const uint32_t ring = base + 2 * C::kTileBytes;
  // columns of P: over S, or behind O
  const auto p_col = [](int i) { return C::kBeside ? 2 * kPos + 2 * D + i * (kPos / 2) : i * kPos; };

  int taken = 0;  // items
  const auto take = [&](Item &item) {  // a whole warp; false: no more, or a wait gave up
    const int at = taken % kItems;
    const bool ok = tc::bar_wait(bar(s_item_full[at]), (taken / kItems) & 1, &s_gone);
    if (!__all_sync(0xffffffffu, ok)) return false;
    item = s_item[at];
    __syncwarp();
    if (lane == 0) tc::bar_arrive(bar(s_item_free[at]));
    ++taken;
    return item.more != 0;
  };

  if (warp >= kSoftmaxWarps) tc::regs_down<kOtherRegs>();
  if (warp == kSoftmaxWarps + 2) {
    // ---------------------------------------------------------------- items, ahead of the others
    if (lane == 0) {
      Walk walk(p, tree, w.tokens, s_spot);
      for (int it = 0;; ++it) {
        const Item item = walk.next();
        if (!tc::bar_wait(bar(s_item_free[it % kItems]), ((it / kItems) & 1) ^ 1, &s_gone)) break;
        s_item[it % kItems] = item;
        tc::bar_arrive(bar(s_item_full[it % kItems]));
        if (!item.more) break;
      }
    }
    __syncwarp();
  } else if (warp == kSoftmaxWarps + 1) {
    // ---------------------------------------------------------------- copies
    // a box is one page's positions of a step (all 128 for larger pages), 64 elements wide; lanes
    // take one each
    const int box_rows = min(1 << p.page_shift, kPos);
    const int per_half = kPos / box_rows, boxes = per_half * (D / 64);
    const int b_row = (lane % per_half) * box_rows, half = lane / per_half;
    int issued = 0, q_loads[2] = {0, 0};  // tiles into the ring, tiles of Q
    // The products' warp goes on to the end of its step when a wait of its has given up, and gives stages back
    // whose copies are still under way: nothing is copied there then.
    const auto free = [&](uint32_t b, int parity) {
      return tc::bar_wait(b, parity, &s_gone, w.limit) && !*static_cast<volatile int *>(&s_gone);
    };
    bool ok = true;
    Item item;
    while (ok && take(item)) {
      const int32_t *pages = p.table + item.seq * p.table_stride;
      const auto page_of = [&](int t) {
        const int pos = t * kPos + b_row;
        return lane < boxes && pos < item.len ? pages[pos >> p.page_shift] : p.n_pages;
      };
      int page = page_of(item.a);
      for (int t = item.a; ok && t < item.a + item.steps; ++t) {
        const int pos = t * kPos + b_row;
        if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.n_pages)) {
          if (lane < boxes && pos < item.len && p.err) atomicOr(p.err, kDevErrBadId);
          page = p.n_pages;  // outside the cache: reads zeros
        }
        const int next_page = page_of(t + 1);  // on its way while this step waits for the ring
        const int in_page = pos & ((1 << p.page_shift) - 1);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int st = issued % C::kStages;
          ok = ok && free(bar(s_empty[st]), ((issued / C::kStages) & 1) ^ 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) continue;
          if (lane == 0) tc::bar_expect(bar(s_full[st]), C::kTileBytes);
          __syncwarp();
          if (lane < boxes)
            tc::copy_4d(ring + st * C::kTileBytes + half * kPos * 128 + b_row * 128,
                        kv ? &w.v : &w.k, 64 * half, in_page, item.kvh, page, bar(s_full[st]));
          ++issued;
          if (kv == 1 || t > item.a) continue;
          // Q between the first K and the first V: its place is free only shortly before
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (item.count[i] == 0) continue;
            ok = ok && free(bar(s_q_free[i]), (q_loads[i] & 1) ^ 1);
            ok = __all_sync(0xffffffffu, ok);
            if (ok && lane == 0) {
              tc::bar_expect(bar(s_q[i]), static_cast<uint32_t>(w.tokens * p.group * D * 2));
              for (int h = 0; h < D / 64; ++h)
                tc::copy_3d(base + i * C::kTileBytes + h * kPos * 128, &w.q, 64 * h,
                            item.kvh * p.group, item.row0 + item.tok0 + i * w.tokens, bar(s_q[i]));
            }
            if (ok) ++q_loads[i];
          }
        }
        page = next_page;
      }
    }
    // The copies under way land before the shared memory goes: those that nobody waits for when some
    // warp gives up, now or after this one has issued its last.
    volatile int never = 0;
    for (int it = issued > C::kStages ? issued - C::kStages : 0; it < issued; ++it)
      tc::bar_wait(bar(s_full[it % C::kStages]), (it / C::kStages) & 1, &never);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (q_loads[i] > 0) tc::bar_wait(bar(s_q[i]), (q_loads[i] - 1) & 1, &never);
  } else if (warp == kSoftmaxWarps) {
    // ---------------------------------------------------------------- products
    // Everything here is the same for all lanes (the shuffles say so to the compiler); `one` issues.
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr uint32_t i_s = tc::instr(kBf16, false, 128, kPos);
    constexpr uint32_t i_o = tc::instr(kBf16, true, 128, D);
    constexpr uint32_t hi = tc::desc_hi(1024);
    const auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    const uint32_t one = tc::elect();
    const uint32_t tm = uniform(tmem), ub = uniform(base);
    const uint32_t q_lo = tc::desc_lo(ub, 16);
    // A wait that gives up shows in s_gone, which ends the loop; what is issued until then only
    // reads and writes this CTA's own shared memory and TMEM.  No branch depends on a wait, so that the
    // descriptors stay in uniform registers.
    const auto wait = [&](uint32_t b, int parity) {
      if (!tc::bar_test(b, parity)) tc::bar_wait(b, parity, &s_gone, w.limit);
      __syncwarp();
    };
    const auto stage = [&](int i) { return ub + (2 + i) * C::kTileBytes; };
    int st = 0, phase = 0;  // the ring's next stage
    const auto turn = [&]() {
      if (++st == C::kStages) st = 0, phase ^= 1;
    };
    int n_q[2] = {0, 0}, n_p[2] = {0, 0};  // tiles of Q, steps so far
    int k_before = 0, v_before = -1;       // stages to give back: this step's K, the last one's V
    bool gone = false;
    Item item;
    while (!gone && take(item)) {
      const int u[2] = {uniform(item.count[0]), uniform(item.count[1])}, last = uniform(item.steps);
      const int valid = uniform(item.len - item.a * kPos);  // positions from the first step on
      const auto issue_s = [&](int i, int t, uint32_t k) {
        const uint32_t k_lo = tc::desc_lo(k, 16);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk / 4) * kPos * 128 + (kk % 4) * 32) / 16;
          tc::mma_smem(one, tm + i * kPos, q_lo + i * (C::kTileBytes / 16) + off, hi, k_lo + off, hi,
                       i_s, kk > 0);
        }
        tc::mma_commit(one, bar(s_s[i]));
        if (t == u[i] - 1) tc::mma_commit(one, bar(s_q_free[i]));
      };
      wait(bar(s_full[st]), phase);
      k_before = st;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (u[i] == 0) continue;
        wait(bar(s_q[i]), n_q[i] & 1);
        ++n_q[i];
        if (C::kBeside && n_p[i] > 0) {  // the last item's S has been read
          wait(bar(s_x[i]), (n_p[i] - 1) & 1);
          tc::fence_after();
        }
        issue_s(i, 0, stage(st));
      }
      turn();
      wait(bar(s_full[st]), phase);
      for (int t = 0; t < last; ++t) {
        const int v_st = st;
        const uint32_t v = stage(v_st);
        if (valid - t * kPos < kPos) {
          // positions behind the sequence have weight 0, but what their page holds may be NaN
          for (int x = (valid - t * kPos) * 128 + lane * 16; x < kPos * 128; x += 512)
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              asm volatile(
                  "st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(v + h * kPos * 128 + x), "r"(0)
                  : "memory");
          tc::fence_async_proxy();
          __syncwarp();
        }
        const uint32_t v_lo = tc::desc_lo(v, kPos * 128);
        turn();
        const int k_st = st, k_phase = phase;
        if (t + 1 < last) turn();
        const auto next_s = [&](int i) {
          if (t + 1 < u[i]) {
            if (i == 0 || t + 1 >= u[0]) wait(bar(s_full[k_st]), k_phase);
            if (C::kBeside) {
              wait(bar(s_x[i]), n_p[i] & 1);
              tc::fence_after();
            }
            issue_s(i, t + 1, stage(k_st));
          }
        };
        const auto add_pv = [&](int i) {
          if (t < u[i]) {
            wait(bar(s_p[i]), n_p[i] & 1);
            tc::fence_after();
#pragma unroll
            for (int kk = 0; kk < kPos / 16; ++kk)
              tc::mma_tmem(one, tm + 2 * kPos + i * D, tm + p_col(i) + kk * 8, v_lo + kk * 128, hi,
                           i_o, t > 0 || kk > 0);
            if (C::kBeside || t == u[i] - 1) tc::mma_commit(one, bar(s_o[i]));
          }
        };
        // While the tensor cores have work queued, this step's K and the last one's V go back to the
        // ring, and the next V is waited for.
        const auto turn_ring = [&]() {
          tc::mma_commit(one, bar(s_empty[k_before]));
          if (v_before >= 0) tc::mma_commit(one, bar(s_empty[v_before]));
          if (t + 1 < last) wait(bar(s_full[st]), phase);
        };
        if (C::kBeside) {
          next_s(0);
          next_s(1);
          add_pv(0);
          turn_ring();
          add_pv(1);
        } else {
          add_pv(0);
          next_s(0);
          turn_ring();
          add_pv(1);
          next_s(1);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (t < u[i]) ++n_p[i];
        k_before = k_st;
        v_before = v_st;
        gone = __any_sync(0xffffffffu, *static_cast<volatile int *>(&s_gone));
        if (gone) break;
      }
    }
    // The products under way end before TMEM and the shared memory go, whoever gives up and when.
    volatile int never = 0;
    tc::mma_commit(one, bar(s_end));
    tc::bar_wait(bar(s_end), 0, &never);
    __syncwarp();
  } else if (warp < kSoftmaxWarps) {
    // ---------------------------------------------------------------- softmax, one row a thread
    tc::regs_up<kSoftmaxRegs>();
    const int i = warp / 4, r = threadIdx.x & 127;
    const uint32_t recip = (65536u + p.group - 1) / p.group;  // x / group = x recip >> 16, x < 128
    const int r_tok = r * recip >> 16;
    const uint32_t lanes = static_cast<uint32_t>(warp % 4) << 21;  // 32 * (warp % 4) << 16
    const uint32_t ts = tmem + lanes + i * kPos, to = tmem + lanes + 2 * kPos + i * D;
    const uint32_t tp = tmem + lanes + p_col(i);
    int n_s = 0, n_o = 0;  // steps, commits of O so far
    bool ok = true;
    Item item;
    while (ok && take(item)) {
      const int n = i ? item.count[1] : item.count[0], tok_first = item.tok0 + i * w.tokens;
      if (n == 0) {
        if (!item.whole && tok_first < item.nq)  // a piece in which this tile has no part
          w.part_ml[(2 * static_cast<int64_t>(blockIdx.x) + (item.a > 0 ? 0 : 1)) * 256 + i * 128 +
                    r] = make_float2(kNegInf, 0.f);
        continue;
      }
      const int tok = tok_first + r_tok;
      const int limit = item.ctx + tok + 1;  // positions that the row sees
      // a warp without rows only keeps the barriers going
      const int rows = min(w.tokens, item.nq - tok_first) * p.group;
      const bool idle = 32 * (warp % 4) >= rows;
      uint64_t row_mask = 0;  // drafted positions that the row sees
      if (tree && tok < item.nq) row_mask = p.mask[item.row0 + tok] & (~0ull >> (64 - item.nq));
      float m = kNegInf, l = 0.f;
      for (int t = 0; t < n; ++t, ++n_s) {
        ok = tc::bar_wait(bar(s_s[i]), n_s & 1, &s_gone);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc::fence_after();
        if (idle) {
          if (C::kBeside && t > 0) {  // its arrival for P must not count for the step before
            ok = tc::bar_wait(bar(s_o[i]), n_o & 1, &s_gone);
            ++n_o;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
          if (lane == 0) {
            if (C::kBeside) tc::bar_arrive(bar(s_x[i]));
            tc::bar_arrive(bar(s_p[i]));
          }
          continue;
        }
        uint32_t x[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::tmem_load32(x[c], ts + 32 * c);
        tc::wait_load(x[0]);
        tc::loaded(x[1]);
        tc::loaded(x[2]);
        tc::loaded(x[3]);
        if (C::kBeside) {
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::bar_arrive(bar(s_x[i]));
        }
        const int pos0 = (item.a + t) * kPos;
        if (tree) {
          if (pos0 + kPos > item.ctx) {  // drafted positions, and those behind the sequence
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int d = pos0 + 32 * c - item.ctx;  // drafted position of the first column
              uint32_t see = d >= 64 ? 0u : static_cast<uint32_t>(row_mask >> (d & 63));
              if (d < 0)
                see = d <= -32 ? ~0u : static_cast<uint32_t>(row_mask << -d) | ((1u << -d) - 1);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(see >> e & 1)) x[c][e] = __float_as_uint(kNegInf);
            }
          }
        } else if (pos0 + kPos > item.ctx + tok_first + 1) {  // some row does not see all positions
          const int see = limit - pos0;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (32 * c + e >= see) x[c][e] = __float_as_uint(kNegInf);
        }
        // The weights are taken relative to m, which goes by the first step: whatever reference they
        // are taken to divides out.  Only when their sum shows that some row has outgrown m (no
        // weight is larger than the sum) is a new one found, O scaled down, and the work done
        // again; finding the maximum in every step took 450 of 1250 cycles.
        // A row that has seen nothing yet (a later piece of an item, a tree without context) has no m.
        if (t == 0 || (tree && __any_sync(0xffffffffu, m == kNegInf))) {
          const float top = reference<T>(row_max(x), p);
          if (m == kNegInf) m = top;
        }
        const float ref = m == kNegInf ? 0.f : m;
        if (C::kBeside && t > 0) {  // the last step's product has read P and written O
          ok = tc::bar_wait(bar(s_o[i]), n_o & 1, &s_gone);
          ++n_o;
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc::fence_after();
        }
        __syncwarp();  // stores and loads of TMEM want converged warps
        float add = store_weights<T>(x, ref * p.scale_log2, p.scale_log2, tp);
        // Rows behind the sequence's hold what is in memory there, or what an earlier kernel left: they have no
        // say.  (Asked first without them: a flag a row in every step costs 1% with heads of 64.)
        if (__any_sync(0xffffffffu, add > kMostWeight<T>) &&
            __any_sync(0xffffffffu, r < rows && add > kMostWeight<T>)) {
          tc::wait_store();  // P is written again below, and stores to TMEM have no order of their own
          const float up = fmaxf(ref, outgrown<T>(row_max(x).max, p));
          const float f = exp2_approx((ref - up) * p.scale_log2);
          if (m != kNegInf) m = up;
          l *= f;
#pragma unroll 1
          for (int c = 0; t > 0 && c < D / 32; ++c) {
            uint32_t o[32];
            tc::tmem_load32(o, to + 32 * c);
            tc::wait_load(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tc::tmem_store32(to + 32 * c, o);
          }
          add = store_weights<T>(x, up * p.scale_log2, p.scale_log2, tp);
        }
        l += add;
        tc::wait_store();  // P is for the tensor cores
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(bar(s_p[i]));
      }
      if (!ok) break;
      ok = tc::bar_wait(bar(s_o[i]), n_o & 1, &s_gone);
      ++n_o;
      ok = __all_sync(0xffffffffu, ok && !s_gone);
      if (!ok) break;
      if (idle) continue;
      tc::fence_after();
      // The next item's first P V overwrites O only after this warp has handed over that P.
      // Short loops: this code runs once an item, and fetching a long stretch of it took longer than
      // running it (16 packed prompts of 1024 tokens 88 us unrolled, 76 so).
      const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (item.a > 0 ? 0 : 1);
      if (!item.whole) {
        float4 *part = reinterpret_cast<float4 *>(w.part) + (slot * 2 + i) * (D / 4) * 128 + r;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          __syncwarp();
          tc::tmem_load32(o, to + 32 * c);
          tc::wait_load(o);
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            if (r < rows)
              part[(8 * c + e / 4) * 128] =
                  make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                              __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
        }
      } else {
        // 32 columns at a time, four lanes exchange 16-byte chunks so that each then has one chunk of
        // four rows, and together they write 64 bytes of a row: a lane writing its own row touches 32
        // lines an instruction.
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const uint64_t inv2 = pair(inv, inv);
        T *dst[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int rr = 32 * (warp % 4) + (lane & 28) + j, rt = rr * recip >> 16;
          dst[j] = rr < rows ? static_cast<T *>(p.out) + (item.row0 + tok_first + rt) * p.o_row +
                                   (item.kvh * p.group + rr - rt * p.group) * p.o_head +
                                   8 * (lane & 3)
                             : nullptr;
        }
#pragma unroll 2
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32], v[4][4];
          __syncwarp();
          tc::tmem_load32(o, to + 32 * c);
          tc::wait_load(o);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 f = unpair(
                mul2(pair(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])), inv2));
            v[e / 4][e % 4] = Half<T>::pack(f.x, f.y);
          }
#pragma unroll
          for (int k = 1; k < 4; k <<= 1) {
            const bool upper = (lane & k) != 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (!(j & k))
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint32_t got =
                      __shfl_xor_sync(0xffffffffu, upper ? v[j][e] : v[j | k][e], k);
                  if (upper) v[j][e] = got; else v[j | k][e] = got;
                }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (dst[j])
              *reinterpret_cast<uint4 *>(dst[j] + 32 * c) =
                  make_uint4(v[j][0], v[j][1], v[j][2], v[j][3]);
        }
      }
      if (!item.whole && r < rows) w.part_ml[slot * 256 + i * 128 + r] = make_float2(m, l);
    }
  }
  tc::fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && s_gone && p.err) atomicOr(p.err, kDevErrTimeout);
  if (warp == kSoftmaxWarps) {
    tc::fence_after();
    tc::tmem_free(tmem, C::kColumns);
  }
}

// Joins the parts of the item that begins in CTA blockIdx.x and ends in a later one: a thread takes
// eight columns of a row.  The parts are added in the order of the positions.  The list of parts
// is found first, 32 CTAs at a time, so that the loads of one part do not wait for another's.
constexpr int kMaxCtas = 512;

template <typename T, int D>
__global__ void __launch_bounds__(256) prompt_join_kernel(const Params p, int tokens,
                                                          const float *part, const float2 *part_ml,
                                                          const Share *share, int ctas) {
  __shared__ int s_slot[kMaxCtas], s_count;
  pdl_wait();
  const Share sh = share[blockIdx.x];
  if (!sh.tail) return;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int n = 1;
    if (lane == 0) s_slot[0] = 2 * blockIdx.x + 1;
    for (int c0 = blockIdx.x + 1; c0 < ctas; c0 += 32) {
      const int c = c0 + lane;
      int head = 0, ends = 0;
      if (c < ctas) head = share[c].head, ends = head && share[c].head_ends;
      const uint32_t stop = __ballot_sync(0xffffffffu, ends);
      uint32_t parts = __ballot_sync(0xffffffffu, head);  // without: a CTA that had no work
      if (stop) parts &= 0xffffffffu >> (32 - __ffs(stop));
      if (parts >> lane & 1) s_slot[n + __popc(parts & ((1u << lane) - 1))] = 2 * c;
      n += __popc(parts);
      if (stop) break;
    }
    if (lane == 0) s_count = n;
  }
  __syncthreads();
  const int n = s_count;
  const int i = threadIdx.x >> 7, r = threadIdx.x & 127;
  const int r_tok = r / p.group, tok = sh.tok0 + i * tokens + r_tok;
  if (r >= tokens * p.group || tok >= sh.nq) return;
  const float2 *ml = part_ml + threadIdx.x;
  float m = kNegInf;
#pragma unroll 4
  for (int c = 0; c < n; ++c) m = fmaxf(m, ml[s_slot[c] * 256].x);
  const float4 *src = reinterpret_cast<const float4 *>(part) + (i * (D / 4) + 2 * blockIdx.y) * 128 + r;
  float l = 0.f, o[8] = {};
#pragma unroll 4
  for (int c = 0; c < n; ++c) {
    const float2 v = ml[s_slot[c] * 256];
    const float4 *q = src + static_cast<int64_t>(s_slot[c]) * 2 * (D / 4) * 128;
    const float4 a = q[0], b = q[128];
    if (!(v.y == 0.f)) {  // a part without weight may not have been written; a sum that is NaN counts
      const float g = exp2_approx((v.x - m) * p.scale_log2);
      l = fmaf(v.y, g, l);
      o[0] = fmaf(a.x, g, o[0]), o[1] = fmaf(a.y, g, o[1]);
      o[2] = fmaf(a.z, g, o[2]), o[3] = fmaf(a.w, g, o[3]);
      o[4] = fmaf(b.x, g, o[4]), o[5] = fmaf(b.y, g, o[5]);
      o[6] = fmaf(b.z, g, o[6]), o[7] = fmaf(b.w, g, o[7]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint4 v;
  v.x = Half<T>::pack(o[0] * inv, o[1] * inv);
  v.y = Half<T>::pack(o[2] * inv, o[3] * inv);
  v.z = Half<T>::pack(o[4] * inv, o[5] * inv);
  v.w = Half<T>::pack(o[6] * inv, o[7] * inv);
  *reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + (sh.row0 + tok) * p.o_row +
                             (sh.kvh * p.group + r - r_tok * p.group) * p.o_head +
                             8 * blockIdx.y) = v;
}

struct PromptPlan {
  int grid;
  int64_t ml, share, bytes;  // offsets in the workspace
};

static int make_plan(const moe_kv_cache *c, const Params &p, PromptPlan *plan) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MOE_ERR_CUDA;
  plan->grid = sms < kMaxCtas ? sms : kMaxCtas;
  plan->ml = plan->share = plan->bytes = 0;
  const int64_t len = static_cast<int64_t>(p.table_width) << p.page_shift;  // of a sequence at most
  // the line's length times the CTAs stays inside 64 bits
  const double items = static_cast<double>(p.n_rows) / (2 * (128 / p.group)) + p.n_seqs;
  if (items * (static_cast<double>(len) + kItemCost) * p.hkv * sms > 4e18) return MOE_ERR_UNSUPPORTED;
  if ((len + kPos - 1) / kPos < kShareSteps) return MOE_OK;
  plan->ml = 4ll * 2 * plan->grid * 256 * c->head_dim;
  plan->share = plan->ml + 8ll * 2 * plan->grid * 256;
  plan->bytes = plan->share + static_cast<int64_t>(sizeof(Share)) * plan->grid;
  return MOE_OK;
}

template <typename T, int D, bool TREE>
static int launch(const moe_kv_cache *c, const Params &p, const PromptPlan &plan, uint8_t *ws,
                  cudaStream_t stream) {
  PromptParams w;
  w.p = p;
  w.tokens = 128 / p.group;
  w.part = reinterpret_cast<float *>(ws);
  w.part_ml = reinterpret_cast<float2 *>(ws + plan.ml);
  w.share = plan.bytes ? reinterpret_cast<Share *>(ws + plan.share) : nullptr;
  if (const int64_t cycles = debug_wait_cycles.load(std::memory_order_relaxed))
    w.limit.cycles = cycles, w.limit.nap_ns = 0;
  const bool bf16 = c->dtype == MOE_DTYPE_BF16;
  const uint64_t q_dims[3] = {D, static_cast<uint64_t>(p.hq), static_cast<uint64_t>(p.n_rows)};
  const int64_t q_str[2] = {p.q_head, p.q_row};
  const uint32_t q_box[3] = {64, static_cast<uint32_t>(p.group), static_cast<uint32_t>(w.tokens)};
  const uint64_t dims[4] = {D, static_cast<uint64_t>(c->page_size), static_cast<uint64_t>(p.hkv),
                            static_cast<uint64_t>(p.n_pages)};
  const int64_t str[3] = {p.tok_stride, p.head_stride, p.page_stride};
  const uint32_t box[4] = {64, static_cast<uint32_t>(c->page_size < kPos ? c->page_size : kPos), 1, 1};
  if (!tc::make_map(&w.q, bf16, p.q, 3, q_dims, q_str, q_box) ||
      !tc::make_map(&w.k, bf16, p.k, 4, dims, str, box) ||
      !tc::make_map(&w.v, bf16, p.v, 4, dims, str, box))
    return MOE_ERR_UNSUPPORTED;
  const auto kern = prompt_kernel<T, D, TREE>;
  static SmemLimit limit;
  cudaError_t e = limit.set(reinterpret_cast<const void *>(kern), Prompt<D>::kSmem);
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  kern<<<plan.grid, kPromptThreads, Prompt<D>::kSmem, stream>>>(w);
  if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
  if (!plan.bytes) return MOE_OK;
  // the joining blocks are set up while the kernel runs and wait for its end
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(plan.grid, D / 8);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, prompt_join_kernel<T, D>, p, w.tokens,
                         static_cast<const float *>(w.part),
                         static_cast<const float2 *>(w.part_ml),
                         static_cast<const Share *>(w.share), plan.grid);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// The kernel for causal (TREE false) or masked (TREE true) attention of one cache type.
template <bool TREE>
static int run(const moe_kv_cache *cache, const Params &p, void *workspace, int64_t workspace_bytes,
               cudaStream_t stream) {
  PromptPlan plan;
  const int rc = make_plan(cache, p, &plan);
  if (rc != MOE_OK) return rc;
  if (plan.bytes && (!workspace || workspace_bytes < plan.bytes)) return MOE_ERR_INVALID_ARG;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  if (cache->dtype == MOE_DTYPE_BF16)
    return cache->head_dim == 64 ? launch<__nv_bfloat16, 64, TREE>(cache, p, plan, ws, stream)
                                 : launch<__nv_bfloat16, 128, TREE>(cache, p, plan, ws, stream);
  return cache->head_dim == 64 ? launch<__half, 64, TREE>(cache, p, plan, ws, stream)
                               : launch<__half, 128, TREE>(cache, p, plan, ws, stream);
}

}  // namespace attn
