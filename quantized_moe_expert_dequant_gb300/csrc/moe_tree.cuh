// moe_tree.cuh -- attention of decoded tokens, or of trees of drafted tokens, over the pages of a
// cache (moe_tree_attention; instantiated by moe_tree.cu and moe_tree_cluster.cu), over pages that are listed
// for each row (moe_sparse.cu, moe_sparse_cluster.cu), and with a group's first pages (moe_prefix_tree.cu).
//
//   out_r = sum_j p_rj v_j / sum_j p_rj,   p_rj = exp(scale * q_r . k_j - m_r)  over the positions j
//   that row r sees, m_r their largest score: one pass over K and V with the running maximum and
//   sum; what was summed before a larger maximum is scaled down to it.  (fp16: all p times 2^15.)
//
// Bound by the bytes of K and V, so what matters is that every SM streams all the time, whatever
// the lengths are.  An item is one sequence and one key/value head, with the queries of all heads
// that share it as rows (row R is query R / group, head R % group; more than 32 rows go to the tiles
// of moe_tiles.cuh); its positions are cut into tiles of 64, of 128 with heads of 64 (tile_of).  All tiles of
// all items, in order, form one
// line that the CTAs share evenly: CTA c takes the tiles [c W / G, (c + 1) W / G).  The lengths are
// read on the device, so a captured graph balances whatever it is replayed on.  An item that ends up in
// one CTA is written by it; one that several CTAs share leaves its partial maxima, sums and outputs
// in the workspace, and join_kernel adds them in order.
//
// With few items that plan and the second kernel are most of the time; there a cluster of 16 or 8 CTAs
// takes each item and joins in distributed shared memory.
//
// A CTA is four warps over 16 WR rows: WR warps split the rows, 4 / WR warps the positions of a
// tile, so a single decoded token (group <= 16 rows) still uses all four.  Copies run two
// tiles ahead and across items, so that one item's end does not empty the pipeline of the next:
// 32 tokens over contexts of 1 to 15991 positions (741 MB) 132 us with a pipeline per item, 125 us
// so (5.8 to 5.9 TB/s); 8 drafts behind 65536 to 131064 positions (1.75 GB) 264 us (6.6 TB/s).
#pragma once

#include <algorithm>
#include <type_traits>

#include "moe_attention.cuh"

namespace attn {

constexpr int kThreads = 128;
constexpr int kSlice = 40;  // 32 output columns of a row on their way between warps, padded

// positions of a tile: 32 KB of K and V each way; with 64 for heads of 64 too, what a tile costs besides
// its copies showed (64 sequences, 16 heads of 64: 148 us, 136 with 128)
constexpr int tile_of(int dim) { return dim == 64 ? 128 : 64; }

template <int D>
struct Tree {
  static constexpr int kTile = tile_of(D);
  // 32 KB a stage; with two CTAs an SM there are 128 KB in flight, more than the 35 KB that latency
  // times bandwidth asks for
  static constexpr int kStages = 3;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kRing = kStages * 2 * kTileBytes;
  static constexpr int kSmem = kRing + 4 * 16 * kSlice * 4;
};
constexpr int kCtasPerSm = 2;
constexpr int kMinPositions = 128, kMaxLeast = 256;  // bounds of the positions that a CTA takes at least

// What one CTA leaves for join_kernel: the item that begins in it and goes on in the next ones.
struct Shared {
  int pieces;  // CTAs that hold a part; 0: nothing to join
  int row0;    // the sequence's first row
  int kvh, rows;
  int slot;    // 0 or 1: which of its CTA's parts is its first
};

struct Work {
  Params p;
  float *part;      // [2 G][ROWS][D] partial outputs: slot 2c the CTA's first item, 2c + 1 its last
  float2 *part_ml;  // [2 G][ROWS] (maximum, sum)
  Shared *shared;   // [G]
  const int32_t *list;  // kListed: [n_rows][hkv][n_list] pages of each row, of its table
  int n_list;
  Prefixes g;           // kGrouped
};

// What an item is: a sequence, a row and its list of pages (moe_sparse_attention), or a sequence whose first
// pages are those of its group's first one (moe_prefix_attention).
enum Items { kSeqs, kListed, kGrouped };

// All threads of the cluster's CTAs.  The aligned form wants converged warps, and the code before it may have
// split them (half a warp of a tile's rows, the last of a loop).
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// Shared memory of the cluster's CTA `rank` at this CTA's address.
__device__ __forceinline__ float4 peer_float4(uint32_t addr, int rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}
__device__ __forceinline__ float2 peer_float2(uint32_t addr, int rank) {
  float2 v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %2, %3;\n\t"
      "ld.shared::cluster.v2.f32 {%0, %1}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}

template <int D>
__device__ __forceinline__ uint32_t swizzled(int row, int chunk) {  // byte offset in a [rows][D] tile
  return static_cast<uint32_t>(row * D * 2 + ((chunk ^ (row & 7)) << 4));
}

// The pages of each 16 positions of a tile (a page has at least 16); -1: nothing there.
template <int TILE>
__device__ __forceinline__ void load_pages(const Params &p, const int32_t *pages, int len, int tile,
                                           int (&pg)[TILE / 16]) {
#pragma unroll
  for (int e = 0; e < TILE / 16; ++e) {
    const int pos = tile * TILE + 16 * e;
    pg[e] = pos < len ? pages[pos >> p.page_shift] : -1;
  }
}

// The same where the first `shared` positions are on other pages than the sequence's own.
template <int TILE>
__device__ __forceinline__ void load_pages(const Params &p, const int32_t *first, int shared,
                                           const int32_t *own, int len, int tile, int (&pg)[TILE / 16]) {
#pragma unroll
  for (int e = 0; e < TILE / 16; ++e) {
    const int pos = tile * TILE + 16 * e;
    pg[e] = pos < len ? (pos < shared ? first : own)[pos >> p.page_shift] : -1;
  }
}

// Copies the positions of tile t of K and V into shared memory; rows past the sequence and on
// a page outside the cache are zeros (what stale pages hold, NaN included, is never multiplied).
template <typename T, int D, int TILE>
__device__ __forceinline__ void load_tile(const Params &p, int len, const int (&pg)[TILE / 16],
                                          int64_t head_off, int tile, uint32_t k_smem,
                                          uint32_t v_smem) {
  constexpr int kChunks = D / 8, kStep = kThreads / kChunks;
  const int c = threadIdx.x % kChunks, r0 = threadIdx.x / kChunks;
#pragma unroll
  for (int i = 0; i < TILE / kStep; ++i) {
    const int r = r0 + i * kStep, pos = tile * TILE + r;
    const int page = pg[i * kStep / 16];
    const bool valid = pos < len && static_cast<unsigned>(page) < static_cast<unsigned>(p.n_pages);
    const int64_t off = valid ? page * p.page_stride + head_off +
                                    (pos & ((1 << p.page_shift) - 1)) * p.tok_stride + 8 * c
                              : 0;
    const uint32_t d = swizzled<D>(r, c);
    cp_async16(k_smem + d, static_cast<const T *>(p.k) + off, valid);
    cp_async16(v_smem + d, static_cast<const T *>(p.v) + off, valid);
  }
#pragma unroll
  for (int e = 0; e < TILE / 16; ++e)  // a used page outside the cache is reported
    if (threadIdx.x == e && tile * TILE + 16 * e < len &&
        static_cast<unsigned>(pg[e]) >= static_cast<unsigned>(p.n_pages) && p.err)
      atomicOr(p.err, kDevErrBadId);
}

// Listed pages.  Each warp copies every fourth run of 16 positions of a tile, so that a thread looks up one
// or two pages a tile and steps through their positions.  (All threads looking up all pages of a tile: a chunk of
// 512 rows over 100 pages of 16, heads of 64, 108 us; 62 so.)
template <int TILE>
struct Listed {
  static constexpr int kRuns = TILE / 64;  // of a warp
  int at[kRuns];    // the next tile's entries of the list
  int page[kRuns];  // the pages that they name
  int see[kRuns];   // how many of the 16 positions are seen (the others are not read)
};

template <int TILE>
__device__ __forceinline__ void load_entries(const Params &p, const int32_t *list, int len, int tile,
                                             Listed<TILE> &l) {
#pragma unroll
  for (int e = 0; e < Listed<TILE>::kRuns; ++e) {
    const int pos = tile * TILE + 16 * ((threadIdx.x >> 5) + 4 * e);
    l.at[e] = pos < len ? list[pos >> p.page_shift] : -1;
  }
}

template <int TILE>
__device__ __forceinline__ void load_listed(const Params &p, int seq, int limit, int tile,
                                            Listed<TILE> &l) {
#pragma unroll
  for (int e = 0; e < Listed<TILE>::kRuns; ++e) {
    const int pos = tile * TILE + 16 * ((threadIdx.x >> 5) + 4 * e), at = l.at[e];
    const bool seen = at >= 0 && at <= (limit - 1) >> p.page_shift;
    l.page[e] = seen ? p.table[seq * p.table_stride + at] : -1;
    const int left = limit - (at << p.page_shift) - (pos & ((1 << p.page_shift) - 1));
    l.see[e] = seen ? max(0, min(left, 16)) : 0;
  }
}

template <typename T, int D, int TILE>
__device__ __forceinline__ void load_listed_tile(const Params &p, const Listed<TILE> &l,
                                                 int64_t head_off, int tile, uint32_t k_smem,
                                                 uint32_t v_smem, int *s_see) {
  constexpr int kChunks = D / 8, kStep = 32 / kChunks;
  const int c = threadIdx.x % kChunks, r0 = (threadIdx.x & 31) / kChunks, warp = threadIdx.x >> 5;
#pragma unroll
  for (int e = 0; e < Listed<TILE>::kRuns; ++e) {
    const int run = warp + 4 * e, page = l.page[e];
    const bool there = static_cast<unsigned>(page) < static_cast<unsigned>(p.n_pages);
    const int see = there ? l.see[e] : 0;
    const int in_page = (tile * TILE + 16 * run) & ((1 << p.page_shift) - 1);
    const int64_t off = there ? page * p.page_stride + head_off + (in_page + r0) * p.tok_stride + 8 * c : 0;
    const T *k = static_cast<const T *>(p.k) + off, *v = static_cast<const T *>(p.v) + off;
    const int64_t step = there ? kStep * p.tok_stride : 0;
#pragma unroll
    for (int i = 0; i < 16 / kStep; ++i) {
      const int r = r0 + i * kStep;
      const uint32_t d = swizzled<D>(16 * run + r, c);
      cp_async16(k_smem + d, k, r < see);
      cp_async16(v_smem + d, v, r < see);
      k += step, v += step;
    }
    if ((threadIdx.x & 31) == 0) {
      s_see[run] = see;
      if (!there && l.see[e] > 0 && p.err) atomicOr(p.err, kDevErrBadId);
    }
  }
}

// Sums v over the block (every thread gets the sum) and gives each thread the sum before it.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *s_warp, int64_t *before) {
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
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) base += s_warp[w];
    all += s_warp[w];
  }
  *before = base + x - v;
  return all;
}

// CS > 0: a cluster of CS CTAs takes an item, each an even part of its tiles, and joins the parts in
// distributed shared memory.
template <typename T, int D, int WR, int CS, int ITEMS>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) tree_kernel(const Work w) {
  constexpr bool SPARSE = ITEMS == kListed;
  constexpr int kTile = Tree<D>::kTile;
  constexpr int ROWS = 16 * WR, WT = 4 / WR, TW = kTile / WT;  // TW positions of a warp per tile
  constexpr int kStages = Tree<D>::kStages, kTileBytes = Tree<D>::kTileBytes;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[4][16], s_l[4][16];
  __shared__ int64_t s_warp[4], s_before;
  __shared__ int s_seq;
  __shared__ float2 s_part_ml[ROWS];
  __shared__ int s_see[SPARSE ? kStages : 1][kTile / 16];
  using Item = std::conditional_t<SPARSE, Row, Seq>;
  const Params &p = w.p;
  const int n_items = SPARSE ? p.n_rows : p.n_seqs;  // a key/value head
  const auto load = [&](int i, bool report) -> Item {
    if constexpr (SPARSE)
      return load_row(p, i, w.n_list);
    else
      return load_seq(p, i, report);
  };
  if constexpr (ITEMS != kSeqs) {
    pdl_wait();
    if (CS > 0) pdl_launch();
  }
  if constexpr (ITEMS == kGrouped) {
    if (blockIdx.x == 0)
      for (int i = threadIdx.x; i < w.g.n_groups; i += kThreads) load_group(p, w.g, i, true);
  }
  if constexpr (SPARSE) {
    if (blockIdx.x == 0)
      for (int i = threadIdx.x; i < p.n_seqs; i += kThreads) load_seq(p, i, true);
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q4 = lane & 3;
  const int wr = warp % WR, wt = warp / WR;

  int64_t at, end, total = 0, ctas = 0;
  if constexpr (CS > 0) {
    const int item = blockIdx.x / CS, rank = blockIdx.x % CS;
    const int sq = item / p.hkv, head = item - sq * p.hkv;
    const Item q = load(sq, rank == 0 && head == 0 && threadIdx.x == 0);
    if (q.nq == 0) return;  // the whole cluster
    const int nt = (q.len + kTile - 1) / kTile;
    // tiles count from the beginning of the sequence's line, as below
    at = static_cast<int64_t>(head) * nt + static_cast<int64_t>(rank) * nt / CS;
    end = static_cast<int64_t>(head) * nt + static_cast<int64_t>(rank + 1) * nt / CS;
    if (threadIdx.x == 0) s_seq = sq, s_before = 0;
  } else {
    pdl_launch();
    // all tiles, and the sequence in which this CTA's part of them begins
    const auto weight = [&](const Item &s) {
      return s.nq ? static_cast<int64_t>(p.hkv) * ((s.len + kTile - 1) / kTile) : 0;
    };
    const bool first_cta = blockIdx.x == 0;
    int64_t before, mine = 0;
    for (int b = 0; b < n_items; b += kThreads) {
      const int i = b + threadIdx.x;
      mine = i < n_items ? weight(load(i, first_cta)) : 0;
      total += block_scan(mine, s_warp, &before);
    }
    // A CTA's time grows with its tiles, that of join_kernel with an item's parts: with n tiles an item the
    // shortest is near sqrt(n) / 2 tiles a CTA.  (One token, positions: us with 2, 4, 8 tiles of 64 at
    // least.  500: 7.8, 9.6, 12.9; 4000: 16.2, 14.4, 15.2; 16384: 21.6, 21.5, 22.9.)
    const float per_item = static_cast<float>(total) / (static_cast<float>(n_items) * p.hkv);
    const int least = min(kMaxLeast / kTile, max(kMinPositions / kTile,
                                                 static_cast<int>(0.5f * sqrtf(per_item) + 0.5f)));
    ctas = min(static_cast<int64_t>(gridDim.x), (total + least - 1) / least);
    if (threadIdx.x == 0) w.shared[blockIdx.x].pieces = 0;
    if (blockIdx.x >= ctas) return;
    at = blockIdx.x * total / ctas;
    end = (blockIdx.x + 1) * total / ctas;
    if (n_items <= kThreads) {
      if (before <= at && at < before + mine) s_seq = threadIdx.x, s_before = before;
    } else {
      int64_t sum = 0;
      for (int b = 0; sum <= at; b += kThreads) {
        const int i = b + threadIdx.x;
        mine = i < n_items ? weight(load(i, false)) : 0;
        const int64_t all = block_scan(mine, s_warp, &before);
        before += sum;
        if (before <= at && at < before + mine) s_seq = i, s_before = before;
        sum += all;
      }
    }
  }
  __syncthreads();
  const int64_t begin = at;
  const uint32_t base = smem_u32(smem);

  // What is copied next: tile `t` of head `kvh` of sequence `seq`; the tile that is computed is
  // kStages - 1 behind.  Tile number k of the CTA waits in stage k % kStages; its pages are read one
  // tile ahead, and a sequence's description one sequence ahead.
  struct Ahead {
    const int32_t *pages;
    int64_t head_off;
    int left, seq, kvh, t, nt, len, stage, pg[kTile / 16];
    Item next;
    int limit, table;  // listed pages: pages is the list, of pages of sequence `table`
    Listed<kTile> list;
    bool ready;        // the next tile's entries have been read
    const int32_t *first;  // grouped: the pages of positions before `limit`
  } ld;
  const auto look_up_group = [&](int ctx) {
    int index;
    const Group group = group_of(p, w.g, ld.seq, &index);
    ld.limit = shared_by(group, ctx);
    ld.first = ld.limit ? p.table + group.begin * p.table_stride : ld.pages;
  };
  const auto look_up = [&]() {
    if constexpr (SPARSE) {
      if (!ld.ready) load_entries<kTile>(p, ld.pages, ld.len, ld.t, ld.list);
      load_listed<kTile>(p, ld.table, ld.limit, ld.t, ld.list);
      ld.ready = ld.t + 1 < ld.nt;
      if (ld.ready) load_entries<kTile>(p, ld.pages, ld.len, ld.t + 1, ld.list);
    } else if constexpr (ITEMS == kGrouped) {
      load_pages<kTile>(p, ld.first, ld.limit, ld.pages, ld.len, ld.t, ld.pg);
    } else {
      load_pages<kTile>(p, ld.pages, ld.len, ld.t, ld.pg);
    }
  };
  {
    const int64_t in_seq = at - s_before;
    const Item q = load(s_seq, false);
    ld.left = static_cast<int>(end - at);
    ld.seq = s_seq, ld.len = q.len, ld.nt = (q.len + kTile - 1) / kTile;
    ld.kvh = static_cast<int>(in_seq / ld.nt);
    ld.t = static_cast<int>(in_seq - static_cast<int64_t>(ld.kvh) * ld.nt);
    ld.stage = 0;
    if constexpr (SPARSE) {
      ld.pages = w.list + (static_cast<int64_t>(ld.seq) * p.hkv + ld.kvh) * w.n_list;
      ld.limit = q.ctx, ld.table = q.seq, ld.ready = false;
    } else {
      ld.pages = p.table + ld.seq * p.table_stride;
    }
    if constexpr (ITEMS == kGrouped) look_up_group(q.ctx);
    ld.head_off = ld.kvh * p.head_stride;
    look_up();
    ld.next = load(min(ld.seq + 1, n_items - 1), false);
  }
  const auto next_item = [&]() {
    ld.t = 0;
    ld.head_off += p.head_stride;
    if (SPARSE) ld.pages += w.n_list;
    if (++ld.kvh < p.hkv) return;
    ld.kvh = 0;
    ld.head_off = 0;
    bool empty = true;  // sequences without rows have no tiles
    int ctx = 0;
    while (empty && ++ld.seq < n_items) {
      ctx = ld.next.ctx;
      ld.len = ld.next.len, ld.nt = (ld.len + kTile - 1) / kTile;
      empty = ld.next.nq == 0;
      if constexpr (SPARSE) ld.limit = ld.next.ctx, ld.table = ld.next.seq;
      ld.next = load(min(ld.seq + 1, n_items - 1), false);
    }
    if (empty) ld.left = 0;
    if constexpr (SPARSE)
      ld.pages = w.list + static_cast<int64_t>(ld.seq) * p.hkv * w.n_list;
    else
      ld.pages = p.table + ld.seq * p.table_stride;
    if constexpr (ITEMS == kGrouped)
      if (!empty) look_up_group(ctx);
  };
  const auto copy_next = [&]() {
    if (ld.left > 0) {
      const uint32_t st = base + ld.stage * 2 * kTileBytes;
      if constexpr (SPARSE)
        load_listed_tile<T, D, kTile>(p, ld.list, ld.head_off, ld.t, st, st + kTileBytes,
                                      s_see[ld.stage]);
      else
        load_tile<T, D, kTile>(p, ld.len, ld.pg, ld.head_off, ld.t, st, st + kTileBytes);
      if (++ld.stage == kStages) ld.stage = 0;
      --ld.left;
      if (++ld.t == ld.nt) next_item();
      if (ld.left > 0) look_up();
    }
    cp_async_commit();
  };

  int seq = ld.seq, kvh = ld.kvh, t0 = ld.t, stage = 0;
  Item s = load(seq, false);
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) copy_next();
  while (at < end) {
    const int nt = (s.len + kTile - 1) / kTile, rows = s.nq * p.group;
    const int64_t item_at = at - t0;
    const int t1 = static_cast<int>(min(static_cast<int64_t>(nt), t0 + (end - at)));
    // this lane's two rows: queries, heads, masks
    int row_q[2];
    uint64_t row_mask[2];
    bool row_ok[2];
    const uint32_t *qp[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int R = wr * 16 + g + 8 * h;
      row_ok[h] = R < rows;
      row_q[h] = row_ok[h] ? R / p.group : 0;
      const int head = kvh * p.group + (row_ok[h] ? R - row_q[h] * p.group : 0);
      qp[h] = reinterpret_cast<const uint32_t *>(static_cast<const T *>(p.q) +
                                                 (s.row0 + row_q[h]) * p.q_row + head * p.q_head);
      // without masks: bits 0 .. query
      if (SPARSE) continue;
      row_mask[h] = p.mask ? p.mask[s.row0 + row_q[h]] : ~0ull >> (63 - row_q[h]);
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

    for (int t = t0; t < t1; ++t) {
      cp_async_wait<kStages - 2>();
      __syncthreads();  // tile t is there, and every warp is done with the tile before
      const uint32_t ks = base + stage * 2 * kTileBytes, vs = ks + kTileBytes;
      int see[TW / 16];
      if constexpr (SPARSE) {
#pragma unroll
        for (int j = 0; j < TW / 16; ++j) see[j] = s_see[stage][wt * (TW / 16) + j];
      }
      if (++stage == kStages) stage = 0;

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
      copy_next();
      if constexpr (SPARSE) {
#pragma unroll
        for (int j = 0; j < TW / 8; ++j)
          if (see[j / 2] < 16)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (8 * (j & 1) + 2 * q4 + (e & 1) >= see[j / 2]) sc[j][e] = kNegInf;
      } else if ((t + 1) * kTile > s.ctx) {  // drafted positions, and those behind the sequence
        const int pos0 = t * kTile + wt * TW + 2 * q4;
#pragma unroll
        for (int j = 0; j < TW / 8; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int d = pos0 + 8 * j + (e & 1) - s.ctx;
            if (d >= 0 && (d >= s.nq || !((row_mask[e >> 1] >> d) & 1))) sc[j][e] = kNegInf;
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
        const float off = ref * p.scale_log2 - Half<T>::kRow;
        float add = 0.f;
#pragma unroll
        for (int j = 0; j < TW / 8; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x = exp2_approx(fmaf(sc[j][2 * h + e], p.scale_log2, -off));
            sc[j][2 * h + e] = x;
            add += x;
          }
        l[h] = l[h] * scale[h] + add;
      }
      if (__any_sync(0xffffffffu, scale[0] != 1.f || scale[1] != 1.f)) {
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          o[j][0] *= scale[0], o[j][1] *= scale[0];
          o[j][2] *= scale[1], o[j][3] *= scale[1];
        }
      }
#pragma unroll
      for (int j = 0; j < TW / 16; ++j) {
        // p enters the product in the cache's type (as v is)
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
    }

    // join the warps that split the positions, 32 columns at a time, and the rows' sums over their
    // four lanes
    float *s_o = reinterpret_cast<float *>(smem + Tree<D>::kRing);  // [4][16][kSlice]
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if (q4 == 0) s_m[warp][g + 8 * h] = m[h], s_l[warp][g + 8 * h] = l[h];
    }
    const bool whole = t0 == 0 && t1 == nt;
    const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (at == begin ? 0 : 1);
    if (CS == 0 && threadIdx.x == 0 && t0 == 0 && t1 < nt) {
      Shared &r = w.shared[blockIdx.x];
      r.pieces = static_cast<int>(((item_at + nt) * ctas - 1) / total) - blockIdx.x + 1;
      r.row0 = s.row0, r.kvh = kvh, r.rows = rows, r.slot = at == begin ? 0 : 1;
    }
    const int r = threadIdx.x / 4, c8 = threadIdx.x % 4;  // eight columns of a row, ROWS * 4 threads
#pragma unroll
    for (int slice = 0; slice < D / 32; ++slice) {
      if (slice > 0) __syncthreads();  // the last slice has been read
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<float2 *>(s_o + (warp * 16 + g + 8 * h) * kSlice + 8 * j + 2 * q4) =
              make_float2(o[4 * slice + j][2 * h], o[4 * slice + j][2 * h + 1]);
      __syncthreads();
      if (r < ROWS && r < rows) {
        float top = kNegInf;
#pragma unroll
        for (int v = 0; v < WT; ++v) top = fmaxf(top, s_m[v * WR + r / 16][r % 16]);
        const float ref = top == kNegInf ? 0.f : top;
        float total_l = 0.f, x[8] = {};
#pragma unroll
        for (int v = 0; v < WT; ++v) {
          const int ww = v * WR + r / 16;
          const float f = exp2_approx((s_m[ww][r % 16] - ref) * p.scale_log2);
          total_l += f * s_l[ww][r % 16];
          const float *src = s_o + (ww * 16 + r % 16) * kSlice + 8 * c8;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = fmaf(f, src[e], x[e]);
        }
        const int col = 32 * slice + 8 * c8;
        if (CS == 0 && whole) {
          const float inv = total_l > 0.f ? 1.f / total_l : 0.f;  // a row that sees nothing is zeros
          const int tok = r / p.group, head = kvh * p.group + r - tok * p.group;
          uint4 v;
          v.x = Half<T>::pack(x[0] * inv, x[1] * inv);
          v.y = Half<T>::pack(x[2] * inv, x[3] * inv);
          v.z = Half<T>::pack(x[4] * inv, x[5] * inv);
          v.w = Half<T>::pack(x[6] * inv, x[7] * inv);
          *reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + (s.row0 + tok) * p.o_row +
                                     head * p.o_head + col) = v;
        } else {
          // (of a cluster, the part goes where the ring was: every tile has been read)
          float *part = CS > 0 ? reinterpret_cast<float *>(smem) + r * D
                               : w.part + (slot * ROWS + r) * D;
          float4 *dst = reinterpret_cast<float4 *>(part + col);
          dst[0] = make_float4(x[0], x[1], x[2], x[3]);
          dst[1] = make_float4(x[4], x[5], x[6], x[7]);
          if (col == 0) {
            float2 *ml = CS > 0 ? s_part_ml + r : w.part_ml + slot * ROWS + r;
            *ml = make_float2(top, total_l);
          }
        }
      }
    }
    __syncthreads();  // s_o, s_m and s_l are free again
    at = item_at + t1;
    t0 = 0;
    if (t1 == nt && ++kvh == p.hkv) {
      kvh = 0;
      do {
        if (CS > 0) break;
        if (++seq >= n_items) return;  // the end of the line
        s = load(seq, false);
      } while (s.nq == 0);
    }
  }

  if constexpr (CS > 0) {
    const int rank = blockIdx.x % CS, rows = s.nq * p.group;
    if (begin == end && threadIdx.x < ROWS) s_part_ml[threadIdx.x] = make_float2(kNegInf, 0.f);
    cluster_sync();
    // eight columns of a row a thread, over all threads of the cluster; parts in the positions' order
    for (int u = rank * kThreads + threadIdx.x; u < ROWS * D / 8; u += CS * kThreads) {
      const int r = u / (D / 8), col = 8 * (u % (D / 8));
      if (r >= rows) break;
      float2 ml[CS];
      float top = kNegInf;
#pragma unroll
      for (int c = 0; c < CS; ++c) {
        ml[c] = peer_float2(smem_u32(s_part_ml + r), c);
        top = fmaxf(top, ml[c].x);
      }
      const float ref = top == kNegInf ? 0.f : top;
      float x[8] = {}, sum = 0.f;
#pragma unroll
      for (int c = 0; c < CS; ++c) {
        if (ml[c].y == 0.f) continue;  // a CTA without tiles has written nothing
        const float f = exp2_approx((ml[c].x - ref) * p.scale_log2);
        sum = fmaf(f, ml[c].y, sum);
        const float4 a = peer_float4(base + (r * D + col) * 4, c);
        const float4 b = peer_float4(base + (r * D + col) * 4 + 16, c);
        x[0] = fmaf(f, a.x, x[0]), x[1] = fmaf(f, a.y, x[1]);
        x[2] = fmaf(f, a.z, x[2]), x[3] = fmaf(f, a.w, x[3]);
        x[4] = fmaf(f, b.x, x[4]), x[5] = fmaf(f, b.y, x[5]);
        x[6] = fmaf(f, b.z, x[6]), x[7] = fmaf(f, b.w, x[7]);
      }
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      const int kvh_c = blockIdx.x / CS % p.hkv;
      const int tok = r / p.group, head = kvh_c * p.group + r - tok * p.group;
      uint4 v;
      v.x = Half<T>::pack(x[0] * inv, x[1] * inv);
      v.y = Half<T>::pack(x[2] * inv, x[3] * inv);
      v.z = Half<T>::pack(x[4] * inv, x[5] * inv);
      v.w = Half<T>::pack(x[6] * inv, x[7] * inv);
      *reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + (s.row0 + tok) * p.o_row + head * p.o_head +
                                 col) = v;
    }
    cluster_sync();  // nobody's shared memory goes while a peer reads it
  }
}

// Joins the parts of the item that begins in CTA blockIdx.x and ends in a later one; a warp takes a
// row.  The parts are added in the order of the positions: repeat calls give the same bytes.
template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(kThreads) join_kernel(const Work w) {
  const Params &p = w.p;
  pdl_wait();
  pdl_launch();
  const Shared sh = w.shared[blockIdx.x];
  const int r = blockIdx.y * (kThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int R = r;
  if (sh.pieces == 0 || R >= sh.rows) return;
  const int64_t c0 = blockIdx.x;
  const int64_t first = 2 * c0 + sh.slot;
  const auto slot = [&](int i) { return i == 0 ? first : 2 * (c0 + i); };
  float top = kNegInf;
  for (int i = lane; i < sh.pieces; i += 32) top = fmaxf(top, w.part_ml[slot(i) * ROWS + r].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float ref = top == kNegInf ? 0.f : top;
  constexpr int V = D / 32;
  float x[V] = {}, sum = 0.f;
#pragma unroll 4
  for (int i = 0; i < sh.pieces; ++i) {
    const int64_t at = slot(i) * ROWS + r;
    const float2 ml = w.part_ml[at];
    const float f = exp2_approx((ml.x - ref) * p.scale_log2);
    sum = fmaf(f, ml.y, sum);
    const float *src = w.part + at * D + V * lane;
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = fmaf(f, src[e], x[e]);
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const int tok = R / p.group, head = sh.kvh * p.group + R - tok * p.group;
  uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<T *>(p.out) + (sh.row0 + tok) * p.o_row +
                                               head * p.o_head + V * lane);
#pragma unroll
  for (int e = 0; e < V / 2; ++e) dst[e] = Half<T>::pack(x[2 * e] * inv, x[2 * e + 1] * inv);
}

struct Plan {
  int sms;
  int grid, rows;  // CTAs, rows of a tile
  int cluster;     // CTAs of an item's cluster; 0: all CTAs share all items
  int64_t part, ml, shared, bytes;  // offsets in the workspace
};

constexpr int64_t kClusterPositions = 16384;  // up to which a cluster takes an item

// Of n items a key/value head with up to `rows` rows and `positions` positions each; `most_items` of them
// at most can have any.
inline int make_plan(const moe_kv_cache *c, const Params &p, int64_t n, int64_t most_items,
                     int64_t rows, int64_t positions, Plan *plan, bool clusters_too = true) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MOE_ERR_CUDA;
  plan->sms = sms;
  plan->rows = rows <= 16 ? 16 : 32;
  // With few items a cluster takes each, when the 16 or 8 CTAs of every one can be resident at once: one
  // kernel instead of two.  (32 query, 8 key/value heads of 128, one token, shared line against clusters
  // of 16: 500 positions 8.5, 6.8 us; 4000 15.1, 10.8; 8000 18.2, 14.8; 16000 21.8, 22.6; 32000 34.7,
  // 39.2.  16 items of 4000: 15.2, clusters of 16 17.2, of 8 12.4; 32 items of 2000: 13.8, of 8 10.1.)
  plan->cluster = 0;
  plan->part = plan->ml = plan->shared = plan->bytes = 0;
  const int64_t clusters = n * p.hkv;
  if (clusters_too && positions <= kClusterPositions)
    plan->cluster = clusters * 16 <= sms ? 16 : clusters * 8 <= sms * kCtasPerSm ? 8 : 0;
  plan->grid = static_cast<int>(clusters) * plan->cluster;
  if (plan->cluster) return MOE_OK;
  // no more CTAs than the largest batch that the arguments allow has work for
  const int64_t len = positions / tile_of(c->head_dim) + 1;
  const int64_t items = most_items * p.hkv;
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

// Whether the CTAs of clusters of 8 are all resident at once: 288 are, 304 are not.
inline bool resident(const Plan &plan) { return 10 * static_cast<int64_t>(plan.grid) <= 19 * plan.sms; }

inline void use_workspace(const Plan &plan, void *workspace, Work *w) {
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  w->part = reinterpret_cast<float *>(ws + plan.part);
  w->part_ml = reinterpret_cast<float2 *>(ws + plan.ml);
  w->shared = reinterpret_cast<Shared *>(ws + plan.shared);
}

// All CTAs share all items.
template <typename T, int D, int WR, int ITEMS>
static cudaError_t launch_line(const Work &w, int grid, cudaStream_t stream) {
  const auto kern = tree_kernel<T, D, WR, 0, ITEMS>;
  static SmemLimit limit;
  cudaError_t e = limit.set(reinterpret_cast<const void *>(kern), Tree<D>::kSmem);
  if (e != cudaSuccess) return e;
  if (ITEMS != kSeqs) {
    e = launch_early(kern, dim3(grid), kThreads, Tree<D>::kSmem, stream, w);
  } else {
    kern<<<grid, kThreads, Tree<D>::kSmem, stream>>>(w);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  // the joining blocks are set up while the kernel runs and wait for its end
  return launch_early(join_kernel<T, D, 16 * WR>, dim3(grid, 16 * WR / (kThreads / 32)), kThreads, 0,
                      stream, w);
}

// A cluster of CS CTAs takes each of `items` items.
template <typename T, int D, int WR, int CS, int ITEMS>
static cudaError_t launch_cluster(const Work &w, int items, cudaStream_t stream) {
  const auto kern = tree_kernel<T, D, WR, CS, ITEMS>;
  static SmemLimit limit;
  cudaError_t e = limit.set(reinterpret_cast<const void *>(kern), Tree<D>::kSmem, CS > 8);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(items * CS);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Tree<D>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CS;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ITEMS != kSeqs ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, w);
}

// A few items: each by a cluster of cs (8 or 16) CTAs.
cudaError_t launch_clusters(const moe_kv_cache *c, const Work &w, int rows, int cs,
                            cudaStream_t stream);

}  // namespace attn
