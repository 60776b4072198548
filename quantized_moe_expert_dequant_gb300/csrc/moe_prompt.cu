// moe_prompt.cu -- causal attention of packed prompts over the pages of a cache, on the 5th-generation
// tensor cores (moe_prompt_attention).
//
//   out_r = sum_j p_rj v_j / sum_j p_rj,   p_rj = exp(scale * q_r . k_j - m_r)  over the positions j
//   that row r sees, in one pass over K and V with a running maximum and sum.
//
// Bound by the two products (4 D flops per row and position).  A CTA takes two tiles of up to 128
// rows of one sequence and one key/value head: row R of a tile is token R / group, query head
// R % group, so all query heads of a key/value head share the K and V that one CTA loads, and a short
// prompt still fills the tiles.  Per 128 positions and tile:
//   S = Q K^T    128 x 128 x D, both operands in shared memory, S in TMEM
//   softmax      four warps, one row a thread: S from TMEM to registers, P back over S in 16 bits
//   O += P V     128 x D x 128, P from TMEM, V from shared memory, O in TMEM
// The two tiles take turns: while four warps are at one tile's softmax, the tensor cores work on
// the other tile.  One thread issues all products in the order S0 S1 | PV0 S0' | PV1 S1' | ..., they
// complete in that order, and one commit after S0' therefore also says that PV0 is done.
// O is only scaled down when a row's maximum has grown by more than 2^8 since O's last scale; the
// weights then stay below 2^8, which 16-bit floats and the fp32 sums hold without loss.
#include "moe_attention.cuh"
#include "moe_tcgen05.cuh"

#include <type_traits>

namespace attn {

constexpr int kPos = 128;               // positions of a step
constexpr int kSoftmaxWarps = 8;        // four a tile
constexpr int kPromptThreads = 32 * (kSoftmaxWarps + 4);  // and products, copies, two idle warps
// 168 registers at launch; 2 x 128 x 208 + 128 x 88 = 384 x 168
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
constexpr float kGrowth = 8.f;          // log2 of how far a maximum may grow before O is rescaled

template <int D>
struct Prompt {
  static constexpr int kTileBytes = kPos * D * 2;             // K, V or a tile of Q
  static constexpr int kStages = D == 128 ? 5 : 8;            // ring of K and V tiles, in turn
  static constexpr int kSmem = (2 + kStages) * kTileBytes + 1024;
  static constexpr int kColumns = 512;                        // S0 S1 (128 each) O0 O1 (D each)
};

struct PromptParams {
  Params p;
  CUtensorMap q, k, v;
  int tokens;  // of a tile: 128 / group
};

// The tile that CTA `index` takes: tiles in the order of falling cost, so that the last ones to
// start are the shortest.  The cost of a tile is its number of steps c; N(c) tiles cost c or more, a
// closed form per sequence, and a binary search finds the cost of the index-th tile.
struct Pick {
  int seq, tile;
};

__device__ __forceinline__ int tiles_at_least(const Seq &s, int per, int c) {
  const int all = (s.nq + per - 1) / per;
  const int64_t below = static_cast<int64_t>(c - 1) * kPos - s.ctx;  // tokens whose tiles cost less
  if (s.nq <= below) return 0;
  return below <= 0 ? all : all - static_cast<int>(below / per);
}

__device__ __forceinline__ int block_sum(int v, int *s_warp) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = v;
  __syncthreads();
  int sum = 0;
#pragma unroll
  for (int w = 0; w < kPromptThreads / 32; ++w) sum += s_warp[w];
  return sum;
}

__device__ __forceinline__ bool pick_tile(const Params &p, int per, int index, bool report,
                                          int *s_warp, Pick *s_pick) {
  const int tid = threadIdx.x;
  Seq mine = {0, 0, 0, 0};
  if (tid < p.n_seqs) mine = load_seq(p, tid, report);
  const auto count = [&](int c) {
    int n = tid < p.n_seqs ? tiles_at_least(mine, per, c) : 0;
    for (int s = tid + kPromptThreads; s < p.n_seqs; s += kPromptThreads)
      n += tiles_at_least(load_seq(p, s, report && c == 1), per, c);
    return block_sum(n, s_warp);
  };
  if (index >= count(1)) return false;
  // the largest cost c with more than `index` tiles of at least c
  int lo = 1;
  int64_t top = (static_cast<int64_t>(p.table_width) << p.page_shift) / kPos + 2;
  int hi = top > INT32_MAX ? INT32_MAX : static_cast<int>(top);
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (count(mid) > index) lo = mid; else hi = mid;
  }
  int rank = index - count(lo + 1);  // among the tiles that cost exactly lo
  // warp 0 walks the sequences in order
  if (tid < 32) {
    for (int b = 0; b < p.n_seqs; b += 32) {
      const int s = b + tid;
      Seq q = {0, 0, 0, 0};
      if (s < p.n_seqs) q = load_seq(p, s, false);
      const int from = s < p.n_seqs ? tiles_at_least(q, per, lo) : 0;
      const int here = from - (s < p.n_seqs ? tiles_at_least(q, per, lo + 1) : 0);
      int before = here;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, o);
        if (tid >= o) before += y;
      }
      const int all = __shfl_sync(0xffffffffu, before, 31);
      before -= here;
      if (rank >= before && rank < before + here) {
        s_pick->seq = s;
        s_pick->tile = (q.nq + per - 1) / per - from + rank - before;
      }
      if (rank < all) break;
      rank -= all;
    }
  }
  __syncthreads();
  return true;
}

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
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

template <typename T, int D>
__global__ void __launch_bounds__(kPromptThreads, 1)
    prompt_kernel(const __grid_constant__ PromptParams w) {
  using C = Prompt<D>;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t s_q[2], s_full[C::kStages], s_empty[C::kStages], s_s[2], s_p[2],
      s_o[2], s_end;
  __shared__ uint32_t s_tmem;
  __shared__ int s_gone, s_warp[kPromptThreads / 32];
  __shared__ Pick s_pick;
  const Params &p = w.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kvh = blockIdx.x % p.hkv, index = blockIdx.x / p.hkv;
  if (!pick_tile(p, 2 * w.tokens, index, index == 0 && kvh == 0, s_warp, &s_pick)) return;
  const int seq = s_pick.seq;
  const Seq s = load_seq(p, seq, false);
  // tokens and steps of the two tiles
  const int tok0 = s_pick.tile * 2 * w.tokens;
  const int tok1 = tok0 + w.tokens;
  const int n0 = (s.ctx + min(tok1, s.nq) + kPos - 1) / kPos;
  const int n1 = tok1 < s.nq ? (s.ctx + min(tok1 + w.tokens, s.nq) + kPos - 1) / kPos : 0;
  const int steps = max(n0, n1);

  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  const auto bar = [](uint64_t &b) { return smem_u32(&b); };
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::bar_init(bar(s_q[i]), 1);
      tc::bar_init(bar(s_s[i]), 1);
      tc::bar_init(bar(s_p[i]), kSoftmaxWarps / 2);
      tc::bar_init(bar(s_o[i]), 1);
    }
    for (int i = 0; i < C::kStages; ++i) {
      tc::bar_init(bar(s_full[i]), 1);
      tc::bar_init(bar(s_empty[i]), 1);
    }
    tc::bar_init(bar(s_end), 1);
    s_gone = 0;
    tc::bar_fence_init();
  }
  if (warp == kSoftmaxWarps) tc::tmem_alloc(smem_u32(&s_tmem), C::kColumns);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = s_tmem;
  const uint32_t ring = base + 2 * C::kTileBytes;

  if (warp >= kSoftmaxWarps) tc::regs_down<kOtherRegs>();
  if (warp == kSoftmaxWarps + 1) {
    // ---------------------------------------------------------------- copies
    if (lane == 0) {
      for (int i = 0; i < (n1 > 0 ? 2 : 1); ++i) {
        const int tok = i ? tok1 : tok0;
        tc::bar_expect(bar(s_q[i]), static_cast<uint32_t>(w.tokens * p.group * D * 2));
        for (int h = 0; h < D / 64; ++h)
          tc::copy_3d(base + i * C::kTileBytes + h * kPos * 128, &w.q, 64 * h, kvh * p.group,
                      s.row0 + tok, bar(s_q[i]));
      }
    }
    // a box is one page's positions of a step (all 128 for larger pages), 64 elements wide; lanes
    // take one each
    const int box_rows = min(1 << p.page_shift, kPos);
    const int per_half = kPos / box_rows, boxes = per_half * (D / 64);
    const int32_t *pages = p.table + seq * p.table_stride;
    const int b_row = (lane % per_half) * box_rows, half = lane / per_half;
    int issued = 0;
    for (int t = 0; t < steps; ++t) {
      int page = p.n_pages;  // outside the cache: reads zeros
      const int pos = t * kPos + b_row;
      if (lane < boxes && pos < s.len) {
        page = pages[pos >> p.page_shift];
        if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.n_pages)) {
          if (p.err) atomicOr(p.err, kDevErrBadId);
          page = p.n_pages;
        }
      }
      const int in_page = pos & ((1 << p.page_shift) - 1);
      bool ok = true;
      for (int kv = 0; kv < 2 && ok; ++kv) {
        const int it = 2 * t + kv, st = it % C::kStages;
        ok = tc::bar_wait(bar(s_empty[st]), ((it / C::kStages) & 1) ^ 1, &s_gone);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) tc::bar_expect(bar(s_full[st]), C::kTileBytes);
        __syncwarp();
        if (lane < boxes)
          tc::copy_4d(ring + st * C::kTileBytes + half * kPos * 128 + b_row * 128,
                      kv ? &w.v : &w.k, 64 * half, in_page, kvh, page, bar(s_full[st]));
        issued = it + 1;
      }
      if (!ok) break;
    }
    if (s_gone) {  // let the copies under way land before the shared memory goes
      volatile int never = 0;
      const int from = issued > C::kStages ? issued - C::kStages : 0;
      for (int it = from; it < issued; ++it)
        tc::bar_wait(bar(s_full[it % C::kStages]), (it / C::kStages) & 1, &never);
      for (int i = 0; i < (n1 > 0 ? 2 : 1); ++i) tc::bar_wait(bar(s_q[i]), 0, &never);
    }
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
    const int u0 = uniform(n0), u1 = uniform(n1), last = uniform(steps), len = uniform(s.len);
    const uint32_t q_lo = tc::desc_lo(ub, 16);
    int st = 0, phase = 0;  // the ring's next stage
    const auto wait = [&](uint32_t b, int parity) {
      return __all_sync(0xffffffffu, tc::bar_wait(b, parity, &s_gone)) != 0;
    };
    const auto stage = [&](int i) { return ub + (2 + i) * C::kTileBytes; };
    const auto issue_s = [&](int i, uint32_t k) {
      const uint32_t k_lo = tc::desc_lo(k, 16);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk / 4) * kPos * 128 + (kk % 4) * 32) / 16;
        tc::mma_smem(one, tm + i * kPos, q_lo + i * (C::kTileBytes / 16) + off, hi, k_lo + off, hi,
                     i_s, kk > 0);
      }
      tc::mma_commit(one, bar(s_s[i]));
    };
    const auto next = [&]() {
      if (++st == C::kStages) st = 0, phase ^= 1;
    };
    bool ok = wait(bar(s_q[0]), 0) && wait(bar(s_full[0]), 0);
    if (ok) issue_s(0, stage(0));
    if (ok && u1 > 0) {
      ok = wait(bar(s_q[1]), 0);
      if (ok) issue_s(1, stage(0));
    }
    if (ok) tc::mma_commit(one, bar(s_empty[0]));
    next();
    for (int t = 0; ok && t < last; ++t) {
      const int v_st = st, v_phase = phase;
      next();
      const int k_st = st, k_phase = phase;
      next();
      const uint32_t v = stage(v_st);
      ok = wait(bar(s_full[v_st]), v_phase);
      const int valid = len - t * kPos;
      if (valid < kPos) {
        // positions behind the sequence have weight 0, but what their page holds may be NaN
        for (int x = valid * 128 + lane * 16; x < kPos * 128; x += 512)
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(v + h * kPos * 128 + x),
                         "r"(0)
                         : "memory");
        tc::fence_async_proxy();
        __syncwarp();
      }
      const uint32_t v_lo = tc::desc_lo(v, kPos * 128);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int n = i ? u1 : u0;
        if (ok && t < n) {
          ok = wait(bar(s_p[i]), t & 1);
          tc::fence_after();
          if (ok) {
#pragma unroll
            for (int kk = 0; kk < kPos / 16; ++kk)
              tc::mma_tmem(one, tm + 2 * kPos + i * D, tm + i * kPos + kk * 8, v_lo + kk * 128, hi,
                           i_o, t > 0 || kk > 0);
            if (t == n - 1) tc::mma_commit(one, bar(s_o[i]));
          }
        }
        if (ok && t + 1 < n) {
          ok = wait(bar(s_full[k_st]), k_phase);
          if (ok) issue_s(i, stage(k_st));
        }
      }
      if (ok) {
        tc::mma_commit(one, bar(s_empty[v_st]));
        if (t + 1 < last) tc::mma_commit(one, bar(s_empty[k_st]));
      }
    }
    if (s_gone) {  // let the products under way end before TMEM goes
      volatile int never = 0;
      tc::mma_commit(one, bar(s_end));
      tc::bar_wait(bar(s_end), 0, &never);
    }
  } else if (warp < kSoftmaxWarps) {
    // ---------------------------------------------------------------- softmax, one row a thread
    tc::regs_up<kSoftmaxRegs>();
    const int i = warp / 4;
    const int n = i ? n1 : n0, tok_first = i ? tok1 : tok0;
    const int r = threadIdx.x & 127;
    const int tok = tok_first + r / p.group;
    const bool row_ok = r < w.tokens * p.group && tok < s.nq;
    const int limit = s.ctx + tok + 1;  // positions that the row sees
    const uint32_t lanes = static_cast<uint32_t>(warp % 4) << 21;  // 32 * (warp % 4) << 16
    const uint32_t ts = tmem + lanes + i * kPos, to = tmem + lanes + 2 * kPos + i * D;
    float m = kNegInf, l = 0.f;
    bool ok = true;
    for (int t = 0; t < n; ++t) {
      ok = tc::bar_wait(bar(s_s[i]), t & 1, &s_gone);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc::fence_after();
      uint32_t x[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tc::tmem_load32(x[c], ts + 32 * c);
      tc::wait_load(x[0]);
      tc::loaded(x[1]);
      tc::loaded(x[2]);
      tc::loaded(x[3]);
      if ((t + 1) * kPos > s.ctx + tok_first + 1) {  // some row does not see all positions
        const int see = limit - t * kPos;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (32 * c + e >= see) x[c][e] = __float_as_uint(kNegInf);
      }
      float tops[4];  // four chains: one of 64 dependent maxima took 500 cycles
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        tops[c] = kNegInf;
#pragma unroll
        for (int e = 0; e < 32; e += 2)
          tops[c] = fmaxf(tops[c], fmaxf(__uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1])));
      }
      const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
      // every row sees position 0, so after the first step m is finite
      const float up = fmaxf(m, top);
      if (t == 0) {
        m = up;
      } else if (__any_sync(0xffffffffu, (up - m) * p.scale_log2 > kGrowth)) {
        const float f = exp2_approx((m - up) * p.scale_log2);
        m = up;
        l *= f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tc::tmem_load32(o, to + 32 * c);
          tc::wait_load(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
          tc::tmem_store32(to + 32 * c, o);
        }
      }
      const uint64_t sc = pair(p.scale_log2, p.scale_log2);
      const float off = -m * p.scale_log2;
      const uint64_t shift = pair(off, off);
      uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t y[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const uint32_t *src = &x[2 * c + e / 16][2 * (e % 16)];
          const float2 a = unpair(fma2(pair(__uint_as_float(src[0]), __uint_as_float(src[1])), sc,
                                       shift));
          const float pa = exp2_approx(a.x), pb = exp2_approx(a.y);
          sum[e & 1] = add2(sum[e & 1], pair(pa, pb));
          // the weights meet v in the cache's type: half a step of it, as large as the output's own
          // rounding
          y[e] = Half<T>::pack(pa, pb);
        }
        tc::tmem_store32(ts + 32 * c, y);
      }
      const float2 total = unpair(add2(sum[0], sum[1]));
      l += total.x + total.y;
      tc::wait_store();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::bar_arrive(bar(s_p[i]));
    }
    if (ok && n > 0) {
      ok = tc::bar_wait(bar(s_o[i]), 0, &s_gone);
      ok = __all_sync(0xffffffffu, ok);
      tc::fence_after();
      if (ok) {
        const float inv = 1.f / l;
        const int head = kvh * p.group + r % p.group;
        T *dst = static_cast<T *>(p.out) + (s.row0 + tok) * p.o_row + head * p.o_head;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tc::tmem_load32(o, to + 32 * c);
          tc::wait_load(o);
          if (row_ok) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint4 v;
              v.x = Half<T>::pack(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv);
              v.y = Half<T>::pack(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
              v.z = Half<T>::pack(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv);
              v.w = Half<T>::pack(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv);
              *reinterpret_cast<uint4 *>(dst + 32 * c + e) = v;
            }
          }
        }
      }
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

template <typename T, int D>
static int launch(const moe_kv_cache *c, const moe_attention *a, const Params &p,
                  cudaStream_t stream) {
  PromptParams w;
  w.p = p;
  w.tokens = 128 / p.group;
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
  const auto kern = prompt_kernel<T, D>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Prompt<D>::kSmem);
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  const int64_t tiles = (p.n_rows / (2 * w.tokens) + static_cast<int64_t>(p.n_seqs)) * p.hkv;
  if (tiles > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  kern<<<static_cast<int>(tiles), kPromptThreads, Prompt<D>::kSmem, stream>>>(w);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace attn

extern "C" int moe_prompt_attention(const moe_kv_cache *cache, const moe_attention *a,
                                    void *stream) {
  attn::Params p;
  const int rc = attn::check_attention(cache, a, &p);
  if (rc != MOE_OK) return rc;
  if (p.n_seqs == 0 || p.n_rows == 0) return MOE_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cache->dtype == MOE_DTYPE_BF16)
    return cache->head_dim == 64 ? attn::launch<__nv_bfloat16, 64>(cache, a, p, st)
                                 : attn::launch<__nv_bfloat16, 128>(cache, a, p, st);
  return cache->head_dim == 64 ? attn::launch<__half, 64>(cache, a, p, st)
                               : attn::launch<__half, 128>(cache, a, p, st);
}
