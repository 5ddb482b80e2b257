// sv_attn.cuh -- attention of drafted trees over the KV cache.
//
// "EAGLE-3 speculative decoding review", "EAGLE-2: Does Every Context Need the
// Same Draft Tree?" and "The Complete EAGLE-3 Inference Process" step 3: all
// nodes of a tree are scored in one pass of the target; a node sees the whole
// committed prefix and its own ancestors (itself among them).  Query head
// h G + g of node v of sequence b reads key-value head h:
//   o = sum_j softmax_j(scale q.k_j) v_j
// over j in the prefix shared by the batch (P entries, one copy), the
// sequence's own positions [0, base_len - 1), and the tree entries
// base_len - 1 + u with bit u of the node's mask row set (mask null: u <= v).
//
// The entries are taken 128 at a time by matrix products on the tensor cores,
// with the nodes' query heads of one key-value head as the rows: a sequence's
// nodes for its own entries (the tree's stand right behind the prefix, and
// only their tiles look at the mask), the whole batch's nodes for the shared
// prefix, so that its entries are read once for all.
//
// The work is cut into equal runs of (rows, 128 entries) tiles, one run per
// SM, whatever the lengths: the tiles of all items (shared prefix first, then
// sequence by sequence) stand in one line of T, CTA c takes [c T / n, (c+1) T / n),
// and an item that is cut (or has a shared prefix to be joined with) leaves one
// partial per CTA for tree_attn_finish_kernel to join: in slot item + c, or,
// where many items of which only cut ones leave partials would take too many
// slots, 2 c (+ 1 if the item begins in CTA c).  Shared and own items have
// slots of their own sizes.
//
// Measured (32 query heads of 8, D = 128; ranges over several runs): plain decoding of
// 64 sequences of about 3000 entries 132-139 us, 5.9 TB/s, bound by HBM; 16 trees
// of 60 nodes over as many 65-71 us (a floor of 33 us of HBM time); 3 trees of 33
// (40 heads) over 49000 entries 121-145 us under the power cap (91 us); 64 trees
// of 16 behind a shared prefix of 8192 180-185 us (77 us of tensor time).  In the
// loop trees are bound by the hand-over between softmax and products: a pair of
// halves takes 3200-3600 clocks a tile, 2048 of them products (16 of K = 16 for
// S, as many for O, 64 clocks each and half), because one half's chain -- its
// scores 490, softmax 1600, its product with V 630 and the hand-overs -- is longer
// than the other half's products beside it.  Outside the loop: start, fills and
// stores 9 of the 16 trees' 70 us, CTAs of unequal length 6, the wait for the
// join 8 and the join 10; behind a shared prefix the CTAs of short own items (15
// items of 4-5 tiles, 20500 clocks each) end at 184 us, those of the prefix at
// 120-153.  D = 64 (half the bytes and products): 107, 56, 114 and 155 us.  What
// was tried against it and lost (16 trees /
// long / shared prefix, us, then 69 / 137 / 182): one issuing warp per half 79 /
// 199 / 197; P handed over in two parts 78 / 153 / 233; scores loaded 64 or 128
// columns at once 81 / 145 / 184 and 78 / 141 / 177 (the products with V slow
// down beside long loads); two softmax warps for 32 rows, 64 entries each, 112 /
// 236 / 277 (96 registers a thread are too few).
#pragma once

#include "sv_lmhead.cuh"
#include "sv_rope.cuh"

namespace sv {

constexpr int kAtRows = 128;     // rows of a half (UMMA M, tensor-memory lanes)
constexpr int kAtKeys = 128;     // cache entries per tile
constexpr int kAtThreads = 384;  // copies, MMAs, segments, an idle warp, 2 x 4 softmax warps
constexpr int kAtMaxStages = 13;
constexpr int kAtMaxCtas = 160;  // partial slots are laid out for at most this many CTAs
constexpr float kAtLazy = 4096.0f;  // a tile's largest sum of a row's weights before its
                                    // reference is renewed
constexpr int kAtFinThreads = 256;
constexpr int kAtSegs = 4;       // segment descriptors ahead of their use
constexpr unsigned kAtTileNs = 20000;  // more than a tile takes (about 2000)

template <int D>
__host__ __device__ constexpr int at_tile_bytes() { return kAtKeys * D * 2; }
// Query tiles (one, or two where items are pairs) and as many K and V tiles as
// fit beside them: with the static arrays, all of an SM's 227 KB.
template <int D>
__host__ __device__ constexpr int at_tiles() { return D == 128 ? 7 : 14; }
template <int D>
__host__ __device__ constexpr int at_smem() { return at_tiles<D>() * at_tile_bytes<D>(); }

struct AttnParams {
  const uint16_t* q;        // [B, N, Hq, D]
  const uint16_t* k;        // [B, L, Hkv, D], sequences seq_stride elements apart
  const uint16_t* v;
  const uint32_t* mask;     // [B, N, W] or null (a chain)
  const int32_t* base_len;  // [B]
  uint16_t* out;            // [B, N, Hq, D]
  float* lse;               // [B, N, Hq] or null
  unsigned* flags;
  long long seq_stride;     // elements
  float scale_log2;         // scale * log2(e)
  int B, N, Hq, Hkv, G, W, L, P;
  // the prefixes' tiles
  int tok;                  // nodes per half: floor(128 / G)
  int pair_s, pair_o;       // shared / own items: two halves of rows (else one, by alternate tiles)
  int mg_s, mg_o;           // items per key-value head (and sequence)
  int tiles_s;              // ceil(P / 128)
  int rows_s, rows_o;       // rows of a slot of a shared / own item
  int by_cta;               // own items' slots by CTA (else by item)
  long long own0;           // row of the own items' slot 0
  int nctas;
  int q_tiles;              // 2 if any item is a pair
  float* opart;             // [slot][D / 4][rows][4]
  float2* ml;               // [slot][rows]: reference (log2) and sum
  unsigned long long wait_ns;  // limit of each wait between the roles, where it was set (else
                               // kWaitLimitNs), as a test does to exercise the timeout path
  int2* span;               // [items]: first and last CTA that holds a part of the item
};

__device__ __forceinline__ bool attn_seq_ok(const AttnParams& p, int base) {
  return base >= 1 && (long long)base + p.N - 1 <= p.L;
}
// 128-entry tiles of a sequence's own entries, prefix and tree
__device__ __forceinline__ int attn_tiles_of(const AttnParams& p, int base) {
  return attn_seq_ok(p, base) ? (base - 1 + p.N + kAtKeys - 1) / kAtKeys : 0;
}

// 1 / l and the log-sum; nothing visible (l = 0): output 0, log-sum -inf.
__device__ __forceinline__ float attn_norm(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }
__device__ __forceinline__ float attn_lse(float m, float l) {
  return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// A CTA's run of tiles is cut into segments, one per item it meets.
struct AttnSeg {
  long long slot;     // first row of the partial's slot
  int b, h;           // sequence (0 for the shared prefix), key-value head
  int node0, ntok;    // first node and number of nodes of the item's rows: of all nodes of the
                      // batch for the shared prefix, else of the sequence's
  int t0, n;          // tiles [t0, t0 + n) of the item; n = 0: no more segments
  int kvlen, plen;    // entries, and the first of them that not every node sees
  int shared, pair, whole;  // whole: all that the item's rows attend to
};
struct AttnWalk {
  long long pos, hi, bstart;  // bstart: first tile of sequence b in the line
  int b;
  __device__ __forceinline__ void next(const AttnParams& p, AttnSeg* s) {
    s->n = 0;
    if (pos >= hi) return;
    const long long items_s = (long long)p.Hkv * p.mg_s;
    const long long shared = items_s * p.tiles_s;
    long long it, item;  // item: among all, the shared ones first
    int tiles;
    s->shared = pos < shared;
    if (s->shared) {
      it = pos / p.tiles_s;
      tiles = p.tiles_s;
      s->t0 = (int)(pos - it * tiles);
      s->b = 0;
      s->kvlen = s->plen = p.P;
      item = it;
      s->slot = (it + blockIdx.x) * p.rows_s;
      s->pair = p.pair_s;
    } else {
      const int per = p.Hkv * p.mg_o;
      int base = p.base_len[b];
      tiles = attn_tiles_of(p, base);
      while (pos >= bstart + (long long)per * tiles) {
        bstart += (long long)per * tiles;
        base = p.base_len[++b];
        tiles = attn_tiles_of(p, base);
      }
      it = (pos - bstart) / tiles;
      s->t0 = (int)(pos - bstart - it * tiles);
      s->b = b;
      s->plen = base - 1;
      s->kvlen = s->plen + p.N;
      item = items_s + (long long)b * per + it;
      s->slot = p.own0 + (p.by_cta ? 2ll * blockIdx.x + (s->t0 == 0)
                                   : (long long)b * per + it + blockIdx.x) * p.rows_o;
      s->pair = p.pair_o;
    }
    const int mg = (int)it / p.Hkv;
    s->h = (int)it - mg * p.Hkv;
    s->node0 = mg * (p.tok << s->pair);
    s->ntok = min(p.tok << s->pair, (s->shared ? p.B * p.N : p.N) - s->node0);
    s->n = (int)min((long long)(tiles - s->t0), hi - pos);
    s->whole = s->n == tiles && p.tiles_s == 0;
    if (s->t0 == 0) p.span[item].x = blockIdx.x;
    if (s->t0 + s->n == tiles) p.span[item].y = blockIdx.x;
    pos += s->n;
  }
};

// --- tcgen05 / TMA forms of one CTA (see sv_lmhead.cuh for the pair's) -------

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                            int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}
// D (tensor memory) = or += A B with both operands in shared memory
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// the same with A in tensor memory (two bf16 per column)
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_addr(bar))
      : "memory");
}
// 16 columns to and from registers; a store's wait is tmem_wait_st
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15}, [%16];\ntcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// Shared-memory descriptor of V [keys, D] as the product's second operand
// with D contiguous (MN-major, 128-byte swizzle): 64-wide column blocks 128
// rows x 128 bytes apart (leading-byte offset), 8-key groups 1024 bytes apart
// (stride-byte offset).  A step of 16 keys advances the start by 2048 bytes.
__device__ __forceinline__ uint64_t umma_desc_mn_sw128(uint32_t smem_byte_addr) {
  return umma_desc_sw128(smem_byte_addr) | ((uint64_t)((kAtKeys * 128) >> 4) << 16);
}

// A wait in the kernel below.  The first test sleeps up to 1 ms in the
// instruction; past that, the wait ends when it has taken its limit or another
// role of the CTA has given up.  As in mbar_wait_bounded, a limit of 1 ns gives
// up as soon as one test finds the phase incomplete.  kSet: the limit is p's
// (instantiations of their own, since a limit that is not a constant makes the
// softmax loop slower: a shared prefix 180 -> 207 us).
template <bool kSet>
__device__ __forceinline__ bool at_try(const AttnParams& p, uint64_t* bar, unsigned parity) {
  if (!kSet) return mbar_try_wait(bar, parity);
  return mbar_try_wait(bar, parity, (uint32_t)min(p.wait_ns, (unsigned long long)kSuspendHintNs));
}
template <bool kSet>
__device__ __forceinline__ bool at_wait_slow(const AttnParams& p, uint64_t* bar, unsigned parity,
                                             const int* abort, uint64_t more_ns = 0) {
  const uint64_t limit = (kSet ? p.wait_ns : kWaitLimitNs) + more_ns;
  if (limit <= 1) return false;
  const uint64_t t0 = global_ns();
  for (unsigned it = 0; it < (1u << 30); ++it) {
    if (at_try<kSet>(p, bar, parity)) return true;
    if (*(const volatile int*)abort || global_ns() - t0 > limit) return false;
  }
  return false;
}
template <bool kSet>
__device__ __forceinline__ bool at_wait(const AttnParams& p, uint64_t* bar, unsigned parity,
                                        const int* abort, uint64_t more_ns = 0) {
  return at_try<kSet>(p, bar, parity) || at_wait_slow<kSet>(p, bar, parity, abort, more_ns);
}
// the same for a whole warp, with one answer
template <bool kSet>
__device__ __forceinline__ bool at_wait_warp(const AttnParams& p, uint64_t* bar, unsigned parity,
                                             const int* abort) {
  if (__all_sync(0xffffffffu, at_try<kSet>(p, bar, parity))) return true;
  return __all_sync(0xffffffffu, at_wait_slow<kSet>(p, bar, parity, abort));
}

// Warp 0 copies (TMA), warp 1 issues the MMAs, warp 2 lists the CTA's
// segments, warps 4-7 and 8-11 are the softmax of half 0 and 1.  A half is
// 128 rows with its own score and output accumulators in tensor memory
// (S0 | S1 | O0 | O1) and its own running reference and sums.  With more rows
// than one tile holds (pair), the halves are two row tiles over the same
// entries; otherwise both take the same rows and alternate tiles, and are
// joined at the end of an item.  Either way one half's softmax runs beside
// the other's products:
//   S = Q K^T -> registers -> P = 2^(S c - m), bf16, over S in tensor memory
//   O += P V   (P from tensor memory)
// The reference m of a row is the maximum of the first tile, and is renewed
// only by a tile whose weights add up to more than 2^12 (up to there they are
// harmless in bf16 and float32): the maximum of a tile is not looked for, the
// sum that softmax needs anyway shows whether the reference still serves, and
// the weights are kept back until it is known.
//   Every wait between the roles is a bounded one on an mbarrier; a role
// that gives up leaves, and the others follow.
template <int D, bool kSet>
__global__ void __launch_bounds__(kAtThreads, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap map_q,
                     const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v,
                     const __grid_constant__ CUtensorMap map_pk,
                     const __grid_constant__ CUtensorMap map_pv, const AttnParams p) {
  constexpr int kTile = at_tile_bytes<D>();
  constexpr int kSub = D / 64;  // 64-element column blocks of a tile (128 rows x 128 bytes)
  constexpr int kWarps = kAtThreads / 32;
  extern __shared__ __align__(1024) uint8_t smem[];
  static_assert(at_tiles<D>() - 1 <= kAtMaxStages, "ring barriers");
  __shared__ uint64_t full[kAtMaxStages], empty[kAtMaxStages];
  __shared__ uint64_t q_full, q_empty, s_full[2], p_full[2], o_full[2], drain;
  __shared__ uint64_t seg_full[kAtSegs], seg_empty[kAtSegs], half_bar[2], pair_bar;
  __shared__ AttnSeg s_seg[kAtSegs];
  __shared__ uint32_t tmem_holder;
  __shared__ int s_abort, s_b;
  __shared__ long long s_bstart, s_sum[kWarps];
  __shared__ float2 s_ml[2][kAtRows];
  __shared__ uint32_t s_bad[2][2][4];  // tree entries of a tile whose V is not finite: by
                                       // turns, half
  __shared__ uint32_t s_spoilt[2][4];  // rows of a half that see one in this segment
  uint8_t* ring = smem + p.q_tiles * kTile;
  const int S = at_tiles<D>() - p.q_tiles;  // ring stages
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (smem_addr(smem) & 1023) {  // swizzled tiles start at 1024-byte boundaries; never expected
    if (threadIdx.x == 0) set_flag(p.flags, kFlagTimeout);
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&q_full, 1);
    mbar_init(&q_empty, 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(&s_full[w], 1);
      mbar_init(&p_full[w], 4);
      mbar_init(&o_full[w], 1);
      mbar_init(&half_bar[w], 4);
    }
    mbar_init(&pair_bar, 8);
    for (int s = 0; s < kAtSegs; ++s) {
      mbar_init(&seg_full[s], 1);
      mbar_init(&seg_empty[s], 10);  // copies, MMAs, eight softmax warps
    }
    mbar_init(&drain, 1);
    s_abort = 0;
    s_b = 0;
    s_bstart = 0;
    mbar_init_fence();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&tmem_holder)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // a programmatic dependent of the kernel before it in the stream: nothing of
  // global memory is touched before that grid has finished
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  // (lengths and masks, which the call before this one may have written, are read
  // with ordinary loads: those that may be taken out of order are for data that
  // stays as it is while a kernel lives)
  // the run [lo, hi) of this CTA and the sequence it starts in: a scan of the
  // sequences' tile counts, kAtThreads sequences at a time
  const int per = p.Hkv * p.mg_o;
  const long long shared = (long long)p.Hkv * p.mg_s * p.tiles_s;
  int mine = (int)threadIdx.x < p.B ? attn_tiles_of(p, p.base_len[threadIdx.x]) : 0;
  long long own = mine;
  for (int b = threadIdx.x + kAtThreads; b < p.B; b += kAtThreads)
    own += attn_tiles_of(p, p.base_len[b]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) own += __shfl_xor_sync(0xffffffffu, own, o);
  if (lane == 0) s_sum[warp] = own;
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  own = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) own += s_sum[w];
  const long long total = shared + own * per;
  const int n = (int)min((long long)p.nctas, total);  // no run is empty; other CTAs have none
  const long long lo = (int)blockIdx.x < n ? total * blockIdx.x / n : 0;
  const long long hi = (int)blockIdx.x < n ? total * (blockIdx.x + 1) / n : 0;
  if (threadIdx.x == 0 && lo < shared) s_bstart = shared;
  {
    long long run = 0;
    for (int b0 = 0; b0 < p.B; b0 += kAtThreads) {
      const int b = b0 + threadIdx.x;
      if (b0 > 0) mine = b < p.B ? attn_tiles_of(p, p.base_len[b]) : 0;
      long long incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      __syncthreads();
      if (lane == 31) s_sum[warp] = incl;
      __syncthreads();
      long long before = run;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_sum[w];
        run += s_sum[w];
      }
      const long long excl = before + incl - mine;
      if (lo >= shared && lo - shared >= excl * per && lo - shared < (excl + mine) * per) {
        s_b = b;
        s_bstart = shared + excl * per;
      }
    }
  }
  __syncthreads();
  const uint32_t tmem = tmem_holder;
  const int* abort = &s_abort;
  auto fail = [&]() {
    s_abort = 1;
    set_flag(p.flags, kFlagTimeout);
  };

  if (warp == 2) {
    if (lane == 0) {
      // ---------------- segments ----------------
      AttnWalk walk{lo, hi, s_bstart, s_b};
      for (unsigned k = 0;; ++k) {
        AttnSeg seg;
        walk.next(p, &seg);
        const unsigned at = k % kAtSegs;
        // (the only wait that lasts as long as an item: until the one four before
        // this is begun, so up to the run's length)
        if (!at_wait<kSet>(p, &seg_empty[at], ((k / kAtSegs) & 1) ^ 1u, abort,
                           (uint64_t)(hi - lo) * kAtTileNs)) {
          fail();
          break;
        }
        s_seg[at] = seg;
        mbar_arrive(&seg_full[at]);
        if (seg.n == 0) break;
      }
    }
    __syncwarp();
  } else if (warp == 0) {
    if (lane == 0) {
      // ---------------- copies ----------------
      int stage = 0, issued = 0;
      unsigned phase = 0, nq = 0;
      for (bool ok = true; ok;) {
        const unsigned at = nq % kAtSegs;
        if (!at_wait<kSet>(p, &seg_full[at], (nq / kAtSegs) & 1, abort)) {
          fail();
          break;
        }
        const AttnSeg seg = s_seg[at];
        mbar_arrive(&seg_empty[at]);
        if (seg.n == 0) break;
        if (!at_wait<kSet>(p, &q_empty, (nq & 1) ^ 1u, abort)) {
          fail();
          break;
        }
        ++nq;
        const int tok0 = seg.b * p.N + seg.node0;
        mbar_expect_tx(&q_full, (unsigned)((1 + seg.pair) * kSub * p.tok * p.G * 128));
        for (int w = 0; w <= seg.pair; ++w)
          for (int c = 0; c < kSub; ++c)
            tma_load_3d(smem + w * kTile + c * (kAtRows * 128), &map_q, c * 64, seg.h * p.G,
                        tok0 + w * p.tok, &q_full);
        const CUtensorMap* mk = seg.shared ? &map_pk : &map_k;
        const CUtensorMap* mv = seg.shared ? &map_pv : &map_v;
        auto put = [&](const CUtensorMap* m, int t) {
          if (!at_wait<kSet>(p, &empty[stage], phase ^ 1u, abort)) {
            ok = false;
            fail();
            return;
          }
          mbar_expect_tx(&full[stage], kTile);
          for (int c = 0; c < kSub; ++c)
            tma_load_4d(ring + stage * kTile + c * (kAtKeys * 128), m, c * 64, seg.h,
                        (seg.t0 + t) * kAtKeys, seg.b, &full[stage]);
          ++issued;
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        };
        // in the order of use: each V tile, then the K tile `ahead` further on
        const int ahead = 2 - seg.pair;
        for (int t = 0; ok && t < seg.n + ahead; ++t) {
          if (t >= ahead) put(mv, t - ahead);
          if (ok && t < seg.n) put(mk, t);
        }
      }
      // every copy has landed before the CTA can leave
      for (int j = max(0, issued - S); j < issued; ++j)
        mbar_wait_bounded(&full[j % S], (unsigned)((j / S) & 1));
      if (nq) mbar_wait_bounded(&q_full, (nq - 1) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------- MMAs ----------------
      const uint32_t id_qk = umma_idesc_bf16_f32(kAtRows, kAtKeys);
      const uint32_t id_pv = umma_idesc_bf16_f32(kAtRows, D) | (1u << 16);  // V: MN-major
      const uint64_t qdesc = umma_desc_sw128(smem_addr(smem));
      const uint64_t kdesc = umma_desc_sw128(smem_addr(ring));
      const uint64_t vdesc = umma_desc_mn_sw128(smem_addr(ring));
      int stage = 0;
      unsigned phase = 0, nq = 0, np0 = 0, np1 = 0;
      bool ok = true;
      auto wait = [&](uint64_t* bar, unsigned parity) {
        if (!at_wait<kSet>(p, bar, parity & 1, abort)) {
          ok = false;
          fail();
        }
        tmem_fence_after();
        return ok;
      };
      auto advance = [&]() {
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      };
      // scores of half w from the K tile in stage st, query tile qt
      auto scores = [&](int w, int qt, int st) {
        const uint64_t a = qdesc + (uint64_t)(qt * kTile >> 4);
        const uint64_t b = kdesc + (uint64_t)(st * kTile >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t o = (uint64_t)((kk >> 2) * (kAtKeys * 128 >> 4) + (kk & 3) * 2);
          umma_ss(tmem + w * kAtKeys, a + o, b + o, id_qk, kk ? 1u : 0u);
        }
        umma_commit(&s_full[w]);
      };
      // output of half w from the V tile in stage st
      auto output = [&](int w, int st, bool first) {
        const uint64_t b = vdesc + (uint64_t)(st * kTile >> 4);
#pragma unroll
        for (int kk = 0; kk < kAtKeys / 16; ++kk)
          umma_ts(tmem + 2 * kAtKeys + w * D, tmem + w * kAtKeys + kk * 8,
                  b + (uint64_t)(kk * (2048 >> 4)), id_pv, (!first || kk) ? 1u : 0u);
      };
      while (ok) {
        const unsigned at = nq % kAtSegs;
        if (!wait(&seg_full[at], nq / kAtSegs)) break;
        const int n = s_seg[at].n, pair = s_seg[at].pair;
        mbar_arrive(&seg_empty[at]);
        if (n == 0 || !wait(&q_full, nq++)) break;
        if (pair) {
          // ring: K0, V0, K1, V1, ...; each tile is waited for as late as its use
          // allows, and where the tensor cores have work
          if (!wait(&full[stage], phase)) break;
          scores(0, 0, stage);
          scores(1, 1, stage);
          if (n == 1) umma_commit(&q_empty);
          advance();
          int vst = stage;
          if (!wait(&full[stage], phase)) break;
          advance();
#pragma unroll 1
          for (int t = 0; t < n; ++t) {
            const bool more = t + 1 < n;
            const int v = vst, k = stage;
            if (more && !wait(&full[stage], phase)) break;
            if (!wait(&p_full[0], np0++)) break;
            output(0, v, t == 0);
            if (more) {
              scores(0, 0, k);
              advance();
              vst = stage;
              if (!wait(&full[stage], phase)) break;
              advance();
            } else {
              umma_commit(&o_full[0]);
            }
            if (!wait(&p_full[1], np1++)) break;
            output(1, v, t == 0);
            if (more) {
              scores(1, 1, k);
              if (t + 2 == n) umma_commit(&q_empty);
            } else {
              umma_commit(&o_full[1]);
            }
          }
        } else {
          for (int t = 0; t < min(2, n); ++t) {
            if (!wait(&full[stage], phase)) break;
            scores(t, 0, stage);
            if (t + 1 == n) umma_commit(&q_empty);
            advance();
          }
#pragma unroll 1
          for (int t = 0; ok && t < n; ++t) {
            const int w = t & 1, vst = stage;
            if (!wait(&full[stage], phase)) break;
            advance();
            if (!wait(&p_full[w], w ? np1++ : np0++)) break;
            output(w, vst, t < 2);
            if (t + 2 < n) {
              if (!wait(&full[stage], phase)) break;
              scores(w, 0, stage);
              if (t + 3 == n) umma_commit(&q_empty);
              advance();
            } else {
              umma_commit(&o_full[w]);
            }
          }
        }
      }
      // every MMA has completed before tensor memory is freed
      umma_commit(&drain);
      mbar_wait_bounded(&drain, 0);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------- softmax ----------------
    const int w = (warp - 4) >> 2;                // half
    const int quad = warp & 3;                    // tensor-memory lanes 32 quad ..
    const int r = quad * 32 + lane;               // row of the half
    const int rtok = r / p.G, rhead = r - rtok * p.G;
    const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
    const uint32_t sbase = lanes + w * kAtKeys;
    unsigned ns = 0, no = 0, nh = 0, npair = 0;  // uses of the barriers so far
    unsigned ring0 = 0;                          // ring uses before this segment
    // Ring uses of a segment, in the order of the copies: K tile t and V tile t
    // (pair: K0 V0 K1 V1 ..; else K0 K1 V0 K2 V1 K3 ..).
    auto k_use = [&](int pair, int t) { return pair ? 2 * t : t < 2 ? t : 2 * t - 1; };
    auto v_use = [&](int pair, int t, int n) { return min(n, t + 2 - pair) + t; };
    // A half whose scores or outputs are complete frees the tiles that made
    // them (of a pair, half 1, whose products come last).
    auto slot_of = [&](int use) {
      const unsigned u = ring0 + use;
      return p.q_tiles == 2 ? u % (at_tiles<D>() - 2) : u % (at_tiles<D>() - 1);
    };
    auto release = [&](int use) {
      if (quad == 0 && lane == 0) mbar_arrive(&empty[slot_of(use)]);
    };
    // all warps of a half, or of both halves, meet
    auto meet = [&](uint64_t* bar, unsigned& uses) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
      return at_wait_warp<kSet>(p, bar, uses++ & 1, abort);
    };
    bool ok = true;
    for (unsigned k = 0; ok; ++k) {
      if (!at_wait_warp<kSet>(p, &seg_full[k % kAtSegs], (k / kAtSegs) & 1, abort)) {
        ok = false;
        break;
      }
      const AttnSeg seg = s_seg[k % kAtSegs];
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_empty[k % kAtSegs]);
      if (seg.n == 0) break;
      const int pair = seg.pair;
      const int node = seg.node0 + (pair ? w * p.tok : 0) + rtok;
      const int nrows = max(0, min(p.tok, seg.ntok - (pair ? w * p.tok : 0))) * p.G;
      const bool busy = quad * 32 < nrows;  // whole warps of unused rows only wait
      const int nt = pair ? seg.n : (seg.n + 1 - w) / 2;
      float m = -1e30f, l = 0.0f;
      if (lane == 0) s_spoilt[w][quad] = 0;
      for (int i = 0; i < nt; ++i) {
        const int t = pair ? i : 2 * i + w;
        const int key0 = (seg.t0 + t) * kAtKeys;
        const bool edge = key0 + kAtKeys > seg.plen;  // not all of the tile is seen by all
        uint32_t see[4];
        if (edge) {
          // the row's view of the tile, 32 entries per word
          const int tree0 = key0 - seg.plen;  // tree number of the tile's first entry
          const uint32_t* mrow = !seg.shared && p.mask && node < p.N
                                     ? p.mask + ((size_t)seg.b * p.N + node) * p.W : nullptr;
          auto word = [&](int j) -> uint32_t {  // tree entries 32 j .. that the node sees
            if (j < 0) return 0xFFFFFFFFu;
            if (seg.shared || j >= p.W) return 0u;
            uint32_t x;
            if (p.mask) {
              x = mrow ? mrow[j] : 0u;
            } else {
              const int c = node + 1 - 32 * j;
              x = c >= 32 ? 0xFFFFFFFFu : c <= 0 ? 0u : (1u << c) - 1u;
            }
            const int left = p.N - 32 * j;
            return left < 32 ? x & ((1u << left) - 1u) : x;
          };
          const int j0 = tree0 >> 5;
          uint32_t x[5];
#pragma unroll
          for (int c = 0; c < 5; ++c) x[c] = word(j0 + c);
#pragma unroll
          for (int c = 0; c < 4; ++c) see[c] = __funnelshift_r(x[c], x[c + 1], tree0 & 31);
        }
        if (!at_wait_warp<kSet>(p, &s_full[w], ns++ & 1, abort)) {
          ok = false;
          break;
        }
        tmem_fence_after();
        if (!pair || w == 1) {
          release(k_use(pair, t));
          if (i > 0) release(v_use(pair, t - (2 - pair), seg.n));
        }
        if (edge) {
          // V entries beyond the last are zeroed, whatever they hold: their
          // products with weights of 0 have to be 0.  So are tree entries that
          // are not finite, and the outputs of rows that see them become NaN
          // (not their log-sums, which V has no part in).
          if (!pair || w == 0) {
            const int use = v_use(pair, t, seg.n);
            const int st = slot_of(use);
            if (!at_wait_warp<kSet>(p, &full[st], ((ring0 + use) / S) & 1, abort)) {
              ok = false;
              break;
            }
            const int at = key0 + r;
            bool bad = false;
            if (at >= seg.plen) {
              uint8_t* row = ring + st * kTile + r * 128;
              if (at < seg.kvlen) {
#pragma unroll
                for (int c = 0; c < kSub; ++c)
#pragma unroll
                  for (int j = 0; j < 8; ++j) {  // by turns, so that rows meet other banks
                    const uint4 x = lds128(row + c * (kAtKeys * 128) + ((j + r) & 7) * 16);
                    auto inf = [](uint32_t y) {
                      return (y & 0x7F80u) == 0x7F80u || (y & 0x7F800000u) == 0x7F800000u;
                    };
                    bad |= inf(x.x) | inf(x.y) | inf(x.z) | inf(x.w);
                  }
              }
              if (bad || at >= seg.kvlen) {
#pragma unroll
                for (int c = 0; c < kSub; ++c)
#pragma unroll
                  for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<uint4*>(row + c * (kAtKeys * 128) + ((j + r) & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
              }
            }
            const unsigned any = __ballot_sync(0xffffffffu, bad);
            if (lane == 0) s_bad[i & 1][w][quad] = any;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          ok = pair ? meet(&pair_bar, npair) : meet(&half_bar[w], nh);
          if (!ok) break;
          uint32_t bad = 0;
#pragma unroll
          for (int c = 0; c < 4; ++c) bad |= see[c] & s_bad[i & 1][pair ? 0 : w][c];
          const unsigned rows_bad = __ballot_sync(0xffffffffu, bad != 0);
          if (rows_bad && lane == 0) s_spoilt[w][quad] |= rows_bad;
        }
        if (busy) {
          const unsigned long long c2 = f2pack(p.scale_log2, p.scale_log2);
          unsigned long long sum0, sum1, nm2;
          auto hide = [&](uint32_t (&a)[32], uint32_t bits) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!((bits >> j) & 1)) a[j] = 0xFF800000u;
          };
          // weights of 32 entries, two to a word
          auto weights = [&](const uint32_t (&a)[32], uint32_t (&pk)[16]) {
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              float e0, e1, e2, e3;
              f2unpack(fma2(f2pack(__uint_as_float(a[2 * j]), __uint_as_float(a[2 * j + 1])), c2,
                            nm2), e0, e1);
              f2unpack(fma2(f2pack(__uint_as_float(a[2 * j + 2]), __uint_as_float(a[2 * j + 3])),
                            c2, nm2), e2, e3);
              e0 = ex2(e0);
              e1 = ex2(e1);
              e2 = ex2(e2);
              e3 = ex2(e3);
              sum0 = add2(sum0, f2pack(e0, e1));
              sum1 = add2(sum1, f2pack(e2, e3));
              pk[j] = pack_bf16(e0, e1);
              pk[j + 1] = pack_bf16(e2, e3);
            }
          };
          auto total = [&]() {
            float x, y;
            f2unpack(add2(sum0, sum1), x, y);
            return x + y;
          };
          bool good = false;
          if (i > 0) {
            uint32_t sa[32], sb[32], p0[16], p1[16], p2[16], p3[16];
            nm2 = f2pack(-m, -m);
            sum0 = sum1 = 0;
            tmem_ld32_async(sbase, sa);
            tmem_wait_ld(sa);
            tmem_ld32_async(sbase + 32, sb);
            if (edge) hide(sa, see[0]);
            weights(sa, p0);
            tmem_wait_ld(sb);
            tmem_ld32_async(sbase + 64, sa);
            if (edge) hide(sb, see[1]);
            weights(sb, p1);
            tmem_wait_ld(sa);
            tmem_ld32_async(sbase + 96, sb);
            if (edge) hide(sa, see[2]);
            weights(sa, p2);
            tmem_wait_ld(sb);
            if (edge) hide(sb, see[3]);
            weights(sb, p3);
            good = __all_sync(0xffffffffu, total() <= kAtLazy || r >= nrows);
            if (good) {
              tmem_st16(sbase, p0);
              tmem_st16(sbase + 16, p1);
              tmem_st16(sbase + 32, p2);
              tmem_st16(sbase + 48, p3);
            }
          }
          if (!good) {
            // the first tile, or a sum that shows the reference to be too old:
            // the row's maximum first
            float x = -INFINITY, y = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t a[32];
              tmem_ld32(sbase + 32 * c, a);
              if (edge) hide(a, c == 0 ? see[0] : c == 1 ? see[1] : c == 2 ? see[2] : see[3]);
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                x = fmaxf(fmaxf(x, __uint_as_float(a[j])), __uint_as_float(a[j + 1]));
                y = fmaxf(fmaxf(y, __uint_as_float(a[j + 2])), __uint_as_float(a[j + 3]));
              }
            }
            const float mn = fmaxf(m, fmaxf(x, y) * p.scale_log2), f = ex2(m - mn);
            m = mn;
            l *= f;
            if (i > 0) {  // the tile before this one is in the output: its product was
                          // issued before this tile's scores
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                uint32_t o[16];
                const uint32_t at = lanes + 2 * kAtKeys + w * D + c;
                tmem_ld16(at, o);
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                tmem_st16(at, o);
              }
            }
            nm2 = f2pack(-m, -m);
            sum0 = sum1 = 0;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {  // P of a chunk goes over scores already taken
              uint32_t a[32], pk[16];
              tmem_ld32(sbase + 32 * c, a);
              if (edge) hide(a, c == 0 ? see[0] : c == 1 ? see[1] : c == 2 ? see[2] : see[3]);
              weights(a, pk);
              tmem_st16(sbase + 16 * c, pk);
            }
          }
          l += total();
          tmem_wait_st();
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[w]);
      }
      if (!ok) break;
      // the item's output, or its partial as [D / 4][rows][4], so that a
      // warp's lanes (rows) store 512 consecutive bytes
      if (nt > 0 && !at_wait_warp<kSet>(p, &o_full[w], no++ & 1, abort)) {
        ok = false;
        break;
      }
      tmem_fence_after();
      if (nt > 0 && (!pair || w == 1)) release(v_use(pair, pair ? nt - 1 : 2 * (nt - 1) + w, seg.n));
      ring0 += 2 * seg.n;
      const bool mine_row = r < nrows;
      float* slot = p.opart + seg.slot * D;
      const int rows = seg.shared ? p.rows_s : p.rows_o;
      const int row = (pair ? w * p.tok * p.G : 0) + r;
      const size_t orow = ((size_t)seg.b * p.N + node) * p.Hq + seg.h * p.G + rhead;
      auto put = [&](int c, const uint32_t (&o)[32], float norm) {
        if (!mine_row) return;
        if (seg.whole) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + orow * D + c);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[e] = pack_bf16(__uint_as_float(o[8 * j + 2 * e]) * norm,
                               __uint_as_float(o[8 * j + 2 * e + 1]) * norm);
            dst[j] = make_uint4(x[0], x[1], x[2], x[3]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(slot + ((c / 4 + j) * rows + row) * 4) =
                make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        }
      };
      // NaN over the columns [c0, c1) that put stored, in a spoilt row
      auto spoil = [&](int c0, int c1, uint32_t rows_bad) {
        if (!((rows_bad >> lane) & 1) || !mine_row) return;
        const uint32_t x = seg.whole ? 0x7FC07FC0u : 0x7FC00000u;
#pragma unroll 1
        for (int c = c0; c < c1; c += 4) {
          if (!seg.whole)
            *reinterpret_cast<uint4*>(slot + (c / 4 * rows + row) * 4) = make_uint4(x, x, x, x);
          else
            *reinterpret_cast<uint2*>(p.out + orow * D + c) = make_uint2(x, x);
        }
      };
      auto put_ml = [&](float mm, float ll) {
        if (!mine_row) return;
        if (!seg.whole)
          p.ml[seg.slot + row] = make_float2(mm, ll);
        else if (p.lse)
          p.lse[orow] = attn_lse(mm, ll);
      };
      const uint32_t obase = lanes + 2 * kAtKeys;
      if (pair) {
        if (busy) {
          const float norm = attn_norm(l);
          put_ml(m, l);
#pragma unroll 1
          for (int c = 0; c < D; c += 64) {
            uint32_t o0[32], o1[32];
            tmem_ld32_async(obase + w * D + c, o0);
            tmem_ld32_async(obase + w * D + c + 32, o1);
            tmem_wait_ld(o0);
            tmem_wait_ld(o1);
            put(c, o0, norm);
            put(c + 32, o1, norm);
          }
          __syncwarp();
          spoil(0, D, s_spoilt[w][quad]);
        }
        tmem_fence_before();
      } else {
        // join the two halves; each takes half of the columns
        s_ml[w][r] = make_float2(m, l);
        if (!(ok = meet(&pair_bar, npair))) break;
        tmem_fence_after();
        if (busy) {
          const float2 a = s_ml[0][r], b = s_ml[1][r];  // half 0 has at least one tile
          const float mm = fmaxf(a.x, b.x);
          const float fa = ex2(a.x - mm), fb = ex2(b.x - mm);
          const float ll = seg.n > 1 ? a.y * fa + b.y * fb : a.y;
          const float norm = attn_norm(ll);
          if (w == 0) put_ml(mm, ll);
#pragma unroll 1
          for (int c = w * (D / 2); c < (w + 1) * (D / 2); c += 32) {
            uint32_t o[32], o1[32];
            tmem_ld32_async(obase + c, o);
            if (seg.n > 1) tmem_ld32_async(obase + D + c, o1);
            tmem_wait_ld(o);
            if (seg.n > 1) {
              tmem_wait_ld(o1);
#pragma unroll
              for (int j = 0; j < 32; ++j)
                o[j] = __float_as_uint(
                    __fmaf_rn(__uint_as_float(o1[j]), fb, __uint_as_float(o[j]) * fa));
            }
            put(c, o, norm);
          }
          spoil(w * (D / 2), (w + 1) * (D / 2), s_spoilt[0][quad] | s_spoilt[1][quad]);
        }
        // neither half's accumulators are written again before both are read
        tmem_fence_before();
        ok = meet(&pair_bar, npair);
      }
    }
    if (!ok) fail();
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (warp == 1) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

// Joins the partials of items that several CTAs share or that have a shared
// prefix; other rows are done.  A thread takes E elements of a row (a node's
// query head), neighbouring lanes neighbouring rows of a key-value head, as
// the partials lie, and reads A partials at once: the kernel is a chain of
// loads (lengths, span, partials), and what counts is how few times a thread
// waits (few items in many parts) or how many threads are resident (many items).
template <int D, int E, int A>
__global__ void __launch_bounds__(kAtFinThreads, E * A <= 32 ? 3 : 2)
    tree_attn_finish_kernel(const AttnParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const unsigned rows = (unsigned)p.B * p.N * p.Hq;  // at most 2^31
  const unsigned blocks = (rows + kAtFinThreads - 1) / kAtFinThreads;
  const unsigned part = blockIdx.x / blocks;  // E elements: part < D / E
  const unsigned at = (blockIdx.x - part * blocks) * kAtFinThreads + threadIdx.x;
  if (at >= rows) return;
  // row = ((b Hkv + h) N + n) G + g
  const unsigned ng = (unsigned)p.N * p.G, bh = at / ng, in_bh = at - bh * ng;
  const int n = (int)(in_bh / p.G), g = (int)(in_bh - (unsigned)n * p.G);
  const int b = (int)(bh / p.Hkv), h = (int)(bh - (unsigned)b * p.Hkv);
  const bool ok = attn_seq_ok(p, p.base_len[b]);
  float m = -1e30f, l = 0.0f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.0f;
  if (ok) {
#pragma unroll 1
    for (int k = p.tiles_s == 0 ? 1 : 0; k < 2; ++k) {  // shared prefix, own entries
      const int cap = p.tok << (k == 0 ? p.pair_s : p.pair_o);
      const int node = k == 0 ? b * p.N + n : n;
      const int mg = node / cap;
      const int row = (node - mg * cap) * p.G + g;  // (half 1 stands behind the tok G of half 0)
      const long long it = ((k == 0 ? 0ll : (long long)b * p.mg_o) + mg) * p.Hkv + h;
      int2 span = p.span[k == 0 ? it : (long long)p.Hkv * p.mg_s + it];
      if (p.tiles_s == 0 && span.x == span.y) return;  // written by its only CTA
      // slots of the workspace, whatever an overlapping call made of the span
      span.x = max(span.x, 0);
      span.y = min(span.y, p.nctas - 1);
      const int slot_rows = k == 0 ? p.rows_s : p.rows_o;
      const bool by_cta = k == 1 && p.by_cta;
      const long long slot0 = (k == 0 ? 0ll : p.own0) + (by_cta ? 0ll : it * slot_rows);
      const int first = span.x;
      const float* base = p.opart + (size_t)part * E * slot_rows + (size_t)row * 4;
      for (int c = span.x; c <= span.y; c += A) {
        float2 x[A];
        float4 y[A][E / 4];
#pragma unroll
        for (int i = 0; i < A; ++i) {
          if (c + i <= span.y) {
            const int at_c = by_cta ? 2 * (c + i) + (c + i == first) : c + i;
            const size_t slot = (size_t)(slot0 + (long long)at_c * slot_rows);
            x[i] = p.ml[slot + row];
#pragma unroll
            for (int j = 0; j < E / 4; ++j)
              y[i][j] = *reinterpret_cast<const float4*>(base + slot * D + (size_t)j * 4 * slot_rows);
          }
        }
#pragma unroll
        for (int i = 0; i < A; ++i) {
          if (c + i <= span.y) {
            const float mn = fmaxf(m, x[i].x);
            const float fa = ex2(m - mn), fb = ex2(x[i].x - mn);
            m = mn;
            l = l * fa + x[i].y * fb;
#pragma unroll
            for (int j = 0; j < E / 4; ++j) {
              acc[4 * j] = acc[4 * j] * fa + y[i][j].x * fb;
              acc[4 * j + 1] = acc[4 * j + 1] * fa + y[i][j].y * fb;
              acc[4 * j + 2] = acc[4 * j + 2] * fa + y[i][j].z * fb;
              acc[4 * j + 3] = acc[4 * j + 3] * fa + y[i][j].w * fb;
            }
          }
        }
      }
    }
  } else if (n == 0 && h == 0 && g == 0 && part == 0) {
    set_flag(p.flags, kFlagBadPath);
  }
  const float norm = attn_norm(l);
  const size_t orow = ((size_t)b * p.N + n) * p.Hq + h * p.G + g;
  uint4* out = reinterpret_cast<uint4*>(p.out + orow * D + part * E);
#pragma unroll
  for (int j = 0; j < E / 8; ++j) {
    uint32_t x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      x[e] = pack_bf16(acc[8 * j + 2 * e] * norm, acc[8 * j + 2 * e + 1] * norm);
    out[j] = make_uint4(x[0], x[1], x[2], x[3]);
  }
  if (p.lse && part == 0) p.lse[orow] = attn_lse(m, l);
}

}  // namespace sv
