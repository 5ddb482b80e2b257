// sv_attn4t.cuh -- attention of drafted trees over a 4-bit cache in pages, on the
// tensor cores' tiles: more rows (nodes x query heads of a key-value head) than
// sv_attn4.cuh serves.
//
// The same tiles, roles and softmax as the attention over a bf16 cache
// (sv_attn.cuh: segments, half tiles, references, hand-overs), with two
// differences.  Entries do not come as tiles that a product can read: a warp
// copies the packed groups of a tile, and two groups of four warps, one for keys
// and one for values, unpack them to fp16 tiles in the layout that a TMA copy
// would have given (K-major and, for the values, MN-major rows of 128 swizzled
// bytes).  And the products are of fp16, in which codes times scales are exact:
// queries are brought into its range by a power of two per row, weights by
// 2^kA4Off (they are rounded to fp16: 2^-11 of a weight, or 2^-32 of the largest).
//
// Bound: products, 4 N Hq D len operations (2048 clocks a pair of half tiles at
// D = 128), more than the pages' bytes.  Measured (D = 128, 8 key-value heads):
// 16 trees of 60 nodes, 32 heads, up to 4096 positions 87-91 us (products 25 us at
// the library's rate, the bf16 kernel 68; D = 64: 69, 13 and 57); 3 trees of 33, 40
// heads, up to 65536 positions 154-184 us (52; bf16 129; D = 64: 142, 23 and 109); 64
// chains of 8 nodes 183 us (35, the bytes; bf16 141).  A chunk of 1000 nodes behind
// each of 4 prompts of up to 4096, D = 128: 402 us (121; bf16 290), of which a chain's
// tiles of nodes that its rows do not see are computed all the same; alone 62.  About 4700 clocks a tile, two chains of
// scores (512), softmax (2050-2400 beside the warps that unpack) and output (512)
// with their hand-overs; and the hand-over of a place of the ring, 2300 clocks
// from the products that free it to the products that read it: query and unpacked
// tiles are 32 KB each, so four or five places are all there is.
// What was gained on the way from 143 / 234 us: queries and nodes by TMA,
// converted in place (115 / 222); no per-entry branches, and loops small enough
// for the instruction caches, which five roles share (96 / 169); the issuing warp
// as a whole (91); eight warps that unpack instead of four (87, long 173); every
// tile waited for right before its use (87-92, long 173 -> 157 in turns); waits of one
// loop, by the clock (90.5 -> 88.8, long 177 -> 173 in turns).
#pragma once

#include "sv_attn4.cuh"

namespace sv {

constexpr int kAtqThreads = 640;  // copies, MMAs, segments, an idle warp; 2 x 4 softmax warps;
                                  // 2 x 4 that unpack
constexpr int kAtqTurns = 16;
constexpr float kAtqLazy = 32768.0f;  // largest sum of a row's weights in 32 entries before its
                                      // reference is renewed: 2^8 times 2^kA4Off, within fp16

// Query and unpacked tiles, and half tiles (keys or values) of packed groups.
template <int D>
__host__ __device__ constexpr int atq_tiles() { return D == 128 ? 6 : 11; }
template <int D>
__host__ __device__ constexpr int atq_raw() { return D == 128 ? 3 : 8; }
template <int D>
__host__ __device__ constexpr int atq_smem() {
  return atq_tiles<D>() * at_tile_bytes<D>() + atq_raw<D>() * 4 * kv4_group(D);
}

struct AttnQParams : AttnParams {
  alignas(64) CUtensorMap map_q;  // [B N, Hq, D]
  CUtensorMap map_k, map_v;       // the nodes' [B, N, Hkv, D]
  const uint8_t* pages;  // [n_pages, Hkv, block]
  const int32_t* table;  // [B, Wt]
  const int32_t* exps;   // [2] or null
  long long n_pages;
  int Wt, lg;            // the table's width; log2 of the page size
  unsigned sleep_ns;     // longest sleep of one test of a wait
};

// The limit of the waits between the roles.  A wait ends at most one test behind it,
// so a test sleeps an eighth of it at most (3.9 us, measured, whatever it is told).
__host__ inline void atq_limit(AttnQParams* p, uint64_t limit_ns) {
  const uint64_t eighth = limit_ns / 8;
  p->wait_ns = limit_ns < (1ull << 62) ? limit_ns : 1ull << 62;
  p->sleep_ns = (unsigned)(eighth < 1 ? 1 : eighth < kSuspendHintNs ? eighth : kSuspendHintNs);
}

// Put i of a segment of n tiles into the ring, in the order of use: pairs K0 V0
// K1 V1 .., else K0 K1 V0 K2 V1 K3 .. (see the softmax's k_use and v_use).
__device__ __forceinline__ void atq_put(int pair, int n, int i, int* t, int* is_v) {
  if (pair) {
    *t = i >> 1;
    *is_v = i & 1;
  } else if (i < 2) {
    *is_v = i >= n;  // (n = 1: K0 V0)
    *t = *is_v ? 0 : i;
  } else {
    const int tk = (i + 1) >> 1;
    *is_v = !(i & 1) || tk >= n;
    *t = (i & 1) ? min(tk, n - 1) : (i - 2) >> 1;
  }
}

// True in one thread of the (converged) warp, the same each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
  return one != 0;
}
// Waits between the roles: tests that sleep in the instruction until the phase
// completes, and after each a look at whether another role has given up and at the
// clock (a wait is a few instructions, since what the roles share here is the
// instruction caches, see below).  end: when the wait is given up, set at the first
// look; a limit of 1 ns gives up there.
__device__ __forceinline__ bool atq_late(const AttnQParams& p, uint64_t& end, uint64_t more_ns) {
  const uint64_t now = global_ns();
  if (end == 0) end = now + p.wait_ns - 1 + more_ns;
  return now >= end;
}
__device__ __forceinline__ bool atq_wait(const AttnQParams& p, uint64_t* bar, unsigned parity,
                                         const int* abort, uint64_t more_ns = 0) {
  uint64_t end = 0;
#pragma unroll 1
  for (unsigned i = 1u << 30; i > 0; --i) {
    if (mbar_try_wait(bar, parity, p.sleep_ns)) return true;
    if (*(const volatile int*)abort || atq_late(p, end, more_ns)) break;
  }
  return false;
}
// the same for a whole warp, with one answer
__device__ __forceinline__ bool atq_wait_warp(const AttnQParams& p, uint64_t* bar, unsigned parity,
                                              const int* abort) {
  uint64_t end = 0;
#pragma unroll 1
  for (unsigned i = 1u << 30; i > 0; --i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity, p.sleep_ns))) return true;
    if (__any_sync(0xffffffffu, *(const volatile int*)abort || atq_late(p, end, 0))) break;
  }
  return false;
}

// fp16 operands, fp32 accumulator (formats 0 of bits 7-9 and 10-12)
__host__ __device__ constexpr uint32_t umma_idesc_f16_f32(int M, int N) {
  return umma_idesc_bf16_f32(M, N) & ~((1u << 7) | (1u << 10));
}

template <int D>
__global__ void __launch_bounds__(kAtqThreads, 1)
    kv4_attn_tiles_kernel(const __grid_constant__ AttnQParams p) {
  constexpr int kTile = at_tile_bytes<D>();
  constexpr int kSub = D / 64;  // 64-element column blocks of a tile (128 rows x 128 bytes)
  constexpr int kWarps = kAtqThreads / 32;
  constexpr int kHalf = 4 * kv4_group(D);  // bytes of the keys (values) of a tile in the pages
  constexpr int kRaw = atq_raw<D>();
  extern __shared__ __align__(1024) uint8_t smem[];
  static_assert(atq_tiles<D>() - 1 <= kAtMaxStages, "ring barriers");
  __shared__ uint64_t full[kAtMaxStages], empty[kAtMaxStages];
  __shared__ uint64_t raw_full[kRaw], raw_empty[kRaw], node_full[2][kAtqTurns], q_raw;
  __shared__ uint64_t q_full, q_empty, s_full[2], p_full[2], o_full[2], drain;
  __shared__ uint64_t seg_full[kAtSegs], seg_empty[kAtSegs], pair_bar;
  __shared__ AttnSeg s_seg[kAtSegs];
  __shared__ uint32_t tmem_holder;
  __shared__ int s_abort, s_b;
  __shared__ long long s_bstart, s_sum[kWarps];
  __shared__ float2 s_ml[2][kAtRows];
  __shared__ float s_fac[2][2][kAtRows];        // score of a row (log2) per unit of its product: by
                                                // turns, half
  __shared__ unsigned s_nopage[kRaw];           // bit j: positions 16 j .. have no page
  // of the K tiles in turn (more than the ring holds: some warps of a half may
  // still look at a tile that its first warp has given back): positions without
  // a page, and tree entries that are not finite
  __shared__ unsigned s_hole[kAtqTurns];
  __shared__ uint32_t s_bad[kAtqTurns][2][4];   // (of keys, of values)
  uint8_t* ring = smem + p.q_tiles * kTile;
  const int S = atq_tiles<D>() - p.q_tiles;  // ring stages
  uint8_t* raw = smem + atq_tiles<D>() * kTile;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (smem_addr(smem) & 1023) {  // swizzled tiles start at 1024-byte boundaries; never expected
    if (threadIdx.x == 0) set_flag(p.flags, kFlagTimeout);
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 4);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kRaw; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], 4);
    }
    for (int s = 0; s < 2 * kAtqTurns; ++s) mbar_init(&node_full[0][s], 1);
    mbar_init(&q_raw, 1);
    mbar_init(&q_full, 8);
    mbar_init(&q_empty, 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(&s_full[w], 2);  // the products, and the issuing thread for what it has waited for
      mbar_init(&p_full[w], 4);
      mbar_init(&o_full[w], 1);
    }
    mbar_init(&pair_bar, 8);
    for (int s = 0; s < kAtSegs; ++s) {
      mbar_init(&seg_full[s], 1);
      mbar_init(&seg_empty[s], 18);  // copies, MMAs, eight softmax warps, eight that unpack
    }
    mbar_init(&drain, 1);
    for (int s = 0; s < kAtqTurns; ++s) s_hole[s] = 0;
    s_abort = 0;
    s_b = 0;
    s_bstart = 0;
    mbar_init_fence();
  }
  if (threadIdx.x < kAtqTurns * 8) (&s_bad[0][0][0])[threadIdx.x] = 0;
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
  // sequences' tile counts, kAtqThreads sequences at a time
  const int per = p.Hkv * p.mg_o;
  int mine = (int)threadIdx.x < p.B ? attn_tiles_of(p, p.base_len[threadIdx.x]) : 0;
  long long own = mine;
  for (int b = threadIdx.x + kAtqThreads; b < p.B; b += kAtqThreads)
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
  const long long total = own * per;
  const int n = (int)min((long long)p.nctas, total);  // no run is empty; other CTAs have none
  const long long lo = (int)blockIdx.x < n ? total * blockIdx.x / n : 0;
  const long long hi = (int)blockIdx.x < n ? total * (blockIdx.x + 1) / n : 0;
  {
    long long run = 0;
    for (int b0 = 0; b0 < p.B; b0 += kAtqThreads) {
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
      if (lo >= excl * per && lo < (excl + mine) * per) {
        s_b = b;
        s_bstart = excl * per;
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

  // registers: 96 a thread at launch, 480 over the five warpgroups
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
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
          if (!atq_wait(p, &seg_empty[at], ((k / kAtSegs) & 1) ^ 1u, abort,
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
      // ---------------- copies ----------------
      // lane j < 8 brings in the keys or values of positions 16 j .. of a tile
      int stage = 0, issued = 0;
      unsigned phase = 0;
      bool ok = true;
      const int page = 1 << p.lg;
      for (unsigned k = 0; ok; ++k) {
        const unsigned at = k % kAtSegs;
        if (!atq_wait_warp(p, &seg_full[at], (k / kAtSegs) & 1, abort)) {
          ok = false;
          break;
        }
        const AttnSeg seg = s_seg[at];
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_empty[at]);
        if (seg.n == 0) break;
        const int32_t* row = p.table + (size_t)seg.b * p.Wt;
        auto page_of = [&](int i) {  // of this lane's positions of put i: -2 none wanted, -1 no page
          if (lane >= 8 || i >= 2 * seg.n) return -2;
          int t, is_v;
          atq_put(seg.pair, seg.n, i, &t, &is_v);
          const int pos = (seg.t0 + t) * kAtKeys + lane * 16;
          if (pos >= seg.plen) return -2;
          const int id = row[pos >> p.lg];
          return id >= 0 && id < p.n_pages ? id : -1;
        };
        // (pages are looked up two puts early)
        int id0 = page_of(0), id1 = page_of(1);
#pragma unroll 1
        for (int i = 0; i < 2 * seg.n; ++i) {
          int t, is_v;
          atq_put(seg.pair, seg.n, i, &t, &is_v);
          const int id = id0;
          id0 = id1;
          id1 = page_of(i + 2);
          const int key0 = (seg.t0 + t) * kAtKeys;
          if (key0 >= seg.plen) continue;  // nodes alone: not in the pages
          if (!atq_wait_warp(p, &raw_empty[stage], phase ^ 1u, abort)) {
            ok = false;
            break;
          }
          const unsigned some = __ballot_sync(0xffffffffu, id >= 0);
          const unsigned none = __ballot_sync(0xffffffffu, id == -1);
          if (lane == 0) {
            if (none) set_flag(p.flags, kFlagBadPage);
            s_nopage[stage] = none;
            mbar_expect_tx(&raw_full[stage], (unsigned)__popc(some) * (kHalf / 8));
          }
          __syncwarp();
          if (id >= 0)
            bulk_g2s(raw + stage * kHalf + lane * (kHalf / 8),
                     p.pages + ((size_t)id * p.Hkv + seg.h) * kv4_block(page, D) +
                         kv4_half((key0 + lane * 16) & (page - 1), is_v, D),
                     kHalf / 8, &raw_full[stage]);
          ++issued;
          if (++stage == kRaw) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && lane == 0) fail();
      // every copy has landed before the CTA can leave
      for (int j = max(0, issued - kRaw); j < issued; ++j)
        mbar_wait_bounded(&raw_full[j % kRaw], (unsigned)((j / kRaw) & 1));
      __syncwarp();
    } else if (warp == 1) {
      // ---------------- MMAs ----------------
      // The whole warp walks along and one elected thread issues, so that what the
      // products are issued with stands in uniform registers (one thread on its own
      // took 3900 clocks a tile to issue 2048 clocks of products).
      const uint32_t id_qk = umma_idesc_f16_f32(kAtRows, kAtKeys);
      const uint32_t id_pv = umma_idesc_f16_f32(kAtRows, D) | (1u << 16);  // V: MN-major
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint64_t qdesc = umma_desc_sw128(smem_addr(smem));
      const uint64_t kdesc = umma_desc_sw128(smem_addr(ring));
      const uint64_t vdesc = umma_desc_mn_sw128(smem_addr(ring));
      int stage = 0;
      unsigned phase = 0, nq = 0, np = 0, np1 = 0;
      bool ok = true;
      auto wait = [&](uint64_t* bar, unsigned parity) {
        if (!atq_wait_warp(p, bar, parity & 1, abort)) {
          ok = false;
          if (lane == 0) fail();
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
      auto commit = [&](uint64_t* bar) {
        if (elect_one()) umma_commit(bar);
        __syncwarp();
      };
      // scores of half w from the K tile in stage st, query tile qt
      auto scores = [&](int w, int qt, int st) {
        const uint64_t a = qdesc + (uint64_t)(qt * kTile >> 4);
        const uint64_t b = kdesc + (uint64_t)(st * kTile >> 4);
        const uint32_t d = tm + w * kAtKeys;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t o = (uint64_t)((kk >> 2) * (kAtKeys * 128 >> 4) + (kk & 3) * 2);
            umma_ss(d, a + o, b + o, id_qk, kk ? 1u : 0u);
          }
          umma_commit(&s_full[w]);
          mbar_arrive(&s_full[w]);
        }
        __syncwarp();
      };
      // output of half w from the V tile in stage st
      auto output = [&](int w, int st, bool first) {
        const uint64_t b = vdesc + (uint64_t)(st * kTile >> 4);
        const uint32_t d = tm + 2 * kAtKeys + w * D, a = tm + w * kAtKeys;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kAtKeys / 16; ++kk)
            umma_ts(d, a + kk * 8, b + (uint64_t)(kk * (2048 >> 4)), id_pv, (!first || kk) ? 1u : 0u);
        }
        __syncwarp();
      };
      while (ok) {
        const unsigned at = nq % kAtSegs;
        if (!wait(&seg_full[at], nq / kAtSegs)) break;
        const int n = __shfl_sync(0xffffffffu, s_seg[at].n, 0);
        const int pair = __shfl_sync(0xffffffffu, s_seg[at].pair, 0);
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_empty[at]);
        if (n == 0 || !wait(&q_full, nq++)) break;
        if (pair) {
          // ring: K0, V0, K1, V1, ...; each tile is waited for right before its use
          if (!wait(&full[stage], phase)) break;
          scores(0, 0, stage);
          scores(1, 1, stage);
          if (n == 1) commit(&q_empty);
          advance();
#pragma unroll 1
          for (int t = 0; t < n; ++t, ++np) {
            const bool more = t + 1 < n;
            const int v = stage;
            if (!wait(&p_full[0], np) || !wait(&full[stage], phase)) break;
            output(0, v, t == 0);
            advance();
            const int k = stage;
            if (more) {
              if (!wait(&full[stage], phase)) break;
              scores(0, 0, k);
              advance();
            } else {
              commit(&o_full[0]);
            }
            if (!wait(&p_full[1], np)) break;
            output(1, v, t == 0);
            if (more) {
              scores(1, 1, k);
              if (t + 2 == n) commit(&q_empty);
            } else {
              commit(&o_full[1]);
            }
          }
        } else {
          for (int t = 0; t < min(2, n); ++t) {
            if (!wait(&full[stage], phase)) break;
            scores(t, 0, stage);
            if (t + 1 == n) commit(&q_empty);
            advance();
          }
#pragma unroll 1
          for (int t = 0; ok && t < n; ++t) {
            const int w = t & 1, vst = stage;
            if (!wait(&full[stage], phase)) break;
            advance();
            if (!wait(&p_full[w], w ? np1++ : np++)) break;
            output(w, vst, t < 2);
            if (t + 2 < n) {
              if (!wait(&full[stage], phase)) break;
              scores(w, 0, stage);
              if (t + 3 == n) commit(&q_empty);
              advance();
            } else {
              commit(&o_full[w]);
            }
          }
        }
      }
      // every MMA has completed before tensor memory is freed
      commit(&drain);
      mbar_wait_bounded(&drain, 0);
      __syncwarp();
    }
  } else if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    // ---------------- unpacking ----------------
    // thread r of a group of four warps: query row r of its half, and node r of its
    // tiles.  (One copy of the code for keys and values: the roles share the
    // instruction caches.)
    const int r = (int)threadIdx.x & 127;
    const int kexp = kv4_exp(p.exps, 0);
    const float kinv = pow2_small(-kexp), vinv = pow2_small(-kv4_exp(p.exps, 1));
    int rst = 0, stage = 0;
    unsigned rphase = 0, phase = 0, nput = 0, tput = 0;  // node tiles and tiles so far
    unsigned noted = 0;           // turns whose words in s_bad and s_hole are not 0
    unsigned nq = 0, nasked = 0;  // (one thread's:) queries and node tiles asked for
    bool ok = true;
    // the tiles' rows of 128 bytes: 16-byte chunk c of row r stands at c ^ (r & 7)
    auto chunk = [&](uint8_t* tile, int r, int c) {  // of D / 8
      return reinterpret_cast<uint4*>(tile + (c >> 3) * (kAtRows * 128) + r * 128 +
                                      (((c & 7) ^ (r & 7)) << 4));
    };
    // Warps 12 to 15 unpack K tiles, 16 to 19 V tiles, so that from a free place to
    // a full one it is short (four warps for both: 16 trees of 60 nodes
    // 91 us, now 87).
    // A warp takes 32 entries: lane 4 s + c (D = 64: 2 s + c) takes
    // channels 32 c .. of entries s, s + kRows, ..: 16 bytes of codes, four chunks of
    // fp16, which start at chunk 4 (c & 1) of column block c >> 1 and lie at places
    // xor s & 7.  Lanes of the second column block store their chunks in the order
    // 2 3 0 1.
    constexpr int kRows = 32 * 32 / D;
    const int is_v = (warp - 12) >> 2, row0 = (warp & 3) * 32;
    const int ucc = lane % (D / 32), usub = lane / (D / 32);
    const bool uswap = ucc >= 2;
    const int udst = (ucc >> 1) * (kAtRows * 128) + (row0 + usub) * 128;
    const int ulow = ((4 * (ucc & 1) + (uswap ? 2 : 0)) ^ (usub & 7)) * 16;
    const bool asks = (threadIdx.x & 127) == 0;
    for (unsigned k = 0; ok; ++k) {
      const unsigned at = k % kAtSegs;
      if (!atq_wait_warp(p, &seg_full[at], (k / kAtSegs) & 1, abort)) {
        ok = false;
        break;
      }
      const AttnSeg seg = s_seg[at];
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_empty[at]);
      if (seg.n == 0) break;
      // the segment's queries and nodes come as bf16 tiles, for one thread to ask
      // for; the queries become fp16 in place, each row times a power of two that
      // brings its largest element to [2^14, 2^15)
      if (threadIdx.x == 384) {
        if (atq_wait(p, &q_empty, (k & 1) ^ 1u, abort)) {
          const int tok0 = seg.b * p.N + seg.node0;
          mbar_expect_tx(&q_raw, (unsigned)((1 + seg.pair) * kSub * p.tok * p.G * 128));
          for (int w = 0; w <= seg.pair; ++w)
            for (int c = 0; c < kSub; ++c)
              tma_load_3d(smem + w * kTile + c * (kAtRows * 128), &p.map_q, c * 64, seg.h * p.G,
                          tok0 + w * p.tok, &q_raw);
          ++nq;
        } else {
          fail();
        }
      }
      __syncwarp();
      if (!atq_wait_warp(p, &q_raw, k & 1, abort)) {
        ok = false;
        break;
      }
      if (is_v <= seg.pair && r < p.tok * p.G) {  // (rows of no node: whatever the copy brought)
        const int w = is_v;  // half
        uint8_t* tile = smem + w * kTile;
        uint32_t a = 0;
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          const uint4 x = lds128(chunk(tile, r, c));
          const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) a = max(a, max(y[e] & 0x7FFFu, (y[e] >> 16) & 0x7FFFu));
        }
        const int e2 = a == 0 || a >= 0x7F80u ? 0 : 14 - ilogbf(__uint_as_float(a << 16));
        const float nan = a >= 0x7F80u ? __int_as_float(0x7FC00000) : 0.0f;
        s_fac[k & 1][w][r] = score_unit(p.scale_log2, kexp - e2);
        const float f0 = pow2_small(e2 / 2), f1 = pow2_small(e2 - e2 / 2);  // (2^e2 may overflow)
#pragma unroll 2
        for (int c = 0; c < D / 8; ++c) {
          uint4* at_c = chunk(tile, r, c);
          const uint4 x = lds128(at_c);
          const uint32_t y[4] = {x.x, x.y, x.z, x.w};
          uint32_t z[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            z[e] = pack_half(bf16_lo(y[e]) * f0 * f1 + nan, bf16_hi(y[e]) * f0 * f1 + nan);
          *at_c = make_uint4(z[0], z[1], z[2], z[3]);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full);
      const int t_nodes = max(0, seg.plen / kAtKeys - seg.t0);  // the first tile with nodes
#pragma unroll 1
      for (int i = 0; i < 2 * seg.n; ++i) {
        int ti, vi;
        atq_put(seg.pair, seg.n, i, &ti, &vi);
        const int key0 = (seg.t0 + ti) * kAtKeys;
        // a tile with nodes: they are in it already (and 0 behind the last)
        const bool nodes = ti >= t_nodes, paged = key0 < seg.plen;
        if (vi == is_v) {
          uint8_t* tile = ring + stage * kTile;
          if (nodes && asks) {
            if (atq_wait(p, &empty[stage], phase ^ 1u, abort)) {
              uint64_t* bar = &node_full[is_v][nasked++ % kAtqTurns];
              mbar_expect_tx(bar, kTile);
              for (int c = 0; c < kSub; ++c)
                tma_load_4d(tile + c * (kAtKeys * 128), is_v ? &p.map_v : &p.map_k, c * 64, seg.h,
                            key0 - seg.plen, seg.b, bar);
            } else {
              fail();
            }
          }
          __syncwarp();
          if (!(nodes ? atq_wait_warp(p, &node_full[is_v][nput % kAtqTurns], (nput / kAtqTurns) & 1, abort)
                      : atq_wait_warp(p, &empty[stage], phase ^ 1u, abort))) {
            ok = false;
            break;
          }
          nput += nodes;
          unsigned hole = 0;
          if (paged) {
            if (!atq_wait_warp(p, &raw_full[rst], rphase, abort)) {
              ok = false;
              break;
            }
            hole = s_nopage[rst];
          }
          const uint8_t* src = raw + rst * kHalf + (row0 >> 4) * (kHalf / 8);
          const uint8_t* codes = src + usub * (D / 2) + ucc * 16;
          const uint8_t* scales = src + 8 * D + usub * (D / 16) + ucc * 2;
          uint8_t* dst = tile + udst;
          auto load = [&](int j, uint4& x, uint32_t& two) {
            const int group = j * kRows / 16, place = j * kRows % 16;
            x = lds128(codes + group * (kHalf / 8) + place * (D / 2));
            two = *reinterpret_cast<const uint16_t*>(scales + group * (kHalf / 8) + place * (D / 16));
          };
          auto unpack = [&](int j, uint4 x, uint32_t two) {
            const uint32_t s01 = kv4_scales(two);
            const uint32_t s0 = prmt(s01, 0, uswap ? 0x3232 : 0x1010);
            const uint32_t s1 = prmt(s01, 0, uswap ? 0x1010 : 0x3232);
            if (uswap) x = make_uint4(x.z, x.w, x.x, x.y);
            const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t h[4];
              kv4_unpack(y[e], h);
              const uint32_t s = e < 2 ? s0 : s1;
              *reinterpret_cast<uint4*>(dst + j * kRows * 128 + (ulow ^ (e * 16))) =
                  make_uint4(hmul2(h[0], s), hmul2(h[1], s), hmul2(h[2], s), hmul2(h[3], s));
            }
          };
          constexpr int kSteps = 32 / kRows;
          if (!nodes && !hole) {  // all of them: loads first, and no branches between
            uint4 x[kSteps];
            uint32_t two[kSteps];
#pragma unroll
            for (int j = 0; j < kSteps; ++j) load(j, x[j], two[j]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&raw_empty[rst]);  // (all that is needed of it is in registers)
#pragma unroll
            for (int j = 0; j < kSteps; ++j) unpack(j, x[j], two[j]);
          } else {
            const int left = seg.plen - key0 - row0 - usub;  // positions from this lane's first on
            if (paged)
#pragma unroll 1
              for (int j = 0; j < kSteps; ++j) {
                if (j * kRows >= left || ((hole >> ((row0 + j * kRows) >> 4)) & 1)) continue;
                uint4 x;
                uint32_t two;
                load(j, x, two);
                unpack(j, x, two);
              }
          }
          const unsigned turn = tput++ % kAtqTurns;
          if (nodes || hole || ((noted >> turn) & 1)) {
            // nodes, bf16 to fp16 in place; 0 if an element is not finite, and where
            // there is no page
            const int row = row0 + lane, key = key0 + row;
            const bool mine = key < seg.plen;
            bool bad = false;
            if (!mine && key < seg.kvlen) {
              const float f = is_v ? vinv : kinv;
#pragma unroll 2
              for (int c = 0; c < D / 8; ++c) {
                uint4* at_c = chunk(tile, row, c);
                const uint4 x = lds128(at_c);
                *at_c = make_uint4(node_half2(x.x, f, bad), node_half2(x.y, f, bad),
                                   node_half2(x.z, f, bad), node_half2(x.w, f, bad));
              }
            }
            if (bad || (mine && ((hole >> (row >> 4)) & 1)))
#pragma unroll 1
              for (int c = 0; c < D / 8; ++c) *chunk(tile, row, c) = make_uint4(0, 0, 0, 0);
            const unsigned any = __ballot_sync(0xffffffffu, bad);
            if (lane == 0) {  // (0 where nothing was noted before)
              s_bad[turn][is_v][row0 >> 5] = any;
              if (warp == 12) s_hole[turn] = hole;
            }
            noted = any || hole ? noted | (1u << turn) : noted & ~(1u << turn);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&full[stage]);
            if (paged && (nodes || hole)) mbar_arrive(&raw_empty[rst]);
          }
        }
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
        if (paged && ++rst == kRaw) {
          rst = 0;
          rphase ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) fail();
    if (asks) {  // every copy has landed before the CTA can leave
      for (unsigned j = nasked > kAtqTurns ? nasked - kAtqTurns : 0; j < nasked; ++j)
        mbar_wait_bounded(&node_full[is_v][j % kAtqTurns], (j / kAtqTurns) & 1);
      if (nq) mbar_wait_bounded(&q_raw, (nq - 1) & 1);
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
    // ---------------- softmax ----------------
    const int w = (warp - 4) >> 2;                // half
    const int quad = warp & 3;                    // tensor-memory lanes 32 quad ..
    const int r = quad * 32 + lane;               // row of the half
    const int rtok = r / p.G, rhead = r - rtok * p.G;
    const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
    const uint32_t sbase = lanes + w * kAtKeys;
    unsigned ns = 0, no = 0, npair = 0;          // uses of the barriers so far
    unsigned ring0 = 0;                          // ring uses before this segment
    // Ring uses of a segment, in the order of the copies: K tile t and V tile t
    // (pair: K0 V0 K1 V1 ..; else K0 K1 V0 K2 V1 K3 ..).
    auto k_use = [&](int pair, int t) { return pair ? 2 * t : t < 2 ? t : 2 * t - 1; };
    auto v_use = [&](int pair, int t, int n) { return min(n, t + 2 - pair) + t; };
    // A half whose scores or outputs are complete frees the tiles that made
    // them (of a pair, half 1, whose products come last).
    auto slot_of = [&](int use) {
      const unsigned u = ring0 + use;
      return p.q_tiles == 2 ? u % (atq_tiles<D>() - 2) : u % (atq_tiles<D>() - 1);
    };
    auto release = [&](int use) {
      if (quad == 0 && lane == 0) mbar_arrive(&empty[slot_of(use)]);
    };
    // all warps of a half, or of both halves, meet
    auto meet = [&](uint64_t* bar, unsigned& uses) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
      return atq_wait_warp(p, bar, uses++ & 1, abort);
    };
    bool ok = true;
    for (unsigned k = 0; ok; ++k) {
      if (!atq_wait_warp(p, &seg_full[k % kAtSegs], (k / kAtSegs) & 1, abort)) {
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
      float m = -1e30f, l = 0.0f, fac = 0.0f;
      for (int i = 0; i < nt; ++i) {
        const int t = pair ? i : 2 * i + w;
        const int key0 = (seg.t0 + t) * kAtKeys;
        bool edge = key0 + kAtKeys > seg.plen;  // not all of the tile is seen by all
        uint32_t see[4];
        if (edge) {
          // the row's view of the tile, 32 entries per word
          const int tree0 = key0 - seg.plen;  // tree number of the tile's first entry
          const uint32_t* mrow = p.mask && node < p.N
                                     ? p.mask + ((size_t)seg.b * p.N + node) * p.W : nullptr;
          auto word = [&](int j) -> uint32_t {  // tree entries 32 j .. that the node sees
            if (j < 0) return 0xFFFFFFFFu;
            if (j >= p.W) return 0u;
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
        const unsigned turn = (ring0 / 2 + t) % kAtqTurns;
        if (!atq_wait_warp(p, &s_full[w], ns++ & 1, abort)) {
          ok = false;
          break;
        }
        tmem_fence_after();
        if (i == 0) fac = s_fac[k & 1][pair ? w : 0][r];
        // positions without a page are hidden from all
        const unsigned hole = s_hole[turn];
        bool spoilt = false;
        if (edge) {
          // tree entries that are not finite are 0 in the tiles, and the sums of
          // the rows that see them become NaN
          const int use = v_use(pair, t, seg.n);
          if (!atq_wait_warp(p, &full[slot_of(use)], ((ring0 + use) / S) & 1, abort)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) spoilt |= ((s_bad[turn][0][c] | s_bad[turn][1][c]) & see[c]) != 0;
        }
        if (hole) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const unsigned two = hole >> (2 * c);
            see[c] = (edge ? see[c] : 0xFFFFFFFFu) &
                     ~((two & 1 ? 0xFFFFu : 0u) | (two & 2 ? 0xFFFF0000u : 0u));
          }
          edge = true;
        }
        __syncwarp();
        if (!pair || w == 1) {
          release(k_use(pair, t));
          if (i > 0) release(v_use(pair, t - (2 - pair), seg.n));
        }
        if (busy) {
          const unsigned long long c2 = f2pack(fac, fac);
          unsigned long long sum0, sum1, nm2;
          auto hide = [&](uint32_t (&a)[32], int c) {
            const uint32_t bits = c == 0 ? see[0] : c == 1 ? see[1] : c == 2 ? see[2] : see[3];
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
              pk[j] = pack_half(e0, e1);
              pk[j + 1] = pack_half(e2, e3);
            }
          };
          auto total = [&]() {
            float x, y;
            f2unpack(add2(sum0, sum1), x, y);
            return x + y;
          };
          // the row's maximum over the chunks from c0 on becomes its reference; what
          // there is of sums, output and weights follows
          auto renew = [&](int c0) {
            float x = -INFINITY, y = -INFINITY;
#pragma unroll 1
            for (int c = c0; c < 4; ++c) {
              uint32_t a[32];
              tmem_ld32(sbase + 32 * c, a);
              if (edge) hide(a, c);
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                x = fmaxf(fmaxf(x, __uint_as_float(a[j])), __uint_as_float(a[j + 1]));
                y = fmaxf(fmaxf(y, __uint_as_float(a[j + 2])), __uint_as_float(a[j + 3]));
              }
            }
            const float mn = fmaxf(m, fmaxf(x, y) * fac), f = ex2(m - mn);
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
            const uint32_t f2 = pack_half(f, f);
#pragma unroll 1
            for (int c = 0; c < c0; ++c) {  // weights that are stored already
              uint32_t o[16];
              tmem_ld16(sbase + 16 * c, o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = hmul2(o[j], f2);
              tmem_st16(sbase + 16 * c, o);
            }
            tmem_wait_st();
          };
          int c = 0;
          bool old = i > 0, stale = i == 0;  // the reference may be too old; it is
#pragma unroll 1
          while (c < 4) {  // weights of a chunk go over scores already taken
            if (stale) renew(c);
            stale = false;
            uint32_t a[32], pk[16];
            tmem_ld32(sbase + 32 * c, a);
            if (edge) hide(a, c);
            nm2 = f2pack(kA4Off - m, kA4Off - m);
            sum0 = sum1 = 0;
            weights(a, pk);
            const float sum = total();
            // a sum that shows the reference to be too old: once more with the
            // maximum of what is left, which serves to the tile's end
            if (old && __any_sync(0xffffffffu, sum > kAtqLazy && r < nrows)) {
              stale = true;
              old = false;
              continue;
            }
            l += sum;
            tmem_st16(sbase + 16 * c, pk);
            ++c;
          }
          if (spoilt) l = __int_as_float(0x7FC00000);
          tmem_wait_st();
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[w]);
      }
      if (!ok) break;
      // the item's output, or its partial as [D / 4][rows][4], so that a
      // warp's lanes (rows) store 512 consecutive bytes
      if (nt > 0 && !atq_wait_warp(p, &o_full[w], no++ & 1, abort)) {
        ok = false;
        break;
      }
      tmem_fence_after();
      if (nt > 0 && (!pair || w == 1)) release(v_use(pair, pair ? nt - 1 : 2 * (nt - 1) + w, seg.n));
      ring0 += 2 * seg.n;
      const bool mine_row = r < nrows;
      float* slot = p.opart + seg.slot * D;
      const int rows = p.rows_o;
      const float vscale = pow2_small(kv4_exp(p.exps, 1));
      const int row = (pair ? w * p.tok * p.G : 0) + r;
      const size_t orow = ((size_t)seg.b * p.N + node) * p.Hq + seg.h * p.G + rhead;
      auto scaled = [&](uint32_t x) { return __float_as_uint(__uint_as_float(x) * vscale); };
      auto put = [&](int c, const uint32_t (&o)[32], float norm) {
        if (!mine_row) return;
        norm *= vscale;
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
                make_uint4(scaled(o[4 * j]), scaled(o[4 * j + 1]), scaled(o[4 * j + 2]),
                           scaled(o[4 * j + 3]));
        }
      };
      auto put_ml = [&](float mm, float ll) {
        if (!mine_row) return;
        if (!seg.whole)
          p.ml[seg.slot + row] = make_float2(mm - kA4Off, ll);
        else if (p.lse)
          p.lse[orow] = attn_lse(mm - kA4Off, ll);
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

}  // namespace sv
