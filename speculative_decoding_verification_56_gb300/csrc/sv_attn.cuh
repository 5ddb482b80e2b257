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
// sequence by sequence) stand in one line, CTA c takes [c T / n, (c+1) T / n),
// and an item that is cut (or has a shared prefix to be joined with) leaves one
// partial per CTA, in slot item + c, for tree_attn_finish_kernel to join.
#pragma once

#include "sv_lmhead.cuh"
#include "sv_rope.cuh"

namespace sv {

constexpr int kAtRows = 128;     // rows of a half (UMMA M, tensor-memory lanes)
constexpr int kAtKeys = 128;     // cache entries per tile
constexpr int kAtThreads = 384;  // producer, MMA issuer, 2 idle warps, 2 x 4 softmax warps
constexpr int kAtMaxStages = 8;
constexpr int kAtMaxCtas = 160;  // partial slots are laid out for at most this many CTAs
constexpr float kAtLazy = 8.0f;  // a row's reference grows only past 2^8
constexpr int kAtFinThreads = 128;
constexpr int kAtFinHeads = 4;  // query heads of a key-value head held by a warp at once

template <int D>
__host__ __device__ constexpr int at_tile_bytes() { return kAtKeys * D * 2; }
// K and V tiles in flight beside the two query tiles, in 195 KB
template <int D>
__host__ __device__ constexpr int at_stages() { return D == 128 ? 4 : 8; }
template <int D>
__host__ __device__ constexpr int at_smem() { return (2 + at_stages<D>()) * at_tile_bytes<D>() + 1024; }

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
  int half_rows;            // rows stored per half
  int slot_rows;            // rows stored per slot
  int nctas;
  float* opart;             // [slot][D / 4][slot_rows][4]
  float2* ml;               // [slot][slot_rows]: reference (log2) and sum
  long long* tstart;        // [B + 1]: tiles of the sequences before b, per item
};

__device__ __forceinline__ bool attn_seq_ok(const AttnParams& p, int base) {
  return base >= 1 && (long long)base + p.N - 1 <= p.L;
}
// 128-entry tiles of a sequence's own entries, prefix and tree
__device__ __forceinline__ int attn_tiles(const AttnParams& p, int b) {
  const int base = __ldg(p.base_len + b);
  return attn_seq_ok(p, base) ? (base - 1 + p.N + kAtKeys - 1) / kAtKeys : 0;
}

// 1 / l and the log-sum; nothing visible (l = 0): output 0, log-sum -inf.
__device__ __forceinline__ float attn_norm(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }
__device__ __forceinline__ float attn_lse(float m, float l) {
  return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// A CTA's run of tiles, item by item.
struct AttnSeg {
  long long slot;     // of the partial: item + CTA
  int b, mg, h;       // b < 0: the shared prefix
  int t0, n, kvlen;   // tiles [t0, t0 + n) of an item with kvlen entries,
  int plen;           // the first plen of them seen by all nodes
  bool whole;         // all that the item's rows attend to
};
struct AttnWalk {
  long long pos, hi, bstart;  // bstart: first tile of sequence b in the line
  int b;
  __device__ __forceinline__ bool next(const AttnParams& p, AttnSeg* s) {
    if (pos >= hi) return false;
    const long long items_s = (long long)p.Hkv * p.mg_s;
    const long long shared = items_s * p.tiles_s;
    long long it;
    int tiles;
    if (pos < shared) {
      it = pos / p.tiles_s;
      tiles = p.tiles_s;
      s->t0 = (int)(pos - it * tiles);
      s->b = -1;
      s->kvlen = s->plen = p.P;
      s->slot = it + blockIdx.x;
    } else {
      const int per = p.Hkv * p.mg_o;
      tiles = attn_tiles(p, b);
      while (pos >= bstart + (long long)per * tiles) {
        bstart += (long long)per * tiles;
        tiles = attn_tiles(p, ++b);
      }
      it = (pos - bstart) / tiles;
      s->t0 = (int)(pos - bstart - it * tiles);
      s->b = b;
      s->plen = __ldg(p.base_len + b) - 1;
      s->kvlen = s->plen + p.N;
      s->slot = items_s + (long long)b * per + it + blockIdx.x;
    }
    s->mg = (int)(it / p.Hkv);
    s->h = (int)(it - (long long)s->mg * p.Hkv);
    s->n = (int)min((long long)(tiles - s->t0), hi - pos);
    s->whole = s->n == tiles && p.tiles_s == 0;
    pos += s->n;
    return true;
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

// Warp 0 copies (TMA), warp 1 issues the MMAs, warps 4-7 and 8-11 are the
// softmax of half 0 and 1.  A half is 128 rows with its own score and output
// accumulators in tensor memory (S0 | S1 | O0 | O1) and its own running
// reference and sums.  With more rows than one tile holds (pair), the halves
// are two row tiles over the same entries; otherwise both take the same rows
// and alternate tiles, and are joined at the end of an item.  Either way one
// half's softmax runs beside the other's products:
//   S = Q K^T -> registers -> P = 2^(S c - m), bf16, over S in tensor memory
//   O += P V   (P from tensor memory)
// The reference m of a row follows the row's maximum only when that has grown
// by more than 2^8 (P then stays below 2^8, harmless in bf16 and float32), so
// that O is rarely rescaled.
template <int D>
__global__ void __launch_bounds__(kAtThreads, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap map_q,
                     const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v,
                     const __grid_constant__ CUtensorMap map_pk,
                     const __grid_constant__ CUtensorMap map_pv, const AttnParams p) {
  constexpr int kTile = at_tile_bytes<D>();
  constexpr int S = at_stages<D>();
  constexpr int kSub = D / 64;  // 64-element column blocks of a tile (128 rows x 128 bytes)
  extern __shared__ uint8_t at_raw[];
  __shared__ uint64_t full[kAtMaxStages], empty[kAtMaxStages];
  __shared__ uint64_t q_full, q_empty, s_full[2], p_full[2], o_full[2], drain;
  __shared__ uint32_t tmem_holder;
  __shared__ int s_abort, s_b;
  __shared__ long long s_bstart, s_sum[kAtThreads / 32];
  __shared__ float2 s_ml[2][kAtRows];
  __shared__ uint32_t s_bad[2][2][4];  // tree entries of a tile whose V is not finite: by
                                       // turns, half
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(at_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* ring = smem + 2 * kTile;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
  // the run [lo, hi) of this CTA and the sequence it starts in
  const int per = p.Hkv * p.mg_o;
  const long long shared = (long long)p.Hkv * p.mg_s * p.tiles_s;
  long long own = 0;
  for (int b = threadIdx.x; b < p.B; b += kAtThreads) own += attn_tiles(p, b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) own += __shfl_xor_sync(0xffffffffu, own, o);
  if (lane == 0) s_sum[warp] = own;
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  own = 0;
  for (int w = 0; w < kAtThreads / 32; ++w) own += s_sum[w];
  const long long total = shared + own * per;
  const long long lo = total * blockIdx.x / p.nctas, hi = total * (blockIdx.x + 1) / p.nctas;
  {
    long long run = 0;
    for (int b0 = 0; b0 < p.B; b0 += kAtThreads) {
      const int b = b0 + threadIdx.x;
      const long long mine = b < p.B ? attn_tiles(p, b) : 0;
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
      for (int w = 0; w < kAtThreads / 32; ++w) {
        if (w < warp) before += s_sum[w];
        run += s_sum[w];
      }
      const long long excl = before + incl - mine;
      if (b < p.B) {
        if (blockIdx.x == 0) p.tstart[b] = excl;
        if (lo >= shared && lo - shared >= excl * per && lo - shared < (excl + mine) * per) {
          s_b = b;
          s_bstart = shared + excl * per;
        }
      }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) p.tstart[p.B] = run;
  }
  if (threadIdx.x == 0 && lo < shared) s_bstart = shared;
  __syncthreads();
  const uint32_t tmem = tmem_holder;
  AttnWalk walk{lo, hi, s_bstart, s_b};
  AttnSeg seg;
  auto fail = [&]() {
    s_abort = 1;
    set_flag(p.flags, kFlagTimeout);
  };

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- copies ----------------
      int stage = 0, issued = 0;
      unsigned phase = 0, nq = 0;
      bool ok = true;
      while (ok && walk.next(p, &seg)) {
        const bool sh = seg.b < 0;
        const int pair = sh ? p.pair_s : p.pair_o;
        const int cap = p.tok << pair;
        const int tok0 = (sh ? 0 : seg.b * p.N) + seg.mg * cap;
        if (*(volatile int*)&s_abort || !mbar_wait_bounded(&q_empty, (nq & 1) ^ 1u)) {
          fail();
          break;
        }
        mbar_expect_tx(&q_full, (unsigned)((1 + pair) * kSub * p.tok * p.G * 128));
        for (int w = 0; w <= pair; ++w)
          for (int c = 0; c < kSub; ++c)
            tma_load_3d(smem + w * kTile + c * (kAtRows * 128), &map_q, c * 64, seg.h * p.G,
                        tok0 + w * p.tok, &q_full);
        ++nq;
        const CUtensorMap* mk = sh ? &map_pk : &map_k;
        const CUtensorMap* mv = sh ? &map_pv : &map_v;
        auto put = [&](const CUtensorMap* m, int t) {
          if (*(volatile int*)&s_abort || !mbar_wait_bounded(&empty[stage], phase ^ 1u)) {
            ok = false;
            fail();
            return;
          }
          mbar_expect_tx(&full[stage], kTile);
          for (int c = 0; c < kSub; ++c)
            tma_load_4d(ring + stage * kTile + c * (kAtKeys * 128), m, c * 64, seg.h,
                        (seg.t0 + t) * kAtKeys, sh ? 0 : seg.b, &full[stage]);
          ++issued;
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        };
        // in the order of use: each V tile, then the K tile `ahead` further on
        const int ahead = 2 - pair;
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
      unsigned phase = 0, nq = 0, np[2] = {0, 0};
      bool ok = true;
      auto wait = [&](uint64_t* bar, unsigned parity) {
        if (ok && (*(volatile int*)&s_abort || !mbar_wait_bounded(bar, parity))) {
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
      // scores of half w from the K tile in the current stage, query tile qt
      auto scores = [&](int w, int qt) {
        const uint64_t a = qdesc + (uint64_t)(qt * kTile >> 4);
        const uint64_t b = kdesc + (uint64_t)(stage * kTile >> 4);
#pragma unroll
        for (int c = 0; c < kSub; ++c)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t o = (uint64_t)((c * kAtKeys * 128 + kk * 32) >> 4);
            umma_ss(tmem + w * kAtKeys, a + o, b + o, id_qk, (c | kk) ? 1u : 0u);
          }
        umma_commit(&s_full[w]);
      };
      // output of half w from the V tile in stage st
      auto output = [&](int w, int st, bool first) {
        const uint64_t b = vdesc + (uint64_t)(st * kTile >> 4);
#pragma unroll
        for (int kk = 0; kk < kAtKeys / 16; ++kk)
          umma_ts(tmem + 2 * kAtKeys + w * D, tmem + w * kAtKeys + kk * 8,
                  b + (uint64_t)(kk * 2048 >> 4), id_pv, (!first || kk) ? 1u : 0u);
      };
      while (ok && walk.next(p, &seg)) {
        const int pair = seg.b < 0 ? p.pair_s : p.pair_o;
        const int n = seg.n;
        if (!wait(&q_full, nq & 1)) break;
        ++nq;
        if (pair) {
          if (!wait(&full[stage], phase)) break;
          scores(0, 0);
          scores(1, 1);
          umma_commit(&empty[stage]);
          if (n == 1) umma_commit(&q_empty);
          advance();
          for (int t = 0; t < n; ++t) {
            const int vst = stage;
            if (!wait(&full[stage], phase)) break;
            advance();
            if (!wait(&p_full[0], np[0]++ & 1)) break;
            output(0, vst, t == 0);
            if (t + 1 < n) {
              if (!wait(&full[stage], phase)) break;
              scores(0, 0);
            } else {
              umma_commit(&o_full[0]);
            }
            if (!wait(&p_full[1], np[1]++ & 1)) break;
            output(1, vst, t == 0);
            umma_commit(&empty[vst]);
            if (t + 1 < n) {
              scores(1, 1);
              umma_commit(&empty[stage]);
              if (t + 2 == n) umma_commit(&q_empty);
              advance();
            } else {
              umma_commit(&o_full[1]);
            }
          }
        } else {
          for (int t = 0; t < min(2, n); ++t) {
            if (!wait(&full[stage], phase)) break;
            scores(t, 0);
            umma_commit(&empty[stage]);
            if (t + 1 == n) umma_commit(&q_empty);
            advance();
          }
          for (int t = 0; ok && t < n; ++t) {
            const int w = t & 1, vst = stage;
            if (!wait(&full[stage], phase)) break;
            advance();
            if (!wait(&p_full[w], np[w]++ & 1)) break;
            output(w, vst, t < 2);
            umma_commit(&empty[vst]);
            if (t + 2 < n) {
              if (!wait(&full[stage], phase)) break;
              scores(w, 0);
              umma_commit(&empty[stage]);
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
    const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
    const uint32_t sbase = lanes + w * kAtKeys;
    unsigned ns = 0, no = 0;  // uses of s_full / o_full so far
    long long ring0 = 0;      // ring uses before this segment
    bool dead = false;        // a wait gave up: only the barriers are kept up
    auto wait = [&](uint64_t* bar, unsigned parity) {
      if (!dead && (*(volatile int*)&s_abort || !mbar_wait_bounded(bar, parity))) {
        dead = true;
        fail();
      }
      dead = __any_sync(0xffffffffu, dead);  // the warp decides as one
      tmem_fence_after();
    };
    while (walk.next(p, &seg)) {
      const bool sh = seg.b < 0;
      const int pair = sh ? p.pair_s : p.pair_o;
      const int cap = p.tok << pair;
      const int ntok = (sh ? p.B * p.N : p.N) - seg.mg * cap - (pair ? w * p.tok : 0);
      const int nrows = max(0, min(p.tok, ntok)) * p.G;  // rows of this half in use
      const bool busy = quad * 32 < nrows;               // whole warps of unused rows only wait
      const int nt = pair ? seg.n : (seg.n + 1 - w) / 2;
      const int node = seg.mg * cap + (pair ? w * p.tok : 0) + r / p.G;  // own items: the row's
      float m = -INFINITY, l = 0.0f;
      for (int i = 0; i < nt; ++i) {
        const int t = pair ? i : 2 * i + w;
        const int key0 = (seg.t0 + t) * kAtKeys;
        const bool edge = key0 + kAtKeys > seg.plen;  // not all of the tile is seen by all
        wait(&s_full[w], ns++ & 1);
        uint32_t see[4];
        bool spoilt = false;
        if (edge) {
          // V entries beyond the last are zeroed, whatever they hold: their
          // products with weights of 0 have to be 0.  So are tree entries that
          // are not finite, and the rows that see them become NaN.
          if (!pair || w == 0) {
            const long long u = ring0 + min(seg.n, t + 2 - pair) + t;  // V tile's ring use
            const int st = (int)(u % S);
            wait(&full[st], (unsigned)((u / S) & 1));
            const int at = key0 + r;
            bool bad = false;
            if (!dead && at >= seg.plen) {
              uint8_t* row = ring + st * kTile + r * 128;
              if (at < seg.kvlen) {
#pragma unroll
                for (int c = 0; c < kSub; ++c)
#pragma unroll
                  for (int j = 0; j < 8; ++j) {
                    const uint4 x = lds128(row + c * (kAtKeys * 128) + j * 16);
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
                    *reinterpret_cast<uint4*>(row + c * (kAtKeys * 128) + j * 16) =
                        make_uint4(0, 0, 0, 0);
              }
            }
            const unsigned any = __ballot_sync(0xffffffffu, bad);
            if (lane == 0) s_bad[i & 1][w][quad] = any;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          if (pair)
            asm volatile("bar.sync 2, 256;" ::: "memory");
          else
            asm volatile("bar.sync %0, 128;" ::"r"(3 + w) : "memory");
          // the row's view of the tile, 32 entries per word
          const int tree0 = key0 - seg.plen;  // tree number of the tile's first entry
          const uint32_t* mrow = !sh && p.mask && node < p.N
                                     ? p.mask + ((size_t)seg.b * p.N + node) * p.W : nullptr;
          auto word = [&](int j) -> uint32_t {  // tree entries 32 j .. that the node sees
            if (j < 0) return 0xFFFFFFFFu;
            if (sh || j >= p.W) return 0u;
            uint32_t x;
            if (p.mask) {
              x = mrow ? __ldg(mrow + j) : 0u;
            } else {
              const int c = node + 1 - 32 * j;
              x = c >= 32 ? 0xFFFFFFFFu : c <= 0 ? 0u : (1u << c) - 1u;
            }
            const int left = p.N - 32 * j;
            return left < 32 ? x & ((1u << left) - 1u) : x;
          };
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int u = tree0 + 32 * c;
            see[c] = __funnelshift_r(word(u >> 5), word((u >> 5) + 1), u & 31);
            spoilt |= (see[c] & s_bad[i & 1][pair ? 0 : w][c]) != 0;
          }
        }
        if (busy && !dead) {
          uint32_t s0[32], s1[32], s2[32], s3[32];
          tmem_ld32_async(sbase, s0);
          tmem_ld32_async(sbase + 32, s1);
          tmem_ld32_async(sbase + 64, s2);
          tmem_ld32_async(sbase + 96, s3);
          tmem_wait_ld(s0);
          tmem_wait_ld(s1);
          tmem_wait_ld(s2);
          tmem_wait_ld(s3);
          if (edge) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              if (!((see[0] >> j) & 1)) s0[j] = 0xFF800000u;
              if (!((see[1] >> j) & 1)) s1[j] = 0xFF800000u;
              if (!((see[2] >> j) & 1)) s2[j] = 0xFF800000u;
              if (!((see[3] >> j) & 1)) s3[j] = 0xFF800000u;
            }
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            mx[0] = fmaxf(fmaxf(mx[0], __uint_as_float(s0[j])), __uint_as_float(s0[j + 1]));
            mx[1] = fmaxf(fmaxf(mx[1], __uint_as_float(s1[j])), __uint_as_float(s1[j + 1]));
            mx[2] = fmaxf(fmaxf(mx[2], __uint_as_float(s2[j])), __uint_as_float(s2[j + 1]));
            mx[3] = fmaxf(fmaxf(mx[3], __uint_as_float(s3[j])), __uint_as_float(s3[j + 1]));
          }
          const float top = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2,
                                  -1e30f);
          if (i == 0) {
            m = top;
          } else if (__any_sync(0xffffffffu, top > m + kAtLazy)) {
            // rescale this row's output; the tile before this one is in it
            // (its product was issued before this tile's scores)
            const float mn = fmaxf(m, top), f = ex2(m - mn);
            m = mn;
            l *= f;
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
          // weights of 16 entries at a time, into 8 columns
          const unsigned long long c2 = f2pack(p.scale_log2, p.scale_log2), nm2 = f2pack(-m, -m);
          unsigned long long sum0 = 0, sum1 = 0;
          auto weights = [&](const uint32_t (&a)[32], uint32_t at) {
            uint32_t pk[16];
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              float x, y, z, u;
              f2unpack(fma2(f2pack(__uint_as_float(a[2 * j]), __uint_as_float(a[2 * j + 1])), c2, nm2), x, y);
              f2unpack(fma2(f2pack(__uint_as_float(a[2 * j + 2]), __uint_as_float(a[2 * j + 3])), c2, nm2), z, u);
              x = ex2(x);
              y = ex2(y);
              z = ex2(z);
              u = ex2(u);
              sum0 = add2(sum0, f2pack(x, y));
              sum1 = add2(sum1, f2pack(z, u));
              pk[j] = pack_bf16(x, y);
              pk[j + 1] = pack_bf16(z, u);
            }
            tmem_st16(at, pk);
          };
          weights(s0, sbase);
          weights(s1, sbase + 16);
          weights(s2, sbase + 32);
          weights(s3, sbase + 48);
          float a0, a1;
          f2unpack(add2(sum0, sum1), a0, a1);
          l += spoilt ? NAN : a0 + a1;
          tmem_wait_st();
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[w]);
      }
      ring0 += 2 * seg.n;
      // the item's output, or its partial as [D / 4][slot_rows][4], so that a
      // warp's lanes (rows) store 512 consecutive bytes
      if (nt > 0) wait(&o_full[w], no++ & 1);
      const bool mine = r < nrows;
      float* slot = p.opart + seg.slot * (long long)p.slot_rows * D;
      const int row = (pair ? w * p.half_rows : 0) + r;
      const size_t orow = ((size_t)max(seg.b, 0) * p.N + node) * p.Hq + seg.h * p.G + r % p.G;
      auto put = [&](int c, const uint32_t (&o)[16], float norm) {
        if (!mine) return;
        if (seg.whole) {
          uint32_t x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            x[j] = pack_bf16(__uint_as_float(o[2 * j]) * norm, __uint_as_float(o[2 * j + 1]) * norm);
          uint4* dst = reinterpret_cast<uint4*>(p.out + orow * D + c);
          dst[0] = make_uint4(x[0], x[1], x[2], x[3]);
          dst[1] = make_uint4(x[4], x[5], x[6], x[7]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(slot + ((c / 4 + j) * p.slot_rows + row) * 4) =
                make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        }
      };
      auto put_ml = [&](float mm, float ll) {
        if (!mine) return;
        if (!seg.whole)
          p.ml[seg.slot * p.slot_rows + row] = make_float2(mm, ll);
        else if (p.lse)
          p.lse[orow] = attn_lse(mm, ll);
      };
      if (pair) {
        if (busy && !dead) {
          const float norm = attn_norm(l);
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            tmem_ld16(lanes + 2 * kAtKeys + w * D + c, o);
            put(c, o, norm);
          }
          put_ml(m, l);
        }
        tmem_fence_before();
      } else {
        // join the two halves; each takes half of the columns
        s_ml[w][r] = make_float2(m, l);
        asm volatile("bar.sync 1, 256;" ::: "memory");
        tmem_fence_after();
        if (busy && !dead) {
          const float2 a = s_ml[0][r], b = s_ml[1][r];  // half 0 has at least one tile
          const float mm = fmaxf(a.x, b.x);
          const float fa = ex2(a.x - mm), fb = ex2(b.x - mm);
          const float ll = seg.n > 1 ? a.y * fa + b.y * fb : a.y;
          const float norm = attn_norm(ll);
#pragma unroll 1
          for (int c = w * (D / 2); c < (w + 1) * (D / 2); c += 16) {
            uint32_t o[16];
            tmem_ld16(lanes + 2 * kAtKeys + c, o);
            if (seg.n > 1) {
              uint32_t o1[16];
              tmem_ld16(lanes + 2 * kAtKeys + D + c, o1);
#pragma unroll
              for (int j = 0; j < 16; ++j)
                o[j] = __float_as_uint(
                    __fmaf_rn(__uint_as_float(o1[j]), fb, __uint_as_float(o[j]) * fa));
            }
            put(c, o, norm);
          }
          if (w == 0) put_ml(mm, ll);
        }
        // neither half's accumulators are written again before both are read
        tmem_fence_before();
        asm volatile("bar.sync 1, 256;" ::: "memory");
      }
    }
  }
  tmem_fence_before();
  __syncthreads();
  if (warp == 1) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

// Joins the partials of items that several CTAs share or that have a shared
// prefix; other rows are done.  One warp per (node, key-value head),
// kAtFinHeads query heads at a time, a lane holding D / 32 elements of a head.
template <int D>
__global__ void __launch_bounds__(kAtFinThreads) tree_attn_finish_kernel(const AttnParams p) {
  constexpr int kE = D / 32;  // elements per lane
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * (kAtFinThreads / 32) + warp;
  if (item >= (long long)p.B * p.N * p.Hkv) return;
  const int h = (int)(item % p.Hkv);
  const long long node = item / p.Hkv;
  const int b = (int)(node / p.N), n = (int)(node - (long long)b * p.N);
  const bool ok = attn_seq_ok(p, __ldg(p.base_len + b));
  if (!ok && n == 0 && h == 0 && lane == 0) set_flag(p.flags, kFlagBadPath);
  // per class (shared prefix, own entries): the partials' first slot, the run
  // of CTAs, and the row in the slot
  long long it[2], total = 1;
  int c0[2] = {0, 0}, c1[2] = {0, 0}, row[2];
  if (ok) {
    const long long items_s = (long long)p.Hkv * p.mg_s, per = (long long)p.Hkv * p.mg_o;
    const long long shared = items_s * p.tiles_s;
    total = shared + p.tstart[p.B] * per;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const long long tiles = k == 0 ? p.tiles_s : p.tstart[b + 1] - p.tstart[b];
      if (tiles == 0) continue;
      const int cap = p.tok << (k == 0 ? p.pair_s : p.pair_o);
      const int tokn = k == 0 ? (int)node : n;
      const int mg = tokn / cap, in = tokn - mg * cap;
      const int half = in / p.tok;
      const int index = mg * p.Hkv + h;
      row[k] = half * p.half_rows + (in - half * p.tok) * p.G;
      it[k] = k == 0 ? index : items_s + (long long)b * per + index;
      const long long s0 = k == 0 ? index * tiles
                                  : shared + p.tstart[b] * per + (long long)index * tiles;
      // the CTAs whose runs [c T / n, (c+1) T / n) meet the item's tiles
      int c = (int)(s0 * p.nctas / total);
      while (total * (c + 1) / p.nctas <= s0) ++c;
      c0[k] = c;
      while (c < p.nctas && total * c / p.nctas < s0 + tiles) ++c;
      c1[k] = c;
    }
    if (p.tiles_s == 0 && c1[1] - c0[1] == 1) return;  // written by its only CTA
  }
  for (int g0 = 0; g0 < p.G; g0 += kAtFinHeads) {
    const int ng = min(kAtFinHeads, p.G - g0);
    float acc[kAtFinHeads][kE], m[kAtFinHeads], l[kAtFinHeads];
#pragma unroll
    for (int g = 0; g < kAtFinHeads; ++g) {
      m[g] = -1e30f;
      l[g] = 0.0f;
#pragma unroll
      for (int e = 0; e < kE; ++e) acc[g][e] = 0.0f;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      for (int c = c0[k]; c < c1[k]; ++c) {
        if (total * c / p.nctas == total * (c + 1) / p.nctas) continue;  // an empty run
        const long long slot = it[k] + c;
        const float* part = p.opart + slot * (long long)p.slot_rows * D;
        const float2* ml = p.ml + slot * p.slot_rows + row[k] + g0;
#pragma unroll
        for (int g = 0; g < kAtFinHeads; ++g) {
          if (g < ng) {
            const float2 x = ml[g];
            float o[kE];
            if constexpr (kE == 4) {
              const float4 y = *reinterpret_cast<const float4*>(
                  part + ((size_t)lane * p.slot_rows + row[k] + g0 + g) * 4);
              o[0] = y.x; o[1] = y.y; o[2] = y.z; o[3] = y.w;
            } else {
              const float2 y = *reinterpret_cast<const float2*>(
                  part + ((size_t)(lane >> 1) * p.slot_rows + row[k] + g0 + g) * 4 + (lane & 1) * 2);
              o[0] = y.x; o[1] = y.y;
            }
            const float mn = fmaxf(m[g], x.x);
            const float fa = ex2(m[g] - mn), fb = ex2(x.x - mn);
            m[g] = mn;
            l[g] = l[g] * fa + x.y * fb;
#pragma unroll
            for (int e = 0; e < kE; ++e) acc[g][e] = acc[g][e] * fa + o[e] * fb;
          }
        }
      }
    }
#pragma unroll
    for (int g = 0; g < kAtFinHeads; ++g) {
      if (g < ng) {
        const float rl = attn_norm(l[g]);
        const size_t at = (size_t)node * p.Hq + h * p.G + g0 + g;
        if constexpr (kE == 4) {
          *reinterpret_cast<uint2*>(p.out + at * D + lane * 4) =
              make_uint2(pack_bf16(acc[g][0] * rl, acc[g][1] * rl),
                         pack_bf16(acc[g][2] * rl, acc[g][3] * rl));
        } else {
          *reinterpret_cast<uint32_t*>(p.out + at * D + lane * 2) =
              pack_bf16(acc[g][0] * rl, acc[g][1] * rl);
        }
        if (p.lse && lane == 0) p.lse[at] = attn_lse(m[g], l[g]);
      }
    }
  }
}

}  // namespace sv
