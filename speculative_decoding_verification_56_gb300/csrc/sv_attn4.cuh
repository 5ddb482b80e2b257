// sv_attn4.cuh -- attention of drafted trees over a 4-bit cache in pages, for
// few rows (a node's query heads of one key-value head) per sequence.
//
//   out = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q . k_j),
//
// over the committed positions in the pages and the nodes that the mask names.
// S = K Q^T and O = V^T P are matrix instructions of 16 entries (channels) by 8
// rows from registers: with 8 to 24 rows, tiles of 128 would be mostly padding,
// and entries would be written to shared memory and read back.  Both operands of
// codes are unpacked into registers from the packed bytes, whose 16 positions of a
// group are placed so that the thread that reads a 4- or 8-byte piece holds what
// its fragment needs; what a product sums over (channels for S, positions for O)
// may come in any order that both its operands share.  P becomes the second
// product's operand by one transposition in registers.
//
// The work is cut into equal runs of 256 positions over two CTAs an SM (one for
// more than 8 rows), whatever the lengths; in a CTA each warp has its own 32
// positions of a run's step, its own ring of bulk copies (nobody waits for a
// producer), reference, sum and output, joined at the item's end; items that
// several CTAs share leave float32 partials for kv4_attn_finish_kernel.  The
// softmax reference is renewed only when a score passes it by 2^kA4Lazy.  Sums,
// references and outputs are float32; weights are rounded to fp16 (2^-11 of a
// weight, or 2^-32 of the largest), queries, brought into its range by a power of
// two per row, lose bits only in elements below 2^-31 of the row's largest.
//
// Bound: latency.  A warp's 32 positions are about 700 instructions at D = 128
// (unpacking, scaling and products), one chain of wait, unpack, product, exponentials,
// unpack, product, and registers leave four warps a scheduler to overlap them (two
// from 9 rows on).  Decoding, while an SM is busy: 54% of the issue slots, the integer
// and logic unit, the busiest, 48%, DRAM 43%; of 6.9 cycles between a warp's
// instructions 1.5 are waits for results of fixed latency, 1.0 barriers of the joins,
// 0.8 a busy unit, 0.5 loads; and SMs are busy for 84% of the kernel's time.
// Measured: decoding 64 sequences of up to 4096 positions, 32 heads of 8, 69-72 us
// where the packed bytes (229 MB) take 34 at the copy rate and the bf16 cache takes
// its kernel 134 (D = 64: 52, 17 and 110); 16 positions a step 104 us, 32 with more
// registers 77.  Chains of 3 and 4 nodes (12 and 16 rows) 113 us, of 5 and 6 (20 and
// 24) 140 (the bf16 cache 136 and 138; D = 64: 87 and 105, 112 and 113).  One chain of 5
// over 300 positions: 10.6 us of kernels.
#pragma once

#include "sv_attn.cuh"
#include "sv_kv4.cuh"

namespace sv {

constexpr int kA4Warps = 8;
constexpr int kA4Step = 32;  // positions that a warp takes at once: two products' 16 entries
constexpr int kA4Tile = kA4Warps * kA4Step;
constexpr int kA4Threads = kA4Warps * 32;
constexpr int kA4MaxCtas = 320;
constexpr float kA4Off = 7.0f;   // weights are held 2^7 times as large: fp16 then has them down
                                 // to 2^-31 of the reference
constexpr float kA4Lazy = 8.0f;  // a score (log2) above its row's reference by more renews it

struct Attn4Params {
  const uint16_t* q;        // [B, N, Hq, D]
  const uint8_t* pages;     // [n_pages, Hkv, block]
  const int32_t* table;     // [B, W]
  const uint16_t* nk;       // [B, N, Hkv, D]
  const uint16_t* nv;
  const uint32_t* mask;     // [B, N, Wm] or null (a chain)
  const int32_t* base_len;  // [B]
  const int32_t* exps;      // [2] or null
  uint16_t* out;            // [B, N, Hq, D]
  float* lse;               // [B, N, Hq] or null
  unsigned* flags;
  float* opart;             // [slot][row][D]
  float2* ml;               // [slot][row]: reference (log2) and sum
  int2* span;               // [items]: first and last CTA that holds a part of the item
  unsigned long long wait_ns;
  long long n_pages;
  float scale_log2;         // scale * log2(e)
  int B, N, Hq, Hkv, G, W, Wm, lg;
  int rows;                 // N G, at most 8 NT: rows of an item (a sequence's key-value head)
  int nctas;
};

// Committed positions of a sequence that can be attended to, or -1.
__device__ __forceinline__ int attn4_len(const Attn4Params& p, int base) {
  return base >= 1 && (long long)base - 1 <= ((long long)p.W << p.lg) ? base - 1 : -1;
}
// Units of work of an item: tiles of committed positions, the first of them together
// with the nodes (kA4Warps times 16 at most).
__device__ __forceinline__ int attn4_units(const Attn4Params& p, int base) {
  const int len = attn4_len(p, base);
  return len < 0 ? 0 : max(1, len / kA4Tile + (len % kA4Tile != 0));
}

// A CTA's run of units is cut into segments, one per item it meets.
struct Attn4Seg {
  int b, h;               // sequence, key-value head
  int t0, n, len;         // units, committed positions
  int slot, whole;        // partial's slot; whole: all units of the item
};
struct Attn4Walk {
  long long pos, hi, bstart;  // bstart: first unit of sequence b in the line
  int b;
  __device__ __forceinline__ bool next(const Attn4Params& p, Attn4Seg* s, bool writes) {
    if (pos >= hi) return false;
    const int per = p.Hkv;
    int base = p.base_len[b];
    int units = attn4_units(p, base);
    while (pos >= bstart + (long long)per * units) {
      bstart += (long long)per * units;
      base = p.base_len[++b];
      units = attn4_units(p, base);
    }
    const int it = (int)((pos - bstart) / units);
    s->t0 = (int)(pos - bstart - (long long)it * units);
    s->n = (int)min((long long)(units - s->t0), hi - pos);
    s->b = b;
    s->h = it;
    s->len = base - 1;
    s->slot = 2 * blockIdx.x + (s->t0 == 0);
    s->whole = s->n == units;
    if (writes) {
      const long long item = (long long)b * per + it;
      if (s->t0 == 0) p.span[item].x = blockIdx.x;
      if (s->t0 + s->n == units) p.span[item].y = blockIdx.x;
    }
    pos += s->n;
    return true;
  }
};

// scale 2^e, kept finite and above 0 (where it would not be, products are 0 or
// scores beyond their limit), so that its products with 0 and -inf are right
__device__ __forceinline__ float score_unit(float scale, int e) {
  return fminf(fmaxf(ldexpf(scale, e), 1.2e-38f), 1e38f);
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  return __byte_perm(a, b, sel);
}
__device__ __forceinline__ uint32_t mov_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
      " {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// whether one of two bf16 is not finite
__device__ __forceinline__ bool bf16_inf(uint32_t x) {
  return (x & 0x7F80u) == 0x7F80u || (x & 0x7F800000u) == 0x7F800000u;
}
// two bf16 times f (a power of two) as two fp16, saturating; bad: one is not finite
__device__ __forceinline__ uint32_t node_half2(uint32_t x, float f, bool& bad) {
  bad |= bf16_inf(x);
  const float lo = fminf(fmaxf(bf16_lo(x) * f, -65504.0f), 65504.0f);
  const float hi = fminf(fmaxf(bf16_hi(x) * f, -65504.0f), 65504.0f);
  return pack_half(lo, hi);
}

template <int D, int NT>
__host__ __device__ constexpr int a4_q_bytes() { return NT * 8 * (D * 2 + 16); }
template <int D, int NT>
__host__ __device__ constexpr int a4_red_bytes() { return kA4Warps / 2 * NT * 8 * D * 4; }
template <int NT>
__host__ __device__ constexpr int a4_per_sm() { return NT == 1 ? 2 : 1; }
// Steps of kA4Step positions that each warp has in shared memory: what fits
// beside the queries, the join's buffer and the static arrays
template <int D, int NT>
__host__ __device__ constexpr int a4_stages() {
  const int room = 232448 / a4_per_sm<NT>() - 1024 - 4096 - a4_q_bytes<D, NT>() - a4_red_bytes<D, NT>();
  const int fit = room / (kA4Warps * 2 * kv4_group(D));
  return fit < 4 ? fit : 4;
}
template <int D, int NT>
__host__ __device__ constexpr int a4_smem() {
  return a4_stages<D, NT>() * kA4Warps * 2 * kv4_group(D) + a4_q_bytes<D, NT>() + a4_red_bytes<D, NT>();
}

template <int D, int NT>
__global__ void __launch_bounds__(kA4Threads, a4_per_sm<NT>())
    kv4_attn_rows_kernel(const Attn4Params p) {
  constexpr int kSteps = D / 16;  // k-steps of S, m-tiles of O
  constexpr int kCh = D / 4;      // channels of a row that a thread multiplies for S
  constexpr int kCv = D / 8;      // channels of a position that it multiplies for O
  constexpr int kQStride = D * 2 + 16;  // bytes of a query row: neighbouring rows in other banks
  constexpr int kGroup = kv4_group(D);
  constexpr int kStages = a4_stages<D, NT>();
  constexpr int kStage = 2 * kGroup;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ uint64_t full[kA4Warps][kStages];
  __shared__ Attn4Walk s_walk[kA4Warps], s_at[kA4Warps];  // of the copies, and of the products
  __shared__ Attn4Seg s_seg[kA4Warps];
  __shared__ long long s_sum[kA4Warps], s_bstart;
  __shared__ int s_b;
  __shared__ float s_m[kA4Warps][NT * 8], s_l[kA4Warps][NT * 8];
  __shared__ float s_fac[NT * 8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = smem + warp * (kStages * kStage);
  uint8_t* s_q = smem + kA4Warps * kStages * kStage;
  float* s_red = reinterpret_cast<float*>(s_q + a4_q_bytes<D, NT>());
  if (lane == 0)
    for (int s = 0; s < kStages; ++s) mbar_init(&full[warp][s], 1);
  if (threadIdx.x == 0) {
    s_b = 0;
    s_bstart = 0;
  }
  mbar_init_fence();
  // a programmatic dependent of the kernel before it in the stream: nothing of
  // global memory is touched before that grid has finished
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  // the run [lo, hi) of this CTA and the sequence it starts in
  const int per = p.Hkv;
  int mine = (int)threadIdx.x < p.B ? attn4_units(p, p.base_len[threadIdx.x]) : 0;
  long long sum = mine;
  for (int b = threadIdx.x + kA4Threads; b < p.B; b += kA4Threads)
    sum += attn4_units(p, p.base_len[b]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  sum = 0;
#pragma unroll
  for (int w = 0; w < kA4Warps; ++w) sum += s_sum[w];
  const long long total = sum * per;
  const int n = (int)min((long long)p.nctas, total);  // no run is empty; other CTAs have none
  const long long lo = (int)blockIdx.x < n ? total * blockIdx.x / n : 0;
  const long long hi = (int)blockIdx.x < n ? total * (blockIdx.x + 1) / n : 0;
  {
    long long run = 0;
    for (int b0 = 0; b0 < p.B; b0 += kA4Threads) {
      const int b = b0 + threadIdx.x;
      if (b0 > 0) mine = b < p.B ? attn4_units(p, p.base_len[b]) : 0;
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
      for (int w = 0; w < kA4Warps; ++w) {
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
  const int page = 1 << p.lg;

  // ---------------- copies ----------------
  // Each warp brings in its own steps, kStages ahead of their use: nobody waits
  // for another warp before the end of an item.  c_at: the next step's first
  // position in the sequence, up to c_end; lane j < 2 brings in its positions 16 j ..,
  // whose page c_id was looked up one step ahead.
  int c_at = 0, c_end = 0, c_h = 0, c_id = -1;
  const int32_t* c_row = p.table;
  unsigned holes = 0;  // bits 2 s, 2 s + 1: stage s's positions have no page; 16 + s: it is in use
  bool dead = false;  // a wait was given up: go on without work, so that all barriers are met
  if (lane == 0) s_walk[warp] = s_at[warp] = Attn4Walk{lo, hi, s_bstart, s_b};
  __syncwarp();
  auto look_up = [&]() {  // -2: no position there
    const int at = c_at + 16 * lane;
    c_id = lane < 2 && at < c_end ? c_row[at >> p.lg] : -2;
  };
  auto next_item = [&]() {  // the next one with a step for this warp; false: none
    Attn4Walk w = s_walk[warp];
    __syncwarp();
    Attn4Seg s;
    bool some = false;
    while (!some && w.next(p, &s, warp == 0 && lane == 0)) {
      c_at = s.t0 * kA4Tile + warp * kA4Step;
      c_end = min(s.len, (s.t0 + s.n) * kA4Tile);
      c_h = s.h;
      c_row = p.table + (size_t)s.b * p.W;
      some = c_at < c_end;
    }
    if (lane == 0) s_walk[warp] = w;
    __syncwarp();
    if (some) look_up();
    return some;
  };
  auto refill = [&](int st) {
    if (c_at >= c_end && !next_item()) return;
    const bool ok = c_id >= 0 && c_id < p.n_pages;
    const unsigned some = __ballot_sync(0xffffffffu, ok);
    const unsigned none = __ballot_sync(0xffffffffu, !ok && c_id != -2);
    if (none && lane == 0) set_flag(p.flags, kFlagBadPage);
    holes = (holes & ~(3u << (2 * st))) | (none << (2 * st)) | (0x10000u << st);
    if (lane == 0) mbar_expect_tx(&full[warp][st], __popc(some) * kGroup);
    __syncwarp();
    if (ok)
      bulk_g2s(ring + st * kStage + lane * kGroup,
               p.pages + ((size_t)c_id * p.Hkv + c_h) * kv4_block(page, D) +
                   (((c_at + 16 * lane) & (page - 1)) >> 4) * kGroup,
               kGroup, &full[warp][st]);
    c_at += kA4Tile;
    look_up();
  };
  for (int s = 0; s < kStages; ++s) refill(s);

  // ---------------- products ----------------
  const int g = lane >> 2, t = lane & 3;
  const int kexp = kv4_exp(p.exps, 0), vexp = kv4_exp(p.exps, 1);
  const float kinv = pow2_small(-kexp), vinv = pow2_small(-vexp);
  const int pi = ((g >> 1) & 3) + 4 * (g & 1);  // place of product row g among the warp's 16
  int stage = 0;
  unsigned phase = 0;
  auto meet = [&]() { __syncthreads(); };

  // (a warp's walk and item stand in shared memory: the loop below has no registers
  // to spare for them)
  Attn4Seg& seg = s_seg[warp];
  for (;;) {
    __syncwarp();
    if (lane == 0) {
      Attn4Walk w = s_at[warp];
      if (!w.next(p, &seg, false)) seg.n = 0;
      s_at[warp] = w;
    }
    __syncwarp();
    if (seg.n == 0) break;
    // queries as fp16, each row times a power of two that brings its largest
    // element to [2^14, 2^15)
    for (int r = warp; r < NT * 8; r += kA4Warps) {
      const bool in = r < p.rows;
      const int v = r / p.G;
      uint32_t x[D / 64];
#pragma unroll
      for (int j = 0; j < D / 64; ++j)
        x[j] = in ? *reinterpret_cast<const uint32_t*>(
                        p.q + (((size_t)seg.b * p.N + v) * p.Hq + seg.h * p.G + (r - v * p.G)) * D +
                        j * 64 + lane * 2)
                  : 0u;
      uint32_t a = 0;
#pragma unroll
      for (int j = 0; j < D / 64; ++j) a = max(a, max(x[j] & 0x7FFFu, (x[j] >> 16) & 0x7FFFu));
      a = __reduce_max_sync(0xffffffffu, a);
      const int e = a == 0 || a >= 0x7F80u ? 0 : 14 - ilogbf(__uint_as_float(a << 16));
      const float bad = a >= 0x7F80u ? __int_as_float(0x7FC00000) : 0.0f;
#pragma unroll
      for (int j = 0; j < D / 64; ++j)
        *reinterpret_cast<uint32_t*>(s_q + r * kQStride + (j * 64 + lane * 2) * 2) =
            pack_half(ldexpf(bf16_lo(x[j]), e) + bad, ldexpf(bf16_hi(x[j]), e) + bad);
      if (lane == 0) s_fac[r] = score_unit(p.scale_log2, kexp - e);
    }
    meet();
    uint32_t qf[NT][kSteps][2];
    float fac[NT][2], m[NT][2], l[NT][2];
    int vis[NT][2];  // node of the thread's two rows of each n-tile
    float o[NT][kSteps][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        const uint2 x = *reinterpret_cast<const uint2*>(s_q + (8 * i + g) * kQStride + (kCh * t + 4 * j) * 2);
        qf[i][j][0] = x.x;
        qf[i][j][1] = x.y;
        o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.0f;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        fac[i][c] = s_fac[8 * i + 2 * t + c];
        m[i][c] = -1e30f;
        l[i][c] = 0.0f;
        vis[i][c] = min(8 * i + 2 * t + c, p.rows - 1) / p.G;
      }
    }
    // products of 16 entries a time (rows g, g + 8), hidden ones -inf, to weights;
    // renews references that their scores outgrow
    auto weights = [&](auto& s, auto& w) {
      constexpr int kTimes = sizeof(s) / sizeof(s[0]);
      float top = -INFINITY;
      float mo[NT][2];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          mo[i][c] = kA4Off - m[i][c];
#pragma unroll
          for (int q = 0; q < kTimes; ++q)
            top = fmaxf(top, fmaf(fmaxf(s[q][i][c], s[q][i][c + 2]), fac[i][c], mo[i][c]));
        }
      if (__any_sync(0xffffffffu, top > kA4Off + kA4Lazy)) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x = fmaxf(s[0][i][c], s[0][i][c + 2]);
#pragma unroll
            for (int q = 1; q < kTimes; ++q) x = fmaxf(x, fmaxf(s[q][i][c], s[q][i][c + 2]));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
            const float mn = fmaxf(m[i][c], x * fac[i][c]);
            const float f = ex2(m[i][c] - mn);
            m[i][c] = mn;
            mo[i][c] = kA4Off - mn;
            l[i][c] *= f;
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
              o[i][j][c] *= f;
              o[i][j][c + 2] *= f;
            }
          }
      }
#pragma unroll
      for (int q = 0; q < kTimes; ++q)
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          float e[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) e[c] = ex2(fmaf(s[q][i][c], fac[i][c & 1], mo[i][c & 1]));
          l[i][0] += e[0] + e[2];
          l[i][1] += e[1] + e[3];
          w[q][i][0] = mov_trans(pack_half(e[0], e[1]));
          w[q][i][1] = mov_trans(pack_half(e[2], e[3]));
        }
    };

    // ---- 16 nodes ----
    const int u0 = warp * 16;
    if (seg.t0 == 0 && u0 < p.N) {
      const size_t node0 = (size_t)seg.b * p.N;
      const size_t stride = (size_t)p.Hkv * D;
      float s[1][NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i) s[0][i][0] = s[0][i][1] = s[0][i][2] = s[0][i][3] = 0.0f;
      const int n0 = u0 + pi, n1 = n0 + 8;
      bool bad0 = false, bad1 = false;
      {
        const uint16_t* k0 = p.nk + (node0 + min(n0, p.N - 1)) * stride + seg.h * D + kCh * t;
        const uint16_t* k1 = p.nk + (node0 + min(n1, p.N - 1)) * stride + seg.h * D + kCh * t;
#pragma unroll
        for (int j = 0; j < kSteps; j += 2) {
          const uint4 x = *reinterpret_cast<const uint4*>(k0 + 4 * j);
          const uint4 y = *reinterpret_cast<const uint4*>(k1 + 4 * j);
          const uint32_t a0[4] = {node_half2(x.x, kinv, bad0), node_half2(y.x, kinv, bad1),
                                  node_half2(x.y, kinv, bad0), node_half2(y.y, kinv, bad1)};
          const uint32_t a1[4] = {node_half2(x.z, kinv, bad0), node_half2(y.z, kinv, bad1),
                                  node_half2(x.w, kinv, bad0), node_half2(y.w, kinv, bad1)};
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            mma_16816(s[0][i], a0, qf[i][j][0], qf[i][j][1]);
            mma_16816(s[0][i], a1, qf[i][j + 1][0], qf[i][j + 1][1]);
          }
        }
      }
      // values: this thread's four nodes 4 i + t of the 16, channels kCv g ..;
      // looked at first, and loaded once more for their product
      const uint16_t* vrow[4];
      unsigned badv = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        vrow[i] = p.nv + (node0 + min(u0 + 4 * i + t, p.N - 1)) * stride + seg.h * D + kCv * g;
        bool bad = false;
#pragma unroll
        for (int c = 0; c < kCv; c += 8) {
          const uint4 x = *reinterpret_cast<const uint4*>(vrow[i] + c);
          bad |= bf16_inf(x.x) || bf16_inf(x.y) || bf16_inf(x.z) || bf16_inf(x.w);
        }
        badv |= bad ? 1u << (4 * i + t) : 0u;
      }
      // entries with an element that is not finite: their values count as 0
      // here, and the scores of the rows that see them become NaN
      badv |= (bad0 ? 1u << pi : 0u) | (bad1 ? 1u << (pi + 8) : 0u);
      badv = __reduce_or_sync(0xffffffffu, badv);
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int v = vis[i][e & 1], nn = e < 2 ? n0 : n1;
          bool see = nn < p.N;
          if (see)
            see = p.mask ? (p.mask[(node0 + v) * p.Wm + (nn >> 5)] >> (nn & 31)) & 1 : nn <= v;
          const bool bad = (badv >> (e < 2 ? pi : pi + 8)) & 1;
          if (!see || bad) s[0][i][e] = see ? __int_as_float(0x7FC00000) : -INFINITY;
        }
      uint32_t w[1][NT][2];
      weights(s, w);
#pragma unroll
      for (int c = 0; c < kCv; c += 8) {
        uint32_t h[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4 x = *reinterpret_cast<const uint4*>(vrow[i] + c);
          if ((badv >> (4 * i + t)) & 1) x = make_uint4(0, 0, 0, 0);
          bool dummy = false;
          h[i][0] = node_half2(x.x, vinv, dummy);
          h[i][1] = node_half2(x.y, vinv, dummy);
          h[i][2] = node_half2(x.z, vinv, dummy);
          h[i][3] = node_half2(x.w, vinv, dummy);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t a[4] = {prmt(h[0][j], h[1][j], 0x5410), prmt(h[0][j], h[1][j], 0x7632),
                                 prmt(h[2][j], h[3][j], 0x5410), prmt(h[2][j], h[3][j], 0x7632)};
#pragma unroll
          for (int i = 0; i < NT; ++i) mma_16816(o[i][c / 2 + j], a, w[0][i][0], w[0][i][1]);
        }
      }
    }

    // ---- 32 committed positions ----
    const int len = seg.len, end = min(len, (seg.t0 + seg.n) * kA4Tile);
#pragma unroll 1
    for (int at = seg.t0 * kA4Tile + warp * kA4Step; at < end && !dead; at += kA4Tile) {
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&full[warp][stage], phase, p.wait_ns))) {
        dead = true;
        if (lane == 0) set_flag(p.flags, kFlagTimeout);
        break;
      }
      holes &= ~(0x10000u << stage);
      const uint8_t* block = ring + stage * kStage;
      const bool edge = at + kA4Step > len || ((holes >> (2 * stage)) & 3);
      float s[2][NT][4];
      uint32_t w[2][NT][2];
      {
        const uint8_t* kc = block + pi * (D / 2) + t * (kCh / 2);
        const uint8_t* ks = block + 8 * D + pi * (D / 16) + t * (kCh / 16);
        uint32_t x[2][2][kCh / 8], sc[2][2];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint8_t* kr = kc + q * kGroup + r * 8 * (D / 2);
            const uint8_t* sr = ks + q * kGroup + r * 8 * (D / 16);
            if constexpr (D == 128) {
              const uint4 y = lds128(kr);
              x[q][r][0] = y.x;
              x[q][r][1] = y.y;
              x[q][r][2] = y.z;
              x[q][r][3] = y.w;
              sc[q][r] = kv4_scales(*reinterpret_cast<const uint16_t*>(sr));
            } else {
              const uint2 y = *reinterpret_cast<const uint2*>(kr);
              x[q][r][0] = y.x;
              x[q][r][1] = y.y;
              sc[q][r] = kv4_scales(*sr);
            }
          }
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int i = 0; i < NT; ++i) s[q][i][0] = s[q][i][1] = s[q][i][2] = s[q][i][3] = 0.0f;
#pragma unroll
        for (int c = 0; c < kCh / 8; ++c)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t h0[4], h1[4];
            kv4_unpack(x[q][0][c], h0);
            kv4_unpack(x[q][1][c], h1);
            const uint32_t s0 = prmt(sc[q][0], 0, c < 2 ? 0x1010 : 0x3232);
            const uint32_t s1 = prmt(sc[q][1], 0, c < 2 ? 0x1010 : 0x3232);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t a[4] = {hmul2(h0[2 * j], s0), hmul2(h1[2 * j], s1),
                                     hmul2(h0[2 * j + 1], s0), hmul2(h1[2 * j + 1], s1)};
#pragma unroll
              for (int i = 0; i < NT; ++i)
                mma_16816(s[q][i], a, qf[i][2 * c + j][0], qf[i][2 * c + j][1]);
            }
          }
      }
      if (edge) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const bool hole = (holes >> (2 * stage + q)) & 1;
          const bool in0 = at + 16 * q + pi < len && !hole;
          const bool in1 = at + 16 * q + pi + 8 < len && !hole;
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!(e < 2 ? in0 : in1)) s[q][i][e] = -INFINITY;
        }
      }
      weights(s, w);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint8_t* vc = block + q * kGroup + kGroup / 2 + t * (D / 2) + g * (kCv / 2);
        const uint8_t* vs = block + q * kGroup + kGroup / 2 + 8 * D + t * (D / 16) + (g * kCv) / 16;
        uint32_t x[4][kCv / 8], sc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (D == 128) {
            const uint2 y = *reinterpret_cast<const uint2*>(vc + 4 * i * (D / 2));
            x[i][0] = y.x;
            x[i][1] = y.y;
          } else {
            x[i][0] = *reinterpret_cast<const uint32_t*>(vc + 4 * i * (D / 2));
          }
          sc[i] = vs[4 * i * (D / 16)];
        }
        if (edge) {  // behind the last position anything may stand: 0 times it is 0
          const bool hole = (holes >> (2 * stage + q)) & 1;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (at + 16 * q + 4 * i + t >= len || hole) sc[i] = 0;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[i] = prmt(kv4_scales(sc[i]), 0, 0x1010);
#pragma unroll
        for (int c = 0; c < kCv / 8; ++c) {
          uint32_t h[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            kv4_unpack(x[i][c], h[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) h[i][j] = hmul2(h[i][j], sc[i]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t a[4] = {prmt(h[0][j], h[1][j], 0x5410), prmt(h[0][j], h[1][j], 0x7632),
                                   prmt(h[2][j], h[3][j], 0x5410), prmt(h[2][j], h[3][j], 0x7632)};
#pragma unroll
            for (int i = 0; i < NT; ++i) mma_16816(o[i][4 * c + j], a, w[q][i][0], w[q][i][1]);
          }
        }
      }
      __syncwarp();
      refill(stage);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }

    // the warps' parts joined, in a fixed order
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[i][c] += __shfl_xor_sync(0xffffffffu, l[i][c], d);
        if (g == 0) {
          s_m[warp][8 * i + 2 * t + c] = m[i][c];
          s_l[warp][8 * i + 2 * t + c] = l[i][c];
        }
      }
    meet();
    float mm[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = -1e30f;
#pragma unroll
        for (int w = 0; w < kA4Warps; ++w) x = fmaxf(x, s_m[w][8 * i + 2 * t + c]);
        const float f = ex2(m[i][c] - x);
        mm[i][c] = x;
        float y = 0.0f;
#pragma unroll
        for (int w = 0; w < kA4Warps; ++w)
          y += s_l[w][8 * i + 2 * t + c] * ex2(s_m[w][8 * i + 2 * t + c] - x);
        l[i][c] = y;
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
          o[i][j][c] *= f;
          o[i][j][c + 2] *= f;
        }
      }
    // outputs: warps [half, 2 half) hand theirs to warps [0, half)
#pragma unroll 1
    for (int half = kA4Warps / 2; half >= 1; half >>= 1) {
      if (warp >= half && warp < 2 * half) {
        float* dst = s_red + (warp - half) * (NT * 8 * D) + lane;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int j = 0; j < kSteps; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) dst[((i * kSteps + j) * 4 + e) * 32] = o[i][j][e];
      }
      meet();
      if (warp < half) {
        const float* src = s_red + warp * (NT * 8 * D) + lane;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int j = 0; j < kSteps; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][j][e] += src[((i * kSteps + j) * 4 + e) * 32];
      }
      meet();
    }
    if (warp == 0) {
      const float vscale = pow2_small(vexp);
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = 8 * i + 2 * t + c;
          if (r >= p.rows) continue;
          if (seg.whole) {
            const float norm = attn_norm(l[i][c]) * vscale;
            const int v = r / p.G;
            const size_t orow = ((size_t)seg.b * p.N + v) * p.Hq + seg.h * p.G + (r - v * p.G);
            uint32_t x[kCv / 2];
#pragma unroll
            for (int j = 0; j < kSteps; ++j) x[j] = pack_bf16(o[i][j][c] * norm, o[i][j][c + 2] * norm);
            uint4* dst = reinterpret_cast<uint4*>(p.out + orow * D + kCv * g);
#pragma unroll
            for (int j = 0; j < kSteps / 4; ++j)
              dst[j] = make_uint4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
            if (p.lse && g == 0) p.lse[orow] = attn_lse(mm[i][c] - kA4Off, l[i][c]);
          } else {
            const size_t row = (size_t)seg.slot * p.rows + r;
            float4* dst = reinterpret_cast<float4*>(p.opart + row * D + kCv * g);
#pragma unroll
            for (int j = 0; j < kSteps / 2; ++j)
              dst[j] = make_float4(o[i][2 * j][c], o[i][2 * j][c + 2], o[i][2 * j + 1][c], o[i][2 * j + 1][c + 2]);
            if (g == 0) p.ml[row] = make_float2(mm[i][c], l[i][c]);
          }
        }
    }
  }
  // every copy has landed before the CTA can leave
  if (dead)
    for (int s = 0; s < kStages; ++s, ++stage) {
      if (stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
      if ((holes >> (16 + stage)) & 1) mbar_wait_bounded(&full[warp][stage], phase);
    }
}

// Joins the partials of items that several CTAs share; other rows are done.  A
// thread takes 4 elements of a row.
template <int D>
__global__ void __launch_bounds__(256) kv4_attn_finish_kernel(const Attn4Params p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long at = id / (D / 4);  // row ((b Hkv + h) N + n) G + g
  const int c = (int)(id - at * (D / 4)) * 4;
  const int ng = p.N * p.G;
  if (at >= (long long)p.B * p.Hkv * ng) return;
  const long long bh = at / ng;
  const int rr = (int)(at - bh * ng);
  const int b = (int)(bh / p.Hkv), h = (int)(bh - (long long)b * p.Hkv);
  const int v = rr / p.G;
  const size_t orow = ((size_t)b * p.N + v) * p.Hq + h * p.G + (rr - v * p.G);
  float m = -1e30f, l = 0.0f;
  float4 acc = make_float4(0, 0, 0, 0);
  if (attn4_len(p, p.base_len[b]) >= 0) {
    const int r = rr;
    int2 span = p.span[bh];
    if (span.x == span.y) return;  // written by its only CTA
    // slots of the workspace, whatever an overlapping call made of the span
    span.x = max(span.x, 0);
    span.y = min(span.y, p.nctas - 1);
    for (int k = span.x; k <= span.y; ++k) {
      const size_t row = (size_t)(2 * k + (k == span.x)) * p.rows + r;
      const float2 x = p.ml[row];
      const float4 y = *reinterpret_cast<const float4*>(p.opart + row * D + c);
      const float mn = fmaxf(m, x.x), fa = ex2(m - mn), fb = ex2(x.x - mn);
      m = mn;
      l = l * fa + x.y * fb;
      acc.x = acc.x * fa + y.x * fb;
      acc.y = acc.y * fa + y.y * fb;
      acc.z = acc.z * fa + y.z * fb;
      acc.w = acc.w * fa + y.w * fb;
    }
  } else if (rr == 0 && h == 0 && c == 0) {
    set_flag(p.flags, kFlagBadPath);
  }
  const float norm = attn_norm(l) * pow2_small(kv4_exp(p.exps, 1));
  *reinterpret_cast<uint2*>(p.out + orow * D + c) =
      make_uint2(pack_bf16(acc.x * norm, acc.y * norm), pack_bf16(acc.z * norm, acc.w * norm));
  if (p.lse && c == 0) p.lse[orow] = attn_lse(m - kA4Off, l);
}

}  // namespace sv
