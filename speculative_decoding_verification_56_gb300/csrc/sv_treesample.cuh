// sv_treesample.cuh -- sampling verification of drafted trees.
//
// The walk starts at the root (node 0).  At a node whose target row is z it
// draws the next token from the target's own distribution with the given
// uniform u of its depth, x = the smallest j with u R < C_j, where
//   w_j = 2^(z_j log2(e) / T),  C_j = w_0 + ... + w_j,  R = C_{V-1},
// and goes on to the lowest-numbered child that holds x, or stops there and
// keeps x as the last token.  The tokens are those that drawing one by one
// from the target with the same uniforms gives, whatever the tree: every
// child x_c is taken with probability p(x_c), and the token after a miss
// follows p without the children -- the accept test and the residual of
// "EAGLE-3 speculative decoding review", "Does Using a Small Model's Answer
// Reduce Quality?" for drafts that are points (the top-K children of
// "EAGLE math", "EAGLE-2: dynamic draft trees").
//
// Only the rows on the walk are read (one per step), so the call is bound by
// the latency of a step, not by the bandwidth of all rows.  One cluster of
// CTAs per sequence splits each row; the CTAs meet twice a step: once to add
// up their sums, once to learn the token.
//
// A token must fall on the right side of every border C_j, also of the
// hundred thousand unlikely ones, which no float32 sum can promise.  So a step
// first screens the row in float32, in one pass: every 256 elements are summed
// as 2^(z_j c - ref) with a power of two near their largest as the reference,
// those sums are added up in turn, and the token of t = u R is taken if t is
// further than R / 2^15 from both of its borders.  The error of such sums is
// bounded: 2^-22.4 of a weight from ex2.approx, 1.5 |r| 2^-24 ln 2 from its
// argument r (its rounding and that of c), where the mean of |r| over the
// row's mass is at most log2(V) + 1, and up to 13 float additions in a step, 69
// over a warp's 2048 steps, 5 over the warps, 5 over the CTAs and 5 in the
// search: together below 8e-6 R for V = 2^26, of t and of a border.  Otherwise
// (a draw among tokens of probability below 6e-5, for the most part) the row is
// summed again in integers, whose sums depend on no order: weights in units of
// 2^-50 of the largest, from a double-float evaluation of 2^x (off by 2^-40 of
// itself, and by |z / T| 2^-46 of itself for the argument's rounding).  The
// roundings to the unit can all go one way (equal tokens), which moves a border
// by V 2^-51; the sums of a warp's 256-element steps are kept whole, and only
// the warps' sums are cut to 2^(extra-50) (so that the row's fit 64 bits), 128 of
// them at most: 2^-29 at V = 2^26.  Together a border is off by less than 2^-24
// of R for every V up to 2^26, one step of a float32 uniform.
// No float64 arithmetic is on the way: it runs at two operations per
// clock and SM here, and the sums of 16 CTAs alone took 16 us of a step.
//
// Measured (V = 128256 bf16): one sequence 8-21 us by the length of its walk, 16
// of them 21-31 (their longest walks count: 5 rows 21, 7 rows 28), 64 of
// V = 151936 float32 60-70 us; about 4.2 us a step (5.8 where V = 128257 has rows
// read element by element) (clocks: screen 1700, the CTA's sum 680, exchange 1650, search
// 480, token 2700, child 460), against 0.1 to 15 us of HBM time for the rows.
// Tried against the exchanges and lost: words counted by mbarriers in place of
// the cluster's barriers 17.5 us at one sequence and 30.1 at 16; the rows of the
// children asked for ahead 19.8 -> 22.5 and 28.2 -> 33.0.
#pragma once

#include "sv_lmhead.cuh"

namespace sv {

constexpr int kTsThreads = 256;
constexpr int kTsWarps = kTsThreads / 32;
constexpr int kTsStep = 256;          // elements of a warp's step: 8 per lane
constexpr int kTsMaxCluster = 16;
constexpr int kTsMant = 45;           // fraction bits of a mantissa in [1, 2)
constexpr int kTsFrac = 50;           // and of a weight: 32 steps' sums stay below 2^64
constexpr unsigned kFlagEmptyRow = 64u;

// 2^(k/64): in units of 2^-45, and as two floats (nearest to the exact values).
__constant__ long long kTsPow[64] = {
    0x200000000000ll, 0x2059347cef01ll, 0x20b361a62b0bll, 0x210e8a30eb38ll,
    0x216ab0d9f312ll, 0x21c7d865a7a3ll, 0x222603a024b7ll, 0x2285355d525cll,
    0x22e57078faa3ll, 0x2346b7d6df97ll, 0x23a90e62d173ll, 0x240c7710c51all,
    0x2470f4dceac4ll, 0x24d68acbc4fall, 0x253d3bea3fbell, 0x25a50b4dc806ll,
    0x260dfc14636ell, 0x26781164c82ell, 0x26e34e6e7554ll, 0x274fb669cb40ll,
    0x27bd4c982468ll, 0x282c1443ee5cll, 0x289c10c0c312ll, 0x290d456b827all,
    0x297fb5aa6c54ll, 0x29f364ed3a59ll, 0x2a6856ad3a9fll, 0x2ade8e6d6a50ll,
    0x2b560fba90a8ll, 0x2bcede2b5a43ll, 0x2c48fd6074abll, 0x2cc47104aa44ll,
    0x2d413cccfe78ll, 0x2dbf6478ca34ll, 0x2e3eebd1d8bfll, 0x2ebfd6ac84d0ll,
    0x2f4228e7d603ll, 0x2fc5e66d9e9dll, 0x304b1332999cll, 0x30d1b3368926ll,
    0x3159ca845542ll, 0x31e35d322aeell, 0x326e6f619b8cll, 0x32fb053fbc9dll,
    0x3389230547e1ll, 0x3418ccf6bbcbll, 0x34aa07647c4bll, 0x353cd6aaf3fbll,
    0x35d13f32b5a7ll, 0x366745709e2cll, 0x36feede5f6bdll, 0x37983d209784ll,
    0x383337bb0aa5ll, 0x38cfe25cafa3ll, 0x396e41b9df21ll, 0x3a0e5a940f13ll,
    0x3ab031b9f749ll, 0x3b53cc07b665ll, 0x3bf92e66f737ll, 0x3ca05dcf1680ll,
    0x3d495f454922ll, 0x3df437dcc2b4ll, 0x3ea0ecb6dc8bll, 0x3f4f83033d22ll,
};
__constant__ float2 kTsPowF[64] = {
    {0x1.0000000000000p+0f, 0x0.0p+0f}, {0x1.02c9a40000000p+0f, -0x1.887fa00000000p-28f},
    {0x1.059b0e0000000p+0f, -0x1.9d4f520000000p-25f}, {0x1.0874520000000p+0f, -0x1.e2990e0000000p-26f},
    {0x1.0b55860000000p+0f, 0x1.9f31220000000p-25f}, {0x1.0e3ec40000000p+0f, -0x1.a585cc0000000p-25f},
    {0x1.11301e0000000p+0f, -0x1.fdb4960000000p-25f}, {0x1.1429aa0000000p+0f, 0x1.d525bc0000000p-25f},
    {0x1.172b840000000p+0f, -0x1.c157420000000p-27f}, {0x1.1a35be0000000p+0f, 0x1.6df96e0000000p-25f},
    {0x1.1d48740000000p+0f, -0x1.d2e8ca0000000p-25f}, {0x1.2063b80000000p+0f, 0x1.0c519a0000000p-25f},
    {0x1.2387a60000000p+0f, 0x1.ceac480000000p-25f}, {0x1.26b4560000000p+0f, 0x1.789f380000000p-26f},
    {0x1.29e9e00000000p+0f, -0x1.5c04240000000p-25f}, {0x1.2d285a0000000p+0f, 0x1.b900c20000000p-26f},
    {0x1.306fe00000000p+0f, 0x1.4636e20000000p-25f}, {0x1.33c08c0000000p+0f, -0x1.b37d200000000p-25f},
    {0x1.371a740000000p+0f, -0x1.18aac60000000p-25f}, {0x1.3a7db40000000p+0f, -0x1.634c020000000p-25f},
    {0x1.3dea640000000p+0f, 0x1.8246840000000p-25f}, {0x1.4160a20000000p+0f, 0x1.f72e2a0000000p-28f},
    {0x1.44e0860000000p+0f, 0x1.8624b40000000p-30f}, {0x1.486a2c0000000p+0f, -0x1.47d8660000000p-25f},
    {0x1.4bfdae0000000p+0f, -0x1.593abc0000000p-25f}, {0x1.4f9b280000000p+0f, -0x1.2c5a6c0000000p-25f},
    {0x1.5342b60000000p+0f, -0x1.2c56100000000p-25f}, {0x1.56f4740000000p+0f, -0x1.295b040000000p-25f},
    {0x1.5ab07e0000000p+0f, -0x1.5bd5ec0000000p-27f}, {0x1.5e76f20000000p+0f, -0x1.4a5bd60000000p-25f},
    {0x1.6247ec0000000p+0f, -0x1.f8b5500000000p-25f}, {0x1.6623880000000p+0f, 0x1.2a91120000000p-27f},
    {0x1.6a09e60000000p+0f, 0x1.9fcef40000000p-26f}, {0x1.6dfb240000000p+0f, -0x1.cd72e80000000p-27f},
    {0x1.71f75e0000000p+0f, 0x1.1d8bee0000000p-25f}, {0x1.75feb60000000p+0f, -0x1.37b3060000000p-25f},
    {0x1.7a11480000000p+0f, -0x1.829fd00000000p-25f}, {0x1.7e2f340000000p+0f, -0x1.2616340000000p-25f},
    {0x1.82589a0000000p+0f, -0x1.accc7c0000000p-26f}, {0x1.868d9a0000000p+0f, -0x1.2edb440000000p-26f},
    {0x1.8ace540000000p+0f, 0x1.15506e0000000p-27f}, {0x1.8f1aea0000000p+0f, -0x1.baa2320000000p-26f},
    {0x1.93737c0000000p+0f, -0x1.e647440000000p-25f}, {0x1.97d82a0000000p+0f, -0x1.0d8d840000000p-31f},
    {0x1.9c49180000000p+0f, 0x1.51f8480000000p-27f}, {0x1.a0c6680000000p+0f, -0x1.2886a60000000p-26f},
    {0x1.a5503c0000000p+0f, -0x1.b83b540000000p-25f}, {0x1.a9e6b60000000p+0f, -0x1.50c0480000000p-25f},
    {0x1.ae89fa0000000p+0f, -0x1.a94b140000000p-26f}, {0x1.b33a2c0000000p+0f, -0x1.ec3a820000000p-26f},
    {0x1.b7f7700000000p+0f, -0x1.a094380000000p-25f}, {0x1.bcc1ea0000000p+0f, -0x1.f687c60000000p-25f},
    {0x1.c199be0000000p+0f, -0x1.3d56b20000000p-27f}, {0x1.c67f120000000p+0f, 0x1.cafa2a0000000p-25f},
    {0x1.cb720e0000000p+0f, -0x1.8837cc0000000p-27f}, {0x1.d072d40000000p+0f, 0x1.40f1300000000p-25f},
    {0x1.d5818e0000000p+0f, -0x1.822dbc0000000p-27f}, {0x1.da9e600000000p+0f, 0x1.ed99420000000p-27f},
    {0x1.dfc9740000000p+0f, -0x1.908c940000000p-25f}, {0x1.e502ee0000000p+0f, 0x1.e2cffe0000000p-26f},
    {0x1.ea4afa0000000p+0f, 0x1.52486c0000000p-27f}, {0x1.efa1be0000000p+0f, 0x1.cc2b440000000p-25f},
    {0x1.f507660000000p+0f, -0x1.246eb00000000p-26f}, {0x1.fa7c180000000p+0f, 0x1.9e90d80000000p-28f},
};

struct TreeSampleParams {
  const void* logits;         // [B, N, V]
  const int32_t* tokens;      // [B, N]
  const int32_t* parents;     // [B, N]
  const float* u;             // [B, max_depth + 1]
  float c_hi, c_lo;           // log2(e) / T as a double-float
  int N, V, max_depth;
  int nsteps;                 // steps of kTsStep elements per warp
  int extra;                  // right shift of the warps' sums: V > 2^12
  int32_t* accepted_len;      // [B]
  int32_t* path;              // [B, max_depth + 1]
  int32_t* out;               // [B, max_depth + 1]
  float* probs;               // [B, max_depth + 1]
  unsigned* flags;
};

// z * log2(e) / T - ref as a normalised double-float: the product's two parts,
// the difference to the reference with its rounding error (two-sum), and a
// renormalisation, so that large logits lose nothing to their common size.
__device__ __forceinline__ void ts_exponent(const TreeSampleParams& p, float z, float ref,
                                            float* hi, float* lo) {
  const float y = __fmul_rn(z, p.c_hi);
  const float y_lo = __fmaf_rn(z, p.c_lo, __fmaf_rn(z, p.c_hi, -y));
  const float d = __fsub_rn(y, ref);
  const float t = __fsub_rn(d, y);  // two-sum of y and -ref
  const float err = __fsub_rn(__fsub_rn(y, __fsub_rn(d, t)), __fadd_rn(ref, t));
  const float l = __fadd_rn(err, y_lo);
  *hi = __fadd_rn(d, l);
  *lo = __fsub_rn(l, __fsub_rn(*hi, d));
}

// Mantissa of 2^(y_hi + y_lo) in fixed point (2^kTsMant stands for 1) and its
// binary exponent *n.  y = n + k/64 + r with |r| <= 1/128: the table gives
// 2^(k/64) (as the integer and as two floats), e^(r ln 2) - 1 is s + s^2/2 + ...
// with s held as a double-float; its product with the table's value is
// brought into the integer in two parts by the rounding of float additions
// (each part below 2^22 of its units, where 1.5 * 2^23 + part keeps all bits).  Relative error about 2^-40.
__device__ __forceinline__ long long ts_mantissa(float y_hi, float y_lo, const long long* tab_i,
                                                 const float2* tab_f, int* n) {
  const float shifter = 12582912.0f;  // 1.5 * 2^23
  const float t = __fmaf_rn(y_hi, 64.0f, shifter);
  const int ki = __float_as_int(t) - 0x4B400000;
  const float r = __fmaf_rn(__fsub_rn(t, shifter), -0.015625f, y_hi);  // exact
  const float ln2_hi = 0.693147182f, ln2_lo = -1.9046542e-9f;
  const float s = __fmul_rn(r, ln2_hi);
  float e = __fmaf_rn(r, ln2_lo, __fmaf_rn(r, ln2_hi, -s));
  e = __fmaf_rn(y_lo, ln2_hi, e);
  e = __fmaf_rn(s, e, e);  // (s + e)^2 / 2 holds s e
  float q = __fmaf_rn(s, 8.3333333e-3f, 4.1666667e-2f);
  q = __fmaf_rn(s, q, 1.6666667e-1f);
  q = __fmaf_rn(s, q, 0.5f);
  e = __fmaf_rn(__fmul_rn(s, s), q, e);  // e^(s + ...) - 1 = s + e
  const int k = ki & 63;
  *n = ki >> 6;
  const float2 f = tab_f[k];                                    // high and low part
  const float h = __fmul_rn(f.x, s);                            // |h| < 2^-6.8
  const float l = __fmaf_rn(f.x, e, __fmaf_rn(f.y, s, __fmaf_rn(f.x, s, -h)));
  const float m1 = __fmaf_rn(__fadd_rn(h, l), 4194304.0f, shifter);  // units of 2^-22
  const float h1 = __fsub_rn(m1, shifter);
  // what is left, below 2^-22.9, in units of 2^-44
  const float rest = __fadd_rn(__fmaf_rn(h1, -2.384185791015625e-7f, h), l);
  const float m2 = __fmaf_rn(rest, 17592186044416.0f, shifter);
  const int i1 = __float_as_int(m1) - 0x4B400000, i2 = __float_as_int(m2) - 0x4B400000;
  return tab_i[k] + ((long long)i1 << 23) + 2ll * i2;
}

// Weight of logit z relative to 2^ref, in units of 2^-kTsFrac, rounded.
__device__ __forceinline__ unsigned long long ts_weight(const TreeSampleParams& p, float z, int ref,
                                                        const long long* tab_i, const float2* tab_f) {
  float hi, lo;
  ts_exponent(p, z, (float)ref, &hi, &lo);
  if (!(hi > -(float)(kTsFrac + 3))) return 0;  // too small, -inf or NaN
  int n;
  const long long m = ts_mantissa(hi, lo, tab_i, tab_f, &n);
  const int sh = kTsMant - kTsFrac - n;
  if (sh <= 0) return (unsigned long long)m << min(-sh, kTsFrac - kTsMant);
  return ((unsigned long long)m + (1ull << (sh - 1))) >> sh;
}

// floor(u * R) for u in [0, 1): below R, so that u R < C means floor < C; and the
// next `extra` bits of u * R, for the warps' uncut sums.
__device__ __forceinline__ unsigned long long ts_threshold(float u, unsigned long long R, int extra,
                                                           unsigned* frac) {
  const unsigned mask = (1u << extra) - 1u;
  *frac = 0;
  if (!(u > 0.0f)) return 0;
  *frac = mask;
  if (u >= 1.0f) return R - 1;
  const unsigned bits = __float_as_uint(u);
  const int ex = (int)(bits >> 23);
  const unsigned man = ex ? (bits & 0x7FFFFFu) | 0x800000u : (bits & 0x7FFFFFu);
  const int sh = 150 - (ex ? ex : 1) - extra;  // u = man * 2^-(sh + extra); sh in [9, 149]
  const unsigned __int128 x = sh < 128 ? (unsigned __int128)man * R >> sh : 0;
  *frac = (unsigned)x & mask;
  return (unsigned long long)(x >> extra);
}

__device__ __forceinline__ unsigned long long warp_sum_u64(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ unsigned long long warp_scan_u64(unsigned long long v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// The lane's 8 elements of a step (-inf past the end of the row).  kVec: rows
// start at 16-byte boundaries and hold whole groups of 8.
template <typename E, bool kVec>
__device__ __forceinline__ void ts_load(const typename E::storage* row, long long at, int V,
                                        float (&z)[8]) {
  if constexpr (kVec) {
    if (at < V) {
#pragma unroll
      for (int i = 0; i < 8 / E::kEPV; ++i) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + at) + i);
#pragma unroll
        for (int e = 0; e < E::kEPV; ++e) z[i * E::kEPV + e] = E::elem(v, e);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = -INFINITY;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = at + e < V ? E::load1(row + at + e) : -INFINITY;
  }
}

// A CTA's part of a row, as every CTA of the cluster holds it.
struct TsPart {
  unsigned long long sum;  // exact: of weights relative to 2^ref, in units of 2^(extra-kTsFrac)
  int ref;
  float fsum;              // screened: of weights relative to 2^ref
};

// All threads of the cluster.  The aligned barrier wants whole warps, so lanes
// that took different ways come together first.
__device__ __forceinline__ void ts_cluster_sync() {
  __syncwarp();
  cluster_sync_all();
}

__device__ __forceinline__ void cluster_st64(uint32_t at, unsigned long long x) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(x) : "memory");
}
__device__ __forceinline__ void cluster_st32(uint32_t at, uint32_t x) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(x) : "memory");
}

constexpr float kTsScreen = 1.0f / 32768.0f;  // of R: draws nearer to a border are decided exactly
constexpr int kTsTreeSmem = 1024;   // trees of up to so many nodes are held in shared memory
constexpr int kTsNone = -1, kTsUnclear = -2;
constexpr int kTsRefBad = 1 << 30;  // of a sum that is not finite

__device__ __forceinline__ unsigned long long ts_shift(unsigned long long x, int sh) {
  return sh < 64 ? x >> sh : 0ull;
}

// The first lane whose inclusive sum of x exceeds t (-1: none); t becomes the
// rest inside that lane.  Every lane gets the answer.
__device__ __forceinline__ int ts_pick(unsigned long long x, unsigned long long* t) {
  const unsigned long long incl = warp_scan_u64(x);
  const unsigned past = __ballot_sync(0xffffffffu, *t < incl);
  if (past == 0) return -1;
  const int at = __ffs(past) - 1;
  *t -= __shfl_sync(0xffffffffu, incl - x, at);
  return at;
}

// The same for float sums (behind all of them: the last lane that is not 0).
__device__ __forceinline__ float warp_scan_f(float v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}
__device__ __forceinline__ int ts_pick_f(float x, float incl, float* t) {
  const unsigned past = __ballot_sync(0xffffffffu, *t < incl && x > 0.0f);
  const unsigned some = __ballot_sync(0xffffffffu, x > 0.0f);
  const int at = past ? __ffs(past) - 1 : some ? 31 - __clz(some) : 0;
  *t = fmaxf(*t - __shfl_sync(0xffffffffu, incl - x, at), 0.0f);
  return at;
}
// 2^d, 0 for d < -126 (d <= 127)
__device__ __forceinline__ float ts_pow2(int d) {
  return d < -126 ? 0.0f : __int_as_float((min(d, 127) + 127) << 23);
}

template <typename E, bool kVec>
__global__ void __launch_bounds__(kTsThreads, 4) tree_sample_kernel(const TreeSampleParams p) {
  extern __shared__ unsigned long long ts_steps[];  // [kTsWarps][nsteps]: sums of the steps
  __shared__ long long tab_i[64];
  __shared__ float2 tab_f[64];
  __shared__ TsPart s_part[2][kTsMaxCluster];  // the cluster's, by turns
  __shared__ TsPart s_warp[kTsWarps];
  __shared__ int s_tok[2];
  __shared__ float s_prob[2];
  __shared__ int s_max[kTsWarps];
  __shared__ int s_child;
  __shared__ int2 s_tree[kTsTreeSmem];  // parent, token
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t C;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(C));
  const uint32_t rank = cluster_rank();
  const int b = blockIdx.x / C;
  if (threadIdx.x < 64) {
    tab_i[threadIdx.x] = kTsPow[threadIdx.x];
    tab_f[threadIdx.x] = kTsPowF[threadIdx.x];
  }
  ts_cluster_sync();  // every CTA runs before its shared memory is written to
  // a programmatic dependent of the kernel before it in the stream: nothing
  // of global memory is touched before that grid has finished
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int32_t* par = p.parents + (size_t)b * p.N;
  const int32_t* tok = p.tokens + (size_t)b * p.N;
  const int W = p.max_depth + 1;
  const bool held = p.N <= kTsTreeSmem;
  if (held || rank == 0) {
    unsigned bad = 0;
    for (int v = threadIdx.x; v < p.N; v += kTsThreads) {
      const int pa = par[v], to = tok[v];
      if (v > 0) {
        if (pa < 0 || pa >= v) bad |= kFlagBadParent;
        if (to < 0 || to >= p.V) bad |= kFlagTokenRange;
      }
      if (held) s_tree[v] = make_int2(pa, to);
    }
    if (bad && rank == 0) set_flag(p.flags, bad);
  }
  const long long span = (long long)p.nsteps * kTsStep;  // elements of a warp
  const long long w0 = ((long long)rank * kTsWarps + warp) * span + lane * 8;
  unsigned long long* steps = ts_steps + (size_t)warp * p.nsteps;
  int2* raw = reinterpret_cast<int2*>(steps);
  unsigned meet = 0;  // exchanges so far: their buffers alternate

  // Exact: adds up the warps' sums (s_warp), tells the cluster, and finds the
  // CTA with t = floor(u R) -- the same answer everywhere -- and in that CTA
  // the warp `own` and the rest t.
  unsigned long long R;
  int gref, owner, own;
  unsigned long long t;
  unsigned t_frac;  // bits of t below the unit of the cut sums
  auto exchange = [&](float u) {
    __syncthreads();  // s_warp is complete
    const TsPart mine = lane < kTsWarps ? s_warp[lane] : TsPart{0ull, kRefEmpty, 0.0f};
    const int top = __reduce_max_sync(0xffffffffu, mine.ref);
    const unsigned long long x = ts_shift(mine.sum, top - mine.ref);
    if (warp == 0) {
      const unsigned long long sum = warp_sum_u64(x);
      if (lane < (int)C) {  // into every CTA of the cluster
        const uint32_t at = cluster_addr(&s_part[meet & 1][rank], lane);
        cluster_st64(at, sum);
        cluster_st32(at + 8, (uint32_t)top);
      }
    }
    ts_cluster_sync();
    const TsPart part = lane < (int)C ? s_part[meet & 1][lane] : TsPart{0ull, kRefEmpty, 0.0f};
    gref = __reduce_max_sync(0xffffffffu, part.ref);
    const unsigned long long y = ts_shift(part.sum, gref - part.ref);
    R = warp_sum_u64(y);
    owner = kTsNone;
    if (R) {
      t = ts_threshold(u, R, p.extra, &t_frac);
      owner = ts_pick(y, &t);
      if (owner == (int)rank) {
        t <<= gref - top;      // in the CTA's own units: below its sum
        own = ts_pick(x, &t);  // (a CTA's warps have one reference)
      }
    }
  };
  // the step of the owning warp that holds t, which becomes the rest in it (in
  // the weights' units; a warp's 2048 steps may add up to more than 64 bits)
  auto find_step = [&]() {
    unsigned __int128 left = (unsigned __int128)t << p.extra | t_frac;
    t = 0;
    for (int s0 = 0; s0 < p.nsteps; s0 += 32) {
      const unsigned long long x = s0 + lane < p.nsteps ? steps[s0 + lane] : 0ull;
      const unsigned long long all = warp_sum_u64(x);
      if (left < all) {
        t = (unsigned long long)left;
        return s0 + ts_pick(x, &t);
      }
      left -= all;
    }
    return p.nsteps - 1;  // never: t is below the steps' sum
  };
  auto tell = [&](int from, int token, float prob) {  // lane `from`'s, to every CTA
    token = __shfl_sync(0xffffffffu, token, from);
    prob = __shfl_sync(0xffffffffu, prob, from);
    if (lane < (int)C) {
      cluster_st32(cluster_addr(&s_tok[meet & 1], lane), (uint32_t)token);
      cluster_st32(cluster_addr(&s_prob[meet & 1], lane), __float_as_uint(prob));
    }
  };

  int cur = 0, d = 0;
  for (;; ++d) {
    const typename E::storage* row =
        static_cast<const typename E::storage*>(p.logits) + ((size_t)b * p.N + cur) * (size_t)p.V;
    const float u = p.u[(size_t)b * W + d];
    if (threadIdx.x == 0) s_child = 0x7FFFFFFF;
    // ---- screen: float32 sums in one pass
#pragma unroll 4
    for (int s = 0; s < p.nsteps; ++s) {
      float z[8];
      ts_load<E, kVec>(row, w0 + (long long)s * kTsStep, p.V, z);
      const float m = fmaxf(fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])),
                            fmaxf(fmaxf(z[4], z[5]), fmaxf(z[6], z[7])));
      const int ref = __reduce_max_sync(0xffffffffu, exp_ref(m, p.c_hi));
      const float nref = -(float)ref;
      float x = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) x += ex2(__fmaf_rn(z[e], p.c_hi, nref));
      x = warp_sum_f(x);
      if (lane == 0) raw[s] = x <= 512.0f ? make_int2(ref, __float_as_int(x)) : make_int2(kTsRefBad, 0);
    }
    __syncwarp();
    {
      int top = kRefEmpty;
      for (int s = lane; s < p.nsteps; s += 32) top = max(top, raw[s].x);
      top = __reduce_max_sync(0xffffffffu, top);
      float sum = 0.0f;
      for (int s = lane; s < p.nsteps; s += 32) {  // brought to the warp's reference
        const float y = __int_as_float(raw[s].y) * ts_pow2(raw[s].x - top);
        raw[s].y = __float_as_int(y);
        sum += y;
      }
      sum = warp_sum_f(sum);
      if (lane == 0) s_warp[warp] = TsPart{0ull, top, sum};
    }
    __syncthreads();
    float R_f = 0.0f, t_f = 0.0f;
    {
      const TsPart mine = lane < kTsWarps ? s_warp[lane] : TsPart{0ull, kRefEmpty, 0.0f};
      const int top = __reduce_max_sync(0xffffffffu, mine.ref);
      if (warp == 0) {
        const float sum = warp_sum_f(mine.fsum * ts_pow2(mine.ref - top));
        if (lane < (int)C)  // into every CTA of the cluster
          cluster_st64(cluster_addr(&s_part[meet & 1][rank].ref, lane),
                       (unsigned long long)__float_as_uint(sum) << 32 | (uint32_t)top);
      }
      ts_cluster_sync();
      const TsPart part = lane < (int)C ? s_part[meet & 1][lane] : TsPart{0ull, kRefEmpty, 0.0f};
      gref = __reduce_max_sync(0xffffffffu, part.ref);
      const float y = part.fsum * ts_pow2(part.ref - gref);
      const float incl = warp_scan_f(y);
      R_f = __shfl_sync(0xffffffffu, incl, 31);
      owner = gref == kTsRefBad ? kTsUnclear : kTsNone;
      if (gref != kTsRefBad && R_f > 0.0f) {
        t_f = fminf(fmaxf(u, 0.0f), 0.99999994f) * R_f;
        owner = ts_pick_f(y, incl, &t_f);
        if (owner == (int)rank) {
          const float x = mine.fsum * ts_pow2(mine.ref - gref);
          own = ts_pick_f(x, warp_scan_f(x), &t_f);
        }
      }
    }
    if (owner == (int)rank && warp == own) {
      const int ref = s_warp[warp].ref;
      const float unit = ts_pow2(ref - gref);  // of the warp's sums
      int s = 0;
      for (int s0 = 0; s0 < p.nsteps; s0 += 32) {
        const float y = s0 + lane < p.nsteps ? __int_as_float(raw[s0 + lane].y) * unit : 0.0f;
        const float incl = warp_scan_f(y);
        const float all = __shfl_sync(0xffffffffu, incl, 31);
        if (t_f < all || s0 + 32 >= p.nsteps) {
          s = s0 + ts_pick_f(y, incl, &t_f);
          break;
        }
        t_f -= all;
      }
      float z[8], w[8], sum = 0.0f;
      ts_load<E, kVec>(row, w0 + (long long)s * kTsStep, p.V, z);
      const float nref = -(float)ref;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        w[e] = ex2(__fmaf_rn(z[e], p.c_hi, nref)) * unit;
        sum += w[e];
      }
      const int at = ts_pick_f(sum, warp_scan_f(sum), &t_f);
      float lo = 0.0f, hi = 0.0f, wx = 0.0f;  // (of the lane that holds t)
      int x = 0;
      bool found = false;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (!found) {
          lo = hi;
          hi += w[e];
          wx = w[e];
          x = e;
          found = t_f < hi;
        }
      }
      const float eps = R_f * kTsScreen;
      const bool clear = found && t_f - lo > eps && hi - t_f > eps;
      tell(at, clear ? (int)(w0 + (long long)s * kTsStep) + x : kTsUnclear, wx / R_f);
    }
    int x = owner;
    float prob = 0.0f;
    if (owner >= 0) {
      ts_cluster_sync();
      x = s_tok[meet & 1];
      prob = s_prob[meet & 1];
    }
    ++meet;
    if (x == kTsUnclear) {
      // ---- exact: fixed-point sums relative to the CTA's largest logit
      int ref = kRefEmpty;
      for (int s = 0; s < p.nsteps; ++s) {
        float z[8], m = -INFINITY;
        ts_load<E, kVec>(row, w0 + (long long)s * kTsStep, p.V, z);
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, z[e]);
        ref = max(ref, exp_ref(m, p.c_hi));
      }
      ref = __reduce_max_sync(0xffffffffu, ref);
      if (lane == 0) s_max[warp] = ref;
      __syncthreads();
      ref = __reduce_max_sync(0xffffffffu, s_max[lane % kTsWarps]);
      if (ref == kTsRefBad) ref = kTsRefBad - 1;  // (an infinite logit: unspecified)
      unsigned __int128 sum = 0;
      for (int s = 0; s < p.nsteps; ++s) {
        float z[8];
        ts_load<E, kVec>(row, w0 + (long long)s * kTsStep, p.V, z);
        unsigned long long part = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) part += ts_weight(p, z[e], ref, tab_i, tab_f);
        part = warp_sum_u64(part);
        if (lane == 0) steps[s] = part;
        sum += part;
      }
      if (lane == 0) s_warp[warp] = TsPart{(unsigned long long)(sum >> p.extra), ref, 0.0f};
      exchange(u);
      if (owner == (int)rank && warp == own) {
        const int s = find_step();
        float z[8];
        unsigned long long w[8], part = 0;
        ts_load<E, kVec>(row, w0 + (long long)s * kTsStep, p.V, z);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          w[e] = ts_weight(p, z[e], ref, tab_i, tab_f);
          part += w[e];
        }
        const int at = ts_pick(part, &t);
        unsigned long long left = 0;
        int e0 = 0;
        float zx = z[0];
        bool found = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          left += w[e];
          if (!found && t < left) {
            found = true;
            e0 = e;
            zx = z[e];
          }
        }
        float hi, lo;
        int n;
        ts_exponent(p, zx, (float)ref, &hi, &lo);
        const float mant = (float)ts_mantissa(hi, lo, tab_i, tab_f, &n);
        tell(max(at, 0), (int)(w0 + (long long)s * kTsStep) + e0,
             mant * (float)(1 << (kTsFrac - kTsMant)) / (float)R *
                 pow2i_f(min(n + ref - gref, 0) - p.extra));
      }
      ts_cluster_sync();
      x = owner < 0 ? kTsNone : s_tok[meet & 1];
      prob = owner < 0 ? 0.0f : s_prob[meet & 1];
      ++meet;
    }
    if (rank == 0 && threadIdx.x == 0) {
      p.path[(size_t)b * W + d] = cur;
      p.out[(size_t)b * W + d] = x;
      p.probs[(size_t)b * W + d] = prob;
      if (x < 0) set_flag(p.flags, kFlagEmptyRow);
    }
    // the lowest-numbered child that holds the token (children come after
    // their parent, so the walk ends)
    int child = 0x7FFFFFFF;
    if (held) {  // every warp for itself
      for (int v = cur + 1; x >= 0 && v < p.N; v += 32) {
        const int2 node = v + lane < p.N ? s_tree[v + lane] : make_int2(-1, -1);
        const unsigned hit = __ballot_sync(0xffffffffu, node.x == cur && node.y == x);
        if (hit) {
          child = v + __ffs(hit) - 1;
          break;
        }
      }
    } else {
      if (x >= 0) {
        for (int v = cur + 1 + threadIdx.x; v < p.N; v += kTsThreads)
          if (par[v] == cur && tok[v] == x) atomicMin(&s_child, v);
      }
      __syncthreads();
      child = s_child;
      __syncthreads();  // s_child is read before the next step resets it
    }
    if (child == 0x7FFFFFFF) break;
    if (d == p.max_depth) {
      if (rank == 0 && threadIdx.x == 0) set_flag(p.flags, kFlagDepth);
      break;
    }
    cur = child;
  }
  if (rank == 0) {
    if (threadIdx.x == 0) p.accepted_len[b] = d;
    for (int i = d + 1 + threadIdx.x; i < W; i += kTsThreads) {
      p.path[(size_t)b * W + i] = -1;
      p.out[(size_t)b * W + i] = -1;
      p.probs[(size_t)b * W + i] = 0.0f;
    }
  }
  // no CTA leaves while a peer may still write into its shared memory: the
  // last writes came before the last cluster barrier
}

}  // namespace sv
