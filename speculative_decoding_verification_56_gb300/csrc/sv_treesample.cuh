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
// hundred thousand unlikely ones, so sums are exact: weights are fixed-point
// 64-bit integers (2^-45 of the largest, from a double-float evaluation of
// 2^x), whose sums depend on no order.  Each CTA scales by its own largest
// logit, rounded up to a power of two, so that one pass needs no exchange of
// maxima and the sums of two CTAs are brought together by shifts.
#pragma once

#include "sv_lmhead.cuh"

namespace sv {

constexpr int kTsThreads = 512;
constexpr int kTsWarps = kTsThreads / 32;
constexpr int kTsStep = 256;          // elements of a warp's step: 8 per lane
constexpr int kTsMaxCluster = 16;
constexpr int kTsFrac = 45;           // fraction bits of a weight
constexpr unsigned kFlagEmptyRow = 64u;

struct TreeSampleParams {
  const void* logits;         // [B, N, V]
  const int32_t* tokens;      // [B, N]
  const int32_t* parents;     // [B, N]
  const float* u;             // [B, max_depth + 1]
  float c_hi, c_lo;           // log2(e) / T as a double-float
  int N, V, max_depth;
  int nsteps;                 // steps of kTsStep elements per warp
  int extra;                  // further right shift of the weights: V > 2^17
  int32_t* accepted_len;      // [B]
  int32_t* path;              // [B, max_depth + 1]
  int32_t* out;               // [B, max_depth + 1]
  float* probs;               // [B, max_depth + 1]
  unsigned* flags;
};

// z * log2(e) / T as a double-float.
__device__ __forceinline__ void ts_exponent(const TreeSampleParams& p, float z, float* hi, float* lo) {
  *hi = __fmul_rn(z, p.c_hi);
  *lo = __fmaf_rn(z, p.c_lo, __fmaf_rn(z, p.c_hi, -*hi));
}

// Mantissa of 2^(y_hi + y_lo) in fixed point (2^45 stands for 1) and its
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

// Weight of logit z relative to 2^ref, in units of 2^-kTsFrac (2^-extra more).
__device__ __forceinline__ unsigned long long ts_weight(const TreeSampleParams& p, float z, int ref,
                                                        const long long* tab_i, const float2* tab_f) {
  float hi, lo;
  ts_exponent(p, z, &hi, &lo);
  if (!(hi > (float)(ref - kTsFrac - 3))) return 0;  // too small, -inf or NaN
  int n;
  const long long m = ts_mantissa(hi, lo, tab_i, tab_f, &n);
  const int sh = ref - n + p.extra;
  if (sh <= 0) return (unsigned long long)m;
  return ((unsigned long long)m + (1ull << (sh - 1))) >> sh;
}

// floor(u * R) for u in [0, 1): below R, so that u R < C means floor < C.
__device__ __forceinline__ unsigned long long ts_threshold(float u, unsigned long long R) {
  if (!(u > 0.0f)) return 0;
  if (u >= 1.0f) return R - 1;
  const unsigned bits = __float_as_uint(u);
  const int ex = (int)(bits >> 23);
  const unsigned long long man = ex ? (bits & 0x7FFFFFu) | 0x800000u : (bits & 0x7FFFFFu);
  const int sh = 150 - (ex ? ex : 1);  // u = man * 2^-sh, sh in [24, 149]
  const unsigned long long lo = man * R, hi = __umul64hi(man, R);
  if (sh < 64) return (hi << (64 - sh)) | (lo >> sh);
  return sh < 128 ? hi >> (sh - 64) : 0;
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

struct TsPart {  // a CTA's part of a row, as every CTA of the cluster holds it
  unsigned long long sum;
  int ref;
  int pad;
};

template <typename E, bool kVec>
__global__ void __launch_bounds__(kTsThreads) tree_sample_kernel(const TreeSampleParams p) {
  extern __shared__ unsigned long long ts_steps[];  // [kTsWarps][nsteps]: sums of the steps
  __shared__ long long tab_i[64];
  __shared__ float2 tab_f[64];
  __shared__ TsPart s_part[2][kTsMaxCluster];
  __shared__ int s_tok[2];
  __shared__ float s_prob[2];
  __shared__ float s_max[kTsWarps];
  __shared__ unsigned long long s_wsum[kTsWarps];
  __shared__ int s_child;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t C;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(C));
  const uint32_t rank = cluster_rank();
  const int b = blockIdx.x / C;
  if (threadIdx.x < 64) {
    const double m = exp2((double)threadIdx.x / 64.0);
    tab_i[threadIdx.x] = __double2ll_rn(m * 35184372088832.0);  // 2^45
    tab_f[threadIdx.x] = make_float2((float)m, (float)(m - (double)(float)m));
  }
  // a programmatic dependent of the kernel before it in the stream: nothing
  // of global memory is touched before that grid has finished
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int32_t* par = p.parents + (size_t)b * p.N;
  const int32_t* tok = p.tokens + (size_t)b * p.N;
  const int W = p.max_depth + 1;
  if (rank == 0) {
    unsigned bad = 0;
    for (int v = threadIdx.x; v < p.N; v += kTsThreads) {
      if (v > 0) {
        if (par[v] < 0 || par[v] >= v) bad |= kFlagBadParent;
        if (tok[v] < 0 || tok[v] >= p.V) bad |= kFlagTokenRange;
      }
    }
    if (bad) set_flag(p.flags, bad);
  }
  __syncthreads();
  const long long span = (long long)p.nsteps * kTsStep;  // elements of a warp
  const long long w0 = ((long long)rank * kTsWarps + warp) * span + lane * 8;
  unsigned long long* steps = ts_steps + (size_t)warp * p.nsteps;
  int cur = 0, d = 0;
  for (;; ++d) {
    const int par_ = d & 1;
    const typename E::storage* row =
        static_cast<const typename E::storage*>(p.logits) + ((size_t)b * p.N + cur) * (size_t)p.V;
    // the CTA's largest logit: the power of two its weights are relative to
    float m = -INFINITY;
    for (int s = 0; s < p.nsteps; ++s) {
      float z[8];
      ts_load<E, kVec>(row, w0 + (long long)s * kTsStep, p.V, z);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, z[e]);
    }
    m = warp_max_f(m);
    if (lane == 0) s_max[warp] = m;
    if (threadIdx.x == 0) s_child = 0x7FFFFFFF;
    __syncthreads();
    m = s_max[lane & (kTsWarps - 1)];
    m = warp_max_f(m);
    const int ref = exp_ref(m, p.c_hi);
    // sums of the weights
    unsigned long long sum = 0;
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
    if (lane == 0) s_wsum[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      unsigned long long t = warp_sum_u64(lane < kTsWarps ? s_wsum[lane] : 0ull);
      if (lane < (int)C) {  // into every CTA of the cluster
        const uint32_t at = cluster_addr(&s_part[par_][rank], lane);
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(t) : "memory");
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at + 8), "r"(ref) : "memory");
      }
    }
    cluster_sync_all();
    // the total, and the CTA that holds the drawn token
    int gref = kRefEmpty;
    for (int c = 0; c < (int)C; ++c) gref = max(gref, s_part[par_][c].ref);
    unsigned long long R = 0;
    for (int c = 0; c < (int)C; ++c) {
      const int sh = gref - s_part[par_][c].ref;
      R += sh < 64 ? s_part[par_][c].sum >> sh : 0ull;
    }
    unsigned long long t = R ? ts_threshold(p.u[(size_t)b * W + d], R) : 0;
    int owner = -1, shift = 0;
    if (R) {
      for (int c = 0; c < (int)C; ++c) {
        const int sh = gref - s_part[par_][c].ref;
        const unsigned long long part = sh < 64 ? s_part[par_][c].sum >> sh : 0ull;
        if (t < part) {
          owner = c;
          shift = sh;
          break;
        }
        t -= part;
      }
    }
    if (owner == (int)rank) {
      t <<= shift;  // in the CTA's own units: below its sum
      int own = 0;
      for (; own < kTsWarps - 1 && t >= s_wsum[own]; ++own) t -= s_wsum[own];
      if (warp == own) {
        int s = 0;
        for (; s < p.nsteps - 1 && t >= steps[s]; ++s) t -= steps[s];
        float z[8];
        unsigned long long w[8], part = 0;
        ts_load<E, kVec>(row, w0 + (long long)s * kTsStep, p.V, z);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          w[e] = ts_weight(p, z[e], ref, tab_i, tab_f);
          part += w[e];
        }
        const unsigned long long incl = warp_scan_u64(part);
        unsigned long long left = incl - part;
        if (t >= left && t < incl) {  // one lane
          int x = 0;
          float zx = z[0];
          bool found = false;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (!found && t < left + w[e]) {
              found = true;
              x = e;
              zx = z[e];
            }
            left += w[e];
          }
          const int token = (int)(w0 + (long long)s * kTsStep) + x;
          float hi, lo;
          int n;
          ts_exponent(p, zx, &hi, &lo);
          const double mant = (double)ts_mantissa(hi, lo, tab_i, tab_f, &n);
          const float prob = (float)(mant * exp2((double)(n - gref - p.extra)) / (double)R);
          for (int c = 0; c < (int)C; ++c) {
            const uint32_t at = cluster_addr(&s_tok[par_], c), ap = cluster_addr(&s_prob[par_], c);
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(token) : "memory");
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(ap), "f"(prob) : "memory");
          }
        }
      }
    }
    cluster_sync_all();
    const int x = owner < 0 ? -1 : s_tok[par_];
    if (rank == 0 && threadIdx.x == 0) {
      p.path[(size_t)b * W + d] = cur;
      p.out[(size_t)b * W + d] = x;
      p.probs[(size_t)b * W + d] = owner < 0 ? 0.0f : s_prob[par_];
      if (owner < 0) set_flag(p.flags, kFlagEmptyRow);
    }
    // the lowest-numbered child that holds the token (children come after
    // their parent, so the walk ends)
    if (x >= 0) {
      for (int v = cur + 1 + threadIdx.x; v < p.N; v += kTsThreads)
        if (__ldg(par + v) == cur && __ldg(tok + v) == x) atomicMin(&s_child, v);
    }
    __syncthreads();
    const int child = s_child;
    if (child == 0x7FFFFFFF) break;
    if (d == p.max_depth) {
      if (rank == 0 && threadIdx.x == 0) set_flag(p.flags, kFlagDepth);
      break;
    }
    cur = child;
    __syncthreads();  // s_child is read before the next step resets it
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
