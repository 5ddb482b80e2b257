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
#pragma once

#include "sv_lmhead.cuh"
#include "sv_rope.cuh"

namespace sv {

constexpr int kAtFinThreads = 128;
constexpr int kAtFinHeads = 8;  // query heads of a key-value head held by a warp at once

struct AttnParams {
  const uint16_t* q;        // [B, N, Hq, D]
  const uint16_t* k;        // [B, L, Hkv, D], sequences seq_stride elements apart
  const uint16_t* v;
  const uint16_t* pk;       // [P, Hkv, D]
  const uint16_t* pv;
  const uint32_t* mask;     // [B, N, W] or null (a chain)
  const int32_t* base_len;  // [B]
  uint16_t* out;            // [B, N, Hq, D]
  float* lse;               // [B, N, Hq] or null
  unsigned* flags;
  long long seq_stride;     // elements
  float scale_log2;         // scale * log2(e)
  int B, N, Hq, Hkv, G, W, L, P;
};

__device__ __forceinline__ bool attn_seq_ok(const AttnParams& p, int base) {
  return base >= 1 && (long long)base + p.N - 1 <= p.L;
}

// One warp per (node, key-value head): running softmax over the visible
// entries in float32, kAtFinHeads query heads at a time; a lane holds D / 32
// elements of the head.
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
  const int base = __ldg(p.base_len + b);
  const bool ok = attn_seq_ok(p, base);
  if (!ok && n == 0 && h == 0 && lane == 0) set_flag(p.flags, kFlagBadPath);
  const int prefix = base - 1;
  const uint16_t* kseq = p.k + (long long)b * p.seq_stride + h * D;
  const uint16_t* vseq = p.v + (long long)b * p.seq_stride + h * D;
  auto load = [&](const uint16_t* src, float (&x)[kE]) {
    if constexpr (kE == 4) {
      const uint2 w = *reinterpret_cast<const uint2*>(src + lane * 4);
      x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
    } else {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(src + lane * 2);
      x[0] = bf16_lo(w); x[1] = bf16_hi(w);
    }
  };
  for (int g0 = 0; g0 < p.G; g0 += kAtFinHeads) {
    const int ng = min(kAtFinHeads, p.G - g0);
    float q[kAtFinHeads][kE], acc[kAtFinHeads][kE], m[kAtFinHeads], l[kAtFinHeads];
    const uint16_t* qrow = p.q + ((size_t)node * p.Hq + h * p.G + g0) * D;
#pragma unroll
    for (int g = 0; g < kAtFinHeads; ++g) {
      m[g] = -INFINITY;
      l[g] = 0.0f;
#pragma unroll
      for (int e = 0; e < kE; ++e) acc[g][e] = q[g][e] = 0.0f;
      if (g < ng) load(qrow + (size_t)g * D, q[g]);
    }
    auto visit = [&](const uint16_t* krow, const uint16_t* vrow) {
      float kx[kE], vx[kE];
      load(krow, kx);
      load(vrow, vx);
#pragma unroll
      for (int g = 0; g < kAtFinHeads; ++g) {
        if (g < ng) {
          float s = 0.0f;
#pragma unroll
          for (int e = 0; e < kE; ++e) s = __fmaf_rn(q[g][e], kx[e], s);
          s = warp_sum_f(s) * p.scale_log2;
          const float mn = fmaxf(m[g], s);
          const float a = ex2(m[g] - mn), w = ex2(s - mn);
          m[g] = mn;
          l[g] = __fmaf_rn(l[g], a, w);
#pragma unroll
          for (int e = 0; e < kE; ++e) acc[g][e] = __fmaf_rn(acc[g][e], a, w * vx[e]);
        }
      }
    };
    const size_t es = (size_t)p.Hkv * D;
    if (ok) {
      for (int j = 0; j < p.P; ++j) visit(p.pk + j * es + h * D, p.pv + j * es + h * D);
      for (int j = 0; j < prefix; ++j) visit(kseq + j * es, vseq + j * es);
      const uint32_t* mrow = p.mask ? p.mask + (size_t)node * p.W : nullptr;
      for (int w = 0; w < p.W; ++w) {
        uint32_t bits;
        if (mrow) {
          bits = __ldg(mrow + w);
        } else {
          const int c = n + 1 - 32 * w;
          bits = c >= 32 ? 0xFFFFFFFFu : c <= 0 ? 0u : (1u << c) - 1u;
        }
        if (p.N - 32 * w < 32) bits &= (1u << (p.N - 32 * w)) - 1u;
        while (bits) {
          const int u = 32 * w + __ffs(bits) - 1;
          bits &= bits - 1;
          visit(kseq + (size_t)(prefix + u) * es, vseq + (size_t)(prefix + u) * es);
        }
      }
    }
#pragma unroll
    for (int g = 0; g < kAtFinHeads; ++g) {
      if (g < ng) {
        const float r = l[g] > 0.0f ? 1.0f / l[g] : (l[g] == 0.0f ? 0.0f : l[g]);
        uint16_t* orow = p.out + ((size_t)node * p.Hq + h * p.G + g0 + g) * D;
        if constexpr (kE == 4) {
          *reinterpret_cast<uint2*>(orow + lane * 4) =
              make_uint2(pack_bf16(acc[g][0] * r, acc[g][1] * r),
                         pack_bf16(acc[g][2] * r, acc[g][3] * r));
        } else {
          *reinterpret_cast<uint32_t*>(orow + lane * 2) = pack_bf16(acc[g][0] * r, acc[g][1] * r);
        }
        if (p.lse && lane == 0)
          p.lse[(size_t)node * p.Hq + h * p.G + g0 + g] =
              l[g] == 0.0f ? -INFINITY : (m[g] + log2f(l[g])) * 0.6931471805599453f;
      }
    }
  }
}

}  // namespace sv
