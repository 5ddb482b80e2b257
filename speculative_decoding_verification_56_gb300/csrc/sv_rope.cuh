// sv_rope.cuh -- head norms, rotary positions and the cache write of a drafted
// tree's query, key and value heads, in one pass.
//
// "EAGLE-3 speculative decoding review", "The Complete EAGLE-3 Inference
// Process" step 3: the target runs once over all tree nodes.  Node v of
// sequence b stands at position pos = offset + base_len[b] - 1 + depth(v) (the
// root is the last committed token), and its key and value go to cache
// position base_len[b] - 1 + v, where spec_kv_commit_path finds them.
//
//   y = x * rsqrt(mean(x^2) + eps) * w          (query and key heads)
//   (a, b) -> (a cos - b sin, b cos + a sin)    angle = pos * inv_freq[i]
//
// in float32, rounded to bf16 once at the end.  Memory-bound: every element
// is read once and written once, so what counts is that the arithmetic in
// between stays below the loads: D/16 threads share a head, each holding the
// two 8-element vectors that a rotation pairs, which needs no exchange (the
// norm is a butterfly over 4 or 8 lanes), and a thread keeps its sines,
// cosines and norm weights in registers over all the heads of the node that
// it takes, as pairs for the two-wide float instructions.  One CTA per node;
// the first threads make the sines and cosines while the first heads' loads
// are in flight.
//
// Measured: 128 trees of 60 nodes, 32 + 8 + 8 heads of 128 (189 MB): 34.8 us,
// 5.4 TB/s, 81% of a plain copy's rate.  64 threads a CTA, so that ends and
// starts of nodes overlap (128 threads 37.2 us, 256 threads 50.8); loads one
// head ahead (two heads ahead 36.0 us: fewer CTAs fit); scalar arithmetic 44.5.
// A single tree of 60 nodes takes what a launch takes.  Other forms at that size:
// pairs side by side 37.2 us; halves that are not whole vectors, whose partners
// are read from memory, 77 us (3 elements) to 103 (60); D = 64 18.5 and, side by
// side, 19.1 (95 MB).
#pragma once

#include "sv_device.cuh"

namespace sv {

constexpr int kRopeThreads = 64;  // at least D / 2: they make the sines (see above for others)

struct RopeParams {
  const uint16_t* qkv;     // [B, N, Hq + 2 Hkv, D] bf16
  const uint16_t* q_norm;  // [D] or null (no norm of the query heads)
  const uint16_t* k_norm;  // [D] or null
  const float* inv_freq;   // [rot / 2]
  const int32_t* base_len; // [B]
  const int32_t* depth;    // [B, N] or null (a chain: node v at depth v)
  uint16_t* q_out;         // [B, N, Hq, D]
  uint16_t* k_cache;       // [B, L, Hkv, D], sequences seq_stride elements apart
  uint16_t* v_cache;
  unsigned* flags;
  long long seq_stride;    // elements
  long long pos_offset;
  float eps;
  int N, Hq, Hkv, L, rot, interleaved;
  int to_nodes;            // keys and values at place v of [B, N, Hkv, D], not behind the prefix
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Sine and cosine of pos * f for an integer position and a float frequency.
// The turns per position f / (2 pi) are a double-float product (off by less
// than 2^-47 of itself: the rounding of its low part and of 1 / (2 pi)), held to
// 2^-64 of a turn, multiplied by pos modulo one turn in 64-bit integers, and
// only the remaining fraction of a turn is rounded to float (2^-26): an angle of
// A turns is off by A 2^-47 + 2^-25 of a turn, and no float64 arithmetic (two
// operations per clock and SM here) is needed.
__device__ __forceinline__ void turn_sincos(long long pos, float f, float* sn, float* cs) {
  const float inv2pi_hi = 0.15915494f;                       // nearest float to 1 / (2 pi)
  const float inv2pi_lo = 6.4206383e-09f;                    // 1 / (2 pi) - inv2pi_hi
  const float sign = copysignf(1.0f, f);
  f = fabsf(f);
  const float hi = __fmul_rn(f, inv2pi_hi);
  const float lo = __fmaf_rn(f, inv2pi_lo, __fmaf_rn(f, inv2pi_hi, -hi));
  const float frac = hi - floorf(hi);  // exact; in [0, 1)
  const float rest = lo - rintf(lo);   // exact; whole turns only past 2^23
  const unsigned long long step = __float2ull_rn(frac * 18446744073709551616.0f) +
                                  (unsigned long long)__float2ll_rn(rest * 18446744073709551616.0f);
  const unsigned long long turns = step * (unsigned long long)pos;
  const float t = (float)(int)(turns >> 32) * 2.3283064365386963e-10f;  // [-1/2, 1/2] turns
  sincospif(2.0f * t, sn, cs);
  *sn *= sign;
}

// mul.rn on both floats of a pair
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// a vector of 8 bf16 as 4 pairs of floats, and back
__device__ __forceinline__ void unpack_pairs(const uint4& v, unsigned long long (&x)[4]) {
  x[0] = f2pack(bf16_lo(v.x), bf16_hi(v.x));
  x[1] = f2pack(bf16_lo(v.y), bf16_hi(v.y));
  x[2] = f2pack(bf16_lo(v.z), bf16_hi(v.z));
  x[3] = f2pack(bf16_lo(v.w), bf16_hi(v.w));
}
__device__ __forceinline__ uint32_t pack_pair(unsigned long long x) {
  float lo, hi;
  f2unpack(x, lo, hi);
  return pack_bf16(lo, hi);
}
__device__ __forceinline__ uint4 pack_pairs(const unsigned long long (&x)[4]) {
  return make_uint4(pack_pair(x[0]), pack_pair(x[1]), pack_pair(x[2]), pack_pair(x[3]));
}
__device__ __forceinline__ unsigned long long swap_pair(unsigned long long x) {
  float lo, hi;
  f2unpack(x, lo, hi);
  return f2pack(hi, lo);
}

// Where a rotation finds its two elements: in the halves of the rotated part,
// a whole number of 8-element vectors apart, or side by side (in either case
// in one thread); or in halves that are not whole vectors, where each thread
// reads an element's partner from memory.
enum RopeMode : int { kRopeHalves = 0, kRopePairs = 1, kRopeOdd = 2 };

template <int D, int kMode>
__global__ void __launch_bounds__(kRopeThreads) tree_qkv_rope_kernel(const RopeParams p) {
  constexpr int kLanes = D / 16;                  // threads per head
  constexpr int kHeads = kRopeThreads / kLanes;   // heads in flight per CTA
  __shared__ float s_sin[D / 2], s_cos[D / 2];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int node = blockIdx.x;
  const int b = node / p.N, v = node - b * p.N;
  const int H = p.Hq + 2 * p.Hkv;
  const int sub = threadIdx.x % kLanes;
  const int half = p.rot / 2;
  const unsigned head_lanes = ((1u << kLanes) - 1u) << ((threadIdx.x & 31) / kLanes * kLanes);
  // the thread's two 8-element vectors: a rotated pair of vectors first, then
  // what is left of the head in order
  int c0 = 2 * sub, c1 = 2 * sub + 1;
  const bool turns = kMode == kRopeHalves && sub < p.rot / 16;
  if (turns) {
    c0 = sub;
    c1 = sub + p.rot / 16;
  }
  const uint16_t* src = p.qkv + (size_t)node * H * D;
  int h = threadIdx.x / kLanes;
  uint4 r0, r1;
  if (h < H) {
    r0 = ldg_stream(src + (size_t)h * D + c0 * 8);
    r1 = ldg_stream(src + (size_t)h * D + c1 * 8);
  }
  // (ordinary loads: the call before this one may have written them)
  const int base = p.base_len[b];
  int dep = p.depth ? p.depth[node] : v;
  const bool ok = base >= 1 && (p.to_nodes || (long long)base + p.N - 1 <= p.L);
  if (threadIdx.x == 0) {
    if (!ok && v == 0) set_flag(p.flags, kFlagBadPath);
    if (dep < 0) set_flag(p.flags, kFlagBadParent);
  }
  if (dep < 0) dep = 0;
  if (threadIdx.x < half) {
    const long long pos = p.pos_offset + base - 1 + dep;
    turn_sincos(pos, __ldg(p.inv_freq + threadIdx.x), &s_sin[threadIdx.x], &s_cos[threadIdx.x]);
  }
  unsigned long long wq[8];  // the query norm's weights of the thread's elements
  if (p.q_norm) {
    unsigned long long t[4];
    unpack_pairs(__ldg(reinterpret_cast<const uint4*>(p.q_norm + c0 * 8)), t);
#pragma unroll
    for (int i = 0; i < 4; ++i) wq[i] = t[i];
    unpack_pairs(__ldg(reinterpret_cast<const uint4*>(p.q_norm + c1 * 8)), t);
#pragma unroll
    for (int i = 0; i < 4; ++i) wq[4 + i] = t[i];
  }
  __syncthreads();
  // halves: cosines and sines of the vector's elements, two to a word; pairs:
  // (c, c) and (-s, s) of the 8 pairs of both vectors
  unsigned long long cs[8], sn[8];
  if (turns) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = c0 * 8 + 2 * i;
      cs[i] = f2pack(s_cos[e], s_cos[e + 1]);
      sn[i] = f2pack(s_sin[e], s_sin[e + 1]);
      sn[4 + i] = f2pack(-s_sin[e], -s_sin[e + 1]);
    }
  } else if (kMode == kRopePairs) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = (i < 4 ? c0 : c1) * 4 + (i & 3);  // the pair's number
      const bool in = e < half;
      const float c = in ? s_cos[e] : 1.0f, s = in ? s_sin[e] : 0.0f;
      cs[i] = f2pack(c, c);
      sn[i] = f2pack(-s, s);
    }
  }
  for (; h < H; h += kHeads) {
    const uint4 a = r0, c = r1;
    const int hn = h + kHeads;
    if (hn < H) {  // the next head's loads
      r0 = ldg_stream(src + (size_t)hn * D + c0 * 8);
      r1 = ldg_stream(src + (size_t)hn * D + c1 * 8);
    }
    const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
    uint16_t* dst = nullptr;
    if (is_q) {
      dst = p.q_out + ((size_t)node * p.Hq + h) * D;
    } else if (ok) {
      const int hk = h - p.Hq - (is_v ? p.Hkv : 0);
      dst = (is_v ? p.v_cache : p.k_cache) + (long long)b * p.seq_stride +
            ((long long)(p.to_nodes ? v : base - 1 + v) * p.Hkv + hk) * D;
    }
    uint4 o0 = a, o1 = c;
    if (!ok) {
      o0 = o1 = make_uint4(0, 0, 0, 0);
    } else if (!is_v) {
      const uint16_t* w = is_q ? p.q_norm : p.k_norm;
      unsigned long long x[4], y[4];
      unpack_pairs(a, x);
      unpack_pairs(c, y);
      float r = 1.0f;
      if (w) {
        unsigned long long s2 = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) s2 = fma2(x[i], x[i], fma2(y[i], y[i], s2));
        float lo, hi;
        f2unpack(s2, lo, hi);
        float ss = lo + hi;
        // butterfly over the head's own lanes (other heads of the warp may be values)
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(head_lanes, ss, o);
        r = rsqrtf(ss * (1.0f / D) + p.eps);
        const unsigned long long r2 = f2pack(r, r);
        if (is_q) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = mul2(x[i], mul2(r2, wq[i]));
            y[i] = mul2(y[i], mul2(r2, wq[4 + i]));
          }
        } else {
          unsigned long long t[4];
          unpack_pairs(__ldg(reinterpret_cast<const uint4*>(w + c0 * 8)), t);
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = mul2(x[i], mul2(r2, t[i]));
          unpack_pairs(__ldg(reinterpret_cast<const uint4*>(w + c1 * 8)), t);
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], mul2(r2, t[i]));
        }
      }
      if constexpr (kMode == kRopeHalves) {
        if (turns) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const unsigned long long u = x[i];
            x[i] = fma2(u, cs[i], mul2(y[i], sn[4 + i]));
            y[i] = fma2(y[i], cs[i], mul2(u, sn[i]));
          }
        }
      } else if constexpr (kMode == kRopePairs) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          unsigned long long& u = i < 4 ? x[i] : y[i - 4];
          const unsigned long long t = fma2(u, cs[i], mul2(swap_pair(u), sn[i]));
          if ((i < 4 ? c0 : c1) * 4 + (i & 3) < half) u = t;
        }
      } else {
        // halves that are not whole vectors: the partner read from memory
        const uint16_t* row = src + (size_t)h * D;
        auto turned = [&](int e, float mine) {
          if (e >= p.rot) return mine;
          const int q = e < half ? e + half : e - half, i = e < half ? e : e - half;
          float other = __uint_as_float((uint32_t)__ldg(row + q) << 16);
          if (w) other = other * r * __uint_as_float((uint32_t)__ldg(w + q) << 16);
          return e < half ? mine * s_cos[i] - other * s_sin[i] : mine * s_cos[i] + other * s_sin[i];
        };
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          unsigned long long& u = i < 4 ? x[i] : y[i - 4];
          const int e = (i < 4 ? c0 : c1) * 8 + 2 * (i & 3);
          float lo, hi;
          f2unpack(u, lo, hi);
          u = f2pack(turned(e, lo), turned(e + 1, hi));
        }
      }
      o0 = pack_pairs(x);
      o1 = pack_pairs(y);
    }
    if (dst) {
      *reinterpret_cast<uint4*>(dst + c0 * 8) = o0;
      *reinterpret_cast<uint4*>(dst + c1 * 8) = o1;
    }
  }
}

}  // namespace sv
