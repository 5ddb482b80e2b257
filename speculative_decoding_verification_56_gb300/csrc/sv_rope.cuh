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
// is read once and written once.  One CTA per node: its first rot/2 threads
// make the node's sines and cosines while the first heads' loads are in
// flight, and D/16 threads share a head, each holding the two 8-element
// vectors that a rotation pairs, so that the rotation needs no exchange and
// the norm a butterfly over 4 or 8 lanes.
#pragma once

#include "sv_device.cuh"

namespace sv {

constexpr int kRopeThreads = 256;

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
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x); x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
  x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z); x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                    pack_bf16(x[6], x[7]));
}

// Sine and cosine of pos * f for an integer position and a float frequency.
// The turns per position f / (2 pi) are held to 2^-64 of a turn (the product
// as a double-float, about 2^-48 relative), multiplied by pos modulo one turn
// in 64-bit integers, and only the remaining fraction of a turn is rounded to
// float: far positions lose no more than near ones, and no float64
// arithmetic (two operations per clock and SM here) is needed.
__device__ __forceinline__ void turn_sincos(long long pos, float f, float* sn, float* cs) {
  const float inv2pi_hi = 0.15915494f;                       // nearest float to 1 / (2 pi)
  const float inv2pi_lo = 6.4206383e-09f;                    // 1 / (2 pi) - inv2pi_hi
  const float sign = copysignf(1.0f, f);
  f = fabsf(f);
  const float hi = __fmul_rn(f, inv2pi_hi);
  const float lo = __fmaf_rn(f, inv2pi_lo, __fmaf_rn(f, inv2pi_hi, -hi));
  const float frac = hi - floorf(hi);  // exact; in [0, 1)
  const unsigned long long step = __float2ull_rn(frac * 18446744073709551616.0f) +
                                  (unsigned long long)__float2ll_rn(lo * 18446744073709551616.0f);
  const unsigned long long turns = step * (unsigned long long)pos;
  const float t = (float)(int)(turns >> 32) * 2.3283064365386963e-10f;  // [-1/2, 1/2] turns
  sincospif(2.0f * t, sn, cs);
  *sn *= sign;
}

// kVec: the vector layout holds both members of every pair in one thread
// (pairs side by side, or halves a whole number of 8-element vectors apart);
// otherwise each thread finds an element's partner in memory.
template <int D, bool kVec>
__global__ void __launch_bounds__(kRopeThreads) tree_qkv_rope_kernel(const RopeParams p) {
  constexpr int kLanes = D / 16;                  // threads per head
  constexpr int kHeads = kRopeThreads / kLanes;   // heads in flight per CTA
  __shared__ float s_sin[D / 2], s_cos[D / 2];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int node = blockIdx.x;
  const int b = node / p.N, v = node - b * p.N;
  const int base = __ldg(p.base_len + b);
  const bool ok = base >= 1 && (long long)base + p.N - 1 <= p.L;
  int dep = p.depth ? __ldg(p.depth + node) : v;
  if (threadIdx.x == 0) {
    if (!ok && v == 0) set_flag(p.flags, kFlagBadPath);
    if (dep < 0) set_flag(p.flags, kFlagBadParent);
  }
  if (dep < 0) dep = 0;
  const int H = p.Hq + 2 * p.Hkv;
  const int sub = threadIdx.x % kLanes;
  const int half = p.rot / 2;
  const unsigned head_lanes = ((1u << kLanes) - 1u) << ((threadIdx.x & 31) / kLanes * kLanes);
  // the thread's two 8-element vectors: a rotated pair of vectors first, then
  // what is left of the head in order
  int c0 = 2 * sub, c1 = 2 * sub + 1;
  if (kVec && !p.interleaved && sub < p.rot / 16) {
    c0 = sub;
    c1 = sub + p.rot / 16;
  }
  const uint16_t* src = p.qkv + (size_t)node * H * D;
  int h = threadIdx.x / kLanes;
  uint4 r0, r1;
  if (h < H) {
    r0 = *reinterpret_cast<const uint4*>(src + (size_t)h * D + c0 * 8);
    r1 = *reinterpret_cast<const uint4*>(src + (size_t)h * D + c1 * 8);
  }
  if (threadIdx.x < half) {
    const long long pos = p.pos_offset + base - 1 + dep;
    turn_sincos(pos, __ldg(p.inv_freq + threadIdx.x), &s_sin[threadIdx.x], &s_cos[threadIdx.x]);
  }
  __syncthreads();
  for (; h < H; h += kHeads) {
    const uint4 a = r0, c = r1;
    const int hn = h + kHeads;
    if (hn < H) {  // the next head's loads
      r0 = *reinterpret_cast<const uint4*>(src + (size_t)hn * D + c0 * 8);
      r1 = *reinterpret_cast<const uint4*>(src + (size_t)hn * D + c1 * 8);
    }
    const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
    uint16_t* dst = nullptr;
    if (is_q) {
      dst = p.q_out + ((size_t)node * p.Hq + h) * D;
    } else if (ok) {
      const int hk = h - p.Hq - (is_v ? p.Hkv : 0);
      dst = (is_v ? p.v_cache : p.k_cache) + (long long)b * p.seq_stride +
            ((long long)(base - 1 + v) * p.Hkv + hk) * D;
    }
    uint4 o0 = a, o1 = c;
    if (!ok) {
      o0 = o1 = make_uint4(0, 0, 0, 0);
    } else if (!is_v) {
      const uint16_t* w = is_q ? p.q_norm : p.k_norm;
      float x[8], y[8];
      unpack8(a, x);
      unpack8(c, y);
      float r = 1.0f;
      {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __fmaf_rn(x[i], x[i], __fmaf_rn(y[i], y[i], ss));
        // butterfly over the head's own lanes (other heads of the warp may be values)
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(head_lanes, ss, o);
        if (w) r = rsqrtf(ss * (1.0f / D) + p.eps);
      }
      if (w) {
        float wx[8], wy[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(w + c0 * 8)), wx);
        unpack8(__ldg(reinterpret_cast<const uint4*>(w + c1 * 8)), wy);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = x[i] * r * wx[i];
          y[i] = y[i] * r * wy[i];
        }
      }
      if constexpr (kVec) {
        if (p.interleaved) {
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const int ex = c0 * 8 + i, ey = c1 * 8 + i;
            if (ex < p.rot) {
              const float cs = s_cos[ex / 2], sn = s_sin[ex / 2], u = x[i], t = x[i + 1];
              x[i] = u * cs - t * sn;
              x[i + 1] = t * cs + u * sn;
            }
            if (ey < p.rot) {
              const float cs = s_cos[ey / 2], sn = s_sin[ey / 2], u = y[i], t = y[i + 1];
              y[i] = u * cs - t * sn;
              y[i + 1] = t * cs + u * sn;
            }
          }
        } else if (sub < p.rot / 16) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float cs = s_cos[c0 * 8 + i], sn = s_sin[c0 * 8 + i], u = x[i], t = y[i];
            x[i] = u * cs - t * sn;
            y[i] = t * cs + u * sn;
          }
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
          x[i] = turned(c0 * 8 + i, x[i]);
          y[i] = turned(c1 * 8 + i, y[i]);
        }
      }
      o0 = pack8(x);
      o1 = pack8(y);
    }
    if (dst) {
      *reinterpret_cast<uint4*>(dst + c0 * 8) = o0;
      *reinterpret_cast<uint4*>(dst + c1 * 8) = o1;
    }
  }
}

}  // namespace sv
