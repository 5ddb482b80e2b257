// sv_kv4.cuh -- a key-value cache in pages of 4-bit values: its format, the
// commit of an accepted path into it, and the way back to bf16.
//
// A page holds `page` positions of all key-value heads of one layer, head by
// head, and a head's positions in groups of 16, each contiguous:
//   key codes [16, D/2], key scales [16, D/16], value codes, value scales
// (18 D bytes), so that whatever the page, one copy brings a warp of the
// attention all that it needs for one matrix product's 16 entries.  16 channels
// of a head share a scale:
//   a = max |x|,  s = e4m3(min(448, a / 6 2^-e)),  code = e2m1(x / (s 2^e)),
//   value = code s 2^e,
// both rounded to nearest even (codes saturate at 6), channel 2 i in the low
// half of byte i; e is one exponent per layer for keys and one for values.
// Codes have 2 significant bits and scales 4, so a value is exact in bf16 and,
// without 2^e, in fp16; and a / 6 and x / (s 2^e) next to a border are decided
// exactly in float32 (see the commit).
//
// Commit reads 4 D bytes of an entry's head and writes 9 D / 8, read the other
// way round.  Measured with 5 prompts of up to 1000 tokens, 8 layers, 8 heads of
// 128: commit 42-44 us, read 43-46 us (6.3-6.6 TB/s); commit took 55 with divisions and
// rounding by integers, and both 119 before the lanes of a warp shared an entry.
#pragma once

#include "sv_rope.cuh"

namespace sv {

constexpr unsigned kFlagBadPage = 128u;
constexpr int kKv4MaxExp = 64;  // exponents beyond are taken as this
constexpr int kKv4Threads = 256;

// Bytes of a group of 16 positions, and of a head's block.
__host__ __device__ constexpr int kv4_group(int D) { return 18 * D; }
__host__ __device__ constexpr int kv4_block(int page, int D) { return page / 16 * kv4_group(D); }
// Byte offset in a block of the key (value) half of place `slot`'s group
__device__ __forceinline__ int kv4_half(int slot, int is_v, int D) {
  return (slot >> 4) * kv4_group(D) + is_v * (kv4_group(D) / 2);
}

__device__ __forceinline__ int kv4_exp(const int32_t* e, int i) {
  return e ? min(max(e[i], -kKv4MaxExp), kKv4MaxExp) : 0;
}
// 2^e for |e| <= 126
__device__ __forceinline__ float pow2_small(int e) { return __int_as_float((e + 127) << 23); }

// 8 codes (a word) as 4 pairs of fp16, in channel order
__device__ __forceinline__ void kv4_unpack(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// two scales (low byte first) as a pair of fp16
__device__ __forceinline__ uint32_t kv4_scales(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float2 half2_to_float2(uint32_t h) {
  float2 f;
  asm("{\n .reg .f16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}\n"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}
// e4m3 of a float in [0, 448], to nearest even
__device__ __forceinline__ uint32_t to_e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(x));
  return r & 0xFFu;
}
// 8 codes (a word), channels in order from the low end, to nearest even, saturating
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&x)[8]) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

struct Kv4Params {
  uint8_t* pages;           // [layers, n_pages, Hkv, block]
  const int32_t* table;     // [B, W]
  const uint16_t* node_k;   // commit: [layers, B, N, Hkv, D] bf16
  const uint16_t* node_v;
  const int32_t* base_len;  // commit: [B]
  const int32_t* accepted;  // commit: [B] or null (all nodes)
  const int32_t* path;      // commit: [B, max_depth + 1] or null (a chain)
  const int32_t* length;    // read: [B]
  const int32_t* exps;      // [layers, 2] or null
  int32_t* new_len;         // commit: [B]
  uint16_t* k_out;          // read: [layers, B, L, Hkv, D] bf16
  uint16_t* v_out;
  unsigned* flags;
  long long n_pages, out_layer, out_seq;  // (elements)
  int B, N, Hkv, W, lg, max_depth, L, layers;
  int blocks;               // of each (layer, sequence)
  int lg_lanes;             // log2 of the lanes that share an entry
};

// Page of position t of sequence b, or -1 (outside the table, or no page).
__device__ __forceinline__ long long kv4_page_of(const Kv4Params& p, int b, long long t) {
  const long long i = t >> p.lg;
  if (i < 0 || i >= p.W) return -1;
  const int id = p.table[(size_t)b * p.W + i];
  return id >= 0 && id < p.n_pages ? id : -1;
}

// Number of entries that sequence b commits; 0 for one that is malformed
// (flagged).  The whole block takes part.
__device__ __forceinline__ int kv4_commit_count(const Kv4Params& p, int b) {
  const int base = p.base_len[b];
  const int acc = p.accepted ? p.accepted[b] : p.N - 1;
  const int most = p.path ? min(p.max_depth, p.N - 1) : p.N - 1;
  bool ok = base >= 1 && acc >= 0 && acc <= most;
  bool paged = true;
  if (ok) {
    if (p.path) {
      const int32_t* path = p.path + (size_t)b * (p.max_depth + 1);
      for (int i = threadIdx.x; i <= acc; i += blockDim.x)
        ok &= i == 0 ? path[0] == 0 : path[i] >= 1 && path[i] < p.N;
    }
    const long long first = (base - 1) >> p.lg, last = ((long long)base - 1 + acc) >> p.lg;
    for (long long i = first + threadIdx.x; i <= last; i += blockDim.x)
      paged &= kv4_page_of(p, b, i << p.lg) >= 0;
  }
  ok = __syncthreads_and(ok);
  paged = __syncthreads_and(paged);
  if (ok && paged) return acc + 1;
  if (threadIdx.x == 0) set_flag(p.flags, ok ? kFlagBadPage : kFlagBadPath);
  return 0;
}

// Where a (layer, sequence)'s threads find their entries: 1 << lg_lanes lanes (as
// many as an entry has groups of 16 channels, a warp at most) share an entry, so
// that what an entry costs -- its page, its addresses -- is paid once for many
// channels.
struct Kv4Lanes {
  int first, step, lane, lanes;
  __device__ __forceinline__ Kv4Lanes(const Kv4Params& p, unsigned part) {
    const int per_block = kKv4Threads >> p.lg_lanes;
    first = (int)part * per_block + (int)(threadIdx.x >> p.lg_lanes);
    step = p.blocks * per_block;
    lanes = 1 << p.lg_lanes;
    lane = threadIdx.x & (lanes - 1);
  }
};

// Commit: a thread takes 16 channels of an entry's key and as many of its value
// -- loads of 32 bytes, stores of 8 and of one -- in turn over the entry's heads.
// How many entries a sequence has is known only to the device.
template <int D>
__global__ void __launch_bounds__(kKv4Threads) kv4_commit_kernel(const Kv4Params p) {
  constexpr int kBlocks = D / 16;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const unsigned lb = blockIdx.x / p.blocks, part = blockIdx.x - lb * p.blocks;
  const int layer = (int)(lb / p.B), b = (int)(lb - (unsigned)layer * p.B);
  const int count = kv4_commit_count(p, b);
  const int base = p.base_len[b];
  if (layer == 0 && part == 0 && threadIdx.x == 0)
    p.new_len[b] = count ? base - 1 + count : max(base, 1) - 1;
  const int blocks = p.Hkv * kBlocks, page = 1 << p.lg;
  const int e[2] = {kv4_exp(p.exps, 2 * layer), kv4_exp(p.exps, 2 * layer + 1)};
  const Kv4Lanes w(p, part);
  for (int at = w.first; at < count; at += w.step) {
    const int node = p.path ? p.path[(size_t)b * (p.max_depth + 1) + at] : at;
    const size_t src = (((size_t)layer * p.B + b) * p.N + node) * (size_t)blocks * 16;
    const long long t = (long long)base - 1 + at;
    const int slot = (int)t & (page - 1);
    uint8_t* dst = p.pages + ((size_t)layer * p.n_pages + kv4_page_of(p, b, t)) * p.Hkv *
                                 kv4_block(page, D) + kv4_half(slot, 0, D);
    const int place = slot & 15;
    for (int hb = w.lane; hb < blocks; hb += w.lanes) {
      uint4 x4[2][2];
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const uint16_t* s = (v ? p.node_v : p.node_k) + src + hb * 16;
        x4[v][0] = ldg_stream(s);
        x4[v][1] = ldg_stream(s + 8);
      }
      const int h = hb / kBlocks, c = hb % kBlocks;
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const uint32_t x[8] = {x4[v][0].x, x4[v][0].y, x4[v][0].z, x4[v][0].w,
                               x4[v][1].x, x4[v][1].y, x4[v][1].z, x4[v][1].w};
        uint32_t a2 = 0;  // largest magnitudes of even and odd channels, as bits
#pragma unroll
        for (int j = 0; j < 8; ++j) a2 = max_u16x2(a2, x[j] & 0x7FFF7FFFu);
        const float a = __uint_as_float(max(a2 & 0xFFFF0000u, a2 << 16));
        // Quotients a / 6 and x / step, by reciprocals (off by 2^-22 of themselves)
        // and rounded so far that those on a border of two scales or codes are
        // exactly that, while the others, further from a border than 2^-8 of it,
        // stay on their side.  (With whole numbers X < 2^8 of a or x, m < 2^4 of the
        // step: X against borders times 6 or m, below 2^8.)  a / 6 to 12 bits; x /
        // step, whose borders are 1/4 and more, to multiples of 2^-11 (by at most a
        // quarter of that distance).
        const float sixth = __uint_as_float((__float_as_uint(a * (1.0f / 6.0f)) + 0x800u) & 0xFFFFF000u);
        const uint32_t sb = to_e4m3(fminf(sixth * pow2_small(-e[v]), 448.0f));
        const float step = half2_to_float2(kv4_scales(sb)).x * pow2_small(e[v]);
        float inv;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(step));
        if (sb == 0) inv = 0.0f;
        constexpr float kGrid = 6144.0f;  // 1.5 2^12, whose last place is 2^-11
        const unsigned long long inv2 = f2pack(inv, inv), up = f2pack(kGrid, kGrid),
                                 down = f2pack(-kGrid, -kGrid);
        uint32_t code[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float q[8];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            f2unpack(add2(fma2(f2pack(bf16_lo(x[4 * j + i]), bf16_hi(x[4 * j + i])), inv2, up), down),
                     q[2 * i], q[2 * i + 1]);
          code[j] = to_e2m1x8(q);
        }
        uint8_t* block = dst + (size_t)h * kv4_block(page, D) + v * (kv4_group(D) / 2);
        *reinterpret_cast<uint2*>(block + place * (D / 2) + c * 8) = make_uint2(code[0], code[1]);
        block[8 * D + place * kBlocks + c] = (uint8_t)sb;
      }
    }
  }
}

// Read: a thread takes 16 channels of a position's key and of its value, in turn
// over the heads, and stores each in one piece where the outputs' alignment allows
// (commit and read of 5 prompts 87 us, with two stores of 16 bytes, whose sectors
// reach L2 half full, 102).
template <int D>
__global__ void __launch_bounds__(kKv4Threads) kv4_read_kernel(const Kv4Params p) {
  constexpr int kBlocks = D / 16;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const unsigned lb = blockIdx.x / p.blocks, part = blockIdx.x - lb * p.blocks;
  const int layer = (int)(lb / p.B), b = (int)(lb - (unsigned)layer * p.B);
  const int len = p.length[b];
  const int count = max(0, min(len, p.L));
  if ((len < 0 || len > p.L) && layer == 0 && part == 0 && threadIdx.x == 0)
    set_flag(p.flags, kFlagBadPath);
  const int blocks = p.Hkv * kBlocks, page = 1 << p.lg;
  const float unit[2] = {pow2_small(kv4_exp(p.exps, 2 * layer)),
                         pow2_small(kv4_exp(p.exps, 2 * layer + 1))};
  const Kv4Lanes w(p, part);
  const bool wide = (((uintptr_t)p.k_out | (uintptr_t)p.v_out | (uintptr_t)(p.out_layer * 2) |
                      (uintptr_t)(p.out_seq * 2)) & 31) == 0;
  for (int t = w.first; t < count; t += w.step) {
    const long long id = kv4_page_of(p, b, t);
    if (id < 0 && w.lane == 0) set_flag(p.flags, kFlagBadPage);
    const int slot = t & (page - 1), place = slot & 15;
    const uint8_t* src = p.pages + ((size_t)layer * p.n_pages + max(id, 0ll)) * p.Hkv *
                                       kv4_block(page, D) + kv4_half(slot, 0, D);
    const size_t dst = layer * p.out_layer + b * p.out_seq + (size_t)t * blocks * 16;
#pragma unroll 2
    for (int hb = w.lane; hb < blocks; hb += w.lanes) {
      const int h = hb / kBlocks, c = hb % kBlocks;
      uint2 code[2];
      uint32_t sb[2];
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const uint8_t* block = src + (size_t)h * kv4_block(page, D) + v * (kv4_group(D) / 2);
        code[v] = *reinterpret_cast<const uint2*>(block + place * (D / 2) + c * 8);
        sb[v] = block[8 * D + place * kBlocks + c];
      }
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const float s = id < 0 ? 0.0f : half2_to_float2(kv4_scales(sb[v])).x * unit[v];
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t h4[4];
          kv4_unpack(e ? code[v].y : code[v].x, h4);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = half2_to_float2(h4[j]);
            o[4 * e + j] = id < 0 ? 0u : pack_bf16(f.x * s, f.y * s);
          }
        }
        uint4* out = reinterpret_cast<uint4*>((v ? p.v_out : p.k_out) + dst + hb * 16);
        if (wide) {
          asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out), "r"(o[0]),
                       "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                       : "memory");
        } else {
          out[0] = make_uint4(o[0], o[1], o[2], o[3]);
          out[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
      }
    }
  }
}

}  // namespace sv
