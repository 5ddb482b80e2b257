// sv_beam.cuh -- beam search's selection: the M best continuations over all
// beams and tokens of a request.
//
//   total[b, k, v] = score[b, k] + z[b, k, v] / T - ln sum_j exp(z[b, k, j] / T)
//
// for the live beams; a finished one has the single candidate (eos, score).
// Larger totals first, then lower beams, then lower tokens.  A request's M best
// are among the M best of its rows, and within a row totals order as logits do.
//
//   beam_rows_*kernel   streams all logits once: per warp and chunk the sum of
//                       exp (relative to the warp's own maximum) and per run of
//                       32 vectors the maximum.  No warp waits for another.
//   beam_select_kernel  a CTA per request, a warp per row: the rows' sums, and
//                       their M best -- which are in the runs with the M largest
//                       maxima, unless one of those shows that a further run
//                       may hold some -- from those runs' logits, read again
//                       (2 M of 500 runs); then the M best of the rows' candidates
//
// Measured: 64 requests of 8 beams, V = 128256 bf16 (115 MB of live beams), 38 us:
// rows 26-27 (4.3 TB/s, instructions), select 11 (a chain of dependent loads and
// exchanges); 4 beams of one request 10.4-11.4 us.  float32 (230 MB) 56; V = 128255 of
// bf16, no whole number of vectors, 69 (a CTA a chunk and plain loads; float32 56).  The sorted lists of tree growth, one
// per thread, took 40.6 us for the rows; a selection that reads the best runs one
// after the other 24 us, and all of a row's M at once 18.
//
// Totals are float64.  A row's ln sum is rounded to 2^-32, and its sum depends
// on its logits alone (references and order are the chunks' own), so equal rows
// have equal totals.  What a total is off by: of the sum, the exponents' rounding
// 2^-24 of themselves (27 ln 2 on the weights' average, the entropy of 2^26 tokens),
// the exponential 2^-22, 15 additions in float32 2^-24 each; and the scale's rounding,
// 2^-24 of what z_v / T lies from the weights' average, itself within ln V <= 18 of
// the largest: 2^-24 (18.7 + 4 + 15 + 18) < 2^-18, and 2^-24 of the distance from
// the largest.
#pragma once

#include "sv_grow.cuh"
#include "sv_kv4.cuh"

namespace sv {

constexpr int kBeamThreads = 512;
constexpr int kBeamWarps = kBeamThreads / 32;
constexpr int kBeamMaxK = 64;   // beams of a request
constexpr int kBeamMaxM = 16;   // candidates
constexpr int kBeamRuns = kVecPerThread * kWarps;  // runs of a chunk
constexpr int kBeamStage = 1280;  // runs of a row that fit in a warp's shared memory

struct BeamParams {
  const void* logits;        // [B, K, V]
  const float* score;        // [B, K]
  const int32_t* finished;   // [B, K] or null
  float2* part;              // [B K, nchunks, kWarps]: reference (bits), sum
  float* runs;               // [B K, nchunks, kBeamRuns]: maxima
  float* out_score;          // [B, M]
  int32_t* out_parent;       // rows b K + k
  int32_t* out_token;
  int32_t* out_finished;
  unsigned* flags;
  float scale;               // log2(e) / T
  int B, K, V, M, eos, nchunks, items;
};

// A warp's sum of 2^(z scale) relative to its reference, the next whole number from
// its largest logit m's power on.  Beyond 2^30 there are no such numbers, and powers of
// two float logits are 64 or more apart (2^30 2^-24): the sum is then the number of
// logits equal to m, relative to m itself, and the reference says so.
constexpr float kBeamFar = 1073741824.0f;
constexpr int kBeamFarRef = 0x7FFFFFFF;
__device__ __forceinline__ bool beam_far(float m, float scale) {
  return !(fabsf(ceilf(m * scale)) < kBeamFar);
}

// A chunk's records, from its logits in registers.
template <typename E>
__device__ __forceinline__ void beam_chunk(const BeamParams& p, const uint4 (&raw)[kVecPerThread],
                                           int item) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float top[kVecPerThread];
#pragma unroll
  for (int q = 0; q < kVecPerThread; ++q)
    top[q] = grow_funkey(__reduce_max_sync(0xffffffffu, grow_fkey(grow_vec_max<E>(raw[q]))));
  const float m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
  int bits = kRefEmpty;
  float total = 0.0f;
  if (!beam_far(m, p.scale)) {
    const float ref = ceilf(m * p.scale);
    const unsigned long long s2 = f2pack(p.scale, p.scale);
    const unsigned long long n2 = f2pack(-ref, -ref);
    constexpr int kP = E::kEPV / 2;
    unsigned long long sum[2] = {0, 0};
#pragma unroll
    for (int q = 0; q < kVecPerThread; ++q) {
      unsigned long long pr[kP];
      vec_pairs<E>(raw[q], pr);
#pragma unroll
      for (int h = 0; h < kP; ++h) {
        float x0, x1;
        f2unpack(fma2(pr[h], s2, n2), x0, x1);
        sum[h & 1] = add2(sum[h & 1], f2pack(ex2(x0), ex2(x1)));
      }
    }
    float a0, a1;
    f2unpack(add2(sum[0], sum[1]), a0, a1);
    total = warp_sum_f(a0 + a1);
    bits = (int)ref;
  } else if (m > -INFINITY) {
    int n = 0;
#pragma unroll
    for (int q = 0; q < kVecPerThread; ++q)
#pragma unroll
      for (int e = 0; e < E::kEPV; ++e) n += E::elem(raw[q], e) == m ? 1 : 0;
    total = (float)__reduce_add_sync(0xffffffffu, n);
    bits = kBeamFarRef;
  }
  if (lane == 0) {
    p.part[(size_t)item * kWarps + warp] = make_float2(__int_as_float(bits), total);
    float* run = p.runs + (size_t)item * kBeamRuns + warp;  // (their order is the tokens')
#pragma unroll
    for (int q = 0; q < kVecPerThread; ++q) run[q * kWarps] = top[q];
  }
}

// One CTA per item (row, chunk), plain loads (any row size and alignment).
template <typename E>
__global__ void __launch_bounds__(kThreads, 2) beam_rows_kernel(const BeamParams p) {
  using St = typename E::storage;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int item = blockIdx.x, row = item / p.nchunks, c = item - row * p.nchunks;
  if (p.finished && p.finished[row]) return;
  const int j0 = c * E::kChunk, j1 = min(p.V, j0 + E::kChunk);
  uint4 raw[kVecPerThread];
  load_chunk_regs<E, false>(reinterpret_cast<const St*>(p.logits) + (size_t)row * p.V, j0, j1, raw);
  beam_chunk<E>(p, raw, item);
}

// Persistent CTAs over contiguous item ranges, the chunks streamed through the
// bulk-copy ring of the verification kernels (rows of whole 16-byte vectors).
template <typename E>
__global__ void __launch_bounds__(kThreads, 2) beam_rows_stream_kernel(const BeamParams p) {
  extern __shared__ __align__(128) uint8_t stage_mem[];
  __shared__ Ring ring;
  using St = typename E::storage;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int i0, i1;
  item_range(p.items, i0, i1);
  asm volatile("griddepcontrol.launch_dependents;");
  if (i0 >= i1) return;
  const int C = p.nchunks;
  int nrow = i0 / C, nc = i0 % C;  // the next item thread 0 issues (in order)
  bool skip = false;               // its beam is finished: nothing of it is needed
  auto look = [&]() { skip = p.finished && p.finished[nrow]; };
  if (threadIdx.x == 0) look();
  auto issue = [&](int item, int slot) {
    const int j0 = nc * E::kChunk, j1 = min(p.V, j0 + E::kChunk);
    const unsigned bytes = skip ? 0u : (unsigned)(j1 - j0) * (unsigned)sizeof(St);
    mbar_expect_tx(&ring.full[slot], bytes);
    if (!skip)
      bulk_g2s(stage_mem + (size_t)slot * kChunkBytes,
               reinterpret_cast<const St*>(p.logits) + (size_t)nrow * p.V + j0, bytes,
               &ring.full[slot]);
    if (++nc == C) {
      nc = 0;
      ++nrow;
      if (item + 1 < i1) look();
    }
  };
  int issued = ring_init(ring, i0, i1, issue);
  int slot = 0;
  unsigned par = 0;
  int c = i0 % C;
  for (int it = i0; it < i1; ++it) {
    const int j0 = c * E::kChunk, j1 = min(p.V, j0 + E::kChunk);
    uint4 raw[kVecPerThread];
    ring_take<E>(ring, stage_mem, slot, par, (j1 - j0) / E::kEPV, p.flags, raw);
    if (threadIdx.x == 0)
      issued = ring_refill(ring, slot, par, it + kStages, i1, issued, p.flags, issue);
    beam_chunk<E>(p, raw, it);  // (of a finished beam: whatever the stage held, unused)
    if (++c == C) c = 0;
    if (++slot == kStages) {
      slot = 0;
      par ^= 1u;
    }
  }
  if (threadIdx.x == 0) ring_drain(ring, i0, issued);
}

// ln(k / 16), k = 16 .. 32
__constant__ double kBeamLn[17] = {
    0.0, 0.06062462181643484, 0.11778303565638346, 0.17185025692665923,
    0.22314355131420976, 0.27193371548364176, 0.3184537311185346, 0.3629054936893685,
    0.4054651081081644, 0.44628710262841953, 0.4855078157817008, 0.5232481437645479,
    0.5596157879354227, 0.5947071077466928, 0.6286086594223741, 0.661398482245365,
    0.6931471805599453};

// ln(S 2^R) of a positive double-float S to 2^-30: S = m 2^n, the nearest
// c = k / 16 to m, and ln(m / c) = 2 atanh((m - c) / (m + c)) in double-floats
// (a float64 logarithm takes 1.3 us of a warp here: two float64 lanes a clock).
__device__ __forceinline__ double beam_ln(const FSum& S, int R) {
  if (!(S.hi > 0.0f)) return -INFINITY;
  const int n = ((__float_as_int(S.hi) >> 23) & 255) - 127;  // (S is normal: at least one term of
                                                              // 1/2 to 1 is in it)
  const float m = __int_as_float((__float_as_int(S.hi) & 0x007FFFFF) | 0x3F800000);
  const float lo = S.lo * pow2_small(-n);
  const int k = (int)(m * 16.0f + 0.5f);
  const float c = (float)k * 0.0625f;
  const float a = m - c;  // exact
  const float den = __fadd_rn(m, c), den_lo = __fadd_rn(c - __fsub_rn(den, m), lo);
  const float q0 = __fdiv_rn(__fadd_rn(a, lo), den);
  const float r = __fadd_rn(__fmaf_rn(-q0, den, a), __fmaf_rn(-q0, den_lo, lo));
  const float q1 = r / den;
  const float u = q0 * q0;
  const float t = q0 * u * (0.66666667f + u * (0.4f + u * 0.2857143f));
  return (double)(R + n) * 0.6931471805599453 + kBeamLn[k - 16] +
         ((double)(2.0f * q0) + (double)(2.0f * q1 + t));
}

// the double of a grow_key
__device__ __forceinline__ double beam_unkey(unsigned long long k) {
  return __longlong_as_double((long long)((k >> 63) ? (k & 0x7FFFFFFFFFFFFFFFull) : ~k));
}

// Warp argmax over lanes of (v, i), lower i first; the winner to every lane.  (-0
// becomes +0: keys are equal exactly where floats are, as the other compares here.)
__device__ __forceinline__ void beam_warp_best(float& v, int& i) {
  const unsigned key = grow_fkey(v == 0.0f ? 0.0f : v);
  const unsigned top = __reduce_max_sync(0xffffffffu, key);
  i = (int)__reduce_min_sync(0xffffffffu, key == top ? (unsigned)i : 0x7FFFFFFFu);
  v = grow_funkey(top);
}

// A warp's M best so far, the r-th best in lane r, and the last of them.
struct BeamBest {
  float v, last_v;
  int i, last_i;
};

// Adds the elements of a run, E::kEPV to a lane from token j on.
template <typename E>
__device__ __forceinline__ void beam_add(BeamBest& best, const uint4& raw, int j, int V, int M) {
  const int lane = threadIdx.x & 31;
  unsigned left = 0;  // this lane's elements not taken yet
#pragma unroll
  for (int e = 0; e < E::kEPV; ++e)
    if (j + e < V && E::elem(raw, e) > -INFINITY) left |= 1u << e;
#pragma unroll 1
  for (int n = 0; n < 32 * E::kEPV; ++n) {
    float bv = -INFINITY;
    int bi = 0x7FFFFFFF;
#pragma unroll
    for (int e = 0; e < E::kEPV; ++e) {
      const float z = E::elem(raw, e);
      if (((left >> e) & 1) && z > bv) {
        bv = z;
        bi = j + e;
      }
    }
    float v = bv;
    int i = bi;
    beam_warp_best(v, i);
    if (i == 0x7FFFFFFF || !grow_better(v, i, best.last_v, best.last_i)) break;
    const int pos = __popc(__ballot_sync(0xffffffffu, lane < M && grow_better(best.v, best.i, v, i)));
    const float uv = __shfl_up_sync(0xffffffffu, best.v, 1);
    const int ui = __shfl_up_sync(0xffffffffu, best.i, 1);
    if (lane == pos) {
      best.v = v;
      best.i = i;
    } else if (lane > pos) {
      best.v = uv;
      best.i = ui;
    }
    best.last_v = __shfl_sync(0xffffffffu, best.v, M - 1);
    best.last_i = __shfl_sync(0xffffffffu, best.i, M - 1);
    if (bi == i) left &= ~(1u << (i - j));
  }
}

template <typename E, bool kVec>
__global__ void __launch_bounds__(kBeamThreads) beam_select_kernel(const BeamParams p) {
  using St = typename E::storage;
  extern __shared__ __align__(16) uint8_t beam_mem[];
  const int M = p.M, K = p.K, C = p.nchunks, nruns = C * kBeamRuns;
  constexpr int kRun = 32 * E::kEPV;  // tokens of a run
  // candidates of the rows, best first: totals, tokens; the warps' runs
  // (totals as order-preserving integers: float64 compares are slow here)
  unsigned long long* s_tot = reinterpret_cast<unsigned long long*>(beam_mem);
  int* s_tok = reinterpret_cast<int*>(s_tot + K * M);
  float* s_runs = reinterpret_cast<float*>(s_tok + K * M);
  __shared__ uint2 s_cand[kBeamWarps][32];
  __shared__ int s_ncand[kBeamWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  for (int k = warp; k < K; k += kBeamWarps) {
    const size_t row = (size_t)b * K + k;
    unsigned long long* tot = s_tot + k * M;
    int* tok = s_tok + k * M;
    const float score = p.score[row];
    if (p.finished && p.finished[row]) {
      if (lane < M) {
        tot[lane] = grow_key(lane == 0 && score > -INFINITY ? (double)score : -INFINITY);
        tok[lane] = lane == 0 ? p.eos : 0x7FFFFFFF;
      }
      continue;
    }
    // the runs' maxima, run r at lane r mod 32; without room for them the row's
    // own records are used up (they are of no use afterwards)
    float* gruns = p.runs + row * nruns;
    float* runs = gruns;
    if (nruns <= kBeamStage) {
      runs = s_runs + warp * min(nruns, kBeamStage);
#pragma unroll 8
      for (int r = lane; r < nruns; r += 32) runs[r] = __ldcg(gruns + r);
    }
    const float2* part = p.part + row * C * kWarps;
    int lref = kRefEmpty;
    FSum acc = FSum::zero();
    bool some_far = false;
#pragma unroll 4
    for (int i = lane; i < C * kWarps; i += 32) {
      const float2 x = __ldcg(part + i);
      const int ref = __float_as_int(x.x);
      if (ref == kBeamFarRef) {  // 2^-64 and less of the others' sums, unless it is the row's largest
        some_far = true;
        continue;
      }
      if (ref > lref) {
        acc.scale(pow2i_f(lref - ref));
        lref = ref;
      }
      acc.add(x.y * pow2i_f(ref - lref));
    }
    float top = 0.0f;  // what the sum is relative to, besides its reference: 0 or the row's largest logit
    if (__any_sync(0xffffffffu, some_far)) {
      float m = -INFINITY;
      for (int r = lane; r < nruns; r += 32) m = fmaxf(m, __ldcg(gruns + r));
      m = grow_funkey(__reduce_max_sync(0xffffffffu, grow_fkey(m)));
      if (beam_far(m, p.scale)) {
        top = m;
        lref = 0;
        acc = FSum::zero();
        for (int i = lane; i < C * kWarps; i += 32) {  // the warps whose largest it is
          const float* run = gruns + i / kWarps * kBeamRuns + i % kWarps;
          float w = -INFINITY;
#pragma unroll
          for (int q = 0; q < kVecPerThread; ++q) w = fmaxf(w, __ldcg(run + q * kWarps));
          if (w == top) acc.add(__ldcg(part + i).y);
        }
      }
    }
    // this lane's best run that is left
    float rv = -INFINITY;
    int ri = 0x7FFFFFFF;
    auto look = [&]() {
      rv = -INFINITY;
      ri = 0x7FFFFFFF;
#pragma unroll 4
      for (int r = lane; r < nruns; r += 32) {
        const float v = nruns <= kBeamStage ? runs[r] : __ldcg(runs + r);
        if (v > rv) {
          rv = v;
          ri = r;
        }
      }
    };
    auto take = [&](float& v, int& r) {  // the best run of all; 0x7FFFFFFF: none
      v = rv;
      r = ri;
      beam_warp_best(v, r);
      if (r != 0x7FFFFFFF && ri == r) {
        runs[r] = -INFINITY;
        look();
      }
    };
    const St* z = reinterpret_cast<const St*>(p.logits) + row * p.V;
    auto load = [&](int r) {
      uint4 x = make_uint4(E::kNegInfWord, E::kNegInfWord, E::kNegInfWord, E::kNegInfWord);
      const long long j = (long long)r * kRun + lane * E::kEPV;
      if (r == 0x7FFFFFFF || j >= p.V) return x;
      if (kVec) return ldg_stream(z + j);
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        w[q] = E::kNegInfWord;
        const long long e = j + q * (E::kEPV / 4);
        if (E::kEPV == 4) {
          if (e < p.V) w[q] = __float_as_uint(E::load1(z + e));
        } else {
          if (e < p.V) w[q] = (w[q] & 0xFFFF0000u) | (__float_as_uint(E::load1(z + e)) >> 16);
          if (e + 1 < p.V) w[q] = (w[q] & 0xFFFFu) | __float_as_uint(E::load1(z + e + 1));
        }
      }
      return make_uint4(w[0], w[1], w[2], w[3]);
    };
    look();
    BeamBest best{-INFINITY, -INFINITY, 0x7FFFFFFF, 0x7FFFFFFF};
    // At least M runs, and so M elements, reach the M-th largest of the lanes' best
    // runs: the M best elements are among those that do, mostly hardly more than M,
    // in few runs.  They get a lane each and are ranked against one another.
    uint2* cand = s_cand[warp];
    int rank = 0;
#pragma unroll 8
    for (int u = 0; u < 32; ++u) {
      const float v = __shfl_sync(0xffffffffu, rv, u);
      rank += v > rv || (v == rv && u < lane) ? 1 : 0;
    }
    const float thr = __shfl_sync(0xffffffffu, rv, __ffs(__ballot_sync(0xffffffffu, rank == M - 1)) - 1);
    if (lane == 0) s_ncand[warp] = 0;
    __syncwarp();
    int ncand = 33;
    if (thr > -INFINITY) {
#pragma unroll 4
      for (int r = lane; r < nruns; r += 32) {
        const float v = nruns <= kBeamStage ? runs[r] : __ldcg(runs + r);
        if (v >= thr) {
          const int at = atomicAdd(&s_ncand[warp], 1);
          if (at < 32) cand[at] = grow_pack(v, r);
        }
      }
      __syncwarp();
      const int n = s_ncand[warp];
      if (n <= 32) {
        const int mine = lane < n ? (int)cand[lane].y : 0x7FFFFFFF;
        __syncwarp();
        if (lane == 0) s_ncand[warp] = 0;
        __syncwarp();
#pragma unroll 1
        for (int m0 = 0; m0 < n; m0 += 8) {
          uint4 x[8];
          int run[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            run[q] = __shfl_sync(0xffffffffu, mine, (m0 + q) & 31);
            if (m0 + q >= n) run[q] = 0x7FFFFFFF;
            x[q] = load(run[q]);
          }
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            if (run[q] == 0x7FFFFFFF) continue;
            if (!(grow_vec_max<E>(x[q]) >= thr)) continue;
            const int j = run[q] * kRun + lane * E::kEPV;
#pragma unroll
            for (int e = 0; e < E::kEPV; ++e) {
              const float z = E::elem(x[q], e);
              if (z >= thr && j + e < p.V) {
                const int at = atomicAdd(&s_ncand[warp], 1);
                if (at < 32) cand[at] = grow_pack(z, j + e);
              }
            }
          }
        }
        __syncwarp();
        ncand = s_ncand[warp];
      }
    }
    if (ncand <= 32) {
      const uint2 mine = lane < ncand ? cand[lane] : grow_pack(-INFINITY, 0x7FFFFFFF);
      const float v = __uint_as_float(mine.x);
      const int i = (int)mine.y;
      int at = 0;
      for (int u = 0; u < ncand; ++u) at += grow_before(cand[u], v, i) ? 1 : 0;
      __syncwarp();
      if (lane < ncand) cand[at] = mine;  // (distinct tokens: ranks are too)
      __syncwarp();
      if (lane < min(M, ncand)) {
        best.v = __uint_as_float(cand[lane].x);
        best.i = (int)cand[lane].y;
      }
    } else {
      // too many of them (equal logits, or a row of few): run by run, the largest
      // maximum first, while the next may hold something better (equal maxima:
      // lower tokens come first)
#pragma unroll 1
      for (int n = 0; n < nruns; ++n) {
        float v;
        int r;
        take(v, r);
        if (r == 0x7FFFFFFF || !(v > best.last_v || (v == best.last_v && r * kRun < best.last_i))) break;
        beam_add<E>(best, load(r), r * kRun + lane * E::kEPV, p.V, M);
      }
    }
    __syncwarp();
    const int R = warp_max_i(lref);
    acc.scale(pow2i_f(lref - R));
    const FSum S = df_norm(warp_sum_df(acc));
    const double ln2 = 0.6931471805599453;
    const double lse = rint(beam_ln(S, R) * 4294967296.0) * (1.0 / 4294967296.0);
    if (lane < M) {
      const double x = (double)score + (((double)best.v - (double)top) * (double)p.scale * ln2 - lse);
      tot[lane] = grow_key(best.i < p.V && x > -INFINITY ? x : -INFINITY);
      tok[lane] = best.i;
    }
  }
  __syncthreads();
  // rank of each candidate among all: those of other rows are sorted
  for (int e = threadIdx.x; e < K * M; e += kBeamThreads) {
    const int k = e / M, r = e - k * M;
    const unsigned long long x = s_tot[e];
    int rank = r;
    for (int q = 0; q < K && rank < M; ++q) {
      if (q == k) continue;
      const unsigned long long* y = s_tot + q * M;
      int lo = 0, hi = M;  // entries of row q before (x, k)
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (y[mid] > x || (y[mid] == x && q < k))
          lo = mid + 1;
        else
          hi = mid;
      }
      rank += lo;
    }
    if (rank >= M) continue;
    const size_t at = (size_t)b * M + rank;
    const size_t row = (size_t)b * K + k;
    const bool none = x == grow_key(-INFINITY);
    p.out_score[at] = none ? -INFINITY : (float)beam_unkey(x);
    p.out_parent[at] = none ? -1 : (int)row;
    p.out_token[at] = none ? -1 : s_tok[e];
    p.out_finished[at] =
        none || s_tok[e] == p.eos || (p.finished && p.finished[row]) ? 1 : 0;
  }
}

}  // namespace sv
