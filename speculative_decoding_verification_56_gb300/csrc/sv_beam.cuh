// sv_beam.cuh -- beam search's selection: the M best continuations over all
// beams and tokens of a request.
//
//   total[b, k, v] = score[b, k] + z[b, k, v] / T - ln sum_j exp(z[b, k, j] / T)
//
// for the live beams; a finished one has the single candidate (eos, score).
// Larger totals first, then lower beams, then lower tokens.  A request's M best
// are among the M best of its rows, and within a row totals order as logits do:
// the rows are reduced by the streaming top-k of the draft trees (sv_grow.cuh)
// to M candidates and the normaliser, and one CTA per request merges them.
// Totals are float64; a row's ln sum is rounded to 2^-32, so that equal rows
// have equal totals although their sums were cut differently (2^-44).
#pragma once

#include "sv_grow.cuh"

namespace sv {

constexpr int kBeamThreads = 512;
constexpr int kBeamWarps = kBeamThreads / 32;
constexpr int kBeamMaxK = 64;  // beams of a request

struct BeamParams {
  GrowParams rows;  // [B K] rows of nchunks records, K = M candidates each
  const float* score;        // [B, K]
  const int32_t* finished;   // [B, K] or null
  float* out_score;          // [B, M]
  int32_t* out_parent;       // rows b K + k
  int32_t* out_token;
  int32_t* out_finished;
  int B, K, M, eos;
};

__global__ void __launch_bounds__(kBeamThreads) beam_select_kernel(const BeamParams p) {
  extern __shared__ __align__(8) uint8_t beam_mem[];
  const int M = p.M, K = p.K, C = p.rows.nchunks;
  // candidates of the rows, best first: totals, tokens; the lists' heads
  double* s_tot = reinterpret_cast<double*>(beam_mem);
  int* s_tok = reinterpret_cast<int*>(s_tot + K * M);
  uint8_t* s_head = reinterpret_cast<uint8_t*>(s_tok + K * M);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  uint8_t* head = s_head + warp * C;
  for (int k = warp; k < K; k += kBeamWarps) {
    const size_t row = (size_t)b * K + k;
    double* tot = s_tot + k * M;
    int* tok = s_tok + k * M;
    const double score = (double)p.score[row];
    if (p.finished && p.finished[row]) {
      for (int r = lane; r < M; r += 32) {
        tot[r] = r == 0 && score > -INFINITY ? score : -INFINITY;
        tok[r] = r == 0 ? p.eos : 0x7FFFFFFF;
      }
      continue;
    }
    const GrowRec* rec = p.rows.rec + row * C;
    int lref = kRefEmpty;
    FSum acc = FSum::zero();
    for (int c = lane; c < C; c += 32) {
      const int gref = __ldcg(&rec[c].ref);
      FSum v;
      v.hi = __ldcg(&rec[c].hi);
      v.lo = __ldcg(&rec[c].lo);
      head[c] = 0;
      if (gref > lref) {
        acc.scale(pow2i_f(lref - gref));
        lref = gref;
      }
      v.scale(pow2i_f(gref - lref));
      acc = df_add(acc, v);
    }
    const int R = warp_max_i(lref);
    acc.scale(pow2i_f(lref - R));
    const FSum S = df_norm(warp_sum_df(acc));
    const double ln2 = 0.6931471805599453;
    const double lse = rint(((double)R + log2(S.value())) * ln2 * 4294967296.0) * (1.0 / 4294967296.0);
    // M rounds over the chunks' sorted lists, list c at lane c mod 32
    float hv = -INFINITY;  // the best head of this lane's lists
    int hi = 0x7FFFFFFF, hc = -1;
    auto look = [&]() {
      hv = -INFINITY;
      hi = 0x7FFFFFFF;
      hc = -1;
      for (int c = lane; c < C; c += 32) {
        const int h = head[c];
        if (h >= M) continue;
        const float v = __ldcg(&rec[c].val[h]);
        const int i = __ldcg(&rec[c].idx[h]);
        if (grow_better(v, i, hv, hi)) {
          hv = v;
          hi = i;
          hc = c;
        }
      }
    };
    look();
    for (int r = 0; r < M; ++r) {
      float v = hv;
      int i = hi;
      grow_warp_best(v, i);
      if (lane == 0) {
        const double x = score + ((double)v * (double)p.rows.scale * ln2 - lse);
        tot[r] = i < p.rows.V && x > -INFINITY ? x : -INFINITY;
        tok[r] = i;
      }
      if (hc >= 0 && hi == i) {
        ++head[hc];
        look();
      }
    }
  }
  __syncthreads();
  // rank of each candidate among all: those of other rows are sorted
  for (int e = threadIdx.x; e < K * M; e += kBeamThreads) {
    const int k = e / M, r = e - k * M;
    const double x = s_tot[e];
    int rank = r;
    for (int q = 0; q < K && rank < M; ++q) {
      if (q == k) continue;
      const double* y = s_tot + q * M;
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
    const bool none = !(x > -INFINITY);
    p.out_score[at] = none ? -INFINITY : (float)x;
    p.out_parent[at] = none ? -1 : (int)row;
    p.out_token[at] = none ? -1 : s_tok[e];
    p.out_finished[at] =
        none || s_tok[e] == p.eos || (p.finished && p.finished[row]) ? 1 : 0;
  }
}

}  // namespace sv
