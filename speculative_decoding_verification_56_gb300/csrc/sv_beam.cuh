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
  int off_stage, stage;  // shared memory: candidates staged per warp (C M, or 0)
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
  float* cval = reinterpret_cast<float*>(beam_mem + p.off_stage) + (size_t)warp * 2 * p.stage;
  int* cidx = reinterpret_cast<int*>(cval + p.stage);
  for (int k = warp; k < K; k += kBeamWarps) {
    const size_t row = (size_t)b * K + k;
    double* tot = s_tot + k * M;
    int* tok = s_tok + k * M;
    const GrowRec* rec = p.rows.rec + row * C;
    // (all loads of a row at once)
    const float score = p.score[row];
    const bool done = p.finished && p.finished[row];
    int lref = kRefEmpty;
    FSum acc = FSum::zero();
    unsigned live = 0;  // of the first 32 records
    for (int c0 = 0; c0 < C; c0 += 32) {
      const int c = c0 + lane;
      int gref = kRefEmpty;
      FSum v = FSum::zero();
      if (c < C) {
        gref = __ldcg(&rec[c].ref);
        v.hi = __ldcg(&rec[c].hi);
        v.lo = __ldcg(&rec[c].lo);
        head[c] = 0;
      }
      if (c0 == 0) live = __ballot_sync(0xffffffffu, gref != kRefEmpty);
      if (gref > lref) {
        acc.scale(pow2i_f(lref - gref));
        lref = gref;
      }
      v.scale(pow2i_f(gref - lref));
      acc = df_add(acc, v);
    }
    const bool staged = C * M <= p.stage;
    if (staged)
      for (int i = lane; i < C * M; i += 32) {
        const int c = i / M, h = i - c * M;
        cval[i] = __ldcg(&rec[c].val[h]);
        cidx[i] = __ldcg(&rec[c].idx[h]);
      }
    if (done) {
      for (int r = lane; r < M; r += 32) {
        tot[r] = r == 0 && score > -INFINITY ? (double)score : -INFINITY;
        tok[r] = r == 0 ? p.eos : 0x7FFFFFFF;
      }
      __syncwarp();
      continue;
    }
    const int R = warp_max_i(lref);
    acc.scale(pow2i_f(lref - R));
    const FSum S = df_norm(warp_sum_df(acc));
    const double ln2 = 0.6931471805599453;
    const double lse = rint(((double)R + log2(S.value())) * ln2 * 4294967296.0) * (1.0 / 4294967296.0);
    auto put = [&](int r, float v, int i) {
      const double x = (double)score + ((double)v * (double)p.rows.scale * ln2 - lse);
      tot[r] = i < p.rows.V && x > -INFINITY ? x : -INFINITY;
      tok[r] = i;
    };
    __syncwarp();
    const int nl = __popc(live);
    if (staged && C <= 32 && nl * M <= 32) {
      // a row's candidates stand in the records of its segments, mostly one or
      // two: a lane each, ranked against one another by shuffles
      const int j = lane / M, e = lane - j * M;
      float v = -INFINITY;
      int x = 0x7FFFFFFF;
      if (j < nl) {
        unsigned m = live;  // drop the j live records before this lane's
        for (int t = 0; t < j; ++t) m &= m - 1;
        const int at = (__ffs(m) - 1) * M + e;
        v = cval[at];
        x = cidx[at];
      }
      int rank = 0;
#pragma unroll 8
      for (int u = 0; u < 32; ++u) {
        const float vu = __shfl_sync(0xffffffffu, v, u);
        const int xu = __shfl_sync(0xffffffffu, x, u);
        rank += (xu != 0x7FFFFFFF && grow_better(vu, xu, v, x)) ? 1 : 0;
      }
      const bool real = x < p.rows.V;
      // (with fewer than M real ones, -inf in records marked empty: the rounds below)
      if (__popc(__ballot_sync(0xffffffffu, real)) >= M) {
        if (real && rank < M) put(rank, v, x);
        __syncwarp();
        continue;
      }
    }
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
        const float v = staged ? cval[c * M + h] : __ldcg(&rec[c].val[h]);
        const int i = staged ? cidx[c * M + h] : __ldcg(&rec[c].idx[h]);
        if (grow_better(v, i, hv, hi)) {
          hv = v;
          hi = i;
          hc = c;
        }
      }
    };
    look();
    float mv = -INFINITY;  // lane r: the r-th best
    int mi = 0x7FFFFFFF;
    for (int r = 0; r < M; ++r) {
      float v = hv;
      int i = hi;
      grow_warp_best(v, i);
      if (lane == r) {
        mv = v;
        mi = i;
      }
      if (hc >= 0 && hi == i) {
        ++head[hc];
        look();
      }
    }
    if (lane < M) put(lane, mv, mi);
    __syncwarp();
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
