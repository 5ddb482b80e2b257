// sv_pages.cuh -- pages of a key-value cache that sequences share: forks (new
// sequences take their parents' pages, copy what both would write, get fresh
// pages to grow into, and what nobody holds is free) and compaction.
//
// Which page is whose follows from the tables alone: no counts or free lists
// are kept between calls.  A plan kernel reads the tables, marks the pages that
// the new ones hold in a bitmap, ranks the free ones by prefix sums over its
// words and writes the new tables and a list of page copies; a second kernel
// carries the copies out over all planes.
//
// Bound: the copies, where there are many (compaction of 24 sequences in 32 planes
// of 64 positions, 993 MB read and written: 144-152 us, up to 98% of the rate of a plain
// copy); else the plan's chain of dependent loads.
#pragma once

#include "spec_verify.h"
#include "sv_kv4.cuh"

namespace sv {

constexpr unsigned kFlagNoPage = 256u;
constexpr int kPgThreads = 1024;
constexpr int kPgMaxCluster = 8;
constexpr int kPgCopyThreads = 256;
constexpr int kPgCopyVecs = 8;  // 16-byte vectors of a thread in flight

struct PagesParams {
  uint8_t* pages;          // [planes][n_pages][page_bytes], planes plane_stride apart
  const int32_t* table;    // [B, W]
  const int32_t* length;   // fork: [B]
  const int32_t* parent;   // fork: [B2] or null (each its own)
  const int32_t* need;     // fork: [B2] or null
  int32_t* new_table;      // [B2, W]
  int32_t* new_len;        // fork: [B2]
  int32_t* used;           // [1]
  unsigned* flags;
  uint32_t* bits;          // [words] pages held
  int32_t* mark;           // [n_pages] fork: lowest taker of an unfinished page; compact: new place
  int32_t* free_ids;       // [n_pages] the free pages, ascending
  int32_t* off;            // [B2] fork: fresh pages of the sequences before
  int2* copies;            // [max(B2, n_pages)] from, to
  int32_t* ncopies;        // [1]
  long long plane_stride, page_bytes;
  int planes, n_pages, B, B2, W, page, words;
};

__device__ __forceinline__ void pg_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ unsigned pg_cluster_rank() {
  unsigned r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ unsigned pg_cluster_size() {
  unsigned r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

// Exclusive prefix of v over the block's threads; *total their sum.  Two block
// barriers.
__device__ __forceinline__ int pg_scan(int v, int* total, int* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  const int mine = s_warp[lane];
  int x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  *total = __shfl_sync(0xffffffffu, x, 31);
  return __shfl_sync(0xffffffffu, x - mine, warp) + incl - v;
}

__device__ __forceinline__ void pg_hold(const PagesParams& p, int id) {
  const uint32_t bit = 1u << (id & 31);
  uint32_t* word = p.bits + (id >> 5);
  if (!(__ldcg(word) & bit)) atomicOr(word, bit);  // shared pages are held many times
}
__device__ __forceinline__ bool pg_held(const PagesParams& p, int id) {
  return (__ldcg(p.bits + (id >> 5)) >> (id & 31)) & 1;
}
// What the sequences want in all may be more than 2^31 pages (2^20 sequences of 2^20);
// that more than the pool's pages are wanted is all that counts then.  So the sum of
// the turns before, of kPgThreads sequences each, stops at kPgMany, above any pool,
// and the place of a sequence's page (the turns before, at most a turn's pages before
// it, its own) stays below 2^31.
constexpr int kPgMany = 2 * SPEC_KV_MAX_PAGES;
static_assert((long long)kPgMany + (long long)kPgThreads * SPEC_KV_MAX_TABLE + SPEC_KV_MAX_TABLE <= 0x7FFFFFFF,
              "places of fresh pages fit 32 bits");
__host__ __device__ constexpr int pg_many(int before, int sum) {
  return before + sum < kPgMany ? before + sum : kPgMany;
}

// bits of word w that stand for pages
__device__ __forceinline__ uint32_t pg_valid(const PagesParams& p, int w) {
  const int left = p.n_pages - 32 * w;
  return left >= 32 ? 0xFFFFFFFFu : (1u << left) - 1u;
}

// What new sequence j takes: its parent's row, length, whole pages, whether an
// unfinished page follows, and the pages it is to have.
struct PgTake {
  int row, len, full, pages;
  bool part;
  int open;  // the unfinished page, -1 if none or not a page
};
__device__ __forceinline__ PgTake pg_take(const PagesParams& p, int j, bool flag) {
  PgTake t;
  const int par = p.parent ? p.parent[j] : j;
  unsigned bad = 0;
  t.row = par;
  t.len = 0;
  if (par < -1 || par >= p.B) {
    bad |= kFlagBadParent;
    t.row = -1;
  }
  const long long most = (long long)p.W * p.page;
  long long need = 0;
  if (t.row >= 0) {
    t.len = p.length[t.row];
    if (t.len < 0 || t.len > most) {
      bad |= kFlagBadPath;
      t.len = 0;
    }
    need = p.need ? max(p.need[j], t.len) : t.len;
    if (need > most) {
      bad |= kFlagBadPath;
      need = most;
    }
  }
  t.full = t.len / p.page;
  t.part = t.len - t.full * p.page > 0;
  t.pages = (int)((need + p.page - 1) / p.page);
  t.open = -1;
  if (t.part) {
    t.open = p.table[(size_t)t.row * p.W + t.full];
    if (t.open < 0 || t.open >= p.n_pages) {
      bad |= kFlagBadPage;
      t.open = -1;
    }
  }
  if (flag && bad) set_flag(p.flags, bad);
  return t;
}

__global__ void __launch_bounds__(kPgThreads) pages_fork_kernel(const PagesParams p) {
  __shared__ int s_warp[32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int rank = (int)pg_cluster_rank(), ranks = (int)pg_cluster_size();
  const int me = rank * kPgThreads + threadIdx.x, all = ranks * kPgThreads;
  const int lane = threadIdx.x & 31;
  for (int w = me; w < p.words; w += all) p.bits[w] = 0;
  for (int j = me; j < p.B2; j += all) {
    const PgTake t = pg_take(p, j, true);
    if (t.open >= 0) p.mark[t.open] = 0x7FFFFFFF;
  }
  if (me == 0) *p.ncopies = 0;
  pg_sync();
  // whole pages are held by all that take them; of those that take an
  // unfinished page, the lowest may go on in it
  for (int j = me >> 5; j < p.B2; j += all >> 5) {
    const PgTake t = pg_take(p, j, false);
    const int32_t* row = p.table + (size_t)max(t.row, 0) * p.W;
    for (int i = lane; i < t.full; i += 32) {
      const int id = row[i];
      if (id >= 0 && id < p.n_pages)
        pg_hold(p, id);
      else
        set_flag(p.flags, kFlagBadPage);
    }
    if (lane == 0 && t.open >= 0) atomicMin(p.mark + t.open, j);
  }
  pg_sync();
  // fresh pages per sequence; an unfinished page that its taker keeps is held
  // (others that take it copy it whatever the bit says, since they are not the
  // lowest).  p.off holds 2 fresh + keep until it is summed up.
  for (int j = me; j < p.B2; j += all) {
    const PgTake t = pg_take(p, j, false);
    const bool keep = t.open >= 0 && __ldcg(p.mark + t.open) == j && !pg_held(p, t.open);
    // (an unfinished page that is none: a fresh one takes its place)
    p.off[j] = 2 * max(0, t.pages - t.full - keep) + keep;
  }
  pg_sync();
  for (int j = me; j < p.B2; j += all)
    if (__ldcg(p.off + j) & 1) {
      const PgTake t = pg_take(p, j, false);
      pg_hold(p, t.open);
    }
  pg_sync();
  // the free pages in order: every CTA sums up all words, and lists those of its turn
  int nfree = 0;
  for (int w0 = 0, turn = 0; w0 < p.words; w0 += kPgThreads, ++turn) {
    const int w = w0 + threadIdx.x;
    uint32_t f = w < p.words ? ~__ldcg(p.bits + w) & pg_valid(p, w) : 0u;
    int sum;
    int at = nfree + pg_scan(__popc(f), &sum, s_warp);
    nfree += sum;
    if (turn % ranks == rank)
      while (f) {
        p.free_ids[at++] = 32 * w + __ffs(f) - 1;
        f &= f - 1;
      }
  }
  pg_sync();
  // the new rows, a warp each: every CTA sums up the fresh pages of the
  // sequences before, 1024 at a time
  __shared__ int s_before[kPgThreads], s_keep[kPgThreads];
  int nfresh = 0;
  for (int j0 = 0; j0 < p.B2; j0 += kPgThreads) {
    const int j = j0 + threadIdx.x;
    const int x = j < p.B2 ? __ldcg(p.off + j) : 0;
    int sum;
    const int before = nfresh + pg_scan(x >> 1, &sum, s_warp);
    nfresh = pg_many(nfresh, sum);
    s_before[threadIdx.x] = before;
    s_keep[threadIdx.x] = x & 1;
    __syncthreads();
    for (int k = (me >> 5); k < min(kPgThreads, p.B2 - j0); k += all >> 5) {
      const int jj = j0 + k;
      const PgTake t = pg_take(p, jj, false);
      const int kept = t.full + s_keep[k];
      const int32_t* row = p.table + (size_t)max(t.row, 0) * p.W;
      for (int i = lane; i < p.W; i += 32) {
        int id = -1;
        if (i < kept) {
          id = row[i];
          if (id < 0 || id >= p.n_pages) id = -1;
        } else if (i < t.pages) {
          const int r = s_before[k] + i - kept;
          if (r < nfree)
            id = __ldcg(p.free_ids + r);
          else
            set_flag(p.flags, kFlagNoPage);
          if (i == t.full && t.open >= 0 && id >= 0)
            p.copies[atomicAdd(p.ncopies, 1)] = make_int2(t.open, id);
        }
        p.new_table[(size_t)jj * p.W + i] = id;
      }
      if (lane == 0) p.new_len[jj] = t.len;
    }
  }
  if (me == 0) *p.used = p.n_pages - nfree + min(nfresh, nfree);
}

__global__ void __launch_bounds__(kPgThreads) pages_compact_kernel(const PagesParams p) {
  __shared__ int s_warp[32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int rank = (int)pg_cluster_rank(), ranks = (int)pg_cluster_size();
  const int me = rank * kPgThreads + threadIdx.x, all = ranks * kPgThreads;
  const long long entries = (long long)p.B * p.W;
  for (int w = me; w < p.words; w += all) p.bits[w] = 0;
  pg_sync();
  for (long long i = me; i < entries; i += all) {
    const int id = p.table[i];
    if (id >= 0 && id < p.n_pages)
      pg_hold(p, id);
    else if (id >= 0)
      set_flag(p.flags, kFlagBadPage);
  }
  pg_sync();
  // pages held, and how many of them stay where they are (below that number)
  int held = 0, below = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int v = 0;
    for (int w = threadIdx.x; w < p.words; w += kPgThreads) {
      const int left = held - 32 * w;
      const uint32_t m = pass == 0 || left >= 32 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << left) - 1u;
      v += __popc(__ldcg(p.bits + w) & m);
    }
    int sum;
    pg_scan(v, &sum, s_warp);
    (pass == 0 ? held : below) = sum;
  }
  // the k-th free place below `held` takes the k-th page from there on
  int run = 0;  // pages held before the words
  for (int w0 = 0, turn = 0; w0 < p.words; w0 += kPgThreads, ++turn) {
    const int w = w0 + threadIdx.x;
    const uint32_t b = w < p.words ? __ldcg(p.bits + w) : 0u;
    int sum;
    int at = run + pg_scan(__popc(b), &sum, s_warp);
    run += sum;
    if (turn % ranks != rank || w >= p.words) continue;
    const int left = held - 32 * w;
    const uint32_t m = left >= 32 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << left) - 1u;
    uint32_t f = ~b & m;
    int k = 32 * w - at;  // free places before the word
    while (f) {
      p.copies[k++].y = 32 * w + __ffs(f) - 1;
      f &= f - 1;
    }
    uint32_t up = b & ~m;
    k = at + __popc(b & m) - below;
    while (up) {
      const int id = 32 * w + __ffs(up) - 1;
      p.copies[k].x = id;
      p.mark[id] = k++;
      up &= up - 1;
    }
  }
  pg_sync();
  for (long long i = me; i < entries; i += all) {
    int id = p.table[i];
    if (id < 0 || id >= p.n_pages)
      id = -1;
    else if (id >= held)
      id = __ldcg(&p.copies[__ldcg(p.mark + id)].y);
    p.new_table[i] = id;
  }
  if (me == 0) {
    *p.used = held;
    *p.ncopies = held - below;
  }
}

// The same two plans in one CTA's shared memory, where the tables are small: a
// plan is a chain of dependent loads, and what counts is how few there are
// (four beams of 19 pages 10.7 -> 5.4 us with the copies, 64 of up to 17 pages
// 28 -> 24, compaction of three sequences 6.1 -> 4.8).
constexpr int kPgSmallRows = 512;     // new sequences
constexpr int kPgSmallWords = kPgThreads;
constexpr int kPgSmallFree = 4096;    // free pages listed in shared memory (others in the workspace)

__global__ void __launch_bounds__(kPgThreads) pages_fork_small_kernel(const PagesParams p) {
  __shared__ int s_warp[32];
  __shared__ uint32_t s_bits[kPgSmallWords];
  __shared__ int s_row[kPgSmallRows], s_len[kPgSmallRows], s_full[kPgSmallRows], s_pages[kPgSmallRows];
  __shared__ int s_open[kPgSmallRows], s_kept[kPgSmallRows], s_before[kPgSmallRows];
  __shared__ int s_free[kPgSmallFree];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  s_bits[threadIdx.x] = 0;
  if (threadIdx.x == 0) *p.ncopies = 0;
  const int j = threadIdx.x;
  const bool mine = j < p.B2;
  PgTake t;
  t.open = -1;
  if (mine) {
    t = pg_take(p, j, true);
    s_row[j] = t.row;
    s_len[j] = t.len;
    s_full[j] = t.full;
    s_pages[j] = t.pages;
    s_open[j] = t.open;
  }
  __syncthreads();
  for (int k = warp; k < p.B2; k += kPgThreads / 32) {
    const int32_t* row = p.table + (size_t)max(s_row[k], 0) * p.W;
    for (int i = lane; i < s_full[k]; i += 32) {
      const int id = row[i];
      if (id >= 0 && id < p.n_pages)
        atomicOr(&s_bits[id >> 5], 1u << (id & 31));
      else
        set_flag(p.flags, kFlagBadPage);
    }
  }
  __syncthreads();
  // of those that take an unfinished page, the lowest may go on in it, unless it
  // is held as a full one
  bool keep = mine && t.open >= 0 && !((s_bits[t.open >> 5] >> (t.open & 31)) & 1);
  if (keep)
    for (int i = 0; i < j; ++i)
      if (s_open[i] == t.open) {
        keep = false;
        break;
      }
  __syncthreads();
  if (keep) atomicOr(&s_bits[t.open >> 5], 1u << (t.open & 31));
  int nfresh;
  const int before = pg_scan(mine ? max(0, t.pages - t.full - keep) : 0, &nfresh, s_warp);
  if (mine) {
    s_kept[j] = t.full + keep;
    s_before[j] = before;
  }
  __syncthreads();
  uint32_t f = j < p.words ? ~s_bits[j] & pg_valid(p, j) : 0u;
  int nfree;
  int at = pg_scan(__popc(f), &nfree, s_warp);
  while (f && at < nfresh) {
    const int id = 32 * j + __ffs(f) - 1;
    if (at < kPgSmallFree)
      s_free[at] = id;
    else
      p.free_ids[at] = id;
    ++at;
    f &= f - 1;
  }
  __syncthreads();
  for (int k = warp; k < p.B2; k += kPgThreads / 32) {
    const int32_t* row = p.table + (size_t)max(s_row[k], 0) * p.W;
    const int kept = s_kept[k], pages = s_pages[k];
    for (int i = lane; i < p.W; i += 32) {
      int id = -1;
      if (i < kept) {
        id = row[i];
        if (id < 0 || id >= p.n_pages) id = -1;
      } else if (i < pages) {
        const int r = s_before[k] + i - kept;
        if (r < nfree)
          id = r < kPgSmallFree ? s_free[r] : __ldcg(p.free_ids + r);
        else
          set_flag(p.flags, kFlagNoPage);
        if (i == s_full[k] && s_open[k] >= 0 && id >= 0)
          p.copies[atomicAdd(p.ncopies, 1)] = make_int2(s_open[k], id);
      }
      p.new_table[(size_t)k * p.W + i] = id;
    }
    if (lane == 0) p.new_len[k] = s_len[k];
  }
  if (threadIdx.x == 0) *p.used = p.n_pages - nfree + min(nfresh, nfree);
}

__global__ void __launch_bounds__(kPgThreads) pages_compact_small_kernel(const PagesParams p) {
  __shared__ int s_warp[32];
  __shared__ uint32_t s_bits[kPgSmallWords];
  __shared__ int s_rank[kPgSmallWords];  // pages held before the word
  __shared__ int s_free[kPgSmallFree];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  s_bits[threadIdx.x] = 0;
  __syncthreads();
  const int entries = p.B * p.W;  // (few)
  for (int i = threadIdx.x; i < entries; i += kPgThreads) {
    const int id = p.table[i];
    if (id >= 0 && id < p.n_pages)
      atomicOr(&s_bits[id >> 5], 1u << (id & 31));
    else if (id >= 0)
      set_flag(p.flags, kFlagBadPage);
  }
  __syncthreads();
  const int w = threadIdx.x;
  const uint32_t b = s_bits[w];
  int held;
  const int before = pg_scan(__popc(b), &held, s_warp);
  s_rank[w] = before;
  const int left = held - 32 * w;
  const uint32_t m = left >= 32 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << left) - 1u;
  // the k-th free place below `held` takes the k-th page from there on
  uint32_t f = ~b & m;
  for (int k = 32 * w - before; f; ++k) {
    const int id = 32 * w + __ffs(f) - 1;
    if (k < kPgSmallFree) s_free[k] = id;
    p.copies[k].y = id;
    f &= f - 1;
  }
  int below;
  pg_scan(__popc(b & m), &below, s_warp);
  uint32_t up = b & ~m;
  for (int k = before + __popc(b & m) - below; up; ++k) {
    p.copies[k].x = 32 * w + __ffs(up) - 1;
    up &= up - 1;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < entries; i += kPgThreads) {
    int id = p.table[i];
    if (id < 0 || id >= p.n_pages) {
      id = -1;
    } else if (id >= held) {
      const int k = s_rank[id >> 5] + __popc(s_bits[id >> 5] & ((1u << (id & 31)) - 1u)) - below;
      id = k < kPgSmallFree ? s_free[k] : __ldcg(&p.copies[k].y);
    }
    p.new_table[i] = id;
  }
  if (threadIdx.x == 0) {
    *p.used = held;
    *p.ncopies = held - below;
  }
}

// The planned copies, over all planes: units of kPgCopyThreads x kPgCopyVecs
// vectors of a page's plane.
__global__ void __launch_bounds__(kPgCopyThreads) pages_copy_kernel(const PagesParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int n = *p.ncopies;
  const long long vecs = p.page_bytes / 16;
  const long long chunks = (vecs + kPgCopyThreads * kPgCopyVecs - 1) / (kPgCopyThreads * kPgCopyVecs);
  const long long units = (long long)n * p.planes * chunks;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const long long pc = u / chunks, chunk = u - pc * chunks;
    const long long k = pc / p.planes, plane = pc - k * p.planes;
    const int2 c = p.copies[k];
    uint8_t* base = p.pages + plane * p.plane_stride;
    const uint4* src = reinterpret_cast<const uint4*>(base + c.x * p.page_bytes);
    uint4* dst = reinterpret_cast<uint4*>(base + c.y * p.page_bytes);
    const long long v0 = chunk * kPgCopyThreads * kPgCopyVecs + threadIdx.x;
    uint4 x[kPgCopyVecs];
#pragma unroll
    for (int i = 0; i < kPgCopyVecs; ++i)
      if (v0 + i * kPgCopyThreads < vecs) x[i] = src[v0 + i * kPgCopyThreads];
#pragma unroll
    for (int i = 0; i < kPgCopyVecs; ++i)
      if (v0 + i * kPgCopyThreads < vecs) dst[v0 + i * kPgCopyThreads] = x[i];
  }
}

}  // namespace sv
