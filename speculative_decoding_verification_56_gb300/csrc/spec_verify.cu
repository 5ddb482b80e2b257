// spec_verify.cu -- C ABI of libspecverify (declared in include/spec_verify.h):
// host-side argument checks, workspace layout and kernel launches.
//
// Workspace layout (all offsets 256-byte aligned):
//   [0, 256)     header; word 0 = sticky device flag bits
//   [256, ...)   per-call scratch records; every record a kernel reads was
//                written earlier in the same call, so the contents on entry
//                do not matter and calls of any shape can share a workspace.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <utility>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "spec_verify.h"
#include "sv_kernels.cuh"
#include "sv_tree.cuh"
#include "sv_lmhead.cuh"
#include "sv_grow.cuh"
#include "sv_rope.cuh"
#include "sv_attn.cuh"
#include "sv_treesample.cuh"
#include "sv_kv4.cuh"
#include "sv_attn4.cuh"
#include "sv_attn4t.cuh"
#include "sv_pages.cuh"
#include "sv_beam.cuh"

static_assert(sv::kMaxDraft == SPEC_MAX_K, "finish kernel buffers are sized for SPEC_MAX_K");

namespace {

std::atomic<uint64_t> g_launches{0};
// limit of the verification kernels' waits on their bulk copies and of the tree
// attention's between its roles (spec_verify_set_wait_limit_ns)
std::atomic<uint64_t> g_wait_limit_ns{sv::kWaitLimitNs};

constexpr size_t kAlign = 256;
constexpr size_t kHeaderBytes = 256;
constexpr size_t kDataOffset = kHeaderBytes;
constexpr int kLmMaxGrid = 1024;  // CTAs (records per row) of the fused LM-head kernel

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

int elem_bytes(int dtype) { return dtype == SPEC_DTYPE_BF16 ? 2 : 4; }
int chunk_elems(int dtype) {
  return dtype == SPEC_DTYPE_BF16 ? sv::BF16::kChunk : sv::F32::kChunk;
}

struct Layout {
  size_t bytes = 0;
  int rows = 0, nchunks = 0;
  size_t off_part = 0, off_desc = 0, off_csum = 0, off_csum_p = 0, off_zx = 0;  // sample
  size_t off_gsum = 0, off_gsum_p = 0;
  size_t off_arg = 0;                                            // greedy / tree
  size_t off_log = 0;  // LM head + sampling: the drawn rows' logits
};

// Returns false for arguments outside the documented limits.
bool make_layout(int mode, int B, int kN, int V, int dtype, Layout* L) {
  if (mode == SPEC_MODE_TREE_MASK || mode == SPEC_MODE_KV_COMMIT ||
      mode == SPEC_MODE_TREE_SAMPLE || mode == SPEC_MODE_TREE_QKV ||
      mode == SPEC_MODE_KV4) {  // the flag header only
    if (B < 0 || kN < 1 || kN > SPEC_MAX_TREE_NODES) return false;
    L->bytes = kHeaderBytes;
    return true;
  }
  if (mode == SPEC_MODE_TREE_GROW) {  // kN = K (children per node); records and node arrays
    const int K = kN;
    if (B < 0 || K < 1 || K > sv::kGrowMaxK || V < K || V > SPEC_MAX_V) return false;
    if (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16) return false;
    const int C = (V + chunk_elems(dtype) - 1) / chunk_elems(dtype);
    if ((long long)C * K > sv::kGrowMaxCand) return false;
    L->nchunks = C;
    size_t off = kDataOffset;
    L->off_part = off;  // GrowRec [B, 1 + (kGrowMaxD - 1) K, C]: every row of up to 16 layers
    off = align_up(off + (size_t)B * (1 + (sv::kGrowMaxD - 1) * K) * C * sizeof(sv::GrowRec));
    L->off_desc = off;  // node values, float64 [B, kGrowMaxNodes]
    off = align_up(off + (size_t)B * sv::kGrowMaxNodes * sizeof(double));
    L->off_gsum = off;  // parent, token, depth [3][B, kGrowMaxNodes]
    off = align_up(off + 3 * (size_t)B * sv::kGrowMaxNodes * sizeof(int32_t));
    L->bytes = off;
    return true;
  }
  if (mode == SPEC_MODE_LM_HEAD_SAMPLE) {
    // statistics records of up to kLmMaxGrid CTAs per row, captured token
    // logits, the draw's structures over fp32 rows, the drawn rows' hidden
    // states [2B, d <= SPEC_LM_MAX_D] and their logits [2B, V] fp32
    if (B < 0 || kN < 0 || kN > SPEC_MAX_K || V < 1 || V > SPEC_MAX_V) return false;
    const long long rows = (long long)B * (2LL * kN + 1);
    if (rows * kLmMaxGrid > 0x7FFFFFFFLL) return false;
    const int C = (V + sv::F32::kChunk - 1) / sv::F32::kChunk;
    if ((long long)B * C * sv::kVecPerChunk > 0x7FFFFFFFLL) return false;
    L->rows = (int)rows;
    L->nchunks = C;
    size_t off = kDataOffset;
    L->off_part = off;
    off = align_up(off + (size_t)rows * kLmMaxGrid * sizeof(sv::SoftmaxPartial));
    L->off_zx = off;
    off = align_up(off + (size_t)rows * sizeof(float));
    L->off_desc = off;
    off = align_up(off + (size_t)B * sizeof(sv::DrawDesc));
    const size_t bc = (size_t)B * C;
    L->off_csum = off;
    off = align_up(off + bc * sizeof(sv::FSum));
    L->off_csum_p = off;
    off = align_up(off + bc * sizeof(sv::FSum));
    L->off_gsum = off;
    off = align_up(off + bc * sv::kVecPerChunk * sizeof(float));
    L->off_gsum_p = off;
    off = align_up(off + bc * sv::kVecPerChunk * sizeof(float));
    L->off_arg = off;
    off = align_up(off + (size_t)2 * B * SPEC_LM_MAX_D * sizeof(uint16_t));
    L->off_log = off;
    off = align_up(off + (size_t)2 * B * V * sizeof(float));
    L->bytes = off;
    return true;
  }
  if (mode == SPEC_MODE_LM_HEAD_GREEDY) {  // argmax records of up to kLmMaxGrid CTAs per row
    if (B < 0 || kN < 0 || kN > SPEC_MAX_K || V < 1 || V > SPEC_MAX_V) return false;
    const long long rows = (long long)B * (kN + 1);
    if (rows * kLmMaxGrid > 0x7FFFFFFFLL) return false;
    L->rows = (int)rows;
    L->nchunks = kLmMaxGrid;
    size_t off = kDataOffset;
    L->off_part = off;
    off = align_up(off + (size_t)rows * kLmMaxGrid * sizeof(sv::ArgPartial));
    L->off_arg = off;
    off = align_up(off + (size_t)rows * sizeof(int32_t));
    L->bytes = off;
    return true;
  }
  if (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16) return false;
  if (B < 0 || V < 1 || V > SPEC_MAX_V) return false;
  const int C = (V + chunk_elems(dtype) - 1) / chunk_elems(dtype);
  long long rows;
  if (mode == SPEC_MODE_SAMPLE) {
    if (kN < 0 || kN > SPEC_MAX_K) return false;
    rows = (long long)B * (2LL * kN + 1);
  } else if (mode == SPEC_MODE_GREEDY) {
    if (kN < 0 || kN > SPEC_MAX_K) return false;
    rows = (long long)B * (kN + 1LL);
  } else if (mode == SPEC_MODE_TREE_GREEDY) {
    if (kN < 1 || kN > SPEC_MAX_TREE_NODES) return false;
    rows = (long long)B * kN;
  } else {
    return false;
  }
  if (rows * C > 0x7FFFFFFFLL || (long long)B * C * sv::kVecPerChunk > 0x7FFFFFFFLL) return false;
  L->rows = (int)rows;
  L->nchunks = C;
  size_t off = kDataOffset;
  if (mode == SPEC_MODE_SAMPLE) {
    L->off_part = off;
    off = align_up(off + (size_t)rows * C * sizeof(sv::SoftmaxPartial));
    L->off_desc = off;
    off = align_up(off + (size_t)B * sizeof(sv::DrawDesc));
    const size_t bc = (size_t)B * C;
    L->off_csum = off;
    off = align_up(off + bc * sizeof(sv::FSum));
    L->off_csum_p = off;
    off = align_up(off + bc * sizeof(sv::FSum));
    L->off_gsum = off;
    off = align_up(off + bc * sv::kVecPerChunk * sizeof(float));
    L->off_gsum_p = off;
    off = align_up(off + bc * sv::kVecPerChunk * sizeof(float));
    L->off_zx = off;
    off = align_up(off + (size_t)rows * sizeof(float));
  } else {
    L->off_part = off;
    off = align_up(off + (size_t)rows * C * sizeof(sv::ArgPartial));
    L->off_arg = off;
    off = align_up(off + (size_t)rows * sizeof(int32_t));
  }
  L->bytes = off;
  return true;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Whether two arrays (null: none) share bytes.
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && x < y + nb && y < x + na;
}

// 16-byte vector path: base aligned and every row a whole number of vectors.
bool vec_ok(const void* p, int V, int dtype) {
  return aligned(p, 16) && ((size_t)V * elem_bytes(dtype)) % 16 == 0;
}

template <typename KernelT, typename ParamT>
spec_status_t launch(KernelT kernel, int grid, size_t smem, const ParamT& prm, void* stream,
                     bool pdl, int cluster = 1, int threads = sv::kThreads) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[2];
  unsigned na = 0;
  if (pdl) {
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
  }
  if (cluster > 1) {
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = (unsigned)cluster;
    attr[na].val.clusterDim.y = 1;
    attr[na].val.clusterDim.z = 1;
    ++na;
  }
  cfg.attrs = na ? attr : nullptr;
  cfg.numAttrs = na;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, prm);
  if (e != cudaSuccess) return SPEC_ERR_CUDA;
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return SPEC_OK;
}

// Launch configuration of a programmatic dependent launch (the kernel waits
// for the preceding kernel in the stream with griddepcontrol.wait).
void pdl_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, dim3 grid, dim3 block,
                size_t smem, void* stream) {
  *cfg = cudaLaunchConfig_t{};
  cfg->gridDim = grid;
  cfg->blockDim = block;
  cfg->dynamicSmemBytes = smem;
  cfg->stream = (cudaStream_t)stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg->attrs = attr;
  cfg->numAttrs = 1;
}

// Per-device state the library caches (shared-memory opt-ins, launch shapes,
// the no-allocation array's address) belongs to the device's current context:
// each cache entry records the context's unique id and is redone when the id
// changes (after cudaDeviceReset, for example).
constexpr int kMaxDevices = 64;
constexpr size_t kStreamSmem = (size_t)sv::kStages * sv::kChunkBytes;
std::mutex g_shape_mu;
std::mutex g_ctx_mu;
CUresult (*g_ctx_current)(CUcontext*) = nullptr;
CUresult (*g_ctx_id)(CUcontext, unsigned long long*) = nullptr;

// The current device and the unique id of its (primary) context, creating
// that context if the runtime has not yet done so.
spec_status_t current_context(int* dev, unsigned long long* id) {
  if (cudaGetDevice(dev) != cudaSuccess || *dev < 0 || *dev >= kMaxDevices) return SPEC_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lock(g_ctx_mu);
    if (!g_ctx_current || !g_ctx_id) {
      void* f1 = nullptr;
      void* f2 = nullptr;
      cudaDriverEntryPointQueryResult q1, q2;
      if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &f1, 4000, cudaEnableDefault,
                                           &q1) != cudaSuccess ||
          q1 != cudaDriverEntryPointSuccess || !f1 ||
          cudaGetDriverEntryPointByVersion("cuCtxGetId", &f2, 12000, cudaEnableDefault, &q2) !=
              cudaSuccess ||
          q2 != cudaDriverEntryPointSuccess || !f2)
        return SPEC_ERR_CUDA;
      g_ctx_current = reinterpret_cast<CUresult (*)(CUcontext*)>(f1);
      g_ctx_id = reinterpret_cast<CUresult (*)(CUcontext, unsigned long long*)>(f2);
    }
  }
  CUcontext ctx = nullptr;
  if (g_ctx_current(&ctx) != CUDA_SUCCESS) return SPEC_ERR_CUDA;
  if (ctx == nullptr) {  // the runtime has not made the device's context current yet
    if (cudaSetDevice(*dev) != cudaSuccess || g_ctx_current(&ctx) != CUDA_SUCCESS || !ctx)
      return SPEC_ERR_CUDA;
  }
  return g_ctx_id(ctx, id) == CUDA_SUCCESS ? SPEC_OK : SPEC_ERR_CUDA;
}

// Per-device launch shape of a persistent streaming kernel: the shared-memory
// opt-in is set once per device context, the grid is SMs x resident CTAs per
// SM.
template <auto kernel>
spec_status_t persistent_grid(int items, int* grid) {
  static int cached[kMaxDevices] = {0};  // one table per kernel instantiation
  static unsigned long long cached_ctx[kMaxDevices] = {0};
  int dev = 0;
  unsigned long long ctx = 0;
  if (current_context(&dev, &ctx) != SPEC_OK) return SPEC_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_shape_mu);
  if (cached[dev] == 0 || cached_ctx[dev] != ctx) {
    int sms = 0, per_sm = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)kStreamSmem) != cudaSuccess)
      return SPEC_ERR_CUDA;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return SPEC_ERR_CUDA;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, sv::kThreads,
                                                      kStreamSmem) != cudaSuccess)
      return SPEC_ERR_CUDA;
    cached[dev] = std::max(1, sms * std::max(1, per_sm));
    cached_ctx[dev] = ctx;
  }
  *grid = std::min(items, cached[dev]);
  return SPEC_OK;
}

// Dynamic shared-memory opt-in for a kernel (and, for clusters of more than
// eight CTAs, the opt-in to those), once per device context.
template <auto kernel>
spec_status_t ensure_smem(size_t bytes, bool big_clusters = false) {
  static bool done[kMaxDevices] = {false};
  static unsigned long long done_ctx[kMaxDevices] = {0};
  int dev = 0;
  unsigned long long ctx = 0;
  if (current_context(&dev, &ctx) != SPEC_OK) return SPEC_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_shape_mu);
  if (!done[dev] || done_ctx[dev] != ctx) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) !=
        cudaSuccess)
      return SPEC_ERR_CUDA;
    if (big_clusters && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed,
                                             1) != cudaSuccess)
      return SPEC_ERR_CUDA;
    done[dev] = true;
    done_ctx[dev] = ctx;
  }
  return SPEC_OK;
}

// TMA descriptors of bf16 arrays (innermost dimension first; strides in bytes,
// of the outer dimensions) read in boxes 64 elements wide with 128-byte
// swizzle, out-of-range elements as zero; encode_bf16_kmajor: a row-major
// matrix [outer, inner] in boxes of 64 x box_outer.  The driver's encoder is
// looked up once.
std::mutex g_encode_mu;
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

spec_status_t encode_bf16(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims,
                          const cuuint64_t* strides, const cuuint32_t* box) {
  {
    std::lock_guard<std::mutex> lock(g_encode_mu);
    if (!g_encode) {
      void* fn = nullptr;
      cudaDriverEntryPointQueryResult q;
      if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                           &q) != cudaSuccess ||
          q != cudaDriverEntryPointSuccess || !fn)
        return SPEC_ERR_CUDA;
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
  }
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r =
      g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base),
               dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SPEC_OK : SPEC_ERR_INVALID_ARG;
}

spec_status_t encode_bf16_kmajor(CUtensorMap* map, const void* base, int inner, int outer,
                                 int box_outer) {
  const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
  const cuuint64_t strides[1] = {(cuuint64_t)inner * 2};
  const cuuint32_t box[2] = {(cuuint32_t)sv::kLmBK, (cuuint32_t)box_outer};
  return encode_bf16(map, base, 2, dims, strides, box);
}

// Row groups of an LM-head GEMM: at most kLmMaxRows rows each, split evenly,
// each a multiple of the 64-row H box (so two MMAs of equal N stay multiples
// of 16).  Returns false when the rows need more groups than a grid allows.
bool lm_row_groups(int rows, int* ngroups, int* grp) {
  if (rows <= 0) {
    *ngroups = 0;
    *grp = sv::kLmHBox;
    return true;
  }
  const int gy = (rows + sv::kLmMaxRows - 1) / sv::kLmMaxRows;
  if (gy > 32768) return false;
  *ngroups = gy;
  *grp = ((rows + gy - 1) / gy + sv::kLmHBox - 1) / sv::kLmHBox * sv::kLmHBox;
  return true;
}

// One CTA per SM (the kernel holds the SM's tensor memory and most of its
// shared memory), in pairs: as many pairs as can be resident at once, at most
// one per 256-entry vocabulary tile.  The number of co-resident pairs is
// asked of the runtime once per device and context.
template <int Mode>
spec_status_t lm_grid_x(int ntiles, int* gx) {
  static int pairs_cached[kMaxDevices] = {0};
  static unsigned long long pairs_ctx[kMaxDevices] = {0};
  int dev = 0;
  unsigned long long ctx = 0;
  if (current_context(&dev, &ctx) != SPEC_OK) return SPEC_ERR_CUDA;
  int pairs = 0;
  {
    std::lock_guard<std::mutex> lock(g_shape_mu);
    if (pairs_ctx[dev] == ctx && pairs_cached[dev] > 0) pairs = pairs_cached[dev];
  }
  if (pairs == 0) {
    // the occupancy query sees the kernel's shared-memory opt-in
    const spec_status_t st = ensure_smem<sv::lmhead_kernel<Mode>>((size_t)sv::kLmRingBytes + 1024);
    if (st != SPEC_OK) return st;
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return SPEC_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(2 * std::max(1, sms / 2)), 1, 1);
    cfg.blockDim = dim3(sv::kLmThreads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)sv::kLmRingBytes + 1024;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, sv::lmhead_kernel<Mode>, &cfg) != cudaSuccess)
      return SPEC_ERR_CUDA;
    pairs = std::max(1, std::min(clusters, sms / 2));
    std::lock_guard<std::mutex> lock(g_shape_mu);
    pairs_cached[dev] = pairs;
    pairs_ctx[dev] = ctx;
  }
  *gx = 2 * std::max(1, std::min(std::min(pairs, ntiles), kLmMaxGrid / 2));
  return SPEC_OK;
}

template <int Mode>
spec_status_t launch_lmhead(const CUtensorMap& map_h, const CUtensorMap& map_h1,
                            const CUtensorMap& map_w, const sv::LmHeadParams& lp, int gx, int gy,
                            void* stream) {
  const spec_status_t st =
      ensure_smem<sv::lmhead_kernel<Mode>>((size_t)sv::kLmRingBytes + 1024);
  if (st != SPEC_OK) return st;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  pdl_config(&cfg, attr, dim3((unsigned)gx, (unsigned)gy, 1), dim3(sv::kLmThreads, 1, 1),
             (size_t)lp.nstages * lp.stage_bytes + 1024, stream);
  if (cudaLaunchKernelEx(&cfg, sv::lmhead_kernel<Mode>, map_h, map_h1, map_w, lp) != cudaSuccess)
    return SPEC_ERR_CUDA;
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return SPEC_OK;
}

template <typename E, bool kVec>
spec_status_t run_finish(const sv::SampleParams& prm, void* stream) {
  if (prm.nchunks <= sv::kClusterMaxChunks) {
    const spec_status_t st = ensure_smem<sv::sample_finish_kernel<E, kVec>>(sv::kFinishSmem);
    if (st != SPEC_OK) return st;
    return launch(sv::sample_finish_kernel<E, kVec>, prm.B * sv::kClusterCTAs, sv::kFinishSmem,
                  prm, stream, true, sv::kClusterCTAs);
  }
  const spec_status_t st =
      launch(sv::draw_kernel<E, kVec>, prm.B * prm.nchunks, 0, prm, stream, true);
  if (st != SPEC_OK) return st;
  return launch(sv::draw_resolve_kernel<E, kVec>, prm.B, 0, prm, stream, true);
}

// L2 budget for the rows streamed with a keep hint (well under the 129 MB L2
// of a GB300, so that the rest of the stream does not evict them).
constexpr double kKeepBytes = 80.0 * (1 << 20);

template <typename E>
spec_status_t run_sample(sv::SampleParams prm, int rows, bool vec, void* stream) {
  prm.items = rows * prm.nchunks;
  prm.wait_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  {
    const double pair = 2.0 * prm.B * (double)prm.V * sizeof(typename E::storage);
    prm.keep_pos = pair > 0 ? std::min(prm.k + 1, (int)(kKeepBytes / pair)) : 0;
  }
  spec_status_t st;
  if (vec) {
    int grid = 0;
    st = persistent_grid<sv::stream_stats_kernel<E, false>>(prm.items, &grid);
    if (st != SPEC_OK) return st;
    if (prm.items / grid < sv::kFrontLoadItems) {  // short ranges: start before the wait
      st = persistent_grid<sv::stream_stats_kernel<E, true>>(prm.items, &grid);
      if (st != SPEC_OK) return st;
      st = launch(sv::stream_stats_kernel<E, true>, grid, kStreamSmem, prm, stream, true);
    } else {
      st = launch(sv::stream_stats_kernel<E, false>, grid, kStreamSmem, prm, stream, true);
    }
  } else {
    st = launch(sv::chunk_stats_kernel<E, false>, prm.items, 0, prm, stream, false);
  }
  if (st != SPEC_OK) return st;
  return vec ? run_finish<E, true>(prm, stream) : run_finish<E, false>(prm, stream);
}

template <typename E>
spec_status_t run_argmax(sv::ArgmaxParams prm, int rows, bool vec, void* stream) {
  prm.items = rows * prm.nchunks;
  prm.wait_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  if (vec) {
    int grid = 0;
    spec_status_t st = persistent_grid<sv::stream_argmax_kernel<E>>(prm.items, &grid);
    if (st != SPEC_OK) return st;
    st = launch(sv::stream_argmax_kernel<E>, grid, kStreamSmem, prm, stream, true);
    if (st != SPEC_OK) return st;
  } else {
    const spec_status_t st =
        launch(sv::chunk_argmax_kernel<E, false>, prm.items, 0, prm, stream, false);
    if (st != SPEC_OK) return st;
  }
  return launch(sv::argmax_resolve_kernel, prm.B, 0, prm, stream, true);
}

// Scratch of spec_verify_greedy_noalloc: a fixed array in the library's own
// device memory (one copy per device that loads the library).  Host code may
// not use the symbol as an address; its device address is looked up with
// cudaGetSymbolAddress while the device is current, once per device context.
static __device__ __align__(256) unsigned char g_noalloc_scratch[SPEC_NOALLOC_SCRATCH_BYTES];
void* g_noalloc_addr[kMaxDevices] = {nullptr};
unsigned long long g_noalloc_ctx[kMaxDevices] = {0};
std::mutex g_noalloc_mu;

spec_status_t noalloc_scratch(void** addr) {
  int dev = 0;
  unsigned long long ctx = 0;
  if (current_context(&dev, &ctx) != SPEC_OK) return SPEC_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_noalloc_mu);
  if (g_noalloc_addr[dev] == nullptr || g_noalloc_ctx[dev] != ctx) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || p == nullptr)
      return SPEC_ERR_CUDA;
    g_noalloc_addr[dev] = p;
    g_noalloc_ctx[dev] = ctx;
  }
  *addr = g_noalloc_addr[dev];
  return SPEC_OK;
}

constexpr int kTsMaxSteps = 2048;  // of a warp, whose sums are held in shared memory
constexpr size_t kTsMaxSmem = (size_t)sv::kTsWarps * kTsMaxSteps * sizeof(unsigned long long);

// Tree sampling: a cluster of CTAs per sequence (16 are more than the portable
// 8); the dynamic shared memory holds the sums of the warps' steps.
template <auto kernel>
spec_status_t launch_tree_sample(const sv::TreeSampleParams& prm, int B, int cluster, size_t smem,
                                 void* stream) {
  const spec_status_t st = ensure_smem<kernel>(kTsMaxSmem, true);
  if (st != SPEC_OK) return st;
  return launch(kernel, B * cluster, smem, prm, stream, true, cluster, sv::kTsThreads);
}

// Tiles and partial slots of spec_tree_attention for one call shape.
struct AttnPlan {
  int tok = 0, pair_s = 0, pair_o = 0, mg_s = 0, mg_o = 0, rows_s = 0, rows_o = 0, by_cta = 0;
  long long own0 = 0;  // row of the own items' slot 0, behind the shared ones
  size_t off_ml = 0, off_part = 0, bytes = 0;
};

// Rows of an item: the G query heads of `tok` nodes fill one 128-row half;
// an item with more nodes takes two halves, with fewer one (both halves of
// the kernel then share it by alternate tiles).  Items of one half throughout:
// 79.6 us instead of 69.4 (16 trees of 60), 181 instead of 133 (65536 cached),
// 254 instead of 184 (a shared prefix); two halves throughout: decoding 154.8
// instead of 136.3 us.
// Slots: shared and own items have slots of their own sizes.  Behind a shared
// prefix every item leaves a partial, and each cut one more: items + CTAs slots
// in all.  If CTA c holds the last shared tile, the shared items' slots (item +
// CTA) end below row (items_s + c) rows_s, and the own items' begin at own0 +
// c rows_o, so own0 = items_s rows_s + CTAs (rows_s - rows_o) keeps them apart
// for every c.  Without a prefix, only cut items leave partials, at most two a
// CTA (the item that it begins with and the one that it ends with), which is
// less from kAtMaxCtas items on (by_cta).
AttnPlan attn_plan(int B, int N, int Hq, int Hkv, int D, int P) {
  AttnPlan a;
  const int G = Hq / Hkv;
  a.tok = sv::kAtRows / G;
  const long long all = (long long)B * N;
  a.pair_o = N > a.tok;
  a.mg_o = (N + (a.tok << a.pair_o) - 1) / (a.tok << a.pair_o);
  a.rows_o = std::min(N, a.tok << a.pair_o) * G;
  const size_t items_o = (size_t)B * Hkv * a.mg_o;
  size_t items_s = 0, slots_o = items_o + sv::kAtMaxCtas;
  if (P > 0) {
    a.pair_s = all > a.tok;
    a.mg_s = (int)((all + (a.tok << a.pair_s) - 1) / (a.tok << a.pair_s));
    a.rows_s = (int)std::min<long long>(all, a.tok << a.pair_s) * G;
    items_s = (size_t)Hkv * a.mg_s;
    a.own0 = (long long)items_s * a.rows_s + (long long)sv::kAtMaxCtas * (a.rows_s - a.rows_o);
  } else if (items_o > (size_t)sv::kAtMaxCtas) {
    a.by_cta = 1;
    slots_o = 2 * (size_t)sv::kAtMaxCtas;
  }
  const size_t rows = (size_t)a.own0 + slots_o * a.rows_o;
  a.off_ml = align_up(kDataOffset + (items_s + items_o) * sizeof(int2));
  a.off_part = align_up(a.off_ml + rows * sizeof(float2));
  a.bytes = align_up(a.off_part + rows * D * sizeof(float));
  return a;
}

// Multiprocessors of the current device, once per device context.
spec_status_t sm_count(int* sms) {
  static int cached[kMaxDevices] = {0};
  static unsigned long long cached_ctx[kMaxDevices] = {0};
  int dev = 0;
  unsigned long long ctx = 0;
  if (current_context(&dev, &ctx) != SPEC_OK) return SPEC_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_shape_mu);
  if (cached[dev] == 0 || cached_ctx[dev] != ctx) {
    if (cudaDeviceGetAttribute(&cached[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return SPEC_ERR_CUDA;
    cached_ctx[dev] = ctx;
  }
  *sms = cached[dev];
  return SPEC_OK;
}

template <int D, bool kSet>
spec_status_t launch_attention(const sv::AttnParams& prm, const CUtensorMap (&map)[5],
                               void* stream) {
  const spec_status_t st = ensure_smem<sv::tree_attn_kernel<D, kSet>>((size_t)sv::at_smem<D>());
  if (st != SPEC_OK) return st;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  pdl_config(&cfg, attr, dim3((unsigned)prm.nctas), dim3(sv::kAtThreads), sv::at_smem<D>(), stream);
  if (cudaLaunchKernelEx(&cfg, sv::tree_attn_kernel<D, kSet>, map[0], map[1], map[2], map[3],
                         map[4], prm) != cudaSuccess)
    return SPEC_ERR_CUDA;
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return SPEC_OK;
}

// The join of cut items.
template <int D>
spec_status_t finish_attention(const sv::AttnParams& prm, void* stream) {
  const long long rows = (long long)prm.B * prm.N * prm.Hq;
  const long long blocks = (rows + sv::kAtFinThreads - 1) / sv::kAtFinThreads;
  // Parts of an item: about 1 + CTAs / items.  Many (3 sequences of 65536, 24
  // items): 8 elements a thread of 8 parts at once 132 us, 16 of 4 134, 16 of 2
  // 137; few (16 trees of 60, 128 items): 16 of 2 68.5 us, 16 of 4 69.9, 8 of 8
  // 74.9; a shared prefix (640 items) 181, 183.5 and 194.
  const long long items = (long long)prm.Hkv * (prm.mg_s + (long long)prm.B * prm.mg_o);
  if (2 * items >= prm.nctas)
    return launch(sv::tree_attn_finish_kernel<D, 16, 2>, (int)(blocks * (D / 16)), 0, prm, stream,
                  true, 1, sv::kAtFinThreads);
  return launch(sv::tree_attn_finish_kernel<D, 8, 8>, (int)(blocks * (D / 8)), 0, prm, stream, true,
                1, sv::kAtFinThreads);
}

template <int D>
spec_status_t run_attention(const sv::AttnParams& prm, const CUtensorMap (&map)[5], void* stream) {
  const spec_status_t st = prm.wait_ns == sv::kWaitLimitNs
                               ? launch_attention<D, false>(prm, map, stream)
                               : launch_attention<D, true>(prm, map, stream);
  if (st != SPEC_OK) return st;
  return finish_attention<D>(prm, stream);
}

template <int D>
spec_status_t run_rope(const sv::RopeParams& prm, int mode, int nodes, void* stream) {
  if (mode == sv::kRopeHalves)
    return launch(sv::tree_qkv_rope_kernel<D, sv::kRopeHalves>, nodes, 0, prm, stream, true, 1,
                  sv::kRopeThreads);
  if (mode == sv::kRopePairs)
    return launch(sv::tree_qkv_rope_kernel<D, sv::kRopePairs>, nodes, 0, prm, stream, true, 1,
                  sv::kRopeThreads);
  return launch(sv::tree_qkv_rope_kernel<D, sv::kRopeOdd>, nodes, 0, prm, stream, true, 1,
                sv::kRopeThreads);
}

bool attn_shape_ok(int B, int N, int Hq, int Hkv, int D, int P) {
  return B >= 0 && N >= 1 && N <= SPEC_ATTN_MAX_NODES && Hkv >= 1 && Hq >= Hkv && Hq <= 65536 &&
         Hq % Hkv == 0 && Hq / Hkv <= 128 && (D == 64 || D == 128) && P >= 0 && P <= INT32_MAX - 256 &&
         (long long)B * N <= INT32_MAX / 128 && (long long)B * N * Hq <= INT32_MAX;
}

// --- the 4-bit cache in pages --------------------------------------------------

int log2_of(int x) {  // of a power of two
  int n = 0;
  while ((1 << n) < x) ++n;
  return n;
}

bool kv4_shape_ok(long long n_pages, int page_size, int Hkv, int D, int W) {
  return n_pages >= 1 && n_pages <= INT32_MAX && Hkv >= 1 && Hkv <= 65536 &&
         (D == 64 || D == 128) && W >= 1 && W <= SPEC_KV_MAX_TABLE &&
         (page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128);
}

// Items and partial slots of spec_tree_attention_kv4 for one call shape.
struct Attn4Plan {
  bool tiles = false;  // more rows than the kernel for few serves
  AttnPlan t;          // tiles: items and slots as spec_tree_attention's
  int nt = 1, rows = 0;
  size_t off_ml = 0, off_part = 0, bytes = 0;
};
// Few rows (matrix instructions from registers, no unpacked tiles) against the
// tensor cores' tiles, 64 sequences of about 3000 positions, 8 key-value heads:
// D = 128, 8 rows 71 us against 186, 16 rows 113 / 187, 24 rows 140-146 / 190; D = 64,
// 53 / 158, 87 / 157, 105 / 158; 2 sequences of 22000, D = 128, 24 rows 48 / 58.
constexpr int kA4MaxRows = 24;
static_assert(kA4MaxRows <= 16 * sv::kA4Warps, "an item's nodes are its first unit's");

Attn4Plan attn4_plan(int B, int N, int Hq, int Hkv, int D) {
  Attn4Plan a;
  const long long all = (long long)N * (Hq / Hkv);
  if (all > kA4MaxRows) {
    a.tiles = true;
    a.t = attn_plan(B, N, Hq, Hkv, D, 0);
    a.bytes = a.t.bytes;
    return a;
  }
  a.nt = all <= 8 ? 1 : all <= 16 ? 2 : 3;
  a.rows = (int)all;
  const size_t items = (size_t)B * Hkv;
  const size_t rows = (size_t)2 * sv::kA4MaxCtas * a.rows;
  a.off_ml = align_up(kDataOffset + items * sizeof(int2));
  a.off_part = align_up(a.off_ml + rows * sizeof(float2));
  a.bytes = align_up(a.off_part + rows * D * sizeof(float));
  return a;
}

template <int D, int NT>
spec_status_t launch_attn4(sv::Attn4Params prm, int sms, void* stream) {
  constexpr size_t smem = sv::a4_smem<D, NT>();
  prm.nctas = std::min(sms * sv::a4_per_sm<NT>(), sv::kA4MaxCtas);
  const spec_status_t st = ensure_smem<sv::kv4_attn_rows_kernel<D, NT>>(smem);
  if (st != SPEC_OK) return st;
  const spec_status_t st2 = launch(sv::kv4_attn_rows_kernel<D, NT>, prm.nctas, smem, prm, stream,
                                   true, 1, sv::kA4Threads);
  if (st2 != SPEC_OK) return st2;
  const long long threads = (long long)prm.B * prm.N * prm.Hq * (D / 4);
  return launch(sv::kv4_attn_finish_kernel<D>, (int)((threads + 255) / 256), 0, prm, stream, true,
                1, 256);
}

template <int D>
spec_status_t run_attn4(const sv::Attn4Params& prm, int nt, int sms, void* stream) {
  if (nt == 1) return launch_attn4<D, 1>(prm, sms, stream);
  if (nt == 2) return launch_attn4<D, 2>(prm, sms, stream);
  return launch_attn4<D, 3>(prm, sms, stream);
}

template <int D>
spec_status_t run_attn4_tiles(const sv::AttnQParams& prm, void* stream) {
  spec_status_t st = ensure_smem<sv::kv4_attn_tiles_kernel<D>>((size_t)sv::atq_smem<D>());
  if (st != SPEC_OK) return st;
  st = launch(sv::kv4_attn_tiles_kernel<D>, prm.nctas, sv::atq_smem<D>(), prm, stream, true, 1,
              sv::kAtqThreads);
  if (st != SPEC_OK) return st;
  return finish_attention<D>(prm, stream);
}

// Lanes of an entry and blocks of a (layer, sequence) of the commit and read
// kernels: enough for its most places, and no more than fill the GPU several times.
void kv4_grid(sv::Kv4Params* prm, long long places, int D) {
  prm->lg_lanes = std::min(5, log2_of(prm->Hkv * (D / 16)));
  const long long per_block = sv::kKv4Threads >> prm->lg_lanes;
  const long long most = std::max(1ll, 4864ll / ((long long)prm->layers * prm->B));
  prm->blocks = (int)std::max(1ll, std::min((places + per_block - 1) / per_block, most));
}

struct PagesLayout {
  size_t off_bits = 0, off_mark = 0, off_free = 0, off_off = 0, off_copies = 0, bytes = 0;
};
bool pages_layout(long long n_pages, long long rows, PagesLayout* L) {
  if (n_pages < 1 || n_pages > SPEC_KV_MAX_PAGES || rows < 0 || rows > SPEC_KV_MAX_TABLE)
    return false;
  size_t off = kDataOffset;  // (word 4 of the header's space holds the number of copies)
  L->off_bits = off;
  off = align_up(off + (size_t)((n_pages + 31) / 32) * 4);
  L->off_mark = off;
  off = align_up(off + (size_t)n_pages * 4);
  L->off_free = off;
  off = align_up(off + (size_t)n_pages * 4);
  L->off_off = off;
  off = align_up(off + (size_t)rows * 4);
  L->off_copies = off;
  off = align_up(off + (size_t)std::max(n_pages, rows) * sizeof(int2));
  L->bytes = off;
  return true;
}

// Arguments that both calls on pages share, checked and laid out.
spec_status_t pages_params(void* pages, int planes, long long plane_stride, long long n_pages,
                           long long page_bytes, const int32_t* table, int B, int rows, int W,
                           int32_t* new_table, int32_t* used, void* workspace,
                           size_t workspace_bytes, sv::PagesParams* prm) {
  PagesLayout L;
  if (planes < 1 || planes > 65535 || page_bytes < 16 || B < 0 || W < 1 ||
      W > SPEC_KV_MAX_TABLE || B > SPEC_KV_MAX_TABLE || !pages_layout(n_pages, rows, &L) ||
      page_bytes > INT64_MAX / n_pages ||
      (planes > 1 && plane_stride < n_pages * page_bytes))
    return SPEC_ERR_INVALID_ARG;
  if (!pages || !used || (B > 0 && !table) || (rows > 0 && !new_table)) return SPEC_ERR_INVALID_ARG;
  if (!aligned(pages, 16) || page_bytes % 16 || plane_stride % 16 || !aligned(table, 4) ||
      !aligned(new_table, 4) || !aligned(used, 4))
    return SPEC_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < L.bytes) return SPEC_ERR_WORKSPACE;
  if (!aligned(workspace, kAlign)) return SPEC_ERR_ALIGNMENT;
  char* ws = static_cast<char*>(workspace);
  std::memset(prm, 0, sizeof *prm);
  prm->pages = static_cast<uint8_t*>(pages);
  prm->table = table;
  prm->new_table = new_table;
  prm->used = used;
  prm->flags = reinterpret_cast<unsigned*>(ws);
  prm->ncopies = reinterpret_cast<int32_t*>(ws + 16);
  prm->bits = reinterpret_cast<uint32_t*>(ws + L.off_bits);
  prm->mark = reinterpret_cast<int32_t*>(ws + L.off_mark);
  prm->free_ids = reinterpret_cast<int32_t*>(ws + L.off_free);
  prm->off = reinterpret_cast<int32_t*>(ws + L.off_off);
  prm->copies = reinterpret_cast<int2*>(ws + L.off_copies);
  prm->plane_stride = plane_stride;
  prm->page_bytes = page_bytes;
  prm->planes = planes;
  prm->n_pages = (int)n_pages;
  prm->B = B;
  prm->B2 = rows;
  prm->W = W;
  prm->words = (int)((n_pages + 31) / 32);
  return SPEC_OK;
}

spec_status_t run_pages(bool fork, const sv::PagesParams& prm, void* stream) {
  // one CTA's shared memory where the tables are small, else a cluster with a CTA
  // per 8192 table entries or 1024 words of the bitmap
  const long long entries = (long long)std::max(prm.B, prm.B2) * prm.W;
  spec_status_t st;
  if (prm.words <= sv::kPgSmallWords && entries <= 65536 && prm.B2 <= sv::kPgSmallRows) {
    st = launch(fork ? sv::pages_fork_small_kernel : sv::pages_compact_small_kernel, 1, 0, prm,
                stream, true, 1, sv::kPgThreads);
  } else {
    int cluster = 1;
    while (cluster < sv::kPgMaxCluster &&
           (entries > 8192ll * cluster || prm.words > sv::kPgThreads * cluster))
      cluster *= 2;
    st = launch(fork ? sv::pages_fork_kernel : sv::pages_compact_kernel, cluster, 0, prm, stream,
                true, cluster, sv::kPgThreads);
  }
  if (st != SPEC_OK) return st;
  int sms = 0;
  st = sm_count(&sms);
  if (st != SPEC_OK) return st;
  // no more CTAs than the most copies have units
  const long long unit = 16ll * sv::kPgCopyThreads * sv::kPgCopyVecs;
  const double units = (double)(fork ? prm.B2 : prm.n_pages) * prm.planes *
                       (double)((prm.page_bytes + unit - 1) / unit);
  const int grid = (int)std::max(1.0, std::min((double)sms * 8, units));
  return launch(sv::pages_copy_kernel, grid, 0, prm, stream, true, 1, sv::kPgCopyThreads);
}

struct BeamLayout {
  int nchunks = 0;
  size_t off_runs = 0, bytes = 0;
};
bool beam_layout(int B, int K, int V, int M, int dtype, BeamLayout* L) {
  if (B < 0 || K < 1 || K > sv::kBeamMaxK || M < 1 || M > sv::kBeamMaxM || V < 1 ||
      V > SPEC_MAX_V || (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16))
    return false;
  const int C = (V + chunk_elems(dtype) - 1) / chunk_elems(dtype);
  if ((long long)B * K * C > INT32_MAX / 64) return false;
  const size_t items = (size_t)B * K * C;
  L->nchunks = C;
  L->off_runs = align_up(kDataOffset + items * sv::kWarps * sizeof(float2));
  L->bytes = align_up(L->off_runs + items * sv::kBeamRuns * sizeof(float));
  return true;
}

template <typename E>
spec_status_t run_beam(const sv::BeamParams& prm, bool vec, void* stream) {
  spec_status_t st;
  if (vec) {
    int grid = 0;
    st = persistent_grid<sv::beam_rows_stream_kernel<E>>(prm.items, &grid);
    if (st == SPEC_OK)
      st = launch(sv::beam_rows_stream_kernel<E>, grid, kStreamSmem, prm, stream, true);
  } else {
    st = launch(sv::beam_rows_kernel<E>, prm.items, 0, prm, stream, true);
  }
  if (st != SPEC_OK) return st;
  const int nruns = prm.nchunks * sv::kBeamRuns;
  constexpr size_t kMost = (size_t)sv::kBeamMaxK * sv::kBeamMaxM * 12 +
                           (size_t)sv::kBeamWarps * sv::kBeamStage * sizeof(float);
  const size_t smem = (size_t)prm.K * prm.M * 12 +
                      (nruns <= sv::kBeamStage
                           ? (size_t)std::min(prm.K, sv::kBeamWarps) * nruns * sizeof(float) : 0);
  if (vec) {
    st = ensure_smem<sv::beam_select_kernel<E, true>>(kMost);
    if (st != SPEC_OK) return st;
    return launch(sv::beam_select_kernel<E, true>, prm.B, smem, prm, stream, true, 1, sv::kBeamThreads);
  }
  st = ensure_smem<sv::beam_select_kernel<E, false>>(kMost);
  if (st != SPEC_OK) return st;
  return launch(sv::beam_select_kernel<E, false>, prm.B, smem, prm, stream, true, 1, sv::kBeamThreads);
}

}  // namespace

extern "C" {

size_t spec_verify_workspace_bytes(int mode, int B, int k_or_N, int V, int dtype) {
  Layout L;
  if (!make_layout(mode, B, k_or_N, V, dtype, &L)) return 0;
  return L.bytes;
}

spec_status_t spec_verify_sample(const void* target_logits, const void* draft_logits, int dtype,
                                 const int32_t* draft_tokens, const float* u_accept,
                                 const float* u_sample, float temperature, int B, int k, int V,
                                 int32_t* accepted_len, int32_t* out_tokens, float* p_out,
                                 float* q_out, float* resid_mass, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  if (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16) return SPEC_ERR_INVALID_ARG;
  if (B < 0 || k < 0 || k > SPEC_MAX_K || V < 1 || V > SPEC_MAX_V) return SPEC_ERR_INVALID_ARG;
  if (!(temperature > 0.0f) || !std::isfinite(temperature)) return SPEC_ERR_INVALID_ARG;
  Layout L;
  if (!make_layout(SPEC_MODE_SAMPLE, B, k, V, dtype, &L)) return SPEC_ERR_INVALID_ARG;
  if (B == 0) return SPEC_OK;
  if (!target_logits || !u_sample || !accepted_len || !out_tokens || !resid_mass)
    return SPEC_ERR_INVALID_ARG;
  if (k > 0 && (!draft_logits || !draft_tokens || !u_accept || !p_out || !q_out))
    return SPEC_ERR_INVALID_ARG;
  const int eb = elem_bytes(dtype);
  if (!aligned(target_logits, eb) || (k > 0 && !aligned(draft_logits, eb)))
    return SPEC_ERR_ALIGNMENT;
  if (!aligned(accepted_len, 4) || !aligned(out_tokens, 4) || !aligned(u_sample, 4) ||
      !aligned(resid_mass, 4) ||
      (k > 0 && (!aligned(draft_tokens, 4) || !aligned(u_accept, 4) || !aligned(p_out, 4) ||
                 !aligned(q_out, 4))))
    return SPEC_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < L.bytes) return SPEC_ERR_WORKSPACE;
  if (!aligned(workspace, kAlign)) return SPEC_ERR_ALIGNMENT;

  char* ws = static_cast<char*>(workspace);
  sv::SampleParams prm;
  prm.target = target_logits;
  prm.draft = draft_logits;
  prm.tokens = draft_tokens;
  prm.u_accept = u_accept;
  prm.u_sample = u_sample;
  prm.scale = (float)(1.4426950408889634 / (double)temperature);
  prm.B = B;
  prm.k = k;
  prm.V = V;
  prm.nchunks = L.nchunks;
  prm.accepted_len = accepted_len;
  prm.out_tokens = out_tokens;
  prm.p_out = p_out;
  prm.q_out = q_out;
  prm.resid_mass = resid_mass;
  prm.flags = reinterpret_cast<unsigned*>(ws);
  prm.part = reinterpret_cast<sv::SoftmaxPartial*>(ws + L.off_part);
  prm.desc = reinterpret_cast<sv::DrawDesc*>(ws + L.off_desc);
  prm.csum = reinterpret_cast<sv::FSum*>(ws + L.off_csum);
  prm.csum_p = reinterpret_cast<sv::FSum*>(ws + L.off_csum_p);
  prm.gsum = reinterpret_cast<float*>(ws + L.off_gsum);
  prm.gsum_p = reinterpret_cast<float*>(ws + L.off_gsum_p);
  prm.zx = reinterpret_cast<float*>(ws + L.off_zx);
  prm.nrec = L.nchunks;
  prm.drawn = nullptr;

  const bool vec = vec_ok(target_logits, V, dtype) && (k == 0 || vec_ok(draft_logits, V, dtype));
  if (dtype == SPEC_DTYPE_BF16) return run_sample<sv::BF16>(prm, L.rows, vec, stream);
  return run_sample<sv::F32>(prm, L.rows, vec, stream);
}

static spec_status_t argmax_common(sv::ArgmaxParams& prm, const Layout& L, void* workspace,
                                   int dtype, void* stream) {
  char* ws = static_cast<char*>(workspace);
  prm.flags = reinterpret_cast<unsigned*>(ws);
  prm.part = reinterpret_cast<sv::ArgPartial*>(ws + L.off_part);
  prm.rowarg = reinterpret_cast<int32_t*>(ws + L.off_arg);
  prm.nchunks = L.nchunks;
  const bool vec = vec_ok(prm.target, prm.V, dtype);
  if (dtype == SPEC_DTYPE_BF16) return run_argmax<sv::BF16>(prm, L.rows, vec, stream);
  return run_argmax<sv::F32>(prm, L.rows, vec, stream);
}

spec_status_t spec_verify_greedy(const void* target_logits, int dtype,
                                 const int32_t* draft_tokens, int B, int k, int V,
                                 int32_t* accepted_len, int32_t* out_tokens, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  if (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16) return SPEC_ERR_INVALID_ARG;
  if (B < 0 || k < 0 || k > SPEC_MAX_K || V < 1 || V > SPEC_MAX_V) return SPEC_ERR_INVALID_ARG;
  Layout L;
  if (!make_layout(SPEC_MODE_GREEDY, B, k, V, dtype, &L)) return SPEC_ERR_INVALID_ARG;
  if (B == 0) return SPEC_OK;
  if (!target_logits || !accepted_len || !out_tokens || (k > 0 && !draft_tokens))
    return SPEC_ERR_INVALID_ARG;
  if (!aligned(target_logits, elem_bytes(dtype)) || !aligned(accepted_len, 4) ||
      !aligned(out_tokens, 4) || (k > 0 && !aligned(draft_tokens, 4)))
    return SPEC_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < L.bytes) return SPEC_ERR_WORKSPACE;
  if (!aligned(workspace, kAlign)) return SPEC_ERR_ALIGNMENT;
  sv::ArgmaxParams prm;
  std::memset(&prm, 0, sizeof prm);
  prm.target = target_logits;
  prm.tokens = draft_tokens;
  prm.parents = nullptr;
  prm.B = B;
  prm.rows_per_seq = k + 1;
  prm.V = V;
  prm.tree = 0;
  prm.max_depth = 0;
  prm.accepted_len = accepted_len;
  prm.out_tokens = out_tokens;
  prm.path_nodes = nullptr;
  return argmax_common(prm, L, workspace, dtype, stream);
}

spec_status_t spec_verify_tree_greedy(const void* target_logits, int dtype,
                                      const int32_t* node_tokens, const int32_t* parents, int B,
                                      int N, int V, int max_depth, int32_t* accepted_len,
                                      int32_t* path_nodes, int32_t* out_tokens, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  if (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16) return SPEC_ERR_INVALID_ARG;
  if (B < 0 || N < 1 || N > SPEC_MAX_TREE_NODES || V < 1 || V > SPEC_MAX_V)
    return SPEC_ERR_INVALID_ARG;
  if (max_depth < 0 || max_depth > SPEC_MAX_TREE_DEPTH) return SPEC_ERR_INVALID_ARG;
  Layout L;
  if (!make_layout(SPEC_MODE_TREE_GREEDY, B, N, V, dtype, &L)) return SPEC_ERR_INVALID_ARG;
  if (B == 0) return SPEC_OK;
  if (!target_logits || !node_tokens || !parents || !accepted_len || !path_nodes || !out_tokens)
    return SPEC_ERR_INVALID_ARG;
  if (!aligned(target_logits, elem_bytes(dtype)) || !aligned(node_tokens, 4) ||
      !aligned(parents, 4) || !aligned(accepted_len, 4) || !aligned(path_nodes, 4) ||
      !aligned(out_tokens, 4))
    return SPEC_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < L.bytes) return SPEC_ERR_WORKSPACE;
  if (!aligned(workspace, kAlign)) return SPEC_ERR_ALIGNMENT;
  sv::ArgmaxParams prm;
  std::memset(&prm, 0, sizeof prm);
  prm.target = target_logits;
  prm.tokens = node_tokens;
  prm.parents = parents;
  prm.B = B;
  prm.rows_per_seq = N;
  prm.V = V;
  prm.tree = 1;
  prm.max_depth = max_depth;
  prm.accepted_len = accepted_len;
  prm.out_tokens = out_tokens;
  prm.path_nodes = path_nodes;
  return argmax_common(prm, L, workspace, dtype, stream);
}

spec_status_t spec_tree_attention_mask(const int32_t* parents, int B, int N, uint32_t* mask,
                                       int32_t* depth, void* workspace, size_t workspace_bytes,
                                       void* stream) {
  if (B < 0 || N < 1 || N > SPEC_MAX_TREE_NODES) return SPEC_ERR_INVALID_ARG;
  if (B == 0) return SPEC_OK;
  if (!parents || !mask) return SPEC_ERR_INVALID_ARG;
  if (!aligned(parents, 4) || !aligned(mask, 4) || (depth && !aligned(depth, 4)))
    return SPEC_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < kHeaderBytes) return SPEC_ERR_WORKSPACE;
  if (!aligned(workspace, kAlign)) return SPEC_ERR_ALIGNMENT;
  const int W = (N + 31) / 32;
  const long long threads = (long long)B * N * W;
  const long long blocks = (threads + sv::kMaskThreads - 1) / sv::kMaskThreads;
  if (blocks > 0x7FFFFFFFLL) return SPEC_ERR_INVALID_ARG;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  pdl_config(&cfg, attr, dim3((unsigned)blocks), dim3(sv::kMaskThreads), 0, stream);
  if (cudaLaunchKernelEx(&cfg, sv::tree_mask_kernel, parents, B, N, W, mask, depth,
                         reinterpret_cast<unsigned*>(workspace)) != cudaSuccess)
    return SPEC_ERR_CUDA;
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return SPEC_OK;
}

spec_status_t spec_kv_commit_path(void* cache, int B, int planes, long long plane_stride,
                                  long long seq_stride, int entry_bytes, int L, int N,
                                  const int32_t* base_len, const int32_t* accepted_len,
                                  const int32_t* path_nodes, int max_depth, int32_t* new_len,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  if (B < 0 || planes < 1 || planes > 65535 || entry_bytes < 16 || L < 1 || N < 1 ||
      N > SPEC_MAX_TREE_NODES || max_depth < 0 || max_depth > SPEC_MAX_TREE_DEPTH ||
      plane_stride < 0 || seq_stride < 0)
    return SPEC_ERR_INVALID_ARG;
  if (B == 0) return SPEC_OK;
  if (!cache || !base_len || !accepted_len || !path_nodes || !new_len)
    return SPEC_ERR_INVALID_ARG;
  if (!aligned(cache, 16) || entry_bytes % 16 || plane_stride % 16 || seq_stride % 16 ||
      !aligned(base_len, 4) || !aligned(accepted_len, 4) || !aligned(path_nodes, 4) ||
      !aligned(new_len, 4))
    return SPEC_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < kHeaderBytes) return SPEC_ERR_WORKSPACE;
  if (!aligned(workspace, kAlign)) return SPEC_ERR_ALIGNMENT;
  sv::KvCommitParams prm;
  prm.cache = static_cast<uint8_t*>(cache);
  prm.plane_stride = plane_stride;
  prm.seq_stride = seq_stride;
  prm.entry_bytes = entry_bytes;
  prm.L = L;
  prm.N = N;
  prm.max_depth = max_depth;
  prm.planes = planes;
  prm.base_len = base_len;
  prm.accepted_len = accepted_len;
  prm.path_nodes = path_nodes;
  prm.new_len = new_len;
  prm.flags = reinterpret_cast<unsigned*>(workspace);
  // stage every moved entry of a pass in at most 40 KB of dynamic shared
  // memory (under the 48 KB default with the kernel's static arrays)
  constexpr int kStageBytes = 40 * 1024;
  const int moves = std::max(1, std::min(max_depth, sv::kKvMaxMoves));
  prm.slice_bytes = std::min(entry_bytes, kStageBytes / moves / 16 * 16);
  const size_t smem = (size_t)prm.slice_bytes * moves;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  pdl_config(&cfg, attr, dim3((unsigned)B, (unsigned)planes), dim3(sv::kKvThreads), smem,
             stream);
  if (cudaLaunchKernelEx(&cfg, sv::kv_commit_kernel, prm) != cudaSuccess) return SPEC_ERR_CUDA;
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return SPEC_OK;
}

spec_status_t spec_lm_head_verify_greedy(const void* hidden, const void* w_lm,
                                         const int32_t* draft_tokens, int B, int k, int d, int V,
                                         int32_t* accepted_len, int32_t* out_tokens,
                                         void* workspace, size_t workspace_bytes, void* stream) {
  if (B < 0 || k < 0 || k > SPEC_MAX_K || d < 8 || d > (1 << 20) || d % 8 || V < 1 ||
      V > SPEC_MAX_V)
    return SPEC_ERR_INVALID_ARG;
  Layout L;
  if (!make_layout(SPEC_MODE_LM_HEAD_GREEDY, B, k, V, SPEC_DTYPE_BF16, &L))
    return SPEC_ERR_INVALID_ARG;
  if (B == 0) return SPEC_OK;
  if (!hidden || !w_lm || !accepted_len || !out_tokens || (k > 0 && !draft_tokens))
    return SPEC_ERR_INVALID_ARG;
  if (!aligned(hidden, 16) || !aligned(w_lm, 16) || !aligned(accepted_len, 4) ||
      !aligned(out_tokens, 4) || (k > 0 && !aligned(draft_tokens, 4)))
    return SPEC_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < L.bytes) return SPEC_ERR_WORKSPACE;
  if (!aligned(workspace, kAlign)) return SPEC_ERR_ALIGNMENT;
  const int rows = L.rows;
  const int ntiles = (V + sv::kLmPairBV - 1) / sv::kLmPairBV;
  int gy = 0, grp = 0, gx = 0;
  if (!lm_row_groups(rows, &gy, &grp)) return SPEC_ERR_INVALID_ARG;
  spec_status_t st = lm_grid_x<sv::kLmArgmax>(ntiles, &gx);
  if (st != SPEC_OK) return st;
  CUtensorMap map_h, map_w;
  st = encode_bf16_kmajor(&map_h, hidden, d, rows, sv::lm_half_rows(grp));
  if (st != SPEC_OK) return st;
  st = encode_bf16_kmajor(&map_w, w_lm, d, V, sv::kLmBV);
  if (st != SPEC_OK) return st;
  char* ws = static_cast<char*>(workspace);
  sv::LmHeadParams lp;
  std::memset(&lp, 0, sizeof lp);
  lp.rows = rows;
  lp.d = d;
  lp.V = V;
  lp.ntiles = ntiles;
  lp.grp_rows = grp;
  lp.stage_bytes = sv::lm_stage_bytes(grp);
  lp.nstages = sv::lm_stages(lp.stage_bytes);
  lp.part = reinterpret_cast<sv::ArgPartial*>(ws + L.off_part);
  lp.flags = reinterpret_cast<unsigned*>(ws);
  lp.ngroups0 = gy;
  lp.grp_rows1 = sv::kLmHBox;
  st = launch_lmhead<sv::kLmArgmax>(map_h, map_h, map_w, lp, gx, gy, stream);
  if (st != SPEC_OK) return st;
  // merge the per-CTA records and resolve the chains (the greedy resolve)
  sv::ArgmaxParams prm;
  std::memset(&prm, 0, sizeof prm);
  prm.tokens = draft_tokens;
  prm.B = B;
  prm.rows_per_seq = k + 1;
  prm.V = V;
  prm.nchunks = gx;
  prm.tree = 0;
  prm.accepted_len = accepted_len;
  prm.out_tokens = out_tokens;
  prm.flags = lp.flags;
  prm.part = lp.part;
  prm.rowarg = reinterpret_cast<int32_t*>(ws + L.off_arg);
  prm.wait_ns = sv::kWaitLimitNs;
  return launch(sv::argmax_resolve_kernel, B, 0, prm, stream, true);
}

spec_status_t spec_lm_head_verify_sample(
    const void* hidden_target, const void* hidden_draft, const void* w_lm,
    const int32_t* draft_tokens, const float* u_accept, const float* u_sample, float temperature,
    int B, int k, int d, int V, int32_t* accepted_len, int32_t* out_tokens, float* p_out,
    float* q_out, float* resid_mass, void* workspace, size_t workspace_bytes, void* stream) {
  if (B < 0 || k < 0 || k > SPEC_MAX_K || d < 8 || d > SPEC_LM_MAX_D || d % 8 || V < 1 ||
      V > SPEC_MAX_V)
    return SPEC_ERR_INVALID_ARG;
  if (!(temperature > 0.0f) || !std::isfinite(temperature)) return SPEC_ERR_INVALID_ARG;
  Layout L;
  if (!make_layout(SPEC_MODE_LM_HEAD_SAMPLE, B, k, V, SPEC_DTYPE_BF16, &L))
    return SPEC_ERR_INVALID_ARG;
  if (B == 0) return SPEC_OK;
  if (!hidden_target || !w_lm || !u_sample || !accepted_len || !out_tokens || !resid_mass)
    return SPEC_ERR_INVALID_ARG;
  if (k > 0 && (!hidden_draft || !draft_tokens || !u_accept || !p_out || !q_out))
    return SPEC_ERR_INVALID_ARG;
  if (!aligned(hidden_target, 16) || !aligned(w_lm, 16) || (k > 0 && !aligned(hidden_draft, 16)))
    return SPEC_ERR_ALIGNMENT;
  if (!aligned(accepted_len, 4) || !aligned(out_tokens, 4) || !aligned(u_sample, 4) ||
      !aligned(resid_mass, 4) ||
      (k > 0 && (!aligned(draft_tokens, 4) || !aligned(u_accept, 4) || !aligned(p_out, 4) ||
                 !aligned(q_out, 4))))
    return SPEC_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < L.bytes) return SPEC_ERR_WORKSPACE;
  if (!aligned(workspace, kAlign)) return SPEC_ERR_ALIGNMENT;
  const int rows_t = B * (k + 1), rows_d = B * k, rows_2 = 2 * B;
  const int ntiles = (V + sv::kLmPairBV - 1) / sv::kLmPairBV;
  int gy0 = 0, grp0 = 0, gy1 = 0, grp1 = 0, gy2 = 0, grp2 = 0, gx = 0;
  if (!lm_row_groups(rows_t, &gy0, &grp0) || !lm_row_groups(rows_d, &gy1, &grp1) ||
      !lm_row_groups(rows_2, &gy2, &grp2) || gy0 + gy1 > 65535)
    return SPEC_ERR_INVALID_ARG;
  spec_status_t st = lm_grid_x<sv::kLmStats>(ntiles, &gx);
  if (st != SPEC_OK) return st;
  char* ws = static_cast<char*>(workspace);
  uint16_t* hbuf = reinterpret_cast<uint16_t*>(ws + L.off_arg);
  float* lbuf = reinterpret_cast<float*>(ws + L.off_log);
  CUtensorMap map_ht, map_hd, map_w, map_hb;
  st = encode_bf16_kmajor(&map_ht, hidden_target, d, rows_t, sv::lm_half_rows(grp0));
  if (st != SPEC_OK) return st;
  st = k > 0 ? encode_bf16_kmajor(&map_hd, hidden_draft, d, rows_d, sv::lm_half_rows(grp1))
             : SPEC_OK;
  if (k == 0) map_hd = map_ht;  // no draft rows: never read
  if (st != SPEC_OK) return st;
  st = encode_bf16_kmajor(&map_w, w_lm, d, V, sv::kLmBV);
  if (st != SPEC_OK) return st;
  st = encode_bf16_kmajor(&map_hb, hbuf, d, rows_2, sv::lm_half_rows(grp2));
  if (st != SPEC_OK) return st;

  // 1. softmax statistics of every target and draft row, and the draft
  // tokens' logits, from the tensor cores' accumulators
  sv::LmHeadParams lp;
  std::memset(&lp, 0, sizeof lp);
  lp.rows = rows_t;
  lp.d = d;
  lp.V = V;
  lp.ntiles = ntiles;
  lp.grp_rows = grp0;
  lp.stage_bytes = sv::lm_stage_bytes(std::max(grp0, grp1));
  lp.nstages = sv::lm_stages(lp.stage_bytes);
  lp.flags = reinterpret_cast<unsigned*>(ws);
  lp.ngroups0 = gy0;
  lp.rows1 = rows_d;
  lp.grp_rows1 = grp1;
  lp.k = k;
  lp.scale = (float)(1.4426950408889634 / (double)temperature);
  lp.tokens = draft_tokens;
  lp.spart = reinterpret_cast<sv::SoftmaxPartial*>(ws + L.off_part);
  lp.zx = reinterpret_cast<float*>(ws + L.off_zx);
  st = launch_lmhead<sv::kLmStats>(map_ht, map_hd, map_w, lp, gx, gy0 + gy1, stream);
  if (st != SPEC_OK) return st;

  // 2. accept test; hidden states of the rows each sequence draws from
  sv::SampleParams prm;
  std::memset(&prm, 0, sizeof prm);
  prm.target = lbuf;
  prm.draft = lbuf;
  prm.tokens = draft_tokens;
  prm.u_accept = u_accept;
  prm.u_sample = u_sample;
  prm.scale = lp.scale;
  prm.B = B;
  prm.k = k;
  prm.V = V;
  prm.nchunks = L.nchunks;
  prm.nrec = gx;
  prm.accepted_len = accepted_len;
  prm.out_tokens = out_tokens;
  prm.p_out = p_out;
  prm.q_out = q_out;
  prm.resid_mass = resid_mass;
  prm.flags = lp.flags;
  prm.part = lp.spart;
  prm.desc = reinterpret_cast<sv::DrawDesc*>(ws + L.off_desc);
  prm.csum = reinterpret_cast<sv::FSum*>(ws + L.off_csum);
  prm.csum_p = reinterpret_cast<sv::FSum*>(ws + L.off_csum_p);
  prm.gsum = reinterpret_cast<float*>(ws + L.off_gsum);
  prm.gsum_p = reinterpret_cast<float*>(ws + L.off_gsum_p);
  prm.zx = lp.zx;
  prm.wait_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  prm.drawn = lbuf;
  {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    pdl_config(&cfg, attr, dim3((unsigned)B, 1, 1), dim3(sv::kThreads, 1, 1), 0, stream);
    if (cudaLaunchKernelEx(&cfg, sv::lm_sample_gather_kernel, prm,
                           static_cast<const uint16_t*>(hidden_target),
                           static_cast<const uint16_t*>(hidden_draft), hbuf, d) != cudaSuccess)
      return SPEC_ERR_CUDA;
    g_launches.fetch_add(1, std::memory_order_relaxed);
  }

  // 3. those rows' logits, fp32
  sv::LmHeadParams lq = lp;
  lq.rows = rows_2;
  lq.grp_rows = grp2;
  lq.stage_bytes = sv::lm_stage_bytes(grp2);
  lq.nstages = sv::lm_stages(lq.stage_bytes);
  lq.ngroups0 = gy2;
  lq.rows1 = 0;
  lq.grp_rows1 = sv::kLmHBox;
  lq.logits = lbuf;
  st = launch_lmhead<sv::kLmLogits>(map_hb, map_hb, map_w, lq, gx, gy2, stream);
  if (st != SPEC_OK) return st;

  // 4. the residual or bonus draw (the accept test again, then the draw over
  // the recomputed rows), as spec_verify_sample's
  if (vec_ok(lbuf, V, SPEC_DTYPE_F32)) return run_finish<sv::F32, true>(prm, stream);
  return run_finish<sv::F32, false>(prm, stream);
}

spec_status_t spec_verify_tree_sample(const void* target_logits, int dtype,
                                      const int32_t* node_tokens, const int32_t* parents,
                                      const float* u_sample, float temperature, int B, int N,
                                      int V, int max_depth, int32_t* accepted_len,
                                      int32_t* path_nodes, int32_t* out_tokens, float* out_probs,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  if (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16) return SPEC_ERR_INVALID_ARG;
  if (B < 0 || N < 1 || N > SPEC_MAX_TREE_NODES || V < 1 || V > SPEC_MAX_V || max_depth < 0 ||
      max_depth > SPEC_MAX_TREE_DEPTH || !(temperature > 0.0f) || !std::isfinite(temperature))
    return SPEC_ERR_INVALID_ARG;
  if ((long long)B * sv::kTsMaxCluster > INT32_MAX) return SPEC_ERR_INVALID_ARG;
  if (B == 0) return SPEC_OK;
  if (!target_logits || !node_tokens || !parents || !u_sample || !accepted_len || !path_nodes ||
      !out_tokens || !out_probs)
    return SPEC_ERR_INVALID_ARG;
  if (!aligned(target_logits, elem_bytes(dtype)) || !aligned(node_tokens, 4) ||
      !aligned(parents, 4) || !aligned(u_sample, 4) || !aligned(accepted_len, 4) ||
      !aligned(path_nodes, 4) || !aligned(out_tokens, 4) || !aligned(out_probs, 4))
    return SPEC_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < kHeaderBytes) return SPEC_ERR_WORKSPACE;
  if (!aligned(workspace, kAlign)) return SPEC_ERR_ALIGNMENT;
  const double scale = 1.4426950408889634 / (double)temperature;
  sv::TreeSampleParams prm;
  std::memset(&prm, 0, sizeof prm);
  prm.logits = target_logits;
  prm.tokens = node_tokens;
  prm.parents = parents;
  prm.u = u_sample;
  prm.c_hi = (float)scale;
  prm.c_lo = (float)(scale - (double)prm.c_hi);
  prm.N = N;
  prm.V = V;
  prm.max_depth = max_depth;
  // the largest weight is below 2^(kTsFrac + 1/2): the sum of 2^bits of them stays below 2^63
  for (int bits = 12; bits < 31 && (1 << bits) < V; ++bits) prm.extra = bits - 11;
  prm.accepted_len = accepted_len;
  prm.path = path_nodes;
  prm.out = out_tokens;
  prm.probs = out_probs;
  prm.flags = reinterpret_cast<unsigned*>(workspace);
  constexpr int kCtaStep = sv::kTsWarps * sv::kTsStep;  // elements of a CTA's step
  // CTAs per sequence.  608 CTAs are resident (four on an SM); clusters beyond
  // that start as others end, which pays where rows are long.  Measured with 4,
  // 8 and 16 CTAs: V = 32000 bf16, B = 40 24.2, 22.1, 22.0 us; 56 26.5, 24.1,
  // 27.7; 112 26.5, 33.6, 50.2; V = 128256 bf16, B = 24 35.6, 23.9, 21.1; 40
  // 53.1, 34.7, 29.6; 80 64.8, 45.7, 52.3; 112 70.2, 57.3, 70.9; 250 101, 102,
  // 138; V = 151936 float32, B = 40 80.7, 55.4, 40.9; 112 87.2, 71.8, 84.3; and 2
  // CTAs at B = 250 44.6, 127 and 170 us against 39.8, 101 and 131 with 4.
  const long long row_bytes = (long long)V * elem_bytes(dtype);
  int most = 1;
  while (most < sv::kTsMaxCluster) {
    const long long beyond = most < 4 ? 608 : row_bytes * (most == 4 ? 12 : 4) / 5120;
    if (2ll * most * B > 608 + std::min(beyond, 608ll)) break;
    most *= 2;
  }
  int cluster = 1;
  while (cluster < most && cluster * kCtaStep < V) cluster *= 2;
  while ((long long)cluster * kCtaStep * kTsMaxSteps < V) cluster *= 2;
  prm.nsteps = (V + cluster * kCtaStep - 1) / (cluster * kCtaStep);
  const size_t smem = (size_t)sv::kTsWarps * prm.nsteps * sizeof(unsigned long long);
  // 16-byte loads: whole groups of 8 elements at 16-byte boundaries (element by
  // element 15.5 us become 18.1 at one stream of V = 128256 bf16, 62.0 become
  // 78.4 at 64 of V = 151936 float32)
  const bool vec = aligned(target_logits, 16) && V % 8 == 0;
  if (dtype == SPEC_DTYPE_BF16)
    return vec ? launch_tree_sample<sv::tree_sample_kernel<sv::BF16, true>>(prm, B, cluster, smem, stream)
               : launch_tree_sample<sv::tree_sample_kernel<sv::BF16, false>>(prm, B, cluster, smem, stream);
  return vec ? launch_tree_sample<sv::tree_sample_kernel<sv::F32, true>>(prm, B, cluster, smem, stream)
             : launch_tree_sample<sv::tree_sample_kernel<sv::F32, false>>(prm, B, cluster, smem, stream);
}

namespace {

// spec_tree_qkv_rope and, with to_nodes, spec_tree_qkv_rope_nodes
spec_status_t tree_qkv_rope(const void* qkv, const void* q_norm, const void* k_norm, float eps,
                            const float* inv_freq, int rot_dim, int interleaved,
                            long long pos_offset, const int32_t* base_len, const int32_t* depth,
                            int B, int N, int Hq, int Hkv, int D, int L, long long seq_stride,
                            void* q_out, void* k_cache, void* v_cache, bool to_nodes,
                            void* workspace, size_t workspace_bytes, void* stream) {
  if (B < 0 || N < 1 || N > SPEC_MAX_TREE_NODES || Hq < 1 || Hkv < 1 || Hq > 65536 ||
      Hkv > 65536 || (D != 64 && D != 128) || L < 1 || rot_dim < 0 || rot_dim > D || rot_dim % 2 ||
      pos_offset < 0 || pos_offset > INT32_MAX || !(eps >= 0.0f) || !std::isfinite(eps) ||
      (long long)B * N > INT32_MAX)
    return SPEC_ERR_INVALID_ARG;
  if (seq_stride < (long long)L * Hkv * D * 2) return SPEC_ERR_INVALID_ARG;
  if (B == 0) return SPEC_OK;
  if (!qkv || !base_len || !q_out || !k_cache || !v_cache || (rot_dim > 0 && !inv_freq))
    return SPEC_ERR_INVALID_ARG;
  if (!aligned(qkv, 16) || !aligned(q_out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(q_norm, 16) || !aligned(k_norm, 16) || seq_stride % 16 || !aligned(base_len, 4) ||
      !aligned(depth, 4) || !aligned(inv_freq, 4))
    return SPEC_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < kHeaderBytes) return SPEC_ERR_WORKSPACE;
  if (!aligned(workspace, kAlign)) return SPEC_ERR_ALIGNMENT;
  sv::RopeParams prm;
  std::memset(&prm, 0, sizeof prm);
  prm.qkv = static_cast<const uint16_t*>(qkv);
  prm.q_norm = static_cast<const uint16_t*>(q_norm);
  prm.k_norm = static_cast<const uint16_t*>(k_norm);
  prm.inv_freq = inv_freq;
  prm.base_len = base_len;
  prm.depth = depth;
  prm.q_out = static_cast<uint16_t*>(q_out);
  prm.k_cache = static_cast<uint16_t*>(k_cache);
  prm.v_cache = static_cast<uint16_t*>(v_cache);
  prm.flags = reinterpret_cast<unsigned*>(workspace);
  prm.seq_stride = seq_stride / 2;
  prm.pos_offset = pos_offset;
  prm.eps = eps;
  prm.N = N;
  prm.Hq = Hq;
  prm.Hkv = Hkv;
  prm.L = L;
  prm.rot = rot_dim;
  prm.interleaved = interleaved != 0;
  prm.to_nodes = to_nodes;
  // an element's partner in the thread's registers where the halves are whole
  // vectors (128 trees of 60, D = 128: 34.8 us; 100.8 with the partner read from
  // memory, as other rotations have to)
  const int mode = interleaved ? sv::kRopePairs : rot_dim % 16 == 0 ? sv::kRopeHalves : sv::kRopeOdd;
  return D == 128 ? run_rope<128>(prm, mode, B * N, stream) : run_rope<64>(prm, mode, B * N, stream);
}

}  // namespace

spec_status_t spec_tree_qkv_rope(const void* qkv, const void* q_norm, const void* k_norm, float eps,
                                 const float* inv_freq, int rot_dim, int interleaved,
                                 long long pos_offset, const int32_t* base_len,
                                 const int32_t* depth, int B, int N, int Hq, int Hkv, int D, int L,
                                 long long seq_stride, void* q_out, void* k_cache, void* v_cache,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  return tree_qkv_rope(qkv, q_norm, k_norm, eps, inv_freq, rot_dim, interleaved, pos_offset,
                       base_len, depth, B, N, Hq, Hkv, D, L, seq_stride, q_out, k_cache, v_cache,
                       false, workspace, workspace_bytes, stream);
}

spec_status_t spec_tree_qkv_rope_nodes(const void* qkv, const void* q_norm, const void* k_norm,
                                       float eps, const float* inv_freq, int rot_dim,
                                       int interleaved, long long pos_offset,
                                       const int32_t* base_len, const int32_t* depth, int B, int N,
                                       int Hq, int Hkv, int D, void* q_out, void* k_out,
                                       void* v_out, void* workspace, size_t workspace_bytes,
                                       void* stream) {
  return tree_qkv_rope(qkv, q_norm, k_norm, eps, inv_freq, rot_dim, interleaved, pos_offset,
                       base_len, depth, B, N, Hq, Hkv, D, N, (long long)N * Hkv * D * 2, q_out,
                       k_out, v_out, true, workspace, workspace_bytes, stream);
}

size_t spec_tree_attention_workspace_bytes(int B, int N, int Hq, int Hkv, int D, int P) {
  if (!attn_shape_ok(B, N, Hq, Hkv, D, P)) return 0;
  return attn_plan(B, N, Hq, Hkv, D, P).bytes;
}

spec_status_t spec_tree_attention(const void* q, const void* k_cache, const void* v_cache,
                                  long long seq_stride, int L, const void* prefix_k,
                                  const void* prefix_v, int P, const uint32_t* mask,
                                  const int32_t* base_len, int B, int N, int Hq, int Hkv, int D,
                                  float scale, void* out, float* lse, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  if (!attn_shape_ok(B, N, Hq, Hkv, D, P) || L < 1 || L > INT32_MAX - 256 || !(scale > 0.0f) ||
      !(scale < 1.7014118e38f))  // 2^127: scale * log2(e) stays finite
    return SPEC_ERR_INVALID_ARG;
  if (seq_stride < (long long)L * Hkv * D * 2) return SPEC_ERR_INVALID_ARG;
  if (B == 0) return SPEC_OK;
  if (!q || !k_cache || !v_cache || !base_len || !out || (P > 0 && (!prefix_k || !prefix_v)))
    return SPEC_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      seq_stride % 16 || (P > 0 && (!aligned(prefix_k, 16) || !aligned(prefix_v, 16))) ||
      !aligned(mask, 4) || !aligned(base_len, 4) || !aligned(lse, 4))
    return SPEC_ERR_ALIGNMENT;
  if (!workspace) return SPEC_ERR_WORKSPACE;
  if (!aligned(workspace, kAlign)) return SPEC_ERR_ALIGNMENT;
  const AttnPlan plan = attn_plan(B, N, Hq, Hkv, D, P);
  if (workspace_bytes < plan.bytes) return SPEC_ERR_WORKSPACE;
  int sms = 0;
  spec_status_t st = sm_count(&sms);
  if (st != SPEC_OK) return st;
  char* ws = static_cast<char*>(workspace);
  sv::AttnParams prm;
  std::memset(&prm, 0, sizeof prm);
  prm.q = static_cast<const uint16_t*>(q);
  prm.k = static_cast<const uint16_t*>(k_cache);
  prm.v = static_cast<const uint16_t*>(v_cache);
  prm.mask = mask;
  prm.base_len = base_len;
  prm.out = static_cast<uint16_t*>(out);
  prm.lse = lse;
  prm.flags = reinterpret_cast<unsigned*>(workspace);
  prm.seq_stride = seq_stride / 2;
  prm.scale_log2 = (float)(1.4426950408889634 * (double)scale);
  prm.B = B;
  prm.N = N;
  prm.Hq = Hq;
  prm.Hkv = Hkv;
  prm.G = Hq / Hkv;
  prm.W = (N + 31) / 32;
  prm.L = L;
  prm.P = P;
  prm.tok = plan.tok;
  prm.pair_s = plan.pair_s;
  prm.pair_o = plan.pair_o;
  prm.mg_s = plan.mg_s;
  prm.mg_o = plan.mg_o;
  prm.tiles_s = P / sv::kAtKeys + (P % sv::kAtKeys != 0);
  prm.rows_s = plan.rows_s;
  prm.rows_o = plan.rows_o;
  prm.by_cta = plan.by_cta;
  prm.own0 = plan.own0;
  prm.nctas = std::min(sms, sv::kAtMaxCtas);
  prm.q_tiles = 1 + std::max(plan.pair_s, plan.pair_o);
  prm.span = reinterpret_cast<int2*>(ws + kDataOffset);
  prm.wait_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  prm.ml = reinterpret_cast<float2*>(ws + plan.off_ml);
  prm.opart = reinterpret_cast<float*>(ws + plan.off_part);
  // queries: boxes of 64 elements x the heads of one key-value head x nodes;
  // caches: 64 elements x one head x 128 positions
  CUtensorMap map[5];
  {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)B * N};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)Hq * D * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)prm.G, (cuuint32_t)prm.tok};
    st = encode_bf16(&map[0], q, 3, dims, strides, box);
    if (st != SPEC_OK) return st;
  }
  const cuuint32_t box[4] = {64, 1, (cuuint32_t)sv::kAtKeys, 1};
  const cuuint64_t row = (cuuint64_t)Hkv * D * 2;
  for (int i = 0; i < 2; ++i) {
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)Hkv, (cuuint64_t)L, (cuuint64_t)B};
    const cuuint64_t strides[3] = {(cuuint64_t)D * 2, row, (cuuint64_t)seq_stride};
    st = encode_bf16(&map[1 + i], i == 0 ? k_cache : v_cache, 4, dims, strides, box);
    if (st != SPEC_OK) return st;
    if (P == 0) {
      map[3 + i] = map[1 + i];  // never read
      continue;
    }
    const cuuint64_t pdims[4] = {(cuuint64_t)D, (cuuint64_t)Hkv, (cuuint64_t)P, 1};
    const cuuint64_t pstrides[3] = {(cuuint64_t)D * 2, row, row * P};
    st = encode_bf16(&map[3 + i], i == 0 ? prefix_k : prefix_v, 4, pdims, pstrides, box);
    if (st != SPEC_OK) return st;
  }
  return D == 128 ? run_attention<128>(prm, map, stream) : run_attention<64>(prm, map, stream);
}

spec_status_t spec_tree_grow(const void* draft_logits, int dtype, float temperature, int B,
                             int D, int K, int V, int M, int32_t* tokens, int32_t* parents,
                             int32_t* depth, float* values, void* workspace,
                             size_t workspace_bytes, void* stream) {
  if (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16) return SPEC_ERR_INVALID_ARG;
  if (B < 0 || D < 1 || D > sv::kGrowMaxD || K < 1 || K > sv::kGrowMaxK || V < K ||
      V > SPEC_MAX_V || !(temperature > 0.0f) || !std::isfinite(temperature))
    return SPEC_ERR_INVALID_ARG;
  const int nnodes = 1 + K + (D - 1) * K * K;
  if (M < 0 || M > nnodes - 1) return SPEC_ERR_INVALID_ARG;
  Layout L;
  if (!make_layout(SPEC_MODE_TREE_GROW, B, K, V, dtype, &L)) return SPEC_ERR_INVALID_ARG;
  if (B == 0) return SPEC_OK;
  if (!draft_logits || !tokens || !parents || !depth || !values) return SPEC_ERR_INVALID_ARG;
  if (!aligned(draft_logits, elem_bytes(dtype)) || !aligned(tokens, 4) || !aligned(parents, 4) ||
      !aligned(depth, 4) || !aligned(values, 4))
    return SPEC_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < L.bytes) return SPEC_ERR_WORKSPACE;
  if (!aligned(workspace, kAlign)) return SPEC_ERR_ALIGNMENT;
  char* ws = static_cast<char*>(workspace);
  sv::GrowParams prm;
  std::memset(&prm, 0, sizeof prm);
  prm.logits = draft_logits;
  prm.scale = (float)(1.4426950408889634 / (double)temperature);
  prm.B = B;
  prm.D = D;
  prm.K = K;
  prm.V = V;
  prm.M = M;
  prm.nchunks = L.nchunks;
  prm.rec = reinterpret_cast<sv::GrowRec*>(ws + L.off_part);
  prm.nval = reinterpret_cast<double*>(ws + L.off_desc);
  prm.npar = reinterpret_cast<int32_t*>(ws + L.off_gsum);
  prm.ntok = prm.npar + (size_t)B * sv::kGrowMaxNodes;
  prm.ndep = prm.ntok + (size_t)B * sv::kGrowMaxNodes;
  prm.tokens = tokens;
  prm.parents = parents;
  prm.depth = depth;
  prm.values = values;
  prm.flags = reinterpret_cast<unsigned*>(ws);
  // every draft row the growth reads, reduced in one streaming launch
  prm.rows_per_tree = 1 + (D - 1) * K;
  if ((long long)B * prm.rows_per_tree * prm.nchunks > INT32_MAX) return SPEC_ERR_INVALID_ARG;
  prm.items = B * prm.rows_per_tree * prm.nchunks;
  const bool vec = vec_ok(draft_logits, V, dtype);  // whole 16-byte vectors per row
  spec_status_t st;
  if (vec) {
    int grid = 0;
    if (dtype == SPEC_DTYPE_BF16) {
      st = persistent_grid<sv::grow_topk_stream_kernel<sv::BF16>>(prm.items, &grid);
      if (st == SPEC_OK)
        st = launch(sv::grow_topk_stream_kernel<sv::BF16>, grid, kStreamSmem, prm, stream, true);
    } else {
      st = persistent_grid<sv::grow_topk_stream_kernel<sv::F32>>(prm.items, &grid);
      if (st == SPEC_OK)
        st = launch(sv::grow_topk_stream_kernel<sv::F32>, grid, kStreamSmem, prm, stream, true);
    }
  } else if (dtype == SPEC_DTYPE_BF16) {
    st = launch(sv::grow_topk_kernel<sv::BF16, false>, prm.items, 0, prm, stream, true);
  } else {
    st = launch(sv::grow_topk_kernel<sv::F32, false>, prm.items, 0, prm, stream, true);
  }
  if (st != SPEC_OK) return st;
  // the node bookkeeping of every layer and the final ranking, one CTA per tree
  st = ensure_smem<sv::grow_tree_kernel>(sv::kGrowTreeSmem);
  if (st != SPEC_OK) return st;
  return launch(sv::grow_tree_kernel, B * sv::kGrowTreeCluster,
                sv::grow_tree_smem(L.nchunks, K, prm.rows_per_tree, nnodes), prm, stream,
                true, sv::kGrowTreeCluster, sv::kGrowTreeThreads);
}

spec_status_t spec_kv4_commit_path(void* pages, int layers, long long n_pages, int page_size,
                                   int Hkv, int D, const int32_t* page_table, int W,
                                   const void* node_k, const void* node_v,
                                   const int32_t* base_len, const int32_t* accepted_len,
                                   const int32_t* path_nodes, int max_depth, const int32_t* kv_exp,
                                   int B, int N, int32_t* new_len, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  if (!kv4_shape_ok(n_pages, page_size, Hkv, D, W) || layers < 1 || layers > 65535 || B < 0 ||
      N < 1 || N > SPEC_MAX_TREE_NODES ||
      (path_nodes && (max_depth < 0 || max_depth > SPEC_MAX_TREE_DEPTH || !accepted_len)) ||
      (long long)B * layers > INT32_MAX / 64)
    return SPEC_ERR_INVALID_ARG;
  if (B == 0) return SPEC_OK;
  if (!pages || !page_table || !node_k || !node_v || !base_len || !new_len)
    return SPEC_ERR_INVALID_ARG;
  if (!aligned(pages, 16) || !aligned(node_k, 16) || !aligned(node_v, 16) ||
      !aligned(page_table, 4) || !aligned(base_len, 4) || !aligned(accepted_len, 4) ||
      !aligned(path_nodes, 4) || !aligned(kv_exp, 4) || !aligned(new_len, 4))
    return SPEC_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < kHeaderBytes) return SPEC_ERR_WORKSPACE;
  if (!aligned(workspace, kAlign)) return SPEC_ERR_ALIGNMENT;
  // (many CTAs read a sequence's inputs, one writes its new length)
  const size_t seqs = 4 * (size_t)B, nodes = 2 * (size_t)layers * B * N * Hkv * D;
  if (overlap(new_len, seqs, base_len, seqs) || overlap(new_len, seqs, accepted_len, seqs) ||
      overlap(new_len, seqs, path_nodes, path_nodes ? seqs * (max_depth + 1) : 0) ||
      overlap(new_len, seqs, page_table, seqs * W) || overlap(new_len, seqs, kv_exp, 8 * (size_t)layers) ||
      overlap(new_len, seqs, node_k, nodes) || overlap(new_len, seqs, node_v, nodes))
    return SPEC_ERR_INVALID_ARG;
  sv::Kv4Params prm;
  std::memset(&prm, 0, sizeof prm);
  prm.pages = static_cast<uint8_t*>(pages);
  prm.table = page_table;
  prm.node_k = static_cast<const uint16_t*>(node_k);
  prm.node_v = static_cast<const uint16_t*>(node_v);
  prm.base_len = base_len;
  prm.accepted = accepted_len;
  prm.path = path_nodes;
  prm.exps = kv_exp;
  prm.new_len = new_len;
  prm.flags = reinterpret_cast<unsigned*>(workspace);
  prm.n_pages = n_pages;
  prm.B = B;
  prm.N = N;
  prm.Hkv = Hkv;
  prm.W = W;
  prm.lg = log2_of(page_size);
  prm.max_depth = max_depth;
  prm.layers = layers;
  kv4_grid(&prm, path_nodes ? std::min(max_depth + 1, N) : N, D);
  const int grid = layers * B * prm.blocks;
  return D == 128 ? launch(sv::kv4_commit_kernel<128>, grid, 0, prm, stream, true, 1, sv::kKv4Threads)
                  : launch(sv::kv4_commit_kernel<64>, grid, 0, prm, stream, true, 1, sv::kKv4Threads);
}

spec_status_t spec_kv4_read(const void* pages, int layers, long long n_pages, int page_size,
                            int Hkv, int D, const int32_t* page_table, int W,
                            const int32_t* length, const int32_t* kv_exp, int B, int L,
                            void* k_out, void* v_out, long long layer_stride,
                            long long seq_stride, void* workspace, size_t workspace_bytes,
                            void* stream) {
  if (!kv4_shape_ok(n_pages, page_size, Hkv, D, W) || layers < 1 || layers > 65535 || B < 0 ||
      L < 1 || (long long)B * layers > INT32_MAX / 64)
    return SPEC_ERR_INVALID_ARG;
  if (seq_stride < (long long)L * Hkv * D * 2 ||
      (layers > 1 && (B > 1 ? seq_stride > INT64_MAX / B : false)) ||
      (layers > 1 && layer_stride < (long long)std::max(B - 1, 0) * seq_stride + (long long)L * Hkv * D * 2))
    return SPEC_ERR_INVALID_ARG;
  if (B == 0) return SPEC_OK;
  if (!pages || !page_table || !length || !k_out || !v_out) return SPEC_ERR_INVALID_ARG;
  if (!aligned(pages, 16) || !aligned(k_out, 16) || !aligned(v_out, 16) || layer_stride % 16 ||
      seq_stride % 16 || !aligned(page_table, 4) || !aligned(length, 4) || !aligned(kv_exp, 4))
    return SPEC_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < kHeaderBytes) return SPEC_ERR_WORKSPACE;
  if (!aligned(workspace, kAlign)) return SPEC_ERR_ALIGNMENT;
  sv::Kv4Params prm;
  std::memset(&prm, 0, sizeof prm);
  prm.pages = static_cast<uint8_t*>(const_cast<void*>(pages));
  prm.table = page_table;
  prm.length = length;
  prm.exps = kv_exp;
  prm.k_out = static_cast<uint16_t*>(k_out);
  prm.v_out = static_cast<uint16_t*>(v_out);
  prm.flags = reinterpret_cast<unsigned*>(workspace);
  prm.n_pages = n_pages;
  prm.out_layer = layer_stride / 2;
  prm.out_seq = seq_stride / 2;
  prm.B = B;
  prm.Hkv = Hkv;
  prm.W = W;
  prm.lg = log2_of(page_size);
  prm.L = L;
  prm.layers = layers;
  kv4_grid(&prm, L, D);
  const int grid = layers * B * prm.blocks;
  return D == 128 ? launch(sv::kv4_read_kernel<128>, grid, 0, prm, stream, true, 1, sv::kKv4Threads)
                  : launch(sv::kv4_read_kernel<64>, grid, 0, prm, stream, true, 1, sv::kKv4Threads);
}

size_t spec_tree_attention_kv4_workspace_bytes(int B, int N, int Hq, int Hkv, int D) {
  if (!attn_shape_ok(B, N, Hq, Hkv, D, 0)) return 0;
  return attn4_plan(B, N, Hq, Hkv, D).bytes;
}

spec_status_t spec_tree_attention_kv4(const void* q, const void* pages, long long n_pages,
                                      int page_size, const int32_t* page_table, int W,
                                      const void* node_k, const void* node_v,
                                      const uint32_t* mask, const int32_t* base_len,
                                      const int32_t* kv_exp, int B, int N, int Hq, int Hkv, int D,
                                      float scale, void* out, float* lse, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  if (!attn_shape_ok(B, N, Hq, Hkv, D, 0) || !kv4_shape_ok(n_pages, page_size, Hkv, D, W) ||
      (long long)W * page_size + N > INT32_MAX - 256 || !(scale > 0.0f) ||
      !(scale < 1.7014118e38f))  // 2^127: scale * log2(e) stays finite
    return SPEC_ERR_INVALID_ARG;
  if (B == 0) return SPEC_OK;
  if (!q || !pages || !page_table || !node_k || !node_v || !base_len || !out)
    return SPEC_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(pages, 16) || !aligned(node_k, 16) || !aligned(node_v, 16) ||
      !aligned(out, 16) || !aligned(page_table, 4) || !aligned(mask, 4) || !aligned(base_len, 4) ||
      !aligned(kv_exp, 4) || !aligned(lse, 4))
    return SPEC_ERR_ALIGNMENT;
  if (!workspace) return SPEC_ERR_WORKSPACE;
  if (!aligned(workspace, kAlign)) return SPEC_ERR_ALIGNMENT;
  const Attn4Plan plan = attn4_plan(B, N, Hq, Hkv, D);
  if (workspace_bytes < plan.bytes) return SPEC_ERR_WORKSPACE;
  // (CTAs that share a sequence's or a node's inputs write their outputs at different times)
  const size_t rows = (size_t)B * N, heads = 2 * rows * D;  // heads: bytes of a head of all nodes
  const std::pair<const void*, size_t> outs[] = {{out, heads * Hq}, {lse, 4 * rows * Hq}};
  const std::pair<const void*, size_t> ins[] = {
      {q, heads * Hq}, {node_k, heads * Hkv}, {node_v, heads * Hkv},
      {pages, (size_t)n_pages * Hkv * sv::kv4_block(page_size, D)}, {page_table, 4 * (size_t)B * W},
      {mask, 4 * rows * ((N + 31) / 32)}, {base_len, 4 * (size_t)B}, {kv_exp, 8}};
  for (const auto& o : outs)
    for (const auto& i : ins)
      if (overlap(o.first, o.second, i.first, i.second)) return SPEC_ERR_INVALID_ARG;
  int sms = 0;
  const spec_status_t st = sm_count(&sms);
  if (st != SPEC_OK) return st;
  char* ws = static_cast<char*>(workspace);
  if (plan.tiles) {
    sv::AttnQParams t;
    std::memset(&t, 0, sizeof t);
    t.q = static_cast<const uint16_t*>(q);
    t.mask = mask;
    t.base_len = base_len;
    t.out = static_cast<uint16_t*>(out);
    t.lse = lse;
    t.flags = reinterpret_cast<unsigned*>(ws);
    t.scale_log2 = (float)(1.4426950408889634 * (double)scale);
    t.B = B;
    t.N = N;
    t.Hq = Hq;
    t.Hkv = Hkv;
    t.G = Hq / Hkv;
    t.W = (N + 31) / 32;
    // positions that a sequence may have: W pages of committed ones, and its nodes
    t.L = W * page_size + N;
    t.tok = plan.t.tok;
    t.pair_o = plan.t.pair_o;
    t.mg_o = plan.t.mg_o;
    t.rows_o = plan.t.rows_o;
    t.by_cta = plan.t.by_cta;
    t.own0 = plan.t.own0;
    t.nctas = std::min(sms, sv::kAtMaxCtas);
    t.q_tiles = 1 + plan.t.pair_o;
    t.span = reinterpret_cast<int2*>(ws + kDataOffset);
    t.ml = reinterpret_cast<float2*>(ws + plan.t.off_ml);
    t.opart = reinterpret_cast<float*>(ws + plan.t.off_part);
    sv::atq_limit(&t, g_wait_limit_ns.load(std::memory_order_relaxed));
    t.pages = static_cast<const uint8_t*>(pages);
    t.table = page_table;
    {
      const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)B * N};
      const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)Hq * D * 2};
      const cuuint32_t box[3] = {64, (cuuint32_t)t.G, (cuuint32_t)t.tok};
      const spec_status_t e = encode_bf16(&t.map_q, q, 3, dims, strides, box);
      if (e != SPEC_OK) return e;
    }
    for (int i = 0; i < 2; ++i) {
      const cuuint64_t row = (cuuint64_t)Hkv * D * 2;
      const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)Hkv, (cuuint64_t)N, (cuuint64_t)B};
      const cuuint64_t strides[3] = {(cuuint64_t)D * 2, row, row * N};
      const cuuint32_t box[4] = {64, 1, (cuuint32_t)sv::kAtKeys, 1};
      const spec_status_t e = encode_bf16(i == 0 ? &t.map_k : &t.map_v, i == 0 ? node_k : node_v,
                                          4, dims, strides, box);
      if (e != SPEC_OK) return e;
    }
    t.exps = kv_exp;
    t.n_pages = n_pages;
    t.Wt = W;
    t.lg = log2_of(page_size);
    return D == 128 ? run_attn4_tiles<128>(t, stream) : run_attn4_tiles<64>(t, stream);
  }
  sv::Attn4Params prm;
  std::memset(&prm, 0, sizeof prm);
  prm.q = static_cast<const uint16_t*>(q);
  prm.pages = static_cast<const uint8_t*>(pages);
  prm.table = page_table;
  prm.nk = static_cast<const uint16_t*>(node_k);
  prm.nv = static_cast<const uint16_t*>(node_v);
  prm.mask = mask;
  prm.base_len = base_len;
  prm.exps = kv_exp;
  prm.out = static_cast<uint16_t*>(out);
  prm.lse = lse;
  prm.flags = reinterpret_cast<unsigned*>(ws);
  prm.span = reinterpret_cast<int2*>(ws + kDataOffset);
  prm.ml = reinterpret_cast<float2*>(ws + plan.off_ml);
  prm.opart = reinterpret_cast<float*>(ws + plan.off_part);
  prm.wait_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  prm.n_pages = n_pages;
  prm.scale_log2 = (float)(1.4426950408889634 * (double)scale);
  prm.B = B;
  prm.N = N;
  prm.Hq = Hq;
  prm.Hkv = Hkv;
  prm.G = Hq / Hkv;
  prm.W = W;
  prm.Wm = (N + 31) / 32;
  prm.lg = log2_of(page_size);
  prm.rows = plan.rows;
  return D == 128 ? run_attn4<128>(prm, plan.nt, sms, stream)
                  : run_attn4<64>(prm, plan.nt, sms, stream);
}

size_t spec_kv_pages_workspace_bytes(long long n_pages, int rows) {
  PagesLayout L;
  return pages_layout(n_pages, rows, &L) ? L.bytes : 0;
}

spec_status_t spec_kv_pages_fork(void* pages, int planes, long long plane_stride,
                                 long long n_pages, long long page_bytes, int page_size,
                                 const int32_t* page_table, const int32_t* length, int B,
                                 const int32_t* parent, const int32_t* need, int B2, int W,
                                 int32_t* new_table, int32_t* new_len, int32_t* used,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  if (page_size < 1 || B2 < 0 || B2 > SPEC_KV_MAX_TABLE || (long long)W * page_size > INT32_MAX ||
      (!parent && B2 > B))
    return SPEC_ERR_INVALID_ARG;
  sv::PagesParams prm;
  const spec_status_t st = pages_params(pages, planes, plane_stride, n_pages, page_bytes,
                                        page_table, B, B2, W, new_table, used, workspace,
                                        workspace_bytes, &prm);
  if (st != SPEC_OK) return st;
  if ((B > 0 && !length) || (B2 > 0 && !new_len)) return SPEC_ERR_INVALID_ARG;
  if (!aligned(length, 4) || !aligned(parent, 4) || !aligned(need, 4) || !aligned(new_len, 4))
    return SPEC_ERR_ALIGNMENT;
  const size_t rows = 4 * (size_t)B, rows2 = 4 * (size_t)B2;
  for (const auto& o : {std::pair<const void*, size_t>(new_table, rows2 * W), {new_len, rows2}, {used, 4}})
    if (overlap(o.first, o.second, page_table, rows * W) || overlap(o.first, o.second, length, rows) ||
        overlap(o.first, o.second, parent, rows2) || overlap(o.first, o.second, need, rows2))
      return SPEC_ERR_INVALID_ARG;
  prm.length = length;
  prm.parent = parent;
  prm.need = need;
  prm.new_len = new_len;
  prm.page = page_size;
  return run_pages(true, prm, stream);
}

spec_status_t spec_kv_pages_compact(void* pages, int planes, long long plane_stride,
                                    long long n_pages, long long page_bytes,
                                    const int32_t* page_table, int B, int W, int32_t* new_table,
                                    int32_t* used, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  sv::PagesParams prm;
  const spec_status_t st = pages_params(pages, planes, plane_stride, n_pages, page_bytes,
                                        page_table, B, B, W, new_table, used, workspace,
                                        workspace_bytes, &prm);
  if (st != SPEC_OK) return st;
  const size_t bytes = 4 * (size_t)B * W;
  if ((new_table != page_table && overlap(new_table, bytes, page_table, bytes)) ||
      overlap(used, 4, page_table, bytes))
    return SPEC_ERR_INVALID_ARG;
  return run_pages(false, prm, stream);
}

size_t spec_beam_select_workspace_bytes(int B, int K, int V, int M, int dtype) {
  BeamLayout L;
  return beam_layout(B, K, V, M, dtype, &L) ? L.bytes : 0;
}

spec_status_t spec_beam_select(const void* logits, int dtype, const float* scores,
                               const int32_t* finished, int eos, float temperature, int B, int K,
                               int V, int M, float* out_scores, int32_t* out_parents,
                               int32_t* out_tokens, int32_t* out_finished, void* workspace,
                               size_t workspace_bytes, void* stream) {
  BeamLayout L;
  if (!beam_layout(B, K, V, M, dtype, &L) || eos < -1 || eos >= V || !(temperature > 0.0f) ||
      !std::isfinite(temperature))
    return SPEC_ERR_INVALID_ARG;
  if (B == 0) return SPEC_OK;
  if (!logits || !scores || !out_scores || !out_parents || !out_tokens || !out_finished)
    return SPEC_ERR_INVALID_ARG;
  if (!aligned(logits, elem_bytes(dtype)) || !aligned(scores, 4) || !aligned(finished, 4) ||
      !aligned(out_scores, 4) || !aligned(out_parents, 4) || !aligned(out_tokens, 4) ||
      !aligned(out_finished, 4))
    return SPEC_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < L.bytes) return SPEC_ERR_WORKSPACE;
  if (!aligned(workspace, kAlign)) return SPEC_ERR_ALIGNMENT;
  const size_t in = 4 * (size_t)B * K, picked = 4 * (size_t)B * M;
  for (const void* o : {(const void*)out_scores, (const void*)out_parents, (const void*)out_tokens,
                        (const void*)out_finished})
    if (overlap(o, picked, scores, in) || overlap(o, picked, finished, in) ||
        overlap(o, picked, logits, (size_t)B * K * V * elem_bytes(dtype)))
      return SPEC_ERR_INVALID_ARG;
  char* ws = static_cast<char*>(workspace);
  sv::BeamParams prm;
  std::memset(&prm, 0, sizeof prm);
  prm.logits = logits;
  prm.score = scores;
  prm.finished = finished;
  prm.part = reinterpret_cast<float2*>(ws + kDataOffset);
  prm.runs = reinterpret_cast<float*>(ws + L.off_runs);
  prm.out_score = out_scores;
  prm.out_parent = out_parents;
  prm.out_token = out_tokens;
  prm.out_finished = out_finished;
  prm.flags = reinterpret_cast<unsigned*>(ws);
  // (finite, so that 0 times it is 0: temperatures below 2^-127 count as that)
  prm.scale = (float)std::min(1.4426950408889634 / (double)temperature, 3.4028234663852886e38);
  prm.B = B;
  prm.K = K;
  prm.V = V;
  prm.M = M;
  prm.eos = eos;
  prm.nchunks = L.nchunks;
  prm.items = B * K * L.nchunks;
  const bool vec = vec_ok(logits, V, dtype);
  return dtype == SPEC_DTYPE_BF16 ? run_beam<sv::BF16>(prm, vec, stream)
                                  : run_beam<sv::F32>(prm, vec, stream);
}

spec_status_t spec_verify_read_flags(void* workspace, uint32_t* host_flags, int clear,
                                     void* stream) {
  if (!workspace || !host_flags) return SPEC_ERR_INVALID_ARG;
  if (!aligned(workspace, kAlign)) return SPEC_ERR_ALIGNMENT;
  cudaStream_t s = (cudaStream_t)stream;
  if (cudaMemcpyAsync(host_flags, workspace, sizeof(uint32_t), cudaMemcpyDeviceToHost, s) !=
      cudaSuccess)
    return SPEC_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return SPEC_ERR_CUDA;
  if (clear && cudaMemsetAsync(workspace, 0, sizeof(uint32_t), s) != cudaSuccess)
    return SPEC_ERR_CUDA;
  return SPEC_OK;
}

spec_status_t spec_verify_greedy_noalloc(const void* target_logits, int dtype,
                                         const int32_t* draft_tokens, int B, int k, int V,
                                         int32_t* accepted_len, int32_t* out_tokens, void* stream) {
  if (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16) return SPEC_ERR_INVALID_ARG;
  if (B < 0 || k < 0 || k > SPEC_MAX_K || V < 1 || V > SPEC_MAX_V) return SPEC_ERR_INVALID_ARG;
  Layout L;
  if (!make_layout(SPEC_MODE_GREEDY, B, k, V, dtype, &L)) return SPEC_ERR_INVALID_ARG;
  if (L.bytes > (size_t)SPEC_NOALLOC_SCRATCH_BYTES) return SPEC_ERR_TOO_LARGE;
  if (B == 0) return SPEC_OK;
  if (!target_logits || !accepted_len || !out_tokens || (k > 0 && !draft_tokens))
    return SPEC_ERR_INVALID_ARG;
  if (!aligned(target_logits, elem_bytes(dtype)) || !aligned(accepted_len, 4) ||
      !aligned(out_tokens, 4) || (k > 0 && !aligned(draft_tokens, 4)))
    return SPEC_ERR_ALIGNMENT;
  void* scratch = nullptr;
  const spec_status_t st = noalloc_scratch(&scratch);
  if (st != SPEC_OK) return st;
  // the flag word starts clear on every call (nothing else needs zeroing)
  if (cudaMemsetAsync(scratch, 0, sizeof(uint32_t), (cudaStream_t)stream) != cudaSuccess)
    return SPEC_ERR_CUDA;
  return spec_verify_greedy(target_logits, dtype, draft_tokens, B, k, V, accepted_len, out_tokens,
                            scratch, (size_t)SPEC_NOALLOC_SCRATCH_BYTES, stream);
}

spec_status_t spec_verify_selftest_exp2(const float* x, float* y_fma, float* y_sfu, int n,
                                        void* stream) {
  if (n < 0 || (n > 0 && (!x || !y_fma || !y_sfu))) return SPEC_ERR_INVALID_ARG;
  if (n == 0) return SPEC_OK;
  sv::selftest_exp2_kernel<<<(n + 255) / 256, 256, 0, (cudaStream_t)stream>>>(x, y_fma, y_sfu, n);
  if (cudaGetLastError() != cudaSuccess) return SPEC_ERR_CUDA;
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return SPEC_OK;
}

uint64_t spec_verify_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

void spec_verify_set_wait_limit_ns(uint64_t limit_ns) {
  g_wait_limit_ns.store(limit_ns == 0 ? sv::kWaitLimitNs : limit_ns, std::memory_order_relaxed);
}

const char* spec_status_string(int status) {
  switch (status) {
    case SPEC_OK: return "ok";
    case SPEC_ERR_INVALID_ARG: return "invalid argument";
    case SPEC_ERR_ALIGNMENT: return "misaligned pointer";
    case SPEC_ERR_WORKSPACE: return "workspace missing or too small";
    case SPEC_ERR_CUDA: return "CUDA error";
    case SPEC_ERR_TOO_LARGE: return "call exceeds the fixed no-allocation scratch";
    default: return "unknown status";
  }
}

int spec_verify_abi_version(void) { return SPEC_VERIFY_ABI_VERSION; }

}  // extern "C"
