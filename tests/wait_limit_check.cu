// How long the tree attention over 4-bit pages waits for a role that does not answer
// (atq_wait, atq_wait_warp of sv_attn4t.cuh), built by tests/test_gpu_wait_limit.py
// with nvcc: one CTA of one warp waits for a phase that nothing completes, with
// limits of its own, and reads the GPU's clock before and behind.  Every wait ends
// by its limit; prints one line per wait.
#include <cstdio>

#include "sv_attn4t.cuh"

__global__ void waits(const __grid_constant__ sv::AttnQParams p, int warp, int gone, int ready,
                      unsigned long long more, unsigned long long* out) {
  __shared__ uint64_t bar;
  __shared__ int abort;
  if (threadIdx.x == 0) {
    sv::mbar_init(&bar, 1);
    abort = gone;
    sv::mbar_init_fence();
  }
  __syncthreads();
  if (threadIdx.x == 0 && ready) sv::mbar_arrive(&bar);
  __syncwarp();
  const uint64_t t0 = sv::global_ns();
  bool ok = false;
  if (warp)
    ok = sv::atq_wait_warp(p, &bar, 0, &abort);
  else if (threadIdx.x == 0)
    ok = sv::atq_wait(p, &bar, 0, &abort, more);
  if (threadIdx.x == 0) {
    out[0] = sv::global_ns() - t0;
    out[1] = ok;
  }
}

int main() {
  unsigned long long *out, host[2];
  if (cudaMalloc(&out, sizeof host) != cudaSuccess) return 1;
  const unsigned long long limits[] = {1, 20, 3000, 50000, 2000000, 30000000, 200000000};
  for (int warp = 0; warp < 2; ++warp)
    for (int kind = 0; kind < 4; ++kind)  // runs out; another role gave up; complete; 5 ms more
      for (const unsigned long long limit : limits) {
        const unsigned long long more = kind == 3 ? 5000000 : 0;
        if (warp && more) continue;
        sv::AttnQParams p{};
        sv::atq_limit(&p, limit);
        for (int i = 0; i < 2; ++i)  // (the first one loads the code)
          waits<<<1, 32>>>(p, warp, kind == 1, kind == 2, more, out);
        if (cudaMemcpy(host, out, sizeof host, cudaMemcpyDeviceToHost) != cudaSuccess) return 1;
        std::printf("%d %d %llu %llu %llu\n", warp, kind, limit, host[0], host[1]);
      }
  return 0;
}
