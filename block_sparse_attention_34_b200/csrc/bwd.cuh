// What the training kernels' files share: the launch arguments and the check
// of a kept list.
#pragma once

#include "common.cuh"

#include <atomic>
#include <mutex>

namespace paro {

// Opts kernel Kern into `bytes` of dynamic shared memory on the current
// device (kClusters: and into clusters of more than 8 CTAs), once for each
// size that grows: the attribute outlives the call, and setting it every
// time is a microsecond of a small call.  (Under a lock: of two threads that
// set it at once the smaller size could stay.)
template <auto Kern, bool kClusters = false>
cudaError_t opt_in_smem(int bytes) {
  constexpr int kDevices = 64;
  static std::atomic<int> done[kDevices];
  static std::mutex mutex;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < kDevices && done[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
  const std::lock_guard<std::mutex> lock(mutex);
  if (dev < kDevices && done[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (kClusters && e == cudaSuccess)
    e = cudaFuncSetAttribute(Kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && dev < kDevices) done[dev].store(bytes, std::memory_order_relaxed);
  return e;
}

struct BwdArgs {
  const __nv_bfloat16 *q, *k, *v;  // permuted [B*heads, Np, d]
  __nv_bfloat16* dop;              // workspace: dO in the permuted order
  float *nlse, *ndel;              // workspace: -lse log2 e and -D of each permuted row
  uint32_t* mask;                  // workspace: [B*heads, NB, words], bit i of row j: i keeps j
  int words;
  int32_t* checked;                // workspace: entries of each kept list, -1 if malformed
  int32_t* counters;               // workspace: two, zero: blocks handed out
  const int32_t *idx, *counts;
  int k_max;
  __nv_bfloat16 *dq, *dk, *dv;  // natural order
  int32_t* status;
};

// Whether a kept list is well formed (count in [0, k_max], entries ascending
// in [0, NB)): one warp, the same answer in every lane.
__device__ __forceinline__ bool list_ok(const int32_t* __restrict__ ids, int cnt, int k_max,
                                        int NB, int lane) {
  bool bad = cnt < 0 || cnt > k_max;
  if (!bad)
    for (int e = lane; e < cnt; e += 32) {
      const int j = __ldg(ids + e);
      const int prev = e > 0 ? __ldg(ids + e - 1) : -1;
      bad |= j <= prev || j >= NB;
    }
  return !__any_sync(0xffffffffu, bad);
}

cudaError_t launch_bwd_prep(const void* out, const void* dout, const float* lse,
                            const float* dlse, const BwdArgs& a, const Grid& g, cudaStream_t s);
// The kernels of block 128 (attn_sm100.cu, attn_bwd_sm100.cu) and of block 64
// (attn_fwd64_sm100.cu, attn_bwd64_sm100.cu).  Of the arguments the forward
// pass uses q, k, v, idx, counts, k_max and status.
cudaError_t launch_fwd_lse_sm100(const BwdArgs& a, const Grid& g, void* out, float* lse,
                                 cudaStream_t s);
cudaError_t launch_bwd_sm100(const BwdArgs& a, const Grid& g, cudaStream_t s);
cudaError_t launch_bwd64_sm100(const BwdArgs& a, const Grid& g, cudaStream_t s);
cudaError_t launch_fwd64_sm100(const BwdArgs& a, const Grid& g, void* out, float* lse,
                               cudaStream_t s);

}  // namespace paro
