// Shared by the serving operators' translation units (declared in
// include/mk_serve.h): error mapping, launches with programmatic dependent
// launch, and the status word.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "../../include/mk_serve.h"

namespace mk {

inline int serve_code(cudaError_t e) {
  if (e == cudaSuccess) return MK_OK;
  cudaGetLastError();
  if (e == cudaErrorMemoryAllocation) return MK_ERR_OUT_OF_MEMORY;
  if (e == cudaErrorLaunchOutOfResources || e == cudaErrorInvalidConfiguration) return MK_ERR_LAUNCH;
  return MK_ERR_CUDA;
}

// Launch fn; `overlap`: its blocks may start while the kernel before it on
// the stream drains (the kernel then calls pdl_wait before it touches what
// that one wrote); `cluster` > 1: blocks of a cluster.
template <class... A, class... B>
int serve_launch(void (*fn)(A...), dim3 grid, int threads, size_t smem, cudaStream_t st, bool overlap, int cluster,
                 B... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  int n = 0;
  if (overlap) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = (unsigned)cluster;
    at[n].val.clusterDim.y = 1;
    at[n++].val.clusterDim.z = 1;
  }
  cfg.attrs = at;
  cfg.numAttrs = (unsigned)n;
  return serve_code(cudaLaunchKernelEx(&cfg, fn, static_cast<std::remove_const_t<A>>(args)...));
}

// Streaming multiprocessors of the current device (asked for once per device:
// the calls here are short enough for the question to show).
inline int serve_sms(int *out) {
  static std::atomic<int> known[64];
  int d = 0;
  cudaError_t e = cudaGetDevice(&d);
  if (e != cudaSuccess) return serve_code(e);
  int n = d < 64 ? known[d].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, d);
    if (e != cudaSuccess) return serve_code(e);
    if (d < 64) known[d].store(n, std::memory_order_relaxed);
  }
  *out = n;
  return MK_OK;
}
// Allow fn `bytes` of dynamic shared memory on the current device (once per
// device and function: `done` is the function's own).
inline int serve_allow_smem(std::atomic<uint64_t> &done, const void *fn, size_t bytes) {
  int d = 0;
  cudaError_t e = cudaGetDevice(&d);
  if (e != cudaSuccess) return serve_code(e);
  const uint64_t bit = d < 64 ? 1ull << d : 0;
  if (bit && (done.load(std::memory_order_relaxed) & bit)) return MK_OK;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) return serve_code(e);
  done.fetch_or(bit, std::memory_order_relaxed);
  return MK_OK;
}

// mk_token_probs with the temperatures `ts` words apart (0: one for all rows).
int token_probs(const void *logits, int32_t dtype, int64_t logits_stride, const float *temperature, int ts, float *probs,
                int64_t probs_stride, int32_t n, int32_t vocab, void *stream);

// mk_attn_shared inside an engine's step (bf16 cache, one token a sequence, scale
// above 0): a->q is the step's q and `out` its attention output, both tagged
// 32-bit words [batch][n_q_heads][head_dim]; a->out is not used (but not NULL).
int attn_shared_tagged(const mk_attn_shared_args *a, float *out, const unsigned *epoch, void *workspace, void *stream);

inline bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

#ifdef __CUDACC__
// The kernel before this one on the stream has finished and its writes are visible.
static __device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel's blocks may be scheduled.
static __device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// First code wins.
static __device__ __forceinline__ void report(int32_t *status, int code) {
  if (status) atomicCAS(status, 0, code);
}
static __device__ __forceinline__ int warp_incl_sum(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}
#endif

}  // namespace mk
