// paged.cuh -- what the paged K/V cache's kernels share: element access and the host-side
// checks of rq_paged_kv (include/rq.h).
#pragma once

#include <limits.h>

#include <atomic>

#include "../../include/rq.h"
#include "common.cuh"

namespace rqk {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The cache's own description: sizes, types, alignment.
inline rq_status paged_kv_check(const rq_paged_kv* kv) {
  if (!kv || !kv->k || !kv->v || !aligned16(kv->k) || !aligned16(kv->v)) return RQ_ERR_ARG;
  if (kv->dtype != RQ_F32 && kv->dtype != RQ_BF16) return RQ_ERR_ARG;
  if (kv->heads < 1 || kv->block_size < 1 || kv->n_blocks < 1) return RQ_ERR_ARG;
  if (kv->head_dim != 32 && kv->head_dim != 64 && kv->head_dim != 128) return RQ_ERR_UNSUPPORTED;
  const int64_t unit = kv->dtype == RQ_BF16 ? 8 : 4;  // elements of 16 bytes
  for (int64_t s : {kv->block_stride, kv->row_stride, kv->head_stride})
    if (s < 0 || s % unit != 0) return RQ_ERR_ARG;
  return RQ_OK;
}

constexpr int kMaxDevices = 64;

// multiprocessors of the current device, looked up once (0 if there is none)
inline int sm_count() {
  static std::atomic<int> known[kMaxDevices];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < kMaxDevices && (sms = known[dev].load(std::memory_order_relaxed)) != 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < kMaxDevices) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

// CTAs of `kernel` that are resident at once on the current device; `cache`: one entry a
// device for this kernel and shared-memory size, 0 until looked up.
template <typename K>
inline cudaError_t resident_ctas(K* kernel, int threads, size_t smem, std::atomic<int>* cache, int* ctas) {
  int dev = 0, sms = 0, per_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  *ctas = dev < kMaxDevices ? cache[dev].load(std::memory_order_relaxed) : 0;
  if (*ctas != 0) return cudaSuccess;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem);
  if (e != cudaSuccess) return e;
  if (per_sm < 1) return cudaErrorInvalidConfiguration;
  *ctas = sms * per_sm;
  if (dev < kMaxDevices) cache[dev].store(*ctas, std::memory_order_relaxed);
  return cudaSuccess;
}

// packed pairs of f32: one instruction for two values
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {  // a * b + c
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Launch with a programmatic dependency on the kernel before it in the stream: the CTAs start
// while that one ends, and wait (pdl_wait, the first thing every kernel here does) until its
// writes are there.  cluster: CTAs of a cluster along x, 0 for none.
template <typename P>
inline cudaError_t launch_dependent(void (*kernel)(P), dim3 grid, int threads, size_t smem, int cluster,
                                    cudaStream_t s, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace rqk
