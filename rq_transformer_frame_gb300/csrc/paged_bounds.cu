// paged_bounds.cu -- the smallest and largest key of the blocks that a step's tokens lie in, by
// dimension (include/rq.h, rq_paged_bounds).
//
// A block's bounds over its rows 0 .. o, o the row of the step's last token there: a prompt's keys
// are read once. No atomics and nothing kept between steps: a block that another request had before
// starts anew. A CTA looks at up to 32 tokens, a lane each, and goes through the blocks whose last token
// is among them; a thread takes 16 bytes of a block's rows, neighbouring threads neighbouring pieces,
// eight rows in flight. HBM-bound for prompts, latency for steps (a token a CTA then).
#include <algorithm>

#include "paged.cuh"

namespace rqk {
namespace {

struct BoundsParams {
  rq_paged_kv kv;
  void* bounds;
  int tokens;
  const int32_t* positions;
  const int64_t* slots;
  int chunk;  // tokens of a CTA
};

constexpr int kThreads = 128;

// Smallest and largest of 16 bytes of elements; a NaN stays.
template <typename T>
struct Range;
template <>
struct Range<float> {
  static __device__ __forceinline__ uint32_t low(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.f32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ uint32_t high(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.f32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
};
template <>
struct Range<uint16_t> {
  static __device__ __forceinline__ uint32_t low(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ uint32_t high(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) bounds_kernel(const __grid_constant__ BoundsParams p) {
  constexpr int E = 16 / (int)sizeof(T);  // elements of a piece
  pdl_wait();
  pdl_trigger();
  const long long P = p.kv.block_size, slots = P * p.kv.n_blocks;
  auto slot_of = [&](int t) {  // -1: the token is not stored
    if (t >= p.tokens || p.positions[t] < 0) return -1ll;
    const long long s = p.slots[t];
    return s < slots ? s : -1ll;
  };
  const int lane = threadIdx.x % 32, pieces = p.kv.head_dim / E, width = p.kv.heads * pieces;
  const long long t = (long long)blockIdx.x * p.chunk + lane;
  const long long slot = lane < p.chunk && t < p.tokens ? slot_of((int)t) : -1;
  const long long block = slot < 0 ? -1 : slot / P;
  // the token behind is the next lane's, but for the last lane
  long long behind = __shfl_down_sync(0xffffffffu, block, 1);
  if (lane == p.chunk - 1) {
    const long long s = slot_of((int)min(t + 1, (long long)p.tokens));
    behind = s < 0 ? -1 : s / P;
  }
  uint32_t last = __ballot_sync(0xffffffffu, block >= 0 && behind != block);
  while (last) {
    const int from = __ffs(last) - 1;
    last &= last - 1;
    const long long n = __shfl_sync(0xffffffffu, block, from);
    const int rows = (int)(__shfl_sync(0xffffffffu, slot, from) - n * P) + 1;
    for (int i = blockIdx.y * kThreads + threadIdx.x; i < width; i += gridDim.y * kThreads) {
      const int h = i / pieces, c = i % pieces;
      const T* k = static_cast<const T*>(p.kv.k) + n * p.kv.block_stride + h * p.kv.head_stride + c * E;
      uint4 lo = *reinterpret_cast<const uint4*>(k), hi = lo;
      auto take = [&](const uint4& x) {
        lo.x = Range<T>::low(lo.x, x.x), lo.y = Range<T>::low(lo.y, x.y);
        lo.z = Range<T>::low(lo.z, x.z), lo.w = Range<T>::low(lo.w, x.w);
        hi.x = Range<T>::high(hi.x, x.x), hi.y = Range<T>::high(hi.y, x.y);
        hi.z = Range<T>::high(hi.z, x.z), hi.w = Range<T>::high(hi.w, x.w);
      };
      int r = 1;
      for (; r + 8 <= rows; r += 8) {
        uint4 x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = *reinterpret_cast<const uint4*>(k + (r + j) * p.kv.row_stride);
#pragma unroll
        for (int j = 0; j < 8; ++j) take(x[j]);
      }
      if (r < rows) {  // the rest: the last row stands in for those that are not there
        uint4 x[7];
#pragma unroll
        for (int j = 0; j < 7; ++j)
          x[j] = *reinterpret_cast<const uint4*>(k + min(r + j, rows - 1) * p.kv.row_stride);
#pragma unroll
        for (int j = 0; j < 7; ++j) take(x[j]);
      }
      T* out = static_cast<T*>(p.bounds) + (n * p.kv.heads + h) * 2 * p.kv.head_dim + c * E;
      *reinterpret_cast<uint4*>(out) = lo;
      *reinterpret_cast<uint4*>(out + p.kv.head_dim) = hi;
    }
  }
}

}  // namespace
}  // namespace rqk

extern "C" rq_status rq_paged_bounds(const rq_paged_kv* kv, void* bounds, int32_t tokens,
                                     const int32_t* positions, const int64_t* slots,
                                     void* cuda_stream) {
  using namespace rqk;
  const rq_status st = paged_kv_check(kv);
  if (st != RQ_OK) return st;
  if (tokens < 0) return RQ_ERR_ARG;
  if (tokens > 1 << 30 || kv->heads > 1 << 23) return RQ_ERR_UNSUPPORTED;
  if (tokens == 0) return RQ_OK;
  if (!bounds || !aligned16(bounds) || !positions || !slots) return RQ_ERR_ARG;
  // a warp's tokens where there are plenty, one where CTAs are few
  const int chunk = std::min(std::max(tokens / (8 * std::max(sm_count(), 1)), 1), 32);
  BoundsParams p{*kv, bounds, tokens, positions, slots, chunk};
  const int pieces = kv->heads * (kv->head_dim * (kv->dtype == RQ_BF16 ? 2 : 4) / 16);
  const dim3 grid((unsigned)((tokens + chunk - 1) / chunk), (unsigned)std::min((pieces + kThreads - 1) / kThreads, 1024), 1);
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = kv->dtype == RQ_BF16
                            ? launch_dependent(bounds_kernel<uint16_t>, grid, kThreads, 0, 0, s, p)
                            : launch_dependent(bounds_kernel<float>, grid, kThreads, 0, 0, s, p);
  return e == cudaSuccess ? RQ_OK : RQ_ERR_CUDA;
}
