// paged_plan.cu -- block tables and token maps of the paged K/V cache, built on the GPU
// from the requests' lengths (include/rq.h, rq_paged_plan).
//
// With pages(c) = min(ceil(c / P), W), request b needs pages(c_b + n_b) - pages(c_b) new
// blocks, or gives back pages(c_b) if it has ended.  Three prefix sums over the requests
// (tokens, blocks taken, blocks given back) place everything: taken block x is entry
// head + x of the free ring, given block x goes to entry head + count + x, token t belongs
// to the last request whose first token is <= t.  Every output element is then computed
// from its index alone, by a binary search in the prefix sums in shared memory.
//
// One CTA does the sums and whatever is written from them; many tokens are a second kernel's,
// which finds everything it needs in the first one's outputs (a CTA of 1024 threads writes
// 262144 tokens in 209 us, the two kernels take 8.2 us).
//
// What may alias needs no order of its own: taken entries of the ring are read at [head,
// head + taken) and given ones written at [head + count, head + count + given), apart because
// count + given <= N; table columns are written from pages(c_b) on and read below. Only the
// lengths and the pool's words are read by all and written by some: those writes follow a
// barrier.
#include "paged.cuh"

namespace rqk {
namespace {

constexpr int kPlanMaxBatch = 8192;  // four prefix arrays of this length fit shared memory
constexpr int kPlanMaxTokens = 1 << 30;  // token numbers and a thread's four stay in 32 bits
constexpr int kPlanMaxBlocks = 1 << 30;  // and so do ring entries and a thread's next one
constexpr int kPlanThreads = 1024, kTokenThreads = 256;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanTokens = 4 * kPlanThreads;  // tokens that the first kernel maps itself

struct PlanParams {
  int B, W, P, N, M;
  const int32_t *new_lens, *lens, *pool;
  int32_t *free_ids, *table, *lens_out, *pool_out, *cu, *requests, *positions;
  int64_t* slots;
};

struct Sums {
  long long tok, need, give;
};

__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return {a.tok + b.tok, a.need + b.need, a.give + b.give};
}

__device__ __forceinline__ Sums shfl_up(const Sums& a, int o) {
  return {__shfl_up_sync(0xffffffffu, a.tok, o), __shfl_up_sync(0xffffffffu, a.need, o),
          __shfl_up_sync(0xffffffffu, a.give, o)};
}

__device__ __forceinline__ Sums shfl(const Sums& a, int l) {
  return {__shfl_sync(0xffffffffu, a.tok, l), __shfl_sync(0xffffffffu, a.need, l),
          __shfl_sync(0xffffffffu, a.give, l)};
}

__device__ __forceinline__ int pages_of(int c, const PlanParams& p) {
  const int n = c / p.P + (c % p.P != 0);
  return n < p.W ? n : p.W;
}

// entry i behind entry `from` of the ring of N, both in [0, N] (from < N)
__device__ __forceinline__ int ring_at(int N, int from, int i) {
  const unsigned x = (unsigned)from + (unsigned)i;
  return (int)(x >= (unsigned)N ? x - (unsigned)N : x);
}

// the last b with first[b] <= x, first[0] = 0
__device__ __forceinline__ int last_at_most(const int* first, int B, int x) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Tokens [t0, t0 + 4) of T: request, position and slot, -1 behind the last. cu: first tokens
// [B + 1]; held(b): the length before; block(b, col): the block in column col.
template <typename Held, typename Block>
__device__ __forceinline__ void map_tokens(const PlanParams& p, const int* cu, int t0, int T, bool wide,
                                           Held held, Block block) {
  int req[4], pos[4], b = 0, len = 0, page = -1, id = -1;
  long long slot[4];
  if (t0 < T) {
    b = last_at_most(cu, p.B, t0);
    len = held(b);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + i;
    req[i] = pos[i] = -1;
    slot[i] = -1;
    if (t >= T) continue;
    if (t >= cu[b + 1]) {
      do ++b; while (t >= cu[b + 1]);
      len = held(b);
      page = -1;
    }
    req[i] = b;
    pos[i] = len + (t - cu[b]);
    const int pg = pos[i] / p.P;
    if (pg != page) {
      page = pg;
      id = block(b, len, pg % p.W);
      // a page that a later token of this call takes over, or a block that is none
      const int last = (len + (cu[b + 1] - cu[b]) - 1) / p.P;
      if (last - pg >= p.W || id >= p.N) id = -1;
    }
    if (id >= 0) slot[i] = (long long)id * p.P + (pos[i] - pg * p.P);
  }
  if (wide && t0 + 4 <= p.M) {
    *reinterpret_cast<int4*>(p.requests + t0) = make_int4(req[0], req[1], req[2], req[3]);
    *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    *reinterpret_cast<longlong2*>(p.slots + t0) = make_longlong2(slot[0], slot[1]);
    *reinterpret_cast<longlong2*>(p.slots + t0 + 2) = make_longlong2(slot[2], slot[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (t0 + i < p.M) {
        p.requests[t0 + i] = req[i];
        p.positions[t0 + i] = pos[i];
        p.slots[t0 + i] = slot[i];
      }
  }
}

__device__ __forceinline__ bool wide_maps(const PlanParams& p) {
  return ((reinterpret_cast<uintptr_t>(p.requests) | reinterpret_cast<uintptr_t>(p.positions) |
           reinterpret_cast<uintptr_t>(p.slots)) & 15u) == 0;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p) {
  extern __shared__ int s_mem[];
  int* const s_cu = s_mem;               // [B + 1] first token
  int* const s_take = s_cu + p.B + 1;    // [B] first taken block
  int* const s_give = s_take + p.B;      // [B] first block given back
  int* const s_held = s_give + p.B;      // [B] length before
  __shared__ Sums s_warp[kPlanWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
  pdl_wait();
  pdl_trigger();
  const int head = p.pool[0], count = p.pool[1];
  Sums run{0, 0, 0};
  int bad = head < 0 || head >= p.N || count < 0 || count > p.N;
  for (int base = 0; base < p.B; base += nt) {
    const int b = base + tid;
    Sums own{0, 0, 0};
    int c = 0;
    if (b < p.B) {
      const int n = p.new_lens[b];
      c = p.lens[b];
      if (n < -1 || c < 0 || (n > 0 && c > INT_MAX - n)) {
        bad = 1;
        c = 0;
      } else if (n < 0) {
        own.give = pages_of(c, p);
      } else {
        own.tok = n;
        own.need = pages_of(c + n, p) - pages_of(c, p);
      }
    }
    Sums inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Sums t = shfl_up(inc, o);
      if (lane >= o) inc = inc + t;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    // every warp scans the warps' sums
    Sums w = lane < nt / 32 ? s_warp[lane] : Sums{0, 0, 0};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Sums t = shfl_up(w, o);
      if (lane >= o) w = w + t;
    }
    const Sums all = shfl(w, 31), below = shfl(w, (warp + 31) & 31);
    if (b < p.B) {
      // a sum past the limits fails the call below: the narrowed value is not used then
      const Sums at = run + (warp ? below : Sums{0, 0, 0}) + inc;
      s_cu[b] = (int)(at.tok - own.tok);
      s_take[b] = (int)(at.need - own.need);
      s_give[b] = (int)(at.give - own.give);
      s_held[b] = c;
    }
    run = run + all;
    __syncthreads();
  }
  bad = __syncthreads_or(bad);
  int status = 0;
  if (bad || (long long)count + run.give > p.N) status |= RQ_PAGED_BAD_INPUT;
  if (run.tok > p.M) status |= RQ_PAGED_NO_TOKENS;
  if (run.need > count) status |= RQ_PAGED_NO_BLOCKS;
  const int T = status ? 0 : (int)run.tok;
  const int taken = status ? 0 : (int)run.need, given = status ? 0 : (int)run.give;
  if (tid == 0) s_cu[p.B] = T;
  __syncthreads();

  for (int b = tid; b < p.B; b += nt) {
    const int n = status ? 0 : p.new_lens[b];
    p.lens_out[b] = n < 0 ? 0 : p.lens[b] + n;
    p.cu[b] = status ? 0 : s_cu[b];
  }
  if (tid == 0) {
    p.cu[p.B] = T;
    p.pool_out[0] = status ? head : ring_at(p.N, head, taken);
    p.pool_out[1] = count - taken + given;
    p.pool_out[2] = status;
    p.pool_out[3] = (int)(run.need < INT_MAX ? run.need : INT_MAX);
  }
  for (int x = tid; x < taken; x += nt) {
    const int b = last_at_most(s_take, p.B, x);
    p.table[(size_t)b * p.W + pages_of(s_held[b], p) + (x - s_take[b])] =
        p.free_ids[ring_at(p.N, head, x)];
  }
  const int tail = given ? ring_at(p.N, head, count) : 0;
  for (int x = tid; x < given; x += nt) {
    const int b = last_at_most(s_give, p.B, x);
    p.free_ids[ring_at(p.N, tail, x)] = p.table[(size_t)b * p.W + (x - s_give[b])];
  }
  if (p.M > kPlanTokens) return;  // the token kernel's
  const bool wide = wide_maps(p);
  for (int t0 = tid * 4; t0 < p.M; t0 += nt * 4)
    map_tokens(p, s_cu, t0, T, wide, [&](int b) { return s_held[b]; },
               [&](int b, int len, int col) {
                 const int before = pages_of(len, p);
                 return col < before
                            ? p.table[(size_t)b * p.W + col]
                            : p.free_ids[ring_at(p.N, head, s_take[b] + (col - before))];
               });
}

// The maps of many tokens, from the first kernel's outputs.
__global__ void __launch_bounds__(kTokenThreads) plan_tokens_kernel(const PlanParams p) {
  extern __shared__ int s_cu[];  // [B + 1]
  pdl_wait();
  pdl_trigger();
  for (int b = threadIdx.x; b <= p.B; b += kTokenThreads) s_cu[b] = p.cu[b];
  __syncthreads();
  const int t0 = (blockIdx.x * kTokenThreads + threadIdx.x) * 4;
  if (t0 >= p.M) return;
  map_tokens(p, s_cu, t0, s_cu[p.B], wide_maps(p),
             [&](int b) { return p.lens_out[b] - (s_cu[b + 1] - s_cu[b]); },
             [&](int b, int, int col) { return p.table[(size_t)b * p.W + col]; });
}

__global__ void pool_init_kernel(int n, int32_t* pool, int32_t* free_ids) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) free_ids[i] = i;
  if (i < 4) pool[i] = i == 1 ? n : 0;
}

}  // namespace
}  // namespace rqk

extern "C" rq_status rq_paged_pool_init(int32_t n_blocks, int32_t* pool, int32_t* free_ids,
                                        void* cuda_stream) {
  if (n_blocks < 1 || !pool || !free_ids) return RQ_ERR_ARG;
  if (n_blocks > rqk::kPlanMaxBlocks) return RQ_ERR_UNSUPPORTED;
  const unsigned grid = ((unsigned)n_blocks + 4 + 255) / 256;
  rqk::pool_init_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(cuda_stream)>>>(n_blocks, pool,
                                                                                  free_ids);
  return cudaGetLastError() == cudaSuccess ? RQ_OK : RQ_ERR_CUDA;
}

extern "C" rq_status rq_paged_plan(int32_t batch, int32_t max_blocks, int32_t block_size,
                                   int32_t n_blocks, int32_t max_tokens, const int32_t* new_lens,
                                   const int32_t* lens, const int32_t* pool, int32_t* free_ids,
                                   int32_t* block_table, int32_t* lens_out, int32_t* pool_out,
                                   int32_t* cu_tokens, int32_t* requests, int32_t* positions,
                                   int64_t* slots, void* cuda_stream) {
  using namespace rqk;
  if (batch < 1 || max_blocks < 1 || block_size < 1 || n_blocks < 1 || max_tokens < 1)
    return RQ_ERR_ARG;
  if (batch > kPlanMaxBatch || max_tokens > kPlanMaxTokens || n_blocks > kPlanMaxBlocks)
    return RQ_ERR_UNSUPPORTED;
  if (!new_lens || !lens || !pool || !free_ids || !block_table || !lens_out || !pool_out ||
      !cu_tokens || !requests || !positions || !slots)
    return RQ_ERR_ARG;
  PlanParams p{batch,       max_blocks, block_size, n_blocks,  max_tokens, new_lens,
               lens,        pool,       free_ids,   block_table, lens_out, pool_out,
               cu_tokens,   requests,   positions,  slots};
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  const size_t smem = ((size_t)4 * batch + 1) * sizeof(int);
  // a block has 48 KB unasked, for these sums and what the kernel declares itself (its warps' sums)
  if (smem + kPlanWarps * sizeof(Sums) > 48 * 1024 &&
      cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)((4 * kPlanMaxBatch + 1) * sizeof(int))) != cudaSuccess)
    return RQ_ERR_CUDA;
  // few requests and tokens: fewer warps to wait for one another (64 tokens: 5.6 us, with 1024 threads 6.4)
  const int threads = batch <= 256 && max_tokens <= 1024 ? 256 : kPlanThreads;
  if (launch_dependent(plan_kernel, dim3(1), threads, smem, 0, s, p) != cudaSuccess) return RQ_ERR_CUDA;
  if (max_tokens <= kPlanTokens) return RQ_OK;
  const unsigned grid = (unsigned)(((long long)max_tokens + kTokenThreads * 4 - 1) / (kTokenThreads * 4));
  return launch_dependent(plan_tokens_kernel, dim3(grid), kTokenThreads, ((size_t)batch + 1) * sizeof(int), 0, s,
                          p) == cudaSuccess ? RQ_OK : RQ_ERR_CUDA;
}
