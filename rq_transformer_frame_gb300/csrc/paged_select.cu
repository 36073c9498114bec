// paged_select.cu -- the pages that each row and K/V head attends to, by a bound of their scores
// (include/rq.h, rq_paged_select).
//
// With u+ = sum over the K/V head's queries of max(q, 0) and u- the same of min(q, 0), a page's
// score is u+ . (largest key) + u- . (smallest key): one product of 2 head_dim terms a page, whatever
// the number of queries. Two kernels: the scores in f32 (the bounds are read once: HBM-bound), then
// for each (row, K/V head) the best ones and the list.
//
// Which pages are taken must not hang on the order of f32 sums, so the second kernel takes only what
// those decide for sure. An f32 score is off by at most
//   E = eps (32 + 2 G) sum_d (|u+_d| + |u-_d|) * max |bound|,  eps = 2^-24
// (sums of 8 terms in a lane and 5 levels of lanes, the G queries' sums before, and half as
// much again), so with t the k-th largest f32 score, a score above t + 2 E is among the k
// best and one below t - 2 E is not; what lies between is scored again in f64 and ordered by that.
// With random keys this is the border page itself and in one row of twenty a second one.
#include "paged.cuh"

namespace rqk {
namespace {

constexpr int kScoreWarps = 8, kSelectThreads = 512, kSelectWarps = kSelectThreads / 32;
constexpr uint32_t kNone = 0u, kUnsure = 0xffffffffu;  // keys: no candidate; a score that f32 does not hold

struct SelectParams {
  const void* bounds;
  const int32_t *table, *requests, *positions;
  const void* q;
  int32_t* pages;
  uint32_t* keys;       // [rows][heads][stride] order of the f32 scores
  unsigned long long* fine;  // the same of the f64 scores, where they are wanted
  float* most;          // [rows][heads][chunks] largest |bound|
  int rows, heads, kv_heads, batch, W, n_blocks, block_size, top, first, last;
  int stride, chunks, chunk;  // pages of a row's keys, chunks of a row, pages of a chunk
};

struct Live {
  int b, lo, n;  // request, lowest live page and their number (0: none)
  bool padding;
};

__device__ __forceinline__ Live live_of(const SelectParams& p, int row) {
  Live x{p.requests ? p.requests[row] : row, 0, 0, false};
  x.padding = x.b < 0 || x.b >= p.batch;
  const int pos = p.positions[row];
  if (x.padding || pos < 0) return x;
  const int newest = pos / p.block_size;
  x.lo = max(0, newest - p.W + 1);
  x.n = newest - x.lo + 1;
  return x;
}

// the table's block of a page, or -1
__device__ __forceinline__ int block_of(const SelectParams& p, const Live& x, int page) {
  const int id = p.table[(size_t)x.b * p.W + (page < p.W ? page : page % p.W)];
  return id >= 0 && id < p.n_blocks ? id : -1;
}

__device__ __forceinline__ float widen(const float* p) { return *p; }
__device__ __forceinline__ float widen(const uint16_t* p) { return bf16lo(*p); }

// f32 bits in the order of the values
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);  // -0 as +0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}
__device__ __forceinline__ unsigned long long order_of(double v) {
  if (!(v == v)) v = -__longlong_as_double(0x7ff0000000000000ll);
  const unsigned long long u = (unsigned long long)__double_as_longlong(v + 0.0);
  return u >> 63 ? ~u : u | 1ull << 63;
}

// ---------------------------------------------------------------- scores
// A warp takes 32 pages of one K/V head at a time. A page's 2 HD values are HD / 4 lanes' (8 each,
// 16 bytes of bf16 or twice 16 of f32), so a warp reads 128 / HD pages in a step; the sums of eight
// steps are reduced together, halving the values with the lanes.
template <typename T, typename QT, int HD>
__global__ void __launch_bounds__(kScoreWarps * 32) score_kernel(const __grid_constant__ SelectParams p) {
  constexpr int L = HD / 4;             // lanes of a page
  constexpr bool kF32 = sizeof(T) == 4;
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int i = lane % L, sub = lane / L;
  const int G = p.heads / p.kv_heads, parts = p.chunk / 32;
  const int page0 = blockIdx.x * p.chunk;
  for (int row = blockIdx.y; row < p.rows; row += gridDim.y) {
  const Live x = live_of(p, row);
  if (x.n <= p.top || page0 >= x.n) continue;  // up to `top` pages all are taken
  for (int item = warp; item < p.kv_heads; item += kScoreWarps) {
    const int h = item;
    // this lane's 8 values of (u-, u+)
    float u[8] = {};
    for (int g = 0; g < G; ++g) {
      const QT* q = static_cast<const QT*>(p.q) + ((size_t)row * p.heads + (size_t)h * G + g) * HD;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const bool up = kF32 ? e >= 4 : i >= L / 2;
        const int d = kF32 ? i * 4 + (e & 3) : (i % (L / 2)) * 8 + e;
        const float y = widen(q + d);
        u[e] += up ? fmaxf(y, 0.f) : fminf(y, 0.f);
      }
    }
    float most = 0.f;
    uint32_t* keys = p.keys + ((size_t)row * p.kv_heads + h) * p.stride;
    for (int part = 0; part < parts; ++part) {
      const int first = page0 + part * 32;
      if (first >= x.n) break;
      const int mine = first + lane < x.n ? block_of(p, x, x.lo + first + lane) : -1;
      float score = 0.f;
#pragma unroll 1
      for (int g = 0; g < L / 8; ++g) {
        float s[8];
        uint4 a[8], b[kF32 ? 8 : 1];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int id = __shfl_sync(0xffffffffu, mine, sub * L + g * 8 + j);
          const T* at = static_cast<const T*>(p.bounds) + ((size_t)max(id, 0) * p.kv_heads + h) * 2 * HD;
          a[j] = id >= 0 ? *reinterpret_cast<const uint4*>(at + i * (kF32 ? 4 : 8)) : make_uint4(0, 0, 0, 0);
          if constexpr (kF32)
            b[j] = id >= 0 ? *reinterpret_cast<const uint4*>(at + HD + i * 4) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float v[8];
          if constexpr (kF32) {
            v[0] = __uint_as_float(a[j].x), v[1] = __uint_as_float(a[j].y);
            v[2] = __uint_as_float(a[j].z), v[3] = __uint_as_float(a[j].w);
            v[4] = __uint_as_float(b[j].x), v[5] = __uint_as_float(b[j].y);
            v[6] = __uint_as_float(b[j].z), v[7] = __uint_as_float(b[j].w);
          } else {
            v[0] = bf16lo(a[j].x), v[1] = bf16hi(a[j].x), v[2] = bf16lo(a[j].y), v[3] = bf16hi(a[j].y);
            v[4] = bf16lo(a[j].z), v[5] = bf16hi(a[j].z), v[6] = bf16lo(a[j].w), v[7] = bf16hi(a[j].w);
          }
          s[j] = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            s[j] = fmaf(v[e], u[e], s[j]);
            const float m = fabsf(v[e]);
            if (m < 3.4028235e38f) most = fmaxf(most, m);  // pages of others are looked at in f64
          }
        }
        // lanes i with i % 8 = j end with step j's sum
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float keep = lane & 4 ? s[j + 4] : s[j], give = lane & 4 ? s[j] : s[j + 4];
          s[j] = keep + __shfl_xor_sync(0xffffffffu, give, 4);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float keep = lane & 2 ? s[j + 2] : s[j], give = lane & 2 ? s[j] : s[j + 2];
          s[j] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
        }
        {
          const float keep = lane & 1 ? s[1] : s[0], give = lane & 1 ? s[0] : s[1];
          s[0] = keep + __shfl_xor_sync(0xffffffffu, give, 1);
        }
#pragma unroll
        for (int o = 8; o < L; o <<= 1) s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
        if (i / 8 == g) score = s[0];
      }
      if (first + lane < x.n) {
        const bool finite = fabsf(score) <= 3.4028235e38f;
        keys[first + lane] = mine < 0 ? kNone : finite ? order_of(score) : kUnsure;
      }
    }
    most = warp_max(most);
    if (lane == 0) p.most[((size_t)row * p.kv_heads + h) * p.chunks + blockIdx.x] = most;
  }
  }
}

// ---------------------------------------------------------------- the best and the list
struct SelectShared {
  int hist[256];
  int warp_a[kSelectWarps], warp_b[kSelectWarps];
  float f[kSelectWarps];
  int digit, left;
};

// sums over the CTA of two counts, the same in every thread
__device__ __forceinline__ int2 block_sum(SelectShared& s, int a, int b) {
  a = __reduce_add_sync(0xffffffffu, a);
  b = __reduce_add_sync(0xffffffffu, b);
  __syncthreads();
  if (threadIdx.x % 32 == 0) s.warp_a[threadIdx.x / 32] = a, s.warp_b[threadIdx.x / 32] = b;
  __syncthreads();
  int2 r = make_int2(0, 0);
  for (int w = 0; w < kSelectWarps; ++w) r.x += s.warp_a[w], r.y += s.warp_b[w];
  return r;
}

// The k-th largest of the keys key(0 .. n-1), k >= 1 and at most the number of those above 0 (zeros
// do not count); `left`: how many of the keys equal to it are among the k. Digits of 8 bits
// from the top, a histogram each.
template <typename Key, typename F>
__device__ Key kth_largest(SelectShared& s, int n, int k, F key, int* left) {
  Key prefix = 0;
  for (int shift = (int)sizeof(Key) * 8 - 8; shift >= 0; shift -= 8) {
    __syncthreads();
    if (threadIdx.x < 256) s.hist[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kSelectThreads) {
      const Key x = key(i);
      if (x != 0 && ((x ^ prefix) >> shift) < 256) atomicAdd(&s.hist[(int)(x >> shift) & 255], 1);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      // bins from the top, 8 a lane
      int own = 0;
      for (int j = 0; j < 8; ++j) own += s.hist[255 - (threadIdx.x * 8 + j)];
      int inc = own;
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if ((int)threadIdx.x >= o) inc += y;
      }
      int before = inc - own;
      if (before < k && k <= inc) {
        for (int j = 0; j < 8; ++j) {
          const int d = 255 - (threadIdx.x * 8 + j), c = s.hist[d];
          if (before + c >= k) {
            s.digit = d;
            s.left = k - before;
            break;
          }
          before += c;
        }
      }
    }
    __syncthreads();
    prefix |= (Key)s.digit << shift;
    k = s.left;
  }
  *left = k;
  return prefix;
}

template <typename T, typename QT>
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const __grid_constant__ SelectParams p, int HD) {
  __shared__ SelectShared s;
  pdl_wait();
  pdl_trigger();
  const int pair = blockIdx.x, row = pair / p.kv_heads, h = pair % p.kv_heads;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const Live x = live_of(p, row);
  if (x.padding) return;
  int32_t* out = p.pages + (size_t)pair * p.top;
  const int G = p.heads / p.kv_heads, want = p.top - p.first - p.last;
  const uint32_t* keys = p.keys + (size_t)pair * p.stride;
  unsigned long long* fine = p.fine + (size_t)pair * p.stride;
  auto always = [&](int i) { return i < p.first || i >= x.n - p.last; };
  // a page's key among those the score decides about
  auto key = [&](int i) { return always(i) ? kNone : keys[i]; };
  // what is taken beside the pages that always are: keys above `sure`; of those in [low, sure]
  // fine keys above `border`, and the first `left` that equal it
  uint32_t low = 1, sure = 0;
  unsigned long long border = 0;
  int left = 0;
  bool all = x.n <= p.top;  // no scores then
  if (!all) {
    int a = 0, b = 0;
    for (int i = tid; i < x.n; i += kSelectThreads) {
      const uint32_t v = key(i);
      a += v != kNone;
      b += v == kUnsure;
    }
    const int2 n = block_sum(s, a, b);
    if (n.x > want && want > 0) {
      // the error of the f32 scores
      float most = 0.f, sum = 0.f;
      for (int i = tid; i < (x.n + p.chunk - 1) / p.chunk; i += kSelectThreads)
        most = fmaxf(most, p.most[(size_t)pair * p.chunks + i]);
      const QT* q = static_cast<const QT*>(p.q) + ((size_t)row * p.heads + (size_t)h * G) * HD;
      for (int i = tid; i < G * HD; i += kSelectThreads) sum += fabsf(widen(q + i));
      most = warp_max(most);
      sum = warp_sum(sum);
      __syncthreads();
      if (lane == 0) s.f[warp] = most, s.warp_a[warp] = __float_as_int(sum);
      __syncthreads();
      sum = 0.f;
      for (int w = 0; w < kSelectWarps; ++w) most = fmaxf(most, s.f[w]), sum += __int_as_float(s.warp_a[w]);
      const float E = (32.f + 2.f * G) * 5.9604645e-8f * sum * most + 1e-36f;
      sure = kUnsure;
      if (n.y == 0 && E < 1e38f) {
        int same;
        const float t = value_of(kth_largest<uint32_t>(s, x.n, want, key, &same));
        low = order_of(t - 2.f * E);
        sure = order_of(t + 2.f * E);
      }
      a = b = 0;
      for (int i = tid; i < x.n; i += kSelectThreads) {
        const uint32_t v = key(i);
        a += v > sure;
        b += v >= low && v <= sure;
      }
      const int2 m = block_sum(s, a, b);
      border = 0, left = 0;
      if (m.x + m.y > want) {
        // the others again in f64, a warp each
        for (int i = warp; i < x.n; i += kSelectWarps) {
          const uint32_t v = key(i);
          if (v < low || v > sure) continue;
          const T* at = static_cast<const T*>(p.bounds) +
                        ((size_t)block_of(p, x, x.lo + i) * p.kv_heads + h) * 2 * HD;
          double sum = 0.0;
          for (int d = lane; d < HD; d += 32) {
            double up = 0.0, down = 0.0;
            for (int g = 0; g < G; ++g) {
              const double y = (double)widen(q + (size_t)g * HD + d);
              // a NaN query stays in both
              up += y < 0.0 ? 0.0 : y;
              down += y > 0.0 ? 0.0 : y;
            }
            sum += up * (double)widen(at + HD + d) + down * (double)widen(at + d);
          }
          for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          if (lane == 0) fine[i] = order_of(sum);
        }
        __syncthreads();
        border = kth_largest<unsigned long long>(
            s, x.n, want - m.x,
            [&](int i) {
              const uint32_t v = key(i);
              return v >= low && v <= sure ? fine[i] : 0ull;
            },
            &left);
      } else {
        sure = low - 1;  // all of them
      }
    } else if (want == 0) {
      low = sure = kUnsure;
      border = ~0ull;  // none
    }
  }
  // ---- the list, page after page
  int done = 0, ties = 0;  // pages written, equal ones met
  const bool fine_used = low <= sure;
  for (int i0 = 0; i0 < x.n; i0 += kSelectThreads) {
    const int i = i0 + tid;
    int take = 0, tie = 0;
    if (i < x.n) {
      if (always(i)) {
        take = 1;
      } else if (all) {
        take = block_of(p, x, x.lo + i) >= 0;
      } else {
        const uint32_t v = keys[i];
        if (v == kNone || want == 0) {
        } else if (!fine_used || v > sure) {
          take = v > sure;
        } else if (v >= low) {
          const unsigned long long f = fine[i];
          take = f > border;
          tie = f == border;
        }
      }
    }
    // equal ones before this page, then pages before it
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t tied = __ballot_sync(0xffffffffu, tie);
    __syncthreads();
    if (lane == 0) s.warp_a[warp] = __popc(tied);
    __syncthreads();
    int before = ties + __popc(tied & below);
    for (int w = 0; w < kSelectWarps; ++w) {
      if (w < warp) before += s.warp_a[w];
      ties += s.warp_a[w];
    }
    if (tie && before < left) take = 1;
    const uint32_t taken = __ballot_sync(0xffffffffu, take);
    if (lane == 0) s.warp_b[warp] = __popc(taken);
    __syncthreads();
    int at = done + __popc(taken & below);
    for (int w = 0; w < kSelectWarps; ++w) {
      if (w < warp) at += s.warp_b[w];
      done += s.warp_b[w];
    }
    if (take && at < p.top) out[at] = x.lo + i;
  }
  for (int i = done + tid; i < p.top; i += kSelectThreads) out[i] = -1;
}

struct Layout {
  int stride, chunk, chunks;
  size_t keys, fine, most, bytes;
};

// chunks: two CTAs an SM at least if the rows are few
inline Layout layout_of(int rows, int kv_heads, int W) {
  Layout x;
  x.stride = (W + 3) & ~3;
  x.chunk = 32;
  x.chunks = (W + x.chunk - 1) / x.chunk;
  const size_t n = (size_t)rows * kv_heads;
  auto up = [](size_t b) { return (b + 255) & ~(size_t)255; };
  x.keys = up(n * x.stride * sizeof(uint32_t));
  x.fine = up(n * x.stride * sizeof(unsigned long long));
  x.most = up(n * x.chunks * sizeof(float));
  x.bytes = x.keys + x.fine + x.most;
  return x;
}

template <typename T, typename QT>
cudaError_t launch(const SelectParams& p, int hd, cudaStream_t s) {
  const dim3 grid((unsigned)p.chunks, (unsigned)(p.rows < 65535 ? p.rows : 65535), 1);
  auto* scores = hd == 32 ? score_kernel<T, QT, 32> : hd == 64 ? score_kernel<T, QT, 64> : score_kernel<T, QT, 128>;
  if (p.W > p.top && p.top > p.first + p.last) {  // some row may have to choose
    const cudaError_t e = launch_dependent(scores, grid, kScoreWarps * 32, 0, 0, s, p);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.rows * p.kv_heads), 1, 1);
  cfg.blockDim = dim3(kSelectThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, select_kernel<T, QT>, p, hd);
}

rq_status check(const rq_paged_kv* kv, int32_t rows, int32_t max_blocks) {
  const rq_status st = paged_kv_check(kv);
  if (st != RQ_OK) return st;
  if (rows < 0 || max_blocks < 1) return RQ_ERR_ARG;
  if (max_blocks > 1 << 30 || kv->heads > 1 << 23 || (long long)rows * kv->heads > INT_MAX) return RQ_ERR_UNSUPPORTED;
  if ((double)rows * kv->heads * max_blocks > 1099511627776.0) return RQ_ERR_UNSUPPORTED;
  return RQ_OK;
}

}  // namespace
}  // namespace rqk

extern "C" size_t rq_paged_select_workspace_size(const rq_paged_kv* kv, int32_t rows, int32_t max_blocks) {
  using namespace rqk;
  return check(kv, rows, max_blocks) == RQ_OK ? layout_of(rows, kv->heads, max_blocks).bytes : 0;
}

extern "C" rq_status rq_paged_select(const rq_paged_kv* kv, const void* bounds, int32_t rows,
                                     int32_t heads, int32_t batch, int32_t max_blocks,
                                     const int32_t* block_table, const int32_t* requests,
                                     const int32_t* positions, int32_t top, int32_t first,
                                     int32_t last, int32_t q_dtype, const void* q, int32_t* pages,
                                     void* workspace, size_t workspace_bytes, void* cuda_stream) {
  using namespace rqk;
  const rq_status st = check(kv, rows, max_blocks);
  if (st != RQ_OK) return st;
  if (heads < 1 || heads % kv->heads != 0 || batch < 1 || first < 0 || last < 1 || top < 1 ||
      (long long)first + last > top)
    return RQ_ERR_ARG;
  if (q_dtype != RQ_F32 && q_dtype != RQ_BF16) return RQ_ERR_ARG;
  if (rows > 1 << 30 || heads > 1 << 23 || (long long)rows * heads > INT_MAX) return RQ_ERR_UNSUPPORTED;
  if (rows == 0) return RQ_OK;
  if (!requests && rows > batch) return RQ_ERR_ARG;
  if (!bounds || !block_table || !positions || !q || !pages || !workspace) return RQ_ERR_ARG;
  if (!aligned16(bounds) || !aligned16(q) || !aligned16(workspace)) return RQ_ERR_ARG;
  const Layout x = layout_of(rows, kv->heads, max_blocks);
  if (workspace_bytes < x.bytes) return RQ_ERR_ARG;
  char* ws = static_cast<char*>(workspace);
  SelectParams p{};
  p.bounds = bounds;
  p.table = block_table;
  p.requests = requests;
  p.positions = positions;
  p.q = q;
  p.pages = pages;
  p.keys = reinterpret_cast<uint32_t*>(ws);
  p.fine = reinterpret_cast<unsigned long long*>(ws + x.keys);
  p.most = reinterpret_cast<float*>(ws + x.keys + x.fine);
  p.rows = rows;
  p.heads = heads;
  p.kv_heads = kv->heads;
  p.batch = batch;
  p.W = max_blocks;
  p.n_blocks = kv->n_blocks;
  p.block_size = kv->block_size;
  p.top = top;
  p.first = first;
  p.last = last;
  p.stride = x.stride;
  p.chunk = x.chunk;
  p.chunks = x.chunks;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  const bool b = kv->dtype == RQ_BF16, qb = q_dtype == RQ_BF16;
  const cudaError_t e = b ? (qb ? launch<uint16_t, uint16_t>(p, kv->head_dim, s) : launch<uint16_t, float>(p, kv->head_dim, s))
                          : (qb ? launch<float, uint16_t>(p, kv->head_dim, s) : launch<float, float>(p, kv->head_dim, s));
  return e == cudaSuccess ? RQ_OK : RQ_ERR_CUDA;
}
