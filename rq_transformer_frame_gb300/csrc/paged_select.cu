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
//   E = eps (16 + G) sum_d (|u+_d| + |u-_d|) * max |bound|,  eps = 2^-24
// (8 terms one after another in a lane, 5 levels of lanes, and the G queries' sums before), so with t the
// k-th largest f32 score, a score above t + 2 E is among the k best and one below t - 2 E is not; what
// lies between is scored again in f64 and ordered by that. With random keys this is the border page
// itself and in one row of ten a second one.
#include <algorithm>
#include <climits>

#include "paged.cuh"

namespace rqk {
namespace {

constexpr int kScoreWarps = 8;
constexpr int kChunk = 32;  // pages of a warp
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
  int stride, chunks, span;  // pages of a row's keys, chunks of kChunk of a row, those of a warp
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
// eight values, or TWICE four
template <bool TWICE>
__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = TWICE ? a : reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <bool TWICE>
__device__ __forceinline__ void load8(const uint16_t* p, float* v) {
  const uint2 a = reinterpret_cast<const uint2*>(p)[0], b = TWICE ? a : reinterpret_cast<const uint2*>(p)[1];
  v[0] = bf16lo(a.x), v[1] = bf16hi(a.x), v[2] = bf16lo(a.y), v[3] = bf16hi(a.y);
  v[4] = bf16lo(b.x), v[5] = bf16hi(b.x), v[6] = bf16lo(b.y), v[7] = bf16hi(b.y);
}

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
// A warp takes a few times 32 pages of one K/V head. A page's 2 HD values are HD / 4 lanes' (8 each, 16
// bytes of bf16 or twice 16 of f32), so a warp reads 128 / HD pages in a step; the sums of eight
// steps are reduced together, halving the values with the lanes, while the next eight are on their way.
template <typename T, typename QT, int HD>
__global__ void __launch_bounds__(kScoreWarps * 32, 2) score_kernel(const __grid_constant__ SelectParams p) {
  constexpr int L = HD / 4;  // lanes of a page
  constexpr bool kF32 = sizeof(T) == 4;
  constexpr int N = kF32 ? 2 : 1;  // 16-byte pieces of a lane
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int i = lane % L, sub = lane / L;
  const int G = p.heads / p.kv_heads;
  constexpr int GP = L / 8;  // groups of eight steps of a chunk
  for (int row = blockIdx.y; row < p.rows; row += gridDim.y) {
    const Live x = live_of(p, row);
    if (x.n <= p.top) continue;  // all of them are taken
    // the CTA's items: p.span chunks of a K/V head each, K/V heads first
    const int live = (x.n + kChunk - 1) / kChunk, runs = (live + p.span - 1) / p.span;
    const long long items = (long long)runs * p.kv_heads;
    for (long long item = (long long)blockIdx.x * kScoreWarps + warp; item < items; item += (long long)gridDim.x * kScoreWarps) {
      const int h = (int)(item % p.kv_heads), chunk0 = (int)(item / p.kv_heads) * p.span;
      const int total = min(p.span, live - chunk0) * GP;
      auto ids_of = [&](int chunk) {
        const int at = chunk * kChunk + lane;
        return at < x.n ? block_of(p, x, x.lo + at) : -1;
      };
      // what is read for a page without a block: another's bounds, so that loads hang on nothing
      auto there = [&](int ids) {
        const uint32_t some = __ballot_sync(0xffffffffu, ids >= 0);
        const int other = __shfl_sync(0xffffffffu, ids, some ? __ffs(some) - 1 : 0);
        return ids >= 0 ? ids : max(other, 0);
      };
      int mine = ids_of(chunk0), next = ids_of(chunk0 + 1), chunk = chunk0;
      int at_mine = there(mine), at_next = there(next);
      const char* const base = static_cast<const char*>(p.bounds) + (size_t)h * 2 * HD * sizeof(T) + i * 16;
      const uint32_t page_bytes = p.kv_heads * 2 * HD * (uint32_t)sizeof(T);
      uint4 a[8][N], b[kF32 ? 1 : 8][N];
      auto load = [&](int ids, int g, auto& v) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int id = __shfl_sync(0xffffffffu, ids, sub * L + g * 8 + j);
          const char* at = base + (size_t)id * page_bytes;
#pragma unroll
          for (int e = 0; e < N; ++e) v[j][e] = *reinterpret_cast<const uint4*>(at + e * HD * sizeof(T));
        }
      };
      load(at_mine, 0, a);
      // this lane's 8 values of (u-, u+)
      float u[8] = {};
      for (int g = 0; g < G; ++g) {
        const QT* q = static_cast<const QT*>(p.q) + ((size_t)row * p.heads + (size_t)h * G + g) * HD;
        float y[8];
        load8<kF32>(q + (kF32 ? i * 4 : (i % (L / 2)) * 8), y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool up = kF32 ? e >= 4 : i >= L / 2;
          u[e] += up ? fmaxf(y[e], 0.f) : fminf(y[e], 0.f);
        }
      }
      float most = 0.f, score = 0.f;
      const size_t pair = (size_t)row * p.kv_heads + h;
      auto reduce = [&](int g, const auto& r) {
        float s[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float v[8];
          if constexpr (kF32) {
            v[0] = __uint_as_float(r[j][0].x), v[1] = __uint_as_float(r[j][0].y);
            v[2] = __uint_as_float(r[j][0].z), v[3] = __uint_as_float(r[j][0].w);
            v[4] = __uint_as_float(r[j][N - 1].x), v[5] = __uint_as_float(r[j][N - 1].y);
            v[6] = __uint_as_float(r[j][N - 1].z), v[7] = __uint_as_float(r[j][N - 1].w);
          } else {
            v[0] = bf16lo(r[j][0].x), v[1] = bf16hi(r[j][0].x), v[2] = bf16lo(r[j][0].y), v[3] = bf16hi(r[j][0].y);
            v[4] = bf16lo(r[j][0].z), v[5] = bf16hi(r[j][0].z), v[6] = bf16lo(r[j][0].w), v[7] = bf16hi(r[j][0].w);
          }
          s[j] = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            s[j] = fmaf(v[e], u[e], s[j]);
            most = fmaxf(most, fabsf(v[e]));
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
        if (g < GP - 1) return;
        // the chunk's last: out with it
        const int at = chunk * kChunk + lane;
        if (at < x.n) {
          const bool finite = fabsf(score) <= 3.4028235e38f;
          p.keys[pair * p.stride + at] = mine < 0 ? kNone : finite ? order_of(score) : kUnsure;
        }
        const float largest = warp_max(most);
        const bool any = __any_sync(0xffffffffu, mine >= 0);
        if (lane == 0) p.most[pair * p.chunks + chunk] = any ? largest : 0.f;
        ++chunk;
        mine = next;
        at_mine = at_next;
        next = ids_of(chunk + 1);
        at_next = there(next);
        most = 0.f;
      };
      // (twice the f32 values do not fit the registers)
      if constexpr (kF32) {
#pragma unroll 1
        for (int k = 0; k < total; ++k) {
          if (k > 0) load(at_mine, k % GP, a);
          reduce(k % GP, a);
        }
      } else {
#pragma unroll 1
        for (int k = 0; k < total; k += 2) {
          if (k + 1 < total) load(k % GP == GP - 1 ? at_next : at_mine, (k + 1) % GP, b);
          reduce(k % GP, a);
          if (k + 1 >= total) break;
          if (k + 2 < total) load((k + 1) % GP == GP - 1 ? at_next : at_mine, (k + 2) % GP, a);
          reduce((k + 1) % GP, b);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- the best and the list
// A CTA of NT threads takes a (row, K/V head); a thread takes a run of its pages. All of it is latency:
// a pass over the keys for their range, one for a histogram over that, one for the keys of the bin that
// holds the k-th largest (the f32 scores of random keys leave some dozens there, sorted out among
// themselves), one that counts what is taken and one that writes it.
constexpr int kBins = 1024, kFew = 1024;

template <int NT>
struct SelectShared {
  int hist[kBins + kBins / 32];  // bin i at i + i / 32: a lane's bins in a bank of their own
  uint32_t few[kFew];       // keys, or pages
  unsigned long long fine[kFew];
  int warp_a[NT / 32], warp_b[NT / 32];
  float warp_f[NT / 32], warp_g[NT / 32];
  uint32_t warp_u[NT / 32], warp_v[NT / 32];
  int bin, above, n_few;
  uint32_t kth;
  unsigned long long border;
};

__device__ __forceinline__ int place(int bin) { return bin + bin / 32; }

// both sums over the CTA, the same in every thread
template <int NT>
__device__ __forceinline__ int2 block_sum(SelectShared<NT>& s, int a, int b) {
  a = __reduce_add_sync(0xffffffffu, a);
  b = __reduce_add_sync(0xffffffffu, b);
  __syncthreads();
  if (threadIdx.x % 32 == 0) s.warp_a[threadIdx.x / 32] = a, s.warp_b[threadIdx.x / 32] = b;
  __syncthreads();
  const int lane = threadIdx.x % 32;
  return make_int2(__reduce_add_sync(0xffffffffu, lane < NT / 32 ? s.warp_a[lane] : 0),
                   __reduce_add_sync(0xffffffffu, lane < NT / 32 ? s.warp_b[lane] : 0));
}
// the sum of the threads' counts before this one, and of all
template <int NT>
__device__ __forceinline__ int2 block_scan(SelectShared<NT>& s, int a) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int inc = a;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();
  if (lane == 31) s.warp_a[warp] = inc;
  __syncthreads();
  const int w = lane < NT / 32 ? s.warp_a[lane] : 0;
  return make_int2(inc - a + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0), __reduce_add_sync(0xffffffffu, w));
}

// The bin of s.hist from the top in which the k-th entry lies, and the number above it, by the first warp.
template <int NT>
__device__ __forceinline__ void find_bin(SelectShared<NT>& s, int k) {
  if (threadIdx.x < 32) {
    constexpr int B = kBins / 32;  // bins of a lane, from the top
    const int top = kBins - 1 - threadIdx.x * B;
    int own = 0;
#pragma unroll 8
    for (int j = 0; j < B; ++j) own += s.hist[place(top - j)];
    int inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if ((int)threadIdx.x >= o) inc += y;
    }
    int before = inc - own;
    if (before < k && k <= inc) {
      for (int j = 0; j < B; ++j) {
        const int c = s.hist[place(top - j)];
        if (before + c >= k) {
          s.bin = top - j;
          s.above = before;
          break;
        }
        before += c;
      }
    }
  }
  __syncthreads();
}

// The k-th largest of the keys that `each` passes to its argument (twice or more: the same each time),
// all in [low, low + range]; k at least 1 and at most their number; `left`: how many of those equal to it are
// among the k.
template <typename Key, int NT, typename Each>
__device__ Key kth_largest(SelectShared<NT>& s, Key low, Key range, int k, Each each, int* left) {
  while (true) {
    const int bits = range == 0 ? 0 : (int)sizeof(Key) * 8 - (sizeof(Key) == 8 ? __clzll((long long)range) : __clz((int)range));
    const int shift = max(bits - 10, 0);
    __syncthreads();
    for (int i = threadIdx.x; i < kBins + kBins / 32; i += NT) s.hist[i] = 0;
    if (threadIdx.x == 0) s.n_few = 0;
    __syncthreads();
    each([&](Key x) {
      if (x - low <= range) atomicAdd(&s.hist[place((int)((x - low) >> shift))], 1);
    });
    __syncthreads();
    find_bin(s, k);
    low += (Key)s.bin << shift;
    k -= s.above;
    range = ((Key)1 << shift) - 1;
    if (shift == 0) break;
    if constexpr (sizeof(Key) == 4) {
      const int n = s.hist[place(s.bin)];
      if (n <= kFew) {  // sorted out among themselves
        each([&](Key x) {
          if (x - low <= range) s.few[atomicAdd(&s.n_few, 1)] = x;
        });
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += NT) {
          const uint32_t x = s.few[i];
          int more = 0, same = 0;
          for (int j = 0; j < n; ++j) {
            more += s.few[j] > x;
            same += s.few[j] == x;
          }
          if (more < k && k <= more + same) s.kth = x, s.above = more;  // of equal ones any
        }
        __syncthreads();
        *left = k - s.above;
        return s.kth;
      }
    }
  }
  *left = k;
  return low;
}

template <typename T, typename QT, int NT>
__global__ void __launch_bounds__(NT) select_kernel(const __grid_constant__ SelectParams p, int HD) {
  __shared__ SelectShared<NT> s;
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
  const bool all = x.n <= p.top;  // no scores then
  auto always = [&](int i) { return i < p.first || i >= x.n - p.last; };
  // the thread's pages [i0, i1), four at a time
  const int run = ((x.n + NT - 1) / NT + 3) & ~3;
  const int i0 = min((long long)tid * run, (long long)x.n), i1 = min(i0 + run, x.n);
  // keys of runs of up to eight stay in registers
  uint4 held[2] = {};
  if (!all && want > 0 && run <= 8)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (i0 + 4 * j < i1) held[j] = *reinterpret_cast<const uint4*>(keys + i0 + 4 * j);
  auto four = [&](int i) {
    if (run <= 8) return i == i0 ? held[0] : held[1];
    return *reinterpret_cast<const uint4*>(keys + i);
  };
  auto each = [&](auto f) {  // f(page, key among those the score decides about)
#pragma unroll 1
    for (int i = i0; i < i1; i += 4) {
      const uint4 v = four(i);
      const uint32_t k[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < i1 && !always(i + j) && k[j] != kNone) f(i + j, k[j]);
    }
  };
  // taken beside the pages that always are: keys above `sure`, and of those in [low, sure] fine keys above
  // `border` and the first `left` that equal it; without a border all from `low` on
  uint32_t low = 1, sure = 0;
  unsigned long long border = 0;
  int left = 0;
  bool ties = false;
  if (!all && want > 0) {
    // range and number of the keys, the largest bound and the sum of the queries' sizes, over the CTA
    uint32_t least = 0xffffffffu, largest = 0;
    int a = 0, b = 0;
    each([&](int, uint32_t k) {
      a += 1;
      b += k == kUnsure;
      least = min(least, k);
      largest = max(largest, k);
    });
    float most = 0.f, sum = 0.f;
    for (int i = tid; i < (x.n + kChunk - 1) / kChunk; i += NT)
      most = fmaxf(most, p.most[(size_t)pair * p.chunks + i]);
    const QT* q = static_cast<const QT*>(p.q) + ((size_t)row * p.heads + (size_t)h * G) * HD;
    for (int i = tid * 4; i < G * HD; i += NT * 4)
      sum += fabsf(widen(q + i)) + fabsf(widen(q + i + 1)) + fabsf(widen(q + i + 2)) + fabsf(widen(q + i + 3));
    least = __reduce_min_sync(0xffffffffu, least);
    largest = __reduce_max_sync(0xffffffffu, largest);
    most = warp_max(most);
    sum = warp_sum(sum);
    if (lane == 0) s.warp_u[warp] = least, s.warp_v[warp] = largest, s.warp_f[warp] = most, s.warp_g[warp] = sum;
    const int2 n = block_sum(s, a, b);
    if (n.x > want) {
      const bool in = lane < NT / 32;
      least = __reduce_min_sync(0xffffffffu, in ? s.warp_u[lane] : 0xffffffffu);
      largest = __reduce_max_sync(0xffffffffu, in ? s.warp_v[lane] : 0u);
      most = warp_max(in ? s.warp_f[lane] : 0.f);
      sum = warp_sum(in ? s.warp_g[lane] : 0.f);
      const float E = (16.f + G) * 5.9604645e-8f * sum * most + 1e-36f;
      sure = kUnsure;
      if (n.y == 0 && E < 1e38f) {
        int same;
        const float t = value_of(kth_largest<uint32_t, NT>(
            s, least, largest - least, want, [&](auto f) { each([&](int, uint32_t k) { f(k); }); }, &same));
        low = order_of(t - 2.f * E);
        sure = order_of(t + 2.f * E);
      }
      // if from `low` on there are as many as are wanted, it is those
      a = b = 0;
      each([&](int, uint32_t k) {
        a += k > sure;
        b += k >= low && k <= sure;
      });
      const int2 m = block_sum(s, a, b);
      if (m.x + m.y > want) {
        // those between again in f64, a warp each
        auto score = [&](int i) {
          const T* at = static_cast<const T*>(p.bounds) +
                        ((size_t)block_of(p, x, x.lo + i) * p.kv_heads + h) * 2 * HD;
          double sum = 0.0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int d = j * 32 + lane;
            if (d >= HD) break;
            double up = 0.0, down = 0.0;
#pragma unroll 4
            for (int g = 0; g < G; ++g) {
              const double y = (double)widen(q + (size_t)g * HD + d);
              // a NaN query stays in both
              up += y < 0.0 ? 0.0 : y;
              down += y > 0.0 ? 0.0 : y;
            }
            sum += up * (double)widen(at + HD + d) + down * (double)widen(at + d);
          }
          for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          return order_of(sum);
        };
        const int wanted = want - m.x;
        if (tid == 0) s.n_few = 0;
        __syncthreads();
        if (m.y <= kFew) {
          each([&](int i, uint32_t k) {
            if (k >= low && k <= sure) s.few[atomicAdd(&s.n_few, 1)] = i;
          });
          __syncthreads();
          for (int e = warp; e < m.y; e += NT / 32) {
            const unsigned long long v = score(s.few[e]);
            if (lane == 0) s.fine[e] = v;
          }
          __syncthreads();
          for (int e = tid; e < m.y; e += NT) {
            const unsigned long long v = s.fine[e];
            int more = 0, same = 0;
            for (int j = 0; j < m.y; ++j) {
              more += s.fine[j] > v;
              same += s.fine[j] == v;
            }
            fine[s.few[e]] = v;
            if (more < wanted && wanted <= more + same) s.border = v, s.above = more;  // of equal ones any
          }
          __syncthreads();
          border = s.border;
          left = wanted - s.above;
        } else {
          // many alike
          for (int i1 = warp * 32; i1 < x.n; i1 += NT) {
            const uint32_t v = i1 + lane < x.n && !always(i1 + lane) ? keys[i1 + lane] : kNone;
            uint32_t some = __ballot_sync(0xffffffffu, v != kNone && v >= low && v <= sure);
            while (some) {
              const int i = i1 + __ffs(some) - 1;
              some &= some - 1;
              const unsigned long long f = score(i);
              if (lane == 0) fine[i] = f;
            }
          }
          __syncthreads();
          border = kth_largest<unsigned long long, NT>(
              s, 0ull, ~0ull, wanted,
              [&](auto f) {
                each([&](int i, uint32_t k) {
                  if (k >= low && k <= sure) f(fine[i]);
                });
              },
              &left);
        }
        ties = true;
      } else {
        sure = low - 1;  // all of them
      }
    }
  }
  // ---- the list: what each thread takes of its run, in order
  int before = 0;  // equal ones in the runs before
  if (ties) {
    int n = 0;
    each([&](int i, uint32_t k) { n += k >= low && k <= sure && fine[i] == border; });
    before = block_scan(s, n).x;
  }
  auto taken = [&](auto f) {
    int tie = before;
    if (all) {
      for (int i = i0; i < i1; ++i)
        if (always(i) || block_of(p, x, x.lo + i) >= 0) f(i);
      return;
    }
#pragma unroll 1
    for (int i = i0; i < i1; i += 4) {
      const uint4 v = want > 0 ? four(i) : make_uint4(0, 0, 0, 0);
      const uint32_t k[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (i + j >= i1) continue;
        bool take = always(i + j);
        if (!take && k[j] != kNone) {
          take = k[j] > sure;
          if (ties && !take && k[j] >= low) {
            const unsigned long long f64 = fine[i + j];
            take = f64 > border || (f64 == border && tie < left);
            tie += f64 == border;
          }
        }
        if (take) f(i + j);
      }
    }
  };
  int n = 0;
  taken([&](int) { ++n; });
  const int2 at = block_scan(s, n);
  int to = at.x;
  taken([&](int i) {
    if (to < p.top) out[to] = x.lo + i;
    ++to;
  });
  for (int i = at.y + tid; i < p.top; i += NT) out[i] = -1;
}

struct Layout {
  int stride, chunks, span;
  size_t keys, fine, most, bytes;
};

inline Layout layout_of(int rows, int kv_heads, int W) {
  Layout x;
  x.stride = (W + 3) & ~3;
  x.chunks = (W + kChunk - 1) / kChunk;
  // a warp's chunks: more than one where those that are resident at once (16 an SM) would have six; rows
  // are seldom as long as their tables, and long items leave warps idle at the end (64 rows of 31 to 2031
  // pages of 2048: 38 us with six chunks an item, 32 with two)
  const long long warps = (long long)rows * kv_heads * x.chunks;
  x.span = (int)std::min<long long>(std::max<long long>(warps / (96ll * std::max(sm_count(), 1)), 1), 4);
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
  const long long items = (long long)((p.chunks + p.span - 1) / p.span) * p.kv_heads;
  const dim3 grid((unsigned)std::min<long long>((items + kScoreWarps - 1) / kScoreWarps, 1 << 20), (unsigned)(p.rows < 65535 ? p.rows : 65535), 1);
  auto* scores = hd == 32 ? score_kernel<T, QT, 32> : hd == 64 ? score_kernel<T, QT, 64> : score_kernel<T, QT, 128>;
  if (p.W > p.top && p.top > p.first + p.last) {  // some row may have to choose
    const cudaError_t e = launch_dependent(scores, grid, kScoreWarps * 32, 0, 0, s, p);
    if (e != cudaSuccess) return e;
  }
  // threads: eight keys each, but few CTAs are wide ones
  const bool wide = p.W > 2048;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.rows * p.kv_heads), 1, 1);
  cfg.blockDim = dim3(wide ? 1024 : 256, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return wide ? cudaLaunchKernelEx(&cfg, select_kernel<T, QT, 1024>, p, hd)
              : cudaLaunchKernelEx(&cfg, select_kernel<T, QT, 256>, p, hd);
}

rq_status check(const rq_paged_kv* kv, int32_t rows, int32_t max_blocks) {
  const rq_status st = paged_kv_check(kv);
  if (st != RQ_OK) return st;
  if (rows < 0 || max_blocks < 1) return RQ_ERR_ARG;
  if (max_blocks > 1 << 30 || kv->heads > 1 << 23 || (long long)rows * kv->heads > INT_MAX) return RQ_ERR_UNSUPPORTED;
  if ((double)rows * kv->heads * max_blocks > 1099511627776.0) return RQ_ERR_UNSUPPORTED;
  // a block's bounds are counted in 32 bits of bytes
  if ((long long)kv->heads * 2 * kv->head_dim * (kv->dtype == RQ_BF16 ? 2 : 4) > UINT_MAX) return RQ_ERR_UNSUPPORTED;
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
  if (rows > 1 << 30 || heads > 1 << 23 || (long long)rows * heads > INT_MAX || top > 1 << 30) return RQ_ERR_UNSUPPORTED;
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
  p.span = x.span;
  p.chunks = x.chunks;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  const bool b = kv->dtype == RQ_BF16, qb = q_dtype == RQ_BF16;
  const cudaError_t e = b ? (qb ? launch<uint16_t, uint16_t>(p, kv->head_dim, s) : launch<uint16_t, float>(p, kv->head_dim, s))
                          : (qb ? launch<float, uint16_t>(p, kv->head_dim, s) : launch<float, float>(p, kv->head_dim, s));
  return e == cudaSuccess ? RQ_OK : RQ_ERR_CUDA;
}
