// paged_attn.cuh -- attention of one query token per row over a paged K/V cache: the kernel
// template (include/rq.h, rq_paged_attention; instantiated by paged_attn_bf16.cu and
// paged_attn_f32.cu, launched by paged_attn.cu).
//
// For row r with position pos and query head h: s_j = scale q . k_j over the live positions
// j, o = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m), in one pass with m the running maximum and
// the sums rescaled when it moves (all in base 2: scale carries log2 e).
//
// Work. A unit is one (row, K/V head, group of up to 8 query heads that read it), a tile 64
// consecutive positions of a unit. All units' tiles form one list, rows outermost; the grid
// (a few CTAs per SM, all resident) cuts it into equal runs, one per CTA, whatever the rows'
// lengths are. A unit that lies in one CTA is finished there; one that is cut leaves a
// partial (m, l, acc) per CTA, joined in order by the merge kernel, so the result does not
// depend on timing. A CTA has at most two cut units (its first and its last), which bounds
// the workspace by the grid.
//
// A tile is split over the CTA's 4 warps, 16 positions each. Every warp streams its own
// K and V rows with 16-byte cp.async into a ring of its own, ahead across units, and meets the others
// only at the end of a unit. Positions outside the live range or in a missing block are
// filled with zeros by the copy and masked, so nothing that lies there is ever used.
#pragma once

#include "paged.cuh"

namespace rqk {
namespace paged_attn {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kKeys = 16;                  // positions of a warp's part of a tile
constexpr int kTile = kWarps * kKeys;      // positions of a tile
constexpr int kHeads = 8;                  // query heads of a unit, at most
constexpr int kMaxGrid = 608;              // CTAs of a launch, at most
constexpr int kMinTiles = 1;               // tiles of a CTA's run, at least

struct Params {
  rq_paged_kv kv;
  const void* q;
  void* out;
  float* lse;
  const int32_t *table, *requests, *positions;
  int rows, heads, batch, W, window;
  int G, HG, GB;       // query heads per K/V head, groups of them, heads in a group
  float scale;         // times log2 e
  float* part;         // [grid][2][GB][HD] partial sums
  float2* part_ml;     // [grid][2][GB] (m, l)
  int4* cut;           // [grid] (row, group, parts, 0) of the unit to join that starts there
};

inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }
inline size_t part_bytes(int gb, int hd) {
  return align256((size_t)kMaxGrid * 2 * gb * hd * sizeof(float));
}
inline size_t ml_bytes(int gb) { return align256((size_t)kMaxGrid * 2 * gb * sizeof(float2)); }
inline size_t workspace_bytes(int gb, int hd) {
  return part_bytes(gb, hd) + ml_bytes(gb) + align256((size_t)kMaxGrid * sizeof(int4));
}

// A unit's shared-memory ring and merge buffer, by element type and head size: the ring is
// as deep as lets two or more CTAs share an SM (K rows of bf16 are padded by 16 bytes, so
// the eight rows an ldmatrix reads fall into different banks).
template <typename KT, int HD>
struct Shape {
  static constexpr int kPitch = sizeof(KT) == 2 ? HD * 2 + 16 : HD * 4;  // bytes of a row
  static constexpr int kStage = 2 * kKeys * kPitch;                      // K rows, then V rows
  static constexpr int kStages = HD == 128 ? 3 : 4;
  static constexpr int kMergeDims = HD > 64 ? 64 : HD;  // dimensions joined at a time
  static constexpr size_t kRing = (size_t)kWarps * kStages * kStage;
  static constexpr size_t kSmem = kRing + (size_t)kWarps * kHeads * kMergeDims * sizeof(float);
};

struct Row {
  int b, lo, pos, t0, nt;  // request, live positions [lo, pos], tiles [t0, t0 + nt)
};

__device__ __forceinline__ Row load_row(const Params& p, int r) {
  Row x;
  x.b = p.requests ? p.requests[r] : r;
  x.pos = p.positions[r];
  x.lo = x.t0 = x.nt = 0;
  if (x.b < 0 || x.b >= p.batch || x.pos < 0) return x;
  const int P = p.kv.block_size, first = x.pos / P - p.W + 1;
  if (first > 0) x.lo = first * P;
  if (p.window > 0) x.lo = max(x.lo, x.pos - p.window + 1);
  x.t0 = x.lo / kTile;
  x.nt = x.pos / kTile - x.t0 + 1;
  return x;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 2^x in one instruction (its error is two steps of the result)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float neg_inf() { return -__int_as_float(0x7f800000); }
// the reference point of a maximum that may still be -inf
__device__ __forceinline__ float finite_or_zero(float m) { return m == neg_inf() ? 0.f : m; }

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) {
  *p = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// ---------------------------------------------------------------- bf16 cache: tensor cores
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// (lo, hi) as bf16 pairs: the rounded values, and what the rounding left
__device__ __forceinline__ uint32_t split_bf16(float& lo, float& hi) {
  const uint32_t u = pack_bf16(lo, hi);
  lo -= bf16lo(u);
  hi -= bf16hi(u);
  return u;
}

// A warp's share of a unit over a bf16 cache. Decode is bound by reading the cache: the
// tensor cores (mma.sync m16n8k16; a unit has at most 8 query rows, far below a tcgen05
// tile) are there so that 8 queries a K/V head cost no more than one. The 16 rows of A hold
// 8 heads twice: rows 0-7 a value's leading bf16 part, rows 8-15 the part that rounding
// left, so both halves of a product come out of one instruction, in one thread (c0 + c2,
// c1 + c3). f32 queries and their weights take a third part in a second instruction: 24
// bits, every product exact. bf16 queries are exact in one part; their weights have two.
template <typename QT, int HD>
struct MmaCore {
  static constexpr bool kF32 = sizeof(QT) == 4;
  static constexpr int kSteps = HD / 16;
  using S = Shape<uint16_t, HD>;
  uint32_t q[kF32 ? 3 : 1][kSteps][2];
  float acc[HD / 8][2];
  float m, l;

  __device__ __forceinline__ void begin(const Params& p, const QT* qrow, int live, int lane) {
    const int g = lane >> 2, c = (lane & 3) * 2;
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int d = k * 16 + c + i * 8;
        if constexpr (kF32) {
          float2 x = make_float2(0.f, 0.f);
          if (g < live) x = *reinterpret_cast<const float2*>(qrow + (size_t)g * HD + d);
          q[0][k][i] = split_bf16(x.x, x.y);
          q[1][k][i] = split_bf16(x.x, x.y);
          q[2][k][i] = pack_bf16(x.x, x.y);
        } else {
          q[0][k][i] = g < live ? *reinterpret_cast<const uint32_t*>(qrow + (size_t)g * HD + d) : 0u;
        }
      }
#pragma unroll
    for (int i = 0; i < HD / 8; ++i) acc[i][0] = acc[i][1] = 0.f;
    m = neg_inf();
    l = 0.f;
  }

  __device__ __forceinline__ void tile(const Params& p, uint32_t ks, uint32_t mask, int lane, float*) {
    const uint32_t vs = ks + kKeys * S::kPitch;
    float c[2][4] = {};
    // B of the first product: K rows as they lie (8 keys x 8 dimensions a matrix)
    const uint32_t kaddr = ks + ((lane >> 4) * 8 + (lane & 7)) * S::kPitch + ((lane >> 3) & 1) * 16;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      uint32_t b[4];
      ldmatrix4(kaddr + k * 32, b);
      if constexpr (kF32) {
        mma16816(c[0], q[0][k][0], q[1][k][0], q[0][k][1], q[1][k][1], b[0], b[1]);
        mma16816(c[1], q[0][k][0], q[1][k][0], q[0][k][1], q[1][k][1], b[2], b[3]);
      } else {
        mma16816(c[0], q[0][k][0], 0u, q[0][k][1], 0u, b[0], b[1]);
        mma16816(c[1], q[0][k][0], 0u, q[0][k][1], 0u, b[2], b[3]);
      }
    }
    float e[2][4] = {};
    if constexpr (kF32) {
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        uint32_t b[4];
        ldmatrix4(kaddr + k * 32, b);
        mma16816(e[0], q[2][k][0], 0u, q[2][k][1], 0u, b[0], b[1]);
        mma16816(e[1], q[2][k][0], 0u, q[2][k][1], 0u, b[2], b[3]);
      }
    }
    // this thread: head lane / 4, keys 8 n + 2 (lane % 4) + i
    float s[2][2], mx = m;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = c[n][i];
        if constexpr (kF32) {
          // an infinite key's product stands: the parts that are 0 would make it NaN
          if (fabsf(x) != __int_as_float(0x7f800000)) x += c[n][2 + i] + e[n][i];
        }
        x *= p.scale;
        s[n][i] = (mask >> (n * 8 + (lane & 3) * 2 + i)) & 1u ? x : neg_inf();
        mx = fmaxf(mx, s[n][i]);
      }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const float ref = finite_or_zero(mx), scale = ex2(m - ref);
    m = mx;
    float w[2][2];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) w[n][i] = ex2(s[n][i] - ref);
    l = l * scale + ((w[0][0] + w[0][1]) + (w[1][0] + w[1][1]));
    const uint32_t a0 = split_bf16(w[0][0], w[0][1]), a2 = split_bf16(w[1][0], w[1][1]);
    uint32_t a1, a3, e0 = 0, e2 = 0;
    if constexpr (kF32) {
      a1 = split_bf16(w[0][0], w[0][1]);
      a3 = split_bf16(w[1][0], w[1][1]);
      e0 = pack_bf16(w[0][0], w[0][1]);
      e2 = pack_bf16(w[1][0], w[1][1]);
    } else {
      a1 = pack_bf16(w[0][0], w[0][1]);
      a3 = pack_bf16(w[1][0], w[1][1]);
    }
    // B of the second product: V rows transposed on the way in
    const uint32_t vaddr = vs + (((lane >> 3) & 1) * 8 + (lane & 7)) * S::kPitch + (lane >> 4) * 16;
#pragma unroll
    for (int d = 0; d < HD / 16; ++d) {
      uint32_t b[4];
      ldmatrix4_trans(vaddr + d * 32, b);
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        float o[4] = {};
        mma16816(o, a0, a1, a2, a3, b[2 * n], b[2 * n + 1]);
        if constexpr (kF32) mma16816(o, e0, 0u, e2, 0u, b[2 * n], b[2 * n + 1]);
        float* a = acc[2 * d + n];
        a[0] = fmaf(a[0], scale, o[0] + o[2]);
        a[1] = fmaf(a[1], scale, o[1] + o[3]);
      }
    }
  }

  // this warp's (m, l) of each head, and its sums of dimensions [d0, d0 + n)
  __device__ __forceinline__ void state(float2* ml, int lane) {
    float t = l + __shfl_xor_sync(0xffffffffu, l, 1);
    t += __shfl_xor_sync(0xffffffffu, t, 2);
    if ((lane & 3) == 0) ml[lane >> 2] = make_float2(m, t);
  }
  template <int N>
  __device__ __forceinline__ void sums(float* dst, int d0, int lane) {
    const int g = lane >> 2, c = (lane & 3) * 2;
#pragma unroll
    for (int i = 0; i < HD / 8; ++i)
      if (i * 8 >= d0 && i * 8 < d0 + N)
        *reinterpret_cast<float2*>(dst + g * N + i * 8 - d0 + c) = make_float2(acc[i][0], acc[i][1]);
  }
};

// ---------------------------------------------------------------- f32 cache: FMA
// A lane holds HD / 32 consecutive dimensions of up to GP heads' queries and sums. Its part
// of each score meets the other lanes' in a transposing butterfly (32 values in 31 shuffles,
// one left per lane); the weights go round through shared memory.
template <typename QT, int HD, int GP>
struct FmaCore {
  static constexpr int E = HD / 32;
  static constexpr int NV = kKeys * GP < 32 ? kKeys * GP : 32;  // scores of a butterfly
  static constexpr int NB = kKeys * GP / NV;                     // butterflies of a tile
  static constexpr int KB = NV / GP;                             // keys of a butterfly
  using S = Shape<float, HD>;
  float q[GP][E], acc[GP][E];
  float m, l;  // of head index % GP, index = lane / (32 / NV)

  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ float one(const uint16_t* p) { return bf16lo(*p); }

  static __device__ __forceinline__ void row(uint32_t addr, float (&v)[E]) {
    if constexpr (E == 4)
      asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(addr) : "memory");
    else if constexpr (E == 2)
      asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "r"(addr) : "memory");
    else
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[0]) : "r"(addr) : "memory");
  }

  __device__ __forceinline__ void begin(const Params& p, const QT* qrow, int live, int lane) {
#pragma unroll
    for (int h = 0; h < GP; ++h)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        q[h][e] = h < live ? one(qrow + (size_t)h * HD + lane * E + e) : 0.f;
        acc[h][e] = 0.f;
      }
    m = neg_inf();
    l = 0.f;
  }

  __device__ __forceinline__ float max_over_keys(float x) const {
#pragma unroll
    for (int o = GP * (32 / NV); o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
  }

  __device__ __forceinline__ void tile(const Params& p, uint32_t ks, uint32_t mask, int lane, float* sw) {
    const uint32_t vs = ks + kKeys * S::kPitch;
    const int vi = lane / (32 / NV);
    float s[NB], mx = m;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float v[NV];
#pragma unroll
      for (int k = 0; k < KB; ++k) {
        float x[E];
        row(ks + (b * KB + k) * S::kPitch + lane * E * 4, x);
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          float d = q[h][0] * x[0];
#pragma unroll
          for (int e = 1; e < E; ++e) d = fmaf(q[h][e], x[e], d);
          v[k * GP + h] = d;
        }
      }
#pragma unroll
      for (int o = 16, n = NV / 2; n >= 1; o >>= 1, n >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < n; ++i) {
          const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
          v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
      }
      if (NV == 16) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
      s[b] = (mask >> (b * KB + vi / GP)) & 1u ? v[0] * p.scale : neg_inf();
      mx = fmaxf(mx, s[b]);
    }
    mx = max_over_keys(mx);
    const float ref = finite_or_zero(mx), scale = ex2(m - ref);
    m = mx;
    l *= scale;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const float w = ex2(s[b] - ref);
      l += w;
      sw[b * NV + vi] = w;
    }
    __syncwarp();
#pragma unroll
    for (int h = 0; h < GP; ++h) {
      const float sc = __shfl_sync(0xffffffffu, scale, h * (32 / NV));
#pragma unroll
      for (int e = 0; e < E; ++e) acc[h][e] *= sc;
    }
#pragma unroll
    for (int k = 0; k < kKeys; ++k) {
      float x[E];
      row(vs + k * S::kPitch + lane * E * 4, x);
#pragma unroll
      for (int h = 0; h < GP; ++h) {
        const float w = sw[k * GP + h];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[h][e] = fmaf(w, x[e], acc[h][e]);
      }
    }
    __syncwarp();
  }

  __device__ __forceinline__ void state(float2* ml, int lane) {
    float t = l;
#pragma unroll
    for (int o = GP * (32 / NV); o < 32; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    const int h = lane / (32 / NV);
    if (lane % (32 / NV) == 0 && h < GP) ml[h] = make_float2(m, t);
    if (lane >= GP && lane < kHeads) ml[lane] = make_float2(neg_inf(), 0.f);
  }
  template <int N>
  __device__ __forceinline__ void sums(float* dst, int d0, int lane) {
#pragma unroll
    for (int h = 0; h < GP; ++h)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int d = lane * E + e - d0;
        if (d >= 0 && d < N) dst[h * N + d] = acc[h][e];
      }
  }
};

// ---------------------------------------------------------------- the kernel
enum : int { kStart = 1, kEnd = 2, kFirst = 4, kLast = 8 };  // of the run's piece; of the unit

template <typename QT, typename KT, int HD, typename Core>
__global__ void __launch_bounds__(kThreads) attend_kernel(const __grid_constant__ Params p) {
  using S = Shape<KT, HD>;
  constexpr int NS = S::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_scan[kWarps];
  __shared__ long long s_off;             // the run's first tile, counted from row s_row's first
  __shared__ int s_row;
  __shared__ int4 s_desc[kWarps][NS];     // row, group, key mask, flags of each stage's part
  __shared__ float2 s_ml[kWarps][kHeads];
  __shared__ __align__(16) float s_w[kWarps][kKeys * kHeads];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int units = p.kv.heads * p.HG;    // units of a row
  float* const s_acc = reinterpret_cast<float*>(smem + S::kRing);

  // where this CTA's run starts: prefix sums of the rows' tiles, a slice of rows per thread
  const int slice = (p.rows + kThreads - 1) / kThreads;
  const int r0 = min(tid * slice, p.rows), r1 = min(r0 + slice, p.rows);
  long long own = 0;
  for (int r = r0; r < r1; ++r) own += (long long)load_row(p, r).nt * units;
  long long inc = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) s_scan[warp] = inc;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) inc += s_scan[w];
    total += s_scan[w];
  }
  long long per = (total + gridDim.x - 1) / gridDim.x;
  if (per < kMinTiles) per = kMinTiles;
  const long long begin = min((long long)blockIdx.x * per, total);
  const int n = (int)(min(begin + per, total) - begin);
  if (n > 0 && inc - own <= begin && begin < inc) {
    long long at = begin - (inc - own);
    for (int r = r0; r < r1; ++r) {
      const long long t = (long long)load_row(p, r).nt * units;
      if (at < t) {
        s_row = r;
        s_off = at;
        break;
      }
      at -= t;
    }
  }
  __syncthreads();
  pdl_trigger();
  // rows of empty requests
  for (int r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const int b = p.requests ? p.requests[r] : r;
    if (b < 0 || b >= p.batch || p.positions[r] >= 0) continue;
    QT* o = static_cast<QT*>(p.out) + (size_t)r * p.heads * HD;
    for (int i = tid; i < p.heads * HD; i += kThreads) put(o + i, 0.f);
    if (p.lse)
      for (int i = tid; i < p.heads; i += kThreads) p.lse[(size_t)r * p.heads + i] = neg_inf();
  }
  int4 cut = make_int4(0, 0, 0, 0);
  if (n > 0) {
    // ---- the warp's stream of parts: a cursor over (row, group, tile), one table entry ahead
    Row x = load_row(p, s_row);
    int r = s_row, u = (int)(s_off / x.nt), t = (int)(s_off % x.nt);
    int issued = 0;
    const int P = p.kv.block_size;
    const uint32_t ring = smem_u32(smem) + warp * NS * S::kStage;
    int key = 0, page = 0, id = -1;  // lane i < 16: the i-th key of the cursor's part
    auto look_up = [&]() {
      key = (x.t0 + t) * kTile + warp * kKeys + (lane & 15);
      page = key / P;
      id = -1;
      if (key >= x.lo && key <= x.pos && key >= 0)
        id = p.table[(size_t)x.b * p.W + (page < p.W ? page : page % p.W)];
    };
    look_up();
    auto issue = [&]() {
      const int s = issued % NS;
      const bool ok = id >= 0 && id < p.kv.n_blocks;
      const uint32_t mask = __ballot_sync(0xffffffffu, ok) & 0xffffu;
      const int kvh = u / p.HG;
      const long long off = ok ? id * p.kv.block_stride + (key - page * P) * p.kv.row_stride +
                                     kvh * p.kv.head_stride
                               : 0;
      if (lane == 0) {
        int f = 0;
        if (issued == 0 || t == 0) f |= kStart;
        if (issued == n - 1 || t == x.nt - 1) f |= kEnd;
        if (t == x.nt - 1) f |= kLast;
        // the unit's first tile is in this run: t steps back are
        if (t <= issued) f |= kFirst;
        s_desc[warp][s] = make_int4(r, u, (int)mask, f);
        if (issued == n - 1 && t < x.nt - 1) {  // the unit goes on in the runs that follow
          const long long end = begin + n - 1 + (x.nt - t);
          cut = make_int4(r, u, t <= issued ? (int)((end - 1) / per - blockIdx.x) + 1 : 0, 0);
        }
      }
      if (mask) {
        constexpr int CH = HD * sizeof(KT) / 16;  // 16-byte pieces of a row
        constexpr int RPI = 32 / CH > 0 ? 32 / CH : 1;
        const uint32_t dst = ring + s * S::kStage;
        const KT* kb = static_cast<const KT*>(p.kv.k);
        const KT* vb = static_cast<const KT*>(p.kv.v);
        const int c = lane % CH;
#pragma unroll
        for (int i = 0; i < kKeys / RPI; ++i) {
          const int row = i * RPI + lane / CH;
          const long long o = __shfl_sync(0xffffffffu, off, row);
          const bool live = (mask >> row) & 1u;
          const long long e = o + c * (16 / (int)sizeof(KT));
          cp_async16(dst + row * S::kPitch + c * 16, kb + e, live);
          cp_async16(dst + (kKeys + row) * S::kPitch + c * 16, vb + e, live);
        }
      }
      // on to the next part
      ++issued;
      if (issued < n) {
        if (++t == x.nt) {
          t = 0;
          if (++u == units) {
            u = 0;
            do {
              x = load_row(p, ++r);
            } while (x.nt == 0 && r + 1 < p.rows);
          }
        }
        look_up();
      }
    };
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) {
      if (issued < n) issue();
      cp_async_commit();
    }
    Core core;
    for (int i = 0; i < n; ++i) {
      if (issued < n) issue();
      cp_async_commit();
      cp_async_wait<NS - 1>();
      __syncwarp();
      const int4 d = s_desc[warp][i % NS];
      const int kvh = d.y / p.HG, g0 = (d.y % p.HG) * kHeads, live = min(kHeads, p.G - g0);
      const size_t head = (size_t)d.x * p.heads + (size_t)kvh * p.G + g0;
      if (d.w & kStart)
        core.begin(p, static_cast<const QT*>(p.q) + head * HD, live, lane);
      if (d.z) core.tile(p, ring + (i % NS) * S::kStage, (uint32_t)d.z, lane, s_w[warp]);
      __syncwarp();  // the stage is free for the next copy
      if (!(d.w & kEnd)) continue;
      // ---- join the warps
      constexpr int N = S::kMergeDims;
      core.state(s_ml[warp], lane);
      const bool whole = (d.w & kFirst) && (d.w & kLast);
      const size_t slot = (size_t)blockIdx.x * 2 + ((d.w & kFirst) ? 1 : 0);
#pragma unroll
      for (int d0 = 0; d0 < HD; d0 += N) {
        core.template sums<N>(s_acc + warp * kHeads * N, d0, lane);
        __syncthreads();
        for (int j = tid; j < live * N; j += kThreads) {
          const int g = j / N, dd = j % N;
          float M = neg_inf();
#pragma unroll
          for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_ml[w][g].x);
          const float ref = finite_or_zero(M);
          float L = 0.f, A = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float c = ex2(s_ml[w][g].x - ref);
            L += s_ml[w][g].y * c;
            A += s_acc[(w * kHeads + g) * N + dd] * c;
          }
          if (whole) {
            put(static_cast<QT*>(p.out) + (head + g) * HD + d0 + dd, L == 0.f ? 0.f : A / L);
            if (p.lse && d0 + dd == 0)
              p.lse[head + g] = L == 0.f ? neg_inf() : (M + log2f(L)) * 0.6931471805599453f;
          } else {
            p.part[(slot * p.GB + g) * HD + d0 + dd] = A;
            if (d0 + dd == 0) p.part_ml[slot * p.GB + g] = make_float2(M, L);
          }
        }
        __syncthreads();
      }
    }
  }
  if (tid == 0) p.cut[blockIdx.x] = cut;
}

// One CTA per (run, head of a group): if a unit starts in run blockIdx.x and goes on, its
// partials -- the run's second slot, then the first slot of each run that follows -- are
// summed in order.
template <typename QT, int HD>
__global__ void __launch_bounds__(HD) join_kernel(const __grid_constant__ Params p) {
  pdl_wait();
  const int4 cut = p.cut[blockIdx.x];
  if (cut.z == 0) return;
  const int kvh = cut.y / p.HG, g0 = (cut.y % p.HG) * kHeads, g = blockIdx.y;
  if (g >= min(kHeads, p.G - g0)) return;
  const size_t head = (size_t)cut.x * p.heads + (size_t)kvh * p.G + g0 + g;
  const int d = threadIdx.x;
  auto slot = [&](int i) { return (size_t)(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0); };
  float M = neg_inf();
  for (int i = 0; i < cut.z; ++i) M = fmaxf(M, p.part_ml[slot(i) * p.GB + g].x);
  const float ref = finite_or_zero(M);
  float L = 0.f, A = 0.f;
#pragma unroll 8
  for (int i = 0; i < cut.z; ++i) {
    const float2 ml = p.part_ml[slot(i) * p.GB + g];
    const float a = p.part[(slot(i) * p.GB + g) * HD + d];
    const float c = ex2(ml.x - ref);
    L += ml.y * c;
    A += a * c;
  }
  put(static_cast<QT*>(p.out) + head * HD + d, L == 0.f ? 0.f : A / L);
  if (p.lse && d == 0) p.lse[head] = L == 0.f ? neg_inf() : (M + log2f(L)) * 0.6931471805599453f;
}

// Launch one instantiation: as many CTAs as are resident at once, at most one per tile that
// the largest rows could have.
template <typename QT, typename KT, int HD, typename Core>
cudaError_t launch(const Params& p, cudaStream_t s) {
  using S = Shape<KT, HD>;
  auto* kernel = attend_kernel<QT, KT, HD, Core>;
  int dev = 0, sms = 0, per_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
  if (e == cudaSuccess)
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, S::kSmem);
  if (e != cudaSuccess) return e;
  if (per_sm < 1) return cudaErrorInvalidConfiguration;
  long long keys = min((long long)p.W * p.kv.block_size, (long long)INT_MAX);
  if (p.window > 0 && p.window < keys) keys = p.window;
  const long long most = (keys / kTile + 2) * p.rows * p.kv.heads * p.HG;
  long long grid = (long long)sms * per_sm;
  if (grid > kMaxGrid) grid = kMaxGrid;
  if (grid > most) grid = most;
  kernel<<<(unsigned)grid, kThreads, S::kSmem, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, (unsigned)p.GB, 1);
  cfg.blockDim = dim3(HD, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<QT, HD>, p);
}

cudaError_t launch_bf16(const Params& p, bool q_bf16, cudaStream_t s);  // over a bf16 cache
cudaError_t launch_f32(const Params& p, bool q_bf16, cudaStream_t s);   // over an f32 cache

}  // namespace paged_attn
}  // namespace rqk
