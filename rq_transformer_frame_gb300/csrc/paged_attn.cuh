// paged_attn.cuh -- attention of one query token per row over a paged K/V cache: the kernel
// template (include/rq.h, rq_paged_attention; instantiated by paged_attn_bf16.cu and
// paged_attn_f32.cu, launched by paged_attn.cu; with lists of pages rq_paged_sparse_attention,
// paged_sparse.cu; with f32 outputs part of rq_paged_prefix_attention, paged_prefix.cu).
//
// For row r with position pos and query head h: s_j = scale q . k_j over the live positions
// j, o = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m), in one pass with m the running maximum and
// the sums rescaled when it moves (all in base 2: scale carries log2 e).
//
// Work. A unit is one (row, K/V head, group of query heads that read it), a tile 4 KB of K
// at most (and as much V) of a unit: 16 positions at head_dim 128 in bf16. All units' tiles form one
// list, rows outermost, in which a unit also counts kUnitCost tiles for its start and end; the
// resident warps cut it into equal runs, one each, whatever the rows' lengths are. Warps work
// alone: each streams its own K and V rows with 16-byte cp.async into a ring of its own,
// ahead across units, and writes what it finished. A unit that is cut leaves a partial
// (m, l, acc) per run, joined in order by a second kernel, so the result does not depend on
// timing. A run has at most two cut units (its first and its last), which bounds the
// workspace by the grid. Where no row can be long, runs are of whole units instead: nothing
// to search and nothing to join.
//
// Positions outside the live range or in a missing block are filled with zeros by the copy
// and masked, so nothing that lies there is ever used.
//
// Lists. In mode kLists a row's positions are not a range but those of the pages that a list names,
// another list for each K/V head: every (row, K/V head) is then a row of its own, of one K/V head
// and its queries, and its key j is position j % block_size of the list's entry j / block_size.
//
// Prefixes. In mode kPrefixes each row of queries is two rows, one over the prefix that its group
// shares and one over its own request. Of the first kind `bundle` rows of a group are one, their queries
// a unit's like those of one row are; the others of the bundle have nothing to do.
#pragma once

#include <type_traits>

#include "paged.cuh"
#include "tc_common.cuh"

namespace rqk {
namespace paged_attn {

constexpr int kWarps = 4, kStages = 2;            // of a CTA of runs; stages of a warp's ring
constexpr int kSplitWarps = 8;                    // of a CTA of one unit
// stages of a split warp's ring, with SCRATCH bytes of a warp beside it: as the CTA's 227 KB
// allow
template <int STAGE, int SCRATCH>
constexpr int split_stages = kSplitWarps * (3 * STAGE + SCRATCH) <= 224 * 1024 ? 3 : 2;
constexpr int kMaxGrid = 304;              // CTAs of a launch, at most
constexpr int kMaxRuns = kMaxGrid * kWarps;
constexpr int kMinRun = 1;                 // tiles of a run, at least
constexpr int kUnitCost = 1;               // what a unit's start and end count, in tiles
enum Mode { kRows, kLists, kPrefixes };

struct Params {
  rq_paged_kv kv;
  const void* q;
  void* out;
  float* lse;
  const int32_t *table, *requests, *positions;
  int rows, heads, batch, W, window;
  int G, GB, HG;       // query heads per K/V head (of all a unit reads), of a unit; units of a K/V head
  int runs;            // runs (warps) of the launch
  int whole;           // units of a run that takes whole ones, 0: runs are cut anywhere
  float scale;         // times log2 e
  float* part;         // [runs][2][GB][HD] partial sums
  float unit;          // what the sums of values are in (a core's kUnit)
  float2* part_ml;     // [runs][2][GB] (m, l)
  int4* cut;           // [runs] (row, first head, heads, parts) of the unit that starts there and goes on
};

// what the other modes have besides (a launch's time goes by the size of its parameters too)
struct MoreParams : Params {
  const int32_t* pages;  // kLists: [rows][list] pages, -1 in empty entries
  int list, kv_heads;    // kLists: entries of a list; rows of one query token
  const int32_t *cu_rows, *prefix_requests, *prefix_lens;  // kPrefixes: rq_paged_prefix_attention's
  int groups, q_rows;    // rows of queries: over prefixes first, then as many over their own requests
  int bundle;            // rows over a prefix that are one
  int row_heads, row_skip;  // queries of a row in a unit, and the heads to the next row's first behind them
};
template <Mode MODE>
using ParamsOf = std::conditional_t<MODE == kRows, Params, MoreParams>;

inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }
inline size_t part_bytes(int gb, int hd) {
  return align256((size_t)kMaxRuns * 2 * gb * hd * sizeof(float));
}
inline size_t ml_bytes(int gb) { return align256((size_t)kMaxRuns * 2 * gb * sizeof(float2)); }
inline size_t workspace_bytes(int gb, int hd) {
  return part_bytes(gb, hd) + ml_bytes(gb) + align256((size_t)kMaxRuns * sizeof(int4));
}

// A warp's ring, by element type and head size: stages of K and V rows. The 16-byte pieces of a
// row are permuted by the row's number, so that one piece of eight rows -- what an ldmatrix
// reads, and what eight lanes with a key each do -- falls into different banks.
template <typename KT, int HD>
struct Shape {
  static constexpr int kPitch = HD * (int)sizeof(KT);  // bytes of a row
  // positions of a tile: 8 KB of K and V, but 32 at most (a lane looks one up; bf16 heads of 32
  // dimensions alone have 4 KB then) and 16 at least in bf16 (the second product's step)
  static constexpr int kKeys = 4096 / kPitch < 32 ? 4096 / kPitch : 32;
  static constexpr int kStage = 2 * kKeys * kPitch;    // K rows, then V rows
  // where piece c of row r lies, in bytes from the tile's first row
  static __device__ __forceinline__ int at(int r, int c) {
    return r * kPitch + (c ^ (kPitch >= 128 ? r & 7 : (r >> 1) & 3)) * 16;
  }
};

struct Row {
  int r;                   // kLists: its number
  int b, lo, pos, t0, nt;  // request, live positions [lo, pos], tiles [t0, t0 + nt)
};

// the group of row r, of groups [cu_rows[g], cu_rows[g + 1]), or -1
__device__ __forceinline__ int group_of(const int32_t* cu_rows, int groups, int r) {
  int lo = 0, hi = groups;  // the last one that starts at the row or before
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (cu_rows[mid] <= r) lo = mid + 1;
    else hi = mid;
  }
  return lo > 0 && r < cu_rows[lo] ? lo - 1 : -1;
}

// row r's request and position as they stand; out of the list: no tiles
template <Mode MODE>
__device__ __forceinline__ int2 row_words(const ParamsOf<MODE>& p, int r) {
  if ((unsigned)r >= (unsigned)p.rows) return make_int2(-1, -1);
  if constexpr (MODE == kLists) r /= p.kv_heads;
  if constexpr (MODE == kPrefixes) {
    if (r >= p.q_rows) {
      r -= p.q_rows;
      return make_int2(p.requests ? p.requests[r] : r, p.positions[r]);
    }
    const int g = group_of(p.cu_rows, p.groups, r);
    if (g >= 0) {
      const int x = p.prefix_requests[g], n = p.prefix_lens[g];
      if (x >= 0 && x < p.batch && n > 0)
        return (r - max(p.cu_rows[g], 0)) % p.bundle == 0 ? make_int2(x, n - 1) : make_int2(-1, -1);
    }
    return make_int2(0, -1);  // no prefix: an empty request
  }
  return make_int2(p.requests ? p.requests[r] : r, p.positions[r]);
}

// rows of a unit of row r
template <Mode MODE>
__device__ __forceinline__ int bundle_of(const ParamsOf<MODE>& p, int r) {
  static_assert(MODE == kPrefixes, "rows of the other modes are one each");
  if (p.bundle == 1 || r >= p.q_rows) return 1;
  const int g = group_of(p.cu_rows, p.groups, r);
  return g < 0 ? 1 : min(p.bundle, min(p.cu_rows[g + 1], p.q_rows) - r);
}
// where query g of a unit is, in heads from its first
struct Next {
  __device__ __forceinline__ size_t operator()(int g) const { return g; }
};
struct Bundled {
  int row_heads, row_skip;
  __device__ __forceinline__ size_t operator()(int g) const { return g + (size_t)(g / row_heads) * row_skip; }
};

template <int kKeys, Mode MODE>
__device__ __forceinline__ Row row_of(const ParamsOf<MODE>& p, int r, int2 words) {
  Row x;
  x.r = r;
  x.b = words.x;
  x.pos = words.y;
  x.lo = x.t0 = x.nt = 0;
  if (x.b < 0 || x.b >= p.batch || x.pos < 0) return x;
  if constexpr (MODE == kLists) {
    x.nt = (p.list * p.kv.block_size - 1) / kKeys + 1;
    return x;
  }
  const int P = p.kv.block_size, first = x.pos / P - p.W + 1;
  if (first > 0) x.lo = first * P;
  if (p.window > 0) x.lo = max(x.lo, x.pos - p.window + 1);
  x.t0 = x.lo / kKeys;
  x.nt = x.pos / kKeys - x.t0 + 1;
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
// the log of the sum of e^s from the base-2 maximum and sum
__device__ __forceinline__ float log_sum(float m, float l) {
  return l == 0.f ? neg_inf() : (m + log2f(l)) * 0.6931471805599453f;
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
__device__ __forceinline__ void put2(float* p, float a, float b) {
  *reinterpret_cast<float2*>(p) = make_float2(a, b);
}
__device__ __forceinline__ void put2(uint16_t* p, float a, float b) {
  *reinterpret_cast<uint32_t*>(p) = pack_bf16(a, b);
}
// (lo, hi) as bf16 pairs: the rounded values, and what the rounding left
__device__ __forceinline__ uint32_t split_bf16(float& lo, float& hi) {
  const uint32_t u = pack_bf16(lo, hi);
  lo -= bf16lo(u);
  hi -= bf16hi(u);
  return u;
}
// A pair of weights' leading bf16 parts, and in lo and hi what is left, all above 0 where the weight
// is: cut just below the weight instead of rounded to nearest. An infinite value times any part of
// a weight then has its own sign; times 0 or a negative part it would make the sum NaN. Three such
// parts are a weight's 24 bits exactly: the first leaves at most 2^-7 of it, 17 bits, the second 8
// of them or a power of two.
__device__ __forceinline__ uint32_t cut_bf16(float& lo, float& hi) {
  const uint32_t a = (uint32_t)__viaddmax_s32(__float_as_int(lo), -1, 0);
  const uint32_t b = (uint32_t)__viaddmax_s32(__float_as_int(hi), -1, 0);
  lo -= __uint_as_float(a & 0xffff0000u);
  hi -= __uint_as_float(b & 0xffff0000u);
  return __byte_perm(a, b, 0x7632);
}
constexpr uint32_t kTiny = 0x00010001u;  // a pair of bf16's smallest number above 0
// x within the finite numbers: infinities and NaN become the largest one, of either sign
__device__ __forceinline__ float finite(float x) {
  float y;
  asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(3.4028234663852886e38f));
  return y;
}

// A warp's unit over a bf16 cache. Decode is bound by reading the cache: the tensor cores
// (mma.sync m16n8k16; a unit has at most 16 query rows, far below a tcgen05 tile) are there so
// that 8 queries a K/V head cost no more than one. The 16 rows of A hold 8 heads twice: rows
// 0-7 a value's leading bf16 part, rows 8-15 the part that rounding left, so both halves of
// a product come out of one instruction, in one thread (c0 + c2, c1 + c3). f32 queries and
// their weights take a third part in a second instruction: 24 bits, every product exact.
// bf16 queries are exact in one part; their weights have two. The weights of f32 queries are cut
// into parts that are all above 0 (cut_bf16): rounded to nearest, with infinite values guarded as
// those of bf16 queries are, 64 rows of 3000 positions took 551 us against 480.
// The rows in shared memory may hold more than this head (SideCore): SHAPE is theirs, a tile's
// FIRST the head's first 16-byte piece.
template <typename QT, int HD, typename SHAPE = Shape<uint16_t, HD>>
struct MmaCore {
  static constexpr bool kF32 = sizeof(QT) == 4;
  static constexpr int kHeads = 8;
  static constexpr float kUnit = 1.f;  // what the sums of values are in
  static constexpr int kLoad = HD;    // dimensions of a row in the ring
  static constexpr int kScratch = 0;  // bytes of shared memory of a warp
  static constexpr int kSteps = HD / 16;
  using S = SHAPE;
  static constexpr int K = S::kKeys, NT = K / 8;  // keys of a tile, in eights
  uint32_t q[kF32 ? 3 : 1][kSteps][2];
  f32x2 acc[HD / 8];
  float m, l;

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < HD / 8; ++i) acc[i] = pack2(0.f, 0.f);
    m = neg_inf();
    l = 0.f;
  }
  template <typename At>
  __device__ __forceinline__ void load(const QT* qrow, int live, int lane, float*, At at) {
    const int g = lane >> 2, c = (lane & 3) * 2;
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int d = k * 16 + c + i * 8;
        if constexpr (kF32) {
          float2 x = make_float2(0.f, 0.f);
          if (g < live) x = *reinterpret_cast<const float2*>(qrow + at(g) * HD + d);
          q[0][k][i] = split_bf16(x.x, x.y);
          q[1][k][i] = split_bf16(x.x, x.y);
          q[2][k][i] = pack_bf16(x.x, x.y);
        } else {
          q[0][k][i] = g < live ? *reinterpret_cast<const uint32_t*>(qrow + at(g) * HD + d) : 0u;
        }
      }
  }

  template <int FIRST = 0>
  __device__ __forceinline__ void tile(float scale_log2, uint32_t ks, uint32_t mask, int lane, float*) {
    const uint32_t vs = ks + K * S::kPitch;
    float c[NT][4] = {};
    // B of the first product: K rows as they lie (8 keys x 8 dimensions a matrix)
    const int krow = (lane >> 4) * 8 + (lane & 7), kpiece = (lane >> 3) & 1;
#pragma unroll
    for (int n = 0; n < NT; n += 2) {
      float e[2][4] = {};
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        uint32_t b[4];
        ldmatrix4(ks + n * 8 * S::kPitch + S::at(krow, FIRST + 2 * k + kpiece), b);
        if constexpr (kF32) {
          mma16816(c[n], q[0][k][0], q[1][k][0], q[0][k][1], q[1][k][1], b[0], b[1]);
          mma16816(c[n + 1], q[0][k][0], q[1][k][0], q[0][k][1], q[1][k][1], b[2], b[3]);
          mma16816(e[0], q[2][k][0], 0u, q[2][k][1], 0u, b[0], b[1]);
          mma16816(e[1], q[2][k][0], 0u, q[2][k][1], 0u, b[2], b[3]);
        } else {
          mma16816(c[n], q[0][k][0], 0u, q[0][k][1], 0u, b[0], b[1]);
          mma16816(c[n + 1], q[0][k][0], 0u, q[0][k][1], 0u, b[2], b[3]);
        }
      }
      if constexpr (kF32) {
        // an infinite key's product stands: the parts that are 0 would make it NaN
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (fabsf(c[n + j][i]) != -neg_inf()) c[n + j][i] += c[n + j][2 + i] + e[j][i];
      }
    }
    // this thread: head lane / 4, keys 8 n + 2 (lane % 4) + i
    float mx = m;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint32_t bits = mask >> (n * 8 + (lane & 3) * 2);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        c[n][i] = (bits >> i) & 1u ? c[n][i] * scale_log2 : neg_inf();
        mx = fmaxf(mx, c[n][i]);
      }
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const float ref = finite_or_zero(mx), scale = ex2(m - ref);
    m = mx;
    l *= scale;
    // A of the second product, 16 keys a step: the weights in their parts
    uint32_t a[K / 16][4], e[K / 16][2];
#pragma unroll
    for (int j = 0; j < K / 16; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = ex2(c[2 * j + i][0] - ref), y = ex2(c[2 * j + i][1] - ref);
        l += x + y;
        if constexpr (kF32) {
          a[j][2 * i] = cut_bf16(x, y);
          a[j][2 * i + 1] = cut_bf16(x, y);
          e[j][i] = pack_bf16(x, y);
        } else {
          a[j][2 * i] = split_bf16(x, y);
          a[j][2 * i + 1] = pack_bf16(x, y);
        }
      }
    // B of the second product: V rows transposed on the way in
    const int vrow = ((lane >> 3) & 1) * 8 + (lane & 7), vpiece = lane >> 4;
    const f32x2 scale2 = pack2(scale, scale);
#pragma unroll
    for (int d = 0; d < HD / 16; ++d) {
      float o[2][4] = {};
#pragma unroll
      for (int j = 0; j < K / 16; ++j) {
        uint32_t b[4];
        ldmatrix4_trans(vs + j * 16 * S::kPitch + S::at(vrow, FIRST + 2 * d + vpiece), b);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          mma16816(o[n], a[j][0], a[j][1], a[j][2], a[j][3], b[2 * n], b[2 * n + 1]);
          // the rows beside the third parts: 2^-133, of whose products nothing comes but an infinite
          // value's own sign (with zeros there NaN); 2^-126 of a value is what ex2 may drop anyway
          if constexpr (kF32) mma16816(o[n], e[j][0], kTiny, e[j][1], kTiny, b[2 * n], b[2 * n + 1]);
        }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        // of two parts rounded to nearest (16 bits and a sign) the second may be 0 or negative: where
        // a value is infinite its product with the first one stands
        const f32x2 rest = kF32 ? pack2(o[n][2], o[n][3]) : pack2(finite(o[n][2]), finite(o[n][3]));
        acc[2 * d + n] = fma2(acc[2 * d + n], scale2, add2(pack2(o[n][0], o[n][1]), rest));
      }
    }
  }

  // the unit's outputs, or with PARTIAL its (m, l) and sums
  template <bool PARTIAL, typename OT, typename At>
  __device__ __forceinline__ void end(OT* out, float* lse, float2* ml, int live, int lane, At at) {
    float t = l + __shfl_xor_sync(0xffffffffu, l, 1);
    t += __shfl_xor_sync(0xffffffffu, t, 2);
    const int g = lane >> 2, c = (lane & 3) * 2;
    if (g >= live) return;
    const float inv = PARTIAL ? 1.f : t == 0.f ? 0.f : 1.f / t;
#pragma unroll
    for (int i = 0; i < HD / 8; ++i) {
      const float2 x = unpack2(acc[i]);
      put2(out + at(g) * HD + i * 8 + c, x.x * inv, x.y * inv);
    }
    if ((lane & 3) != 0) return;
    if (PARTIAL) ml[g] = make_float2(m, t);
    else if (lse) lse[at(g)] = log_sum(m, t);
  }
};

// The same with 9 to 16 heads of a K/V head: the 16 rows of A are one head each, and each part
// of a value is an instruction of its own, into the same sums. One pass over the cache instead of
// two: 512 rows of 3000 positions, 16 heads of 128, take 139 us (84% of the measured copy rate), 256
// rows of 4 x 12 heads 255 (91%), 256 rows of 2 x 16 heads with f32 queries 178 (65%). All weights
// are in parts above 0, so two parts (bf16 queries) are within 2^-16 of them. Rounded to nearest
// they would be within 2^-17, but the second part wants sums of its own against infinite values (the
// first case above: 145 us), and these outputs are rounded to 2^-9.
template <typename QT, int HD>
struct WideCore {
  static constexpr bool kF32 = sizeof(QT) == 4;
  static constexpr int kHeads = 16;
  static constexpr float kUnit = 1.f;
  static constexpr int kLoad = HD;
  static constexpr int kSteps = HD / 16, QP = kF32 ? 3 : 1, WP = kF32 ? 3 : 2;  // parts
  static constexpr int kScratch = 0;
  using S = Shape<uint16_t, HD>;
  static constexpr int K = S::kKeys, NT = K / 8;
  uint32_t q[QP][kSteps][4];
  float acc[HD / 8][4];
  float m[2], l[2];  // heads lane / 4, lane / 4 + 8

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < HD / 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    m[0] = m[1] = neg_inf();
    l[0] = l[1] = 0.f;
  }
  template <typename At>
  __device__ __forceinline__ void load(const QT* qrow, int live, int lane, float*, At at) {
    const int c = (lane & 3) * 2;
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int g = (lane >> 2) + (i & 1) * 8, d = k * 16 + c + (i >> 1) * 8;
        if constexpr (kF32) {
          float2 x = make_float2(0.f, 0.f);
          if (g < live) x = *reinterpret_cast<const float2*>(qrow + at(g) * HD + d);
#pragma unroll
          for (int j = 0; j < QP; ++j) q[j][k][i] = split_bf16(x.x, x.y);
        } else {
          q[0][k][i] = g < live ? *reinterpret_cast<const uint32_t*>(qrow + at(g) * HD + d) : 0u;
        }
      }
  }

  __device__ __forceinline__ void tile(float scale_log2, uint32_t ks, uint32_t mask, int lane, float*) {
    const uint32_t vs = ks + K * S::kPitch;
    float c[NT][4] = {};
    const int krow = (lane >> 4) * 8 + (lane & 7), kpiece = (lane >> 3) & 1;
#pragma unroll
    for (int n = 0; n < NT; n += 2) {
      float e[2][4] = {};
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        uint32_t b[4];
        ldmatrix4(ks + n * 8 * S::kPitch + S::at(krow, 2 * k + kpiece), b);
#pragma unroll
        for (int j = 0; j < QP; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            mma16816(j == 0 ? c[n + i] : e[i], q[j][k][0], q[j][k][1], q[j][k][2], q[j][k][3], b[2 * i],
                     b[2 * i + 1]);
      }
      if constexpr (kF32) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (fabsf(c[n + j][i]) != -neg_inf()) c[n + j][i] += e[j][i];
      }
    }
    float scale[2], ref[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float mx = m[h];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint32_t bits = mask >> (n * 8 + (lane & 3) * 2);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float& x = c[n][2 * h + i];
          x = (bits >> i) & 1u ? x * scale_log2 : neg_inf();
          mx = fmaxf(mx, x);
        }
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      ref[h] = finite_or_zero(mx);
      scale[h] = ex2(m[h] - ref[h]);
      m[h] = mx;
      l[h] *= scale[h];
    }
    uint32_t a[WP][K / 16][4];
#pragma unroll
    for (int j = 0; j < K / 16; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // A register i: head (i & 1), keys + 8 (i >> 1)
        const int h = i & 1;
        float x = ex2(c[2 * j + (i >> 1)][2 * h] - ref[h]);
        float y = ex2(c[2 * j + (i >> 1)][2 * h + 1] - ref[h]);
        l[h] += x + y;
#pragma unroll
        for (int w = 0; w < WP - 1; ++w) a[w][j][i] = cut_bf16(x, y);
        a[WP - 1][j][i] = pack_bf16(x, y);
      }
    const int vrow = ((lane >> 3) & 1) * 8 + (lane & 7), vpiece = lane >> 4;
#pragma unroll
    for (int d = 0; d < HD / 16; ++d) {
      float o[2][4] = {};
#pragma unroll
      for (int j = 0; j < K / 16; ++j) {
        uint32_t b[4];
        ldmatrix4_trans(vs + j * 16 * S::kPitch + S::at(vrow, 2 * d + vpiece), b);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int w = 0; w < WP; ++w)
            mma16816(o[n], a[w][j][0], a[w][j][1], a[w][j][2], a[w][j][3], b[2 * n], b[2 * n + 1]);
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[2 * d + n][i] = fmaf(acc[2 * d + n][i], scale[i >> 1], o[n][i]);
    }
  }

  template <bool PARTIAL, typename OT, typename At>
  __device__ __forceinline__ void end(OT* out, float* lse, float2* ml, int live, int lane, At at) {
    const int c = (lane & 3) * 2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float t = l[h] + __shfl_xor_sync(0xffffffffu, l[h], 1);
      t += __shfl_xor_sync(0xffffffffu, t, 2);
      const int g = (lane >> 2) + h * 8;
      if (g >= live) continue;
      const float inv = PARTIAL ? 1.f : t == 0.f ? 0.f : 1.f / t;
#pragma unroll
      for (int i = 0; i < HD / 8; ++i)
        put2(out + at(g) * HD + i * 8 + c, acc[i][2 * h] * inv, acc[i][2 * h + 1] * inv);
      if ((lane & 3) != 0) continue;
      if (PARTIAL) ml[g] = make_float2(m[h], t);
      else if (lse) lse[at(g)] = log_sum(m[h], t);
    }
  }
};

// N neighbouring K/V heads of 32 or 64 dimensions in bf16, up to 8 query heads each, as one unit
// whose rows hold them all. A head of 32 dimensions alone is half of a line, and by the time
// another warp wants the other half it has left the L2 (128 rows of 3000 positions, 8 heads:
// 703 MB read for 393; 256 rows 237 us, in twos 137, in fours 140 and with f32 queries 10 to
// 25% longer); one of 64 is a line, but short pieces of a DRAM page cost more than their bytes
// (256 rows of 3000 positions, 8 heads: 280 us, in twos 251).
template <typename QT, int HD, int N>
struct SideCore {
  static constexpr int kHeads = 8 * N;
  static constexpr float kUnit = 1.f;
  static constexpr int kLoad = N * HD;
  static constexpr int kScratch = 0;
  using S = Shape<uint16_t, kLoad>;
  MmaCore<QT, HD, S> core[N];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N; ++i) core[i].clear();
  }
  template <typename At>
  __device__ __forceinline__ void load(const QT* qrow, int live, int lane, float*, At at) {
#pragma unroll
    for (int i = 0; i < N; ++i) core[i].load(qrow + (size_t)i * (live / N) * HD, live / N, lane, nullptr, at);
  }
  template <int I = 0>
  __device__ __forceinline__ void tile(float scale_log2, uint32_t ks, uint32_t mask, int lane, float*) {
    core[I].template tile<I * HD / 8>(scale_log2, ks, mask, lane, nullptr);
    if constexpr (I + 1 < N) tile<I + 1>(scale_log2, ks, mask, lane, nullptr);
  }
  template <bool PARTIAL, typename OT, typename At>
  __device__ __forceinline__ void end(OT* out, float* lse, float2* ml, int live, int lane, At at) {
    const int g = live / N;
#pragma unroll
    for (int i = 0; i < N; ++i)
      core[i].template end<PARTIAL>(out + (size_t)i * g * HD, lse ? lse + i * g : nullptr,
                                    ml ? ml + i * g : nullptr, g, lane, at);
  }
};

// ---------------------------------------------------------------- f32 cache: FMA
__device__ __forceinline__ void lds2(uint32_t addr, f32x2& a, f32x2& b) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr) : "memory");
}

// A tile is 1024 elements of K and of V whatever the head size. For the scores a lane takes 32
// dimensions of one key (key lane % K, dimensions 32 (lane / K) ..) and all GP heads, the
// queries read from shared memory, where all lanes of a slice read the same address. For
// the sums a lane takes 4 dimensions and 8 of the keys, the weights through shared memory,
// each stored twice (a packed pair).
//
// The reference that weights are taken against moves only when a score passes it by more than kSlack,
// instead of by finding each tile's maximum. A weight may be up to 2^kSlack then; it enters the sums
// of values divided by that (exactly), so they stay in range wherever a softmax's own would, and
// what is written is multiplied by it again.
template <typename QT, int HD, int GP>
struct FmaCore {
  static constexpr int kHeads = GP;
  static constexpr int kLoad = HD;
  using S = Shape<float, HD>;
  static constexpr int K = S::kKeys;              // 8, 16, 32
  static constexpr int SL = 32 / K;               // slices of 32 dimensions of a key
  static constexpr int KS = 128 / HD;             // slices of 8 keys of a tile
  static constexpr int kQPitch = 32 + 4;          // floats of a query slice: apart in banks
  static constexpr int kWPitch = 8 * GP * 2 + 4;  // floats of a key slice's weights
  static constexpr int kScratch = (GP * SL * kQPitch + KS * kWPitch) * 4;  // bytes of a warp
  static constexpr float kSlack = 10.f, kUnit = 1024.f;  // 2^kSlack
  f32x2 acc[GP][2];
  float m[GP], l[GP];

  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ float one(const uint16_t* p) { return bf16lo(*p); }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int h = 0; h < GP; ++h) {
      acc[h][0] = acc[h][1] = pack2(0.f, 0.f);
      m[h] = neg_inf();
      l[h] = 0.f;
    }
  }
  template <typename At>
  __device__ __forceinline__ void load(const QT* qrow, int live, int lane, float* scratch, At at) {
#pragma unroll
    for (int h = 0; h < GP; ++h)
#pragma unroll
      for (int sl = 0; sl < SL; ++sl)
        scratch[(h * SL + sl) * kQPitch + lane] =
            h < live ? one(qrow + at(h) * HD + sl * 32 + lane) : 0.f;
    __syncwarp();
  }

  __device__ __forceinline__ void tile(float scale_log2, uint32_t ks, uint32_t mask, int lane,
                                       float* scratch) {
    const uint32_t vs = ks + K * S::kPitch, qs = smem_u32(scratch);
    float* const sw = scratch + GP * SL * kQPitch;
    const int key = lane % K, sl = lane / K;
    f32x2 d[GP];
#pragma unroll
    for (int h = 0; h < GP; ++h) d[h] = pack2(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      f32x2 k0, k1;
      lds2(ks + S::at(key, sl * 8 + c), k0, k1);
#pragma unroll
      for (int h = 0; h < GP; ++h) {
        f32x2 q0, q1;
        lds2(qs + ((h * SL + sl) * kQPitch + c * 4) * 4, q0, q1);
        d[h] = fma2(q0, k0, d[h]);
        d[h] = fma2(q1, k1, d[h]);
      }
    }
    const bool live = (mask >> key) & 1u;
    float s[GP];
    bool over = false;
#pragma unroll
    for (int h = 0; h < GP; ++h) {
      const float2 x = unpack2(d[h]);
      s[h] = x.x + x.y;
#pragma unroll
      for (int o = K; o < 32; o <<= 1) s[h] += __shfl_xor_sync(0xffffffffu, s[h], o);
      s[h] = live ? s[h] * scale_log2 : neg_inf();
      over |= s[h] > m[h] + kSlack;
    }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int h = 0; h < GP; ++h) {
        float mx = fmaxf(m[h], s[h]);
#pragma unroll
        for (int o = 1; o < K; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float f = ex2(m[h] - finite_or_zero(mx));
        m[h] = mx;
        l[h] *= f;
        const f32x2 f2 = pack2(f, f);
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[h][i] = mul2(acc[h][i], f2);
      }
    }
    // weights: slice key / 8, entry key % 8
    if (sl == 0) {
#pragma unroll
      for (int h = 0; h < GP; ++h) {
        const float w = ex2(s[h] - finite_or_zero(m[h]));
        l[h] += w;
        const float u = w * (1.f / kUnit);
        *reinterpret_cast<float2*>(sw + (key / 8) * kWPitch + ((key % 8) * GP + h) * 2) = make_float2(u, u);
      }
    }
    __syncwarp();
    const int piece = lane % (HD / 4), slice = lane / (HD / 4);
    const uint32_t ws = smem_u32(sw + slice * kWPitch);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f32x2 v0, v1;
      lds2(vs + S::at(slice * 8 + i, piece), v0, v1);
      f32x2 w[GP];
      if constexpr (GP == 1) {
        asm volatile("ld.shared.b64 %0, [%1];" : "=l"(w[0]) : "r"(ws + i * 8) : "memory");
      } else {
#pragma unroll
        for (int h = 0; h < GP; h += 2) lds2(ws + (i * GP + h) * 8, w[h], w[h + 1]);
      }
#pragma unroll
      for (int h = 0; h < GP; ++h) {
        acc[h][0] = fma2(w[h], v0, acc[h][0]);
        acc[h][1] = fma2(w[h], v1, acc[h][1]);
      }
    }
    __syncwarp();
  }

  template <bool PARTIAL, typename OT, typename At>
  __device__ __forceinline__ void end(OT* out, float* lse, float2* ml, int live, int lane, At at) {
#pragma unroll
    for (int h = 0; h < GP; ++h) {
      float t = l[h];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      float2 a = unpack2(acc[h][0]), b = unpack2(acc[h][1]);
#pragma unroll
      for (int o = HD / 4; o < 32; o <<= 1) {
        a.x += __shfl_xor_sync(0xffffffffu, a.x, o);
        a.y += __shfl_xor_sync(0xffffffffu, a.y, o);
        b.x += __shfl_xor_sync(0xffffffffu, b.x, o);
        b.y += __shfl_xor_sync(0xffffffffu, b.y, o);
      }
      if (h >= live) continue;
      const float inv = PARTIAL ? 1.f : t == 0.f ? 0.f : kUnit / t;
      if (lane < HD / 4) {
        put2(out + at(h) * HD + lane * 4, a.x * inv, a.y * inv);
        put2(out + at(h) * HD + lane * 4 + 2, b.x * inv, b.y * inv);
      }
      if (lane != 0) continue;
      if (PARTIAL) ml[h] = make_float2(m[h], t);
      else if (lse) lse[at(h)] = log_sum(m[h], t);
    }
  }
};

// ---------------------------------------------------------------- the kernel
// flags of a tile: begins / ends its run's piece of the unit; that piece has the unit's first
// / last tile
enum : int { kStart = 1, kEnd = 2, kFirst = 4, kLast = 8 };

// SPLIT: not a list of runs, but one unit for each cluster of gridDim.x CTAs, its tiles spread
// evenly over their warps and joined through shared memory at the end: no join kernel and
// no search, for few units.
//
// At least two CTAs an SM are asked for so that registers are not held back further: the
// f32-query kernel takes 255 with the bound of two, 185 without one, and reads 64 sessions of
// 3000 positions in 476 us against 563.
//
// OT: the outputs' type, QT but for sums that are joined with others.
template <typename QT, typename KT, int HD, typename Core, bool SPLIT, Mode MODE, typename OT>
__global__ void __launch_bounds__(SPLIT ? kSplitWarps * 32 : kWarps * 32, SPLIT ? 1 : 2)
    attend_kernel(const __grid_constant__ ParamsOf<MODE> p) {
  using S = Shape<KT, Core::kLoad>;
  constexpr int NW = SPLIT ? kSplitWarps : kWarps, NT = NW * 32;
  constexpr int NS = SPLIT ? split_stages<S::kStage, Core::kScratch> : kStages, K = S::kKeys;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int4 s_desc[NW][NS];  // each stage's tile: row, K/V head, group * 16 + flags, key mask
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int units = p.kv.heads * p.HG;  // units of a row
  const int run = blockIdx.x * NW + warp;
  const int P = p.kv.block_size;
  auto empty_row = [&](int r, int h0, int h1, int i0, int step) {  // a row without a live position
    OT* o = static_cast<OT*>(p.out) + (size_t)r * p.heads * HD;
    for (int i = h0 * HD + i0; i < h1 * HD; i += step) put(o + i, 0.f);
    if (p.lse)
      for (int i = h0 + i0; i < h1; i += step) p.lse[(size_t)r * p.heads + i] = neg_inf();
  };
  pdl_wait();
  pdl_trigger();
  int4 cut = make_int4(0, 0, 0, 0);
  // the warp's tiles: the list's entries [at, stop), the first of them tile t of unit (kvh, hg)
  // of row r; a run of the list is `per` entries
  int r = 0, kvh = 0, hg = 0, t = 0;
  long long at = 0, stop = 0, per = 1, unit_end = LLONG_MAX;
  Row x;
  int2 next_words = make_int2(-1, -1);
  if constexpr (SPLIT) {
    const int u = blockIdx.y % units;
    r = blockIdx.y / units;
    kvh = u / p.HG;
    hg = u % p.HG;
    const int2 words = row_words<MODE>(p, r);
    x = row_of<K, MODE>(p, r, words);
    if (x.nt == 0) {  // the whole cluster's
      const int h0 = kvh * p.G + hg * Core::kHeads;
      if (blockIdx.x == 0 && words.x >= 0 && words.x < p.batch)
        empty_row(r, h0, min(h0 + Core::kHeads, (kvh + 1) * p.G), tid, NT);
      return;
    }
    const long long n = (long long)gridDim.x * NW;
    t = (int)(x.nt * (long long)run / n);
    at = t;
    stop = x.nt * (long long)(run + 1) / n;
  } else {
    if (p.whole) {
      // units [first, last): rows without tiles have units too, of no work
      const long long all = (long long)p.rows * units, from = min((long long)run * p.whole, all);
      unit_end = min(from + p.whole, all);
      if (from < unit_end) {
        r = (int)(from / units);
        int u = (int)(from % units);
        x = row_of<K, MODE>(p, r, row_words<MODE>(p, r));
        while (x.nt == 0 && (long long)(r + 1) * units < unit_end) {
          ++r;
          x = row_of<K, MODE>(p, r, row_words<MODE>(p, r));
          u = 0;
        }
        next_words = row_words<MODE>(p, r + 1);
        kvh = u / p.HG;
        hg = u % p.HG;
        stop = x.nt ? LLONG_MAX : 0;  // ends by unit_end
      }
    } else {
      __shared__ long long s_scan[NW];
      __shared__ long long s_off[NW];  // each run's start, counted from its row's start
      __shared__ int s_row[NW];
      // where each run starts: prefix sums of the rows' costs, a slice of rows per thread
      auto cost = [&](int r) {
        const int nt = row_of<K, MODE>(p, r, row_words<MODE>(p, r)).nt;
        return nt ? (long long)(nt + kUnitCost) * units : 0ll;
      };
      const int slice = (p.rows + NT - 1) / NT;
      const int r0 = min(tid * slice, p.rows), r1 = min(r0 + slice, p.rows);
      long long own = 0;
#pragma unroll 4
      for (int i = r0; i < r1; ++i) own += cost(i);
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
      for (int w = 0; w < NW; ++w) {
        if (w < warp) inc += s_scan[w];
        total += s_scan[w];
      }
      per = (total + p.runs - 1) / p.runs;
      if (per < kMinRun + kUnitCost) per = kMinRun + kUnitCost;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const long long begin = (blockIdx.x * NW + w) * per;
        if (inc - own <= begin && begin < inc) {
          long long at = begin - (inc - own);
          for (int i = r0; i < r1; ++i) {
            const long long c = cost(i);
            if (at < c) {
              s_row[w] = i;
              s_off[w] = at;
              break;
            }
            at -= c;
          }
        }
      }
      __syncthreads();
      const long long begin = run * per;
      stop = min(begin + per, total);
      at = stop;
      if (begin < total) {
        r = s_row[warp];
        x = row_of<K, MODE>(p, r, row_words<MODE>(p, r));
        next_words = row_words<MODE>(p, r + 1);
        const int unit_cost = x.nt + kUnitCost, u = (int)(s_off[warp] / unit_cost);
        const int in = (int)(s_off[warp] % unit_cost);
        kvh = u / p.HG;
        hg = u % p.HG;
        t = max(in - kUnitCost, 0);
        at = begin + (t - (in - kUnitCost));
      }
    }
    // rows of empty requests
    for (int i = run; i < p.rows; i += p.runs) {
      const int2 words = row_words<MODE>(p, i);
      if (words.x < 0 || words.x >= p.batch || words.y >= 0) continue;
      empty_row(i, 0, p.heads, lane, 32);
    }
  }
  Core core;
  core.clear();
  using At = std::conditional_t<MODE == kPrefixes, Bundled, Next>;
  At place{};
  if constexpr (MODE == kPrefixes) place = Bundled{p.row_heads, p.row_skip};
  auto behind = [&](int r) {  // rows from that of the queries to this one
    if constexpr (MODE == kPrefixes) return r >= p.q_rows ? p.q_rows : 0;
    else return 0;
  };
  if (at < stop) {
    // ---- the cursor over the tiles. Table entries are read 32 pages at a time, a lane each,
    // well ahead of their use: ids of pages [base, base + 32), then the 32 that follow, the
    // first 32 of the row (every unit of it begins there) and of the next row.
    //
    // Of a list, entries stand for pages: an id's complement is that of the row's own, newest page,
    // which holds positions behind the row's, and INT_MIN, the complement of no block, that of none.
    auto ids_from = [&](const Row& y, int first) {
      const int page = first + lane;  // past 2^31: a large unsigned number
      if constexpr (MODE == kLists) {
        if (y.nt == 0 || (unsigned)page >= (unsigned)p.list) return INT_MIN;
        const int at = p.pages[(size_t)y.r * p.list + page], newest = y.pos / P;
        if (at < 0 || at > newest || at <= newest - p.W) return INT_MIN;
        const int id = p.table[(size_t)y.b * p.W + (at < p.W ? at : at % p.W)];
        return id < 0 ? INT_MIN : at == newest ? ~id : id;
      }
      if (y.nt == 0 || (unsigned)page > (unsigned)(y.pos / P)) return -1;
      return p.table[(size_t)y.b * p.W + (page < p.W ? page : page % p.W)];
    };
    int base = (x.t0 + t) * K / P, ids = ids_from(x, base), ids_after = ids_from(x, base + 32);
    int ids0 = SPLIT || t == 0 ? ids : ids_from(x, x.t0 * K / P), ids_next = -1;
    bool next_known = SPLIT, more = true, start = true, first = false;
    int issued = 0, n = 0;  // kPrefixes: rows of the unit
    const uint32_t ring = smem_u32(smem) + warp * NS * S::kStage;
    float* const scratch = reinterpret_cast<float*>(smem + NW * NS * S::kStage + warp * Core::kScratch);
    auto issue = [&]() {
      const int s = issued % NS, key = (x.t0 + t) * K + (K < 32 ? lane % K : lane), page = key / P;
      if (!next_known) {  // its words came with this row's: its first pages
        const Row y = row_of<K, MODE>(p, r + 1, next_words);
        ids_next = ids_from(y, y.t0 * K / P);
        next_known = true;
      }
      const int rel = page - base;
      const int id0 = __shfl_sync(0xffffffffu, ids, rel & 31);
      const int id1 = __shfl_sync(0xffffffffu, ids_after, rel & 31);
      int id = rel < 32 ? id0 : id1, kv_head = kvh;
      bool ok;
      if constexpr (MODE == kLists) {
        ok = id >= 0 || key - page * P <= x.pos % P;
        if (id < 0) id = ~id;
        ok = ok && id < p.kv.n_blocks && page < p.list;
        kv_head = r % p.kv_heads;
      } else {
        ok = key >= x.lo && key <= x.pos && id >= 0 && id < p.kv.n_blocks;
      }
      const uint32_t mask = __ballot_sync(0xffffffffu, ok) & (K < 32 ? (1u << (K & 31)) - 1u : ~0u);
      const long long off = ok ? id * p.kv.block_stride + (key - page * P) * p.kv.row_stride +
                                     kv_head * p.kv.head_stride
                               : 0;
      if (t == 0) first = true;
      const bool last = t == x.nt - 1, end = last || at + 1 >= stop;
      if constexpr (MODE == kPrefixes)
        if (start) n = bundle_of<MODE>(p, r);
      if (lane == 0)
        s_desc[warp][s] = make_int4(r, kvh | n << 24, hg * 16 + ((start ? kStart : 0) | (end ? kEnd : 0) |
                                                       (first ? kFirst : 0) | (last ? kLast : 0)),
                                    (int)mask);
      if (start) {  // the unit's queries will be wanted soon
        const int g0 = hg * Core::kHeads, n = min(Core::kHeads, p.G - g0) * HD * (int)sizeof(QT);
        const char* q = static_cast<const char*>(p.q) +
                        ((size_t)(r - behind(r)) * p.heads + (size_t)kvh * p.G + g0) * HD * sizeof(QT);
        if (lane * 128 < n) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + lane * 128));
      }
      if (end && !last && first)  // goes on in the runs that follow
        cut = make_int4(r, kvh * p.G + hg * Core::kHeads,
                        n > 1 ? n * p.G : min(Core::kHeads, p.G - hg * Core::kHeads),
                        (int)((at + (x.nt - t) - 1) / per - run) + 1);
      if (mask) {
        constexpr int CH = S::kPitch / 16;        // 16-byte pieces of a row
        constexpr int RPI = 32 / CH;              // rows of a warp's copy instruction
        const uint32_t dst = ring + s * S::kStage;
        const KT* kb = static_cast<const KT*>(p.kv.k);
        const KT* vb = static_cast<const KT*>(p.kv.v);
        const int c = lane % CH;
#pragma unroll
        for (int i = 0; i < K / RPI; ++i) {
          const int row = i * RPI + lane / CH;
          const long long e = __shfl_sync(0xffffffffu, off, row) + c * (16 / (int)sizeof(KT));
          const bool live = (mask >> row) & 1u;
          cp_async16(dst + S::at(row, c), kb + e, live);
          cp_async16(dst + K * S::kPitch + S::at(row, c), vb + e, live);
        }
      }
      // on to the next tile
      ++issued;
      ++at;
      start = last;
      if (++t == x.nt) {
        if (SPLIT) {
          more = false;
          return;
        }
        t = 0;
        first = false;
        at += kUnitCost;
        bool one_window = x.pos / P - x.t0 * K / P < 32;
        if constexpr (MODE == kLists) one_window = p.list <= 32;
        if (++hg == p.HG) {
          hg = 0;
          if (++kvh == p.kv.heads) {
            kvh = 0;
            // nothing is looked for behind the run's own rows: padding may be long (64 rows and
            // 8000 of padding took 1.42 ms when it was walked, now 0.07 as with the padding in front)
            if (p.whole ? (long long)(r + 1) * units >= unit_end : at >= stop) {
              more = false;
              return;
            }
            ++r;
            x = row_of<K, MODE>(p, r, next_words);
            ids0 = ids_next;
            // empty rows between, 32 at a time (of a run that is not whole units a row follows)
            while (x.nt == 0 && r < p.rows - 1 && (!p.whole || (long long)(r + 1) * units < unit_end)) {
              const int2 words = row_words<MODE>(p, r + 1 + lane);
              const uint32_t some = __ballot_sync(0xffffffffu, row_of<K, MODE>(p, 0, words).nt > 0);
              const int n = some ? __ffs(some) : min(32, p.rows - 1 - r);
              r += n;
              x = row_of<K, MODE>(p, r, make_int2(__shfl_sync(0xffffffffu, words.x, n - 1),
                                                   __shfl_sync(0xffffffffu, words.y, n - 1)));
              ids0 = ids_from(x, x.t0 * K / P);
            }
            next_words = row_words<MODE>(p, r + 1);
            next_known = false;
          }
        }
        base = x.t0 * K / P;
        ids = ids0;
        if (!(one_window && kvh + hg > 0)) ids_after = ids_from(x, base + 32);
      } else if ((x.t0 + t) * K / P - base >= 32) {
        base += 32;
        ids = ids_after;
        ids_after = ids_from(x, base + 32);
      }
      more = at < stop && x.nt > 0 &&
             (!p.whole || (long long)r * units + kvh * p.HG + hg < unit_end);
    };
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) {
      if (more) issue();
      cp_async_commit();
    }
    for (int i = 0; i < issued; ++i) {
      if (more) issue();
      cp_async_commit();
      __syncwarp();
      const int4 d = s_desc[warp][i % NS];
      const int g0 = (d.z >> 4) * Core::kHeads, n = MODE == kPrefixes ? d.y >> 24 : 0;
      const int live = n > 1 ? n * p.G : min(Core::kHeads, p.G - g0);
      const size_t head = (size_t)d.x * p.heads + (size_t)(MODE == kPrefixes ? d.y & 0xffffff : d.y) * p.G + g0;
      if (d.z & kStart) {
        core.clear();
        const size_t q_head = head - (size_t)behind(d.x) * p.heads;
        core.load(static_cast<const QT*>(p.q) + q_head * HD, live, lane, scratch, place);
      }
      cp_async_wait<NS - 1>();
      __syncwarp();
      if (d.w) core.tile(p.scale, ring + (i % NS) * S::kStage, (uint32_t)d.w, lane, scratch);
      __syncwarp();  // the stage is free for the next copy
      if (SPLIT || !(d.z & kEnd)) continue;
      if ((d.z & kFirst) && (d.z & kLast)) {
        core.template end<false>(static_cast<OT*>(p.out) + head * HD, p.lse ? p.lse + head : nullptr,
                                 nullptr, live, lane, place);
      } else {
        const size_t slot = ((size_t)run * 2 + ((d.z & kFirst) ? 1 : 0)) * p.GB;
        core.template end<true>(p.part + slot * HD, nullptr, p.part_ml + slot, live, lane, Next());
      }
    }
  }
  if constexpr (!SPLIT) {
    if (lane == 0 && !p.whole) p.cut[run] = cut;
  } else {
    // ---- join: the warps' sums in this CTA's shared memory (its ring is free), then each CTA
    // of the cluster finishes a share of the outputs from every CTA's sums
    int rows = 1;
    if constexpr (MODE == kPrefixes) rows = bundle_of<MODE>(p, r);
    const int live = rows > 1 ? rows * p.G : min(Core::kHeads, p.G - hg * Core::kHeads), n = live * HD;
    float* const s_sum = reinterpret_cast<float*>(smem);              // [NW][kHeads][HD]
    float* const s_cta = s_sum + NW * Core::kHeads * HD;              // [kHeads][HD]
    float2* const s_ml = reinterpret_cast<float2*>(s_cta + Core::kHeads * HD);  // [NW][kHeads]
    float2* const s_cta_ml = s_ml + NW * Core::kHeads;                // [kHeads]
    __syncthreads();
    core.template end<true>(s_sum + warp * Core::kHeads * HD, nullptr, s_ml + warp * Core::kHeads, live, lane, Next());
    __syncthreads();
    const size_t head = (size_t)r * p.heads + (size_t)kvh * p.G + hg * Core::kHeads;
    auto at_out = [&](int i, int g) {  // element i, of query g, behind the first head
      if constexpr (MODE == kPrefixes) return place(g) * HD + i % HD;
      else return i;
    };
    auto at_lse = [&](int g) {
      if constexpr (MODE == kPrefixes) return place(g);
      else return g;
    };
    const int ctas = gridDim.x;
    for (int i = tid; i < n; i += NT) {
      const int g = i / HD;
      float m = neg_inf(), l = 0.f, a = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) m = fmaxf(m, s_ml[w * Core::kHeads + g].x);
      const float ref = finite_or_zero(m);
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float f = ex2(s_ml[w * Core::kHeads + g].x - ref);
        l += s_ml[w * Core::kHeads + g].y * f;
        a = fmaf(s_sum[w * Core::kHeads * HD + i], f, a);
      }
      if (ctas > 1) {
        s_cta[i] = a;
        if (i % HD == 0) s_cta_ml[g] = make_float2(m, l);
      } else {
        put(static_cast<OT*>(p.out) + head * HD + at_out(i, g),
            l == 0.f ? 0.f : a / l * Core::kUnit);
        if (p.lse && i % HD == 0) p.lse[head + at_lse(g)] = log_sum(m, l);
      }
    }
    if (ctas == 1) return;
    tc::cluster_sync();
    const uint32_t sums = smem_u32(s_cta), mls = smem_u32(s_cta_ml);
    for (int i = blockIdx.x * NT + tid; i < n; i += ctas * NT) {
      const int g = i / HD;
      float m = neg_inf(), l = 0.f, a = 0.f;
      for (int c = 0; c < ctas; ++c) m = fmaxf(m, tc::ld_cluster(tc::mapa(mls + g * 8, c)));
      const float ref = finite_or_zero(m);
#pragma unroll 4
      for (int c = 0; c < ctas; ++c) {
        const float f = ex2(tc::ld_cluster(tc::mapa(mls + g * 8, c)) - ref);
        l += tc::ld_cluster(tc::mapa(mls + g * 8 + 4, c)) * f;
        a = fmaf(tc::ld_cluster(tc::mapa(sums + i * 4, c)), f, a);
      }
      put(static_cast<OT*>(p.out) + head * HD + at_out(i, g),
          l == 0.f ? 0.f : a / l * Core::kUnit);
      if (p.lse && i % HD == 0) p.lse[head + at_lse(g)] = log_sum(m, l);
    }
    tc::cluster_sync();  // no CTA leaves while another reads its sums
  }
}

// Units that were cut: if a unit starts in run c and goes on, its partials -- run c's second
// slot, then the first slot of each run that follows -- are summed in order. A CTA takes
// kJoinWarps consecutive runs (blockIdx.x) and head blockIdx.y of their units. A unit of few
// parts is a warp's, all sixteen at once; one of many parts (a long row over many runs, so
// at most one or two among them) is the whole CTA's: each warp sums a share of the parts.
// All of it is latency, a chain of reads in L2 behind the main kernel's end, so the CTAs are
// held to 64 registers: 1216 cut units of 8 heads want all their warps resident at once.
constexpr int kJoinWarps = 16, kJoinFew = 12;

template <int E>
struct alignas(4 * E) Floats {
  float v[E];
};

// (m, l, a) += the parts [i0, i1) of one head: m and l alike in every lane, a the lane's E
// dimensions. `slot(i)`: where part i is. U sums are in flight, the first of them beside their
// (m, l).
template <int E, int U, typename Slot>
__device__ __forceinline__ void join_parts(const Params& p, int i0, int i1, Slot slot, int lane, float& m,
                                           float& l, float (&a)[E]) {
  auto part = [&](int i) { return *reinterpret_cast<const Floats<E>*>(p.part + slot(i) * (E * 32) + lane * E); };
  for (int b = i0; b < i1; b += 32) {
    const int n = min(i1 - b, 32);
    float2 ml = make_float2(neg_inf(), 0.f);
    if (lane < n) ml = p.part_ml[slot(b + lane)];
    Floats<E> x[U];
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (j < n) x[j] = part(b + j);
    const float mx = fmaxf(m, warp_max(ml.x)), ref = finite_or_zero(mx);
    const float f = ex2(ml.x - ref), old = ex2(m - ref);
    m = mx;
    l = l * old + warp_sum(ml.y * f);
#pragma unroll
    for (int e = 0; e < E; ++e) a[e] *= old;
#pragma unroll 1
    for (int j0 = 0; j0 < n; j0 += U) {
      if (j0 > 0) {
#pragma unroll
        for (int j = 0; j < U; ++j)
          if (j0 + j < n) x[j] = part(b + j0 + j);
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (j0 + j >= n) break;
        const float fj = __shfl_sync(0xffffffffu, f, j0 + j);
#pragma unroll
        for (int e = 0; e < E; ++e) a[e] = fmaf(x[j].v[e], fj, a[e]);
      }
    }
  }
}

template <typename OT, int HD, Mode MODE>
__global__ void __launch_bounds__(kJoinWarps * 32, 2) join_kernel(const __grid_constant__ ParamsOf<MODE> p) {
  constexpr int E = HD / 32;
  __shared__ int4 s_cut[kJoinWarps];
  __shared__ float s_m[kJoinWarps], s_l[kJoinWarps], s_a[kJoinWarps][HD];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = blockIdx.y;
  const int run0 = blockIdx.x * kJoinWarps;
  pdl_wait();
  pdl_trigger();
  auto write = [&](const int4& cut, float m, float l, const float (&a)[E]) {
    size_t head = (size_t)cut.x * p.heads + cut.y + g;
    if constexpr (MODE == kPrefixes) head += Bundled{p.row_heads, p.row_skip}(g) - g;
    const float inv = l == 0.f ? 0.f : p.unit / l;
#pragma unroll
    for (int e = 0; e < E; ++e) put(static_cast<OT*>(p.out) + head * HD + lane * E + e, a[e] * inv);
    if (p.lse && lane == 0) p.lse[head] = log_sum(m, l);
  };
  auto slots_of = [&](int run) {
    return [=](int i) { return ((size_t)(run + i) * 2 + (i == 0 ? 1 : 0)) * p.GB + g; };
  };
  int4 own = make_int4(0, 0, 0, 0);
  if (run0 + warp < p.runs) own = p.cut[run0 + warp];
  const bool many = g < own.z && own.w > kJoinFew;
  if (g < own.z && !many) {
    float m = neg_inf(), l = 0.f, a[E] = {};
    join_parts<E, 4>(p, 0, own.w, slots_of(run0 + warp), lane, m, l, a);
    write(own, m, l, a);
  }
  if (lane == 0) s_cut[warp] = many ? own : make_int4(0, 0, 0, 0);
  if (!__syncthreads_or(many)) return;
  for (int c = 0; c < kJoinWarps; ++c) {
    const int4 cut = s_cut[c];
    if (cut.w == 0) continue;
    float m = neg_inf(), l = 0.f, a[E] = {};
    join_parts<E, 6>(p, (int)((long long)cut.w * warp / kJoinWarps),
                     (int)((long long)cut.w * (warp + 1) / kJoinWarps), slots_of(run0 + c), lane, m, l, a);
    if (lane == 0) {
      s_m[warp] = m;
      s_l[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s_a[warp][lane * E + e] = a[e];
    __syncthreads();
    if (warp == 0) {
      m = neg_inf();
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, s_m[w]);
      const float ref = finite_or_zero(m);
      l = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) a[e] = 0.f;
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) {
        const float f = ex2(s_m[w] - ref);
        l += s_l[w] * f;
#pragma unroll
        for (int e = 0; e < E; ++e) a[e] = fmaf(s_a[w][lane * E + e], f, a[e]);
      }
      write(cut, m, l, a);
    }
    __syncthreads();
  }
}

// How a call is launched, from what the host knows: the shapes, and how long a row may be.
struct Choice {
  int side;                // K/V heads of a unit (SideCore), or 1
  int unit_heads;          // query heads of a unit, at most
  int units_of_kv;         // units of a K/V head (or of `side` of them)
  long long units, tiles;  // units of all rows, tiles of a unit, at most
  int split;               // CTAs of a unit in a split launch, or 0
  bool whole;              // runs of whole units
  size_t workspace;
};

// A split launch's CTAs per unit for `units` units of up to `tiles` tiles, or 0 for a launch of
// runs. Measured (head_dim 128, bf16): one row of 8 K/V heads takes 5.8 / 6.6 / 9.9 / 23 us
// split at 16 / 1000 / 4000 / 16000 positions against 9.4 / 16.0 / 16.2 / 23 us in runs, and
// 136 against 92 us at 131071; 16 rows of 1000 positions 15.4 against 21.2 us. But 16 rows
// of 1 to 16000 take 132 against 46 us: a split launch lasts as long as its longest unit. So
// several rows are split up to 8 tiles a warp (1024 positions of one CTA), one row up to 24, half
// more than where the two meet, as a row is seldom as long as its table allows (3 K/V heads whose
// table allows 25000 positions: 8.6 us split and 12.3 in runs at 3000, 31.1 and 20.9 at 24951;
// f32, whose tiles take longer: 8), or up to 128 where the clusters fill three quarters of the
// card (32 K/V heads: 5.5 / 7.9 / 19 / 53 / 99 us at 16 / 1000 / 4000 / 16000 / 32768
// positions against 8.5 / 13 / 23 / 53 / 92).
inline int split_ctas(long long units, long long tiles, int rows, bool bf16, int sms) {
  if (units > sms) return 0;
  int c = 1;
  // clusters that are all resident: with one CTA an SM 15 clusters of eight fit this card at
  // once, 36 of four, 76 of two; a sixteenth cluster of eight waits for the others (16 units
  // of 16 positions took 8.8 us in eights, 5.6 in fours)
  while (c < 8 && (units + 4) * c * 2 <= sms) c *= 2;
  // every warp of the cluster a tile at least
  while (c > 1 && (long long)c * kSplitWarps > tiles * 2) c /= 2;
  const long long most = tiles / (c * kSplitWarps);  // tiles of a warp, at most
  const bool full = 4 * units * c >= 3 * sms;        // the clusters fill the card
  return most <= (rows > 1 ? 8 : full ? 128 : bf16 ? 24 : 8) ? c : 0;
}

// bundle: rows whose queries are one unit's (g * bundle at most eight)
inline Choice choose(const rq_paged_kv& kv, int rows, int heads, int max_blocks, int window, int bundle = 1) {
  Choice x{};
  const int g = heads / kv.heads;
  const bool bf16 = kv.dtype == RQ_BF16;
  const int most = bf16 ? 16 : 8;  // query heads of a unit
  long long keys = (long long)max_blocks * kv.block_size;
  if (keys > INT_MAX) keys = INT_MAX;
  if (window > 0 && window < keys) keys = window;
  const int row_bytes = kv.head_dim * (bf16 ? 2 : 4), tile = 4096 / row_bytes < 32 ? 4096 / row_bytes : 32;
  x.side = 1;
  x.unit_heads = g < most ? g * bundle : most;
  x.units_of_kv = (g + most - 1) / most;
  x.units = (long long)rows * kv.heads * x.units_of_kv;
  x.tiles = keys / tile + 2;
  x.split = split_ctas(x.units, x.tiles, rows, bf16, sm_count());
  // rows of at most eight whole tiles: no search and no join (182 rows of up to 192 positions,
  // head_dim 64, 12.9 us with them and 8.4 without; longer units would be uneven shares)
  x.whole = !x.split && x.tiles <= 10;
  x.workspace = 0;
  if (x.split || x.whole) return x;
  // runs that the memory bounds: two heads at a time where they lie side by side
  if (bf16 && bundle == 1 && kv.head_dim < 128 && g <= 8 && kv.head_stride == kv.head_dim && kv.heads % 2 == 0) {
    x.side = 2;
    x.unit_heads = 2 * g;
    x.units /= 2;
    x.tiles = keys / (2048 / (2 * kv.head_dim)) + 2;
  }
  x.workspace = workspace_bytes(x.unit_heads, kv.head_dim);
  return x;
}

template <typename QT, typename KT, int HD, typename Core, Mode MODE = kRows, typename OT = QT>
cudaError_t launch(ParamsOf<MODE> p, const Choice& x, cudaStream_t s) {
  using S = Shape<KT, Core::kLoad>;
  cudaError_t e;
  if (x.unit_heads > Core::kHeads) return cudaErrorInvalidValue;
  p.HG = x.units_of_kv;
  p.GB = x.unit_heads;
  p.unit = Core::kUnit;
  if constexpr (Core::kLoad == HD) {  // units of one K/V head
    if (x.split) {
      auto* kernel = attend_kernel<QT, KT, HD, Core, true, MODE, OT>;
      constexpr size_t ring = (size_t)kSplitWarps *
                              (split_stages<S::kStage, Core::kScratch> * S::kStage + Core::kScratch);
      constexpr size_t sums = (size_t)(kSplitWarps + 1) * Core::kHeads * (HD * 4 + 8);
      constexpr size_t smem = ring > sums ? ring : sums;
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
      return launch_dependent(kernel, dim3((unsigned)x.split, (unsigned)x.units, 1), kSplitWarps * 32, smem, x.split,
                              s, p);
    }
  }
  // as many CTAs as are resident at once, at most as many as the largest rows could fill
  auto* kernel = attend_kernel<QT, KT, HD, Core, false, MODE, OT>;
  constexpr size_t smem = (size_t)kWarps * (kStages * S::kStage + Core::kScratch);
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  static std::atomic<int> resident[kMaxDevices];
  int ctas = 0;
  if ((e = resident_ctas(kernel, kWarps * 32, smem, resident, &ctas)) != cudaSuccess) return e;
  if (ctas > kMaxGrid) ctas = kMaxGrid;
  if (x.whole) {
    const long long runs = (long long)ctas * kWarps, share = (x.units + runs - 1) / runs;
    if (share > INT_MAX) return cudaErrorInvalidValue;
    p.whole = (int)share;
    p.runs = (int)((x.units + share - 1) / share);
    const int grid = (p.runs + kWarps - 1) / kWarps;
    p.runs = grid * kWarps;
    return launch_dependent(kernel, dim3((unsigned)grid), kWarps * 32, smem, 0, s, p);
  }
  const long long most = (x.tiles * x.units + kWarps * kMinRun - 1) / (kWarps * kMinRun);
  const int grid = (int)(ctas < most ? ctas : most);
  p.runs = grid * kWarps;
  if ((e = launch_dependent(kernel, dim3((unsigned)grid), kWarps * 32, smem, 0, s, p)) != cudaSuccess) return e;
  const dim3 joins((unsigned)((p.runs + kJoinWarps - 1) / kJoinWarps), (unsigned)p.GB, 1);
  return launch_dependent(join_kernel<OT, HD, MODE>, joins, kJoinWarps * 32, 0, 0, s, p);
}

// a launch's scratch in its workspace
inline void place(Params& p, const Choice& x, void* workspace) {
  char* ws = static_cast<char*>(workspace);
  p.part = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + part_bytes(x.unit_heads, p.kv.head_dim));
  p.cut = reinterpret_cast<int4*>(ws + part_bytes(x.unit_heads, p.kv.head_dim) + ml_bytes(x.unit_heads));
}

// over a bf16 cache, over an f32 cache; with lists; with f32 outputs whatever the queries are; and of rows
// over prefixes too
cudaError_t launch_bf16(const Params& p, const Choice& x, bool q_bf16, cudaStream_t s);
cudaError_t launch_f32(const Params& p, const Choice& x, bool q_bf16, cudaStream_t s);
cudaError_t launch_lists_bf16(const MoreParams& p, const Choice& x, bool q_bf16, cudaStream_t s);
cudaError_t launch_lists_f32(const MoreParams& p, const Choice& x, bool q_bf16, cudaStream_t s);
cudaError_t launch_sums_bf16(const Params& p, const Choice& x, bool q_bf16, cudaStream_t s);
cudaError_t launch_prefixes_bf16(const MoreParams& p, const Choice& x, bool q_bf16, cudaStream_t s);
cudaError_t launch_prefixes_f32(const MoreParams& p, const Choice& x, bool q_bf16, cudaStream_t s);

}  // namespace paged_attn
}  // namespace rqk
