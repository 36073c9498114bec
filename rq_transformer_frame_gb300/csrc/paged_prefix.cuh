// paged_prefix.cuh -- attention of groups of rows over a prefix that each group shares, on the tcgen05
// tensor cores: the kernel template (include/rq.h, rq_paged_prefix_attention; launched by
// paged_prefix.cu, instantiated by paged_prefix_bf16.cu and paged_prefix_f32.cu).
//
// The queries that read a K/V head's keys are those of all rows of a group: rows x G of them, one
// matrix product with the prefix. For a tile of keys
//   S = Q K^T (f32 in tensor memory), P = 2^(scale S - ref), O += P V, l += sum P,
// ref a running bound of the maximum: it moves, and O and l are scaled, only when a score passes it. It
// is set kSlack above the maximum met, so that P stays at most 1 and sums in range, and is a whole number, so
// that what is scaled is scaled exactly.
//
// A unit is (group, K/V head, 128 queries). All units' tiles, of 128 keys for bf16 queries and 64 for f32
// ones, form one list, cut into equal runs, a CTA each, one CTA an SM. A unit inside one run leaves its sums in row order; of a unit
// that is cut each piece leaves (ref, l, O) in its CTA's scratch, and paged_prefix.cu joins them with
// the rows' own requests.
//
// A CTA is 12 warps (168 registers a thread, of which the bf16-query kernels spill 4 to 24 bytes; with 13 it is
// 128, and spills that miss the little L1 beside 227 KB of shared memory):
//   0-7       softmax. Scores come in two streams, each with its S and P in tensor memory, that take
//             turns by tiles. All eight warps form one stream's P, two threads a row, while the tensor
//             cores work for the other, and add the other's O before they hand P over. (Four warps a stream
//             came into step: both at P, then both at their products, 48 us where either alone took 26)
//   8, 9      the loaders: K and V rows by the block table into a ring, in the swizzled layouts that
//             the tensor cores read (K with dimensions inside, V with dimensions outside: the same
//             rows, read transposed). Blocks of a multiple of eight positions come by TMA, a lane
//             a box; rows of other blocks by 16-byte cp.async
//   10, 11    issue the tensor cores' work, a stream each: S of the next tile behind O of this one,
//             in order: it takes the place of the P that O is made of. (One warp for both streams:
//             2800 cycles a tile, 900 of them its waits)
//
// bf16 queries enter as they are, f32 queries and all P in three bf16 parts (24 bits, every product exact),
// smallest first. The tensor cores cut the sum after each product of 16 terms, towards 0: a bias that
// grows with the sum's length, so O is a tile's alone and the tiles are added in registers, rounded to
// nearest (in one O the cuts of 20 tiles were 2.6e-6 of the result, now it is within 3.3e-7 whatever the
// length). The first two parts are cut, not rounded to nearest, so that all three are of the value's sign
// and an infinite key or value is met by no zero part. P lies in tensor memory, in the columns of the S it
// was made of.
//
// What bounds it: a tile of 128 queries and 128 keys is 32 products of 64 cycles (24 of them P's three parts),
// 1.1 us, beside the softmax, some 3000 cycles or 1.5 us: 410 for scores and maxima, 130 for the exchange of
// these, 1850 for exponentials (1024 of the unit that makes them) and parts, 420 for sums, the rest waits. A
// loader is busy for 2600 of them with blocks of 16 positions. 64 rows of 32 heads over 8 K/V heads behind
// 32768 positions, two units a head: 58 us, 27 tiles a CTA, tensor pipe 53% of the time; the second unit's
// keys come from HBM again (243 MB of 134). One O for all tiles of a piece, two parts of P and 256 queries a unit
// took 1.15 us a tile, 47 us in all, and was off by 1e-4 behind 50000 positions.
#pragma once

#include <type_traits>

#include "paged_attn.cuh"

namespace rqk {
namespace prefix {

using paged_attn::cp_async16;
using paged_attn::cp_async_commit;
using paged_attn::cp_async_wait;
using paged_attn::cut_bf16;
using paged_attn::ex2;
using paged_attn::finite_or_zero;
using paged_attn::neg_inf;
using paged_attn::pack_bf16;

constexpr int kThreads = 384, kLoaders = 64;
constexpr int kRows = 128;       // queries of a unit
// What a tile, and a unit's start and end count in the list: between what is best for bf16 and for f32 queries (250
// rows of five groups with bf16 ones, 64 rows behind 2500 positions with f32 ones: 192 and 57.7 us where a unit
// counts 9, 185 and 57.5 with 12, 180 and 58.9 with 16, 177 and 59.6 with 20)
constexpr int kTileCost = 2, kUnitCost = 14;
constexpr float kSlack = 8.f;
constexpr int kMasks = 8;        // tiles whose masks are kept
// columns of tensor memory: the two streams' scores, and P's first two parts, at 0 and 128; O; P's third parts
constexpr int kSumsAt = 256, kThirdAt = 384;

struct alignas(16) Group {  // what the joining kernel needs of a group
  long long list0;          // its first entry of the list
  int row0, queries, tiles;
};

struct Params {
  rq_paged_kv kv;
  const void* q;
  const int32_t *table, *cu_rows, *prefix_requests, *prefix_lens;
  int rows, heads, batch, W, groups, G;
  float scale;      // |scale| times log2 e
  uint32_t flip;    // 1: the scale is negative, queries enter negated
  float* whole;     // [rows][heads][HD] sums of units of one run
  float2* whole_ml; // [rows][heads] (ref, l)
  float* part;      // [ctas][2][HD / 4][kRows][4]
  float2* part_ml;  // [ctas][2][kRows]
  Group* group;     // [groups]
  long long* per;   // entries of a run
  uint32_t* gave_up;  // [ctas] 1: a wait of the CTA ran out, 0: none did
  unsigned long long wait_ns;  // after which one does
  int stall;        // a test's: the CTA whose loaders load nothing, or -1
  int box;          // rows of a TMA box, 0: copies by threads
  CUtensorMap kmap, vmap;  // [block][head][row][dimension]
};

template <typename QT, int HD>
struct Shape {
  static constexpr bool kF32 = sizeof(QT) == 4;
  static constexpr int kQParts = kF32 ? 3 : 1, kPParts = 3;
  static constexpr int KT = kF32 ? 64 : 128;           // keys of a tile
  static constexpr int kHalf = KT * HD * 2;            // bytes of a tile's keys, or values
  static constexpr int kQ = kQParts * kRows * HD * 2;  // of the queries
  static constexpr int kRoom = (224 * 1024 - kQ) / kHalf;
  static constexpr int NH = kRoom < 8 ? kRoom : 8;     // halves of the ring
  static constexpr int kRing = kQ + NH * kHalf;
  // a row's bytes in shared memory: 64 dimensions, or all 32
  static constexpr int kPitch = HD < 64 ? 64 : 128;
  static_assert(NH >= 5, "two tiles and the next one's keys");
  // where 16-byte piece c of row r of R rows lies
  template <int R>
  static __device__ __forceinline__ int at(int r, int c) {
    if constexpr (HD < 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    return (c >> 3) * (R * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
  }
};

// A pair of weights' leading bf16 parts, cut towards 0, and in p what is left, and 2^-126 with it: above 0
// where the weight is, however few bits that has. (cut_bf16 cuts just below the weight instead, by three
// more instructions of the busiest pipe a pair.)
__device__ __forceinline__ uint32_t cut_part(f32x2& p) {
  const float2 x = unpack2(p);
  uint32_t u;
  asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(x.y), "f"(x.x));
  const float tiny = 1.17549435e-38f;
  p = add2(add2(p, pack2(-bf16lo(u), -bf16hi(u))), pack2(tiny, tiny));
  return u;
}

// ---------------------------------------------------------------- tensor memory
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
// what was loaded is there; passing the values through keeps their uses behind it
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
      "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
      "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
      "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
      :
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// One lane of the warp. With a lane chosen by comparing lane numbers the compiler does not know that it is
// one alone, and each tensor instruction becomes a loop over lanes.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_from_tmem(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Shared-memory matrix descriptor (tc_common.cuh has the fields) of rows of 128 or 64 bytes in the
// swizzle of that size: SBO between groups of eight rows, LBO between the 64-dimension
// halves where dimensions are the outer ones.
template <int PITCH>
__device__ __forceinline__ uint64_t desc(uint32_t saddr, uint32_t lbo) {
  return (uint64_t)((saddr >> 4) & 0x3fffu) | (uint64_t)((lbo >> 4) & 0x3fffu) << 16 |
         (uint64_t)((8 * PITCH) >> 4) << 32 | (uint64_t)1u << 46 | (uint64_t)(PITCH == 128 ? 2u : 4u) << 61;
}
// Between threads' writes and the tensor cores' reads of them. Behind copies the reader has it: a
// loader's own would wait for all of its copies in flight.
__device__ __forceinline__ void fence_proxy_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// one arrival once this thread's copies so far have landed
__device__ __forceinline__ void arrive_behind_copies(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// A box of a 4-D tensor map into 16-byte aligned shared memory. x times the element size is a multiple
// of 16 bytes; what lies past an extent is filled with zeros.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int row, int head, int block,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(row), "r"(head), "r"(block), "r"(smem_u32(bar))
      : "memory");
}

// ---------------------------------------------------------------- units and pieces
// A group as the list has it. tiles: key tiles [t0, t0 + tiles) of request b, live positions [lo, end)
struct View {
  int row0, queries, b, lo, end, t0, tiles;
};

template <int KT>
__device__ __noinline__ View view_of(const Params& p, int g) {
  View v{};
  v.row0 = min(max(p.cu_rows[g], 0), p.rows);
  const int row1 = min(max(p.cu_rows[g + 1], v.row0), p.rows);
  v.b = p.prefix_requests[g];
  v.end = p.prefix_lens[g];
  if (row1 == v.row0 || v.b < 0 || v.b >= p.batch || v.end < 1) return v;
  v.queries = (row1 - v.row0) * p.G;
  const int P = p.kv.block_size, first = (v.end - 1) / P - p.W + 1;
  v.lo = max(first, 0) * P;
  v.t0 = v.lo / KT;
  v.tiles = (v.end - 1) / KT - v.t0 + 1;
  return v;
}

// what a group's units of a K/V head count in the list
struct Costs {
  long long unit, head;
};

__host__ __device__ __forceinline__ Costs costs_of(int queries, int tiles) {
  if (tiles == 0) return Costs{0, 0};
  const long long unit = (long long)tiles * kTileCost + kUnitCost;
  return Costs{unit, ((queries - 1) / kRows + 1) * unit};
}

struct Small {  // behind the tiles
  uint64_t full[8], empty[8], q_full, s_full[2], p_full[2], o_full, drain;
  uint32_t mask[kMasks][4];
  float row[2][2][kRows];  // of halves of a row, for its other half: [stream][half], maxima, then sums
  long long scan[kThreads / 32], start0;
  int start_group;
  View start_view;
  uint32_t tmem;
  volatile int abort;
};

template <typename QT, int HD>
constexpr size_t smem_bytes = Shape<QT, HD>::kRing + sizeof(Small);
static_assert(smem_bytes<uint16_t, 128> <= 227 * 1024 && smem_bytes<float, 128> <= 227 * 1024, "a CTA's shared memory");

struct Piece {
  View v;
  int h, unit, t, n;  // K/V head, unit of it, tiles [t, t + n)
  bool first, last;
};

// a CTA's walk over its run, the same in every thread
template <int KT>
struct Cursor {
  long long at, stop, list0;
  int g, of;  // the group, and that of `v`
  View v;
  // To the start of the CTA's run: prefix sums of the groups' costs, a slice of the groups a thread. False
  // where the list ends before.
  __device__ __noinline__ bool start(const Params& p, Small& s) {
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int slice = (p.groups + kThreads - 1) / kThreads;
    const int g0 = min(tid * slice, p.groups), g1 = min(g0 + slice, p.groups);
    long long own = 0;
    View seen{};
#pragma unroll 1
    for (int i = g0; i < g1; ++i) {
      seen = view_of<KT>(p, i);
      own += costs_of(seen.queries, seen.tiles).head * p.kv.heads;
    }
    long long inc = own;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) s.scan[warp] = inc;
    __syncthreads();
    long long total = 0;
#pragma unroll 1
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) inc += s.scan[w];
      total += s.scan[w];
    }
    const long long per = max((total + gridDim.x - 1) / gridDim.x, (long long)(kUnitCost + kTileCost));
    at = blockIdx.x * per;
    stop = min(at + per, total);
    long long first = inc - own;
    if (blockIdx.x == 0 && tid == 0) *p.per = per;
    if (blockIdx.x == 0 || (first <= at && at < inc)) {
#pragma unroll 1
      for (int i = g0; i < g1; ++i) {
        const View v = slice == 1 ? seen : view_of<KT>(p, i);
        const long long c = costs_of(v.queries, v.tiles).head * p.kv.heads;
        if (blockIdx.x == 0) p.group[i] = Group{first, v.row0, v.queries, v.tiles};
        if (first <= at && at < first + c) s.start_group = i, s.start0 = first, s.start_view = v;
        first += c;
      }
    }
    __syncthreads();
    g = of = s.start_group;
    list0 = s.start0;
    v = s.start_view;
    return at < total;
  }
  __device__ __noinline__ bool next(const Params& p, Piece& x) {
    while (at < stop && g < p.groups) {
      if (of != g) v = view_of<KT>(p, of = g);
      x.v = v;
      const Costs c = costs_of(x.v.queries, x.v.tiles);
      const long long cost = c.head * p.kv.heads;
      if (at >= list0 + cost) {
        list0 += cost;
        ++g;
        continue;
      }
      long long in = at - list0;
      x.h = (int)(in / c.head);
      in -= x.h * c.head;
      x.unit = (int)(in / c.unit);
      in -= x.unit * c.unit;
      const long long begin = at - in;  // the unit's first entry
      x.t = in <= kUnitCost ? 0 : (int)((in - kUnitCost + kTileCost - 1) / kTileCost);
      at = begin + c.unit;
      if (x.t >= x.v.tiles) continue;
      const long long room = stop - begin - kUnitCost - (long long)x.t * kTileCost;
      if (room <= 0) return false;  // its first tile is the next run's
      x.n = (int)min((room + kTileCost - 1) / kTileCost, (long long)(x.v.tiles - x.t));
      x.first = x.t == 0;
      x.last = x.t + x.n == x.v.tiles;
      return true;
    }
    return false;
  }
};

// out of line, as is all that runs once a piece: 140 KB of code took 8 us to arrive at each launch
static __device__ __noinline__ bool slow_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
  if (*abort) return false;
  if (mbar_wait_for(bar, parity, limit_ns)) return true;
  *abort = 1;
  return false;
}

// A unit's queries into shared memory by the 256 softmax threads, negated where the scale is negative (the
// scores then have its size alone); rows that are not there are 0. bf16 ones are copied, all copies in
// flight at once, and are there once the caller has waited for them; f32 ones are cut into parts.
template <typename QT, int HD>
__device__ __noinline__ void load_queries(const Params& p, const Piece& x, uint8_t* smem, int tid) {
  using S = Shape<QT, HD>;
  constexpr int CH = HD / 8, STEP = 2 * kRows / CH, kAhead = 4;
  const int c = tid % CH, last = x.v.queries - 1 - x.unit * kRows;
  // the query's row and head of the group, step by step
  const int first = x.unit * kRows + tid / CH, rows_step = STEP / p.G, heads_step = STEP % p.G;
  int row = first / p.G, head = first % p.G;
  const QT* base = static_cast<const QT*>(p.q) + ((size_t)x.v.row0 * p.heads + (size_t)x.h * p.G) * HD + c * 8;
  auto next = [&] {
    const QT* q = base + ((size_t)row * p.heads + head) * HD;
    row += rows_step;
    head += heads_step;
    if (head >= p.G) head -= p.G, ++row;
    return q;
  };
  if constexpr (!S::kF32) {
#pragma unroll 2
    for (int r = tid / CH; r < kRows; r += STEP) {
      const QT* q = next();
      cp_async16(smem_u32(smem) + S::template at<kRows>(r, c), r <= last ? q : base, r <= last);
    }
    cp_async_commit();
  } else {
    const uint32_t flip = p.flip ? 0x80008000u : 0u;
#pragma unroll 1
    for (int r0 = tid / CH; r0 < kRows; r0 += STEP * kAhead) {
      uint4 v[kAhead][2];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const QT* q = next();
        if (r0 + k * STEP > last) q = base;  // of a row that is there, not used
        v[k][0] = reinterpret_cast<const uint4*>(q)[0];
        v[k][1] = reinterpret_cast<const uint4*>(q)[1];
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int r = r0 + k * STEP;
        if (r >= kRows) break;
        uint8_t* to = smem + S::template at<kRows>(r, c);
        const uint32_t f[8] = {v[k][0].x, v[k][0].y, v[k][0].z, v[k][0].w, v[k][1].x, v[k][1].y, v[k][1].z, v[k][1].w};
        uint32_t o[3][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float lo = __uint_as_float(f[2 * e] & 0x7fffffffu), hi = __uint_as_float(f[2 * e + 1] & 0x7fffffffu);
          const uint32_t sign = (__byte_perm(f[2 * e], f[2 * e + 1], 0x7632) & 0x80008000u) ^ flip;
          o[0][e] = cut_bf16(lo, hi) ^ sign;
          o[1][e] = cut_bf16(lo, hi) ^ sign;
          o[2][e] = pack_bf16(lo, hi) ^ sign;
        }
#pragma unroll
        for (int j = 0; j < 3; ++j)
          *reinterpret_cast<uint4*>(to + j * kRows * HD * 2) =
              r <= last ? make_uint4(o[j][0], o[j][1], o[j][2], o[j][3]) : make_uint4(0, 0, 0, 0);
      }
    }
  }
}

// ... and once they are there
template <typename QT, int HD>
__device__ __noinline__ void queries_loaded(const Params& p, uint8_t* smem, int tid) {
  using S = Shape<QT, HD>;
  if constexpr (!S::kF32) {
    cp_async_wait<0>();
    if (p.flip) {
      constexpr int CH = HD / 8;
      for (int r = tid / CH; r < kRows; r += 2 * kRows / CH) {
        uint4* v = reinterpret_cast<uint4*>(smem + S::template at<kRows>(r, tid % CH));
        v->x ^= 0x80008000u, v->y ^= 0x80008000u, v->z ^= 0x80008000u, v->w ^= 0x80008000u;
      }
    }
  }
  fence_proxy_async();
}

// BOX: blocks come by TMA
template <typename QT, int HD, bool BOX>
__global__ void __launch_bounds__(kThreads, 1) prefix_kernel(const __grid_constant__ Params p) {
  using S = Shape<QT, HD>;
  constexpr int KT = S::KT, NH = S::NH;
  extern __shared__ __align__(1024) uint8_t smem[];
  Small& s = *reinterpret_cast<Small*>(smem + S::kRing);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_trigger();

  Cursor<KT> cur;
  if (!cur.start(p, s)) {
    if (tid == 0) p.gave_up[blockIdx.x] = 0;
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < NH; ++i) {
      mbar_init(&s.full[i], BOX ? 1 : kLoaders + kLoaders / 32);
      mbar_init(&s.empty[i], 2);  // both streams
    }
    mbar_init(&s.q_full, 2 * kRows);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.s_full[i], 2);
      mbar_init(&s.p_full[i], 2 * kRows);
    }
    mbar_init(&s.o_full, 1);
    mbar_init(&s.drain, 2);
    fence_barrier_init();
    s.abort = (smem_u32(smem) & 1023u) != 0;  // the swizzles go by the address
  }
  if (warp == 10) {
    tc::tmem_alloc(&s.tmem, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s.tmem;
  // of a warp, all of whose lanes go on or none; a wait that runs out ends the CTA's work: its sums
  // become NaN, and it says so
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity & 1u))) return true;
    return __all_sync(0xffffffffu, slow_wait(bar, parity & 1u, &s.abort, p.wait_ns)) != 0;
  };
  Piece x;

  if ((warp == 8 || warp == 9) && BOX) {
    // ------------------------------------------------------------ loaders: TMA, one the keys, one the values
    // Lane i has box i of a half (a copy takes some 110 cycles of its warp, 16 of them are a tile's keys of
    // blocks of 16 positions): rows [g BR, g BR + BR) of the tile, 64 dimensions (or all 32). A box is
    // of one page; where that has no block it is read past the last one and filled with zeros. What
    // lies in a box behind the prefix's end must not be read, so that box's rows are copied by the warp.
    constexpr int kSubs = HD < 64 ? 1 : HD / 64;
    const int BR = p.box, box_log = __ffs(BR) - 1, nb = KT >> box_log, g = lane & (nb - 1), sub = lane / nb;
    const int P = p.kv.block_size, step_pages = KT / P % p.W, step_rows = KT % P;
    const uint32_t ring = smem_u32(smem) + S::kQ;
    const int side = warp - 8;
    const CUtensorMap* const map = side == 0 ? &p.kmap : &p.vmap;
    int tile = 0;
    bool ok = (int)blockIdx.x != p.stall;
    if (lane == 0) tc::prefetch_tmap(map);
    while (ok && cur.next(p, x)) {
      // the lane's box's first key, column of the table and row of the block, a tile ahead. Divided once a piece:
      // with divisions every tile a loader, which has 16 copies of 110 cycles to make for one, took 3200 cycles
      const int32_t* const table = p.table + (size_t)x.v.b * p.W;
      int ahead = (x.v.t0 + x.t) * KT + g * BR, column = ahead / P % p.W, in_block = ahead % P;
      auto id_of = [&](int t) { return t >= x.n || ahead < x.v.lo || ahead >= x.v.end ? -1 : table[column]; };
      int next = id_of(0);
      for (int t = 0; ok && t < x.n; ++t, ++tile) {
        const int key0 = (x.v.t0 + x.t + t) * KT, key = key0 + g * BR, id = next, at_row = in_block;
        ahead += KT;
        in_block += step_rows;
        column += step_pages;
        if (in_block >= P) in_block -= P, ++column;
        if (column >= p.W) column -= p.W;
        next = id_of(t + 1);
        const bool live = id >= 0 && id < p.kv.n_blocks;
        const uint32_t boxes = __ballot_sync(0xffffffffu, live) & (nb < 32 ? (1u << nb) - 1u : ~0u);
        const uint32_t torn = __ballot_sync(0xffffffffu, live && x.v.end - key < BR) & boxes;
        if (side == 0 && lane < KT / 32) {
          uint32_t m = BR >= 32 && ((boxes >> (lane * 32 >> box_log)) & 1u) ? ~0u : 0u;
#pragma unroll 1
          for (int r = 0; BR < 32 && r < 32; r += BR)
            if ((boxes >> ((lane * 32 + r) >> box_log)) & 1u) m |= ((1u << BR) - 1u) << r;
          const int left = x.v.end - key0 - lane * 32;  // keys of the word
          s.mask[tile % kMasks][lane] = left >= 32 ? m : left <= 0 ? 0u : m & ((1u << left) - 1u);
        }
        const int half = 2 * tile + side, slot = half % NH;
        if (half >= NH && !(ok = wait_warp(&s.empty[slot], half / NH - 1))) break;
        if (torn) {
          const int b = __ffs(torn) - 1, r0 = key0 + b * BR, rows = x.v.end - r0;
          const long long at = __shfl_sync(0xffffffffu, id, b) * p.kv.block_stride + x.h * p.kv.head_stride +
                               (r0 % P) * p.kv.row_stride;
          const uint16_t* from = static_cast<const uint16_t*>(side == 0 ? p.kv.k : p.kv.v) + at;
#pragma unroll 1
          for (int i = lane; i < BR * (HD / 8); i += 32) {
            const int r = i / (HD / 8), c = i % (HD / 8);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < rows) v = *reinterpret_cast<const uint4*>(from + r * p.kv.row_stride + c * 8);
            *reinterpret_cast<uint4*>(smem + S::kQ + slot * S::kHalf + S::template at<KT>(b * BR + r, c)) = v;
          }
          fence_proxy_async();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&s.full[slot], (uint32_t)((nb - (torn ? 1 : 0)) * BR * HD * 2));
        __syncwarp();
        if (sub < kSubs && !((torn >> g) & 1u))
          tma_load_4d(ring + slot * S::kHalf + sub * (KT * 128) + g * BR * S::kPitch, map, sub * 64, live ? at_row : 0,
                      x.h, live ? id : p.kv.n_blocks, &s.full[slot]);
      }
    }
    // whatever happened: nothing lands behind the CTA's end
#pragma unroll 1
    for (int i = max(tile - NH / 2 - 1, 0); i < tile; ++i) {
      const int half = 2 * i + side;
      if (half >= 2 * tile - NH) mbar_wait(&s.full[half % NH], (uint32_t)(half / NH) & 1u);
    }
  } else if ((warp == 8 || warp == 9) && !BOX) {
    // ------------------------------------------------------------ loaders: copies
    constexpr int RW = KT / 2;          // rows of a warp
    constexpr int RL = RW / 32;         // of them a lane looks up
    constexpr int CH = HD / 8;          // 16-byte pieces of a row
    constexpr int RPI = 32 / CH;        // rows of a warp's copy instruction
    const int w = warp - 8, P = p.kv.block_size;
    const uint32_t ring = smem_u32(smem) + S::kQ;
    int half = 0, tile = 0;
    bool ok = (int)blockIdx.x != p.stall;
    while (ok && cur.next(p, x)) {
      const uint16_t* kb = static_cast<const uint16_t*>(p.kv.k) + x.h * p.kv.head_stride;
      const uint16_t* vb = static_cast<const uint16_t*>(p.kv.v) + x.h * p.kv.head_stride;
      auto key_of = [&](int t, int i) { return (x.v.t0 + x.t + t) * KT + w * RW + i * 32 + lane; };
      auto id_of = [&](int t, int i) {
        const int key = key_of(t, i), page = key / P;
        if (t >= x.n || key < x.v.lo || key >= x.v.end) return -1;
        return p.table[(size_t)x.v.b * p.W + (page < p.W ? page : page % p.W)];
      };
      int next[RL];
#pragma unroll
      for (int i = 0; i < RL; ++i) next[i] = id_of(0, i);
      for (int t = 0; ok && t < x.n; ++t, ++tile) {
        uint32_t mask[RL];
        long long off[RL];
#pragma unroll
        for (int i = 0; i < RL; ++i) {
          const int id = next[i];
          next[i] = id_of(t + 1, i);
          const bool live = id >= 0 && id < p.kv.n_blocks;
          mask[i] = __ballot_sync(0xffffffffu, live);
          if (lane == 0) s.mask[tile % kMasks][w * RL + i] = mask[i];
          off[i] = live ? id * p.kv.block_stride + (key_of(t, i) % P) * p.kv.row_stride : 0;
        }
#pragma unroll
        for (int side = 0; side < 2; ++side) {
          const int slot = half % NH;
          if (half >= NH && !(ok = wait_warp(&s.empty[slot], half / NH - 1))) break;
          const uint32_t dst = ring + slot * S::kHalf;
          const uint16_t* base = side == 0 ? kb : vb;
          const int c = lane % CH;
#pragma unroll
          for (int i = 0; i < RW / RPI; ++i) {
            const int r = i * RPI + lane / CH;
            const long long e = __shfl_sync(0xffffffffu, off[i * RPI / 32], r % 32);
            cp_async16(dst + S::template at<KT>(w * RW + r, c), base + e + c * 8, (mask[i * RPI / 32] >> (r % 32)) & 1u);
          }
          ++half;
          arrive_behind_copies(&s.full[slot]);
          if (lane == 0) mbar_arrive(&s.full[slot]);  // the mask's
        }
      }
    }
    cp_async_commit();
    cp_async_wait<0>();
  } else if (warp == 8 || warp == 9) {
  } else if (warp >= 10) {
    // ------------------------------------------------------------ tensor cores
    // The whole warp walks along, so that addresses stay in uniform registers; one lane issues. Loops
    // that stay loops: unrolled, the instructions came late, once each in 3000 cycles.
    const int st = warp - 10;
    const uint32_t qs = smem_u32(smem), ring = qs + S::kQ, ts = tmem + st * 128, to = tmem + kSumsAt;
    const uint32_t is = tc::idesc_bf16_f32(kRows, KT);
    const uint32_t io = tc::idesc_bf16_f32(kRows, HD) | 1u << 16;  // B: dimensions outside
    constexpr int kSub = HD < 64 ? 2 : 4;  // steps of 16 dimensions of a row in shared memory
    int base = 0, made = 0, piece = 0;
    bool ok = true;
    auto behind = [&] {
      if (!BOX) fence_proxy_async();
      tc::fence_after_sync();
    };
    while (ok && cur.next(p, x)) {
      // Each half is passed by both streams, also where only one reads it, in its turn: a barrier's parity
      // tells two uses of a slot apart, and a stream that went on to the next use while the other's half
      // were still on its way would take that one's phase for its own.
      auto pass = [&](int t) {
#pragma unroll 1
        for (int half = base + 2 * t; half < base + 2 * t + 2; ++half) {
          if (!wait_warp(&s.full[half % NH], half / NH)) return false;
          if (lane == 0) mbar_arrive(&s.empty[half % NH]);
          __syncwarp();
        }
        return true;
      };
      ok = wait_warp(&s.q_full, piece);
#pragma unroll 1
      for (int t = st - 2; ok && t < x.n; t += 2) {
        if (t >= 0) {  // O of tile t
          const int half = base + 2 * t + 1;
          if (t > 0 && !(ok = pass(t - 1))) break;
          if (!(ok = wait_warp(&s.full[half % NH], half / NH) && wait_warp(&s.p_full[st], made))) break;
          ++made;
          behind();
          if (elect_one()) {
            uint32_t acc = 0;
#pragma unroll 1
            for (int part = S::kPParts - 1; part >= 0; --part) {
              uint64_t v = desc<S::kPitch>(ring + (half % NH) * S::kHalf, KT * 128);
              uint32_t at = part < 2 ? ts + 16 * part : tmem + kThirdAt + st * 64;
#pragma unroll 1
              for (int i = 0; i < KT / 32; ++i) {
                mma_from_tmem(to, at, v, io, acc);
                mma_from_tmem(to, at + 8, v + ((16 * S::kPitch) >> 4), io, 1);
                v += (32 * S::kPitch) >> 4;
                at += part < 2 ? 32 : 16;
                acc = 1;
              }
            }
            tc::commit(&s.empty[half % NH]);
            tc::commit(&s.o_full);
          }
          __syncwarp();
        }
        if (t + 2 < x.n) {  // S of this stream's next one
          const int half = base + 2 * (t + 2);
          if (!(ok = wait_warp(&s.full[half % NH], half / NH))) break;
          behind();
          if (elect_one()) {
            uint64_t q = desc<S::kPitch>(qs + (S::kQParts - 1) * (kRows * HD * 2), 16);
#pragma unroll 1
            for (int part = S::kQParts - 1; part >= 0; --part) {
              const uint64_t k = desc<S::kPitch>(ring + (half % NH) * S::kHalf, 16);
#pragma unroll 1
              for (int sub = 0; sub < HD / 16 / kSub; ++sub)
#pragma unroll
                for (int i = 0; i < kSub; ++i)
                  tc::mma_bf16(ts, q + ((sub * (kRows * 128) + i * 32) >> 4), k + ((sub * (KT * 128) + i * 32) >> 4), is,
                               part < S::kQParts - 1 || sub + i > 0);
              q -= (kRows * HD * 2) >> 4;
            }
            tc::commit(&s.empty[half % NH]);
            tc::commit(&s.s_full[st]);
            mbar_arrive(&s.s_full[st]);  // passes on what the loaders wrote beside the tile
          }
          __syncwarp();
        }
      }
      if (ok && ((x.n - 1) & 1) != st) ok = pass(x.n - 1);
      base += 2 * x.n;
      ++piece;
    }
    if (elect_one()) tc::commit(&s.drain);
    __syncwarp();
    // whatever happened: tensor memory is given back behind it
    if (!mbar_wait(&s.drain, 0)) s.abort = 1;
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    // Warps w and w + 4 share rows (and tensor memory lanes): each has half of a tile's keys, and of O's
    // dimensions.
    constexpr int C = KT / 64;  // 32 keys at a time
    const int side = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16), to = lanes + kSumsAt + side * (HD / 2);
    const f32x2 scale2 = pack2(p.scale, p.scale);
    uint32_t seen[2] = {0, 0};  // tiles of a stream
    int tile = 0;
    bool ok = true;
    Piece y;
    bool more = cur.next(p, y);
    auto queries = [&] {
      load_queries<QT, HD>(p, y, smem, tid);
      queries_loaded<QT, HD>(p, smem, tid);
      mbar_arrive(&s.q_full);
    };
    if (more) queries();
    while (more) {
      x = y;
      float ref = neg_inf(), l = 0.f;
      constexpr int D = HD / 2;
      float o[D] = {};  // sums of the tiles so far
      uint32_t r[32];
      // the sums of the tile before, times f
      auto add_tile = [&](float f) {
        if (ok) ok = wait_warp(&s.o_full, tile - 1);
        tc::fence_after_sync();
        if constexpr (D >= 32) {
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            tmem_ld32(to + c, r);
            tmem_wait_ld(r);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[c + e] = fmaf(__uint_as_float(r[e]), f, o[c + e]);
          }
        } else {
          float v[16];
          tc::tmem_ld16(to, v);
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = fmaf(v[e], f, o[e]);
        }
      };
#pragma unroll 1
      for (int j = 0; j < x.n; ++j, ++tile) {
        const int st = j & 1;
        const uint32_t ts = lanes + st * 128;
        // (a partner warp whose wait ran out is still met at the barrier below)
        if (ok) ok = wait_warp(&s.s_full[st], st ? seen[1]++ : seen[0]++);
        tc::fence_after_sync();
        auto scores = [&](int c) {
          tmem_ld32(ts + (side * C + c) * 32, r);
          tmem_wait_ld(r);
          const uint32_t m = s.mask[tile % kMasks][side * C + c];
          if (m == 0xffffffffu) return;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!((m >> i) & 1u)) r[i] = 0xff800000u;
        };
        float mx = neg_inf();
#pragma unroll
        for (int c = 0; c < C; ++c) {
          scores(c);
          float m0 = neg_inf(), m1 = neg_inf();
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            m0 = fmaxf(fmaxf(m0, __uint_as_float(r[i])), __uint_as_float(r[i + 1]));
            m1 = fmaxf(fmaxf(m1, __uint_as_float(r[i + 2])), __uint_as_float(r[i + 3]));
          }
          mx = fmaxf(mx, fmaxf(m0, m1));
        }
        s.row[st][side][row] = mx;
        bar_sync(1 + (warp & 3), 64);
        mx = fmaxf(mx, s.row[st][side ^ 1][row]);
        mx = mx == neg_inf() ? mx : mx * p.scale;
        float f = 1.f;
        if (__any_sync(0xffffffffu, mx > ref)) {
          const float was = ref;
          if (mx > was) ref = ceilf(mx) + kSlack;  // whole: sums are scaled exactly
          if (ref > was) f = ex2(was - ref);
          l *= f;
#pragma unroll
          for (int e = 0; e < D; ++e) o[e] *= f;
        }
        const f32x2 sub2 = pack2(-finite_or_zero(ref), -finite_or_zero(ref));
        f32x2 sum2 = pack2(0.f, 0.f);
        // P, two parts over the scores, the third one behind them; the scores read last are still there
#pragma unroll
        for (int c = C - 1; c >= 0; --c) {
          if (c < C - 1) scores(c);
          uint32_t w[32], w3[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float2 y = unpack2(fma2(pack2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), scale2, sub2));
            f32x2 p2 = pack2(ex2(y.x), ex2(y.y));
            sum2 = add2(sum2, p2);
            w[i] = cut_part(p2);
            w[16 + i] = cut_part(p2);
            y = unpack2(p2);
            w3[i] = pack_bf16(y.x, y.y);
          }
          tmem_st32(ts + (side * C + c) * 32, w);
          tmem_st16(lanes + kThirdAt + st * 64 + (side * C + c) * 16, w3);
        }
        const float2 sum = unpack2(sum2);
        l += sum.x + sum.y;
        // the products of this tile go where those of the one before are
        if (j > 0) add_tile(f);
        tmem_wait_st();
        tc::fence_before_sync();
        mbar_arrive(&s.p_full[st]);
      }
      // ---- the piece's sums
      bar_sync(1 + (warp & 3), 64);  // the last maxima have been read
      s.row[0][side][row] = l;
      bar_sync(1 + (warp & 3), 64);
      l += s.row[0][side ^ 1][row];
      more = cur.next(p, y);
      add_tile(1.f);
      // the unit's products are done: the next one's first scores are made while its sums are written
      if (more) queries();
      if (!ok) ref = 0.f, l = __int_as_float(0x7fc00000);
      const bool cut = !(x.first && x.last);
      const size_t slot = (size_t)blockIdx.x * 2 + (x.first ? 1 : 0);
      const int i = x.unit * kRows + row;  // of the group
      if (i < x.v.queries) {
        const size_t head = (size_t)(x.v.row0 + i / p.G) * p.heads + (size_t)x.h * p.G + i % p.G;
        float* out = cut ? p.part + slot * kRows * HD + row * 4 : p.whole + head * HD;
        const size_t step = cut ? kRows * 4 : 4;  // floats from four dimensions to the next four
        if (side == 0) *(cut ? p.part_ml + slot * kRows + row : p.whole_ml + head) = make_float2(ref, l);
#pragma unroll
        for (int e = 0; e < D / 4; ++e)
          *reinterpret_cast<float4*>(out + (side * (HD / 8) + e) * step) =
              make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 10) tc::tmem_dealloc(tmem, 512);
  if (tid == 0) p.gave_up[blockIdx.x] = s.abort != 0;
}

// The TMA boxes of a cache: p.box and the maps, or box 0 where there are none for it. Rows of a box: the
// most of a power of two that divides a block and the tile.
inline cudaError_t set_maps(Params& p, int tile) {
  p.box = 0;
  if (p.kv.block_size % 8 != 0) return cudaSuccess;
  int box = 8;
  while (box < tile && p.kv.block_size % (2 * box) == 0) box *= 2;
  static std::atomic<void*> fn{nullptr};
  void* f = fn.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !f) return cudaErrorNotSupported;
    fn.store(f, std::memory_order_release);
  }
  const int hd = p.kv.head_dim;
  const cuuint64_t extent[4] = {(cuuint64_t)hd, (cuuint64_t)p.kv.block_size, (cuuint64_t)p.kv.heads,
                                (cuuint64_t)p.kv.n_blocks};
  // the stride of an extent of one is never used; a map takes none of 0
  auto bytes = [&](int64_t stride, int64_t n) { return (cuuint64_t)(n > 1 ? stride : hd) * 2; };
  const cuuint64_t stride[3] = {bytes(p.kv.row_stride, p.kv.block_size), bytes(p.kv.head_stride, p.kv.heads),
                                bytes(p.kv.block_stride, p.kv.n_blocks)};
  for (cuuint64_t x : stride)
    if (x == 0 || x >= 1ull << 40) return cudaSuccess;  // rows that are one, or too far apart: copies
  const cuuint32_t dims[4] = {(cuuint32_t)(hd < 64 ? hd : 64), (cuuint32_t)box, 1, 1}, ones[4] = {1, 1, 1, 1};
  auto encode = reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(f);
  for (int i = 0; i < 2; ++i)
    if (encode(i == 0 ? &p.kmap : &p.vmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, i == 0 ? p.kv.k : p.kv.v, extent, stride,
               dims, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
               hd < 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaSuccess;
  p.box = box;
  return cudaSuccess;
}

template <typename QT, int HD>
cudaError_t launch(Params p, int ctas, cudaStream_t s) {
  cudaError_t err = set_maps(p, Shape<QT, HD>::KT);
  if (err != cudaSuccess) return err;
  auto* kernel = p.box ? prefix_kernel<QT, HD, true> : prefix_kernel<QT, HD, false>;
  err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<QT, HD>);
  if (err != cudaSuccess) return err;
  return launch_dependent(kernel, dim3((unsigned)ctas), kThreads, smem_bytes<QT, HD>, 0, s, p);
}

cudaError_t launch_bf16(const Params& p, int ctas, cudaStream_t s);  // bf16 queries
cudaError_t launch_f32(const Params& p, int ctas, cudaStream_t s);   // f32 queries

}  // namespace prefix
}  // namespace rqk
