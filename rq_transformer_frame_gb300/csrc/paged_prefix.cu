// paged_prefix.cu -- attention over a prefix that a group of rows shares and over each row's own
// request (include/rq.h, rq_paged_prefix_attention).
//
// Where the cache is bf16 and there is work for it, paged_prefix.cuh multiplies all queries of a group with
// its prefix at once, and the rows' own requests are paged_attn.cuh's work, with f32 outputs. Else both
// parts of every row are that, as two rows of one launch. Then all parts of a row are joined: with o_i, lse_i
// of a part, lse = log sum e^lse_i and o = sum e^(lse_i - lse) o_i. All parts are f32, the output is
// rounded once. The last launch of a call leaves its status in the workspace's first word.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "paged_prefix.cuh"

namespace rqk {
namespace {

using paged_attn::finite_or_zero;
using paged_attn::neg_inf;
using paged_attn::put;

struct MergeParams {
  const int32_t* requests;
  int rows, heads, batch, hd;
  const float *o1, *o2, *lse1, *lse2;  // prefix, own
  void* out;
  float* lse;
  int32_t* status;
};

template <typename OT>
__global__ void __launch_bounds__(256) merge_kernel(const __grid_constant__ MergeParams p) {
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;  // nothing waits in this form
  const int warps = gridDim.x * 8;
  for (long long i = (long long)blockIdx.x * 8 + threadIdx.x / 32; i < (long long)p.rows * p.heads; i += warps) {
    const int r = (int)(i / p.heads), lane = threadIdx.x % 32;
    const int b = p.requests ? p.requests[r] : r;
    if (b < 0 || b >= p.batch) continue;
    const float a = p.lse1[i], c = p.lse2[i];
    const float m = finite_or_zero(fmaxf(a, c));
    const float x = a == neg_inf() ? 0.f : expf(a - m), y = c == neg_inf() ? 0.f : expf(c - m);
    const float sum = x + y;
    for (int d = lane; d < p.hd; d += 32) {
      const size_t at = (size_t)i * p.hd + d;
      float o = 0.f;
      if (a != neg_inf()) o = x * p.o1[at];
      if (c != neg_inf()) o += y * p.o2[at];
      put(static_cast<OT*>(p.out) + at, sum == 0.f ? 0.f : o / sum);
    }
    if (p.lse && lane == 0) p.lse[i] = sum == 0.f ? neg_inf() : m + logf(sum);
  }
}

// The prefix kernel's pieces and the own request's part of each query. A lane has one query -- those of
// a K/V head one after another, as they lie in the pieces -- and four dimensions, eight pieces in flight.
// (32 dimensions of each query a CTA: 64 CTAs of all 128 took 24 us for 2048 queries of 10 pieces.)
struct JoinParams {
  prefix::Params t;
  const int32_t* requests;
  const float *own, *own_lse;
  void* out;
  float* lse;
  int32_t* status;
  int ctas;
};

constexpr int kJoinWarps = 8;

template <typename OT, int HD>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ JoinParams p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % 32, four = blockIdx.y * kJoinWarps + threadIdx.x / 32;
  if (blockIdx.x == 0 && four == 0) {
    uint32_t gave_up = 0;
    for (int i = lane; i < p.ctas; i += 32) gave_up |= p.t.gave_up[i];
    gave_up = __any_sync(0xffffffffu, gave_up != 0);
    if (lane == 0) *p.status = gave_up ? RQ_PAGED_TIMEOUT : 0;
  }
  const uint32_t of_head = (uint32_t)p.t.rows * p.t.G, idx = blockIdx.x * 32 + lane;
  if (idx >= of_head * p.t.kv.heads) return;
  const int h = idx / of_head, in = idx % of_head, r = in / p.t.G, g = in % p.t.G;
  const size_t head = (size_t)r * p.t.heads + (size_t)h * p.t.G + g;
  const int b = p.requests ? p.requests[r] : r;
  const float own = p.own_lse[head] * 1.4426950408889634f;
  const float4 own_o = *reinterpret_cast<const float4*>(p.own + head * HD + four * 4);
  const long long per = *p.t.per;
  if (b < 0 || b >= p.t.batch) return;
  // the query's pieces, `count` of them: the first at ml[0] and part[0], the others one run after another
  int count = 0;
  const float2 *ml = nullptr, *ml_rest = nullptr;
  const float *part = nullptr, *part_rest = nullptr;
  size_t ml_step = 0, part_step = 0;
  {
    const int of = paged_attn::group_of(p.t.cu_rows, p.t.groups, r);
    if (of >= 0) {
      const prefix::Group x = p.t.group[of];
      if (x.tiles > 0) {
        const int i = (r - x.row0) * p.t.G + g, u = i / prefix::kRows, at = i % prefix::kRows;
        const prefix::Costs c = prefix::costs_of(x.queries, x.tiles);
        const long long first = x.list0 + h * c.head + u * c.unit + prefix::kUnitCost;
        const long long c0 = first / per;
        count = (int)((first + (long long)(x.tiles - 1) * prefix::kTileCost) / per - c0) + 1;
        ml_step = 2 * prefix::kRows;
        part_step = ml_step * HD;
        const size_t slot = (size_t)c0 * 2 * prefix::kRows;
        const size_t in_part = (size_t)four * (prefix::kRows * 4) + at * 4;
        if (count == 1) {
          ml = p.t.whole_ml + head;
          part = p.t.whole + head * HD + four * 4;
        } else {
          ml = p.t.part_ml + slot + prefix::kRows + at;
          part = p.t.part + (slot + prefix::kRows) * HD + in_part;
        }
        ml_rest = p.t.part_ml + slot + at;
        part_rest = p.t.part + slot * HD + in_part;
      }
    }
  }
  // from the own request's part on; four pieces at once, the last one again in place of those behind it
  float m = own, sum = own == neg_inf() ? 0.f : 1.f;
  float o[4] = {sum * own_o.x, sum * own_o.y, sum * own_o.z, sum * own_o.w};
  if (own == neg_inf()) o[0] = o[1] = o[2] = o[3] = 0.f;
  for (int c0 = 0; c0 < count; c0 += 4) {
    float2 x[4];
    float4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = min(c0 + j, count - 1);
      x[j] = *(c == 0 ? ml : ml_rest + c * ml_step);
      v[j] = *reinterpret_cast<const float4*>(c == 0 ? part : part_rest + c * part_step);
    }
    float next = m;
#pragma unroll
    for (int j = 0; j < 4; ++j) next = fmaxf(next, x[j].x);
    const float ref = finite_or_zero(next), old = exp2f(m - ref);
    m = next;
    sum *= old;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] *= old;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (c0 + j >= count) break;
      const float f = exp2f(x[j].x - ref);
      sum = fmaf(x[j].y, f, sum);
      o[0] = fmaf(v[j].x, f, o[0]), o[1] = fmaf(v[j].y, f, o[1]);
      o[2] = fmaf(v[j].z, f, o[2]), o[3] = fmaf(v[j].w, f, o[3]);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  OT* out = static_cast<OT*>(p.out) + head * HD + four * 4;
  paged_attn::put2(out, o[0] * inv, o[1] * inv);
  paged_attn::put2(out + 2, o[2] * inv, o[3] * inv);
  if (p.lse && four == 0) p.lse[head] = sum == 0.f ? neg_inf() : (m + log2f(sum)) * 0.6931471805599453f;
}

constexpr size_t kHead = 256;  // bytes of the workspace for the status, in front
// what rq_paged_set_wait_limit set
std::atomic<unsigned long long> g_wait_ns{0};
std::atomic<int> g_stall{-1};

struct Layout {
  paged_attn::Choice x;
  bool tc;         // prefixes by matrix products
  int ctas;        // of the prefix kernel
  int bundle;      // else: rows of a group whose queries are a unit's
  size_t o, lse, part, part_ml, group, gave_up, bytes;
};

Layout layout_of(const rq_paged_kv& kv, int rows, int heads, int max_blocks, int groups) {
  using paged_attn::align256;
  Layout l{};
  const size_t hd = kv.head_dim;
  // What the tables allow all rows to read for themselves, in bytes: a launch over few short rows is over
  // before the prefix kernel has its first tile (8 rows of 16 heads, 64 dimensions, 200 positions before 40:
  // 20 us against 22).
  const double most = 4.0 * rows * kv.heads * hd * max_blocks * kv.block_size;
  l.tc = groups > 0 && kv.dtype == RQ_BF16 && most > 32e6;
  if (l.tc || groups == 0) {
    l.x = paged_attn::choose(kv, rows, heads, max_blocks, 0);
  } else {
    // the rows' own, and a bundle of them each over a prefix: that is the work, but all are rows of the launch
    const int g = heads / kv.heads;
    l.bundle = std::min(g <= 8 ? 8 / g : 1, rows);
    l.x = paged_attn::choose(kv, rows + (rows + l.bundle - 1) / l.bundle, heads, max_blocks, 0, l.bundle);
    l.x.units = 2ll * rows * kv.heads * l.x.units_of_kv;
  }
  l.o = align256((size_t)rows * heads * hd * sizeof(float));
  l.lse = align256((size_t)rows * heads * sizeof(float2));
  l.ctas = std::max(sm_count(), 1);
  l.part = align256((size_t)l.ctas * 2 * prefix::kRows * hd * sizeof(float));
  l.part_ml = align256((size_t)l.ctas * 2 * prefix::kRows * sizeof(float2));
  l.group = align256((size_t)groups * sizeof(prefix::Group)) + 256;
  l.gave_up = align256((size_t)l.ctas * sizeof(uint32_t));
  l.bytes = kHead + 2 * (l.o + l.lse) + l.x.workspace + (l.tc ? l.part + l.part_ml + l.group + l.gave_up : 0);
  return l;
}

rq_status check(const rq_paged_kv* kv, int32_t rows, int32_t heads, int32_t max_blocks, int32_t groups) {
  const rq_status st = paged_kv_check(kv);
  if (st != RQ_OK) return st;
  if (rows < 0 || heads < 1 || heads % kv->heads != 0 || max_blocks < 1 || groups < 0) return RQ_ERR_ARG;
  // a row is two rows of a launch
  if (rows > 1 << 29 || heads > 1 << 23 || (long long)rows * heads > 1 << 30 || groups > 1 << 16)
    return RQ_ERR_UNSUPPORTED;
  return RQ_OK;
}

}  // namespace
}  // namespace rqk

extern "C" rq_status rq_paged_set_wait_limit(uint64_t limit_ns, int32_t stall) {
  if (stall < -1) return RQ_ERR_ARG;
  rqk::g_wait_ns.store(limit_ns, std::memory_order_relaxed);
  rqk::g_stall.store(stall, std::memory_order_relaxed);
  return RQ_OK;
}

extern "C" size_t rq_paged_prefix_attention_workspace_size(const rq_paged_kv* kv, int32_t rows,
                                                           int32_t heads, int32_t max_blocks,
                                                           int32_t groups) {
  using namespace rqk;
  if (check(kv, rows, heads, max_blocks, groups) != RQ_OK || rows < 1) return 0;
  return layout_of(*kv, rows, heads, max_blocks, groups).bytes;
}

extern "C" rq_status rq_paged_prefix_attention(const rq_paged_kv* kv, int32_t rows, int32_t heads,
                                               int32_t batch, int32_t max_blocks,
                                               const int32_t* block_table, const int32_t* requests,
                                               const int32_t* positions, int32_t groups,
                                               const int32_t* cu_rows,
                                               const int32_t* prefix_requests,
                                               const int32_t* prefix_lens, float scale,
                                               int32_t q_dtype, const void* q, void* out, float* lse,
                                               void* workspace, size_t workspace_bytes,
                                               void* cuda_stream) {
  using namespace rqk;
  const rq_status st = check(kv, rows, heads, max_blocks, groups);
  if (st != RQ_OK) return st;
  const float scale_log2 =
      (float)((scale != 0.f ? (double)scale : 1.0 / std::sqrt((double)kv->head_dim)) * 1.4426950408889634);
  if (batch < 1 || !std::isfinite(scale_log2)) return RQ_ERR_ARG;
  if (q_dtype != RQ_F32 && q_dtype != RQ_BF16) return RQ_ERR_ARG;
  if (rows == 0) return RQ_OK;
  if (!requests && rows > batch) return RQ_ERR_ARG;
  if (!block_table || !positions || !q || !out || !workspace) return RQ_ERR_ARG;
  if (groups > 0 && (!cu_rows || !prefix_requests || !prefix_lens)) return RQ_ERR_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace)) return RQ_ERR_ARG;
  const bool qb = q_dtype == RQ_BF16;
  const Layout l = layout_of(*kv, rows, heads, max_blocks, groups);
  if (workspace_bytes < l.bytes) return RQ_ERR_ARG;
  char* ws = static_cast<char*>(workspace);
  auto take = [&](size_t n) {
    char* at = ws;
    ws += n;
    return at;
  };
  int32_t* const status = reinterpret_cast<int32_t*>(take(kHead));
  // [2][rows][heads][head_dim] sums and [2][rows][heads] lse: of the prefixes, of the rows' own requests
  float* const o = reinterpret_cast<float*>(take(2 * l.o));
  float* const ls = reinterpret_cast<float*>(take(2 * l.lse));
  float* const own_o = o + (size_t)rows * heads * kv->head_dim;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  paged_attn::MoreParams p{};
  p.kv = *kv;
  p.q = q;
  p.table = block_table;
  p.requests = requests;
  p.positions = positions;
  p.rows = rows;
  p.heads = heads;
  p.batch = batch;
  p.W = max_blocks;
  p.G = heads / kv->heads;
  p.scale = scale_log2;
  paged_attn::place(p, l.x, take(l.x.workspace));
  const bool bf16 = kv->dtype == RQ_BF16;
  cudaError_t e;
  if (groups == 0) {
    p.out = out;
    p.lse = lse;
    e = cudaMemsetAsync(status, 0, sizeof(int32_t), s);
    if (e != cudaSuccess) return RQ_ERR_CUDA;
    e = bf16 ? paged_attn::launch_bf16(p, l.x, qb, s) : paged_attn::launch_f32(p, l.x, qb, s);
  } else if (l.tc) {
    float* const own_lse = ls + 2 * (size_t)rows * heads;
    prefix::Params t{};
    t.kv = *kv;
    t.q = q;
    t.table = block_table;
    t.cu_rows = cu_rows;
    t.prefix_requests = prefix_requests;
    t.prefix_lens = prefix_lens;
    t.rows = rows;
    t.heads = heads;
    t.batch = batch;
    t.W = max_blocks;
    t.groups = groups;
    t.G = p.G;
    t.scale = std::fabs(scale_log2);
    t.flip = scale_log2 < 0.f ? 1u : 0u;
    t.whole = o;
    t.whole_ml = reinterpret_cast<float2*>(ls);
    t.part = reinterpret_cast<float*>(take(l.part));
    t.part_ml = reinterpret_cast<float2*>(take(l.part_ml));
    t.group = reinterpret_cast<prefix::Group*>(take(l.group));
    t.per = reinterpret_cast<long long*>(reinterpret_cast<char*>(t.group) + l.group - 256);
    t.gave_up = reinterpret_cast<uint32_t*>(take(l.gave_up));
    const unsigned long long wait_ns = g_wait_ns.load(std::memory_order_relaxed);
    t.wait_ns = wait_ns ? wait_ns : kWaitLimitNs;
    t.stall = g_stall.load(std::memory_order_relaxed);
    p.out = own_o;
    p.lse = own_lse;
    e = qb ? prefix::launch_bf16(t, l.ctas, s) : prefix::launch_f32(t, l.ctas, s);
    if (e == cudaSuccess) e = paged_attn::launch_sums_bf16(p, l.x, qb, s);
    if (e != cudaSuccess) return RQ_ERR_CUDA;
    JoinParams j{t, requests, own_o, own_lse, out, lse, status, l.ctas};
    const dim3 grid((unsigned)(((long long)rows * heads + 31) / 32), (unsigned)(kv->head_dim / (4 * kJoinWarps)));
    auto join = [&](auto* kernel) { return launch_dependent(kernel, grid, kJoinWarps * 32, 0, 0, s, j); };
    switch (kv->head_dim) {
      case 32: e = qb ? join(join_kernel<uint16_t, 32>) : join(join_kernel<float, 32>); break;
      case 64: e = qb ? join(join_kernel<uint16_t, 64>) : join(join_kernel<float, 64>); break;
      default: e = qb ? join(join_kernel<uint16_t, 128>) : join(join_kernel<float, 128>);
    }
  } else {
    const MergeParams m{requests, rows, heads, batch, kv->head_dim, o, own_o, ls, ls + (size_t)rows * heads, out, lse, status};
    p.rows = 2 * rows;
    p.q_rows = rows;
    p.bundle = l.bundle;
    p.row_heads = p.G;
    p.row_skip = heads - p.G;
    p.groups = groups;
    p.cu_rows = cu_rows;
    p.prefix_requests = prefix_requests;
    p.prefix_lens = prefix_lens;
    p.out = o;
    p.lse = ls;
    e = bf16 ? paged_attn::launch_prefixes_bf16(p, l.x, qb, s) : paged_attn::launch_prefixes_f32(p, l.x, qb, s);
    if (e != cudaSuccess) return RQ_ERR_CUDA;
    const long long pairs = (long long)rows * heads;
    const int grid = (int)std::min<long long>((pairs + 7) / 8, 8ll * sm_count() + 1);
    e = qb ? launch_dependent(merge_kernel<uint16_t>, dim3((unsigned)grid), 256, 0, 0, s, m)
           : launch_dependent(merge_kernel<float>, dim3((unsigned)grid), 256, 0, 0, s, m);
  }
  return e == cudaSuccess ? RQ_OK : RQ_ERR_CUDA;
}
