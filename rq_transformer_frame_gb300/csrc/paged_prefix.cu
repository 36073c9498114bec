// paged_prefix.cu -- attention over a prefix that a group of rows shares and over each row's own
// request (include/rq.h, rq_paged_prefix_attention).
//
// Softmax over two sets of positions from the two apart: with o_i, lse_i of set i,
// lse = log(e^lse_1 + e^lse_2) and o = e^(lse_1 - lse) o_1 + e^(lse_2 - lse) o_2. Both parts are f32;
// the output is rounded once.
#include <algorithm>
#include <cmath>

#include "paged_attn.cuh"

namespace rqk {
namespace {

using paged_attn::finite_or_zero;
using paged_attn::neg_inf;
using paged_attn::put;

struct PrefixParams {
  const int32_t *requests, *cu_rows, *prefix_requests, *prefix_lens;
  int rows, heads, batch, groups, hd;
  int32_t *row_request, *row_position;  // of the prefix, for each row
  const float *o1, *o2, *lse1, *lse2;   // prefix, own
  void* out;
  float* lse;
};

// each row's prefix as a request and the last position read of it
__global__ void __launch_bounds__(256) rows_kernel(const __grid_constant__ PrefixParams p) {
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x * 256 + threadIdx.x;
  if (r >= p.rows) return;
  const int b = p.requests ? p.requests[r] : r;
  int request = -1, position = -1;
  if (b >= 0 && b < p.batch) {
    request = 0;  // without a prefix: an empty request
    int lo = 0, hi = p.groups;  // the last group that starts at r or before
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (p.cu_rows[mid] <= r) lo = mid + 1;
      else hi = mid;
    }
    if (lo > 0 && r < p.cu_rows[lo]) {
      const int x = p.prefix_requests[lo - 1], n = p.prefix_lens[lo - 1];
      if (x >= 0 && x < p.batch && n > 0) request = x, position = n - 1;
    }
  }
  p.row_request[r] = request;
  p.row_position[r] = position;
}

template <typename OT>
__global__ void __launch_bounds__(256) merge_kernel(const __grid_constant__ PrefixParams p) {
  pdl_wait();
  pdl_trigger();
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

struct Layout {
  paged_attn::Choice x;
  size_t o, lse, map, bytes;
};

Layout layout_of(const rq_paged_kv& kv, int rows, int heads, int max_blocks) {
  Layout l{};
  l.x = paged_attn::choose(kv, rows, heads, max_blocks, 0);
  l.o = paged_attn::align256((size_t)rows * heads * kv.head_dim * sizeof(float));
  l.lse = paged_attn::align256((size_t)rows * heads * sizeof(float));
  l.map = paged_attn::align256((size_t)rows * sizeof(int32_t));
  l.bytes = 2 * (l.o + l.lse + l.map) + l.x.workspace;
  return l;
}

rq_status check(const rq_paged_kv* kv, int32_t rows, int32_t heads, int32_t max_blocks, int32_t groups) {
  const rq_status st = paged_kv_check(kv);
  if (st != RQ_OK) return st;
  if (rows < 0 || heads < 1 || heads % kv->heads != 0 || max_blocks < 1 || groups < 0) return RQ_ERR_ARG;
  if (rows > 1 << 30 || heads > 1 << 23 || (long long)rows * heads > INT_MAX || groups > 1 << 20)
    return RQ_ERR_UNSUPPORTED;
  return RQ_OK;
}

}  // namespace
}  // namespace rqk

extern "C" size_t rq_paged_prefix_attention_workspace_size(const rq_paged_kv* kv, int32_t rows,
                                                           int32_t heads, int32_t max_blocks,
                                                           int32_t groups) {
  using namespace rqk;
  if (check(kv, rows, heads, max_blocks, groups) != RQ_OK || rows < 1) return 0;
  return layout_of(*kv, rows, heads, max_blocks).bytes;
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
  const Layout l = layout_of(*kv, rows, heads, max_blocks);
  if (workspace_bytes < l.bytes) return RQ_ERR_ARG;
  char* ws = static_cast<char*>(workspace);
  float* o[2] = {reinterpret_cast<float*>(ws), reinterpret_cast<float*>(ws + l.o)};
  ws += 2 * l.o;
  float* ls[2] = {reinterpret_cast<float*>(ws), reinterpret_cast<float*>(ws + l.lse)};
  ws += 2 * l.lse;
  int32_t* map[2] = {reinterpret_cast<int32_t*>(ws), reinterpret_cast<int32_t*>(ws + l.map)};
  ws += 2 * l.map;
  PrefixParams pp{requests, cu_rows, prefix_requests, prefix_lens, rows, heads, batch, groups, kv->head_dim,
                  map[0], map[1], o[0], o[1], ls[0], ls[1], out, lse};
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e = launch_dependent(rows_kernel, dim3((unsigned)((rows + 255) / 256)), 256, 0, 0, s, pp);
  if (e != cudaSuccess) return RQ_ERR_CUDA;
  paged_attn::Params p{};
  p.kv = *kv;
  p.q = q;
  p.table = block_table;
  p.rows = rows;
  p.heads = heads;
  p.batch = batch;
  p.W = max_blocks;
  p.G = heads / kv->heads;
  p.scale = scale_log2;
  paged_attn::place(p, l.x, ws);
  const bool qb = q_dtype == RQ_BF16;
  for (int i = 0; i < 2; ++i) {
    p.requests = i == 0 ? map[0] : requests;
    p.positions = i == 0 ? map[1] : positions;
    p.out = o[i];
    p.lse = ls[i];
    e = kv->dtype == RQ_BF16 ? paged_attn::launch_sums_bf16(p, l.x, qb, s)
                             : paged_attn::launch_sums_f32(p, l.x, qb, s);
    if (e != cudaSuccess) return RQ_ERR_CUDA;
  }
  const long long pairs = (long long)rows * heads;
  const int grid = (int)std::min<long long>((pairs + 7) / 8, 8ll * sm_count() + 1);
  e = qb ? launch_dependent(merge_kernel<uint16_t>, dim3((unsigned)grid), 256, 0, 0, s, pp)
         : launch_dependent(merge_kernel<float>, dim3((unsigned)grid), 256, 0, 0, s, pp);
  return e == cudaSuccess ? RQ_OK : RQ_ERR_CUDA;
}
