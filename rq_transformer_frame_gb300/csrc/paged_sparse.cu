// paged_sparse.cu -- rq_paged_sparse_attention (include/rq.h): checks, workspace and launch of the
// kernels in paged_attn.cuh with lists of pages.
//
// Each (row, K/V head) is a row of one K/V head, with a list of its own, and launches are chosen as for
// such rows: few units are split up to 8 tiles a warp where there are several lists, as one request with
// several K/V heads has, and further for one list alone (paged_attn.cuh, split_ctas).
#include <cmath>

#include "paged_attn.cuh"

namespace rqk {
namespace paged_attn {
namespace {

Choice choose_lists(rq_paged_kv kv, int rows, int heads, int list) {
  const int lists = rows * kv.heads;
  heads /= kv.heads;
  kv.heads = 1;
  return choose(kv, lists, heads, list, 0);
}

}  // namespace
}  // namespace paged_attn
}  // namespace rqk

static rq_status check(const rq_paged_kv* kv, int32_t rows, int32_t heads, int32_t list) {
  using namespace rqk;
  const rq_status st = paged_kv_check(kv);
  if (st != RQ_OK) return st;
  if (rows < 0 || heads < 1 || heads % kv->heads != 0 || list < 1) return RQ_ERR_ARG;
  if (rows > 1 << 30 || heads > 1 << 23 || (long long)rows * heads > INT_MAX ||
      (long long)rows * kv->heads >= 1 << 30 || (long long)list * kv->block_size >= INT_MAX - 64)
    return RQ_ERR_UNSUPPORTED;
  return RQ_OK;
}

extern "C" size_t rq_paged_sparse_attention_workspace_size(const rq_paged_kv* kv, int32_t rows,
                                                           int32_t heads, int32_t list) {
  if (check(kv, rows, heads, list) != RQ_OK || rows < 1) return 0;
  return rqk::paged_attn::choose_lists(*kv, rows, heads, list).workspace;
}

extern "C" rq_status rq_paged_sparse_attention(const rq_paged_kv* kv, int32_t rows, int32_t heads,
                                               int32_t batch, int32_t max_blocks,
                                               const int32_t* block_table, const int32_t* requests,
                                               const int32_t* positions, int32_t list,
                                               const int32_t* pages, float scale, int32_t q_dtype,
                                               const void* q, void* out, float* lse, void* workspace,
                                               size_t workspace_bytes, void* cuda_stream) {
  using namespace rqk;
  const rq_status st = check(kv, rows, heads, list);
  if (st != RQ_OK) return st;
  const float scale_log2 =
      (float)((scale != 0.f ? (double)scale : 1.0 / std::sqrt((double)kv->head_dim)) * 1.4426950408889634);
  if (batch < 1 || max_blocks < 1 || !std::isfinite(scale_log2)) return RQ_ERR_ARG;
  if (q_dtype != RQ_F32 && q_dtype != RQ_BF16) return RQ_ERR_ARG;
  if (rows == 0) return RQ_OK;
  if (!requests && rows > batch) return RQ_ERR_ARG;
  if (!block_table || !positions || !pages || !q || !out) return RQ_ERR_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace)) return RQ_ERR_ARG;
  const paged_attn::Choice x = paged_attn::choose_lists(*kv, rows, heads, list);
  if (workspace_bytes < x.workspace || (x.workspace && !workspace)) return RQ_ERR_ARG;
  paged_attn::MoreParams p{};
  p.kv = *kv;
  p.kv.heads = 1;
  p.kv_heads = kv->heads;
  p.q = q;
  p.out = out;
  p.lse = lse;
  p.table = block_table;
  p.requests = requests;
  p.positions = positions;
  p.rows = rows * kv->heads;
  p.heads = p.G = heads / kv->heads;
  p.batch = batch;
  p.W = max_blocks;
  p.pages = pages;
  p.list = list;
  p.scale = scale_log2;
  paged_attn::place(p, x, workspace);
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  const bool qb = q_dtype == RQ_BF16;
  const cudaError_t e = kv->dtype == RQ_BF16 ? paged_attn::launch_lists_bf16(p, x, qb, s)
                                             : paged_attn::launch_lists_f32(p, x, qb, s);
  return e == cudaSuccess ? RQ_OK : RQ_ERR_CUDA;
}
