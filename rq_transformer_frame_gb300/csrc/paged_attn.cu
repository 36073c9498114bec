// paged_attn.cu -- rq_paged_attention (include/rq.h): checks, workspace and launch of the
// kernels in paged_attn.cuh.
#include <cmath>

#include "paged_attn.cuh"

extern "C" size_t rq_paged_attention_workspace_size(const rq_paged_kv* kv, int32_t rows,
                                                    int32_t heads, int32_t max_blocks,
                                                    int32_t window) {
  using namespace rqk;
  if (paged_kv_check(kv) != RQ_OK || rows < 1 || heads < 1 || heads % kv->heads != 0 ||
      max_blocks < 1 || window < 0)
    return 0;
  return paged_attn::choose(*kv, rows, heads, max_blocks, window).workspace;
}

extern "C" rq_status rq_paged_attention(const rq_paged_kv* kv, int32_t rows, int32_t heads,
                                        int32_t batch, int32_t max_blocks,
                                        const int32_t* block_table, const int32_t* requests,
                                        const int32_t* positions, int32_t window, float scale,
                                        int32_t q_dtype, const void* q, void* out, float* lse,
                                        void* workspace, size_t workspace_bytes,
                                        void* cuda_stream) {
  using namespace rqk;
  const rq_status st = paged_kv_check(kv);
  if (st != RQ_OK) return st;
  const float scale_log2 =
      (float)((scale != 0.f ? (double)scale : 1.0 / std::sqrt((double)kv->head_dim)) * 1.4426950408889634);
  if (rows < 0 || heads < 1 || heads % kv->heads != 0 || batch < 1 || max_blocks < 1 ||
      window < 0 || !std::isfinite(scale_log2))
    return RQ_ERR_ARG;
  if (q_dtype != RQ_F32 && q_dtype != RQ_BF16) return RQ_ERR_ARG;
  // rows, a row's elements and (row, head) pairs are counted in 32 bits, a thread's next one too
  if (rows > 1 << 30 || heads > 1 << 23 || (long long)rows * heads > INT_MAX) return RQ_ERR_UNSUPPORTED;
  if (rows == 0) return RQ_OK;
  if (!requests && rows > batch) return RQ_ERR_ARG;
  if (!block_table || !positions || !q || !out) return RQ_ERR_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace)) return RQ_ERR_ARG;
  const paged_attn::Choice x = paged_attn::choose(*kv, rows, heads, max_blocks, window);
  if (workspace_bytes < x.workspace || (x.workspace && !workspace)) return RQ_ERR_ARG;
  paged_attn::Params p{};
  p.kv = *kv;
  p.q = q;
  p.out = out;
  p.lse = lse;
  p.table = block_table;
  p.requests = requests;
  p.positions = positions;
  p.rows = rows;
  p.heads = heads;
  p.batch = batch;
  p.W = max_blocks;
  p.window = window;
  p.G = heads / kv->heads;
  p.scale = scale_log2;
  paged_attn::place(p, x, workspace);
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  const bool qb = q_dtype == RQ_BF16;
  const cudaError_t e = kv->dtype == RQ_BF16 ? paged_attn::launch_bf16(p, x, qb, s)
                                             : paged_attn::launch_f32(p, x, qb, s);
  return e == cudaSuccess ? RQ_OK : RQ_ERR_CUDA;
}
