// paged_attn.cu -- attention of one query token per row over a paged K/V cache
// (include/rq.h, rq_paged_attention).
//
// For row r with position pos and query head h: s_j = scale q . k_j over the live positions
// j, o = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m), m the running maximum.  One CTA per (row,
// head), its warps taking every fourth key.
#include <cmath>

#include "paged.cuh"

namespace rqk {
namespace {

constexpr int kWarps = 4;

struct PagedAttnParams {
  rq_paged_kv kv;
  const void* q;
  void* out;
  float* lse;
  const int32_t *table, *requests, *positions;
  int rows, heads, batch, W, window;
  float scale;
};

template <typename T>
__device__ __forceinline__ float elem(const T* p, long long i);
template <>
__device__ __forceinline__ float elem<float>(const float* p, long long i) { return p[i]; }
template <>
__device__ __forceinline__ float elem<uint16_t>(const uint16_t* p, long long i) {
  return bf16lo(p[i]);
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) {
  *p = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

template <typename QT, typename KT, int HD>
__global__ void __launch_bounds__(kWarps * 32) paged_attn_kernel(const PagedAttnParams p) {
  constexpr int E = HD / 32;
  __shared__ float s_m[kWarps], s_l[kWarps], s_acc[kWarps][HD];
  const int h = blockIdx.x % p.heads, r = blockIdx.x / p.heads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = p.requests ? p.requests[r] : r, pos = p.positions[r];
  if (b < 0 || b >= p.batch) return;
  const int P = p.kv.block_size, kh = h / (p.heads / p.kv.heads);
  const float ninf = -__int_as_float(0x7f800000);
  const QT* q = static_cast<const QT*>(p.q) + ((long long)r * p.heads + h) * HD;
  float qv[E], acc[E], m = ninf, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qv[e] = elem<QT>(q, lane + 32 * e);
    acc[e] = 0.f;
  }
  if (pos >= 0) {
    const int first = pos / P - p.W + 1;
    int lo = first > 0 ? first * P : 0;
    if (p.window > 0 && pos - p.window + 1 > lo) lo = pos - p.window + 1;
    const KT* kc = static_cast<const KT*>(p.kv.k) + kh * p.kv.head_stride;
    const KT* vc = static_cast<const KT*>(p.kv.v) + kh * p.kv.head_stride;
    for (long long j = (long long)lo + warp; j <= pos; j += kWarps) {
      const int page = (int)(j / P);
      const int id = p.table[(size_t)b * p.W + page % p.W];
      if (id < 0 || id >= p.kv.n_blocks) continue;
      const long long at = id * p.kv.block_stride + (j - (long long)page * P) * p.kv.row_stride;
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(qv[e], elem<KT>(kc + at, lane + 32 * e), s);
      s = warp_sum(s) * p.scale;
      const float mn = fmaxf(m, s);
      if (mn == ninf) continue;
      const float c = expf(m - mn), w = expf(s - mn);
      l = l * c + w;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = acc[e] * c + w * elem<KT>(vc + at, lane + 32 * e);
      m = mn;
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_acc[warp][lane + 32 * e] = acc[e];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  float M = ninf, L = 0.f;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w]);
  for (int w = 0; w < kWarps; ++w) L += s_l[w] > 0.f ? s_l[w] * expf(s_m[w] - M) : 0.f;
  QT* out = static_cast<QT*>(p.out) + ((long long)r * p.heads + h) * HD;
  for (int d = threadIdx.x; d < HD; d += kWarps * 32) {
    float a = 0.f;
    for (int w = 0; w < kWarps; ++w)
      if (s_l[w] > 0.f) a += s_acc[w][d] * expf(s_m[w] - M);
    put(out + d, L > 0.f ? a / L : 0.f);
  }
  if (p.lse && threadIdx.x == 0)
    p.lse[(long long)r * p.heads + h] = L > 0.f ? M + logf(L) : ninf;
}

template <typename QT, typename KT>
cudaError_t launch(const PagedAttnParams& p, cudaStream_t s) {
  const unsigned grid = (unsigned)p.rows * (unsigned)p.heads;
  switch (p.kv.head_dim) {
    case 32: paged_attn_kernel<QT, KT, 32><<<grid, kWarps * 32, 0, s>>>(p); break;
    case 64: paged_attn_kernel<QT, KT, 64><<<grid, kWarps * 32, 0, s>>>(p); break;
    default: paged_attn_kernel<QT, KT, 128><<<grid, kWarps * 32, 0, s>>>(p); break;
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace rqk

extern "C" size_t rq_paged_attention_workspace_size(int32_t heads, int32_t kv_heads,
                                                    int32_t head_dim) {
  if (heads < 1 || kv_heads < 1 || heads % kv_heads != 0 || head_dim < 1) return 0;
  return 16;
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
  if (rows < 0 || heads < 1 || heads % kv->heads != 0 || batch < 1 || max_blocks < 1 ||
      window < 0 || !std::isfinite(scale))
    return RQ_ERR_ARG;
  if (q_dtype != RQ_F32 && q_dtype != RQ_BF16) return RQ_ERR_ARG;
  if ((long long)rows * heads > INT_MAX) return RQ_ERR_UNSUPPORTED;
  if (rows == 0) return RQ_OK;
  if (!requests && rows > batch) return RQ_ERR_ARG;
  if (!block_table || !positions || !q || !out || !workspace) return RQ_ERR_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace)) return RQ_ERR_ARG;
  if (workspace_bytes < rq_paged_attention_workspace_size(heads, kv->heads, kv->head_dim))
    return RQ_ERR_ARG;
  PagedAttnParams p{};
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
  p.scale = scale != 0.f ? scale : 1.0f / sqrtf((float)kv->head_dim);
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e;
  if (q_dtype == RQ_BF16)
    e = kv->dtype == RQ_BF16 ? launch<uint16_t, uint16_t>(p, s) : launch<uint16_t, float>(p, s);
  else
    e = kv->dtype == RQ_BF16 ? launch<float, uint16_t>(p, s) : launch<float, float>(p, s);
  return e == cudaSuccess ? RQ_OK : RQ_ERR_CUDA;
}
