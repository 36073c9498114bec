// paged_append.cu -- per-head norm of queries and keys, position rotation, and the store of
// keys and values into the paged cache, in one pass over the rows of a qkv projection
// (include/rq.h, rq_paged_append).
//
// Per head y = x * alpha / sqrt(mean(x^2) + eps); a pair (a, b) of y's first rope_dim
// dimensions becomes (a cos w - b sin w, a sin w + b cos w), w = pos * theta^(-2i/rope_dim).
// The angle is formed in turns, as a 64-bit fixed-point fraction: pos * F_i mod 2^64 with
// F_i = theta^(-2i/rope_dim) / (2 pi) * 2^64 is exact in the position, so far positions
// lose nothing (an f32 product pos * frequency is off by 0.06 rad at position 10^6).
//
// Each element is read once and written once: HBM-bound for many rows, latency for few.
#include <cmath>

#include "paged.cuh"

namespace rqk {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kMaxPairs = 64;

struct AppendParams {
  rq_paged_kv kv;
  const void* qkv;
  long long qkv_stride;
  const float *q_alpha, *k_alpha;
  float eps;
  int heads, style, rope_dim;
  const int32_t* positions;
  const int64_t* slots;
  void* q_out;
  unsigned long long turns[kMaxPairs];  // F_i
};

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
template <>
__device__ __forceinline__ float4 load4<uint16_t>(const uint16_t* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y));
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T>
__device__ __forceinline__ void store4(T* p, float4 v);
template <>
__device__ __forceinline__ void store4<float>(float* p, float4 v) {
  *reinterpret_cast<float4*>(p) = v;
}
template <>
__device__ __forceinline__ void store4<uint16_t>(uint16_t* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(bf16_pair(v.x, v.y), bf16_pair(v.z, v.w));
}

// One CTA per row; HD / 4 lanes share a head, four consecutive dimensions each.
template <typename IT, typename OT, typename KT, int HD>
__global__ void __launch_bounds__(kAppendThreads)
    append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LPH = HD / 4;                   // lanes per head
  constexpr int HPS = kAppendThreads / LPH;     // heads per step of the CTA
  __shared__ float2 s_cs[kMaxPairs];            // (cos, sin) of each pair's angle
  const int tid = threadIdx.x, gl = tid % LPH;
  const int t = blockIdx.x;
  const int pos = p.positions[t];
  if (pos < 0) return;
  if (tid < p.rope_dim / 2) {
    const long long frac = (long long)((unsigned long long)pos * p.turns[tid]);
    float s, c;
    sincospif(__ll2float_rn(frac) * 1.0842021724855044e-19f /* 2^-63: half turns */, &s, &c);
    s_cs[tid] = make_float2(c, s);
  }
  __syncthreads();
  const long long slot = p.slots[t];
  const bool stored = slot >= 0 && slot < (long long)p.kv.n_blocks * p.kv.block_size;
  const long long block = stored ? slot / p.kv.block_size : 0;
  const long long at = block * p.kv.block_stride + (slot - block * p.kv.block_size) * p.kv.row_stride;
  const IT* row = static_cast<const IT*>(p.qkv) + (long long)t * p.qkv_stride;
  const int Hk = p.kv.heads, total = p.heads + 2 * Hk, d = gl * 4;
  const int half = p.rope_dim / 2;
  // heads in steps of HPS over the CTA: every lane of a warp takes part in each shuffle
  for (int base = 0; base < total; base += HPS) {
    const int h = base + tid / LPH;
    const bool live = h < total;
    float4 x = live ? load4<IT>(row + (long long)h * HD + d) : make_float4(0.f, 0.f, 0.f, 0.f);
    const bool is_v = h >= p.heads + Hk;
    const float* alpha = h < p.heads ? p.q_alpha : p.k_alpha;
    float ss = x.x * x.x + x.y * x.y + x.z * x.z + x.w * x.w;
#pragma unroll
    for (int o = LPH / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (!is_v && alpha) {
      const float r = rsqrtf(ss * (1.0f / HD) + p.eps);
      const float4 a = *reinterpret_cast<const float4*>(alpha + d);
      x = make_float4(x.x * r * a.x, x.y * r * a.y, x.z * r * a.z, x.w * r * a.w);
    }
    // the partner of dimension d in the halves pairing is rope_dim / 2 (half / 4 lanes) away
    const int lane = tid & 31, src = p.style == RQ_ROPE_HALVES
                                         ? (d < half ? lane + half / 4 : lane - half / 4) : lane;
    float4 y;
    y.x = __shfl_sync(0xffffffffu, x.x, src);
    y.y = __shfl_sync(0xffffffffu, x.y, src);
    y.z = __shfl_sync(0xffffffffu, x.z, src);
    y.w = __shfl_sync(0xffffffffu, x.w, src);
    if (!is_v && d < p.rope_dim) {
      if (p.style == RQ_ROPE_INTERLEAVED) {
        const float2 c0 = s_cs[d / 2], c1 = s_cs[d / 2 + 1];
        x = make_float4(x.x * c0.x - x.y * c0.y, x.x * c0.y + x.y * c0.x,
                        x.z * c1.x - x.w * c1.y, x.z * c1.y + x.w * c1.x);
      } else {
        const int i = d < half ? d : d - half;
        const float g = d < half ? -1.f : 1.f;  // a cos - b sin, b cos + a sin
        const float2 c0 = s_cs[i], c1 = s_cs[i + 1], c2 = s_cs[i + 2], c3 = s_cs[i + 3];
        x = make_float4(x.x * c0.x + g * y.x * c0.y, x.y * c1.x + g * y.y * c1.y,
                        x.z * c2.x + g * y.z * c2.y, x.w * c3.x + g * y.w * c3.y);
      }
    }
    if (!live) continue;
    if (h < p.heads) {
      store4<OT>(static_cast<OT*>(p.q_out) + ((long long)t * p.heads + h) * HD + d, x);
    } else if (stored) {
      KT* base_kv = static_cast<KT*>(is_v ? p.kv.v : p.kv.k);
      const int kh = h - p.heads - (is_v ? Hk : 0);
      store4<KT>(base_kv + at + kh * p.kv.head_stride + d, x);
    }
  }
}

template <typename IT, typename OT, typename KT>
cudaError_t launch_append(const AppendParams& p, int tokens, cudaStream_t s) {
  switch (p.kv.head_dim) {
    case 32: append_kernel<IT, OT, KT, 32><<<tokens, kAppendThreads, 0, s>>>(p); break;
    case 64: append_kernel<IT, OT, KT, 64><<<tokens, kAppendThreads, 0, s>>>(p); break;
    default: append_kernel<IT, OT, KT, 128><<<tokens, kAppendThreads, 0, s>>>(p); break;
  }
  return cudaGetLastError();
}

template <typename IT, typename OT>
cudaError_t launch_append_kv(const AppendParams& p, int tokens, cudaStream_t s) {
  return p.kv.dtype == RQ_BF16 ? launch_append<IT, OT, uint16_t>(p, tokens, s)
                               : launch_append<IT, OT, float>(p, tokens, s);
}

// F_i = theta^(-2i/rd) / (2 pi) * 2^64 for i < rd / 2, each a product of at most six powers
// g^(2^k), g = theta^(-2/rd) (one call of pow), so within 2^-49 of its value.
void rope_turns(unsigned long long* turns, int rd, double theta) {
  double power[6];
  power[0] = std::pow(theta, -2.0 / rd);
  for (int k = 1; k < 6; ++k) power[k] = power[k - 1] * power[k - 1];
  for (int i = 0; i < rd / 2; ++i) {
    double f = 0.15915494309189535;  // 1 / (2 pi)
    for (int k = 0; k < 6; ++k)
      if (i >> k & 1) f *= power[k];
    turns[i] = (unsigned long long)(f * 18446744073709551616.0);  // f < 1/6: in range
  }
}

}  // namespace
}  // namespace rqk

extern "C" rq_status rq_paged_append(const rq_paged_kv* kv, int32_t tokens, int32_t heads,
                                     int32_t qkv_dtype, const void* qkv, int64_t qkv_stride,
                                     const float* q_alpha, const float* k_alpha, float eps,
                                     int32_t rope_style, int32_t rope_dim, double rope_theta,
                                     const int32_t* positions, const int64_t* slots,
                                     int32_t q_dtype, void* q_out, void* cuda_stream) {
  using namespace rqk;
  const rq_status st = paged_kv_check(kv);
  if (st != RQ_OK) return st;
  if (tokens < 0 || heads < 1 || (long long)heads + 2ll * kv->heads > INT_MAX / 128)
    return RQ_ERR_ARG;
  if ((qkv_dtype != RQ_F32 && qkv_dtype != RQ_BF16) || (q_dtype != RQ_F32 && q_dtype != RQ_BF16))
    return RQ_ERR_ARG;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return RQ_ERR_ARG;
  if (rope_style != RQ_ROPE_INTERLEAVED && rope_style != RQ_ROPE_HALVES) return RQ_ERR_ARG;
  if (rope_dim < 0 || rope_dim > kv->head_dim || rope_dim % 8 != 0) return RQ_ERR_ARG;
  if (rope_dim > 0 && !(rope_theta > 1.0 && std::isfinite(rope_theta))) return RQ_ERR_ARG;
  if (tokens == 0) return RQ_OK;
  if (!qkv || !positions || !slots || !q_out) return RQ_ERR_ARG;
  if (!aligned16(qkv) || !aligned16(q_out) || !aligned16(q_alpha) || !aligned16(k_alpha))
    return RQ_ERR_ARG;
  const int64_t width = ((int64_t)heads + 2 * kv->heads) * kv->head_dim;
  if (qkv_stride < width || qkv_stride % (qkv_dtype == RQ_BF16 ? 8 : 4) != 0) return RQ_ERR_ARG;
  AppendParams p{};
  p.kv = *kv;
  p.qkv = qkv;
  p.qkv_stride = qkv_stride;
  p.q_alpha = q_alpha;
  p.k_alpha = k_alpha;
  p.eps = eps;
  p.heads = heads;
  p.style = rope_style;
  p.rope_dim = rope_dim;
  p.positions = positions;
  p.slots = slots;
  p.q_out = q_out;
  if (rope_dim > 0) rope_turns(p.turns, rope_dim, rope_theta);
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e;
  if (qkv_dtype == RQ_BF16)
    e = q_dtype == RQ_BF16 ? launch_append_kv<uint16_t, uint16_t>(p, tokens, s)
                           : launch_append_kv<uint16_t, float>(p, tokens, s);
  else
    e = q_dtype == RQ_BF16 ? launch_append_kv<float, uint16_t>(p, tokens, s)
                           : launch_append_kv<float, float>(p, tokens, s);
  return e == cudaSuccess ? RQ_OK : RQ_ERR_CUDA;
}
