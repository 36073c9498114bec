// paged_append.cu -- per-head norm of queries and keys, position rotation, and the store of
// keys and values into the paged cache, in one pass over the rows of a qkv projection
// (include/rq.h, rq_paged_append).
//
// Per head y = x * alpha / sqrt(mean(x^2) + eps); a pair (a, b) of y's first rope_dim
// dimensions becomes (a cos w - b sin w, a sin w + b cos w), w = pos * theta^(-2i/rope_dim).
// The angle is formed in turns, as a 64-bit fixed-point fraction: pos * F_i mod 2^64 with
// F_i = theta^(-2i/rope_dim) / (2 pi) * 2^64 to 2^-62, so it is within 2^-31 of a turn at any
// position (an f32 product pos * frequency is off by 0.06 rad at position 10^6). It is rounded
// once, to the f32 half turns that sine and cosine are taken of (2^-26 of a turn).
//
// Each element is read once and written once: HBM-bound for many rows, latency for few. A CTA
// takes a row, or a slice of its heads where there are too few rows to fill the card: the
// row's angles are computed once and shared. HD / 8 lanes share a head; a lane holds two pieces
// of four dimensions such that both dimensions of each of its pairs are its own: 8
// consecutive ones, or with the halves pairing 4 j and rope_dim / 2 + 4 j, so no value changes
// lanes. The loads of a few steps (a step is a head for each HD / 8 lanes) are always in flight,
// the first of them before the position is known.
#include <cmath>

#include "paged.cuh"

namespace rqk {
namespace {

constexpr int kMaxWarps = 2;  // of a CTA
constexpr int kMaxPairs = 64;
// steps of a warp whose loads are in flight: 16 registers of bf16, 24 of f32
template <typename IT>
constexpr int kAheadOf = sizeof(IT) == 2 ? 4 : 3;

struct AppendParams {
  rq_paged_kv kv;
  const void* qkv;
  long long qkv_stride;
  const float *q_alpha, *k_alpha;
  float eps;
  int heads, rope_dim;
  int slices, steps;  // CTAs of a row, and steps (of 256 / HD heads) of each of their warps
  const int32_t* positions;
  const int64_t* slots;
  void* q_out;
  unsigned long long turns[kMaxPairs];  // F_i
};

// four values as they lie in memory
template <typename T>
struct Piece;
template <>
struct Piece<float> {
  float4 v;
  __device__ __forceinline__ void widen(float* x) const { x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w; }
};
template <>
struct Piece<uint16_t> {
  uint2 v;
  __device__ __forceinline__ void widen(float* x) const {
    x[0] = bf16lo(v.x), x[1] = bf16hi(v.x), x[2] = bf16lo(v.y), x[3] = bf16hi(v.y);
  }
};

__device__ __forceinline__ void store4(float* p, const float* x) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(uint16_t* p, const float* x) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// A lane's eight values of a head as the first and second members of its four pairs, packed by
// two: one instruction works on two values (the kernel issues more than it waits otherwise).
// HALVES: the first members are the piece at lo; else every second value from there.
struct Pairs {
  f32x2 u[2], v[2];
};
template <bool HALVES>
__device__ __forceinline__ Pairs pairs_of(const float (&x)[8]) {
  if (HALVES) return {{pack2(x[0], x[1]), pack2(x[2], x[3])}, {pack2(x[4], x[5]), pack2(x[6], x[7])}};
  return {{pack2(x[0], x[2]), pack2(x[4], x[6])}, {pack2(x[1], x[3]), pack2(x[5], x[7])}};
}
template <bool HALVES>
__device__ __forceinline__ void values_of(const Pairs& p, float (&x)[8]) {
  const float2 a = unpack2(p.u[0]), b = unpack2(p.u[1]), c = unpack2(p.v[0]), d = unpack2(p.v[1]);
  if (HALVES) {
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y, x[4] = c.x, x[5] = c.y, x[6] = d.x, x[7] = d.y;
  } else {
    x[0] = a.x, x[2] = a.y, x[4] = b.x, x[6] = b.y, x[1] = c.x, x[3] = c.y, x[5] = d.x, x[7] = d.y;
  }
}

template <typename IT, typename OT, typename KT, int HD, bool HALVES>
__global__ void __launch_bounds__(kMaxWarps * 32, 28 / kMaxWarps)
    append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LPH = HD / 8, HPS = 32 / LPH;  // lanes of a head, heads of a step
  constexpr int kAhead = kAheadOf<IT>;
  __shared__ float2 s_cs[kMaxPairs];
  const int tid = threadIdx.x, lane = tid & 31, sub = lane / LPH, j = lane % LPH;
  const int t = blockIdx.x / p.slices, slice = blockIdx.x - t * p.slices;
  const int total = p.heads + 2 * p.kv.heads, half = p.rope_dim / 2;
  const bool turned = j * 8 < p.rope_dim;
  // this lane's dimensions: lo .. lo + 3 and hi .. hi + 3; its pairs are 4 j .. 4 j + 3
  const int lo = HALVES && turned ? 4 * j : 8 * j, hi = HALVES && turned ? half + 4 * j : 8 * j + 4;
  // the warp's heads: step i from h0 + i * HPS, this lane's head `sub` further, below h1
  const int h0 = (slice * ((int)blockDim.x / 32) + tid / 32) * p.steps * HPS, h1 = min(h0 + p.steps * HPS, total);
  pdl_wait();
  pdl_trigger();
  const IT* const row = static_cast<const IT*>(p.qkv) + t * p.qkv_stride + (long long)sub * HD;
  Piece<IT> in[kAhead][2];
  auto load = [&](Piece<IT> (&d)[2], int h) {
    if (h + sub >= h1) return;
    const IT* x = row + (long long)h * HD;
    d[0] = *reinterpret_cast<const Piece<IT>*>(x + lo);
    d[1] = *reinterpret_cast<const Piece<IT>*>(x + hi);
  };
#pragma unroll
  for (int b = 0; b < kAhead; ++b) load(in[b], h0 + b * HPS);
  const int pos = p.positions[t];
  const long long slot = p.slots[t];
  if (pos < 0) return;
  auto alpha_of = [&](const float* alpha) {
    float a[8];
    reinterpret_cast<const Piece<float>*>(alpha + lo)->widen(a);
    reinterpret_cast<const Piece<float>*>(alpha + hi)->widen(a + 4);
    return pairs_of<HALVES>(a);
  };
  for (int i = tid; i < half; i += blockDim.x) {
    const long long frac = (long long)((unsigned long long)pos * p.turns[i]);
    float sn, cs;  // of half turns: 2^-63 of the fraction
    sincospif(__ll2float_rn(frac) * 1.0842021724855044e-19f, &sn, &cs);
    s_cs[i] = make_float2(cs, sn);
  }
  __syncthreads();
  f32x2 c[2], s[2], ns[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = turned ? s_cs[4 * j + 2 * i] : make_float2(1.f, 0.f);
    const float2 b = turned ? s_cs[4 * j + 2 * i + 1] : make_float2(1.f, 0.f);
    c[i] = pack2(a.x, b.x);
    s[i] = pack2(a.y, b.y);
    ns[i] = pack2(-a.y, -b.y);
  }
  const bool stored = slot >= 0 && slot < (long long)p.kv.n_blocks * p.kv.block_size;
  const long long block = !stored ? 0 : slot <= INT_MAX ? (int)slot / p.kv.block_size
                                                        : slot / p.kv.block_size;
  const long long at = block * p.kv.block_stride +
                       (stored ? slot - block * p.kv.block_size : 0) * p.kv.row_stride;
  OT* const out = static_cast<OT*>(p.q_out) + (long long)t * p.heads * HD;
  for (int h = h0; h < h1; h += kAhead * HPS) {
#pragma unroll
    for (int b = 0; b < kAhead; ++b) {
      if (h + b * HPS >= h1) break;  // the whole step is past the slice
      const int head = h + b * HPS + sub;
      const bool live = head < h1, is_q = head < p.heads, is_v = head >= p.heads + p.kv.heads;
      float x[8] = {};
      if (live) {
        in[b][0].widen(x);
        in[b][1].widen(x + 4);
      }
      load(in[b], h + (b + kAhead) * HPS);
      Pairs y = pairs_of<HALVES>(x);
      f32x2 sq = mul2(y.u[0], y.u[0]);
      sq = fma2(y.u[1], y.u[1], sq);
      sq = fma2(y.v[0], y.v[0], sq);
      sq = fma2(y.v[1], y.v[1], sq);
      float ss = unpack2(sq).x + unpack2(sq).y;
#pragma unroll
      for (int o = LPH / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (!is_v) {
        if (const float* alpha = is_q ? p.q_alpha : p.k_alpha) {
          const Pairs a = alpha_of(alpha);
          const float r = rsqrtf(ss * (1.0f / HD) + p.eps);
          const f32x2 r2 = pack2(r, r);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            y.u[i] = mul2(y.u[i], mul2(r2, a.u[i]));
            y.v[i] = mul2(y.v[i], mul2(r2, a.v[i]));
          }
        }
        if (turned) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const f32x2 u = y.u[i];
            y.u[i] = fma2(u, c[i], mul2(y.v[i], ns[i]));
            y.v[i] = fma2(u, s[i], mul2(y.v[i], c[i]));
          }
        }
        values_of<HALVES>(y, x);
      }
      if (!live) continue;
      if (is_q) {
        OT* o = out + (long long)head * HD;
        store4(o + lo, x);
        store4(o + hi, x + 4);
      } else if (stored) {
        KT* o = static_cast<KT*>(is_v ? p.kv.v : p.kv.k) + at +
                (head - p.heads - (is_v ? p.kv.heads : 0)) * p.kv.head_stride;
        store4(o + lo, x);
        store4(o + hi, x + 4);
      }
    }
  }
}

template <typename IT, typename OT, typename KT, int HD, bool HALVES>
cudaError_t launch_append(AppendParams& p, int tokens, cudaStream_t s) {
  // Rows in plenty are a CTA of one warp each: no warp waits for another's angles (16384 rows
  // of 48 heads of 128 in bf16: 67 us; 69 with two warps a row, 73 with four; 4300 rows 26
  // and 23). Fewer rows are CTAs of two warps, and below eight rows a multiprocessor each is divided
  // over several, down to one step a warp (64 such rows: 2.7 us, with CTAs of one warp 3.2).
  constexpr int HPS = 32 / (HD / 8);
  const int sms = sm_count();
  if (sms == 0) return cudaErrorInvalidDevice;
  const int steps = (p.heads + 2 * p.kv.heads + HPS - 1) / HPS, warps = tokens >= sms * 48 ? 1 : 2;
  const int whole = (steps + warps - 1) / warps;  // of a warp, with one CTA a row
  int slices = tokens >= sms * 8 ? 1 : (sms * 8 + tokens - 1) / tokens;
  if (slices > whole) slices = whole;
  p.steps = (whole + slices - 1) / slices;
  p.slices = (steps + p.steps * warps - 1) / (p.steps * warps);
  const long long grid = (long long)tokens * p.slices;
  if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
  return launch_dependent(append_kernel<IT, OT, KT, HD, HALVES>, dim3((unsigned)grid), warps * 32, 0, 0, s, p);
}

template <typename IT, typename OT, typename KT, int HD>
cudaError_t by_rope(AppendParams& p, int tokens, int style, cudaStream_t s) {
  return style == RQ_ROPE_HALVES ? launch_append<IT, OT, KT, HD, true>(p, tokens, s)
                                 : launch_append<IT, OT, KT, HD, false>(p, tokens, s);
}

template <typename IT, typename OT, typename KT>
cudaError_t by_head_dim(AppendParams& p, int tokens, int style, cudaStream_t s) {
  switch (p.kv.head_dim) {
    case 32: return by_rope<IT, OT, KT, 32>(p, tokens, style, s);
    case 64: return by_rope<IT, OT, KT, 64>(p, tokens, style, s);
    default: return by_rope<IT, OT, KT, 128>(p, tokens, style, s);
  }
}

template <typename IT, typename OT>
cudaError_t by_cache(AppendParams& p, int tokens, int style, cudaStream_t s) {
  return p.kv.dtype == RQ_BF16 ? by_head_dim<IT, OT, uint16_t>(p, tokens, style, s)
                               : by_head_dim<IT, OT, float>(p, tokens, style, s);
}

// hi + lo: a number in two doubles, 100 bits and more of it
struct Double2 {
  double hi, lo;
};
// The product's rounding error comes from a fused multiply-add, the sum's from T. J. Dekker, "A
// floating-point technique for extending the available precision" (1971).
Double2 times(const Double2& a, const Double2& b) {
  const double p = a.hi * b.hi;
  const double e = std::fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi);
  const double s = p + e;
  return {s, e - (s - p)};
}
// v in (0, 1) times 2^64, to nearest (hi may be 1 already, lo is below 0 then)
unsigned long long fixed64(const Double2& v) {
  const double h = v.hi * 18446744073709551616.0;
  const unsigned long long whole = v.hi < 1.0 ? (unsigned long long)h : 0;
  const double rest = (v.hi < 1.0 ? h - (double)whole : 0.0) + v.lo * 18446744073709551616.0;
  return whole + (unsigned long long)std::llround(rest);
}

// F_i = theta^(-2i/rd) / (2 pi) * 2^64 for i < n = rd / 2, within 4 (2^-62 of a turn): F_0 times
// powers g^(2^k) of g = theta^(-2/rd), at most six of them, each and each product to nearest in
// 64 bits. A double's g would be off by 2^-53 and its powers by n times that, which position 2^31
// makes 2^-21 of a turn; but g^n theta = 1 in exact arithmetic, so what it is in two doubles says
// by how much g, and each of its powers, is off.
void rope_turns(unsigned long long* turns, int rd, double theta) {
  const int n = rd / 2;  // 64 at most
  Double2 power[7], all{1.0, 0.0};
  power[0] = {std::pow(theta, -2.0 / rd), 0.0};
  for (int k = 1; n >> k; ++k) power[k] = times(power[k - 1], power[k - 1]);
  for (int k = 0; n >> k; ++k)
    if (n >> k & 1) all = times(all, power[k]);
  all = times(all, {theta, 0.0});
  const double off = ((all.hi - 1.0) + all.lo) / n;  // of g, relative
  turns[0] = 0x28BE60DB9391054Aull;  // 2^64 / (2 pi)
  for (int k = 0; 1 << k < n; ++k) {
    power[k].lo -= power[k].hi * off * (1 << k);
    const unsigned long long g = fixed64(power[k]);
    for (int i = 0; i < 1 << k && i + (1 << k) < n; ++i)
      turns[i + (1 << k)] =
          (unsigned long long)(((unsigned __int128)turns[i] * g + (1ull << 63)) >> 64);
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
  p.rope_dim = rope_dim;
  p.positions = positions;
  p.slots = slots;
  p.q_out = q_out;
  if (rope_dim > 0) rope_turns(p.turns, rope_dim, rope_theta);
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e;
  if (qkv_dtype == RQ_BF16)
    e = q_dtype == RQ_BF16 ? by_cache<uint16_t, uint16_t>(p, tokens, rope_style, s)
                           : by_cache<uint16_t, float>(p, tokens, rope_style, s);
  else
    e = q_dtype == RQ_BF16 ? by_cache<float, uint16_t>(p, tokens, rope_style, s)
                           : by_cache<float, float>(p, tokens, rope_style, s);
  return e == cudaSuccess ? RQ_OK : RQ_ERR_CUDA;
}
