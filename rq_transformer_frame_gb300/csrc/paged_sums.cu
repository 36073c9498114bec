// paged_sums.cu -- paged attention with bf16 queries and f32 outputs (paged_attn.cuh): a part of an
// attention over two requests, joined with the other before it is rounded.
#include "paged_attn.cuh"

namespace rqk {
namespace paged_attn {

template <int HD>
static cudaError_t bf16_by_heads(const Params& p, const Choice& x, cudaStream_t s) {
  using T = uint16_t;
  if constexpr (HD < 128)
    if (x.side > 1) {
      constexpr int N = 2;
      Params side = p;
      side.kv.heads /= N;
      side.kv.head_stride *= N;
      side.G *= N;
      return launch<T, T, HD, SideCore<T, HD, N>, false, float>(side, x, s);
    }
  return p.G <= 8 ? launch<T, T, HD, MmaCore<T, HD>, false, float>(p, x, s)
                  : launch<T, T, HD, WideCore<T, HD>, false, float>(p, x, s);
}

template <int HD>
static cudaError_t f32_by_heads(const Params& p, const Choice& x, cudaStream_t s) {
  using T = uint16_t;
  if (p.G == 1) return launch<T, float, HD, FmaCore<T, HD, 1>, false, float>(p, x, s);
  if (p.G == 2) return launch<T, float, HD, FmaCore<T, HD, 2>, false, float>(p, x, s);
  if (p.G <= 4) return launch<T, float, HD, FmaCore<T, HD, 4>, false, float>(p, x, s);
  return launch<T, float, HD, FmaCore<T, HD, 8>, false, float>(p, x, s);
}

cudaError_t launch_sums_bf16(const Params& p, const Choice& x, bool q_bf16, cudaStream_t s) {
  if (!q_bf16) return launch_bf16(p, x, false, s);
  switch (p.kv.head_dim) {
    case 32: return bf16_by_heads<32>(p, x, s);
    case 64: return bf16_by_heads<64>(p, x, s);
    default: return bf16_by_heads<128>(p, x, s);
  }
}

cudaError_t launch_sums_f32(const Params& p, const Choice& x, bool q_bf16, cudaStream_t s) {
  if (!q_bf16) return launch_f32(p, x, false, s);
  switch (p.kv.head_dim) {
    case 32: return f32_by_heads<32>(p, x, s);
    case 64: return f32_by_heads<64>(p, x, s);
    default: return f32_by_heads<128>(p, x, s);
  }
}

}  // namespace paged_attn
}  // namespace rqk
