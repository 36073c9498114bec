// paged_sums.cu -- paged attention with f32 outputs (paged_attn.cuh): a part of an attention over two
// requests, joined with the other before it is rounded. Over a bf16 cache with bf16 queries (f32 ones have
// f32 outputs as it is).
#include "paged_attn.cuh"

namespace rqk {
namespace paged_attn {

template <int HD>
static cudaError_t by_heads(const Params& p, const Choice& x, cudaStream_t s) {
  using T = uint16_t;
  if constexpr (HD < 128)
    if (x.side > 1) {
      constexpr int N = 2;
      Params side = p;
      side.kv.heads /= N;
      side.kv.head_stride *= N;
      side.G *= N;
      return launch<T, T, HD, SideCore<T, HD, N>, kRows, float>(side, x, s);
    }
  return p.G <= 8 ? launch<T, T, HD, MmaCore<T, HD>, kRows, float>(p, x, s)
                  : launch<T, T, HD, WideCore<T, HD>, kRows, float>(p, x, s);
}

cudaError_t launch_sums_bf16(const Params& p, const Choice& x, bool q_bf16, cudaStream_t s) {
  if (!q_bf16) return launch_bf16(p, x, false, s);
  switch (p.kv.head_dim) {
    case 32: return by_heads<32>(p, x, s);
    case 64: return by_heads<64>(p, x, s);
    default: return by_heads<128>(p, x, s);
  }
}

}  // namespace paged_attn
}  // namespace rqk
