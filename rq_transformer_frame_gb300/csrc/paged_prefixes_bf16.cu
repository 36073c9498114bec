// paged_prefixes_bf16.cu -- paged attention of rows over prefixes and over their own requests, bf16 cache, f32
// outputs (paged_attn.cuh).
#include "paged_attn.cuh"

namespace rqk {
namespace paged_attn {

template <typename QT, int HD>
static cudaError_t by_heads(const MoreParams& p, const Choice& x, cudaStream_t s) {
  if constexpr (HD < 128)
    if (x.side > 1) {
      constexpr int N = 2;
      MoreParams side = p;
      side.kv.heads /= N;
      side.kv.head_stride *= N;
      side.G *= N;
      side.row_heads = side.G;
      return launch<QT, uint16_t, HD, SideCore<QT, HD, N>, kPrefixes, float>(side, x, s);
    }
  return x.unit_heads <= 8 ? launch<QT, uint16_t, HD, MmaCore<QT, HD>, kPrefixes, float>(p, x, s)
                  : launch<QT, uint16_t, HD, WideCore<QT, HD>, kPrefixes, float>(p, x, s);
}

template <typename QT>
static cudaError_t by_head_dim(const MoreParams& p, const Choice& x, cudaStream_t s) {
  switch (p.kv.head_dim) {
    case 32: return by_heads<QT, 32>(p, x, s);
    case 64: return by_heads<QT, 64>(p, x, s);
    default: return by_heads<QT, 128>(p, x, s);
  }
}

cudaError_t launch_prefixes_bf16(const MoreParams& p, const Choice& x, bool q_bf16, cudaStream_t s) {
  return q_bf16 ? by_head_dim<uint16_t>(p, x, s) : by_head_dim<float>(p, x, s);
}

}  // namespace paged_attn
}  // namespace rqk
