// paged_prefixes_f32.cu -- paged attention of rows over prefixes and over their own requests, f32 cache, f32
// outputs (paged_attn.cuh).
#include "paged_attn.cuh"

namespace rqk {
namespace paged_attn {

template <typename QT, int HD>
static cudaError_t by_heads(const MoreParams& p, const Choice& x, cudaStream_t s) {
  if (x.unit_heads == 1) return launch<QT, float, HD, FmaCore<QT, HD, 1>, kPrefixes, float>(p, x, s);
  if (x.unit_heads == 2) return launch<QT, float, HD, FmaCore<QT, HD, 2>, kPrefixes, float>(p, x, s);
  if (x.unit_heads <= 4) return launch<QT, float, HD, FmaCore<QT, HD, 4>, kPrefixes, float>(p, x, s);
  return launch<QT, float, HD, FmaCore<QT, HD, 8>, kPrefixes, float>(p, x, s);
}

template <typename QT>
static cudaError_t by_head_dim(const MoreParams& p, const Choice& x, cudaStream_t s) {
  switch (p.kv.head_dim) {
    case 32: return by_heads<QT, 32>(p, x, s);
    case 64: return by_heads<QT, 64>(p, x, s);
    default: return by_heads<QT, 128>(p, x, s);
  }
}

cudaError_t launch_prefixes_f32(const MoreParams& p, const Choice& x, bool q_bf16, cudaStream_t s) {
  return q_bf16 ? by_head_dim<uint16_t>(p, x, s) : by_head_dim<float>(p, x, s);
}

}  // namespace paged_attn
}  // namespace rqk
