// paged_attn_f32.cu -- paged attention over an f32 cache (paged_attn.cuh, FmaCore).
#include "paged_attn.cuh"

namespace rqk {
namespace paged_attn {

template <typename QT, int HD>
static cudaError_t by_heads(const Params& p, const Choice& x, cudaStream_t s) {
  if (p.G == 1) return launch<QT, float, HD, FmaCore<QT, HD, 1>>(p, x, s);
  if (p.G == 2) return launch<QT, float, HD, FmaCore<QT, HD, 2>>(p, x, s);
  if (p.G <= 4) return launch<QT, float, HD, FmaCore<QT, HD, 4>>(p, x, s);
  return launch<QT, float, HD, FmaCore<QT, HD, 8>>(p, x, s);
}

template <typename QT>
static cudaError_t by_head_dim(const Params& p, const Choice& x, cudaStream_t s) {
  switch (p.kv.head_dim) {
    case 32: return by_heads<QT, 32>(p, x, s);
    case 64: return by_heads<QT, 64>(p, x, s);
    default: return by_heads<QT, 128>(p, x, s);
  }
}

cudaError_t launch_f32(const Params& p, const Choice& x, bool q_bf16, cudaStream_t s) {
  return q_bf16 ? by_head_dim<uint16_t>(p, x, s) : by_head_dim<float>(p, x, s);
}

}  // namespace paged_attn
}  // namespace rqk
