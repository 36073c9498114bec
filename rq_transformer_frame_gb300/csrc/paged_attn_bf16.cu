// paged_attn_bf16.cu -- paged attention over a bf16 cache (paged_attn.cuh, MmaCore and WideCore).
#include "paged_attn.cuh"

namespace rqk {
namespace paged_attn {

template <typename QT, int HD>
static cudaError_t by_heads(const Params& p, cudaStream_t s) {
  return p.G <= 8 ? launch<QT, uint16_t, HD, MmaCore<QT, HD>>(p, s)
                  : launch<QT, uint16_t, HD, WideCore<QT, HD>>(p, s);
}

template <typename QT>
static cudaError_t by_head_dim(const Params& p, cudaStream_t s) {
  switch (p.kv.head_dim) {
    case 32: return by_heads<QT, 32>(p, s);
    case 64: return by_heads<QT, 64>(p, s);
    default: return by_heads<QT, 128>(p, s);
  }
}

cudaError_t launch_bf16(const Params& p, bool q_bf16, cudaStream_t s) {
  return q_bf16 ? by_head_dim<uint16_t>(p, s) : by_head_dim<float>(p, s);
}

}  // namespace paged_attn
}  // namespace rqk
