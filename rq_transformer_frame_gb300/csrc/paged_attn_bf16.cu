// paged_attn_bf16.cu -- paged attention over a bf16 cache (paged_attn.cuh, MmaCore).
#include "paged_attn.cuh"

namespace rqk {
namespace paged_attn {

template <typename QT>
static cudaError_t by_head_dim(const Params& p, cudaStream_t s) {
  switch (p.kv.head_dim) {
    case 32: return launch<QT, uint16_t, 32, MmaCore<QT, 32>>(p, s);
    case 64: return launch<QT, uint16_t, 64, MmaCore<QT, 64>>(p, s);
    default: return launch<QT, uint16_t, 128, MmaCore<QT, 128>>(p, s);
  }
}

cudaError_t launch_bf16(const Params& p, bool q_bf16, cudaStream_t s) {
  return q_bf16 ? by_head_dim<uint16_t>(p, s) : by_head_dim<float>(p, s);
}

}  // namespace paged_attn
}  // namespace rqk
