// paged_prefix_bf16.cu -- the shared prefix's kernel with bf16 queries (paged_prefix.cuh).
#include "paged_prefix.cuh"

namespace rqk {
namespace prefix {

cudaError_t launch_bf16(const Params& p, int ctas, cudaStream_t s) {
  switch (p.kv.head_dim) {
    case 32: return launch<uint16_t, 32>(p, ctas, s);
    case 64: return launch<uint16_t, 64>(p, ctas, s);
    default: return launch<uint16_t, 128>(p, ctas, s);
  }
}

}  // namespace prefix
}  // namespace rqk
