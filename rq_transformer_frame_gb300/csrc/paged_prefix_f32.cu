// paged_prefix_f32.cu -- the shared prefix's kernel with f32 queries (paged_prefix.cuh).
#include "paged_prefix.cuh"

namespace rqk {
namespace prefix {

cudaError_t launch_f32(const Params& p, int ctas, cudaStream_t s) {
  switch (p.kv.head_dim) {
    case 32: return launch<float, 32>(p, ctas, s);
    case 64: return launch<float, 64>(p, ctas, s);
    default: return launch<float, 128>(p, ctas, s);
  }
}

}  // namespace prefix
}  // namespace rqk
