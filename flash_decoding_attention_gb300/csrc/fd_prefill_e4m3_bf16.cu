// fd_prefill_e4m3_bf16.cu -- the attention kernel's variants (fd_prefill.cuh)
// for e4m3 caches with bf16 queries.
#include "fd_prefill.cuh"

namespace fd {
namespace pf {

cudaError_t launch_e4m3_bf16(const Prefill& p, const CUtensorMap* maps, cudaStream_t stream) {
  return p.head_dim == 128 ? launch_8<128, 1, true>(p, maps, stream)
                           : launch_8<64, 1, true>(p, maps, stream);
}

}  // namespace pf
}  // namespace fd
