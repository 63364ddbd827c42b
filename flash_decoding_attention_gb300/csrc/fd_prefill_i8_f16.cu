// fd_prefill_i8_f16.cu -- the attention kernel's variants (fd_prefill.cuh)
// for i8 caches with f16 queries.
#include "fd_prefill.cuh"

namespace fd {
namespace pf {

cudaError_t launch_i8_f16(const Prefill& p, const CUtensorMap* maps, cudaStream_t stream) {
  return p.head_dim == 128 ? launch_8<128, 2, false>(p, maps, stream)
                           : launch_8<64, 2, false>(p, maps, stream);
}

}  // namespace pf
}  // namespace fd
