// fd_prefill_16bit.cu -- the attention kernel's variants (fd_prefill.cuh) for
// 16-bit caches.
#include "fd_prefill.cuh"

namespace fd {
namespace pf {

cudaError_t launch_16bit(const Prefill& p, const CUtensorMap* maps, cudaStream_t stream) {
  if (p.q_dtype == FD_BF16)
    return p.head_dim == 128 ? launch_16<128, true>(p, maps, stream)
                             : launch_16<64, true>(p, maps, stream);
  return p.head_dim == 128 ? launch_16<128, false>(p, maps, stream)
                           : launch_16<64, false>(p, maps, stream);
}

}  // namespace pf
}  // namespace fd
