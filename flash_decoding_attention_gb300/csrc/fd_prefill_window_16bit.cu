// fd_prefill_window_16bit.cu -- the attention kernel's variants (fd_prefill.cuh) with a sliding window
// for 16-bit caches.
#include "fd_prefill.cuh"

namespace fd {
namespace pf {

cudaError_t launch_window_16bit(const Prefill& p, const CUtensorMap* maps, cudaStream_t stream) {
  return launch_16bit<true>(p, maps, stream);
}

}  // namespace pf
}  // namespace fd
