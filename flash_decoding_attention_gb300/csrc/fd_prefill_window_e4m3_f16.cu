// fd_prefill_window_e4m3_f16.cu -- the attention kernel's variants (fd_prefill.cuh) with a sliding window
// for e4m3 caches with f16 queries.
#include "fd_prefill.cuh"

namespace fd {
namespace pf {

cudaError_t launch_window_e4m3_f16(const Prefill& p, const CUtensorMap* maps, cudaStream_t stream) {
  return launch_8<1, false, true>(p, maps, stream);
}

}  // namespace pf
}  // namespace fd
