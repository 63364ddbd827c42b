// fd_prefill_window_i8_bf16.cu -- the attention kernel's variants (fd_prefill.cuh) with a sliding window
// for i8 caches with bf16 queries.
#include "fd_prefill.cuh"

namespace fd {
namespace pf {

cudaError_t launch_window_i8_bf16(const Prefill& p, const CUtensorMap* maps, cudaStream_t stream) {
  return launch_8<2, true, true>(p, maps, stream);
}

}  // namespace pf
}  // namespace fd
