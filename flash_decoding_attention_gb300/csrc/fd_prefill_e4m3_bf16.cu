// fd_prefill_e4m3_bf16.cu -- the attention kernel's variants (fd_prefill.cuh)
// for e4m3 caches with bf16 queries.
#include "fd_prefill.cuh"

namespace fd {
namespace pf {

cudaError_t launch_plain_e4m3_bf16(const Prefill& p, const CUtensorMap* maps, cudaStream_t stream) {
  return launch_8<1, true, false>(p, maps, stream);
}

}  // namespace pf
}  // namespace fd
