// fd_split_mma_window_e4m3.cu -- the tensor-core split kernel's sliding-window variants for
// e4m3 caches (see fd_split_mma.cuh).
#include "fd_split_mma.cuh"

namespace fd {
namespace mma {

cudaError_t launch_window_e4m3(const Params& p, const Shape& sh, const Maps& m, cudaStream_t st) {
  const bool tok = p.scale_kind == FD_SCALE_TOKEN;
  if (p.q_dtype == FD_F16)
    return tok ? launch_window<FD_E4M3, __half, true>(p, sh, m, st)
               : launch_window<FD_E4M3, __half, false>(p, sh, m, st);
  return tok ? launch_window<FD_E4M3, __nv_bfloat16, true>(p, sh, m, st)
             : launch_window<FD_E4M3, __nv_bfloat16, false>(p, sh, m, st);
}

}  // namespace mma
}  // namespace fd
