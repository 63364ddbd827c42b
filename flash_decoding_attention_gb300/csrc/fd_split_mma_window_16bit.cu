// fd_split_mma_window_16bit.cu -- the tensor-core split kernel's sliding-window variants for
// fp16 and bf16 caches (see fd_split_mma.cuh).
#include "fd_split_mma.cuh"

namespace fd {
namespace mma {

cudaError_t launch_window_16bit(const Params& p, const Shape& sh, const Maps& m, cudaStream_t st) {
  return p.kv_dtype == FD_F16 ? launch_window<FD_F16, __half, false>(p, sh, m, st)
                              : launch_window<FD_BF16, __nv_bfloat16, false>(p, sh, m, st);
}

}  // namespace mma
}  // namespace fd
