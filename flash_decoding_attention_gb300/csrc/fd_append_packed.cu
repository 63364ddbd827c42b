// fd_append_packed.cu -- the packed append's variants (fd_append_packed.cuh)
// without norms and axes, and the choice between these and the others.
#include "fd_append_packed.cuh"

namespace fd {

cudaError_t launch_append_packed_ext(const AppendPacked& p, int sms, cudaStream_t stream);

cudaError_t launch_append_packed(const AppendPacked& p, int sms, cudaStream_t stream) {
  if (p.q_norm || p.k_norm || p.num_axes > 0) return launch_append_packed_ext(p, sms, stream);
  return p.new_dtype == FD_F16 ? launch_x<__half, false>(p, sms, stream)
                               : launch_x<__nv_bfloat16, false>(p, sms, stream);
}

}  // namespace fd
