// fd_append_packed_ext.cu -- the packed append's variants (fd_append_packed.cuh)
// with norms of query and key heads and rotary positions on several axes.
#include "fd_append_packed.cuh"

namespace fd {

cudaError_t launch_append_packed_ext(const AppendPacked& p, int sms, cudaStream_t stream) {
  return p.new_dtype == FD_F16 ? launch_x<__half, true>(p, sms, stream)
                               : launch_x<__nv_bfloat16, true>(p, sms, stream);
}

}  // namespace fd
