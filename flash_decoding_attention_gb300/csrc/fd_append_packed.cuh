// fd_append_packed.cuh -- elements of a head's row in the packed append's
// kernels (fd_append_packed.cu, fd_append_normed.cu): 16-bit elements in and
// out, and 8-bit codes.
//
// Each product, sum and quotient is a separate round-to-nearest fp32
// operation, so the codes can be reproduced off the device.
#pragma once

#include <type_traits>

#include "fd_prompt.cuh"

namespace fd {

template <typename XT>
__device__ __forceinline__ void unpack8(const uint4& w, float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 f;
    if constexpr (std::is_same<XT, __half>::value)
      f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    else
      f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <typename XT>
__device__ __forceinline__ uint4 pack8(const float* x) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same<XT, __half>::value) {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// Eight quotients x / s as 8-bit codes.
template <int KVT>
__device__ __forceinline__ uint2 encode8(const float* x, float s) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float a = __fdiv_rn(x[i], s), b = __fdiv_rn(x[i + 1], s);
    uint32_t two;
    if constexpr (KVT == FD_E4M3) {
      two = static_cast<uint32_t>(
          __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3));
    } else {
      const int ia = min(max(__float2int_rn(a), -127), 127);
      const int ib = min(max(__float2int_rn(b), -127), 127);
      two = (static_cast<uint32_t>(ia) & 0xffu) | ((static_cast<uint32_t>(ib) & 0xffu) << 8);
    }
    w[i >> 2] |= two << (16 * ((i >> 1) & 1));
  }
  return make_uint2(w[0], w[1]);
}

}  // namespace fd
