// fd_prefill.cu -- attention of packed new tokens over the cache.
//
//   s_t = softmax_scale k_scale ks_t (q . k_t),  t <= position of the token,
//   out = v_scale sum_t 2^(s_t log2 e - m) vs_t v_t / l,
//   l = sum_t 2^(s_t log2 e - m),  lse = (m + log2 l) ln 2,
// in one pass over the keys with the running maximum m and sum l.
//
// One warp per (token, query head): the lanes share the head's dims, a dot
// product is a warp reduction, everything in fp32.
#include <type_traits>

#include "fd_prompt.cuh"

namespace fd {
namespace {

constexpr int kWarps = 8;

template <int KVT, typename QT, int DPL>
__device__ __forceinline__ void load_dims(const void* cache, long long at, float* x) {
#pragma unroll
  for (int i = 0; i < DPL; ++i) {
    if constexpr (KVT == FD_E4M3) {
      __nv_fp8_e4m3 c;
      c.__x = static_cast<const uint8_t*>(cache)[at + i];
      x[i] = static_cast<float>(c);
    } else if constexpr (KVT == FD_I8) {
      x[i] = static_cast<float>(static_cast<const int8_t*>(cache)[at + i]);
    } else {
      x[i] = QType<QT>::to_f32(static_cast<const QT*>(cache)[at + i]);
    }
  }
}

template <int KVT, typename QT, int D>
__global__ void __launch_bounds__(kWarps * 32) prefill_kernel(const __grid_constant__ Prefill p) {
  constexpr int DPL = D / 32;
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (item >= (long long)p.tokens * p.num_q_heads) return;
  const int i = (int)(item / p.num_q_heads), h = (int)(item - (long long)i * p.num_q_heads);
  const int b = owner_of(p.q_start, p.at.batch, i);
  if (b < 0) return;
  const int lo = __ldg(p.q_start + b), hi = __ldg(p.q_start + b + 1);
  if (lo < 0 || hi > p.tokens) {
    raise_error(p.at.ws, kErrBounds, lo < 0 ? lo : hi);
    return;
  }
  const int T = max(0, __ldg(p.seq_len + b));
  const int seen = T - (hi - 1 - i);   // keys this token attends to
  const int kvh = h / p.group;
  float q[DPL], o[DPL];
  const QT* qp = static_cast<const QT*>(p.q) + (long long)i * p.q_stride + (long long)h * D;
#pragma unroll
  for (int k = 0; k < DPL; ++k) {
    q[k] = QType<QT>::to_f32(qp[lane * DPL + k]);
    o[k] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int t = 0; t < seen; ++t) {
    const long long row = placed_row(p.at, b, t);
    if (row < 0) continue;
    const long long at = (row * p.num_kv_heads + kvh) * D + lane * DPL;
    float x[DPL];
    load_dims<KVT, QT, DPL>(p.k, at, x);
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < DPL; ++k) s = fmaf(q[k], x[k], s);
#pragma unroll
    for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    s *= p.score_scale;
    float vs = p.v_scale;
    if (p.scale_kind != FD_SCALE_TENSOR) {
      const long long sa = p.scale_kind == FD_SCALE_HEAD ? kvh : row * p.num_kv_heads + kvh;
      s *= __ldg(p.k_scales + sa);
      vs *= __ldg(p.v_scales + sa);
    }
    const float mn = fmaxf(m, s);
    const float f = m == -INFINITY ? 0.f : exp2f(m - mn), e = exp2f(s - mn);
    m = mn;
    l = fmaf(l, f, e);
    load_dims<KVT, QT, DPL>(p.v, at, x);
#pragma unroll
    for (int k = 0; k < DPL; ++k) o[k] = fmaf(o[k], f, e * vs * x[k]);
  }
  QT* op = static_cast<QT*>(p.out) + ((long long)i * p.num_q_heads + h) * D;
  const float r = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int k = 0; k < DPL; ++k) op[lane * DPL + k] = QType<QT>::from_f32(o[k] * r);
  if (p.lse && lane == 0)
    p.lse[(long long)i * p.num_q_heads + h] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

template <int KVT, typename QT>
cudaError_t launch_t(const Prefill& p, cudaStream_t stream) {
  const long long items = (long long)p.tokens * p.num_q_heads;
  const unsigned blocks = (unsigned)((items + kWarps - 1) / kWarps);
  if (p.head_dim == 128) prefill_kernel<KVT, QT, 128><<<blocks, kWarps * 32, 0, stream>>>(p);
  else prefill_kernel<KVT, QT, 64><<<blocks, kWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename QT>
cudaError_t launch_q(const Prefill& p, cudaStream_t stream) {
  if (p.kv_dtype == FD_E4M3) return launch_t<FD_E4M3, QT>(p, stream);
  if (p.kv_dtype == FD_I8) return launch_t<FD_I8, QT>(p, stream);
  if constexpr (std::is_same<QT, __half>::value) return launch_t<FD_F16, QT>(p, stream);
  else return launch_t<FD_BF16, QT>(p, stream);
}

}  // namespace

size_t prefill_workspace(int head_dim, int sms) {
  (void)head_dim;
  (void)sms;
  return sizeof(WsHeader);
}

cudaError_t launch_prefill(const Prefill& p, cudaStream_t stream) {
  return p.q_dtype == FD_F16 ? launch_q<__half>(p, stream) : launch_q<__nv_bfloat16>(p, stream);
}

}  // namespace fd
