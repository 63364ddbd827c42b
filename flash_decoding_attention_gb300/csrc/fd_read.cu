// fd_read.cu -- reads cached K and V rows back as packed 16-bit rows.
//
//   k = round16(k_scale * ks * dec(code)), v likewise, every product one fp32
//   operation; ks per tensor (1), KV head or token.
//
// A copy with a widening: the floor is the DRAM traffic of codes, scales and
// output rows.  A thread takes 16 elements of one head of K and of V (one
// 16-byte load of 8-bit codes each, two of 16-bit elements), so a head's row
// is read and written by neighbouring threads in full lines.
#include <type_traits>

#include "fd_prompt.cuh"

namespace fd {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 64;   // packed rows of a block

// Four 8-bit codes (low byte first) as fp32.
__device__ __forceinline__ void decode4(uint32_t w, int kvt, float* x) {
  if (kvt == FD_E4M3) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
          static_cast<__nv_fp8x2_storage_t>((w >> (16 * i)) & 0xffffu), __NV_E4M3);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = i8_to_f32(w >> (8 * i));
  }
}

template <typename T>
__device__ __forceinline__ float2 two_of(uint32_t w) {
  if constexpr (std::is_same<T, __half>::value)
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  else
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}

template <typename T>
__device__ __forceinline__ uint32_t round2(float a, float b) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

template <int KVT, typename OT>
__device__ __forceinline__ void load16(const void* cache, long long at, uint4& w0, uint4& w1) {
  if constexpr (KVT == FD_E4M3 || KVT == FD_I8) {
    w0 = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(cache) + at);
  } else {
    w0 = *reinterpret_cast<const uint4*>(static_cast<const OT*>(cache) + at);
    w1 = *reinterpret_cast<const uint4*>(static_cast<const OT*>(cache) + at + 8);
  }
}

template <int KVT, typename OT>
__device__ __forceinline__ void store16(void* out, long long at, const uint4& w0, const uint4& w1,
                                        float scale) {
  const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
  uint32_t r[8];
  if constexpr (KVT == FD_E4M3 || KVT == FD_I8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x[4];
      decode4(w[i], KVT, x);
      r[2 * i] = round2<OT>(__fmul_rn(x[0], scale), __fmul_rn(x[1], scale));
      r[2 * i + 1] = round2<OT>(__fmul_rn(x[2], scale), __fmul_rn(x[3], scale));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = two_of<OT>(w[i]);
      r[i] = round2<OT>(__fmul_rn(f.x, scale), __fmul_rn(f.y, scale));
    }
  }
  uint4* d = reinterpret_cast<uint4*>(static_cast<OT*>(out) + at);
  d[0] = make_uint4(r[0], r[1], r[2], r[3]);
  d[1] = make_uint4(r[4], r[5], r[6], r[7]);
}

constexpr long long kSkip = -2;   // the row belongs to no sequence: left as it was

template <int KVT, typename OT, int D>
__global__ void __launch_bounds__(kThreads) read_kv_kernel(const __grid_constant__ ReadKv p,
                                                           int per_block) {
  constexpr int TPH = D / 16;
  __shared__ long long src_row[kMaxRows];
  const int i0 = blockIdx.x * per_block;
  const int n = min(per_block, p.rows - i0);
  if (threadIdx.x < n) {
    const int i = i0 + threadIdx.x;
    long long row = kSkip;
    const int b = owner_of(p.out_start, p.at.batch, i);
    if (b >= 0) {
      const int lo = __ldg(p.out_start + b), hi = __ldg(p.out_start + b + 1);
      const int f = p.first ? __ldg(p.first + b) : 0;
      if (lo < 0 || hi > p.rows) {
        raise_error(p.at.ws, kErrBounds, lo < 0 ? lo : hi);
      } else if (f >= 0) {
        const long long t = (long long)f + (i - lo);
        if (t > 0x7fffffffll) {
          raise_error(p.at.ws, kErrBounds, t);
          row = -1;
        } else {
          row = placed_row(p.at, b, (int)t);
        }
      }
    }
    src_row[threadIdx.x] = row;
  }
  __syncthreads();
  const int per_row = p.num_kv_heads * TPH;
  const int items = n * per_row;
  for (int x = threadIdx.x; x < items; x += kThreads) {
    const int r = x / per_row, e = x - r * per_row;   // e = head * TPH + part
    const long long row = src_row[r];
    if (row == kSkip) continue;
    const long long to = ((long long)(i0 + r) * per_row + e) * 16;
    uint4 ka = make_uint4(0, 0, 0, 0), kb = ka, va = ka, vb = ka;
    float ks = p.k_scale, vs = p.v_scale;
    if (row >= 0) {
      const long long from = (row * per_row + e) * 16;
      load16<KVT, OT>(p.k_cache, from, ka, kb);
      load16<KVT, OT>(p.v_cache, from, va, vb);
      if (p.scale_kind != FD_SCALE_TENSOR) {
        const int h = e / TPH;
        const long long at = p.scale_kind == FD_SCALE_HEAD ? h : row * p.num_kv_heads + h;
        ks = __fmul_rn(ks, __ldg(p.k_scales + at));
        vs = __fmul_rn(vs, __ldg(p.v_scales + at));
      }
      store16<KVT, OT>(p.k_out, to, ka, kb, ks);
      store16<KVT, OT>(p.v_out, to, va, vb, vs);
    } else {
      uint4* dk = reinterpret_cast<uint4*>(static_cast<OT*>(p.k_out) + to);
      uint4* dv = reinterpret_cast<uint4*>(static_cast<OT*>(p.v_out) + to);
      dk[0] = dk[1] = dv[0] = dv[1] = ka;
    }
  }
}

template <int KVT, typename OT>
cudaError_t launch_t(const ReadKv& p, int sms, cudaStream_t stream) {
  // rows enough for eight blocks per SM, at most kMaxRows a block
  int per_block = p.rows / (8 * sms);
  per_block = per_block < 1 ? 1 : per_block > kMaxRows ? kMaxRows : per_block;
  const unsigned blocks = (unsigned)((p.rows + per_block - 1) / per_block);
  if (p.head_dim == 128)
    read_kv_kernel<KVT, OT, 128><<<blocks, kThreads, 0, stream>>>(p, per_block);
  else
    read_kv_kernel<KVT, OT, 64><<<blocks, kThreads, 0, stream>>>(p, per_block);
  return cudaGetLastError();
}

template <typename OT>
cudaError_t launch_o(const ReadKv& p, int sms, cudaStream_t stream) {
  if (p.kv_dtype == FD_E4M3) return launch_t<FD_E4M3, OT>(p, sms, stream);
  if (p.kv_dtype == FD_I8) return launch_t<FD_I8, OT>(p, sms, stream);
  if constexpr (std::is_same<OT, __half>::value) return launch_t<FD_F16, OT>(p, sms, stream);
  else return launch_t<FD_BF16, OT>(p, sms, stream);
}

}  // namespace

cudaError_t launch_read_kv(const ReadKv& p, int sms, cudaStream_t stream) {
  return p.out_dtype == FD_F16 ? launch_o<__half>(p, sms, stream)
                               : launch_o<__nv_bfloat16>(p, sms, stream);
}

}  // namespace fd
