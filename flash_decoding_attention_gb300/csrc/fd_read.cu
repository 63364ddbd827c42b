// fd_read.cu -- reads cached K and V rows back as packed 16-bit rows.
//
//   k = round16(k_scale * ks * dec(code)), v likewise, every product one fp32
//   operation; ks per tensor (1), KV head or token.
//
// A copy with a widening: the floor is the DRAM traffic of codes, scales and
// output rows.  A thread takes 8 elements of one head of K and of V, so its
// stores are 16 bytes beside its neighbours' (whole lines) and its loads 8 or
// 16; four rows are in flight at a time.  Its place in a row is fixed, so the
// head is known once.  1.1 GB (e4m3 pages to bf16) take 175 us, 6.3 TB/s, 0.93
// of the measured copy rate; 16 elements a thread took 208 us.
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

// 8 elements from `at` on: 8-bit codes in w.x, w.y, or 16-bit elements.
template <int KVT, typename OT>
__device__ __forceinline__ uint4 load8(const void* cache, long long at) {
  if constexpr (KVT == FD_E4M3 || KVT == FD_I8) {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(cache) + at);
    return make_uint4(w.x, w.y, 0, 0);
  } else {
    return *reinterpret_cast<const uint4*>(static_cast<const OT*>(cache) + at);
  }
}

template <int KVT, typename OT>
__device__ __forceinline__ uint4 decode8(const uint4& v, float scale) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t r[4];
  if constexpr (KVT == FD_E4M3 || KVT == FD_I8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float x[4];
      decode4(w[i], KVT, x);
      r[2 * i] = round2<OT>(__fmul_rn(x[0], scale), __fmul_rn(x[1], scale));
      r[2 * i + 1] = round2<OT>(__fmul_rn(x[2], scale), __fmul_rn(x[3], scale));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = two_of<OT>(w[i]);
      r[i] = round2<OT>(__fmul_rn(f.x, scale), __fmul_rn(f.y, scale));
    }
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

constexpr long long kSkip = -2;   // the row belongs to no sequence: left as it was

template <int KVT, typename OT, int D>
__global__ void __launch_bounds__(kThreads) read_kv_kernel(const __grid_constant__ ReadKv p,
                                                           int per_block) {
  constexpr int TPH = D / 8, kFlight = 4;
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
      if (lo >= 0 && hi <= p.rows && f >= 0) {   // (else recorded by check_starts)
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
  if (blockIdx.x == 0) check_starts(p.at, p.out_start, p.rows);
  __syncthreads();
  const int per_row = p.num_kv_heads * TPH;   // threads of a row
  // narrow rows: several at a time; wide ones: several passes over each
  const int rows_at_once = per_row < kThreads ? kThreads / per_row : 1;
  const int r0 = per_row < kThreads ? threadIdx.x / per_row : 0;
  if (r0 >= rows_at_once) return;
  for (int e = threadIdx.x - r0 * per_row; e < per_row; e += kThreads) {
    const int h = e / TPH;
    for (int r = r0; r < n; r += kFlight * rows_at_once) {
      uint4 k[kFlight], v[kFlight];
      float ks[kFlight], vs[kFlight];
      long long row[kFlight];
#pragma unroll
      for (int x = 0; x < kFlight; ++x) {
        const int q = r + x * rows_at_once;
        row[x] = q < n ? src_row[q] : kSkip;
        k[x] = v[x] = make_uint4(0, 0, 0, 0);
        ks[x] = p.k_scale;
        vs[x] = p.v_scale;
        if (row[x] < 0) continue;
        const long long from = (row[x] * per_row + e) * 8;
        k[x] = load8<KVT, OT>(p.k_cache, from);
        v[x] = load8<KVT, OT>(p.v_cache, from);
        if (p.scale_kind != FD_SCALE_TENSOR) {
          const long long at = p.scale_kind == FD_SCALE_HEAD ? h : row[x] * p.num_kv_heads + h;
          ks[x] = __fmul_rn(ks[x], __ldg(p.k_scales + at));
          vs[x] = __fmul_rn(vs[x], __ldg(p.v_scales + at));
        }
      }
#pragma unroll
      for (int x = 0; x < kFlight; ++x) {
        if (row[x] == kSkip) continue;
        const long long to = ((long long)(i0 + r + x * rows_at_once) * per_row + e) * 8;
        // (a row that is not there: zero bits stay zero)
        *reinterpret_cast<uint4*>(static_cast<OT*>(p.k_out) + to) =
            row[x] < 0 ? k[x] : decode8<KVT, OT>(k[x], ks[x]);
        *reinterpret_cast<uint4*>(static_cast<OT*>(p.v_out) + to) =
            row[x] < 0 ? v[x] : decode8<KVT, OT>(v[x], vs[x]);
      }
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
