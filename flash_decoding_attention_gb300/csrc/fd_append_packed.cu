// fd_append_packed.cu -- packed new tokens into the KV cache: rotary
// positions on query and key heads, 16-bit or quantised cache rows.
//
// A token's work is its query, key and value heads; a thread takes 16
// elements of one head as two 16-byte chunks, one of each half of the rotated
// part, so both members of every rotary pair are in its hands (pairs half the
// rotated part apart: element by element; neighbouring pairs: inside each
// chunk) and a head's threads touch whole lines.  The D / 16 threads of a head
// sit in one warp, so the per-token scale is a warp reduction.  A thread keeps
// its place inside the head for the whole block, so the 8 + 8 table values of
// a token are loaded once and serve all its heads; two heads are in flight at
// a time.  Everything is read and written once: DRAM traffic is the floor.
// About 14000 tokens of 32 query and 8 KV heads of 128, bf16 into bf16 (347 MB
// both ways), take 63 us, 5.5 TB/s; small batches are bound by the launch.
//
// Each product, sum and quotient is a separate round-to-nearest fp32
// operation, so the codes can be reproduced off the device.
#include "fd_append_packed.cuh"

namespace fd {
namespace {

constexpr int kMaxThreads = 512;

// The pairs of the thread's 16 elements turned by their angles (interleaved:
// chunk a holds pairs 0..3 of c and s, chunk b pairs 4..7).
template <bool INTERLEAVED>
__device__ __forceinline__ void rotate16(float* a, float* b, const float* c, const float* s) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float* x = INTERLEAVED ? (i < 4 ? a + 2 * i : b + 2 * (i - 4)) : a + i;
    float* y = INTERLEAVED ? x + 1 : b + i;
    const float x1 = *x, x2 = *y;
    *x = __fsub_rn(__fmul_rn(x1, c[i]), __fmul_rn(x2, s[i]));
    *y = __fadd_rn(__fmul_rn(x2, c[i]), __fmul_rn(x1, s[i]));
  }
}

struct TokenAt {
  long long row;   // cache row, < 0: leave the token alone
  int pos;
};

// Token i's cache row and position; every reason to leave it alone gives -1.
__device__ __forceinline__ TokenAt place_token(const AppendPacked& p, int i) {
  TokenAt t{-1, 0};
  const int b = owner_of(p.q_start, p.at.batch, i);
  if (b < 0) return t;
  const int lo = __ldg(p.q_start + b), hi = __ldg(p.q_start + b + 1);
  if (lo < 0 || hi > p.tokens) return t;   // (recorded by check_starts)
  const int first = __ldg(p.positions + b);
  if (first < 0) return t;
  const long long pos = (long long)first + (i - lo);
  if (pos > 0x7fffffffll || (p.rotary && pos >= p.rotary_positions)) {
    raise_error(p.at.ws, kErrBounds, pos);
    return t;
  }
  t.pos = (int)pos;
  t.row = placed_row(p.at, b, t.pos);
  return t;
}

constexpr int kMaxTokens = 4;   // of a block (8: 69 us for those 347 MB, 4: 63 us)

// gridDim.x blocks of `per_block` tokens; gridDim.y parts of a token's heads.
template <typename XT, int KVT, int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kMaxThreads, 2) append_packed_kernel(const __grid_constant__ AppendPacked p,
                                                                    int per_block) {
  constexpr int TPH = D / 16;                        // threads per head
  const int hpp = blockDim.x / TPH;                  // heads per pass
  __shared__ TokenAt at[kMaxTokens];
  const int t0 = blockIdx.x * per_block;
  const int n = min(per_block, p.tokens - t0);
  if (threadIdx.x < n) at[threadIdx.x] = place_token(p, t0 + threadIdx.x);
  if (blockIdx.x == 0 && blockIdx.y == 0) check_starts(p.at, p.q_start, p.tokens);
  __syncthreads();
  const int u = threadIdx.x % TPH, h0 = threadIdx.x / TPH;
  const int half = p.rot_dim / 2;
  const int turned = p.rot_dim / 16;                 // threads of a head that rotate
  // this thread's chunks (8 elements each): one of each half of the rotated
  // part, or of the rest
  const bool turns = u < turned;
  const int ea = turns ? 8 * u : p.rot_dim + 8 * (u - turned);
  const int eb = ea + (turns ? half : (D - p.rot_dim) / 2);
  const int heads = p.num_q_heads + 2 * p.num_kv_heads;
  const int per_part = (heads + gridDim.y - 1) / gridDim.y;
  const int h_begin = blockIdx.y * per_part, h_end = min(heads, h_begin + per_part);

  auto is_query = [&](int h) { return h < p.num_q_heads; };
  auto is_key = [&](int h) { return h >= p.num_q_heads && h < p.num_q_heads + p.num_kv_heads; };
  auto kv_head = [&](int h) { return h - p.num_q_heads - (is_key(h) ? 0 : p.num_kv_heads); };
  auto load = [&](long long token, int h, uint4& wa, uint4& wb) {
    wa = wb = make_uint4(0, 0, 0, 0);
    if (h >= h_end) return;
    const XT* src = is_query(h)
                        ? static_cast<const XT*>(p.q) + token * p.q_stride + (long long)h * D
                        : static_cast<const XT*>(is_key(h) ? p.k_new : p.v_new) +
                              token * p.kv_stride + (long long)kv_head(h) * D;
    wa = *reinterpret_cast<const uint4*>(src + ea);
    wb = *reinterpret_cast<const uint4*>(src + eb);
  };
  for (int i = 0; i < n; ++i) {
    const TokenAt where = at[i];
    if (where.row < 0) continue;
    const long long token = t0 + i;
    float c[8], s[8];
    if (turns) {
      const float* r = p.rotary + (long long)where.pos * p.rot_dim;
#pragma unroll
      for (int k = 0; k < 8; k += 4) {
        // pairs of chunk a and b: 8 u .. 8 u + 7, or 4 u .. and half / 2 + 4 u ..
        const int pair = INTERLEAVED ? 4 * u + (k ? half / 2 : 0) : 8 * u + k;
        const float4 x = __ldg(reinterpret_cast<const float4*>(r + pair));
        const float4 y = __ldg(reinterpret_cast<const float4*>(r + half + pair));
        c[k] = x.x; c[k + 1] = x.y; c[k + 2] = x.z; c[k + 3] = x.w;
        s[k] = y.x; s[k + 1] = y.y; s[k + 2] = y.z; s[k + 3] = y.w;
      }
    }
    // one head, loaded: turned, rounded or quantised, stored.  Every lane of
    // the warp comes here (the amax is a warp reduction).
    auto finish = [&](int h, const uint4& wa, const uint4& wb) {
      const bool live = h < h_end, is_q = is_query(h), is_k = is_key(h);
      const int kvh = kv_head(h);
      const bool rot = turns && (is_q || is_k);
      float a[8], b[8];
      unpack8<XT>(wa, a);
      unpack8<XT>(wb, b);
      if (rot) rotate16<INTERLEAVED>(a, b, c, s);
      const long long srow = where.row * p.num_kv_heads + kvh;
      if (live && (is_q || KVT == FD_F16 || KVT == FD_BF16)) {
        XT* dst = is_q ? static_cast<XT*>(p.q_out) + (token * p.num_q_heads + h) * D
                       : static_cast<XT*>(is_k ? p.k_cache : p.v_cache) + srow * D;
        *reinterpret_cast<uint4*>(dst + ea) = rot ? pack8<XT>(a) : wa;
        *reinterpret_cast<uint4*>(dst + eb) = rot ? pack8<XT>(b) : wb;
      }
      if constexpr (KVT == FD_E4M3 || KVT == FD_I8) {
        float scale = is_k ? p.k_scale : p.v_scale;
        if (p.scale_kind == FD_SCALE_TOKEN) {
          float amax = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fmaxf(fabsf(a[k]), fabsf(b[k])));
#pragma unroll
          for (int o = TPH / 2; o; o >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          const float qmax = KVT == FD_I8 ? 127.f : 448.f;
          const float ks = amax > 0.f ? __fdiv_rn(amax, __fmul_rn(qmax, scale)) : 1.f;
          if (live && !is_q && u == 0) (is_k ? p.k_scales : p.v_scales)[srow] = ks;
          scale = __fmul_rn(scale, ks);
        } else if (p.scale_kind == FD_SCALE_HEAD && live && !is_q) {
          scale = __fmul_rn(scale, __ldg((is_k ? p.k_scales : p.v_scales) + kvh));
        }
        if (live && !is_q) {
          uint8_t* dst = static_cast<uint8_t*>(is_k ? p.k_cache : p.v_cache) + srow * D;
          *reinterpret_cast<uint2*>(dst + ea) = encode8<KVT>(a, scale);
          *reinterpret_cast<uint2*>(dst + eb) = encode8<KVT>(b, scale);
        }
      }
    };
    for (int h = h_begin + h0; h - h0 < h_end; h += 2 * hpp) {
      uint4 wa[2], wb[2];
      load(token, h, wa[0], wb[0]);
      load(token, h + hpp, wa[1], wb[1]);
      finish(h, wa[0], wb[0]);
      if (h - h0 + hpp < h_end) finish(h + hpp, wa[1], wb[1]);
    }
  }
}

template <typename XT, int KVT, int D>
cudaError_t launch_d(const AppendPacked& p, int sms, cudaStream_t stream) {
  // Blocks enough to fill the SMs: several tokens a block when there are many,
  // several blocks a token when there are few.
  const int heads = p.num_q_heads + 2 * p.num_kv_heads;
  int per_block = p.tokens / (8 * sms);
  per_block = per_block < 1 ? 1 : per_block > kMaxTokens ? kMaxTokens : per_block;
  const int blocks = (p.tokens + per_block - 1) / per_block;
  const int warps_token = (heads * (D / 16) + 31) / 32;   // warps of one token
  int parts = blocks >= 4 * sms ? 1 : (4 * sms + blocks - 1) / blocks;
  const int most = (warps_token + 3) / 4;                 // parts of four warps at least
  if (parts > most) parts = most;
  // threads that pass a part's heads in equal, full passes of two heads each
  const int warps_part = ((heads + parts - 1) / parts * (D / 16) + 31) / 32;
  const int passes = (warps_part + kMaxThreads / 32 - 1) / (kMaxThreads / 32);
  int warps = (warps_part + passes - 1) / passes;
  if (passes == 1 && warps > 4) warps = (warps + 1) / 2;  // two heads a thread
  const dim3 grid((unsigned)blocks, (unsigned)parts);
  if (p.interleaved)
    append_packed_kernel<XT, KVT, D, true><<<grid, warps * 32, 0, stream>>>(p, per_block);
  else
    append_packed_kernel<XT, KVT, D, false><<<grid, warps * 32, 0, stream>>>(p, per_block);
  return cudaGetLastError();
}

template <typename XT, int KVT>
cudaError_t launch_t(const AppendPacked& p, int sms, cudaStream_t stream) {
  return p.head_dim == 128 ? launch_d<XT, KVT, 128>(p, sms, stream)
                           : launch_d<XT, KVT, 64>(p, sms, stream);
}

template <typename XT>
cudaError_t launch_x(const AppendPacked& p, int sms, cudaStream_t stream) {
  if (p.kv_dtype == FD_E4M3) return launch_t<XT, FD_E4M3>(p, sms, stream);
  if (p.kv_dtype == FD_I8) return launch_t<XT, FD_I8>(p, sms, stream);
  if constexpr (std::is_same<XT, __half>::value) return launch_t<XT, FD_F16>(p, sms, stream);
  else return launch_t<XT, FD_BF16>(p, sms, stream);
}

}  // namespace

cudaError_t launch_append_packed(const AppendPacked& p, int sms, cudaStream_t stream) {
  if (p.q_norm || p.k_norm || p.num_axes > 0) return launch_append_normed(p, sms, stream);
  return p.new_dtype == FD_F16 ? launch_x<__half>(p, sms, stream)
                               : launch_x<__nv_bfloat16>(p, sms, stream);
}

}  // namespace fd
