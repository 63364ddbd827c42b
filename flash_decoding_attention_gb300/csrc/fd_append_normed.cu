// fd_append_normed.cu -- packed new tokens into the KV cache with norms of query
// and key heads and rotary positions on several axes.
//
// A head of D elements is y = x / sqrt(sum x^2 / D + eps) * w, then its pairs are
// turned, then it is rounded or quantised.  As in the plain append a thread takes
// 16 elements of a head as two 16-byte chunks, one of each half of the rotated
// part; a head's D / 16 threads sit in one warp, so the norm and the per-token
// scale are warp reductions.
//
// A square of a 16-bit element is exact in fp32 (from 2^-149 up), and their sum is
// kept as two floats: the rounding error of every addition, itself exact, is added
// up beside it.  What the second float's own additions lose is below 2^-40 of the
// sum (a thread's 8 additions a lane lose 8 * 2^-24 of errors up to 8 * 2^-24, the
// tree's some 100 * 2^-48), so that the sum rounds like the exact one unless that
// lies as near to the middle of two floats: a plain fp32 sum would move every
// value next to a border of the codes to either side.  The arithmetic runs on
// packed pairs, 3.5 instructions an element for the sum.
//
// An axis only changes which row of the table a pair's cosine and sine come from.
// A block gathers them for its few tokens into shared memory first.  Blocks are
// small, so that some look their tokens up while others work.
//
// Everything is read and written once: DRAM traffic is the floor.  21000 tokens of
// 32 query and 8 KV heads of 128, bf16 into bf16 with both norms (528 MB both
// ways), take 110 us, 4.8 TB/s (the plain append 6.0): issue slots are two thirds
// busy, a third of them with the two-float sum and the division, and 24 warps an SM
// do not hide the rest.  (That is what this kernel executes, 354 instructions a
// thread for 16 elements, not a bound: a thread fetches and packs its weights
// anew for every head.)  Without norms (64 registers, 32 warps) 10000 tokens of 16
// and 4 heads (123 MB) take 27 us, 4.6 TB/s; 64 tokens 4.7 us, a launch and five
// dependent loads.  What did not pay: 128 registers and four heads in flight (171
// us for those 528 MB), 64 and spills (131), persistent blocks with a warp that
// looks tokens up for the others (136).
#include "fd_append_packed.cuh"

namespace fd {
namespace {

constexpr int kThreads = 128;    // of a block at most (256: 1 to 4 % slower)
// Blocks of that size on an SM: 80 registers a thread, or 64 with axes alone
template <bool NORM>
constexpr int kBlocks = NORM ? 6 : 8;
constexpr int kMaxTokens = 4;    // of a block
constexpr int kMaxAxes = 4;

// Eight 16-bit elements <-> four pairs of fp32.
template <typename XT>
__device__ __forceinline__ void unpack_pairs(const uint4& w, uint64_t* x) {
  float f[8];
  unpack8<XT>(w, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = pack2(f[2 * i], f[2 * i + 1]);
}

__device__ __forceinline__ void to_floats(const uint64_t* x, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = unpack2(x[i]);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}

__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {   // a - b, one rounding
  return fma2(b, pack2(-1.f, -1.f), a);
}

// (s, e) += x^2: s + e keeps the sum (but for e's own roundings, 2^-24 of it).
// The error of an addition is itself a float, found by four more operations
// (Knuth's two-sum; x^2 is exact, so the multiplications fold into the additions).
__device__ __forceinline__ void add_square(uint64_t& s, uint64_t& e, uint64_t x) {
  const uint64_t t = fma2(x, x, s), w = sub2(s, t);
  e = add2(e, add2(sub2(s, add2(t, w)), fma2(x, x, w)));
  s = t;
}

// The same for (s, e) += (s2, e2), both non-negative.
__device__ __forceinline__ void add_exact(float& s, float& e, float s2, float e2) {
  // (the larger first: the error is then two operations, and both lanes of an
  // exchange do the same)
  const float hi = fmaxf(s, s2), lo = fminf(s, s2), t = __fadd_rn(s, s2);
  e = __fadd_rn(__fadd_rn(e, e2), __fsub_rn(lo, __fsub_rn(t, hi)));
  s = t;
}

// The factor 1 / sqrt(sum x^2 / D + eps) of a head whose TPH threads hold 16
// elements each; all lanes of the warp take part and get their head's.
template <int D, int TPH>
__device__ __forceinline__ float norm_factor(const uint64_t* a, const uint64_t* b, float eps) {
  uint64_t ss = pack2(0.f, 0.f), ee = ss;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    add_square(ss, ee, a[k]);
    add_square(ss, ee, b[k]);
  }
  const float2 sv = unpack2(ss), ev = unpack2(ee);
  float s = sv.x, e = ev.x;
  add_exact(s, e, sv.y, ev.y);
#pragma unroll
  for (int o = TPH / 2; o; o >>= 1) {
    const float s2 = __shfl_xor_sync(0xffffffffu, s, o), e2 = __shfl_xor_sync(0xffffffffu, e, o);
    add_exact(s, e, s2, e2);
  }
  // past fp32's range (or with a NaN) the errors are NaN: the sum is what it is
  const float sum = fabsf(s) < INFINITY ? __fadd_rn(s, e) : s;
  return __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(sum, 1.f / D), eps)));
}

// a + b and a - b of two products, each rounded by itself (ptxas 13.0 fuses a
// packed product into a packed sum that follows it, rounding modes or not; it
// keeps its hands off single ones).
__device__ __forceinline__ uint64_t sum_apart(uint64_t a, uint64_t b) {
  const float2 x = unpack2(a), y = unpack2(b);
  return pack2(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y));
}
__device__ __forceinline__ uint64_t difference_apart(uint64_t a, uint64_t b) {
  const float2 x = unpack2(a), y = unpack2(b);
  return pack2(__fsub_rn(x.x, y.x), __fsub_rn(x.y, y.y));
}

// The thread's pairs turned by the token's cosines and sines (of `half` pairs each,
// in shared memory): chunk a and chunk b hold the members of pairs 8 u .., or
// with neighbouring pairs 4 u .. and half / 2 + 4 u ...
template <bool INTERLEAVED>
__device__ __forceinline__ void rotate(uint64_t* a, uint64_t* b, const float* cs, int u, int half) {
  if constexpr (INTERLEAVED) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      uint64_t* v = r ? b : a;
      const float* at = cs + 4 * u + (r ? half / 2 : 0);
      const float4 c = *reinterpret_cast<const float4*>(at);
      const float4 s = *reinterpret_cast<const float4*>(at + half);
      const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {   // v[i] is a whole pair (x, y)
        const float2 xy = unpack2(v[i]);
        const float2 c2 = unpack2(mul2(v[i], pack2(cc[i], cc[i])));
        const float2 s2 = unpack2(mul2(pack2(xy.y, xy.x), pack2(ss[i], ss[i])));
        v[i] = pack2(__fsub_rn(c2.x, s2.x), __fadd_rn(c2.y, s2.y));
      }
    }
  } else {
    const float* at = cs + 4 * u;   // (see turn_at)
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(at + i * half / 4);
      const ulonglong2 s = *reinterpret_cast<const ulonglong2*>(at + half + i * half / 4);
      const uint64_t x0 = a[i], y0 = b[i], x1 = a[i + 1], y1 = b[i + 1];
      a[i] = difference_apart(mul2(x0, c.x), mul2(y0, s.x));
      b[i] = sum_apart(mul2(y0, c.x), mul2(x0, s.x));
      a[i + 1] = difference_apart(mul2(x1, c.y), mul2(y1, s.y));
      b[i + 1] = sum_apart(mul2(y1, c.y), mul2(x1, s.y));
    }
  }
}

// Where a pair's cosine lies among the token's (its sine as far behind them): a
// thread's eight pairs half the rotated part apart are two quads, whose first
// ones lie behind one another and so do the second ones (read 16 bytes a lane
// without bank conflicts).
template <bool INTERLEAVED>
__device__ __forceinline__ int turn_at(int pair, int half) {
  return INTERLEAVED ? pair : ((pair >> 2) & 1) * (half / 2) + ((pair >> 3) << 2) + (pair & 3);
}

struct TokenAt {
  long long row;   // cache row, < 0: leave the token alone
  int pos[kMaxAxes];
};

// Token i's cache row and positions, by a warp (lane 0 has the answer); every
// reason to leave it alone gives row -1.
__device__ __forceinline__ TokenAt place_token(const AppendPacked& p, int i) {
  const int lane = threadIdx.x & 31;
  // the last sequence that starts at or before i: 32 probes at a time
  int lo = 0, hi = p.at.batch;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const bool below = at < hi && __ldg(p.q_start + at) <= i;
    const unsigned set = __ballot_sync(0xffffffffu, below);
    // (starts ascend; where they do not, any answer in range will do)
    const int n = set ? 31 - __clz(set) : 0;
    lo += n * step;
    hi = min(hi, lo + step);
  }
  TokenAt t;
  t.row = -1;
  if (lane != 0) return t;
  const int b = lo, first_token = __ldg(p.q_start + b), end = __ldg(p.q_start + b + 1);
  const int first = __ldg(p.positions + b);
  for (int a = 0; a < kMaxAxes; ++a)
    t.pos[a] = a < p.num_axes ? __ldg(p.axis_positions + a * p.axis_stride + i) : 0;
  if (i < first_token || i >= end) return t;                      // nobody's
  if (first_token < 0 || end > p.tokens) return t;                // (recorded by check_starts)
  if (first < 0) return t;
  const long long pos = (long long)first + (i - first_token);
  if (pos > 0x7fffffffll || (p.rotary && p.num_axes == 0 && pos >= p.rotary_positions)) {
    raise_error(p.at.ws, kErrBounds, pos);
    return t;
  }
  if (p.num_axes == 0) t.pos[0] = (int)pos;
  for (int a = 0; a < p.num_axes; ++a)
    if (t.pos[a] < 0 || t.pos[a] >= p.rotary_positions) {
      raise_error(p.at.ws, kErrBounds, t.pos[a]);
      return t;
    }
  t.row = placed_row(p.at, b, (int)pos);
  return t;
}

// gridDim.x blocks of `per_block` tokens; gridDim.y parts of a token's heads.  A
// thread takes its place in a head and passes the block's tokens there, then
// goes to its next head: the head's addresses and weights serve all tokens.
template <typename XT, int KVT, int D, bool INTERLEAVED, bool NORM>
__global__ void __launch_bounds__(kThreads, kBlocks<NORM>)
    append_normed_kernel(const __grid_constant__ AppendPacked p, int per_block) {
  constexpr int TPH = D / 16;                        // threads per head
  __shared__ TokenAt at[kMaxTokens];
  __shared__ __align__(16) float turns_of[kMaxTokens][D];   // cosines, then sines
  const int hpp = blockDim.x / TPH;                  // heads per pass
  const int warp = threadIdx.x >> 5;
  const int t0 = blockIdx.x * per_block;
  const int n = min(per_block, p.tokens - t0);
  const int half = p.rot_dim / 2;
  for (int i = warp; i < n; i += blockDim.x >> 5) {
    const TokenAt t = place_token(p, t0 + i);
    if ((threadIdx.x & 31) == 0) at[i] = t;
  }
  if (blockIdx.x == 0 && blockIdx.y == 0) check_starts(p.at, p.q_start, p.tokens);
  __syncthreads();
  const int u = threadIdx.x % TPH, h0 = threadIdx.x / TPH;
  const int turned = p.rot_dim / 16;                 // threads of a head that rotate
  // this thread's chunks (8 elements each): one of each half of the rotated
  // part, or of the rest
  const bool turns = u < turned;
  const int ea = turns ? 8 * u : p.rot_dim + 8 * (u - turned);
  const int eb = ea + (turns ? half : (D - p.rot_dim) / 2);
  const int heads = p.num_q_heads + 2 * p.num_kv_heads;
  const int per_part = (heads + gridDim.y - 1) / gridDim.y;
  const int h_begin = blockIdx.y * per_part, h_end = min(heads, h_begin + per_part);

  // a head's elements in the packed arrays: of token t0, and from token to token
  struct Source {
    const XT* at;
    long long step;
  };
  auto source = [&](int h) {
    const int kv = h - p.num_q_heads;
    Source s{static_cast<const XT*>(p.q) + (long long)h * D, p.q_stride};
    if (kv >= 0) {
      const bool is_k = kv < p.num_kv_heads;
      s.at = static_cast<const XT*>(is_k ? p.k_new : p.v_new) +
             (long long)(is_k ? kv : kv - p.num_kv_heads) * D;
      s.step = p.kv_stride;
    }
    s.at += t0 * s.step + ea;
    return s;
  };
  const int apart = eb - ea;
  struct Elements {
    uint4 a, b;
  };
  auto load = [&](const Source& s, int h, int i) {
    Elements w{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (i < n && h < h_end && at[i].row >= 0) {
      const XT* src = s.at + i * s.step;
      w.a = *reinterpret_cast<const uint4*>(src);
      w.b = *reinterpret_cast<const uint4*>(src + apart);
    }
    return w;
  };
  // two tokens ahead, over the end of a head into the next one
  int h = h_begin + h0;
  Source src = source(h);
  Elements w0 = load(src, h, 0), w1 = n > 1 ? load(src, h, 1) : load(source(h + hpp), h + hpp, 0);

  // the tokens' cosines and sines, while the first heads are on their way
  for (int x = threadIdx.x; x < n * half; x += blockDim.x) {
    const int k = x / half, pair = x - k * half;
    if (at[k].row < 0) continue;
    const int axis = p.num_axes > 0 ? p.pair_axis[pair] : 0;
    const float* row = p.rotary + (long long)at[k].pos[axis] * p.rot_dim + pair;
    const int to = turn_at<INTERLEAVED>(pair, half);
    turns_of[k][to] = __ldg(row);
    turns_of[k][half + to] = __ldg(row + half);
  }
  __syncthreads();

  for (; h - h0 < h_end; h += hpp) {
    const bool live = h < h_end, is_q = h < p.num_q_heads;
    const bool is_k = !is_q && h < p.num_q_heads + p.num_kv_heads;
    const bool rot = turns && (is_q || is_k);
    const void* norm = !NORM ? nullptr : is_q ? p.q_norm : is_k ? p.k_norm : nullptr;
    const bool any_normed = NORM && __any_sync(0xffffffffu, live && norm);
    const int kvh = h - p.num_q_heads - (is_k ? 0 : p.num_kv_heads);
    uint64_t wt[8];
    if (NORM && norm && live) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int e = k < 4 ? ea + 2 * k : eb + 2 * (k - 4);
        float2 v;
        if (p.norm_f32) {
          // (one by one: weights may start at any element of a larger array)
          const float* x = static_cast<const float*>(norm) + e;
          v = make_float2(__ldg(x), __ldg(x + 1));
        } else {
          const XT* x = static_cast<const XT*>(norm) + e;
          v = make_float2(QType<XT>::to_f32(x[0]), QType<XT>::to_f32(x[1]));
        }
        wt[k] = pack2(v.x, v.y);
      }
    }
    // 8-bit caches: the scale, but for the token's part of it
    float head_scale = is_k ? p.k_scale : p.v_scale;
    if constexpr (KVT == FD_E4M3 || KVT == FD_I8)
      if (p.scale_kind == FD_SCALE_HEAD && live && !is_q)
        head_scale = __fmul_rn(head_scale, __ldg((is_k ? p.k_scales : p.v_scales) + kvh));
    const Source next = source(h + hpp);
    for (int i = 0; i < n; ++i) {
      const Elements w = w0;
      w0 = w1;
      w1 = i + 2 < n ? load(src, h, i + 2)
           : n > 1   ? load(next, h + hpp, i + 2 - n)
                     : load(source(h + 2 * hpp), h + 2 * hpp, 0);
      const long long row = at[i].row;
      if (row < 0) continue;
      // one head, loaded: normed, turned, rounded or quantised, stored.  Every
      // lane of the warp comes here (the reductions).
      uint64_t a[4], b[4];
      unpack_pairs<XT>(w.a, a);
      unpack_pairs<XT>(w.b, b);
      if (any_normed) {
        const float f = norm_factor<D, TPH>(a, b, p.norm_eps);
        if (norm) {
          const uint64_t f2 = pack2(f, f);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            a[k] = mul2(mul2(a[k], f2), wt[k]);
            b[k] = mul2(mul2(b[k], f2), wt[k + 4]);
          }
        }
      }
      if (rot) rotate<INTERLEAVED>(a, b, turns_of[i], u, half);
      const long long srow = row * p.num_kv_heads + kvh;
      float x[8], y[8];
      to_floats(a, x);
      to_floats(b, y);
      if (live && (is_q || KVT == FD_F16 || KVT == FD_BF16)) {
        XT* dst = is_q ? static_cast<XT*>(p.q_out) + ((long long)(t0 + i) * p.num_q_heads + h) * D
                       : static_cast<XT*>(is_k ? p.k_cache : p.v_cache) + srow * D;
        const bool same = !rot && !norm;
        *reinterpret_cast<uint4*>(dst + ea) = same ? w.a : pack8<XT>(x);
        *reinterpret_cast<uint4*>(dst + eb) = same ? w.b : pack8<XT>(y);
      }
      if constexpr (KVT == FD_E4M3 || KVT == FD_I8) {
        float scale = head_scale;
        if (p.scale_kind == FD_SCALE_TOKEN) {
          float amax = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fmaxf(fabsf(x[k]), fabsf(y[k])));
#pragma unroll
          for (int o = TPH / 2; o; o >>= 1)
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          const float qmax = KVT == FD_I8 ? 127.f : 448.f;
          const float ks = amax > 0.f ? __fdiv_rn(amax, __fmul_rn(qmax, scale)) : 1.f;
          if (live && !is_q && u == 0) (is_k ? p.k_scales : p.v_scales)[srow] = ks;
          scale = __fmul_rn(scale, ks);
        }
        if (live && !is_q) {
          uint8_t* dst = static_cast<uint8_t*>(is_k ? p.k_cache : p.v_cache) + srow * D;
          *reinterpret_cast<uint2*>(dst + ea) = encode8<KVT>(x, scale);
          *reinterpret_cast<uint2*>(dst + eb) = encode8<KVT>(y, scale);
        }
      }
    }
    src = next;
  }
}

template <typename XT, int KVT, int D>
cudaError_t launch_d(const AppendPacked& p, int sms, cudaStream_t stream) {
  // Blocks enough to fill the SMs: several tokens a block when there are many,
  // several blocks a token when there are few.
  const int heads = p.num_q_heads + 2 * p.num_kv_heads;
  // (as many tokens a block as make a whole number of rounds of the GPU)
  const bool norm = p.q_norm || p.k_norm;
  const long long room = (norm ? kBlocks<true> : kBlocks<false>) * sms;
  const long long rounds = (p.tokens + room * kMaxTokens - 1) / (room * kMaxTokens);
  const int per_block = (int)((p.tokens + rounds * room - 1) / (rounds * room));
  const int blocks = (int)(((long long)p.tokens + per_block - 1) / per_block);
  const int warps_token = (heads * (D / 16) + 31) / 32;   // warps of one token
  int parts = blocks >= 4 * sms ? 1 : (4 * sms + blocks - 1) / blocks;
  const int most = (warps_token + 3) / 4;                 // parts of four warps at least
  if (parts > most) parts = most;
  // threads that pass a part's heads in equal, full passes
  const int warps_part = ((heads + parts - 1) / parts * (D / 16) + 31) / 32;
  const int passes = (warps_part + kThreads / 32 - 1) / (kThreads / 32);
  const int warps = (warps_part + passes - 1) / passes;
  const dim3 grid((unsigned)blocks, (unsigned)parts);
  const auto kern = p.interleaved ? (norm ? append_normed_kernel<XT, KVT, D, true, true>
                                          : append_normed_kernel<XT, KVT, D, true, false>)
                                  : (norm ? append_normed_kernel<XT, KVT, D, false, true>
                                          : append_normed_kernel<XT, KVT, D, false, false>);
  kern<<<grid, warps * 32, 0, stream>>>(p, per_block);
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

cudaError_t launch_append_normed(const AppendPacked& p, int sms, cudaStream_t stream) {
  return p.new_dtype == FD_F16 ? launch_x<__half>(p, sms, stream)
                               : launch_x<__nv_bfloat16>(p, sms, stream);
}

}  // namespace fd
