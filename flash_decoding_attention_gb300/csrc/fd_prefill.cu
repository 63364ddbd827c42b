// fd_prefill.cu -- host side of the attention of packed new tokens: tensor
// maps, workspace, dispatch; and the merge of streams cut between CTAs.
#include <cstring>
#include <mutex>

#include "fd_prefill.cuh"

namespace fd {
namespace pf {
namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &qr) == cudaSuccess &&
        qr == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// {dims, heads, tokens or rows} with boxes of `elems` dims, `heads_box` heads
// and `rows_box` rows.
bool make_map(CUtensorMap* m, const void* base, int elem, int head_dim, int heads, long long rows,
              long long row_stride, int elems, int heads_box, int rows_box) {
  const auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)head_dim * elem, (cuuint64_t)row_stride * elem};
  const cuuint32_t box[3] = {(cuuint32_t)elems, (cuuint32_t)heads_box, (cuuint32_t)rows_box};
  const cuuint32_t step[3] = {1u, 1u, 1u};
  return fn(m, elem == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 3,
            const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            elems * elem == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ---------------------------------------------------------------------------
// Merge
// ---------------------------------------------------------------------------
// A stream cut between CTAs c - 1, c, ... left its beginning in slot
// 2 (c - 1) + 1 and its continuations in slots 2 c, 2 (c + 1), ...:
//   M = max_k m_k, L = sum_k l_k 2^(m_k - M), A = sum_k acc_k 2^(m_k - M),
//   out = v_scale A / L, lse = (M + log2 L) ln 2,
// in a fixed order.  Every CTA finds all cut streams from the slots' notes (one
// per boundary between CTAs at most) and lays their work end to end: items of
// 32 rows (a row per lane, as the states are laid out) times 16 dims.  A warp
// takes an item of a stream cut into few parts; the warps of a CTA share the
// states of an item of a stream cut into many.
constexpr int kMergeThreads = 256;
constexpr int kMergeWarps = kMergeThreads / 32;
constexpr int kMaxGrid = 512;   // boundaries (SMs)
constexpr int kFew = 6;         // parts one warp passes alone

struct Part {
  int c, X, row0, dim0, parts;   // boundary, query tile, first row, first dim, parts
  int4 id;
};

// Running state of one row and 16 dims.
struct State {
  float m, l, a[16];
  __device__ __forceinline__ void clear() {
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) a[i] = 0.f;
  }
  __device__ __forceinline__ void add(float mk, float lk, const float (&x)[16]) {
    const float M = fmaxf(m, mk);
    const float f = m == -INFINITY ? 0.f : fast_exp2(m - M);
    const float g = mk == -INFINITY ? 0.f : fast_exp2(mk - M);
    m = M;
    l = l * f + lk * g;
#pragma unroll
    for (int i = 0; i < 16; ++i) a[i] = fmaf(x[i], g, a[i] * f);
  }
};

template <int D, bool BF16>
struct Merge {
  const Prefill& p;
  int lane;

  __device__ __forceinline__ int live_rows(const Seq& s, int m, int X) const {
    const long long left = (long long)s.n - (long long)m * s.span - (long long)X * p.tile_tokens;
    return (int)(left < p.tile_tokens ? (left > 0 ? left : 0) : p.tile_tokens) * p.group;
  }

  // Adds parts first, first + step, ... of `it` to `st`.
  __device__ __forceinline__ void gather(const Part& it, int first, int step, bool live,
                                         State& st) const {
    constexpr int kAhead = 2;
    for (int k0 = first; k0 < it.parts; k0 += kAhead * step) {
      float2 ml[kAhead];
      float4 x[kAhead][4];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int k = k0 + u * step;
        ml[u] = make_float2(-INFINITY, 0.f);
        if (live && k < it.parts) {
          // (a sum, not a choice by k: nvcc 13.0 translates
          // k == 0 ? 2 * (c - 1) + 1 : 2 * (c + k - 1) wrongly where such a loop
          // is unrolled by four; a kernel of nothing else shows it)
          const int slot = 2 * (it.c - 1 + k) + (k == 0 ? 1 : 0);
          const long long tile = 2ll * slot + it.X;
          ml[u] = p.part_ml[tile * kRowsTile + it.row0 + lane];
          const float4* src = reinterpret_cast<const float4*>(p.part_acc) +
                              (tile * (D / 4) + it.dim0 / 4) * kRowsTile + it.row0 + lane;
#pragma unroll
          for (int i = 0; i < 4; ++i) x[u][i] = src[i * kRowsTile];
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (!live || k0 + u * step >= it.parts) continue;
        float y[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[4 * i] = x[u][i].x;
          y[4 * i + 1] = x[u][i].y;
          y[4 * i + 2] = x[u][i].z;
          y[4 * i + 3] = x[u][i].w;
        }
        st.add(ml[u].x, ml[u].y, y);
      }
    }
  }

  __device__ __forceinline__ void write(const Part& it, const Seq& s, const State& st) const {
    const int r = it.row0 + lane;
    const long long tok = (long long)s.q0 + (long long)(2 * it.id.z + it.X) * p.tile_tokens +
                          r / p.group;
    const long long orow = tok * p.num_q_heads + (long long)it.id.y * p.group + r % p.group;
    float vsc = p.v_scale;
    if (p.scale_kind == FD_SCALE_HEAD) vsc *= __ldg(p.v_scales + it.id.y);
    const float q = st.l == 0.f ? 0.f : vsc / st.l;
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack16<BF16>(st.a[2 * i] * q, st.a[2 * i + 1] * q);
    uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + orow * D + it.dim0);
    o[0] = make_uint4(w[0], w[1], w[2], w[3]);
    o[1] = make_uint4(w[4], w[5], w[6], w[7]);
    if (p.lse && it.dim0 == 0)
      p.lse[orow] = st.l == 0.f ? -INFINITY : (st.m + log2f(st.l)) * kLn2;
  }
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const __grid_constant__ Prefill p) {
  __shared__ int4 first[kMaxGrid];                  // stream of slot 2 c
  __shared__ short parts_of[kMaxGrid];
  __shared__ int before[2][kMaxGrid + 1];           // items before c: few parts, many parts
  __shared__ int wsum[2][kMergeWarps];
  __shared__ float red[kMergeWarps][18][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Merge<D, BF16> mg{p, lane};
  for (int c = tid; c < p.grid; c += kMergeThreads) first[c] = p.meta[2 * c];
  __syncthreads();
  auto same = [](const int4& a, const int4& b) { return a.x == b.x && a.y == b.y && a.z == b.z; };
  int carry[2] = {0, 0};
  for (int base = 0; base < p.grid; base += kMergeThreads) {
    const int c = base + tid;
    int items[2] = {0, 0};
    if (c > 0 && c < p.grid) {
      const int4 id = first[c], begun = p.meta[2 * c - 1];
      if (id.x >= 0 && id.x < p.at.batch && same(id, begun)) {
        int parts = 2;   // the beginning and this continuation
        while (c + parts - 1 < p.grid && same(first[c + parts - 1], id)) ++parts;
        parts_of[c] = (short)parts;
        const Seq s = load_seq<false>(p, id.x, false);
        const int blocks = (mg.live_rows(s, id.z, 0) + 31) / 32 + (mg.live_rows(s, id.z, 1) + 31) / 32;
        items[parts <= kFew ? 0 : 1] = blocks * (D / 16);
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      int x = items[k];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) wsum[k][warp] = x;
      __syncthreads();
      int b = carry[k];
      for (int w = 0; w < kMergeWarps; ++w) {
        if (w < warp) b += wsum[k][w];
        carry[k] += wsum[k][w];
      }
      if (c < p.grid) before[k][c] = b + x - items[k];
    }
    __syncthreads();
  }
  auto part_at = [&](int k, int item) {
    int lo = 0, hi = p.grid;   // the last boundary with before <= item
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (before[k][mid] <= item) lo = mid;
      else hi = mid;
    }
    Part it;
    it.c = lo;
    it.id = first[lo];
    it.parts = parts_of[lo];
    const int w = item - before[k][lo];
    it.dim0 = (w % (D / 16)) * 16;
    it.row0 = w / (D / 16) * 32;   // over both query tiles for now
    return it;
  };
  for (int item = blockIdx.x * kMergeWarps + warp; item < carry[0];
       item += gridDim.x * kMergeWarps) {
    Part it = part_at(0, item);
    const Seq s = load_seq<false>(p, it.id.x, false);
    const int rows_a = (mg.live_rows(s, it.id.z, 0) + 31) / 32 * 32;
    it.X = it.row0 >= rows_a ? 1 : 0;
    if (it.X) it.row0 -= rows_a;
    const bool live = it.row0 + lane < mg.live_rows(s, it.id.z, it.X);
    State st;
    st.clear();
    mg.gather(it, 0, 1, live, st);
    if (live) mg.write(it, s, st);
  }
  for (int item = blockIdx.x; item < carry[1]; item += gridDim.x) {
    Part it = part_at(1, item);
    const Seq s = load_seq<false>(p, it.id.x, false);
    const int rows_a = (mg.live_rows(s, it.id.z, 0) + 31) / 32 * 32;
    it.X = it.row0 >= rows_a ? 1 : 0;
    if (it.X) it.row0 -= rows_a;
    const bool live = it.row0 + lane < mg.live_rows(s, it.id.z, it.X);
    State st;
    st.clear();
    mg.gather(it, warp, kMergeWarps, live, st);
    red[warp][16][lane] = st.m;
    red[warp][17][lane] = st.l;
#pragma unroll
    for (int i = 0; i < 16; ++i) red[warp][i][lane] = st.a[i];
    __syncthreads();
    if (warp == 0 && live) {
      for (int w = 1; w < kMergeWarps; ++w) {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = red[w][i][lane];
        st.add(red[w][16][lane], red[w][17][lane], x);
      }
      mg.write(it, s, st);
    }
    __syncthreads();
  }
}

// Launched as a programmatic dependent of the attention kernel.
template <int D, bool BF16>
cudaError_t launch_merge(const Prefill& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(4 * p.grid));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, merge_kernel<D, BF16>, p);
}

}  // namespace
}  // namespace pf

PrefillLayout prefill_layout(int head_dim, int sms) {
  PrefillLayout l;
  const size_t slots = 2 * (size_t)sms;
  l.meta_off = sizeof(WsHeader);
  l.ml_off = align_up(l.meta_off + slots * sizeof(int4), 256);
  l.acc_off = align_up(l.ml_off + slots * pf::kRowsPair * sizeof(float2), 256);
  l.total = align_up(l.acc_off + slots * pf::kRowsPair * head_dim * sizeof(float), 256);
  return l;
}

cudaError_t launch_prefill(Prefill p, void* workspace, cudaStream_t stream) {
  if (p.grid > pf::kMaxGrid) p.grid = pf::kMaxGrid;
  const PrefillLayout l = prefill_layout(p.head_dim, p.grid);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.meta = reinterpret_cast<int4*>(ws + l.meta_off);
  p.part_ml = reinterpret_cast<float2*>(ws + l.ml_off);
  p.part_acc = reinterpret_cast<float*>(ws + l.acc_off);
  p.tile_tokens = pf::kRowsTile / p.group;
  const bool wide = kv_elem_bytes(p.kv_dtype) == 2;
  // a box of page rows must fill whole swizzle atoms of 8 rows
  p.gather = p.at.block_table && p.at.page_size < 8 ? 1 : 0;
  CUtensorMap maps[3];
  std::memset(maps, 0, sizeof(maps));
  if (!pf::make_map(&maps[0], p.q, 2, p.head_dim, p.num_q_heads, p.tokens, p.q_stride, 64, p.group,
                    p.tile_tokens))
    return cudaErrorInvalidValue;
  if (!p.gather) {
    const int box = p.at.block_table && p.at.page_size < pf::kTile ? p.at.page_size : pf::kTile;
    const int elem = wide ? 2 : 1, elems = wide ? 64 : p.head_dim;
    const long long stride = (long long)p.num_kv_heads * p.head_dim;
    if (!pf::make_map(&maps[1], p.k, elem, p.head_dim, p.num_kv_heads, p.at.kv_rows, stride, elems,
                      1, box) ||
        !pf::make_map(&maps[2], p.v, elem, p.head_dim, p.num_kv_heads, p.at.kv_rows, stride, elems,
                      1, box))
      return cudaErrorInvalidValue;
  }
  const bool bf16 = p.q_dtype == FD_BF16;
  cudaError_t e;
  if (wide) e = pf::launch_16bit(p, maps, stream);
  else if (p.kv_dtype == FD_E4M3)
    e = bf16 ? pf::launch_e4m3_bf16(p, maps, stream) : pf::launch_e4m3_f16(p, maps, stream);
  else e = bf16 ? pf::launch_i8_bf16(p, maps, stream) : pf::launch_i8_f16(p, maps, stream);
  if (e != cudaSuccess) return e;
  if (p.head_dim == 128)
    return bf16 ? pf::launch_merge<128, true>(p, stream) : pf::launch_merge<128, false>(p, stream);
  return bf16 ? pf::launch_merge<64, true>(p, stream) : pf::launch_merge<64, false>(p, stream);
}

}  // namespace fd
