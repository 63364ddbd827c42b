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
// in the order of k.  Every CTA finds all cut streams from the slots' notes
// (one per boundary between CTAs at most), lays their rows end to end and
// takes its share.
constexpr int kMergeThreads = 256;
constexpr int kMaxGrid = 512;   // boundaries (SMs)

template <int D, bool BF16, int WPI>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const __grid_constant__ Prefill p) {
  constexpr int DPL = D / 32, kWarps = kMergeThreads / 32;
  __shared__ int4 first[kMaxGrid];     // slot 2 c
  __shared__ int rows_before[kMaxGrid + 1];
  __shared__ int wsum[kWarps];
  __shared__ float red_m[kWarps], red_l[kWarps], red_a[kWarps][D];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int c = tid; c < p.grid; c += kMergeThreads) first[c] = p.meta[2 * c];
  int carry = 0;
  for (int base = 0; base < p.grid; base += kMergeThreads) {
    const int c = base + tid;
    int rows = 0;
    if (c > 0 && c < p.grid) {
      const int4 a = p.meta[2 * c - 1], b = p.meta[2 * c];
      if (b.x >= 0 && b.x < p.at.batch && a.x == b.x && a.y == b.y && a.z == b.z) {
        // whole tokens of both query tiles, as the attention kernel lays them
        const Seq s = load_seq(p, b.x, false);
        const long long left = (long long)s.n - (long long)b.z * s.span;
        rows = (int)(left < s.span ? (left > 0 ? left : 0) : s.span) * p.group;
      }
    }
    int x = rows;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    int before = carry, all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += wsum[w];
      all += wsum[w];
    }
    if (c < p.grid) rows_before[c] = before + x - rows;
    carry += all;
    __syncthreads();
  }
  if (tid == 0) rows_before[p.grid] = carry;
  __syncthreads();
  const int total = carry;
  constexpr int kItems = kWarps / WPI;   // rows a CTA merges at a time
  const int part = warp % WPI, slot_in_cta = warp / WPI;
  for (int it0 = blockIdx.x * kItems; it0 < total; it0 += gridDim.x * kItems) {
    const int item = it0 + slot_in_cta;
    const bool live = item < total;
    int c = 0, nseg = 0, row = 0;
    int4 id = make_int4(0, 0, 0, 0);
    if (live) {
      int lo = 0, hi = p.grid;   // the last boundary with rows_before <= item
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (rows_before[mid] <= item) lo = mid;
        else hi = mid;
      }
      c = lo;
      id = first[c];
      nseg = 2;   // the beginning and this continuation
      while (c + nseg - 1 < p.grid && first[c + nseg - 1].x == id.x &&
             first[c + nseg - 1].y == id.y && first[c + nseg - 1].z == id.z)
        ++nseg;
      row = item - rows_before[c];
    }
    // row of the pair: query tile, token of the tile, head of the group
    const int per_tile = p.tile_tokens * p.group;
    const int X = row >= per_tile ? 1 : 0;
    const int r = row - X * per_tile;
    auto at = [&](int k) -> long long {
      // (written as a sum: with a choice between two addresses the compiled
      // loop read the wrong slot from its second state on)
      const int slot = 2 * (c - 1 + k) + (k == 0 ? 1 : 0);
      return (long long)slot * kRowsPair + X * kRowsTile + r;
    };
    // this warp's states: part, part + WPI, ...; the lanes share a state's dims
    const int nu = nseg > part ? (nseg - part + WPI - 1) / WPI : 0;
    float M = -INFINITY;
    for (int u = lane; u < nu; u += 32) M = fmaxf(M, p.part_ml[at(part + WPI * u)].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if constexpr (WPI > 1) {
      if (lane == 0) red_m[warp] = M;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < WPI; ++w) M = fmaxf(M, red_m[slot_in_cta * WPI + w]);
    }
    float L = 0.f, a[DPL];
#pragma unroll
    for (int k = 0; k < DPL; ++k) a[k] = 0.f;
#pragma unroll 4
    for (int u = 0; u < nu; ++u) {
      const long long i = at(part + WPI * u);
      const float2 ml = p.part_ml[i];
      const float* src = p.part_acc + i * D + lane * DPL;
      float x[DPL];
      if constexpr (DPL == 4) {
        const float4 y = *reinterpret_cast<const float4*>(src);
        x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w;
      } else {
        const float2 y = *reinterpret_cast<const float2*>(src);
        x[0] = y.x; x[1] = y.y;
      }
      const float w = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - M);
      L = fmaf(ml.y, w, L);
#pragma unroll
      for (int k = 0; k < DPL; ++k) a[k] = fmaf(x[k], w, a[k]);
    }
    if constexpr (WPI > 1) {
      if (lane == 0) red_l[warp] = L;
#pragma unroll
      for (int k = 0; k < DPL; ++k) red_a[warp][lane * DPL + k] = a[k];
      __syncthreads();
      L = 0.f;
#pragma unroll
      for (int k = 0; k < DPL; ++k) a[k] = 0.f;
#pragma unroll
      for (int w = 0; w < WPI; ++w) {
        L += red_l[slot_in_cta * WPI + w];
#pragma unroll
        for (int k = 0; k < DPL; ++k) a[k] += red_a[slot_in_cta * WPI + w][lane * DPL + k];
      }
      __syncthreads();
    }
    if (!live || part != 0) continue;
    const Seq s = load_seq(p, id.x, false);
    const long long tok = (long long)s.q0 + (long long)(2 * id.z + X) * p.tile_tokens + r / p.group;
    const long long orow = tok * p.num_q_heads + (long long)id.y * p.group + r % p.group;
    float vsc = p.v_scale;
    if (p.scale_kind == FD_SCALE_HEAD) vsc *= __ldg(p.v_scales + id.y);
    const float q = L > 0.f ? vsc / L : 0.f;
    uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + orow * D + lane * DPL);
    if constexpr (DPL == 4)
      *reinterpret_cast<uint2*>(o) =
          make_uint2(pack16<BF16>(a[0] * q, a[1] * q), pack16<BF16>(a[2] * q, a[3] * q));
    else
      *o = pack16<BF16>(a[0] * q, a[1] * q);
    if (p.lse && lane == 0) p.lse[orow] = L > 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
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
  return cudaLaunchKernelEx(&cfg, merge_kernel<D, BF16, 2>, p);
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
