// fd_prompt_api.cu -- the prompt path's entry points: argument checks and
// launches of fd_rotary_table, fd_append_kv_packed, fd_append_kv_normed,
// fd_read_kv, fd_assign_pages, fd_prefill_attention and their variants.
#include <cmath>
#include <cstring>

#include "fd_prompt.cuh"

namespace fd {
namespace {

constexpr int64_t kMaxPacked = int64_t(1) << 31;
constexpr double kTwoPi = 6.283185307179586476925;

// Layout, sizes and dtypes that every packed entry point takes.
fd_status check_placement(const void* k_cache, const void* v_cache, const int32_t* kv_start_idx,
                          const int32_t* block_table, int block_table_stride,
                          const int32_t* starts, int64_t num_tokens, int64_t kv_rows, int batch,
                          int num_kv_heads, int head_dim, int page_size, fd_scale_kind scale_kind,
                          const float* k_scales, const float* v_scales, fd_dtype dtype16,
                          fd_dtype kv_dtype, const void* workspace) {
  if (scale_kind != FD_SCALE_TENSOR && scale_kind != FD_SCALE_HEAD &&
      scale_kind != FD_SCALE_TOKEN)
    return FD_ERR_INVALID_ARG;
  if (dtype16 != FD_F16 && dtype16 != FD_BF16) return FD_ERR_INVALID_ARG;
  if (kv_dtype != FD_F16 && kv_dtype != FD_BF16 && kv_dtype != FD_E4M3 && kv_dtype != FD_I8)
    return FD_ERR_INVALID_ARG;
  if (scale_kind != FD_SCALE_TENSOR) {
    if (!k_scales || !v_scales || !aligned(k_scales, 4) || !aligned(v_scales, 4))
      return FD_ERR_INVALID_ARG;
    if (kv_elem_bytes(kv_dtype) != 1) return FD_ERR_UNSUPPORTED;
  }
  if (!k_cache || !v_cache || !starts || !workspace) return FD_ERR_INVALID_ARG;
  if ((kv_start_idx == nullptr) == (block_table == nullptr)) return FD_ERR_INVALID_ARG;
  if (batch <= 0 || batch > (1 << 24)) return FD_ERR_INVALID_ARG;
  if (num_tokens < 0 || num_tokens >= kMaxPacked) return FD_ERR_INVALID_ARG;
  if (num_kv_heads <= 0 || num_kv_heads > 4096) return FD_ERR_INVALID_ARG;
  if (kv_rows <= 0 || kv_rows > (int64_t(1) << 40)) return FD_ERR_INVALID_ARG;
  if (block_table) {
    if (!is_pow2(page_size) || page_size > 256) return FD_ERR_UNSUPPORTED;
    if (block_table_stride <= 0 || kv_rows % page_size != 0) return FD_ERR_INVALID_ARG;
  }
  if (!dtypes_ok(dtype16, kv_dtype)) return FD_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return FD_ERR_UNSUPPORTED;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(workspace, 256) ||
      !aligned(starts, 4) || (kv_start_idx && !aligned(kv_start_idx, 4)) ||
      (block_table && !aligned(block_table, 4)))
    return FD_ERR_INVALID_ARG;
  return FD_OK;
}

Placement placement(const int32_t* kv_start_idx, const int32_t* block_table,
                    int block_table_stride, int64_t kv_rows, int batch, int page_size,
                    void* workspace) {
  Placement at;
  std::memset(&at, 0, sizeof(at));
  at.kv_start = kv_start_idx;
  at.block_table = block_table;
  at.kv_rows = kv_rows;
  at.bt_stride = block_table ? block_table_stride : 0;
  at.page_size = block_table ? page_size : 1;
  at.page_shift = block_table ? log2i(page_size) : 0;
  at.batch = batch;
  at.ws = static_cast<WsHeader*>(workspace);
  return at;
}

// Tokens `stride` elements apart, `heads` heads each: 16-byte vectors and TMA
// rows need a multiple of 8 elements.
bool stride_ok(int64_t stride, int heads, int head_dim) {
  return stride >= (int64_t)heads * head_dim && stride % 8 == 0 && stride < (int64_t(1) << 32);
}

// Do `tokens` dense rows of `width` bytes at `a` and rows of `b_width` bytes,
// `b_stride` apart, at `b` share an address range?
bool overlap(const void* a, int64_t width, const void* b, int64_t b_width, int64_t b_stride,
             int64_t tokens) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return tokens > 0 && a0 < b0 + (uintptr_t)((tokens - 1) * b_stride + b_width) &&
         b0 < a0 + (uintptr_t)(tokens * width);
}

}  // namespace
}  // namespace fd

using namespace fd;

extern "C" {

fd_status fd_rotary_table(float* table, int64_t positions, int rot_dim, double theta,
                          fd_rotary_scaling scaling, double factor, double original_positions,
                          double low_turns, double high_turns, float amplitude,
                          fd_stream_t stream) {
  if (!table || !aligned(table, 16)) return FD_ERR_INVALID_ARG;
  if (positions <= 0 || positions >= kMaxPacked) return FD_ERR_INVALID_ARG;
  if (rot_dim < 16 || rot_dim > kMaxRotDim || rot_dim % 16 != 0) return FD_ERR_UNSUPPORTED;
  if (!std::isfinite(theta) || !(theta > 1.0) || !std::isfinite(amplitude))
    return FD_ERR_INVALID_ARG;
  if (scaling != FD_ROTARY_PLAIN && scaling != FD_ROTARY_LINEAR && scaling != FD_ROTARY_BY_PARTS)
    return FD_ERR_INVALID_ARG;
  if (scaling != FD_ROTARY_PLAIN && !(std::isfinite(factor) && factor >= 1.0))
    return FD_ERR_INVALID_ARG;
  if (scaling == FD_ROTARY_BY_PARTS &&
      !(std::isfinite(original_positions) && original_positions > 0.0 && low_turns >= 0.0 &&
        std::isfinite(high_turns) && high_turns > low_turns))
    return FD_ERR_INVALID_ARG;
  const int sms = current_sms();
  if (sms <= 0) return FD_ERR_CUDA;
  RotaryTable p;
  std::memset(&p, 0, sizeof(p));
  p.table = table;
  p.positions = positions;
  p.rot_dim = rot_dim;
  p.amplitude = amplitude;
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / rot_dim);
    if (scaling == FD_ROTARY_LINEAR) {
      f /= factor;
    } else if (scaling == FD_ROTARY_BY_PARTS) {
      const double r = original_positions * f / kTwoPi;
      const double g = std::fmin(std::fmax((r - low_turns) / (high_turns - low_turns), 0.0), 1.0);
      f = g * f + (1.0 - g) * f / factor;
    }
    // f <= 1, so at most 2^64 / (2 pi): scaling by 2^64 is exact in a double
    p.turns[i] = (unsigned long long)std::ldexp(f / kTwoPi, 64);
  }
  return launch_rotary_table(p, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FD_OK
             : FD_ERR_CUDA;
}

// What fd_append_kv_normed has beside the packed append's arguments.
struct AppendExtra {
  const void *q_norm, *k_norm;
  int norm_f32;
  float norm_eps;
  const int32_t* axis_positions;
  int num_axes;
  int64_t axis_stride;
  const uint8_t* pair_axis;
};

static fd_status append_impl(const void* q, int64_t q_stride, void* q_out, const void* k_new,
                             const void* v_new, int64_t kv_stride, void* k_cache, void* v_cache,
                             const int32_t* kv_start_idx, const int32_t* block_table,
                             int block_table_stride, const int32_t* q_start,
                             const int32_t* positions, int64_t num_tokens, int64_t kv_rows,
                             int batch, int num_q_heads, int num_kv_heads, int head_dim,
                             int page_size, const float* rotary, int64_t rotary_positions,
                             int rot_dim, int interleaved, float k_scale, float v_scale,
                             fd_scale_kind scale_kind, float* k_scales, float* v_scales,
                             fd_dtype new_dtype, fd_dtype kv_dtype, void* workspace,
                             size_t workspace_bytes, fd_stream_t stream, const AppendExtra& x) {
  const fd_status chk = check_placement(
      k_cache, v_cache, kv_start_idx, block_table, block_table_stride, q_start, num_tokens,
      kv_rows, batch, num_kv_heads, head_dim, page_size, scale_kind, k_scales, v_scales, new_dtype,
      kv_dtype, workspace);
  if (chk != FD_OK) return chk;
  if (!positions || !aligned(positions, 4)) return FD_ERR_INVALID_ARG;
  // (packed arrays without rows may have no address)
  if (num_tokens > 0 && (!k_new || !v_new)) return FD_ERR_INVALID_ARG;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !stride_ok(kv_stride, num_kv_heads, head_dim))
    return FD_ERR_INVALID_ARG;
  if (q) {
    if ((!q_out && num_tokens > 0) || num_q_heads <= 0 || num_q_heads > 4096)
      return FD_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(q_out, 16) || !stride_ok(q_stride, num_q_heads, head_dim))
      return FD_ERR_INVALID_ARG;
    // in place only where a token's rows are its own
    if (q == q_out && num_tokens > 0 && q_stride != (int64_t)num_q_heads * head_dim) return FD_ERR_INVALID_ARG;
  }
  if (rotary) {
    if (!aligned(rotary, 16) || rotary_positions <= 0) return FD_ERR_INVALID_ARG;
    if (rot_dim < 16 || rot_dim > head_dim || rot_dim % 16 != 0) return FD_ERR_UNSUPPORTED;
  }
  if (x.q_norm || x.k_norm) {
    if (x.q_norm && !q && num_tokens > 0) return FD_ERR_INVALID_ARG;
    const size_t elem = x.norm_f32 ? 4 : 2;
    if (!aligned(x.q_norm, elem) || !aligned(x.k_norm, elem)) return FD_ERR_INVALID_ARG;
    if (!std::isfinite(x.norm_eps) || !(x.norm_eps > 0.f)) return FD_ERR_INVALID_ARG;
  }
  if (x.num_axes != 0) {
    if (x.num_axes < 0 || x.num_axes > 4) return FD_ERR_UNSUPPORTED;
    if (!rotary || !x.pair_axis) return FD_ERR_INVALID_ARG;
    if ((!x.axis_positions && num_tokens > 0) || !aligned(x.axis_positions, 4) ||
        x.axis_stride < num_tokens || x.axis_stride >= kMaxPacked)
      return FD_ERR_INVALID_ARG;
    for (int i = 0; i < rot_dim / 2; ++i)
      if (x.pair_axis[i] >= x.num_axes) return FD_ERR_INVALID_ARG;
  }
  if (!std::isfinite(k_scale) || !std::isfinite(v_scale)) return FD_ERR_INVALID_ARG;
  if (kv_elem_bytes(kv_dtype) == 1 && !(k_scale > 0.f && v_scale > 0.f)) return FD_ERR_INVALID_ARG;
  if (workspace_bytes < sizeof(WsHeader)) return FD_ERR_WORKSPACE_TOO_SMALL;
  if (num_tokens == 0) return FD_OK;
  if (q) {   // written by blocks while others read (in place: their own rows)
    const int64_t width = (int64_t)num_q_heads * head_dim * 2;
    const int64_t kv_width = (int64_t)num_kv_heads * head_dim * 2;
    if ((q != q_out && overlap(q_out, width, q, width, 2 * q_stride, num_tokens)) ||
        overlap(q_out, width, k_new, kv_width, 2 * kv_stride, num_tokens) ||
        overlap(q_out, width, v_new, kv_width, 2 * kv_stride, num_tokens))
      return FD_ERR_INVALID_ARG;
  }
  const int sms = current_sms();
  if (sms <= 0) return FD_ERR_CUDA;

  AppendPacked p;
  std::memset(&p, 0, sizeof(p));
  p.at = placement(kv_start_idx, block_table, block_table_stride, kv_rows, batch, page_size,
                   workspace);
  p.q = q;
  p.q_out = q_out;
  p.q_stride = q_stride;
  p.k_new = k_new;
  p.v_new = v_new;
  p.kv_stride = kv_stride;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.q_start = q_start;
  p.positions = positions;
  p.tokens = (int)num_tokens;
  p.num_q_heads = q ? num_q_heads : 0;
  p.num_kv_heads = num_kv_heads;
  p.head_dim = head_dim;
  p.rotary = rotary;
  p.rotary_positions = rotary_positions;
  p.rot_dim = rotary ? rot_dim : 0;
  p.interleaved = interleaved ? 1 : 0;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.scale_kind = scale_kind;
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.new_dtype = new_dtype;
  p.kv_dtype = kv_dtype;
  p.q_norm = x.q_norm;
  p.k_norm = x.k_norm;
  p.norm_f32 = x.norm_f32 ? 1 : 0;
  p.norm_eps = x.norm_eps;
  if (x.num_axes > 0) {
    p.num_axes = x.num_axes;
    p.axis_stride = x.axis_stride;
    p.axis_positions = x.axis_positions;
    std::memcpy(p.pair_axis, x.pair_axis, rot_dim / 2);
  }
  return launch_append_packed(p, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FD_OK
             : FD_ERR_CUDA;
}

fd_status fd_append_kv_packed(const void* q, int64_t q_stride, void* q_out, const void* k_new,
                              const void* v_new, int64_t kv_stride, void* k_cache, void* v_cache,
                              const int32_t* kv_start_idx, const int32_t* block_table,
                              int block_table_stride, const int32_t* q_start,
                              const int32_t* positions, int64_t num_tokens, int64_t kv_rows,
                              int batch, int num_q_heads, int num_kv_heads, int head_dim,
                              int page_size, const float* rotary, int64_t rotary_positions,
                              int rot_dim, int interleaved, float k_scale, float v_scale,
                              fd_scale_kind scale_kind, float* k_scales, float* v_scales,
                              fd_dtype new_dtype, fd_dtype kv_dtype, void* workspace,
                              size_t workspace_bytes, fd_stream_t stream) {
  return append_impl(q, q_stride, q_out, k_new, v_new, kv_stride, k_cache, v_cache, kv_start_idx,
                     block_table, block_table_stride, q_start, positions, num_tokens, kv_rows,
                     batch, num_q_heads, num_kv_heads, head_dim, page_size, rotary,
                     rotary_positions, rot_dim, interleaved, k_scale, v_scale, scale_kind,
                     k_scales, v_scales, new_dtype, kv_dtype, workspace, workspace_bytes, stream,
                     AppendExtra{});
}

fd_status fd_append_kv_normed(const void* q, int64_t q_stride, void* q_out, const void* k_new,
                              const void* v_new, int64_t kv_stride, void* k_cache, void* v_cache,
                              const int32_t* kv_start_idx, const int32_t* block_table,
                              int block_table_stride, const int32_t* q_start,
                              const int32_t* positions, int64_t num_tokens, int64_t kv_rows,
                              int batch, int num_q_heads, int num_kv_heads, int head_dim,
                              int page_size, const float* rotary, int64_t rotary_positions,
                              int rot_dim, int interleaved, const void* q_norm, const void* k_norm,
                              int norm_f32, float norm_eps, const int32_t* axis_positions,
                              int num_axes, int64_t axis_stride, const uint8_t* pair_axis,
                              float k_scale, float v_scale, fd_scale_kind scale_kind,
                              float* k_scales, float* v_scales, fd_dtype new_dtype,
                              fd_dtype kv_dtype, void* workspace, size_t workspace_bytes,
                              fd_stream_t stream) {
  const AppendExtra x{q_norm,   k_norm,      norm_f32,  norm_eps, axis_positions,
                      num_axes, axis_stride, pair_axis};
  return append_impl(q, q_stride, q_out, k_new, v_new, kv_stride, k_cache, v_cache, kv_start_idx,
                     block_table, block_table_stride, q_start, positions, num_tokens, kv_rows,
                     batch, num_q_heads, num_kv_heads, head_dim, page_size, rotary,
                     rotary_positions, rot_dim, interleaved, k_scale, v_scale, scale_kind,
                     k_scales, v_scales, new_dtype, kv_dtype, workspace, workspace_bytes, stream,
                     x);
}

fd_status fd_read_kv(const void* k_cache, const void* v_cache, const int32_t* kv_start_idx,
                     const int32_t* block_table, int block_table_stride,
                     const int32_t* out_start, const int32_t* first, int64_t num_rows,
                     int64_t kv_rows, int batch, int num_kv_heads, int head_dim, int page_size,
                     float k_scale, float v_scale, fd_scale_kind scale_kind,
                     const float* k_scales, const float* v_scales, fd_dtype kv_dtype,
                     fd_dtype out_dtype, void* k_out, void* v_out, void* workspace,
                     size_t workspace_bytes, fd_stream_t stream) {
  const fd_status chk = check_placement(
      k_cache, v_cache, kv_start_idx, block_table, block_table_stride, out_start, num_rows,
      kv_rows, batch, num_kv_heads, head_dim, page_size, scale_kind, k_scales, v_scales, out_dtype,
      kv_dtype, workspace);
  if (chk != FD_OK) return chk;
  if (num_rows > 0 && (!k_out || !v_out)) return FD_ERR_INVALID_ARG;
  if (!aligned(k_out, 16) || !aligned(v_out, 16) ||
      (first && !aligned(first, 4)))
    return FD_ERR_INVALID_ARG;
  if (!std::isfinite(k_scale) || !std::isfinite(v_scale)) return FD_ERR_INVALID_ARG;
  if (workspace_bytes < sizeof(WsHeader)) return FD_ERR_WORKSPACE_TOO_SMALL;
  if (num_rows == 0) return FD_OK;
  const int sms = current_sms();
  if (sms <= 0) return FD_ERR_CUDA;

  ReadKv p;
  std::memset(&p, 0, sizeof(p));
  p.at = placement(kv_start_idx, block_table, block_table_stride, kv_rows, batch, page_size,
                   workspace);
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_out = k_out;
  p.v_out = v_out;
  p.out_start = out_start;
  p.first = first;
  p.rows = (int)num_rows;
  p.num_kv_heads = num_kv_heads;
  p.head_dim = head_dim;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.scale_kind = scale_kind;
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.kv_dtype = kv_dtype;
  p.out_dtype = out_dtype;
  return launch_read_kv(p, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FD_OK
             : FD_ERR_CUDA;
}

size_t fd_assign_pages_workspace_bytes(int batch) {
  return batch > 0 && batch <= (1 << 24) ? assign_pages_bytes(batch) : 0;
}

fd_status fd_assign_pages(int32_t* block_table, int block_table_stride, const int32_t* seq_len,
                          const int32_t* new_tokens, int32_t* free_pages, int64_t free_capacity,
                          const int32_t* free_count, int batch, int page_size, int window,
                          int sinks, const int32_t* released, int32_t* seq_len_out,
                          int32_t* free_count_out, int32_t* released_out, int32_t* q_start,
                          int32_t* positions, int64_t* slots, int64_t num_slots, void* workspace,
                          size_t workspace_bytes, fd_stream_t stream) {
  return fd_assign_pages_attended(block_table, block_table_stride, seq_len, new_tokens, free_pages,
                                  free_capacity, free_count, batch, page_size, window, sinks,
                                  released, seq_len_out, free_count_out, released_out, q_start,
                                  positions, slots, num_slots, nullptr, workspace,
                                  workspace_bytes, stream);
}

fd_status fd_assign_pages_attended(int32_t* block_table, int block_table_stride,
                                   const int32_t* seq_len, const int32_t* new_tokens,
                                   int32_t* free_pages, int64_t free_capacity,
                                   const int32_t* free_count, int batch, int page_size, int window,
                                   int sinks, const int32_t* released, int32_t* seq_len_out,
                                   int32_t* free_count_out, int32_t* released_out,
                                   int32_t* q_start, int32_t* positions, int64_t* slots,
                                   int64_t num_slots, int32_t* attend_len, void* workspace,
                                   size_t workspace_bytes, fd_stream_t stream) {
  if (!block_table || !seq_len || !new_tokens || !free_pages || !free_count || !seq_len_out ||
      !free_count_out || !q_start || !positions || !workspace)
    return FD_ERR_INVALID_ARG;
  if (batch <= 0 || batch > (1 << 24) || block_table_stride <= 0) return FD_ERR_INVALID_ARG;
  if (free_capacity <= 0 || free_capacity >= kMaxPacked) return FD_ERR_INVALID_ARG;
  if ((int64_t)batch * block_table_stride >= kMaxPacked) return FD_ERR_UNSUPPORTED;
  if (!is_pow2(page_size) || page_size > 256) return FD_ERR_UNSUPPORTED;
  if (window < 0 || sinks < 0 || (window == 0 && sinks != 0)) return FD_ERR_INVALID_ARG;
  if ((window > 0) != (released != nullptr) || (window > 0) != (released_out != nullptr))
    return FD_ERR_INVALID_ARG;
  if (num_slots < 0 || num_slots >= kMaxPacked || (!slots && num_slots > 0))
    return FD_ERR_INVALID_ARG;
  for (const int32_t* a : {(const int32_t*)block_table, seq_len, new_tokens,
                           (const int32_t*)free_pages, free_count, released,
                           (const int32_t*)seq_len_out, (const int32_t*)free_count_out,
                           (const int32_t*)released_out, (const int32_t*)q_start,
                           (const int32_t*)positions, (const int32_t*)attend_len})
    if (!aligned(a, 4)) return FD_ERR_INVALID_ARG;
  if (!aligned(slots, 8) || !aligned(workspace, 256)) return FD_ERR_INVALID_ARG;
  if (workspace_bytes < assign_pages_bytes(batch)) return FD_ERR_WORKSPACE_TOO_SMALL;
  // Arrays lie apart, but for a state that takes the old one's place (starts
  // overwritten by another array would send the fill outside the table).
  const struct {
    const void* at;
    int64_t bytes;
    int old;   // entry whose array this one may be
  } all[] = {
      {seq_len, 4ll * batch, -1},
      {new_tokens, 4ll * batch, -1},
      {free_count, 4, -1},
      {released, 4ll * batch, -1},
      {block_table, 4ll * batch * block_table_stride, -1},   // from here on written
      {free_pages, 4 * free_capacity, -1},
      {seq_len_out, 4ll * batch, 0},
      {free_count_out, 4, 2},
      {released_out, 4ll * batch, 3},
      {q_start, 4 * (batch + 1ll), -1},
      {positions, 4ll * batch, -1},
      {slots, 8 * num_slots, -1},
      {attend_len, 4ll * batch, -1},
      {workspace, (int64_t)assign_pages_bytes(batch), -1},
  };
  for (int i = 4; i < (int)(sizeof(all) / sizeof(all[0])); ++i)
    for (int j = 0; j < i; ++j)
      if (all[i].at && all[j].at && !(all[i].old == j && all[i].at == all[j].at) &&
          all[i].bytes > 0 && overlap(all[i].at, all[i].bytes, all[j].at, all[j].bytes, 0, 1))
        return FD_ERR_INVALID_ARG;
  const int sms = current_sms();
  if (sms <= 0) return FD_ERR_CUDA;
  AssignPages p;
  std::memset(&p, 0, sizeof(p));
  p.table = block_table;
  p.stride = block_table_stride;
  p.seq_len = seq_len;
  p.new_tokens = new_tokens;
  p.free_pages = free_pages;
  p.capacity = free_capacity;
  p.free_count = free_count;
  p.released = released;
  p.seq_len_out = seq_len_out;
  p.free_count_out = free_count_out;
  p.released_out = released_out;
  p.q_start = q_start;
  p.positions = positions;
  p.attend_len = attend_len;
  static_assert(sizeof(long long) == sizeof(int64_t), "slots");
  p.slots = reinterpret_cast<long long*>(slots);
  p.num_slots = num_slots;
  p.batch = batch;
  p.page_shift = log2i(page_size);
  p.window = window;
  p.keep = (int)(((int64_t)sinks + page_size - 1) / page_size);
  p.ws = static_cast<WsHeader*>(workspace);
  return launch_assign_pages(p, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FD_OK
             : FD_ERR_CUDA;
}

size_t fd_prefill_workspace_bytes(int head_dim) {
  if (head_dim != 64 && head_dim != 128) return 0;
  const int sms = current_sms();
  return sms > 0 ? prefill_layout(head_dim, sms).total : 0;
}

static fd_status prefill_impl(const void* q, int64_t q_stride, const void* k_cache,
                              const void* v_cache, const int32_t* kv_start_idx,
                              const int32_t* block_table, int block_table_stride,
                              const int32_t* q_start, const int32_t* seq_len,
                              int64_t num_tokens, int64_t kv_rows, int batch, int num_q_heads,
                              int num_kv_heads, int head_dim, int page_size,
                              float softmax_scale, float k_scale, float v_scale,
                              fd_scale_kind scale_kind, const float* k_scales,
                              const float* v_scales, fd_dtype q_dtype, fd_dtype kv_dtype,
                              void* out, float* lse, void* workspace, size_t workspace_bytes,
                              fd_stream_t stream, int window, int sinks) {
  const fd_status chk = check_placement(
      k_cache, v_cache, kv_start_idx, block_table, block_table_stride, q_start, num_tokens,
      kv_rows, batch, num_kv_heads, head_dim, page_size, scale_kind, k_scales, v_scales, q_dtype,
      kv_dtype, workspace);
  if (chk != FD_OK) return chk;
  if (!seq_len || (num_tokens > 0 && (!q || !out))) return FD_ERR_INVALID_ARG;
  if (num_q_heads <= 0 || num_q_heads % num_kv_heads != 0) return FD_ERR_INVALID_ARG;
  if (num_q_heads / num_kv_heads > 128 || num_q_heads > 4096) return FD_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(seq_len, 4) || (lse && !aligned(lse, 4)) ||
      !stride_ok(q_stride, num_q_heads, head_dim))
    return FD_ERR_INVALID_ARG;
  if (!std::isfinite(softmax_scale) || !std::isfinite(k_scale) || !std::isfinite(v_scale))
    return FD_ERR_INVALID_ARG;
  if (kv_rows >= kMaxPacked) return FD_ERR_UNSUPPORTED;   // 32-bit TMA coordinates
  const int64_t width = (int64_t)num_q_heads * head_dim * 2;
  if (overlap(out, width, q, width, 2 * q_stride, num_tokens)) return FD_ERR_INVALID_ARG;
  const int sms = current_sms();
  if (sms <= 0) return FD_ERR_CUDA;
  if (workspace_bytes < prefill_layout(head_dim, sms).total) return FD_ERR_WORKSPACE_TOO_SMALL;
  if (num_tokens == 0) return FD_OK;

  Prefill p;
  std::memset(&p, 0, sizeof(p));
  p.at = placement(kv_start_idx, block_table, block_table_stride, kv_rows, batch, page_size,
                   workspace);
  p.q = q;
  p.q_stride = q_stride;
  p.k = k_cache;
  p.v = v_cache;
  p.out = out;
  p.lse = lse;
  p.q_start = q_start;
  p.seq_len = seq_len;
  p.tokens = (int)num_tokens;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.head_dim = head_dim;
  p.group = num_q_heads / num_kv_heads;
  p.score_scale = softmax_scale * k_scale * kLog2e;
  p.v_scale = v_scale;
  p.scale_kind = scale_kind;
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.q_dtype = q_dtype;
  p.kv_dtype = kv_dtype;
  p.window = window;
  // (so that whole tiles of them are still an int; longer sequences are refused)
  p.sinks = sinks < 0x7fffff00 ? sinks : 0x7fffff00;
  p.wait_ns = wait_limit_ns();
  p.starve = starve_switch();
  p.grid = sms;
  return launch_prefill(p, workspace, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FD_OK
             : FD_ERR_CUDA;
}

fd_status fd_prefill_attention(const void* q, int64_t q_stride, const void* k_cache,
                               const void* v_cache, const int32_t* kv_start_idx,
                               const int32_t* block_table, int block_table_stride,
                               const int32_t* q_start, const int32_t* seq_len,
                               int64_t num_tokens, int64_t kv_rows, int batch, int num_q_heads,
                               int num_kv_heads, int head_dim, int page_size, float softmax_scale,
                               float k_scale, float v_scale, fd_scale_kind scale_kind,
                               const float* k_scales, const float* v_scales, fd_dtype q_dtype,
                               fd_dtype kv_dtype, void* out, float* lse, void* workspace,
                               size_t workspace_bytes, fd_stream_t stream) {
  return prefill_impl(q, q_stride, k_cache, v_cache, kv_start_idx, block_table, block_table_stride,
                      q_start, seq_len, num_tokens, kv_rows, batch, num_q_heads, num_kv_heads,
                      head_dim, page_size, softmax_scale, k_scale, v_scale, scale_kind, k_scales,
                      v_scales, q_dtype, kv_dtype, out, lse, workspace, workspace_bytes, stream,
                      0, 0);
}

fd_status fd_prefill_attention_window(const void* q, int64_t q_stride, const void* k_cache,
                                      const void* v_cache, const int32_t* kv_start_idx,
                                      const int32_t* block_table, int block_table_stride,
                                      const int32_t* q_start, const int32_t* seq_len,
                                      int64_t num_tokens, int64_t kv_rows, int batch, int num_q_heads,
                                      int num_kv_heads, int head_dim, int page_size, int window, int sinks, float softmax_scale,
                                      float k_scale, float v_scale, fd_scale_kind scale_kind,
                                      const float* k_scales, const float* v_scales, fd_dtype q_dtype,
                                      fd_dtype kv_dtype, void* out, float* lse, void* workspace,
                                      size_t workspace_bytes, fd_stream_t stream) {
  if (window < 1 || sinks < 0) return FD_ERR_INVALID_ARG;
  return prefill_impl(q, q_stride, k_cache, v_cache, kv_start_idx, block_table, block_table_stride,
                      q_start, seq_len, num_tokens, kv_rows, batch, num_q_heads, num_kv_heads,
                      head_dim, page_size, softmax_scale, k_scale, v_scale, scale_kind, k_scales,
                      v_scales, q_dtype, kv_dtype, out, lse, workspace, workspace_bytes, stream,
                      window, sinks);
}

}  // extern "C"
