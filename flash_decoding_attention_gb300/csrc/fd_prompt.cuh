// fd_prompt.cuh -- pieces shared by the prompt path's kernels (packed append,
// cache read-back, rotary table, attention of packed new tokens): the
// placement of cached tokens, the search of a packed token's sequence, and
// the launchers that fd_prompt_api.cu calls.
#pragma once

#include "fd_common.cuh"

namespace fd {

// Where a batch's cached tokens lie.
struct Placement {
  const int32_t* kv_start;      // contiguous caches
  const int32_t* block_table;   // paged caches
  long long kv_rows;
  int bt_stride, page_shift, page_size, batch;
  WsHeader* ws;
};

// Row of token t of sequence b, or -1 (recorded) when it lies outside the
// cache or past the block table's row.
__device__ __forceinline__ long long placed_row(const Placement& pl, int b, int t) {
  if (pl.block_table) {
    const int col = t >> pl.page_shift;
    if (t < 0 || col >= pl.bt_stride) {
      raise_error(pl.ws, kErrBounds, t);
      return -1;
    }
    const int page = __ldg(pl.block_table + (long long)b * pl.bt_stride + col);
    const long long row = ((long long)page << pl.page_shift) + (t & (pl.page_size - 1));
    if (page < 0 || row >= pl.kv_rows) {
      raise_error(pl.ws, kErrBounds, page);
      return -1;
    }
    return row;
  }
  const long long row = (long long)__ldg(pl.kv_start + b) + t;
  if (t < 0 || row < 0 || row >= pl.kv_rows) {
    raise_error(pl.ws, kErrBounds, row);
    return -1;
  }
  return row;
}

// The sequence that owns packed token i (start[b] <= i < start[b + 1]), or -1
// when none does.  Binary search for the last start <= i; sequences without
// tokens are passed over because their successor starts at the same token.
__device__ __forceinline__ int owner_of(const int32_t* start, int batch, int i) {
  if (i < __ldg(start)) return -1;
  int lo = 0, hi = batch;   // start[lo] <= i
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(start + mid) <= i) lo = mid;
    else hi = mid;
  }
  return i < __ldg(start + lo + 1) ? lo : -1;
}

// Records the sequences whose starts descend or lie outside the `rows` packed
// rows, by the threads of one block.  (The search of a token's owner never
// meets a sequence that owns no token.)
__device__ __forceinline__ void check_starts(const Placement& pl, const int32_t* start, int rows) {
  for (int b = threadIdx.x; b < pl.batch; b += blockDim.x) {
    const int lo = __ldg(start + b), hi = __ldg(start + b + 1);
    if (lo < 0 || hi < lo || hi > rows) raise_error(pl.ws, kErrBounds, lo < 0 ? lo : hi);
  }
}

constexpr int kMaxRotDim = 128;

struct AppendPacked {
  Placement at;
  const void *q, *k_new, *v_new;
  void *q_out, *k_cache, *v_cache;
  const int32_t *q_start, *positions;
  const float* rotary;
  long long q_stride, kv_stride, rotary_positions;
  int tokens, num_q_heads, num_kv_heads, head_dim, rot_dim, interleaved;
  float k_scale, v_scale;
  int scale_kind;
  float *k_scales, *v_scales;
  int new_dtype, kv_dtype;
  // norms of heads (weights [head_dim] of new_dtype, or fp32 with norm_f32)
  const void *q_norm, *k_norm;
  int norm_f32;
  float norm_eps;
  // positions [num_axes] rows of axis_stride, and the axis of every pair
  int num_axes;
  long long axis_stride;
  const int32_t* axis_positions;
  uint8_t pair_axis[kMaxRotDim / 2];
};

struct ReadKv {
  Placement at;
  const void *k_cache, *v_cache;
  void *k_out, *v_out;
  const int32_t *out_start, *first;
  int rows, num_kv_heads, head_dim;
  float k_scale, v_scale;
  int scale_kind;
  const float *k_scales, *v_scales;
  int kv_dtype, out_dtype;
};

// The scaled frequencies as fixed-point turns per position (2^64 = one turn).
struct RotaryTable {
  float* table;
  long long positions;
  int rot_dim;
  float amplitude;
  unsigned long long turns[kMaxRotDim / 2];
};

struct Prefill {
  Placement at;
  const void *q, *k, *v;
  void* out;
  float* lse;
  const int32_t *q_start, *seq_len;
  long long q_stride;
  int tokens, num_q_heads, num_kv_heads, head_dim, group;
  float score_scale;   // softmax_scale * k_scale * log2(e)
  float v_scale;
  int scale_kind;
  const float *k_scales, *v_scales;
  int q_dtype, kv_dtype;
  // Sliding window (0: none): position q sees keys t with q - window < t <= q
  // and the first `sinks` ones.  sink_keys: sinks rounded up to whole tiles;
  // win_align: window tiles start at a multiple of it (a box's rows; 1: anywhere)
  int window, sinks, sink_keys, win_align;
  unsigned long long wait_ns;
  int starve;
  int grid;            // CTAs of the attention kernel
  int tile_tokens;     // tokens of a 128-row query tile: 128 / group
  int gather;          // pages too small for TMA boxes: rows copied by threads
  // workspace: partial states of streams cut between CTAs
  int4* meta;          // [grid][2]: stream {sequence, KV head, tile pair} of a slot
  float2* part_ml;     // [grid][2][query tile][128 rows]: m (log2 units), l
  float* part_acc;     // [grid][2][query tile][head_dim / 4][128 rows][4]
};

struct PrefillLayout {
  size_t meta_off, ml_off, acc_off, total;
};
PrefillLayout prefill_layout(int head_dim, int sms);

struct PageRec {
  int L, held;   // cached tokens, pages held
  int need;      // pages handed out; -1: its tokens are not served
  int keep, lo;  // columns that go back: [0, keep), then from lo on
};

struct PageTotals {
  long long count, avail;   // of the stack: before, and with what returns
  long long back, handed;   // pages
};

struct AssignPages {
  int32_t *table, *free_pages;
  const int32_t *seq_len, *new_tokens, *free_count, *released;
  int32_t *seq_len_out, *free_count_out, *released_out, *q_start, *positions;
  int32_t* attend_len;   // or null
  long long* slots;
  long long num_slots, capacity;
  int batch, stride, page_shift;
  int window, keep;   // 0: none; columns [0, keep) hold first tokens and stay
  WsHeader* ws;
  // workspace of the two-launch form: what each sequence gives and takes, and
  // the sums before it
  PageTotals* totals;
  PageRec* rec;
  int32_t *back, *handed;
};

size_t assign_pages_bytes(int batch);
cudaError_t launch_assign_pages(AssignPages p, int sms, cudaStream_t stream);
cudaError_t launch_append_normed(const AppendPacked& p, int sms, cudaStream_t stream);
cudaError_t launch_append_packed(const AppendPacked& p, int sms, cudaStream_t stream);
cudaError_t launch_read_kv(const ReadKv& p, int sms, cudaStream_t stream);
cudaError_t launch_rotary_table(const RotaryTable& p, int sms, cudaStream_t stream);
cudaError_t launch_prefill(Prefill p, void* workspace, cudaStream_t stream);

}  // namespace fd
