// fd_prefill.cuh -- attention of packed new tokens over the cache, on the
// fifth-generation tensor cores; included by one translation unit per format
// (fd_prefill_*.cu), which instantiate its variants, and by fd_prefill.cu
// (tensor maps, dispatch, merge).
//
//   s_t = softmax_scale k_scale ks_t (q . k_t),  t <= position of the token,
//   m = max_t s_t log2 e,  p_t = 2^(s_t log2 e - m),  l = sum_t p_t,
//   out = v_scale sum_t p_t vs_t v_t / l,  lse = (m + log2 l) ln 2,
// one pass over the keys in tiles of 128 with a running m and l.
//
// Rows.  A KV head's group of g query heads times the tokens of a sequence
// are the rows of a product with that head's keys; a query tile is 128 / g
// whole tokens (at most 128 rows), and a CTA works on two neighbouring query
// tiles A and B at a time against the same stream of K and V tiles, so that
// the softmax of one runs while the tensor cores work for the other.
//
// Split.  (sequence, KV head, pair of query tiles) are the streams.  Their
// costs (keys to pass plus a start) are laid end to end and cut into one
// equal range per CTA, whatever the lengths: a long prompt's causal triangle,
// a chunk over a long context and single tokens beside them all fill the GPU.
// A stream cut between CTAs leaves partial states (m, l, unnormalised out)
// that fd_prefill.cu merges in a fixed order.  A pair with rows in A only (a solo segment: single tokens, a
// chunk's end) has its keys shared between the two halves of the CTA instead,
// which merge their states through shared memory: the time of a tile is a
// chain (S, softmax, P V), the same for one query tile as for two.
//
// What bounds it, on GB300 (152 SMs), bf16, 32 query / 8 KV heads, D = 128:
// 2048 new tokens over 30000 cached ones run at 1.70 PFLOP/s, 0.87 of the
// cuBLAS burst rate and 0.99 of its sustained one: the tensor cores (and the
// power limit).  Whole prompts, with a start and an end for every 26 tiles or
// so, run at 1.52 PFLOP/s replayed from a graph, 1.41 called one by one.  With
// 8-bit caches the widened copies compete with the products for shared
// memory's port (e4m3 under f16 1.6 PFLOP/s).  Decode-like batches (one token
// over 4096 keys, bf16) read the cache at 5.5 TB/s.
//
// Roles (one persistent CTA per SM):
//   warps 0-3, 4-7  softmax of query tile A, B: one row per thread, its scores
//                   read from tensor memory twice (maximum, probabilities);
//                   P overwrites S there as 16-bit pairs;
//   warp 8          TMA producer: Q tiles, K and V tiles through one ring;
//   warp 9          issues S = Q K^T and O += P V for A and B as their inputs
//                   become ready (O and S: 2 x 128 columns each, all 512);
//   warps 10-11     repair V tiles that some row may not see (see below); with
//                   a scale per token they fetch the scales instead;
//   warps 12-15     (8-bit caches, or pages of fewer than 8 rows) widen or
//                   copy the cache rows into the ring; the producer then feeds
//                   raw tiles to them.
//
// A tile in which some row sees fewer than all keys: scores of unseen keys
// are excluded by selection, so K may hold any bits there, but in O += P V an
// unseen non-finite V element would reach every row as 0 * NaN.  V elements
// of such tiles are therefore zeroed when no row sees them, and when some
// rows do, non-finite ones are zeroed and the segment is marked; its epilogue
// then adds the non-finite elements of a row's own keys to that row.
//
// Sliding window (WIN, instantiations of their own): a pair's stream leaves out the
// tiles between the first tokens' and its window's (pair_gap); in the remaining
// ones some rows hide keys at the lower end as others do at the upper, and both
// are treated alike (Sight).  Segments are short, so what surrounds their tiles
// counts: 16384 bf16 tokens of 32/8 heads take 1.07 ms with a window of 8192 (1.54
// PFLOP/s) and 289 us with 1024 (0.92), 9 tiles of 1.38 us a segment beside 6 us
// of masks, last product, epilogue and restart, which nothing overlaps because
// both query tiles of a pair begin and end on the same keys.  An edge tile is put
// right in tensor memory in those blocks of 32 keys that some row of the warp sees
// and some does not (3.7 -> 2.2 us for a first tile), the next segment is walked to
// under the last product, and the usual epilogue loads ahead of its stores (2.5 ->
// 1.4).
//
// Roundings below 32 bits: P to the query's 16-bit type (the tensor cores
// take 16-bit operands; an error of half a step of each probability, the
// size of the output's own rounding; l sums P unrounded, so that the lse keeps
// 32 bits), and the output.  With f16, P is scaled by 2^6 so that small
// probabilities stay above f16's subnormals; the running maximum is moved only
// when exceeded by 2^8 (O is then rescaled in tensor memory), which keeps P
// below 2^14 (so P of a row's largest score need not be exact).  With a scale per token as well,
// P times the V scale is what is rounded, divided by the power of two of the
// largest scale that the row itself has seen: taken over the whole tile, a
// later token's scale would push an earlier row's P out of f16's range.
#pragma once

#include "fd_prompt.cuh"
#include "fd_tcgen05.cuh"

namespace fd {
namespace pf {

using mma::mbar_arrive;
using mma::mbar_arrive_tx;
using mma::mbar_init;
using mma::mbar_try_wait;
using mma::mbar_wait;
using mma::smem_u32;
using namespace tc;

constexpr int kTile = 128;          // keys per tile
constexpr int kRowsTile = 128;      // rows of a query tile
constexpr int kRowsPair = 2 * kRowsTile;
constexpr int kProducerWarp = 8, kMmaWarp = 9, kFixWarp0 = 10, kConvWarp0 = 12;
constexpr int kPages = 20;          // block-table entries staged at a time (a tile has 16)
constexpr int kMaxSlots = 8, kMaxRaw = 4;
// What the split counts, in keys: a segment's start (Q load, first product,
// epilogue: about 7 us, against 1.4 to 2.5 for a tile) and a tile that only
// query tile A passes.  Neither is sharp: four bf16 prompts (10824 tokens) take
// 421 us with a start of 320, 390 with 400, 382 with 560, 384 with 640, 399 with
// 800 and 400 with 1000; e4m3 chunks 128, 126, 124, 122, 118 and 122.  Without a
// scale per token a solo tile costs as much as a full one where it matters
// (8-bit: the widening bounds both).  With one, the softmax of a full tile is
// the longer chain, 2.3 against 1.9 us: a mixed INT8 batch takes 243 us with
// 320 and 128, 239 with 320 and 92, 229 with 384 and 92, 240 with 448 and 92.
template <bool TOK>
struct Cost {
  static constexpr int kStart = TOK ? 448 : 640;
  static constexpr int kSolo = TOK ? 92 : kTile;
};

// ---------------------------------------------------------------------------
// Streams and their split
// ---------------------------------------------------------------------------
struct Seq {
  int b, q0, n, T, ctx, pairs, span;   // span: tokens of a pair
  bool solo;                           // (TOK) the last pair has rows in A only
  long long head;                      // cost of one KV head
};

// The last key that a token of pair m sees, plus one.
__device__ __forceinline__ int pair_end(const Seq& s, int m) {
  const long long t = (long long)(m + 1) * s.span;
  const int e = s.ctx + (t < s.n ? (int)t : s.n);
  return e > 0 ? e : 0;
}

// With a window (WIN; position q sees key t when q - window < t <= q or t <
// sinks) a pair's stream leaves out the middle that none of its tokens sees:
// key x of the stream is key x of the sequence below sink_keys (the first
// tokens, rounded up to whole tiles), and x + gap from there on.
__device__ __forceinline__ long long window_start(const Prefill& p, const Seq& s, int m) {
  return (long long)s.ctx + (long long)m * s.span - p.window + 1;   // of its first token
}

template <bool WIN>
__device__ __forceinline__ int pair_gap(const Prefill& p, const Seq& s, int m) {
  if constexpr (!WIN) return 0;
  const long long first = window_start(p, s, m);
  return first > 0 ? max(0, ((int)first & ~(p.win_align - 1)) - p.sink_keys) : 0;
}

// The keys that a pair's cost leaves out: at most the gap (which jumps by
// win_align, where this grows by one a token and so can be summed).
__device__ __forceinline__ long long skipped(const Prefill& p, const Seq& s, int m) {
  return max(0ll, window_start(p, s, m) - p.sink_keys - (p.win_align - 1));
}

template <bool TOK, bool WIN>
__device__ __forceinline__ long long pair_cost(const Prefill& p, const Seq& s, int m) {
  const long long end = pair_end(s, m) - (WIN ? skipped(p, s, m) : 0ll);
  if constexpr (TOK) {
    if (s.solo && m == s.pairs - 1)
      return Cost<TOK>::kStart + (end * Cost<TOK>::kSolo + kTile - 1) / kTile;
  }
  return Cost<TOK>::kStart + end;
}

// Cost of pairs 0 .. m - 1 (m < pairs: all of them are full).
template <bool TOK, bool WIN>
__device__ __forceinline__ long long pairs_before(const Prefill& p, const Seq& s, int m) {
  long long c = (long long)m * Cost<TOK>::kStart;
  const int m0 = s.ctx >= 0 ? 0 : -s.ctx / s.span;   // pairs without keys
  if (m > m0) {
    const long long a = m, b = m0;
    c += (a - b) * s.ctx + (long long)s.span * ((a * (a + 1) - b * (b + 1)) / 2);
  }
  if constexpr (WIN) {   // less skipped(i) = first + i span, i < m, where positive
    const long long first = window_start(p, s, 0) - p.sink_keys - (p.win_align - 1);
    const long long a = m, b = first > 0 ? 0 : -first / s.span + 1;
    if (a > b) c -= (a - b) * first + (long long)s.span * ((a * (a - 1) - b * (b - 1)) / 2);
  }
  return c;
}

template <bool TOK, bool WIN>
__device__ inline Seq load_seq(const Prefill& p, int b, bool report) {
  Seq s;
  s.b = b;
  const int lo = __ldg(p.q_start + b), hi = __ldg(p.q_start + b + 1);
  s.T = max(0, __ldg(p.seq_len + b));
  s.q0 = lo;
  s.n = hi - lo;
  if (lo < 0 || hi < lo || hi > p.tokens || s.T > 0x7fffff00) {   // (tile ends stay int)
    if (report) raise_error(p.at.ws, kErrBounds, lo < 0 ? lo : hi < lo || hi > p.tokens ? hi : s.T);
    s.n = 0;
  }
  s.ctx = s.T - s.n;
  s.span = 2 * p.tile_tokens;
  s.pairs = (int)(((unsigned)s.n + (unsigned)s.span - 1u) / (unsigned)s.span);
  if constexpr (TOK)
    s.solo = s.n > 0 && s.n - (long long)(s.pairs - 1) * s.span <= p.tile_tokens;
  s.head = s.n > 0 ? pairs_before<TOK, WIN>(p, s, s.pairs - 1) +
                         pair_cost<TOK, WIN>(p, s, s.pairs - 1)
                   : 0;
  return s;
}

struct Plan {
  long long total, per_cta;   // cost, and cost per CTA
  long long first;            // cost before sequence b
  int b;                      // sequence holding this CTA's first unit
};

// Every thread of the CTA gets the plan; `red` is 34 long longs of shared memory.
template <bool TOK, bool WIN>
__device__ inline Plan make_plan(const Prefill& p, long long* red) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  const int B = p.at.batch;
  long long mine = 0, v0 = 0;
  for (int b = tid; b < B; b += blockDim.x) {
    const long long v = load_seq<TOK, WIN>(p, b, blockIdx.x == 0).head * p.num_kv_heads;
    if (b == tid) v0 = v;
    mine += v;
  }
  for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) red[warp] = mine;
  __syncthreads();
  Plan r;
  r.total = 0;
  for (int w = 0; w < nw; ++w) r.total += red[w];
  // every CTA but the last takes at least one tile, so a range inside a
  // stream always holds one
  r.per_cta = (r.total + p.grid - 1) / p.grid;
  if (r.per_cta < kTile) r.per_cta = kTile;
  const long long target = (long long)blockIdx.x * r.per_cta;
  __syncthreads();
  if (tid == 0) {
    red[32] = B;
    red[33] = r.total;
  }
  long long carry = 0;
  for (int base = 0; base < B; base += blockDim.x) {
    const int b = base + tid;
    const long long v = b >= B ? 0 : base == 0 ? v0 : load_seq<TOK, WIN>(p, b, false).head * p.num_kv_heads;
    long long x = v;
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) red[warp] = x;
    __syncthreads();
    long long before = carry, all = 0;
    for (int w = 0; w < nw; ++w) {
      if (w < warp) before += red[w];
      all += red[w];
    }
    const long long excl = before + x - v;
    if (v > 0 && excl <= target && target < excl + v) {
      red[32] = b;
      red[33] = excl;
    }
    carry += all;
    __syncthreads();
  }
  r.b = (int)red[32];
  r.first = red[33];
  fence_async_smem();   // `red` lies where the first Q tile lands
  __syncthreads();
  return r;
}

struct Seg {
  int b, q0, n, ctx, h, m;   // sequence (first packed token, tokens, cached before), KV head, pair
  int tb, te;                // tiles [tb, te) of the pair's stream
  int end;                   // the last key of the stream, plus one
  int gap;                   // (WIN) keys left out behind sink_keys
  int nt[2];                 // tiles of query tile A, B in the stream (0: no rows or no keys)
  bool solo;                 // no rows in B: its softmax takes A's odd tiles (see below)
  bool complete;             // the whole stream
  int slot;                  // partial slot otherwise
};

// The first sequence behind b whose entries differ, or the batch's end; by a
// whole warp, 32 sequences at a time (a batch may hold millions of empty ones,
// and the other warps' waits have their limit).
static __device__ __forceinline__ int next_owner(const int32_t* start, int batch, int b) {
  for (++b; b < batch; b += 32) {
    const int i = b + (threadIdx.x & 31);
    const bool owns = i < batch && __ldg(start + i) != __ldg(start + i + 1);
    const unsigned any = __ballot_sync(0xffffffffu, owns);
    if (any) return b + __ffs(any) - 1;
  }
  return batch;
}

// The segments of this CTA, in order; every role walks its own copy.
template <bool TOK, bool WIN>
struct Walk {
  long long g, g_end, ps;
  Seq s;
  int h, m;

  __device__ void init(const Prefill& p, const Plan& pl) {
    g = (long long)blockIdx.x * pl.per_cta;
    g_end = min(g + pl.per_cta, pl.total);
    ps = g_end;
    if (g >= pl.total || pl.b >= p.at.batch) return;
    s = load_seq<TOK, WIN>(p, pl.b, false);
    const long long off = g - pl.first;
    h = (int)(off / s.head);
    const long long r = off - h * s.head;
    int lo = 0, hi = s.pairs;   // the last pair that begins at or before r
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pairs_before<TOK, WIN>(p, s, mid) <= r) lo = mid;
      else hi = mid;
    }
    m = lo;
    ps = pl.first + h * s.head + pairs_before<TOK, WIN>(p, s, m);
  }

  __device__ __forceinline__ bool next(const Prefill& p, Seg& o) {
    while (ps < g_end) {
      const int end = pair_end(s, m);
      const long long cost = pair_cost<TOK, WIN>(p, s, m);
      const int gap = pair_gap<WIN>(p, s, m);
      const int n = (end - gap + kTile - 1) / kTile;
      const long long a = g > ps ? g : ps, e = ps + cost < g_end ? ps + cost : g_end;
      // tile i stands at ps + the start + i times its cost and belongs to the
      // range that holds this point
      const long long xa = a - ps - Cost<TOK>::kStart, xe = e - ps - Cost<TOK>::kStart;
      auto tiles_at = [&](long long x) -> int {   // (a stream costs less than 2^32)
        if constexpr (TOK) {
          constexpr unsigned kSolo = Cost<TOK>::kSolo;
          if (s.solo && m == s.pairs - 1) return (int)(((unsigned)x + kSolo - 1u) / kSolo);
        }
        return (int)((x + kTile - 1) >> 7);
      };
      const int tb = xa <= 0 ? 0 : min(n, tiles_at(xa));
      const int te = xe <= 0 ? 0 : min(n, tiles_at(xe));
      const bool yields = n > 0 ? te > tb : g <= ps;
      if (yields) {
        o.b = s.b;
        o.q0 = s.q0;
        o.n = s.n;
        o.ctx = s.ctx;
        o.h = h;
        o.m = m;
        o.tb = tb;
        o.te = te;
        o.end = end;
        o.gap = gap;
        const int half = s.span >> 1;
        const int ea = s.ctx + (int)min((long long)s.n, (long long)m * s.span + half);
        o.nt[0] = ea > 0 ? (ea - gap + kTile - 1) / kTile : 0;
        o.solo = (long long)m * s.span + half >= s.n;
        o.nt[1] = o.solo ? 0 : n;
        o.complete = tb == 0 && te == n;
        o.slot = 2 * (int)blockIdx.x + (tb > 0 ? 0 : 1);
      }
      ps += cost;
      if (++m == s.pairs) {
        m = 0;
        if (++h == p.num_kv_heads) {
          h = 0;
          if (ps < g_end) {
            int b = s.b;
            do {
              b = next_owner(p.q_start, p.at.batch, b);
              if (b >= p.at.batch) break;
              s = load_seq<TOK, WIN>(p, b, false);
            } while (s.n == 0);
          }
        }
      }
      if (yields) return true;
    }
    return false;
  }
};

// First key of the stream that some row of the pair does not see.
__device__ __forceinline__ int first_unseen(const Seg& s, int span) {
  const long long t = (long long)s.ctx + (long long)s.m * span + 1;
  return t > 0 ? (int)t : 0;
}

// What the rows of a segment's pair see of its tiles.  Without a window: all
// rows see the keys below `unseen`, and none those behind the stream's end.
template <bool WIN>
struct Sight {
  int unseen;
  // with a window: keys [sinks, any) are hidden from some row, [sinks, all) from all
  int sinks, sink_keys, any, all;
  __device__ __forceinline__ void init(const Prefill& p, const Seg& s) {
    const int span = 2 * p.tile_tokens;
    unseen = first_unseen(s, span);
    if constexpr (WIN) {
      sinks = p.sinks;
      sink_keys = p.sink_keys;
      const long long first = (long long)s.m * span;
      const long long last = min((long long)s.n, first + span) - 1;
      all = (int)max(0ll, s.ctx + first - p.window + 1);
      any = (int)max(0ll, s.ctx + last - p.window + 1);
    }
  }
  // first key of tile j, and its keys that belong to the stream
  __device__ __forceinline__ int key(const Seg& s, int j) const {
    const int x = j * kTile;
    return WIN && x >= sink_keys ? x + s.gap : x;
  }
  __device__ __forceinline__ int valid(const Seg& s, int j) const {
    if (WIN && s.gap > 0 && j * kTile < sink_keys) return min(kTile, sinks - j * kTile);
    return min(kTile, s.end - key(s, j));
  }
  // keys that some row, or no row, sees (of those that belong to the stream)
  __device__ __forceinline__ bool partly(int k) const {
    return k >= unseen || (WIN && k >= sinks && k < any);
  }
  __device__ __forceinline__ bool hidden(int k) const { return WIN && k >= sinks && k < all; }
  __device__ __forceinline__ bool hidden(int k, int n) const {
    return WIN && k >= sinks && k + n <= all;
  }
  // a tile with a key that some row does not see
  __device__ __forceinline__ bool fix(const Seg& s, int j) const {
    const int k = key(s, j);
    return k + kTile > unseen || (WIN && max(k, sinks) < min(k + kTile, any));
  }
};

// ---------------------------------------------------------------------------
// Shape and shared memory
// ---------------------------------------------------------------------------
// KV: 0 16-bit cache in the query's type, 1 e4m3, 2 int8.  CONV: the
// converter warps fill the ring.
template <int D, int KV, bool CONV>
struct Shape {
  static constexpr int kThreads = CONV ? 512 : 384;
  static constexpr uint32_t kQTile = kRowsTile * D * 2u;
  static constexpr uint32_t kSlot = kTile * D * 2u;
  static constexpr uint32_t kRaw = KV == 0 ? 0u : kTile * D * 1u;
  static constexpr int kSlots = D == 128 ? (CONV ? 4 : 5) : (CONV ? 6 : 8);
  static constexpr int kRawSlots = KV == 0 ? 0 : D == 128 ? 2 : 4;
  static constexpr uint32_t kOffSlot = 2u * kQTile;
  static constexpr uint32_t kOffRaw = kOffSlot + kSlots * kSlot;
  static constexpr uint32_t kOffCtl = kOffRaw + kRawSlots * kRaw;
};

// A tile's info, written with its K tile: the query tiles that take part, the
// ends of its segment, and what its rows are.  An entry behind the last tile
// says stop.
enum : int {
  kInfoA = 1, kInfoB = 2,            // products for query tile A, B
  kInfoLastA = 4, kInfoLastB = 8,    // their last of the segment
  kInfoStart = 16,                   // first tile of the segment
  kInfoFix = 32,                     // V is repaired before use (no converters)
  kInfoBad = 64,                     // a row lies outside the cache: the tile is absent
  kInfoSolo = 128,                   // A and B take turns on query tile A
  kInfoEnd = 256,                    // last tile of the segment
  kInfoStop = 512
};

struct Control {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t raw_full[kMaxRaw], raw_empty[kMaxRaw];
  uint64_t fixed[4];   // V tiles repaired (no converters), or V scales written (converters)
  uint64_t q_full[2], q_empty[2], s_full[2], p_half[2], p_full[2], o_full[2], fin;
  uint64_t x_full, x_empty;   // exchange between the softmax halves of a solo segment
  int info[8];      // what the tensor cores do with tile j (slot j mod 8), kInfo bits
  int nf[8];        // i + 1 (slot i mod 8) when V of segment i, of those with tiles, held
                    // non-finite elements that some row does not see
  int abort_flag;
  int swaps;        // exchanges of solo segments that are over
  uint32_t tmem_base;
  int pages[kPages];
};

constexpr uint32_t kCtlBytes = (sizeof(Control) + 15) / 16 * 16;

// Per-token scales of a tile's 128 keys: rings of kKeyRing K arrays, then
// kValRing V arrays, written when the tile's operand slots are free.  A V slot
// is free once P V is done, for which the softmax has read the V scales.  A K
// slot is free once S is done, but its scales are read after that.  The warps
// that write tile n's have waited before, for tile n - 1's V, until P V of tile
// n - 1 - kSlots / 2 was done, whose softmax had read its K scales: one array
// more than the slots hold, and the order of those waits, keep them apart.
template <int D, int KV>
struct ScaleRing {
  static constexpr int kKeyRing = Shape<D, KV, true>::kSlots / 2 + 1;
  static constexpr int kValRing = Shape<D, KV, true>::kSlots / 2;
  static constexpr uint32_t kBytes = (kKeyRing + kValRing) * kTile * 4u;
  static __device__ __forceinline__ int key(int n) { return (n % kKeyRing) * kTile; }
  static __device__ __forceinline__ int val(int n) { return (kKeyRing + n % kValRing) * kTile; }
};

template <int D, int KV, bool CONV, bool TOK>
constexpr uint32_t smem_bytes() {
  return Shape<D, KV, CONV>::kOffCtl + kCtlBytes + (TOK ? ScaleRing<D, KV>::kBytes : 0u);
}
static_assert(smem_bytes<128, 1, true, true>() <= 227u * 1024u, "shared memory");
static_assert(smem_bytes<128, 0, false, false>() <= 227u * 1024u, "shared memory");

__device__ __forceinline__ bool aborted(const Control& c) {
  return *(volatile const int*)&c.abort_flag != 0;
}

__device__ __forceinline__ void record_abort(Control& c, const Prefill& p, int role) {
  if (!aborted(c)) {
    raise_error(p.at.ws, kErrTimeout, role);
    *(volatile int*)&c.abort_flag = 1;
  }
}

static __device__ __noinline__ bool wait_slow(Control& c, const Prefill& p, uint64_t* bar,
                                       uint32_t parity, int role) {
  // a try takes a microsecond at most; once a warp has given up, all do
  const unsigned long long t0 = mma::global_ns();
  do {
    if (aborted(c)) return false;
    if (mbar_try_wait(bar, parity)) return true;
  } while (mma::global_ns() - t0 <= p.wait_ns);
  record_abort(c, p, role);
  return false;
}

// A bounded wait; on expiry the timeout is recorded and the CTA aborts.
__device__ __forceinline__ bool wait_for(Control& c, const Prefill& p, uint64_t* bar,
                                         uint32_t parity, int role) {
  if (mbar_try_wait(bar, parity)) return true;
  return wait_slow(c, p, bar, parity, role);
}

// The same by a whole warp, whose lanes all get one answer.
__device__ __forceinline__ bool wait_warp(Control& c, const Prefill& p, uint64_t* bar,
                                          uint32_t parity, int role) {
  return __all_sync(0xffffffffu, wait_for(c, p, bar, parity, role));
}

// ---------------------------------------------------------------------------
// Small pieces
// ---------------------------------------------------------------------------
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Four floats of shared memory, all lanes at one address (in program order:
// gathered ahead they would not fit beside a row's scores).
__device__ __forceinline__ void lds_pairs(const float* a, uint64_t& x, uint64_t& y) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(x), "=l"(y) : "r"(smem_u32(a)));
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// Non-finite 16-bit elements of a word zeroed; true if there was one.
template <bool BF16>
__device__ __forceinline__ bool drop_nonfinite(uint32_t& w) {
  constexpr uint32_t e = BF16 ? 0x7F80u : 0x7C00u;
  const bool lo = (w & e) == e, hi = (w & (e << 16)) == (e << 16);
  if (lo) w &= 0xFFFF0000u;
  if (hi) w &= 0x0000FFFFu;
  return lo || hi;
}

// NaN codes of an e4m3 word (S.1111.111) zeroed; true if there was one.
__device__ __forceinline__ bool drop_nan_e4m3(uint32_t& w) {
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (((w >> (8 * i)) & 0x7Fu) == 0x7Fu) {
      w &= ~(0xFFu << (8 * i));
      any = true;
    }
  return any;
}

// Solo segments of two tiles or more: the two softmax halves exchange their
// states through query tile B's place in shared memory.
__device__ __forceinline__ bool swaps_in(const Seg& s) { return s.solo && s.te - s.tb > 1; }

// Waits until `want` exchanges are over; bounded like every wait.
__device__ __forceinline__ bool wait_swaps(Control& c, const Prefill& p, int want) {
  if (*(volatile int*)&c.swaps >= want) return true;
  const unsigned long long t0 = mma::global_ns();
  while (*(volatile int*)&c.swaps < want) {
    if (aborted(c)) return false;
    if (mma::global_ns() - t0 > p.wait_ns) {
      record_abort(c, p, 4);
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ int tile_info(const Seg& s, int j, bool fix, bool bad) {
  int w = bad ? kInfoBad : 0;
  if (s.solo) {
    const int x = (j - s.tb) & 1;
    w |= kInfoSolo | (x ? kInfoB : kInfoA);
    if (j + 2 >= s.te) w |= x ? kInfoLastB : kInfoLastA;
  } else {
    if (j < s.nt[0]) w |= kInfoA | (j + 1 == min(s.te, s.nt[0]) ? kInfoLastA : 0);
    if (j < s.nt[1]) w |= kInfoB | (j + 1 == min(s.te, s.nt[1]) ? kInfoLastB : 0);
  }
  if (j == s.tb) w |= kInfoStart;
  if (j + 1 == s.te) w |= kInfoEnd;
  if (fix) w |= kInfoFix;
  return w;
}

// ---------------------------------------------------------------------------
// Producer warp
// ---------------------------------------------------------------------------
// The boxes that bring a K or V tile: of D / 64 blocks of 128-byte rows
// (16-bit), or of rows of D bytes (8-bit).
template <int D, int KV>
struct TileCopy {
  static constexpr int kRowBytes = KV == 0 || D == 128 ? 128 : 64;   // of a box
  static constexpr int kBlocks = KV == 0 ? D / 64 : 1;
  static constexpr int kBoxElems = KV == 0 ? 64 : D;
};

// Copies in flight must land before the CTA ends, which after a timeout the
// other warps do not wait for.  By one lane.
static __device__ __forceinline__ void land_copies(Control& c, const Prefill& p, uint64_t* full,
                                                   int slots, int issued, int q0, int q1) {
  bool late = false;
  for (int e = max(0, issued - slots); e < issued; ++e)
    late |= !mbar_wait(&full[e % slots], (uint32_t)((e / slots) & 1), mma::kDrainNs);
  if (q0 > 0) late |= !mbar_wait(&c.q_full[0], (uint32_t)((q0 - 1) & 1), mma::kDrainNs);
  if (q1 > 0) late |= !mbar_wait(&c.q_full[1], (uint32_t)((q1 - 1) & 1), mma::kDrainNs);
  if (late) raise_error(p.at.ws, kErrDrain, 3);
}

template <int D, int KV, bool CONV, bool TOK, bool WIN>
__device__ __forceinline__ void producer(const Prefill& p, Walk<TOK, WIN> walk, Control& c,
                                         uint8_t* base, const CUtensorMap* tmq,
                                         const CUtensorMap* tmk, const CUtensorMap* tmv) {
  using SH = Shape<D, KV, CONV>;
  using TC = TileCopy<D, KV>;
  const int lane = threadIdx.x & 31;
  // the ring that TMA fills: the operand ring, or the converters' raw ring
  constexpr int NS = KV == 0 ? SH::kSlots : SH::kRawSlots;
  uint64_t* full = KV == 0 ? c.full : c.raw_full;
  uint64_t* empty = KV == 0 ? c.empty : c.raw_empty;
  uint8_t* ring = base + (KV == 0 ? SH::kOffSlot : SH::kOffRaw);
  constexpr uint32_t kSlot = KV == 0 ? SH::kSlot : SH::kRaw;
  const bool tiles = !p.gather;   // gathered rows are the converters' business
  uint64_t keep;
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(keep));
  Seg seg;
  int n = 0, issued = 0, qn[2] = {0, 0}, swaps = 0;   // issued: stages of the ring
  bool stop = p.starve != 0;
  const int box_rows = p.at.block_table && p.at.page_size < kTile ? p.at.page_size : kTile;
  while (!stop && walk.next(p, seg)) {
    if (lane == 0) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (stop || seg.tb >= min(seg.te, seg.nt[x])) continue;
        // tile B's place may still serve an exchange of an earlier segment
        if (x == 1 && !wait_swaps(c, p, swaps)) {
          stop = true;
          continue;
        }
        if (!wait_for(c, p, &c.q_empty[x], (uint32_t)((qn[x] & 1) ^ 1), 1)) {
          stop = true;
          continue;
        }
        ++qn[x];
        const uint32_t rows = (uint32_t)(p.tile_tokens * p.group);
        mbar_arrive_tx(&c.q_full[x], rows * D * 2u);
        const int tok = seg.q0 + (2 * seg.m + x) * p.tile_tokens;
#pragma unroll
        for (int d = 0; d < D / 64; ++d)
          mma::tma_load_3d_hint(base + x * SH::kQTile + d * (kRowsTile * 128), tmq, 64 * d,
                                seg.h * p.group, tok, &c.q_full[x], keep);
      }
    }
    stop = __shfl_sync(0xffffffffu, stop, 0);
    if (swaps_in(seg)) ++swaps;
    if (!tiles || stop) continue;
    const long long start = p.at.block_table ? 0 : (long long)__ldg(p.at.kv_start + seg.b);
    Sight<WIN> sight;
    sight.init(p, seg);
    int win_lo = 0, win_hi = 0;
    for (int j = seg.tb; j < seg.te; ++j, ++n) {
      const int t0 = sight.key(seg, j);
      const int valid = sight.valid(seg, j);
      const bool fix = sight.fix(seg, j);
      const int nbox = (valid + box_rows - 1) / box_rows;
      if (p.at.block_table) {
        const int lo = t0 >> p.at.page_shift, hi = ((t0 + valid - 1) >> p.at.page_shift) + 1;
        if (lo < win_lo || hi > win_hi) {
          const int last = ((seg.end - 1) >> p.at.page_shift) + 1;
          win_lo = lo;
          win_hi = min(lo + kPages, last);
          __syncwarp();
          for (int k = lane; k < win_hi - win_lo; k += 32)
            c.pages[k] = win_lo + k < p.at.bt_stride
                             ? __ldg(p.at.block_table + (long long)seg.b * p.at.bt_stride + win_lo + k)
                             : -1;
          __syncwarp();
        }
      }
      // one box per lane (at most 16): its row, and whether it lies in the cache
      // (one that no row sees is not loaded: its page may be gone)
      long long row = 0;
      bool ok = true, loads = lane < nbox;
      if (lane < nbox) {
        const int t = t0 + lane * box_rows;
        const int nval = min(box_rows, valid - lane * box_rows);
        if (sight.hidden(t, nval)) {
          loads = false;
        } else if (p.at.block_table) {
          const int page = c.pages[(t >> p.at.page_shift) - win_lo];
          row = ((long long)page << p.at.page_shift) + (t & (p.at.page_size - 1));
          ok = page >= 0 && row + nval <= p.at.kv_rows;
          if (!ok) raise_error(p.at.ws, kErrBounds, page);
        } else {
          row = start + t;
          ok = row >= 0 && row + nval <= p.at.kv_rows;
          if (!ok) raise_error(p.at.ws, kErrBounds, row < 0 ? row : row + nval - 1);
        }
      }
      const bool bad = __any_sync(0xffffffffu, !ok);
      const int boxes = WIN ? __popc(__ballot_sync(0xffffffffu, loads)) : nbox;
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        const int e = 2 * n + kv, slot = e % NS;
        if (!wait_warp(c, p, &empty[slot], (uint32_t)(((e / NS) & 1) ^ 1), 2)) {
          stop = true;
          break;
        }
        issued = e + 1;
        uint8_t* dst = ring + (size_t)slot * kSlot;
        if (bad) {
          // a row outside the cache: the tile counts as absent (all scores
          // excluded), its operands only have to be finite
          for (uint32_t o = lane * 16; o < kSlot; o += 512)
            *reinterpret_cast<uint4*>(dst + o) = make_uint4(0, 0, 0, 0);
          fence_async_smem();
          if (lane == 0 && kv == 0) c.info[n & 7] = tile_info(seg, j, fix, true);
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[slot]);
          continue;
        }
        if (lane == 0) {
          if (kv == 0) c.info[n & 7] = tile_info(seg, j, fix, false);
          mbar_arrive_tx(&full[slot], (uint32_t)boxes * box_rows * TC::kRowBytes * TC::kBlocks);
        }
        __syncwarp();
        if (loads) {
#pragma unroll
          for (int d = 0; d < TC::kBlocks; ++d)
            mma::tma_load_3d_hint(dst + d * (kTile * TC::kRowBytes) +
                                      (size_t)lane * box_rows * TC::kRowBytes,
                                  kv ? tmv : tmk, d * TC::kBoxElems, seg.h, (int)row, &full[slot],
                                  keep);
        }
      }
      if (stop) break;
    }
    stop = __any_sync(0xffffffffu, stop);
  }
  if (lane == 0) land_copies(c, p, full, NS, issued, qn[0], qn[1]);
  __syncwarp();
  if (!stop && KV == 0 && !CONV) {   // (with converters they write the end)
    const int e = 2 * n, slot = e % NS;
    if (wait_warp(c, p, &empty[slot], (uint32_t)(((e / NS) & 1) ^ 1), 2) && lane == 0) {
      c.info[n & 7] = kInfoStop;
      mbar_arrive(&full[slot]);
    }
  }
  __syncwarp();
}

// ---------------------------------------------------------------------------
// MMA warp
// ---------------------------------------------------------------------------
// The whole warp walks the tiles, so that the operands' descriptors stay in
// uniform registers; one elected lane issues.  For tile n, in this order:
//   P V of A, S of A for tile n + 1, P V of B, S of B for tile n + 1,
// so the softmax of one query tile has the other's two products to run in.
// In a solo segment (rows in A only) A and B take the tiles in turns:
//   P V of A for tile n, S of A for n + 2, P V of B for n + 1, S of B for n + 3.
// Products of one thread run in issue order, so S may overwrite the P that
// the P V before it reads.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(e));
  return e;
}

template <int D, int KV, bool CONV, bool BF16>
struct Mma {
  using SH = Shape<D, KV, CONV>;
  static constexpr int NS = SH::kSlots;
  const Prefill& p;
  Control& c;
  uint32_t tbase, base, lead;   // lead: this lane issues
  uint32_t qph[2], pph[2];      // phases of Q and of P
  int fixes;                    // repaired V tiles so far

  // S of X with Q tile `qt` and the K tile in `slot`.
  template <int X>
  __device__ __forceinline__ void scores(int slot, int qt) const {
    constexpr uint32_t id = idesc_f16(kRowsTile, kTile, 0, BF16 ? 1 : 0);
    const uint64_t a = sdesc(base + (uint32_t)qt * SH::kQTile, 0, 1024);
    const uint64_t b = sdesc(base + SH::kOffSlot + (uint32_t)slot * SH::kSlot, 0, 1024);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      const uint32_t off = ((ks >> 2) * (128 * 128) + (ks & 3) * 32) >> 4;
      umma_lead(lead, tbase + X * kTile, a + off, b + off, id, ks > 0);
    }
    commit(&c.s_full[X]);
  }

  // P V of X with the V tile in `slot`: the first half of the keys as soon as
  // their P is there, then the others.
  template <int X>
  __device__ __forceinline__ bool values(int slot, int accumulate) {
    constexpr uint32_t id = idesc_f16(kRowsTile, D, 1, BF16 ? 1 : 0);
    const uint64_t b = sdesc(base + SH::kOffSlot + (uint32_t)slot * SH::kSlot, kTile * 128u, 1024);
    constexpr int kHalf = kTile / 32;
    if (!wait_warp(c, p, &c.p_half[X], pph[X], 7)) return false;
    tc_fence_after();
#pragma unroll
    for (int ks = 0; ks < kHalf; ++ks)
      umma_ts_lead(lead, tbase + (2 + X) * kTile, tbase + X * kTile + ks * 8,
                   b + ((ks * 2048) >> 4), id, ks > 0 ? 1 : accumulate);
    if (!wait_warp(c, p, &c.p_full[X], pph[X], 7)) return false;
    pph[X] ^= 1;
    tc_fence_after();
#pragma unroll
    for (int ks = kHalf; ks < 2 * kHalf; ++ks)
      umma_ts_lead(lead, tbase + (2 + X) * kTile, tbase + X * kTile + ks * 8,
                   b + ((ks * 2048) >> 4), id, 1);
    return true;
  }

  __device__ __forceinline__ void commit(uint64_t* bar) const {
    umma_commit_lead(lead, bar);
  }

  static __device__ __forceinline__ int slot_of(int e) { return e % NS; }

  __device__ __forceinline__ bool key_there(int n) {   // without waiting
    return __all_sync(0xffffffffu, mbar_test(&c.full[slot_of(2 * n)], (uint32_t)((2 * n / NS) & 1)));
  }
  __device__ __forceinline__ bool wait_key(int n) {
    return wait_warp(c, p, &c.full[slot_of(2 * n)], (uint32_t)((2 * n / NS) & 1), 7);
  }
  // V of tile n with info w
  __device__ __forceinline__ bool wait_value(int n, int w) {
    if (!CONV && (w & kInfoFix)) {
      const int f = fixes++;
      return wait_warp(c, p, &c.fixed[f & 3], (uint32_t)((f >> 2) & 1), 7);
    }
    const int e = 2 * n + 1;
    return wait_warp(c, p, &c.full[slot_of(e)], (uint32_t)((e / NS) & 1), 7);
  }
  // A tile's info, which every lane reads from shared memory, in a uniform
  // register; valid once its K tile is there.
  __device__ __forceinline__ int info_of(int n) const {
    return (int)__reduce_or_sync(0xffffffffu, (unsigned)*(volatile int*)&c.info[n & 7]);
  }
  __device__ __forceinline__ bool wait_q(int x) {
    const bool ok = wait_warp(c, p, &c.q_full[x], qph[x], 7);
    qph[x] ^= 1;
    tc_fence_after();
    return ok;
  }

  // A segment whose first tile n has info w; n and w become those of the next
  // segment's first tile (or the end's).  False after a timeout.
  __device__ __forceinline__ bool dual(int& n, int& w) {
    int slot = slot_of(2 * n);
    if (w & kInfoA) {
      if (!wait_q(0)) return false;
      scores<0>(slot, 0);
      if (w & kInfoLastA) commit(&c.q_empty[0]);
    }
    if (w & kInfoB) {
      if (!wait_q(1)) return false;
      scores<1>(slot, 1);
      if (w & kInfoLastB) commit(&c.q_empty[1]);
    }
    commit(&c.empty[slot]);
    int acc = 0;
    for (;;) {
      const int vs = slot_of(2 * n + 1);
      if (!wait_value(n, w)) return false;
      // the next tile, if it is there already (else after P V of A)
      const bool known = key_there(n + 1);
      int next = known ? info_of(n + 1) : 0;
      if (w & kInfoA) {
        if (!values<0>(vs, acc)) return false;
        if (w & kInfoLastA) commit(&c.o_full[0]);
      }
      if (!known) {
        if (!wait_key(n + 1)) return false;
        next = info_of(n + 1);
      }
      const bool follows = !(next & (kInfoStart | kInfoStop));
      slot = slot_of(2 * n + 2);
      if (follows && (next & kInfoA)) {
        tc_fence_after();
        scores<0>(slot, 0);
        if (next & kInfoLastA) commit(&c.q_empty[0]);
      }
      if (w & kInfoB) {
        if (!values<1>(vs, acc)) return false;
        if (w & kInfoLastB) commit(&c.o_full[1]);
      }
      commit(&c.empty[vs]);
      ++n;
      w = next;
      if (!follows) return true;
      if (next & kInfoB) {
        tc_fence_after();
        scores<1>(slot, 1);
        if (next & kInfoLastB) commit(&c.q_empty[1]);
      }
      commit(&c.empty[slot]);
      acc = 1;
    }
  }

  // S of X for tile n (info w) of a solo segment.
  template <int X>
  __device__ __forceinline__ void solo_scores(int n, int w) {
    tc_fence_after();
    scores<X>(slot_of(2 * n), 0);
    commit(&c.empty[slot_of(2 * n)]);
    if (w & kInfoEnd) commit(&c.q_empty[0]);
  }

  // P V of X for tile n (info w) of a solo segment.
  template <int X>
  __device__ __forceinline__ bool solo_values(int n, int w, int acc) {
    const int vs = slot_of(2 * n + 1);
    if (!wait_value(n, w) || !values<X>(vs, acc)) return false;
    commit(&c.empty[vs]);
    if (w & (X ? kInfoLastB : kInfoLastA)) commit(&c.o_full[X]);
    return true;
  }

  // The same for a solo segment.
  __device__ __forceinline__ bool solo(int& n, int& w) {
    if (!wait_q(0)) return false;
    solo_scores<0>(n, w);
    int na = n++, wa = w, nb = 0, wb = 0;   // tiles whose P V is due
    bool a_due = true, b_due = false, more = !(w & kInfoEnd);
    int acc = 0;
    if (more) {
      if (!wait_key(n)) return false;
      w = info_of(n);
      solo_scores<1>(n, w);
      nb = n++;
      wb = w;
      b_due = true;
      more = !(w & kInfoEnd);
    }
    while (a_due || b_due) {
      if (a_due) {
        if (!solo_values<0>(na, wa, acc)) return false;
        a_due = more;
        if (more) {
          if (!wait_key(n)) return false;
          wa = info_of(n);
          solo_scores<0>(n, wa);
          na = n++;
          more = !(wa & kInfoEnd);
        }
      }
      if (b_due) {
        if (!solo_values<1>(nb, wb, acc)) return false;
        b_due = more;
        if (more) {
          if (!wait_key(n)) return false;
          wb = info_of(n);
          solo_scores<1>(n, wb);
          nb = n++;
          more = !(wb & kInfoEnd);
        }
      }
      acc = 1;
    }
    if (!wait_key(n)) return false;
    w = info_of(n);
    return true;
  }

  __device__ __forceinline__ void run() {
    int n = 0;
    bool ok = wait_key(0);
    int w = ok ? info_of(0) : kInfoStop;
    while (ok && !(w & kInfoStop)) ok = w & kInfoSolo ? solo(n, w) : dual(n, w);
    // every issued product is done before the tensor memory is freed
    commit(&c.fin);
    if (!wait_drain(&c.fin) && lead) raise_error(p.at.ws, kErrDrain, 10);
  }

  static __device__ __forceinline__ bool wait_drain(uint64_t* bar) {
    return __all_sync(0xffffffffu, mbar_wait(bar, 0, mma::kDrainNs));
  }
};

// ---------------------------------------------------------------------------
// Repair of V tiles in the ring (16-bit caches by TMA)
// ---------------------------------------------------------------------------
template <int D, bool BF16, bool WIN>
__device__ __forceinline__ void fixers(const Prefill& p, Walk<false, WIN> walk, Control& c,
                                       uint8_t* base) {
  using SH = Shape<D, 0, false>;
  constexpr int NS = SH::kSlots;
  const int lane = threadIdx.x & 31, ft = threadIdx.x - kFixWarp0 * 32;
  Seg seg;
  int n = 0, fixes = 0, sn = 0;
  // (sn counts the segments that have tiles)
  for (; walk.next(p, seg); sn += seg.te > seg.tb) {
    Sight<WIN> sight;
    sight.init(p, seg);
    for (int j = seg.tb; j < seg.te; ++j, ++n) {
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        const int e = 2 * n + kv, slot = e % NS;
        if (!wait_warp(c, p, &c.full[slot], (uint32_t)((e / NS) & 1), 20)) return;
        if (kv == 1 && sight.fix(seg, j)) {
          const int k0 = sight.key(seg, j), valid = sight.valid(seg, j);
          // rows from here on are not seen by all; with a window also those of a
          // first range [lo, hi), which is passed in front of them
          const int from = max(0, min(kTile, sight.unseen - k0));
          int lo = 0, early = 0;
          if constexpr (WIN) {
            lo = max(0, sight.sinks - k0);
            early = max(0, min(from, sight.any - k0) - lo);
          }
          uint8_t* v = base + SH::kOffSlot + (size_t)slot * SH::kSlot;
          bool found = false;
          const int items = (early + kTile - from) * 8;
#pragma unroll
          for (int d = 0; d < D / 64; ++d) {
#pragma unroll 2
            for (int i = ft; i < items; i += 64) {
              int r = from + (i >> 3);
              if constexpr (WIN) r = (i >> 3) < early ? lo + (i >> 3) : r - early;
              uint4* at = reinterpret_cast<uint4*>(v + d * (kTile * 128) + r * 128 + (i & 7) * 16);
              if (r >= valid || sight.hidden(k0 + r)) {
                *at = make_uint4(0, 0, 0, 0);
              } else {
                uint4 w = *at;
                bool hit = drop_nonfinite<BF16>(w.x);
                hit |= drop_nonfinite<BF16>(w.y);
                hit |= drop_nonfinite<BF16>(w.z);
                hit |= drop_nonfinite<BF16>(w.w);
                if (hit) {
                  *at = w;
                  found = true;
                }
              }
            }
          }
          if (found) *(volatile int*)&c.nf[sn & 7] = sn + 1;
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&c.fixed[fixes & 3]);
          ++fixes;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.empty[slot]);
      }
    }
  }
}

// Four 8-bit codes (low byte first) as two registers of 16-bit pairs, exact.
// int8 as bf16: with m the low seven bits, 128 + m is 0x43 above m, and code =
// (128 + m) - (128 or, with the sign bit set, 256), which is 0x43 above 0x00
// or 0x80: the sign bit itself.
template <int KVT, bool BF16>
__device__ __forceinline__ uint2 widen(uint32_t w) {
  if constexpr (KVT == FD_I8 && BF16) {
    const uint32_t m = w & 0x7F7F7F7Fu, s = w & 0x80808080u;
    uint32_t r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t a = __byte_perm(m, 0x43u, i ? 0x4342 : 0x4140);
      const uint32_t b = __byte_perm(s, 0x43u, i ? 0x4342 : 0x4140);
      const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                       *reinterpret_cast<const __nv_bfloat162*>(&b));
      r[i] = *reinterpret_cast<const uint32_t*>(&d);
    }
    return make_uint2(r[0], r[1]);
  } else {
    return mma::widen8x4<KVT, BF16>(w);
  }
}

// ---------------------------------------------------------------------------
// Converter warps: thread = key of the tile
// ---------------------------------------------------------------------------
template <int D, int KV, bool BF16, bool TOK, bool WIN>
__device__ __forceinline__ void converters(const Prefill& p, Walk<TOK, WIN> walk, Control& c,
                                           uint8_t* base) {
  using SH = Shape<D, KV, true>;
  constexpr int NS = SH::kSlots;
  constexpr int NR = SH::kRawSlots > 0 ? SH::kRawSlots : 1;
  constexpr int kChunks = KV == 0 ? D / 8 : D / 16;   // 16-byte chunks of a cache row
  const int lane = threadIdx.x & 31, t = threadIdx.x - kConvWarp0 * 32;
  const uint32_t ring = smem_u32(base) + SH::kOffSlot, raw = smem_u32(base) + SH::kOffRaw;
  Seg seg;
  int n = 0, sn = 0;
  for (; walk.next(p, seg); sn += seg.te > seg.tb) {
    Sight<WIN> sight;
    sight.init(p, seg);
    for (int j = seg.tb; j < seg.te; ++j, ++n) {
      const int k0 = sight.key(seg, j), valid = sight.valid(seg, j);
      const bool fix = sight.fix(seg, j);
      long long row = -1;
      int bad = 0;
      if (p.gather) {
        // a row outside the cache: the tile counts as absent; every warp looks
        // at all 128 rows and so comes to the same answer
        bool wrong = false;
        for (int k = lane; k < valid; k += 32)
          wrong |= !sight.hidden(k0 + k) && placed_row(p.at, seg.b, k0 + k) < 0;
        bad = __any_sync(0xffffffffu, wrong) ? 1 : 0;
        if (t < valid && !sight.hidden(k0 + t)) row = placed_row(p.at, seg.b, k0 + t);
        if (t == 0) c.info[n & 7] = tile_info(seg, j, fix, bad != 0);
      }
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        const int e = 2 * n + kv, slot = e % NS, rs = e % NR;
        const uint32_t dst = ring + (uint32_t)slot * SH::kSlot;
        uint4 w[kChunks];
        if (p.gather) {
          const uint8_t* src = static_cast<const uint8_t*>(kv ? p.v : p.k) +
                               (row * p.num_kv_heads + seg.h) * (long long)(kChunks * 16);
#pragma unroll
          for (int i = 0; i < kChunks; ++i)
            w[i] = row >= 0 && !bad ? __ldg(reinterpret_cast<const uint4*>(src) + i)
                                    : make_uint4(0, 0, 0, 0);
        } else if constexpr (KV != 0) {
          if (!wait_warp(c, p, &c.raw_full[rs], (uint32_t)((e / NR) & 1), 21)) return;
          const uint32_t src = raw + (uint32_t)rs * SH::kRaw + (uint32_t)t * D;
#pragma unroll
          for (int i = 0; i < kChunks; ++i) {
            const int swz = D == 128 ? i ^ (t & 7) : i ^ ((t >> 1) & 3);
            w[i] = lds128(src + (uint32_t)swz * 16);
          }
        }
        // V rows that some query row does not see (see the file comment)
        if (kv == 1 && fix && (sight.partly(k0 + t) || (WIN && t >= valid))) {
          bool found = false;
#pragma unroll
          for (int i = 0; i < kChunks; ++i) {
            if (t >= valid || sight.hidden(k0 + t)) {
              w[i] = make_uint4(0, 0, 0, 0);
            } else if constexpr (KV == 0) {
              found |= drop_nonfinite<BF16>(w[i].x);
              found |= drop_nonfinite<BF16>(w[i].y);
              found |= drop_nonfinite<BF16>(w[i].z);
              found |= drop_nonfinite<BF16>(w[i].w);
            } else if constexpr (KV == 1) {
              found |= drop_nan_e4m3(w[i].x);
              found |= drop_nan_e4m3(w[i].y);
              found |= drop_nan_e4m3(w[i].z);
              found |= drop_nan_e4m3(w[i].w);
            }
          }
          if (found) *(volatile int*)&c.nf[sn & 7] = sn + 1;
        }
        if (!wait_warp(c, p, &c.empty[slot], (uint32_t)(((e / NS) & 1) ^ 1), 22)) return;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          if constexpr (KV == 0) {
            sts128(dst + kmajor_chunk(kTile, t, i), w[i]);
          } else {
            constexpr int KVT = KV == 1 ? FD_E4M3 : FD_I8;
            const uint2 a = widen<KVT, BF16>(w[i].x), b = widen<KVT, BF16>(w[i].y);
            const uint2 d = widen<KVT, BF16>(w[i].z), f = widen<KVT, BF16>(w[i].w);
            sts128(dst + kmajor_chunk(kTile, t, 2 * i), make_uint4(a.x, a.y, b.x, b.y));
            sts128(dst + kmajor_chunk(kTile, t, 2 * i + 1), make_uint4(d.x, d.y, f.x, f.y));
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (!p.gather && KV != 0) mbar_arrive(&c.raw_empty[rs]);
          mbar_arrive(&c.full[slot]);
        }
      }
    }
  }
  const int e = 2 * n, slot = e % NS;   // the end
  if (!wait_warp(c, p, &c.empty[slot], (uint32_t)(((e / NS) & 1) ^ 1), 22)) return;
  if (t == 0) c.info[n & 7] = kInfoStop;
  __syncwarp();
  if (lane == 0) mbar_arrive(&c.full[slot]);
}

// Does tile j of a segment hold a row outside the cache (that some row sees)?
// By one thread; off every fast path.
template <bool WIN>
static __device__ __noinline__ bool tile_absent(const Prefill& p, const Seg& s,
                                                const Sight<WIN>& sight, int j) {
  const int k0 = sight.key(s, j), end = k0 + sight.valid(s, j);
  for (int k = k0; k < end; ++k)
    if (!sight.hidden(k) && placed_row(p.at, s.b, k) < 0) return true;
  return false;
}

// ---------------------------------------------------------------------------
// Per-token scales: warps 10 and 11, keys t and t + 64 of the tile per thread
// ---------------------------------------------------------------------------
// Values are loaded one tile ahead, their block-table entries two.  Loaded by
// the converters, between their other loads, they cost each tile a memory
// latency: single tokens over INT8, 2.56 us a tile in place of 1.9 (the time
// without scales per token), full tiles 0.2 more.  Widening is not a work for
// these two warps: with six warps at it the products wait for shared memory's
// port (e4m3 under f16 at three quarters of the rate).
template <int D, int KV, bool WIN>
__device__ __forceinline__ void token_scales(const Prefill& p, Walk<true, WIN> walk, Control& c,
                                             float* scales) {
  using SH = Shape<D, KV, true>;
  using SR = ScaleRing<D, KV>;
  constexpr int NS = SH::kSlots;
  static_assert(NS % 2 == 0, "K tiles lie in the even slots");
  const int lane = threadIdx.x & 31, t = threadIdx.x - kFixWarp0 * 32;
  // page of key k of the stream, or -1 behind the last key of the segment, and
  // where no row sees the key (its page may be gone)
  auto page_of = [&](const Seg& g, const Sight<WIN>& sight, int j, int k) -> int {
    if (j >= g.te || k >= g.end || sight.hidden(k)) return -1;
    if (!p.at.block_table) return 0;
    const int col = k >> p.at.page_shift;
    return col < p.at.bt_stride
               ? __ldg(p.at.block_table + (long long)g.b * p.at.bt_stride + col)
               : -1;
  };
  Seg seg;
  int n = 0, sn = 0;
  for (; walk.next(p, seg); sn += seg.te > seg.tb) {
    Sight<WIN> sight;
    sight.init(p, seg);
    const long long start = p.at.block_table ? 0 : (long long)__ldg(p.at.kv_start + seg.b);
    float ks[2], vs[2];
    int page[2];
    auto load = [&](int j) {   // of tile j, whose pages are at hand
      const int k0 = sight.key(seg, j), next = WIN ? sight.key(seg, j + 1) : k0 + kTile;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = k0 + t + 64 * i;
        const long long row = p.at.block_table
                                  ? ((long long)page[i] << p.at.page_shift) + (k & (p.at.page_size - 1))
                                  : start + k;
        ks[i] = vs[i] = 0.f;
        if (page[i] >= 0 && row >= 0 && row < p.at.kv_rows) {
          ks[i] = __ldg(p.k_scales + row * p.num_kv_heads + seg.h);
          vs[i] = __ldg(p.v_scales + row * p.num_kv_heads + seg.h);
        }
        page[i] = page_of(seg, sight, j + 1, next + t + 64 * i);
      }
    };
#pragma unroll
    for (int i = 0; i < 2; ++i)
      page[i] = page_of(seg, sight, seg.tb, sight.key(seg, seg.tb) + t + 64 * i);
    if (seg.te > seg.tb) load(seg.tb);
    for (int j = seg.tb; j < seg.te; ++j, ++n) {
      float k[2], v[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        k[i] = ks[i] * p.score_scale;
        v[i] = vs[i];
        // the V scale of a key that some row does not see: as V's elements
        if (!isfinite(v[i])) {
          if (sight.partly(sight.key(seg, j) + t + 64 * i)) {
            v[i] = 0.f;
            *(volatile int*)&c.nf[sn & 7] = sn + 1;
          } else if (tile_absent<WIN>(p, seg, sight, j)) {   // (its P is zero: 0 * NaN would be seen)
            v[i] = 0.f;
          }
        }
      }
      load(j + 1);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const int e = 2 * n + kv, slot = e % NS;
        if (!wait_warp(c, p, &c.empty[slot], (uint32_t)(((e / NS) & 1) ^ 1), 23)) return;
        float* to = scales + (kv ? SR::val(n) : SR::key(n)) + t;
        to[0] = kv ? v[0] : k[0];
        to[64] = kv ? v[1] : k[1];
        __syncwarp();
        if (lane == 0) mbar_arrive(kv ? &c.fixed[n % SR::kValRing] : &c.full[slot]);
      }
    }
  }
  const int e = 2 * n, slot = e % NS;   // the end
  if (!wait_warp(c, p, &c.empty[slot], (uint32_t)(((e / NS) & 1) ^ 1), 23)) return;
  if (lane == 0) mbar_arrive(&c.full[slot]);
}

// ---------------------------------------------------------------------------
// Softmax warps: thread = row of query tile X
// ---------------------------------------------------------------------------
// Elements of V that are not finite, in the keys [lo, hi) of a sequence: added
// to this row's 32 dims from d0 (see the file comment; off every fast path).
// (with a window: those that the row, whose window starts at `first`, sees and
// another row does not)
template <int D, int KV, bool BF16, bool TOK, bool WIN>
__device__ __noinline__ void add_nonfinite(const Prefill& p, const Seg& seg,
                                           const Sight<WIN>& sight, int lo, int hi, int first,
                                           int d0, float* o) {
  float vsc = 1.f;   // (a cut stream's merge brings v_scale)
  if (seg.complete) {
    vsc = p.v_scale;
    if (KV != 0 && p.scale_kind == FD_SCALE_HEAD) vsc *= __ldg(p.v_scales + seg.h);
  }
  for (int t = lo; t < hi; ++t) {
    if (WIN && ((t >= sight.sinks && t < first) || !sight.partly(t))) continue;
    const long long row = placed_row(p.at, seg.b, t);
    if (row < 0) continue;
    const long long at = (row * p.num_kv_heads + seg.h) * D + d0;
    const float scale = TOK ? __ldg(p.v_scales + row * p.num_kv_heads + seg.h) : 1.f;
    for (int i = 0; i < 32; ++i) {
      float x;
      if constexpr (KV == 0) {
        if constexpr (BF16) x = __bfloat162float(static_cast<const __nv_bfloat16*>(p.v)[at + i]);
        else x = __half2float(static_cast<const __half*>(p.v)[at + i]);
      } else if constexpr (KV == 1) {
        __nv_fp8_e4m3 e;
        e.__x = static_cast<const uint8_t*>(p.v)[at + i];
        x = static_cast<float>(e);
      } else {
        x = static_cast<float>(static_cast<const int8_t*>(p.v)[at + i]);
      }
      x *= scale;
      if (!isfinite(x)) o[i] += x * vsc;
    }
  }
}

// 32 bytes in one store (a whole sector) where the address allows it.
__device__ __forceinline__ void store32(void* at, const uint4& a, const uint4& b, bool whole) {
  if (whole)
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(at), "r"(a.x), "r"(a.y),
                 "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  else {
    static_cast<uint4*>(at)[0] = a;
    static_cast<uint4*>(at)[1] = b;
  }
}

template <int D, int KV, bool CONV, bool BF16, bool TOK, bool WIN>
struct Softmax {
  using SH = Shape<D, KV, CONV>;
  using SR = ScaleRing<D, KV>;
  // f16: a factor of P (see the file comment)
  static constexpr float kLift = BF16 ? 0.f : 6.f;
  // exchange of a solo segment: dims per round, and where the states' (m, l) go
  static constexpr int kRound = D / 4;
  static constexpr uint32_t kOffMl = SH::kQTile / 2;

  const Prefill& p;
  Control& c;
  uint8_t* base;
  const float* scales;
  int X, lane, w4, r;
  uint32_t tS, tO;
  // the row's state in the segment
  float m_ref, l, sc;
  int vexp;   // TOK with f16: P's factor carries 2^-vexp against the V scales that
              // the row has seen in the segment

  // P and l carry a factor 2^lift()
  __device__ __forceinline__ float lift() const { return TOK && !BF16 ? kLift - vexp : kLift; }

  __device__ __forceinline__ static void fetch(uint32_t tS, float (&x)[32], int k) {
    tmem_ld32<128>(tS + 32 * k, x);
  }
  // the loads before this have arrived: nothing may read x earlier
  __device__ __forceinline__ static void arrived(float (&x)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+f"(x[i]));
  }
  // scores 32 k .. 32 k + 31 into log2 units by their keys' scales
  __device__ __forceinline__ static void key_scales(float (&x)[32], const float* ks) {
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      uint64_t k01, k23;
      lds_pairs(ks + i, k01, k23);
      const float2 u = unpack2(mul2(pack2(x[i], x[i + 1]), k01));
      const float2 v = unpack2(mul2(pack2(x[i + 2], x[i + 3]), k23));
      x[i] = u.x;
      x[i + 1] = u.y;
      x[i + 2] = v.x;
      x[i + 3] = v.y;
    }
  }
  // off the straight path: the sign of the scale, and -inf for keys that the
  // row does not see (from `left` of the 32 on)
  __device__ __forceinline__ void exclude(float (&x)[32], int left) const {
    if (!TOK && sc <= 0.f) {
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = sc == 0.f ? 0.f : -x[i];
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = i < left ? x[i] : -INFINITY;
  }

  // The same with a window: `seen` has a bit for every key that the row sees.
  __device__ __forceinline__ void exclude_but(float (&x)[32], unsigned seen) const {
    if (!TOK && sc <= 0.f) {
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = sc == 0.f ? 0.f : -x[i];
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = seen & (1u << i) ? x[i] : -INFINITY;
  }
  // bits 0 .. n - 1
  static __device__ __forceinline__ unsigned low_bits(int n) {
    return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
  }
  __device__ __forceinline__ static void row_max(const float (&x)[32], float (&mx)[4]) {
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
#pragma unroll
      for (int k = 0; k < 4; ++k) mx[k] = max3(mx[k], x[i + 2 * k], x[i + 2 * k + 1]);
    }
  }
  // P of scores 32 k .. into 16 columns of tensor memory, over scores that
  // were read before; their sum into `sum`.
  __device__ __forceinline__ void exponents(const float (&x)[32], int k, uint64_t sc2, uint64_t nm2,
                                            const float* vs, uint64_t (&sum)[4]) const {
    uint32_t pk[16];
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      const float2 u = unpack2(fma2(pack2(x[i], x[i + 1]), sc2, nm2));
      const float2 v = unpack2(fma2(pack2(x[i + 2], x[i + 3]), sc2, nm2));
      uint64_t pa = pack2(fast_exp2(u.x), fast_exp2(u.y));
      uint64_t pb = pack2(fast_exp2(v.x), fast_exp2(v.y));
      sum[(i >> 1) & 2] = add2(sum[(i >> 1) & 2], pa);
      sum[((i >> 1) & 2) + 1] = add2(sum[((i >> 1) & 2) + 1], pb);
      if constexpr (TOK) {
        uint64_t va, vb;
        lds_pairs(vs + 32 * k + i, va, vb);
        pa = mul2(pa, va);
        pb = mul2(pb, vb);
      }
      const float2 qa = unpack2(pa), qb = unpack2(pb);
      pk[i / 2] = pack16<BF16>(qa.x, qa.y);
      pk[i / 2 + 1] = pack16<BF16>(qb.x, qb.y);
    }
    tmem_st16u(tS + 16 * k, pk);
  }

  // Largest |V scale| among a tile's first `left` keys, per lane: prefix maxima
  // over four keys a lane, of which each row takes its own.
  static __device__ __forceinline__ float seen_scale(const float* vs, int left) {
    const int lane = threadIdx.x & 31;
    float4 v = reinterpret_cast<const float4*>(vs)[lane];
    v.x = fabsf(v.x);
    v.y = fmaxf(v.x, fabsf(v.y));
    v.z = fmaxf(v.y, fabsf(v.z));
    v.w = fmaxf(v.z, fabsf(v.w));
    float before = v.w;   // of this lane's keys and all earlier ones
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float y = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before = fmaxf(before, y);
    }
    before = __shfl_up_sync(0xffffffffu, before, 1);
    if (lane == 0) before = 0.f;
    const int last = max(left - 1, 0), src = last >> 2;
    const float b = __shfl_sync(0xffffffffu, before, src);
    const float x = __shfl_sync(0xffffffffu, v.x, src), y = __shfl_sync(0xffffffffu, v.y, src);
    const float z = __shfl_sync(0xffffffffu, v.z, src), w = __shfl_sync(0xffffffffu, v.w, src);
    const int i = last & 3;
    return left > 0 ? fmaxf(b, i == 0 ? x : i == 1 ? y : i == 2 ? z : w) : 0.f;
  }

  // The same with keys [hl, hh) hidden, key by key (the window's edge tiles).
  static __device__ __noinline__ float seen_scale(const float* vs, int left, int hl, int hh) {
    float m = 0.f;
    for (int i = 0; i < kTile; ++i)
      if (i < left && !(i >= hl && i < hh)) m = fmaxf(m, fabsf(vs[i]));
    return m;
  }

  // P is in tensor memory up to here: one of this warp's two arrivals a tile.
  __device__ __forceinline__ void publish(uint64_t* bar) const {
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  }

  // One tile (tile jn of the CTA), of whose 128 keys the row sees the first
  // `left`, less [hl, hh) with a window.  False after a timeout.  The scores are read from tensor memory
  // twice, 32 at a time: a thread that kept all 128 would spill.
  __device__ __forceinline__ bool tile(int jn, int left, int hl, int hh, bool mine) {
    const bool whole = __all_sync(0xffffffffu, left == kTile && !(WIN && hl < min(hh, kTile)));
    const float* ks = scales + SR::key(jn);   // written before the tile's S was issued
    const float* vs = scales + SR::val(jn);
    // |sc| is factored out of the scores (a negative scale: the maximum of -s
    // is sought; zero: all scores alike, as 0 * -inf would not be)
    const float scl = TOK || sc == 0.f ? 1.f : fabsf(sc);
    // Other tiles than those whose keys every row of the warp sees (or with
    // the scale's sign turned) are put right in tensor memory first, so that
    // one stretch of code, kept in the instruction cache, serves all.  Scores
    // with per-token scales always go back scaled, and are read once more.
    const bool fast = whole && (TOK || sc > 0.f);
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if (TOK || !fast) {
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        float x[32];
        // with a window, most of an edge tile's blocks of 32 keys are seen or
        // hidden by all rows of the warp, which lie few tokens apart
        unsigned seen = 0;
        if constexpr (WIN) {
          seen = low_bits(left - 32 * k) & (low_bits(hl - 32 * k) | ~low_bits(hh - 32 * k));
          if (!TOK && sc > 0.f && __all_sync(0xffffffffu, seen == 0xffffffffu)) continue;
          if (__all_sync(0xffffffffu, seen == 0u)) {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = -INFINITY;
            tmem_st32<128>(tS + 32 * k, x);
            continue;
          }
        }
        fetch(tS, x, k);
        tmem_wait_ld();
        arrived(x);
        if constexpr (TOK) key_scales(x, ks + 32 * k);
        if constexpr (WIN) {
          if (!TOK || !whole) exclude_but(x, seen);
        } else {
          if (!TOK || !whole) exclude(x, left - 32 * k);
        }
        tmem_st32<128>(tS + 32 * k, x);
        if constexpr (TOK) row_max(x, mx);
      }
      tmem_wait_st();
    }
    if constexpr (!TOK) {
      float x[2][32];
      fetch(tS, x[0], 0);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        tmem_wait_ld();
        arrived(x[k & 1]);
        if (k < 3) fetch(tS, x[(k + 1) & 1], k + 1);
        row_max(x[k & 1], mx);
      }
    }
    const float smax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
    const float mt = smax == -INFINITY ? -INFINITY : smax * scl;
    float fac = 1.f;
    bool resc = false;
    const bool fresh = m_ref == -INFINITY;   // nothing has reached the row's O yet
    if (mt > m_ref + 8.f || fresh) {
      if (!fresh) {
        fac = exp2f(m_ref - mt);
        l *= fac;
        resc = mine;
      }
      m_ref = mt;
    }
    if constexpr (TOK) {
      if (!wait_warp(c, p, &c.fixed[jn % SR::kValRing], (uint32_t)((jn / SR::kValRing) & 1), 12))
        return false;
      if constexpr (!BF16) {
        // largest V scale that the row sees in the tile -> its exponent, which
        // P's factor takes back, so that P times a V scale stays below 2^15
        float vm = 0.f;
        if (whole) {
#pragma unroll
          for (int i = 0; i < 4; ++i) vm = fmaxf(vm, fabsf(vs[lane + 32 * i]));
#pragma unroll
          for (int o = 16; o; o >>= 1) vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, o));
        } else if (WIN) {
          vm = seen_scale(vs, left, hl, hh);
        } else {
          vm = seen_scale(vs, left);
        }
        int ev = (int)((__float_as_uint(vm) >> 23) & 255u) - 127;
        ev = max(-60, min(60, ev));
        if (fresh) {
          vexp = ev;
        } else if (ev > vexp) {
          const float f = exp2f((float)(vexp - ev));
          fac *= f;
          l *= f;
          resc = true;
          vexp = ev;
        }
      }
    }
    if (__any_sync(0xffffffffu, resc)) {
      // the S commit that the caller waited for follows the last P V
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        float o[32];
        tmem_ld32<128>(tO + c0, o);
        tmem_wait_ld();
        arrived(o);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] *= fac;
        tmem_st32<128>(tO + c0, o);
      }
      tmem_wait_st();
    }
    // P = 2^(s - m_ref + kLift); excluded scores are -inf and give 0 (a row
    // that has seen no key has m_ref = -inf: everything is excluded)
    const float nm = m_ref == -INFINITY ? 0.f : lift() - m_ref;
    const uint64_t sc2 = pack2(scl, scl), nm2 = pack2(nm, nm);
    uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
    float x[2][32];
    fetch(tS, x[0], 0);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      tmem_wait_ld();
      arrived(x[k & 1]);
      if (k < 3) fetch(tS, x[(k + 1) & 1], k + 1);
      exponents(x[k & 1], k, sc2, nm2, vs, sum);
      if (k == 1) publish(&c.p_half[X]);
    }
    publish(&c.p_full[X]);
    const float2 sa = unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
    l += sa.x + sa.y;
    return true;
  }

  // Solo segments: A merges B's state (m, l, O) into its own, in rounds of
  // kRound dims through query tile B's place.  `o` takes A's dims as they are
  // read from tensor memory.
  __device__ __forceinline__ float4* swap_at(int d4) const {
    return reinterpret_cast<float4*>(base + SH::kQTile) + d4 * kRowsTile + r;
  }

  __device__ void run(Walk<TOK, WIN> walk) {
    const int rtok = r / p.group, rhead = r - rtok * p.group;
    Seg seg;
    int n = 0, done = 0, segs = 0, sn = 0;
    uint32_t xph = 0;   // phase of the exchange barriers
    // streams of the two partial slots, for the merge
    int4 used0 = make_int4(-1, 0, 0, 0), used1 = used0;
    bool dead = false;
    // with a window, whose segments are short, the next one is walked to while
    // the last product of the present one runs
    Seg ahead;
    bool more = WIN && walk.next(p, ahead);
    for (; !dead && (WIN ? more : walk.next(p, seg)); sn += seg.te > seg.tb) {
      if constexpr (WIN) seg = ahead;
      const int qt = seg.solo ? 0 : X;                     // query tile of this half
      const int tok0 = (2 * seg.m + qt) * p.tile_tokens;   // its first token
      const int live_rows = min(p.tile_tokens, max(0, seg.n - tok0)) * p.group;
      const bool mine = r < live_rows;
      const bool warp_live = 32 * w4 < live_rows;
      // keys this row sees; a row of nobody never restricts its warp
      const int lim = mine ? max(0, seg.ctx + tok0 + rtok + 1) : 0x7fffffff;
      // first key of its window (in 64 bits: a window may be longer than any cache)
      const int wfirst =
          WIN && mine ? (int)max(0ll, (long long)seg.ctx + tok0 + rtok - p.window + 1) : 0;
      Sight<WIN> sight;
      sight.init(p, seg);
      const int te = min(seg.te, qt ? seg.nt[1] : seg.nt[0]);
      const int first = seg.tb + (seg.solo ? X : 0), step = seg.solo ? 2 : 1;
      float vsc = p.v_scale;
      sc = p.score_scale;
      if (KV != 0 && p.scale_kind == FD_SCALE_HEAD) {
        sc *= __ldg(p.k_scales + seg.h);
        vsc *= __ldg(p.v_scales + seg.h);
      }
      m_ref = -INFINITY;
      l = 0.f;
      vexp = 0;
      for (int j = first; j < te; j += step, ++done) {
        const int jn = n + (j - seg.tb);   // tile of the CTA
        if (!wait_warp(c, p, &c.s_full[X], (uint32_t)(done & 1), 11)) {
          dead = true;
          break;
        }
        tc_fence_after();
        if (warp_live) {
          const bool bad = (*(volatile int*)&c.info[jn & 7] & kInfoBad) != 0;
          const int k0 = sight.key(seg, j);
          const int left = WIN ? min(sight.valid(seg, j), lim - k0) : min(kTile, lim - k0);
          if (!tile(jn, bad ? 0 : max(0, left), WIN ? max(0, p.sinks - k0) : 0, wfirst - k0,
                    mine)) {
            dead = true;
            break;
          }
        } else {   // no row of this warp: P may be anything
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&c.p_half[X]);
            mbar_arrive(&c.p_full[X]);
          }
        }
      }
      if (dead) break;
      n += seg.te - seg.tb;
      // ---------------------------------------------------------- segment end
      if constexpr (WIN) more = walk.next(p, ahead);
      const bool any = first < te;   // O of this half was accumulated
      if (any) {
        if (!wait_warp(c, p, &c.o_full[X], (uint32_t)(segs & 1), 15)) {
          dead = true;
          break;
        }
        ++segs;
        tc_fence_after();
      }
      if (!seg.complete) {
        if (seg.slot & 1) used1 = make_int4(seg.b, seg.h, seg.m, 0);
        else used0 = make_int4(seg.b, seg.h, seg.m, 0);
      }
      float m_out = m_ref == -INFINITY ? -INFINITY : m_ref - lift();
      float osc = 1.f;   // of this half's O
      const bool swap = swaps_in(seg);
      float bsc = 0.f;   // of the other half's O (A of a solo segment)
      if (swap) {
        float2* ml = reinterpret_cast<float2*>(base + SH::kQTile + kOffMl) + r;
        if (X == 1) {
          *ml = make_float2(m_out, l);
          for (int q = 0; q < 4 && !dead; ++q) {   // rounds of kRound dims
            if (warp_live) {
#pragma unroll
              for (int d0 = 0; d0 < kRound; d0 += 16) {
                float o[16];
                load16(tO + q * kRound + d0, o);
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                  *swap_at((d0 + i) / 4) =
                      make_float4(o[i] * osc, o[i + 1] * osc, o[i + 2] * osc, o[i + 3] * osc);
              }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&c.x_full);
            dead = !wait_warp(c, p, &c.x_empty, xph, 16);
            xph ^= 1;
          }
          if (dead) break;
          fence_async_smem();   // a later query tile B lands here
          if (w4 == 0 && lane == 0) *(volatile int*)&c.swaps = c.swaps + 1;
        } else {
          if (!wait_warp(c, p, &c.x_full, xph, 17)) {
            dead = true;
            break;
          }
          const float2 b = *ml;
          const float M = fmaxf(m_out, b.x);
          const float fa = m_out == -INFINITY ? 0.f : fast_exp2(m_out - M);
          bsc = b.x == -INFINITY ? 0.f : fast_exp2(b.x - M);
          l = l * fa + b.y * bsc;
          osc *= fa;
          m_out = M;
        }
      }
      const bool writes = !(seg.solo && X == 1);
      if (seg.complete) {
        const float q = l == 0.f ? 0.f : vsc / l;
        osc *= q;
        bsc *= q;
      }
      const bool nonfinite = seg.te > seg.tb && *(volatile int*)&c.nf[sn & 7] == sn + 1;
      if (writes && (warp_live || swap)) {
        const long long out_at = ((long long)(seg.q0 + tok0 + rtok) * p.num_q_heads +
                                  (long long)seg.h * p.group + rhead) * D;
        const bool sectors = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
        const bool plain = WIN && seg.complete && !swap && !nonfinite && any;
        if (plain) {   // the usual end of a short segment: loads ahead of stores
          float o[2][32];
          tmem_ld32<128>(tO, o[0]);
          const uint64_t q2 = pack2(osc, osc);
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            tmem_wait_ld();
            arrived(o[k & 1]);
            if (k + 1 < D / 32) tmem_ld32<128>(tO + 32 * (k + 1), o[(k + 1) & 1]);
            uint32_t v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 x = unpack2(mul2(pack2(o[k & 1][2 * i], o[k & 1][2 * i + 1]), q2));
              v[i] = pack16<BF16>(x.x, x.y);
            }
            if (mine) {
              uint16_t* to = static_cast<uint16_t*>(p.out) + out_at + 32 * k;
              store32(to, make_uint4(v[0], v[1], v[2], v[3]), make_uint4(v[4], v[5], v[6], v[7]),
                      sectors);
              store32(to + 16, make_uint4(v[8], v[9], v[10], v[11]),
                      make_uint4(v[12], v[13], v[14], v[15]), sectors);
            }
            __syncwarp();
          }
        }
#pragma unroll(D == 64 ? 2 : 1)
        for (int c0 = plain ? D : 0; c0 < D; c0 += 32) {
          float o[32];
          if (any && warp_live) {
            tmem_ld32<128>(tO + c0, o);
            tmem_wait_ld();
            arrived(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= osc;
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0.f;
          }
          if (swap) {   // 32 dims are one round, or two of 16
#pragma unroll
            for (int q = 0; q < 32 / kRound; ++q) {
              const int round = c0 / kRound + q;
              if (round > 0) dead = dead || !wait_warp(c, p, &c.x_full, xph, 17);
              xph ^= 1;
              if (warp_live && bsc != 0.f) {
#pragma unroll
                for (int i = 0; i < kRound; i += 4) {
                  const float4 y = *swap_at(i / 4);
                  const int k = q * kRound + i;
                  o[k] = fmaf(y.x, bsc, o[k]);
                  o[k + 1] = fmaf(y.y, bsc, o[k + 1]);
                  o[k + 2] = fmaf(y.z, bsc, o[k + 2]);
                  o[k + 3] = fmaf(y.w, bsc, o[k + 3]);
                }
              }
              fence_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&c.x_empty);
            }
          }
          if (!warp_live) continue;
          if ((KV != 2 || TOK) && nonfinite && mine) {
            float x[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = o[i];
            // tile by tile: an absent one has no elements
            const int lo = WIN ? 0 : sight.unseen;
#pragma unroll 1
            for (int j = max(seg.tb, lo / kTile); j < seg.te; ++j) {
              const int k0 = sight.key(seg, j);
              if (k0 >= lim || !sight.fix(seg, j) || tile_absent<WIN>(p, seg, sight, j)) continue;
              add_nonfinite<D, KV, BF16, TOK, WIN>(
                  p, seg, sight, max(lo, k0),
                  min(lim, k0 + (WIN ? sight.valid(seg, j) : kTile)), wfirst, c0, x);
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = x[i];
          }
          if (!mine) continue;
          if (seg.complete) {
            uint4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              v[i] = make_uint4(pack16<BF16>(o[8 * i], o[8 * i + 1]),
                                pack16<BF16>(o[8 * i + 2], o[8 * i + 3]),
                                pack16<BF16>(o[8 * i + 4], o[8 * i + 5]),
                                pack16<BF16>(o[8 * i + 6], o[8 * i + 7]));
            uint16_t* at = static_cast<uint16_t*>(p.out) + out_at + c0;
            store32(at, v[0], v[1], sectors);
            store32(at + 16, v[2], v[3], sectors);
          } else {
            // partial states: [slot][query tile][dim / 4][row][4]
            float4* pa = reinterpret_cast<float4*>(p.part_acc) +
                         ((long long)(2 * seg.slot + qt) * (D / 4) + c0 / 4) * kRowsTile + r;
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              pa[(i / 4) * kRowsTile] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
        }
        if (mine) {
          if (!seg.complete) {
            p.part_ml[(long long)(2 * seg.slot + qt) * kRowsTile + r] = make_float2(m_out, l);
          } else if (p.lse) {
            p.lse[out_at / D] = l == 0.f ? -INFINITY : (m_out + log2f(l)) * kLn2;
          }
        }
      }
      tc_fence_before();
    }
    if (X == 0 && r == 0) {
      // after a timeout nothing is merged: the outputs are undefined
      if (dead) used0.x = used1.x = -1;
      p.meta[2 * blockIdx.x] = used0;
      p.meta[2 * blockIdx.x + 1] = used1;
    }
  }

  __device__ __forceinline__ static void load16(uint32_t taddr, float (&v)[16]) {
    uint32_t w[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]),
          "=r"(w[7]), "=r"(w[8]), "=r"(w[9]), "=r"(w[10]), "=r"(w[11]), "=r"(w[12]), "=r"(w[13]),
          "=r"(w[14]), "=r"(w[15])
        : "r"(taddr));
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      v[i] = __uint_as_float(w[i]);
      asm volatile("" : "+f"(v[i]));
    }
  }
};

// ---------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------
template <int D, int KV, bool CONV, bool BF16, bool TOK, bool WIN>
__global__ void __launch_bounds__(Shape<D, KV, CONV>::kThreads, 1)
    prefill_kernel(const __grid_constant__ Prefill p, const __grid_constant__ CUtensorMap tmq,
                   const __grid_constant__ CUtensorMap tmk,
                   const __grid_constant__ CUtensorMap tmv) {
  using SH = Shape<D, KV, CONV>;
  extern __shared__ __align__(1024) uint8_t base[];
  Control& c = *reinterpret_cast<Control*>(base + SH::kOffCtl);
  float* scales = reinterpret_cast<float*>(base + SH::kOffCtl + kCtlBytes);
  const int warp = threadIdx.x >> 5;
  if (smem_u32(base) & 1023u) {   // the swizzled operands need whole atoms
    if (threadIdx.x == 0) {
      raise_error(p.at.ws, kErrPlan, 0);
      p.meta[2 * blockIdx.x].x = p.meta[2 * blockIdx.x + 1].x = -1;
    }
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < SH::kSlots; ++i) {
      // the producer, or the converter warps and, with K tiles, the scale warps
      mbar_init(&c.full[i], !CONV ? 1 : TOK && i % 2 == 0 ? 6 : 4);
      mbar_init(&c.empty[i], CONV ? 1 : 3);       // the last product (and the two repair warps)
    }
    for (int i = 0; i < kMaxRaw; ++i) {
      mbar_init(&c.raw_full[i], 1);
      mbar_init(&c.raw_empty[i], 4);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&c.fixed[i], 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.q_full[i], 1);
      mbar_init(&c.q_empty[i], 1);
      mbar_init(&c.s_full[i], 1);
      mbar_init(&c.p_half[i], 4);
      mbar_init(&c.p_full[i], 4);
      mbar_init(&c.o_full[i], 1);
    }
    mbar_init(&c.fin, 1);
    mbar_init(&c.x_full, 4);
    mbar_init(&c.x_empty, 4);
    for (int i = 0; i < 8; ++i) c.info[i] = c.nf[i] = 0;
    c.abort_flag = 0;
    c.swaps = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&c.tmem_base)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == kProducerWarp * 32) {
    mma::prefetch_map(&tmq);
    if (!p.gather) {
      mma::prefetch_map(&tmk);
      mma::prefetch_map(&tmv);
    }
  }
  tc_fence_before();
  const Plan plan = make_plan<TOK, WIN>(p, reinterpret_cast<long long*>(base));   // (barriers)
  tc_fence_after();
  Walk<TOK, WIN> walk;   // every role walks its own copy
  walk.init(p, plan);
  const uint32_t tbase = c.tmem_base;
  allow_dependent_launch();

  if (warp < 8) {
    const int X = warp >> 2, w4 = warp & 3, lane = threadIdx.x & 31;
    const uint32_t tl = tbase + ((uint32_t)(32 * w4) << 16);
    Softmax<D, KV, CONV, BF16, TOK, WIN> sm{p, c, base, scales, X, lane, w4, 32 * w4 + lane,
                                       tl + X * kTile, tl + (2 + X) * kTile};
    sm.run(walk);
  } else if (warp < kConvWarp0) {
    if (warp == kProducerWarp) {
      producer<D, KV, CONV, TOK, WIN>(p, walk, c, base, &tmq, &tmk, &tmv);
    } else if (warp == kMmaWarp) {
      Mma<D, KV, CONV, BF16> mm{p, c, tbase, smem_u32(base), elect_one(), {0, 0}, {0, 0}, 0};
      mm.run();
    } else if constexpr (!CONV) {
      fixers<D, BF16, WIN>(p, walk, c, base);
    } else if constexpr (TOK) {
      token_scales<D, KV, WIN>(p, walk, c, scales);
    }
  } else if constexpr (CONV) {
    converters<D, KV, BF16, TOK, WIN>(p, walk, c, base);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(512)
                 : "memory");
  }
}

template <int D, int KV, bool CONV, bool BF16, bool TOK, bool WIN>
cudaError_t launch_one(const Prefill& p, const CUtensorMap* maps, cudaStream_t stream) {
  constexpr uint32_t smem = smem_bytes<D, KV, CONV, TOK>();
  static std::atomic<unsigned long long> limit_set{0};
  const auto kern = prefill_kernel<D, KV, CONV, BF16, TOK, WIN>;
  const cudaError_t e = ensure_smem_limit(kern, (int)smem, &limit_set);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)p.grid, Shape<D, KV, CONV>::kThreads, smem, stream>>>(p, maps[0], maps[1],
                                                                        maps[2]);
  return cudaGetLastError();
}

// 16-bit caches: by TMA, or gathered row by row.
template <int D, bool BF16, bool WIN>
cudaError_t launch_16(const Prefill& p, const CUtensorMap* maps, cudaStream_t stream) {
  return p.gather ? launch_one<D, 0, true, BF16, false, WIN>(p, maps, stream)
                  : launch_one<D, 0, false, BF16, false, WIN>(p, maps, stream);
}

// 8-bit caches: with per-token scales or not.
template <int KV, bool BF16, bool WIN>
cudaError_t launch_8(const Prefill& p, const CUtensorMap* maps, cudaStream_t stream) {
  const bool tok = p.scale_kind == FD_SCALE_TOKEN;
  if (p.head_dim == 128)
    return tok ? launch_one<128, KV, true, BF16, true, WIN>(p, maps, stream)
               : launch_one<128, KV, true, BF16, false, WIN>(p, maps, stream);
  return tok ? launch_one<64, KV, true, BF16, true, WIN>(p, maps, stream)
             : launch_one<64, KV, true, BF16, false, WIN>(p, maps, stream);
}

// One per translation unit; WIN: with a window.
template <bool WIN>
cudaError_t launch_16bit(const Prefill& p, const CUtensorMap* maps, cudaStream_t stream) {
  if (p.q_dtype == FD_BF16)
    return p.head_dim == 128 ? launch_16<128, true, WIN>(p, maps, stream)
                             : launch_16<64, true, WIN>(p, maps, stream);
  return p.head_dim == 128 ? launch_16<128, false, WIN>(p, maps, stream)
                           : launch_16<64, false, WIN>(p, maps, stream);
}

using Launch = cudaError_t(const Prefill& p, const CUtensorMap* maps, cudaStream_t stream);
Launch launch_plain_16bit, launch_plain_e4m3_f16, launch_plain_e4m3_bf16, launch_plain_i8_f16,
    launch_plain_i8_bf16;
Launch launch_window_16bit, launch_window_e4m3_f16, launch_window_e4m3_bf16, launch_window_i8_f16,
    launch_window_i8_bf16;

}  // namespace pf
}  // namespace fd
