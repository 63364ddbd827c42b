// fd_pages.cu -- pages of a step's requests: block tables, the stack of free
// pages and the packed tokens' cache rows, from the requests' lengths.
//
// Plan.  A sequence of L cached tokens holds ceil(L / P) pages; it gives pages
// back (all when it ends, with a window those that no later token sees) and
// wants ceil((L + n) / P) - ceil(L / P) more for n new tokens.  Three running
// sums over the sequences (tokens, pages back, pages wanted) say where each
// one's tokens begin in the packed arrays, where its pages go on the stack and
// which entries it takes from there; it gets its pages if the sum up to and with
// it does not pass what the stack holds, so the answer does not depend on any
// order of execution and no atomics are needed.
//
// Fill.  Every page that goes back, every page handed out and every slot is
// then one item of its own, found by a search in those sums.  The k-th page
// handed out is entry avail - 1 - k of the stack with all returned pages on it;
// an item that needs one which returns in this call reads it from the table
// entry that it returns from, so that items do not wait for one another: what
// is read (columns that are held, entries below the old count) is never written
// in the same call.
//
// What bounds it: latency.  Small steps run in one block, its sums in shared
// memory (one launch); others in two launches, the plan in one block and the fill
// on all SMs, the second launched as a programmatic dependent.  1024 requests
// with 800000 new tokens (7 MB) take 16.3 us, 5 to 6 of them the plan (19.9 with
// the sums searched in global memory and the kinds of items one after the other).
#include "fd_prompt.cuh"

namespace fd {
namespace {

constexpr int kThreads = 1024;      // of the plan's block
constexpr int kFillThreads = 256;
// One block fills a slot or moves a page about every nanosecond; a second launch
// costs 1.2 to 1.8 us and fills on all SMs.  One token each of 64 sequences:
// 5.2 us in one launch, 6.4 in two; of 1024: 8.0 and 9.7; four each: 12.6 and
// 9.5.  128 ended sequences of 8000 tokens: 60 us and 7.4, so one launch is kept
// for tables that hold few pages to give back.
constexpr int kFusedSlots = 2048, kFusedEntries = 4096;

using Rec = PageRec;
using Totals = PageTotals;

struct Sums {   // of all sequences before b, [batch + 1]; in shared or global memory
  Rec* rec;
  int32_t *back, *handed, *tokens;
};

// The last b with start[b] <= i < start[b + 1] (start[0] = 0, ascending).
__device__ __forceinline__ int owner(const int32_t* start, int batch, long long i) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The same for i = first + lane of a whole warp: one search for the warp's first
// (32 probes at a time), which serves the lanes of the same sequence.
__device__ __forceinline__ int owner_in_warp(const int32_t* start, int batch, long long first) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const unsigned below = __ballot_sync(0xffffffffu, at < hi && start[at] <= first);
    lo += (31 - __clz(below)) * step;   // (start[lo] <= first: never empty)
    hi = min(hi, lo + step);
  }
  return first + lane < start[lo + 1] ? lo : owner(start, batch, first + lane);
}

// Page r of those that go back.
__device__ __forceinline__ int returned(const AssignPages& p, const Sums& s, long long r) {
  const int b = owner(s.back, p.batch, r);
  const Rec& t = s.rec[b];
  const int j = (int)(r - s.back[b]);
  return p.table[(long long)b * p.stride + (j < t.keep ? j : t.lo + j - t.keep)];
}

// Page k of those handed out.
__device__ __forceinline__ int handed(const AssignPages& p, const Sums& s, const Totals& t,
                                      long long k) {
  const long long i = t.avail - 1 - k;
  return i < t.count ? p.free_pages[i] : returned(p, s, i - t.count);
}

// One range of items, so that no thread passes one kind after the other: slots
// (whole warps of them), pages handed out, pages that go back.  (Table and stack
// are read and written by one launch: plain loads.)
__device__ __forceinline__ void fill(const AssignPages& p, const Sums& s, const Totals& t,
                                     long long first, long long step) {
  const long long tokens = s.tokens[p.batch], slots = (p.num_slots + 31) / 32 * 32;
  const long long items = slots + t.handed + t.back;
  for (long long i = first; i - (threadIdx.x & 31) < items; i += step) {
    if (i >= slots) {
      const long long k = i - slots, r = k - t.handed;
      if (k < t.handed) {
        const int b = owner(s.handed, p.batch, k);
        p.table[(long long)b * p.stride + s.rec[b].held + (k - s.handed[b])] = handed(p, s, t, k);
      } else if (r < t.back && t.count + r < p.capacity) {
        p.free_pages[t.count + r] = returned(p, s, r);
      }
      continue;
    }
    long long slot = -1;
    // (lane 0's item is a multiple of 32)
    const long long w = i - (threadIdx.x & 31);
    const int b = w < tokens ? owner_in_warp(s.tokens, p.batch, w) : 0;
    if (i < tokens) {
      const Rec& x = s.rec[b];
      if (x.need >= 0) {
        const int pos = x.L + (int)(i - s.tokens[b]);
        const int col = pos >> p.page_shift;
        const int page = col < x.held ? p.table[(long long)b * p.stride + col]
                                      : handed(p, s, t, (long long)s.handed[b] + col - x.held);
        if (page >= 0)
          slot = ((long long)page << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
      }
    }
    if (i < p.num_slots) p.slots[i] = slot;
  }
}

// Inclusive sums of x over the block's threads; `all` gets the block's.
__device__ __forceinline__ long long block_sum(long long x, long long& all, long long* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();   // (the last sum's readers are done)
  if (lane == 31) red[warp] = x;
  __syncthreads();
  long long w = lane < kThreads / 32 ? red[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  all = __shfl_sync(0xffffffffu, w, 31);
  const long long before = __shfl_sync(0xffffffffu, w, max(0, warp - 1));
  return x + (warp > 0 ? before : 0);
}

struct Look {
  Rec rec;
  int n, back, released;   // new tokens (< 0: it ends), pages back, columns given back after it
  long long total, want;   // tokens and pages wanted
  bool fits;
};

__device__ __forceinline__ Look look_at(const AssignPages& p, int b, bool report) {
  Look x;
  const int L = max(0, p.seq_len[b]);
  const long long round = (1ll << p.page_shift) - 1;
  long long held = (L + round) >> p.page_shift;
  x.fits = held <= p.stride;
  if (!x.fits) {
    if (report) raise_error(p.ws, kErrBounds, held);
    held = p.stride;
  }
  x.rec.L = L;
  x.rec.held = (int)held;
  x.n = p.new_tokens[b];
  x.released = 0;
  if (p.window) {
    const int gone = max(p.keep, p.released[b]);
    x.rec.lo = gone;
    if (x.n < 0) {
      x.rec.keep = min(p.keep, x.rec.held);
      x.back = x.rec.keep + max(0, x.rec.held - gone);
    } else {
      x.rec.keep = 0;
      x.released = max(gone, min(max(0, L - p.window + 1) >> p.page_shift, x.rec.held));
      x.back = x.released - gone;
    }
  } else {
    x.rec.keep = x.back = x.n < 0 ? x.rec.held : 0;
    x.rec.lo = x.rec.held;
  }
  x.total = (long long)L + max(0, x.n);
  const long long pages = (x.total + round) >> p.page_shift;
  if (x.fits && (pages > p.stride || x.total > 0x7fffffffll)) {
    if (report) raise_error(p.ws, kErrBounds, pages);
    x.fits = false;
  }
  if (x.n < 0) x.fits = false;
  x.want = x.fits ? pages - held : 0;
  return x;
}

// The plan, by one block; the sums go to `s`.
__device__ __forceinline__ Totals plan(const AssignPages& p, const Sums& s, long long* red) {
  const int tid = threadIdx.x;
  Totals t;
  t.count = max(0, p.free_count[0]);
  if (t.count > p.capacity) {
    if (tid == 0) raise_error(p.ws, kErrBounds, t.count);
    t.count = p.capacity;
  }
  t.back = 0;
  if (p.batch > kThreads) {   // what returns in all is needed before the first grant
    long long mine = 0;
    for (int b = tid; b < p.batch; b += kThreads) mine += look_at(p, b, false).back;
    block_sum(mine, t.back, red);
  }
  long long tokens = 0, back = 0, wanted = 0, given = 0;   // of the chunks before
  for (int base = 0; base < p.batch; base += kThreads) {
    const int b = base + tid;
    const bool live = b < p.batch;
    Look x = {};
    if (live) x = look_at(p, b, true);
    long long all_tokens, all_back, all_wanted, all_given;
    const long long tok = tokens + block_sum(live ? max(0, x.n) : 0, all_tokens, red);
    const long long bk = back + block_sum(x.back, all_back, red);
    if (p.batch <= kThreads) t.back = all_back;
    t.avail = min(t.count + t.back, p.capacity);
    if (tid == 0 && base == 0 && t.count + t.back > p.capacity)
      raise_error(p.ws, kErrBounds, t.count + t.back);
    // packed tokens behind the slots, or behind what an int32 counts
    if (live && x.n > 0 && (tok > 0x7fffffffll || (p.slots && tok > p.num_slots))) {
      if (x.fits) raise_error(p.ws, kErrBounds, tok);
      x.fits = false;
      x.want = 0;
    }
    const long long upto = wanted + block_sum(x.want, all_wanted, red);
    const bool granted = x.fits && (x.want == 0 || upto <= t.avail);
    const long long need = granted ? x.want : 0;
    const long long gv = given + block_sum(need, all_given, red);
    if (live) {
      x.rec.need = granted ? (int)need : -1;
      s.rec[b] = x.rec;
      s.back[b] = (int)(bk - x.back);
      s.handed[b] = (int)(gv - need);
      const int start = (int)min(tok - max(0, x.n), 0x7fffffffll);
      p.q_start[b] = start;
      if (s.tokens != p.q_start) s.tokens[b] = start;
      p.positions[b] = granted ? x.rec.L : -1;
      p.seq_len_out[b] = x.n < 0 ? 0 : granted ? (int)x.total : x.rec.L;
      if (p.window) p.released_out[b] = x.released;
      // (what goes back with a window is what tokens from L on do not see:
      // sequences without any in this step are not for its attention)
      if (p.attend_len) p.attend_len[b] = granted && x.n > 0 ? (int)x.total : 0;
    }
    tokens += all_tokens;
    back += all_back;
    wanted += all_wanted;
    given += all_given;
  }
  t.handed = given;
  if (tid == 0) {
    const int end = (int)min(tokens, 0x7fffffffll);
    s.back[p.batch] = (int)min(t.back, 0x7fffffffll);
    s.handed[p.batch] = (int)given;
    p.q_start[p.batch] = end;
    if (s.tokens != p.q_start) s.tokens[p.batch] = end;
    p.free_count_out[0] = (int)(t.avail - given);
  }
  return t;
}

// Few slots: everything in one block.
__global__ void __launch_bounds__(kThreads) assign_pages_fused(const __grid_constant__ AssignPages p) {
  __shared__ Rec rec[kThreads];
  __shared__ int32_t back[kThreads + 1], handed_[kThreads + 1], tokens[kThreads + 1];
  __shared__ long long red[32];
  const Sums s{rec, back, handed_, tokens};
  const Totals t = plan(p, s, red);
  __syncthreads();
  fill(p, s, t, threadIdx.x, kThreads);
}

__global__ void __launch_bounds__(kThreads) assign_pages_plan(const __grid_constant__ AssignPages p) {
  __shared__ long long red[32];
  allow_dependent_launch();
  const Totals t = plan(p, Sums{p.rec, p.back, p.handed, p.q_start}, red);
  if (threadIdx.x == 0) *p.totals = t;
}

// LOCAL: at most kThreads sequences, whose sums are searched in shared memory.
template <bool LOCAL>
__global__ void __launch_bounds__(kFillThreads) assign_pages_fill(const __grid_constant__ AssignPages p) {
  __shared__ Rec rec[LOCAL ? kThreads : 1];
  __shared__ int32_t sums[3][LOCAL ? kThreads + 1 : 1];
  wait_prior_grid();
  const Totals t = *p.totals;
  Sums s{p.rec, p.back, p.handed, p.q_start};
  if constexpr (LOCAL) {
    for (int b = threadIdx.x; b <= p.batch; b += kFillThreads) {
      if (b < p.batch) rec[b] = s.rec[b];
      sums[0][b] = s.back[b];
      sums[1][b] = s.handed[b];
      sums[2][b] = s.tokens[b];
    }
    s = Sums{rec, sums[0], sums[1], sums[2]};
    __syncthreads();
  }
  fill(p, s, t, (long long)blockIdx.x * kFillThreads + threadIdx.x,
       (long long)gridDim.x * kFillThreads);
}

struct Layout {
  size_t totals, rec, back, handed, total;
};

Layout layout(int batch) {
  Layout l;
  l.totals = sizeof(WsHeader);
  l.rec = align_up(l.totals + sizeof(Totals), 256);
  l.back = align_up(l.rec + sizeof(Rec) * (size_t)batch, 256);
  l.handed = align_up(l.back + 4 * ((size_t)batch + 1), 256);
  l.total = align_up(l.handed + 4 * ((size_t)batch + 1), 256);
  return l;
}

}  // namespace

size_t assign_pages_bytes(int batch) { return layout(batch).total; }

cudaError_t launch_assign_pages(AssignPages p, int sms, cudaStream_t stream) {
  if (p.batch <= kThreads && p.slots && p.num_slots <= kFusedSlots &&
      (long long)p.batch * p.stride <= kFusedEntries) {
    assign_pages_fused<<<1, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
  }
  const Layout l = layout(p.batch);
  uint8_t* ws = reinterpret_cast<uint8_t*>(p.ws);
  p.totals = reinterpret_cast<Totals*>(ws + l.totals);
  p.rec = reinterpret_cast<Rec*>(ws + l.rec);
  p.back = reinterpret_cast<int32_t*>(ws + l.back);
  p.handed = reinterpret_cast<int32_t*>(ws + l.handed);
  assign_pages_plan<<<1, kThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(4 * sms));
  cfg.blockDim = dim3(kFillThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.batch <= kThreads ? cudaLaunchKernelEx(&cfg, assign_pages_fill<true>, p)
                             : cudaLaunchKernelEx(&cfg, assign_pages_fill<false>, p);
}

}  // namespace fd
