// pages.cu — page bookkeeping of the paged cache: forking, freeing, trimming
// and growing slots, compaction, page copies (include/pi_serve.h).
//
// References are counted anew from the tables in each call, so no count can
// drift: a page is live while a used table entry or a holder names it.  Both
// calls are the same few passes:
//
//   clear   references = held
//   count   references += one per used table entry (integer atomics: the sum
//           does not depend on their order)
//   rank    per 1024 pages, how many are free (live); the last block to
//           arrive turns these into positions and settles what concerns the
//           slots
//   place   every page of a block knows its rank now: fresh pages go to their
//           slots, or movers and holes to their pairs
//   copy    page contents in all layers
//
// Bound: for small pools launches and memory latency, so one block runs all
// passes but the copy with the pool's counts in its shared memory; for large
// ones the chain of dependent reads and the tables; with real pages the copy,
// at HBM bandwidth (each byte once in, once out).
//
// Measured: a fork of 4 slots 7 us, of 1024 slots of 12000 tokens 20 us (8 of
// them the 768 K atomics of the count); a compaction of 64 slots with 16
// layers 207 us, the copy in it 189, 93 % of a copy's 6.8 TB/s.
#include "serve.cuh"

namespace pis {

struct PageArgs {
  const int *parent, *grow, *held, *table_in, *len_in;
  int *table, *len, *ref, *map, *pairs, *counts, *status;
  int *arrived, *blocks, *owner, *rank, *first, *before, *src, *sums;
  int slots, max_pages, pages, page_tokens;
};

constexpr int kPageThreads = 256;
constexpr int kNobody = 0x7fffffff;
enum { kSumNeed, kSumLive, kSumLow };  // places in `sums`

// A pool and tables this small are left to one block of 1024 threads, with
// both counts of every page in shared memory.
constexpr int kSmallPages = 8192, kSmallEntries = 16384;
inline bool is_small(const PageArgs& a) {
  return a.pages <= kSmallPages && (long long)a.slots * a.max_pages <= kSmallEntries;
}

// What becomes of slot s (pi_cache_fork): the parent's row, the tokens kept,
// the tokens wanted.
struct Fate {
  int parent, keep, want;
};

__device__ __forceinline__ Fate fate_of(const PageArgs& a, int s) {
  Fate f{a.parent[s], 0, 0};
  const int grow = a.grow[s];
  const long long most = (long long)a.max_pages * a.page_tokens;
  long long base = 0;
  if (f.parent >= a.slots || f.parent < -1) {
    set_status(a.status, PI_ERR_INDEX);
    f.parent = -1;
  }
  if (f.parent >= 0) {
    base = a.len_in[f.parent];
    if (base < 0 || base > most) {
      set_status(a.status, PI_ERR_INDEX);
      f.parent = -1;
      base = 0;
    }
  }
  long long want = base + grow;
  want = want < 0 ? 0 : want;
  if (want > most) {
    set_status(a.status, PI_ERR_CAPACITY);
    want = most;
  }
  f.want = (int)want;
  f.keep = (int)(base < want ? base : want);
  return f;
}

__device__ __forceinline__ int used_pages(const PageArgs& a, int s) {
  const int n = a.len_in[s];
  if (n < 0 || n > a.max_pages * a.page_tokens) {
    set_status(a.status, PI_ERR_INDEX);
    return 0;
  }
  return pages_of(n, a.page_tokens);
}

// Sum over the block, and the sum of the threads before this one.  T threads.
template <int T, typename V>
__device__ __forceinline__ V block_scan(V v, V* total) {
  __shared__ V sh[T / 32 + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  V upto = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V w = __shfl_up_sync(~0u, upto, o);
    if (lane >= o) upto += w;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = upto;
  __syncthreads();
  if (warp == 0) {
    V w = lane < T / 32 ? sh[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const V x = __shfl_up_sync(~0u, w, o);
      if (lane >= o) w += x;
    }
    __syncwarp();
    if (lane < T / 32) sh[lane] = w;
  }
  __syncthreads();
  *total = sh[T / 32 - 1];
  return upto - v + (warp ? sh[warp - 1] : 0);
}

// ------------------------------------------------------------------ passes
// Work items [first, end) in steps of `step`.  FORK: else compaction.
template <bool FORK>
__device__ __forceinline__ void clear_pass(const PageArgs& a, int first, int step) {
  for (int p = first; p < a.pages; p += step) {
    (FORK ? a.ref : a.owner)[p] = a.held ? a.held[p] : 0;
    if (FORK) a.owner[p] = kNobody;
  }
}

// Entries [first, end) of slot s, four at a time where rows are aligned to
// that.  Fork: full pages are shared, the lowest slot bids for each partly
// filled one, and the slot's full pages, partly filled page and wanted length
// are noted.  A row may end at 2^31 - 1: loops count from `first`.
template <bool FORK>
__device__ __forceinline__ void count_pass(const PageArgs& a, int s, int first, int end) {
  if (FORK) {
    const Fate f = fate_of(a, s);
    const int whole = f.keep / a.page_tokens;
    const int* src = a.table_in + (size_t)max(f.parent, 0) * a.max_pages;
    int* dst = a.table + (size_t)s * a.max_pages;
    if (first == 0 && threadIdx.x == 0) {
      int p = -1;
      if (f.keep % a.page_tokens) p = checked_page(src[whole], a.pages, a.status);
      if (p >= 0) atomicMin(a.owner + p, s);
      a.first[s] = whole;
      a.src[s] = p;
      a.before[s] = f.want;
    }
    auto take = [&](int j, int p) {
      if (j >= whole) return -1;
      p = checked_page(p, a.pages, a.status);
      if (p >= 0) atomicAdd(a.ref + p, 1);
      return p;
    };
    if ((a.max_pages & 3) == 0) {
      for (int i = 4 * threadIdx.x; i < end - first; i += 4 * kPageThreads) {
        const int j = first + i;
        int4 p = make_int4(-1, -1, -1, -1);
        if (j < whole) p = __ldg(reinterpret_cast<const int4*>(src + j));
        p = make_int4(take(j, p.x), take(j + 1, p.y), take(j + 2, p.z), take(j + 3, p.w));
        *reinterpret_cast<int4*>(dst + j) = p;
      }
    } else {
      for (int i = threadIdx.x; i < end - first; i += kPageThreads) {
        const int j = first + i;
        dst[j] = take(j, j < whole ? __ldg(src + j) : -1);
      }
    }
  } else {
    const int used = used_pages(a, s);
    const int* src = a.table_in + (size_t)s * a.max_pages;
    for (int i = threadIdx.x; i < min(end, used) - first; i += kPageThreads) {
      const int p = checked_page(src[first + i], a.pages, a.status);
      if (p >= 0) atomicAdd(a.owner + p, 1);
    }
  }
}

// Whether page p counts: free pages in a fork, live ones in a compaction.
// rank_pass settles a fork's partly filled pages: one that nobody shares in
// full stays with its lowest slot.
template <bool FORK, bool SETTLE>
__device__ __forceinline__ bool counts(const PageArgs& a, int p) {
  if (!FORK) return __ldcg(a.owner + p) > 0;
  const int ref = __ldcg(a.ref + p);
  if (!SETTLE) return ref == 0;
  const int owner = __ldcg(a.owner + p);
  if (owner == kNobody) return ref == 0;
  if (ref > 0)
    a.owner[p] = kNobody;
  else
    a.ref[p] = 1;
  return false;
}

// Positions of the 1024-page blocks, and of the slots; by one thread block.
template <bool FORK, int T>
__device__ void settle(const PageArgs& a, int nb) {
  int sum = 0;
  for (int b0 = 0; b0 < nb; b0 += T) {
    const int b = b0 + threadIdx.x;
    const int v = b < nb ? __ldcg(a.blocks + b) : 0;
    int total;
    const int at = block_scan<T>(v, &total);
    if (b < nb) a.blocks[b] = sum + at;
    sum += total;
  }
  if (!FORK) {
    // live pages below c = sum: those of the blocks before c's, and of its own
    __syncthreads();
    int n = 0;
    const int b = sum / kScanPages;
    for (int p = b * kScanPages + (int)threadIdx.x; p < sum; p += T) n += __ldcg(a.owner + p) > 0;
    int low;
    block_scan<T>(n, &low);
    if (threadIdx.x == 0) {
      low = b < nb ? low + a.blocks[b] : sum;
      a.sums[kSumLive] = sum;
      a.sums[kSumLow] = low;
      a.counts[0] = sum - low;
      a.counts[1] = sum;
    }
    return;
  }
  // slots <= T
  const int s = threadIdx.x;
  int first = 0, need = 0, from = -1, want = 0;
  if (s < a.slots) {
    first = __ldcg(a.first + s);
    want = __ldcg(a.before + s);
    from = __ldcg(a.src + s);
    if (from >= 0 && __ldcg(a.owner + from) == s) {
      a.table[(size_t)s * a.max_pages + first++] = from;
      from = -1;
    }
    need = max(0, pages_of(want, a.page_tokens) - first);
  }
  // 1024 slots may want more pages than 2^31; `sum` of them at most are there
  long long need_sum;
  int pair_sum;
  const int before = (int)min(block_scan<T>((long long)need, &need_sum), (long long)sum);
  const int got = min(need, sum - before);
  const bool copied = from >= 0 && got > 0;
  const int pair = block_scan<T>((int)copied, &pair_sum);
  if (s < a.slots) {
    a.first[s] = first;
    a.before[s] = before;
    a.src[s] = copied ? pair : -1;
    if (copied) a.pairs[2 * pair] = from;
    a.len[s] = got < need ? min(want, (first + got) * a.page_tokens) : want;
  }
  if (threadIdx.x == 0) {
    const int taken = (int)min(need_sum, (long long)sum);
    a.sums[kSumNeed] = taken;
    a.counts[0] = pair_sum;
    a.counts[1] = a.pages - sum + taken;
    if (need_sum > sum) set_status(a.status, PI_ERR_CAPACITY);
  }
}

// The last slot whose fresh pages begin at or before the at-th.
__device__ __forceinline__ int slot_of(const int* before, int slots, int at) {
  int lo = 0, hi = slots - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (before[mid] <= at) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Compaction: the new numbers, references and tables.
__device__ __forceinline__ int moved_to(const PageArgs& a, int p, int live) {
  if (__ldcg(a.owner + p) <= 0) return -1;
  return p < live ? p : __ldcg(a.pairs + 2 * __ldcg(a.rank + p) + 1);
}
__device__ __forceinline__ void map_pass(const PageArgs& a, long long first, long long step) {
  const int live = __ldcg(a.sums + kSumLive);
  for (long long p = first; p < a.pages; p += step) {
    const int to = moved_to(a, (int)p, live);
    a.map[p] = to;
    if (to >= 0) a.ref[to] = __ldcg(a.owner + p);
    if (p >= live) a.ref[p] = 0;
  }
  const long long entries = (long long)a.slots * a.max_pages;
  for (long long e = first; e < entries; e += step) {
    const int s = (int)quotient(e, a.max_pages), j = (int)(e - (long long)s * a.max_pages);
    const int n = a.len_in[s];
    int p = -1;
    if (n > 0 && n <= a.max_pages * a.page_tokens && j < pages_of(n, a.page_tokens)) p = a.table_in[e];
    a.table[e] = (unsigned)p < (unsigned)a.pages ? moved_to(a, p, live) : -1;
  }
}

// ------------------------------------------------------------------ kernels
template <bool FORK>
__global__ void __launch_bounds__(kPageThreads) clear_kernel(const PageArgs a) {
  pdl_enter();
  clear_pass<FORK>(a, blockIdx.x * kPageThreads + threadIdx.x, gridDim.x * kPageThreads);
}

constexpr int kCountEntries = 1024;  // table entries of one block

template <bool FORK>
__global__ void __launch_bounds__(kPageThreads) count_kernel(const PageArgs a) {
  pdl_enter();
  for (long long at = (long long)blockIdx.y * kCountEntries; at < a.max_pages;
       at += (long long)gridDim.y * kCountEntries)
    count_pass<FORK>(a, blockIdx.x, (int)at, (int)min((long long)a.max_pages, at + kCountEntries));
}

// A thread per page.
template <bool FORK>
__global__ void __launch_bounds__(kScanPages) rank_kernel(const PageArgs a) {
  pdl_enter();
  __shared__ int last;
  const int p = blockIdx.x * kScanPages + threadIdx.x;
  const int n = __syncthreads_count(p < a.pages && counts<FORK, true>(a, p));
  if (threadIdx.x == 0) a.blocks[blockIdx.x] = n;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(a.arrived, 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  if (threadIdx.x == 0) *a.arrived = 0;
  settle<FORK, kScanPages>(a, gridDim.x);
}

template <bool FORK>
__global__ void __launch_bounds__(kScanPages) place_kernel(const PageArgs a) {
  pdl_enter();
  __shared__ int before[PI_CACHE_MAX_SLOTS];
  int at = __ldcg(a.blocks + blockIdx.x);
  const int need = __ldcg(a.sums + kSumNeed), live = __ldcg(a.sums + kSumLive);
  const int low = __ldcg(a.sums + kSumLow);
  if (FORK && at >= need) return;
  if (FORK && (int)threadIdx.x < a.slots) before[threadIdx.x] = __ldcg(a.before + threadIdx.x);
  const int p = blockIdx.x * kScanPages + threadIdx.x;
  const bool in = p < a.pages && counts<FORK, false>(a, p);
  int total;
  at += block_scan<kScanPages>((int)in, &total);
  if (FORK) {
    if (!in || at >= need) return;
    const int s = slot_of(before, a.slots, at), j = at - before[s];
    a.table[(size_t)s * a.max_pages + __ldcg(a.first + s) + j] = p;
    a.ref[p] = 1;
    const int pair = __ldcg(a.src + s);
    if (j == 0 && pair >= 0) a.pairs[2 * pair + 1] = p;
  } else if (p < a.pages) {
    if (in && p >= live) {
      a.rank[p] = at - low;
      a.pairs[2 * (at - low)] = p;
    } else if (!in && p < live) {
      a.pairs[2 * (p - at) + 1] = p;
    }
  }
}

// All passes but the copy in one block, for small pools.  Thread t ranks the
// pages [t k, t k + k).
template <bool FORK>
__global__ void __launch_bounds__(1024) small_kernel(const PageArgs a) {
  constexpr int T = 1024;
  extern __shared__ int sh[];
  int* ref = sh;              // [pages]
  int* owner = sh + a.pages;  // [pages]: fork: the lowest bidder; else the new number
  __shared__ int sh_from[T], sh_whole[T], sh_before[T], sh_pair[T];
  __shared__ int sh_low;
  pdl_enter();
  const int tid = threadIdx.x;
  const int entries = a.slots * a.max_pages;
  // what becomes of the slots; the pages' references
  int last = -1, want = 0;
  if (tid < a.slots) {
    if (FORK) {
      const Fate f = fate_of(a, tid);
      sh_whole[tid] = f.keep / a.page_tokens;
      sh_from[tid] = f.parent;
      want = f.want;
      if (f.keep % a.page_tokens)
        last = checked_page(a.table_in[(size_t)f.parent * a.max_pages + f.keep / a.page_tokens],
                            a.pages, a.status);
    } else {
      sh_whole[tid] = used_pages(a, tid);
      sh_from[tid] = tid;
    }
  }
  for (int p = tid; p < a.pages; p += T) {
    ref[p] = a.held ? a.held[p] : 0;
    owner[p] = kNobody;
  }
  __syncthreads();
#pragma unroll 4
  for (int e = tid; e < entries; e += T) {
    const int s = e / a.max_pages, j = e - s * a.max_pages;
    int p = -1;
    if (j < sh_whole[s])
      p = checked_page(a.table_in[(size_t)sh_from[s] * a.max_pages + j], a.pages, a.status);
    if (p >= 0) atomicAdd(ref + p, 1);
    if (FORK) a.table[e] = p;
  }
  if (last >= 0) atomicMin(owner + last, tid);
  __syncthreads();
  // ranks
  const int k = (a.pages + T - 1) / T, p0 = min(a.pages, tid * k), p1 = min(a.pages, p0 + k);
  int n = 0;
  for (int p = p0; p < p1; ++p) {
    if (FORK) {
      if (ref[p] > 0) owner[p] = kNobody;
      else if (owner[p] != kNobody) ref[p] = 1;
    }
    n += FORK ? ref[p] == 0 : ref[p] > 0;
  }
  int sum;
  int at = block_scan<T>(n, &sum);
  if (FORK) {
    int first = 0, need = 0;
    if (tid < a.slots) {
      first = sh_whole[tid];
      if (last >= 0 && owner[last] == tid) {
        a.table[(size_t)tid * a.max_pages + first++] = last;
        last = -1;
      }
      need = max(0, pages_of(want, a.page_tokens) - first);
    }
    int need_sum, pair_sum;
    const int before = block_scan<T>(need, &need_sum);
    const int got = max(0, min(need, sum - before));
    const bool copied = last >= 0 && got > 0;
    const int pair = block_scan<T>((int)copied, &pair_sum);
    if (tid < a.slots) {
      sh_whole[tid] = first;
      sh_before[tid] = before;
      sh_pair[tid] = copied ? pair : -1;
      if (copied) a.pairs[2 * pair] = last;
      a.len[tid] = got < need ? min(want, (first + got) * a.page_tokens) : want;
    }
    need_sum = min(need_sum, sum);
    if (tid == 0) {
      a.counts[0] = pair_sum;
      a.counts[1] = a.pages - sum + need_sum;
    }
    if (got < need) set_status(a.status, PI_ERR_CAPACITY);
    __syncthreads();
    for (int p = p0; p < p1; ++p) {
      if (ref[p]) continue;
      if (at < need_sum) {
        const int s = slot_of(sh_before, a.slots, at), j = at - sh_before[s];
        a.table[(size_t)s * a.max_pages + sh_whole[s] + j] = p;
        ref[p] = 1;
        if (j == 0 && sh_pair[s] >= 0) a.pairs[2 * sh_pair[s] + 1] = p;
      }
      ++at;
    }
    __syncthreads();
    for (int p = tid; p < a.pages; p += T) a.ref[p] = ref[p];
  } else {
    // `sum` pages are live; `low` of them are below that number
    if (p0 <= sum && (sum < p1 || tid == T - 1)) {
      int low = at;
      for (int p = p0; p < min(p1, sum); ++p) low += ref[p] > 0;
      if (sum < p1 || p1 == a.pages) sh_low = low;
    }
    __syncthreads();
    const int low = sh_low;
    if (tid == 0) {
      a.counts[0] = sum - low;
      a.counts[1] = sum;
    }
    for (int p = p0; p < p1; ++p) {
      if (ref[p] > 0) {
        if (p >= sum) a.pairs[2 * (at - low)] = p;
        owner[p] = p < sum ? p : at - low;  // a mover's place among them
        ++at;
      } else if (p < sum) {
        a.pairs[2 * (p - at) + 1] = p;
      }
    }
    __syncthreads();
    for (int p = tid; p < a.pages; p += T) {
      int to = -1;
      if (ref[p] > 0) {
        to = p < sum ? p : a.pairs[2 * owner[p] + 1];
        owner[p] = to;
        a.ref[to] = ref[p];
      }
      a.map[p] = to;
      if (p >= sum) a.ref[p] = 0;
    }
    __syncthreads();
    for (int e = tid; e < entries; e += T) {
      const int s = e / a.max_pages, j = e - s * a.max_pages;
      const int p = j < sh_whole[s] ? a.table_in[e] : -1;
      a.table[e] = (unsigned)p < (unsigned)a.pages && ref[p] > 0 ? owner[p] : -1;
    }
  }
}

// Page pairs x layers, a warp moving 2 KB at a time.
struct CopyArgs {
  const int *pairs, *count;
  uint4* pool;
  int* status;
  long long page16;  // 16-byte pieces of a page
  int cap, pages, layers, parts;  // parts of 128 pieces of a page
};

constexpr int kCopyThreads = 256;

__device__ __forceinline__ void copy_pass(const CopyArgs& c) {
  int n = __ldcg(c.count);
  if (n > c.cap) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_status(c.status, PI_ERR_CAPACITY);
    n = c.cap;
  }
  const int lane = threadIdx.x & 31;
  const long long items = (long long)n * c.layers * c.parts;
  const long long step = (long long)gridDim.x * (kCopyThreads / 32);
  for (long long it = blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); it < items; it += step) {
    const long long r = quotient(it, c.parts);
    const int part = (int)(it - r * c.parts);
    const int i = (int)quotient(r, c.layers), layer = (int)(r - (long long)i * c.layers);
    const int2 pr = __ldcg(reinterpret_cast<const int2*>(c.pairs) + i);
    if ((unsigned)pr.x >= (unsigned)c.pages || (unsigned)pr.y >= (unsigned)c.pages) {
      if (lane == 0) set_status(c.status, PI_ERR_INDEX);
      continue;
    }
    const uint4* src = c.pool + ((size_t)layer * c.pages + pr.x) * c.page16;
    uint4* dst = c.pool + ((size_t)layer * c.pages + pr.y) * c.page16;
    const long long e = part * 128ll + lane;
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (e + 32 * k < c.page16) v[k] = __ldcs(src + e + 32 * k);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (e + 32 * k < c.page16) __stcs(dst + e + 32 * k, v[k]);
  }
}

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const CopyArgs c) {
  pdl_enter();
  copy_pass(c);
}

// The last passes of a compaction: both follow from the pairs.
__global__ void __launch_bounds__(kCopyThreads) map_copy_kernel(const PageArgs a, const CopyArgs c) {
  pdl_enter();
  map_pass(a, blockIdx.x * kCopyThreads + threadIdx.x, (long long)gridDim.x * kCopyThreads);
  if (c.pool) copy_pass(c);
}

// ------------------------------------------------------------------ launches
static CopyArgs copy_args(const pi_cache_desc& C, const int* pairs, const int* count, int cap,
                          void* pool, int* status) {
  const long long page16 = (long long)(page_elems(C) / 8);
  return CopyArgs{pairs, count, static_cast<uint4*>(pool), status, page16, cap, C.pages, C.layers,
                  (int)((page16 + 127) / 128)};
}

// Eight blocks per SM, or what `cap` pairs can use.
static unsigned copy_grid(const CopyArgs& c) {
  DevInfo di;
  if (dev_info(&di) != PI_OK) return 0;
  const long long most = ((long long)c.cap * c.layers * c.parts + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
  return (unsigned)(most < di.sms * 8 ? (most > 0 ? most : 1) : di.sms * 8);
}

static pi_status launch_copy(const CopyArgs& c, pi_stream stream) {
  const unsigned grid = copy_grid(c);
  return grid ? launch(copy_kernel, dim3(grid), kCopyThreads, 0, stream, c) : PI_ERR_CUDA;
}

// The passes up to `place` (and a small compaction's map).
template <bool FORK>
static pi_status launch_passes(const PageArgs& a, pi_stream stream) {
  if (is_small(a)) {
    const pi_status st = ensure_smem(reinterpret_cast<const void*>(small_kernel<FORK>), 8 * kSmallPages);
    return st == PI_OK ? launch(small_kernel<FORK>, dim3(1), 1024, 8 * (size_t)a.pages, stream, a) : st;
  }
  const unsigned nb = (unsigned)((a.pages + kScanPages - 1) / kScanPages);
  const unsigned parts = ((unsigned)a.max_pages + kCountEntries - 1) / kCountEntries;
  const dim3 entries((unsigned)a.slots, parts < 65535 ? parts : 65535);
  const unsigned clear = (unsigned)((a.pages + kPageThreads - 1) / kPageThreads);
  pi_status st = launch(clear_kernel<FORK>, dim3(clear < 1216 ? clear : 1216), kPageThreads, 0, stream, a);
  if (st == PI_OK) st = launch(count_kernel<FORK>, entries, kPageThreads, 0, stream, a);
  if (st == PI_OK) st = launch(rank_kernel<FORK>, dim3(nb), kScanPages, 0, stream, a);
  if (st == PI_OK) st = launch(place_kernel<FORK>, dim3(nb), kScanPages, 0, stream, a);
  return st;
}

static void bind(PageArgs& a, const pi_cache_desc& C, int slots, int max_pages, void* ws) {
  const CacheWs w = cache_ws(C, slots, 0);
  char* b = static_cast<char*>(ws);
  auto at = [&](size_t o) { return reinterpret_cast<int*>(b + o); };
  a.arrived = at(w.arrived);
  a.blocks = at(w.blocks);
  a.owner = at(w.owner);
  a.rank = at(w.rank);
  a.first = at(w.first);
  a.before = at(w.before);
  a.src = at(w.src);
  a.sums = at(w.sums);
  a.slots = slots;
  a.max_pages = max_pages;
  a.pages = C.pages;
  a.page_tokens = C.page_tokens;
}

}  // namespace pis

using namespace pis;

extern "C" {

pi_status pi_cache_fork(const pi_cache_desc* cache, int32_t slots, int32_t max_pages,
                        const int32_t* parent, const int32_t* grow, const int32_t* held,
                        const int32_t* table_in, const int32_t* len_in, int32_t* table,
                        int32_t* len, int32_t* ref, void* pool, int32_t* pairs, int32_t* counts,
                        int32_t* dev_status, void* ws, size_t ws_bytes, pi_stream stream) {
  pi_status st = check_cache(cache);
  if (st != PI_OK) return st;
  const pi_cache_desc& C = *cache;
  st = check_slots(C, slots, max_pages);
  if (st != PI_OK) return st;
  if (!parent || !grow || !table_in || !len_in || !table || !len || !ref || !pairs || !counts ||
      !dev_status || !ws)
    return PI_ERR_NULL;
  if (!all_aligned(parent, grow, held, table_in, len_in, table, len, ref, pool, pairs, counts,
                   dev_status, ws))
    return PI_ERR_ALIGN;
  if (table == table_in || len == len_in || ref == held) return PI_ERR_SHAPE;
  if (ws_bytes < cache_ws(C, slots, 0).total) return PI_ERR_WORKSPACE;
  PageArgs a{};
  bind(a, C, slots, max_pages, ws);
  a.parent = parent;
  a.grow = grow;
  a.held = held;
  a.table_in = table_in;
  a.len_in = len_in;
  a.table = table;
  a.len = len;
  a.ref = ref;
  a.pairs = pairs;
  a.counts = counts;
  a.status = dev_status;
  st = launch_passes<true>(a, stream);
  if (st == PI_OK && pool)
    st = launch_copy(copy_args(C, pairs, counts, slots, pool, dev_status), stream);
  return st;
}

pi_status pi_cache_compact(const pi_cache_desc* cache, int32_t slots, int32_t max_pages,
                           const int32_t* held, const int32_t* table_in, const int32_t* len,
                           int32_t* table, int32_t* ref, int32_t* map, void* pool,
                           int32_t* pairs, int32_t* counts, int32_t* dev_status, void* ws,
                           size_t ws_bytes, pi_stream stream) {
  pi_status st = check_cache(cache);
  if (st != PI_OK) return st;
  const pi_cache_desc& C = *cache;
  st = check_slots(C, slots, max_pages);
  if (st != PI_OK) return st;
  if (!table_in || !len || !table || !ref || !map || !pairs || !counts || !dev_status || !ws)
    return PI_ERR_NULL;
  if (!all_aligned(held, table_in, len, table, ref, map, pool, pairs, counts, dev_status, ws))
    return PI_ERR_ALIGN;
  if (ref == held) return PI_ERR_SHAPE;
  if (ws_bytes < cache_ws(C, slots, 0).total) return PI_ERR_WORKSPACE;
  PageArgs a{};
  bind(a, C, slots, max_pages, ws);
  a.held = held;
  a.table_in = table_in;
  a.len_in = len;
  a.table = table;
  a.ref = ref;
  a.map = map;
  a.pairs = pairs;
  a.counts = counts;
  a.status = dev_status;
  st = launch_passes<false>(a, stream);
  if (st != PI_OK) return st;
  const CopyArgs c = copy_args(C, pairs, counts, C.pages / 2, pool, dev_status);
  if (is_small(a)) return pool ? launch_copy(c, stream) : PI_OK;
  const unsigned grid = copy_grid(c);
  return grid ? launch(map_copy_kernel, dim3(grid), kCopyThreads, 0, stream, a, c) : PI_ERR_CUDA;
}

pi_status pi_cache_copy(const pi_cache_desc* cache, const int32_t* pairs, const int32_t* count,
                        int32_t cap, void* pool, int32_t* dev_status, pi_stream stream) {
  pi_status st = check_cache(cache);
  if (st != PI_OK) return st;
  if (cap < 0) return PI_ERR_SHAPE;
  if (!pairs || !count || !pool || !dev_status) return PI_ERR_NULL;
  if (!all_aligned(pairs, count, pool, dev_status)) return PI_ERR_ALIGN;
  return launch_copy(copy_args(*cache, pairs, count, cap, pool, dev_status), stream);
}

}  // extern "C"
