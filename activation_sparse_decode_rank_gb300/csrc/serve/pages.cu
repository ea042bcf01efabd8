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
// Bound: for small tables launches and memory latency, so one block runs all
// passes but the copy; for large ones the reading of the tables; with real
// pages the copy, at HBM bandwidth (each byte once in, once out).
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
enum { kSumNeed, kSumFree, kSumLive, kSumLow };  // places in `sums`

// A table this small is left to one block of 1024 threads: its passes take a
// microsecond or less each, a launch two.
inline bool one_block(const PageArgs& a) {
  return a.pages <= 16384 && (long long)a.slots * a.max_pages <= 16384;
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
template <int T>
__device__ __forceinline__ int block_scan(int v, int* total) {
  __shared__ int sh[T / 32 + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int upto = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int w = __shfl_up_sync(~0u, upto, o);
    if (lane >= o) upto += w;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = upto;
  __syncthreads();
  if (warp == 0) {
    int w = lane < T / 32 ? sh[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(~0u, w, o);
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

// Entries [first, ...) of slot s.  Fork: full pages are shared, and the
// lowest slot bids for each partly filled one.
template <bool FORK>
__device__ __forceinline__ void count_pass(const PageArgs& a, int s, int first, int end, int step) {
  if (FORK) {
    const Fate f = fate_of(a, s);
    const int whole = f.keep / a.page_tokens;
    const int* src = a.table_in + (size_t)max(f.parent, 0) * a.max_pages;
    int* dst = a.table + (size_t)s * a.max_pages;
    for (int j = first; j < end; j += step) {
      int p = -1;
      if (j <= whole && f.keep > 0 && (j < whole || f.keep % a.page_tokens)) {
        p = checked_page(src[j], a.pages, a.status);
        if (p >= 0) {
          if (j < whole) {
            atomicAdd(a.ref + p, 1);
          } else {
            atomicMin(a.owner + p, s);
            p = -1;
          }
        }
      }
      dst[j] = p;
    }
  } else {
    const int used = used_pages(a, s);
    const int* src = a.table_in + (size_t)s * a.max_pages;
    for (int j = first; j < min(end, used); j += step) {
      const int p = checked_page(src[j], a.pages, a.status);
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
      low = b < nb ? low + __ldcg(a.blocks + b) : sum;
      a.sums[kSumLive] = sum;
      a.sums[kSumLow] = low;
      a.counts[0] = sum - low;
      a.counts[1] = sum;
    }
    return;
  }
  int need_sum = 0, pair_sum = 0;
  for (int s0 = 0; s0 < a.slots; s0 += T) {
    const int s = s0 + threadIdx.x;
    int first = 0, need = 0, from = -1, want = 0;
    if (s < a.slots) {
      const Fate f = fate_of(a, s);
      want = f.want;
      first = f.keep / a.page_tokens;
      if (f.keep % a.page_tokens) {
        const int p = a.table_in[(size_t)f.parent * a.max_pages + first];
        if ((unsigned)p < (unsigned)a.pages) {
          if (__ldcg(a.owner + p) == s)
            a.table[(size_t)s * a.max_pages + first++] = p;
          else
            from = p;
        }
      }
      need = max(0, pages_of(want, a.page_tokens) - first);
    }
    int total;
    const int before = need_sum + block_scan<T>(need, &total);
    need_sum += total;
    const int got = max(0, min(need, sum - before));
    const bool copied = from >= 0 && got > 0;
    const int pair = pair_sum + block_scan<T>(copied, &total);
    pair_sum += total;
    if (s < a.slots) {
      a.first[s] = first;
      a.before[s] = before;
      a.src[s] = copied ? pair : -1;
      if (copied) a.pairs[2 * pair] = from;
      a.len[s] = got < need ? min(want, (first + got) * a.page_tokens) : want;
    }
  }
  if (threadIdx.x == 0) {
    a.sums[kSumNeed] = min(need_sum, sum);
    a.counts[0] = pair_sum;
    a.counts[1] = a.pages - sum + min(need_sum, sum);
    if (need_sum > sum) set_status(a.status, PI_ERR_CAPACITY);
  }
}

// Page p, the at-th of those that count, finds its place.
template <bool FORK>
__device__ __forceinline__ void place(const PageArgs& a, int p, int at, bool in) {
  if (FORK) {
    if (!in || at >= __ldcg(a.sums + kSumNeed)) return;
    int lo = 0, hi = a.slots - 1;  // the last slot whose pages begin at or before `at`
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldcg(a.before + mid) <= at) lo = mid;
      else hi = mid - 1;
    }
    const int j = at - __ldcg(a.before + lo);
    a.table[(size_t)lo * a.max_pages + __ldcg(a.first + lo) + j] = p;
    a.ref[p] = 1;
    const int pair = __ldcg(a.src + lo);
    if (j == 0 && pair >= 0) a.pairs[2 * pair + 1] = p;
  } else {
    const int live = __ldcg(a.sums + kSumLive);
    if (in && p >= live) {
      const int r = at - __ldcg(a.sums + kSumLow);
      a.rank[p] = r;
      a.pairs[2 * r] = p;
    } else if (!in && p < live) {
      a.pairs[2 * (p - at) + 1] = p;
    }
  }
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
    count_pass<FORK>(a, blockIdx.x, (int)at + threadIdx.x,
                     (int)min((long long)a.max_pages, at + kCountEntries), kPageThreads);
}

template <bool FORK>
__global__ void __launch_bounds__(kPageThreads) rank_kernel(const PageArgs a) {
  pdl_enter();
  __shared__ int last;
  int n = 0;
  const int p0 = blockIdx.x * kScanPages;
  for (int p = p0 + threadIdx.x; p < min(a.pages, p0 + kScanPages); p += kPageThreads)
    n += counts<FORK, true>(a, p);
  int total;
  block_scan<kPageThreads>(n, &total);
  if (threadIdx.x == 0) {
    a.blocks[blockIdx.x] = total;
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(a.arrived, 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  if (threadIdx.x == 0) *a.arrived = 0;
  settle<FORK, kPageThreads>(a, gridDim.x);
}

template <bool FORK>
__global__ void __launch_bounds__(kPageThreads) place_kernel(const PageArgs a) {
  pdl_enter();
  int at = __ldcg(a.blocks + blockIdx.x);
  if (FORK && at >= __ldcg(a.sums + kSumNeed)) return;
  const int p0 = blockIdx.x * kScanPages;
  for (int q = 0; q < kScanPages; q += kPageThreads) {
    const int p = p0 + q + threadIdx.x;
    const bool in = p < a.pages && counts<FORK, false>(a, p);
    int total;
    const int mine = block_scan<kPageThreads>(in, &total);
    if (p < a.pages) place<FORK>(a, p, at + mine, in);
    at += total;
  }
}

// All passes but the copy, in one block.
template <bool FORK>
__global__ void __launch_bounds__(1024) small_kernel(const PageArgs a) {
  pdl_enter();
  const int tid = threadIdx.x;
  clear_pass<FORK>(a, tid, 1024);
  __syncthreads();
  for (int s = tid >> 5; s < a.slots; s += 32) count_pass<FORK>(a, s, tid & 31, a.max_pages, 32);
  __syncthreads();
  const int nb = (a.pages + kScanPages - 1) / kScanPages;
  for (int b = 0; b < nb; ++b) {
    const int p = b * kScanPages + tid;
    const int n = __syncthreads_count(p < a.pages && counts<FORK, true>(a, p));
    if (tid == 0) a.blocks[b] = n;
  }
  __syncthreads();
  settle<FORK, 1024>(a, nb);
  __syncthreads();
  for (int b = 0; b < nb; ++b) {
    const int p = b * kScanPages + tid;
    const bool in = p < a.pages && counts<FORK, false>(a, p);
    int total;
    const int mine = block_scan<1024>(in, &total);
    if (p < a.pages) place<FORK>(a, p, __ldcg(a.blocks + b) + mine, in);
  }
  if (!FORK) {
    __syncthreads();
    map_pass(a, tid, 1024);
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

static unsigned copy_grid() {
  DevInfo di;
  return dev_info(&di) == PI_OK ? (unsigned)di.sms * 8 : 0;
}

static pi_status launch_copy(const CopyArgs& c, pi_stream stream) {
  const unsigned grid = copy_grid();
  return grid ? launch(copy_kernel, dim3(grid), kCopyThreads, 0, stream, c) : PI_ERR_CUDA;
}

// The passes up to `place` (and a small compaction's map).
template <bool FORK>
static pi_status launch_passes(const PageArgs& a, pi_stream stream) {
  if (one_block(a)) return launch(small_kernel<FORK>, dim3(1), 1024, 0, stream, a);
  const unsigned nb = (unsigned)((a.pages + kScanPages - 1) / kScanPages);
  const unsigned parts = (unsigned)a.max_pages / kCountEntries + 1;
  const dim3 entries((unsigned)a.slots, parts < 65535 ? parts : 65535);
  const unsigned clear = (unsigned)((a.pages + kPageThreads - 1) / kPageThreads);
  pi_status st = launch(clear_kernel<FORK>, dim3(clear < 1216 ? clear : 1216), kPageThreads, 0, stream, a);
  if (st == PI_OK) st = launch(count_kernel<FORK>, entries, kPageThreads, 0, stream, a);
  if (st == PI_OK) st = launch(rank_kernel<FORK>, dim3(nb), kPageThreads, 0, stream, a);
  if (st == PI_OK) st = launch(place_kernel<FORK>, dim3(nb), kPageThreads, 0, stream, a);
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
  if (one_block(a)) return pool ? launch_copy(c, stream) : PI_OK;
  const unsigned grid = copy_grid();
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
