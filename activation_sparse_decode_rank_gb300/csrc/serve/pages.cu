// pages.cu — page bookkeeping of the paged cache: forking, freeing, trimming
// and growing slots, compaction, page copies (include/pi_serve.h).
//
// References are counted anew from the tables in each call, so no count can
// drift: a page is live while a used table entry or a holder names it.
#include "serve.cuh"

namespace pis {

struct PageArgs {
  const int *parent, *grow, *held, *table_in, *len_in;
  int *table, *len, *ref, *map, *pairs, *counts, *status;
  int *blocks, *owner, *free_list;
  int slots, max_pages, pages, page_tokens;
};

// What becomes of slot s (pi_cache_fork): the parent's row, the tokens kept,
// the tokens wanted.
struct Fate {
  int parent, keep, want;
};

__device__ __forceinline__ Fate fate_of(const PageArgs& a, int s) {
  Fate f{a.parent[s], 0, 0};
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
  long long want = base + a.grow[s];
  want = want < 0 ? 0 : want;
  if (want > most) {
    set_status(a.status, PI_ERR_CAPACITY);
    want = most;
  }
  f.want = (int)want;
  f.keep = (int)(base < want ? base : want);
  return f;
}

__global__ void __launch_bounds__(256) fork_init_kernel(const PageArgs a) {
  pdl_enter();
  for (int p = blockIdx.x * 256 + threadIdx.x; p < a.pages; p += gridDim.x * 256) {
    a.ref[p] = a.held ? a.held[p] : 0;
    a.owner[p] = a.slots;
  }
}

// Full pages are shared; the lowest slot bids for each partly filled one.
__global__ void __launch_bounds__(256) fork_share_kernel(const PageArgs a) {
  pdl_enter();
  const int s = blockIdx.x;
  const Fate f = fate_of(a, s);
  const int whole = f.keep / a.page_tokens;
  const int* src = a.table_in + (size_t)max(f.parent, 0) * a.max_pages;
  int* dst = a.table + (size_t)s * a.max_pages;
  for (int j = threadIdx.x; j < a.max_pages; j += 256) {
    int p = -1;
    if (j < whole) {
      p = checked_page(src[j], a.pages, a.status);
      if (p >= 0) atomicAdd(a.ref + p, 1);
    }
    dst[j] = p;
  }
  if (threadIdx.x == 0 && f.keep % a.page_tokens) {
    const int p = checked_page(src[whole], a.pages, a.status);
    if (p >= 0) atomicMin(a.owner + p, s);
  }
}

// One block: who keeps its last page, how many fresh pages each slot needs,
// the free pages in ascending order, and their assignment in slot order.
__global__ void __launch_bounds__(1024) fork_assign_kernel(const PageArgs a) {
  pdl_enter();
  __shared__ int s_first[PI_CACHE_MAX_SLOTS], s_need[PI_CACHE_MAX_SLOTS], s_src[PI_CACHE_MAX_SLOTS];
  const int tid = threadIdx.x;
  for (int s = tid; s < a.slots; s += 1024) {
    const Fate f = fate_of(a, s);
    const int whole = f.keep / a.page_tokens;
    int first = whole, from = -1;
    if (f.keep % a.page_tokens) {
      const int p = a.table_in[(size_t)max(f.parent, 0) * a.max_pages + whole];
      if ((unsigned)p < (unsigned)a.pages) {
        if (a.owner[p] == s && __ldcg(a.ref + p) == 0) {
          a.table[(size_t)s * a.max_pages + whole] = p;
          first = whole + 1;
        } else {
          from = p;
        }
      }
    }
    s_first[s] = first;
    s_need[s] = max(0, pages_of(f.want, a.page_tokens) - first);
    s_src[s] = from;
    a.len[s] = f.want;
  }
  __syncthreads();
  // the pages kept by their owner count from here on
  for (int s = tid; s < a.slots; s += 1024) {
    const int j = s_first[s] - 1;
    if (j >= 0 && s_first[s] > 0) {
      const Fate f = fate_of(a, s);
      if (j == f.keep / a.page_tokens && f.keep % a.page_tokens)
        a.ref[a.table[(size_t)s * a.max_pages + j]] = 1;
    }
  }
  __syncthreads();
  if (tid == 0) {
    int total = 0, n = 0, live = 0, copies = 0;
    for (int s = 0; s < a.slots; ++s) total += s_need[s];
    for (int p = 0; p < a.pages; ++p) {
      if (a.ref[p] == 0) {
        if (n < total) a.free_list[n++] = p;
      } else {
        ++live;
      }
    }
    if (n < total) set_status(a.status, PI_ERR_CAPACITY);
    int at = 0;
    for (int s = 0; s < a.slots; ++s) {
      for (int j = 0; j < s_need[s]; ++j) {
        if (at == n) {
          a.len[s] = min(a.len[s], (s_first[s] + j) * a.page_tokens);
          break;
        }
        const int p = a.free_list[at++];
        a.table[(size_t)s * a.max_pages + s_first[s] + j] = p;
        a.ref[p] = 1;
        ++live;
        if (j == 0 && s_src[s] >= 0) {
          a.pairs[2 * copies] = s_src[s];
          a.pairs[2 * copies + 1] = p;
          ++copies;
        }
      }
    }
    a.counts[0] = copies;
    a.counts[1] = live;
  }
}

__global__ void __launch_bounds__(256) compact_count_kernel(const PageArgs a) {
  pdl_enter();
  const int s = blockIdx.x;
  int n = a.len_in[s];
  if (n < 0 || n > a.max_pages * a.page_tokens) {
    if (threadIdx.x == 0) set_status(a.status, PI_ERR_INDEX);
    n = 0;
  }
  const int used = pages_of(n, a.page_tokens);
  for (int j = threadIdx.x; j < used; j += 256) {
    const int p = checked_page(a.table_in[(size_t)s * a.max_pages + j], a.pages, a.status);
    if (p >= 0) atomicAdd(a.owner + p, 1);
  }
}

__global__ void __launch_bounds__(256) compact_init_kernel(const PageArgs a) {
  pdl_enter();
  for (int p = blockIdx.x * 256 + threadIdx.x; p < a.pages; p += gridDim.x * 256) {
    a.owner[p] = a.held ? a.held[p] : 0;
    a.ref[p] = 0;
  }
}

__global__ void compact_map_kernel(const PageArgs a) {
  pdl_enter();
  int live = 0;
  for (int p = 0; p < a.pages; ++p) live += a.owner[p] > 0;
  int hole = 0, moved = 0;
  for (int p = 0; p < a.pages; ++p) {
    const int r = a.owner[p];
    int to = -1;
    if (r > 0) {
      to = p;
      if (p >= live) {
        while (a.owner[hole] > 0) ++hole;
        to = hole++;
        a.pairs[2 * moved] = p;
        a.pairs[2 * moved + 1] = to;
        ++moved;
      }
      a.ref[to] = r;
    }
    a.map[p] = to;
  }
  a.counts[0] = moved;
  a.counts[1] = live;
}

__global__ void __launch_bounds__(256) compact_table_kernel(const PageArgs a) {
  pdl_enter();
  const int s = blockIdx.x;
  const int n = a.len_in[s];
  const int used = n < 0 || n > a.max_pages * a.page_tokens ? 0 : pages_of(n, a.page_tokens);
  for (int j = threadIdx.x; j < a.max_pages; j += 256) {
    const size_t e = (size_t)s * a.max_pages + j;
    const int p = j < used ? a.table_in[e] : -1;
    a.table[e] = (unsigned)p < (unsigned)a.pages ? a.map[p] : -1;
  }
}

// Page pairs x layers in pieces of 16 bytes.
__global__ void __launch_bounds__(256) copy_kernel(const int* pairs, const int* count, int cap,
                                                   uint4* pool, int pages, int layers,
                                                   long long page16, int* status) {
  pdl_enter();
  int n = *count;
  if (n > cap) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_status(status, PI_ERR_CAPACITY);
    n = cap;
  }
  const long long rows = (long long)n * layers;
  for (long long r = blockIdx.x; r < rows; r += gridDim.x) {
    const int i = (int)(r / layers), layer = (int)(r % layers);
    const int from = pairs[2 * i], to = pairs[2 * i + 1];
    if ((unsigned)from >= (unsigned)pages || (unsigned)to >= (unsigned)pages) {
      if (threadIdx.x == 0) set_status(status, PI_ERR_INDEX);
      continue;
    }
    const uint4* src = pool + ((size_t)layer * pages + from) * page16;
    uint4* dst = pool + ((size_t)layer * pages + to) * page16;
    for (long long e = threadIdx.x; e < page16; e += 256) dst[e] = src[e];
  }
}

static pi_status launch_copy(const pi_cache_desc& C, const int* pairs, const int* count, int cap,
                             void* pool, int* status, pi_stream stream) {
  return launch(copy_kernel, dim3(152 * 8), 256, 0, stream, pairs, count, cap,
                static_cast<uint4*>(pool), C.pages, C.layers, (long long)(page_elems(C) / 8),
                status);
}

static void bind_ws(PageArgs& a, const pi_cache_desc& C, int slots, void* ws) {
  const CacheWs w = cache_ws(C, slots, 0);
  char* b = static_cast<char*>(ws);
  a.blocks = reinterpret_cast<int*>(b + w.blocks);
  a.owner = reinterpret_cast<int*>(b + w.owner);
  a.free_list = reinterpret_cast<int*>(b + w.free_list);
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
  bind_ws(a, C, slots, ws);
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
  a.slots = slots;
  a.max_pages = max_pages;
  a.pages = C.pages;
  a.page_tokens = C.page_tokens;
  st = launch(fork_init_kernel, dim3((unsigned)((C.pages + 255) / 256)), 256, 0, stream, a);
  if (st == PI_OK) st = launch(fork_share_kernel, dim3((unsigned)slots), 256, 0, stream, a);
  if (st == PI_OK) st = launch(fork_assign_kernel, dim3(1), 1024, 0, stream, a);
  if (st == PI_OK && pool) st = launch_copy(C, pairs, counts, slots, pool, dev_status, stream);
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
  bind_ws(a, C, slots, ws);
  a.held = held;
  a.table_in = table_in;
  a.len_in = len;
  a.table = table;
  a.ref = ref;
  a.map = map;
  a.pairs = pairs;
  a.counts = counts;
  a.status = dev_status;
  a.slots = slots;
  a.max_pages = max_pages;
  a.pages = C.pages;
  a.page_tokens = C.page_tokens;
  st = launch(compact_init_kernel, dim3((unsigned)((C.pages + 255) / 256)), 256, 0, stream, a);
  if (st == PI_OK) st = launch(compact_count_kernel, dim3((unsigned)slots), 256, 0, stream, a);
  if (st == PI_OK) st = launch(compact_map_kernel, dim3(1), 1, 0, stream, a);
  if (st == PI_OK) st = launch(compact_table_kernel, dim3((unsigned)slots), 256, 0, stream, a);
  if (st == PI_OK && pool)
    st = launch_copy(C, pairs, counts, C.pages / 2, pool, dev_status, stream);
  return st;
}

pi_status pi_cache_copy(const pi_cache_desc* cache, const int32_t* pairs, const int32_t* count,
                        int32_t cap, void* pool, int32_t* dev_status, pi_stream stream) {
  pi_status st = check_cache(cache);
  if (st != PI_OK) return st;
  if (cap < 0) return PI_ERR_SHAPE;
  if (!pairs || !count || !pool || !dev_status) return PI_ERR_NULL;
  if (!all_aligned(pairs, count, pool, dev_status)) return PI_ERR_ALIGN;
  return launch_copy(*cache, pairs, count, cap, pool, dev_status, stream);
}

}  // extern "C"
