// tree.cu — attention of drafted tokens over a paged cache, and the drafts
// that stay in it (include/pi_draft.h).
#include "serve.cuh"

namespace pis {

struct TreeArgs {
  const float *q, *k_new, *v_new;
  const int *parent, *count, *table, *len;
  uint16_t* pool;  // the layer's pages
  float *y, *lse;
  int* status;
  int slots, drafts, heads, kv_heads, group, head_dim, page_tokens, pages, max_pages, window, sinks;
  float scale;  // scale log2(e)
};

// What a slot's drafts see: the tokens [tail, base) and [0, first) before
// them, and one another.  The drafts begin at token base; the one of depth d (0
// without a parent) stands at position base + d, and a window hides from it the
// tokens below base + d + 1 - window but for the first `sinks`.
struct TreeSlot {
  int base, count, tail, first;
};
__device__ __forceinline__ TreeSlot tree_slot(const TreeArgs& a, int slot) {
  TreeSlot v;
  const int n = __ldg(a.len + slot), c = a.count ? __ldg(a.count + slot) : a.drafts;
  const bool ok = n >= 0 && n <= a.max_pages * a.page_tokens && c >= 0 && c <= a.drafts && c <= n;
  v.count = ok ? c : 0;
  v.base = ok ? n - c : 0;
  v.tail = a.window > 0 ? max(0, v.base + 1 - a.window) : 0;
  v.first = min(v.tail, a.sinks);
  return v;
}
__device__ __forceinline__ bool tree_slot_bad(const TreeArgs& a, int slot) {
  const int n = __ldg(a.len + slot), c = a.count ? __ldg(a.count + slot) : a.drafts;
  return n < 0 || n > a.max_pages * a.page_tokens || c < 0 || c > a.drafts || c > n;
}

// The drafts that draft i sees, as bits: itself and its ancestors, in the
// window.  `parent(j)` gives a draft's parent; one that is not -1 .. j - 1
// counts as -1 (reported).
template <typename F>
__device__ __forceinline__ unsigned long long tree_path(const TreeArgs& a, int i, F parent) {
  unsigned long long path = 0;
  for (int j = i; j >= 0;) {
    path |= 1ull << j;
    int p = parent(j);
    if (p < -1 || p >= j) {
      set_status(a.status, PI_ERR_INDEX);
      p = -1;
    }
    j = p;
  }
  return path;
}
__device__ __forceinline__ unsigned long long tree_seen(const TreeArgs& a, int base, unsigned long long path) {
  const int hidden = a.window > 0 ? __popcll(path) - a.window : 0;  // the path's first ones
  unsigned long long seen = path;
  for (int d = 0; d < hidden; ++d) {  // the one of depth d
    const unsigned long long bit = path & -path;
    path ^= bit;
    if (base + d >= a.sinks) seen ^= bit;
  }
  return seen;
}

// A query row's sums over some of its tokens: the running maximum m of the
// scores (in base 2), l = sum 2^(a - m), o = sum 2^(a - m) v.
struct RowSums {
  float m, l;
  float o[8];  // of elements 8 lane + i
};

// Adds 32 tokens, one per lane, by the formulas in fp32 (any operand, infinite
// ones too).  `key`: the lane's key, null where its token is not seen; `val`:
// its value; fp32 rows (NEW) are taken as rounded to the cache's type.
template <int DT, bool NEW>
__device__ __forceinline__ void row_add32(const TreeArgs& a, const float* q, const void* key, const void* val,
                                          RowSums& r) {
  const int lane = threadIdx.x & 31, D = a.head_dim;
  auto piece = [](const void* row, int e, float (&x)[8]) {
    if (NEW) {
      const float4 u = __ldg(reinterpret_cast<const float4*>(row) + (e >> 2));
      const float4 w = __ldg(reinterpret_cast<const float4*>(row) + (e >> 2) + 1);
      const float f[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = from_bits<DT>(to_bits<DT>(f[i]));
    } else {
      const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(row) + e);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = from_bits<DT>((uint16_t)(w[i >> 1] >> 16 * (i & 1)));
    }
  };
  float s = -INFINITY;
  if (key) {
    s = 0.f;
    for (int e = 0; e < D; e += 8) {
      float k[8];
      piece(key, e, k);
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(__ldg(q + e + i), k[i], s);
    }
    s *= a.scale;
  }
  float up = s;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) up = fmaxf(up, __shfl_xor_sync(~0u, up, o));
  up = fmaxf(up, r.m);
  const float ref = up == -INFINITY ? 0.f : up;
  const float was = part_weight(r.m - ref), p = key ? ex2(s - ref) : 0.f;
  // an infinite value's weight is not 0 unless its score is -infinity
  const float w = key && s != -INFINITY ? fmaxf(p, 0x1p-126f) : p;
  r.m = up;
  r.l = fmaf(r.l, was, warp_sum(p));
#pragma unroll
  for (int i = 0; i < 8; ++i) r.o[i] *= was;
  for (uint32_t left = __ballot_sync(~0u, key != nullptr); left; left &= left - 1) {
    const int j = __ffs(left) - 1;
    const float wj = __shfl_sync(~0u, w, j);
    const void* row = reinterpret_cast<const void*>(
        __shfl_sync(~0u, reinterpret_cast<unsigned long long>(val), j));
    if (8 * lane < D) {
      float v[8];
      piece(row, 8 * lane, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) r.o[i] = fmaf(wj, v[i], r.o[i]);
    }
  }
}

// Adds the cached tokens [t0, t1), of which those at or past `lo` and the
// first `sinks` are seen.
template <int DT>
__device__ __forceinline__ void row_add_cached(const TreeArgs& a, int slot, int g, const float* q, int t0, int t1,
                                               int lo, RowSums& r) {
  const int lane = threadIdx.x & 31;
  for (int t = t0 + lane; t - lane < t1; t += 32) {
    const uint16_t* key = nullptr;
    if (t < t1 && (t >= lo || t < a.sinks)) {
      const int j = t / a.page_tokens;
      const int page = checked_page(__ldg(a.table + (size_t)slot * a.max_pages + j), a.pages, a.status);
      if (page >= 0)
        key = a.pool + (((size_t)page * 2 * a.kv_heads + g) * a.page_tokens + t - j * a.page_tokens) * a.head_dim;
    }
    row_add32<DT, false>(a, q, key, key + (size_t)a.kv_heads * a.page_tokens * a.head_dim, r);
  }
}

// Adds the drafts `seen`.
template <int DT>
__device__ __forceinline__ void row_add_drafts(const TreeArgs& a, int slot, const TreeSlot& v, int g, const float* q,
                                               unsigned long long seen, RowSums& r) {
  const int lane = threadIdx.x & 31;
  if (!a.k_new) {
    for (int j0 = 0; j0 < v.count; j0 += 32) {
      const int t = v.base + j0 + lane;
      const uint16_t* key = nullptr;
      if (j0 + lane < v.count && seen >> (j0 + lane) & 1) {
        const int j = t / a.page_tokens;
        const int page = checked_page(__ldg(a.table + (size_t)slot * a.max_pages + j), a.pages, a.status);
        if (page >= 0)
          key = a.pool + (((size_t)page * 2 * a.kv_heads + g) * a.page_tokens + t - j * a.page_tokens) * a.head_dim;
      }
      row_add32<DT, false>(a, q, key, key + (size_t)a.kv_heads * a.page_tokens * a.head_dim, r);
    }
    return;
  }
  for (int j0 = 0; j0 < v.count; j0 += 32) {
    const bool ok = j0 + lane < v.count && seen >> (j0 + lane) & 1;
    const size_t row = (((size_t)slot * a.drafts + min(j0 + lane, v.count - 1)) * a.kv_heads + g) * a.head_dim;
    row_add32<DT, true>(a, q, ok ? a.k_new + row : nullptr, a.v_new + row, r);
  }
}

// One warp per query row, in fp32.
template <int DT>
__global__ void __launch_bounds__(128) tree_rows_kernel(const __grid_constant__ TreeArgs a) {
  pdl_enter();
  const int lane = threadIdx.x & 31, D = a.head_dim;
  const long long rows = (long long)a.slots * a.drafts * a.heads;
  for (long long row = blockIdx.x * 4ll + (threadIdx.x >> 5); row < rows; row += gridDim.x * 4ll) {
    const int slot = (int)(row / (a.drafts * a.heads)), i = (int)(row / a.heads) % a.drafts, h = (int)(row % a.heads);
    const int g = h / a.group;
    const TreeSlot v = tree_slot(a, slot);
    if (lane == 0 && i == 0 && h == 0 && tree_slot_bad(a, slot)) set_status(a.status, PI_ERR_INDEX);
    if (i >= v.count) continue;
    const unsigned long long path = a.parent
        ? tree_path(a, i, [&](int j) { return __ldg(a.parent + (size_t)slot * a.drafts + j); })
        : (2ull << i) - 1;
    if (a.k_new && h % a.group == 0) {
      const int t = v.base + i, j = t / a.page_tokens;
      const int page = checked_page(__ldg(a.table + (size_t)slot * a.max_pages + j), a.pages, a.status);
      const size_t from = (((size_t)slot * a.drafts + i) * a.kv_heads + g) * D;
      if (page >= 0)
        for (int e = lane; e < D; e += 32) {
          uint16_t* to = a.pool + (((size_t)page * 2 * a.kv_heads + g) * a.page_tokens + t - j * a.page_tokens) * D + e;
          *to = to_bits<DT>(__ldg(a.k_new + from + e));
          to[(size_t)a.kv_heads * a.page_tokens * D] = to_bits<DT>(__ldg(a.v_new + from + e));
        }
    }
    const float* q = a.q + row * D;
    RowSums r = {-INFINITY, 0.f, {}};
    const int lo = a.window > 0 ? v.base + __popcll(path) - a.window : 0;
    row_add_cached<DT>(a, slot, g, q, 0, v.first, lo, r);
    row_add_cached<DT>(a, slot, g, q, v.tail, v.base, lo, r);
    row_add_drafts<DT>(a, slot, v, g, q, tree_seen(a, v.base, path), r);
    const float inv = r.l > 0.f ? 1.f / r.l : r.l == r.l ? 0.f : r.l;
    if (8 * lane < D) {
      float4* to = reinterpret_cast<float4*>(a.y + row * D + 8 * lane);
      to[0] = make_float4(r.o[0] * inv, r.o[1] * inv, r.o[2] * inv, r.o[3] * inv);
      to[1] = make_float4(r.o[4] * inv, r.o[5] * inv, r.o[6] * inv, r.o[7] * inv);
    }
    if (lane == 0 && a.lse) a.lse[row] = (r.m + log2f(r.l)) * kLn2;
  }
}

// ------------------------------------------------------------------ acceptance
//
// The root is taken; from a draft that is taken, the first child whose token is
// the one chosen there.  A block walks the path of one slot by itself: of the
// drafts that fit, the lowest child of the current one is a ballot away.
// Confirmed drafts move up behind one another: step j's row goes to place j
// <= its own, so a thread that copies its piece of the rows in the path's order,
// reading a batch before writing it, overwrites no row that is still needed.
// Bound: the moved rows' bytes.
struct AcceptArgs {
  const int *parent, *count, *tokens, *choice, *table, *len;
  uint16_t* pool;
  int *len_out, *path, *accepted, *next, *status;
  int slots, drafts, max_pages, layers, kv_heads, head_dim, page_tokens, pages;
  int blocks;  // per slot
};

constexpr int kAcceptThreads = 256;

__global__ void __launch_bounds__(kAcceptThreads) tree_accept_kernel(const __grid_constant__ AcceptArgs a) {
  pdl_enter();
  __shared__ int s_path[64], s_n;
  __shared__ long long s_row[64];  // first of the row's elements in a layer, of K and kv head 0
  const int slot = blockIdx.x / a.blocks, part = blockIdx.x - slot * a.blocks;
  const int tid = threadIdx.x, lane = tid & 31;
  const int P = a.page_tokens, most = a.max_pages * P;
  const int n = __ldg(a.len + slot), c = a.count ? __ldg(a.count + slot) : a.drafts;
  const bool ok = n >= 0 && n <= most && c >= 0 && c <= a.drafts && c <= n;
  const int count = ok ? c : 0, base = n - c;
  if (tid < 32) {
    bool bad = !ok;
    int par[2], tok[2], want[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = lane + 32 * k;
      const size_t at = (size_t)slot * a.drafts + i;
      const bool in = i < count;
      par[k] = in ? a.parent ? __ldg(a.parent + at) : i - 1 : -1;
      tok[k] = in ? __ldg(a.tokens + at) : 0;
      want[k] = in ? __ldg(a.choice + at) : -1;
      if (in && (par[k] < -1 || par[k] >= i)) {
        bad = true;
        par[k] = -1;
      }
    }
    int at = 0, steps = 0, chosen = -1;
    while (steps < count) {
      if (lane == 0) s_path[steps] = at;
      ++steps;
      const int w0 = __shfl_sync(~0u, want[0], at & 31), w1 = __shfl_sync(~0u, want[1], at & 31);
      chosen = at < 32 ? w0 : w1;
      const unsigned f0 = __ballot_sync(~0u, chosen >= 0 && lane < count && par[0] == at && tok[0] == chosen);
      const unsigned f1 = __ballot_sync(~0u, chosen >= 0 && lane + 32 < count && par[1] == at && tok[1] == chosen);
      if (!(f0 | f1)) break;
      at = f0 ? __ffs(f0) - 1 : 31 + __ffs(f1);
    }
    __syncwarp();
    if (part == 0) {
      if (bad) set_status(a.status, PI_ERR_INDEX);
      for (int i = lane; i < a.drafts; i += 32)
        a.path[(size_t)slot * a.drafts + i] = i < steps ? s_path[i] : -1;
      if (lane == 0) {
        a.len_out[slot] = ok ? base + steps : 0;
        a.accepted[slot] = steps;
        a.next[slot] = chosen;
      }
    }
    if (lane == 0) s_n = steps;
  }
  __syncthreads();
  if (!a.pool) return;
  (void)P;
  // rows that stay where they are come first on the path
  const int steps = s_n;
  int first = 0;
  while (first < steps && s_path[first] == first) ++first;
  if (first == steps) return;
  const size_t half = (size_t)a.kv_heads * P * a.head_dim;
  auto row_of = [&](int t) -> long long {
    const int j = t / P;
    const int page = checked_page(__ldg(a.table + (size_t)slot * a.max_pages + j), a.pages, a.status);
    return page < 0 ? -1 : (long long)page * 2 * (long long)half + (long long)(t - j * P) * a.head_dim;
  };
  __shared__ long long s_to[64];
  for (int j = first + tid; j < steps; j += kAcceptThreads) {
    s_row[j] = row_of(base + s_path[j]);
    s_to[j] = row_of(base + j);
  }
  __syncthreads();
  const int pieces = a.head_dim >> 3;
  const long long layer = (long long)a.pages * 2 * half, total = 2ll * a.layers * a.kv_heads * pieces;
  for (long long e = (long long)part * kAcceptThreads + tid; e < total; e += (long long)a.blocks * kAcceptThreads) {
    const long long r = e / pieces;
    const int piece = (int)(e - r * pieces), g = (int)(r % a.kv_heads);
    const long long kv = r / a.kv_heads;  // 2 layer + (K, V)
    uint16_t* at = a.pool + (kv >> 1) * layer + (kv & 1) * half + (size_t)g * P * a.head_dim + 8 * piece;
    constexpr int B = 8;
    for (int j0 = first; j0 < steps; j0 += B) {
      uint4 x[B];
#pragma unroll
      for (int j = 0; j < B; ++j)
        if (j0 + j < steps && s_row[j0 + j] >= 0) x[j] = *reinterpret_cast<const uint4*>(at + s_row[j0 + j]);
#pragma unroll
      for (int j = 0; j < B; ++j)
        if (j0 + j < steps && s_row[j0 + j] >= 0 && s_to[j0 + j] >= 0)
          *reinterpret_cast<uint4*>(at + s_to[j0 + j]) = x[j];
    }
  }
}

}  // namespace pis

using namespace pis;

extern "C" {

size_t pi_tree_workspace_size(const pi_cache_desc* cache, int32_t slots, int32_t heads, int32_t drafts) {
  if (check_cache(cache) != PI_OK || slots < 1 || slots > PI_CACHE_MAX_SLOTS) return 0;
  if (heads < 1 || heads > kMaxHeads || heads % cache->kv_heads || drafts < 1 || drafts > PI_TREE_MAX) return 0;
  return kAlign;
}

pi_status pi_tree_attention(const pi_cache_desc* cache, int32_t layer, int32_t slots, int32_t heads,
                            int32_t max_pages, int32_t drafts, const int32_t* parent, const int32_t* count,
                            const float* q, const float* k_new, const float* v_new, const int32_t* table,
                            const int32_t* len, void* pool, float scale, int32_t window, int32_t sinks,
                            float* y, float* lse, int32_t* dev_status, void* ws, size_t ws_bytes,
                            pi_stream stream) {
  pi_status st = check_cache(cache);
  if (st != PI_OK) return st;
  const pi_cache_desc& C = *cache;
  st = check_slots(C, slots, max_pages);
  if (st != PI_OK) return st;
  if (layer < 0 || layer >= C.layers || heads < 1 || heads > kMaxHeads || heads % C.kv_heads) return PI_ERR_SHAPE;
  if (drafts < 1 || drafts > PI_TREE_MAX || window < 0 || sinks < 0) return PI_ERR_SHAPE;
  if (!q || !table || !len || !pool || !y || !dev_status || !ws || !k_new != !v_new) return PI_ERR_NULL;
  if (!all_aligned(parent, count, q, k_new, v_new, table, len, pool, y, lse, dev_status, ws)) return PI_ERR_ALIGN;
  if (ws_bytes < pi_tree_workspace_size(cache, slots, heads, drafts)) return PI_ERR_WORKSPACE;
  TreeArgs a{};
  a.q = q;
  a.k_new = k_new;
  a.v_new = v_new;
  a.parent = parent;
  a.count = count;
  a.table = table;
  a.len = len;
  a.pool = static_cast<uint16_t*>(pool) + (size_t)layer * C.pages * page_elems(C);
  a.y = y;
  a.lse = lse;
  a.status = dev_status;
  a.slots = slots;
  a.drafts = drafts;
  a.heads = heads;
  a.kv_heads = C.kv_heads;
  a.group = heads / C.kv_heads;
  a.head_dim = C.head_dim;
  a.page_tokens = C.page_tokens;
  a.pages = C.pages;
  a.max_pages = max_pages;
  a.window = window;
  a.sinks = sinks;
  a.scale = scale * 1.4426950408889634f;
  const long long rows = (long long)slots * drafts * heads, blocks = (rows + 3) / 4;
  return launch(C.dtype == PI_F16 ? tree_rows_kernel<0> : tree_rows_kernel<1>,
                dim3((unsigned)(blocks < 65536 ? blocks : 65536)), 128, 0, stream, a);
}

pi_status pi_tree_accept(const pi_cache_desc* cache, int32_t slots, int32_t max_pages, int32_t drafts,
                         const int32_t* parent, const int32_t* count, const int32_t* tokens,
                         const int32_t* choice, const int32_t* table, const int32_t* len, void* pool,
                         int32_t* len_out, int32_t* path, int32_t* accepted, int32_t* next,
                         int32_t* dev_status, pi_stream stream) {
  pi_status st = check_cache(cache);
  if (st != PI_OK) return st;
  const pi_cache_desc& C = *cache;
  st = check_slots(C, slots, max_pages);
  if (st != PI_OK) return st;
  if (drafts < 1 || drafts > PI_TREE_MAX) return PI_ERR_SHAPE;
  if (!tokens || !choice || !table || !len || !len_out || !path || !accepted || !next || !dev_status)
    return PI_ERR_NULL;
  if (!all_aligned(parent, count, tokens, choice, table, len, pool, len_out, path, accepted, next, dev_status))
    return PI_ERR_ALIGN;
  // every block of a slot reads what these hold
  for (const void* out : {(const void*)len_out, (const void*)path, (const void*)accepted, (const void*)next})
    for (const void* in : {(const void*)parent, (const void*)count, (const void*)tokens, (const void*)choice,
                           (const void*)table, (const void*)len})
      if (out == in) return PI_ERR_SHAPE;
  AcceptArgs a{parent, count, tokens, choice, table, len, static_cast<uint16_t*>(pool), len_out, path, accepted,
               next, dev_status, slots, drafts, max_pages, C.layers, C.kv_heads, C.head_dim, C.page_tokens,
               C.pages, 1};
  DevInfo di;
  st = dev_info(&di);
  if (st != PI_OK) return st;
  // enough blocks to fill the GPU, while each thread has a piece of the rows
  const long long work = pool ? (2ll * C.layers * C.kv_heads * (C.head_dim / 8) + kAcceptThreads - 1) / kAcceptThreads : 1;
  const long long fill = (8ll * di.sms + slots - 1) / slots;
  a.blocks = (int)(work < fill ? work : fill);
  return launch(tree_accept_kernel, dim3((unsigned)(a.blocks * slots)), kAcceptThreads, 0, stream, a);
}

}  // extern "C"
