// accept.cu — the drafts that the chosen tokens confirm stay in the cache
// (include/pi_draft.h).
#include "serve.cuh"

namespace pis {

// The root is taken; from a draft that is taken, the first child whose token is
// the one chosen there.  A block walks the path of one slot by itself: of the
// drafts that fit, the lowest child of the current one is a ballot away.
// Confirmed drafts move up behind one another: step j's row goes to place j
// <= its own, so a thread that copies its piece of the rows in the path's order,
// reading a batch before writing it, overwrites no row that is still needed.
// Bound: the moved rows' bytes (64 slots, 48 layers of 8 heads of 128, some 100 rows:
// 13.4 us, 52 % of a copy's rate; one slot 6.1 us, all of it the call).
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
