// attend.cu — attention of one new token per slot over a paged cache, and
// the stores of new keys and values (include/pi_serve.h).
#include "serve.cuh"

namespace pis {

struct AttendArgs {
  const float *q, *k_new, *v_new;
  const int *table, *len;
  uint16_t* pool;  // the layer's pages
  float *y, *lse;
  int* status;
  int slots, heads, kv_heads, group, head_dim, page_tokens, pages, max_pages, window, sinks;
  float scale;
};

// One block per (slot, query head): warp w takes the visible tokens w, w + 8,
// ..., lane l the head's dimensions l, l + 32, ...; each warp keeps a running
// maximum, sum and output, joined in warp order at the end.
template <int DT>
__global__ void __launch_bounds__(256) attend_kernel(const AttendArgs a) {
  pdl_enter();
  __shared__ float so[8][256], sm[8], sl[8];
  const int s = blockIdx.y, h = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = h / a.group, D = a.head_dim;
  int n = a.len[s];
  if (n < 0 || n > a.max_pages * a.page_tokens) {
    if (threadIdx.x == 0) set_status(a.status, PI_ERR_INDEX);
    n = 0;
  }
  const int tail = a.window > 0 ? max(0, n - a.window) : 0;  // first token of the window
  const int first = a.window > 0 ? min(tail, a.sinks) : 0;   // visible tokens before it
  const int seen = n - tail + first;
  float q[8], o[8];
  for (int i = 0; i < 8; ++i) {
    const int d = lane + 32 * i;
    q[i] = d < D ? a.q[((size_t)s * a.heads + h) * D + d] * a.scale : 0.f;
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int v = warp; v < seen; v += 8) {
    const int t = v < first ? v : v - first + tail;
    const int page = checked_page(a.table[(size_t)s * a.max_pages + t / a.page_tokens], a.pages,
                                  a.status);
    if (page < 0) continue;
    const size_t row = ((size_t)page * 2 * a.kv_heads + g) * a.page_tokens + t % a.page_tokens;
    uint16_t* kr = a.pool + row * D;
    uint16_t* vr = kr + (size_t)a.kv_heads * a.page_tokens * D;
    const bool fresh = a.k_new != nullptr && t == n - 1;
    const size_t nrow = ((size_t)s * a.kv_heads + g) * D;
    float dot = 0.f, vv[8];
    for (int i = 0; i < 8; ++i) {
      const int d = lane + 32 * i;
      if (d >= D) continue;
      uint16_t kb, vb;
      if (fresh) {
        kb = to_bits<DT>(a.k_new[nrow + d]);
        vb = to_bits<DT>(a.v_new[nrow + d]);
        if (h % a.group == 0) {
          kr[d] = kb;
          vr[d] = vb;
        }
      } else {
        kb = kr[d];
        vb = vr[d];
      }
      dot += q[i] * from_bits<DT>(kb);
      vv[i] = from_bits<DT>(vb);
    }
    dot = warp_sum(dot);
    const float mn = fmaxf(m, dot);
    const float c = m == -INFINITY ? 0.f : __expf(m - mn);
    const float p = __expf(dot - mn);
    l = l * c + p;
    for (int i = 0; i < 8; ++i)
      if (lane + 32 * i < D) o[i] = o[i] * c + p * vv[i];
    m = mn;
  }
  for (int i = 0; i < 8; ++i) so[warp][lane + 32 * i] = o[i];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  float mx = -INFINITY, tot = 0.f;
  for (int w = 0; w < 8; ++w) mx = fmaxf(mx, sm[w]);
  for (int w = 0; w < 8; ++w) tot += sl[w] > 0.f ? sl[w] * __expf(sm[w] - mx) : 0.f;
  for (int d = threadIdx.x; d < D; d += 256) {
    float r = 0.f;
    for (int w = 0; w < 8; ++w)
      if (sl[w] > 0.f) r += so[w][d] * __expf(sm[w] - mx);
    a.y[((size_t)s * a.heads + h) * D + d] = tot > 0.f ? r / tot : 0.f;
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[(size_t)s * a.heads + h] = tot > 0.f ? mx + logf(tot) : -INFINITY;
}

// Thread = eight elements of one (token, K or V, kv head) row.
template <int DT>
__global__ void __launch_bounds__(256) append_kernel(const float* k, const float* v,
                                                     const int* slot, const int* pos,
                                                     const int* table, uint16_t* pool,
                                                     long long total, int kv_heads, int head_dim,
                                                     int page_tokens, int pages, int slots,
                                                     int max_pages, int* status) {
  pdl_enter();
  const int pieces = head_dim >> 3;
  for (long long e = blockIdx.x * 256ll + threadIdx.x; e < total; e += gridDim.x * 256ll) {
    const int pc = (int)(e % pieces);
    const long long r = e / pieces;  // (token, kind, head)
    const int g = (int)(r % kv_heads);
    const long long tk = r / kv_heads;
    const int kind = (int)(tk & 1);
    const int i = (int)(tk >> 1);
    const int s = slot[i], p = pos[i];
    if (s == -1) continue;
    if (s < 0 || s >= slots || p < 0 || p >= max_pages * page_tokens) {
      set_status(status, PI_ERR_INDEX);
      continue;
    }
    const int page = checked_page(table[(size_t)s * max_pages + p / page_tokens], pages, status);
    if (page < 0) continue;
    const float4* src = reinterpret_cast<const float4*>((kind ? v : k) +
                                                        ((size_t)i * kv_heads + g) * head_dim) + 2 * pc;
    const float4 f0 = src[0], f1 = src[1];
    uint16_t* dst = pool + ((((size_t)page * 2 + kind) * kv_heads + g) * page_tokens +
                            p % page_tokens) * head_dim + 8 * pc;
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bits<DT>(f0.x, f0.y), pack_bits<DT>(f0.z, f0.w),
                                                pack_bits<DT>(f1.x, f1.y), pack_bits<DT>(f1.z, f1.w));
  }
}

}  // namespace pis

using namespace pis;

extern "C" {

size_t pi_cache_workspace_size(const pi_cache_desc* cache, int32_t slots, int32_t heads) {
  if (check_cache(cache) != PI_OK || slots < 1 || slots > PI_CACHE_MAX_SLOTS) return 0;
  if (heads < 0 || heads > kMaxHeads || heads % cache->kv_heads) return 0;
  return cache_ws(*cache, slots, heads).total;
}

pi_status pi_paged_attention(const pi_cache_desc* cache, int32_t layer, int32_t slots,
                             int32_t heads, int32_t max_pages, const float* q,
                             const float* k_new, const float* v_new, const int32_t* table,
                             const int32_t* len, void* pool, float scale, int32_t window,
                             int32_t sinks, float* y, float* lse, int32_t* dev_status, void* ws,
                             size_t ws_bytes, pi_stream stream) {
  pi_status st = check_cache(cache);
  if (st != PI_OK) return st;
  const pi_cache_desc& C = *cache;
  st = check_slots(C, slots, max_pages);
  if (st != PI_OK) return st;
  if (layer < 0 || layer >= C.layers || heads < 1 || heads > kMaxHeads || heads % C.kv_heads)
    return PI_ERR_SHAPE;
  if (window < 0 || sinks < 0) return PI_ERR_SHAPE;
  if (!q || !table || !len || !pool || !y || !dev_status || !ws || !k_new != !v_new)
    return PI_ERR_NULL;
  if (!all_aligned(q, k_new, v_new, table, len, pool, y, lse, dev_status, ws)) return PI_ERR_ALIGN;
  if (ws_bytes < cache_ws(C, slots, heads).total) return PI_ERR_WORKSPACE;
  AttendArgs a{};
  a.q = q;
  a.k_new = k_new;
  a.v_new = v_new;
  a.table = table;
  a.len = len;
  a.pool = static_cast<uint16_t*>(pool) + (size_t)layer * C.pages * page_elems(C);
  a.y = y;
  a.lse = lse;
  a.status = dev_status;
  a.slots = slots;
  a.heads = heads;
  a.kv_heads = C.kv_heads;
  a.group = heads / C.kv_heads;
  a.head_dim = C.head_dim;
  a.page_tokens = C.page_tokens;
  a.pages = C.pages;
  a.max_pages = max_pages;
  a.window = window;
  a.sinks = sinks;
  a.scale = scale;
  return launch(C.dtype == PI_F16 ? attend_kernel<0> : attend_kernel<1>,
                dim3((unsigned)heads, (unsigned)slots), 256, 0, stream, a);
}

pi_status pi_cache_append(const pi_cache_desc* cache, int32_t layer, int32_t slots,
                          int32_t max_pages, int32_t tokens, const int32_t* slot,
                          const int32_t* pos, const float* k, const float* v,
                          const int32_t* table, void* pool, int32_t* dev_status,
                          pi_stream stream) {
  pi_status st = check_cache(cache);
  if (st != PI_OK) return st;
  const pi_cache_desc& C = *cache;
  st = check_slots(C, slots, max_pages);
  if (st != PI_OK) return st;
  if (layer < 0 || layer >= C.layers || tokens < 0) return PI_ERR_SHAPE;
  if (!table || !pool || !dev_status) return PI_ERR_NULL;
  if (tokens > 0 && (!slot || !pos || !k || !v)) return PI_ERR_NULL;
  if (!all_aligned(slot, pos, k, v, table, pool, dev_status)) return PI_ERR_ALIGN;
  if (tokens == 0) return PI_OK;
  const long long total = 2ll * tokens * C.kv_heads * (C.head_dim / 8);
  const long long blocks = (total + 255) / 256;
  uint16_t* base = static_cast<uint16_t*>(pool) + (size_t)layer * C.pages * page_elems(C);
  return launch(C.dtype == PI_F16 ? append_kernel<0> : append_kernel<1>,
                dim3((unsigned)(blocks < 152 * 64 ? blocks : 152 * 64)), 256, 0, stream, k, v, slot,
                pos, table, base, total, C.kv_heads, C.head_dim, C.page_tokens, C.pages, slots,
                max_pages, dev_status);
}

}  // extern "C"
