// logprob.cu — log probabilities of given tokens, entropy and the largest
// alternatives of rows of logits (include/pi_serve.h).
//
// Mathematics.  One pass keeps, per thread, a running maximum m and the sums
// s = sum exp(x - m), t = sum exp(x - m)(x - m), rescaled when m grows; parts
// join the same way.  Then log p_i = x_i - m - log s and the entropy is
// log s - t / s, with no large terms to cancel.
//
// Alternatives without a second pass: order all elements by a unique key
// (value, then lowest index).  Threads own disjoint sets of elements, and the
// pass leaves each thread's largest key (the batch that held it is noted when
// the maximum grows, which is rare).  Let tau be the k-th largest of these.
// At least k elements are >= tau, so every one of the k largest is; and an
// element >= tau can only belong to the k threads whose largest key is >= tau.
// Only their elements are looked at again (k / 256 of the row, from L2).
// Selection is by sorted lists of 32 keys in the lanes of a warp: sort 32,
// merge two lists, a tree over the warps.
//
// Bound: HBM bandwidth (each logit read once); for 16-bit logits the pass
// issues some 7 instructions per logit, near the machine's rate at that
// bandwidth.  Few rows: a row is split over several blocks, and the last of
// them to arrive joins the parts in order.
#include "serve.cuh"

namespace pis {

typedef unsigned long long u64;

struct ScoreArgs {
  const void* logits;
  long long stride;
  const int* tokens;
  float *logprob, *entropy, *top_logprob;
  int* top_idx;
  int* status;
  int* arrived;  // per row, zero between calls
  float* psum;   // [rows][parts][4]: m, s, t
  u64* pkeys;    // [rows][parts][32]
  int rows, vocab, topk, parts;
};

constexpr int kScoreThreads = 256;
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kScoreBlocks = 4;        // per SM
constexpr int kScoreParts = 2048;      // most parts of rows in flight
constexpr int kBatch = 4;              // 16-byte vectors of a thread's batch
constexpr float kLog2e = 1.4426950408889634f;

template <int DT>
__device__ __forceinline__ float logit_at(const void* p, long long i) {
  if (DT == 2) return static_cast<const float*>(p)[i];
  return from_bits<DT>(static_cast<const uint16_t*>(p)[i]);
}

// Rank of (value, index): larger values first, equal ones (-0 = +0) by lower
// index, NaN below everything; 0 is no element.
__device__ __forceinline__ u64 rank_key(float v, int i) {
  uint32_t b = __float_as_uint(v + 0.f);
  b = v != v ? 0u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return ((u64)b << 32) | (uint32_t)~i;
}
__device__ __forceinline__ int key_index(u64 k) { return (int)~(uint32_t)k; }
__device__ __forceinline__ float key_value(u64 k) {
  const uint32_t b = (uint32_t)(k >> 32);
  return __uint_as_float((b & 0x80000000u) ? b & 0x7fffffffu : ~b);
}

// ------------------------------------------------------------------ lists of 32 keys
__device__ __forceinline__ u64 keep(u64 v, u64 w, bool larger) { return (v > w) == larger ? v : w; }

__device__ __forceinline__ u64 merge_down(u64 v) {  // a bitonic sequence, sorted descending
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) v = keep(v, __shfl_xor_sync(~0u, v, j), (lane & j) == 0);
  return v;
}
__device__ __forceinline__ u64 sort32(u64 v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 2; k < 32; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1)
      v = keep(v, __shfl_xor_sync(~0u, v, j), ((lane & j) == 0) == ((lane & k) == 0));
  return merge_down(v);
}
// The 32 largest of two sorted lists, sorted.
__device__ __forceinline__ u64 merge32(u64 a, u64 b) {
  const u64 r = __shfl_sync(~0u, b, 31 - (threadIdx.x & 31));
  return merge_down(a > r ? a : r);
}
// The warps' lists into one, left in warp 0.
__device__ __forceinline__ u64 block_merge(u64 v, u64 (*sh)[32]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll 1
  for (int half = kScoreWarps / 2; half > 0; half >>= 1) {
    if (warp >= half && warp < 2 * half) sh[warp][lane] = v;
    __syncthreads();
    if (warp < half) v = merge32(v, sh[warp + half][lane]);
  }
  return v;
}

// ------------------------------------------------------------------ sums
struct Sums {
  float m, s, t;
};
// The same sums with the maximum `top` >= a.m.
__device__ __forceinline__ Sums raised(const Sums& a, float top) {
  if (a.m == top || a.m == -INFINITY) return Sums{top, a.s, a.m == top ? a.t : 0.f};
  const float d = a.m - top, f = exp2f(d * kLog2e);
  return Sums{top, a.s * f, f * fmaf(d, a.s, a.t)};
}

template <int DT>
struct Vec {
  static constexpr int n = DT == 2 ? 4 : 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[n]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == 2) {
        f[i] = __uint_as_float(w[i]);
      } else if constexpr (DT == 1) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
      }
    }
  }
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void add_one(Sums& a, float ref, float x) {
  // exp underflows to 0 below -1000 anyway; keeps 0 * infinity out of t
  const float d = max_nan(x - ref, -1000.f);
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(d * kLog2e));
  a.s += e;
  a.t = fmaf(e, d, a.t);
}

// One block per (row, part).
template <int DT>
__global__ void __launch_bounds__(kScoreThreads, kScoreBlocks) score_kernel(const ScoreArgs a) {
  constexpr int VN = Vec<DT>::n, T = kScoreThreads;
  constexpr int kSize = DT == 2 ? 4 : 2;
  __shared__ u64 sh_keys[kScoreWarps][32], sh_tau;
  __shared__ float sh_sums[kScoreWarps][3];
  __shared__ int sh_win[32], sh_nwin, sh_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_enter();
  const long long row = blockIdx.x;
  const int part = blockIdx.y;
  const char* base = static_cast<const char*>(a.logits) + row * a.stride * kSize;
  // Vectors of 16 aligned bytes; vector j holds the elements j VN - shift ...
  const int shift = (int)(reinterpret_cast<uintptr_t>(base) & 15) / kSize;
  const uint4* vecs = reinterpret_cast<const uint4*>(base - shift * kSize);
  const int nvec = (a.vocab + shift + VN - 1) / VN;
  const int v0 = (int)((long long)part * nvec / a.parts);
  const int v1 = (int)((long long)(part + 1) * nvec / a.parts);
  // whole vectors [w0, w1); the row's first and last, where cut, go to threads 0 and 1
  const int w0 = v0 == 0 && shift ? 1 : v0;
  const bool cut_last = v1 == nvec && (a.vocab + shift) % VN && nvec - 1 >= w0;
  const int w1 = cut_last ? v1 - 1 : v1;

  Sums sum{-INFINITY, 0.f, 0.f};
  int at = -1;  // batch of the thread's largest element; cut vectors: -2, -3
  auto raise = [&](float top, int where) {
    if (top > sum.m || (at == -1 && top == top)) {
      at = where;
      if (top > sum.m) sum = raised(sum, top);
    }
  };
  // elements of a cut vector
  auto cut = [&](int j, auto&& use) {
    for (int e = 0; e < VN; ++e) {
      const int i = j * VN + e - shift;
      if (i >= 0 && i < a.vocab) use(logit_at<DT>(base, i), i);
    }
  };
  const int steps = w1 > w0 ? (w1 - w0 + T * kBatch - 1) / (T * kBatch) : 0;
  const uint4* mine = vecs + w0 + tid;
  uint4 raw[kBatch];
  auto load = [&](int it) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int j = (it * kBatch + u) * T;
      if (w0 + tid + j < w1) raw[u] = __ldcs(mine + j);
    }
  };
  if (steps > 0) load(0);
  for (int it = 0; it < steps; ++it) {
    float x[kBatch][VN];
    bool have[kBatch];
    float top = -INFINITY;
    bool any = false;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      have[u] = w0 + tid + (it * kBatch + u) * T < w1;
      Vec<DT>::unpack(raw[u], x[u]);
    }
    const bool full = have[kBatch - 1];
    if (it + 1 < steps) load(it + 1);
    if (full) {
      float m4[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        m4[u] = x[u][0];
#pragma unroll
        for (int e = 1; e < VN; ++e) m4[u] = fmaxf(m4[u], x[u][e]);
      }
      top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
      any = true;
    } else {
      top = NAN;
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (have[u]) {
          any = true;
#pragma unroll
          for (int e = 0; e < VN; ++e) top = fmaxf(top, x[u][e]);
        }
    }
    if (any) raise(top, it);
    const float ref = sum.m == -INFINITY ? 0.f : sum.m;
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (full || have[u]) {
#pragma unroll
        for (int e = 0; e < VN; ++e) add_one(sum, ref, x[u][e]);
      }
  }
  if (tid == 0 && w0 > v0) {
    float top = NAN;
    cut(0, [&](float x, int) { top = fmaxf(top, x); });
    raise(top, -2);
    const float ref = sum.m == -INFINITY ? 0.f : sum.m;
    cut(0, [&](float x, int) { add_one(sum, ref, x); });
  }
  if (tid == 1 && cut_last) {
    float top = NAN;
    cut(nvec - 1, [&](float x, int) { top = fmaxf(top, x); });
    raise(top, -3);
    const float ref = sum.m == -INFINITY ? 0.f : sum.m;
    cut(nvec - 1, [&](float x, int) { add_one(sum, ref, x); });
  }

  // the block's sums
  float top = sum.m;
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  if (lane == 0) sh_sums[warp][0] = top;
  if (tid == 0) sh_nwin = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kScoreWarps; ++w) top = fmaxf(top, sh_sums[w][0]);
  {
    const Sums up = raised(sum, top);
    const float s = warp_sum(up.s), t = warp_sum(up.t);
    if (lane == 0) {
      sh_sums[warp][1] = s;
      sh_sums[warp][2] = t;
    }
  }

  // elements of thread w's set, one vector at a time
  auto each = [&](int w, int i, auto&& use) {  // i-th whole vector of thread w
    const int j = w0 + w + i * T;
    if (j >= w1) return;
    float x[VN];
    Vec<DT>::unpack(__ldg(vecs + j), x);
#pragma unroll
    for (int e = 0; e < VN; ++e) use(x[e], j * VN + e - shift);
  };
  u64 list = 0;  // this warp's 32 largest keys
  if (a.topk > 0) {
    u64 key = 0;
    auto best = [&](float x, int i) {
      const u64 k = rank_key(x, i);
      key = k > key ? k : key;
    };
    if (at == -1) {  // nothing but NaN: the first elements will do
      if (tid == 0 && w0 > v0) cut(0, best);
      each(tid, 0, best);
      if (key == 0 && tid == 1 && cut_last) cut(nvec - 1, best);
    } else if (at >= 0) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) each(tid, at * kBatch + u, best);
    } else {
      cut(at == -2 ? 0 : nvec - 1, best);
    }
    // equal values elsewhere in the thread's cut vector may come earlier
    if (tid == 0 && w0 > v0) cut(0, best);
    const u64 sorted = block_merge(sort32(key), sh_keys);
    if (warp == 0 && lane == a.topk - 1) sh_tau = sorted;
    __syncthreads();
    const u64 tau = sh_tau;
    if (key >= tau && key > 0) sh_win[atomicAdd(&sh_nwin, 1)] = tid;
    __syncthreads();
    const int nwin = sh_nwin, per = (max(0, w1 - w0) + T - 1) / T;
    u64 least = tau > 0 ? tau - 1 : 0;  // what enters is larger
    auto enter = [&](u64 k) {
      if (__any_sync(~0u, k > least)) {
        list = merge32(list, sort32(k > least ? k : 0));
        const u64 kth = __shfl_sync(~0u, list, a.topk - 1);
        least = kth > least ? kth : least;
      }
    };
    const int items = nwin * per;
    for (int i0 = warp * 32; i0 < items; i0 += T) {
      const int i = i0 + lane, w = min(i, items - 1) / per;
      const int j = w0 + sh_win[w] + (min(i, items - 1) - w * per) * T;
      const bool in = i < items && j < w1;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (in) v = __ldg(vecs + j);
      float x[VN];
      Vec<DT>::unpack(v, x);
#pragma unroll
      for (int e = 0; e < VN; ++e) enter(in ? rank_key(x[e], j * VN + e - shift) : 0);
    }
    if (warp == 0 && w0 > v0) {
      const int i = lane - shift;
      enter(lane < VN && i >= 0 && i < a.vocab ? rank_key(logit_at<DT>(base, i), i) : 0);
    }
    if (warp == 1 && cut_last) {
      const int i = (nvec - 1) * VN + lane - shift;
      enter(lane < VN && i >= 0 && i < a.vocab ? rank_key(logit_at<DT>(base, i), i) : 0);
    }
    list = block_merge(list, sh_keys);
  }
  __syncthreads();
  if (warp == 0) {
    sum = Sums{top, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kScoreWarps; ++w) {
      sum.s += sh_sums[w][1];
      sum.t += sh_sums[w][2];
    }
  }

  if (a.parts > 1) {
    const long long slot = row * a.parts + part;
    if (warp == 0) {
      if (lane == 0) __stcg(reinterpret_cast<float4*>(a.psum) + slot, make_float4(sum.m, sum.s, sum.t, 0.f));
      if (a.topk > 0) __stcg(a.pkeys + slot * 32 + lane, list);
      __threadfence();
      __syncwarp();
      if (lane == 0) sh_last = atomicAdd(a.arrived + row, 1) == a.parts - 1;
    }
    __syncthreads();
    if (!sh_last) return;
    __threadfence();
    if (tid == 0) a.arrived[row] = 0;
    // all parts, by one warp in order for the sums and by all for the lists
    if (warp == 0) {
      float up = -INFINITY;
      const float4* ps = reinterpret_cast<const float4*>(a.psum) + row * a.parts;
      for (int p = lane; p < a.parts; p += 32) up = fmaxf(up, __ldcg(ps + p).x);
#pragma unroll
      for (int o = 16; o; o >>= 1) up = fmaxf(up, __shfl_xor_sync(~0u, up, o));
      Sums all{up, 0.f, 0.f};
      for (int p = lane; p < a.parts; p += 32) {
        const float4 v = __ldcg(ps + p);
        const Sums one = raised(Sums{v.x, v.y, v.z}, up);
        all.s += one.s;
        all.t += one.t;
      }
      all.s = warp_sum(all.s);
      all.t = warp_sum(all.t);
      sum = all;
    }
    if (a.topk > 0) {
      list = 0;
      for (int p = warp; p < a.parts; p += kScoreWarps)
        list = merge32(list, __ldcg(a.pkeys + (row * a.parts + p) * 32 + lane));
      list = block_merge(list, sh_keys);
    }
  }

  if (warp == 0) {
    const bool bad = sum.s != sum.s, none = sum.m == -INFINITY;
    const float ls = logf(sum.s);
    auto lp = [&](float x) { return bad ? NAN : none ? -INFINITY : x - sum.m - ls; };
    if (lane == 0) {
      if (a.entropy) a.entropy[row] = bad ? NAN : none ? 0.f : ls - sum.t / sum.s;
      if (a.logprob) {
        const int tok = a.tokens[row];
        float r = 0.f;
        if (tok < -1 || tok >= a.vocab) {
          set_status(a.status, PI_ERR_INDEX);
          r = NAN;
        } else if (tok >= 0) {
          r = lp(logit_at<DT>(base, tok));
        }
        a.logprob[row] = r;
      }
    }
    if (lane < a.topk) {
      a.top_idx[row * a.topk + lane] = key_index(list);
      a.top_logprob[row * a.topk + lane] = lp(key_value(list));
    }
  }
}

// Parts of a row: enough blocks to fill the GPU, each with a batch at least.
static int score_parts(int rows, int vocab, int dtype, int sms) {
  const int slots = sms * kScoreBlocks;
  int parts = rows < slots ? slots / rows : 1;
  const int batches = vocab / (kScoreThreads * kBatch * (dtype == PI_F32 ? 4 : 8));
  if (parts > batches) parts = batches;
  if (parts > kScoreParts / rows) parts = kScoreParts / rows;
  return parts > 1 ? parts : 1;
}

}  // namespace pis

using namespace pis;

extern "C" {

size_t pi_logprob_workspace_size(int32_t rows, int32_t vocab, int32_t topk) {
  if (rows < 0 || vocab < 1 || vocab > (1 << 24) || topk < 0 || topk > PI_TOPK_MAX || topk > vocab)
    return 0;
  // arrivals, zero between calls; parts' sums and lists
  return (size_t)kScoreParts * (4 + 16 + 32 * 8);
}

pi_status pi_token_logprobs(const void* logits, int32_t dtype, int32_t rows, int32_t vocab,
                            int64_t stride, const int32_t* tokens, int32_t topk, float* logprob,
                            float* entropy, int32_t* top_idx, float* top_logprob,
                            int32_t* dev_status, void* ws, size_t ws_bytes, pi_stream stream) {
  if (dtype != PI_F16 && dtype != PI_BF16 && dtype != PI_F32) return PI_ERR_DTYPE;
  const size_t need = pi_logprob_workspace_size(rows, vocab, topk);
  if (need == 0 || stride < vocab) return PI_ERR_SHAPE;
  if (!dev_status || !ws || !tokens != !logprob) return PI_ERR_NULL;
  if (rows > 0 && !logits) return PI_ERR_NULL;
  if (topk > 0 && rows > 0 && (!top_idx || !top_logprob)) return PI_ERR_NULL;
  if (!all_aligned(logits, tokens, logprob, entropy, top_idx, top_logprob, dev_status, ws))
    return PI_ERR_ALIGN;
  if (ws_bytes < need) return PI_ERR_WORKSPACE;
  if (rows == 0) return PI_OK;
  DevInfo di;
  const pi_status st = dev_info(&di);
  if (st != PI_OK) return st;
  char* w = static_cast<char*>(ws);
  ScoreArgs a{logits,  stride,      tokens,  logprob,
              entropy, top_logprob, top_idx, dev_status,
              reinterpret_cast<int*>(w),
              reinterpret_cast<float*>(w + kScoreParts * 4),
              reinterpret_cast<u64*>(w + kScoreParts * (4 + 16)),
              rows, vocab, topk, score_parts(rows, vocab, dtype, di.sms)};
  return launch(dtype == PI_F16 ? score_kernel<0> : dtype == PI_BF16 ? score_kernel<1> : score_kernel<2>,
                dim3((unsigned)rows, (unsigned)a.parts), kScoreThreads, 0, stream, a);
}

}  // extern "C"
