// logprob.cu — log probabilities of given tokens, entropy and the largest
// alternatives of rows of logits (include/pi_serve.h).
//
// Mathematics.  In units of log 2, with L = log2(e) and any reference M near
// the largest logit's L x, one pass keeps s = sum 2^d and t = sum 2^d d with
// d = L x - M.  Then log p_i = ln 2 (d_i - log2 s) and the entropy is
// ln 2 (log2 s - t / s): no large terms cancel, and since every d is one
// fused multiply-add with the same rounded M, what M and L were rounded by
// drops out.  Each thread's M follows its running maximum.
//
// Alternatives without a second pass.  Threads own disjoint sets of elements,
// so at least k elements are >= tau, the k-th largest of the maxima of 64
// sets of threads, and all of the k largest are.  Each thread leaves the
// maxima of its batches (which the sums need anyway) in shared memory, so that
// only the batches that reach tau, some k of them, are read again; their elements >= tau are
// ranked by a unique key (value, then lowest index).  Where ties make more of
// either than the block has room for, the whole part is read again: slower,
// as exact, by sorted lists of 32 keys in the lanes of a warp.  Few keys are
// ordered by counting, each thread, the keys larger than its own: one pass
// of broadcast reads instead of a chain of exchanges (128 keys at most).
//
// Bound: HBM bandwidth (each logit read once); for 16-bit logits the pass
// issues 9 instructions per logit, selection and start included (two thirds of
// the issue slots at that bandwidth), hence the packed forms (two FP32
// operations per instruction).  Few rows: a row is split over several blocks, and the last
// of them to arrive joins the parts.
//
// Measured: 4096 x 128256 bf16 with 20 alternatives 182 to 185 us, 84 % of a
// copy's 6.8 TB/s (some 20 of it the selection); 7 x 50273 fp32 with 8
// alternatives 8.3 us, a chain of reads, selection and join.  Rows with ties or
// so few finite logits that the part is read again: 4096 x 32000 fp16 with three
// allowed tokens 245 us (60 where all, 1 in 100 or 1 in 1000 are allowed).
#include "serve.cuh"

namespace pis {

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

// Threads of a block.  256 for rows that are few beside the SMs.  From
// kManyRows rows per SM on 128 with twice the blocks: while one block selects
// its alternatives, seven others read (4096 x 128256 bf16, 20 alternatives:
// 182 us against 189; x 32000 fp16: 60 against 73; but 600 rows of 128256, one
// wave of 256-thread blocks, 36 against 32).
constexpr int kManyRows = 10;
constexpr int kScoreThreads = 1024;    // resident threads per SM
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

// A maximum's rank as a thread's; 0 where it has none.
__device__ __forceinline__ uint32_t value_key(float v) { return (uint32_t)(rank_key(v, 0) >> 32); }

// ------------------------------------------------------------------ lists of 32 keys
template <typename K>
__device__ __forceinline__ K keep(K v, K w, bool larger) { return (v > w) == larger ? v : w; }

template <typename K>
__device__ __forceinline__ K merge_down(K v) {  // a bitonic sequence, sorted descending
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) v = keep(v, __shfl_xor_sync(~0u, v, j), (lane & j) == 0);
  return v;
}
template <typename K>
__device__ __forceinline__ K sort32(K v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 2; k < 32; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1)
      v = keep(v, __shfl_xor_sync(~0u, v, j), ((lane & j) == 0) == ((lane & k) == 0));
  return merge_down(v);
}
// The 32 largest of two sorted lists, sorted.
template <typename K>
__device__ __forceinline__ K merge32(K a, K b) {
  const K r = __shfl_sync(~0u, b, 31 - (threadIdx.x & 31));
  return merge_down(a > r ? a : r);
}
// The warps' lists into one, left in warp 0.
template <int WARPS, typename K>
__device__ __forceinline__ K block_merge(K v, u64 (*sh)[32]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll 1
  for (int half = WARPS / 2; half > 0; half >>= 1) {
    if (warp >= half && warp < 2 * half) sh[warp][lane] = v;
    __syncthreads();
    if (warp < half) v = merge32(v, (K)sh[warp + half][lane]);
  }
  return v;
}

// ------------------------------------------------------------------ sums
// Sums relative to the logit m (s = t = 0 for m = -infinity).
struct Sums {
  float m, s, t;
};
// L x would overflow beside the reference: differences are taken first.
__device__ __forceinline__ bool huge(float ref) { return !(fabsf(ref) < 1e38f); }
// d of a logit x.  At least -1500 (2^d is 0 below -150): keeps 0 * infinity
// out of t.  NaN stays NaN; +infinity against itself is NaN.
__device__ __forceinline__ float floor_nan(float d) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(d), "f"(-1500.f));
  return r;
}
__device__ __forceinline__ float distance(float x, float ref) {
  return huge(ref) ? (x - ref) * kLog2e : fmaf(x, kLog2e, -__fmul_rn(ref, kLog2e));
}
// The same sums relative to top >= a.m.
__device__ __forceinline__ Sums raised(const Sums& a, float top) {
  if (a.m == top) return a;
  if (a.m == -INFINITY) return Sums{top, a.s, 0.f};
  const float d = huge(top) ? (a.m - top) * kLog2e
                            : __fsub_rn(__fmul_rn(a.m, kLog2e), __fmul_rn(top, kLog2e));
  const float f = ex2(d);
  return Sums{top, a.s * f, f > 0.f ? f * fmaf(d, a.s, a.t) : 0.f};
}
__device__ __forceinline__ void add_one(Sums& a, float ref, float x) {
  const float d = floor_nan(distance(x, ref)), e = ex2(d);
  a.s += e;
  a.t = fmaf(e, d, a.t);
}

template <int DT>
struct Vec {  // 16 bytes of logits
  static constexpr int n = DT == 2 ? 4 : 8, pairs = n / 2;
  static __device__ __forceinline__ float2 get(const uint4& v, int i) {  // elements 2i, 2i + 1
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (DT == 2) return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    else if constexpr (DT == 1) return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    else return __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
  }
  // packed lower bound for logits beside a reference: 2^d is 0 there, and no
  // rounding takes it near the reference; NaN where the type cannot hold it
  static __device__ __forceinline__ uint32_t floor_at(float ref) {
    const float f = ref - (1040.f + fabsf(ref) * 0.02f);
    if constexpr (DT == 2) return __float_as_uint(f);
    if (DT == 0 && f < -65000.f) return 0x7fff7fffu;
    return pack_bits<DT>(f, f);
  }
  // the larger, NaN if one is NaN
  static __device__ __forceinline__ uint32_t raise(uint32_t a, uint32_t floor) {
    uint32_t r;
    if constexpr (DT == 2) asm("max.NaN.f32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(floor));
    else if constexpr (DT == 1) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(floor));
    else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(floor));
    return r;
  }
  static __device__ __forceinline__ uint4 raise(const uint4& v, uint32_t floor) {
    return make_uint4(raise(v.x, floor), raise(v.y, floor), raise(v.z, floor), raise(v.w, floor));
  }
  // elementwise maximum of packed values (the number where one is NaN)
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (DT == 2) r = __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    else if constexpr (DT == 1) asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ uint32_t max(const uint4& v) {
    return max(max(v.x, v.y), max(v.z, v.w));
  }
  static __device__ __forceinline__ float top(uint32_t w) {
    if constexpr (DT == 2) return __uint_as_float(w);
    return fmaxf(from_bits<DT>((uint16_t)w), from_bits<DT>((uint16_t)(w >> 16)));
  }
};

template <int N>
struct Count {
  static constexpr int value = N;
};

constexpr int kGroups = 16;  // groups of batches whose maxima a thread leaves
constexpr int kPicks = 128;  // groups, then elements, that reach tau

// One block per (row, part).
template <int DT, int T>
__global__ void __launch_bounds__(T, kScoreThreads / T) score_kernel(const ScoreArgs a) {
  using V = Vec<DT>;
  constexpr int VN = V::n, WARPS = T / 32;
  constexpr int kSets = 64;  // sets of threads whose maxima bound the k-th
  constexpr int kSize = DT == 2 ? 4 : 2;
  __shared__ u64 sh_keys[WARPS][32];
  __shared__ float sh_sums[WARPS][3];
  __shared__ float sh_top[kGroups][T];
  __shared__ uint32_t sh_group[kPicks];
  __shared__ u64 sh_pick[kPicks];
  __shared__ __align__(16) uint32_t sh_set[kSets];
  __shared__ uint32_t sh_max[T];
  __shared__ uint32_t sh_tau;
  __shared__ u64 sh_list[32];
  __shared__ int sh_groups, sh_picks, sh_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) sh_groups = sh_picks = 0;
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
  // whole vectors [w0, w1); the elements of the row's first and last, where cut,
  // go to lanes of the warps 0 and 1, which read them before all else (6294 rows
  // of 23150, fp16, one alternative: 66 us; read by one thread each at the end 80)
  const bool cut_first = v0 == 0 && shift;
  const int w0 = cut_first ? 1 : v0;
  const bool cut_last = v1 == nvec && (a.vocab + shift) % VN && nvec - 1 >= w0;
  const int w1 = cut_last ? v1 - 1 : v1;

  Sums sum{-INFINITY, 0.f, 0.f};
  bool some = false;  // an element that is not NaN
  auto raise = [&](float top) {
    if (top > sum.m) sum = raised(sum, top);
    some |= top == top;
  };
  int cut_at = -1;  // the thread's cut element
  float cut_value = NAN;
  if (lane < VN && ((warp == 0 && cut_first) || (warp == 1 && cut_last))) {
    const int i = (warp ? (nvec - 1) * VN : 0) + lane - shift;
    if (i >= 0 && i < a.vocab) {
      cut_at = i;
      cut_value = logit_at<DT>(base, i);
    }
  }
  // Batches: `whole` full ones of every thread, then what is left.
  const int nwhole = max(0, w1 - w0), whole = nwhole / (T * kBatch);
  const int left = nwhole - whole * (T * kBatch) - tid;  // the thread's vectors: tid, + T, ... < left + tid
  const int steps = whole + (nwhole > whole * T * kBatch);
  const uint4* mine = vecs + w0 + tid;
  // batches of a group: the least power of two that kGroups groups suffice for
  const int group_shift = 32 - __clz((max(steps, 1) - 1) / kGroups), group = 1 << group_shift;
  float group_top = NAN;
  auto leave = [&](int it, float top) {
    group_top = it & (group - 1) ? fmaxf(group_top, top) : top;
    sh_top[it >> group_shift][tid] = group_top;
  };
  uint4 raw[kBatch];
  auto load = [&](int it) {
    const uint4* p = mine + it * (T * kBatch);
    if (it < whole) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) raw[u] = __ldg(p + u * T);
    } else {
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (u * T < left) raw[u] = __ldg(p + u * T);
    }
  };
  // Sums of N vectors beside ref, packed where the type can hold the floor.
  auto add = [&](const uint4* v, auto n) {
    constexpr int N = decltype(n)::value;
    const float ref = sum.m == -INFINITY ? 0.f : sum.m;
    const uint32_t low = V::floor_at(ref);
    if (!huge(ref) && (DT != 0 || low != 0x7fff7fffu)) {
      const float M = -__fmul_rn(ref, kLog2e);
      const u64 L2 = pair(kLog2e, kLog2e), M2 = pair(M, M);
      u64 s2 = 0, t2 = 0;
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const uint4 q = V::raise(v[u], low);
#pragma unroll
        for (int p = 0; p < V::pairs; ++p) {
          const float2 x = V::get(q, p);
          const u64 d2 = fma2(pair(x.x, x.y), L2, M2);
          const float2 d = halves(d2);
          const u64 e = pair(ex2(d.x), ex2(d.y));
          s2 = add2(s2, e);
          t2 = fma2(e, d2, t2);
        }
      }
      const float2 s = halves(s2), t = halves(t2);
      sum.s += s.x + s.y;
      sum.t += t.x + t.y;
    } else {
#pragma unroll
      for (int u = 0; u < N; ++u)
#pragma unroll 1
        for (int p = 0; p < V::pairs; ++p) {
          const float2 x = V::get(v[u], p);
          add_one(sum, ref, x.x);
          add_one(sum, ref, x.y);
        }
    }
  };
  if (steps > 0) load(0);
#pragma unroll 1
  for (int it = 0; it < whole; ++it) {
    uint4 v[kBatch];
    uint32_t w[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      v[u] = raw[u];
      w[u] = V::max(v[u]);
    }
    if (it + 1 < steps) load(it + 1);
    const float top = V::top(V::max(V::max(w[0], w[1]), V::max(w[2], w[3])));
    leave(it, top);
    raise(top);
    add(v, Count<kBatch>());
  }
  if (steps > whole) {
    float top = NAN;
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (u * T < left) top = fmaxf(top, V::top(V::max(raw[u])));
    leave(whole, top);
    raise(top);
#pragma unroll 1
    for (int u = 0; u * T < left; ++u) {
      const uint4 q = u == 0 ? raw[0] : u == 1 ? raw[1] : u == 2 ? raw[2] : raw[3];
      add(&q, Count<1>());
    }
  }
  if (cut_at >= 0) {
    raise(cut_value);
    add_one(sum, sum.m == -INFINITY ? 0.f : sum.m, cut_value);
  }

  // the block's sums
  float top = sum.m;
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  if (lane == 0) sh_sums[warp][0] = top;
  if (a.topk > 0) sh_max[tid] = some ? value_key(sum.m) : 0u;  // 0: only NaN, or nothing
  __syncthreads();
  if (a.topk > 0 && tid < kSets) {  // set s: the threads s, s + 64, ...
    uint32_t k = sh_max[tid];
#pragma unroll
    for (int o = kSets; o < T; o += kSets) k = max(k, sh_max[tid + o]);
    sh_set[tid] = k;
    asm volatile("bar.sync 1, %0;" ::"n"(kSets) : "memory");  // the first two warps
    int ahead = 0;  // the one with topk - 1 ahead of it
#pragma unroll 4
    for (int i = 0; i < kSets; i += 4) {
      const uint4 o = *reinterpret_cast<const uint4*>(sh_set + i);
      ahead += (o.x > k || (o.x == k && i < tid)) + (o.y > k || (o.y == k && i + 1 < tid)) +
               (o.z > k || (o.z == k && i + 2 < tid)) + (o.w > k || (o.w == k && i + 3 < tid));
    }
    if (ahead == a.topk - 1) sh_tau = k;
  }
#pragma unroll
  for (int w = 0; w < WARPS; ++w) top = fmaxf(top, sh_sums[w][0]);
  {
    const Sums up = raised(sum, top);
    const float s = warp_sum(up.s), t = warp_sum(up.t);
    if (lane == 0) {
      sh_sums[warp][1] = s;
      sh_sums[warp][2] = t;
    }
  }

  auto order = [&](const u64* keys, int n) {  // the first 32 of n <= T keys into sh_list
    if (tid >= n) return;
    const u64 k = keys[tid];
    int ahead = 0;
#pragma unroll 4
    for (int i = 0; i < n; ++i) ahead += keys[i] > k;
    if (ahead < 32) sh_list[ahead] = k;
  };
  u64 list = 0;  // warp 0: the 32 largest keys (only the first topk count)
  if (a.topk > 0) {
    __syncthreads();
    const uint32_t tau = sh_tau;
    const float tau_value = key_value((u64)tau << 32);
    u64 least = (u64)tau << 32;  // a key that enters is larger
    auto enter = [&](u64 k) {
      if (__any_sync(~0u, k > least)) {
        list = merge32(list, sort32(k > least ? k : (u64)0));
        const u64 kth = __shfl_sync(~0u, list, a.topk - 1);
        least = kth > least ? kth : least;
      }
    };
    auto pick = [&](float x, int i) {
      if (!(x >= tau_value)) return;
      const int n = atomicAdd(&sh_picks, 1);
      if (n < kPicks) sh_pick[n] = rank_key(x, i);
    };
    bool all = tau == 0;  // then everything counts, NaN too
    if (!all) {
      for (int q = 0; q << group_shift < steps; ++q)
        if (sh_top[q][tid] >= tau_value) {
          const int i = atomicAdd(&sh_groups, 1);
          if (i < kPicks) sh_group[i] = (uint32_t)(q * T + tid);
        }
      __syncthreads();
      const int groups = sh_groups, per = group * kBatch, items = groups * per;
      all = groups > kPicks;
      if (!all)
        for (int i = tid; i < items; i += T) {
          const int q = i / per;
          const uint32_t who = sh_group[q];
          const int j = w0 + (int)(who % T) + ((int)(who / T) * per + (i - q * per)) * T;
          if (j >= w1) continue;
          const uint4 v = __ldg(vecs + j);
          if (!(V::top(V::max(v)) >= tau_value)) continue;
#pragma unroll
          for (int p = 0; p < V::pairs; ++p) {
            const float2 x = V::get(v, p);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              pick(h ? x.y : x.x, j * VN + 2 * p + h - shift);
            }
          }
        }
      if (cut_at >= 0) pick(cut_value, cut_at);
      __syncthreads();
      const int picks = sh_picks;
      all |= picks > kPicks;
      if (!all) {
        order(sh_pick, picks);
        __syncthreads();
        if (warp == 0) list = lane < picks ? sh_list[lane] : 0;
      }
    }
    if (all) {
      for (int j0 = w0 + warp * 32; j0 < w1; j0 += T) {
        const bool in = j0 + lane < w1;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (in) v = __ldg(vecs + j0 + lane);
        if (!__any_sync(~0u, in && (tau == 0 || V::top(V::max(v)) >= tau_value))) continue;
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll 1
        for (int e = 0; e < VN; ++e) {
          float x;
          if constexpr (DT == 2) x = __uint_as_float(w[e]);
          else x = from_bits<DT>((uint16_t)(w[e >> 1] >> (16 * (e & 1))));
          enter(in ? rank_key(x, (j0 + lane) * VN + e - shift) : 0);
        }
      }
      list = block_merge<WARPS>(list, sh_keys);
      if (warp == 0 && cut_first) {
        const int i = lane - shift;
        enter(lane < VN && i >= 0 && i < a.vocab ? rank_key(logit_at<DT>(base, i), i) : 0);
      }
      if (warp == 0 && cut_last) {
        const int i = (nvec - 1) * VN + lane - shift;
        enter(lane < VN && i >= 0 && i < a.vocab ? rank_key(logit_at<DT>(base, i), i) : 0);
      }
    }
  }
  __syncthreads();
  if (warp == 0) {
    sum = Sums{top, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
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
    // all parts: the sums by one warp, the lists by all
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
      for (int p = warp; p < a.parts; p += WARPS)
        list = merge32(list, __ldcg(a.pkeys + (row * a.parts + p) * 32 + lane));
      list = block_merge<WARPS>(list, sh_keys);
    }
  }

  if (warp == 0) {
    const bool bad = sum.s != sum.s, none = sum.m == -INFINITY;
    const float ls = log2f(sum.s);
    auto lp = [&](float x) {
      return bad ? NAN : none ? -INFINITY : (distance(x, sum.m) - ls) * kLn2;
    };
    if (lane == 0) {
      if (a.entropy) a.entropy[row] = bad ? NAN : none ? 0.f : (ls - sum.t / sum.s) * kLn2;
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
  const int slots = sms * (kScoreThreads / 256);
  int parts = rows < slots ? slots / rows : 1;
  const int batches = vocab / (256 * kBatch * (dtype == PI_F32 ? 4 : 8));
  if (parts > batches) parts = batches;
  if (parts > kScoreParts / rows) parts = kScoreParts / rows;
  return parts > 1 ? parts : 1;
}

template <int T>
static pi_status launch_score(const ScoreArgs& a, int dtype, pi_stream stream) {
  return launch(dtype == PI_F16    ? score_kernel<0, T>
                : dtype == PI_BF16 ? score_kernel<1, T>
                                   : score_kernel<2, T>,
                dim3((unsigned)a.rows, (unsigned)a.parts), T, 0, stream, a);
}

}  // namespace pis

using namespace pis;

extern "C" {

size_t pi_logprob_workspace_size(int32_t rows, int32_t vocab, int32_t topk) {
  if (rows < 0 || vocab < 1 || vocab > (1 << 24) || topk < 0 || topk > PI_TOPK_MAX || topk > vocab)
    return 0;
  // arrivals, zero between calls; parts' sums and lists
  static_assert(kScoreParts * 4 == kCounters, "one workspace may serve several calls");
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
  return rows >= kManyRows * di.sms ? launch_score<128>(a, dtype, stream)
                                    : launch_score<256>(a, dtype, stream);
}

}  // extern "C"
