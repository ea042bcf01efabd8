// sample.cu — tokens drawn from rows of logits by temperature, top-k, min-p and
// top-p with given random numbers (include/pi_draft.h).
//
// Mathematics.  With M the largest logit, the weight of x is 2^-t, t = (M - x)
// log2(e) / T.  The draw is a place in the running sum of the weights in
// descending order, and so is the end of what top-p keeps, so sums have to be
// those of 64 bits: two borders of a vocabulary lie 1e-6 apart or less.  64-bit
// arithmetic per logit is out of the question here (2 operations per SM and cycle),
// so t is a sum of two fp32 numbers, split into a bin b = floor(32 t) and a rest
// r in [0, 1/32), and 2^-r = 1 - q with q < 0.0215 is a 36-bit fixed-point number:
// z = r ln 2 and z^2 / 2 of the series of 1 - e^-z as sums of two fp32 numbers, the
// rest (2^-19) in one.  A bin's weight is 2^(-b/32) (count - sum q): whole-number
// sums, the same in any order, and one product of 64 bits per bin, not per logit.  The
// sums over bins have 128 bits, with 2^-99 of the largest weight as their unit: cut to
// 64 bits, a vocabulary of 2^24 would leave weights below 2^-37 nothing.
//
// Order without sorting.  Running sums over the 2048 bins (64 octaves; what lies
// below weighs nothing) say in which bin a border lies.  The bin's logits alone are
// collected, ordered by (logit, index) and gone through.  Where ties make them more
// than the list holds, the bin is divided again by the bits of that key.  Rows that
// top-k or min-p leave few logits of need no sums: they are counted by bin, and the
// list holds all that are kept (1024 x 128256 fp32, such rows three of five: 575 us).
//
// A row is a thread-block cluster's.  Its logits stay in the cluster's shared
// memory, so that memory is read once, and few rows still use many SMs.  Rows
// that do not fit are read again from global memory.
//
// Bound: instructions, some 50 per logit for its weight and bin, on one block of 1024
// threads per SM, which issues in 60 % of its cycles: barriers between the phases take
// the rest.  Measured: 832 x 50272 fp16 without filters 202 us (memory 12), 64 x 128256 bf16
// 47 to 60 us, 1 x 50273 fp32 21 to 25 us: a chain of eleven phases of a cluster.
#include <cooperative_groups.h>

#include "sample_weight.cuh"
#include "serve.cuh"

namespace pis {

namespace cg = cooperative_groups;

struct SampleArgs {
  const void* logits;
  long long stride;
  const float *temperature, *top_p, *min_p, *u;
  const int* top_k;
  int* token;
  float* logprob;
  int* status;
  int rows, vocab;
  int held;  // the row's logits fit the cluster's shared memory
};

constexpr int kSampleThreads = 1024;
constexpr int kBinsPerThread = kBins / kSampleThreads;
constexpr int kList = 1024;          // logits that are ordered at once
constexpr uint32_t kBias = 1u << 20; // of q, which rounding may take below 0

typedef unsigned __int128 u128;

// A bin's logits: their number and the sum of q + kBias.
struct Bins {
  uint32_t count[kBins], low[kBins], high[kBins];
};
struct SampleShared {
  Bins local, total;
  u64 list[kList], spare[kList];
  u128 scan[kSampleThreads / 32];
  u64 scale[kBinsPerOctave];  // 2^(63 - i/32)
  float warp_top[kSampleThreads / 32];
  float top, least;  // this block's maximum; the row's least logit that min-p keeps
  int bad, first;    // NaN or +infinity; lowest index of the row's maximum
  int list_n;
  // where a border was found: its bin, the sums before it, what is in it
  int at_bin;
  u128 before_w, at_upto;  // at_upto: the sum up to its logit
  u64 before_n, before_q, inside_n, at_key;
};

template <int DT>
__device__ __forceinline__ float sample_at(const void* p, long long i) {
  if (DT == 2) return static_cast<const float*>(p)[i];
  return from_bits<DT>(static_cast<const uint16_t*>(p)[i]);
}

// Descending logits, equal ones (-0 = +0) by ascending index: ascending keys.
__device__ __forceinline__ u64 order_key(float v, int i) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return ((u64)(b & 0x80000000u ? b : ~(b | 0x80000000u)) << 32) | (uint32_t)i;
}
__device__ __forceinline__ float key_logit(u64 k) {
  const uint32_t b = (uint32_t)(k >> 32);
  return __uint_as_float(b & 0x80000000u ? b : ~b & 0x7fffffffu);
}

__device__ __forceinline__ void bin_add(Bins& h, int b, int q) {
  const uint32_t v = (uint32_t)q + kBias;
  atomicAdd(&h.count[b], 1u);
  if (atomicAdd(&h.low[b], v) > ~v) atomicAdd(&h.high[b], 1u);
}
// A bin's weights as a whole number: kOne each, less q.
__device__ __forceinline__ u64 bin_sum(const Bins& h, int b) {
  const u64 n = h.count[b], q = ((u64)h.high[b] << 32) + h.low[b];
  return n * ((u64)kOne + kBias) - q;
}

__device__ __forceinline__ u64 shfl_from(u64 v, int l) { return __shfl_sync(~0u, v, l); }
__device__ __forceinline__ u128 shfl_from(u128 v, int l) {
  return (u128)__shfl_sync(~0u, (u64)(v >> 64), l) << 64 | __shfl_sync(~0u, (u64)v, l);
}
__device__ __forceinline__ double as_double(u128 v) { return (double)(u64)(v >> 64) * 0x1p64 + (double)(u64)v; }

// floor(f sum), or (up) the least whole number not below f sum, 1 at least, for 0 <= f < 1
// and sums below 2^124: exact, by f's 24 bits.  Below 2^-40 f counts as 0: the largest
// logit alone weighs more than that of any row.
__device__ __forceinline__ u128 part_of(float f, u128 sum, bool up) {
  const uint32_t bits = __float_as_uint(f), s = 150 - (bits >> 23);  // f = m 2^-s
  if (s > 63) return up;
  const uint32_t m = (bits & 0x7fffffu) | 0x800000u;
  const u128 low = (u128)m * (u64)sum, high = (u128)m * (u64)(sum >> 64) + (u64)(low >> 64);
  const u64 rest = (u64)low & ((1ull << s) - 1);
  return (high << (64 - s)) + ((u64)low >> s) + (up && rest ? 1 : 0);
}

// Sorts list[0, n), n <= kList, ascending, a key per thread: few by counting the
// smaller ones, more by a bitonic network whose short steps are exchanges in a warp and
// whose others go through list and spare in turn.
__device__ __forceinline__ void sort_list(u64* list, u64* spare, int n) {
  static_assert(kList == kSampleThreads, "a key per thread");
  const int tid = threadIdx.x;
  if (n <= 384) {
    if (tid < n) {
      const u64 v = list[tid];
      int less = 0;
#pragma unroll 4
      for (int i = 0; i < n; ++i) less += list[i] < v;
      spare[less] = v;
    }
    __syncthreads();
    if (tid < n) list[tid] = spare[tid];
    __syncthreads();
    return;
  }
  int size = 32;
  while (size < n) size *= 2;
  u64 v = tid < n ? list[tid] : ~0ull;
  u64 *to = spare, *other = list;
  __syncthreads();
  for (int k = 2; k <= size; k *= 2) {
    const bool up = (tid & k) == 0;
    for (int j = k / 2; j >= 32; j /= 2) {
      to[tid] = v;
      __syncthreads();
      const u64 w = to[tid ^ j];
      v = ((tid & j) == 0) == up ? (v < w ? v : w) : (v > w ? v : w);
      u64* const t = to;
      to = other;
      other = t;
    }
    if ((tid & ~31) < size)
      for (int j = min(k / 2, 16); j > 0; j /= 2) {
        const u64 w = __shfl_xor_sync(~0u, v, j);
        v = ((tid & j) == 0) == up ? (v < w ? v : w) : (v > w ? v : w);
      }
  }
  __syncthreads();
  if (tid < n) list[tid] = v;
  __syncthreads();
}

// One cluster per row (and those after it).
template <int DT>
__global__ void __launch_bounds__(kSampleThreads, 1) sample_kernel(const __grid_constant__ SampleArgs a) {
  constexpr int T = kSampleThreads, kSize = DT == 2 ? 4 : 2, VN = 16 / kSize;
  extern __shared__ __align__(16) unsigned char smem[];
  SampleShared& S = *reinterpret_cast<SampleShared*>(smem);
  unsigned char* const cache = smem + (sizeof(SampleShared) + 15) / 16 * 16;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_enter();
  if (tid < kBinsPerOctave) S.scale[tid] = (u64)(exp2(-(double)tid / kBinsPerOctave) * 0x1p63);
  // A sum of whole-number weights of bin b, at most 2^24 2^36, in units of 2^-99 of the
  // largest weight: bins of 64 octaves keep the bits that their logits have.
  auto weight = [&](u64 sum, int b) {
    return (u128)sum * S.scale[b & (kBinsPerOctave - 1)] >> (b / kBinsPerOctave);
  };

  // 64 bits: up to 2^31 - 1 rows, and a step of up to 2^20 past the last
  for (long long row = blockIdx.x / C; row < a.rows; row += gridDim.x / C) {
    cluster.sync();  // the last row's results are read
    float temp = a.temperature ? __ldg(a.temperature + row) : 1.f;
    const float u = __ldg(a.u + row);
    const float top_p = a.top_p ? __ldg(a.top_p + row) : 1.f, min_p = a.min_p ? __ldg(a.min_p + row) : 0.f;
    const int top_k = a.top_k ? __ldg(a.top_k + row) : 0;
    const bool good = temp >= 0.f && temp < INFINITY && u >= 0.f && u < 1.f && top_p >= 0.f && min_p >= 0.f &&
                      min_p <= 1.f;
    // the block's vectors [v0, v1) of the row: whole and aligned but at the row's ends
    const char* base = static_cast<const char*>(a.logits) + row * a.stride * kSize;
    const int shift = (int)(reinterpret_cast<uintptr_t>(base) & 15) / kSize;
    const int nvec = (a.vocab + shift + VN - 1) / VN;
    const int v0 = (int)((long long)rank * nvec / C), v1 = (int)((long long)(rank + 1) * nvec / C);
    const uint4* vecs = reinterpret_cast<const uint4*>(base - shift * kSize);
    // f(logit, index) for each
    auto each = [&](auto f) {
      const uint4* from = a.held ? reinterpret_cast<const uint4*>(cache) - v0 : vecs;
      for (int v = v0 + tid; v < v1; v += T) {
        const int at = v * VN - shift;
        if (at >= 0 && at + VN <= a.vocab) {
          const uint4 w = from[v];
#pragma unroll
          for (int i = 0; i < VN; ++i) f(sample_at<DT>(&w, i), at + i);
        } else {
          for (int i = max(0, -at); i < VN && at + i < a.vocab; ++i) f(sample_at<DT>(base, at + i), at + i);
        }
      }
    };

    // ---- the maximum, and the logits into shared memory
    float top = -INFINITY;
    bool bad = false;
    for (int v = v0 + tid; v < v1; v += T) {
      const int at = v * VN - shift;
      if (at >= 0 && at + VN <= a.vocab) {
        const uint4 w = __ldg(vecs + v);
        if (a.held) reinterpret_cast<uint4*>(cache)[v - v0] = w;
#pragma unroll
        for (int i = 0; i < VN; ++i) {
          const float x = sample_at<DT>(&w, i);
          bad |= !(x < INFINITY);
          top = fmaxf(top, x);
        }
      } else {
        for (int i = max(0, -at); i < VN && at + i < a.vocab; ++i) {
          const float x = sample_at<DT>(base, at + i);
          bad |= !(x < INFINITY);
          top = fmaxf(top, x);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    if (lane == 0) S.warp_top[warp] = top;
    bad = __syncthreads_or(bad);
    if (tid == 0) {
      for (int w = 1; w < T / 32; ++w) top = fmaxf(top, S.warp_top[w]);
      S.top = top;
      S.bad = bad;
      S.first = a.vocab;
      S.list_n = 0;
    }
    for (int b = tid; b < kBins; b += T) S.local.count[b] = S.local.low[b] = S.local.high[b] = 0;
    cluster.sync();
    bad = false;
    for (int r = 0; r < C; ++r) {
      const SampleShared& o = *cluster.map_shared_rank(&S, r);
      top = r ? fmaxf(top, o.top) : o.top;
      bad |= o.bad;
    }
    if (!good || bad || top == -INFINITY) {  // the same in every block
      if (rank == 0 && tid == 0) {
        a.token[row] = -1;
        if (a.logprob) a.logprob[row] = NAN;
        set_status(a.status, PI_ERR_RANGE);
      }
      continue;
    }
    if (temp == 0.f || top_k == 1) {
      int first = a.vocab;
      each([&](float x, int i) { first = x == top ? min(first, i) : first; });
      first = (int)__reduce_min_sync(~0u, (uint32_t)first);
      if (lane == 0) atomicMin(&S.first, first);
      cluster.sync();
      if (rank == 0 && tid == 0) {
        for (int r = 0; r < C; ++r) first = min(r ? first : a.vocab, cluster.map_shared_rank(&S, r)->first);
        a.token[row] = first;
        if (a.logprob) a.logprob[row] = 0.f;
      }
      continue;
    }
    temp = fmaxf(temp, 1e-30f);
    if (tid == 0) S.least = min_p > 0.f ? __double2float_ru(top + (double)temp * log((double)min_p)) : -INFINITY;
    __syncthreads();
    Weights W;
    W.set(top, temp, S.least);

    // ---- bins: sums of every block's
    auto bins_of = [&](bool sums, auto which) {  // which(x, i): bin, or kBins; q is that of x's own bin
      if (sums)
        each([&](float x, int i) {
          const int own = W.bin(x);
          if (own < kBins) {
            const int b = which(x, i, own);
            if (b < kBins) bin_add(S.local, b, W.q(x, own));
          }
        });
      else
        each([&](float x, int) {
          const int own = W.bin(x);
          if (own < kBins) atomicAdd(&S.local.count[own], 1u);
        });
      cluster.sync();
      for (int b = rank * T + tid; b < kBins; b += C * T) {
        uint32_t n = 0, h = 0;
        u64 low = 0;
        for (int r = 0; r < C; ++r) {
          const Bins& o = cluster.map_shared_rank(&S, r)->local;
          n += o.count[b];
          low += o.low[b];
          h += o.high[b];
        }
        h += (uint32_t)(low >> 32);
        for (int r = 0; r < C; ++r) {
          Bins& o = cluster.map_shared_rank(&S, r)->total;
          o.count[b] = n;
          o.low[b] = (uint32_t)low;
          o.high[b] = h;
        }
      }
      cluster.sync();
      for (int b = tid; b < kBins; b += T) S.local.count[b] = S.local.low[b] = S.local.high[b] = 0;
      __syncthreads();
    };
    // Exclusive sums over the threads; returns the sum of all.
    auto scan_n = [&](auto v, auto& before) {
      static_assert(T / 32 == 32, "a lane per warp");
      auto in_warp = [&](auto x) {  // inclusive
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const auto w = shfl_from(x, lane - o);
          if (lane >= o) x += w;
        }
        return x;
      };
      const auto upto = in_warp(v);
      if (lane == 31) S.scan[warp] = upto;
      __syncthreads();
      const auto warps = in_warp((decltype(v))S.scan[lane]);
      __syncthreads();
      before = upto - v + (warp ? shfl_from(warps, warp - 1) : 0);
      return shfl_from(warps, 31);
    };
    auto weight_of = [&](u64 key) {  // of one logit
      const float x = key_logit(key);
      const int b = W.bin(x);
      return weight((u64)kOne - (long long)W.q(x, b), b);
    };
    auto finish = [&](u64 key, u128 sum) {
      a.token[row] = (int)(uint32_t)key;
      if (a.logprob) {
        const double p = as_double(weight_of(key)) / as_double(sum);
        a.logprob[row] = p > 0.5 ? log1pf((float)(p - 1.0)) : logf((float)p);
      }
    };
    // ---- few logits are kept before top-p: those alone, in one list
    if ((top_k > 0 && top_k <= kList) || min_p > 0.f) {
      bins_of(false, [&](float, int, int own) { return own; });
      u64 n = 0, before;
      for (int k = 0; k < kBinsPerThread; ++k) n += S.total.count[tid * kBinsPerThread + k];
      const u64 all = scan_n(n, before), want = top_k > 0 && (u64)top_k < all ? (u64)top_k : all;
      for (int k = 0; k < kBinsPerThread && before < want; ++k) {
        const int b = tid * kBinsPerThread + k;
        const u64 c = S.total.count[b];
        if (before + c >= want && c) {
          S.at_bin = b;
          S.inside_n = before + c;
        }
        before += c;
      }
      __syncthreads();
      const int bin = S.at_bin;
      if (S.inside_n <= kList) {  // the same in every block
        SampleShared& F = *cluster.map_shared_rank(&S, 0);
        each([&](float x, int i) {
          if (W.bin(x) <= bin) {
            const int at = atomicAdd(&F.list_n, 1);
            if (at < kList) F.list[at] = order_key(x, i);
          }
        });
        cluster.sync();
        if (rank == 0) {
          sort_list(S.list, S.spare, (int)S.inside_n);
          constexpr int each_n = kList / T;
          u128 v[each_n], mine = 0, v0;
          for (int k = 0; k < each_n; ++k) {
            const int i = tid * each_n + k;
            v[k] = i < (int)want ? weight_of(S.list[i]) : 0;
            mine += v[k];
          }
          u128 sum = scan_n(mine, v0);
          const u128 ahead = v0;
          auto find = [&](u128 target) {  // the place where the running sum reaches it: S.at_key, ...
            v0 = ahead;
            for (int k = 0; k < each_n; ++k) {
              if (v0 < target && v0 + v[k] >= target) {
                S.at_key = S.list[tid * each_n + k];
                S.at_upto = v0 + v[k];
              }
              v0 += v[k];
            }
            __syncthreads();
          };
          if (top_p < 1.f) {
            find(part_of(top_p, sum, true));
            sum = S.at_upto;
            __syncthreads();
          }
          find(part_of(u, sum, false) + 1);
          if (tid == 0) finish(S.at_key, sum);
        }
        continue;
      }
      __syncthreads();
    }
    bins_of(true, [&](float, int, int own) { return own; });

    // The bins' running sums: those before the thread's bins, and of all.
    u64 bins_n, row_n;
    u128 bins_w, row_w;
    auto thread_sums = [&](auto f, u64& before_n, u64& all_n, auto& before_w, auto& all_w) {
      u64 n = 0;
      auto w = all_w;
      w = 0;
      for (int k = 0; k < kBinsPerThread; ++k) {
        const int b = tid * kBinsPerThread + k;
        if (!S.total.count[b]) continue;
        n += S.total.count[b];
        w += f(b);
      }
      all_n = scan_n(n, before_n);
      all_w = scan_n(w, before_w);
    };
    row_w = 0;
    thread_sums([&](int b) { return weight(bin_sum(S.total, b), b); }, bins_n, row_n, bins_w, row_w);
    bool whole = true;  // S.total holds the bins of all logits
    // Finds the logit at which the running count (COUNT) or sum reaches
    // `target`, 1 .. that of the row: S.at_key and S.at_upto.
    auto locate = [&](bool count, u128 target) {
      if (!whole) {
        bins_of(true, [&](float, int, int own) { return own; });
        whole = true;
      }
      {
        u64 n = bins_n;
        u128 w = bins_w;
        for (int k = 0; k < kBinsPerThread && (count ? n : w) < target; ++k) {
          const int b = tid * kBinsPerThread + k;
          const u64 c = S.total.count[b];
          if (!c) continue;
          const u128 next = w + weight(bin_sum(S.total, b), b);
          if ((count ? n + c : next) >= target) {
            S.at_bin = b;
            S.before_n = n;
            S.before_w = w;
            S.inside_n = c;
          }
          n += c;
          w = next;
        }
      }
      __syncthreads();
      const int bin = S.at_bin;
      const u128 before_w = S.before_w;
      u64 before_n = S.before_n, before_q = 0, inside = S.inside_n;
      __syncthreads();
      // keys [lo, lo + size), divided until few logits are left
      u64 lo = 0, size = ~0ull;
      while (inside > kList) {
        whole = false;
        const int sh = max(0, 64 - 11 - __clzll(size));  // 2048 parts
        bins_of(true, [&](float x, int i, int own) {
          const u64 k = order_key(x, i) - lo;
          return own == bin && k < size ? (int)(k >> sh) : kBins;
        });
        u64 n, q, all_n, all_q = 0;
        thread_sums([&](int b) { return bin_sum(S.total, b); }, n, all_n, q, all_q);
        n += before_n;
        q += before_q;
        for (int k = 0; k < kBinsPerThread && (count ? n : before_w + weight(q, bin)) < target; ++k) {
          const int b = tid * kBinsPerThread + k;
          const u64 c = S.total.count[b], next = q + bin_sum(S.total, b);
          if (!c) continue;
          if ((count ? n + c : before_w + weight(next, bin)) >= target) {
            S.at_bin = b;
            S.before_n = n;
            S.before_q = q;
            S.inside_n = c;
          }
          n += c;
          q = next;
        }
        __syncthreads();
        lo += (u64)S.at_bin << sh;
        size = 1ull << sh;
        before_n = S.before_n;
        before_q = S.before_q;
        inside = S.inside_n;
        __syncthreads();
      }
      // the logits themselves, into the first block's list
      SampleShared& F = *cluster.map_shared_rank(&S, 0);
      each([&](float x, int i) {
        if (W.bin(x) == bin) {
          const u64 k = order_key(x, i);
          if (k - lo < size) {
            const int at = atomicAdd(&F.list_n, 1);
            if (at < kList) F.list[at] = k;
          }
        }
      });
      cluster.sync();
      if (rank == 0) {
        const int n = min(S.list_n, kList);
        sort_list(S.list, S.spare, n);
        constexpr int each_n = kList / T;
        u64 q[each_n], mine = 0, q0;
#pragma unroll
        for (int k = 0; k < each_n; ++k) {
          const int i = tid * each_n + k;
          q[k] = i < n ? (u64)kOne - (long long)W.q(key_logit(S.list[i]), bin) : 0;
          mine += q[k];
        }
        scan_n(mine, q0);
        q0 += before_q;
#pragma unroll
        for (int k = 0; k < each_n; ++k) {
          const int i = tid * each_n + k;
          const u128 was = count ? before_n + i : before_w + weight(q0, bin);
          const u128 is = count ? before_n + i + 1 : before_w + weight(q0 + q[k], bin);
          if (i < n && was < target && is >= target) {
            S.at_key = S.list[i];
            S.at_upto = before_w + weight(q0 + q[k], bin);
          }
          q0 += q[k];
        }
        __syncthreads();
        if (tid == 0) {
          S.list_n = 0;
          for (int r = 1; r < C; ++r) {
            SampleShared& o = *cluster.map_shared_rank(&S, r);
            o.at_key = S.at_key;
            o.at_upto = S.at_upto;
          }
        }
      }
      cluster.sync();
    };

    u128 sum = row_w;
    if (top_k > 0 && (u64)top_k < row_n) {
      locate(true, top_k);
      sum = S.at_upto;
    }
    if (top_p < 1.f) {
      locate(false, part_of(top_p, sum, true));
      sum = S.at_upto;
    }
    locate(false, part_of(u, sum, false) + 1);
    if (rank == 0 && tid == 0) finish(S.at_key, sum);
  }
  cluster.sync();  // no block leaves while another reads its memory
}

// Blocks of a row's cluster: as many as its logits need, and more while SMs are idle and a
// block has more than 4096 logits left (1 x 50273 fp32: 25.3 us; from 1024 on 27.1, from
// 16384 on 27.9).
static int sample_cluster(int rows, int vocab, int size, int sms, int room) {
  int c = 1;
  while (c < 8 && (long long)vocab * size > (long long)c * (room - 64)) c *= 2;
  while (c < 8 && (long long)rows * c * 2 <= sms && vocab / c > 4096) c *= 2;
  return c;
}

template <int DT>
static pi_status launch_sample(SampleArgs a, pi_stream stream) {
  DevInfo di;
  pi_status st = dev_info(&di);
  if (st != PI_OK) return st;
  constexpr int size = DT == 2 ? 4 : 2, fixed = (sizeof(SampleShared) + 15) / 16 * 16;
  const int room = di.smem_optin - fixed;
  const int c = sample_cluster(a.rows, a.vocab, size, di.sms, room);
  const int need = (int)(((long long)a.vocab * size / 16 + 3) / c + 2) * 16;
  a.held = (long long)a.vocab * size <= (long long)c * (room - 64) && need <= room;
  const int smem = fixed + (a.held ? need : 0);
  st = ensure_smem(reinterpret_cast<const void*>(sample_kernel<DT>), di.smem_optin);
  if (st != PI_OK) return st;
  cudaLaunchConfig_t cfg = {};
  const long long rows = a.rows < (1 << 20) ? a.rows : 1 << 20;
  cfg.gridDim = dim3((unsigned)(rows * c));
  cfg.blockDim = dim3(kSampleThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = c;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sample_kernel<DT>, a) == cudaSuccess ? PI_OK : PI_ERR_CUDA;
}

}  // namespace pis

using namespace pis;

extern "C" {

size_t pi_sample_workspace_size(int32_t rows, int32_t vocab) {
  return rows < 0 || vocab < 1 || vocab > (1 << 24) ? 0 : kAlign;
}

pi_status pi_token_sample(const void* logits, int32_t dtype, int32_t rows, int32_t vocab, int64_t stride,
                          const float* temperature, const int32_t* top_k, const float* top_p,
                          const float* min_p, const float* u, int32_t* token, float* logprob,
                          int32_t* dev_status, void* ws, size_t ws_bytes, pi_stream stream) {
  if (dtype != PI_F16 && dtype != PI_BF16 && dtype != PI_F32) return PI_ERR_DTYPE;
  if (rows < 0 || vocab < 1 || vocab > (1 << 24) || stride < vocab) return PI_ERR_SHAPE;
  if (!dev_status || !ws || (rows > 0 && (!logits || !u || !token))) return PI_ERR_NULL;
  if (!all_aligned(logits, temperature, top_k, top_p, min_p, u, token, logprob, dev_status, ws)) return PI_ERR_ALIGN;
  if (ws_bytes < pi_sample_workspace_size(rows, vocab)) return PI_ERR_WORKSPACE;
  if (rows == 0) return PI_OK;
  SampleArgs a{logits, stride, temperature, top_p, min_p, u, top_k, token, logprob, dev_status, rows, vocab, 0};
  return dtype == PI_F16 ? launch_sample<0>(a, stream)
                         : dtype == PI_BF16 ? launch_sample<1>(a, stream) : launch_sample<2>(a, stream);
}

}  // extern "C"
