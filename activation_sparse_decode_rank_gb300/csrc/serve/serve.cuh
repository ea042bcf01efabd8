// serve.cuh — what the serving operators (declared in include/pi_serve.h)
// share: argument checks, workspace layout, launches, small device helpers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>
#include <unordered_map>
#include <utility>

#include "../../../include/pi_serve.h"

namespace pis {

// ------------------------------------------------------------------ host
constexpr size_t kAlign = 256;
constexpr int kMaxHeads = 1024;

inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename... Ps>
bool all_aligned(Ps... ps) {
  return (aligned16(ps) && ...);
}

inline pi_status check_cache(const pi_cache_desc* C) {
  if (!C) return PI_ERR_NULL;
  if (C->dtype != PI_F16 && C->dtype != PI_BF16) return PI_ERR_DTYPE;
  if (C->layers < 1 || C->layers > 256 || C->kv_heads < 1 || C->kv_heads > 256) return PI_ERR_SHAPE;
  if (C->head_dim < 8 || C->head_dim > 256 || (C->head_dim & 7)) return PI_ERR_SHAPE;
  if (C->page_tokens < 1 || C->page_tokens > 256) return PI_ERR_SHAPE;
  if (C->pages < 1 || C->pages > (1 << 26)) return PI_ERR_SHAPE;
  return PI_OK;
}

inline pi_status check_slots(const pi_cache_desc& C, int slots, int max_pages) {
  if (slots < 1 || slots > PI_CACHE_MAX_SLOTS || max_pages < 1) return PI_ERR_SHAPE;
  if ((long long)max_pages * C.page_tokens >= (1ll << 31)) return PI_ERR_SHAPE;
  return PI_OK;
}

// 16-bit elements of one page in one layer (K and V of every kv head).
inline size_t page_elems(const pi_cache_desc& C) {
  return (size_t)2 * C.kv_heads * C.page_tokens * C.head_dim;
}

struct DevInfo {
  int sms = 0;
  int smem_optin = 0;
};

inline pi_status dev_info(DevInfo* out) {
  static std::mutex mu;
  static std::unordered_map<int, DevInfo> known;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PI_ERR_CUDA;
  std::lock_guard<std::mutex> lk(mu);
  auto it = known.find(dev);
  if (it == known.end()) {
    DevInfo d;
    if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d.smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) !=
            cudaSuccess)
      return PI_ERR_CUDA;
    it = known.emplace(dev, d).first;
  }
  *out = it->second;
  return PI_OK;
}

// A launch that may be scheduled while the kernel before it in the stream
// still runs; the kernel waits for that one at its pdl_enter.
template <typename... KArgs, typename... Args>
pi_status launch(void (*k)(KArgs...), dim3 grid, unsigned block, size_t smem, pi_stream stream,
                 Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, std::forward<Args>(args)...) == cudaSuccess ? PI_OK
                                                                                 : PI_ERR_CUDA;
}

// Raises a kernel's dynamic shared-memory limit on the current device, once.
inline pi_status ensure_smem(const void* fn, int bytes) {
  static std::mutex mu;
  static std::unordered_map<const void*, unsigned long long> done;  // devices, as bits
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PI_ERR_CUDA;
  std::lock_guard<std::mutex> lk(mu);
  unsigned long long& bits = done[fn];
  if (dev < 64 && (bits >> dev & 1)) return PI_OK;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return PI_ERR_CUDA;
  if (dev < 64) bits |= 1ull << dev;
  return PI_OK;
}

constexpr int kAttendGrid = 1024;  // most thread blocks of the attention

// Byte offsets of the regions of a cache workspace.  `arrived` is zero
// between calls and has one place and size for every cache, so that a
// workspace may serve calls of several shapes; the rest is scratch.
struct CacheWs {
  size_t arrived, part, blocks, owner, rank, first, before, src, sums, total;
};

constexpr int kScanPages = 1024;  // pages of one block of the page scans

inline CacheWs cache_ws(const pi_cache_desc& C, int slots, int heads) {
  CacheWs w{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += round_up(bytes > 0 ? bytes : 1, kAlign);
    return o;
  };
  (void)slots;
  w.arrived = take(8 * kAttendGrid);
  const size_t scratch = off;
  w.part = take(heads ? (size_t)kAttendGrid * 2 * 8 * (C.head_dim + 4) * 4 : 0);
  const size_t end = off;
  off = scratch;  // the page calls use the same bytes
  w.blocks = take(4 * (((size_t)C.pages + kScanPages - 1) / kScanPages + 1));
  w.owner = take(4 * (size_t)C.pages);
  w.rank = take(4 * (size_t)C.pages);
  w.first = take(4 * PI_CACHE_MAX_SLOTS);
  w.before = take(4 * PI_CACHE_MAX_SLOTS);
  w.src = take(4 * PI_CACHE_MAX_SLOTS);
  w.sums = take(16);
  w.total = off > end ? off : end;
  return w;
}

// ------------------------------------------------------------------ device
// First statement of every kernel: wait until the kernel before it in the
// stream has completed (its writes visible), then let the next one be
// scheduled (it waits at its own first statement).
__device__ __forceinline__ void pdl_enter() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ void set_status(int* st, int code) { atomicCAS(st, 0, code); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One value rounded to the cache's type, as its bits.
template <int DT>
__device__ __forceinline__ uint16_t to_bits(float v) {
  return DT == 0 ? __half_as_ushort(__float2half_rn(v))
                 : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

template <int DT>
__device__ __forceinline__ float from_bits(uint16_t b) {
  return DT == 0 ? __half2float(__ushort_as_half(b)) : __uint_as_float((uint32_t)b << 16);
}

template <int DT>
__device__ __forceinline__ uint32_t pack_bits(float a, float b) {
  return (uint32_t)to_bits<DT>(a) | ((uint32_t)to_bits<DT>(b) << 16);
}

// a / b for a >= 0, b > 0: in 32 bits where a allows it.
__device__ __forceinline__ long long quotient(long long a, int b) {
  return a >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

__device__ __forceinline__ int pages_of(int tokens, int page_tokens) {
  return (int)(((unsigned)tokens + (unsigned)page_tokens - 1u) / (unsigned)page_tokens);
}

// Number of a page, or -1 (with the status set) where it is out of range.
__device__ __forceinline__ int checked_page(int p, int pages, int* status) {
  if ((unsigned)p < (unsigned)pages) return p;
  set_status(status, PI_ERR_INDEX);
  return -1;
}

}  // namespace pis
