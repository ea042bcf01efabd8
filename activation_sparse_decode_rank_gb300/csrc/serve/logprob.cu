// logprob.cu — log probabilities of given tokens, entropy and the largest
// alternatives of rows of logits (include/pi_serve.h).
#include "serve.cuh"

namespace pis {

struct ScoreArgs {
  const void* logits;
  long long stride;
  const int* tokens;
  float *logprob, *entropy, *top_logprob;
  int* top_idx;
  int* status;
  int rows, vocab, topk;
};

template <int DT>
__device__ __forceinline__ float logit_at(const void* p, long long i) {
  if (DT == 2) return static_cast<const float*>(p)[i];
  return from_bits<DT>(static_cast<const uint16_t*>(p)[i]);
}

// Descending rank of (value, index) as one unsigned key: larger values
// first, equal ones (-0 = +0) by lower index, NaN below everything.
__device__ __forceinline__ unsigned long long rank_key(float v, int i) {
  uint32_t b = __float_as_uint(v + 0.f);
  b = v != v ? 0u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return ((unsigned long long)b << 32) | (uint32_t)~i;
}

__device__ __forceinline__ unsigned long long block_max(unsigned long long v,
                                                        unsigned long long* sh) {
  for (int o = 16; o; o >>= 1) {
    const unsigned long long w = __shfl_xor_sync(~0u, v, o);
    v = w > v ? w : v;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  v = sh[0];
  for (int w = 1; w < 16; ++w) v = sh[w] > v ? sh[w] : v;
  return v;
}

__device__ __forceinline__ float block_sum(float v, float* sh) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int w = 0; w < 16; ++w) v += sh[w];
  return v;
}

// One block per row: the maximum, the sums, then the alternatives one by one.
template <int DT>
__global__ void __launch_bounds__(512) score_kernel(const ScoreArgs a) {
  pdl_enter();
  __shared__ unsigned long long shk[16];
  __shared__ float shf[16];
  const long long r = blockIdx.x;
  const long long base = r * a.stride;
  unsigned long long best = 0;
  float bad = 0.f;
  for (int i = threadIdx.x; i < a.vocab; i += 512) {
    const float x = logit_at<DT>(a.logits, base + i);
    const unsigned long long k = rank_key(x, i);
    best = k > best ? k : best;
    if (x != x || x == INFINITY) bad = 1.f;
  }
  best = block_max(best, shk);
  bad = block_sum(bad, shf);
  const float m = logit_at<DT>(a.logits, base + (int)~(uint32_t)best);
  float s = 0.f, t = 0.f;
  for (int i = threadIdx.x; i < a.vocab; i += 512) {
    const float d = logit_at<DT>(a.logits, base + i) - m;
    if (d > -INFINITY) {
      const float e = expf(d);
      s += e;
      t += e * d;
    }
  }
  s = block_sum(s, shf);
  t = block_sum(t, shf);
  const bool none = m == -INFINITY;
  const float ls = bad > 0.f ? NAN : logf(s);
  if (threadIdx.x == 0) {
    if (a.entropy) a.entropy[r] = bad > 0.f ? NAN : none ? 0.f : ls - t / s;
    if (a.logprob) {
      const int tok = a.tokens[r];
      float lp = 0.f;
      if (tok < -1 || tok >= a.vocab) {
        set_status(a.status, PI_ERR_INDEX);
        lp = NAN;
      } else if (tok >= 0) {
        lp = bad > 0.f ? NAN : none ? -INFINITY : logit_at<DT>(a.logits, base + tok) - m - ls;
      }
      a.logprob[r] = lp;
    }
  }
  unsigned long long last = ~0ull;
  for (int j = 0; j < a.topk; ++j) {
    unsigned long long k = 0;
    for (int i = threadIdx.x; i < a.vocab; i += 512) {
      const unsigned long long c = rank_key(logit_at<DT>(a.logits, base + i), i);
      if (c < last && c > k) k = c;
    }
    last = block_max(k, shk);
    if (threadIdx.x == 0) {
      const int i = (int)~(uint32_t)last;
      a.top_idx[r * a.topk + j] = i;
      const float x = logit_at<DT>(a.logits, base + i);
      a.top_logprob[r * a.topk + j] = bad > 0.f ? NAN : none ? -INFINITY : x - m - ls;
    }
  }
}

}  // namespace pis

using namespace pis;

extern "C" {

size_t pi_logprob_workspace_size(int32_t rows, int32_t vocab, int32_t topk) {
  if (rows < 0 || vocab < 1 || vocab > (1 << 24) || topk < 0 || topk > PI_TOPK_MAX || topk > vocab)
    return 0;
  return kAlign;
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
  ScoreArgs a{logits, stride, tokens, logprob, entropy, top_logprob, top_idx, dev_status, rows,
              vocab, topk};
  return launch(dtype == PI_F16 ? score_kernel<0> : dtype == PI_BF16 ? score_kernel<1> : score_kernel<2>,
                dim3((unsigned)rows), 512, 0, stream, a);
}

}  // extern "C"
