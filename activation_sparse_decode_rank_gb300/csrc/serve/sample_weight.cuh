// sample_weight.cuh — a logit's weight as a whole number (sample.cu).  Host code
// too, the same bit for bit (products that must not be fused are calls of their own,
// all others are in an fmaf), so that its error can be measured without a GPU.
#pragma once

#include <math.h>

#ifdef __CUDACC__
#define PI_WEIGHT_FN __host__ __device__ __forceinline__
#else
#define PI_WEIGHT_FN inline
#endif

namespace pis {

constexpr int kBins = 2048;
constexpr int kBinsPerOctave = 32;
constexpr float kOne = 0x1p36f;  // of a weight's fixed-point part

PI_WEIGHT_FN float product(float a, float b) {
#ifdef __CUDA_ARCH__
  return __fmul_rn(a, b);
#else
  return a * b;
#endif
}
PI_WEIGHT_FN int nearest(float v) {
#ifdef __CUDA_ARCH__
  return __float2int_rn(v);
#else
  return (int)lrintf(v);
#endif
}

// Weights of one row.  Logits, their maximum and T are multiplied by 2^-64 where T is
// above 2^64: two finite logits may be more than the largest float apart, and the low
// part of log2(e) / T would have no bits left (what falls below 2^-149 is nothing beside
// such a T).  With T <= 2^64 a difference that overflows weighs less than 2^-64.
struct Weights {
  float top, least;   // least logit that min-p keeps
  float unit;         // 2^-64 or 1
  float ch, cl;       // log2(e) / T
  PI_WEIGHT_FN void set(float maximum, float temperature, float least_kept) {
    constexpr float L = 1.4426950408889634f, Ll = 1.9259630e-8f;  // log2(e) - L
    unit = temperature > 0x1p64f ? 0x1p-64f : 1.f;
    top = maximum * unit;
    temperature *= unit;
    least = least_kept;
    ch = L / temperature;
    cl = (fmaf(-ch, temperature, L) + Ll) / temperature;
  }
  // bin of a logit; kBins where its weight counts for nothing
  PI_WEIGHT_FN int bin(float x) const {
    const float t = product(fmaf(-unit, x, top), ch);
    return x >= least && t < (float)(kBins / kBinsPerOctave) ? (int)(t * kBinsPerOctave) : kBins;
  }
  // q of a logit of bin b, as a whole number.  With z = zh + zl, 1 - e^-z = zh - zh^2/2 +
  // zh^3/6 - .. + zl (1 - zh + zh^2/2 - zh^3/6) - zl^2/2: zl is up to 6e-6 (the error of
  // t and of log2(e) / T at t near 64), so that zl^2 and zl zh^3 count in units of 2^-36.
  // Off by less than 1.25 for all t < 64: 1 for the two roundings, the rest fp32's (0.1;
  // the largest of 6e7 random logits, 1.04).
  PI_WEIGHT_FN int q(float x, int b) const {
    const float d = fmaf(-unit, x, top), dx = d - top;
    const float e = (top - (d - dx)) - fmaf(unit, x, dx);  // d + e = top - unit x
    const float th = product(d, ch);
    const float rl = fmaf(d, ch, -th) + fmaf(d, cl, product(e, ch));
    const float rh = fmaf((float)b, -1.f / kBinsPerOctave, th);
    constexpr float L = 0.6931471805599453f, Ll = -1.9046542e-9f;  // ln 2 - L
    const float zh = product(rh, L), zl = fmaf(rh, L, -zh) + fmaf(rh, Ll, product(rl, L));
    const float half = 0.5f * zh, sq = product(half, zh);
    const float sl = fmaf(zl, fmaf(0.5f, zl, zh), fmaf(half, zh, -sq));  // sq + sl = z^2 / 2
    const float more = fmaf(zl, -1.f / 3.f, fmaf(zh, fmaf(zh, 1.f / 60.f, -1.f / 12.f), 1.f / 3.f));
    const float high = zh - sq, low = ((zh - high) - sq) + fmaf(product(zh, sq), more, fmaf(sq, zl, zl - sl));
    return nearest(high * kOne) + nearest(low * kOne);
  }
};

}  // namespace pis
