// Powers of a head's decay a = exp(log_decay), shared by the decayed passes
// and the single-token step.
//
// Every factor is a^n for a row distance n >= 0, taken from the logarithm,
// never as a product of rounded factors over a long distance: a itself is
// rounded by up to 2^-25, so a running product over the 1 / (1 - a) rows a
// state remembers would be off by that many roundings.  Where a state has to
// be scaled step by step, its factor is held as a sum of two (Factor), from
// expm1 while it is near 1.
#pragma once

#include <cfloat>
#include <cstdint>

namespace spanla {

// log_decay of -infinity (a = 0, a state that forgets at once) becomes a large
// finite number, so that a distance of 0 still gives a^0 = 1.  NaN stays NaN.
constexpr float kMinLogDecay = -6000.f;   // exp of it is 0 in fp32 and fp64

__device__ __forceinline__ float load_log_decay(const float* log_decay, int head) {
  const float x = __ldg(log_decay + head);
  return x < kMinLogDecay ? kMinLogDecay : x;
}

__device__ __forceinline__ float decay_log2(float ld) { return ld * 1.4426950408889634f; }

// a^n from log2 a.
__device__ __forceinline__ float decay_pow(float l2, float n) { return exp2f(l2 * n); }

// As decay_pow, by the hardware's 2^x alone: within 2^-22 of it; 0 below 2^-126.
__device__ __forceinline__ float decay_pow_fast(float l2, float n) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(l2 * n));
  return y;
}

// a^n as hi + lo, lo of hi's sign and 0 only with it, so that an infinite state
// stays infinite (hi s and lo s agree; with lo = 0, or of the other sign, their
// sum would be NaN).  Where a^n is hi, lo is too small to be seen beside it.
struct Factor {
  float hi, lo;
  // a^n s + x, with one rounding of a^n in effect.
  __device__ __forceinline__ float step(float s, float x) const { return fmaf(hi, s, fmaf(lo, s, x)); }
};

constexpr Factor kNoDecay = {1.f, FLT_MIN};

__device__ __forceinline__ Factor decay_factor(float ld, float n) {
  const float m1 = expm1f(ld * n);   // a^n - 1
  if (m1 > -0.5f) {
    const float hi = __fadd_rd(1.f, m1);
    return {hi, fmaxf(m1 - (hi - 1.f), FLT_MIN)};   // (both differences exact for hi in [1/2, 2])
  }
  // Below 1/2, where nothing is remembered for long, hi alone.
  const float hi = expf(ld * n);
  return {hi, hi > 0.f ? fmaxf(hi * 0x1p-40f, 0x1p-149f) : 0.f};
}

}  // namespace spanla
