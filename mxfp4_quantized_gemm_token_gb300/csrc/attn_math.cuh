// attn_math.cuh — small pieces the attention kernels share.
#pragma once

#include <math.h>
#include <stdint.h>

namespace mxq {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A finished row's sum and output factor.  ms: the row's reference in natural
// units (-inf: no key), l: the sum of its weights relative to it.  The sink's
// logit joins the sum; both are taken relative to the larger of the two, so
// neither overflows, and a tiny factor is not flushed to zero.
struct RowEnd {
  float factor;   // of the accumulated values
  float lse;
  bool none;      // no key and no sink
};
__device__ __forceinline__ RowEnd finish_row(float ms, float l, const float* sink) {
  RowEnd r;
  float f = 1.f, top = ms;
  if (sink != nullptr) {
    const float s = __ldg(sink);
    top = fmaxf(ms, s);
    f = ms == -INFINITY ? 0.f : expf(ms - top);
    l = l * f + (s == -INFINITY ? 0.f : expf(s - top));
  }
  r.none = l == 0.f;
  r.factor = r.none ? 0.f : f / l;
  r.lse = r.none ? -INFINITY : top + logf(l);
  return r;
}

}  // namespace mxq
