// attn_math.cuh — small pieces the attention kernels share.
#pragma once

#include <math.h>
#include <stdint.h>

#include "ptx.cuh"

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

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float* a, float* b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// bits 0 .. n-1
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}

// four e4m3 -> two f16x2
__device__ __forceinline__ void e4m3x4_f16(uint32_t x, uint32_t* lo, uint32_t* hi) {
  asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2;"
      " cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b; }"
      : "=r"(*lo), "=r"(*hi)
      : "r"(x));
}

// 16 bytes to shared memory, zeros if !valid (the source is not read then)
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

// mbar_wait_warp that calls what follows a first try without success.  The roles of a kernel
// share the instructions' supply, and the warp that issues the MMAs, which find their operands
// ready nearly always, is the one whose turns the others wait for: it fetches no more than
// the try (a prompt of 8192 tokens 324 -> 307 us, a tree's two tiles of e4m3 286 -> 259; one prompt of
// 2048 tokens 65.5 -> 67.5, whichever of the waits are calls; the softmax has no registers for one).
struct LeanWait {
  static __device__ __noinline__ bool longer(uint64_t* bar, uint32_t parity, const WaitCtx& w) {
    return mbar_wait(bar, parity, w);
  }
};
__device__ __forceinline__ bool wait_lean(uint64_t* bar, uint32_t parity, const WaitCtx& w) {
  const bool ok = mbar_try_wait(bar, parity);
  return __all_sync(0xffffffffu, ok) ||
         __all_sync(0xffffffffu, LeanWait::longer(bar, parity, w));
}

}  // namespace mxq
