// attn_simple.cuh — one warp, one query row: the online softmax over a row's
// keys, one key at a time.  A lane holds D/32 consecutive elements.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

namespace mxq {

template <int N, bool FP8>
__device__ __forceinline__ void load_row(const void* row, int lane, float* x) {
  if constexpr (FP8) {
    const uint8_t* s = static_cast<const uint8_t*>(row) + lane * N;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      uint32_t r;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(*reinterpret_cast<const uint16_t*>(s + i)));
      const float2 f = __half22float2(*reinterpret_cast<__half2*>(&r));
      x[i] = f.x, x[i + 1] = f.y;
    }
  } else {
    const __nv_bfloat16* s = static_cast<const __nv_bfloat16*>(row) + lane * N;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __bfloat162float(s[i]);
  }
}

template <int N>
struct SoftmaxRow {
  float m = -INFINITY, l = 0.f, o[N] = {};
  __device__ __forceinline__ void add(const float* q, const float* k, const float* v) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) s += q[i] * k[i];
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    const float n = fmaxf(m, s);
    const float a = n == -INFINITY ? 1.f : expf(m - n);
    const float p = n == -INFINITY ? 0.f : expf(s - n);
    l = l * a + p;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = o[i] * a + p * v[i];
    m = n;
  }
  __device__ __forceinline__ void sink(float s) {
    const float n = fmaxf(m, s);
    if (n == -INFINITY) return;
    const float a = expf(m - n);
    l = l * a + expf(s - n);
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] *= a;
    m = n;
  }
  __device__ __forceinline__ void store(void* row, int lane, float* lse, float vscale) {
    __nv_bfloat16* d = static_cast<__nv_bfloat16*>(row) + lane * N;
    const float r = l == 0.f ? 0.f : vscale / l;
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = __float2bfloat16_rn(o[i] * r);
    if (lse && lane == 0) *lse = l == 0.f ? -INFINITY : m + logf(l);
  }
};

}  // namespace mxq
