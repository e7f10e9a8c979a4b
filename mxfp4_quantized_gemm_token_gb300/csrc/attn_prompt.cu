// attn_prompt.cu — attention of whole prompts: packed sequences of different
// lengths, grouped heads, causal and windowed masks.
#include "attn.h"
#include "attn_simple.cuh"
#include "internal.h"

namespace mxq {

namespace {

// [start, start + len) of sequence b in cu, held inside [0, total]
__device__ __forceinline__ bool seq_range(const int32_t* cu, int b, int64_t total, int64_t* start,
                                          int64_t* len) {
  const int64_t a = cu[b], e = cu[b + 1];
  const bool ok = a >= 0 && e >= a && e <= total;
  *start = ok ? a : 0;
  *len = ok ? e - a : 0;
  return ok;
}

template <int D>
__global__ void prompt_kernel(const PromptParams p) {
  constexpr int N = D / 32;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int h = blockIdx.y;
  const int hk = h / (p.Hq / p.Hkv);
  const int b = blockIdx.z;
  int64_t q0, nq, k0, nk;
  const bool okq = seq_range(p.cu_q, b, p.Tq, &q0, &nq);
  const bool okk = seq_range(p.cu_k, b, p.Tk, &k0, &nk);
  if (!(okq && okk) && threadIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
       i < nq; i += static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5)) {
    float q[N];
    load_row<N, false>(static_cast<const __nv_bfloat16*>(p.q) + (q0 + i) * p.q_t + h * p.q_h, lane,
                       q);
#pragma unroll
    for (int e = 0; e < N; ++e) q[e] *= p.scale;
    const int64_t at = i + nk - nq;
    const int64_t hi = p.causal ? (at + 1 < nk ? at + 1 : nk) : nk;
    const int64_t lo = p.window > 0 && at - p.window + 1 > 0 ? at - p.window + 1 : 0;
    SoftmaxRow<N> row;
    for (int64_t j = lo; j < hi; ++j) {
      float k[N], v[N];
      load_row<N, false>(static_cast<const __nv_bfloat16*>(p.k) + (k0 + j) * p.k_t + hk * p.k_h,
                         lane, k);
      load_row<N, false>(static_cast<const __nv_bfloat16*>(p.v) + (k0 + j) * p.v_t + hk * p.v_h,
                         lane, v);
      row.add(q, k, v);
    }
    if (p.sinks) row.sink(p.sinks[h]);
    row.store(static_cast<__nv_bfloat16*>(p.out) + (q0 + i) * p.o_t + h * p.o_h, lane,
              p.lse ? p.lse + (q0 + i) * p.Hq + h : nullptr, 1.f);
  }
}

}  // namespace

size_t prompt_workspace_bytes(int64_t, int64_t, int, int, int, int) { return 0; }

cudaError_t launch_prompt(const PromptParams& p, int, cudaStream_t stream) {
  int64_t gx = (p.Tq + 3) / 4;
  if (gx > 2048) gx = 2048;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(p.Hq),
                  static_cast<unsigned>(p.B));
  if (p.D == 128) return launch_k(prompt_kernel<128>, grid, dim3(128), 0, stream, p);
  return launch_k(prompt_kernel<64>, grid, dim3(128), 0, stream, p);
}

}  // namespace mxq
