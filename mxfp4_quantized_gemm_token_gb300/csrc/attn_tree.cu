// attn_tree.cu — attention of several new tokens per sequence over a paged key/value
// cache: drafted tokens that form a tree, or a chunk of a prompt.
//
// Row i of a sequence stands behind the P keys of its context; it sees them (a window
// counts from its own position, P + its depth in the tree) and the drafts on its path: itself,
// its parent, its parent's parent and so on.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "attn.h"
#include "attn_math.cuh"
#include "internal.h"

namespace mxq {

namespace {

constexpr int kThreads = 128;

// One warp a (row, query head): scores, maximum and sum key by key.
template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads) tree_kernel(const TreeParams p) {
  constexpr int N = D / 32;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  if (item >= p.T * p.Hq) return;
  const int64_t t = item / p.Hq;
  const int h = static_cast<int>(item - t * p.Hq), hk = h / (p.Hq / p.Hkv);
  // the sequence of the row
  int b = -1;
  for (int i = lane; i < p.B; i += 32)
    if (p.cu_q[i] <= t && t < p.cu_q[i + 1]) b = i;
  b = __reduce_max_sync(0xffffffffu, b);
  if (b < 0) return;
  const int q0 = p.cu_q[b], nq = p.cu_q[b + 1] - q0;
  const int64_t cap = p.max_pages * p.page_size;
  const int given = p.seq_lens[b];
  const int len = static_cast<int>(max(static_cast<int64_t>(0),
                                       min(static_cast<int64_t>(given), cap)));
  bool bad = len != given || q0 < 0 || q0 + static_cast<int64_t>(nq) > p.T || len < nq;
  if (bad && lane == 0) atomicOr(p.status, kStatusBadIndex);
  if (q0 < 0 || q0 + static_cast<int64_t>(nq) > p.T || len < nq) return;
  const int P = len - nq, row = static_cast<int>(t) - q0;
  auto parent = [&](int i) {
    if (p.parents == nullptr) return i - 1;
    const int r = p.parents[q0 + i];
    if (r < -1 || r >= i) {
      if (lane == 0) atomicOr(p.status, kStatusBadIndex);
      return -1;
    }
    return r;
  };
  int depth = -1;
  for (int i = row; i >= 0; i = parent(i)) ++depth;
  const float ks = FP8 && p.k_scale != nullptr ? p.k_scale[hk] : 1.f;
  const float vs = FP8 && p.v_scale != nullptr ? p.v_scale[hk] : 1.f;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + t * p.q_t + h * p.q_h;
  float qv[N], o[N] = {}, m = -INFINITY, l = 0.f;
  for (int i = 0; i < N; ++i) qv[i] = __bfloat162float(q[lane + 32 * i]);
  auto value = [](const void* base, int64_t at) {
    if constexpr (FP8)
      return static_cast<float>(static_cast<const __nv_fp8_e4m3*>(base)[at]);
    else
      return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at]);
  };
  auto take = [&](int j) {
    const int page = p.page_table[b * p.ld_table + j / p.page_size];
    if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.pages)) {
      if (lane == 0) atomicOr(p.status, kStatusBadIndex);
      return;
    }
    const int off = j % p.page_size;
    const int64_t ka = page * p.ck_p + off * p.ck_t + hk * p.ck_h;
    const int64_t va = page * p.cv_p + off * p.cv_t + hk * p.cv_h;
    float s = 0.f;
    for (int i = 0; i < N; ++i) s += qv[i] * value(p.k_cache, ka + lane + 32 * i);
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale * ks;
    const float top = fmaxf(m, s), ref = top == -INFINITY ? 0.f : top;
    const float f = expf(m - ref), w = expf(s - ref);
    l = l * f + w;
    for (int i = 0; i < N; ++i) o[i] = o[i] * f + w * value(p.v_cache, va + lane + 32 * i);
    m = top;
  };
  const int lo = p.window > 0 ? max(0, P + depth - p.window + 1) : 0;
  for (int j = 0; j < min(P, min(p.first, lo)); ++j) take(j);
  for (int j = lo; j < P; ++j) take(j);
  int up = 0;
  for (int i = row; i >= 0; i = parent(i), ++up)
    if (p.window == 0 || up < p.window || P + depth - up < p.first) take(P + i);
  const RowEnd end = finish_row(m, l, p.sinks ? p.sinks + h : nullptr);
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + t * p.o_t + h * p.o_h;
  for (int i = 0; i < N; ++i) out[lane + 32 * i] = __float2bfloat16_rn(o[i] * (end.factor * vs));
  if (p.lse != nullptr && lane == 0) p.lse[t * p.Hq + h] = end.lse;
}

template <int D, bool FP8>
cudaError_t launch(const TreeParams& p, cudaStream_t stream) {
  const int64_t blocks = (p.T * p.Hq + kThreads / 32 - 1) / (kThreads / 32);
  return launch_k(tree_kernel<D, FP8>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0,
                  stream, p);
}

}  // namespace

size_t tree_workspace_bytes(int64_t, int64_t, int, int, int, int) { return 0; }

cudaError_t launch_tree(const TreeParams& p, int, cudaStream_t stream) {
  if (p.D == 128) return p.fp8 ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
  return p.fp8 ? launch<64, true>(p, stream) : launch<64, false>(p, stream);
}

}  // namespace mxq
