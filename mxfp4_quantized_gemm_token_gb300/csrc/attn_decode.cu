// attn_decode.cu — attention of one new token per sequence over a paged
// key/value cache.
#include "attn.h"
#include "attn_simple.cuh"
#include "internal.h"

namespace mxq {

namespace {

template <int D, bool FP8>
__global__ void decode_kernel(const DecodeParams p) {
  constexpr int N = D / 32;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (w >= static_cast<int64_t>(p.B) * p.Hq) return;
  const int64_t b = w / p.Hq;
  const int h = static_cast<int>(w - b * p.Hq);
  const int hk = h / (p.Hq / p.Hkv);
  int64_t len = p.seq_lens[b];
  const int64_t cap = p.max_pages * p.page_size;
  if (len < 0 || len > cap) {
    if (lane == 0) atomicOr(p.status, kStatusBadIndex);
    len = len < 0 ? 0 : cap;
  }
  float q[N];
  load_row<N, false>(static_cast<const __nv_bfloat16*>(p.q) + b * p.q_b + h * p.q_h, lane, q);
  const float ks = p.scale * (p.k_scale ? p.k_scale[hk] : 1.f);
#pragma unroll
  for (int i = 0; i < N; ++i) q[i] *= ks;
  SoftmaxRow<N> row;
  constexpr int es = FP8 ? 1 : 2;
  int64_t j = p.window > 0 && len > p.window ? len - p.window : 0;
  for (; j < len; ++j) {
    const int64_t page = p.page_table[b * p.ld_table + j / p.page_size];
    const int64_t off = j % p.page_size;
    if (page < 0 || page >= p.pages) {
      if (lane == 0) atomicOr(p.status, kStatusBadIndex);
      continue;
    }
    float k[N], v[N];
    load_row<N, FP8>(static_cast<const char*>(p.k_cache) +
                         (page * p.ck_p + off * p.ck_t + hk * p.ck_h) * es, lane, k);
    load_row<N, FP8>(static_cast<const char*>(p.v_cache) +
                         (page * p.cv_p + off * p.cv_t + hk * p.cv_h) * es, lane, v);
    row.add(q, k, v);
  }
  if (p.sinks) row.sink(p.sinks[h]);
  row.store(static_cast<__nv_bfloat16*>(p.out) + b * p.o_b + h * p.o_h, lane,
            p.lse ? p.lse + b * p.Hq + h : nullptr, p.v_scale ? p.v_scale[hk] : 1.f);
}

}  // namespace

size_t decode_workspace_bytes(int64_t, int, int, int, int) { return 0; }

cudaError_t launch_decode(const DecodeParams& p, int, cudaStream_t stream) {
  const int64_t warps = static_cast<int64_t>(p.B) * p.Hq;
  const dim3 grid(static_cast<unsigned>((warps + 3) / 4)), block(128);
  if (p.D == 128)
    return p.fp8 ? launch_k(decode_kernel<128, true>, grid, block, 0, stream, p)
                 : launch_k(decode_kernel<128, false>, grid, block, 0, stream, p);
  return p.fp8 ? launch_k(decode_kernel<64, true>, grid, block, 0, stream, p)
               : launch_k(decode_kernel<64, false>, grid, block, 0, stream, p);
}

}  // namespace mxq
