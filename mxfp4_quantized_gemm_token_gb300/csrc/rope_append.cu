// rope_append.cu — position rotation of q and k, and the append of k and v
// to a paged cache (bf16, or e4m3 with one scale per key/value head).
//
// For token t at position p, with c = cos_sin[p, i] and s = cos_sin[p, R/2 + i],
// every pair (x1, x2) of the first R elements of a head becomes
//     y1 = x1 c - x2 s,   y2 = x2 c + x1 s
// in fp32 with every product and sum rounded on its own (no fused
// multiply-add), so the result does not depend on how it is scheduled.  q and
// the bf16 cache round y once; the e4m3 cache holds e4m3(clamp(y / scale, +-448)),
// the library's quantization rule (IEEE division).
//
// Memory-bound: each element is read and written once; what held the kernel back
// was its arithmetic.  A thread takes 16 elements of a head, so that both
// members of its pairs and two 16-byte loads are its own: elements [8c, 8c + 8) of
// both halves of the rotated part, or 16 adjacent ones (adjacent pairs, the
// part past R, v).  Its position in the head is the same for every head it
// takes, so its cosines and sines are loaded once, and its heads' elements are
// on their way before the slot and the position are known.  The quotient is x r + (x - x r s) r with r = 1/s rounded (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990): three operations an element instead of a division's, and the same
// e4m3 codes as the division for 1.4e11 quotients, half of them around the codes' midpoints.
#include <cuda_bf16.h>

#include "attn.h"
#include "internal.h"

namespace mxq {

namespace {

constexpr int kThreads = 128;
constexpr int kUnroll = 3;   // heads in flight per thread

__device__ __forceinline__ void unpack8(const uint4& w, float* v) {
  const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(a[i] << 16);
    v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8_bf16(const float* v) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    r[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// e4m3 codes of 8 elements over the scale s; r = 1/s, or 0 where the quotient
// has to be a division (the conversion itself clamps to +-448, NaN stays NaN)
__device__ __forceinline__ uint2 pack8_e4m3(const float* v, float s, float r) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q0 = __fmul_rn(v[i], r);
    const float q1 = fmaf(fmaf(-q0, s, v[i]), r, q0);
    q[i] = fabsf(q0) < 1024.f ? q1 : q0;
  }
  if (r == 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = clamp448(__fdiv_rn(v[i], s));
  }
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = static_cast<uint32_t>(e4m3x2_rn(q[4 * i], q[4 * i + 1])) |
           (static_cast<uint32_t>(e4m3x2_rn(q[4 * i + 2], q[4 * i + 3])) << 16);
  return make_uint2(w[0], w[1]);
}

// y1 = a c - b s, y2 = b c + a s over 8 pairs (one at a time: packed products and
// sums came out fused)
__device__ __forceinline__ void rotate(float* a, float* b, const float* c, const float* s) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = a[i], y = b[i];
    a[i] = __fsub_rn(__fmul_rn(x, c[i]), __fmul_rn(y, s[i]));
    b[i] = __fadd_rn(__fmul_rn(y, c[i]), __fmul_rn(x, s[i]));
  }
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const RopeAppendParams p) {
  const int nchunk = p.D / 16;
  const int lanes = kThreads / nchunk;         // heads a block takes at once
  const int c = threadIdx.x % nchunk;
  const int h0 = threadIdx.x / nchunk;
  pdl_wait();
  pdl_launch_dependents();
  if (h0 >= lanes) return;
  const int heads = p.Hq + 2 * p.Hkv;          // q heads, then k, then v
  const bool turn = c < p.rot / 16;
  // offsets of the thread's two groups of 8 elements in a head of q or k
  const int e0 = turn && !p.interleaved ? 8 * c : 16 * c;
  const int e1 = turn && !p.interleaved ? p.rot / 2 + 8 * c : 16 * c + 8;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    // the first heads' elements are on their way before the slot, the position and
    // (which depends on it) the rotation's row are looked at
    uint4 lo[kUnroll], hi[kUnroll];
    auto load = [&](int hb) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = hb + u * lanes;
        if (h >= heads) continue;
        const __nv_bfloat16* src;
        int a = e0, b = e1;
        if (h < p.Hq) {
          src = static_cast<const __nv_bfloat16*>(p.q) + t * p.q_t + h * p.q_h;
        } else if (h < p.Hq + p.Hkv) {
          src = static_cast<const __nv_bfloat16*>(p.k) + t * p.k_t + (h - p.Hq) * p.k_h;
        } else {
          src = static_cast<const __nv_bfloat16*>(p.v) + t * p.v_t + (h - p.Hq - p.Hkv) * p.v_h;
          a = 16 * c, b = 16 * c + 8;
        }
        // plain loads: q may be rotated in place
        lo[u] = *reinterpret_cast<const uint4*>(src + a);
        hi[u] = *reinterpret_cast<const uint4*>(src + b);
      }
    };
    load(h0);
    const int64_t slot = p.slots[t];
    const int64_t pos = p.rot > 0 ? p.positions[t] : 0;
    const bool rows = p.rot == 0 || (pos >= 0 && pos < p.max_pos);   // the table has this row
    float cs[8], sn[8];
    if (turn && rows) {
      const float4* cp = reinterpret_cast<const float4*>(p.cos_sin + pos * p.rot + 8 * c);
      const float4* sp =
          reinterpret_cast<const float4*>(p.cos_sin + pos * p.rot + p.rot / 2 + 8 * c);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 a = __ldg(cp + i), b = __ldg(sp + i);
        cs[4 * i] = a.x, cs[4 * i + 1] = a.y, cs[4 * i + 2] = a.z, cs[4 * i + 3] = a.w;
        sn[4 * i] = b.x, sn[4 * i + 1] = b.y, sn[4 * i + 2] = b.z, sn[4 * i + 3] = b.w;
      }
    }
    const bool stored = slot >= 0 && slot < p.slots_total;   // negative: a token not cached
    int64_t page = 0, off = 0;
    if (stored) {
      if (p.slots_total <= 0x7fffffff) {               // 32-bit division where it is enough
        const uint32_t s32 = static_cast<uint32_t>(slot);
        page = s32 / static_cast<uint32_t>(p.page_size);
        off = s32 - static_cast<uint32_t>(page) * static_cast<uint32_t>(p.page_size);
      } else {
        page = slot / p.page_size;
        off = slot - page * p.page_size;
      }
    }
    if ((!rows || slot >= p.slots_total) && threadIdx.x == 0)
      atomicOr(p.status, kStatusBadIndex);
    if (!rows) continue;                               // flagged: nothing is written
    for (int hb = h0; hb < heads; hb += lanes * kUnroll) {
      if (hb != h0) load(hb);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = hb + u * lanes;
        if (h >= heads || (h >= p.Hq && !stored)) continue;
        const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
        float x[16];
        unpack8(lo[u], x);
        unpack8(hi[u], x + 8);
        int a = e0, b = e1;
        if (is_v) {
          a = 16 * c, b = 16 * c + 8;
        } else if (turn) {
          if (p.interleaved) {
            float y[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = x[2 * i], y[8 + i] = x[2 * i + 1];
            rotate(y, y + 8, cs, sn);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[2 * i] = y[i], x[2 * i + 1] = y[8 + i];
          } else {
            rotate(x, x + 8, cs, sn);
          }
        }
        if (is_q) {
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.q_out) + t * p.o_t + h * p.o_h;
          *reinterpret_cast<uint4*>(dst + a) = pack8_bf16(x);
          *reinterpret_cast<uint4*>(dst + b) = pack8_bf16(x + 8);
          continue;
        }
        const int hk = h - p.Hq - (is_v ? p.Hkv : 0);
        const int64_t at = is_v ? page * p.cv_p + off * p.cv_t + hk * p.cv_h
                                : page * p.ck_p + off * p.ck_t + hk * p.ck_h;
        void* cache = is_v ? p.v_cache : p.k_cache;
        if (FP8) {
          const float* sc = is_v ? p.v_scale : p.k_scale;
          const float s = sc ? __ldg(sc + hk) : 1.f;
          const float r = fabsf(s) > 0x1p-60f && fabsf(s) < 0x1p60f ? __frcp_rn(s) : 0.f;
          uint8_t* dst = static_cast<uint8_t*>(cache) + at;
          *reinterpret_cast<uint2*>(dst + a) = pack8_e4m3(x, s, r);
          *reinterpret_cast<uint2*>(dst + b) = pack8_e4m3(x + 8, s, r);
        } else {
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(cache) + at;
          *reinterpret_cast<uint4*>(dst + a) = pack8_bf16(x);
          *reinterpret_cast<uint4*>(dst + b) = pack8_bf16(x + 8);
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendParams& p, int num_sms, cudaStream_t stream) {
  const int64_t cap = static_cast<int64_t>(num_sms) * 64;
  const unsigned blocks = static_cast<unsigned>(p.T < cap ? p.T : cap);
  if (p.fp8)
    return launch_k(rope_append_kernel<true>, dim3(blocks), dim3(kThreads), 0, stream, p);
  return launch_k(rope_append_kernel<false>, dim3(blocks), dim3(kThreads), 0, stream, p);
}

}  // namespace mxq
