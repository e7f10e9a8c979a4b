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
// was its arithmetic, and loads that waited for it.  A thread takes 16 elements
// of a head, so that both members of its pairs and two 16-byte loads are its own:
// elements [8c, 8c + 8) of both halves of the rotated part, or 16 adjacent ones
// (adjacent pairs, the part past R, v).  Its position in the head is the same for
// every head it takes, so its cosines and sines are loaded once a token.  The
// blocks are persistent: while a token is worked on, the elements of the next
// two are on their way to shared memory (asynchronous copies that only the
// issuing thread reads, so nothing waits for the block), and the next one's
// rotation to registers.  8192 tokens of 32 + 2 x 8 heads of 128 into an e4m3
// cache: 34 us, 5.5 TB/s; bf16 33 us, 6.2 TB/s; of 24 + 2 x 3 heads of 64 bf16 15.6 us,
// 4.2 TB/s, with less in flight (one token a block, loads in registers: 41 us at best; with
// a division an element 49 us).  The quotient is x r + (x - x r s) r with
// r = 1/s rounded (P. Markstein, "Computation of elementary functions on the IBM
// RISC System/6000 processor", 1990): three operations an element instead of a
// division's, and the same e4m3 codes (tests compare six million quotients on and next
// to the codes' midpoints).
#include <cuda_bf16.h>

#include "attn.h"
#include "internal.h"

namespace mxq {

namespace {

constexpr int kThreads = 128;
constexpr int kStages = 3;   // steps in shared memory

// Blocks per SM by the heads a thread takes in a step.  A token of few heads has a step
// of one or two: more blocks, with fewer tokens each (1777 tokens of 24 + 2 x 3 heads of
// 64: 5.1 us with one, 6.2 with steps of three; 3000 tokens of 16 + 2 x 4 heads of 128:
// 8.2 with two, 8.5 with three).
constexpr int blocks_of(int unroll) { return unroll == 1 ? 6 : 5; }

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
// has to be a division (the conversion itself clamps to +-448, NaN stays NaN).  The
// residual is formed so that a zero keeps its sign: over a positive s its correction is
// -0.  (Copying the sign instead costs 3 % of 8192 tokens.)
__device__ __forceinline__ uint2 pack8_e4m3(const float* v, float s, float r) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q0 = __fmul_rn(v[i], r);
    const float q1 = fmaf(-fmaf(q0, s, -v[i]), r, q0);
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

__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}

// kUnroll: heads of a thread in a step
template <bool FP8, int kUnroll>
__global__ void __launch_bounds__(kThreads, blocks_of(kUnroll))
    rope_append_kernel(const RopeAppendParams p) {
  __shared__ uint4 ring[kStages][kUnroll][2][kThreads];
  const int nchunk = p.D / 16;
  const int lanes = kThreads / nchunk;         // heads a block takes at once
  const int c = threadIdx.x % nchunk;
  const int h0 = threadIdx.x / nchunk;
  pdl_wait();
  pdl_launch_dependents();
  if (h0 >= lanes) return;
  const int heads = p.Hq + 2 * p.Hkv;          // q heads, then k, then v
  const int steps = (heads + lanes * kUnroll - 1) / (lanes * kUnroll);   // of a token
  const bool turn = c < p.rot / 16;
  // offsets of the thread's two groups of 8 elements in a head of q or k
  const int e0 = turn && !p.interleaved ? 8 * c : 16 * c;
  const int e1 = turn && !p.interleaved ? p.rot / 2 + 8 * c : 16 * c + 8;

  // a step: token, its first head, its slot and position
  struct Step {
    int64_t t, slot;
    int64_t pos;
    int k;
  };
  auto next = [&](Step& s) {
    if (++s.k == steps) {
      s.k = 0;
      s.t += gridDim.x;
    }
  };
  int fill = 0;
  auto copy = [&](Step& s) {
    if (s.t < p.T) {
      s.slot = p.slots[s.t];
      s.pos = p.rot > 0 ? p.positions[s.t] : 0;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = h0 + (s.k * kUnroll + u) * lanes;
        if (h >= heads) continue;
        const __nv_bfloat16* src;
        int a = e0, b = e1;
        if (h < p.Hq) {
          src = static_cast<const __nv_bfloat16*>(p.q) + s.t * p.q_t + h * p.q_h;
        } else if (h < p.Hq + p.Hkv) {
          src = static_cast<const __nv_bfloat16*>(p.k) + s.t * p.k_t + (h - p.Hq) * p.k_h;
        } else {
          src = static_cast<const __nv_bfloat16*>(p.v) + s.t * p.v_t + (h - p.Hq - p.Hkv) * p.v_h;
          a = 16 * c, b = 16 * c + 8;
        }
        copy16(&ring[fill][u][0][threadIdx.x], src + a);
        copy16(&ring[fill][u][1][threadIdx.x], src + b);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    fill = fill + 1 == kStages ? 0 : fill + 1;
  };
  float cs[8], sn[8], cs_next[8], sn_next[8];
  auto rotation = [&](const Step& s, float* co, float* si) {
    if (!turn || s.t >= p.T || s.pos < 0 || s.pos >= p.max_pos) return;
    const float4* cp = reinterpret_cast<const float4*>(p.cos_sin + s.pos * p.rot + 8 * c);
    const float4* sp =
        reinterpret_cast<const float4*>(p.cos_sin + s.pos * p.rot + p.rot / 2 + 8 * c);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 a = __ldg(cp + i), b = __ldg(sp + i);
      co[4 * i] = a.x, co[4 * i + 1] = a.y, co[4 * i + 2] = a.z, co[4 * i + 3] = a.w;
      si[4 * i] = b.x, si[4 * i + 1] = b.y, si[4 * i + 2] = b.z, si[4 * i + 3] = b.w;
    }
  };
  static_assert(kStages == 3, "the steps ahead are named one by one");
  Step now = {static_cast<int64_t>(blockIdx.x), 0, 0, 0}, ahead, far;
  copy(now);
  ahead = now;
  next(ahead);
  copy(ahead);
  rotation(now, cs_next, sn_next);
  int use = 0;
  while (now.t < p.T) {
    far = ahead;
    next(far);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = cs_next[i], sn[i] = sn_next[i];
    copy(far);                                         // into the stage used one step ago
    rotation(ahead, cs_next, sn_next);
    const bool rows = p.rot == 0 || (now.pos >= 0 && now.pos < p.max_pos);   // the table's
    const bool stored = now.slot >= 0 && now.slot < p.slots_total;   // negative: not cached
    int64_t page = 0, off = 0;
    if (stored) {
      if (p.slots_total <= 0x7fffffff) {               // 32-bit division where it is enough
        const uint32_t s32 = static_cast<uint32_t>(now.slot);
        page = s32 / static_cast<uint32_t>(p.page_size);
        off = s32 - static_cast<uint32_t>(page) * static_cast<uint32_t>(p.page_size);
      } else {
        page = now.slot / p.page_size;
        off = now.slot - page * p.page_size;
      }
    }
    if ((!rows || now.slot >= p.slots_total) && threadIdx.x == 0)
      atomicOr(p.status, kStatusBadIndex);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + (now.k * kUnroll + u) * lanes;
      // a position without a row was flagged: nothing of the token is written
      if (!rows || h >= heads || (h >= p.Hq && !stored)) continue;
      const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
      float x[16];
      unpack8(ring[use][u][0][threadIdx.x], x);
      unpack8(ring[use][u][1][threadIdx.x], x + 8);
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
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.q_out) + now.t * p.o_t + h * p.o_h;
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
        // a negative scale divides: 40 us for 8192 tokens, 34 over a positive one
        const float r = s > 0x1p-60f && s < 0x1p60f ? __frcp_rn(s) : 0.f;
        uint8_t* dst = static_cast<uint8_t*>(cache) + at;
        *reinterpret_cast<uint2*>(dst + a) = pack8_e4m3(x, s, r);
        *reinterpret_cast<uint2*>(dst + b) = pack8_e4m3(x + 8, s, r);
      } else {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(cache) + at;
        *reinterpret_cast<uint4*>(dst + a) = pack8_bf16(x);
        *reinterpret_cast<uint4*>(dst + b) = pack8_bf16(x + 8);
      }
    }
    use = use + 1 == kStages ? 0 : use + 1;
    now = ahead;
    ahead = far;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <bool FP8, int kUnroll>
cudaError_t launch(const RopeAppendParams& p, int num_sms, cudaStream_t stream) {
  const int64_t cap = static_cast<int64_t>(num_sms) * blocks_of(kUnroll);
  const unsigned blocks = static_cast<unsigned>(p.T < cap ? p.T : cap);
  return launch_k(rope_append_kernel<FP8, kUnroll>, dim3(blocks), dim3(kThreads), 0, stream, p);
}

template <bool FP8>
cudaError_t launch_unroll(const RopeAppendParams& p, int num_sms, cudaStream_t stream) {
  const int64_t parts = (p.Hq + 2 * static_cast<int64_t>(p.Hkv)) * (p.D / 16);
  if (parts <= kThreads) return launch<FP8, 1>(p, num_sms, stream);
  if (parts <= 2 * kThreads) return launch<FP8, 2>(p, num_sms, stream);
  return launch<FP8, 3>(p, num_sms, stream);
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendParams& p, int num_sms, cudaStream_t stream) {
  return p.fp8 ? launch_unroll<true>(p, num_sms, stream) : launch_unroll<false>(p, num_sms, stream);
}

}  // namespace mxq
