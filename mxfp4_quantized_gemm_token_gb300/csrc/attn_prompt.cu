// attn_prompt.cu — attention of whole prompts: packed sequences of different
// lengths, grouped heads, causal and windowed masks.
//
//   S = Q K^T,  P = 2^(c S - c m),  l = rowsum P,  O = P V / l   (c = scale log2 e)
//
// one pass over the keys with the running maximum m and sum l of each row.
//
// Rows.  The G query heads of a key/value head read the same keys, so a tile's
// 128 rows are (token, head of the group) pairs, token-major: TB = 128 / G tokens.  A
// tile then spans few positions, which keeps both the masked part of the
// diagonal tiles and the waste of short sequences small, and one 3-D TMA box
// [64, G, TB] brings it in that order.  A CTA takes two tiles (2 TB
// consecutive tokens) against 128-key blocks.
//
// Both products run on the tensor cores with their accumulators in tensor
// memory: S0, S1 (128 columns each, later overwritten by P as bf16) and O0, O1 (D
// columns each).  Q and K are K-major operands; V keeps its [key, d] rows and
// enters as an MN-major operand; P is read from tensor memory.  While the
// softmax of one tile runs on its warpgroup (one thread per row), the tensor
// core works on the other tile.
//   warps 0-3, 4-7   softmax of tile 0 and 1, and their output
//   warp 8           issues the MMAs
//   warp 9           loads Q, K and V with TMA (one ring; K and V alternate)
// The maximum a row subtracts is only raised when it grows by more than 2^8 in the
// exponent: O is rescaled (by the row's own thread) in few blocks,
// and l and O stay far from the range's ends.  l and O use the same reference, so
// the result does not depend on it.
//
// Work.  A kernel of one block first lists the work items (sequence, pair of
// tiles, its blocks of keys) with the costliest first; the persistent CTAs
// take them in turn, in alternating direction, which balances lengths.
#include <cuda_bf16.h>
#include <math.h>

#include <string>

#include "attn.h"
#include "attn_math.cuh"
#include "internal.h"

namespace mxq {

namespace {

constexpr int kBM = 128;             // rows of a tile, keys of a block
constexpr int kPromptThreads = 384;
// registers a thread: the launch gives 168 to each of the 384; the softmax
// warpgroups keep a row of 128 scores and take what the third one gives up
constexpr int kSoftmaxRegs = 208, kOtherRegs = 80;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * 168, "register split above the launch's");

struct PromptMaps {
  CUtensorMap q, k, v;
};

// One pair of tiles: tokens [q_row, q_row + ntok) of the packed queries, the
// first of which stands at key position at0 of its sequence's nk keys, and the
// key blocks [kb0, kb1) that any of them sees.
struct __align__(16) PromptItem {
  int q_row, ntok, at0, k_row;
  int nk, kb0, kb1, pad;
};

struct PromptArgs {
  PromptParams p;
  const int* n_items;                // header of the workspace
  const PromptItem* items;
  int G, TB;
  unsigned long long budget_ns;
  int inject_stall;
};

constexpr int kBuckets = 512;

// [start, start + len) of sequence b in cu, or nothing if it leaves [0, total]
__device__ __forceinline__ bool seq_range(const int32_t* cu, int b, int64_t total, int* start,
                                          int* len) {
  const int64_t a = cu[b], e = cu[b + 1];
  const bool ok = a >= 0 && e >= a && e <= total;
  *start = ok ? static_cast<int>(a) : 0;
  *len = ok ? static_cast<int>(e - a) : 0;
  return ok;
}

// Lists the items, ordered by falling number of key blocks (a counting sort; more than
// 511 blocks count as 511).
__global__ void __launch_bounds__(1024) prompt_plan_kernel(const PromptParams p, int tokens_per_item,
                                                           int* n_items, PromptItem* items,
                                                           int cap) {
  __shared__ int count[kBuckets];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < kBuckets; i += blockDim.x) count[i] = 0;
  __syncthreads();
  for (int pass = 0; pass < 2; ++pass) {
    for (int b = warp; b < p.B; b += 32) {
      int q0, nq, k0, nk;
      const bool okq = seq_range(p.cu_q, b, p.Tq, &q0, &nq);
      const bool okk = seq_range(p.cu_k, b, p.Tk, &k0, &nk);
      if (!(okq && okk)) {
        if (lane == 0) atomicOr(p.status, kStatusBadIndex);
        continue;
      }
      const int pairs = (nq + tokens_per_item - 1) / tokens_per_item;
      for (int i = lane; i < pairs; i += 32) {
        PromptItem it;
        const int first = i * tokens_per_item;
        it.q_row = q0 + first;
        it.ntok = min(tokens_per_item, nq - first);
        it.at0 = first + nk - nq;
        it.k_row = k0;
        it.nk = nk;
        const int hi = p.causal ? min(nk, it.at0 + it.ntok) : nk;
        it.kb1 = hi > 0 ? (hi + kBM - 1) / kBM : 0;
        it.kb0 = p.window > 0 ? max(0, it.at0 - p.window + 1) / kBM : 0;
        it.pad = 0;
        const int bucket = kBuckets - 1 - min(kBuckets - 1, max(0, it.kb1 - it.kb0));
        if (pass == 0) {
          atomicAdd(&count[bucket], 1);
        } else {
          const int at = atomicAdd(&count[bucket], 1);
          if (at < cap) items[at] = it;
        }
      }
    }
    __syncthreads();
    if (pass == 0) {
      // exclusive prefix sum over the buckets, by one warp
      if (warp == 0) {
        int run = 0;
        for (int i = 0; i < kBuckets; i += 32) {
          const int c = count[i + lane];
          int x = c;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
          }
          count[i + lane] = run + x - c;
          run += __shfl_sync(0xffffffffu, x, 31);
        }
        // only offsets that run backwards give more items than there is room for
        if (lane == 0) {
          if (run > cap) atomicOr(p.status, kStatusBadIndex);
          *n_items = min(run, cap);
        }
      }
      __syncthreads();
    }
  }
}

template <int D>
struct PromptLayout {
  static constexpr int kChunks = D / 64;
  static constexpr int kChunkBytes = kBM * 128;          // 128 rows of 64 elements
  static constexpr int kTileBytes = kChunks * kChunkBytes;
  static constexpr int kStages = D == 128 ? 4 : 8;       // five measured no faster than four
  static constexpr int kOutBytes = 8 * 32 * 128;         // output staging: 32 rows x 128 B a warp
  static constexpr int kBars = 2 * 6 + 2 * kStages + 1;
  static constexpr int kSmem =
      (2 + kStages) * kTileBytes + kOutBytes + 8 * kBars + 16;
  static_assert(kSmem + 1024 <= 227 * 1024, "shared memory over budget");
};

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

// position r of the sequence of items that this CTA takes, in alternating direction
__device__ __forceinline__ int item_index(int r) {
  return r * gridDim.x + ((r & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

// The items this CTA takes, each read one ahead of its use.
struct Items {
  const PromptArgs& a;
  int total, r = 0, head = 0, next_head = 0;
  bool more;
  PromptItem it, ahead;
  __device__ __forceinline__ Items(const PromptArgs& args, int n) : a(args), total(n) { fetch(); }
  __device__ __forceinline__ void fetch() {
    const int idx = item_index(r++);
    more = idx < total;
    if (more) {
      const int i = idx / a.p.Hkv;
      next_head = idx - i * a.p.Hkv;
      ahead = a.items[i];
    }
  }
  __device__ __forceinline__ bool next() {
    if (!more) return false;
    it = ahead;
    head = next_head;
    fetch();
    return true;
  }
};

template <int D>
__global__ void __launch_bounds__(kPromptThreads, 1)
    prompt_kernel(const __grid_constant__ PromptMaps maps, const PromptArgs a) {
  using L = PromptLayout<D>;
  constexpr int ST = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* ring = smem + 2 * L::kTileBytes;
  uint8_t* sOut = ring + ST * L::kTileBytes;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(sOut + L::kOutBytes);
  uint64_t* q_empty = q_full + 2;
  uint64_t* s_full = q_empty + 2;
  uint64_t* p_full = s_full + 2;
  // an item's O has a barrier of its own: its commit is followed by the next
  // item's S without a word from the softmax, which would let one barrier run
  // two phases ahead of its waiter
  uint64_t* o_full = p_full + 4;
  uint64_t* kv_full = o_full + 2;
  uint64_t* kv_empty = kv_full + ST;
  uint64_t* drain = kv_empty + ST;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const PromptParams& p = a.p;
  WaitCtx wc{p.status, abort_flag, a.budget_ns};

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&o_full[i], 1);
      mbar_init(&p_full[2 * i], 4);       // the warps of the tile's warpgroup; P
      mbar_init(&p_full[2 * i + 1], 4);   // of keys 0-63 and of 64-127
    }
    for (int i = 0; i < ST; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 9 && lane == 0) {
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_launch_dependents();
  const int total = *a.n_items * p.Hkv;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 9) {
      // ------------------------------------------------------------ loads
      if (lane == 0 && !a.inject_stall) {
        uint32_t fill = 0, nq = 0;
        const uint32_t q_bytes = static_cast<uint32_t>(a.G * a.TB) * 128 * L::kChunks;
        bool ok = true;
        Items items(a, total);
        while (ok && items.next()) {
          const PromptItem& it = items.it;
          const int hk = items.head;
          if (it.kb1 <= it.kb0) continue;
          auto load_q = [&](int s) {
            if (!mbar_wait(&q_empty[s], (nq & 1) ^ 1, wc)) return false;
            mbar_expect_tx(&q_full[s], q_bytes);
            for (int c = 0; c < L::kChunks; ++c)
              tma_load_3d(sQ + s * L::kTileBytes + c * L::kChunkBytes, &maps.q, &q_full[s], c * 64,
                          hk * a.G, it.q_row + s * a.TB);
            return true;
          };
          auto load_kv = [&](const CUtensorMap* map, int kb) {
            const int st = fill % ST;
            if (!mbar_wait(&kv_empty[st], ((fill / ST) & 1) ^ 1, wc)) return false;
            mbar_expect_tx(&kv_full[st], L::kTileBytes);
            for (int c = 0; c < L::kChunks; ++c)
              tma_load_3d(ring + st * L::kTileBytes + c * L::kChunkBytes, map, &kv_full[st], c * 64,
                          hk, it.k_row + kb * kBM);
            ++fill;
            return true;
          };
          ok = load_q(0) && load_kv(&maps.k, it.kb1 - 1) && load_q(1) &&
               load_kv(&maps.v, it.kb1 - 1);
          ++nq;
          for (int kb = it.kb1 - 2; ok && kb >= it.kb0; --kb)
            ok = load_kv(&maps.k, kb) && load_kv(&maps.v, kb);
        }
        if (*abort_flag) {
          // let every copy already issued land before the CTA goes away
          volatile int zero = 0;
          WaitCtx dw{p.status, &zero, 1000000000ull};
          for (uint32_t i = fill > ST ? fill - ST : 0; i < fill; ++i)
            mbar_wait(&kv_full[i % ST], (i / ST) & 1, dw);
          for (int s = 0; s < 2; ++s)
            if (nq > 0) mbar_wait(&q_full[s], (nq - 1) & 1, dw);
        }
      }
    } else if (warp == 8) {
      // -------------------------------------------------------------- MMAs
      constexpr uint32_t kDescS = idesc_bf16(kBM, kBM);
      constexpr uint32_t kDescO = idesc_bf16_bmn(kBM, D);
      const bool leader = elect_one();
      // descriptors of the first tiles; offsets are added in 16-byte units
      const uint64_t q_desc = sw128_desc(smem_u32(sQ)), k_desc = sw128_desc(smem_u32(ring));
      const uint64_t v_desc = sw128_desc_mn(smem_u32(ring), L::kChunkBytes);
      uint32_t base = 0, nq = 0, np = 0;     // ring position of K_0, items, blocks so far
      auto issue_s = [&](int s, uint32_t fill) {
        const uint64_t qd = q_desc + s * (L::kTileBytes / 16);
        const uint64_t kd = k_desc + (fill % ST) * (L::kTileBytes / 16);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const int off = (k / 4) * (L::kChunkBytes / 16) + (k % 4) * 2;
          mma_f16(tmem + s * 128, qd + off, kd + off, kDescS, k > 0);
        }
      };
      // the keys of half `part` of a block
      auto issue_o = [&](int s, uint32_t fill, int part, bool accumulate) {
        const uint64_t vd = v_desc + (fill % ST) * (L::kTileBytes / 16) + part * (4 * 2048 / 16);
        const uint32_t pa = tmem + s * 128 + part * 32;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f16_ts(tmem + 256 + s * 128, pa + k * 8, vd + k * (2048 / 16), kDescO,
                     accumulate || k > 0);
      };
      auto wait_kv = [&](uint32_t fill) {
        return mbar_wait_warp(&kv_full[fill % ST], (fill / ST) & 1, wc);
      };
      Items items(a, total);
      while (items.next()) {
        const int n = items.it.kb1 - items.it.kb0;
        if (n <= 0) continue;
        if (!wait_kv(base)) goto mma_done;
        for (int s = 0; s < 2; ++s) {
          if (!mbar_wait_warp(&q_full[s], nq & 1, wc)) goto mma_done;
          if (leader) {
            tc_fence_after();
            issue_s(s, base);
            mma_commit(&s_full[s]);
            if (n == 1) mma_commit(&q_empty[s]);
            if (s == 1) mma_commit(&kv_empty[base % ST]);
          }
          __syncwarp();
        }
        for (int j = 0; j < n; ++j, ++np) {
          const uint32_t vf = base + 2 * j + 1, kf = vf + 1;
          if (!wait_kv(vf)) goto mma_done;
          for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              if (!mbar_wait_warp(&p_full[2 * s + part], np & 1, wc)) goto mma_done;
              if (leader) {
                tc_fence_after();
                issue_o(s, vf, part, j > 0 || part > 0);
              }
              __syncwarp();
            }
            if (leader && s == 1) mma_commit(&kv_empty[vf % ST]);
            if (j + 1 < n) {
              if (s == 0 && !wait_kv(kf)) goto mma_done;
              if (leader) {
                tc_fence_after();
                issue_s(s, kf);
                mma_commit(&s_full[s]);
                if (j + 2 == n) mma_commit(&q_empty[s]);
                if (s == 1) mma_commit(&kv_empty[kf % ST]);
              }
            } else if (leader) {
              mma_commit(&o_full[s]);        // the item's O is complete
            }
            __syncwarp();
          }
        }
        base += 2 * n;
        ++nq;
      }
    mma_done:
      if (*abort_flag) {
        // wait for the MMAs in flight before the tensor memory is freed
        if (leader) mma_commit(drain);
        volatile int zero = 0;
        WaitCtx dw{p.status, &zero, 1000000000ull};
        mbar_wait(drain, 0, dw);
      }
    }
  } else {
    // ----------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int s = warp >> 2;                            // tile
    const int row = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + s * 128 + lanes, tO = tmem + 256 + s * 128 + lanes;
    const int tok = row / a.G, g = row - tok * a.G;
    const float c = p.scale * kLog2e;
    uint32_t ns = 0, no = 0, base = 0;
    Items items(a, total);
    while (items.next()) {
      const PromptItem& it = items.it;
      const int n = it.kb1 - it.kb0;
      const int h = items.head * a.G + g;
      const int i = s * a.TB + tok;
      const bool valid = tok < a.TB && i < it.ntok;
      // visible keys [lo, hi) of this row, and those every row of the warp sees;
      // a row that is not stored may see anything
      const int at = it.at0 + i;
      const int hi = !valid ? 1 << 30 : (p.causal ? min(it.nk, at + 1) : it.nk);
      const int lo = valid && p.window > 0 ? max(0, at - p.window + 1) : 0;
      const int all_lo = __reduce_max_sync(0xffffffffu, lo);
      const int all_hi = __reduce_min_sync(0xffffffffu, hi);
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j) {
        const int k0 = (it.kb1 - 1 - j) * kBM;
        if (!mbar_wait_warp(&s_full[s], ns & 1, wc)) goto softmax_done;
        ++ns;
        tc_fence_after();
        // the row's scores and their maximum
        float x[128], mq[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32_async(tS + 32 * q, x + 32 * q);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float* v = x + 32 * q;
          tmem_wait32(v);
          const int kq = k0 + 32 * q;
          if (kq + 32 > all_hi || kq < all_lo) {
            // a warp's rows span few positions: most chunks need no mask
            const uint32_t vis = low_bits(hi - kq) & ~low_bits(lo - kq);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = (vis >> e) & 1 ? v[e] : -INFINITY;
          }
          mq[q] = fmaxf(v[0], v[1]);
#pragma unroll
          for (int e = 2; e < 32; e += 2) mq[q] = fmaxf(mq[q], fmaxf(v[e], v[e + 1]));
        }
        const float mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
        // raise the reference if it grows by more than 2^8 (at first: from -inf)
        const bool raise = (mx - m) * c > 8.f;
        if (__any_sync(0xffffffffu, raise)) {
          const float f = raise ? ex2((m - mx) * c) : 1.f;
          if (__any_sync(0xffffffffu, raise && m > -INFINITY)) {
            // the products of the blocks before are complete: their commit came
            // before this block's scores
#pragma unroll 1
            for (int q = 0; q < D; q += 32) {
              float o[32];
              tmem_ld32(tO + q, o);
              uint32_t w[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(o[e] * f);
              tmem_st32(tO + q, w);
            }
          }
          l *= f;
          if (raise) m = mx;
        }
        const float mc = m == -INFINITY ? 0.f : m * c;
        const uint64_t c2 = pack2(c, c), n2 = pack2(-mc, -mc);
        if (j == 0 && s == 0 && it.nk < k0 + kBM) {
          // the last block's rows past the sequence are other keys' (or none): their
          // weights are 0, and the values become 0 too, as 0 * inf is not 0
          const uint32_t vf = base + 1;
          if (!mbar_wait_warp(&kv_full[vf % ST], (vf / ST) & 1, wc)) goto softmax_done;
          if (k0 + row >= it.nk) {
            uint8_t* vr = ring + (vf % ST) * L::kTileBytes + row * 128;
            for (int ch = 0; ch < L::kChunks; ++ch)
#pragma unroll
              for (int q = 0; q < 8; ++q)
                *reinterpret_cast<uint4*>(vr + ch * L::kChunkBytes + 16 * q) =
                    make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        // weights, in two halves of 64 keys; the first is handed over a little
        // into the second, when its store is surely complete
        uint64_t sum[4] = {};
        auto weights = [&](uint32_t* w, int first, int last) {
#pragma unroll
          for (int e = first; e < last; e += 2) {
            float u, v;
            unpack2(fma2(pack2(x[e], x[e + 1]), c2, n2), &u, &v);
            u = ex2(u), v = ex2(v);
            w[(e & 63) / 2] = bf16x2(u, v);
            sum[(e / 2) & 3] = add2(sum[(e / 2) & 3], pack2(u, v));
          }
        };
        auto hand_over = [&](int part) {
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * s + part]);
        };
        uint32_t w0[32], w1[32];
        weights(w0, 0, 64);
        tmem_st32(tS, w0);
        weights(w1, 64, 80);
        hand_over(0);
        weights(w1, 80, 128);
        tmem_st32(tS + 32, w1);
        hand_over(1);
        float s0, s1;
        unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), &s0, &s1);
        l += s0 + s1;
      }
      base += n > 0 ? 2 * n : 0;
      if (n > 0) {
        if (!mbar_wait_warp(&o_full[s], no & 1, wc)) goto softmax_done;
        ++no;
        tc_fence_after();
      }
      const RowEnd end =
          finish_row(m * p.scale, l, p.sinks != nullptr && valid ? p.sinks + h : nullptr);
      const float inv = end.factor;
      const bool none = end.none;
      // through shared memory, so that 8 lanes write 128 adjacent bytes of a row
      const int64_t tokr = it.q_row + i;
      const int64_t dst = tokr * p.o_t + static_cast<int64_t>(h) * p.o_h;
      const uint32_t stored = __ballot_sync(0xffffffffu, valid);
      uint8_t* stage = sOut + warp * (32 * 128);
      for (int d0 = 0; d0 < D; d0 += 64) {
        float o[64];
        if (n > 0) {
          tmem_ld64(tO + d0, o);
        } else {
#pragma unroll
          for (int e = 0; e < 64; ++e) o[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = none ? 0u : bf16x2(o[8 * e + 2 * k] * inv, o[8 * e + 2 * k + 1] * inv);
          *reinterpret_cast<uint4*>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int rw = 4 * e + (lane >> 3), ch = lane & 7;
          const uint4 w = *reinterpret_cast<const uint4*>(stage + rw * 128 + ((ch ^ (rw & 7)) << 4));
          const int64_t to = __shfl_sync(0xffffffffu, dst, rw);
          if ((stored >> rw) & 1)
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + to + d0 + 8 * ch) = w;
        }
        __syncwarp();
      }
      if (p.lse != nullptr && valid)
        p.lse[tokr * p.Hq + h] = end.lse;
      tc_fence_before();
    }
  softmax_done:;
  }

  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

int tokens_per_tile(int Hq, int Hkv) { return kBM / (Hq / Hkv); }

int64_t max_items(int64_t Tq, int64_t B, int Hq, int Hkv) {
  const int64_t per = 2 * tokens_per_tile(Hq, Hkv);
  // each sequence's last item may be ragged
  return Tq / per + (B < Tq ? B : Tq) + 1;
}

template <int D>
cudaError_t launch(const PromptMaps& maps, const PromptArgs& a, int grid, cudaStream_t stream) {
  const int smem = PromptLayout<D>::kSmem + 1024;
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  return launch_k(prompt_kernel<D>, dim3(grid), dim3(kPromptThreads), static_cast<size_t>(smem),
                  stream, maps, a);
}

}  // namespace

size_t prompt_workspace_bytes(int64_t Tq, int64_t B, int Hq, int Hkv, int, int) {
  return 256 + static_cast<size_t>(max_items(Tq, B, Hq, Hkv)) * sizeof(PromptItem);
}

cudaError_t launch_prompt(const PromptParams& p, int num_sms, cudaStream_t stream,
                          std::string* err) {
  PromptArgs a = {};
  a.p = p;
  a.G = p.Hq / p.Hkv;
  a.TB = tokens_per_tile(p.Hq, p.Hkv);
  a.n_items = static_cast<const int*>(p.workspace);
  a.items = reinterpret_cast<const PromptItem*>(static_cast<const char*>(p.workspace) + 256);
  a.budget_ns = static_cast<unsigned long long>(option(MXQ_OPT_WAIT_BUDGET_NS));
  a.inject_stall = static_cast<int>(option(MXQ_OPT_INJECT_STALL));
  // [n, heads, D] as (D, heads, n); a dimension of one takes any legal stride
  auto map3 = [&](CUtensorMap* m, const void* base, int heads, int64_t n, int64_t st, int64_t sh,
                  int box_h, int box_n) {
    const int64_t row = static_cast<int64_t>(p.D) * 2;
    const uint64_t dims[3] = {static_cast<uint64_t>(p.D), static_cast<uint64_t>(heads),
                              static_cast<uint64_t>(n)};
    const uint64_t strides[2] = {static_cast<uint64_t>(heads > 1 ? sh * 2 : row),
                                 static_cast<uint64_t>(n > 1 ? st * 2 : row)};
    const uint32_t box[3] = {64, static_cast<uint32_t>(box_h), static_cast<uint32_t>(box_n)};
    return make_map_bf16_3d(m, base, dims, strides, box, err);
  };
  PromptMaps maps;
  // without keys no block is loaded: any tensor serves as the maps' base
  const bool keys = p.Tk > 0;
  if (!map3(&maps.q, p.q, p.Hq, p.Tq, p.q_t, p.q_h, a.G, a.TB) ||
      !map3(&maps.k, keys ? p.k : p.q, p.Hkv, keys ? p.Tk : 1, p.k_t, keys ? p.k_h : p.D, 1, kBM) ||
      !map3(&maps.v, keys ? p.v : p.q, p.Hkv, keys ? p.Tk : 1, p.v_t, keys ? p.v_h : p.D, 1, kBM))
    return cudaErrorInvalidValue;
  const cudaError_t e =
      launch_k(prompt_plan_kernel, dim3(1), dim3(1024), 0, stream, p, 2 * a.TB,
               static_cast<int*>(p.workspace), const_cast<PromptItem*>(a.items),
               static_cast<int>(max_items(p.Tq, p.B, p.Hq, p.Hkv)));
  if (e != cudaSuccess) return e;
  const int64_t most = max_items(p.Tq, p.B, p.Hq, p.Hkv) * p.Hkv;
  const int grid = static_cast<int>(most < num_sms ? most : num_sms);
  return p.D == 128 ? launch<128>(maps, a, grid, stream) : launch<64>(maps, a, grid, stream);
}

}  // namespace mxq
