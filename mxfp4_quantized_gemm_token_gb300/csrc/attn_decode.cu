// attn_decode.cu — attention of one new token per sequence over a paged
// key/value cache.
//
// Every visible key and value is read once (2 D elements a key and key/value
// head) for 4 D multiply-adds per query head: HBM-bound, so the kernel is built
// around keeping loads in flight.
//
// Work.  A sequence's visible keys are cut into steps of KS keys; the steps of
// all sequences form one line, cut into equal parts whatever the lengths, and a
// (part, key/value head) pair is one warp's.  The heads of a part are at work at
// the same time: their rows of a key are adjacent in memory.  (With all heads' steps on
// one line, each head at another place of a sequence, the 128-byte rows of an e4m3
// cache came at 4.8 TB/s on some devices.)  A warp is on its own: its
// ring of shared-memory stages filled with 16-byte asynchronous copies, its own
// running maximum, sum and accumulators, no block-wide barrier.  A
// sequence that lies inside one part is written out by its warp; the others
// leave at most two partial results per warp in the workspace, which
// a second kernel joins in a fixed order.  A part's end that falls into a
// sequence no longer than a part moves to the nearer end of it: splitting a few steps
// costs more than it balances (24 sequences of 50-250 keys: 12.3 us; whole up to two
// parts' steps 13.1, up to eight steps whatever the parts 16.0).  Where no sequence can be long, by
// the page table's width or the window, all stay whole and there is no join.
//
// Arithmetic.  The G query heads of a key/value head are the rows of 16-row
// tensor-core products (mma.sync m16n8k16: with at most 16 rows to a key the
// products take a fraction of the load time, and their operands come from
// registers and ldmatrix without a pass through tensor memory); every 16 query
// heads of a larger G count as a head of their own above.  Scores and outputs
// accumulate in fp32.  The reference a row's weights are relative to is raised only
// when a score exceeds it by 2^8
// in the exponent, so most steps need no exchange between lanes.
//   bf16 cache: bf16 products, weights rounded to bf16.
//   e4m3 cache: keys and values converted to f16 (exact), q scaled per row by
//   a power of two to use f16's range (exact for elements within 2^31 of the
//   row's largest), weights rounded to f16.
// The order of the elements of D inside a product is free as long as both
// operands agree: the e4m3 path takes the order that ldmatrix delivers.
//
// Measured.  64 sequences of 5-8192 keys, 32 query and 8 key/value heads of 128, bf16:
// 158 us, 6.6 TB/s of keys and values, 97 % of a plain copy's rate.  16 sequences
// of 9000-32768 keys, 64 / 8 heads, e4m3: 110 us, 5.8 TB/s.  D 64, 64 / 8 heads, whose rows
// are half as long: the 64 sequences 91 us, 5.7 TB/s, in e4m3 66 us, 4.0 TB/s; the 16 in
// e4m3 78 us, 4.2 TB/s.  One sequence of 1500 keys: 10.4 us; 128 sequences with a window
// of 128 keys, D 64: 13.9 us: there the chain length -> page -> key, a load each, and the
// launches count.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>

#include "attn.h"
#include "attn_math.cuh"
#include "internal.h"

namespace mxq {

namespace {

constexpr int kWarps = 8;
constexpr int kEntries = 2048;      // entries of the shared prefix table
constexpr int kRows = 16;           // rows of a product
constexpr int kAllWhole = 9;        // calls whose sequences have at most this many steps: all whole
constexpr int kWhole = 8;           // others: sequences of at most this many steps and a part's

struct DecodeArgs {
  DecodeParams p;
  int G, tiles, rows;               // per kv head: query heads, 16-row tiles; rows stored
  int chunk, entries;               // sequences per entry of the prefix table, its entries
  int parts;                        // of the line, at most
  int min_steps;
  int join_rows;                    // rows of a block of the join: 8, or 1
  bool all_whole;                   // no sequence is split
  bool alike;                       // both caches have the same page and token strides
  int64_t* cum;                     // workspace: steps before each sequence [B + 1], then `per`
  float2* part_ml;                  // [task][2][rows]
  float* part_o;                    // [task][2][rows][D]
};

template <int D, bool FP8>
struct DecodeShape {
  static constexpr int kRowBytes = FP8 ? D : 2 * D;
  static constexpr int KS = kRowBytes == 256 ? 16 : 32;        // keys per step
  static constexpr int kTile = KS * kRowBytes;                 // K (or V) of a step
  static constexpr int kStages = kTile == 4096 ? 3 : 6;
  static constexpr int kLPR = kRowBytes / 16;                  // lanes per row
  static constexpr int kSmem =
      kWarps * kStages * 2 * kTile + 12 * kEntries + 4 * kWarps * kStages;
};

struct SeqRange {
  int lo, len, first, steps;        // visible keys [lo, len); the first step's key; its steps
};

// The visible keys of a sequence of `len` keys, in steps from a multiple of 16; at
// least one step (without keys), so that every output is written.
template <int KS>
__device__ __forceinline__ SeqRange seq_steps(const DecodeParams& p, int len) {
  SeqRange r;
  r.len = min(max(len, 0), static_cast<int>(p.max_pages * p.page_size));
  r.lo = p.window > 0 ? max(0, r.len - p.window) : 0;
  r.first = r.lo & ~15;
  r.steps = max(1, (r.len - r.first + KS - 1) / KS);
  return r;
}

// byte offset of 16-byte chunk c of row r in a tile, conflict-free for ldmatrix
template <int ROWB>
__device__ __forceinline__ uint32_t tile_off(int r, int c) {
  if constexpr (ROWB == 64)
    return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  else
    return r * ROWB + ((c ^ (r & 7)) << 4);
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <bool F16>
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void prefetch(const void* at) {
  asm volatile("prefetch.global.L1 [%0];" ::"l"(at));
}

// A place on the line of steps.
struct Cursor {
  int b, step;
  SeqRange s;
};

// a / b for a >= 0, b > 0: 64-bit division only where it is needed
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// steps of the longest sequence that stays whole, with `per` steps a part
__device__ __forceinline__ int whole_steps(int64_t per) {
  return static_cast<int>(min(static_cast<int64_t>(kWhole), per));
}

// lens: the lengths in shared memory, where the prefix table has an entry for each sequence
__device__ __forceinline__ int length_of(const DecodeArgs& a, const int* lens, int b) {
  return a.chunk == 1 ? lens[b] : a.p.seq_lens[b];
}

template <int KS>
__device__ __forceinline__ void advance(Cursor& c, const DecodeArgs& a, const int* lens) {
  if (++c.step < c.s.steps) return;
  c.step = 0;
  if (++c.b < a.p.B) c.s = seq_steps<KS>(a.p, length_of(a, lens, c.b));
}

template <int D, bool FP8>
__global__ void __launch_bounds__(32 * kWarps, 1) decode_kernel(const DecodeArgs a) {
  using S = DecodeShape<D, FP8>;
  constexpr int KS = S::KS, ROWB = S::kRowBytes, ST = S::kStages;
  constexpr int NT = KS / 8;                           // score tiles of 8 keys
  constexpr int DT = D / 8;                            // output tiles of 8 elements
  extern __shared__ __align__(128) uint8_t smem[];
  const DecodeParams& p = a.p;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int quad = lane & 3, r0 = lane >> 2;
  int64_t* table = reinterpret_cast<int64_t*>(smem + kWarps * ST * 2 * S::kTile);
  int* lens = reinterpret_cast<int*>(table + kEntries);
  uint32_t* masks = reinterpret_cast<uint32_t*>(lens + kEntries) + warp * ST;
  __shared__ int64_t warp_sum[kWarps];
  __shared__ int warp_longest[kWarps];
  pdl_wait();
  pdl_launch_dependents();

  // ---- steps before each entry (a.chunk sequences) of the prefix table
  const int per_thread = (a.entries + 32 * kWarps - 1) / (32 * kWarps);
  const int e0 = threadIdx.x * per_thread;
  int64_t mine = 0;
  int longest = 0;
  for (int e = e0; e < min(a.entries, e0 + per_thread); ++e)
    for (int b = e * a.chunk; b < min(p.B, (e + 1) * a.chunk); ++b) {
      const int len = p.seq_lens[b];
      if (a.chunk == 1) lens[b] = len;
      const SeqRange r = seq_steps<KS>(p, len);
      if (len != r.len && blockIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
      mine += r.steps;
      longest = max(longest, r.steps);
    }
  longest = __reduce_max_sync(0xffffffffu, longest);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sum[warp] = incl, warp_longest[warp] = longest;
  __syncthreads();
  int64_t before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
    longest = max(longest, warp_longest[w]);
  }
  const int heads = p.Hkv * a.tiles;
  const int workers = gridDim.x * kWarps;
  int64_t per = max(divide(total + a.parts - 1, a.parts), static_cast<int64_t>(a.min_steps));
  // where all stay whole, a part has room for the longest, or some would get two
  if (a.all_whole && per < longest) per = longest;
  const int whole = a.all_whole ? longest : whole_steps(per);
  for (int e = e0; e < min(a.entries, e0 + per_thread); ++e) {
    table[e] = before;
    for (int b = e * a.chunk; b < min(p.B, (e + 1) * a.chunk); ++b) {
      if (blockIdx.x == 0) a.cum[b] = before;
      if (blockIdx.x == 0 || a.chunk * per_thread > 1)
        before += seq_steps<KS>(p, length_of(a, lens, b)).steps;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.cum[p.B] = total;
    a.cum[p.B + 1] = per;
  }
  __syncthreads();

  // the part's end `pos` on the line, moved out of a short sequence, and where that
  // is; `at`: steps before sequence c->b
  auto locate = [&](int64_t pos, Cursor* c, int64_t at) {
    if (pos >= total) return total;
    while (at + c->s.steps <= pos) {
      at += c->s.steps;
      ++c->b;
      c->s = seq_steps<KS>(p, length_of(a, lens, c->b));
    }
    const int n = c->s.steps;
    c->step = static_cast<int>(pos - at);
    if (n <= whole && c->step > 0) {
      pos -= c->step;
      const bool up = 2 * c->step >= n;
      c->step = up ? n - 1 : 0;
      if (up) {
        pos += n;
        advance<KS>(*c, a, lens);
      }
    }
    return pos;
  };
  // the last entry of the prefix table at or before a position, 32 candidates at a time
  auto entry = [&](int64_t pos, int lo) {
    for (int n = a.entries - lo; n > 1;) {
      const int step = (n + 31) >> 5, k = lane * step;
      const uint32_t at = __ballot_sync(0xffffffffu, k < n && table[lo + k] <= pos);
      const int skip = max(0, __popc(at) - 1) * step;
      lo += skip;
      n = min(step, n - skip);
    }
    return lo;
  };
  const uint32_t ring = smem_u32(smem) + warp * ST * 2 * S::kTile;
  constexpr int es = FP8 ? 1 : 2;
  const int row_in = lane / S::kLPR, ch_in = lane % S::kLPR;
  constexpr int kRPI = 32 / S::kLPR;                   // rows per copy instruction
  const int64_t tasks = divide(total + per - 1, per) * heads;

  // ---- this warp's tasks (one, unless there are more heads than warps).  They are
  // spread over the SMs; with 256-byte rows and work for (nearly) every warp the heads of a part
  // run on one SM (64 sequences of 5-8192 keys: 157.7 us, spread 161.1; an e4m3 cache's
  // 128-byte rows: 111.4 and 109.3).
  const bool together = ROWB == 256 && tasks > workers - static_cast<int>(gridDim.x);
  const int first = together ? blockIdx.x * kWarps + warp : warp * gridDim.x + blockIdx.x;
  for (int64_t task = first; task < tasks; task += workers) {
    const int64_t part = divide(task, heads);
    const int head = static_cast<int>(task - part * heads);
    const int hk = head / a.tiles, tile = head - hk * a.tiles;
    const int64_t raw0 = part * per;
    Cursor in, end;                                      // of the copies
    const int e_in = entry(raw0, 0);
    in.b = e_in * a.chunk;
    in.s = seq_steps<KS>(p, length_of(a, lens, in.b));
    end.b = in.b, end.s = in.s;
    int64_t at_end = table[e_in];
    const int64_t s0 = locate(raw0, &in, at_end);
    const int64_t raw1 = min(raw0 + per, total - 1);
    if (e_in + 1 < a.entries && table[e_in + 1] <= raw1) {
      const int e = entry(raw1, e_in + 1);
      end.b = e * a.chunk;
      end.s = seq_steps<KS>(p, length_of(a, lens, end.b));
      at_end = table[e];
    }
    const int64_t s1 = locate(raw0 + per, &end, at_end);
    if (s0 >= s1) continue;
    {
      // on their way while the pages are looked up: q and what its output needs
      const int gr = tile * kRows + (lane & 15);
      if (gr < a.G) {
        const int hq = hk * a.G + gr;
        if ((lane >> 4) * 64 < D)
          prefetch(static_cast<const __nv_bfloat16*>(p.q) + in.b * p.q_b +
                   static_cast<int64_t>(hq) * p.q_h + (lane >> 4) * 64);
        if (lane < 16 && p.sinks != nullptr) prefetch(p.sinks + hq);
      }
    }
    Cursor at = in;                                      // of the arithmetic
    const char* k_base =
        static_cast<const char*>(p.k_cache) + (hk * p.ck_h) * es + ch_in * 16;
    const char* v_base =
        static_cast<const char*>(p.v_cache) + (hk * p.cv_h) * es + ch_in * 16;

    // the page of this lane's key of a step: looked up two steps before it is copied
    struct Spot {
      int page, off;
      bool seen;
    };
    auto look_up = [&]() {
      Spot r = {0, 0, false};
      const int key = in.s.first + in.step * KS + lane;
      r.seen = lane < KS && key >= in.s.lo && key < in.s.len;
      if (r.seen) {
        const uint32_t n = static_cast<uint32_t>(key) / static_cast<uint32_t>(p.page_size);
        r.off = key - static_cast<int>(n) * p.page_size;
        r.page = __ldg(p.page_table + in.b * p.ld_table + n);
      }
      return r;
    };
    int64_t left = s1 - s0;                              // steps still to be copied
    uint32_t fill = 0;
    Spot now = {0, 0, false}, next = now;
    auto copy_step = [&]() {
      if (left > 0) {
        int page = now.page, off = now.off;
        const bool ok = now.seen && static_cast<uint32_t>(page) < static_cast<uint32_t>(p.pages);
        if (now.seen && !ok) {
          atomicOr(p.status, kStatusBadIndex);
          page = off = 0;
        }
        const uint32_t mask = __ballot_sync(0xffffffffu, ok);
        const int st = fill % ST;
        if (lane == 0) masks[st] = mask;
        const uint32_t dst = ring + st * 2 * S::kTile;
        // the lane's key's row, in both caches if they are laid out alike
        const int64_t ko = (page * p.ck_p + off * p.ck_t) * es;
        if (a.alike) {
#pragma unroll
          for (int i = 0; i < KS / kRPI; ++i) {
            const int r = i * kRPI + row_in;
            const int64_t from = __shfl_sync(0xffffffffu, ko, r);
            const uint32_t d = dst + tile_off<ROWB>(r, ch_in);
            cp16(d, k_base + from, (mask >> r) & 1);
            cp16(d + S::kTile, v_base + from, (mask >> r) & 1);
          }
        } else {
          const int64_t vo = (page * p.cv_p + off * p.cv_t) * es;
#pragma unroll
          for (int i = 0; i < KS / kRPI; ++i) {
            const int r = i * kRPI + row_in;
            const uint32_t d = dst + tile_off<ROWB>(r, ch_in);
            cp16(d, k_base + __shfl_sync(0xffffffffu, ko, r), (mask >> r) & 1);
            cp16(d + S::kTile, v_base + __shfl_sync(0xffffffffu, vo, r), (mask >> r) & 1);
          }
        }
        ++fill;
        now = next;
        if (--left > 1) {
          advance<KS>(in, a, lens);
          next = look_up();
        }
      }
      cp_commit();
    };
    now = look_up();
    if (left > 1) {
      advance<KS>(in, a, lens);
      next = look_up();
    }
#pragma unroll 1
    for (int i = 0; i < ST - 1; ++i) copy_step();

    uint32_t qf[D / 16][4];                              // rows r0, r0 + 8 of q
    float o[DT][4];
    float m[2], l[2], cs[2];
    uint32_t use = 0;
    bool fresh = true, opened = false;                   // opened: the sequence began in this part
    for (int64_t s = s0; s < s1; ++s, ++use) {
      if (fresh) {
        // a new sequence: its q, and nothing summed yet
        fresh = false;
        opened = at.step == 0;
        const float ks = FP8 && p.k_scale != nullptr ? __ldg(p.k_scale + hk) : 1.f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int gr = tile * kRows + r0 + 8 * half;
          const bool in_group = gr < a.G;
          const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + at.b * p.q_b +
                                   static_cast<int64_t>(hk * a.G + gr) * p.q_h;
          float unscale = 1.f;
          if constexpr (FP8) {
            float big = 0.f;
            uint2 raw[D / 16];
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              raw[k] = in_group ? __ldg(reinterpret_cast<const uint2*>(q + 16 * k + 4 * quad))
                                : make_uint2(0u, 0u);
              const uint32_t w[2] = {raw[k].x, raw[k].y};
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                big = fmaxf(big, fabsf(__uint_as_float(w[i] << 16)));
                big = fmaxf(big, fabsf(__uint_as_float(w[i] & 0xFFFF0000u)));
              }
            }
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
            // the power of two that brings the largest to [2^14, 2^15) (a largest below
            // 2^-86: nearer to it; both powers are normal numbers)
            const int e = big > 0.f && big < INFINITY ? min(14 - ilogbf(big), 100) : 0;
            // the key scale's sign goes into q, and so does a scale of 0 or NaN: what
            // multiplies the scores below stays positive and keeps a masked key's -inf
            const float up = (ks > 0.f ? 1.f : ks < 0.f ? -1.f : ks) * ldexpf(1.f, e);
            unscale = ldexpf(1.f, -e);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t w[2] = {raw[k].x, raw[k].y};
#pragma unroll
              for (int i = 0; i < 2; ++i)
                qf[k][half + 2 * i] = f16x2(__uint_as_float(w[i] << 16) * up,
                                            __uint_as_float(w[i] & 0xFFFF0000u) * up);
            }
          } else {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                qf[k][half + 2 * i] =
                    in_group
                        ? __ldg(reinterpret_cast<const uint32_t*>(q + 16 * k + 8 * i + 2 * quad))
                        : 0u;
          }
          if constexpr (FP8)
            // the scores of the scaled q are below 2^32: 1e-30 of them is nothing
            cs[half] = fmaxf(p.scale * fabsf(ks) * kLog2e * unscale, 1e-30f);
          else
            cs[half] = p.scale * kLog2e;
          m[half] = -INFINITY;
          l[half] = 0.f;
        }
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[t][i] = 0.f;
      }
      cp_wait<ST - 2>();
      __syncwarp();
      copy_step();                                       // into the stage used one step ago
      const int st = use % ST;
      const uint32_t mask = masks[st];
      const uint32_t kt = ring + st * 2 * S::kTile, vt = kt + S::kTile;

      // ---- scores: rows x keys
      float x[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[n][i] = 0.f;
      // (elements outside, keys inside: the products that follow one another are independent)
#pragma unroll
      for (int k = 0; k < D / 16; k += FP8 ? 2 : 1) {
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
          uint32_t f[4];
          if constexpr (FP8) {
            // matrices: keys 8n.. and 8(n+1).. of chunk k (16 elements), then of k + 1
            ldsm4(kt + tile_off<ROWB>(8 * n + (lane & 15), k + (lane >> 4)), f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t b0, b1;
              e4m3x4_f16(f[i], &b0, &b1);
              mma16816<true>(x[n + (i & 1)], qf[k + (i >> 1)], b0, b1);
            }
          } else {
            // matrices: (keys 8n.., chunks 2k and 2k + 1), (keys 8(n+1).., the same)
            ldsm4(kt + tile_off<ROWB>(8 * n + ((lane >> 4) << 3) + (lane & 7),
                                      2 * k + ((lane >> 3) & 1)), f);
            mma16816<false>(x[n], qf[k], f[0], f[1]);
            mma16816<false>(x[n + 1], qf[k], f[2], f[3]);
          }
        }
      }

      // ---- weights, relative to the reference m (of the unscaled scores)
      constexpr uint32_t kAll = KS == 32 ? 0xffffffffu : (1u << KS) - 1;
      if (mask != kAll) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!((mask >> (8 * n + 2 * quad + (i & 1))) & 1)) x[n][i] = -INFINITY;
      }
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) mx[h] = fmaxf(mx[h], fmaxf(x[n][2 * h], x[n][2 * h + 1]));
      if (__any_sync(0xffffffffu, (mx[0] - m[0]) * cs[0] > 8.f || (mx[1] - m[1]) * cs[1] > 8.f ||
                                      (m[0] == -INFINITY && mx[0] > m[0]) ||
                                      (m[1] == -INFINITY && mx[1] > m[1]))) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
          const float n = fmaxf(m[h], mx[h]);
          const float f = m[h] == -INFINITY ? 0.f : ex2((m[h] - n) * cs[h]);
          m[h] = n;
          l[h] *= f;
#pragma unroll
          for (int t = 0; t < DT; ++t) {
            o[t][2 * h] *= f;
            o[t][2 * h + 1] *= f;
          }
        }
      }
      const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0] * cs[0],
                            m[1] == -INFINITY ? 0.f : m[1] * cs[1]};
      uint32_t pf[KS / 16][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[n][i] = ex2(fmaf(x[n][i], cs[i >> 1], -ref[i >> 1]));
          l[i >> 1] += x[n][i];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
          pf[n / 2][h + 2 * (n & 1)] = FP8 ? f16x2(x[n][2 * h], x[n][2 * h + 1])
                                           : bf16x2(x[n][2 * h], x[n][2 * h + 1]);
      }

      // ---- values
#pragma unroll
      for (int kk = 0; kk < KS / 16; ++kk) {
        // matrices: keys 16kk.. and 16kk + 8.. of chunk c, then of c + 1
        const int r = 16 * kk + (lane & 15);
        constexpr int kChunks = ROWB / 16;
#pragma unroll
        for (int c = 0; c < kChunks; c += 2) {
          uint32_t f[4];
          ldsm4_t(vt + tile_off<ROWB>(r, c + (lane >> 4)), f);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if constexpr (FP8) {
              // a register holds keys 2q, 2q + 1 of two elements: even elements
              // make one output tile, odd ones the next
              uint32_t e0, o0, e1, o1;
              e4m3x4_f16(__byte_perm(f[2 * i], 0, 0x3120), &e0, &o0);
              e4m3x4_f16(__byte_perm(f[2 * i + 1], 0, 0x3120), &e1, &o1);
              mma16816<true>(o[2 * (c + i)], pf[kk], e0, e1);
              mma16816<true>(o[2 * (c + i) + 1], pf[kk], o0, o1);
            } else {
              mma16816<false>(o[c + i], pf[kk], f[2 * i], f[2 * i + 1]);
            }
          }
        }
      }

      // ---- the sequence's or the part's end
      const bool closed = at.step + 1 == at.s.steps;
      if (!closed && s + 1 < s1) {
        ++at.step;
        continue;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        const int gl = r0 + 8 * h, gr = tile * kRows + gl;
        if (gr >= a.G) continue;
        const float top = m[h] == -INFINITY ? m[h] : m[h] * cs[h];
        if (opened && closed) {
          const int hq = hk * a.G + gr;
          const RowEnd end = finish_row(top * kLn2, l[h], p.sinks ? p.sinks + hq : nullptr);
          const float f = end.factor * (p.v_scale != nullptr ? __ldg(p.v_scale + hk) : 1.f);
          __nv_bfloat16* dst =
              static_cast<__nv_bfloat16*>(p.out) + at.b * p.o_b + static_cast<int64_t>(hq) * p.o_h;
#pragma unroll
          for (int t = 0; t < DT; t += 2) {
            if constexpr (FP8) {
              *reinterpret_cast<uint2*>(dst + 8 * t + 4 * quad) =
                  make_uint2(bf16x2(o[t][2 * h] * f, o[t + 1][2 * h] * f),
                             bf16x2(o[t][2 * h + 1] * f, o[t + 1][2 * h + 1] * f));
            } else {
              *reinterpret_cast<uint32_t*>(dst + 8 * t + 2 * quad) =
                  bf16x2(o[t][2 * h] * f, o[t][2 * h + 1] * f);
              *reinterpret_cast<uint32_t*>(dst + 8 * t + 8 + 2 * quad) =
                  bf16x2(o[t + 1][2 * h] * f, o[t + 1][2 * h + 1] * f);
            }
          }
          if (p.lse != nullptr && quad == 0)
            p.lse[static_cast<int64_t>(at.b) * p.Hq + hq] = end.lse;
        } else {
          // a sequence that begins after the part's (unmoved) begin goes to slot 1 (parts
          // are split at all only with a warp for each task)
          const int64_t slot = (task * 2 + (opened && raw0 < s - at.step ? 1 : 0)) * a.rows + gl;
          if (quad == 0) a.part_ml[slot] = make_float2(top, l[h]);
          float* dst = a.part_o + slot * D;
#pragma unroll
          for (int t = 0; t < DT; t += 2) {
            if constexpr (FP8) {
              *reinterpret_cast<float4*>(dst + 8 * t + 4 * quad) = make_float4(
                  o[t][2 * h], o[t + 1][2 * h], o[t][2 * h + 1], o[t + 1][2 * h + 1]);
            } else {
              *reinterpret_cast<float2*>(dst + 8 * t + 2 * quad) =
                  make_float2(o[t][2 * h], o[t][2 * h + 1]);
              *reinterpret_cast<float2*>(dst + 8 * t + 8 + 2 * quad) =
                  make_float2(o[t + 1][2 * h], o[t + 1][2 * h + 1]);
            }
          }
        }
      }
      fresh = true;
      advance<KS>(at, a, lens);
    }
    cp_wait<0>();
    __syncwarp();
  }
}

// Joins the partial results of the rows of sequences that several parts share, in the
// parts' order: out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i.  A warp takes a row,
// reading eight parts at a time; a row of more than 32 parts, and of more than four
// where there are too few rows to fill the SMs with warps, is shared by a
// block's eight warps (24 parts of each of 32 rows: 4.9 us by one warp a row).
template <int D>
struct JoinRow {
  static constexpr int N = D / 32;
  float m = -INFINITY, l = 0.f, o[N] = {};
  __device__ __forceinline__ void add(float pm, float pl, const float* v) {
    // a part whose scores are all NaN has no reference, but a sum: it counts
    const float n = fmaxf(m, pm), ref = n == -INFINITY ? 0.f : n;
    const float f = ex2(m - ref), g = ex2(pm - ref);
    l = l * f + pl * g;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = o[i] * f + v[i] * g;
    m = n;
  }
  // parts w, w + stride, ... up to w1 of the sequence that begins at u0
  __device__ __forceinline__ void read(const DecodeArgs& a, int64_t w, int64_t w1, int stride,
                                       int64_t per, int64_t u0, int head, int row, int lane) {
    const int heads = a.p.Hkv * a.tiles;
    constexpr int U = 8;
    for (; w <= w1; w += U * stride) {
      float2 ml[U];
      float v[U][N];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t k = w + u * stride;
        ml[u] = make_float2(-INFINITY, 0.f);
        if (k > w1) continue;
        const int64_t slot = ((k * heads + head) * 2 + (k * per < u0 ? 1 : 0)) * a.rows + row;
        ml[u] = a.part_ml[slot];
#pragma unroll
        for (int i = 0; i < N; ++i) v[u][i] = a.part_o[slot * D + lane + 32 * i];
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (w + u * stride <= w1) add(ml[u].x, ml[u].y, v[u]);
    }
  }
  __device__ __forceinline__ void write(const DecodeArgs& a, int b, int hk, int gr, int lane) {
    const DecodeParams& p = a.p;
    const int hq = hk * a.G + gr;
    const RowEnd end = finish_row(m * kLn2, l, p.sinks ? p.sinks + hq : nullptr);
    const float f = end.factor * (p.v_scale != nullptr ? __ldg(p.v_scale + hk) : 1.f);
    __nv_bfloat16* dst =
        static_cast<__nv_bfloat16*>(p.out) + b * p.o_b + static_cast<int64_t>(hq) * p.o_h;
#pragma unroll
    for (int i = 0; i < N; ++i) dst[lane + 32 * i] = __float2bfloat16_rn(o[i] * f);
    if (p.lse != nullptr && lane == 0) p.lse[static_cast<int64_t>(b) * p.Hq + hq] = end.lse;
  }
};

template <int D>
__global__ void __launch_bounds__(32 * kWarps) decode_join_kernel(const DecodeArgs a) {
  constexpr int N = D / 32;
  const int alone = a.join_rows == 1 ? 4 : 32;         // parts that one warp reads
  const DecodeParams& p = a.p;
  __shared__ float so[kWarps][D];
  __shared__ float2 sml[kWarps];
  __shared__ int shared_rows;                          // bit k: row k needs the block
  if (threadIdx.x == 0) shared_rows = 0;
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int heads = p.Hkv * a.tiles;
  const int64_t per = a.cum[p.B + 1];
  struct Where {
    int b, head, hk, gr, row;
    int64_t u0, w0, w1;
    bool split;
  };
  auto where = [&](int64_t item) {
    Where r = {};
    if (item >= static_cast<int64_t>(p.B) * heads * a.rows) return r;
    const int64_t unit = divide(item, a.rows);
    r.row = static_cast<int>(item - unit * a.rows);
    r.b = static_cast<int>(divide(unit, heads));
    r.head = static_cast<int>(unit - static_cast<int64_t>(r.b) * heads);
    r.hk = r.head / a.tiles;
    r.gr = (r.head - r.hk * a.tiles) * kRows + r.row;
    r.u0 = a.cum[r.b];
    const int64_t steps = a.cum[r.b + 1] - r.u0;
    r.w0 = divide(r.u0, per);
    r.w1 = divide(r.u0 + steps - 1, per);
    r.split = steps > whole_steps(per) && r.w0 < r.w1 && r.gr < a.G;
    return r;
  };
  const int64_t first = static_cast<int64_t>(blockIdx.x) * a.join_rows;
  if (warp < a.join_rows) {
    const Where mine = where(first + warp);
    if (mine.split && mine.w1 - mine.w0 < alone) {
      JoinRow<D> r;
      r.read(a, mine.w0, mine.w1, 1, per, mine.u0, mine.head, mine.row, lane);
      r.write(a, mine.b, mine.hk, mine.gr, lane);
    } else if (mine.split && lane == 0) {
      atomicOr(&shared_rows, 1 << warp);
    }
  }
  __syncthreads();
  for (int k = 0; k < a.join_rows; ++k) {
    if (!((shared_rows >> k) & 1)) continue;
    const Where at = where(first + k);
    JoinRow<D> r;
    r.read(a, at.w0 + warp, at.w1, kWarps, per, at.u0, at.head, at.row, lane);
    if (lane == 0) sml[warp] = make_float2(r.m, r.l);
#pragma unroll
    for (int i = 0; i < N; ++i) so[warp][lane + 32 * i] = r.o[i];
    __syncthreads();
    if (warp == 0) {
      JoinRow<D> all;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        float v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = so[w][lane + 32 * i];
        all.add(sml[w].x, sml[w].y, v);
      }
      all.write(a, at.b, at.hk, at.gr, lane);
    }
    __syncthreads();
  }
}

int stored_rows(int Hq, int Hkv) { return std::min(kRows, Hq / Hkv); }

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// bytes of the workspace before the partial maxima, and before the partial outputs
size_t cum_bytes(int64_t B) { return round256(static_cast<size_t>(B + 2) * 8); }
size_t ml_bytes(int rows, int num_sms) {
  return round256(static_cast<size_t>(num_sms) * kWarps * 2 * rows * sizeof(float2));
}

template <int D, bool FP8>
cudaError_t launch(const DecodeArgs& a, int grid, cudaStream_t stream) {
  using S = DecodeShape<D, FP8>;
  static_assert(S::kSmem <= 226 * 1024, "shared memory over budget");
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(decode_kernel<D, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             S::kSmem);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  DecodeArgs b = a;
  b.min_steps = std::max(1, 32 / S::KS);
  b.parts = std::max(1, grid * kWarps / (a.p.Hkv * a.tiles));
  // Where no sequence can have more steps there is nothing to join, and a join's launch takes
  // as long as eight steps (a window of 128 keys, D 128, 128 sequences: 32.0 us split and
  // joined, 23.1 whole; 4 sequences: 10.0 and 10.8).
  int64_t keys = a.p.max_pages * a.p.page_size;
  if (a.p.window > 0) keys = std::min<int64_t>(keys, static_cast<int64_t>(a.p.window) + 15);
  b.all_whole = keys <= kAllWhole * S::KS;
  e = launch_k(decode_kernel<D, FP8>, dim3(grid), dim3(32 * kWarps),
               static_cast<size_t>(S::kSmem), stream, b);
  if (e != cudaSuccess || b.all_whole) return e;
  const int64_t rows = static_cast<int64_t>(a.p.B) * a.p.Hkv * a.tiles * a.rows;
  b.join_rows = rows <= 4 * grid ? 1 : kWarps;
  return launch_k(decode_join_kernel<D>,
                  dim3(static_cast<unsigned>((rows + b.join_rows - 1) / b.join_rows)),
                  dim3(32 * kWarps), 0, stream, b);
}

}  // namespace

size_t decode_workspace_bytes(int64_t B, int Hq, int Hkv, int D, int num_sms) {
  const int rows = stored_rows(Hq, Hkv);
  return cum_bytes(B) + ml_bytes(rows, num_sms) +
         static_cast<size_t>(num_sms) * kWarps * 2 * rows * D * sizeof(float);
}

cudaError_t launch_decode(const DecodeParams& p, int num_sms, cudaStream_t stream) {
  DecodeArgs a = {};
  a.p = p;
  a.G = p.Hq / p.Hkv;
  a.tiles = (a.G + kRows - 1) / kRows;
  a.rows = stored_rows(p.Hq, p.Hkv);
  a.alike = p.ck_p == p.cv_p && p.ck_t == p.cv_t;
  a.chunk = (p.B + kEntries - 1) / kEntries;
  a.entries = (p.B + a.chunk - 1) / a.chunk;
  char* ws = static_cast<char*>(p.workspace);
  a.cum = reinterpret_cast<int64_t*>(ws);
  a.part_ml = reinterpret_cast<float2*>(ws + cum_bytes(p.B));
  a.part_o = reinterpret_cast<float*>(ws + cum_bytes(p.B) + ml_bytes(a.rows, num_sms));
  if (p.D == 128)
    return p.fp8 ? launch<128, true>(a, num_sms, stream) : launch<128, false>(a, num_sms, stream);
  return p.fp8 ? launch<64, true>(a, num_sms, stream) : launch<64, false>(a, num_sms, stream);
}

}  // namespace mxq
