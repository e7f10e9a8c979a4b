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
// the result does not depend on it.  (Two tiles in turn and a reference that is seldom
// raised are published techniques for attention on this generation.)
//
// Work.  A kernel of one block first lists the work items (sequence, pair of
// tiles, its blocks of keys) with the costliest first; the persistent CTAs
// take them in turn, in alternating direction, which balances lengths.  Where
// the longest item is longer than a CTA's share of all blocks (few rows, many keys), the
// blocks of all items form one line instead, cut into equal parts, one per CTA; items
// that parts share leave partial results in the workspace, at most two per
// CTA, and whichever warp is the last to finish its 32 rows of an item joins them,
// in the parts' order, so the result does not depend on who was last.  One
// sequence with enough rows needs no list: its items are in order as they stand.
//
// Bound.  Arithmetic: 4 D operations a visible (query head, key) pair, on the
// tensor cores at best.  One causal prompt of 8192 tokens, 32 query and 8 key/value
// heads of 128: 323 us, 1.70 PFLOP/s, 87 % of a plain bf16 product's burst rate (342-364 us
// when run for seconds, by the device: 87-93 % of its sustained rate under the power limit);
// the tensor pipe is busy 72 % of the time, the rest is the chain scores -> maximum ->
// weights -> product of each tile, ~3000 cycles for a block of both against 2048 of products;
// at D 64 ~2500 against 1280, and the same prompt takes 276 us (141 at the burst rate).
// 11 packed prompts of 8192 tokens: 80 us (42 at the burst rate), 65 at D 64 (21); here an
// item's beginning and end count, ~2 us.  Two chunks of 300 rows over 7892 keys, in pieces:
// 71 us (40).  One prompt of 2048 tokens is cut into pieces too: 65 us (18).
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

// One pair of tiles of a key/value head: tokens [q_row, q_row + ntok) of the packed
// queries, the first of which stands at key position at0 of its sequence's nk
// keys, against the key blocks [kb0, kb1).
struct __align__(16) PromptItem {
  int q_row, ntok, at0, k_row;
  int nk, kb0, kb1;
  int head;                          // + kPiece: only some of the item's blocks
};
constexpr int kPiece = 1 << 30;

// Where a piece's result goes, and who has the item's others: part w0 in its slot
// `first`, parts w0 + 1 .. w1 in their slot 0.
struct __align__(16) PromptPiece {
  int slot;                          // part * 2 + 0 or 1
  int w0, w1;
  int key;                           // 2 * (counter of the item's finished pieces) + first
};

// What the plan leaves at the head of the workspace.
struct __align__(8) PromptHeader {
  int n;                             // entries of the list
  int per;                           // blocks of a part; 0: whole items
};

constexpr int kRowsPerItem = 2 * kBM;
constexpr int kMinSplit = 8;         // items of at most this many blocks stay whole
constexpr int kMaxSplitItems = 16;   // items per SM above which all do
constexpr int kRankItems = 512;      // items of a call, before their heads, above which all do

struct PromptArgs {
  PromptParams p;
  PromptHeader* header;              // in the workspace; null: one sequence, no list
  PromptItem* list;                  // what the CTAs work on
  PromptPiece* pieces;               // for the list's entries; null: items stay whole
  int2* part;                        // each part's first entry, and one past its last
  int* done;                         // [item][8 warps]: finished pieces
  float2* part_ml;                   // [slot][256]: reference and sum
  float* part_o;                     // [slot][256][D]
  int cap;                           // room for items, before their heads
  int grid;                          // CTAs
  int G, TB;
  unsigned long long budget_ns;
  int inject_stall;
};

constexpr int kBuckets = 512;

__device__ __forceinline__ int item_blocks(const PromptItem& it) { return max(1, it.kb1 - it.kb0); }

// [start, start + len) of sequence b in cu, or nothing if it leaves [0, total]
__device__ __forceinline__ bool seq_range(const int32_t* cu, int b, int64_t total, int* start,
                                          int* len) {
  const int64_t a = cu[b], e = cu[b + 1];
  const bool ok = a >= 0 && e >= a && e <= total;
  *start = ok ? static_cast<int>(a) : 0;
  *len = ok ? static_cast<int>(e - a) : 0;
  return ok;
}

// Item i of a sequence.
__device__ __forceinline__ PromptItem make_item(const PromptParams& p, int tokens_per_item, int q0,
                                                int nq, int k0, int nk, int i) {
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
  it.head = 0;
  return it;
}

// Writes the list's entries of one item, for its heads first, first + step, ...: whole at
// rank * Hkv + head, or, with `per` blocks to a part, its pieces.  The line holds all
// items' blocks, heads inside items (an item without keys counts as one block); `before`
// of them, of one head, come before this item's.  The piece of item and head idx that
// lies in part w is entry idx + w: a part's are adjacent, and each is placed without the others.
__device__ __forceinline__ void list_item(const PromptArgs& a, PromptItem it, int rank, int before,
                                          int total, int per, int first, int step) {
  const int Hkv = a.p.Hkv;
  if (per == 0) {
    for (it.head = first; it.head < Hkv; it.head += step) a.list[rank * Hkv + it.head] = it;
    return;
  }
  const int n = item_blocks(it), kb1 = it.kb1, line = total * Hkv;
  const bool keys = it.kb1 > it.kb0;
  for (int h = first; h < Hkv; h += step) {
    const int idx = rank * Hkv + h, p0 = before * Hkv + h * n, p1 = p0 + n;
    const int w0 = p0 / per, w1 = (p1 - 1) / per;
    const bool whole = w0 == w1;
    if (!whole)
      for (int k = 0; k < 2; ++k) reinterpret_cast<int4*>(a.done)[idx * 2 + k] = {0, 0, 0, 0};
    it.head = h + (whole ? 0 : kPiece);
    for (int w = w0; w <= w1; ++w) {
      const int from = max(p0, w * per), to = min(p1, (w + 1) * per);
      if (keys) {
        it.kb1 = kb1 - (from - p0);
        it.kb0 = it.kb1 - (to - from);
      }
      a.list[idx + w] = it;
      if (!whole)
        a.pieces[idx + w] = {2 * w + (from == w * per ? 0 : 1), w0, w1,
                             2 * idx + (w0 * per < p0 ? 1 : 0)};
      if (from == w * per) a.part[w].x = idx + w;
      if (to == min(line, (w + 1) * per)) a.part[w].y = idx + w + 1;
    }
  }
}

// Lists the items, ordered by falling number of key blocks, and cuts them into pieces
// where one is too long.  An item's place is the number of items before it, by
// comparison with each: for up to kRankItems of them no longer than the passes and
// barriers of a sort, and the order, and with it the cuts, is always the same.  Bound by
// the latency of one block's few steps, a call's first use of each instruction among
// them: 5 us from the offsets to the kernel's first item (130 items; or 10 items cut into
// pieces, which took 9 us by a counting sort and three prefix sums).
__global__ void __launch_bounds__(1024) prompt_rank_kernel(const PromptArgs a) {
  const PromptParams& p = a.p;
  __shared__ __align__(16) unsigned long long keys[kRankItems];
  __shared__ PromptItem items[kRankItems];
  __shared__ int count, longest, all_blocks;
  for (int i = threadIdx.x; i < kRankItems; i += 1024) keys[i] = 0;
  if (threadIdx.x == 0) count = longest = all_blocks = 0;
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int b = warp; b < p.B; b += 32) {
    int q0, nq, k0, nk;
    const bool okq = seq_range(p.cu_q, b, p.Tq, &q0, &nq);
    const bool okk = seq_range(p.cu_k, b, p.Tk, &k0, &nk);
    if (!(okq && okk)) {
      if (lane == 0) atomicOr(p.status, kStatusBadIndex);
      continue;
    }
    const int n = (nq + 2 * a.TB - 1) / (2 * a.TB);
    int at = 0, sum = 0, most = 0;
    if (lane == 0) at = atomicAdd(&count, n);
    at = __shfl_sync(0xffffffffu, at, 0);
    for (int i = lane; i < n && at + i < a.cap; i += 32) {
      const PromptItem it = make_item(p, 2 * a.TB, q0, nq, k0, nk, i);
      const int blocks = item_blocks(it);
      items[at + i] = it;
      keys[at + i] =
          static_cast<unsigned long long>(blocks) << 32 | ~static_cast<uint32_t>(it.q_row);
      sum += blocks;
      most = max(most, blocks);
    }
    sum = __reduce_add_sync(0xffffffffu, sum);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) {
      atomicAdd(&all_blocks, sum);
      atomicMax(&longest, most);
    }
  }
  __syncthreads();
  const int n = min(count, a.cap), total = all_blocks;
  const int share = (total * p.Hkv + a.grid - 1) / a.grid;    // of a CTA
  const bool split =
      a.pieces != nullptr && count <= a.cap && longest > kMinSplit && longest > share;
  const int per = split ? max(kMinSplit / 2, share) : 0;
  if (threadIdx.x == 0) {
    // only offsets that run backwards give more items than there is room for
    if (count > a.cap) atomicOr(p.status, kStatusBadIndex);
    *a.header = {n * p.Hkv, per};
  }
  // eight, four or two threads compare an item with the others
  const int threads = n <= 128 ? 8 : n <= 256 ? 4 : 2;
  const int i = threadIdx.x / threads, sub = threadIdx.x & (threads - 1);
  int rank = 0, before = 0;
  if (i < n) {
    const unsigned long long mine = keys[i];
    // the keys of sequences that overlap, of offsets that run backwards, may be equal
    auto count_key = [&](unsigned long long k, int j) {
      const int first = (k > mine) | ((k == mine) & (j < i));
      rank += first;
      before += static_cast<int>(k >> 32) & -first;
    };
    for (int j = 2 * sub; j < n; j += 2 * threads) {
      const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(keys + j);
      count_key(k.x, j);
      count_key(k.y, j + 1);
    }
  }
  for (int o = 1; o < threads; o <<= 1) {
    rank += __shfl_xor_sync(0xffffffffu, rank, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  if (i < n) list_item(a, items[i], rank, before, total, per, sub, threads);
  // parts past the line's end are empty
  if (split)
    for (int w = (total * p.Hkv + per - 1) / per + threadIdx.x; w < a.grid; w += 1024)
      a.part[w] = {0, 0};
}

// The list for more items: a counting sort (more than 511 blocks count as 511), whole items
// only.  Sequences that overlap, of offsets that run backwards, may have more items than there
// is room for, up to 2^44: they are added up in 64 bits, none is counted past the room, and
// then none is listed.
__global__ void __launch_bounds__(1024) prompt_plan_kernel(const PromptArgs a) {
  const PromptParams& p = a.p;
  __shared__ int count[kBuckets];
  __shared__ int sums[kBuckets / 32];
  __shared__ unsigned long long all_items;
  if (threadIdx.x == 0) all_items = 0;
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
      const int n = (nq + 2 * a.TB - 1) / (2 * a.TB);
      if (pass == 0) {
        unsigned long long before = 0;
        if (lane == 0) before = atomicAdd(&all_items, static_cast<unsigned long long>(n));
        before = __shfl_sync(0xffffffffu, before, 0);
        if (before + n > static_cast<unsigned long long>(a.cap)) continue;
      }
      for (int i = lane; i < n; i += 32) {
        PromptItem it = make_item(p, 2 * a.TB, q0, nq, k0, nk, i);
        const int at = atomicAdd(
            &count[kBuckets - 1 - min(kBuckets - 1, max(0, it.kb1 - it.kb0))], 1);
        if (pass == 0) continue;
        for (; it.head < p.Hkv; ++it.head) a.list[static_cast<int64_t>(at) * p.Hkv + it.head] = it;
      }
    }
    __syncthreads();
    if (pass == 1) break;
    if (all_items > static_cast<unsigned long long>(a.cap)) {
      if (threadIdx.x == 0) {
        atomicOr(p.status, kStatusBadIndex);
        *a.header = {0, 0};
      }
      return;
    }
    // items before each bucket
    int x = 0, c = 0;
    if (threadIdx.x < kBuckets) {
      x = c = count[threadIdx.x];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) sums[warp] = x;
    }
    __syncthreads();
    if (threadIdx.x < kBuckets) {
      for (int w = 0; w < warp; ++w) x += sums[w];
      count[threadIdx.x] = x - c;
      if (threadIdx.x == kBuckets - 1) *a.header = {x * p.Hkv, 0};
    }
    __syncthreads();
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

// The entries this CTA takes, each read one ahead of its use: in turn, or
// those of its part of the line.
struct Items {
  const PromptArgs& a;
  PromptItem it, ahead;
  int entry = 0, next_entry = 0;     // of the list
  int r = 0, first = 0, limit = 0;
  bool more = false, parts = false;
  int q0 = 0, nq = 0, k0 = 0, nk = 0;     // without a list: the sequence
  __device__ __forceinline__ explicit Items(const PromptArgs& args) : a(args) {
    if (a.header == nullptr) {
      const bool okq = seq_range(a.p.cu_q, 0, a.p.Tq, &q0, &nq);
      const bool okk = seq_range(a.p.cu_k, 0, a.p.Tk, &k0, &nk);
      if (okq && okk)
        limit = (nq + 2 * a.TB - 1) / (2 * a.TB) * a.p.Hkv;
      else if (threadIdx.x == 0)
        atomicOr(a.p.status, kStatusBadIndex);
    } else {
      // what the first entry needs is read along with the header
      const PromptItem guess = a.list[blockIdx.x];
      const int2 part = a.pieces != nullptr ? a.part[blockIdx.x] : make_int2(0, 0);
      const PromptHeader head = *a.header;
      limit = head.n;
      parts = head.per > 0;
      if (!parts) {
        r = 1;
        next_entry = blockIdx.x;
        more = next_entry < limit;
        ahead = guess;
        return;
      }
      first = part.x;
      limit = part.y;
    }
    fetch();
  }
  __device__ __forceinline__ void fetch() {
    next_entry = parts ? first + r : item_index(r);
    ++r;
    more = next_entry < limit;
    if (!more) return;
    if (a.header != nullptr) {
      ahead = a.list[next_entry];
    } else {
      // the last rows see most keys
      const int k = next_entry / a.p.Hkv;
      ahead = make_item(a.p, 2 * a.TB, q0, nq, k0, nk, limit / a.p.Hkv - 1 - k);
      ahead.head = next_entry - k * a.p.Hkv;
    }
  }
  __device__ __forceinline__ bool next() {
    if (!more) return false;
    it = ahead;
    entry = next_entry;
    fetch();
    return true;
  }
};

// Joins a warp's 32 rows of an item from the parts that hold its blocks:
// out = sum_i 2^(c (m_i - M)) O_i / sum_i 2^(c (m_i - M)) l_i.  A lane weighs
// one row and sums four columns of each; 16 loads are in flight.
template <int D>
__device__ __forceinline__ void join_rows(const PromptArgs& a, const PromptPiece& piece, int row0,
                                          float c, int h, int64_t dst, int64_t lse_at, bool valid) {
  constexpr int kLPR = D / 4, kRPI = 32 / kLPR, kBatch = 16;
  const PromptParams& p = a.p;
  const int lane = threadIdx.x & 31;
  const int w0 = piece.w0, w1 = piece.w1;
  auto first_row = [&](int w) {
    return static_cast<int64_t>(2 * w + (w == w0 ? piece.key & 1 : 0)) * kRowsPerItem + row0;
  };
  float m = -INFINITY, l = 0.f;
  for (int w = w0; w <= w1; ++w) m = fmaxf(m, __ldcg(a.part_ml + first_row(w) + lane).x);
  const float top = m == -INFINITY ? 0.f : m;
  for (int w = w0; w <= w1; ++w) {
    const float2 ml = __ldcg(a.part_ml + first_row(w) + lane);
    l += ml.y * ex2((ml.x - top) * c);
  }
  const RowEnd end =
      finish_row(m * p.scale, l, p.sinks != nullptr && valid ? p.sinks + h : nullptr);
  if (p.lse != nullptr && valid) p.lse[lse_at] = end.lse;
  const uint32_t stored = __ballot_sync(0xffffffffu, valid);
  const int sub = lane / kLPR, col = 4 * (lane % kLPR);
#pragma unroll 1
  for (int r0 = 0; r0 < 32; r0 += kBatch * kRPI) {
    float4 acc[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int w = w0; w <= w1; ++w) {
      const float g = ex2((__ldcg(a.part_ml + first_row(w) + lane).x - top) * c);
      const float* src = a.part_o + (first_row(w) + r0 + sub) * D + col;
      float4 v[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        v[k] = __ldcg(reinterpret_cast<const float4*>(src + k * kRPI * D));
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float f = __shfl_sync(0xffffffffu, g, r0 + k * kRPI + sub);
        acc[k].x += v[k].x * f;
        acc[k].y += v[k].y * f;
        acc[k].z += v[k].z * f;
        acc[k].w += v[k].w * f;
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int rw = r0 + k * kRPI + sub;
      const float f = __shfl_sync(0xffffffffu, end.factor, rw);
      const bool none = __shfl_sync(0xffffffffu, end.none ? 1 : 0, rw) != 0;
      const int64_t to = __shfl_sync(0xffffffffu, dst, rw);
      if ((stored >> rw) & 1)
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + to + col) =
            none ? make_uint2(0u, 0u)
                 : make_uint2(bf16x2(acc[k].x * f, acc[k].y * f),
                              bf16x2(acc[k].z * f, acc[k].w * f));
    }
  }
}

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

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 9) {
      // ------------------------------------------------------------ loads
      if (lane == 0 && !a.inject_stall) {
        uint32_t fill = 0, nq[2] = {0, 0};              // copies of K and V, of each tile's Q
        const uint32_t q_bytes = static_cast<uint32_t>(a.G * a.TB) * 128 * L::kChunks;
        bool ok = true;
        Items items(a);
        while (ok && items.next()) {
          const PromptItem& it = items.it;
          const int hk = it.head & ~kPiece;
          if (it.kb1 <= it.kb0) continue;
          auto load_q = [&](int s) {
            if (!mbar_wait(&q_empty[s], (nq[s] & 1) ^ 1, wc)) return false;
            mbar_expect_tx(&q_full[s], q_bytes);
            for (int c = 0; c < L::kChunks; ++c)
              tma_load_3d(sQ + s * L::kTileBytes + c * L::kChunkBytes, &maps.q, &q_full[s], c * 64,
                          hk * a.G, it.q_row + s * a.TB);
            ++nq[s];
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
          for (int kb = it.kb1 - 2; ok && kb >= it.kb0; --kb)
            ok = load_kv(&maps.k, kb) && load_kv(&maps.v, kb);
        }
        // Every copy issued lands before the CTA goes away, whichever wait of whichever warp
        // gives up, and when.
        volatile int zero = 0;
        WaitCtx dw{p.status, &zero, 1000000000ull};
        for (uint32_t i = fill > ST ? fill - ST : 0; i < fill; ++i)
          mbar_wait(&kv_full[i % ST], (i / ST) & 1, dw);
        for (int s = 0; s < 2; ++s)
          if (nq[s] > 0) mbar_wait(&q_full[s], (nq[s] - 1) & 1, dw);
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
      Items items(a);
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
      // the products in flight end before the tensor memory is freed, as above
      if (leader) mma_commit(drain);
      volatile int zero = 0;
      WaitCtx dw{p.status, &zero, 1000000000ull};
      mbar_wait(drain, 0, dw);
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
    Items items(a);
    while (items.next()) {
      const PromptItem& it = items.it;
      const int n = it.kb1 - it.kb0;
      const int h = (it.head & ~kPiece) * a.G + g;
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
        for (int q = 0; q < 4; ++q) tmem_wait32(x + 32 * q);
        if (__builtin_expect(k0 + kBM > all_hi || k0 < all_lo, 0)) {
          // A warp's rows span few positions: most blocks need no mask.  One test a block,
          // out of line: the loop is short of instructions (a test for each 32 keys: D 128 1 %
          // slower, D 64 6 %).
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int kq = k0 + 32 * q;
            if (kq + 32 <= all_hi && kq >= all_lo) continue;
            const uint32_t vis = low_bits(hi - kq) & ~low_bits(lo - kq);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              x[32 * q + e] = (vis >> e) & 1 ? x[32 * q + e] : -INFINITY;
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float* v = x + 32 * q;
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
        uint64_t sum[4];
        auto weights = [&](uint32_t* w, int first, int last) {
#pragma unroll
          for (int e = first; e < last; e += 2) {
            float u, v;
            unpack2(fma2(pack2(x[e], x[e + 1]), c2, n2), &u, &v);
            u = ex2(u), v = ex2(v);
            w[(e & 63) / 2] = bf16x2(u, v);
            sum[(e / 2) & 3] = e < 8 ? pack2(u, v) : add2(sum[(e / 2) & 3], pack2(u, v));
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
      const int64_t tokr = it.q_row + i;
      const int64_t dst = tokr * p.o_t + static_cast<int64_t>(h) * p.o_h;
      uint8_t* stage = sOut + warp * (32 * 128);
      const RowEnd row_end =
          finish_row(m * p.scale, l, p.sinks != nullptr && valid ? p.sinks + h : nullptr);
      if (n > 0) {
        if (!mbar_wait_warp(&o_full[s], no & 1, wc)) goto softmax_done;
        ++no;
        tc_fence_after();
      }
      if (it.head & kPiece) {
        const PromptPiece piece = a.pieces[items.entry];
        // a piece: its reference, sum and unscaled output, 32 columns at a time
        const int64_t first = static_cast<int64_t>(piece.slot) * kRowsPerItem + warp * 32;
        a.part_ml[first + lane] = make_float2(m, l);
        for (int d0 = 0; d0 < D; d0 += 32) {
          float o[32];
          tmem_ld32(tO + d0, o);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<float4*>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) =
                make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          __syncwarp();
          const int sub = lane >> 3, ch = lane & 7;
          float4 w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            w[e] = *reinterpret_cast<const float4*>(stage + (4 * e + sub) * 128 +
                                                    ((ch ^ ((4 * e + sub) & 7)) << 4));
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<float4*>(a.part_o + (first + 4 * e + sub) * D + d0 + 4 * ch) = w[e];
        }
        tc_fence_before();
        // the last of the item's pieces joins them
        __threadfence();
        __syncwarp();
        int last = 0;
        if (lane == 0)
          last = atomicAdd(a.done + (piece.key >> 1) * 8 + warp, 1) == piece.w1 - piece.w0;
        if (__shfl_sync(0xffffffffu, last, 0)) {
          __threadfence();
          join_rows<D>(a, piece, warp * 32, c, h, dst, tokr * p.Hq + h, valid);
        }
        continue;
      }
      // through shared memory, so that 8 lanes write 128 adjacent bytes of a row
      const uint32_t stored = __ballot_sync(0xffffffffu, valid);
      const int sub = lane >> 3, ch = lane & 7;
      int64_t to[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        to[e] = __shfl_sync(0xffffffffu, dst, 4 * e + sub) + 8 * ch;
#pragma unroll
      for (int d0 = 0; d0 < D; d0 += 64) {
        float o[64];
        if (n > 0) {
          tmem_ld64(tO + d0, o);
        } else {
#pragma unroll
          for (int e = 0; e < 64; ++e) o[e] = 0.f;
        }
        const float f = row_end.factor;
        uint4 w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float* v = o + 8 * e;
          w[e] = row_end.none ? make_uint4(0u, 0u, 0u, 0u)
                              : make_uint4(bf16x2(v[0] * f, v[1] * f), bf16x2(v[2] * f, v[3] * f),
                                           bf16x2(v[4] * f, v[5] * f), bf16x2(v[6] * f, v[7] * f));
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          *reinterpret_cast<uint4*>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) = w[e];
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e)
          w[e] = *reinterpret_cast<const uint4*>(stage + (4 * e + sub) * 128 +
                                                 ((ch ^ ((4 * e + sub) & 7)) << 4));
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if ((stored >> (4 * e + sub)) & 1)
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + to[e] + d0) = w[e];
      }
      if (p.lse != nullptr && valid) p.lse[tokr * p.Hq + h] = row_end.lse;
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

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

struct PromptSpace {
  size_t list, pieces, part, done, ml, o, total;   // offsets
  bool split;
};
PromptSpace prompt_space(int64_t Tq, int64_t B, int Hq, int Hkv, int D, int num_sms) {
  const size_t items = static_cast<size_t>(max_items(Tq, B, Hq, Hkv)), n = items * Hkv;
  PromptSpace s;
  s.split = items <= kRankItems && n <= static_cast<size_t>(kMaxSplitItems) * num_sms;
  size_t at = 256;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round256(bytes);
    return here;
  };
  // with an entry more for each part
  s.list = take((n + (s.split ? num_sms : 0)) * sizeof(PromptItem));
  s.pieces = s.part = s.done = s.ml = s.o = at;
  if (s.split) {
    s.pieces = take((n + num_sms) * sizeof(PromptPiece));
    s.part = take(num_sms * sizeof(int2));
    s.done = take(n * 8 * sizeof(int));
    const size_t rows = static_cast<size_t>(num_sms) * 2 * kRowsPerItem;
    s.ml = take(rows * sizeof(float2));
    s.o = take(rows * D * sizeof(float));
  }
  s.total = at;
  return s;
}

template <int D>
cudaError_t launch(const PromptMaps& maps, const PromptArgs& a, cudaStream_t stream) {
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
  return launch_k(prompt_kernel<D>, dim3(a.grid), dim3(kPromptThreads), static_cast<size_t>(smem),
                  stream, maps, a);
}

}  // namespace

size_t prompt_workspace_bytes(int64_t Tq, int64_t B, int Hq, int Hkv, int D, int num_sms) {
  return prompt_space(Tq, B, Hq, Hkv, D, num_sms).total;
}

cudaError_t launch_prompt(const PromptParams& p, int num_sms, cudaStream_t stream,
                          std::string* err) {
  const PromptSpace space = prompt_space(p.Tq, p.B, p.Hq, p.Hkv, p.D, num_sms);
  char* ws = static_cast<char*>(p.workspace);
  PromptArgs a = {};
  a.p = p;
  a.G = p.Hq / p.Hkv;
  a.TB = tokens_per_tile(p.Hq, p.Hkv);
  const int64_t most = max_items(p.Tq, p.B, p.Hq, p.Hkv);
  a.cap = static_cast<int>(most);
  // Splitting: no sequence has more keys than there are, so there is nothing to
  // split below kMinSplit blocks; the line's length stays below 2^31 (at most kMaxSplitItems
  // pairs per SM).  One causal sequence with two items per SM or more has none longer
  // than a CTA's share.
  const bool keys_long = p.Tk > kMinSplit * kBM && p.Tk <= (1 << 26);
  const bool alone = p.B == 1 && (!keys_long || most * p.Hkv >= 2 * num_sms);
  const bool split = space.split && keys_long && !alone;
  if (!alone) {
    a.header = reinterpret_cast<PromptHeader*>(ws);
    a.list = reinterpret_cast<PromptItem*>(ws + space.list);
  }
  if (split) {
    a.pieces = reinterpret_cast<PromptPiece*>(ws + space.pieces);
    a.part = reinterpret_cast<int2*>(ws + space.part);
    a.done = reinterpret_cast<int*>(ws + space.done);
    a.part_ml = reinterpret_cast<float2*>(ws + space.ml);
    a.part_o = reinterpret_cast<float*>(ws + space.o);
  }
  a.grid = split || most * p.Hkv > num_sms ? num_sms : static_cast<int>(most * p.Hkv);
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
  if (!alone) {
    const cudaError_t e = launch_k(most <= kRankItems ? prompt_rank_kernel : prompt_plan_kernel,
                                   dim3(1), dim3(1024), 0, stream, a);
    if (e != cudaSuccess) return e;
  }
  return p.D == 128 ? launch<128>(maps, a, stream) : launch<64>(maps, a, stream);
}

}  // namespace mxq
