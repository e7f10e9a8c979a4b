// attn_tree.cu — attention of several new tokens per sequence over a paged key/value
// cache: drafted tokens that form a tree, or a chunk of a prompt.
//
//   S = Q K^T,  P = 2^(c S - c m),  l = rowsum P,  O = P V / l   (c = scale log2 e)
//
// over one pass of the keys, with the running maximum m and sum l of each row.  Row i of
// a sequence stands behind the P keys of its context; it sees them (a window counts from its
// own position, P + its depth in the tree) and the rows on its path: itself, its parent, its
// parent's parent and so on.
//
// Rows.  The G query heads of a key/value head read the same keys: a tile's 128 rows
// are (token, head of the group) pairs, TB = 128 / G tokens, against blocks of 128 keys on the
// tensor cores.  Few rows to a key make the operator HBM-bound (a tile takes 1024 tensor
// cycles a block of bf16 at D 128, whose 64 KB take ~3000 of an SM's share of the memory), so the
// kernel is built around loads in flight, and every key is read once by an item of up
// to two tiles.  An item of two tiles (more than TB tokens) takes each block with
// both.  An item of one has both softmax warpgroups take its blocks in turn, each with its own
// maximum, sum and output, which meet at the end.  Either way the work of the tensor cores is one
// list of turns: turn t belongs to warpgroup t & 1.
//   warps 0-3, 4-7   softmax of the even and odd turns, one thread a row, and the output
//   warp 8           issues the MMAs
//   warp 12          finds the pieces of items that the CTA works on (next to warp 8, which needs its
//                    scheduler's turns: two tiles 2 % faster than with a loading warp there)
//   the other six    load keys and values with 16-byte asynchronous copies, row by row, as pages
//                    are of any size; for an e4m3 cache two of them, and four convert to f16 (exact)
// S0, S1, O0 and O1 are in tensor memory, P takes the place of S.  The reference a
// row subtracts is raised only when its maximum grows by more than 2^8.
//   bf16 cache: bf16 products.  e4m3 cache: f16 products, q scaled per row by a power of two to
//   use f16's range (exact for elements within 2^31 of the row's largest).
//
// A row's path is followed while its blocks are taken, from the last key down: the thread holds
// the next ancestor, and a block's part of the path becomes a bit mask.
//
// Work.  The key blocks of all items form one line, cut into parts of equal cost; a (part,
// key/value head) pair is one CTA's, the heads of a part at work at the same time.  Items that parts
// share leave at most two partial results per CTA in the workspace, which a second kernel joins in
// a fixed order.  A part's end inside a short item moves to the nearer end of it.
//
// Measured.  64 sequences of 5-8192 keys with trees of up to 32, 32 / 8 heads of 128, bf16: 184 us
// (178 before the join: 6.0 TB/s of keys and values, 90 % of a plain copy's rate); 16 sequences of
// 9000-32768 keys with 16 rows, 64 / 8 heads: 202 us, 6.4 TB/s, at D 64 124 us.  What bounds the
// rest: of two tiles (32 rows of those) the warp that issues the products, 251 us.  It finds its
// operands ready nearly always, but the roles share the supply of instructions, and a turn costs it
// ~1800 cycles against 1024 of products (at D 64 ~1450 against 640).  With e4m3 that and the
// conversion, 1800 cycles of shared memory a block (16 rows 179 us, 32 rows 258, up to 48 rows 348).
// One tree over 1500 keys: 13.5 us, half of it launches, the chain length -> page -> key, and a
// call's first use of each instruction.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>

#include "attn.h"
#include "attn_math.cuh"
#include "internal.h"

namespace mxq {

namespace {

constexpr int kBM = 128;             // rows of a tile, keys of a block
constexpr int kRows = 2 * kBM;       // of an item
constexpr int kTreeThreads = 512;
constexpr int kTreeWarps = kTreeThreads / 32;
constexpr int kMmaWarp = 8, kWalkWarp = 12;
// registers a thread: the launch gives 128 to each; the softmax warpgroups keep most of a row of
// 128 scores and take what the other two give up
constexpr int kSoftmaxRegs = 168, kOtherRegs = 88;
static_assert(2 * kSoftmaxRegs + 2 * kOtherRegs <= 4 * 128, "register split above the launch's");
constexpr int kPieces = 8;           // pieces of items that may be under way
constexpr int kSeen = 16;            // blocks whose masks of loaded keys are kept
// Items of at most this many blocks stay whole, so that no piece of theirs is joined; in calls that are
// cut anyway it makes no difference in time (64 ragged sequences 184 us, 16 of 200-600 keys 21.5,
// with 0, 1 and 2 alike).
constexpr int kWhole = 2;
// Calls of at most this many sequences: one warp cuts the line, a lane has one at most (one tree over 1500
// keys 13.5 us, by the whole block 14.0; 100 sequences of 300-700 keys, four a lane, 67.5, by the block
// 66.3).
constexpr int kAloneSequences = 32;
// Calls whose items have at most this many blocks: none is cut, and there is nothing to join (one
// sequence of 300 keys 10.3 us, cut 12.6; 64 of 50-300 32.4 and 38.4; 48 of 200-250 26.1 and 32.1).
constexpr int kAllWhole = 3;

// What joins an item that several parts share: written by the CTA that begins it.
struct __align__(16) TreeJoin {
  int q_row, ntok;                   // ntok 0: nothing
  int w0, w1;                        // its parts
  int first;                         // slot of the first one's result
  int pad[3];
};

struct TreeArgs {
  TreeParams p;
  int G, TB;
  int parts;
  bool all_whole;                    // no item is cut
  uint32_t k_page, k_key, v_page, v_key;   // strides of the caches, in 16 bytes
  bool far;                          // a row may begin 2^32 of them or more from the first
  uint32_t page_mul, page_shift;     // key / page_size = (mulhi(key, mul) + key) >> shift
  TreeJoin* joins;                   // [part * Hkv + head]
  float2* part_ml;                   // [task][2][256]: reference (log2) and sum
  float* part_o;                     // [task][2][256][D]
  unsigned long long budget_ns;
  int inject_stall;
};

template <int D, bool FP8>
struct TreeLayout {
  static constexpr int kChunks = D / 64;
  static constexpr int kChunkBytes = kBM * 128;          // 128 rows of 64 elements
  static constexpr int kTileBytes = kChunks * kChunkBytes;
  static constexpr int kRowBytes = FP8 ? D : 2 * D;      // of a cached key
  static constexpr int kLPR = kRowBytes / 16;            // lanes a row
  static constexpr int kRPI = 32 / kLPR;                 // rows a copy instruction
  static constexpr int kCopies = 32 / kRPI;              // copies a thread for 32 rows
  static constexpr int kStages = FP8 ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 10);
  // Beside the warps that convert e4m3 rows of 128 the instructions' supply is short: there a mask
  // is written to the scores in a pass of its own, and the weights' code stands once for both
  // halves (16 long e4m3 sequences 368 -> 360 us; bf16 is 1 % slower so, D 64 up to 4 %).
  static constexpr bool kRolled = FP8 && D == 128;
  static constexpr int kLoaders = 6;                     // warps that load
  // e4m3: two of them copy rows as they are cached into stages of their own, the other four
  // convert a quarter of each to f16 (all six doing both took 253 us for 16 long sequences of 16
  // drafts)
  static constexpr int kFetchers = 2;
  static constexpr int kRawStages = FP8 ? (D == 128 ? 4 : 8) : 0;
  static constexpr int kUnitBytes = 32 * kRowBytes, kRawBytes = 4 * kUnitBytes;
  static constexpr int kBars = 2 * 7 + 2 * kStages + 2 * kPieces + 2 * kRawStages + 1;
  static constexpr int kSmem = (2 + kStages) * kTileBytes + kRawStages * kRawBytes + 16 * kSeen +
                               64 * kPieces + 8 * kBars + 16;
  static_assert(kSmem + 1024 + 512 <= 227 * 1024, "shared memory over budget");
  static_assert(kMmaWarp + 2 + kLoaders <= kTreeWarps, "more warps than there are");
  // Block b's masks are read until its weights are handed over, and so while its values, copy 2 b + 2
  // at most, keep their place: a warp has begun at most kStages + kRawStages + 1 copies behind those
  // (+ 1: the units of six warps reach into a second copy), and the keys of block x are copy 2 x - 1
  // at least.
  static_assert(kSeen > (kStages + kRawStages) / 2 + 2, "masks overwritten by copies ahead");
};

// A sequence: its rows [q0, q0 + nq) of the packed queries, behind len - nq keys.
struct TreeSeq {
  int q0, nq, len;
  bool bad;
};
__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, int from, int to, int given) {
  TreeSeq s;
  const int64_t cap = p.max_pages * p.page_size;
  s.len = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(given), cap)));
  const bool ok = from >= 0 && to >= from && to <= p.T && s.len >= to - from;
  s.bad = !ok || s.len != given;
  s.q0 = from;
  s.nq = ok ? to - from : 0;
  return s;
}

// Item i of a sequence: tokens [i 2 TB, + ntok), its n blocks of keys numbered from the last:
// block v (from the first) is the keys' block v, or v + skip from block `head` on, those in
// between being visible to none of its rows.
struct TreeItem {
  int ntok, hi, lo;                  // keys [0, first) and [lo, hi) are loaded
  int n, head, skip;
};
__device__ __forceinline__ TreeItem tree_item(const TreeArgs& a, const TreeSeq& s, int i) {
  const TreeParams& p = a.p;
  TreeItem it;
  const int first = i * 2 * a.TB, P = s.len - s.nq;
  it.ntok = min(2 * a.TB, s.nq - first);
  it.hi = P + first + it.ntok;
  // a row of a tree may stand right behind the context
  const int at = p.parents != nullptr ? P : P + first;
  it.lo = p.window > 0 ? max(0, at - p.window + 1) : 0;
  it.head = min((p.first + kBM - 1) / kBM, it.lo / kBM);
  it.skip = it.lo / kBM - it.head;
  it.n = (it.hi + kBM - 1) / kBM - it.skip;
  return it;
}

// What an item counts on the line: a block of one tile 3 (bf16 at D 128: ~3000 cycles, its bytes'
// share of the memory), of two 4 (~3600), at D 64 3 and 5; its begin and end as
// much as two blocks (64 ragged sequences: 182 us, with one 184, without 188).
constexpr int kItemCost = 6, kMinCost = 6;
template <int D>
__device__ __forceinline__ int block_cost(const TreeArgs& a, const TreeItem& it) {
  return it.ntok <= a.TB ? 3 : D == 128 ? 4 : 5;
}
template <int D>
__device__ __forceinline__ int item_cost(const TreeArgs& a, const TreeItem& it) {
  return kItemCost + it.n * block_cost<D>(a, it);
}

// A piece of an item: what a CTA's part of the line holds of it.  cnt 0: there are no more.
// Its keys and values are copied in the order K_0, K_1, V_0, K_2, V_1, ..., V_(cnt-1).
struct __align__(16) TreePiece {
  int q_row, ntok, P, first;         // the item's first row (of all, and of its sequence's)
  int hi, lo, head, skip;            // as in TreeItem
  int v1, cnt, flags, task;          // its blocks v1 - 1, v1 - 2, ...
  int b, pad[3];
  // first key of the piece's block j
  __device__ __forceinline__ int key(int j) const {
    const int v = v1 - 1 - j;
    return (v < head ? v : v + skip) * kBM;
  }
  // copy f: whether it is of values, and its block
  __device__ __forceinline__ bool is_value(int f) const {
    return (f > 0 && (f & 1) == 0) || f == 2 * cnt - 1;
  }
  __device__ __forceinline__ int block(int f) const {
    return f == 0 ? 0 : is_value(f) ? (f - 1) / 2 : (f + 1) / 2;
  }
};
static_assert(sizeof(TreePiece) == 64, "four 16-byte words");
constexpr int kOpened = 1, kClosed = 2, kSingle = 4, kSlot1 = 8;

// The pieces that one warp hands to the others through a ring in shared memory; their fields are
// read there as they are needed (registers are short).
struct Pieces {
  const TreePiece* ring;
  uint64_t *full, *empty;
  uint32_t n = 0;
  __device__ __forceinline__ Pieces(const TreePiece* r, uint64_t* f, uint64_t* e)
      : ring(r), full(f), empty(e) {}
  // the next piece; null: there are none, or a wait gave up
  template <bool kLean = true>
  __device__ __forceinline__ const TreePiece* next(const WaitCtx& wc) {
    const int at = n % kPieces;
    const uint32_t phase = (n / kPieces) & 1;
    if (!(kLean ? wait_lean(&full[at], phase, wc) : mbar_wait_warp(&full[at], phase, wc)))
      return nullptr;
    return ring[at].cnt > 0 ? ring + at : nullptr;
  }
  __device__ __forceinline__ void done() {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[n % kPieces]);
    ++n;
  }
};

// a / b for a >= 0, b > 0: 64-bit division only where it is needed
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

__device__ __forceinline__ void prefetch(const void* at) {
  asm volatile("prefetch.global.L1 [%0];" ::"l"(at));
}

// where a key's row begins in a cache, in 16 bytes
__device__ __forceinline__ uint64_t row_at(uint32_t page, uint32_t off, uint32_t page_stride,
                                           uint32_t key_stride) {
  return static_cast<uint64_t>(page) * page_stride + static_cast<uint64_t>(off) * key_stride;
}

// 32 rows of a cache, kRPI at a time: lane r's row begins 16 * at bytes from base (of this lane's 16
// bytes); copy i of this lane goes to to(i).  Usually all rows are there and the cache spans less
// than 2^32 of 16 bytes: then a copy is a shuffle, a product and itself.  The places of several rows
// come first: a shuffle before each copy held the copies back.
template <int kCopies, int kRPI, typename F>
__device__ __forceinline__ void copy_rows(const char* base, uint64_t at, uint32_t mask, int row_in,
                                          bool far, F to) {
  if (mask == 0xffffffffu && !far) {
#pragma unroll
    for (int i0 = 0; i0 < kCopies; i0 += 4) {
      uint32_t from[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        from[i] = __shfl_sync(0xffffffffu, static_cast<uint32_t>(at), (i0 + i) * kRPI + row_in);
#pragma unroll
      for (int i = 0; i < 4; ++i) cp16(to(i0 + i), base + static_cast<uint64_t>(from[i]) * 16);
    }
  } else {
    mask >>= row_in;
#pragma unroll
    for (int i0 = 0; i0 < kCopies; i0 += 4) {
      uint64_t from[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        from[i] = __shfl_sync(0xffffffffu, at, (i0 + i) * kRPI + row_in);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        cp16(to(i0 + i), base + from[i] * 16, (mask >> ((i0 + i) * kRPI)) & 1);
    }
  }
}

// one arrival of this thread on `bar` when its copies so far have landed
__device__ __forceinline__ void cp_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_kernel(const TreeArgs a) {
  using L = TreeLayout<D, FP8>;
  constexpr int ST = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* ring = smem + 2 * L::kTileBytes;
  uint8_t* raw = ring + ST * L::kTileBytes;
  uint32_t* seen = reinterpret_cast<uint32_t*>(raw + L::kRawStages * L::kRawBytes);   // [kSeen][4]
  TreePiece* piece_ring = reinterpret_cast<TreePiece*>(seen + 4 * kSeen);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(piece_ring + kPieces);
  uint64_t* s_full = q_full + 2;
  uint64_t* p_full = s_full + 2;      // [s][half]
  uint64_t* o_full = p_full + 4;
  uint64_t* merge = o_full + 2;       // both results there, both read
  uint64_t* kv_full = merge + 2;
  uint64_t* kv_empty = kv_full + ST;
  uint64_t* piece_full = kv_empty + ST;
  uint64_t* piece_empty = piece_full + kPieces;
  [[maybe_unused]] uint64_t* raw_full = piece_empty + kPieces;
  [[maybe_unused]] uint64_t* raw_empty = raw_full + L::kRawStages;
  uint64_t* drain = raw_full + 2 * L::kRawStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  __shared__ unsigned long long warp_sum[kTreeWarps];
  __shared__ int warp_longest[kTreeWarps];
  __shared__ int ends[2][3];          // the part's begin and end: sequence, item and block of that
  __shared__ long long start_at;      // the line up to the first item
  __shared__ TreeSeq start_seq;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int loader = warp - kMmaWarp - 1 - (warp > kWalkWarp);
  const TreeParams& p = a.p;
  WaitCtx wc{p.status, abort_flag, a.budget_ns};

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 4);           // the warps of the warpgroup
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[2 * i], 4);
      mbar_init(&p_full[2 * i + 1], 4);
      mbar_init(&o_full[i], 1);
      mbar_init(&merge[i], 8);            // the warps of both
    }
    for (int i = 0; i < ST; ++i) {
      // four units of 32 rows: an arrival each, and one of every thread's copies
      mbar_init(&kv_full[i], FP8 ? 4 : 4 + 128);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(&piece_full[i], 1);
      mbar_init(&piece_empty[i], 8 + 1 + L::kLoaders);
    }
    for (int i = 0; i < L::kRawStages; ++i) {
      mbar_init(&raw_full[i], 33 * L::kFetchers);
      mbar_init(&raw_empty[i], 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_launch_dependents();

  // The barriers and the tensor memory are there.
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // ---- the line, and this CTA's part of it: found by the warp that needs it, where a lane has
  // few sequences (no word to the other warps: a tree over 1500 keys 13.6 us, by the whole
  // block 14.2), or by all
  const bool alone = p.B <= kAloneSequences;
  const int part = static_cast<int>(blockIdx.x) / p.Hkv;
  int64_t per = 0, raw0 = 0;
  auto seq = [&](int b) { return tree_seq(p, p.cu_q[b], p.cu_q[b + 1], p.seq_lens[b]); };
  auto sync = [&]() {
    if (alone)
      __syncwarp();
    else
      __syncthreads();
  };
  if (!alone || warp == kWalkWarp) {
    const int team = alone ? 32 : kTreeThreads, me = alone ? lane : threadIdx.x;
    const int per_thread = (p.B + team - 1) / team;
    const int b0 = me * per_thread, b1 = min(p.B, b0 + per_thread);
    unsigned long long mine = 0;
    int longest = 0;
    TreeSeq kept = {0, 0, 0, false};  // where a thread has one sequence, it is read once
    for (int b = b0; b < b1; ++b) {
      const TreeSeq s = seq(b);
      kept = s;
      if (s.bad && blockIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
      for (int i = 0; i * 2 * a.TB < s.nq; ++i) {
        const int cost = item_cost<D>(a, tree_item(a, s, i));
        mine += cost;
        longest = max(longest, cost);
      }
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    unsigned long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (me < 2) ends[me][0] = p.B, ends[me][1] = ends[me][2] = 0;
    if (!alone && lane == 31) warp_sum[warp] = incl, warp_longest[warp] = longest;
    sync();
    int64_t before = static_cast<int64_t>(incl - mine), total = 0;
    if (alone) {
      total = static_cast<int64_t>(__shfl_sync(0xffffffffu, incl, 31));
    } else {
      for (int w = 0; w < kTreeWarps; ++w) {
        if (w < warp) before += static_cast<int64_t>(warp_sum[w]);
        total += static_cast<int64_t>(warp_sum[w]);
        longest = max(longest, warp_longest[w]);
      }
    }
    per = max(divide(total + a.parts - 1, a.parts), static_cast<int64_t>(kMinCost));
    // where all stay whole, a part has room for the longest, or some would get two
    if (a.all_whole && per < longest) per = longest;
    raw0 = part * per;
    // The thread that holds an end of the part finds its item and the block there; inside an item
    // that stays whole it is the nearer end of it.
    for (int end = 0; end < 2; ++end) {
      const int64_t pos = raw0 + end * per;
      if (pos < before || pos >= before + static_cast<int64_t>(mine)) continue;
      int64_t at = before;
      bool found = false;
      for (int b = b0; b < b1 && !found; ++b) {
        const TreeSeq s = per_thread == 1 ? kept : seq(b);
        for (int i = 0; i * 2 * a.TB < s.nq && !found; ++i) {
          const TreeItem it = tree_item(a, s, i);
          const int cost = item_cost<D>(a, it);
          if (at + cost <= pos) {
            at += cost;
            continue;
          }
          found = true;
          const int in = max(0, static_cast<int>(pos - at) - kItemCost);
          int off = in / block_cost<D>(a, it);
          if (a.all_whole || it.n <= kWhole) off = 2 * off >= it.n && off > 0 ? it.n : 0;
          ends[end][0] = b, ends[end][1] = i, ends[end][2] = off;
          if (end == 0) {
            start_at = at;
            start_seq = s;
            // on its way: the page of its last keys
            if (s.len > 0) prefetch(p.page_table + b * p.ld_table + (s.len - 1) / p.page_size);
          }
        }
      }
    }
    sync();
  }
  const int tasks = a.parts * p.Hkv;

  Pieces pieces(piece_ring, piece_full, piece_empty);
  if (warp >= kMmaWarp) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == kWalkWarp) {
    // ----------------------------------------------------- the part's pieces
    if (lane == 0) {
      uint32_t n = 0;
      auto put = [&](const TreePiece& it) {
        const int at = n % kPieces;
        if (!mbar_wait(&piece_empty[at], ((n / kPieces) & 1) ^ 1, wc)) return false;
        piece_ring[at] = it;
        mbar_arrive(&piece_full[at]);
        ++n;
        return true;
      };
      bool ok = true;
      for (int task = blockIdx.x; ok && task < tasks; task += gridDim.x) {
        a.joins[task].ntok = 0;
        int b = ends[0][0], i = ends[0][1], off = ends[0][2];
        const int last_b = ends[1][0], last_i = ends[1][1], last_off = ends[1][2];
        if (b >= p.B) continue;
        int64_t begin = start_at;
        TreeSeq sq = start_seq;
        while (ok) {
          if (i * 2 * a.TB >= sq.nq) {
            if (++b >= p.B) break;
            sq = seq(b);
            i = 0;
            continue;
          }
          const TreeItem it = tree_item(a, sq, i);
          const bool at_end = b > last_b || (b == last_b && i >= last_i);
          const int to_block = !at_end ? it.n : b == last_b && i == last_i ? last_off : 0;
          if (off < to_block) {
            TreePiece t = {};
            t.first = i * 2 * a.TB;
            t.q_row = sq.q0 + t.first;
            t.ntok = it.ntok;
            t.P = sq.len - sq.nq;
            t.hi = it.hi, t.lo = it.lo, t.head = it.head, t.skip = it.skip;
            t.v1 = it.n - off;
            t.cnt = to_block - off;
            t.task = task, t.b = b;
            const bool opened = off == 0, closed = to_block == it.n;
            t.flags = (opened ? kOpened : 0) | (closed ? kClosed : 0) |
                      (it.ntok <= a.TB ? kSingle : 0) | (opened && raw0 < begin ? kSlot1 : 0);
            ok = put(t);
            if (opened && !closed) {
              TreeJoin& to = a.joins[task];
              to.q_row = t.q_row;
              to.ntok = t.ntok;
              to.w0 = part;
              to.w1 = static_cast<int>(divide(begin + item_cost<D>(a, it) - 1, per));
              to.first = raw0 < begin ? 1 : 0;
            }
          }
          if (at_end) break;
          begin += item_cost<D>(a, it);
          off = 0;
          ++i;
        }
      }
      if (ok) put(TreePiece{});
    }
    __syncwarp();
  } else if (FP8 && loader >= L::kFetchers) {
    // ------------------------------------------------- e4m3 rows to f16
    if constexpr (FP8) {
      const int quarter = loader - L::kFetchers;
      const int rows = quarter * 32 + lane / L::kLPR, piece = lane % L::kLPR;
      const uint8_t* src = raw + quarter * L::kUnitBytes + lane * 16;
      uint8_t* dst = ring + (piece >> 2) * L::kChunkBytes + rows * 128;
      // (the second chunk's lanes write their 16-byte pieces the other way round: the first's are
      // in the same banks)
      const int c0 = (2 * piece) & 7, swap = piece >> 2;
      uint32_t fill = 0;
      while (!a.inject_stall) {
        const TreePiece* it = pieces.next(wc);
        if (it == nullptr) break;
        for (const uint32_t end = fill + 2 * it->cnt; fill != end; ++fill) {
          const int from = fill % L::kRawStages, to = fill % ST;
          if (!wait_lean(&raw_full[from], (fill / L::kRawStages) & 1, wc)) goto convert_done;
          uint4 x[L::kCopies];
#pragma unroll
          for (int i = 0; i < L::kCopies; ++i)
            x[i] = *reinterpret_cast<const uint4*>(src + from * L::kRawBytes + i * 512);
          if (!wait_lean(&kv_empty[to], ((fill / ST) & 1) ^ 1, wc)) goto convert_done;
#pragma unroll
          for (int i = 0; i < L::kCopies; ++i) {
            uint4 lo, hi;
            e4m3x4_f16(x[i].x, &lo.x, &lo.y);
            e4m3x4_f16(x[i].y, &lo.z, &lo.w);
            e4m3x4_f16(x[i].z, &hi.x, &hi.y);
            e4m3x4_f16(x[i].w, &hi.z, &hi.w);
            const int r7 = (rows + i * L::kRPI) & 7;
            uint8_t* at = dst + to * L::kTileBytes + i * L::kRPI * 128;
            *reinterpret_cast<uint4*>(at + (((c0 + swap) ^ r7) << 4)) = swap ? hi : lo;
            *reinterpret_cast<uint4*>(at + (((c0 + 1 - swap) ^ r7) << 4)) = swap ? lo : hi;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&kv_full[to]);
            mbar_arrive(&raw_empty[from]);
          }
        }
        pieces.done();
      }
    convert_done:;
    }
  } else if (FP8 && loader >= 0) {
    // ------------------------------------------------------- e4m3 rows
    // A warp takes two quarters of a block (32 rows each), keys and, from the same places,
    // values.
    if constexpr (FP8) {
      constexpr int NF = L::kFetchers, NQ = 4 / NF;
      const int first = loader;
      const int row_in = lane / L::kLPR, piece = lane % L::kLPR;
      const uint32_t raw_at = smem_u32(raw) + first * L::kUnitBytes + lane * 16;
      uint32_t fill = 0, blocks = 0;
      while (!a.inject_stall) {
        const TreePiece* at_piece = pieces.next(wc);
        if (at_piece == nullptr) break;
        const TreePiece& it = *at_piece;
        const int hk = it.task % p.Hkv;
        const char* k_base = static_cast<const char*>(p.k_cache) + hk * p.ck_h + piece * 16;
        const char* v_base = static_cast<const char*>(p.v_cache) + hk * p.cv_h + piece * 16;
        const int32_t* table = p.page_table + it.b * p.ld_table;
        const int hi = it.hi, lo = it.lo, head = it.head, skip = it.skip, v1 = it.v1, cnt = it.cnt;
        // this lane's keys of a block, looked up a block ahead; off -1: not loaded (nothing is
        // done to a page here: it would be waited for)
        struct Spot {
          int page[NQ], off[NQ];
        };
        auto look_up = [&](int j) {
          Spot r;
          const int v = v1 - 1 - j;
          const int key0 = j < cnt ? (v < head ? v : v + skip) * kBM + first * 32 + lane : 1 << 30;
#pragma unroll
          for (int i = 0; i < NQ; ++i) {
            const int key = key0 + i * NF * 32;
            r.page[i] = 0, r.off[i] = -1;
            if (key < hi && (key >= lo || key < p.first)) {
              const uint32_t n = (__umulhi(key, a.page_mul) + key) >> a.page_shift;
              r.off[i] = key - static_cast<int>(n) * p.page_size;
              r.page[i] = __ldg(table + n);
            }
          }
          return r;
        };
        Spot next = look_up(0);
        // of the block whose values are to come, and of the one whose keys are
        uint64_t v_at[NQ] = {}, k_at[NQ] = {}, at[NQ] = {};
        uint32_t v_mask[NQ] = {}, mask[NQ] = {};
        bool ok = true;
        for (int j = 0; ok && j <= cnt; ++j) {
#pragma unroll
          for (int i = 0; i < NQ; ++i) v_at[i] = at[i], v_mask[i] = mask[i];
          if (j < cnt) {
            const Spot now = next;
            next = look_up(j + 1);
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
              const bool there =
                  now.off[i] >= 0 &&
                  static_cast<uint32_t>(now.page[i]) < static_cast<uint32_t>(p.pages);
              if (now.off[i] >= 0 && !there) atomicOr(p.status, kStatusBadIndex);
              // (the source of a row that is not there is not read)
              k_at[i] = there ? row_at(now.page[i], now.off[i], a.k_page, a.k_key) : 0;
              at[i] = there ? row_at(now.page[i], now.off[i], a.v_page, a.v_key) : 0;
              mask[i] = __ballot_sync(0xffffffffu, there);
              if (lane == 0) seen[((blocks + j) % kSeen) * 4 + first + i * NF] = mask[i];
            }
          }
          // K_j, then V_(j-1) (in one place of the code 16 long sequences of 16 drafts 196 us, in two 179)
#pragma unroll
          for (int kind = 0; kind < 2; ++kind) {
            if (kind == 0 ? j >= cnt : j == 0) continue;
            const int st = fill % L::kRawStages;
            ok = wait_lean(&raw_empty[st], ((fill / L::kRawStages) & 1) ^ 1, wc);
            if (!ok) break;
            const uint32_t dst = raw_at + st * L::kRawBytes;
#pragma unroll
            for (int q = 0; q < NQ; ++q)
              copy_rows<L::kCopies, L::kRPI>(
                  kind ? v_base : k_base, kind ? v_at[q] : k_at[q], kind ? v_mask[q] : mask[q],
                  row_in, a.far,
                  [&](int i) { return dst + q * NF * L::kUnitBytes + i * 512; });
            cp_arrive(&raw_full[st]);
            if (lane == 0) mbar_arrive(&raw_full[st]);
            ++fill;
          }
        }
        if (!ok) break;
        blocks += cnt;
        pieces.done();
      }
      cp_wait<0>();
    }
  } else if (loader >= 0) {
    // ------------------------------------------------------- bf16 rows
    // A copy of a block's keys or values is four units of 32 rows; the units of all copies go
    // round the loading warps.
    if constexpr (!FP8) {
      constexpr int NW = L::kLoaders;
      const int row_in = lane / L::kLPR, piece = lane % L::kLPR;
      const uint32_t sw = ((piece & 7) ^ row_in) << 4;
      uint32_t unit = loader;                  // the next one of this warp, of all
      uint32_t base = 0, blocks = 0;                     // copies and blocks before the piece
      while (!a.inject_stall) {
        const TreePiece* at_piece = pieces.next(wc);
        if (at_piece == nullptr) break;
        const TreePiece& it = *at_piece;
        const int hk = it.task % p.Hkv;
        const char* k_base = static_cast<const char*>(p.k_cache) + hk * p.ck_h * 2 + piece * 16;
        const char* v_base = static_cast<const char*>(p.v_cache) + hk * p.cv_h * 2 + piece * 16;
        const int32_t* table = p.page_table + it.b * p.ld_table;
        // A unit: its copy's kind and block, and this lane's key's place, looked up a unit ahead
        // (nothing is done to the page here: it would be waited for).
        struct Unit {
          int j, page, off;              // off -1: not loaded
          bool value;
        };
        auto look_up = [&](uint32_t u) {
          const int f = static_cast<int>((u >> 2) - base);
          Unit r;
          r.value = it.is_value(f);
          r.j = it.block(f);
          r.page = 0, r.off = -1;
          const int key = it.key(r.j) + (u & 3) * 32 + lane;
          if (f < 2 * it.cnt && key < it.hi && (key >= it.lo || key < p.first)) {
            const uint32_t n = (__umulhi(key, a.page_mul) + key) >> a.page_shift;
            r.off = key - static_cast<int>(n) * p.page_size;
            r.page = __ldg(table + n);
          }
          return r;
        };
        Unit next = look_up(unit);
        for (; (unit >> 2) - base < 2u * it.cnt; unit += NW) {
          const Unit now = next;
          next = look_up(unit + NW);
          const bool there =
              now.off >= 0 && static_cast<uint32_t>(now.page) < static_cast<uint32_t>(p.pages);
          if (now.off >= 0 && !there) atomicOr(p.status, kStatusBadIndex);
          const uint64_t at = !there ? 0
                              : now.value ? row_at(now.page, now.off, a.v_page, a.v_key)
                                          : row_at(now.page, now.off, a.k_page, a.k_key);
          const uint32_t mask = __ballot_sync(0xffffffffu, there);
          if (lane == 0 && !now.value)
            seen[((blocks + now.j) % kSeen) * 4 + (unit & 3)] = mask;
          const char* src = now.value ? v_base : k_base;
          const uint32_t fill = unit >> 2;
          const int st = fill % ST, rows = (unit & 3) * 32 + row_in;
          if (!wait_lean(&kv_empty[st], ((fill / ST) & 1) ^ 1, wc)) goto loads_done;
          const uint32_t dst = smem_u32(ring) + st * L::kTileBytes +
                               (piece >> 3) * L::kChunkBytes + rows * 128;
          copy_rows<L::kCopies, L::kRPI>(src, at, mask, row_in, a.far, [&](int i) {
            // (no carry: row_in is below kRPI, which divides the row)
            return dst + i * L::kRPI * 128 + (sw ^ ((i * L::kRPI & 7) << 4));
          });
          cp_arrive(&kv_full[st]);
          if (lane == 0) mbar_arrive(&kv_full[st]);
        }
        base += 2 * it.cnt;
        blocks += it.cnt;
        pieces.done();
      }
    loads_done:
      cp_wait<0>();
    }
  } else if (warp == kMmaWarp) {
    // -------------------------------------------------------------- MMAs
    constexpr uint32_t kDescS = FP8 ? idesc_f16(kBM, kBM) : idesc_bf16(kBM, kBM);
    constexpr uint32_t kDescO = (FP8 ? idesc_f16(kBM, D) : idesc_bf16(kBM, D)) | (1u << 16);
    const bool leader = elect_one();
    const uint64_t q_desc = sw128_desc(smem_u32(sQ)), k_desc = sw128_desc(smem_u32(ring));
    const uint64_t v_desc = sw128_desc_mn(smem_u32(ring), L::kChunkBytes);
    // (All that this warp waits for is usually there: what a turn costs it in instructions bounds
    // the kernel where the memory does not.)
    uint32_t base = 0, nq[2] = {0, 0}, np[2] = {0, 0};   // ring position, items, turns so far
    // What the operands' rows were written by: the copies of other threads, which have arrived
    // on the barrier, become visible to the tensor core's reads here; converted rows, and
    // q, have been made so by their writers.
    auto see = [&]() {
      tc_fence_after();
      if constexpr (!FP8) fence_proxy_async_smem();
    };
    auto issue_s = [&](int s, uint32_t fill) {
      const uint64_t qd = q_desc + s * (L::kTileBytes / 16);
      const uint64_t kd = k_desc + (fill % ST) * (L::kTileBytes / 16);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const int off = (k / 4) * (L::kChunkBytes / 16) + (k % 4) * 2;
        mma_f16(tmem + s * 128, qd + off, kd + off, kDescS, k > 0);
      }
    };
    // the keys of half `part` of a block; P of keys 64-127 lies where their scores began
    auto issue_o = [&](int s, uint32_t fill, int part, bool accumulate) {
      const uint64_t vd = v_desc + (fill % ST) * (L::kTileBytes / 16) + part * (4 * 2048 / 16);
      const uint32_t pa = tmem + s * 128 + part * 64;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        mma_f16_ts(tmem + 256 + s * 128, pa + k * 8, vd + k * (2048 / 16), kDescO,
                   accumulate || k > 0);
    };
    auto wait_kv = [&](uint32_t fill) {
      return wait_lean(&kv_full[fill % ST], (fill / ST) & 1, wc);
    };
    while (const TreePiece* it = pieces.next(wc)) {
      const bool single = it->flags & kSingle;
      const int cnt = it->cnt, turns = single ? cnt : 2 * cnt;
      auto block_of = [&](int t) { return single ? t : t >> 1; };
      auto k_fill = [&](int j) { return base + (j == 0 ? 0 : 2 * j - 1); };
      auto v_fill = [&](int j) { return base + (j + 1 < cnt ? 2 * j + 2 : 2 * j + 1); };
      for (int t = 0; t < 2 && t < turns; ++t) {
        const uint32_t f = k_fill(block_of(t));
        if (!wait_kv(f)) goto mma_done;
        if (!wait_lean(&q_full[t], nq[t] & 1, wc)) goto mma_done;
        ++nq[t];
        if (leader) {
          see();
          issue_s(t, f);
          mma_commit(&s_full[t]);
          if (single || t == 1) mma_commit(&kv_empty[f % ST]);
        }
      }
      for (int t = 0; t < turns; ++t) {
        const int s = t & 1;
        const uint32_t vf = v_fill(block_of(t));
        if (!wait_kv(vf)) goto mma_done;
#pragma unroll
        for (int part = 1; part >= 0; --part) {
          if (!wait_lean(&p_full[2 * s + part], np[s] & 1, wc)) goto mma_done;
          if (leader) {
            see();
            issue_o(s, vf, part, t > 1 || part == 0);
          }
        }
        ++np[s];
        if (leader && (single || s == 1)) mma_commit(&kv_empty[vf % ST]);
        if (t + 2 < turns) {
          const uint32_t kf = k_fill(block_of(t + 2));
          if (!wait_kv(kf)) goto mma_done;
          if (leader) {
            see();
            issue_s(s, kf);
            mma_commit(&s_full[s]);
            if (single || s == 1) mma_commit(&kv_empty[kf % ST]);
          }
        } else if (leader) {
          mma_commit(&o_full[s]);          // the piece's O is complete
        }
      }
      base += 2 * cnt;
      pieces.done();
    }
  mma_done:
    // the products in flight end before the tensor memory is freed
    if (leader) mma_commit(drain);
    volatile int zero = 0;
    WaitCtx dw{p.status, &zero, 1000000000ull};
    mbar_wait(drain, 0, dw);
  } else if (warp < kMmaWarp) {
    // ----------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int s = warp >> 2;                            // warpgroup
    const int row = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + s * 128 + lanes, tO = tmem + 256 + lanes;
    const int tok = row / a.G, g = row - tok * a.G;
    uint8_t* q_tile = sQ + s * L::kTileBytes;
    uint32_t ns = 0, no = 0, nm = 0, blocks = 0;
    while (const TreePiece* at_piece = pieces.next<false>(wc)) {
      const TreePiece& it = *at_piece;
      {
        const int hk = it.task % p.Hkv, h = hk * a.G + g;
        const float ks = FP8 && p.k_scale != nullptr ? __ldg(p.k_scale + hk) : 1.f;
        const float vs = FP8 && p.v_scale != nullptr ? __ldg(p.v_scale + hk) : 1.f;
        const bool single = it.flags & kSingle;
        const int cnt = it.cnt;
        const int turns = single ? (cnt - s + 1) / 2 : cnt;      // of this warpgroup
        const int i = (single ? 0 : s * a.TB) + tok;             // of the item's tokens
        const bool valid = tok < a.TB && i < it.ntok;
        const int64_t tokr = static_cast<int64_t>(it.q_row) + i;
        const int me = it.first + i, P = it.P;
        float c = p.scale * kLog2e;
        if (turns > 0) {
          // q, in the layout of the K operand's rows (16-byte pieces swizzled by the row)
          const uint4* src = reinterpret_cast<const uint4*>(
              static_cast<const __nv_bfloat16*>(p.q) + (valid ? tokr : 0) * p.q_t +
              static_cast<int64_t>(valid ? h : 0) * p.q_h);
          uint4 w[D / 8];
#pragma unroll
          for (int e = 0; e < D / 8; ++e) w[e] = valid ? __ldg(src + e) : make_uint4(0, 0, 0, 0);
          if constexpr (FP8) {
            float big = 0.f;
#pragma unroll
            for (int e = 0; e < D / 8; ++e) {
              const uint32_t x[4] = {w[e].x, w[e].y, w[e].z, w[e].w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                big = fmaxf(big, fabsf(__uint_as_float(x[k] << 16)));
                big = fmaxf(big, fabsf(__uint_as_float(x[k] & 0xFFFF0000u)));
              }
            }
            // the power of two that brings the largest to [2^14, 2^15) (a largest below
            // 2^-86: nearer to it; both powers are normal numbers)
            const int e2 = big > 0.f && big < INFINITY ? min(14 - ilogbf(big), 100) : 0;
            // the key scale's sign goes into q, and so does a scale of 0 or NaN: what
            // multiplies the scores below stays positive and keeps a masked key's -inf
            const float up = (ks > 0.f ? 1.f : ks < 0.f ? -1.f : ks) * ldexpf(1.f, e2);
            // the scores of the scaled q are below 2^32: 1e-30 of them is nothing
            c = fmaxf(c * fabsf(ks) * ldexpf(1.f, -e2), 1e-30f);
            auto half = [&](uint32_t x) {
              return f16x2(__uint_as_float(x << 16) * up, __uint_as_float(x & 0xFFFF0000u) * up);
            };
#pragma unroll
            for (int e = 0; e < D / 8; ++e)
              w[e] = make_uint4(half(w[e].x), half(w[e].y), half(w[e].z), half(w[e].w));
          }
#pragma unroll
          for (int e = 0; e < D / 8; ++e)
            *reinterpret_cast<uint4*>(q_tile + (e >> 3) * L::kChunkBytes + row * 128 +
                                      (((e & 7) ^ (row & 7)) << 4)) = w[e];
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&q_full[s]);
        }
        // the row's place: visible keys [0, first) and [lo, hi), and the path `cur`, its
        // parent, ... of which `up` steps are behind (a row that is not stored may see anything)
        const bool tree = p.parents != nullptr;
        const int32_t* parents = p.parents + (it.q_row - it.first);
        auto parent = [&](int k) {
          const int r = __ldg(parents + k);
          if (r >= -1 && r < k) return r;
          atomicOr(p.status, kStatusBadIndex);
          return -1;
        };
        int depth = me, cur = tree && valid ? me : -1, up = 0;
        if (tree && valid && p.window > 0) {
          depth = -1;
          for (int k = me; k >= 0; k = parent(k)) ++depth;
        }
        const int hi = !valid ? 1 << 30 : tree ? P : P + me + 1;
        const int lo = valid && p.window > 0 ? max(0, P + depth - p.window + 1) : 0;
        const int all_lo = __reduce_max_sync(0xffffffffu, lo);
        const int all_hi = __reduce_min_sync(0xffffffffu, hi);
        float m = -INFINITY, l = 0.f;
        for (int t = 0; t < turns; ++t) {
          const int j = single ? 2 * t + s : t;
          const int k0 = it.key(j);
          if (!mbar_wait_warp(&s_full[s], ns & 1, wc)) goto softmax_done;
          ++ns;
          tc_fence_after();
          const uint4 there = *reinterpret_cast<const uint4*>(seen + ((blocks + j) % kSeen) * 4);
          uint32_t vis[4] = {there.x, there.y, there.z, there.w};
          const bool masked = k0 + kBM > all_hi || k0 < all_lo ||
                              (there.x & there.y & there.z & there.w) != 0xffffffffu;
          if (masked) {
            uint32_t own[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int kq = k0 + 32 * q;
              own[q] = (~low_bits(lo - kq) | low_bits(p.first - kq)) & low_bits(hi - kq);
            }
            while (cur >= 0 && P + cur >= k0) {
              const int d = P + cur - k0;
              const bool sees = p.window == 0 || up < p.window || P + depth - up < p.first;
#pragma unroll
              for (int q = 0; q < 4; ++q)
                if (sees && (d >> 5) == q) own[q] |= 1u << (d & 31);
              cur = parent(cur);
              ++up;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) vis[q] &= own[q];
            __syncwarp();
            if constexpr (L::kRolled) {
#pragma unroll 1
              for (int q = 0; q < 4; ++q) {
                const uint32_t word = q < 2 ? vis[q == 0 ? 0 : 1] : vis[q == 2 ? 2 : 3];
                if (__all_sync(0xffffffffu, word == 0xffffffffu)) continue;
                float y[32];
                tmem_ld32(tS + 32 * q, y);
                uint32_t z[32];
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  z[e] = __float_as_uint((word >> e) & 1 ? y[e] : -INFINITY);
                tmem_st32(tS + 32 * q, z);
              }
              tmem_st_wait();
            }
          }
          // 64 scores, those that the mask hides as -inf, and their maximum
          auto scores = [&](float* x, int half) {
            tmem_ld32_async(tS + 64 * half, x);
            tmem_ld32_async(tS + 64 * half + 32, x + 32);
            tmem_wait32(x);
            tmem_wait32(x + 32);
            if (!L::kRolled && masked) {
#pragma unroll
              for (int e = 0; e < 64; ++e)
                x[e] = (vis[2 * half + (e >> 5)] >> (e & 31)) & 1 ? x[e] : -INFINITY;
            }
          };
          auto top = [&](const float* x) {
            float mq[2] = {fmaxf(x[0], x[1]), fmaxf(x[2], x[3])};
#pragma unroll
            for (int e = 4; e < 64; e += 4) {
              mq[0] = fmaxf(mq[0], fmaxf(x[e], x[e + 1]));
              mq[1] = fmaxf(mq[1], fmaxf(x[e + 2], x[e + 3]));
            }
            return fmaxf(mq[0], mq[1]);
          };
          // the row's scores; those of the first half are read again below (a row of 128
          // does not fit)
          float x[64];
          scores(x, 0);
          float mx = top(x);
          scores(x, 1);
          mx = fmaxf(mx, top(x));
          // raise the reference if it grows by more than 2^8 (at first: from -inf)
          const bool raise = (mx - m) * c > 8.f;
          if (__any_sync(0xffffffffu, raise)) {
            const float f = raise ? ex2((m - mx) * c) : 1.f;
            if (__any_sync(0xffffffffu, raise && m > -INFINITY)) {
              // the products of the turns before are complete: their commit came
              // before this turn's scores
#pragma unroll 1
              for (int q = 0; q < D; q += 32) {
                float o[32];
                tmem_ld32(tO + s * 128 + q, o);
                uint32_t w[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(o[e] * f);
                tmem_st32(tO + s * 128 + q, w);
              }
            }
            l *= f;
            if (raise) m = mx;
          }
          const float mc = m == -INFINITY ? 0.f : m * c;
          const uint64_t c2 = pack2(c, c), n2 = pack2(-mc, -mc);
          // weights, the second half of the keys first
          uint64_t sum[2] = {0, 0};
          auto weights = [&](uint32_t* w, const float* v) {
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float y, z;
              unpack2(fma2(pack2(v[e], v[e + 1]), c2, n2), &y, &z);
              y = ex2(y), z = ex2(z);
              w[e / 2] = FP8 ? f16x2(y, z) : bf16x2(y, z);
              sum[(e / 2) & 1] = add2(sum[(e / 2) & 1], pack2(y, z));
            }
          };
          auto hand_over = [&](int half) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[2 * s + half]);
          };
          if constexpr (L::kRolled) {
#pragma unroll 1
            for (int half = 1; half >= 0; --half) {
              uint32_t w[32];
              scores(x, half);
              weights(w, x);
              weights(w + 16, x + 32);
              tmem_st32(tS + 64 * half, w);
              hand_over(half);
            }
          } else {
            uint32_t w[32];
            weights(w, x);
            weights(w + 16, x + 32);
            tmem_st32(tS + 64, w);
            scores(x, 0);
            hand_over(1);
            weights(w, x);
            weights(w + 16, x + 32);
            tmem_st32(tS, w);
            hand_over(0);
          }
          float y, z;
          unpack2(add2(sum[0], sum[1]), &y, &z);
          l += y + z;
        }
        blocks += cnt;
        if (turns > 0) {
          if (!mbar_wait_warp(&o_full[s], no & 1, wc)) goto softmax_done;
          ++no;
          tc_fence_after();
        }
        // ---- the piece's end: columns [d0, d1) of the row, out of one or both outputs
        float ref = m == -INFINITY ? m : m * c;
        float f0 = 1.f, f1 = 0.f;
        bool both = false;
        int d0 = 0, d1 = D;
        if (single) {
          float2* ml = reinterpret_cast<float2*>(sQ);            // the q tiles are done with
          constexpr int kOther = L::kTileBytes / sizeof(float2);
          ml[s * kOther + row] = make_float2(ref, l);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&merge[0]);
          if (!mbar_wait_warp(&merge[0], nm & 1, wc)) goto softmax_done;
          tc_fence_after();
          const float2 m0 = ml[row], m1 = ml[kOther + row];
          both = cnt > 1;
          ref = both ? fmaxf(m0.x, m1.x) : m0.x;
          const float at = ref == -INFINITY ? 0.f : ref;
          f0 = ex2(m0.x - at), f1 = both ? ex2(m1.x - at) : 0.f;
          l = both ? m0.y * f0 + m1.y * f1 : m0.y;
          if (!both) f0 = 1.f;
          d0 = s * (D / 2), d1 = d0 + D / 2;
        }
        const uint32_t from = tO + (single ? 0 : s * 128);
        const bool direct = (it.flags & (kOpened | kClosed)) == (kOpened | kClosed);
        RowEnd end = {1.f, 0.f, false};
        float f = 1.f;
        if (direct) {
          end = finish_row(ref * kLn2, l, p.sinks != nullptr && valid ? p.sinks + h : nullptr);
          f = end.factor * vs;
        }
        const int64_t slot0 =
            (static_cast<int64_t>(it.task) * 2 + (it.flags & kSlot1 ? 1 : 0)) * kRows +
            (single ? 0 : s * kBM);
        const int64_t slot = slot0 + row;
        // Through shared memory (the tile of q is done with), so that four lanes write 64
        // adjacent bytes of a row: 32 columns of the output, or 16 of a partial result.  In the
        // warp's own rows of q, behind the references: after an item of two tiles no barrier keeps
        // the next one's q, which another warp may write at once, from other rows.
        uint8_t* stage = q_tile + 1024 + (warp & 3) * 4096;
        const uint32_t stored = __ballot_sync(0xffffffffu, valid);
        const int sub = lane >> 2, ch = lane & 3;
        const int64_t out_at = tokr * p.o_t + static_cast<int64_t>(h) * p.o_h;
        auto write_rows = [&](const uint4* v, char* base, auto at_of) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint4*>(stage + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4)) = v[e];
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = 8 * e + sub;
            const uint4 w = *reinterpret_cast<const uint4*>(stage + r * 64 +
                                                            ((ch ^ ((r >> 1) & 3)) << 4));
            const int64_t to = at_of(r);
            if ((stored >> r) & 1) *reinterpret_cast<uint4*>(base + to + ch * 16) = w;
          }
          __syncwarp();
        };
        for (int d = d0; d < d1; d += 32) {
          float o[32];
          tmem_ld32(from + d, o);
          if (both) {
            float o1[32];
            tmem_ld32(from + 128 + d, o1);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = o[e] * f0 + o1[e] * f1;
          }
          uint4 v[4];
          if (direct) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[e] = end.none ? make_uint4(0u, 0u, 0u, 0u)
                              : make_uint4(bf16x2(o[8 * e] * f, o[8 * e + 1] * f),
                                           bf16x2(o[8 * e + 2] * f, o[8 * e + 3] * f),
                                           bf16x2(o[8 * e + 4] * f, o[8 * e + 5] * f),
                                           bf16x2(o[8 * e + 6] * f, o[8 * e + 7] * f));
            write_rows(v, static_cast<char*>(p.out), [&](int r) {
              return 2 * (__shfl_sync(0xffffffffu, out_at, r) + d);
            });
          } else {
            const int64_t first = (slot0 + (warp & 3) * 32) * D + d;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float* x = o + 16 * half + 4 * e;
                v[e] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]),
                                  __float_as_uint(x[2]), __float_as_uint(x[3]));
              }
              write_rows(v, reinterpret_cast<char*>(a.part_o),
                         [&](int r) { return 4 * (first + r * D + 16 * half); });
            }
          }
        }
        if (valid && d0 == 0) {
          if (direct) {
            if (p.lse != nullptr) p.lse[tokr * p.Hq + h] = end.lse;
          } else {
            a.part_ml[slot] = make_float2(ref, l);
          }
        }
        tc_fence_before();
        if (single) {
          // neither output nor reference is written again before both have read them
          __syncwarp();
          if (lane == 0) mbar_arrive(&merge[1]);
          if (!mbar_wait_warp(&merge[1], nm & 1, wc)) goto softmax_done;
          ++nm;
        }
      }
      pieces.done();
    }
  softmax_done:;
  }

  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the partial results of an item that several parts share, in the parts' order:
// out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i.  D / 4 lanes take two rows, four columns
// each, reading four parts of both at a time: what counts is one chain of loads.  (A warp a row:
// 16 us for two chunks of 300 rows.)  A block's y is its rows, its x the head and the part that
// begins the item.  kSplit: few rows, whose parts the block's warps share, and few items, so that x
// counts those that are shared (one tree over 20000 keys in 19 parts: 25.7 us, without 35.2; over 4000
// keys 14.0 and 21.5; finding them costs 64 ragged sequences 4 us).  "Few" is 8 blocks an SM: with 2 or
// 32 none of 17 shapes of 1 to 200 sequences is faster or slower.
constexpr int kJoinWarps = 4;
template <int D>
struct JoinShape {
  static constexpr int kLPR = D / 4, kRPW = 2 * (32 / kLPR);      // rows of a warp
};
struct JoinSum {
  float m = -INFINITY, l = 0.f;
  float4 o = {0.f, 0.f, 0.f, 0.f};
  __device__ __forceinline__ void add(float2 ml, float4 v) {
    // a part whose scores are all NaN has no reference, but a sum: it counts
    const float n = fmaxf(m, ml.x), at = n == -INFINITY ? 0.f : n;
    const float f = ex2(m - at), k = ex2(ml.x - at);
    l = l * f + ml.y * k;
    o.x = o.x * f + v.x * k;
    o.y = o.y * f + v.y * k;
    o.z = o.z * f + v.z * k;
    o.w = o.w * f + v.w * k;
    m = n;
  }
};
template <int D, bool kSplit>
__global__ void __launch_bounds__(32 * kJoinWarps) tree_join_kernel(const TreeArgs a) {
  using S = JoinShape<D>;
  constexpr int U = 4;
  const TreeParams& p = a.p;
  __shared__ float4 so[kSplit ? kJoinWarps : 1][2][32];
  __shared__ float2 sml[kSplit ? kJoinWarps : 1][2][32];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hk = blockIdx.x % p.Hkv;
  // the part that begins the item
  int which = blockIdx.x / p.Hkv, begins = kSplit ? -1 : which;
  for (int w = 0; w < a.parts && begins < 0; w += 32) {
    const bool one = w + lane < a.parts && a.joins[(w + lane) * p.Hkv + hk].ntok > 0;
    uint32_t mask = __ballot_sync(0xffffffffu, one);
    const int n = __popc(mask);
    if (which < n) {
      for (; which > 0; --which) mask &= mask - 1;
      begins = w + __ffs(mask) - 1;
    }
    which -= n;
  }
  if (begins < 0) return;
  const TreeJoin j = a.joins[begins * p.Hkv + hk];
  if (j.ntok == 0) return;
  const int col = 4 * (lane % S::kLPR);
  const int row0 = (kSplit ? blockIdx.y : blockIdx.y * kJoinWarps + warp) * S::kRPW +
                   2 * (lane / S::kLPR);
  bool valid[2];
  int token[2], head[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = row0 + r, s = row / kBM, in = row - s * kBM, tok = in / a.G;
    token[r] = s * a.TB + tok;
    head[r] = hk * a.G + in - tok * a.G;
    valid[r] = row < kRows && tok < a.TB && token[r] < j.ntok;
  }
  JoinSum sum[2];
  const int step = kSplit ? kJoinWarps : 1;
  for (int w = j.w0 + (kSplit ? warp : 0); w <= j.w1; w += U * step) {
    float2 ml[U][2];
    float4 v[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int k = w + u * step;
        if (k > j.w1 || !valid[r]) continue;
        const int64_t task = static_cast<int64_t>(k) * p.Hkv + hk;
        const int64_t slot = (task * 2 + (k == j.w0 ? j.first : 0)) * kRows + row0 + r;
        ml[u][r] = a.part_ml[slot];
        v[u][r] = *reinterpret_cast<const float4*>(a.part_o + slot * D + col);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (w + u * step <= j.w1 && valid[r]) sum[r].add(ml[u][r], v[u][r]);
  }
  if constexpr (kSplit) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      sml[warp][r][lane] = make_float2(sum[r].m, sum[r].l);
      so[warp][r][lane] = sum[r].o;
    }
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int w = 1; w < kJoinWarps; ++w) sum[r].add(sml[w][r][lane], so[w][r][lane]);
  }
  const float vs = p.v_scale != nullptr ? __ldg(p.v_scale + hk) : 1.f;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    if (!valid[r]) continue;
    const int64_t tokr = static_cast<int64_t>(j.q_row) + token[r];
    const float4 o = sum[r].o;
    const RowEnd end =
        finish_row(sum[r].m * kLn2, sum[r].l, p.sinks ? p.sinks + head[r] : nullptr);
    const float f = end.factor * vs;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + tokr * p.o_t +
                         static_cast<int64_t>(head[r]) * p.o_h + col;
    *reinterpret_cast<uint2*>(dst) = end.none
                                         ? make_uint2(0u, 0u)
                                         : make_uint2(bf16x2(o.x * f, o.y * f),
                                                      bf16x2(o.z * f, o.w * f));
    if (p.lse != nullptr && col == 0) p.lse[tokr * p.Hq + head[r]] = end.lse;
  }
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

int parts_of(int Hkv, int num_sms) { return std::max(1, num_sms / Hkv); }

size_t joins_bytes(int Hkv, int num_sms) {
  return round256(static_cast<size_t>(parts_of(Hkv, num_sms)) * Hkv * sizeof(TreeJoin));
}
// results of pieces: none where there is one part
int64_t part_rows(int Hkv, int num_sms) {
  const int parts = parts_of(Hkv, num_sms);
  return parts > 1 ? static_cast<int64_t>(parts) * Hkv * 2 * kRows : 0;
}

template <int D, bool FP8>
cudaError_t launch(const TreeArgs& a, int num_sms, cudaStream_t stream) {
  using L = TreeLayout<D, FP8>;
  const int smem = L::kSmem + 1024;
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(tree_kernel<D, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  const int tasks = a.parts * a.p.Hkv;
  e = launch_k(tree_kernel<D, FP8>, dim3(std::min(tasks, num_sms)), dim3(kTreeThreads),
               static_cast<size_t>(smem), stream, a);
  if (e != cudaSuccess || a.all_whole) return e;
  // rows that an item can have, and items that parts may share
  const int64_t T = a.p.T;
  const int rows = T > a.TB ? kRows : static_cast<int>(T) * a.G;
  const int64_t items = std::min<int64_t>(a.parts, T / (2 * a.TB) + a.p.B);
  constexpr int kRPW = JoinShape<D>::kRPW, kPerBlock = kJoinWarps * kRPW;
  const unsigned fine = static_cast<unsigned>((rows + kRPW - 1) / kRPW);
  if (items * a.p.Hkv * fine <= 8 * num_sms)
    return launch_k(tree_join_kernel<D, true>,
                    dim3(static_cast<unsigned>(items * a.p.Hkv), fine), dim3(32 * kJoinWarps), 0,
                    stream, a);
  return launch_k(tree_join_kernel<D, false>,
                  dim3(static_cast<unsigned>(tasks),
                       static_cast<unsigned>((rows + kPerBlock - 1) / kPerBlock)),
                  dim3(32 * kJoinWarps), 0, stream, a);
}

}  // namespace

size_t tree_workspace_bytes(int64_t, int64_t, int, int Hkv, int D, int num_sms) {
  const int64_t rows = part_rows(Hkv, num_sms);
  return joins_bytes(Hkv, num_sms) + round256(rows * sizeof(float2)) + rows * D * sizeof(float);
}

cudaError_t launch_tree(const TreeParams& p, int num_sms, cudaStream_t stream) {
  TreeArgs a = {};
  a.p = p;
  a.G = p.Hq / p.Hkv;
  a.TB = kBM / a.G;
  a.parts = parts_of(p.Hkv, num_sms);
  const int64_t unit = p.fp8 ? 16 : 8;                   // elements in 16 bytes
  a.k_page = static_cast<uint32_t>(p.ck_p / unit), a.k_key = static_cast<uint32_t>(p.ck_t / unit);
  a.v_page = static_cast<uint32_t>(p.cv_p / unit), a.v_key = static_cast<uint32_t>(p.cv_t / unit);
  auto span = [&](uint32_t page, uint32_t key) {
    return static_cast<uint64_t>(p.pages - 1) * (p.pages > 1 ? page : 0) +
           static_cast<uint64_t>(p.page_size - 1) * (p.page_size > 1 ? key : 0);
  };
  a.far = std::max(span(a.k_page, a.k_key), span(a.v_page, a.v_key)) >> 32 != 0;
  while ((1u << a.page_shift) < static_cast<uint32_t>(p.page_size)) ++a.page_shift;
  a.page_mul = static_cast<uint32_t>(
      ((1ull << 32) * ((1ull << a.page_shift) - p.page_size)) / p.page_size + 1);
  // Blocks of the longest item that there can be
  int64_t blocks = (p.max_pages * p.page_size + kBM - 1) / kBM;
  if (p.window > 0)
    blocks = std::min<int64_t>(blocks, (static_cast<int64_t>(p.window) + p.T + kBM - 1) / kBM + 1 +
                                           (p.first + kBM - 1) / kBM);
  a.all_whole = blocks <= kAllWhole || a.parts == 1;
  char* ws = static_cast<char*>(p.workspace);
  a.joins = reinterpret_cast<TreeJoin*>(ws);
  ws += joins_bytes(p.Hkv, num_sms);
  a.part_ml = reinterpret_cast<float2*>(ws);
  a.part_o = reinterpret_cast<float*>(
      ws + round256(part_rows(p.Hkv, num_sms) * sizeof(float2)));
  a.budget_ns = static_cast<unsigned long long>(option(MXQ_OPT_WAIT_BUDGET_NS));
  a.inject_stall = static_cast<int>(option(MXQ_OPT_INJECT_STALL));
  if (p.D == 128)
    return p.fp8 ? launch<128, true>(a, num_sms, stream) : launch<128, false>(a, num_sms, stream);
  return p.fp8 ? launch<64, true>(a, num_sms, stream) : launch<64, false>(a, num_sms, stream);
}

}  // namespace mxq
