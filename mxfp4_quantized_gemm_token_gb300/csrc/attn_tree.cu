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
//   warps 8-11       load keys and values with 16-byte asynchronous copies, row by row, as pages
//                    are of any size; e4m3 is converted to f16 (exact) on its way
//   warp 12          issues the MMAs
// S0, S1, O0 and O1 are in tensor memory, P takes the place of S.  The reference a
// row subtracts is raised only when its maximum grows by more than 2^8.
//   bf16 cache: bf16 products.  e4m3 cache: f16 products, q scaled per row by a power of two to
//   use f16's range (exact for elements within 2^31 of the row's largest).
//
// A row's path is followed while its blocks are taken, from the last key down: the thread holds
// the next ancestor, and a block's part of the path becomes a bit mask.
//
// Work.  The key blocks of all items form one line, cut into equal parts; a (part, key/value
// head) pair is one CTA's, the heads of a part at work at the same time.  Items that parts share
// leave at most two partial results per CTA in the workspace, which a second kernel joins in
// a fixed order.  A part's end inside a short item moves to the nearer end of it.
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
constexpr int kTreeThreads = 416;
constexpr int kTreeWarps = kTreeThreads / 32;
constexpr int kLoadWarp = 8, kMmaWarp = 12;
constexpr int kSeen = 16;            // blocks whose masks of loaded keys are kept: at most 8 are in use
constexpr int kWhole = 2;            // items of at most this many blocks stay whole
constexpr int kAllWhole = 3;         // calls whose items have at most this many: all do

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
  int parts, min_blocks;
  bool all_whole;                    // no item is cut
  bool alike;                        // both caches have the same page and token strides
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
  static constexpr int kCopies = 32 / kRPI;              // copies a thread and stage
  // stages of 16-bit operands; copies ahead of what is handed over
  static constexpr int kStages = FP8 ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 10);
  static constexpr int kLag = FP8 ? (D == 128 ? 3 : 6) : (D == 128 ? 3 : 6);
  static constexpr int kRaw = FP8 ? (kLag + 1) * kBM * kRowBytes : 0;
  static constexpr int kBars = 2 * 7 + 2 * kStages + 1;
  static constexpr int kSmem = (2 + kStages) * kTileBytes + kRaw + 8 * kBars + 16 + 16 * kSeen;
  static_assert(kSmem + 1024 <= 226 * 1024, "shared memory over budget");
  // a stage is released once the copy after it has been handed over (see the loads)
  static_assert(FP8 || kLag + 2 <= kStages, "the loads would wait for themselves");
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

// The pieces of items in a CTA's part of the line, in order.
struct TreeWalk {
  const TreeArgs& a;
  int b, i, off;
  int64_t pos, left;
  TreeSeq s;
  int next_to, next_len;             // of sequence b + 1
  // the piece
  TreeItem it;
  int first;                         // its first token, of the sequence's
  int v1, cnt;                       // its blocks v1 - 1, v1 - 2, ...
  int64_t begin;                     // the item's place on the line
  bool opened, closed;
  __device__ __forceinline__ TreeWalk(const TreeArgs& args, int b0, int i0, int off0, int64_t s0,
                                      int64_t s1)
      : a(args), b(b0), i(i0), off(off0), pos(s0), left(s1 - s0) {
    if (left <= 0) return;
    s = tree_seq(a.p, a.p.cu_q[b], a.p.cu_q[b + 1], a.p.seq_lens[b]);
    ahead();
  }
  __device__ __forceinline__ void ahead() {
    const bool more = b + 1 < a.p.B;
    next_to = more ? a.p.cu_q[b + 2] : 0;
    next_len = more ? a.p.seq_lens[b + 1] : 0;
  }
  __device__ __forceinline__ bool next() {
    if (left <= 0) return false;
    while (true) {
      if (i * 2 * a.TB >= s.nq) {
        if (b + 1 >= a.p.B) return false;
        const int from = a.p.cu_q[b + 1];
        ++b;
        s = tree_seq(a.p, from, next_to, next_len);
        ahead();
        i = 0;
        continue;
      }
      it = tree_item(a, s, i);
      if (off < it.n) break;
      off = 0;
      ++i;
    }
    first = i * 2 * a.TB;
    begin = pos - off;
    cnt = static_cast<int>(min(static_cast<int64_t>(it.n - off), left));
    v1 = it.n - off;
    opened = off == 0;
    closed = off + cnt == it.n;
    pos += cnt;
    left -= cnt;
    off += cnt;
    return true;
  }
  // first key of the piece's block j
  __device__ __forceinline__ int key(int j) const {
    const int v = v1 - 1 - j;
    return (v < it.head ? v : v + it.skip) * kBM;
  }
  __device__ __forceinline__ bool single() const { return it.ntok <= a.TB; }
};

template <int N>
__device__ __forceinline__ void cp_wait_upto(int n) {
  // all but the last n of at most N groups
  if constexpr (N > 0) {
    if (n >= N) {
      cp_wait<N>();
      return;
    }
    cp_wait_upto<N - 1>(n);
  } else {
    cp_wait<0>();
  }
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
  uint32_t* seen = reinterpret_cast<uint32_t*>(raw + L::kRaw);   // [kSeen][4]
  uint64_t* q_full = reinterpret_cast<uint64_t*>(seen + 4 * kSeen);
  uint64_t* s_full = q_full + 2;
  uint64_t* p_full = s_full + 2;      // [s][half]
  uint64_t* o_full = p_full + 4;
  uint64_t* merge = o_full + 2;       // both results there, both read
  uint64_t* kv_full = merge + 2;
  uint64_t* kv_empty = kv_full + ST;
  uint64_t* drain = kv_empty + ST;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  __shared__ unsigned long long warp_sum[kTreeWarps];
  __shared__ int warp_longest[kTreeWarps];
  __shared__ long long range[2];      // the part's blocks on the line
  __shared__ int start[3];            // its first sequence, item and block of that
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
      mbar_init(&kv_full[i], 4);          // the loading warps
      mbar_init(&kv_empty[i], 1);
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

  // ---- the line, and this CTA's part of it
  const int per_thread = (p.B + kTreeThreads - 1) / kTreeThreads;
  const int b0 = threadIdx.x * per_thread, b1 = min(p.B, b0 + per_thread);
  auto seq = [&](int b) { return tree_seq(p, p.cu_q[b], p.cu_q[b + 1], p.seq_lens[b]); };
  unsigned long long mine = 0;
  int longest = 0;
  for (int b = b0; b < b1; ++b) {
    const TreeSeq s = seq(b);
    if (s.bad && blockIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
    for (int i = 0; i * 2 * a.TB < s.nq; ++i) {
      const int n = tree_item(a, s, i).n;
      mine += n;
      longest = max(longest, n);
    }
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  unsigned long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sum[warp] = incl, warp_longest[warp] = longest;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int64_t before = static_cast<int64_t>(incl - mine), total = 0;
  for (int w = 0; w < kTreeWarps; ++w) {
    if (w < warp) before += static_cast<int64_t>(warp_sum[w]);
    total += static_cast<int64_t>(warp_sum[w]);
    longest = max(longest, warp_longest[w]);
  }
  int64_t per = max((total + a.parts - 1) / a.parts, static_cast<int64_t>(a.min_blocks));
  // where all stay whole, a part has room for the longest, or some would get two
  if (a.all_whole && per < longest) per = longest;
  const int whole =
      a.all_whole ? longest : static_cast<int>(min(static_cast<int64_t>(kWhole), per));
  const int part = static_cast<int>(blockIdx.x) / p.Hkv;
  const int64_t raw0 = part * per;
  if (threadIdx.x < 2) range[threadIdx.x] = total;
  __syncthreads();
  {
    // the thread that holds an end of the part finds its item; inside a short one it moves to
    // the nearer end
    int64_t at = before;
    for (int end = 0; end < 2; ++end) {
      const int64_t pos = raw0 + end * per;
      if (pos < before || pos >= before + static_cast<int64_t>(mine)) continue;
      at = before;
      bool found = false;
      for (int b = b0; b < b1 && !found; ++b) {
        const TreeSeq s = seq(b);
        for (int i = 0; i * 2 * a.TB < s.nq && !found; ++i) {
          const int n = tree_item(a, s, i).n;
          if (at + n <= pos) {
            at += n;
            continue;
          }
          found = true;
          int off = static_cast<int>(pos - at);
          if (n <= whole) off = 2 * off >= n && off > 0 ? n : 0;
          range[end] = at + off;
          if (end == 0) start[0] = b, start[1] = i, start[2] = off;
        }
      }
    }
  }
  __syncthreads();
  const int64_t s0 = range[0], s1 = range[1];
  const int tasks = a.parts * p.Hkv;

  if (warp >= kLoadWarp && warp < kMmaWarp) {
    // ------------------------------------------------------------ loads
    constexpr int es = FP8 ? 1 : 2;
    const int lw = warp - kLoadWarp;                     // rows [32 lw, + 32) of a block
    const int row_in = lane / L::kLPR, piece = lane % L::kLPR;
    uint32_t issued = 0, given = 0, blocks = 0;          // copies begun and handed over
    bool ok = true;
    // Hands over the oldest copy.  It is released by the MMAs no later than after the copy
    // that follows it has been handed over, so a stage's wait ends.
    auto hand_over = [&]() {
      cp_wait_upto<L::kLag>(static_cast<int>(issued - given) - 1);
      const int st = given % ST;
      if constexpr (FP8) {
        if (!mbar_wait_warp(&kv_empty[st], ((given / ST) & 1) ^ 1, wc)) return false;
        const uint8_t* src = raw + (given % (L::kLag + 1)) * (kBM * L::kRowBytes) +
                             (lw * L::kCopies * 32 + lane) * 16;
        uint8_t* dst = ring + st * L::kTileBytes + (piece >> 2) * L::kChunkBytes;
#pragma unroll
        for (int i = 0; i < L::kCopies; ++i) {
          const uint4 x = *reinterpret_cast<const uint4*>(src + i * 512);
          const int r = lw * 32 + i * L::kRPI + row_in;
          uint4 lo, hi;
          e4m3x4_f16(x.x, &lo.x, &lo.y);
          e4m3x4_f16(x.y, &lo.z, &lo.w);
          e4m3x4_f16(x.z, &hi.x, &hi.y);
          e4m3x4_f16(x.w, &hi.z, &hi.w);
          // (the second chunk's lanes write their pieces the other way round: the first's
          // are in the same banks)
          const int c0 = (2 * piece) & 7, swap = piece >> 2;
          uint8_t* to = dst + r * 128;
          *reinterpret_cast<uint4*>(to + (((c0 + swap) ^ (r & 7)) << 4)) = swap ? hi : lo;
          *reinterpret_cast<uint4*>(to + (((c0 + 1 - swap) ^ (r & 7)) << 4)) = swap ? lo : hi;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&kv_full[st]);
      ++given;
      return true;
    };
    if (a.inject_stall) goto loads_done;
    for (int task = blockIdx.x; ok && task < tasks; task += gridDim.x) {
      const int hk = task % p.Hkv;
      const char* k_base = static_cast<const char*>(p.k_cache) + hk * p.ck_h * es + piece * 16;
      const char* v_base = static_cast<const char*>(p.v_cache) + hk * p.cv_h * es + piece * 16;
      TreeWalk walk(a, start[0], start[1], start[2], s0, s1);
      while (ok && walk.next()) {
        // this lane's key of a block: its page, looked up a block ahead
        struct Spot {
          int page, off;
          bool wanted;
        };
        const int32_t* table = p.page_table + walk.b * p.ld_table;
        auto look_up = [&](int j) {
          Spot r = {0, 0, false};
          if (j >= walk.cnt) return r;
          const int key = walk.key(j) + lw * 32 + lane;
          r.wanted = key < walk.it.hi && (key >= walk.it.lo || key < p.first);
          if (r.wanted) {
            const uint32_t n = static_cast<uint32_t>(key) / static_cast<uint32_t>(p.page_size);
            r.off = key - static_cast<int>(n) * p.page_size;
            r.page = __ldg(table + n);
          }
          return r;
        };
        // a copy of 32 rows; mask: those that exist
        auto copy = [&](const char* base, int64_t at, uint32_t mask) {
          uint32_t dst;
          if constexpr (FP8) {
            dst = smem_u32(raw) + (issued % (L::kLag + 1)) * (kBM * L::kRowBytes) +
                  (lw * L::kCopies * 32 + lane) * 16;
#pragma unroll
            for (int i = 0; i < L::kCopies; ++i) {
              const int r = i * L::kRPI + row_in;
              cp16(dst + i * 512, base + __shfl_sync(0xffffffffu, at, r), (mask >> r) & 1);
            }
          } else {
            const int st = issued % ST;
            if (!mbar_wait_warp(&kv_empty[st], ((issued / ST) & 1) ^ 1, wc)) return false;
            dst = smem_u32(ring) + st * L::kTileBytes + (piece >> 3) * L::kChunkBytes;
#pragma unroll
            for (int i = 0; i < L::kCopies; ++i) {
              const int r = i * L::kRPI + row_in, rt = lw * 32 + r;
              cp16(dst + rt * 128 + (((piece & 7) ^ (rt & 7)) << 4),
                   base + __shfl_sync(0xffffffffu, at, r), (mask >> r) & 1);
            }
          }
          cp_commit();
          ++issued;
          return issued - given <= L::kLag || hand_over();
        };
        Spot next = look_up(0);
        int64_t v_at = 0;
        uint32_t v_mask = 0;
        // K_0, K_1, V_0, K_2, V_1, ...
        for (int j = 0; ok && j <= walk.cnt; ++j) {
          const int64_t vo = v_at;
          const uint32_t vm = v_mask;
          if (j < walk.cnt) {
            const Spot now = next;
            next = look_up(j + 1);
            const bool there =
                now.wanted && static_cast<uint32_t>(now.page) < static_cast<uint32_t>(p.pages);
            if (now.wanted && !there) atomicOr(p.status, kStatusBadIndex);
            const int64_t page = there ? now.page : 0, off = there ? now.off : 0;
            const int64_t ko = (page * p.ck_p + off * p.ck_t) * es;
            v_at = a.alike ? ko : (page * p.cv_p + off * p.cv_t) * es;
            v_mask = __ballot_sync(0xffffffffu, there);
            if (lane == 0) seen[(blocks % kSeen) * 4 + lw] = v_mask;
            ++blocks;
            ok = copy(k_base, ko, v_mask);
          }
          if (ok && j > 0) ok = copy(v_base, vo, vm);
        }
      }
    }
    while (ok && given < issued) ok = hand_over();
  loads_done:
    cp_wait<0>();
  } else if (warp == kMmaWarp) {
    // -------------------------------------------------------------- MMAs
    constexpr uint32_t kDescS = FP8 ? idesc_f16(kBM, kBM) : idesc_bf16(kBM, kBM);
    constexpr uint32_t kDescO = (FP8 ? idesc_f16(kBM, D) : idesc_bf16(kBM, D)) | (1u << 16);
    const bool leader = elect_one();
    const uint64_t q_desc = sw128_desc(smem_u32(sQ)), k_desc = sw128_desc(smem_u32(ring));
    const uint64_t v_desc = sw128_desc_mn(smem_u32(ring), L::kChunkBytes);
    uint32_t base = 0, nq[2] = {0, 0}, np[2] = {0, 0};   // ring position, items, turns so far
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
      return mbar_wait_warp(&kv_full[fill % ST], (fill / ST) & 1, wc);
    };
    for (int task = blockIdx.x; task < tasks; task += gridDim.x) {
      TreeWalk walk(a, start[0], start[1], start[2], s0, s1);
      while (walk.next()) {
        const bool single = walk.single();
        const int cnt = walk.cnt, turns = single ? cnt : 2 * cnt;
        auto block_of = [&](int t) { return single ? t : t >> 1; };
        auto k_fill = [&](int j) { return base + (j == 0 ? 0 : 2 * j - 1); };
        auto v_fill = [&](int j) { return base + (j + 1 < cnt ? 2 * j + 2 : 2 * j + 1); };
        for (int t = 0; t < 2 && t < turns; ++t) {
          const uint32_t f = k_fill(block_of(t));
          if (!wait_kv(f)) goto mma_done;
          if (!mbar_wait_warp(&q_full[t], nq[t] & 1, wc)) goto mma_done;
          ++nq[t];
          if (leader) {
            tc_fence_after();
            issue_s(t, f);
            mma_commit(&s_full[t]);
            if (single || t == 1) mma_commit(&kv_empty[f % ST]);
          }
          __syncwarp();
        }
        for (int t = 0; t < turns; ++t) {
          const int s = t & 1;
          const uint32_t vf = v_fill(block_of(t));
          if (!wait_kv(vf)) goto mma_done;
#pragma unroll
          for (int part = 1; part >= 0; --part) {
            if (!mbar_wait_warp(&p_full[2 * s + part], np[s] & 1, wc)) goto mma_done;
            if (leader) {
              tc_fence_after();
              issue_o(s, vf, part, t > 1 || part == 0);
            }
            __syncwarp();
          }
          ++np[s];
          if (leader && (single || s == 1)) mma_commit(&kv_empty[vf % ST]);
          if (t + 2 < turns) {
            const uint32_t kf = k_fill(block_of(t + 2));
            if (!wait_kv(kf)) goto mma_done;
            if (leader) {
              tc_fence_after();
              issue_s(s, kf);
              mma_commit(&s_full[s]);
              if (single || s == 1) mma_commit(&kv_empty[kf % ST]);
            }
          } else if (leader) {
            mma_commit(&o_full[s]);          // the piece's O is complete
          }
          __syncwarp();
        }
        base += 2 * cnt;
      }
    }
  mma_done:
    // the products in flight end before the tensor memory is freed
    if (leader) mma_commit(drain);
    volatile int zero = 0;
    WaitCtx dw{p.status, &zero, 1000000000ull};
    mbar_wait(drain, 0, dw);
  } else {
    // ----------------------------------------------------------- softmax
    const int s = warp >> 2;                            // warpgroup
    const int row = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + s * 128 + lanes, tO = tmem + 256 + lanes;
    const int tok = row / a.G, g = row - tok * a.G;
    uint8_t* q_tile = sQ + s * L::kTileBytes;
    uint32_t ns = 0, no = 0, nm = 0, blocks = 0;
    for (int task = blockIdx.x; task < tasks; task += gridDim.x) {
      const int hk = task % p.Hkv, h = hk * a.G + g;
      const float ks = FP8 && p.k_scale != nullptr ? __ldg(p.k_scale + hk) : 1.f;
      const float vs = FP8 && p.v_scale != nullptr ? __ldg(p.v_scale + hk) : 1.f;
      if (threadIdx.x == 0) a.joins[task].ntok = 0;
      TreeWalk walk(a, start[0], start[1], start[2], s0, s1);
      while (walk.next()) {
        const bool single = walk.single();
        const int cnt = walk.cnt;
        const int turns = single ? (cnt - s + 1) / 2 : cnt;      // of this warpgroup
        const int i = (single ? 0 : s * a.TB) + tok;             // of the item's tokens
        const bool valid = tok < a.TB && i < walk.it.ntok;
        const int64_t tokr = static_cast<int64_t>(walk.s.q0) + walk.first + i;
        const int me = walk.first + i, P = walk.s.len - walk.s.nq;
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
        const int32_t* parents = p.parents + walk.s.q0;
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
          const int k0 = walk.key(j);
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
          }
          // 64 scores, those that the mask hides as -inf, and their maximum
          auto scores = [&](float* x, int half) {
            tmem_ld32_async(tS + 64 * half, x);
            tmem_ld32_async(tS + 64 * half + 32, x + 32);
            tmem_wait32(x);
            tmem_wait32(x + 32);
            if (masked) {
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
          // weights, the second half first: it is in registers, the first one's scores are
          // read again (a row of 128 would not fit)
          uint64_t sum[2] = {0, 0};
          auto weights = [&](const float* v, int half) {
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 64; e += 2) {
              float y, z;
              unpack2(fma2(pack2(v[e], v[e + 1]), c2, n2), &y, &z);
              y = ex2(y), z = ex2(z);
              w[e / 2] = FP8 ? f16x2(y, z) : bf16x2(y, z);
              sum[(e / 2) & 1] = add2(sum[(e / 2) & 1], pack2(y, z));
            }
            tmem_st32(tS + 64 * half, w);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[2 * s + half]);
          };
          weights(x, 1);
          scores(x, 0);
          weights(x, 0);
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
        const bool direct = walk.opened && walk.closed;
        RowEnd end = {1.f, 0.f, false};
        float f = 1.f;
        if (direct) {
          end = finish_row(ref * kLn2, l, p.sinks != nullptr && valid ? p.sinks + h : nullptr);
          f = end.factor * vs;
        }
        const int64_t slot =
            (static_cast<int64_t>(task) * 2 + (walk.opened && raw0 < walk.begin ? 1 : 0)) * kRows +
            (single ? 0 : s * kBM) + row;
        __nv_bfloat16* dst =
            static_cast<__nv_bfloat16*>(p.out) + tokr * p.o_t + static_cast<int64_t>(h) * p.o_h;
        for (int d = d0; d < d1; d += 32) {
          float o[32];
          tmem_ld32(from + d, o);
          if (both) {
            float o1[32];
            tmem_ld32(from + 128 + d, o1);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = o[e] * f0 + o1[e] * f1;
          }
          if (valid && direct) {
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              *reinterpret_cast<uint4*>(dst + d + e) =
                  end.none ? make_uint4(0u, 0u, 0u, 0u)
                           : make_uint4(bf16x2(o[e] * f, o[e + 1] * f),
                                        bf16x2(o[e + 2] * f, o[e + 3] * f),
                                        bf16x2(o[e + 4] * f, o[e + 5] * f),
                                        bf16x2(o[e + 6] * f, o[e + 7] * f));
          } else if (valid) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4*>(a.part_o + slot * D + d + e) =
                  make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
          __syncwarp();
        }
        if (valid && d0 == 0) {
          if (direct) {
            if (p.lse != nullptr) p.lse[tokr * p.Hq + h] = end.lse;
          } else {
            a.part_ml[slot] = make_float2(ref, l);
          }
        }
        if (threadIdx.x == 0 && walk.opened && !walk.closed) {
          TreeJoin& to = a.joins[task];
          to.q_row = walk.s.q0 + walk.first;
          to.ntok = walk.it.ntok;
          to.w0 = part;
          to.w1 = static_cast<int>((walk.begin + walk.it.n - 1) / per);
          to.first = raw0 < walk.begin ? 1 : 0;
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
// out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i, a warp a row.
template <int D>
__global__ void __launch_bounds__(256) tree_join_kernel(const TreeArgs a) {
  constexpr int N = D / 32, U = 8;
  const TreeParams& p = a.p;
  pdl_wait();
  pdl_launch_dependents();
  const TreeJoin j = a.joins[blockIdx.x];
  if (j.ntok == 0) return;
  const int lane = threadIdx.x & 31, hk = blockIdx.x % p.Hkv;
  const int row = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int s = row / kBM, in = row - s * kBM;
  const int tok = in / a.G, g = in - tok * a.G, i = s * a.TB + tok;
  if (tok >= a.TB || i >= j.ntok) return;
  float m = -INFINITY, l = 0.f, o[N] = {};
  for (int w = j.w0; w <= j.w1; w += U) {
    float2 ml[U];
    float v[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      ml[u] = make_float2(-INFINITY, 0.f);
      if (w + u > j.w1) continue;
      const int64_t task = static_cast<int64_t>(w + u) * p.Hkv + hk;
      const int64_t slot = (task * 2 + (w + u == j.w0 ? j.first : 0)) * kRows + row;
      ml[u] = a.part_ml[slot];
#pragma unroll
      for (int e = 0; e < N; ++e) v[u][e] = a.part_o[slot * D + lane + 32 * e];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (w + u > j.w1) continue;
      // a part whose scores are all NaN has no reference, but a sum: it counts
      const float n = fmaxf(m, ml[u].x), at = n == -INFINITY ? 0.f : n;
      const float f = ex2(m - at), k = ex2(ml[u].x - at);
      l = l * f + ml[u].y * k;
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = o[e] * f + v[u][e] * k;
      m = n;
    }
  }
  const int h = hk * a.G + g;
  const int64_t tokr = static_cast<int64_t>(j.q_row) + i;
  const RowEnd end = finish_row(m * kLn2, l, p.sinks ? p.sinks + h : nullptr);
  const float f = end.factor * (p.v_scale != nullptr ? __ldg(p.v_scale + hk) : 1.f);
  __nv_bfloat16* dst =
      static_cast<__nv_bfloat16*>(p.out) + tokr * p.o_t + static_cast<int64_t>(h) * p.o_h;
#pragma unroll
  for (int e = 0; e < N; ++e)
    dst[lane + 32 * e] = end.none ? __float2bfloat16_rn(0.f) : __float2bfloat16_rn(o[e] * f);
  if (p.lse != nullptr && lane == 0) p.lse[tokr * p.Hq + h] = end.lse;
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
  return launch_k(tree_join_kernel<D>, dim3(tasks, kRows / 8), dim3(256), 0, stream, a);
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
  a.min_blocks = 2;
  a.alike = p.ck_p == p.cv_p && p.ck_t == p.cv_t;
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
