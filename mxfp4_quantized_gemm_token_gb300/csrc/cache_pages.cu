// cache_pages.cu — the pages of a key/value cache: taken and freed, forked, copied, and the
// rows that stay of a sequence moved together.
//
// Pages are counted, not listed: refs[p] is the number of page-table entries that hold page
// p, and a page is free where that is 0.  A call takes the lowest free pages, in the order
// of its rows, so its result does not depend on timing; a page that a call frees is not taken
// by the same call.  The atomics here add to counts, in any order.
#include "attn.h"
#include "internal.h"

namespace mxq {

namespace {

// ------------------------------------------------------------- tables and counts
// One cluster of blocks: the steps below depend on one another over all rows and pages, a
// cluster's barrier takes a fraction of a launch, and a table and its counts are small (64K
// pages: 256 KB).  Latency-bound: chains of loads and barriers, so a step's two sums are made
// together, and what a thread finds out about its rows it leaves for itself in the workspace.
// A single block where rows, entries and pages are few.  Fork of 64 x 4 beams of ~2000 tokens: 9 us,
// of 2 x 4 beams 5.7 (a cluster 11.6, a single block for the former 20); resize 6.5 and 3.4.
constexpr int kCluster = 8;
constexpr int kTableThreads = 1024;
constexpr int kWarps = kTableThreads / 32;
constexpr int kChildren = 4096;       // old rows whose children are counted in shared memory

template <int C>
__device__ __forceinline__ void all_sync() {
  if constexpr (C == 1)
    __syncthreads();
  else
    asm volatile(
        "barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::
            : "memory");
}

// a 64-bit value of the same variable in block `rank` of the cluster
__device__ __forceinline__ unsigned long long of_block(const unsigned long long* at, int rank) {
  uint32_t there;
  unsigned long long v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(smem_u32(at)), "r"(rank));
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(there) : "memory");
  return v;
}

// Two sums over all threads in their order: what comes before this thread, and all.  Every
// thread calls it, once a kernel; a barrier has to follow before its block ends.
struct Sums {
  unsigned long long before[2], total[2];
};
template <int C>
__device__ __forceinline__ Sums scan_all(unsigned long long first, unsigned long long second) {
  __shared__ unsigned long long warp_sums[2][kWarps], block_sums[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long incl[2] = {first, second};
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, incl[k], o);
      if (lane >= o) incl[k] += y;
    }
  if (lane == 31) warp_sums[0][warp] = incl[0], warp_sums[1][warp] = incl[1];
  __syncthreads();
  Sums r;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const unsigned long long w = warp_sums[k][lane];
    unsigned long long winc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, winc, o);
      if (lane >= o) winc += y;
    }
    r.total[k] = __shfl_sync(0xffffffffu, winc, 31);
    r.before[k] = __shfl_sync(0xffffffffu, winc - w, warp) + incl[k] - (k == 0 ? first : second);
  }
  if constexpr (C > 1) {
    if (threadIdx.x == 0) block_sums[0] = r.total[0], block_sums[1] = r.total[1];
    all_sync<C>();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const unsigned long long other = lane < C ? of_block(&block_sums[k], lane) : 0;
      unsigned long long oinc = other;
#pragma unroll
      for (int o = 1; o < C; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, oinc, o);
        if (lane >= o) oinc += y;
      }
      r.total[k] = __shfl_sync(0xffffffffu, oinc, C - 1);
      r.before[k] += __shfl_sync(0xffffffffu, oinc - other, static_cast<int>(blockIdx.x));
    }
  }
  return r;
}

// Rows or pages of a thread, adjacent ones
template <int C>
struct Span {
  int64_t from, to;
  __device__ __forceinline__ Span(int64_t n, int unit) {
    constexpr int64_t all = static_cast<int64_t>(C) * kTableThreads;
    const int64_t each = n <= all * unit ? unit : (n + all * unit - 1) / (all * unit) * unit;
    const int64_t me = static_cast<int64_t>(blockIdx.x) * kTableThreads + threadIdx.x;
    from = min(n, me * each);
    to = min(n, from + each);
  }
};

__device__ __forceinline__ int pages_of(int len, int page_size) {
  return static_cast<int>((static_cast<uint32_t>(len) + static_cast<uint32_t>(page_size) - 1) /
                          static_cast<uint32_t>(page_size));
}

// a length inside the table's width (at most 2^30 keys)
__device__ __forceinline__ int clamp_len(const PagesParams& p, int len, bool* bad) {
  const int most = static_cast<int>(p.max_pages) * p.page_size;
  if (len < 0 || len > most) *bad = true;
  return max(0, min(len, most));
}

__device__ __forceinline__ int count_free(const PagesParams& p, int64_t from, int64_t to) {
  int n = 0;
  int64_t i = from;
#pragma unroll 4
  for (; i + 4 <= to; i += 4) {
    // (a span begins at a multiple of four pages; the counts at 16 bytes)
    const int4 r = *reinterpret_cast<const int4*>(p.refs + i);
    n += (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
  }
  for (; i < to; ++i) n += p.refs[i] == 0;
  return n;
}
// The first `need` free pages, ascending, into fresh[]; their counts become 1.  `before`: free
// pages of the threads before this one.
__device__ __forceinline__ void take_free(const PagesParams& p, int64_t from, int64_t to,
                                          unsigned long long before, unsigned long long need) {
  for (int64_t i = from; i < to && before < need; ++i)
    if (p.refs[i] == 0) {
      p.fresh[before++] = static_cast<int>(i);
      p.refs[i] = 1;
    }
}

// a count changed by n; one that falls below 0 was wrong before
__device__ __forceinline__ void add_ref(const PagesParams& p, int page, int n, bool* bad) {
  if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.pages)) {
    if (page >= 0) *bad = true;
    return;
  }
  if (n != 0 && atomicAdd(p.refs + page, n) + n < 0) *bad = true;
}

template <int C>
__device__ __forceinline__ void resize(const PagesParams& p) {
  pdl_wait();
  pdl_launch_dependents();
  bool bad = false;
  // pages that each row takes
  const Span<C> rows(p.B, 1), pages(p.pages, 4);
  unsigned long long need = 0;
  for (int64_t b = rows.from; b < rows.to; ++b) {
    const int more = max(0, pages_of(clamp_len(p, p.new_lens[b], &bad), p.page_size) -
                                pages_of(clamp_len(p, p.lens[b], &bad), p.page_size));
    p.row_begin[b] = more;
    need += more;
  }
  const Sums sums = scan_all<C>(need, count_free(p, pages.from, pages.to));
  unsigned long long at = sums.before[0];
  for (int64_t b = rows.from; b < rows.to; ++b) {
    const int64_t more = p.row_begin[b];
    p.row_begin[b] = static_cast<int64_t>(at);
    at += more;
  }
  take_free(p, pages.from, pages.to, sums.before[1], sums.total[0]);
  all_sync<C>();
  const int lane = threadIdx.x & 31;
  const int64_t have = static_cast<int64_t>(sums.total[1]);
  for (int64_t b = blockIdx.x * kWarps + (threadIdx.x >> 5); b < p.B; b += C * kWarps) {
    int* row = p.table + b * p.ld;
    const int len = clamp_len(p, p.new_lens[b], &bad);
    const int n0 = pages_of(clamp_len(p, p.lens[b], &bad), p.page_size);
    const int n1 = pages_of(len, p.page_size);
    const int64_t first = p.row_begin[b];
    for (int i = n0 + lane; i < n1; i += 32) {
      const int64_t k = first + i - n0;
      row[i] = k < have ? p.fresh[k] : -1;
      if (k >= have) bad = true;
    }
    auto drop = [&](int i) {
      add_ref(p, row[i], -1, &bad);
      row[i] = -1;
    };
    for (int i = n1 + lane; i < n0; i += 32) drop(i);
    if (p.window > 0) {
      // pages that end before the window and begin behind the first keys
      const int from = pages_of(p.first, p.page_size);
      const int to = min(min(n0, n1), max(0, len - p.window) / p.page_size);
      for (int i = from + lane; i < to; i += 32)
        if (row[i] != -1) drop(i);
    }
  }
  if (bad) atomicOr(p.status, kStatusBadIndex);
}

template <int C>
__device__ __forceinline__ void fork(const PagesParams& p) {
  __shared__ int near_children[kChildren], near_first[kChildren];
  const bool near = p.B <= kChildren;      // each block counts all children for itself
  int* children = near ? near_children : p.children;
  int* first_child = near ? near_first : p.first_child;
  const int lane = threadIdx.x & 31;
  const int warp = blockIdx.x * kWarps + (threadIdx.x >> 5);
  pdl_wait();
  pdl_launch_dependents();
  bool bad = false;
  const Span<C> rows(p.n, 1), pages(p.pages, 4);
  // children of every old row, and the first of them
  const int64_t me = near ? threadIdx.x : static_cast<int64_t>(blockIdx.x) * kTableThreads + threadIdx.x;
  const int64_t step = near ? kTableThreads : C * kTableThreads;
  for (int64_t r = me; r < p.B; r += step) children[r] = 0, first_child[r] = 0x7fffffff;
  auto parent_of = [&](int64_t b) {
    const int r = p.parents[b];
    if (r < -1 || r >= p.B) bad = true;
    return r >= 0 && r < p.B ? r : -1;
  };
  if (near)
    __syncthreads();
  else
    all_sync<C>();
  for (int64_t b = me; b < p.n; b += step) {
    const int r = parent_of(b);
    if (r < 0) continue;
    atomicAdd(children + r, 1);
    atomicMin(first_child + r, static_cast<int>(b));
  }
  if (near)
    __syncthreads();
  else
    all_sync<C>();
  // Rows whose open page (the one that the next key goes to) has to be a page of their own
  unsigned long long need = 0;
  for (int64_t b = rows.from; b < rows.to; ++b) {
    const int r = parent_of(b), len = r < 0 ? 0 : clamp_len(p, p.lens[r], &bad);
    bool wants = false;
    if (len % p.page_size != 0) {
      const int page = p.table[r * p.ld + len / p.page_size];
      wants = static_cast<uint32_t>(page) < static_cast<uint32_t>(p.pages) &&
              (p.refs[page] != 1 || first_child[r] != b);
    }
    need += wants;
    p.row_begin[b] = wants ? 0 : -1;
    p.new_lens_out[b] = len;
  }
  const Sums sums = scan_all<C>(need, count_free(p, pages.from, pages.to));
  unsigned long long at = sums.before[0];
  // (-1: the row keeps its parent's pages as they are)
  for (int64_t b = rows.from; b < rows.to; ++b)
    if (p.row_begin[b] == 0) p.row_begin[b] = static_cast<int64_t>(at++);
  // (every row has seen its open page's count: the sums' barrier lies behind that)
  take_free(p, pages.from, pages.to, sums.before[1], sums.total[0]);
  all_sync<C>();
  const int64_t have = static_cast<int64_t>(sums.total[1]);
  for (int64_t b = warp; b < p.n; b += C * kWarps) {
    const int r = parent_of(b), len = p.new_lens_out[b];
    const int n = pages_of(len, p.page_size);
    const int64_t k = p.row_begin[b];
    const int* from = p.table + static_cast<int64_t>(max(r, 0)) * p.ld;
    int* to = p.new_table + b * p.ld_new;
    for (int64_t i = lane; i < p.max_pages; i += 32) {
      int page = i < n ? from[i] : -1;
      if (i == n - 1 && k >= 0) {
        const int src = page;
        page = k < have ? p.fresh[k] : -1;
        if (k >= have) bad = true;
        p.copies[3 * b] = k < have ? src : -1;
        p.copies[3 * b + 1] = page;
        p.copies[3 * b + 2] = k < have ? len % p.page_size : 0;
      }
      to[i] = page;
    }
    if (k < 0 && lane < 3) p.copies[3 * b + lane] = lane < 2 ? -1 : 0;
  }
  // a row's pages are held by its children instead of by itself; its open page by the first
  // child at most
  for (int64_t r = warp; r < p.B; r += C * kWarps) {
    const int len = clamp_len(p, p.lens[r], &bad);
    const int n = pages_of(len, p.page_size), full = len / p.page_size;
    const int more = children[r] - 1;
    const int* row = p.table + r * p.ld;
    if (more != 0)
      for (int i = lane; i < full; i += 32) add_ref(p, row[i], more, &bad);
    if (full < n && lane == 0) {
      const bool kept = more >= 0 && p.row_begin[first_child[r]] < 0;
      if (!kept) add_ref(p, row[full], -1, &bad);
    }
  }
  if (bad) atomicOr(p.status, kStatusBadIndex);
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kTableThreads)
    resize_kernel(const PagesParams p) {
  resize<kCluster>(p);
}
__global__ void __launch_bounds__(kTableThreads) resize_small_kernel(const PagesParams p) {
  resize<1>(p);
}
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kTableThreads)
    fork_kernel(const PagesParams p) {
  fork<kCluster>(p);
}
__global__ void __launch_bounds__(kTableThreads) fork_small_kernel(const PagesParams p) {
  fork<1>(p);
}

// ------------------------------------------------------------------- moving rows
// A token's keys (or values) are `cols` pieces of 16 bytes: head h = col / per_head.
constexpr int kMoveThreads = 256;
constexpr int kDepth = 8;             // loads in flight a thread
constexpr int kCopyBlocks = 8;        // blocks an SM, at least, where pages are long enough
constexpr int kMinWidth = 2;          // columns of a block, at least: a sector

struct Column {
  bool value;                         // of the values' cache
  int64_t at;                         // bytes from a token's begin
};
__device__ __forceinline__ Column column_of(const MoveParams& p, int col) {
  Column c;
  c.value = col >= p.cols;
  col -= c.value ? p.cols : 0;
  const int h = static_cast<int>(static_cast<uint32_t>(col) / static_cast<uint32_t>(p.per_head));
  c.at = h * (c.value ? p.cv_h : p.ck_h) * p.es + (col - h * p.per_head) * 16;
  return c;
}

// Pages copied: block (part of the page, pair).  A thread keeps its column, of the keys or of the
// values, and takes tokens, eight on their way.  HBM-bound where there are many (the places by a
// division a piece: 83 open pages of 2713 tokens 9.6 us, now 6.2; 1000 whole pages 78 us, a copy's rate).
__global__ void __launch_bounds__(kMoveThreads) copy_pages_kernel(const MoveParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t pair = static_cast<int64_t>(blockIdx.y) + static_cast<int64_t>(blockIdx.z) * 65535;
  if (pair >= p.n) return;
  const int src = p.copies[3 * pair], dst = p.copies[3 * pair + 1];
  const int tokens = p.copies[3 * pair + 2];
  if (src < 0 || dst < 0 || tokens <= 0) return;
  const int count = min(tokens, p.page_size);
  const bool bad = src >= p.pages || dst >= p.pages;
  if ((bad || tokens > p.page_size) && blockIdx.x == 0 && threadIdx.x == 0)
    atomicOr(p.status, kStatusBadIndex);
  if (bad) return;
  const int rows = kMoveThreads / p.width;            // at once
  const int r0 = blockIdx.x * rows + threadIdx.x / p.width, step = gridDim.x * rows;
  for (int col = threadIdx.x % p.width; col < 2 * p.cols; col += p.width) {
    const Column c = column_of(p, col);
    char* base = static_cast<char*>(c.value ? p.v_cache : p.k_cache) + c.at;
    const int64_t sp = (c.value ? p.cv_p : p.ck_p) * p.es, st = (c.value ? p.cv_t : p.ck_t) * p.es;
    const char* from = base + src * sp;
    char* to = base + dst * sp;
    for (int64_t t0 = r0; t0 < count; t0 += static_cast<int64_t>(step) * kDepth) {
      uint4 v[kDepth];
#pragma unroll
      for (int u = 0; u < kDepth; ++u) {
        const int64_t t = t0 + static_cast<int64_t>(u) * step;
        if (t < count) v[u] = *reinterpret_cast<const uint4*>(from + t * st);
      }
#pragma unroll
      for (int u = 0; u < kDepth; ++u) {
        const int64_t t = t0 + static_cast<int64_t>(u) * step;
        if (t < count) *reinterpret_cast<uint4*>(to + t * st) = v[u];
      }
    }
  }
}

// Rows moved together, in place: row start + kept[i] becomes row start + i.  A block owns
// `width` columns of a sequence and takes its rows in turn, kDepth x 256 / width at a time:
// all are read before any is written.  As kept[i] >= i, what is read later lies behind all
// that is written, so no block waits for another, and a long list of few sequences
// is shared out by columns (down to 32 bytes).  HBM-bound where it is long: 4096 of
// 9000-16384 keys of 8 sequences, 8 heads of 128, 52 us (78 % of a copy's rate), half of the keys of
// one sequence of 16384 29 us (34 %: 32 bytes of each row a block).
// kFind: rows of a step a thread, at most (1 where a block is 8 columns wide or more: registers
// for two blocks an SM).
template <int kFind>
__global__ void __launch_bounds__(kMoveThreads, kFind == 1 ? 2 : 1)
    compact_kernel(const MoveParams p) {
  extern __shared__ int2 places[];    // [3] of a step's rows: from, then to (page, row of it)
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.y;
  const int rows = kMoveThreads / p.width;            // at once
  const int step = rows * kDepth;
  const int col = blockIdx.x * p.width + threadIdx.x % p.width, r0 = threadIdx.x / p.width;
  const bool mine = col < 2 * p.cols;
  const Column c = column_of(p, mine ? col : 0);
  char* base = static_cast<char*>(c.value ? p.v_cache : p.k_cache) + c.at;
  const int64_t sp = (c.value ? p.cv_p : p.ck_p) * p.es, st = (c.value ? p.cv_t : p.ck_t) * p.es;
  const int start = p.starts[b], given = p.counts[b];
  const int count = max(0, min(given, static_cast<int>(p.most)));
  const int64_t slots = p.max_pages * p.page_size;
  bool bad = given != count || start < 0;
  const int* kept = p.kept + b * p.ld_kept;
  const int* table = p.table + b * p.ld;
  // a key's page (not looked at here: it would be waited for) and its row of it; row -1: none
  auto place = [&](int64_t key) {
    if (key >= slots) {
      bad = true;
      return make_int2(0, -1);
    }
    const uint32_t k = static_cast<uint32_t>(key), s = static_cast<uint32_t>(p.page_size);
    const uint32_t n = k / s;
    return make_int2(table[n], static_cast<int>(k - n * s));
  };
  auto there = [&](int2 at) {
    if (at.y < 0) return false;
    const bool ok = static_cast<uint32_t>(at.x) < static_cast<uint32_t>(p.pages);
    if (!ok) bad = true;
    return ok;
  };
  // Where the rows of a step come from and go to is found a step ahead, in one of three tables
  // (one is being read by the stores of the step before), and the list is read two ahead.
  int listed[kFind];
  auto read_list = [&](int i0) {
#pragma unroll
    for (int f = 0; f < kFind; ++f) {
      const int i = threadIdx.x + f * kMoveThreads;
      if (i < min(step, count - i0)) listed[f] = kept[i0 + i];
    }
  };
  auto find = [&](int i0, int which) {
    int2* from = places + which * 2 * step;
    int2 a[kFind], b[kFind];
#pragma unroll
    for (int f = 0; f < kFind; ++f) {
      const int i = threadIdx.x + f * kMoveThreads;
      a[f] = b[f] = make_int2(0, -1);
      if (i >= min(step, count - i0)) continue;
      const int k = listed[f];
      if (k < i0 + i) {
        bad = true;                   // would be overwritten before it is read
      } else if (k != i0 + i) {
        a[f] = place(static_cast<int64_t>(start) + k);
        b[f] = place(static_cast<int64_t>(start) + i0 + i);
      }
    }
    read_list(i0 + step);
#pragma unroll
    for (int f = 0; f < kFind; ++f) {
      const int i = threadIdx.x + f * kMoveThreads;
      if (i < step) from[i] = a[f], from[step + i] = b[f];
    }
  };
  auto load = [&](uint4* v, int i0, int which) {
    const int2* from = places + which * 2 * step;
#pragma unroll
    for (int u = 0; u < kDepth; ++u) {
      const int i = u * rows + r0;
      if (!mine || i >= min(step, count - i0)) continue;
      const int2 at = from[i];
      if (there(at)) v[u] = *reinterpret_cast<const uint4*>(base + at.x * sp + at.y * st);
    }
  };
  auto store = [&](const uint4* v, int i0, int which) {
    const int2* from = places + which * 2 * step;
#pragma unroll
    for (int u = 0; u < kDepth; ++u) {
      const int i = u * rows + r0;
      if (!mine || i >= min(step, count - i0)) continue;
      const int2 a = from[i], b = from[step + i];
      if (there(a) && there(b)) *reinterpret_cast<uint4*>(base + b.x * sp + b.y * st) = v[u];
    }
  };
  if (start >= 0 && count > 0) {
    uint4 v[kDepth], w[kDepth];
    read_list(0);
    find(0, 0);
    __syncthreads();
    load(v, 0, 0);
    find(step, 1);
    __syncthreads();
    // Of the step, all is read before the barrier and written behind it; the next one's rows,
    // which lie behind all that is written here, are on their way meanwhile.
    int which = 0;
    auto turn = [&](const uint4* now, uint4* next, int i0) {
      const int ahead = which == 2 ? 0 : which + 1, far = ahead == 2 ? 0 : ahead + 1;
      load(next, i0 + step, ahead);
      store(now, i0, which);
      find(i0 + 2 * step, far);
      __syncthreads();
      which = ahead;
    };
    for (int i0 = 0; i0 < count; i0 += 2 * step) {
      turn(v, w, i0);
      if (i0 + step < count) turn(w, v, i0 + step);
    }
  }
  if (bad) atomicOr(p.status, kStatusBadIndex);
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

// [rows] begins, [pages] fresh pages, [rows] children, [rows] first children
size_t pages_workspace_bytes(int64_t rows, int64_t pages) {
  return round256(rows * 8) + round256(pages * 4) + 2 * round256(rows * 4);
}

namespace {
void spread(PagesParams* p, int64_t rows) {
  char* ws = static_cast<char*>(p->workspace);
  p->row_begin = reinterpret_cast<int64_t*>(ws);
  ws += round256(rows * 8);
  p->fresh = reinterpret_cast<int*>(ws);
  ws += round256(p->pages * 4);
  p->children = reinterpret_cast<int*>(ws);
  p->first_child = reinterpret_cast<int*>(ws + round256(rows * 4));
}
}  // namespace

// One block: rows of a warp each and pages of a few loads
static bool small(const PagesParams& p, int64_t rows) {
  return rows <= 64 && p.max_pages <= 1024 && p.pages <= 16384;
}

cudaError_t launch_resize_pages(const PagesParams& given, cudaStream_t stream) {
  PagesParams p = given;
  spread(&p, p.B);
  return small(p, p.B)
             ? launch_k(resize_small_kernel, dim3(1), dim3(kTableThreads), 0, stream, p)
             : launch_k(resize_kernel, dim3(kCluster), dim3(kTableThreads), 0, stream, p);
}

cudaError_t launch_fork_pages(const PagesParams& given, cudaStream_t stream) {
  PagesParams p = given;
  const int64_t rows = p.n > p.B ? p.n : p.B;
  spread(&p, rows);
  return small(p, rows) ? launch_k(fork_small_kernel, dim3(1), dim3(kTableThreads), 0, stream, p)
                        : launch_k(fork_kernel, dim3(kCluster), dim3(kTableThreads), 0, stream, p);
}

cudaError_t launch_copy_pages(const MoveParams& given, int num_sms, cudaStream_t stream) {
  MoveParams p = given;
  p.width = 2;
  while (p.width < kMoveThreads && p.width < 2 * p.cols) p.width *= 2;
  // parts of a page: enough blocks for the SMs, none with less than a pass
  const int64_t pass = static_cast<int64_t>(kMoveThreads / p.width) * kDepth;
  const int64_t passes = (p.page_size + pass - 1) / pass;
  int64_t parts = (kCopyBlocks * static_cast<int64_t>(num_sms) + p.n - 1) / p.n;
  if (parts > passes) parts = passes;
  const int64_t y = p.n < 65535 ? p.n : 65535, z = (p.n + 65534) / 65535;
  return launch_k(copy_pages_kernel,
                  dim3(static_cast<unsigned>(parts), static_cast<unsigned>(y),
                       static_cast<unsigned>(z)),
                  dim3(kMoveThreads), 0, stream, p);
}

cudaError_t launch_compact(const MoveParams& given, int num_sms, cudaStream_t stream) {
  MoveParams p = given;
  // as wide as the longest list allows in one step, and narrower until there is a block an SM
  int width = 128;
  while (width > 2 && (static_cast<int64_t>(kMoveThreads / width) * kDepth < p.most)) width /= 2;
  auto blocks = [&](int w) { return (2 * static_cast<int64_t>(p.cols) + w - 1) / w * p.B; };
  if (width < 16) width = 16;
  while (width > kMinWidth && blocks(width) < num_sms) width /= 2;
  p.width = width;
  const size_t smem = static_cast<size_t>(kMoveThreads / width) * kDepth * 6 * sizeof(int2);
  return launch_k(width >= kDepth ? compact_kernel<1> : compact_kernel<kDepth / kMinWidth>,
                  dim3(static_cast<unsigned>(blocks(width) / p.B), static_cast<unsigned>(p.B)),
                  dim3(kMoveThreads), smem, stream, p);
}

}  // namespace mxq
