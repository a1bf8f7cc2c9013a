// The pages of the cache: pka_copy_pages, pka_alloc_pages, pka_free_pages,
// pka_fork_pages and pka_compact_pages.
//
// The only state is page_refs, a reference count per page (0: free), so there
// is no free list to keep in step with it: the free pages are found by
// counting.  Every answer is the one of lowest page ids, whatever order the
// blocks run in.  The calls that count run as one thread-block cluster: its
// hardware barrier orders the passes over page_refs and the counts of the
// blocks meet in distributed shared memory, with no workspace and no waiting
// on flags.
#include <cooperative_groups.h>

#include <atomic>
#include <mutex>

#include "pka_cache.h"
#include "pka_internal.h"

namespace pka {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxCluster = 16;  // blocks of the largest counting launch
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kAll = 0xffffffffu;

// A call's second launch starts when the blocks of its first are all running
// (start_next) and waits (after_previous) for their end before it reads or
// writes what they write; what it does before that overlaps with them.
__device__ __forceinline__ void start_next() { cudaTriggerProgrammaticLaunchCompletion(); }
__device__ __forceinline__ void after_previous() { cudaGridDependencySynchronize(); }

// ---------------------------------------------------------------------------
// Counting
// ---------------------------------------------------------------------------

// page_refs split among the warps of the cluster, tile by tile in turn (so
// that every block has its part of the lowest pages, which a call wants
// first): row i of tiles is tiles i * warps .. i * warps + warps - 1, one a
// warp, at most kRows rows.
constexpr int kRows = 32;
constexpr uint32_t kTile = 512;  // pages; less where one row suffices, else multiples of it

struct Share {
  uint32_t lo, hi;  // the pages of this warp's tile
  int lane;
  bool vec;         // page_refs is 16-byte aligned
};

struct Tiling {
  uint32_t tile;    // pages of a tile
  int rows;
};

__device__ __forceinline__ Share tile_at(const int32_t* refs, uint32_t num_pages, const Tiling& t,
                                         int row) {
  const uint32_t warps = gridDim.x * kWarps;
  const uint64_t lo =
      (uint64_t)(row * warps + blockIdx.x * kWarps + (threadIdx.x >> 5)) * t.tile;
  Share s;
  s.lo = (uint32_t)min(lo, (uint64_t)num_pages);
  s.hi = (uint32_t)min(lo + t.tile, (uint64_t)num_pages);
  s.lane = threadIdx.x & 31;
  s.vec = (reinterpret_cast<uintptr_t>(refs) & 15) == 0;
  return s;
}

// References of pages p .. p+3 (those past `hi` come as `past`).
__device__ __forceinline__ int4 refs_at(const int32_t* refs, const Share& s, uint32_t p, int past) {
  if (s.vec && p + 4 <= s.hi) return *reinterpret_cast<const int4*>(refs + p);
  int4 r;
  r.x = p < s.hi ? refs[p] : past;
  r.y = p + 1 < s.hi ? refs[p + 1] : past;
  r.z = p + 2 < s.hi ? refs[p + 2] : past;
  r.w = p + 3 < s.hi ? refs[p + 3] : past;
  return r;
}

// Walk a tile in order, 128 pages a step, the loads of four steps in flight:
// use(p, r) with this lane's pages p .. p+3 and their references; a false
// result (of the whole warp) ends the walk.
template <class F>
__device__ __forceinline__ void walk(const int32_t* refs, const Share& s, int past, F use) {
  constexpr int U = 4;
  uint32_t p = s.lo + 4 * s.lane;
  for (uint32_t left = s.hi - s.lo; left > 0; left -= min(left, 128u * U), p += 128 * U) {
    int4 r[U];
    if (s.vec && left >= 128 * U) {
#pragma unroll
      for (int i = 0; i < U; ++i) r[i] = *reinterpret_cast<const int4*>(refs + p + 128 * i);
    } else {
#pragma unroll
      for (int i = 0; i < U; ++i) r[i] = refs_at(refs, s, p + 128 * i, past);
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (128u * i < left && !use(p + 128 * i, r[i])) return;
  }
}

// Bit k: page p + k is free (has no reference); pages past the tile are not.
__device__ __forceinline__ unsigned free_bits(const int4& r) {
  return (r.x <= 0 ? 1u : 0u) | (r.y <= 0 ? 2u : 0u) | (r.z <= 0 ? 4u : 0u) |
         (r.w <= 0 ? 8u : 0u);
}

__device__ __forceinline__ int count_free(const int32_t* refs, const Share& s) {
  int n = 0;
  walk(refs, s, 1, [&](uint32_t, const int4& r) {
    n += (r.x <= 0) + (r.y <= 0) + (r.z <= 0) + (r.w <= 0);
    return true;
  });
  return __reduce_add_sync(kAll, n);
}

// Of the set bits of a step's lanes, taken lane by lane: how many come before
// this lane's first, and how many there are.  A lane has 0 to 4; three ballots
// carry the binary digits.
__device__ __forceinline__ void rank_bits(unsigned bits, int lane, int* before, int* all) {
  const unsigned below = (1u << lane) - 1;
  const int n = __popc(bits);
  const unsigned b0 = __ballot_sync(kAll, n & 1), b1 = __ballot_sync(kAll, n & 2),
                 b2 = __ballot_sync(kAll, n & 4);
  *before = __popc(b0 & below) + 2 * __popc(b1 & below) + 4 * __popc(b2 & below);
  *all = __popc(b0) + 2 * __popc(b1) + 4 * __popc(b2);
}

__device__ __forceinline__ int inclusive_sum(int x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(kAll, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

struct Counts {
  int tile[kRows][kWarps];  // pages counted in a tile; then in the block's tiles before it
  int block[kRows];         // in the block's tiles of a row
  int before[kRows];        // in the row's tiles of the blocks before
  int row[kRows];           // in a row
  int flag;                 // FLAG: set by the block before it counts
  int any_flag;             // FLAG: set by any block of the cluster
};

// Counts the free (or live) pages of this warp's tiles.
__device__ __forceinline__ void count_tiles(Counts& c, const int32_t* refs, uint32_t num_pages,
                                            const Tiling& t, bool live) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = 0; i < t.rows; ++i) {
    const Share s = tile_at(refs, num_pages, t, i);
    const int n = count_free(refs, s);
    if (lane == 0) c.tile[i][warp] = live ? (int)(s.hi - s.lo) - n : n;
  }
}

// Adds up what count_tiles counted.  Lane i gets the number of such pages
// before this warp's tile of row i, and every lane their total.  Leaves the
// cluster barrier armed: the caller ends with leave(), so that no block is gone
// while its counts are read.  FLAG: c.any_flag, which the caller set to its own
// c.flag, becomes that of any block.
template <bool FLAG>
__device__ __forceinline__ int add_counts(Counts& c, const Tiling& t, int* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();
  int block = 0;
  if (warp < t.rows) {  // a warp a row
    const int n = c.tile[warp][lane], upto = inclusive_sum(n, lane);
    c.tile[warp][lane] = upto - n;
    block = __shfl_sync(kAll, upto, 31);
    if (lane == 0) {
      c.block[warp] = c.row[warp] = block;
      c.before[warp] = 0;
    }
  }
  if (gridDim.x > 1) {
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    if (warp < t.rows) {
      const int there = lane < gridDim.x ? cluster.map_shared_rank(&c, lane)->block[warp] : 0;
      const int row = __reduce_add_sync(kAll, there);
      const int before = __reduce_add_sync(kAll, lane < blockIdx.x ? there : 0);
      if (lane == 0) {
        c.row[warp] = row;
        c.before[warp] = before;
      }
    }
    if (FLAG && warp == 0) {
      const int there = lane < gridDim.x ? cluster.map_shared_rank(&c, lane)->flag : 0;
      const bool any = __any_sync(kAll, there != 0);
      if (lane == 0) c.any_flag = any;
    }
    cluster.barrier_arrive();
  }
  __syncthreads();
  const int row = lane < t.rows ? c.row[lane] : 0;
  const int upto = inclusive_sum(row, lane);
  *total = __shfl_sync(kAll, upto, 31);
  return lane < t.rows ? upto - row + c.before[lane] + c.tile[lane][warp] : 0;
}

__device__ __forceinline__ int count_pages(Counts& c, const int32_t* refs, uint32_t num_pages,
                                           const Tiling& t, bool live, int* total) {
  count_tiles(c, refs, num_pages, t, live);
  return add_counts<false>(c, t, total);
}

__device__ __forceinline__ void leave() {
  if (gridDim.x > 1) cg::this_cluster().barrier_wait();
}

// Take the free ones (`bits`) of a step's pages, the first with rank *rank, as
// long as ranks stay below `stop`: use(rank, page) and one reference each.
// False when there is nothing left to take.  ALONE: nobody else changes a
// reference meanwhile, so a lane stores its four pages at once.
template <bool ALONE, class F>
__device__ __forceinline__ bool take_step(int32_t* refs, const Share& s, uint32_t p, const int4& r,
                                          unsigned bits, int* rank, int stop, F use) {
  int first, all;
  rank_bits(bits, s.lane, &first, &all);
  first += *rank;
  unsigned taken = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int at = first + __popc(bits & ((1u << k) - 1));
    if ((bits >> k & 1) && at < stop) {
      use(at, (int32_t)(p + k));
      taken |= 1u << k;
    }
  }
  if (taken) {
    if (ALONE && s.vec && p + 4 <= s.hi) {
      *reinterpret_cast<int4*>(refs + p) =
          make_int4(taken & 1 ? 1 : r.x, taken & 2 ? 1 : r.y, taken & 4 ? 1 : r.z,
                    taken & 8 ? 1 : r.w);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (taken >> k & 1) refs[p + k] = 1;
    }
  }
  *rank += all;
  return *rank < stop;
}

// Take the first `stop` free pages of all: use(rank, page) for those of this
// warp's tiles.  `before` is add_counts' answer.
template <bool ALONE, class F>
__device__ __forceinline__ void take_free(int32_t* refs, uint32_t num_pages, const Tiling& t,
                                          int before, int stop, F use) {
  for (int i = 0; i < t.rows; ++i) {
    int rank = __shfl_sync(kAll, before, i);
    if (rank >= stop) return;
    const Share s = tile_at(refs, num_pages, t, i);
    walk(refs, s, 1, [&](uint32_t p, const int4& r) {
      return take_step<ALONE>(refs, s, p, r, free_bits(r), &rank, stop, use);
    });
  }
}

// ---------------------------------------------------------------------------
// Taking and returning pages
// ---------------------------------------------------------------------------

struct AllocArgs {
  int32_t* refs;
  int32_t* pages;
  int32_t* err;
  int32_t num_pages, n;
  Tiling tiling;
};

// More pages than these, in a pool of more than a row of tiles, are taken by a
// launch of their own.  Taken from 1,500,007 pages and returned, in us, in
// place / in a second launch: 8,192 pages 11.4 / 11.9, 32,768 11.6 / 12.1,
// 131,072 17.4 / 15.0.
constexpr int kTakeInPlace = 65536;

// SPLIT: the taking is left to take_kernel, over the whole GPU.  Each tile's
// count before it travels in the tile's first free page, whose reference count
// holds -1 - count until that page, the first of its tile to be taken, gets
// its reference; tiles that give nothing stay as they are.
template <bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) alloc_kernel(const AllocArgs a) {
  __shared__ Counts c;
  if (SPLIT) start_next();
  int total;
  const int before = count_pages(c, a.refs, a.num_pages, a.tiling, false, &total);
  if (total < a.n) {
    for (int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x; i < a.n;
         i += (int64_t)gridDim.x * kThreads)
      a.pages[i] = -1;
    if (blockIdx.x == 0 && threadIdx.x == 0) note_error(a.err, PKA_ERR_WORKSPACE);
  } else if (!SPLIT) {
    take_free<true>(a.refs, a.num_pages, a.tiling, before, a.n, [&](int rank, int32_t page) {
      a.pages[rank] = page;
    });
  } else {
    for (int i = 0; i < a.tiling.rows; ++i) {
      const int rank = __shfl_sync(kAll, before, i);
      if (rank >= a.n) break;
      const Share s = tile_at(a.refs, a.num_pages, a.tiling, i);
      walk(a.refs, s, 1, [&](uint32_t p, const int4& r) {
        const unsigned bits = free_bits(r), lanes = __ballot_sync(kAll, bits != 0);
        if (lanes && s.lane == __ffs(lanes) - 1) a.refs[p + __ffs(bits) - 1] = -1 - rank;
        return lanes == 0;
      });
    }
  }
  leave();
}

// A warp a tile: the first free page carries the tile's first rank, or 0 in a
// tile that gives nothing.
__global__ void __launch_bounds__(256) take_kernel(const AllocArgs a) {
  const uint64_t lo = (blockIdx.x * 8ull + (threadIdx.x >> 5)) * a.tiling.tile;
  after_previous();
  if (lo >= (uint64_t)a.num_pages) return;
  Share s;
  s.lo = (uint32_t)lo;
  s.hi = (uint32_t)min(lo + a.tiling.tile, (uint64_t)a.num_pages);
  s.lane = threadIdx.x & 31;
  s.vec = (reinterpret_cast<uintptr_t>(a.refs) & 15) == 0;
  int rank = -1;  // not met the first free page yet
  walk(a.refs, s, 1, [&](uint32_t p, const int4& r) {
    const unsigned bits = free_bits(r);
    if (rank < 0) {
      const unsigned lanes = __ballot_sync(kAll, bits != 0);
      if (!lanes) return true;
      const int k = __ffs(bits) - 1;
      const int mark = k == 0 ? r.x : k == 1 ? r.y : k == 2 ? r.z : r.w;
      rank = -1 - __shfl_sync(kAll, mark, __ffs(lanes) - 1);
      if (rank < 0) return false;
    }
    return take_step<true>(a.refs, s, p, r, bits, &rank, a.n, [&](int at, int32_t page) {
      a.pages[at] = page;
    });
  });
}

// A page's count never stays below zero: a decrement that finds none left is
// taken back and noted.  Exactly as many decrements succeed as there were
// references, in whatever order they come.  Four entries a thread, so that
// four atomics are in flight.
__global__ void __launch_bounds__(256) free_kernel(int32_t* refs, int32_t num_pages,
                                                   const int32_t* pages, int64_t n, int32_t* err) {
  constexpr int U = 4;
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  bool bad = false;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += U * step) {
    int32_t p[U], had[U];
#pragma unroll
    for (int u = 0; u < U; ++u) p[u] = i + u * step < n ? pages[i + u * step] : -1;
#pragma unroll
    for (int u = 0; u < U; ++u)
      had[u] = p[u] >= 0 && p[u] < num_pages ? atomicSub(refs + p[u], 1) : 1;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (had[u] <= 0) atomicAdd(refs + p[u], 1);
      bad = bad || had[u] <= 0 || (i + u * step < n && (p[u] < 0 || p[u] >= num_pages));
    }
  }
  if (bad) note_error(err, PKA_ERR_METADATA);
}

// ---------------------------------------------------------------------------
// Fork
// ---------------------------------------------------------------------------

struct ForkArgs {
  int32_t* refs;
  const int32_t* kv_indptr;
  const int32_t* kv_indices;
  const int32_t* last_page_len;
  const int32_t* parent;
  const int32_t* child_indptr;
  int32_t* child_indices;
  int32_t* copy_src;
  int32_t* copy_dst;
  int32_t* copy_slots;
  int32_t* counts;
  int32_t* err;
  int32_t page_size, num_pages, num_parents, num_children;
  int32_t num_indices, num_child_indices;
  Tiling tiling;
};

// What one child takes: the first `shared` entries of its parent's table,
// then fresh pages; the first of those receives the parent's partly filled
// last page, if it has one.
struct Child {
  int first;        // its first entry in child_indices
  int shared;
  int fresh;
  int parent_first; // its parent's first entry in kv_indices
  int slots;        // filled slots of the parent's partial page, or 0
  bool ok;
};

__device__ __forceinline__ Child child_at(const ForkArgs& a, int32_t c0, int32_t c1, int32_t p) {
  Child x{};
  x.first = c0;
  x.ok = c0 >= 0 && c1 >= c0 && c1 <= a.num_child_indices && p >= -1 && p < a.num_parents;
  int32_t k0 = 0, k1 = 0, last = 1;
  if (x.ok && p >= 0) {
    k0 = a.kv_indptr[p];
    k1 = a.kv_indptr[p + 1];
    last = a.last_page_len[p];
  }
  const int pages = k1 - k0;
  x.ok = x.ok && k0 >= 0 && pages >= 0 && k1 <= a.num_indices && pages <= c1 - c0 &&
         (pages == 0 || (last >= 1 && last <= a.page_size));
  if (!x.ok) return x;
  x.parent_first = k0;
  x.slots = pages > 0 && last < a.page_size ? last : 0;
  x.shared = pages - (x.slots > 0);
  x.fresh = c1 - c0 - x.shared;
  return x;
}

__device__ __forceinline__ Child child_at(const ForkArgs& a, int c) {
  return child_at(a, a.child_indptr[c], a.child_indptr[c + 1], a.parent[c]);
}

// Shared memory of fork_take_kernel, one element a child.
struct ChildSums {
  int32_t* fresh_before;   // [num_children + 1] fresh pages of the children before
  int32_t* copies_before;  // copies of the children before
  int32_t* first;          // as in Child
  int32_t* shared;
  int32_t* parent_first;
  int32_t* slots;
};

constexpr int kChildWords = 6;

__device__ __forceinline__ ChildSums child_sums(int32_t* mem, int n) {
  return {mem, mem + n + 1, mem + 2 * n + 1, mem + 3 * n + 1, mem + 4 * n + 1, mem + 5 * n + 1};
}

// The last i in [lo, hi] with ptr[i] <= x.
__device__ __forceinline__ int find_between(const int32_t* ptr, int lo, int hi, int64_t x) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (ptr[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// At most this many entries are shared by the launch that takes the fresh
// pages; more go to a launch over the whole GPU.  Fork and return, in us, in
// one / in two launches: 32 entries 7.2 / 7.6, 1,032 7.7 / 8.6, 4,004 9.9 / 9.6
// (and a launch less for the host), 16,008 9.6 / 9.6 and 64,016 14.8 / 10.5
// before the one looked for pages that nobody holds, which costs it 0.3 to 0.8.
constexpr int kShareInTake = PKA_FORK_CHECKED_INDICES;

// Checks every child, takes the lowest free pages for all of them and writes
// the entries that these fill, the copy list and the counts; nothing at all
// when a child is malformed or the pages do not suffice.  Every block of the
// cluster scans the children for itself into shared memory, then writes for
// the free pages of its share.  SHARE: the parents' pages are looked up before
// the counts meet, whose barrier then tells every block whether all are held;
// so no page is free to one block and shared by another, and the references
// that the shared entries add leave the free pages as they were counted.
template <bool SHARE>
__global__ void __launch_bounds__(kThreads, 1) fork_take_kernel(const ForkArgs a) {
  extern __shared__ int32_t mem[];
  const ChildSums sums = child_sums(mem, a.num_children);
  __shared__ Counts c;
  __shared__ int64_t warp_sum[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (!SHARE) start_next();
  // (the first round's loads go out before the counting)
  const int i0 = min((int)threadIdx.x, a.num_children - 1);
  const int32_t first = a.child_indptr[i0], end = a.child_indptr[i0 + 1], parent = a.parent[i0];
  int total = 0, before = 0;
  count_tiles(c, a.refs, a.num_pages, a.tiling, false);
  if (!SHARE) before = add_counts<false>(c, a.tiling, &total);

  // running sums over the children: fresh pages in the upper 32 bits, copies
  // in the lower
  int64_t carry = 0;
  bool ok = true;
  for (int c0 = 0; c0 < a.num_children; c0 += kThreads) {
    const int i = c0 + threadIdx.x;
    int64_t x = 0;
    if (i < a.num_children) {
      const Child ch = c0 == 0 ? child_at(a, first, end, parent) : child_at(a, i);
      ok = ok && ch.ok;
      if (ch.ok) x = ((int64_t)ch.fresh << 32) | (ch.slots > 0 ? 1 : 0);
      sums.first[i] = ch.first;
      sums.shared[i] = ch.shared;
      sums.parent_first[i] = ch.parent_first;
      sums.slots[i] = ch.slots;
    }
    int64_t incl = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(kAll, incl, d);
      if (lane >= d) incl += y;
    }
    __syncthreads();  // the previous round's warp_sum has been read
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int64_t sum = warp_sum[lane];  // and, in every warp, of the warps
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(kAll, sum, d);
      if (lane >= d) sum += y;
    }
    const int64_t base = carry + (warp > 0 ? __shfl_sync(kAll, sum, warp - 1) : 0);
    const int64_t all = carry + __shfl_sync(kAll, sum, 31);
    if (i < a.num_children) {
      const int64_t excl = base + incl - x;
      sums.fresh_before[i] = (int32_t)(excl >> 32);
      sums.copies_before[i] = (int32_t)excl;
    }
    carry = all;
  }
  ok = __syncthreads_and(ok);
  constexpr int U = kShareInTake / kThreads;
  static_assert(U * kThreads == kShareInTake, "entries of the smallest launch");
  const int e0 = sums.first[0] + blockIdx.x * kThreads + threadIdx.x;
  int32_t page_of[U];
  unsigned named = 0, shares = 0;  // bit u: entry e0 + u * (threads of the launch) names or shares
  if (SHARE) {                     // page_of[u] of its parent
    const int stop = a.child_indptr[a.num_children];  // at most kShareInTake when ok
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = e0 + u * gridDim.x * kThreads;
      if (!ok || e >= stop) break;
      const int i = find_between(sums.first, 0, a.num_children - 1, e);
      const int j = e - sums.first[i], shared = sums.shared[i];
      if (j >= shared + (sums.slots[i] > 0)) continue;
      page_of[u] = a.kv_indices[sums.parent_first[i] + j];
      named |= 1u << u;
      if (j < shared) shares |= 1u << u;
    }
    bool unheld = false;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if ((named >> u & 1) && page_of[u] >= 0 && page_of[u] < a.num_pages)
        unheld |= a.refs[page_of[u]] <= 0;
    unheld = __syncthreads_or(unheld);
    if (threadIdx.x == 0) c.flag = c.any_flag = unheld;
    before = add_counts<true>(c, a.tiling, &total);
    ok = ok && !c.any_flag;
  }
  const int64_t needed = carry >> 32;
  const int copies = (int)(uint32_t)carry;
  const bool refused = !ok || total < needed;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.counts[0] = refused ? -1 : copies;
    a.counts[1] = refused ? -1 : (int32_t)needed;
    if (refused) note_error(a.err, ok ? PKA_ERR_WORKSPACE : PKA_ERR_METADATA);
  }
  if (!refused) {
    const float per_rank = needed > 0 ? (float)a.num_children / (float)needed : 0.f;
    const auto fill = [&](int rank, int32_t page) {
      // where every child takes equally many, this is the child of that rank
      int i = min((int)(((float)rank + 0.5f) * per_rank), a.num_children - 1);
      const int upto = i + 1 < a.num_children ? sums.fresh_before[i + 1] : (int)needed;
      if (rank < sums.fresh_before[i] || rank >= upto)
        i = find_between(sums.fresh_before, 0, a.num_children - 1, rank);
      const int nth = rank - sums.fresh_before[i];
      a.child_indices[sums.first[i] + sums.shared[i] + nth] = page;
      if (nth == 0 && sums.slots[i] > 0) {
        const int to = sums.copies_before[i];
        a.copy_src[to] = a.kv_indices[sums.parent_first[i] + sums.shared[i]];
        a.copy_dst[to] = page;
        a.copy_slots[to] = sums.slots[i];
      }
    };
    take_free<!SHARE>(a.refs, a.num_pages, a.tiling, before, (int)needed, fill);
    if (SHARE) {
      bool bad = false;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!(shares >> u & 1)) continue;
        a.child_indices[e0 + u * gridDim.x * kThreads] = page_of[u];
        if (page_of[u] >= 0 && page_of[u] < a.num_pages) atomicAdd(a.refs + page_of[u], 1);
        else bad = true;
      }
      if (bad) note_error(a.err, PKA_ERR_METADATA);
    }
  }
  leave();
}

// References that an entry of child c adds.  Children of one parent share the
// same pages, so where that saves atomics (a parent of kLongTable pages or
// more; few enough children to look through) the first of its children adds
// for all of them and the others nothing (64 tables of 3,584 pages into 256 and
// back: 23.0 us against 25.7).
constexpr int kLongTable = 256, kFewChildren = 1024;

__device__ __forceinline__ int adds_of(const ForkArgs& a, int c, const Child& ch, int lane) {
  if (ch.shared < kLongTable || a.num_children > kFewChildren) return 1;
  const int32_t p = a.parent[c];
  int kids = 0, earlier = 0;
  for (int i = lane; i < a.num_children; i += 32) {
    const bool same = a.parent[i] == p;
    kids += same;
    earlier += same && i < c;
  }
  kids = __reduce_add_sync(kAll, kids);
  return __reduce_add_sync(kAll, earlier) > 0 ? 0 : kids;
}

// The shared entries of every child's table and their references.  A warp
// takes 256 entries; where they belong to one child it is looked up once, else
// each lane looks its own up between the children of the first and the last
// (of which alone may be longer than the 256).
__global__ void __launch_bounds__(256) fork_share_kernel(const ForkArgs a) {
  constexpr int U = 8, CHUNK = 32 * U;
  static_assert(CHUNK <= kLongTable, "a long table inside a chunk would be missed");
  const int lane = threadIdx.x & 31;
  bool waited = false;
  const int64_t end = a.child_indptr[a.num_children];
  bool bad = false;
  for (int64_t e0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * CHUNK; e0 < end;
       e0 += (int64_t)gridDim.x * 8 * CHUNK) {
    const int64_t e1 = min(e0 + CHUNK, end);
    const int first = warp_find(a.child_indptr, a.num_children, e0, lane);
    const bool one = first + 1 >= a.num_children || a.child_indptr[first + 1] >= e1;
    const int last = one ? first : warp_find(a.child_indptr, a.num_children, e1 - 1, lane);
    Child ch = child_at(a, first);
    const int adds_first = adds_of(a, first, ch, lane);
    const int adds_last = one ? adds_first : adds_of(a, last, child_at(a, last), lane);
    int32_t page[U];
    int adds[U];  // -1: not a shared entry
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t e = e0 + 32 * u + lane;
      int c = first;
      if (!one && e < e1) {
        c = find_between(a.child_indptr, first, last, e);
        ch = child_at(a, c);
      }
      const int64_t j = e - ch.first;
      adds[u] = -1;
      if (e < e1 && j >= 0 && j < ch.shared) {
        page[u] = a.kv_indices[ch.parent_first + j];
        adds[u] = c == first ? adds_first : c == last ? adds_last : 1;
      }
    }
    if (!waited) {  // the first chunk was read while the fresh pages were taken
      after_previous();
      if (*const_cast<volatile int32_t*>(a.counts) < 0) return;  // refused
      waited = true;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (adds[u] >= 0) {
        a.child_indices[e0 + 32 * u + lane] = page[u];
        if (page[u] < 0 || page[u] >= a.num_pages) bad = true;
        else if (adds[u] > 0) atomicAdd(a.refs + page[u], adds[u]);
      }
  }
  if (!waited) after_previous();  // no warp ends the launch before its first ended
  if (bad) note_error(a.err, PKA_ERR_METADATA);
}

// ---------------------------------------------------------------------------
// Compact
// ---------------------------------------------------------------------------

struct CompactArgs {
  const int32_t* refs;   // may be refs_out
  int32_t* refs_out;
  int32_t* map;
  int32_t* copy_src;
  int32_t* copy_dst;
  int32_t* counts;
  const int32_t* in;     // table entries; may be out
  int32_t* out;
  int32_t* err;
  int64_t num_indices;
  int32_t num_pages;
  Tiling tiling;
};

// With L live pages, the live pages at L and above move to the free pages
// below L: as many of the one as of the other.  Before page p lie r(p) live
// pages (one pass of counting), so the free page p < L is number p - r(p) of
// its kind from below and the live page p >= L number L - 1 - r(p) of its kind
// from above; equal numbers pair up.  number_tile writes the two lists by
// those numbers; a moving page's entry of the map holds -2 - number until
// move_kernel, which needs both lists whole, turns it into the new id.  `rank`
// is r of the tile's first page, `live` is L.
__device__ __forceinline__ void number_tile(const CompactArgs& a, const Share& s, int rank,
                                            int live) {
  const bool apart = a.refs != a.refs_out;
  const bool vec_map = (reinterpret_cast<uintptr_t>(a.map) & 15) == 0;
  const bool vec_out = (reinterpret_cast<uintptr_t>(a.refs_out) & 15) == 0;
  walk(a.refs, s, 0, [&](uint32_t p, const int4& r4) {
    const int r[4] = {r4.x, r4.y, r4.z, r4.w};
    const unsigned bits = ~free_bits(r4) & 15u;  // live
    int at, all;
    rank_bits(bits, s.lane, &at, &all);
    at += rank;
    int m[4], o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int32_t page = (int32_t)(p + k);
      const bool held = bits >> k & 1;
      m[k] = !held ? -1 : page < live ? page : -2 - (live - 1 - at);
      o[k] = page < live ? max(r[k], 0) : 0;  // a free page below L: its mover's, later
      if (p + k < s.hi) {
        if (page == live) {
          a.counts[0] = live - at;
          a.counts[1] = live;
        }
        if (!held && page < live) a.copy_dst[page - at] = page;
        if (held && page >= live) a.copy_src[live - 1 - at] = page;
      }
      at += held;
    }
    rank += all;
    if (vec_map && p + 4 <= s.hi) {
      *reinterpret_cast<int4*>(a.map + p) = make_int4(m[0], m[1], m[2], m[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (p + k < s.hi) a.map[p + k] = m[k];
    }
    if (apart && vec_out && p + 4 <= s.hi) {
      *reinterpret_cast<int4*>(a.refs_out + p) = make_int4(o[0], o[1], o[2], o[3]);
    } else if (apart) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (p + k < s.hi) a.refs_out[p + k] = o[k];
    }
    return true;
  });
}

// The moves' references and map entries, and the table entries through the
// map.  An entry whose page moves reads its map entry before or after it is
// turned; either gives the new id.  An entry that names no live page stays as
// it is and is noted.  (In the first launch, for one block and a small table,
// this took as long: 5.6 us against 3.2 + 2.7.)
__global__ void __launch_bounds__(256) move_kernel(const CompactArgs a) {
  after_previous();
  const int64_t at = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  bool bad = false;
  for (int64_t i = at; i < a.num_indices; i += step) {
    const int32_t p = a.in[i];
    int32_t to = -1;
    if (p >= 0 && p < a.num_pages) {
      to = *const_cast<volatile int32_t*>(a.map + p);
      if (to < -1) to = a.copy_dst[-2 - to];
    }
    bad = bad || to < 0;
    a.out[i] = to < 0 ? p : to;
  }
  const int moves = a.counts[0];
  for (int64_t i = at; i < moves; i += step) {
    const int32_t src = a.copy_src[i], dst = a.copy_dst[i];
    a.refs_out[dst] = a.refs[src];
    if (a.refs == a.refs_out) a.refs_out[src] = 0;
    *const_cast<volatile int32_t*>(a.map + src) = dst;
  }
  if (bad) note_error(a.err, PKA_ERR_METADATA);
}

// One row of tiles is numbered where it was counted.  More are too much for
// the cluster's few blocks: they go to number_kernel, each tile's count before
// it in the map entry of its first page (which that tile alone reads and
// overwrites) and L in counts[1].  500,009 pages: 14.4 us in this launch, 9.8
// in the two, which overlap with the next.
__global__ void __launch_bounds__(kThreads, 1) compact_kernel(const CompactArgs a) {
  __shared__ Counts c;
  start_next();
  int live;
  const int before = count_pages(c, a.refs, a.num_pages, a.tiling, true, &live);
  if (blockIdx.x == 0 && threadIdx.x == 0 && (a.tiling.rows > 1 || live == a.num_pages)) {
    a.counts[0] = 0;  // unless a page has the number L
    a.counts[1] = live;
  }
  for (int i = 0; i < a.tiling.rows; ++i) {
    const int rank = __shfl_sync(kAll, before, i);
    const Share s = tile_at(a.refs, a.num_pages, a.tiling, i);
    if (a.tiling.rows == 1)
      number_tile(a, s, rank, live);
    else if (s.lane == 0 && s.lo < s.hi)
      a.map[s.lo] = rank;
  }
  leave();
}

__global__ void __launch_bounds__(256) number_kernel(const CompactArgs a) {
  start_next();
  const uint64_t lo = (blockIdx.x * 8ull + (threadIdx.x >> 5)) * a.tiling.tile;
  after_previous();
  if (lo >= (uint64_t)a.num_pages) return;
  Share s;
  s.lo = (uint32_t)lo;
  s.hi = (uint32_t)min(lo + a.tiling.tile, (uint64_t)a.num_pages);
  s.lane = threadIdx.x & 31;
  s.vec = (reinterpret_cast<uintptr_t>(a.refs) & 15) == 0;
  const int live = *const_cast<volatile int32_t*>(a.counts + 1);
  const int rank = __shfl_sync(kAll, *const_cast<volatile int32_t*>(a.map + s.lo), 0);
  number_tile(a, s, rank, live);
}

// ---------------------------------------------------------------------------
// Copy
// ---------------------------------------------------------------------------

struct CopyArgs {
  uint8_t* k;
  uint8_t* v;
  int64_t page_bytes;        // between pages
  int64_t layer_bytes;       // between layers
  int64_t num_pages;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* slots;      // null: whole pages
  const int32_t* count;      // null: max_copies
  int64_t max_copies;
  int32_t page_size;
  int32_t layout;
  int32_t head_row;          // bytes of one head's row of a slot
  int32_t slot_row;          // bytes of all heads' rows of a slot
  int32_t* err;
};

// Whether piece `off` (bytes into the page) lies in the first `slots` slots:
// NHD pages hold them slot by slot, HND pages in every head.
__device__ __forceinline__ bool in_slots(const CopyArgs& a, uint32_t off, int slots) {
  if (slots == a.page_size) return true;
  const uint32_t slot = a.layout == PKA_NHD
                            ? off / (uint32_t)a.slot_row
                            : off / (uint32_t)a.head_row % (uint32_t)a.page_size;
  return slot < (uint32_t)slots;
}

// Entry i of the list, or false for one that is skipped.
__device__ __forceinline__ bool copy_at(const CopyArgs& a, int64_t i, int64_t* from, int64_t* to,
                                        int* slots, bool* bad) {
  const int32_t src = a.src[i], dst = a.dst[i];
  *slots = a.slots ? a.slots[i] : a.page_size;
  if (src < 0 || src >= a.num_pages || dst < 0 || dst >= a.num_pages || *slots < 0 ||
      *slots > a.page_size) {
    *bad = true;
    return false;
  }
  *from = src * a.page_bytes;
  *to = dst * a.page_bytes;
  return src != dst;
}

// blockIdx.y is (layer, K or V).  A warp moves 4 KB, eight 16-byte pieces a
// lane in flight: a stretch of one page, or (SMALL) pieces of as many pages as
// that takes, each lane with its own list entries.  Bound by memory bandwidth:
// 4,001 pages of 32 KB, K and V in four layers, take 310 us, 6.77 TB/s.  In us,
// a stretch / SMALL: 60,000 pages of 64 B 18.9 / 5.7, of 1 KB 44.9 / 39.9, of
// 2 KB 76.4 / 76.5, 20,000 of 8 KB 100.1 / 100.0.
template <bool SMALL>
__global__ void __launch_bounds__(256) copy_kernel(const CopyArgs a) {
  constexpr int PIECES = 8, CHUNK = PIECES * 512;
  const int lane = threadIdx.x & 31;
  uint8_t* pool = (blockIdx.y & 1 ? a.v : a.k) + (blockIdx.y >> 1) * a.layer_bytes;
  const uint32_t whole = (uint32_t)a.page_size * a.slot_row;
  const uint32_t chunks = (whole + CHUNK - 1) / CHUNK, pieces = whole / 16;
  int64_t n = a.max_copies;
  if (a.count) n = min(n, (int64_t)max(*a.count, 0));
  const int64_t units = SMALL ? (n * pieces + 32 * PIECES - 1) / (32 * PIECES) : n * chunks;
  bool bad = false;
  for (int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); w < units;
       w += (int64_t)gridDim.x * 8) {
    uint4 x[PIECES];
    if constexpr (SMALL) {
      int64_t put[PIECES];
      const int64_t at = w * (32 * PIECES) + lane;
      int64_t i = at <= UINT32_MAX ? (uint32_t)at / pieces : at / pieces;
      uint32_t piece = (uint32_t)(at - i * pieces);
#pragma unroll
      for (int u = 0; u < PIECES; ++u) {
        int64_t from, to;
        int slots;
        put[u] = -1;
        if (i < n && copy_at(a, i, &from, &to, &slots, &bad) && in_slots(a, piece * 16, slots)) {
          x[u] = *reinterpret_cast<const uint4*>(pool + from + piece * 16);
          put[u] = to + piece * 16;
        }
        i += 32 / pieces;  // 32 pieces on
        piece += 32 % pieces;
        if (piece >= pieces) {
          piece -= pieces;
          ++i;
        }
      }
#pragma unroll
      for (int u = 0; u < PIECES; ++u)
        if (put[u] >= 0) *reinterpret_cast<uint4*>(pool + put[u]) = x[u];
    } else {
      const int64_t i = w <= UINT32_MAX ? (uint32_t)w / chunks : w / chunks;
      const uint32_t off0 = (uint32_t)(w - i * chunks) * CHUNK + lane * 16;
      int64_t from, to;
      int slots;
      if (!copy_at(a, i, &from, &to, &slots, &bad)) continue;
      bool take[PIECES];
#pragma unroll
      for (int u = 0; u < PIECES; ++u) {
        const uint32_t off = off0 + u * 512;
        take[u] = off < whole && in_slots(a, off, slots);
        if (take[u]) x[u] = *reinterpret_cast<const uint4*>(pool + from + off);
      }
#pragma unroll
      for (int u = 0; u < PIECES; ++u)
        if (take[u]) *reinterpret_cast<uint4*>(pool + to + off0 + u * 512) = x[u];
    }
  }
  if (bad) note_error(a.err, PKA_ERR_METADATA);
}

int blocks_for(int64_t work, int per_block, int per_sm) {
  const int sms = current_device_sms();
  const int64_t cap = (int64_t)per_sm * (sms > 0 ? sms : 1);
  const int64_t b = (work + per_block - 1) / per_block;
  return (int)(b < 1 ? 1 : b > cap ? cap : b);
}

// Blocks of a launch that counts the references of num_pages pages.  Taking
// one page / an 11th of them and returning it, in us, with 1 and with 16
// blocks: pool of 1,024 4.1 / 4.1 and 4.7 / 4.8, 8,192 4.3 / 5.4 and 5.0 / 6.3,
// 32,768 5.3 / 7.6 and 5.6 / 6.6, 131,072 8.9 / 13.5 and 5.6 / 7.2, 1,500,007
// 46 / 63 and 9.0 / 14.3.  Compacting 16,384: 9.4 and 7.2.
int cluster_ctas(int32_t num_pages) { return num_pages <= 8192 ? 1 : kMaxCluster; }

Tiling tiling_of(int32_t num_pages) {
  const uint64_t warps = (uint64_t)cluster_ctas(num_pages) * kWarps, n = (uint64_t)num_pages;
  const uint64_t share = (n + warps * 128 - 1) / (warps * 128) * 128;  // of one row, in steps
  Tiling t;
  t.tile = share <= kTile ? (uint32_t)share
                          : (uint32_t)((n + warps * kRows * kTile - 1) / (warps * kRows * kTile)) *
                                kTile;
  t.rows = n == 0 ? 0 : (int)((n + warps * t.tile - 1) / (warps * t.tile));
  return t;
}

// Launch as one cluster.
template <auto Kernel, class A>
cudaError_t launch_cluster(int ctas, int smem, cudaStream_t stream, const A& args) {
  if (ctas > 1) {  // past the portable size of 8: allowed once per device
    static std::atomic<bool> set[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool tracked = dev >= 0 && dev < 64;
    if (!tracked || !set[dev].load(std::memory_order_acquire)) {
      e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      if (tracked) set[dev].store(true, std::memory_order_release);
    }
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)ctas;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, Kernel, args);
}

// Launch behind the call's previous launch, which lets it start early.
template <class A>
cudaError_t launch_behind(void (*kernel)(A), int blocks, cudaStream_t stream, const A& args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

pka_status done(cudaError_t e, const char* where) {
  return e == cudaSuccess ? PKA_OK : cuda_failure(e, where);
}

// Held by every call on an array of counts while it launches.  A large take
// keeps marks in the counts between its two launches, and a compaction relies
// on what it counted until its last one, so no other thread's call on the array
// may come between them in the stream that the threads share.
std::mutex& launches_of(const int32_t* refs) {
  static std::mutex table[64];
  const uint64_t a = reinterpret_cast<uintptr_t>(refs) >> 8;
  return table[(a ^ a >> 6 ^ a >> 12 ^ a >> 18) % 64];
}

}  // namespace
}  // namespace pka

extern "C" {

pka_status pka_copy_pages(const pka_params* p, int32_t num_layers, void* k, void* v,
                          int64_t page_stride, int64_t layer_stride, int64_t num_pool_pages,
                          const int32_t* src_d, const int32_t* dst_d, const int32_t* slots_d,
                          int64_t max_copies, const int32_t* num_copies_d, void* stream) {
  if (!pka::params_valid(p) || num_layers < 0 || max_copies < 0 || num_pool_pages < 0)
    return PKA_ERR_INVALID_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return PKA_ERR_UNSUPPORTED;
  if (p->kv_ragged || num_layers > 32767) return PKA_ERR_UNSUPPORTED;
  if (num_layers == 0 || max_copies == 0) return PKA_OK;
  if (!k || !v || !src_d || !dst_d || page_stride <= 0) return PKA_ERR_INVALID_ARG;
  if (pka::unaligned(src_d) || pka::unaligned(dst_d) || pka::unaligned(slots_d) ||
      pka::unaligned(num_copies_d))
    return PKA_ERR_INVALID_ARG;
  const bool f8 = p->kv_dtype == PKA_KV_FP8_E4M3;
  const int item = f8 ? 1 : 2;
  const uintptr_t mis = reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v);
  const int64_t whole16 = f8 ? 15 : 7;
  if ((mis & 15) || (page_stride & whole16)) return PKA_ERR_INVALID_ARG;
  if (num_layers > 1 && (layer_stride <= 0 || (layer_stride & whole16)))
    return PKA_ERR_INVALID_ARG;
  pka::CopyArgs a{};
  const int64_t slot_row = (int64_t)p->num_kv_heads * p->head_dim * item;
  if (slot_row > INT32_MAX / p->page_size) return PKA_ERR_UNSUPPORTED;  // a page of 2 GB
  a.k = static_cast<uint8_t*>(k);
  a.v = static_cast<uint8_t*>(v);
  a.page_bytes = page_stride * item;
  a.layer_bytes = num_layers > 1 ? layer_stride * item : 0;
  a.num_pages = num_pool_pages;
  a.src = src_d;
  a.dst = dst_d;
  a.slots = slots_d;
  a.count = num_copies_d;
  a.max_copies = max_copies;
  a.page_size = p->page_size;
  a.layout = p->layout;
  a.head_row = p->head_dim * item;
  a.slot_row = (int32_t)slot_row;
  a.err = pka::device_error_word();
  const int64_t page = p->page_size * slot_row;
  const bool small = page < 2048;
  const int64_t units = small ? (max_copies * page + 4095) / 4096
                              : max_copies * ((page + 4095) / 4096);
  const int per_sm = 16 / (2 * num_layers) > 1 ? 16 / (2 * num_layers) : 1;
  const dim3 grid((unsigned)pka::blocks_for(units, 8, per_sm), (unsigned)(2 * num_layers));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (small)
    pka::copy_kernel<true><<<grid, 256, 0, st>>>(a);
  else
    pka::copy_kernel<false><<<grid, 256, 0, st>>>(a);
  return pka::done(cudaGetLastError(), "page copy launch");
}

pka_status pka_alloc_pages(int32_t* page_refs_d, int32_t num_pages, int32_t n, int32_t* pages_d,
                           void* stream) {
  if (num_pages < 0 || n < 0) return PKA_ERR_INVALID_ARG;
  if (n == 0) return PKA_OK;
  if (n > num_pages) return PKA_ERR_WORKSPACE;
  if (!page_refs_d || !pages_d || pka::unaligned(page_refs_d) || pka::unaligned(pages_d))
    return PKA_ERR_INVALID_ARG;
  const pka::AllocArgs a{page_refs_d, pages_d, pka::device_error_word(), num_pages, n,
                         pka::tiling_of(num_pages)};
  const int ctas = pka::cluster_ctas(num_pages);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const std::lock_guard<std::mutex> lock(pka::launches_of(page_refs_d));
  if (a.tiling.rows == 1 || n <= pka::kTakeInPlace)
    return pka::done(pka::launch_cluster<pka::alloc_kernel<false>>(ctas, 0, st, a),
                     "page alloc launch");
  cudaError_t e = pka::launch_cluster<pka::alloc_kernel<true>>(ctas, 0, st, a);
  const int64_t tiles = (num_pages + (int64_t)a.tiling.tile - 1) / a.tiling.tile;
  if (e == cudaSuccess) e = pka::launch_behind(pka::take_kernel, (int)((tiles + 7) / 8), st, a);
  return pka::done(e, "page alloc launch");
}

pka_status pka_free_pages(int32_t* page_refs_d, int32_t num_pages, const int32_t* pages_d,
                          int64_t n, void* stream) {
  if (num_pages < 0 || n < 0) return PKA_ERR_INVALID_ARG;
  if (n == 0) return PKA_OK;
  if (!page_refs_d || !pages_d || pka::unaligned(page_refs_d) || pka::unaligned(pages_d))
    return PKA_ERR_INVALID_ARG;
  const std::lock_guard<std::mutex> lock(pka::launches_of(page_refs_d));
  pka::free_kernel<<<pka::blocks_for(n, 256, 8), 256, 0, static_cast<cudaStream_t>(stream)>>>(
      page_refs_d, num_pages, pages_d, n, pka::device_error_word());
  return pka::done(cudaGetLastError(), "page free launch");
}

pka_status pka_fork_pages(int32_t page_size, int32_t* page_refs_d, int32_t num_pages,
                          int32_t num_parents, const int32_t* kv_indptr_d,
                          const int32_t* kv_indices_d, int32_t num_indices,
                          const int32_t* last_page_len_d, int32_t num_children,
                          const int32_t* parent_d, const int32_t* child_indptr_d,
                          int32_t* child_indices_d, int32_t num_child_indices,
                          int32_t* copy_src_d, int32_t* copy_dst_d, int32_t* copy_slots_d,
                          int32_t* counts_d, void* stream) {
  if (page_size < 1 || num_pages < 0 || num_parents < 0 || num_indices < 0 || num_children < 0 ||
      num_child_indices < 0)
    return PKA_ERR_INVALID_ARG;
  const uintptr_t table = reinterpret_cast<uintptr_t>(child_indices_d);
  const uintptr_t parents_table = reinterpret_cast<uintptr_t>(kv_indices_d);
  if (table < parents_table + 4 * (uintptr_t)num_indices &&
      parents_table < table + 4 * (uintptr_t)num_child_indices)
    return PKA_ERR_INVALID_ARG;
  if (num_children > PKA_MAX_FORK_CHILDREN) return PKA_ERR_UNSUPPORTED;
  if (!counts_d || pka::unaligned(counts_d)) return PKA_ERR_INVALID_ARG;
  const bool parents = num_parents > 0 && (!kv_indptr_d || !last_page_len_d);
  const bool children = num_children > 0 && (!parent_d || !child_indptr_d || !copy_src_d ||
                                             !copy_dst_d || !copy_slots_d);
  if (parents || children || (num_indices > 0 && !kv_indices_d) ||
      (num_child_indices > 0 && !child_indices_d) || (num_pages > 0 && !page_refs_d))
    return PKA_ERR_INVALID_ARG;
  const void* arrays[] = {page_refs_d,    kv_indptr_d,     kv_indices_d, last_page_len_d,
                          parent_d,       child_indptr_d,  child_indices_d, copy_src_d,
                          copy_dst_d,     copy_slots_d};
  for (const void* x : arrays)
    if (pka::unaligned(x)) return PKA_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (num_children == 0) return pka::done(cudaMemsetAsync(counts_d, 0, 8, st), "page fork counts");
  pka::ForkArgs a{};
  a.refs = page_refs_d;
  a.kv_indptr = kv_indptr_d;
  a.kv_indices = kv_indices_d;
  a.last_page_len = last_page_len_d;
  a.parent = parent_d;
  a.child_indptr = child_indptr_d;
  a.child_indices = child_indices_d;
  a.copy_src = copy_src_d;
  a.copy_dst = copy_dst_d;
  a.copy_slots = copy_slots_d;
  a.counts = counts_d;
  a.err = pka::device_error_word();
  a.page_size = page_size;
  a.num_pages = num_pages;
  a.num_parents = num_parents;
  a.num_children = num_children;
  a.num_indices = num_indices;
  a.num_child_indices = num_child_indices;
  a.tiling = pka::tiling_of(num_pages);
  const int smem = (pka::kChildWords * num_children + 1) * (int)sizeof(int32_t);
  const int ctas = pka::cluster_ctas(num_pages);
  const std::lock_guard<std::mutex> lock(pka::launches_of(page_refs_d));
  if (num_child_indices <= pka::kShareInTake) {
    cudaError_t e = pka::ensure_dynamic_smem<pka::fork_take_kernel<true>>(smem);
    if (e == cudaSuccess)
      e = pka::launch_cluster<pka::fork_take_kernel<true>>(ctas, smem, st, a);
    return pka::done(e, "page fork launch");
  }
  cudaError_t e = pka::ensure_dynamic_smem<pka::fork_take_kernel<false>>(smem);
  if (e == cudaSuccess) e = pka::launch_cluster<pka::fork_take_kernel<false>>(ctas, smem, st, a);
  if (e != cudaSuccess) return pka::cuda_failure(e, "page fork launch");
  return pka::done(pka::launch_behind(pka::fork_share_kernel,
                                      pka::blocks_for(num_child_indices, 8 * 256, 8), st, a),
                   "page fork launch");
}

pka_status pka_compact_pages(const int32_t* page_refs_d, int32_t num_pages,
                             const int32_t* kv_indices_d, int64_t num_indices,
                             int32_t* page_refs_out_d, int32_t* kv_indices_out_d,
                             int32_t* page_map_d, int32_t* copy_src_d, int32_t* copy_dst_d,
                             int32_t* counts_d, void* stream) {
  if (num_pages < 0 || num_indices < 0) return PKA_ERR_INVALID_ARG;
  if (!counts_d || pka::unaligned(counts_d)) return PKA_ERR_INVALID_ARG;
  if (num_pages > 0 && (!page_refs_d || !page_refs_out_d || !page_map_d))
    return PKA_ERR_INVALID_ARG;
  if (num_pages > 1 && (!copy_src_d || !copy_dst_d)) return PKA_ERR_INVALID_ARG;
  if (num_indices > 0 && (!kv_indices_d || !kv_indices_out_d)) return PKA_ERR_INVALID_ARG;
  const void* arrays[] = {page_refs_d, kv_indices_d, page_refs_out_d, kv_indices_out_d,
                          page_map_d,  copy_src_d,   copy_dst_d};
  for (const void* x : arrays)
    if (pka::unaligned(x)) return PKA_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  pka::CompactArgs a{};
  a.refs = page_refs_d;
  a.refs_out = page_refs_out_d;
  a.map = page_map_d;
  a.copy_src = copy_src_d;
  a.copy_dst = copy_dst_d;
  a.counts = counts_d;
  a.in = kv_indices_d;
  a.out = kv_indices_out_d;
  a.err = pka::device_error_word();
  a.num_indices = num_indices;
  a.num_pages = num_pages;
  a.tiling = pka::tiling_of(num_pages);
  if (num_pages == 0) {  // every entry names a page that is not there
    cudaError_t e = cudaMemsetAsync(counts_d, 0, 8, st);
    if (e == cudaSuccess && num_indices > 0) {
      pka::move_kernel<<<pka::blocks_for(num_indices, 256, 8), 256, 0, st>>>(a);
      e = cudaGetLastError();
    }
    return pka::done(e, "page compact launch");
  }
  std::mutex& in = pka::launches_of(page_refs_d);
  std::mutex& out = pka::launches_of(page_refs_out_d);
  std::unique_lock<std::mutex> lock_in(in, std::defer_lock), lock_out(out, std::defer_lock);
  if (&in == &out)
    lock_in.lock();
  else
    std::lock(lock_in, lock_out);
  cudaError_t e =
      pka::launch_cluster<pka::compact_kernel>(pka::cluster_ctas(num_pages), 0, st, a);
  if (e != cudaSuccess) return pka::cuda_failure(e, "page compact launch");
  if (a.tiling.rows > 1) {
    const int64_t tiles = (num_pages + (int64_t)a.tiling.tile - 1) / a.tiling.tile;
    e = pka::launch_behind(pka::number_kernel, (int)((tiles + 7) / 8), st, a);
    if (e != cudaSuccess) return pka::cuda_failure(e, "page numbering launch");
  }
  const int64_t work = num_indices > num_pages / 2 ? num_indices : num_pages / 2;
  if (work == 0) return PKA_OK;  // one page, no entry: nothing moves
  return pka::done(pka::launch_behind(pka::move_kernel, pka::blocks_for(work, 256, 8), st, a),
                   "page move launch");
}

}  // extern "C"
