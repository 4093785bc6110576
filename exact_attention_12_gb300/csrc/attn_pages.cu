// Upkeep of a paged key/value cache on the device: copying pages, growing,
// forking and freeing sequences, and compacting the pages in use.
//
// State (include/attn.h): a table of page indices per sequence, the sequences'
// lengths, and a reference count per page (0: free).  Every operation reads
// and writes it in device memory, so a serving loop needs no round trip to
// the host and can be captured in a CUDA graph.
//
// Bound: the page copies, 2 bytes moved a byte, at HBM rate; next to them the
// table and counts are small, but a call on a small cache is bound by its
// launches, so an operation takes one kernel, or two where copies follow from
// a decision: a one-CTA plan kernel (which pages are taken, which move: ranks
// by ballots and a scan, so the choice is the lowest free page first and does
// not depend on timing), then a copy kernel over the whole GPU.  (A fork has a
// third before them, which looks at every page of the parents.)  Copies are
// cut into pieces of 16 KB, one per CTA turn, four 16-byte loads in flight a
// thread.
//
// Measured: closing the gaps of 8194 pages of 64 keys (8 heads, d = 128, keys
// and values; 0.93 GB read and written) 143 us = 6.5 TB/s, the plan before it
// 8 us; 512 forks of 64 sequences, each with its last page copied, 36 us; four
// forks of a short prompt 7 us, which is the three launches.
#include <climits>
#include <cstdio>

#include "attn.h"
#include "attn_kernels.cuh"
#include "attn_paged.cuh"

namespace attn {
using namespace sm103;

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kCopyBytes = kCopyThreads * 16 * 4;        // a copy piece
constexpr int kPoolsPerLaunch = 64;
constexpr int kStatusFull = 7;                           // equals ATTN_ERR_FULL in attn.h

struct Table {
  int32_t* table;
  int64_t stride;
  int32_t* lens;
  int32_t* refs;
  int rows, max_pages, page_size, num_pages;
  int* status;
};

struct Pool {
  char* base;
  int64_t stride, bytes;   // between pages, of a page
};
struct Pools {
  Pool p[kPoolsPerLaunch];
  int n;
  int64_t pieces;          // copy pieces per page, all pools
};

__device__ void report(int* status, int code) {
  if (atomicCAS(status, 0, code) == 0) atomicExch(status + 1, kSitePageIndex);
}

__device__ __forceinline__ bool in_range(int i, int n) {
  return static_cast<unsigned>(i) < static_cast<unsigned>(n);
}

__device__ __forceinline__ int held_pages(const Table& t, int len) {
  const int64_t cap = static_cast<int64_t>(t.max_pages) * t.page_size;
  const int64_t n = min(static_cast<int64_t>(max(len, 0)), cap);
  return static_cast<int>((n + t.page_size - 1) / t.page_size);
}

// Exclusive rank of each thread's `x` over the block and the block's total.
// `scratch`: 33 values.
template <typename T>
__device__ __forceinline__ T block_rank(T x, T* scratch, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const T mine = lane < static_cast<int>(blockDim.x) / 32 ? scratch[lane] : 0;
    T s = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    __syncwarp();
    scratch[lane] = s - mine;
    if (lane == 31) scratch[32] = s;
  }
  __syncthreads();
  const T before = scratch[warp];
  *total = scratch[32];
  __syncthreads();   // scratch is free again
  return before + inc - x;
}

// The pages that a plan looks at together: a warp has `words` runs of 32 (up to
// 32 of them, so that all warps have their share of a small cache), lane l of
// it run l.
struct Batch {
  int words;
  __device__ explicit Batch(int num_pages)
      : words(min(32, (num_pages + kPlanThreads - 1) / kPlanThreads)) {}
  __device__ int size() const { return kPlanThreads * words; }
  // The first page of this thread's run, if it has one.
  __device__ int first(int base) const {
    return base + 32 * (static_cast<int>(threadIdx.x >> 5) * words + static_cast<int>(threadIdx.x & 31));
  }
  // Which of its pages are in use, a bit each (0 past the last page).  The warp
  // reads its counts in order, 32 at a time.
  __device__ uint32_t used(const Table& t, int base) const {
    const int lane = threadIdx.x & 31, start = base + 32 * static_cast<int>(threadIdx.x >> 5) * words;
    uint32_t mask = 0;
#pragma unroll 8
    for (int k = 0; k < words; ++k) {
      const int i = start + 32 * k + lane;
      const uint32_t word = __ballot_sync(0xffffffffu, i < t.num_pages && t.refs[i] != 0);
      if (lane == k) mask = word;
    }
    return mask;
  }
  // The bits of its pages that lie below page `end`.
  __device__ uint32_t below(int base, int end) const {
    const int n = static_cast<int>(threadIdx.x & 31) < words ? end - first(base) : 0;
    return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
  }
};

// The lowest `need` free pages into `list`, ascending; how many there are (at
// most `need`).  The whole block.
__device__ int lowest_free(const Table& t, int need, int32_t* list, int* scratch) {
  const Batch batch(t.num_pages);
  int found = 0;
  for (int base = 0; base < t.num_pages && found < need; base += batch.size()) {
    uint32_t free = ~batch.used(t, base) & batch.below(base, t.num_pages);
    int total;
    int at = found + block_rank(__popc(free), scratch, &total);
    for (; free != 0 && at < need; free &= free - 1) list[at++] = batch.first(base) + __ffs(free) - 1;
    found += total;
  }
  __syncthreads();   // list is visible to the block
  return min(found, need);
}

// Whether item i of a list is the first that names `row` (claims of an
// earlier item win); an invalid row is nobody's.  The whole block.
__device__ void claim_rows(const int32_t* rows_list, int n, int rows, int32_t* claim) {
  for (int i = threadIdx.x; i < n; i += blockDim.x)
    if (in_range(rows_list[i], rows)) claim[rows_list[i]] = INT_MAX;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x)
    if (in_range(rows_list[i], rows)) atomicMin(&claim[rows_list[i]], i);
  __syncthreads();
}

// ------------------------------------------------------------------- extend --

// Sequence seqs[i] grows to new_lens[i] keys: the pages it needs are the
// lowest free ones, in the list's order.
__global__ void __launch_bounds__(kPlanThreads)
    extend_kernel(Table t, const int32_t* seqs, const int32_t* new_lens, int n, int32_t* claim,
                  int32_t* rank, int32_t* list) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ int64_t sums[33];
  __shared__ int scratch[33];
  claim_rows(seqs, n, t.rows, claim);
  const int64_t cap = static_cast<int64_t>(t.max_pages) * t.page_size;
  int64_t need = 0;   // pages of all items, far more than there are perhaps
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    int64_t want = 0;
    bool ok = false;
    if (i < n) {
      const int s = seqs[i];
      ok = in_range(s, t.rows) && claim[s] == i && t.lens[s] >= 0 && new_lens[i] >= t.lens[s] &&
           new_lens[i] <= cap;
      if (ok) want = held_pages(t, new_lens[i]) - held_pages(t, t.lens[s]);
      else report(t.status, kStatusPage);
    }
    int64_t total;
    const int64_t at = need + block_rank(want, sums, &total);
    if (i < n)   // (a rank past every page: there are too few)
      rank[i] = ok ? static_cast<int>(min(at, static_cast<int64_t>(INT_MAX))) : -1;
    need += total;
  }
  const int have = lowest_free(
      t, static_cast<int>(min(need, static_cast<int64_t>(t.num_pages))), list, scratch);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = warp; i < n; i += kPlanThreads / 32) {
    const int at = rank[i];
    if (at < 0) continue;
    const int s = seqs[i], from = held_pages(t, t.lens[s]), to = held_pages(t, new_lens[i]);
    if (at > have - (to - from)) {   // too few pages are left: the sequence stays as it was
      if (to > from) {
        if (lane == 0) report(t.status, kStatusFull);
        continue;
      }
    }
    for (int j = from + lane; j < to; j += 32) {
      const int pg = list[at + j - from];
      t.table[s * t.stride + j] = pg;
      t.refs[pg] = 1;
    }
    __syncwarp();
    if (lane == 0) t.lens[s] = new_lens[i];
  }
}

// --------------------------------------------------------------------- fork --

// Whether fork i can be made, as far as it does not depend on the others: its
// rows exist, the child is empty, and every page that the parent holds is in
// use (one that is free could be handed out as new in this very call).
// plen[i]: the parent's length, -1 if not.  A CTA per fork: the plan's one CTA
// would read all the parents' rows one after another.
__global__ void __launch_bounds__(128)
    fork_check_kernel(Table t, const int32_t* parents, const int32_t* children, int32_t* plen) {
  grid_dep_wait();
  grid_dep_launch();
  const int i = blockIdx.x, c = children[i], p = parents[i];
  bool ok = in_range(c, t.rows) && in_range(p, t.rows);
  const int len = ok ? t.lens[p] : -1;
  if (ok)
    ok = t.lens[c] == 0 && len >= 0 && len <= static_cast<int64_t>(t.max_pages) * t.page_size;
  if (ok) {
    const int held = held_pages(t, len);
    for (int j = threadIdx.x; j < held; j += 128) {
      const int pg = t.table[p * t.stride + j];
      ok = ok && in_range(pg, t.num_pages) && t.refs[pg] > 0;
    }
  }
  ok = __syncthreads_and(ok);
  if (threadIdx.x == 0) {
    plen[i] = ok ? len : -1;
    if (!ok) report(t.status, kStatusPage);
  }
}

// Fork i: children[i] becomes a copy of parents[i].  Its full pages are
// shared, a part-filled last page gets a page of its own: new_pages[i] (-1:
// none is needed, -2: the fork is refused or no page is free).
__global__ void __launch_bounds__(kPlanThreads)
    fork_plan_kernel(Table t, const int32_t* children, int n, int32_t* new_pages,
                     int32_t* plen, int32_t* claim, int32_t* list) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ int scratch[33];
  claim_rows(children, n, t.rows, claim);
  int need = 0;
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    int part = 0, len = -1;
    if (i < n) {
      len = plen[i];
      if (len >= 0 && claim[children[i]] != i) {   // an earlier fork has the child
        len = plen[i] = -1;
        report(t.status, kStatusPage);
      }
      part = len > 0 && len % t.page_size != 0;
    }
    int total;
    const int at = need + block_rank(part, scratch, &total);
    if (i < n) new_pages[i] = part ? at : (len < 0 ? -2 : -1);
    need += total;
  }
  __syncthreads();
  const int have = lowest_free(t, need, list, scratch);
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int at = new_pages[i];
    if (at < 0) continue;
    if (at < have) {
      new_pages[i] = list[at];
    } else {
      new_pages[i] = -2;
      plen[i] = -1;
      report(t.status, kStatusFull);
    }
  }
}

// One piece of a page copy: bytes [off, off + kCopyBytes) of a page.
__device__ __forceinline__ void copy_piece(const Pool& p, int64_t src, int64_t dst, int64_t off) {
  const char* from = p.base + src * p.stride + off;
  char* to = p.base + dst * p.stride + off;
  const int64_t left = p.bytes - off;
  uint4 x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t at = (static_cast<int64_t>(k) * kCopyThreads + threadIdx.x) * 16;
    if (at < left) x[k] = __ldcs(reinterpret_cast<const uint4*>(from + at));
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t at = (static_cast<int64_t>(k) * kCopyThreads + threadIdx.x) * 16;
    if (at < left) __stcs(reinterpret_cast<uint4*>(to + at), x[k]);
  }
}

// Piece `piece` of pages.pieces: which pool and offset.
__device__ __forceinline__ void copy_page(const Pools& pools, int64_t src, int64_t dst, int64_t piece) {
  int k = 0;
  for (; k < pools.n - 1; ++k) {
    const int64_t here = (pools.p[k].bytes + kCopyBytes - 1) / kCopyBytes;
    if (piece < here) break;
    piece -= here;
  }
  copy_piece(pools.p[k], src, dst, piece * kCopyBytes);
}

// The rows of the children (`rows`: with the first group of pools only), and
// the copies of the part-filled pages.
__global__ void __launch_bounds__(kCopyThreads)
    fork_apply_kernel(Table t, const __grid_constant__ Pools pools, const int32_t* parents,
                      const int32_t* children, int n, const int32_t* new_pages,
                      const int32_t* plen, int rows) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t heads = rows ? n : 0, all = heads + n * pools.pieces;
  for (int64_t w = blockIdx.x; w < all; w += gridDim.x) {
    if (w < heads) {
      const int i = static_cast<int>(w), len = plen[i];
      if (len < 0) continue;
      const int32_t* from = t.table + parents[i] * t.stride;
      int32_t* to = t.table + children[i] * t.stride;
      const int full = len / t.page_size;
      for (int j = threadIdx.x; j < full; j += kCopyThreads) {
        const int pg = from[j];
        to[j] = pg;
        atomicAdd(&t.refs[pg], 1);
      }
      if (threadIdx.x == 0) {
        if (new_pages[i] >= 0) {
          to[full] = new_pages[i];
          t.refs[new_pages[i]] = 1;
        }
        t.lens[children[i]] = len;
      }
    } else {
      const int64_t c = w - heads;
      const int i = static_cast<int>(c / pools.pieces);
      if (new_pages[i] < 0) continue;
      copy_page(pools, t.table[parents[i] * t.stride + plen[i] / t.page_size], new_pages[i],
                c - i * pools.pieces);
    }
  }
}

// --------------------------------------------------------------------- free --

// A CTA per list entry.  The exchange hands a sequence's pages to one entry
// only, so a sequence that is named twice is freed once.
__global__ void __launch_bounds__(128) free_kernel(Table t, const int32_t* seqs) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ int len;
  const int s = seqs[blockIdx.x];
  if (!in_range(s, t.rows)) {
    if (threadIdx.x == 0) report(t.status, kStatusPage);
    return;
  }
  if (threadIdx.x == 0) len = atomicExch(&t.lens[s], 0);
  __syncthreads();
  const int n = held_pages(t, len);
  int32_t* row = t.table + s * t.stride;
  for (int j = threadIdx.x; j < n; j += 128) {
    const int pg = row[j];
    row[j] = -1;
    if (!in_range(pg, t.num_pages)) {
      report(t.status, kStatusPage);
    } else if (atomicSub(&t.refs[pg], 1) <= 0) {   // was free already
      atomicAdd(&t.refs[pg], 1);
      report(t.status, kStatusPage);
    }
  }
}

// ------------------------------------------------------------------ compact --

// The n_used pages in use come to lie in the first n_used places: those
// behind them move, ascending, to the free places before, ascending.
__global__ void __launch_bounds__(kPlanThreads)
    compact_plan_kernel(Table t, int32_t* moved, int32_t* holes, int32_t* movers, int32_t* count) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ int scratch[33];
  __shared__ uint32_t ranks[33];
  const int P = t.num_pages;
  const Batch batch(P);
  int used = 0;
  uint32_t mask = 0;   // (of the only batch, where there is one)
  for (int base = 0; base < P; base += batch.size()) {
    mask = batch.used(t, base);
    int total;
    block_rank(__popc(mask), scratch, &total);
    used += total;
  }
  const int lane = threadIdx.x & 31;
  int n_holes = 0, n_movers = 0;
  for (int base = 0; base < P; base += batch.size()) {
    if (P > batch.size()) mask = batch.used(t, base);
    const int i0 = batch.first(base);
    const uint32_t low = batch.below(base, used);
    uint32_t hole = ~mask & low, mover = mask & ~low;
    // both ranks in one scan: the counts of a batch fit 16 bits each
    uint32_t total;
    const uint32_t rank = block_rank(
        static_cast<uint32_t>(__popc(hole) | __popc(mover) << 16), ranks, &total);
    int at = n_holes + static_cast<int>(rank & 0xffffu);
    for (; hole != 0; hole &= hole - 1) holes[at++] = i0 + __ffs(hole) - 1;
    at = n_movers + static_cast<int>(rank >> 16);
    for (; mover != 0; mover &= mover - 1) movers[at++] = i0 + __ffs(mover) - 1;
    n_holes += static_cast<int>(total & 0xffffu);
    n_movers += static_cast<int>(total >> 16);
    const int start = base + 32 * static_cast<int>(threadIdx.x >> 5) * batch.words;
    for (int k = 0; k < batch.words; ++k) {
      const uint32_t word = __shfl_sync(0xffffffffu, mask, k);
      const int i = start + 32 * k + lane;
      if (i < P) moved[i] = (word >> lane) & 1u ? i : -1;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n_movers; i += kPlanThreads) {
    moved[movers[i]] = holes[i];
    t.refs[holes[i]] = t.refs[movers[i]];
    t.refs[movers[i]] = 0;
  }
  if (threadIdx.x == 0) *count = n_movers;
}

__global__ void __launch_bounds__(kCopyThreads)
    compact_apply_kernel(Table t, const __grid_constant__ Pools pools, const int32_t* moved,
                         const int32_t* holes, const int32_t* movers, const int32_t* count,
                         int rows) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t heads = rows ? t.rows : 0, all = heads + *count * pools.pieces;
  for (int64_t w = blockIdx.x; w < all; w += gridDim.x) {
    if (w < heads) {
      const int s = static_cast<int>(w), n = held_pages(t, t.lens[s]);
      int32_t* row = t.table + s * t.stride;
      for (int j = threadIdx.x; j < n; j += kCopyThreads) {
        const int pg = row[j];
        const bool there = in_range(pg, t.num_pages);
        const int to = there ? moved[pg] : -1;   // -1: a free page, which is nobody's now
        if (there) row[j] = to;
        if (to < 0) report(t.status, kStatusPage);
      }
    } else {
      const int64_t c = w - heads, i = c / pools.pieces;
      copy_page(pools, movers[i], holes[i], c - i * pools.pieces);
    }
  }
}

// --------------------------------------------------------------------- copy --

__global__ void __launch_bounds__(kCopyThreads)
    copy_kernel(const __grid_constant__ Pools pools, const int32_t* src, const int32_t* dst, int n,
                int num_pages, int* status) {
  grid_dep_wait();
  grid_dep_launch();
  for (int64_t w = blockIdx.x; w < n * pools.pieces; w += gridDim.x) {
    const int64_t i = w / pools.pieces;
    const int s = src[i], d = dst[i];
    if (!in_range(s, num_pages) || !in_range(d, num_pages)) {
      if (threadIdx.x == 0) report(status, kStatusPage);
      continue;
    }
    if (s != d) copy_page(pools, s, d, w - i * pools.pieces);
  }
}

// --------------------------------------------------------------------- host --

constexpr size_t kHeader = 256;

int bad(int status, const char* msg) { return record_error(status, msg); }

int check_table(const attn_page_table* t) {
  if (t == nullptr) return bad(ATTN_ERR_INVALID_ARG, "page table is NULL");
  if (t->rows < 0 || t->max_pages < 0 || t->num_pages < 0)
    return bad(ATTN_ERR_INVALID_ARG, "page table: negative size");
  if (t->page_size < 1 || static_cast<int64_t>(t->max_pages) * t->page_size > (int64_t{1} << 30))
    return bad(ATTN_ERR_INVALID_ARG, "page table: page_size must be positive, a row at most 2^30 keys");
  if (t->table_stride < t->max_pages)
    return bad(ATTN_ERR_INVALID_ARG, "page table: table_stride < max_pages");
  if (t->num_pages > (1 << 30)) return bad(ATTN_ERR_UNSUPPORTED, "page table: too many pages");
  if ((t->rows > 0 && t->max_pages > 0 && t->table == nullptr) ||
      (t->rows > 0 && t->lens == nullptr) || (t->num_pages > 0 && t->refs == nullptr))
    return bad(ATTN_ERR_INVALID_ARG, "page table: NULL pointer");
  return ATTN_OK;
}

int check_pools(const attn_pool* pools, int n_pools, int num_pages) {
  if (n_pools < 0 || (n_pools > 0 && pools == nullptr))
    return bad(ATTN_ERR_INVALID_ARG, "pools: bad count or NULL");
  for (int i = 0; i < n_pools; ++i) {
    const attn_pool& p = pools[i];
    if ((p.base == nullptr && num_pages > 0) || (reinterpret_cast<uintptr_t>(p.base) & 15u) != 0)
      return bad(ATTN_ERR_INVALID_ARG, "pools: base must be 16-byte aligned");
    if (p.page_bytes <= 0 || p.page_bytes % 16 != 0 || p.page_stride % 16 != 0 ||
        p.page_stride < p.page_bytes)
      return bad(ATTN_ERR_INVALID_ARG,
                 "pools: page_bytes and page_stride must be multiples of 16, pages apart");
  }
  return ATTN_OK;
}

int check_ws_bytes(const void* ws, size_t ws_bytes, size_t need) {
  if (ws == nullptr) return bad(ATTN_ERR_WORKSPACE, "workspace is NULL");
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
    return bad(ATTN_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (ws_bytes < need) return bad(ATTN_ERR_WORKSPACE, "workspace too small");
  return ATTN_OK;
}

int check_list(int n, const void* a, const void* b) {
  if (n < 0) return bad(ATTN_ERR_INVALID_ARG, "negative list length");
  if (n > 0 && (a == nullptr || b == nullptr)) return bad(ATTN_ERR_INVALID_ARG, "list is NULL");
  return ATTN_OK;
}

Table dev_table(const attn_page_table* t, void* ws) {
  return Table{t->table,     t->table_stride, t->lens,      t->refs,
               t->rows,      t->max_pages,    t->page_size, t->num_pages,
               static_cast<int*>(ws)};
}

int launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return ATTN_OK;
  char msg[256];
  snprintf(msg, sizeof(msg), "%s: %s", what, cudaGetErrorString(e));
  return bad(ATTN_ERR_CUDA, msg);
}

// Pools [i0, ...) of the list, as many as fit a launch.
Pools group(const attn_pool* pools, int n_pools, int i0) {
  Pools g{};
  for (int i = i0; i < n_pools && g.n < kPoolsPerLaunch; ++i) {
    g.p[g.n++] = Pool{static_cast<char*>(pools[i].base), pools[i].page_stride, pools[i].page_bytes};
    g.pieces += (pools[i].page_bytes + kCopyBytes - 1) / kCopyBytes;
  }
  return g;
}

// CTAs for `work` turns: at most eight per SM.
unsigned copy_grid(int64_t work) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    sms = 148;
  return static_cast<unsigned>(work < 1 ? 1 : (work < 8ll * sms ? work : 8ll * sms));
}

int32_t* ints(void* ws, size_t at) {
  return reinterpret_cast<int32_t*>(static_cast<char*>(ws) + kHeader) + at;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

size_t attn_pages_workspace_size(const attn_page_table* t, int32_t n) {
  if (check_table(t) != ATTN_OK || check_list(n, t, t) != ATTN_OK) return 0;
  // header, then ints: claims per row, two per list entry, two lists of
  // pages, a count
  return kHeader + 4 * (static_cast<size_t>(t->rows) + 2 * static_cast<size_t>(n) +
                        2 * static_cast<size_t>(t->num_pages) + 1);
}

attn_status attn_pages_copy(const attn_pool* pools, int32_t n_pools, int32_t num_pages,
                            const int32_t* src, const int32_t* dst, int32_t n, void* ws,
                            size_t ws_bytes, void* stream) {
  int st;
  if ((st = check_pools(pools, n_pools, num_pages)) != ATTN_OK ||
      (st = check_list(n, src, dst)) != ATTN_OK ||
      (st = check_ws_bytes(ws, ws_bytes, kHeader)) != ATTN_OK)
    return static_cast<attn_status>(st);
  if (num_pages < 0) return static_cast<attn_status>(bad(ATTN_ERR_INVALID_ARG, "negative num_pages"));
  if (n == 0) return ATTN_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  for (int i0 = 0; i0 < n_pools; i0 += kPoolsPerLaunch) {
    const Pools g = group(pools, n_pools, i0);
    const cudaError_t e = launch_pdl(copy_kernel, dim3(copy_grid(n * g.pieces)), dim3(kCopyThreads), 0,
                                     s, g, src, dst, static_cast<int>(n),
                                     static_cast<int>(num_pages), static_cast<int*>(ws));
    if (e != cudaSuccess) return static_cast<attn_status>(launched(e, "page copy launch"));
  }
  return ATTN_OK;
}

attn_status attn_pages_extend(const attn_page_table* t, const int32_t* seqs,
                              const int32_t* new_lens, int32_t n, void* ws, size_t ws_bytes,
                              void* stream) {
  int st;
  if ((st = check_table(t)) != ATTN_OK || (st = check_list(n, seqs, new_lens)) != ATTN_OK ||
      (st = check_ws_bytes(ws, ws_bytes, attn_pages_workspace_size(t, n))) != ATTN_OK)
    return static_cast<attn_status>(st);
  if (n == 0) return ATTN_OK;
  const size_t rows = static_cast<size_t>(t->rows);
  return static_cast<attn_status>(launched(
      launch_pdl(extend_kernel, dim3(1), dim3(kPlanThreads), 0, static_cast<cudaStream_t>(stream),
                 dev_table(t, ws), seqs, new_lens, static_cast<int>(n), ints(ws, 0),
                 ints(ws, rows), ints(ws, rows + 2 * static_cast<size_t>(n))),
      "page extend launch"));
}

attn_status attn_pages_fork(const attn_page_table* t, const attn_pool* pools, int32_t n_pools,
                            const int32_t* parents, const int32_t* children, int32_t n,
                            int32_t* new_pages, void* ws, size_t ws_bytes, void* stream) {
  int st;
  if ((st = check_table(t)) != ATTN_OK ||
      (st = check_pools(pools, n_pools, t->num_pages)) != ATTN_OK ||
      (st = check_list(n, parents, children)) != ATTN_OK ||
      (st = check_list(n, new_pages, new_pages)) != ATTN_OK ||
      (st = check_ws_bytes(ws, ws_bytes, attn_pages_workspace_size(t, n))) != ATTN_OK)
    return static_cast<attn_status>(st);
  if (n == 0) return ATTN_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Table d = dev_table(t, ws);
  const size_t rows = static_cast<size_t>(t->rows);
  int32_t* plen = ints(ws, rows);
  cudaError_t e = launch_pdl(fork_check_kernel, dim3(static_cast<unsigned>(n)), dim3(128), 0, s, d,
                             parents, children, plen);
  if (e == cudaSuccess)
    e = launch_pdl(fork_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, d, children,
                   static_cast<int>(n), new_pages, plen, ints(ws, 0),
                   ints(ws, rows + 2 * static_cast<size_t>(n)));
  for (int i0 = 0; e == cudaSuccess && (i0 < n_pools || i0 == 0); i0 += kPoolsPerLaunch) {
    const Pools g = group(pools, n_pools, i0);
    e = launch_pdl(fork_apply_kernel, dim3(copy_grid(n * (g.pieces + (i0 == 0 ? 1 : 0)))),
                   dim3(kCopyThreads), 0, s, d, g, parents, children, static_cast<int>(n),
                   static_cast<const int32_t*>(new_pages), static_cast<const int32_t*>(plen),
                   i0 == 0 ? 1 : 0);
  }
  return static_cast<attn_status>(launched(e, "page fork launch"));
}

attn_status attn_pages_free(const attn_page_table* t, const int32_t* seqs, int32_t n, void* ws,
                            size_t ws_bytes, void* stream) {
  int st;
  if ((st = check_table(t)) != ATTN_OK || (st = check_list(n, seqs, seqs)) != ATTN_OK ||
      (st = check_ws_bytes(ws, ws_bytes, kHeader)) != ATTN_OK)
    return static_cast<attn_status>(st);
  if (n == 0) return ATTN_OK;
  return static_cast<attn_status>(launched(
      launch_pdl(free_kernel, dim3(static_cast<unsigned>(n)), dim3(128), 0,
                 static_cast<cudaStream_t>(stream), dev_table(t, ws), seqs),
      "page free launch"));
}

attn_status attn_pages_compact(const attn_page_table* t, const attn_pool* pools, int32_t n_pools,
                               int32_t* moved, void* ws, size_t ws_bytes, void* stream) {
  int st;
  if ((st = check_table(t)) != ATTN_OK ||
      (st = check_pools(pools, n_pools, t->num_pages)) != ATTN_OK ||
      (st = check_ws_bytes(ws, ws_bytes, attn_pages_workspace_size(t, 0))) != ATTN_OK)
    return static_cast<attn_status>(st);
  if (moved == nullptr && t->num_pages > 0)
    return static_cast<attn_status>(bad(ATTN_ERR_INVALID_ARG, "moved is NULL"));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Table d = dev_table(t, ws);
  const size_t P = static_cast<size_t>(t->num_pages);
  int32_t *holes = ints(ws, 0), *movers = ints(ws, P), *count = ints(ws, 2 * P);
  cudaError_t e = launch_pdl(compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, d, moved, holes,
                             movers, count);
  for (int i0 = 0; e == cudaSuccess && (i0 < n_pools || i0 == 0); i0 += kPoolsPerLaunch) {
    const Pools g = group(pools, n_pools, i0);
    // at most half of the pages move
    e = launch_pdl(compact_apply_kernel,
                   dim3(copy_grid((i0 == 0 ? t->rows : 0) + static_cast<int64_t>(P / 2) * g.pieces)),
                   dim3(kCopyThreads), 0, s, d, g, static_cast<const int32_t*>(moved),
                   static_cast<const int32_t*>(holes), static_cast<const int32_t*>(movers),
                   static_cast<const int32_t*>(count), i0 == 0 ? 1 : 0);
  }
  return static_cast<attn_status>(launched(e, "page compact launch"));
}

}  // extern "C"
