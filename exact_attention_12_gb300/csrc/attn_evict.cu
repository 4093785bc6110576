// Eviction from a paged cache by gathered attention weight.
//
// What it computes (include/attn.h): of a sequence of `old` keys that shrinks to
// `len`, each head keeps its last r = min(recent, len) keys and the len - r of the
// others that have the largest weights, in their order, at the front.
//
// Two kernels:
//   1. select, a cluster of CTAs per (sequence, head): the weights as 32-bit keys
//      in the order of the numbers; the (len - r)-th largest by three rounds of
//      counting digits (11, 11, 10 bits), every CTA its own part, the counts
//      added up through the cluster's shared memory; then where each kept key
//      goes, by ballots and running counts, and its weight with it.
//   2. move, in place.  Key j comes from slots[j] >= j, and slots ascends, so the
//      keys are moved in chunks of T: a CTA reads a chunk's rows of all pools
//      into shared memory, says so, waits until the chunks in front of it whose
//      rows lie where it writes have been read too, and writes.  Chunks are given
//      out by a ticket, front to back, so what a CTA waits for is always being
//      worked on, whichever CTAs are resident; a row is read and written once,
//      and what stays where it is is not touched.  Behind the chunks a ticket for
//      each sequence: once all its chunks have been read, its left-over pages go
//      back, its length and table follow.
//
// Bound: HBM, the moved rows twice and the weights once; on a short cache the
// two launches.
// Measured (8 heads, d = 128; 4 us of each are copies that put the state back): 32
// sequences of 2048-8192 bf16 keys to 4096, 656 MB moved (96 us at the copy rate), 149 us, of
// them 22 the selection; 4 of 95000 4-bit keys to 24000, 87 us, of them 26 the selection;
// one of 333 keys to 256, 14 us.  With a kernel of its own for the pages and the weights
// behind the new length: 156, 91, 16.
// The choice of variants goes by the room of the table and of the weights, as the lengths
// are on the device: the 32 sequences with room for 40960, 65536, 131072 keys take 155, 159,
// 172 us without those copies, 145 with room for their 8192 (slots are written as far as
// the weights reach; from 40961 on the weights stay in global memory and the moves take
// them along).  One sequence of 400000 keys to 100000, one head, d = 64: 123 us.
#include <climits>
#include <cstdio>

#include "attn.h"
#include "attn_kernels.cuh"
#include "attn_paged.cuh"

namespace attn {
using namespace sm103;

namespace {

constexpr int kSelectThreads = 512;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kMoveThreads = 256;
constexpr int kMoveBytes = 40960;         // of a chunk, all pools
constexpr int kMaxChunk = 512;            // keys of a chunk
constexpr int kMaxPools = 16;
constexpr uint64_t kTimeoutNs = 2000000000ull;

struct RowPool {
  char* base;
  int64_t page, head, row;   // bytes between pages, heads, rows
  int bytes;                 // of a row
  int unit;                  // bytes of one copy: 16, 8 or 4
  int shift;                 // log2 of the copies of a row, -1: no power of two
  int at;                    // where its rows begin in a chunk's buffer
};

struct EvictArgs {
  int32_t* table;
  int64_t table_stride;
  int32_t* lens;
  int32_t* refs;
  int rows, max_pages, page_shift, num_pages;
  int heads, n, recent, width;
  float* weights;
  int64_t weight_row, weight_head;
  const int32_t* seqs;
  const int32_t* new_lens;
  int32_t* slots;            // [n][heads][width]
  // workspace
  int32_t* old_len;          // [n]: -1 where nothing is done
  int32_t* new_len;          // [n]
  int32_t* ticket;
  int32_t* read;             // [n][heads][chunks]: the chunk's rows have been read
  int32_t* bound;            // [n][heads][chunks + 1]: kept keys before slot c T
  int chunk, chunk_shift;    // T, a power of two
  int chunks;                // of a row of the table
  int cluster;               // CTAs per (sequence, head) of the first kernel
  int n_pools;
  RowPool pools[kMaxPools];
  int buffer;                // bytes of a chunk, all pools
  int stall;                 // kStallEvictRead: see attn_debug_stall
  int* status;
  uint64_t timeout_ns;
};

__device__ void report(int* status, int code, int site) {
  if (atomicCAS(status, 0, code) == 0) atomicExch(status + 1, site);
}

__device__ __forceinline__ bool in_range(int i, int n) {
  return static_cast<unsigned>(i) < static_cast<unsigned>(n);
}

// A weight as an unsigned number of the same order; a NaN above all.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t b = __float_as_uint(w + 0.f);   // (-0 is 0)
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The weight of a key (-0 as 0, a NaN as a NaN).
__device__ __forceinline__ float weight_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// Entry i of the list: its sequence's length, and the new one; whether they hold
// together.  (Every thread by itself.)
__device__ __forceinline__ bool entry_lengths(const EvictArgs& a, int i, int* old, int* len) {
  const int s = a.seqs[i], want = a.new_lens[i];
  bool ok = in_range(s, a.rows) && want >= 0;
  *old = ok ? a.lens[s] : 0;
  ok = ok && *old >= 0 && *old <= static_cast<int64_t>(a.max_pages) << a.page_shift;
  if (!ok) *old = 0;
  *len = min(want, *old);
  return ok;
}

// Whether the sequence is named for the first time, and its pages are what they
// should be.  The whole CTA.
__device__ bool check_pages(const EvictArgs& a, int i, int old, int len) {
  const int s = a.seqs[i];
  bool ok = true;
  for (int j = threadIdx.x; j < i; j += kSelectThreads) ok = ok && a.seqs[j] != s;
  const int size = 1 << a.page_shift;
  const int held = (old + size - 1) >> a.page_shift;
  const int stay = len < old ? (len + size - 1) >> a.page_shift : 0;   // pages that are written
  const int32_t* row = a.table + s * a.table_stride;
  for (int j = threadIdx.x; j < held; j += kSelectThreads) {
    const int pg = row[j];
    ok = ok && in_range(pg, a.num_pages);
    if (ok) {
      const int refs = a.refs[pg];
      ok = j < stay ? refs == 1 : refs > 0;
    }
  }
  return __syncthreads_and(ok);
}

struct SelectShared {
  alignas(16) uint32_t bins[3][kBins];
  uint32_t sums[3][kBins / 32];
  uint32_t digit, left;              // the round's digit; how many are still to choose in it
  uint32_t above[kSelectWarps], equal[kSelectWarps];
  uint32_t cta_above, cta_equal;     // of this CTA's part, for the others
};

__device__ __forceinline__ uint32_t cluster_ld_u32(uint32_t addr) {
  uint32_t x;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(addr) : "memory");
  return x;
}

// CACHED: the CTA's part of the weights stays in shared memory, and the weights are
// moved from there.
template <bool CACHED>
__global__ void __launch_bounds__(kSelectThreads, 2) select_kernel(const EvictArgs a) {
  extern __shared__ __align__(16) uint32_t cache[];
  __shared__ SelectShared sh;
  grid_dep_wait();
  grid_dep_launch();
  const int C = a.cluster, rank = C > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int item = blockIdx.x / C, i = item / a.heads, h = item - i * a.heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int old, len;
  bool ok = entry_lengths(a, i, &old, &len);
  // this CTA's part of the slots: a multiple of 32 per warp
  const int per_warp = (old + C * kSelectThreads - 1) / (C * kSelectThreads) * 32;
  const int lo = rank * per_warp * kSelectWarps;
  const int part = max(0, min(per_warp * kSelectWarps, old - lo));
  float* w = ok ? a.weights + a.seqs[i] * a.weight_row + h * a.weight_head : nullptr;
  auto key_at = [&](int j) { return CACHED ? cache[j] : order_key(w[lo + j]); };
  for (int k = threadIdx.x; k < 3 * kBins; k += kSelectThreads) (&sh.bins[0][0])[k] = 0;
  if constexpr (CACHED) {
    if (len < old) {
#pragma unroll 8
      for (int j = threadIdx.x; j < part; j += kSelectThreads) cache[j] = order_key(w[lo + j]);
    }
  }
  ok = ok && check_pages(a, i, old, len);   // (and the CTA's keys are there)
  const bool first = h == 0 && rank == 0 && threadIdx.x == 0;
  if (first && !ok) report(a.status, kStatusPage, kSitePageIndex);
  if (first) {
    a.old_len[i] = ok && len < old ? old : -1;
    a.new_len[i] = len;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
  int32_t* slots = a.slots + static_cast<int64_t>(item) * a.width;
  const int all = C * kSelectThreads, me = rank * kSelectThreads + static_cast<int>(threadIdx.x);
  if (!ok || len == old) {   // (the same in all CTAs of the cluster)
    // (64 bits: `width` may be as large as 32 hold)
    for (int64_t j = me; j < a.width; j += all)
      slots[j] = ok ? (j < old ? static_cast<int32_t>(j) : -1) : -2;
    return;
  }
  const int chunks = (len + a.chunk - 1) / a.chunk;
  int32_t* read = a.read + static_cast<int64_t>(item) * a.chunks;
  int32_t* bound = a.bound + static_cast<int64_t>(item) * (a.chunks + 1);
  for (int c = me; c < chunks; c += all) read[c] = 0;
  const int r = min(a.recent, len), m = old - r;   // slots from m on stay
  uint32_t left = static_cast<uint32_t>(len - r);  // to be chosen of the m

  // the left-th largest key of slots [0, m): digit by digit from the top
  const int mine = max(0, min(part, m - lo));
  uint32_t prefix = 0;
  if (left > 0) {
#pragma unroll
    for (int round = 0; round < 3; ++round) {
      const int shift = round == 0 ? 21 : round == 1 ? 10 : 0;
      const int bits = round == 2 ? 10 : 11, known = round == 0 ? 32 : shift + bits;
      for (int j = threadIdx.x; j < mine; j += kSelectThreads) {
        const uint32_t k = key_at(j);
        if (known == 32 || (k >> known) == (prefix >> known))
          atomicAdd(&sh.bins[round][(k >> shift) & ((1u << bits) - 1u)], 1u);
      }
      __syncthreads();
      {   // sums of 32 bins, which are all that most of the search needs
        const uint4 x = *reinterpret_cast<const uint4*>(&sh.bins[round][4 * threadIdx.x]);
        uint32_t sum = x.x + x.y + x.z + x.w;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if ((lane & 7) == 0) sh.sums[round][threadIdx.x >> 3] = sum;
      }
      if (C > 1) cluster_sync();
      else __syncthreads();
      if (warp == 0) {
        // over the cluster: lane l has the sums 63 - 2 l and 62 - 2 l, then bin 31 - l of
        // the run that holds the digit
        auto over_cluster = [&](const uint32_t* at) {
          uint32_t got[kMaxCluster], n = 0;
#pragma unroll
          for (int q = 0; q < kMaxCluster; ++q)   // (all on their way before the first is used)
            got[q] = q >= C ? 0u : C > 1 ? cluster_ld_u32(cluster_addr(at, q)) : *at;
#pragma unroll
          for (int q = 0; q < kMaxCluster; ++q) n += got[q];
          return n;
        };
        auto inclusive = [&](uint32_t x) {
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
          }
          return x;
        };
        const uint32_t s0 = over_cluster(&sh.sums[round][63 - 2 * lane]);
        const uint32_t s1 = over_cluster(&sh.sums[round][62 - 2 * lane]);
        uint32_t end = inclusive(s0 + s1);
        bool here = end - s0 - s1 < left && left <= end;
        int from = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
        const bool second = left > end - s1;
        const int run = __shfl_sync(0xffffffffu, second ? 62 - 2 * lane : 63 - 2 * lane, from);
        const uint32_t rest = __shfl_sync(
            0xffffffffu, left - (end - s0 - s1) - (second ? s0 : 0u), from);
        const uint32_t n = over_cluster(&sh.bins[round][32 * run + 31 - lane]);
        end = inclusive(n);
        here = end - n < rest && rest <= end;
        if (here) {   // one lane
          sh.digit = static_cast<uint32_t>(32 * run + 31 - lane);
          sh.left = rest - (end - n);
        }
      }
      __syncthreads();
      prefix |= sh.digit << shift;
      left = sh.left;
    }
  }
  // kept: slots from m on, keys above `prefix`, and the first `left` that equal it
  const bool any = len > r;
  uint32_t above = 0, equal = 0;
  const int begin = warp * per_warp, stop = min(begin + per_warp, part);
  for (int j0 = begin; j0 < stop; j0 += 32) {
    const int j = j0 + lane;
    bool up = false, same = false;
    if (j < stop) {
      if (lo + j >= m) {
        up = true;
      } else if (any) {
        const uint32_t k = key_at(j);
        up = k > prefix;
        same = k == prefix;
      }
    }
    above += __popc(__ballot_sync(0xffffffffu, up));
    equal += __popc(__ballot_sync(0xffffffffu, same));
  }
  if (lane == 0) {
    sh.above[warp] = above;
    sh.equal[warp] = equal;
  }
  __syncthreads();
  above = equal = 0;   // of the warps before
  for (int q = 0; q < warp; ++q) {
    above += sh.above[q];
    equal += sh.equal[q];
  }
  if (C > 1) {
    if (threadIdx.x == kSelectThreads - 1) {
      sh.cta_above = above + sh.above[kSelectWarps - 1];
      sh.cta_equal = equal + sh.equal[kSelectWarps - 1];
    }
    cluster_sync();
    for (int q = 0; q < rank; ++q) {
      above += cluster_ld_u32(cluster_addr(&sh.cta_above, q));
      equal += cluster_ld_u32(cluster_addr(&sh.cta_equal, q));
    }
  }
  for (int j0 = begin; j0 < stop; j0 += 32) {
    const int j = j0 + lane;
    bool up = false, same = false;
    if (j < stop) {
      if (lo + j >= m) {
        up = true;
      } else if (any) {
        const uint32_t k = key_at(j);
        up = k > prefix;
        same = k == prefix;
      }
    }
    const uint32_t ups = __ballot_sync(0xffffffffu, up), sames = __ballot_sync(0xffffffffu, same);
    const uint32_t low = (1u << lane) - 1u;
    const uint32_t e = equal + __popc(sames & low);
    const int to = static_cast<int>(above + __popc(ups & low) + min(e, left));
    if (j < stop) {
      const int slot = lo + j;
      if (up || (same && e < left)) {
        slots[to] = slot;
        if (CACHED && to != slot) w[to] = weight_of(cache[j]);   // (all parts are read)
      }
      if ((slot & (a.chunk - 1)) == 0 && slot >> a.chunk_shift <= chunks)
        bound[slot >> a.chunk_shift] = to;
    }
    above += __popc(ups);
    equal += __popc(sames);
  }
  for (int c = (old + a.chunk - 1) / a.chunk + me; c <= chunks; c += all) bound[c] = len;
  for (int64_t j = len + me; j < a.width; j += all) slots[j] = -1;
  if constexpr (CACHED) {
    for (int j = len + me; j < old; j += all) w[j] = 0.f;
  }
  if (C > 1) cluster_sync();   // the others have read this CTA's counts
}

// (Rows lie scattered, and L2 fetches 128 bytes where it is not told otherwise: 4
// sequences of 95000 4-bit keys 98 us, with 64 bytes 92.)
__device__ __forceinline__ void copy_async(uint8_t* dst, const char* src, int unit) {
  const uint32_t d = smem_u32(dst);
  const uint64_t s = reinterpret_cast<uint64_t>(src);
  if (unit == 16) asm volatile("cp.async.cg.shared.global.L2::64B [%0], [%1], 16;" ::"r"(d), "l"(s) : "memory");
  else if (unit == 8) asm volatile("cp.async.ca.shared.global.L2::64B [%0], [%1], 8;" ::"r"(d), "l"(s) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d), "l"(s) : "memory");
}

// A chunk that has been looked up: where its keys come from and go to.
struct ChunkKeys {
  int page[2][kMaxChunk];    // of a key's old and new place
  int row[kMaxChunk];        // in the old page
  float weight[kMaxChunk];   // (WEIGHTS)
};
constexpr int kMoveEntries = 256;   // of the list that are kept at hand
struct MoveShared {
  ChunkKeys keys[2];
  int2 entries[kMoveEntries];       // new length (0: nothing to do), sequence
  int ticket, give_up;
};

// WEIGHTS: the weights are still where they were.
template <bool WEIGHTS>
__global__ void __launch_bounds__(kMoveThreads, 4) move_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ __align__(16) uint8_t buffer[];
  __shared__ MoveShared sh;
  grid_dep_wait();
  grid_dep_launch();
  const int T = a.chunk;
  auto entry_of = [&](int i) { return make_int2(a.old_len[i] < 0 ? 0 : a.new_len[i], a.seqs[i]); };
  int most = 0;
  for (int i = threadIdx.x; i < a.n; i += kMoveThreads) {
    const int2 entry = entry_of(i);
    if (i < kMoveEntries) sh.entries[i] = entry;
    most = max(most, (entry.x + T - 1) >> a.chunk_shift);
  }
  if (threadIdx.x == 0) sh.ticket = sh.give_up = 0;
  __syncthreads();
  atomicMax(&sh.ticket, most);
  __syncthreads();
  most = sh.ticket;
  const int items = a.n * a.heads;
  const int last = most * items;

  struct Chunk {
    int item, c, h, first, count;   // count 0: nothing to move; -1: entry `item` ends
    int from, until;                // chunks to wait for
    float* w;
  };
  // Looks chunk `ticket` up, into keys[buf].  One that stays where it is counts as
  // read.
  auto look_up = [&](int ticket, int buf) {
    Chunk k{};
    if (ticket >= last) {
      k.item = ticket - last;
      k.count = -1;
      return k;
    }
    k.c = ticket / items;
    k.item = ticket - k.c * items;
    const int i = k.item / a.heads;
    k.h = k.item - i * a.heads;
    const int2 entry = i < kMoveEntries ? sh.entries[i] : entry_of(i);
    k.first = k.c * T;
    const int count = min(T, entry.x - k.first);
    if (count <= 0) return k;
    const int32_t* slots = a.slots + static_cast<int64_t>(k.item) * a.width + k.first;
    const int32_t* bound = a.bound + static_cast<int64_t>(k.item) * (a.chunks + 1) + k.c;
    const int b0 = bound[0], b1 = bound[1];
    const int32_t* table = a.table + entry.y * a.table_stride;
    k.w = a.weights + entry.y * a.weight_row + k.h * a.weight_head;
    ChunkKeys& to = sh.keys[buf];
    for (int j = threadIdx.x; j < count; j += kMoveThreads) {
      const int from = slots[j];
      to.page[0][j] = table[from >> a.page_shift];
      to.page[1][j] = table[(k.first + j) >> a.page_shift];
      to.row[j] = from & ((1 << a.page_shift) - 1);
      if constexpr (WEIGHTS) {
        to.weight[j] = k.w[from];
      }
    }
    if (b1 == k.first + T) {   // every key so far is kept: it stays
      if (threadIdx.x == 0) a.read[static_cast<int64_t>(k.item) * a.chunks + k.c] = 1;
      return k;
    }
    k.count = count;
    k.from = b0 >> a.chunk_shift;
    k.until = min((b1 + T - 1) >> a.chunk_shift, k.c);
    return k;
  };
  auto row_of = [](const RowPool& pool, int e, int per) {
    return pool.shift >= 0 ? e >> pool.shift : e / per;
  };

  auto wait_read = [&](const volatile int32_t* flag) {
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1; *flag == 0; ++it)
      if ((it & 63u) == 0 && globaltimer_ns() - t0 > a.timeout_ns) {
        report(a.status, kStatusTimeout, kSiteEvictRead);
        sh.give_up = 1;
        return;
      }
  };
  // Entry i, all of whose chunks are taken: when they have been read, its pages behind
  // the new length go back.
  auto end_entry = [&](int i) {
    const int old = a.old_len[i], len = a.new_len[i], seq = a.seqs[i];
    if (old < 0) return;
    const int chunks = (len + T - 1) >> a.chunk_shift;
    for (int q = threadIdx.x; q < a.heads * chunks; q += kMoveThreads) {
      const int h = q / chunks;
      wait_read(a.read + (static_cast<int64_t>(i) * a.heads + h) * a.chunks + q - h * chunks);
    }
    __syncthreads();
    if (sh.give_up) return;
    const int size = 1 << a.page_shift;
    int32_t* row = a.table + seq * a.table_stride;
    const int held = (old + size - 1) >> a.page_shift;
    for (int j = ((len + size - 1) >> a.page_shift) + static_cast<int>(threadIdx.x); j < held;
         j += kMoveThreads) {
      atomicSub(&a.refs[row[j]], 1);   // (checked by the first kernel)
      row[j] = -1;
    }
    if (threadIdx.x == 0) a.lens[seq] = len;
    if constexpr (WEIGHTS) {
      for (int h = 0; h < a.heads; ++h) {
        float* w = a.weights + seq * a.weight_row + h * a.weight_head;
        for (int j = len + static_cast<int>(threadIdx.x); j < old; j += kMoveThreads) w[j] = 0.f;
      }
    }
  };

  // One chunk's rows are on their way while the next one is looked up.
  __syncthreads();
  if (threadIdx.x == 0) sh.ticket = atomicAdd(a.ticket, 1);
  __syncthreads();
  int ticket = sh.ticket;
  Chunk now = look_up(ticket, 0);
  for (int buf = 0; ticket < last + a.n; buf ^= 1) {
    __syncthreads();   // its keys are there; the buffer is free; sh.ticket has been read
    int next_ticket = 0;
    if (threadIdx.x == 0) next_ticket = atomicAdd(a.ticket, 1);
    const ChunkKeys& keys = sh.keys[buf];
    if (now.count > 0)
      for (int k = 0; k < a.n_pools; ++k) {
        const RowPool& pool = a.pools[k];
        const int per = pool.bytes / pool.unit;
        const char* base = pool.base + now.h * pool.head;
        for (int e = threadIdx.x; e < now.count * per; e += kMoveThreads) {
          const int j = row_of(pool, e, per), at = (e - j * per) * pool.unit;
          copy_async(buffer + pool.at + j * pool.bytes + at,
                     base + keys.page[0][j] * pool.page + keys.row[j] * pool.row + at, pool.unit);
        }
      }
    if (threadIdx.x == 0) sh.ticket = next_ticket;
    __syncthreads();
    ticket = sh.ticket;
    const Chunk next = look_up(ticket, buf ^ 1);
    if (now.count > 0) {
      copies_wait();
      __syncthreads();
      int32_t* read = a.read + static_cast<int64_t>(now.item) * a.chunks;
      // (The rows have arrived, so the flag needs no fence before it; and whoever
      // sees it set writes only after that.)
      // (An armed test stall: the first chunks never say so.)
      if (threadIdx.x == 0 && !(a.stall != 0 && now.c == 0)) atomicExch(read + now.c, 1);
      // chunks in front of this one that have rows where it writes
      for (int q = now.from + static_cast<int>(threadIdx.x); q < now.until; q += kMoveThreads)
        wait_read(read + q);
      __syncthreads();
      if (sh.give_up) break;
      for (int k = 0; k < a.n_pools; ++k) {
        const RowPool& pool = a.pools[k];
        const int per = pool.bytes / pool.unit;
        char* base = pool.base + now.h * pool.head;
        for (int e = threadIdx.x; e < now.count * per; e += kMoveThreads) {
          const int j = row_of(pool, e, per), at = (e - j * per) * pool.unit;
          char* to = base + keys.page[1][j] * pool.page +
                     ((now.first + j) & ((1 << a.page_shift) - 1)) * pool.row + at;
          const uint8_t* from = buffer + pool.at + j * pool.bytes + at;
          if (pool.unit == 16) *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(from);
          else if (pool.unit == 8) *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(from);
          else *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(from);
        }
      }
      if constexpr (WEIGHTS) {
        for (int j = threadIdx.x; j < now.count; j += kMoveThreads) now.w[now.first + j] = keys.weight[j];
      }
    } else if (now.count < 0) {
      end_entry(now.item);
      if (sh.give_up) break;
    }
    now = next;
  }
}

// --------------------------------------------------------------------- host --

constexpr size_t kHeader = 256;

int bad(int status, const char* msg) { return record_error(status, msg); }

int multiprocessors() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    sms = 148;
  return sms;
}

int check_evict(const attn_page_table* t, int32_t heads, int32_t n, const attn_rows* pools,
                int32_t n_pools) {
  if (t == nullptr) return bad(ATTN_ERR_INVALID_ARG, "page table is NULL");
  if (t->rows < 0 || t->max_pages < 0 || t->num_pages < 0 || heads < 0 || n < 0)
    return bad(ATTN_ERR_INVALID_ARG, "page table or list: negative size");
  if (t->page_size < 16 || t->page_size > 32768 || (t->page_size & (t->page_size - 1)) != 0)
    return bad(ATTN_ERR_INVALID_ARG, "page_size must be a power of two, 16 to 32768");
  if (static_cast<int64_t>(t->max_pages) * t->page_size > (int64_t{1} << 30))
    return bad(ATTN_ERR_UNSUPPORTED, "page table: more than 2^30 keys per row");
  if (t->table_stride < t->max_pages)
    return bad(ATTN_ERR_INVALID_ARG, "page table: table_stride < max_pages");
  if ((t->rows > 0 && t->max_pages > 0 && t->table == nullptr) ||
      (t->rows > 0 && t->lens == nullptr) || (t->num_pages > 0 && t->refs == nullptr))
    return bad(ATTN_ERR_INVALID_ARG, "page table: NULL pointer");
  // (a ticket counts chunks of at least one key over all heads and entries)
  if (static_cast<int64_t>(heads) * n >= (1 << 20))
    return bad(ATTN_ERR_UNSUPPORTED, "heads * n must stay below 2^20");
  if (n_pools < 0 || (n_pools > 0 && pools == nullptr))
    return bad(ATTN_ERR_INVALID_ARG, "pools: bad count or NULL");
  if (n_pools > kMaxPools) return bad(ATTN_ERR_UNSUPPORTED, "more than 16 pools");
  int64_t total = 0;
  for (int i = 0; i < n_pools; ++i) {
    const attn_rows& p = pools[i];
    if (p.reserved != 0) return bad(ATTN_ERR_INVALID_ARG, "pools: reserved field must be 0");
    if ((p.base == nullptr && t->num_pages > 0 && heads > 0) || (reinterpret_cast<uintptr_t>(p.base) & 3u) != 0 ||
        p.row_bytes <= 0 || p.row_bytes % 4 != 0 || p.page_stride % 4 != 0 ||
        p.head_stride % 4 != 0 || p.row_stride % 4 != 0 || p.page_stride < 0 ||
        p.head_stride < 0 || p.row_stride < p.row_bytes)
      return bad(ATTN_ERR_INVALID_ARG,
                 "pools: base, row_bytes and strides must be multiples of 4, rows apart");
    total += p.row_bytes;
  }
  if (total > 32768) return bad(ATTN_ERR_UNSUPPORTED, "pools: more than 32768 bytes a row");
  for (int i = 0; i < n_pools && heads > 0; ++i)
    if (!apart({{t->num_pages, pools[i].page_stride}, {heads, pools[i].head_stride},
                {t->page_size, pools[i].row_stride}}, pools[i].row_bytes))
      return bad(ATTN_ERR_INVALID_ARG, "pools: rows, heads and pages must lie apart");
  return ATTN_OK;
}

struct EvictLayout {
  int chunk, chunks, buffer;
  size_t old_len, new_len, ticket, read, bound, total;
};

EvictLayout evict_layout(const attn_page_table* t, int heads, int n, const attn_rows* pools,
                         int n_pools) {
  EvictLayout L{};
  int64_t bytes = 0, units = 0;
  for (int i = 0; i < n_pools; ++i) bytes += pools[i].row_bytes;
  L.chunk = kMaxChunk;
  while (L.chunk > 1 && L.chunk * bytes > kMoveBytes) L.chunk /= 2;
  const int64_t cap = static_cast<int64_t>(t->max_pages) * t->page_size;
  // fewer keys a chunk where that leaves SMs without one
  units = static_cast<int64_t>(heads) * n;
  while (L.chunk > 16 && units * ((cap + L.chunk - 1) / L.chunk) < 2 * multiprocessors()) L.chunk /= 2;
  L.chunks = static_cast<int>((cap + L.chunk - 1) / L.chunk);
  L.buffer = static_cast<int>(L.chunk * bytes) + 16 * n_pools;
  size_t at = kHeader;
  L.ticket = at;
  L.old_len = at += 4;
  L.new_len = at += 4 * static_cast<size_t>(n);
  L.read = at += 4 * static_cast<size_t>(n);
  L.bound = at += 4 * static_cast<size_t>(units) * L.chunks;
  L.total = at + 4 * static_cast<size_t>(units) * (static_cast<size_t>(L.chunks) + 1);
  return L;
}

// CTAs per (sequence, head) of the first kernel: as many as leave each some
// thousands of weights, while the GPU has room for them.  4096 / 1024 / 16384 weights: one
// sequence of 8192 keys 24.1 / 22.7 / 25.2 us, 4 of 16384 69 / 70 / 77.  Two CTAs an SM / one /
// six: 32 of 2048-8192 149 / 149 / 159, 4 of 95000 87 / 93 / 87.
int select_cluster(int64_t cap, int64_t items) {
  int c = 1;
  while (c < kMaxCluster && cap > 4096ll * c && items * c * 2 <= 2 * multiprocessors()) c *= 2;
  return c;
}

template <bool CACHED>
cudaError_t launch_select(const EvictArgs& a, size_t bytes, cudaStream_t s) {
  static std::atomic<uint64_t> set_up{0};
  int dev = 0;
  bool todo = false;
  cudaError_t e = needs_setup(set_up, &dev, &todo);
  if (e != cudaSuccess) return e;
  if (todo) {
    e = cudaFuncSetAttribute(select_kernel<CACHED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             192 * 1024);
    if (e != cudaSuccess) return e;
    mark_done(set_up, dev);
  }
  const dim3 grid(static_cast<unsigned>(a.n * a.heads * a.cluster));
  return launch_clusters(select_kernel<CACHED>, grid, dim3(kSelectThreads), bytes, a.cluster, s, a);
}

template <bool WEIGHTS>
cudaError_t launch_move(const EvictArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> set_up{0};
  int dev = 0;
  bool todo = false;
  cudaError_t e = needs_setup(set_up, &dev, &todo);
  if (e != cudaSuccess) return e;
  if (todo) {
    e = cudaFuncSetAttribute(move_kernel<WEIGHTS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMoveBytes + 16 * kMaxPools);
    if (e != cudaSuccess) return e;
    mark_done(set_up, dev);
  }
  const int64_t work = static_cast<int64_t>(a.n) * a.heads * a.chunks, room = 4ll * multiprocessors();
  return launch_pdl(move_kernel<WEIGHTS>, dim3(static_cast<unsigned>(work < room ? work : room)),
                    dim3(kMoveThreads), a.buffer, s, a);
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

size_t attn_pages_evict_workspace_size(const attn_page_table* t, int32_t heads, int32_t n,
                                       const attn_rows* pools, int32_t n_pools) {
  if (check_evict(t, heads, n, pools, n_pools) != ATTN_OK) return 0;
  return evict_layout(t, heads, n, pools, n_pools).total;
}

attn_status attn_pages_evict(const attn_page_table* t, const attn_rows* pools, int32_t n_pools,
                             int32_t heads, float* weights, int64_t weight_stride_row,
                             int64_t weight_stride_head, int32_t width, const int32_t* seqs,
                             const int32_t* new_lens, int32_t n, int32_t recent, int32_t* slots,
                             void* ws, size_t ws_bytes, void* stream) {
  const int st = check_evict(t, heads, n, pools, n_pools);
  if (st != ATTN_OK) return static_cast<attn_status>(st);
  if (recent < 0) return static_cast<attn_status>(bad(ATTN_ERR_INVALID_ARG, "recent is negative"));
  const int64_t cap = static_cast<int64_t>(t->max_pages) * t->page_size;
  if (width < cap || weight_stride_row < 0 || weight_stride_head < 0 ||
      !apart({{t->rows, weight_stride_row}, {heads, weight_stride_head}}, cap))
    return static_cast<attn_status>(bad(
        ATTN_ERR_INVALID_ARG,
        "weights: width or strides below max_pages * page_size, or rows and heads not apart"));
  const EvictLayout L = evict_layout(t, heads, n, pools, n_pools);
  if (static_cast<int64_t>(n) * heads * L.chunks >= (int64_t{1} << 30))
    return static_cast<attn_status>(bad(ATTN_ERR_UNSUPPORTED, "more than 2^30 chunks to move"));
  if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
    return static_cast<attn_status>(
        bad(ATTN_ERR_WORKSPACE, "workspace is NULL or not 256-byte aligned"));
  if (ws_bytes < L.total)
    return static_cast<attn_status>(bad(ATTN_ERR_WORKSPACE, "workspace too small"));
  if (n == 0 || heads == 0) return ATTN_OK;
  // (slots are written as far as `width`, without any page too)
  if (seqs == nullptr || new_lens == nullptr || (cap > 0 && weights == nullptr) ||
      (width > 0 && slots == nullptr))
    return static_cast<attn_status>(bad(ATTN_ERR_INVALID_ARG, "list, weights or slots is NULL"));
  char* w = static_cast<char*>(ws);
  auto ints = [&](size_t at) { return reinterpret_cast<int32_t*>(w + at); };
  EvictArgs a{};
  a.table = t->table;
  a.table_stride = t->table_stride;
  a.lens = t->lens;
  a.refs = t->refs;
  a.rows = t->rows;
  a.max_pages = t->max_pages;
  while ((1 << a.page_shift) < t->page_size) ++a.page_shift;
  a.num_pages = t->num_pages;
  a.heads = heads;
  a.n = n;
  a.recent = recent;
  a.width = width;
  a.weights = weights;
  a.weight_row = weight_stride_row;
  a.weight_head = weight_stride_head;
  a.seqs = seqs;
  a.new_lens = new_lens;
  a.slots = slots;
  a.old_len = ints(L.old_len);
  a.new_len = ints(L.new_len);
  a.ticket = ints(L.ticket);
  a.read = ints(L.read);
  a.bound = ints(L.bound);
  a.chunk = L.chunk;
  while ((1 << a.chunk_shift) < L.chunk) ++a.chunk_shift;
  a.chunks = L.chunks;
  a.buffer = L.buffer;
  a.cluster = select_cluster(cap, static_cast<int64_t>(n) * heads);
  a.n_pools = n_pools;
  int at = 0;
  for (int i = 0; i < n_pools; ++i) {
    const attn_rows& p = pools[i];
    const int64_t all = static_cast<int64_t>(reinterpret_cast<uintptr_t>(p.base)) | p.row_bytes |
                        p.page_stride | p.head_stride | p.row_stride;
    a.pools[i] = RowPool{static_cast<char*>(p.base), p.page_stride,
                         p.head_stride,              p.row_stride,
                         p.row_bytes,                all % 16 == 0 ? 16 : all % 8 == 0 ? 8 : 4,
                         -1,                 at};
    const int per = p.row_bytes / a.pools[i].unit;
    for (int x = 0; x < 16; ++x)
      if (per == 1 << x) a.pools[i].shift = x;
    at = (at + L.chunk * p.row_bytes + 15) / 16 * 16;
  }
  a.status = reinterpret_cast<int*>(ws);
  a.timeout_ns = kTimeoutNs;
  a.stall = take_stall(kStallEvictRead, &a.timeout_ns);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  // a CTA's part of the weights, if it fits
  const int64_t part = (cap + a.cluster * kSelectThreads - 1) / (a.cluster * kSelectThreads) *
                       kSelectThreads * 4;
  const bool cached = part <= 160 * 1024;
  cudaError_t e = cached ? launch_select<true>(a, static_cast<size_t>(part), s)
                         : launch_select<false>(a, 0, s);
  if (e == cudaSuccess && cap > 0) e = cached ? launch_move<false>(a, s) : launch_move<true>(a, s);
  if (e == cudaSuccess) return ATTN_OK;
  char msg[256];
  snprintf(msg, sizeof(msg), "page evict launch: %s", cudaGetErrorString(e));
  return static_cast<attn_status>(bad(ATTN_ERR_CUDA, msg));
}

}  // extern "C"
