// Kernel argument blocks, launchers and the work split of the kernels that
// read a paged key/value cache: the paged decode step (attn_paged.cu), its
// shared prefix (attn_prefix.cu) and the latent decode step (attn_latent.cu).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn_kernels.cuh"
#include "sm103_async.cuh"

namespace attn {

// Device status code of a page index outside the cache (equals ATTN_ERR_PAGE
// in attn.h).  The page reads as zeros.
constexpr int kStatusPage = 6;

// The split of a decode step over its CTAs.  The problem is a list of
// segments, one per (sequence, head group), sequence by sequence; a segment
// of n key tiles costs n + overhead units (its set-up and write-out, in
// tiles).  The units are dealt to the CTAs in equal runs (of all CTAs
// launched, or of fewer when the lengths leave less than MIN_UNITS each;
// the others return): every CTA gets the same share whatever the lengths are,
// and none waits for keys a short sequence does not have.  A segment that
// falls to one CTA is finished by it; one that is cut leaves a partial (O, L)
// per CTA, merged afterwards by the logsumexp rule.  A CTA cuts at most its
// first and its last segment, so it has two partial slots: slot 0 for a
// segment that began before the CTA's run, slot 1 for one that begins in it.
// The CTA that holds a cut segment's first tile leaves a note of the merge.
struct MergeNote {
  int b, h;      // the segment; b < 0: nothing to merge (per segment: more < 0)
  int slot;      // partial slot of the first piece, 2 CTA + 0 or 1; the next
                 // CTAs' pieces are in their slot 0
  int more;      // how many CTAs follow
};

// Where the caches are short there is nothing to balance, and the merge's own
// launch costs as much as the keys: then a segment falls to a cluster of CTAs,
// each takes an equal part of its tiles, and they merge through their shared
// memory (PagedArgs::cluster > 0; the notes and the partials stay unused).  Of
// many short ones each falls to one CTA, or (paged decode) to a part of one
// (cluster == 1).
struct PagedArgs {
  int B, H, heads;                // heads: segments per sequence, H_kv * blocks
  int blocks;                     // segments per key/value head (1 up to 64 query rows)
  int n_q, rows;                  // query rows per segment (the last of a head may have fewer)
  int head_rows, all_rows;        // of a key/value head, (H / H_kv) * n_q; of a sequence
  int causal, d;
  const int32_t* key_lens;        // [B]
  const int32_t* table;           // [B][table_stride]
  int64_t table_stride;
  int cap;                        // keys a row of the table can name
  int page_shift, num_pages;
  int first;                      // keys below it are left out (they are the shared prefix)
  float scale, scale_log2;        // c, c log2(e)
  const __nv_bfloat16* q;
  int64_t stride_b, stride_h, stride_n;      // q (and o, but for latent)
  __nv_bfloat16* o;
  float* lse;                     // [B][H][n_q]
  // latent: the cache, for copies that go without its tensor map
  const __nv_bfloat16* pages;
  int64_t stride_page;
  int dense;                      // a page's rows follow one another without gaps
  MergeNote* notes;               // workspace: one per segment, or one per CTA, as
  int by_segment;                 // fewer are (with a prefix always per segment)
  int cluster;                    // CTAs of a segment's cluster; 0: the work split above
  float* part_o;                  // workspace [2 G][rows][d]
  float* part_l;                  // workspace [2 G][rows]
  // a shared prefix: its pieces' partials and, behind them, those of the
  // segments that one CTA has finished (pre_splits = 0: no prefix)
  float* pre_o;                   // workspace [pre_splits + 1][B*H*n_q][d]
  float* pre_l;                   // workspace [pre_splits + 1][B*H*n_q]
  int pre_splits;
  int ctas;                       // G, the CTAs with partial slots
  int stall;                      // kStallPagedTile, kStallLatentSoftmax: see attn_debug_stall
  int* status;
  uint64_t timeout_ns;
};

// Whether the merges can follow a note.  A CTA whose wait has run out writes no
// more notes, and one whose shared memory is misaligned none at all; what the
// workspace holds in their place may be another call's.
__device__ __forceinline__ bool note_holds(const PagedArgs& a, const MergeNote& n) {
  return static_cast<unsigned>(n.b) < static_cast<unsigned>(a.B) &&
         static_cast<unsigned>(n.h) < static_cast<unsigned>(a.heads) &&
         static_cast<unsigned>(n.slot) < 2u * static_cast<unsigned>(a.ctas) && n.more >= -1 &&
         n.more < a.ctas - (n.slot >> 1);
}

// Where segment h of a sequence begins among the sequence's rows (head * n_q +
// query), and how many it has.
__device__ __forceinline__ int segment_row(const PagedArgs& a, int h) {
  const int head = h / a.blocks;
  return head * a.head_rows + (h - head * a.blocks) * a.rows;
}

__device__ __forceinline__ int segment_rows(const PagedArgs& a, int h) {
  return min(a.rows, a.head_rows - h % a.blocks * a.rows);
}

struct PrefixArgs {
  int B, H, H_kv, group, n_q, causal, d;
  const int32_t* key_lens;
  const int32_t* table;           // [B][table_stride]; the longest sequence's row names the prefix
  int64_t table_stride;
  int cap;                        // keys a row of the table can name
  int page_shift, num_pages;
  int shared_len;
  int splits, tiles;              // pieces of the prefix; 128-key tiles in all
  int rows;                       // B * group * n_q: query rows of one key/value head
  float scale, scale_log2;        // c, c log2(e)
  const __nv_bfloat16* q;
  int64_t stride_b, stride_h, stride_n;
  float* pre_o;
  float* pre_l;
  int stall;                      // kStallPrefixSoftmax: see attn_debug_stall
  int* status;
  uint64_t timeout_ns;
};

// The constants below were swept on whole steps.  Overhead (units a segment
// costs beside its tiles) 8 / 12, neither best throughout: 48 sequences of
// 250-1000 keys 30.8 / 31.5 us, 4 of 10000-20000 45.4 / 45.6, 16 of 4096-8192
// 70.9 / 70.6, 64 of 0-16384 with 32 rows 330 / 320, 2 of 30000 with 64 rows
// 27.2 / 24.3, a batch of short ones under a prefix 86.8 / 86.1.  8 is what the
// other constants were swept with.  Least share 6 or 9 units of 32 keys: one sequence of 517 keys 10.4 / 11.7 us; latent
// 2 / 3 / 6 units of 64: 13.6 / 15.1 / 21.3 us with 700 tokens.  Clusters: at
// most 24 / 48 key tiles a CTA (d = 128): 64 sequences of 200-800 keys 32.4 /
// 34.5 us; at most 4 / 8 latent tiles: 3000 tokens 13.0 / 15.9 us.  A segment
// to itself for a slot up to 16 / 32 tiles: 64 sequences of 250-1000 keys 37.6 /
// 41.0 us, of 125-500 keys 23.3 where 8 tiles give 25.8.
constexpr int kPagedKeys = 32;        // keys per tile of the paged decode kernel
constexpr int kPagedOverhead = 8;     // a segment's fixed cost in such tiles
constexpr int kPagedMinUnits = 6;     // units a CTA takes at least
constexpr int kLatentKeys = 64;       // keys per tile of the latent kernel
constexpr int kLatentOverhead = 2;
constexpr int kLatentMinUnits = 2;
constexpr int kPagedSoloTiles = 16;      // ... of a slot that has a segment to itself
constexpr int kPagedClusterTiles = 24;   // tiles of a cluster's CTA at most, at full caches
constexpr int kLatentClusterTiles = 4;
constexpr int kLatentRows = 64;       // query rows of one CTA
constexpr int kLatentRope = 64;       // columns of a latent vector that are not values

enum PagedSite : int {
  kSitePagedTile = 60, kSitePagedFree, kSitePrefixQ, kSitePrefixK, kSitePrefixV, kSitePrefixS,
  kSitePrefixP, kSitePrefixFree, kSitePrefixDone,
  kSiteLatentTile = 70, kSiteLatentS, kSiteLatentP, kSiteLatentFree, kSiteLatentDone, kSiteLatentQ,
  kSiteLatentSmem,
  kSitePageIndex = 80
};

// What the weights of a merge, e^(L_i - base), are taken against: the largest
// L_i, or 0 where all are -inf (no keys: the weights and partials are 0) or NaN
// (which fmaxf passes over, and the weights then carry).
__device__ __forceinline__ float merge_base(float top) { return top == -INFINITY ? 0.f : top; }

__device__ __forceinline__ int paged_len(const PagedArgs& a, int b) {
  return min(max(a.key_lens[b], 0), a.cap);
}

// Key tiles of one segment of sequence b.
template <int KEYS>
__device__ __forceinline__ int paged_tiles(const PagedArgs& a, int b) {
  const int n = paged_len(a, b) - a.first;
  return n > 0 ? (n + KEYS - 1) / KEYS : 0;
}

// The page that holds key `key` of a table row; an index outside the cache is
// recorded and read as the (all-zero) page past the last one.
__device__ __forceinline__ int checked_page(int page, int num_pages, int* status) {
  if (static_cast<unsigned>(page) < static_cast<unsigned>(num_pages)) return page;
  if (status != nullptr && atomicCAS(status, 0, kStatusPage) == 0)
    atomicExch(status + 1, kSitePageIndex);
  return max(num_pages, 1);   // (the tensor map of an empty cache has one page)
}

// A CTA's run [lo, hi) of the units, and where it starts.  (All units together
// are less than 2^31: the host sees to that.)
struct PagedShare {
  int lo, hi;
  int q;          // units of a CTA: q + 1 of the first `extra` CTAs, q of the others
  int extra, cta;
  int b;          // the sequence that holds unit lo
  int s;          // its first unit
  // The CTA whose run holds `unit`.
  __device__ __forceinline__ int owner(int unit) const {
    const int big = extra * (q + 1);
    return unit < big ? unit / (q + 1) : extra + (unit - big) / q;
  }
};

// Every warp by itself (each needs the answer, and barriers would cost more
// than the lengths that are read again).  Lane l adds up a run of consecutive
// sequences, the runs' sums are scanned, and the lane whose run holds unit lo
// walks it.
template <int KEYS, int OVERHEAD, int MIN_UNITS>
__device__ __forceinline__ PagedShare paged_share(const PagedArgs& a, int cta, int launched) {
  const int lane = threadIdx.x & 31;
  const int per = (a.B + 31) / 32;
  const int b0 = min(lane * per, a.B), b1 = min(b0 + per, a.B);
  int mine = 0;
#pragma unroll 4
  for (int b = b0; b < b1; ++b) mine += a.heads * (paged_tiles<KEYS>(a, b) + OVERHEAD);
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  const int total = __shfl_sync(0xffffffffu, inc, 31);
  PagedShare sh;
  const int ctas = max(1, min(launched, total / MIN_UNITS));
  sh.cta = cta;
  sh.q = total / ctas;
  sh.extra = total - sh.q * ctas;
  if (cta >= ctas) {   // (uniform over the CTA)
    sh.lo = sh.hi = sh.s = total;
    sh.b = a.B;
    return sh;
  }
  sh.lo = sh.q * cta + min(cta, sh.extra);
  sh.hi = sh.lo + sh.q + (cta < sh.extra ? 1 : 0);
  const bool here = inc - mine <= sh.lo && sh.lo < inc;
  int s = inc - mine, b = b0;
  if (here)
    for (; b + 1 < b1; ++b) {
      const int c = a.heads * (paged_tiles<KEYS>(a, b) + OVERHEAD);
      if (sh.lo < s + c) break;
      s += c;
    }
  const int from = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
  sh.b = __shfl_sync(0xffffffffu, b, from);
  sh.s = __shfl_sync(0xffffffffu, s, from);
  return sh;
}

// One CTA's piece of a segment: key tiles [t0, t1) of the n tiles of segment
// (b, h), whose first unit is s.
struct PagedPiece {
  int b, h, n, len;
  int s;
  int t0, t1;
  bool valid;
  // this CTA alone has the segment
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == n; }
};

template <int OVERHEAD>
__device__ __forceinline__ void paged_clip(PagedPiece& p, const PagedShare& sh) {
  const int first = p.s + OVERHEAD;   // unit of tile 0
  p.t0 = max(0, min(sh.lo - first, p.n));
  p.t1 = max(0, min(sh.hi - first, p.n));
}

// The first piece at or after segment (b, h) at unit s that gives this CTA
// something to do: tiles, or the rows of an empty segment that begins here.
template <int KEYS, int OVERHEAD>
__device__ __forceinline__ PagedPiece paged_piece(const PagedArgs& a, const PagedShare& sh, int b,
                                                  int h, int s) {
  PagedPiece p;
  p.valid = false;
  p.b = b;
  p.h = h;
  p.s = s;
  if (b >= a.B) return p;
  p.len = paged_len(a, b);
  p.n = paged_tiles<KEYS>(a, b);
  while (p.s < sh.hi) {
    paged_clip<OVERHEAD>(p, sh);
    if (p.t1 > p.t0 || (p.n == 0 && p.s >= sh.lo)) {
      p.valid = true;
      return p;
    }
    p.s += p.n + OVERHEAD;
    if (++p.h == a.heads) {
      p.h = 0;
      if (++p.b == a.B) return p;
      p.len = paged_len(a, p.b);
      p.n = paged_tiles<KEYS>(a, p.b);
    }
  }
  return p;
}

template <int KEYS, int OVERHEAD>
__device__ __forceinline__ PagedPiece paged_next(const PagedArgs& a, const PagedShare& sh,
                                                 const PagedPiece& p) {
  int b = p.b, h = p.h + 1;
  if (h == a.heads) {
    h = 0;
    ++b;
  }
  return paged_piece<KEYS, OVERHEAD>(a, sh, b, h, p.s + p.n + OVERHEAD);
}

// Part `rank` of `parts` of segment (b, h).
template <int KEYS>
__device__ __forceinline__ PagedPiece paged_part(const PagedArgs& a, int b, int h, int rank,
                                                 int parts) {
  PagedPiece p;
  p.b = b;
  p.h = h;
  p.len = paged_len(a, b);
  p.n = paged_tiles<KEYS>(a, b);
  p.s = 0;
  p.t0 = static_cast<int>(static_cast<int64_t>(p.n) * rank / parts);
  p.t1 = static_cast<int>(static_cast<int64_t>(p.n) * (rank + 1) / parts);
  p.valid = true;
  return p;
}

// The note of the merge that begins with piece p.
template <int OVERHEAD>
__device__ __forceinline__ MergeNote paged_note(const PagedShare& sh, const PagedPiece& p) {
  return MergeNote{p.b, p.h, 2 * sh.cta + (p.s < sh.lo ? 0 : 1),
                   sh.owner(p.s + OVERHEAD + p.n - 1) - sh.cta};
}

// launch_pdl with clusters of `cluster` CTAs.
template <typename... P, typename... A>
inline cudaError_t launch_clusters(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                                   unsigned cluster, cudaStream_t s, A&&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

cudaError_t launch_paged(const CUtensorMap& tk, const CUtensorMap& tv, const PagedArgs& a, int ctas,
                         cudaStream_t s);
cudaError_t launch_prefix(const CUtensorMap& tk, const CUtensorMap& tv, const PrefixArgs& a,
                          cudaStream_t s);
cudaError_t launch_latent(const CUtensorMap& tc, const PagedArgs& a, int ctas, cudaStream_t s);
cudaError_t launch_paged_merge(const PagedArgs& a, int notes, int ctas, cudaStream_t s);
cudaError_t launch_paged_finish(const PagedArgs& a, int ctas, cudaStream_t s);

// Whether attn_debug_stall armed `which` for this launch; then its wait limit.
bool take_stall(int which, uint64_t* limit_ns);

// Tensor map of a paged cache for the host code (an attn_status).
int encode_pages(CUtensorMap* map, const void* ptr, int num_pages, int heads, int page_size, int d,
                 int64_t stride_p, int64_t stride_h, int64_t stride_n, int box_rows);

}  // namespace attn
