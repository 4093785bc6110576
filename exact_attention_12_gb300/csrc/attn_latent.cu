// Decode step of latent attention in its absorbed form, against a paged cache
// of latent vectors.
//
// What it computes: all heads share one cached vector c_j a token, of
// d_v + 64 columns.  It is the key of every head as it stands, and its first
// d_v columns are the value (the per-head up-projections of keys and values
// are folded into the query and into what follows O):
//   S = scale * q c^T,  O = softmax(S) c[:, :d_v],  L = logsumexp(S),
// with the positions, masks and pages of the paged decode step.
//
// Bound: a token's 2 (d_v + 64) bytes serve 2 (2 d_v + 64) operations per
// query row: at d_v = 512 that is 1.9 rows operations a byte, so 16 heads are
// bound by HBM and 128 heads lie near the ridge (277): unlike the ordinary
// decode step this one needs the tensor cores at full width.
//
// Mapping.  The products are computed transposed, with keys and value
// columns as the 128-row side of the MMA and the query rows as its N:
//   S^T [64 keys x 64 rows]    = c  (K-major)  * q^T   36 MMAs at d_v = 512
//   O^T [d_v x 64 rows]       += c^T (MN-major) * P^T   16 MMAs a tile
// because the other way round the accumulator of 128 rows x 512 columns would
// fill TMEM, and q alone would take 147 KB of shared memory.  So O^T takes
// d_v / 128 * 64 TMEM columns, q 72 KB, and two 64-key tiles of 72 KB are in
// flight, each used as both operands.  H * n_q rows are cut into groups of 64;
// the CTAs of a sequence's groups run side by side on the same keys, of which
// each copies its own tiles (all but the first reading then comes from L2).
// The keys are divided over the CTAs as in the paged decode step.
//   warps 0-7  load q; softmax of 16 keys x 32 columns each, in the MMA's
//              fragment layout; the sums stay in registers, a partial per
//              thread, until the end; rescale O^T when some column's max has
//              grown by 2^8; write O
//   warp 8     copies (a lane per page)
//   warp 9     MMA issue: the scores of the next tile run under this tile's
//              softmax (it looks for whichever comes first, the tile or P)
// A tile is copied, waited for and released in groups of columns, so that its
// scores begin while the rest is on the way, and the next copies while its
// last products run: two 72 KB tiles are few for 1.6 us of latency.
// P is rounded to bf16 for the second product (relative 2^-8 per element);
// m, l, O are fp32.  Rows past the end of a sequence are zeroed in shared
// memory, by the softmax warps, before they are used as values (0 * NaN is NaN).
//
// Measured (d_v = 512, whole steps replayed from a CUDA graph): up to 64 rows
// the kernel streams at the copy rate once it runs (16 sequences, 16 heads:
// 16384 more tokens each cost 44 us = 6.8 TB/s); what remains is 12 us of
// set-up, first and last tiles and the merge (4096 tokens each: 23 us).  With
// 128 rows each tile is worked on by two CTAs, and shared memory bounds it: a
// tile's operand reads, its copy and P take 2600 cycles of its bandwidth, its
// MMAs 1900, and a tile takes 3100 (64 sequences of 4096-8192 tokens: 152 us,
// where the tokens' bytes need 69 and the operations 58).
#include "attn_paged.cuh"

namespace attn {
using namespace sm103;

namespace {

constexpr int kLooks = 4096;   // at two barriers in turn, before the wait (which is limited) for one

template <int DV>
struct LatentCfg {
  static constexpr int kCols = DV + kLatentRope;
  static constexpr int kBoxes = kCols / 64;               // 64-column boxes of a vector
  static constexpr int kBoxBytes = kLatentKeys * 128;
  static constexpr int kTileBytes = kBoxes * kBoxBytes;   // a key tile, and q
  static constexpr int kStages = DV == 512 ? 2 : 4;
  static constexpr int kBlocks = DV / 128;                // 128-row blocks of O^T
  // what is copied, waited for and released together: the 64 key-only columns
  // (group 0), then 128 columns = a block of O^T (groups 1 ..)
  static constexpr int kGroups = kBlocks + 1;
  // P^T of a tile takes the place of its key-only columns (64 keys x 64 rows of
  // bf16 either way): its scores are complete when P is written
  static constexpr int kPOffset = (kBoxes - 1) * kBoxBytes;
  static constexpr int kSmem = (1 + kStages) * kTileBytes;
  static constexpr int kCtl = 3 * 1024;                   // LatentCtl, in whole kilobytes
  static_assert(kSmem + kCtl <= 227 * 1024, "shared memory of a CTA");
  // warpgroups 0, 1: the eight warps of the softmax; warpgroup 2: copies, MMA
  // issue, two idle warps.  Registers re-split after the start: 256 * 208 +
  // 128 * 88 <= 384 * 168 (216 and 72: 16 sequences of 16384 tokens 58.1 against
  // 57.3 us).
  static constexpr int kThreads = 384;
  static constexpr uint32_t kRegsLaunch = 168;
  static constexpr uint32_t kRegsSoftmax = 208, kRegsOther = 88;
  static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= kThreads * kRegsLaunch,
                "register re-split exceeds the launch allocation");
  // S^T of tile t at 64 (t mod 2), block i of O^T at 128 + 64 i
  static constexpr uint32_t kOCol = 128;
};

// (aligned, so that what follows it, the dynamic shared memory, is too)
template <int ST>
struct __align__(1024) LatentCtl {
  // pfull, pvdone of tile T: [T mod 2], because the softmax may be done with
  // tile T + 1 before anyone has looked at tile T's (one barrier's phase would
  // then be two on, which a parity cannot tell from none)
  uint64_t full[ST][5], empty[ST][5], sfull[2], pfull[2], pvdone[2], qfull, final_bar;
  // [tile mod 2][16-key quarter][column]: the tile's maxima; behind the last
  // tile of a piece, in the buffer of the next, the columns' sums
  float wmax[2][4][64];
  float L[64];              // of the rows, for the cluster
  uint32_t tmem_base;
  int abort_flag;
};

// 16 TMEM lanes x 32 columns: thread 4 g + q receives, for i = 0 .. 15, row
// g + 8 ((i / 2) mod 2), column 8 (i / 4) + 2 q + i mod 2.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// How the keys are given out.
//   kAlone  the balanced split
//   kSeq    a sequence per cluster (a.cluster CTAs)
enum LatentMode { kAlone, kSeq };

template <int DV, LatentMode MODE>
__global__ void __launch_bounds__(LatentCfg<DV>::kThreads, 1)
    latent_kernel(const __grid_constant__ CUtensorMap tc, const PagedArgs a, int groups) {
  using C = LatentCfg<DV>;
  constexpr bool CLUSTER = MODE == kSeq;
  constexpr int ST = C::kStages, KT = kLatentKeys;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ LatentCtl<ST> ctl;
  static_assert(sizeof(LatentCtl<ST>) == C::kCtl, "the size that the limit is checked with");
  if ((smem_u32(smem) & 1023u) != 0) {   // swizzled tiles need 1024-byte alignment
    grid_dep_wait();
    if (threadIdx.x == 0 && atomicCAS(a.status, 0, kStatusSmemAlign) == 0)
      atomicExch(a.status + 1, kSiteLatentSmem);
    return;
  }
  uint8_t* sQ = smem;
  uint8_t* sC = smem + C::kTileBytes;

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  // row groups side by side; of clusters, the clusters
  const int unit = CLUSTER ? blockIdx.x / a.cluster : blockIdx.x;
  const int r0 = unit % groups * kLatentRows;   // first query row
  const int cta = unit / groups, ctas = gridDim.x / groups;
  const int rank = CLUSTER ? static_cast<int>(cluster_rank()) : 0;
  const int live = min(kLatentRows, a.all_rows - r0);

  if (threadIdx.x == 0) {
    ctl.abort_flag = 0;
    for (int s = 0; s < ST; ++s)
      for (int x = 0; x < C::kGroups; ++x) {
        mbar_init(&ctl.full[s][x], 1);
        mbar_init(&ctl.empty[s][x], 1);
      }
    mbar_init(&ctl.sfull[0], 1);
    mbar_init(&ctl.sfull[1], 1);
    mbar_init(&ctl.pfull[0], 8);
    mbar_init(&ctl.pfull[1], 8);
    mbar_init(&ctl.pvdone[0], 1);
    mbar_init(&ctl.pvdone[1], 1);
    mbar_init(&ctl.qfull, 8);
    mbar_init(&ctl.final_bar, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tc);
  }
  if (warp == 9) {
    tmem_alloc(&ctl.tmem_base, 512);
    tmem_relinquish();
  }
  // q's rows past the live ones stay zero; the maxima of a half without live
  // rows -inf (what its columns of P and O^T hold reaches no other column)
  for (int i = threadIdx.x; i < C::kTileBytes / 16; i += C::kThreads)
    reinterpret_cast<uint4*>(sQ)[i] = make_uint4(0u, 0u, 0u, 0u);
  for (int i = threadIdx.x; i < 512; i += C::kThreads) (&ctl.wmax[0][0][0])[i] = -INFINITY;
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_wait();
  grid_dep_launch();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl.tmem_base, 0);
  PagedShare share{};
  if constexpr (!CLUSTER)
    share = paged_share<KT, kLatentOverhead, kLatentMinUnits>(a, cta, ctas);
  const WaitCtx wc{&ctl.abort_flag, a.status, a.timeout_ns};
  PagedPiece p;
  if constexpr (CLUSTER) p = paged_part<KT>(a, cta, 0, rank, a.cluster);
  else p = paged_piece<KT, kLatentOverhead>(a, share, share.b, 0, share.s);
  auto next_of = [&](const PagedPiece& w) {
    PagedPiece x = w;
    if constexpr (CLUSTER) x.valid = false;
    else x = paged_next<KT, kLatentOverhead>(a, share, w);
    return x;
  };

  if (warp >= 8) {
    regs_decrease<C::kRegsOther>();
  if (warp == 8) {
    // ------------------------------------------------------------ copies
    const int rows = min(KT, 1 << a.page_shift), parts = KT / rows;
    bool ok = true;
    uint32_t T = 0;   // tiles issued, over all pieces
    PagedPiece nx = p;
    // Tile t of piece p, or past its end of the piece behind it, on its way to
    // L2: the two tiles in shared memory are too few to cover the latency of
    // HBM, and their copies go through a tile's memory 256 bytes of a token at
    // a time, where this reads it in one run.  (Two tiles ahead: 38.7 -> 40.4 us.)
    auto ahead = [&](int t) {
      int b = p.b, len = p.len;
      if (t >= p.t1) {
        if (!nx.valid) return;
        t += nx.t0 - p.t1;
        if (t >= nx.t1) return;
        b = nx.b;
        len = nx.len;
      }
      const int key = t * KT + lane * rows;
      if (lane >= parts || key >= len) return;
      const int page = a.table[b * a.table_stride + (key >> a.page_shift)];
      if (static_cast<unsigned>(page) < static_cast<unsigned>(a.num_pages))
        prefetch_l2(a.pages + page * a.stride_page + (key & ((1 << a.page_shift) - 1)) * C::kCols,
                    rows * C::kCols * 2);
    };
    // (the other row groups' CTAs read the same tiles)
    const bool fetch = a.dense && r0 == 0;
    for (; ok && p.valid; p = nx) {
      nx = next_of(p);
      const int32_t* row = a.table + p.b * a.table_stride;
      for (int t = p.t0; t < p.t1; ++t, ++T) {
        const int s = T % ST;
        const int key = t * KT + lane * rows;
        // a page past the sequence's end: the tile's first page in its place
        const int at = key < p.len ? key : t * KT;
        int page = 0;
        if (lane < parts) page = checked_page(row[at >> a.page_shift], a.num_pages, a.status);
        // the key-only columns last: P lies there until the last product
#pragma unroll
        for (int y = 1; y <= C::kGroups; ++y) {
          const int x = y % C::kGroups;
          if (T >= ST && !(ok = __all_sync(0xffffffffu, mbar_wait(&ctl.empty[s][x], ((T / ST) - 1) & 1,
                                                                  wc, kSiteLatentFree))))
            break;
          const int box = x == 0 ? C::kBoxes - 1 : 2 * (x - 1), boxes = x == 0 ? 1 : 2;
          if (lane == 0) mbar_arrive_expect_tx(&ctl.full[s][x], boxes * C::kBoxBytes);
          __syncwarp();
          if (lane < parts) {
            for (int k = box; k < box + boxes; ++k)
              tma_load_4d(sC + s * C::kTileBytes + k * C::kBoxBytes + lane * rows * 128, &tc,
                          &ctl.full[s][x], k * 64, at & ((1 << a.page_shift) - 1), 0, page);
          }
        }
        if (!ok) break;
        // (a CTA's first tiles themselves go out before any of this)
        if (fetch && T + 1 >= ST) ahead(t + 1);
      }
    }
    if (!ok && lane == 0)   // let issued copies land before the CTA exits
      for (uint32_t u = T > ST ? T - ST : 0; u <= T; ++u)   // (of tile T some groups, perhaps)
        for (int x = 0; x < C::kGroups; ++x)
          if (u < T || mbar_test(&ctl.empty[u % ST][x], ((u / ST) - 1) & 1))
            mbar_wait_drain(&ctl.full[u % ST][x], (u / ST) & 1, a.timeout_ns);
  } else if (warp == 9) {
    // --------------------------------------------------------- MMA issue
    // One elected lane issues, in code that the whole warp runs, from values
    // that are known to be the same in all its lanes (the shuffles): the
    // operands' descriptors then stay in uniform registers, and an MMA goes out
    // every 31 cycles (64 x 64 x 16) or 46 (128 x 64 x 16) instead of every 58.
    // Only as many of the 64 rows as live, in sixteens: 16 rows read 162 KB of
    // operands a tile instead of 245 (32 sequences of 0-8192 tokens 43.0 -> 41.9
    // us).
    const int wide = (live + 15) / 16 * 16;
    const uint32_t id_s = idesc_bf16(64, wide, false, false);
    const uint32_t id_o = idesc_bf16(128, wide, true, true);
    const bool one = elect_one_lane();
    const uint64_t dq = smem_desc(smem_u32(sQ), 16, 1024);
    bool ok = true;
    uint32_t T = 0;   // tiles before this piece
    int k = 0;        // pieces with tiles
    for (; ok && __shfl_sync(0xffffffffu, p.valid, 0);
         p = next_of(p)) {
      const int n = __shfl_sync(0xffffffffu, p.t1 - p.t0, 0);
      if (n == 0) continue;
      // S^T of the piece's tile i, group by group as they land
      // which groups of tile i have landed: all of them?
      auto landed = [&](int i) {
        const uint32_t u = T + i;
        const bool all = __all_sync(0xffffffffu, lane >= C::kGroups ||
                                                     mbar_test(&ctl.full[u % ST][lane], (u / ST) & 1));
        __syncwarp();   // what these lanes have seen the issuing lane may use
        return all;
      };
      auto scores = [&](int i, bool all) {
        const uint32_t u = T + i, s = u % ST;
        uint8_t* tile = sC + s * C::kTileBytes;
        const uint64_t dc = smem_desc(smem_u32(tile), 16, 1024);
#pragma unroll
        for (int y = 1; y <= C::kGroups; ++y) {
          const int x = y % C::kGroups;
          if (!all) {
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(&ctl.full[s][x], (u / ST) & 1, wc,
                                                         kSiteLatentTile))))
              return;
            tc_fence_after();
          }
          const int box = x == 0 ? C::kBoxes - 1 : 2 * (x - 1), boxes = x == 0 ? 1 : 2;
          if (one) {
#pragma unroll
            for (int kk = 4 * box; kk < 4 * (box + boxes); ++kk) {
              const uint64_t off =
                  static_cast<uint64_t>(((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4);
              mma_ss(tmem + 64 * (u & 1), dc + off, dq + off, id_s, x != 1 || kk > 0 ? 1u : 0u);
            }
          }
        }
        if (one) mma_commit(&ctl.sfull[u & 1]);
        __syncwarp();
      };
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&ctl.qfull, k & 1, wc, kSiteLatentQ)))) break;
      tc_fence_after();
      scores(0, landed(0));
      for (int i = 0; ok && i < n; ++i) {
        // the next tile's scores first if it lands before P is there
        const uint32_t u = T + i, s = u % ST;
        bool next = i + 1 < n;
        for (int looks = 0; next && looks < kLooks; ++looks) {
          if (landed(i + 1)) {
            scores(i + 1, true);
            next = false;
          } else if (__all_sync(0xffffffffu, mbar_test(&ctl.pfull[u & 1], (u >> 1) & 1))) {
            break;
          }
        }
        if (!ok || !(ok = __all_sync(0xffffffffu, mbar_wait(&ctl.pfull[u & 1], (u >> 1) & 1, wc,
                                                            kSiteLatentP))))
          break;
        tc_fence_after();
        const uint64_t dp = smem_desc(smem_u32(sC + s * C::kTileBytes + C::kPOffset), 16, 1024);
#pragma unroll
        for (int blk = 0; blk < C::kBlocks; ++blk) {   // O^T += c^T P^T, 128 value columns at a time
          const uint64_t dv = smem_desc(smem_u32(sC + s * C::kTileBytes + 2 * blk * C::kBoxBytes),
                                        C::kBoxBytes, 1024);
          if (one) {
#pragma unroll
            for (int kk = 0; kk < KT / 16; ++kk) {
              const uint64_t off = static_cast<uint64_t>((kk * 2048) >> 4);
              mma_ss(tmem + C::kOCol + 64 * blk, dv + off, dp + off, id_o, i > 0 || kk > 0 ? 1u : 0u);
            }
            mma_commit(&ctl.empty[s][1 + blk]);
          }
        }
        if (one) {
          mma_commit(&ctl.pvdone[u & 1]);
          mma_commit(&ctl.empty[s][0]);
        }
        __syncwarp();
        if (next) scores(i + 1, false);
      }
      T += n;
      ++k;
    }
    if (one) {
      mma_commit(&ctl.final_bar);   // every MMA of this CTA done before TMEM is freed
      mbar_wait_drain(&ctl.final_bar, 0, a.timeout_ns);
    }
    __syncwarp();
  }
  } else {
    regs_increase<C::kRegsSoftmax>();
    // ------------------------------------------- q, softmax, rescale, output
    // softmax: 16 keys and 32 of the columns a warp, in the MMA's fragment
    // layout: keys g, g + 8 and columns 8 b + 2 q, + 1 (b = 0 .. 3) a thread
    const int quad = warp & 3, half = warp >> 2;
    const bool soft = half == 0 || live > 32;
    const int g = lane >> 2, q4 = lane & 3;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float c2 = a.scale_log2;
    bool ok = true;
    uint32_t T = 0;
    MergeNote note{-1, 0, 0, 0};
    // q rows r0 .. of the piece's sequence, K-major (asynchronous copies: all
    // are in flight together)
    auto load_q = [&](const PagedPiece& w) {
      if (!w.valid || w.t0 == w.t1) return;
      for (int r = warp; r < live; r += 8) {
        const int h = (r0 + r) / a.n_q, qt = (r0 + r) - h * a.n_q;
        const __nv_bfloat16* src = a.q + w.b * a.stride_b + h * a.stride_h +
                                   static_cast<int64_t>(qt) * a.stride_n;
        for (int c = lane; c < C::kBoxes * 8; c += 32)
          copy16_async(sQ + (c >> 3) * C::kBoxBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                       src + c * 8, true);
      }
    };
    auto q_ready = [&](const PagedPiece& w) {
      if (!w.valid || w.t0 == w.t1) return;
      copies_wait();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.qfull);
    };
    load_q(p);
    q_ready(p);
    for (PagedPiece nx = p; p.valid; p = nx) {
      nx = next_of(p);
      const int n = p.t1 - p.t0;
      float mref[2] = {-INFINITY, -INFINITY};   // columns lane, lane + 32: reference maxima
      float mc[8], l[8];                        // softmax: this thread's columns
#pragma unroll
      for (int j = 0; j < 8; ++j) mc[j] = l[j] = 0.f;
      const int open = a.causal ? p.len - a.n_q + 1 : p.len;   // every row is allowed keys below it
      for (int i = 0; i < n; ++i, ++T) {
        const int buf = T & 1;
        uint32_t sr[16];
        if (soft) {
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&ctl.sfull[buf], (T >> 1) & 1, wc,
                                                         kSiteLatentS));
          tc_fence_after();
          tmem_ld_16x32(tmem + lanes + 64 * buf + 32 * half, sr);
          tmem_wait_ld();
          const int k0 = (p.t0 + i) * KT;
          if (k0 + KT > open) {
            const int kj = k0 + 16 * quad + g;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int qt = (r0 + 32 * half + 8 * (j >> 2) + 2 * q4 + (j & 1)) % a.n_q;
              const int lim = a.causal ? p.len - a.n_q + qt + 1 : p.len;
              if (kj + 8 * ((j >> 1) & 1) >= lim) sr[j] = __float_as_uint(-INFINITY);
            }
          }
          float top[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int at = 4 * (j >> 1) + (j & 1);
            top[j] = fmaxf(__uint_as_float(sr[at]), __uint_as_float(sr[at + 2]));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1)
              top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], o));
          }
          if (g == 0) {
#pragma unroll
            for (int b = 0; b < 4; ++b)
              *reinterpret_cast<float2*>(&ctl.wmax[buf][quad][32 * half + 8 * b + 2 * q4]) =
                  make_float2(top[2 * b], top[2 * b + 1]);
          }
        }
        named_barrier_sync(1, 256);
        // (the tile's scores are complete) what lies past the sequence's end: zero,
        // before it is used as value rows
        const int from = p.len - (p.t0 + i) * KT;
        if (from < KT) {
          uint8_t* tile = sC + (T % ST) * C::kTileBytes;
          for (int e = threadIdx.x; e < (KT - from) * (DV / 8); e += 256) {
            const int j = from + e / (DV / 8), c = e % (DV / 8);
            *reinterpret_cast<uint4*>(tile + (c >> 3) * C::kBoxBytes + j * 128 + ((c & 7) << 4)) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        float alpha[2];
        bool grown[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float x = fmaxf(fmaxf(ctl.wmax[buf][0][lane + 32 * e], ctl.wmax[buf][1][lane + 32 * e]),
                                fmaxf(ctl.wmax[buf][2][lane + 32 * e], ctl.wmax[buf][3][lane + 32 * e]));
          grown[e] = x > mref[e] && (mref[e] == -INFINITY || (x - mref[e]) * c2 > kRescaleTau);
          alpha[e] = grown[e] ? ex2_approx((mref[e] - x) * c2) : 1.f;
          if (grown[e]) mref[e] = x;
        }
        const bool rescale = __any_sync(0xffffffffu, grown[0] || grown[1]);   // alike in every warp
        if (rescale) {
          if (soft) {
            const float al = half ? alpha[1] : alpha[0], mr = half ? mref[1] : mref[0];
            const float mrc = mr == -INFINITY ? 0.f : mr * c2;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int from = 8 * (j >> 1) + 2 * q4 + (j & 1);
              l[j] *= __shfl_sync(0xffffffffu, al, from);
              mc[j] = __shfl_sync(0xffffffffu, mrc, from);
            }
          }
          if (i > 0) {
            if (ok)   // O^T holds the sum through the tile before
              ok = __all_sync(0xffffffffu, mbar_wait(&ctl.pvdone[(T - 1) & 1], ((T - 1) >> 1) & 1, wc,
                                                     kSiteLatentDone));
            tc_fence_after();
#pragma unroll
            for (int bb = 0; bb < C::kBlocks / 2; ++bb) {
              const uint32_t col = tmem + lanes + C::kOCol + 64 * (half * (C::kBlocks / 2) + bb);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                uint32_t o[32];
                tmem_ld32(col + 32 * e, o);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  o[j] = __float_as_uint(__uint_as_float(o[j]) * __shfl_sync(0xffffffffu, alpha[e], j));
                tmem_st32(col + 32 * e, o);
              }
            }
            tmem_wait_st();
          }
        }
        if (soft) {   // P^T: two columns of keys g and g + 8 at a time
#pragma unroll
          for (int b = 0; b < 4; ++b) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int row = 16 * quad + g + 8 * e;
              const float p0 = ex2_approx(fmaf(__uint_as_float(sr[4 * b + 2 * e]), c2, -mc[2 * b]));
              const float p1 =
                  ex2_approx(fmaf(__uint_as_float(sr[4 * b + 2 * e + 1]), c2, -mc[2 * b + 1]));
              l[2 * b] += p0;
              l[2 * b + 1] += p1;
              *reinterpret_cast<uint32_t*>(sC + (T % ST) * C::kTileBytes + C::kPOffset + row * 128 +
                                           (((4 * half + b) ^ (row & 7)) << 4) + 4 * q4) =
                  pack_bf16x2(p0, p1);
            }
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        // (an armed test stall: warp 0 withholds its first arrive, so the MMA
        // warp's wait runs out)
        if (lane == 0 && !(a.stall != 0 && warp == 0 && T == 0)) mbar_arrive(&ctl.pfull[buf]);
      }

      // ---- O = O^T / l and L of the piece; every score MMA of the piece is
      // complete (a warp waited for the last before the last barrier), so the
      // next piece's q can come
      load_q(nx);
      if (n > 0 && soft) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) l[j] += __shfl_xor_sync(0xffffffffu, l[j], o);
        if (g == 0) {
#pragma unroll
          for (int b = 0; b < 4; ++b)
            *reinterpret_cast<float2*>(&ctl.wmax[T & 1][quad][32 * half + 8 * b + 2 * q4]) =
                make_float2(l[2 * b], l[2 * b + 1]);
        }
      }
      if (n > 0 && ok) {
        ok = __all_sync(0xffffffffu, mbar_wait(&ctl.pvdone[(T - 1) & 1], ((T - 1) >> 1) & 1, wc,
                                                     kSiteLatentDone));
        tc_fence_after();
      }
      named_barrier_sync(1, 256);
      float inv[2], L[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float(*sum)[64] = ctl.wmax[T & 1];
        const int c = lane + 32 * e;
        const float s = n > 0 ? (sum[0][c] + sum[1][c]) + (sum[2][c] + sum[3][c]) : 0.f;
        inv[e] = s != 0.f ? 1.f / s : 0.f;
        L[e] = s != 0.f ? fmaf(mref[e], a.scale, logf(s)) : -INFINITY;
      }
      // the next piece's scores can run under the write-out (its maxima go where
      // the sums were: those are read)
      q_ready(nx);
      const bool whole = !CLUSTER && p.whole();
      if constexpr (!CLUSTER) {
        if (p.t0 == 0 && !whole) note = paged_note<kLatentOverhead>(share, p);
        if (a.by_segment && p.t0 == 0 && threadIdx.x == 0 && r0 == 0)
          a.notes[p.b] = whole ? MergeNote{p.b, 0, 0, -1} : note;
      }
      const int64_t part = 2 * static_cast<int64_t>(cta) + (p.s < share.lo ? 0 : 1);
      if (warp == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = r0 + lane + 32 * e;
          if (lane + 32 * e < live) {
            if (CLUSTER) ctl.L[lane + 32 * e] = L[e];
            else if (whole) a.lse[static_cast<int64_t>(p.b) * a.all_rows + r] = L[e];
            else a.part_l[part * a.rows + r] = L[e];
          }
        }
      }
#pragma unroll
      for (int bb = 0; bb < C::kBlocks / 2; ++bb) {
        const int blk = half * (C::kBlocks / 2) + bb;
        const int dim = 128 * blk + (warp & 3) * 32 + lane;
        // 16 rows (columns of O^T) at a time
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (16 * e >= live) break;
          uint32_t o[16];
          if (n > 0) {
            tmem_ld16(tmem + lanes + C::kOCol + 64 * blk + 16 * e, o);
            tmem_wait_ld();
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float w = __shfl_sync(0xffffffffu, inv[e >> 1], 16 * (e & 1) + j);
            o[j] = n > 0 && w != 0.f ? __float_as_uint(__uint_as_float(o[j]) * w) : 0u;
          }
          if (whole) {
            // lanes 2 i, 2 i + 1 trade: the even one stores its two columns of
            // row j, the odd one those of row j + 1
            __nv_bfloat16* to = a.o + (static_cast<int64_t>(p.b) * a.all_rows + r0 + 16 * e) * DV +
                                (dim & ~1);
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const uint32_t give = (lane & 1) ? o[j] : o[j + 1];
              const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 1);
              const uint32_t v = (lane & 1) ? pack_bf16x2(__uint_as_float(got), __uint_as_float(o[j + 1]))
                                            : pack_bf16x2(__uint_as_float(o[j]), __uint_as_float(got));
              const int r = j + (lane & 1);
              if (16 * e + r < live) *reinterpret_cast<uint32_t*>(to + r * DV) = v;
            }
          } else {
            // (a cluster's CTA: to where its tiles were)
            float* to = CLUSTER ? reinterpret_cast<float*>(sC) + 16 * e * DV + dim
                                : a.part_o + (part * a.rows + r0 + 16 * e) * DV + dim;
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (16 * e + j < live) to[j * DV] = __uint_as_float(o[j]);
          }
        }
      }
      tc_fence_before();
    }
    if (!CLUSTER && !a.by_segment && threadIdx.x == 0 && r0 == 0) a.notes[cta] = note;
  }
  if constexpr (CLUSTER) {
    // the cluster's rows merged: each CTA writes a part of the items
    static_assert(kLatentRows * DV * 4 <= ST * C::kTileBytes, "a CTA's O fits where its tiles were");
    __syncwarp();
    cluster_sync();
    const float* o = reinterpret_cast<const float*>(sC);
    for (int e = rank * C::kThreads + threadIdx.x; e < live * (DV / 4);
         e += a.cluster * C::kThreads) {
      const int r = e / (DV / 4), c = 4 * (e - r * (DV / 4));
      float top = -INFINITY, sum = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
      for (int k = 0; k < a.cluster; ++k) top = fmaxf(top, cluster_ld(cluster_addr(&ctl.L[r], k)));
      top = merge_base(top);
      for (int k = 0; k < a.cluster; ++k) {
        float y[4];
        cluster_ld4(cluster_addr(o + r * DV + c, k), y);
        const float w = __expf(cluster_ld(cluster_addr(&ctl.L[r], k)) - top);
        sum += w;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = fmaf(w, y[i], x[i]);
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const int64_t row = static_cast<int64_t>(cta) * a.all_rows + r0 + r;
      *reinterpret_cast<uint2*>(a.o + row * DV + c) =
          make_uint2(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv));
      if (c == 0) a.lse[row] = sum == 0.f ? -INFINITY : top + logf(sum);
    }
    cluster_sync();   // the others have read this CTA's rows
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int DV, LatentMode MODE>
cudaError_t launch_dv(const CUtensorMap& tc, const PagedArgs& a, int ctas, cudaStream_t s) {
  using C = LatentCfg<DV>;
  static std::atomic<uint64_t> set_up{0};
  int dev = 0;
  bool todo = false;
  cudaError_t e = needs_setup(set_up, &dev, &todo);
  if (e != cudaSuccess) return e;
  if (todo) {
    e = cudaFuncSetAttribute(latent_kernel<DV, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::kSmem);
    if (e != cudaSuccess) return e;
    // the register re-split inside the kernel assumes the launch allocation
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, latent_kernel<DV, MODE>)) != cudaSuccess) return e;
    if (static_cast<uint32_t>(fa.numRegs) < C::kRegsLaunch) return cudaErrorInvalidConfiguration;
    mark_done(set_up, dev);
  }
  const int groups = a.rows / kLatentRows;
  if (MODE == kSeq)
    return launch_clusters(latent_kernel<DV, MODE>,
                           dim3(static_cast<unsigned>(a.B * groups * a.cluster)), dim3(C::kThreads),
                           C::kSmem, a.cluster, s, tc, a, groups);
  return launch_pdl(latent_kernel<DV, MODE>, dim3(ctas * groups), dim3(C::kThreads), C::kSmem, s,
                    tc, a, groups);
}

}  // namespace

cudaError_t launch_latent(const CUtensorMap& tc, const PagedArgs& a, int ctas, cudaStream_t s) {
  const bool wide = a.d == 512;
  if (a.cluster > 0)
    return wide ? launch_dv<512, kSeq>(tc, a, ctas, s) : launch_dv<256, kSeq>(tc, a, ctas, s);
  return wide ? launch_dv<512, kAlone>(tc, a, ctas, s) : launch_dv<256, kAlone>(tc, a, ctas, s);
}

}  // namespace attn
