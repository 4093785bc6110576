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
// flight, each read from global memory once and used as both operands.  (The
// MMA of S^T has M = 128: its rows 64-127 are whatever lies behind the tile,
// and nothing reads them.)  H * n_q rows are cut into groups of 64; the CTAs
// of a sequence's groups run side by side on the same keys, so that the
// second read of a tile finds it in L2.  The keys are divided over the CTAs
// as in the paged decode step.
//   warps 0, 1, 4, 5   softmax: thread = key, 32 of the 64 columns each; a
//                      column's max is a warp reduction; the row sums stay in
//                      registers, a partial per key lane, until the end
//   warps 0-7          load q, rescale O^T when some column's max has grown
//                      by 2^8, write O
//   warp 8             copies (a lane per page), warp 9 MMA issue: the scores of
//                      the next tile run under this tile's softmax
// P is rounded to bf16 for the second product (relative 2^-8 per element);
// m, l, O are fp32.  Rows past the end of a sequence are zeroed in shared
// memory before they are used as values (0 * NaN is NaN).
#include "attn_paged.cuh"

namespace attn {
using namespace sm103;

namespace {

constexpr float kLn2 = 0.693147180559945309f;

template <int DV>
struct LatentCfg {
  static constexpr int kCols = DV + kLatentRope;
  static constexpr int kBoxes = kCols / 64;               // 64-column boxes of a vector
  static constexpr int kBoxBytes = kLatentKeys * 128;
  static constexpr int kTileBytes = kBoxes * kBoxBytes;   // a key tile, and q
  static constexpr int kStages = DV == 512 ? 2 : 4;
  static constexpr int kBlocks = DV / 128;                // 128-row blocks of O^T
  static constexpr int kPBytes = kLatentKeys * 128;
  static constexpr int kSmem = 1024 + (1 + kStages) * kTileBytes + kPBytes;
  static constexpr int kThreads = 320;
  // S^T of tile t at 64 (t mod 2), block i of O^T at 128 + 64 i
  static constexpr uint32_t kOCol = 128;
};

template <int ST>
struct LatentCtl {
  uint64_t full[ST], empty[ST], sfull[2], pfull, pvdone, qfull, final_bar;
  float wmax[2][2][64];     // [tile mod 2][32-key half][column]
  float lsum[2][64];
  int64_t sums[10];
  PagedShare share;
  uint32_t tmem_base;
  int abort_flag;
};

__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

template <int DV>
__global__ void __launch_bounds__(LatentCfg<DV>::kThreads, 1)
    latent_kernel(const __grid_constant__ CUtensorMap tc, const PagedArgs a, int groups) {
  using C = LatentCfg<DV>;
  constexpr int ST = C::kStages, KT = kLatentKeys;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sC = smem + C::kTileBytes;
  uint8_t* sP = sC + ST * C::kTileBytes;
  __shared__ LatentCtl<ST> ctl;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r0 = static_cast<int>(blockIdx.x % groups) * kLatentRows;   // first query row
  const int cta = blockIdx.x / groups, ctas = gridDim.x / groups;
  const int live = min(kLatentRows, a.all_rows - r0);

  if (threadIdx.x == 0) {
    ctl.abort_flag = 0;
    for (int s = 0; s < ST; ++s) {
      mbar_init(&ctl.full[s], 1);
      mbar_init(&ctl.empty[s], 1);
    }
    mbar_init(&ctl.sfull[0], 1);
    mbar_init(&ctl.sfull[1], 1);
    mbar_init(&ctl.pfull, 8);
    mbar_init(&ctl.pvdone, 1);
    mbar_init(&ctl.qfull, 8);
    mbar_init(&ctl.final_bar, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tc);
  }
  if (warp == 9) {
    tmem_alloc(&ctl.tmem_base, 512);
    tmem_relinquish();
  }
  // P's columns past the live rows stay zero; their maxima -inf
  for (int i = threadIdx.x; i < C::kPBytes / 16; i += C::kThreads)
    reinterpret_cast<uint4*>(sP)[i] = make_uint4(0u, 0u, 0u, 0u);
  for (int i = threadIdx.x; i < 256; i += C::kThreads) (&ctl.wmax[0][0][0])[i] = -INFINITY;
  for (int i = threadIdx.x; i < 128; i += C::kThreads) (&ctl.lsum[0][0])[i] = 0.f;
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_wait();
  grid_dep_launch();
  const uint32_t tmem = ctl.tmem_base;
  const PagedShare share =
      paged_share<C::kThreads, KT, kLatentOverhead>(a, cta, ctas, ctl.sums, &ctl.share);
  if (blockIdx.x == 0 && threadIdx.x == 0) a.starts[a.B] = share.total;
  const WaitCtx wc{&ctl.abort_flag, a.status, a.timeout_ns};
  PagedPiece p = paged_piece<KT, kLatentOverhead>(a, share, share.b, 0, share.s,
                                                  threadIdx.x == 0 && r0 == 0);

  if (warp == 8) {
    // ------------------------------------------------------------ copies
    const int rows = min(KT, 1 << a.page_shift), parts = KT / rows;
    bool ok = true;
    uint32_t T = 0;   // tiles issued, over all pieces
    for (; ok && p.valid; p = paged_next<KT, kLatentOverhead>(a, share, p, false)) {
      const int32_t* row = a.table + p.b * a.table_stride;
      for (int t = p.t0; t < p.t1; ++t, ++T) {
        const int s = T % ST;
        const int key = t * KT + lane * rows;
        // a page past the sequence's end: the tile's first page in its place
        const int at = key < p.len ? key : t * KT;
        int page = 0;
        if (lane < parts) page = checked_page(row[at >> a.page_shift], a.num_pages, a.status);
        if (T >= ST && !(ok = __all_sync(0xffffffffu, mbar_wait(&ctl.empty[s], ((T / ST) - 1) & 1,
                                                                wc, kSiteLatentFree))))
          break;
        if (lane == 0) mbar_arrive_expect_tx(&ctl.full[s], C::kTileBytes);
        __syncwarp();
        if (lane < parts) {
#pragma unroll
          for (int x = 0; x < C::kBoxes; ++x)
            tma_load_4d(sC + s * C::kTileBytes + x * C::kBoxBytes + lane * rows * 128, &tc,
                        &ctl.full[s], x * 64, at & ((1 << a.page_shift) - 1), 0, page);
        }
      }
    }
    if (!ok && lane == 0)   // let issued copies land before the CTA exits
      for (uint32_t u = T > ST ? T - ST : 0; u < T; ++u)
        mbar_wait_drain(&ctl.full[u % ST], (u / ST) & 1, a.timeout_ns);
  } else if (warp == 9) {
    // --------------------------------------------------------- MMA issue
    constexpr uint32_t kIdS = idesc_bf16(128, kLatentRows, false, false);
    constexpr uint32_t kIdO = idesc_bf16(128, kLatentRows, true, true);
    const uint64_t dq = smem_desc(smem_u32(sQ), 16, 1024);
    const uint64_t dp = smem_desc(smem_u32(sP), 16, 1024);
    bool ok = true;
    uint32_t T = 0;   // tiles before this piece
    int k = 0;        // pieces with tiles
    for (; ok && p.valid; p = paged_next<KT, kLatentOverhead>(a, share, p, false)) {
      const int n = p.t1 - p.t0;
      if (n == 0) continue;
      // S^T of the piece's tile i (the tile has landed): zero what lies past
      // the sequence's end, then issue
      auto scores = [&](int i) {
        const uint32_t u = T + i, s = u % ST;
        uint8_t* tile = sC + s * C::kTileBytes;
        const int from = p.len - (p.t0 + i) * KT;
        if (from < KT) {
          for (int e = lane; e < (KT - from) * C::kBoxes * 8; e += 32) {
            const int j = from + e / (C::kBoxes * 8), c = e % (C::kBoxes * 8);
            *reinterpret_cast<uint4*>(tile + (c >> 3) * C::kBoxBytes + j * 128 + ((c & 7) << 4)) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        tc_fence_after();
        if (lane == 0) {
          const uint64_t dc = smem_desc(smem_u32(tile), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < C::kCols / 16; ++kk) {
            const uint64_t off = static_cast<uint64_t>(((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4);
            mma_ss(tmem + 64 * (u & 1), dc + off, dq + off, kIdS, kk > 0 ? 1u : 0u);
          }
          mma_commit(&ctl.sfull[u & 1]);
        }
        __syncwarp();
      };
      auto landed = [&](int i, bool wait) {
        const uint32_t u = T + i;
        if (!wait)
          return __all_sync(0xffffffffu, mbar_test(&ctl.full[u % ST], (u / ST) & 1)) != 0;
        return (ok = __all_sync(0xffffffffu, mbar_wait(&ctl.full[u % ST], (u / ST) & 1, wc,
                                                       kSiteLatentTile)));
      };
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&ctl.qfull, k & 1, wc, kSiteLatentQ)))) break;
      if (!landed(0, true)) break;
      scores(0);
      for (int i = 0; i < n; ++i) {
        // the next tile's scores first if it has landed; P of this tile does
        // not wait for it
        bool next = i + 1 < n;
        if (next && landed(i + 1, false)) {
          scores(i + 1);
          next = false;
        }
        const uint32_t u = T + i, s = u % ST;
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&ctl.pfull, u & 1, wc, kSiteLatentP)))) break;
        tc_fence_after();
        if (lane == 0) {   // O^T += c^T P^T, 128 value columns at a time
#pragma unroll
          for (int blk = 0; blk < C::kBlocks; ++blk) {
            const uint64_t dv = smem_desc(smem_u32(sC + s * C::kTileBytes + 2 * blk * C::kBoxBytes),
                                          C::kBoxBytes, 1024);
#pragma unroll
            for (int kk = 0; kk < KT / 16; ++kk) {
              const uint64_t off = static_cast<uint64_t>((kk * 2048) >> 4);
              mma_ss(tmem + C::kOCol + 64 * blk, dv + off, dp + off, kIdO, i > 0 || kk > 0 ? 1u : 0u);
            }
          }
          mma_commit(&ctl.empty[s]);
          mma_commit(&ctl.pvdone);
        }
        __syncwarp();
        if (next) {
          if (!landed(i + 1, true)) break;
          scores(i + 1);
        }
      }
      T += n;
      ++k;
    }
    if (lane == 0) {
      mma_commit(&ctl.final_bar);   // every MMA of this CTA done before TMEM is freed
      mbar_wait_drain(&ctl.final_bar, 0, a.timeout_ns);
    }
    __syncwarp();
  } else {
    // ------------------------------------------- q, softmax, rescale, output
    const bool soft = (warp & 2) == 0 && ((warp >> 2) == 0 || live > 32);
    const int key_row = (warp & 1) * 32 + lane;    // softmax: this thread's key of a tile
    const int half = warp >> 2;                    // ... and columns 32 half .. 32 half + 31
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float c2 = a.scale_log2;
    bool ok = true;
    uint32_t T = 0;
    for (; p.valid; p = paged_next<KT, kLatentOverhead>(a, share, p, threadIdx.x == 0 && r0 == 0)) {
      const int n = p.t1 - p.t0;
      float mref[2] = {-INFINITY, -INFINITY};   // columns lane, lane + 32: reference maxima
      float mc[32], l[32];                      // softmax: this half's columns
#pragma unroll
      for (int j = 0; j < 32; ++j) mc[j] = l[j] = 0.f;
      if (n > 0) {
        // q rows r0 .. r0 + 63 of the sequence (zero past the last), K-major
        for (int e = threadIdx.x; e < kLatentRows * C::kBoxes * 8; e += 256) {
          const int r = e / (C::kBoxes * 8), c = e - r * (C::kBoxes * 8);
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (r < live) {
            const int h = (r0 + r) / a.n_q, qt = (r0 + r) - h * a.n_q;
            v = *reinterpret_cast<const uint4*>(a.q + p.b * a.stride_b + h * a.stride_h +
                                                static_cast<int64_t>(qt) * a.stride_n + c * 8);
          }
          *reinterpret_cast<uint4*>(sQ + (c >> 3) * C::kBoxBytes + r * 128 +
                                    (((c & 7) ^ (r & 7)) << 4)) = v;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.qfull);
      }
      const int open = a.causal ? p.len - a.n_q + 1 : p.len;   // every row is allowed keys below it
      for (int i = 0; i < n; ++i, ++T) {
        const int buf = T & 1;
        uint32_t sr[32];
        if (soft) {
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&ctl.sfull[buf], (T >> 1) & 1, wc,
                                                         kSiteLatentS));
          tc_fence_after();
          tmem_ld32(tmem + lanes + 64 * buf + 32 * half, sr);
          tmem_wait_ld();
          const int k0 = (p.t0 + i) * KT, kj = k0 + key_row;
          if (k0 + KT > open) {
            int qt = (r0 + 32 * half) % a.n_q;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const int lim = a.causal ? p.len - a.n_q + qt + 1 : p.len;
              if (kj >= lim) sr[j] = __float_as_uint(-INFINITY);
              if (++qt == a.n_q) qt = 0;
            }
          }
          float top = -INFINITY;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float x = warp_max(__uint_as_float(sr[j]));
            if (lane == j) top = x;
          }
          ctl.wmax[buf][warp & 1][32 * half + lane] = top;
        }
        named_barrier_sync(1, 256);
        float alpha[2];
        bool grown[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float x = fmaxf(ctl.wmax[buf][0][lane + 32 * e], ctl.wmax[buf][1][lane + 32 * e]);
          grown[e] = x > mref[e] && (mref[e] == -INFINITY || (x - mref[e]) * c2 > kRescaleTau);
          alpha[e] = grown[e] ? ex2_approx((mref[e] - x) * c2) : 1.f;
          if (grown[e]) mref[e] = x;
        }
        const bool rescale = __any_sync(0xffffffffu, grown[0] || grown[1]);   // alike in every warp
        if (i > 0 && ok)   // O^T holds the sum through the tile before; P is free
          ok = __all_sync(0xffffffffu, mbar_wait(&ctl.pvdone, (T - 1) & 1, wc, kSiteLatentDone));
        tc_fence_after();
        if (rescale) {
          if (soft) {
            const float al = half ? alpha[1] : alpha[0], mr = half ? mref[1] : mref[0];
            const float mrc = mr == -INFINITY ? 0.f : mr * c2;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              l[j] *= __shfl_sync(0xffffffffu, al, j);
              mc[j] = __shfl_sync(0xffffffffu, mrc, j);
            }
          }
          if (i > 0) {
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
        if (soft) {   // P^T row of this thread's key: 32 columns, 64 bytes
#pragma unroll
          for (int c8 = 0; c8 < 4; ++c8) {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int j = 8 * c8 + 2 * q;
              const float p0 = ex2_approx(fmaf(__uint_as_float(sr[j]), c2, -mc[j]));
              const float p1 = ex2_approx(fmaf(__uint_as_float(sr[j + 1]), c2, -mc[j + 1]));
              l[j] += p0;
              l[j + 1] += p1;
              w[q] = pack_bf16x2(p0, p1);
            }
            *reinterpret_cast<uint4*>(sP + key_row * 128 + (((4 * half + c8) ^ (key_row & 7)) << 4)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.pfull);
      }

      // ---- O = O^T / l and L of the piece
      if (n > 0 && soft) {
        float mine = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          float x = l[j];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
          if (lane == j) mine = x;
        }
        ctl.lsum[warp & 1][32 * half + lane] = mine;
      }
      if (n > 0 && ok) {
        ok = __all_sync(0xffffffffu, mbar_wait(&ctl.pvdone, (T - 1) & 1, wc, kSiteLatentDone));
        tc_fence_after();
      }
      named_barrier_sync(1, 256);
      float inv[2], L[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float s = n > 0 ? ctl.lsum[0][lane + 32 * e] + ctl.lsum[1][lane + 32 * e] : 0.f;
        inv[e] = s != 0.f ? 1.f / s : 0.f;
        L[e] = s != 0.f ? (mref[e] * c2 + __log2f(s)) * kLn2 : -INFINITY;
      }
      const bool whole = p.whole();
      const int64_t part = 2 * static_cast<int64_t>(cta) + (p.s < share.lo ? 0 : 1);
      if (warp == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = r0 + lane + 32 * e;
          if (lane + 32 * e < live) {
            if (whole) a.lse[static_cast<int64_t>(p.b) * a.all_rows + r] = L[e];
            else a.part_l[part * a.rows + r] = L[e];
          }
        }
      }
#pragma unroll
      for (int bb = 0; bb < C::kBlocks / 2; ++bb) {
        const int blk = half * (C::kBlocks / 2) + bb;
        const int dim = 128 * blk + (warp & 3) * 32 + lane;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (32 * e >= live) break;
          uint32_t o[32];
          if (n > 0) {
            tmem_ld32(tmem + lanes + C::kOCol + 64 * blk + 32 * e, o);
            tmem_wait_ld();
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float w = __shfl_sync(0xffffffffu, inv[e], j);
            o[j] = n > 0 && w != 0.f ? __float_as_uint(__uint_as_float(o[j]) * w) : 0u;
          }
          if (whole) {
            // lanes 2 i, 2 i + 1 trade: the even one stores its two columns of
            // row j, the odd one those of row j + 1
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const uint32_t give = (lane & 1) ? o[j] : o[j + 1];
              const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 1);
              const uint32_t v = (lane & 1) ? pack_bf16x2(__uint_as_float(got), __uint_as_float(o[j + 1]))
                                            : pack_bf16x2(__uint_as_float(o[j]), __uint_as_float(got));
              const int r = 32 * e + j + (lane & 1);
              if (r < live)
                *reinterpret_cast<uint32_t*>(
                    a.o + (static_cast<int64_t>(p.b) * a.all_rows + r0 + r) * DV + (dim & ~1)) = v;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (32 * e + j < live)
                a.part_o[(part * a.rows + r0 + 32 * e + j) * DV + dim] = __uint_as_float(o[j]);
          }
        }
      }
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int DV>
cudaError_t launch_dv(const CUtensorMap& tc, const PagedArgs& a, int ctas, cudaStream_t s) {
  using C = LatentCfg<DV>;
  static std::atomic<uint64_t> set_up{0};
  int dev = 0;
  bool todo = false;
  cudaError_t e = needs_setup(set_up, &dev, &todo);
  if (e != cudaSuccess) return e;
  if (todo) {
    e = cudaFuncSetAttribute(latent_kernel<DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    mark_done(set_up, dev);
  }
  const int groups = a.rows / kLatentRows;
  return launch_pdl(latent_kernel<DV>, dim3(ctas * groups), dim3(C::kThreads), C::kSmem, s, tc, a,
                    groups);
}

}  // namespace

cudaError_t launch_latent(const CUtensorMap& tc, const PagedArgs& a, int ctas, cudaStream_t s) {
  return a.d == 256 ? launch_dv<256>(tc, a, ctas, s) : launch_dv<512>(tc, a, ctas, s);
}

}  // namespace attn
