// Decode step against a paged key/value cache.
//
// What it computes: the decode step of attn_decode.cu (query row t of
// sequence b at position len_b - n_q + t attends the cached keys j < len_b,
// j <= its position when causal; O = softmax(c q K^T) V, L = logsumexp) with
// key j of sequence b in row j mod s of page table[b][j / s].
//
// Bound: HBM.  Every cached key and value is read once, 4 d bytes a key, for
// 4 d rows operations: 1 to 64 operations a byte at 1 to 64 rows, below the
// ridge of 277.  So what counts is that all SMs stream all the time:
//   * the keys of all sequences are divided evenly over a fixed number of
//     CTAs (two per SM) by their real lengths (attn_paged.cuh), which makes
//     the step as fast for ragged batches as for even ones, and leaves at
//     most two partial results per CTA however long the caches are;
//   * each warp streams its own 32-key tiles of K and V by TMA through its
//     own ring, a page's rows at a time, the page indices prefetched 32 tiles
//     at a time, and the first tiles of the next segment are on their way
//     before the write-out of the last one begins;
//   * the two products are 16 x 8 x 16 warp MMAs: with at most 64 rows a
//     128-row tcgen05 tile would be mostly padding, and the products' time is
//     hidden behind the copies.  Above 16 rows MT = 2 or 4 warps share a tile,
//     16 rows each.
// Values of rows past the end of a sequence may be anything, infinities and
// NaN included: their scores are replaced, not added to, and their value
// rows are zeroed in shared memory before the product (0 * NaN is NaN).
// P is rounded to bf16 for the second product (relative 2^-8 per element;
// the row sums are of the unrounded fp32 values), m, l, O are fp32.
//
// Measured (whole steps replayed from a CUDA graph, measured copy rate 6.8
// TB/s): 16 sequences of 4096-8192 keys, 32 heads over 8, d = 128, 403 MB in
// 70 us = 5.8 TB/s, of it 2.7 us the merge; 64 sequences of 0-16384 keys, 4
// queries, 64 heads over 8, 2.2 GB in 332 us = 6.5 TB/s; one sequence of 517
// keys 8.2 us, two reads of lengths and pages, a tile's copy and the merge one
// after another.  DRAM traffic is the algorithmic bytes plus 1 %.
#include <type_traits>

#include "attn_paged.cuh"

namespace attn {
using namespace sm103;

namespace {

constexpr int kSlots = 3;   // tiles worked on at a time by a CTA

template <int D, int MT>
struct PagedCfg {
  static constexpr int kWarps = kSlots * MT;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kKeys = kPagedKeys;
  static constexpr int kBoxes = D / 64;
  static constexpr int kBoxBytes = kKeys * 128;
  static constexpr int kTileBytes = kKeys * D * 2;
  // four row tiles leave one CTA per SM, which then has twice the stages
  static constexpr int kCtasPerSm = MT == 4 ? 1 : 2;
  static constexpr int kStages = (D == 128 ? 2 : 4) * (MT == 4 ? 2 : 1);   // per slot
  static constexpr int kRingBytes = 2 * kSlots * kStages * kTileBytes;
  static constexpr int kRedStride = D + 8;   // floats; the pad spreads the rows over the banks
  static constexpr int kRedBytes = 16 * kRedStride * 4;
  static constexpr int kSmem = 1024 + kRingBytes + kRedBytes;
  static_assert(kCtasPerSm * (kSmem + 1024 + 2560) <= 228 * 1024, "shared memory of an SM");
};

template <int D, int MT>
struct PagedShared {
  uint64_t full[kSlots * PagedCfg<D, MT>::kStages];
  uint64_t empty[kSlots * PagedCfg<D, MT>::kStages];
  float m[kSlots][MT * 16], l[kSlots][MT * 16];
  float L[16];   // of the rows in `red`, for the cluster
  int abort_flag;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2,
                                      uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2,
                                        uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr)
               : "memory");
}

// c += a b, 16 x 8 x 16, bf16 inputs, fp32 accumulators
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// How the segments are given out.
//   kSplit    the balanced split
//   kCluster  a segment per cluster (a.cluster CTAs), merged in shared memory
//   kSolo     a segment per slot, which has nobody to merge with: for many short
//             sequences (64 of 50-200 keys, 8 heads: 13.0 against 19.4 us)
enum PagedMode { kSplit, kCluster, kSolo };

template <int D, int MT, PagedMode MODE>
__global__ void __launch_bounds__(PagedCfg<D, MT>::kThreads, PagedCfg<D, MT>::kCtasPerSm)
    paged_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                 const PagedArgs a) {
  using C = PagedCfg<D, MT>;
  constexpr bool CLUSTER = MODE == kCluster, SOLO = MODE == kSolo;
  constexpr int ST = C::kStages, KT = C::kKeys, NT = D / 8;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* red = reinterpret_cast<float*>(smem + C::kRingBytes);   // [16][kRedStride]
  __shared__ PagedShared<D, MT> sh;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slot = warp / MT, mt = warp % MT;   // which tiles, which 16 rows
  auto sK = [&](int st) { return smem + (slot * ST + st) * 2 * C::kTileBytes; };
  auto sV = [&](int st) { return sK(st) + C::kTileBytes; };

  if (threadIdx.x == 0) {
    sh.abort_flag = 0;
    for (int s = 0; s < kSlots * ST; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], MT);
    }
    fence_mbar_init();
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  __syncthreads();
  // With a prefix the kernel before this one attends it, and only the merge
  // needs its results: so the wait for it comes at the end, and this kernel's
  // CTAs run beside it as SMs fall free.  (That all kernels before it are
  // complete is known here: each of its CTAs had waited for them before it let
  // this kernel start.)
  const bool late = a.pre_splits > 0;
  if (!late) grid_dep_wait();
  grid_dep_launch();
  PagedShare share{};
  if constexpr (MODE == kSplit)
    share = paged_share<KT, kPagedOverhead, kPagedMinUnits>(a, blockIdx.x, gridDim.x);
  MergeNote note{-1, 0, 0, 0};
  const WaitCtx wc{&sh.abort_flag, a.status, a.timeout_ns};
  const int box_rows = min(KT, 1 << a.page_shift);
  // Behind a shared prefix a sequence's own keys go by once, and leave L2 to the
  // partials: 128 sequences 94.7 -> 90.9 us.  Without one, sequences may name
  // the same pages (forks): 8 that share all of 8192 keys, 64 in all, take 149 us,
  // and 202 where what they read is the first to leave.
  const uint64_t policy = l2_policy(a.pre_splits > 0);
  bool ok = true;

  // ---- the copies: tile u of this slot is tile t0 + slot + kSlots u of the
  // piece (of a segment of its own: tile u); lane l of the issuing warp holds the page indices of tile
  // 32 * (batch) + l (two where a tile spans two 16-key pages)
  uint32_t issued = 0, done = 0;   // tiles of this slot issued / used, over all pieces
  int page_of[2] = {0, 0};
  constexpr int kStep = SOLO ? 1 : kSlots;
  const int first_tile = SOLO ? 0 : slot;
  auto slot_tiles = [&](const PagedPiece& p) {
    const int n = p.t1 - p.t0 - first_tile;
    return n > 0 ? (n + kStep - 1) / kStep : 0;
  };
  auto load_pages = [&](const PagedPiece& p, int u0, int nu) {
    const int u = u0 + lane;
    if (u < nu) {
      const int key = a.first + (p.t0 + first_tile + kStep * u) * KT;
      const int32_t* row = a.table + p.b * a.table_stride;
      page_of[0] = checked_page(row[key >> a.page_shift], a.num_pages, a.status);
      // (a page of 16 keys: the tile's second half, where the sequence reaches it)
      page_of[1] = box_rows == KT || key + box_rows >= p.len
                       ? page_of[0]
                       : checked_page(row[(key >> a.page_shift) + 1], a.num_pages, a.status);
    }
  };
  auto issue = [&](const PagedPiece& p, int u) {   // the whole issuing warp
    const int pg0 = __shfl_sync(0xffffffffu, page_of[0], u & 31);
    const int pg1 = __shfl_sync(0xffffffffu, page_of[1], u & 31);
    const int st = issued % ST;
    if (MT > 1 && issued >= ST) {   // the slot's warps are done with the stage
      ok = __all_sync(0xffffffffu, mbar_wait(&sh.empty[slot * ST + st], ((issued / ST) - 1) & 1, wc,
                                             kSitePagedFree));
      if (!ok) return;
    }
    // (an armed test stall: slot 0's first tile is not copied, so the wait for it
    // runs out)
    if (lane == 0 && !(a.stall != 0 && slot == 0 && issued == 0)) {
      uint64_t* bar = &sh.full[slot * ST + st];
      const int row = (a.first + (p.t0 + first_tile + kStep * u) * KT) & ((1 << a.page_shift) - 1);
      const int head = p.h / a.blocks;
      fence_proxy_async_smem();
      mbar_arrive_expect_tx(bar, 2 * C::kTileBytes);
#pragma unroll
      for (int x = 0; x < C::kBoxes; ++x) {
        tma_load_4d(sK(st) + x * C::kBoxBytes, &tk, bar, x * 64, row, head, pg0, policy);
        tma_load_4d(sV(st) + x * C::kBoxBytes, &tv, bar, x * 64, row, head, pg0, policy);
        if (box_rows < KT) {
          tma_load_4d(sK(st) + x * C::kBoxBytes + 16 * 128, &tk, bar, x * 64, 0, head, pg1, policy);
          tma_load_4d(sV(st) + x * C::kBoxBytes + 16 * 128, &tv, bar, x * 64, 0, head, pg1, policy);
        }
      }
    }
    ++issued;
  };
  auto prefetch = [&](const PagedPiece& p) {   // the first tiles of a piece
    if (mt != 0 || !p.valid) return;
    const int nu = slot_tiles(p);
    if (nu == 0) return;
    load_pages(p, 0, nu);
    for (int u = 0; ok && u < ST && u < nu; ++u) issue(p, u);
  };

  const int g = lane >> 2, q4 = lane & 3;
  const int rows[2] = {mt * 16 + g, mt * 16 + g + 8};
  const int lb = lane >> 3, lr = lane & 7;
  const float c2 = a.scale_log2;

  const int rank = CLUSTER ? static_cast<int>(cluster_rank()) : 0;
  PagedPiece p;
  if constexpr (CLUSTER) {
    const int segment = blockIdx.x / a.cluster, b = segment / a.heads;
    p = paged_part<KT>(a, b, segment - b * a.heads, rank, a.cluster);
  } else if constexpr (SOLO) {
    const int segment = blockIdx.x * kSlots + slot, b = segment / a.heads;
    if (b < a.B) p = paged_part<KT>(a, b, segment - b * a.heads, 0, 1);
    else p.valid = false;
  } else {
    p = paged_piece<KT, kPagedOverhead>(a, share, share.b, 0, share.s);
  }
  prefetch(p);
  while (p.valid) {   // (the same pieces in every warp)
    const int nu = slot_tiles(p);
    // Q fragments of rows g and g + 8 of the warp's 16 (zero past the last row)
    uint32_t qa[D / 16][4];
    int lim[2];   // keys below lim are allowed
    const int row0 = segment_row(a, p.h), nrows = segment_rows(a, p.h);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = rows[i];
      const bool live = r < nrows;
      const int h = (row0 + r) / a.n_q, qt = row0 + r - h * a.n_q;
      const __nv_bfloat16* qr =
          a.q + p.b * a.stride_b + h * a.stride_h + static_cast<int64_t>(qt) * a.stride_n;
      lim[i] = !live ? 0 : (a.causal ? min(p.len, p.len - a.n_q + qt + 1) : p.len);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qa[kk][i] = live ? *reinterpret_cast<const uint32_t*>(qr + kk * 16 + 2 * q4) : 0u;
        qa[kk][i + 2] = live ? *reinterpret_cast<const uint32_t*>(qr + kk * 16 + 8 + 2 * q4) : 0u;
      }
    }
    const int open = a.causal ? p.len - a.n_q + 1 : p.len;   // every row is allowed keys below it
    float mrow[2] = {-INFINITY, -INFINITY}, lrow[2] = {0.f, 0.f};
    float o[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;

    for (int u = 0; ok && u < nu; ++u) {
      const int st = done % ST;
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&sh.full[slot * ST + st], (done / ST) & 1, wc,
                                                   kSitePagedTile))))
        break;
      const uint32_t kb = smem_u32(sK(st)), vb = smem_u32(sV(st));
      const int k0 = a.first + (p.t0 + first_tile + kStep * u) * KT;
      if (k0 + KT > p.len) {   // value rows past the end: zero
        const int from = p.len - k0;
        for (int i = lane; i < (KT - from) * (D / 8); i += 32) {
          const int key = from + i / (D / 8), c8 = i % (D / 8);
          *reinterpret_cast<uint4*>(sV(st) + (c8 >> 3) * C::kBoxBytes + key * 128 +
                                    ((c8 & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
        }
        __syncwarp();
      }
      // S = Q K^T: per 16 columns of d one ldmatrix.x4 gives two key blocks of 8
      float sc[KT / 8][4];
#pragma unroll
      for (int n = 0; n < KT / 8; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int n = 0; n < KT / 8; n += 2) {
          const int key = 8 * n + 8 * (lb >> 1) + lr, col = 16 * kk + 8 * (lb & 1);
          uint32_t b0, b1, b2, b3;
          ldsm4(kb + (col >> 6) * C::kBoxBytes + key * 128 + ((((col & 63) >> 3) ^ (key & 7)) << 4),
                b0, b1, b2, b3);
          mma16816(sc[n], qa[kk], b0, b1);
          mma16816(sc[n + 1], qa[kk], b2, b3);
        }
      if (k0 + KT > open) {
#pragma unroll
        for (int n = 0; n < KT / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (k0 + 8 * n + 2 * q4 + (e & 1) >= lim[e >> 1]) sc[n][e] = -INFINITY;
      }
      float tmax[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < KT / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) tmax[e >> 1] = fmaxf(tmax[e >> 1], sc[n][e]);
      float alpha[2], base[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        tmax[i] = fmaxf(tmax[i], __shfl_xor_sync(0xffffffffu, tmax[i], 1));
        tmax[i] = fmaxf(tmax[i], __shfl_xor_sync(0xffffffffu, tmax[i], 2));
        const float mn = fmaxf(mrow[i], tmax[i]);
        base[i] = mn == -INFINITY ? 0.f : mn * c2;   // -inf: no allowed key seen yet
        alpha[i] = mrow[i] == -INFINITY ? 0.f : ex2_approx(mrow[i] * c2 - base[i]);
        mrow[i] = mn;
      }
      // P = 2^(S c - m c) as bf16 A fragments; row sums from the same fp32 values
      uint32_t pa[KT / 16][4];
      float psum[2] = {0.f, 0.f};
#pragma unroll
      for (int n = 0; n < KT / 8; ++n) {
        const float p0 = ex2_approx(fmaf(sc[n][0], c2, -base[0]));
        const float p1 = ex2_approx(fmaf(sc[n][1], c2, -base[0]));
        const float p2 = ex2_approx(fmaf(sc[n][2], c2, -base[1]));
        const float p3 = ex2_approx(fmaf(sc[n][3], c2, -base[1]));
        psum[0] += p0 + p1;
        psum[1] += p2 + p3;
        pa[n >> 1][(n & 1) * 2] = pack_bf16x2(p0, p1);
        pa[n >> 1][(n & 1) * 2 + 1] = pack_bf16x2(p2, p3);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) lrow[i] = lrow[i] * alpha[i] + psum[i];
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          o[n][0] *= alpha[0];
          o[n][1] *= alpha[0];
          o[n][2] *= alpha[1];
          o[n][3] *= alpha[1];
        }
      }
#pragma unroll
      for (int kp = 0; kp < KT / 16; ++kp)
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
          const int key = 16 * kp + 8 * (lb & 1) + lr, col = 8 * n + 8 * (lb >> 1);
          uint32_t b0, b1, b2, b3;
          ldsm4_t(vb + (col >> 6) * C::kBoxBytes + key * 128 +
                      ((((col & 63) >> 3) ^ (key & 7)) << 4),
                  b0, b1, b2, b3);
          mma16816(o[n], pa[kp], b0, b1);
          mma16816(o[n + 1], pa[kp], b2, b3);
        }
      ++done;
      __syncwarp();
      if (MT > 1 && lane == 0) mbar_arrive(&sh.empty[slot * ST + st]);
      if (mt == 0 && u + ST < nu) {   // refill the stage with the slot's tile u + ST
        if (((u + ST) & 31) == 0) load_pages(p, u + ST, nu);
        issue(p, u + ST);
      }
    }

    PagedPiece next = p;
    if constexpr (MODE == kSplit) {
      next = paged_next<KT, kPagedOverhead>(a, share, p);
      if (ok) prefetch(next);
    } else {
      next.valid = false;
    }
    if constexpr (SOLO) {
      // rows g, g + 8 straight from the registers, with a prefix's pieces
      if (late) grid_dep_wait();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float l = lrow[i];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (rows[i] >= nrows) continue;
        const int h = (row0 + rows[i]) / a.n_q, qt = row0 + rows[i] - h * a.n_q;
        const int64_t row = static_cast<int64_t>(p.b) * a.all_rows + row0 + rows[i];
        const int64_t all = static_cast<int64_t>(a.B) * a.all_rows;
        const float L = l == 0.f ? -INFINITY : fmaf(mrow[i], a.scale, logf(l));
        float top = L;
        for (int k = 0; k < a.pre_splits; ++k) top = fmaxf(top, a.pre_l[k * all + row]);
        top = merge_base(top);
        // (without a prefix the weight is 1)
        float sum = a.pre_splits > 0 ? __expf(L - top) : L == -INFINITY ? 0.f : 1.f;
        const float own = sum == 0.f ? 0.f : sum / l;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          o[n][2 * i] *= own;
          o[n][2 * i + 1] *= own;
        }
        for (int k = 0; k < a.pre_splits; ++k) {
          const float w = __expf(a.pre_l[k * all + row] - top);
          const float* y = a.pre_o + (k * all + row) * D + 2 * q4;
          sum += w;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float2 z = *reinterpret_cast<const float2*>(y + 8 * n);
            o[n][2 * i] = fmaf(w, z.x, o[n][2 * i]);
            o[n][2 * i + 1] = fmaf(w, z.y, o[n][2 * i + 1]);
          }
        }
        const float inv = sum == 0.f ? 0.f : a.pre_splits > 0 ? 1.f / sum : 1.f;
        __nv_bfloat16* to =
            a.o + p.b * a.stride_b + h * a.stride_h + static_cast<int64_t>(qt) * a.stride_n + 2 * q4;
#pragma unroll
        for (int n = 0; n < NT; ++n)
          *reinterpret_cast<uint32_t*>(to + 8 * n) =
              pack_bf16x2(o[n][2 * i] * inv, o[n][2 * i + 1] * inv);
        if (q4 == 0)
          a.lse[row] = sum == 0.f ? -INFINITY : a.pre_splits > 0 ? top + logf(sum) : L;
      }
    } else {
      // ---- the slots' states merged: m, l per row, then O through shared memory
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        lrow[i] += __shfl_xor_sync(0xffffffffu, lrow[i], 1);
        lrow[i] += __shfl_xor_sync(0xffffffffu, lrow[i], 2);
        if (lrow[i] != lrow[i]) mrow[i] = 0.f;   // a row of NaN scores has seen keys
        if (q4 == 0) {
          sh.m[slot][rows[i]] = mrow[i];
          sh.l[slot][rows[i]] = lrow[i];
        }
      }
      ok = __syncthreads_and(ok);
      float scale[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx = -INFINITY, lt = 0.f;
#pragma unroll
        for (int w = 0; w < kSlots; ++w) mx = fmaxf(mx, sh.m[w][rows[i]]);
#pragma unroll
        for (int w = 0; w < kSlots; ++w) {
          const float mw = sh.m[w][rows[i]];
          if (mw != -INFINITY) lt += sh.l[w][rows[i]] * ex2_approx((mw - mx) * c2);
        }
        // this slot's weight, with the 1 / l folded in
        scale[i] = mrow[i] == -INFINITY ? 0.f : ex2_approx((mrow[i] - mx) * c2) / lt;
      }
      const bool whole = p.whole();
      const bool apart = a.pre_splits > 0;   // a prefix is merged afterwards
      if constexpr (MODE == kSplit) {
        if (p.t0 == 0 && !whole) note = paged_note<kPagedOverhead>(share, p);
        if (a.by_segment && p.t0 == 0 && threadIdx.x == 0)
          a.notes[p.b * a.heads + p.h] = whole ? MergeNote{p.b, p.h, 0, -1} : note;
      }
      const int64_t part = 2 * static_cast<int64_t>(blockIdx.x) + (p.s < share.lo ? 0 : 1);
      for (int m = 0; m < MT; ++m) {   // 16 rows at a time
        for (int w = 0; w < kSlots; ++w) {   // in turn: the sum has a fixed order
          if (slot == w && mt == m) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float2* dst = reinterpret_cast<float2*>(&red[(g + 8 * i) * C::kRedStride + 8 * n + 2 * q4]);
                float2 x = make_float2(o[n][2 * i] * scale[i], o[n][2 * i + 1] * scale[i]);
                if (w > 0) {
                  const float2 y = *dst;
                  x.x += y.x;
                  x.y += y.y;
                }
                *dst = x;
              }
          }
          __syncthreads();
        }
        const int live = min(16, nrows - 16 * m);   // (negative where a tile has no rows)
        auto logsumexp = [&](int r) {
          float mx = -INFINITY, lt = 0.f;
#pragma unroll
          for (int w = 0; w < kSlots; ++w) mx = fmaxf(mx, sh.m[w][r]);
#pragma unroll
          for (int w = 0; w < kSlots; ++w) {
            const float mw = sh.m[w][r];
            if (mw != -INFINITY) lt += sh.l[w][r] * ex2_approx((mw - mx) * c2);
          }
          return lt == 0.f ? -INFINITY : fmaf(mx, a.scale, logf(lt));
        };
        if constexpr (CLUSTER) {
          // the cluster's rows, and a prefix's pieces, merged: each CTA writes a
          // part of the items
          if (static_cast<int>(threadIdx.x) < live)
            sh.L[threadIdx.x] = logsumexp(16 * m + threadIdx.x);
          if (late) grid_dep_wait();
          cluster_sync();
          for (int e = rank * C::kThreads + threadIdx.x; e < live * (D / 4);
               e += a.cluster * C::kThreads) {
            const int rr = e / (D / 4), c = 4 * (e - rr * (D / 4)), r = 16 * m + rr;
            const int h = (row0 + r) / a.n_q, qt = row0 + r - h * a.n_q;
            const int64_t row = static_cast<int64_t>(p.b) * a.all_rows + row0 + r;
            const int64_t all = static_cast<int64_t>(a.B) * a.all_rows;
            float top = -INFINITY, sum = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
            for (int k = 0; k < a.cluster; ++k)
              top = fmaxf(top, cluster_ld(cluster_addr(&sh.L[rr], k)));
            for (int k = 0; k < a.pre_splits; ++k) top = fmaxf(top, a.pre_l[k * all + row]);
            top = merge_base(top);
            auto add = [&](float L, const float* y) {
              const float w = __expf(L - top);
              sum += w;
#pragma unroll
              for (int i = 0; i < 4; ++i) x[i] = fmaf(w, y[i], x[i]);
            };
            for (int k = 0; k < a.cluster; ++k) {
              float y[4];
              cluster_ld4(cluster_addr(&red[rr * C::kRedStride + c], k), y);
              add(cluster_ld(cluster_addr(&sh.L[rr], k)), y);
            }
            for (int k = 0; k < a.pre_splits; ++k) {
              const float4 y = *reinterpret_cast<const float4*>(a.pre_o + (k * all + row) * D + c);
              const float z[4] = {y.x, y.y, y.z, y.w};
              add(a.pre_l[k * all + row], z);
            }
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            *reinterpret_cast<uint2*>(a.o + p.b * a.stride_b + h * a.stride_h +
                                      static_cast<int64_t>(qt) * a.stride_n + c) =
                make_uint2(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv));
            if (c == 0) a.lse[row] = sum == 0.f ? -INFINITY : top + logf(sum);
          }
          cluster_sync();   // the others have read this CTA's rows
        } else {
          for (int e = threadIdx.x; e < live * (D / 4); e += C::kThreads) {
            const int rr = e / (D / 4), c = 4 * (e - rr * (D / 4)), r = 16 * m + rr;
            const float4 x = *reinterpret_cast<const float4*>(&red[rr * C::kRedStride + c]);
            if (whole) {
              const int h = (row0 + r) / a.n_q, qt = row0 + r - h * a.n_q;
              const int64_t row = static_cast<int64_t>(p.b) * a.all_rows + row0 + r;
              if (apart) {
                const int64_t at = a.pre_splits * (static_cast<int64_t>(a.B) * a.all_rows) + row;
                *reinterpret_cast<float4*>(a.pre_o + at * D + c) = x;
                if (c == 0) a.pre_l[at] = logsumexp(r);
                continue;
              }
              *reinterpret_cast<uint2*>(a.o + p.b * a.stride_b + h * a.stride_h +
                                        static_cast<int64_t>(qt) * a.stride_n + c) =
                  make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
              if (c == 0) a.lse[row] = logsumexp(r);
            } else {
              *reinterpret_cast<float4*>(a.part_o + (part * a.rows + r) * D + c) = x;
              if (c == 0) a.part_l[part * a.rows + r] = logsumexp(r);
            }
          }
          __syncthreads();   // red (and after the last rows m, l) is free
        }
      }
    }
    if (!ok) break;
    p = next;
  }
  if (MODE == kSplit && !a.by_segment && threadIdx.x == 0) a.notes[blockIdx.x] = note;
  if (late) grid_dep_wait();   // the merge, and whatever follows, waits for this kernel only
  if (!ok && mt == 0 && lane == 0) {   // let issued copies land before the CTA exits
    for (uint32_t t = issued > ST ? issued - ST : 0; t < issued; ++t)
      mbar_wait_drain(&sh.full[slot * ST + t % ST], (t / ST) & 1, a.timeout_ns);
  }
}

struct Partial {
  const float *o, *l;   // a row's columns; its L
};

constexpr int kMergeThreads = 256;
// pieces of a segment that sixteen threads share (one sequence of 100000 latent
// vectors: 34.1 us a step, with four threads 41.4; two sequences of 30000 keys,
// 64 rows: 26.2 against 29.5; 6 or 12 pieces are alike)
constexpr int kMergeMany = 6;

// Four columns of a row's O merged from `n` partials, O = sum e^(L_i - L) O_i,
// and the parts of L = log sum e^(L_i) = top + log(sum) (-inf if sum = 0).
// GROUPS threads share an item (threads kMergeThreads / GROUPS apart), each
// takes every GROUPS-th partial, two of them at once so that their L
// and O are on the way together, with a running maximum; the first thread has
// the result.  `live`: the item exists.  The whole CTA.
template <int GROUPS, typename From>
__device__ __forceinline__ void merge_row(bool live, int n, const From& from, float4& x, float& top,
                                          float& sum) {
  constexpr int kItems = kMergeThreads / GROUPS, kAtOnce = 2;
  const int group = threadIdx.x / kItems, item = threadIdx.x % kItems;
  if (!live) n = 0;
  x = make_float4(0.f, 0.f, 0.f, 0.f);
  float most = -INFINITY;
  top = sum = 0.f;
  // what is there weighs e^(before - top), then w y comes on top
  auto scale = [&](float before) {
    top = merge_base(most);
    const float w = __expf(before - top);
    sum *= w;
    x.x *= w;
    x.y *= w;
    x.z *= w;
    x.w *= w;
  };
  auto add = [&](float w, float s, const float4& y) {
    sum = fmaf(w, s, sum);
    x.x = fmaf(w, y.x, x.x);
    x.y = fmaf(w, y.y, x.y);
    x.z = fmaf(w, y.z, x.z);
    x.w = fmaf(w, y.w, x.w);
  };
  for (int i0 = group; i0 < n; i0 += GROUPS * kAtOnce) {
    float l[kAtOnce];
    float4 y[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const bool in = i0 + k * GROUPS < n;
      l[k] = -INFINITY;
      y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (in) {
        const Partial part = from(i0 + k * GROUPS);
        l[k] = *part.l;
        y[k] = *reinterpret_cast<const float4*>(part.o);
      }
    }
    const float before = most;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) most = fmaxf(most, l[k]);
    scale(before);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) add(__expf(l[k] - top), 1.f, y[k]);
  }
  if constexpr (GROUPS > 1) {
    __shared__ float mosts[kMergeThreads], sums[kMergeThreads];
    __shared__ float4 xs[kMergeThreads];
    if (group > 0) {
      mosts[threadIdx.x] = most;
      sums[threadIdx.x] = sum;
      xs[threadIdx.x] = x;
    }
    __syncthreads();
    if (group == 0) {
      const float before = most;
#pragma unroll
      for (int k = 1; k < GROUPS; ++k) most = fmaxf(most, mosts[item + k * kItems]);
      scale(before);
#pragma unroll
      for (int k = 1; k < GROUPS; ++k) {
        const int at = item + k * kItems;
        add(__expf(mosts[at] - top), sums[at], xs[at]);
      }
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  x.x *= inv;
  x.y *= inv;
  x.z *= inv;
  x.w *= inv;
}

// Row hr (head * n_q + query) of sequence b.
__device__ __forceinline__ void write_row(const PagedArgs& a, int b, int hr, int c, const float4& x,
                                          float top, float sum) {
  const int h = hr / a.n_q, qt = hr - h * a.n_q;
  *reinterpret_cast<uint2*>(a.o + b * a.stride_b + h * a.stride_h +
                            static_cast<int64_t>(qt) * a.stride_n + c) =
      make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
  if (c == 0)
    a.lse[static_cast<int64_t>(b) * a.all_rows + hr] = sum == 0.f ? -INFINITY : top + logf(sum);
}

// Segments that were cut: their pieces merged, four columns of a row per item.
// A CTA per (note, kMergeThreads / GROUPS items).  Bound by the latency of its
// loads (the pieces come from L2) and by the launch of CTAs that find nothing
// to do, hence notes per segment where there are fewer of those, and four
// threads per item where a segment has many pieces.
template <int D, int GROUPS>
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const PagedArgs a) {
  constexpr int kItems = kMergeThreads / GROUPS;
  grid_dep_wait();
  grid_dep_launch();
  const int4 raw = *reinterpret_cast<const int4*>(a.notes + blockIdx.x);
  const MergeNote note{raw.x, raw.y, raw.z, raw.w};
  if (note.more < 0 || !note_holds(a, note)) return;   // (uniform over the CTA)
  const int e = blockIdx.y * kItems + threadIdx.x % kItems;
  const int r = e / (D / 4), c = 4 * (e % (D / 4)), hr = segment_row(a, note.h) + r;
  const bool live = r < segment_rows(a, note.h);
  auto piece = [&](int i) {
    const int64_t at =
        static_cast<int64_t>(i == 0 ? note.slot : (note.slot & ~1) + 2 * i) * a.rows + r;
    return Partial{a.part_o + at * D + c, a.part_l + at};
  };
  float4 x;
  float top, sum;
  merge_row<GROUPS>(live, note.more + 1, piece, x, top, sum);
  if (live && threadIdx.x < kItems) write_row(a, note.b, hr, c, x, top, sum);
}

// With a shared prefix: every row from the prefix's pieces and its own
// segment, in one piece or cut.  A CTA per (segment, kMergeThreads / GROUPS items).
template <int D, int GROUPS>
__global__ void __launch_bounds__(kMergeThreads) paged_finish_kernel(const PagedArgs a) {
  constexpr int kItems = kMergeThreads / GROUPS;
  grid_dep_wait();
  grid_dep_launch();
  const int4 raw = *reinterpret_cast<const int4*>(a.notes + blockIdx.x);
  const MergeNote note{raw.x, raw.y, raw.z, raw.w};
  if (!note_holds(a, note)) return;
  const int e = blockIdx.y * kItems + threadIdx.x % kItems;
  const int r = e / (D / 4), c = 4 * (e % (D / 4)), hr = segment_row(a, note.h) + r;
  const bool live = r < segment_rows(a, note.h);
  const int64_t row = static_cast<int64_t>(note.b) * a.all_rows + hr;
  const int64_t all = static_cast<int64_t>(a.B) * a.all_rows;
  const int pre = a.pre_splits + (note.more < 0 ? 1 : 0);
  auto part = [&](int i) {
    if (i < pre) {
      const int64_t at = i * all + row;
      return Partial{a.pre_o + at * D + c, a.pre_l + at};
    }
    i -= pre;
    const int64_t at =
        static_cast<int64_t>(i == 0 ? note.slot : (note.slot & ~1) + 2 * i) * a.rows + r;
    return Partial{a.part_o + at * D + c, a.part_l + at};
  };
  float4 x;
  float top, sum;
  merge_row<GROUPS>(live, pre + note.more + 1, part, x, top, sum);
  if (live && threadIdx.x < kItems) write_row(a, note.b, hr, c, x, top, sum);
}

template <int D, int MT, PagedMode MODE>
cudaError_t launch_mt(const CUtensorMap& tk, const CUtensorMap& tv, const PagedArgs& a, int ctas,
                      cudaStream_t s) {
  using C = PagedCfg<D, MT>;
  static std::atomic<uint64_t> set_up{0};
  int dev = 0;
  bool todo = false;
  cudaError_t e = needs_setup(set_up, &dev, &todo);
  if (e != cudaSuccess) return e;
  if (todo) {
    e = cudaFuncSetAttribute(paged_kernel<D, MT, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::kSmem);
    if (e != cudaSuccess) return e;
    mark_done(set_up, dev);
  }
  const unsigned segments = static_cast<unsigned>(a.B * a.heads);
  if (MODE == kCluster)
    return launch_clusters(paged_kernel<D, MT, MODE>, dim3(segments * a.cluster), dim3(C::kThreads),
                           C::kSmem, a.cluster, s, tk, tv, a);
  const unsigned grid = MODE == kSolo ? (segments + kSlots - 1) / kSlots : ctas;
  return launch_pdl(paged_kernel<D, MT, MODE>, dim3(grid), dim3(C::kThreads), C::kSmem, s, tk, tv, a);
}

template <int D, PagedMode MODE>
cudaError_t launch_d(const CUtensorMap& tk, const CUtensorMap& tv, const PagedArgs& a, int ctas,
                     cudaStream_t s) {
  if (a.rows <= 16) return launch_mt<D, 1, MODE>(tk, tv, a, ctas, s);
  if (a.rows <= 32) return launch_mt<D, 2, MODE>(tk, tv, a, ctas, s);
  return launch_mt<D, 4, MODE>(tk, tv, a, ctas, s);
}

template <int D>
cudaError_t launch_mode(const CUtensorMap& tk, const CUtensorMap& tv, const PagedArgs& a, int ctas,
                        cudaStream_t s) {
  if (a.cluster == 1) return launch_d<D, kSolo>(tk, tv, a, ctas, s);
  if (a.cluster > 1) return launch_d<D, kCluster>(tk, tv, a, ctas, s);
  return launch_d<D, kSplit>(tk, tv, a, ctas, s);
}

}  // namespace

cudaError_t launch_paged(const CUtensorMap& tk, const CUtensorMap& tv, const PagedArgs& a, int ctas,
                         cudaStream_t s) {
  return a.d == 64 ? launch_mode<64>(tk, tv, a, ctas, s) : launch_mode<128>(tk, tv, a, ctas, s);
}

namespace {

template <int GROUPS>
using Groups = std::integral_constant<int, GROUPS>;

// `go` with the number of threads that share an item, 16, 4 or 1: 16 where a
// segment has many pieces (kMergeMany), which one thread would read one
// after the other, and the items are few; 4 if `some`.
template <typename Go>
cudaError_t with_groups(int64_t items, int64_t pieces, bool some, const Go& go) {
  if (pieces >= kMergeMany && items <= (1 << 14)) return go(Groups<16>());
  return some ? go(Groups<4>()) : go(Groups<1>());
}

}  // namespace

cudaError_t launch_paged_merge(const PagedArgs& a, int notes, int ctas, cudaStream_t s) {
  // Four threads an item while the items are too few to fill the GPU: 16
  // sequences of 4096 latent vectors, 16 heads (32 K items of 10 pieces) 25.1
  // against 27.1 us a step, but with 64 heads (131 K items) 38.3 against 35.6.
  const int rows = min(a.rows, a.all_rows);
  const int64_t items = static_cast<int64_t>(notes) * rows * (a.d / 4);
  return with_groups(items, a.by_segment ? ctas / notes : 1, items <= (1 << 16), [&](auto g) {
    constexpr int kGroups = decltype(g)::value, kPer = kMergeThreads / kGroups;
    const dim3 grid(static_cast<unsigned>(notes),
                    static_cast<unsigned>((rows * (a.d / 4) + kPer - 1) / kPer));
    auto kernel = a.d == 64    ? paged_merge_kernel<64, kGroups>
                  : a.d == 128 ? paged_merge_kernel<128, kGroups>
                  : a.d == 256 ? paged_merge_kernel<256, kGroups>
                               : paged_merge_kernel<512, kGroups>;
    return launch_pdl(kernel, grid, dim3(kMergeThreads), 0, s, a);
  });
}

cudaError_t launch_paged_finish(const PagedArgs& a, int ctas, cudaStream_t s) {
  // (92 against 93 us a step with 9 pieces of the prefix and 131 K items)
  const int segments = a.B * a.heads;
  const int64_t items = static_cast<int64_t>(segments) * a.rows * (a.d / 4);
  return with_groups(items, a.pre_splits + ctas / segments, a.pre_splits >= 3, [&](auto g) {
    constexpr int kGroups = decltype(g)::value, kPer = kMergeThreads / kGroups;
    const dim3 grid(static_cast<unsigned>(segments),
                    static_cast<unsigned>((a.rows * (a.d / 4) + kPer - 1) / kPer));
    auto kernel = a.d == 64 ? paged_finish_kernel<64, kGroups> : paged_finish_kernel<128, kGroups>;
    return launch_pdl(kernel, grid, dim3(kMergeThreads), 0, s, a);
  });
}

}  // namespace attn
