// The shared prefix of a decode batch, attended once for all sequences.
//
// When the sequences of a batch begin with the same cached keys (one system
// prompt, one document, samples of one prompt), a decode step that treats
// them apart reads and multiplies the prefix once per sequence.  Here the
// query rows of all sequences that share a key/value head are stacked into
// one tall problem of rows = B * (H / H_kv) * n_q against the prefix: the
// prefix is read once, and the product is a matrix product with up to
// thousands of rows.  It leaves, per row, O normalised over the prefix and
// L = logsumexp of its scores there; the decode step over the sequences' own
// keys folds them in by L = log(e^L1 + e^L2), O = e^(L1 - L) O1 + e^(L2 - L) O2.
//
// Bound: at 256 rows a CTA does 4 * 256 * d operations per 4 d bytes, close
// to the ridge, and the prefix comes from L2 after the first row block, so
// the tensor cores bound it from a few hundred rows on; below, HBM.
//
// Mapping: a CTA takes two 128-row query tiles A, B of one key/value head and
// one piece of the prefix's 128-key tiles (pieces: as many as fill the SMs).
//   warps 0-3, 4-7  softmax of A, B: gather and store their tile's query rows
//                   in swizzled shared memory, then per key tile read S from
//                   TMEM, mask, exponentiate, write P (bf16) over S; O is
//                   rescaled in TMEM only when a row's max has grown by 2^8
//   warp 8          copies: K, V pages into a ring of stages, one lane per page
//   warp 9          MMA issue: O_A += P_A V, S_A' = Q_A K', O_B += ..., S_B' = ...
//                   so one tile's softmax runs under the other's products
// A query row's own limit (its cache length, or its position when causal)
// masks the prefix too, so a sequence shorter than the prefix is right; value
// rows past every sequence's end and past the prefix are zeroed in shared
// memory, because 0 * NaN would spread what lies there.
// P is rounded to bf16 (relative 2^-8 per element); m, l, O are fp32.
//
// Measured: 4096 rows (128 sequences, 32 heads over 8) against 16384 keys, d =
// 128, in about 28 us = 1.2 PFLOP/s; a CTA's tile pair takes 2900 cycles a key
// tile, of which its MMAs fill 2100: the chain S, softmax (1070 cycles), P V of
// one tile is longer than the other tile's MMAs that run under it.
#include "attn_paged.cuh"

namespace attn {
using namespace sm103;

namespace {


template <int D>
struct PrefixCfg {
  static constexpr int kBoxes = D / 64;
  static constexpr int kBoxBytes = kTile * 128;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr int kSmem = 1024 + kTileBytes * (2 + 2 * kStages);
  static constexpr uint32_t kSCol = 0, kOCol = 256;   // S_X at 128 X, O_X at 256 + D X
  // registers re-split after the start: 256 * 208 + 128 * 88 <= 384 * 168 (216 and
  // 72: 86.9 against 86.4 us a step; 224 and 56: 87.8)
  static constexpr int kThreads = 384;
  static constexpr uint32_t kRegsLaunch = 168, kRegsSoftmax = 208, kRegsOther = 88;
  static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= kThreads * kRegsLaunch,
                "register re-split exceeds the launch allocation");
};

template <int ST>
struct PrefixCtl {
  uint64_t qfull, kfull[ST], vfull[ST], kempty[ST], vempty[ST];
  uint64_t sfull[2], pfull[2], done, final_bar;
  uint32_t tmem_base;
  int abort_flag;
};

template <int D>
__global__ void __launch_bounds__(PrefixCfg<D>::kThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                  const PrefixArgs a) {
  using C = PrefixCfg<D>;
  constexpr int ST = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = smem + 2 * C::kTileBytes;
  uint8_t* sV = sK + ST * C::kTileBytes;
  __shared__ PrefixCtl<ST> ctl;

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const int hk = blockIdx.x % a.H_kv, pair = blockIdx.x / a.H_kv, piece = blockIdx.y;
  const int r0 = pair * 2 * kTile;
  const bool two = r0 + kTile < a.rows;   // there is a second query tile
  const int t0 = static_cast<int>(static_cast<int64_t>(a.tiles) * piece / a.splits);
  const int n = static_cast<int>(static_cast<int64_t>(a.tiles) * (piece + 1) / a.splits) - t0;

  if (threadIdx.x == 0) {
    ctl.abort_flag = 0;
    mbar_init(&ctl.qfull, 8);
    for (int s = 0; s < ST; ++s) {
      mbar_init(&ctl.kfull[s], 1);
      mbar_init(&ctl.vfull[s], 1);
      mbar_init(&ctl.kempty[s], 1);
      mbar_init(&ctl.vempty[s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&ctl.sfull[x], 1);
      mbar_init(&ctl.pfull[x], 4);
    }
    mbar_init(&ctl.done, 1);
    mbar_init(&ctl.final_bar, 1);
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(&ctl.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // In this order: the decode kernel behind this one does not wait for it before
  // it reads and writes (attn_paged.cu), it relies on every CTA here having
  // waited for what comes before.
  grid_dep_wait();
  grid_dep_launch();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl.tmem_base, 0);
  const WaitCtx wc{&ctl.abort_flag, a.status, a.timeout_ns};
  const int wg = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) / 128, 0);

  if (wg == 2) {
    regs_decrease<C::kRegsOther>();
    if (warp == 8) {
      // ---------------------------------------------------------- copies
      // keys at or past `end` belong to no sequence; those before it are named by
      // the row of the longest sequence (the first of equals), which holds them all
      int end = 0, from = 0;
      for (int b = lane; b < a.B; b += 32) {
        const int len = a.key_lens[b];
        if (len > end) end = len, from = b;
      }
      const int most = __reduce_max_sync(0xffffffffu, end);
      from = __reduce_min_sync(0xffffffffu, end == most ? from : a.B - 1);
      end = min(most, a.shared_len);
      const int32_t* table = a.table + from * a.table_stride;
      const int rows = min(kTile, 1 << a.page_shift);   // keys per copy
      const int parts = kTile / rows;
      bool ok = true;
      int t = 0;
      for (; t < n; ++t) {
        const int s = t % ST;
        const int k0 = (t0 + t) * kTile;
        const int key = k0 + lane * rows;
        const bool mine = lane < parts && key < end;   // this lane's page of the tile
        int page = 0;
        if (mine) page = checked_page(table[key >> a.page_shift], a.num_pages, a.status);
        // (the keys are free once both tiles' scores are complete, a tile's
        // products before the values)
        if (t >= ST && !(ok = __all_sync(0xffffffffu, mbar_wait(&ctl.kempty[s], ((t / ST) - 1) & 1, wc,
                                                                kSitePrefixFree))))
          break;
        uint8_t* dk = sK + s * C::kTileBytes;
        uint8_t* dv = sV + s * C::kTileBytes;
        const int copies = __popc(__ballot_sync(0xffffffffu, mine));
        const uint32_t bytes = static_cast<uint32_t>(copies * rows * D * 2);
        if (lane == 0) mbar_arrive_expect_tx(&ctl.kfull[s], bytes);
        __syncwarp();
        const int row = key & ((1 << a.page_shift) - 1);
        if (mine) {
#pragma unroll
          for (int x = 0; x < C::kBoxes; ++x)
            tma_load_4d(dk + x * C::kBoxBytes + lane * rows * 128, &tk, &ctl.kfull[s], x * 64, row,
                        hk, page);
        }
        if (t >= ST && !(ok = __all_sync(0xffffffffu, mbar_wait(&ctl.vempty[s], ((t / ST) - 1) & 1, wc,
                                                                kSitePrefixFree))))
          break;
        // value rows past `end` that no copy writes are zeroed before the
        // barrier's arrive, those inside a copied page after the copy (below)
        if (copies < parts) {
          for (int i = lane; i < (kTile - copies * rows) * (D / 8); i += 32) {
            const int j = copies * rows + i / (D / 8), c8 = i % (D / 8);
            *reinterpret_cast<uint4*>(dv + (c8 >> 3) * C::kBoxBytes + j * 128 + ((c8 & 7) << 4)) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive_expect_tx(&ctl.vfull[s], bytes);
        __syncwarp();
        if (mine) {
#pragma unroll
          for (int x = 0; x < C::kBoxes; ++x)
            tma_load_4d(dv + x * C::kBoxBytes + lane * rows * 128, &tv, &ctl.vfull[s], x * 64, row,
                        hk, page);
        }
      }
      if (!ok && lane == 0) {   // let issued copies land before the CTA exits
        for (int u = max(0, t - ST); u < t; ++u) {
          mbar_wait_drain(&ctl.kfull[u % ST], (u / ST) & 1, a.timeout_ns);
          mbar_wait_drain(&ctl.vfull[u % ST], (u / ST) & 1, a.timeout_ns);
        }
        // (tile t's keys perhaps, which have gone out when kempty was passed)
        if (mbar_test(&ctl.kempty[t % ST], ((t / ST) - 1) & 1))
          mbar_wait_drain(&ctl.kfull[t % ST], (t / ST) & 1, a.timeout_ns);
      }
    } else if (warp == 9) {
      // ------------------------------------------------------- MMA issue
      int end = 0;
      for (int b = lane; b < a.B; b += 32) end = max(end, a.key_lens[b]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) end = max(end, __shfl_xor_sync(0xffffffffu, end, o));
      end = min(end, a.shared_len);
      const int rows = min(kTile, 1 << a.page_shift);
      // One elected lane issues, in code that the whole warp runs, so that the
      // descriptors stay in uniform registers: a group of eight MMAs goes out
      // in 520 cycles instead of 900, which had bound the kernel.
      constexpr uint32_t kIdS = idesc_bf16(128, 128, false, false);
      constexpr uint32_t kIdO = idesc_bf16(128, D, false, true);
      const bool one = elect_one_lane();
      auto scores = [&](int x, int s) {
        const uint64_t dq = smem_desc(smem_u32(sQ + x * C::kTileBytes), 16, 1024);
        const uint64_t dk = smem_desc(smem_u32(sK + s * C::kTileBytes), 16, 1024);
        if (one) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t off = static_cast<uint64_t>(((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4);
            mma_ss(tmem + C::kSCol + 128 * x, dq + off, dk + off, kIdS, kk > 0 ? 1u : 0u);
          }
          mma_commit(&ctl.sfull[x]);
        }
      };
      // the whole warp walks the tiles (it zeroes value rows)
      const int tiles_x[2] = {n, two ? n : 0};
      bool ok = n == 0 || __all_sync(0xffffffffu, mbar_wait(&ctl.qfull, 0, wc, kSitePrefixQ));
      if (ok && n > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&ctl.kfull[0], 0, wc, kSitePrefixK));
        tc_fence_after();
        if (ok) {
          scores(0, 0);
          if (two) scores(1, 0);
          if (one) mma_commit(&ctl.kempty[0]);
        }
      }
      for (int t = 0; ok && t < n; ++t) {
        const int s = t % ST, s1 = (t + 1) % ST;
        ok = __all_sync(0xffffffffu, mbar_wait(&ctl.vfull[s], (t / ST) & 1, wc, kSitePrefixV));
        if (!ok) break;
        // a page that ends past `end`: zero its value rows there
        const int k0 = (t0 + t) * kTile;
        if (end > k0 && end < k0 + kTile && ((end - k0) & (rows - 1)) != 0) {
          uint8_t* dv = sV + s * C::kTileBytes;
          const int from = end - k0, to = (from + rows - 1) / rows * rows;
          for (int i = lane; i < (to - from) * (D / 8); i += 32) {
            const int j = from + i / (D / 8), c8 = i % (D / 8);
            *reinterpret_cast<uint4*>(dv + (c8 >> 3) * C::kBoxBytes + j * 128 + ((c8 & 7) << 4)) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        const bool more = t + 1 < n;
        bool k_ready = false;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (tiles_x[x] == 0) continue;
          ok = __all_sync(0xffffffffu, mbar_wait(&ctl.pfull[x], t & 1, wc, kSitePrefixP));
          if (!ok) break;
          tc_fence_after();
          const uint64_t dv = smem_desc(smem_u32(sV + s * C::kTileBytes), C::kBoxBytes, 1024);
          if (one) {   // O_X += P_X V
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
              mma_ts(tmem + C::kOCol + D * x, tmem + C::kSCol + 128 * x + kk * 8,
                     dv + static_cast<uint64_t>((kk * 2048) >> 4), kIdO, t > 0 || kk > 0 ? 1u : 0u);
            if (x == (two ? 1 : 0)) mma_commit(&ctl.vempty[s]);
          }
          if (more) {
            if (!k_ready) {
              ok = k_ready = __all_sync(0xffffffffu, mbar_wait(&ctl.kfull[s1], ((t + 1) / ST) & 1,
                                                               wc, kSitePrefixK));
              if (!ok) break;
              tc_fence_after();
            }
            scores(x, s1);   // S_X of the next key tile
            if (one && x == (two ? 1 : 0)) mma_commit(&ctl.kempty[s1]);
          }
        }
      }
      if (one) {
        if (ok) mma_commit(&ctl.done);
        mma_commit(&ctl.final_bar);   // every MMA of this CTA done before TMEM is freed
        mbar_wait_drain(&ctl.final_bar, 0, a.timeout_ns);
      }
      __syncwarp();
    }
  } else {
    regs_increase<C::kRegsSoftmax>();
    // ------------------------------------------------- query rows, softmax
    const int x = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const int r = r0 + x * kTile + row;          // row of the key/value head's stack
    const bool live = r < a.rows;
    const int per = a.group * a.n_q;
    const int b = live ? r / per : 0;
    const int rem = live ? r - b * per : 0;
    const int hl = rem / a.n_q, qt = rem - hl * a.n_q, h = hk * a.group + hl;
    {
      // the warp's 32 rows, kPerRow lanes a row (asynchronous copies: all are
      // in flight together); rows past the last are zero
      constexpr int kPerRow = D / 8, kAtOnce = 32 / kPerRow;
      const int64_t mine = b * a.stride_b + h * a.stride_h + static_cast<int64_t>(qt) * a.stride_n;
      uint8_t* dst = sQ + x * C::kTileBytes + (warp & 3) * 32 * 128;
      const int c8 = lane % kPerRow;
#pragma unroll
      for (int i = 0; i < kPerRow; ++i) {
        const int rr = i * kAtOnce + lane / kPerRow;
        const int64_t from = __shfl_sync(0xffffffffu, mine, rr);
        const bool there = __shfl_sync(0xffffffffu, live ? 1 : 0, rr) != 0;
        copy16_async(dst + (c8 >> 3) * C::kBoxBytes + rr * 128 + (((c8 & 7) ^ (rr & 7)) << 4),
                     a.q + from + c8 * 8, there);
      }
      copies_wait();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.qfull);
    }
    int lim = 0;   // keys below lim are allowed
    if (live) {
      lim = min(max(a.key_lens[b], 0), a.cap);
      if (a.causal) lim = min(lim, lim - a.n_q + qt + 1);
      lim = min(lim, a.shared_len);
    }
    const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t sc = tl + C::kSCol + 128 * x, oc = tl + C::kOCol + D * x;
    const float c2 = a.scale_log2;
    float m_used = -INFINITY, l_sum = 0.f;
    const int mine = x == 0 || two ? n : 0;
    bool ok = true;
    for (int t = 0; t < mine; ++t) {
      ok = __all_sync(0xffffffffu, mbar_wait(&ctl.sfull[x], t & 1, wc, kSitePrefixS));
      if (!ok) break;
      tc_fence_after();
      uint32_t sr[128];
#pragma unroll
      for (int c = 0; c < 128; c += 32) tmem_ld32(sc + c, sr + c);
      tmem_wait_ld();
      const int col_lim = lim - (t0 + t) * kTile;
      if (col_lim < kTile) {
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c >= col_lim) sr[c] = __float_as_uint(-INFINITY);
      }
      float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
      for (int c = 0; c < 128; c += 8) {
        mx0 = max3f(mx0, __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
        mx1 = max3f(mx1, __uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3]));
        mx2 = max3f(mx2, __uint_as_float(sr[c + 4]), __uint_as_float(sr[c + 5]));
        mx3 = max3f(mx3, __uint_as_float(sr[c + 6]), __uint_as_float(sr[c + 7]));
      }
      const float m_new = max3f(m_used, max3f(mx0, mx1, mx2), mx3);
      const bool need =
          m_new > m_used && (m_used == -INFINITY || (m_new - m_used) * c2 > kRescaleTau);
      float alpha = 1.f;
      if (need) {
        alpha = ex2_approx((m_used - m_new) * c2);
        m_used = m_new;
        l_sum *= alpha;
      }
      const float mc = m_used == -INFINITY ? 0.f : m_used * c2;
      const uint64_t c2x2 = f2_pack(c2, c2), nmc2 = f2_pack(-mc, -mc);
      uint64_t acc0 = f2_pack(0.f, 0.f), acc1 = acc0;
#pragma unroll
      for (int c = 0; c < 128; c += 32) {
        uint32_t pk[16];
#pragma unroll
        for (int u = 0; u < 32; u += 4) {
          float x0, x1, x2, x3;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[c + u]), __uint_as_float(sr[c + u + 1])), c2x2,
                           nmc2), x0, x1);
          f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[c + u + 2]), __uint_as_float(sr[c + u + 3])),
                           c2x2, nmc2), x2, x3);
          const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
          const float p2 = ex2_approx(x2), p3 = ex2_approx(x3);
          acc0 = f2_add(acc0, f2_pack(p0, p1));
          acc1 = f2_add(acc1, f2_pack(p2, p3));
          pk[u / 2] = pack_bf16x2(p0, p1);
          pk[u / 2 + 1] = pack_bf16x2(p2, p3);
        }
        tmem_st16(sc + c / 2, pk);   // S columns [c / 2, c / 2 + 16) are already in registers
      }
      // "S of this tile is complete" implies that O holds the sum through
      // the tile before (one thread issues the MMAs in order)
      if (t >= 1 && __any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_ld32(oc + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * alpha);
          tmem_st32(oc + c, o);
        }
      }
      float s0, s1, s2, s3;
      f2_unpack(acc0, s0, s1);
      f2_unpack(acc1, s2, s3);
      l_sum += (s0 + s2) + (s1 + s3);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      // (an armed test stall: warp 0 withholds its first arrive, so the MMA warp's
      // wait runs out)
      if (lane == 0 && !(a.stall != 0 && warp == 0 && t == 0)) mbar_arrive(&ctl.pfull[x]);
    }
    if (ok && mine > 0) {
      ok = __all_sync(0xffffffffu, mbar_wait(&ctl.done, 0, wc, kSitePrefixDone));
      tc_fence_after();
    }
    // (after a time-out the outputs are undefined, but written)
    const bool some = l_sum != 0.f;
    const float inv = some ? 1.f / l_sum : 0.f;
    const int64_t rows_all = static_cast<int64_t>(a.B) * a.H * a.n_q;
    const int64_t out = piece * rows_all + (static_cast<int64_t>(b) * a.H + h) * a.n_q + qt;
    // O through shared memory (q, k, v are done with), so that a row goes out in
    // one piece: a thread's own stores of its row had taken 5 us
    constexpr int kStride = D + 4;   // floats; the pad spreads the rows over the banks
    static_assert(256 * kStride * 4 <= C::kSmem - 1024, "O fits where the operands were");
    float* mine_o = reinterpret_cast<float*>(smem) + warp * 32 * kStride;
    // (every warp of the two groups is past its last use of them: `done` covers
    // the products; a group without a tile has none)
    named_barrier_sync(1, 256);
#pragma unroll
    for (int c = 0; c < D; c += 32) {
      uint32_t o[32];
      if (mine > 0) {   // (uniform over the warp)
        tmem_ld32(oc + c, o);
        tmem_wait_ld();
      }
      float4* dst = reinterpret_cast<float4*>(mine_o + lane * kStride + c);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        dst[u] = mine > 0 && some
                     ? make_float4(__uint_as_float(o[4 * u]) * inv, __uint_as_float(o[4 * u + 1]) * inv,
                                   __uint_as_float(o[4 * u + 2]) * inv, __uint_as_float(o[4 * u + 3]) * inv)
                     : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncwarp();
    constexpr int kLanes = D / 4;   // float4 lanes a row
#pragma unroll 4
    for (int i = 0; i < kLanes; ++i) {
      const int rr = i * (32 / kLanes) + lane / kLanes, c = lane % kLanes;
      const int64_t to = __shfl_sync(0xffffffffu, out, rr);
      const bool there = __shfl_sync(0xffffffffu, live ? 1 : 0, rr) != 0;
      if (there)
        *reinterpret_cast<float4*>(a.pre_o + to * D + 4 * c) =
            *reinterpret_cast<const float4*>(mine_o + rr * kStride + 4 * c);
    }
    if (live) a.pre_l[out] = some ? fmaf(m_used, a.scale, logf(l_sum)) : -INFINITY;
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch_d(const CUtensorMap& tk, const CUtensorMap& tv, const PrefixArgs& a,
                     cudaStream_t s) {
  using C = PrefixCfg<D>;
  static std::atomic<uint64_t> set_up{0};
  int dev = 0;
  bool todo = false;
  cudaError_t e = needs_setup(set_up, &dev, &todo);
  if (e != cudaSuccess) return e;
  if (todo) {
    e = cudaFuncSetAttribute(prefix_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    // the register re-split inside the kernel assumes the launch allocation
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, prefix_kernel<D>)) != cudaSuccess) return e;
    if (static_cast<uint32_t>(fa.numRegs) < C::kRegsLaunch) return cudaErrorInvalidConfiguration;
    mark_done(set_up, dev);
  }
  const int pairs = (a.rows + 2 * kTile - 1) / (2 * kTile);
  const dim3 grid(static_cast<unsigned>(pairs * a.H_kv), static_cast<unsigned>(a.splits));
  return launch_pdl(prefix_kernel<D>, grid, dim3(C::kThreads), C::kSmem, s, tk, tv, a);
}

}  // namespace

cudaError_t launch_prefix(const CUtensorMap& tk, const CUtensorMap& tv, const PrefixArgs& a,
                          cudaStream_t s) {
  return a.d == 64 ? launch_d<64>(tk, tv, a, s) : launch_d<128>(tk, tv, a, s);
}

}  // namespace attn
