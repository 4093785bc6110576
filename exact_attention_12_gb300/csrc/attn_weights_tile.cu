// The attention weight that cached keys receive from many query rows (an
// observation window, a batch of drafts): attn_weights.cu's sum on the tensor cores.
//
// With hundreds of rows a key/value head the products and the exponentials take
// longer than the keys' way here, and warp MMAs reach a quarter of what tcgen05
// does.  A CTA takes a run of a head's 128-key tiles; all its query rows stay in
// shared memory (in passes of 512).  Per tile and block of 128 rows
//   S^T = K Q^T    one 128 x N x d product into one of the two TMEM stages of the
//                  group of warps whose tile it is,
//   W += sum_r exp(c S^T - L_r)
// with the keys as TMEM's lanes, so that a thread has a key and sums over its own
// columns: no exchange between lanes, and rows of K that hold nothing (a page's
// end, a place the copies left out) reach no other key.
//   warps 0-3, 4-7   every other tile's exponentials and sums
//   warp 8           MMA issue
//   warp 9           copies: K pages into a ring, one lane per page (TMA, swizzled)
//   warps 9-12       of a cache in 4 bits: a key a thread, unpacked to fp16 (exactly)
//                    and stored where TMA would have put it
// Bound: the exponentials and what goes with them (a part of them by a polynomial
// instead of ex2 was slower, 29.6 against 26.7 us at 512 rows); below about 100 rows
// HBM.
//
// Measured: two prompts of 16384 keys under their last 32 queries, 32 heads over 8, d =
// 128 (128 rows a head), 67 MB in 18.5 us: 13 us of a CTA's tiles, the rest the launch,
// Q, and the first tile's way here.  512 rows a head, 34 GFLOP, 20.7 us.
// 16 sequences of 8192 keys, 8 heads, 128 rows: 61 us (floor 41), of a cache in 4 bits 80
// (18): a thread's 64 bytes of a key lie a key apart from its neighbour's, and the packed
// variant spills 96 bytes at 128 registers.
#include "attn_fp4.cuh"

namespace attn {
using namespace sm103;

namespace {

constexpr int kSumWarps = 8;                 // two groups of four
constexpr int kMmaWarp = 8, kCopyWarp = 9;
constexpr int kGroupStages = 2;              // of scores in TMEM, per group of warps
constexpr int kTmemStages = 2 * kGroupStages;
constexpr int kMaxRing = 4;
constexpr int kRowsAtOnce = 128;             // rows of a block
constexpr int kUnpackThreads = 128;
constexpr int kRowBytes = 12;                // what is kept of a row beside Q: see the kernel

template <int D, bool PACKED>
struct TileCfg {
  static constexpr int kThreads = 32 * kCopyWarp + (PACKED ? kUnpackThreads : 32);
  static constexpr int kBoxBytes = 128 * 128;          // 64 columns of 128 rows
  static constexpr int kTileBytes = D / 64 * kBoxBytes;   // of keys, and of a block of Q
  static constexpr int kMaxBlocks = 512 / D;
  static constexpr int kMaxSmem = 1024 + 6 * 128 * D * 2 + kMaxBlocks * kRowsAtOnce * kRowBytes;
};

struct TileCtl {
  uint64_t kfull[kMaxRing], kempty[kMaxRing];
  uint64_t sfull[kTmemStages], sempty[kTmemStages];
  uint64_t final_bar;
  uint32_t tmem_base;
  int abort_flag;
};

// Instruction descriptor as idesc_bf16, with fp16 operands (format code 0).
__device__ __forceinline__ uint32_t idesc_half(int M, int N) {
  return (1u << 4) | ((static_cast<uint32_t>(N) >> 3) << 17) | ((static_cast<uint32_t>(M) >> 4) << 24);
}

// Whether x holds for any thread of the summing warps.
__device__ __forceinline__ bool any_of_sums(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "barrier.cta.red.or.pred p, 2, %2, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(x ? 1u : 0u), "n"(32 * kSumWarps)
      : "memory");
  return r != 0;
}

// A position in a ring of n stages, over the whole kernel.
struct RingAt {
  int stage = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void next(int n) {
    if (++stage == n) {
      stage = 0;
      ++round;
    }
  }
};

template <int D, bool PACKED>
__global__ void __launch_bounds__(TileCfg<D, PACKED>::kThreads, 1)
    key_weights_tile_kernel(const __grid_constant__ CUtensorMap tk, const PagedArgs a,
                            const WeightArgs f) {
  using C = TileCfg<D, PACKED>;
  constexpr int kPerRow = D / 8;   // 16-byte pieces
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int ring = f.ring, blocks_max = f.pass_rows / kRowsAtOnce;
  uint8_t* sQ = smem;
  uint8_t* sK = smem + blocks_max * C::kTileBytes;
  // of each row: -L in log2 units (-inf where it gives nothing), what turns a score
  // into them, the keys that it attends
  float* row_l = reinterpret_cast<float*>(sK + ring * C::kTileBytes);
  float* row_c = row_l + f.pass_rows;
  int* row_lim = reinterpret_cast<int*>(row_c + f.pass_rows);
  __shared__ TileCtl ctl;

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    ctl.abort_flag = 0;
    for (int s = 0; s < kMaxRing; ++s) {
      mbar_init(&ctl.kfull[s], PACKED ? kUnpackThreads / 32 : 1);
      mbar_init(&ctl.kempty[s], 1);
    }
    for (int s = 0; s < kTmemStages; ++s) {
      mbar_init(&ctl.sfull[s], 1);
      mbar_init(&ctl.sempty[s], 4);
    }
    mbar_init(&ctl.final_bar, 1);
    fence_mbar_init();
  }
  if (!PACKED && threadIdx.x == 32 * kCopyWarp) tma_prefetch_desc(&tk);
  if (warp == kMmaWarp) {
    tmem_alloc(&ctl.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_wait();
  grid_dep_launch();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl.tmem_base, 0);
  const WaitCtx wc{&ctl.abort_flag, a.status, a.timeout_ns};
  const PagedShare share =
      paged_share<kTile, kWeightTileOverhead, 1>(a, blockIdx.x, gridDim.x);

  RingAt k_at;         // the next tile's place
  RingAt s_at[2];      // the next score block's, of each group (a stage is one group's only,
                       // so no wait can fall a round behind)
  int k_seen = 0;      // tiles so far: whose turn it is
  bool ok = true;
  for (PagedPiece p = paged_piece<kTile, kWeightTileOverhead>(a, share, share.b, 0, share.s);
       ok && p.valid; p = paged_next<kTile, kWeightTileOverhead>(a, share, p)) {
    const int n = p.t1 - p.t0;
    if (n == 0) continue;
    for (int r0 = 0; ok && r0 < a.head_rows; r0 += f.pass_rows) {
      const int nrows = min(a.head_rows - r0, f.pass_rows);
      const int blocks = (nrows + kRowsAtOnce - 1) / kRowsAtOnce;
      // ---- Q and its rows' limits; what lies past the last row is zero.  A row that gives
      // nothing may hold anything, and an infinite key makes NaN of zeros as well: where
      // there is one, what a row gives is chosen by its limit.
      // (the scores of the pass before have all been read, so its products are complete)
      bool some_dead = false;
      if (warp < kSumWarps) {
        for (int i = threadIdx.x; i < blocks * kRowsAtOnce * kPerRow; i += 32 * kSumWarps) {
          const int r = i / kPerRow, c8 = i % kPerRow, at = p.h * a.head_rows + r0 + r;
          const bool live = r < nrows;
          const int h = at / a.n_q, qt = at - h * a.n_q;
          const __nv_bfloat16* from = a.q + p.b * a.stride_b + h * a.stride_h +
                                      static_cast<int64_t>(qt) * a.stride_n + 8 * c8;
          const int in = r % kRowsAtOnce;
          uint8_t* to = sQ + r / kRowsAtOnce * C::kTileBytes + (c8 >> 3) * C::kBoxBytes + in * 128 +
                        (((c8 & 7) ^ (in & 7)) << 4);
          float c2 = 0.f;
          if constexpr (PACKED) {   // as half_rows, over the row's kPerRow lanes
            const uint4 x = live ? *reinterpret_cast<const uint4*>(from) : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[k] << 16)),
                                     fabsf(__uint_as_float(w[k] & 0xffff0000u))));
#pragma unroll
            for (int o = 1; o < kPerRow; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const int e = row_exponent(top);
            const float up = ldexpf(1.f, e);
            uint32_t y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              y[k] = pack_half2(__uint_as_float(w[k] << 16) * up, __uint_as_float(w[k] & 0xffff0000u) * up);
            *reinterpret_cast<uint4*>(to) = make_uint4(y[0], y[1], y[2], y[3]);
            c2 = score_factor(a.scale_log2 * f.k_descale, e);
          } else {
            copy16_async(to, live ? from : a.q, live);
          }
          if (PACKED && c8 == 0) row_c[r] = c2;
        }
        bool dead = false;
        for (int r = threadIdx.x; r < blocks * kRowsAtOnce; r += 32 * kSumWarps) {
          const int at = p.h * a.head_rows + r0 + r;
          const float L = r < nrows ? f.lse[static_cast<int64_t>(p.b) * a.all_rows + at] : -INFINITY;
          const bool gives = L != -INFINITY;
          dead = dead || (r < nrows && !gives);
          row_l[r] = gives ? -L * kLog2Of : -INFINITY;
          row_lim[r] =
              gives ? (a.causal ? min(p.len, p.len - a.n_q + at % a.n_q + 1) : p.len) : 0;
        }
        some_dead = any_of_sums(dead);
        copies_wait();
        fence_proxy_async_smem();
      }
      // (the copies need not wait for Q)
      if (warp <= kMmaWarp) named_barrier_sync(1, 32 * (kMmaWarp + 1));
      if (warp < kSumWarps) {
        // ------------------------------------------------ exponentials, sums
        const int group = warp >> 2;
        RingAt& mine = s_at[0];
        const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        // every row attends keys below it
        const int open = some_dead ? 0 : a.causal ? p.len - a.n_q + 1 : p.len;
        const bool add = f.add || r0 > 0;
        for (int t = 0; ok && t < n; ++t, ++k_seen) {
          if ((k_seen & 1) != group) continue;
          const int k0 = (p.t0 + t) * kTile, key = k0 + (warp & 3) * 32 + lane;
          float* to = f.weights + p.b * f.stride_b + p.h * f.stride_h + key;
          const float before = add && key < p.len ? *to : 0.f;
          uint64_t sum2[4];   // packed pairs
#pragma unroll
          for (int i = 0; i < 4; ++i) sum2[i] = f2_pack(0.f, 0.f);
          for (int x = 0; x < blocks; ++x) {
            ok = __all_sync(0xffffffffu, mbar_wait(&ctl.sfull[kGroupStages * group + mine.stage],
                                                   mine.round & 1, wc, kSiteWeightsS));
            if (!ok) break;
            tc_fence_after();
            const int first = x * kRowsAtOnce, count = min(kRowsAtOnce, nrows - first);
            const uint32_t sc = tl + (kGroupStages * group + mine.stage) * kRowsAtOnce;
            const bool whole = k0 + kTile <= open;   // every row attends every key of the tile
            // 32 rows' scores s; the next ones are on their way
            auto take = [&](const uint32_t* s, int c) {
              const bool masked = !whole || c + 32 > count;
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const float4 l = *reinterpret_cast<const float4*>(&row_l[first + c + i]);
                float4 k = make_float4(a.scale_log2, a.scale_log2, a.scale_log2, a.scale_log2);
                if constexpr (PACKED) k = *reinterpret_cast<const float4*>(&row_c[first + c + i]);
                float y[4];
                f2_unpack(f2_fma(f2_pack(__uint_as_float(s[i]), __uint_as_float(s[i + 1])),
                                 f2_pack(k.x, k.y), f2_pack(l.x, l.y)), y[0], y[1]);
                f2_unpack(f2_fma(f2_pack(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])),
                                 f2_pack(k.z, k.w), f2_pack(l.z, l.w)), y[2], y[3]);
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = ex2_approx(y[j]);
                if (masked) {
                  const int4 lim = *reinterpret_cast<const int4*>(&row_lim[first + c + i]);
                  y[0] = key < lim.x ? y[0] : 0.f;
                  y[1] = key < lim.y ? y[1] : 0.f;
                  y[2] = key < lim.z ? y[2] : 0.f;
                  y[3] = key < lim.w ? y[3] : 0.f;
                }
                sum2[i / 2 & 3] = f2_add(sum2[i / 2 & 3], f2_pack(y[0], y[1]));
                sum2[(i / 2 + 1) & 3] = f2_add(sum2[(i / 2 + 1) & 3], f2_pack(y[2], y[3]));
              }
            };
            uint32_t s[2][32];
            tmem_ld32(sc, s[0]);
#pragma unroll
            for (int c = 0; c < kRowsAtOnce; c += 32) {
              if (c >= count) break;   // (uniform)
              tmem_wait_ld();
              if (c + 32 < count) tmem_ld32(sc + c + 32, s[(c / 32 + 1) & 1]);
              take(s[c / 32 & 1], c);
            }
            tc_fence_before();
            __syncwarp();
            // (an armed test stall: warp 0 withholds its first arrive)
            if (lane == 0 && !(f.stall != 0 && warp == 0 && t == 0))
              mbar_arrive(&ctl.sempty[kGroupStages * group + mine.stage]);
            mine.next(kGroupStages);
          }
          float sum[2];
          f2_unpack(f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3])), sum[0], sum[1]);
          if (ok && key < p.len) *to = before + (sum[0] + sum[1]);
        }
      } else if (warp == kMmaWarp) {
        // --------------------------------------------------------- MMA issue
        const bool one = elect_one_lane();
        for (int t = 0; ok && t < n; ++t, ++k_seen) {
          ok = __all_sync(0xffffffffu, mbar_wait(&ctl.kfull[k_at.stage], k_at.round & 1, wc, kSiteWeightsK));
          if (!ok) break;
          const uint64_t dk = smem_desc(smem_u32(sK + k_at.stage * C::kTileBytes), 16, 1024);
          const int group = k_seen & 1;
          RingAt& at = s_at[group];
          for (int x = 0; x < blocks; ++x) {
            const int stage = kGroupStages * group + at.stage;
            if (at.round > 0 &&
                !(ok = __all_sync(0xffffffffu, mbar_wait(&ctl.sempty[stage], (at.round - 1) & 1,
                                                         wc, kSiteWeightsFree))))
              break;
            tc_fence_after();
            const int cols = (min(kRowsAtOnce, nrows - x * kRowsAtOnce) + 15) & ~15;
            const uint32_t id = PACKED ? idesc_half(kTile, cols) : idesc_bf16(kTile, cols, false, false);
            const uint64_t dq = smem_desc(smem_u32(sQ + x * C::kTileBytes), 16, 1024);
            if (one) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t off = static_cast<uint64_t>(((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4);
                mma_ss(tmem + stage * kRowsAtOnce, dk + off, dq + off, id, kk > 0 ? 1u : 0u);
              }
              mma_commit(&ctl.sfull[stage]);
            }
            at.next(kGroupStages);
          }
          if (!ok) break;
          if (one) mma_commit(&ctl.kempty[k_at.stage]);
          k_at.next(ring);
        }
      } else if constexpr (!PACKED) {
        // ------------------------------------------------------------ copies
        const int per = min(kTile, 1 << a.page_shift);   // keys per copy
        const int32_t* table = a.table + p.b * a.table_stride;
        for (int t = 0; t < n; ++t) {
          const int key = (p.t0 + t) * kTile + lane * per;
          const bool mine = lane < kTile / per && key < p.len;   // this lane's page of the tile
          const int page = mine ? checked_page(table[key >> a.page_shift], a.num_pages, a.status) : 0;
          if (k_at.round > 0 &&
              !(ok = __all_sync(0xffffffffu, mbar_wait(&ctl.kempty[k_at.stage], (k_at.round - 1) & 1,
                                                       wc, kSiteWeightsRing))))
            break;
          const int copies = __popc(__ballot_sync(0xffffffffu, mine));
          if (lane == 0)
            mbar_arrive_expect_tx(&ctl.kfull[k_at.stage], static_cast<uint32_t>(copies * per * D * 2));
          __syncwarp();
          uint8_t* dk = sK + k_at.stage * C::kTileBytes + lane * per * 128;
          if (mine) {
#pragma unroll
            for (int x = 0; x < D / 64; ++x)
              tma_load_4d(dk + x * C::kBoxBytes, &tk, &ctl.kfull[k_at.stage], x * 64,
                          key & ((1 << a.page_shift) - 1), p.h, page);
          }
          k_at.next(ring);
        }
      } else {
        // --------------------------------- keys in 4 bits: unpacked, a thread a key
        const int me = threadIdx.x - 32 * kCopyWarp;
        const int32_t* table = a.table + p.b * a.table_stride;
        uint32_t w[D / 8], units[D / 64];   // codes; four scales a word
        auto load = [&](int t) {
          const int key = (p.t0 + t) * kTile + me;
          int page = a.num_pages;
          if (t < n && key < p.len) page = checked_page(table[key >> a.page_shift], a.num_pages, a.status);
          const bool there = page < a.num_pages;
          const int row = key & ((1 << a.page_shift) - 1);
          const uint4* from = reinterpret_cast<const uint4*>(
              f.cache.codes + (there ? page * f.cache.code_page : 0) + p.h * f.cache.code_head + row * (D / 2));
          const uint32_t* scales = reinterpret_cast<const uint32_t*>(
              f.cache.scales + (there ? page * f.cache.scale_page : 0) + p.h * f.cache.scale_head +
              row * (D / kFp4Block));
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const uint4 x = there ? __ldcs(from + i) : make_uint4(0u, 0u, 0u, 0u);
            w[4 * i] = x.x;
            w[4 * i + 1] = x.y;
            w[4 * i + 2] = x.z;
            w[4 * i + 3] = x.w;
          }
#pragma unroll
          for (int i = 0; i < D / 64; ++i) units[i] = there ? scales[i] : 0u;
        };
        load(0);
        for (int t = 0; t < n; ++t) {
          if (k_at.round > 0 &&
              !(ok = __all_sync(0xffffffffu, mbar_wait(&ctl.kempty[k_at.stage], (k_at.round - 1) & 1,
                                                       wc, kSiteWeightsRing))))
            break;
          uint8_t* dk = sK + k_at.stage * C::kTileBytes + me * 128;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {   // 8 columns, half a scale's
            uint32_t y[4];
            e2m1_to_half(w[i], y);
            const uint32_t unit =
                e4m3_to_half(((units[i >> 3] >> (8 * ((i >> 1) & 3))) & 0xffu) * 0x0101u);
            *reinterpret_cast<uint4*>(dk + (i >> 3) * C::kBoxBytes + (((i & 7) ^ (me & 7)) << 4)) =
                make_uint4(mul_half2(y[0], unit), mul_half2(y[1], unit), mul_half2(y[2], unit),
                           mul_half2(y[3], unit));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl.kfull[k_at.stage]);
          k_at.next(ring);
          if (t + 1 < n) load(t + 1);
        }
      }
      ok = __syncthreads_and(ok);
    }
  }
  if (!ok) {   // let what is in flight land before shared and tensor memory go
    if (!PACKED && warp == kCopyWarp && lane == 0)
      for (int i = 0; i < ring; ++i) {
        // (a stage's last copy: of this round for those in front, of the one before behind)
        const uint32_t round = i < k_at.stage ? k_at.round : k_at.round - 1;
        if (i < k_at.stage || k_at.round > 0) mbar_wait_drain(&ctl.kfull[i], round & 1, a.timeout_ns);
      }
    if (warp == kMmaWarp) {
      if (elect_one_lane()) {
        mma_commit(&ctl.final_bar);
        mbar_wait_drain(&ctl.final_bar, 0, a.timeout_ns);
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool PACKED>
cudaError_t launch_kind(const CUtensorMap& tk, const PagedArgs& a, WeightArgs f, int ctas,
                        cudaStream_t s) {
  using C = TileCfg<D, PACKED>;
  static std::atomic<uint64_t> set_up{0};
  int dev = 0;
  bool todo = false;
  cudaError_t e = needs_setup(set_up, &dev, &todo);
  if (e != cudaSuccess) return e;
  auto kernel = key_weights_tile_kernel<D, PACKED>;
  if (todo) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kMaxSmem);
    if (e != cudaSuccess) return e;
    mark_done(set_up, dev);
  }
  // blocks of 128 rows of a pass, and what is left of six tiles for the keys
  const int blocks = min((a.head_rows + kRowsAtOnce - 1) / kRowsAtOnce, min(C::kMaxBlocks, 4));
  f.pass_rows = blocks * kRowsAtOnce;
  f.ring = min(6 - blocks, kMaxRing);
  const size_t bytes = 1024 + static_cast<size_t>(blocks + f.ring) * C::kTileBytes +
                       static_cast<size_t>(f.pass_rows) * kRowBytes;
  return launch_pdl(kernel, dim3(ctas), dim3(C::kThreads), bytes, s, tk, a, f);
}

}  // namespace

cudaError_t launch_key_weights_tile(const CUtensorMap& tk, const PagedArgs& a, const WeightArgs& f,
                                    int ctas, cudaStream_t s) {
  if (f.k == nullptr)
    return a.d == 64 ? launch_kind<64, true>(tk, a, f, ctas, s) : launch_kind<128, true>(tk, a, f, ctas, s);
  return a.d == 64 ? launch_kind<64, false>(tk, a, f, ctas, s) : launch_kind<128, false>(tk, a, f, ctas, s);
}

}  // namespace attn
