// The decode step against a cache in 4 bits for many query rows (more than 32 of a
// key/value head, d = 128, long caches): attn_fp4.cu's sums on tcgen05.
//
// Warp MMAs need every value unpacked once per 32 rows, and reach a quarter of
// tcgen05's rate: 32 rows of 16384 keys went at 250 clocks for 16 keys (the copy rate
// is 98), 64 rows at 500.  Here each key and value is unpacked once, to fp16 in
// shared memory, and a CTA (one per SM, the keys divided as in attn_paged.cuh) does
// per tile of 128 keys
//   S^T = K Q^T      128 keys x rows, TMEM's lanes are keys
//   P^T = 2^(S c - m)  a thread has a key: no exchange between lanes for a row's
//                    maximum either, as long as no score is 2^8 above the last one
//                    that was taken
//   O^T += V^T P^T   128 columns x rows; V and P lie as they were written, a key's
//                    columns (rows) side by side, which tcgen05 takes as M- and
//                    N-major operands
//   warps 0-15   Q, softmax, write-out: four groups of 16 rows each (two of 32: 348 us)
//   warp 16      MMA issue, the next tile's S before this one's O
//   warps 20-27  unpacking, four K and four V: four lanes a key, their 16 bytes of codes
//                and two scales a tile ahead in registers and six in L2
// 64 sequences of 16384 keys, 4 heads, 64 rows (604 MB): 303 us, 2.0 TB/s; 2900 clocks a
// tile.  Its 7150 warp instructions take 67 % of the issue slots (136 bytes of spills at 72
// registers), its way through shared
// memory (unpacked values in, operands out) 1400 clocks, and the groups go from a score
// to its weight in step; the tensor cores are busy for a sixth.  S and O from two
// issuing warps: 318.
// Rounding and what may lie where no key is attended: as in attn_fp4.cu.
#include "attn_fp4.cuh"

namespace attn {
using namespace sm103;

namespace {

constexpr int kD = 128;
constexpr int kGroups = 4, kSoftWarps = 4;         // softmax groups; warps of one
constexpr int kIssueWarp = 16, kUnpackWarp = 20;   // then four for K, four for V
constexpr int kTileThreads = 32 * (kUnpackWarp + 8);
// registers re-split between the seven warpgroups after the start
constexpr uint32_t kRegsLaunch = 72, kRegsSoft = 80, kRegsIssue = 40;
static_assert(kGroups * kRegsSoft + kRegsIssue + 2 * kRegsLaunch <= 7 * kRegsLaunch,
              "register re-split exceeds the launch allocation");
constexpr int kTileStages = 2;                     // of every ring
constexpr int kRowsMax = 64;
constexpr int kGroupRows = kRowsMax / kGroups;     // rows of a softmax group
constexpr int kBox = kTile * 128;                  // 64 columns of 128 keys
constexpr int kKeysBytes = kD / 64 * kBox;         // a tile's keys, or values
constexpr int kQBox = kRowsMax * 128;
constexpr int kQBytes = kD / 64 * kQBox;
constexpr int kPBytes = kTile * 2 * kRowsMax;
constexpr int kTileSmem = 1024 + kTileStages * (2 * kKeysBytes + kPBytes) + kQBytes;
constexpr uint32_t kSCol = 0, kOCol = kTileStages * kRowsMax, kTmemCols = 256;
constexpr float kNoScore = -3e38f;                 // a row's maximum before its first key
constexpr int kAhead = 6;                          // tiles that are fetched into L2 ahead

struct FpTileCtl {
  uint64_t kfull[kTileStages], kempty[kTileStages], vfull[kTileStages], vempty[kTileStages];
  uint64_t sfull[kTileStages], sempty[kTileStages], pfull[kTileStages], pempty[kTileStages];
  uint64_t qfull, final_bar;
  uint32_t tmem_base;
  int abort_flag;
  // the rows: score -> log2 units, the maximum taken (negative, in them), the keys
  // attended, where O and L go
  alignas(16) float c2[kRowsMax];
  alignas(16) float negm[kRowsMax];
  alignas(16) int lim[kRowsMax];
  alignas(16) float alpha[kRowsMax];   // then O's factor
  int64_t to[kRowsMax];
  float part[kSoftWarps][kRowsMax];
};

// Instruction descriptor: fp16 operands, fp32 accumulators (fields as in idesc_bf16).
__device__ __forceinline__ uint32_t idesc_half(int M, int N, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | ((a_mn_major ? 1u : 0u) << 15) | ((b_mn_major ? 1u : 0u) << 16) |
         ((static_cast<uint32_t>(N) >> 3) << 17) | ((static_cast<uint32_t>(M) >> 4) << 24);
}

// Whether x holds for any thread of softmax group `group`.
__device__ __forceinline__ bool any_of_group(int group, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "barrier.cta.red.or.pred p, %2, 128, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(x ? 1u : 0u), "r"(1 + group)
      : "memory");
  return r != 0;
}

// The largest x of the warp (NaN left out; -inf if nothing else is).
__device__ __forceinline__ float warp_max(float x) {
  const int b = x != x ? __float_as_int(-INFINITY) : __float_as_int(x);
  const int key = b ^ ((b >> 31) & 0x7fffffff);   // in the order of the numbers
  const int top = __reduce_max_sync(0xffffffffu, key);
  return __int_as_float(top ^ ((top >> 31) & 0x7fffffff));
}

// A group's rows of the warp's 32 lanes.
__device__ __forceinline__ void tmem_read(uint32_t at, uint32_t* r) {
  tmem_ld16(at, r);
  tmem_wait_ld();
}

__global__ void __launch_bounds__(kTileThreads, 1)
    fp4_tile_kernel(const PagedArgs a, const Fp4Args f) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sK = smem;
  uint8_t* sV = sK + kTileStages * kKeysBytes;
  uint8_t* sP = sV + kTileStages * kKeysBytes;
  uint8_t* sQ = sP + kTileStages * kPBytes;
  __shared__ FpTileCtl ctl;

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    ctl.abort_flag = 0;
    for (int s = 0; s < kTileStages; ++s) {
      mbar_init(&ctl.kfull[s], 4);
      mbar_init(&ctl.kempty[s], 1);
      mbar_init(&ctl.vfull[s], 4);
      mbar_init(&ctl.vempty[s], 1);
      mbar_init(&ctl.sfull[s], 1);
      mbar_init(&ctl.sempty[s], kGroups * kSoftWarps);
      mbar_init(&ctl.pfull[s], kGroups * kSoftWarps);
      mbar_init(&ctl.pempty[s], 1);
    }
    mbar_init(&ctl.qfull, kGroups * kSoftWarps);
    mbar_init(&ctl.final_bar, 1);
    fence_mbar_init();
  }
  if (warp == kIssueWarp) {
    tmem_alloc(&ctl.tmem_base, kTmemCols);
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
      paged_share<kTile, kFp4TileOverhead, kFp4TileMinUnits>(a, blockIdx.x, gridDim.x);
  PagedPiece p = paged_piece<kTile, kFp4TileOverhead>(a, share, share.b, 0, share.s);
  auto next_piece = [&] { p = paged_next<kTile, kFp4TileOverhead>(a, share, p); };
  // Tiles are counted over all pieces: tile kt is in stage kt % 2, its stage's kt / 2-th.
  auto filled = [&](uint64_t* bar, uint32_t kt, int site) {
    return __all_sync(0xffffffffu, mbar_wait(&bar[kt & 1], (kt >> 1) & 1, wc, site));
  };
  auto freed = [&](uint64_t* bar, uint32_t kt, int site) {   // what was there before kt
    return kt < kTileStages ||
           __all_sync(0xffffffffu, mbar_wait(&bar[kt & 1], ((kt >> 1) - 1) & 1, wc, site));
  };
  bool ok = true;
  uint32_t kt = 0;
  const int wg = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) / 128, 0);

  if (wg > kGroups) {
    // ------------------------------------------------------------ unpacking
    const bool values = warp >= kUnpackWarp + 4;
    const Fp4Cache& c = values ? f.v : f.k;
    uint64_t* full = values ? ctl.vfull : ctl.kfull;
    uint64_t* empty = values ? ctl.vempty : ctl.kempty;
    uint8_t* base = values ? sV : sK;
    // lane (g, t): quarter t of keys 8 i + g of the warp's 32
    const int w4 = (warp - kUnpackWarp) & 3, g = lane >> 2, t4 = lane & 3;
    const bool small = a.page_shift < 5;   // pages of 16 keys
    struct Raw {
      uint32_t w[4][4], unit[4];
    };
    // the pages of the warp's 32 keys, two where pages have 16: lane l has those of tile
    // 32 * batch + l, of this batch and the next
    int pages[2][2] = {{0, 0}, {0, 0}};
    auto look_up = [&](const PagedPiece& q, int n, int batch, int* to) {
      const int u = 32 * batch + lane, key = (q.t0 + u) * kTile + 32 * w4;
      const int32_t* row = a.table + q.b * a.table_stride;
      to[0] = to[1] = a.num_pages;
      if (u < n && key < q.len) to[0] = checked_page(row[key >> a.page_shift], a.num_pages, a.status);
      if (small && u < n && key + 16 < q.len)
        to[1] = checked_page(row[(key + 16) >> a.page_shift], a.num_pages, a.status);
    };
    auto page_of = [&](int u, int half) {
      const int first = __shfl_sync(0xffffffffu, pages[0][half], u & 31);
      const int second = __shfl_sync(0xffffffffu, pages[1][half], u & 31);
      return u & 32 ? second : first;
    };
    const int size = 1 << a.page_shift;
    const uint8_t *head_codes = nullptr, *head_scales = nullptr;   // of the piece's head
    auto load = [&](const PagedPiece& q, int t, Raw& x) {
      const int k0 = (q.t0 + t) * kTile + 32 * w4, row = k0 & (size - 1);
      const int left = q.len - k0 - g;   // (rows past the end: zeros)
      const int pg0 = page_of(t, 0);
      bool in0 = pg0 < a.num_pages, in1 = in0;
      const uint8_t *c0 = page_at(head_codes, in0 ? pg0 : 0, c.code_page) + row * (kD / 2) + g * (kD / 2) + 16 * t4;
      const uint8_t *s0 = page_at(head_scales, in0 ? pg0 : 0, c.scale_page) + (row + g) * (kD / kFp4Block) + 2 * t4;
      const uint8_t *c1 = c0 + 16 * (kD / 2), *s1 = s0 + 16 * (kD / kFp4Block);
      if (small) {
        const int pg1 = page_of(t, 1);
        in1 = pg1 < a.num_pages;
        c1 = page_at(head_codes, in1 ? pg1 : 0, c.code_page) + g * (kD / 2) + 16 * t4;
        s1 = page_at(head_scales, in1 ? pg1 : 0, c.scale_page) + g * (kD / kFp4Block) + 2 * t4;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool in = (i < 2 ? in0 : in1) && 8 * i < left;
        const uint4 y = in ? __ldcs(reinterpret_cast<const uint4*>((i < 2 ? c0 : c1) + (i & 1) * 8 * (kD / 2)))
                           : make_uint4(0u, 0u, 0u, 0u);
        x.w[i][0] = y.x;
        x.w[i][1] = y.y;
        x.w[i][2] = y.z;
        x.w[i][3] = y.w;
        x.unit[i] = in ? *reinterpret_cast<const uint16_t*>((i < 2 ? s0 : s1) + (i & 1) * 8 * (kD / kFp4Block))
                       : 0u;
      }
    };
    // the warp's keys of a later tile into L2 (of small pages the first half)
    auto fetch = [&](const PagedPiece& q, int t) {
      const int pg = page_of(t, 0);
      if (lane > 0 || pg >= a.num_pages) return;
      const int row = ((q.t0 + t) * kTile + 32 * w4) & (size - 1), rows = small ? 16 : 32;
      prefetch_l2(page_at(head_codes, pg, c.code_page) + row * (kD / 2), rows * (kD / 2));
      prefetch_l2(page_at(head_scales, pg, c.scale_page) + row * (kD / kFp4Block), rows * (kD / kFp4Block));
    };
    for (; ok && p.valid; next_piece()) {
      const int n = p.t1 - p.t0;
      if (n == 0) continue;
      head_codes = c.codes + p.h / a.blocks * c.code_head;
      head_scales = c.scales + p.h / a.blocks * c.scale_head;
      look_up(p, n, 0, pages[0]);
      look_up(p, n, 1, pages[1]);
      Raw now;
      load(p, 0, now);
      for (int t = 1; t < kAhead && t < n; ++t) fetch(p, t);
      for (int t = 0; t < n; ++t, ++kt) {
        Raw next;
        if (t > 0 && (t & 31) == 0) {   // the batch before is done with
          if (t & 32) look_up(p, n, (t >> 5) + 1, pages[0]);
          else look_up(p, n, (t >> 5) + 1, pages[1]);
        }
        load(p, t + 1, next);   // (no page, no load, past the last tile)
        if (t + kAhead < n) fetch(p, t + kAhead);
        if (!(ok = freed(empty, kt, kSiteFp4Ring))) break;
        uint8_t* to = base + (kt & 1) * kKeysBytes + (t4 >> 1) * kBox;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = 32 * w4 + 8 * i + g;
          const uint32_t s = e4m3_to_half(now.unit[i]);
          const uint32_t u[2] = {__byte_perm(s, 0, 0x1010), __byte_perm(s, 0, 0x3232)};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // (in an order in which eight lanes write different banks)
            const int jj = j ^ (t4 & 2);
            const uint32_t word = t4 & 2 ? now.w[i][j ^ 2] : now.w[i][j];
            uint32_t y[4];
            e2m1_to_half(word, y);
            const uint32_t unit2 = jj & 2 ? u[1] : u[0];
            *reinterpret_cast<uint4*>(to + key * 128 + ((((t4 & 1) * 4 + jj) ^ (key & 7)) << 4)) =
                make_uint4(mul_half2(y[0], unit2), mul_half2(y[1], unit2), mul_half2(y[2], unit2),
                           mul_half2(y[3], unit2));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        // (an armed test stall: the first values never arrive)
        if (lane == 0 && !(a.stall != 0 && values && kt == 0)) mbar_arrive(&full[kt & 1]);
        now = next;
      }
    }
  } else if (wg == kGroups) {
    // --------------------------------------------------------------- MMA issue
    regs_decrease<kRegsIssue>();
    // One elected lane issues, in code that the whole warp runs, on values that the
    // compiler knows to be the warp's (from a shuffle or a vote): the descriptors then
    // stay in uniform registers.
    auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    const bool one = warp == kIssueWarp && elect_one_lane();
    uint32_t piece = 0;
    while (warp == kIssueWarp && __all_sync(0xffffffffu, ok && p.valid)) {
      const int n = uniform(p.t1 - p.t0);
      const int cols = uniform((segment_rows(a, p.h) + 15) & ~15);
      const uint32_t id_s = idesc_half(kTile, cols, false, false), id_o = idesc_half(kD, cols, true, true);
      auto scores = [&](uint32_t k) {
        if (!filled(ctl.kfull, k, kSiteFp4K) || !freed(ctl.sempty, k, kSiteFp4Free)) return false;
        tc_fence_after();
        const int st = uniform(static_cast<int>(k & 1));
        const uint64_t dk = smem_desc(smem_u32(sK + st * kKeysBytes), 16, 1024);
        const uint64_t dq = smem_desc(smem_u32(sQ), 16, 1024);
        if (one) {
#pragma unroll
          for (int kk = 0; kk < kD / 16; ++kk)
            mma_ss(tmem + kSCol + st * kRowsMax,
                   dk + static_cast<uint64_t>(((kk >> 2) * kBox + (kk & 3) * 32) >> 4),
                   dq + static_cast<uint64_t>(((kk >> 2) * kQBox + (kk & 3) * 32) >> 4), id_s,
                   kk > 0 ? 1u : 0u);
          mma_commit(&ctl.sfull[st]);
          mma_commit(&ctl.kempty[st]);
        }
        return true;
      };
      if (n > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&ctl.qfull, piece & 1, wc, kSiteFp4Q)) && scores(kt);
        ++piece;
      }
      for (int t = 0; ok && t < n; ++t, ++kt) {
        if (t + 1 < n && !(ok = scores(kt + 1))) break;
        if (!(ok = filled(ctl.vfull, kt, kSiteFp4V) && filled(ctl.pfull, kt, kSiteFp4P))) break;
        tc_fence_after();
        const int st = uniform(static_cast<int>(kt & 1));
        const uint64_t dv = smem_desc(smem_u32(sV + st * kKeysBytes), kBox, 1024);
        const uint64_t dp = smem_desc(smem_u32(sP + st * kPBytes), kBox, 1024);
        if (one) {
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            mma_ss(tmem + kOCol, dv + static_cast<uint64_t>((kk * 2048) >> 4),
                   dp + static_cast<uint64_t>((kk * 2048) >> 4), id_o, t > 0 || kk > 0 ? 1u : 0u);
          mma_commit(&ctl.vempty[st]);
          mma_commit(&ctl.pempty[st]);
        }
      }
      next_piece();
    }
    if (one) {
      mma_commit(&ctl.final_bar);   // every MMA of this CTA done before TMEM is freed
      mbar_wait_drain(&ctl.final_bar, 0, a.timeout_ns);
    }
    __syncwarp();
  } else {
    // --------------------------------------------- Q, softmax, write-out
    regs_increase<kRegsSoft>();
    // (A wait that runs out leaves `ok` false in some warps; they go on to the next
    // any_of_group, where all four leave together.)
    const int me = threadIdx.x & 127, r0 = wg * kGroupRows;   // a tile's key; the group's first row
    const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + r0;
    auto group_sync = [&] { named_barrier_sync(1 + wg, 128); };
    MergeNote note{-1, 0, 0, 0};
    for (; p.valid; next_piece()) {
      const int n = p.t1 - p.t0;
      const int row0 = segment_row(a, p.h), nrows = segment_rows(a, p.h);
      // ---- Q, 16 lanes a row, as fp16 times 2^e
      for (int r = r0 + (me >> 4); r < r0 + kGroupRows; r += 8) {
        const int c8 = me & 15;
        const bool live = r < nrows;
        const int h = (row0 + r) / a.n_q, qt = row0 + r - h * a.n_q;
        const int64_t at = p.b * a.stride_b + h * a.stride_h + static_cast<int64_t>(qt) * a.stride_n;
        const uint4 x = live ? *reinterpret_cast<const uint4*>(a.q + at + 8 * c8)
                             : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[k] << 16)),
                                 fabsf(__uint_as_float(w[k] & 0xffff0000u))));
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int e = row_exponent(top);
        const float up = ldexpf(1.f, e);
        uint32_t y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          y[k] = pack_half2(__uint_as_float(w[k] << 16) * up, __uint_as_float(w[k] & 0xffff0000u) * up);
        *reinterpret_cast<uint4*>(sQ + (c8 >> 3) * kQBox + r * 128 + (((c8 & 7) ^ (r & 7)) << 4)) =
            make_uint4(y[0], y[1], y[2], y[3]);
        if (c8 == 0) {
          ctl.c2[r] = score_factor(a.scale_log2 * f.k_descale, e);
          ctl.negm[r] = live ? -kNoScore : -INFINITY;
          ctl.lim[r] = live ? (a.causal ? min(p.len, p.len - a.n_q + qt + 1) : p.len) : 0;
          ctl.to[r] = at;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && n > 0) mbar_arrive(&ctl.qfull);
      const int open = a.causal ? p.len - a.n_q + 1 : p.len;   // every row attends keys below it
      uint64_t l[kGroupRows / 2];   // this key's share of the rows' sums, packed pairs
#pragma unroll
      for (int i = 0; i < kGroupRows / 2; ++i) l[i] = f2_pack(0.f, 0.f);
      bool bad = any_of_group(wg, !ok);   // (and the rows' values are there)
      for (int t = 0; !bad && t < n; ++t, ++kt) {
        ok = ok && filled(ctl.sfull, kt, kSiteFp4S);
        tc_fence_after();
        const int k0 = (p.t0 + t) * kTile, key = k0 + me;
        const uint32_t sc = tl + kSCol + (kt & 1) * kRowsMax;
        const bool masked = k0 + kTile > open;
        uint32_t s[kGroupRows];
        tmem_read(sc, s);
        // scores in log2 units less the maximum
        auto shift = [&] {
#pragma unroll
          for (int i = 0; i < kGroupRows; i += 4) {
            const float4 k = *reinterpret_cast<const float4*>(&ctl.c2[r0 + i]);
            const float4 m = *reinterpret_cast<const float4*>(&ctl.negm[r0 + i]);
            float x[4];
            f2_unpack(f2_fma(f2_pack(__uint_as_float(s[i]), __uint_as_float(s[i + 1])),
                             f2_pack(k.x, k.y), f2_pack(m.x, m.y)), x[0], x[1]);
            f2_unpack(f2_fma(f2_pack(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])),
                             f2_pack(k.z, k.w), f2_pack(m.z, m.w)), x[2], x[3]);
            if (masked) {
              const int4 lim = *reinterpret_cast<const int4*>(&ctl.lim[r0 + i]);
              x[0] = key < lim.x ? x[0] : -INFINITY;
              x[1] = key < lim.y ? x[1] : -INFINITY;
              x[2] = key < lim.z ? x[2] : -INFINITY;
              x[3] = key < lim.w ? x[3] : -INFINITY;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i + j] = __float_as_uint(x[j]);
          }
        };
        shift();
        float most = -INFINITY;
#pragma unroll
        for (int i = 0; i < kGroupRows; i += 2)
          most = max3f(most, __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
        if (any_of_group(wg, most > kPLazy || !ok)) {
          if ((bad = any_of_group(wg, !ok))) break;
          // new maxima: of the tile's scores, row by row
          tmem_read(sc, s);
          float mine = -INFINITY;
#pragma unroll
          for (int i = 0; i < kGroupRows; ++i) {
            const float top = warp_max(
                key < ctl.lim[r0 + i] ? fmaf(__uint_as_float(s[i]), ctl.c2[r0 + i], -kPTop) : -INFINITY);
            if (lane == i) mine = top;
          }
          if (lane < kGroupRows) ctl.part[warp & 3][r0 + lane] = mine;
          group_sync();
          if (me < kGroupRows) {
            const int r = r0 + me;
            const float m = -ctl.negm[r];
            float alpha = 1.f;
            if (r < nrows) {
              float top = m;
#pragma unroll
              for (int k = 0; k < kSoftWarps; ++k) top = fmaxf(top, ctl.part[k][r]);
              alpha = ex2_approx(m - top);
              ctl.negm[r] = -top;
            }
            ctl.alpha[r] = alpha;
          }
          group_sync();
#pragma unroll
          for (int i = 0; i < kGroupRows; i += 2) {
            const float2 alpha = *reinterpret_cast<const float2*>(&ctl.alpha[r0 + i]);
            l[i / 2] = f2_mul(l[i / 2], f2_pack(alpha.x, alpha.y));
          }
          if (t > 0) {   // O stands still once the tile before this one has been added
            ok = ok && filled(ctl.pempty, kt - 1, kSiteFp4Done);
            tc_fence_after();
            uint32_t o[16];
#pragma unroll
            for (int c = 0; c < kGroupRows; c += 16) {
              tmem_ld16(tl + kOCol + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i)
                o[i] = __float_as_uint(__uint_as_float(o[i]) * ctl.alpha[r0 + c + i]);
              tmem_st16(tl + kOCol + c, o);
            }
            tmem_wait_st();
          }
          shift();   // (s still holds the scores)
        }
        ok = ok && freed(ctl.pempty, kt, kSiteFp4Done);
        uint8_t* to = sP + (kt & 1) * kPBytes + me * 128;
#pragma unroll
        for (int i = 0; i < kGroupRows; i += 8) {
          uint32_t y[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float p0 = ex2_approx(__uint_as_float(s[i + 2 * j]));
            const float p1 = ex2_approx(__uint_as_float(s[i + 2 * j + 1]));
            l[i / 2 + j] = f2_add(l[i / 2 + j], f2_pack(p0, p1));
            y[j] = pack_half2(p0, p1);
          }
          *reinterpret_cast<uint4*>(to + ((((r0 + i) >> 3) ^ (me & 7)) << 4)) =
              make_uint4(y[0], y[1], y[2], y[3]);
        }
        tc_fence_before();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&ctl.sempty[kt & 1]);
          mbar_arrive(&ctl.pfull[kt & 1]);
        }
      }
      if (n > 0 && !bad) ok = ok && filled(ctl.pempty, kt - 1, kSiteFp4Done);
      if (bad || any_of_group(wg, !ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // ---- the rows' sums: lane i of a warp gets row i's, by halves
      {
        float v[kGroupRows];
#pragma unroll
        for (int i = 0; i < kGroupRows / 2; ++i) f2_unpack(l[i], v[2 * i], v[2 * i + 1]);
#pragma unroll
        for (int o = kGroupRows / 2; o > 0; o >>= 1) {
          const bool high = (lane & o) != 0;
#pragma unroll
          for (int i = 0; i < o; ++i) {
            const float give = high ? v[i] : v[i + o], keep = high ? v[i + o] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
          }
        }
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], 16);   // (two lanes a row)
        if (lane < kGroupRows) ctl.part[warp & 3][r0 + lane] = v[0];
      }
      group_sync();
      const bool whole = p.whole();
      if (wg == 0) {
        if (p.t0 == 0 && !whole) note = paged_note<kFp4TileOverhead>(share, p);
        if (a.by_segment && p.t0 == 0 && me == 0)
          a.notes[p.b * a.heads + p.h] = whole ? MergeNote{p.b, p.h, 0, -1} : note;
      }
      const int64_t part = 2 * static_cast<int64_t>(blockIdx.x) + (p.s < share.lo ? 0 : 1);
      if (me < kGroupRows && r0 + me < nrows) {
        const int r = r0 + me;
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < kSoftWarps; ++k) sum += ctl.part[k][r];
        // (a row of NaN scores has a maximum of none, and a sum that is NaN)
        const float m = -ctl.negm[r];
        const float L = sum == 0.f ? -INFINITY : fmaf(m == kNoScore ? 0.f : m, 0.69314718f, logf(sum));
        ctl.alpha[r] = sum == 0.f ? 0.f : f.v_descale / sum;
        if (whole) a.lse[static_cast<int64_t>(p.b) * a.all_rows + row0 + r] = L;
        else a.part_l[part * a.rows + r] = L;
      }
      group_sync();
      {
        uint32_t o[kGroupRows];
        if (n > 0) tmem_read(tl + kOCol, o);
#pragma unroll
        for (int i = 0; i < kGroupRows; ++i) {   // column `me` of row r0 + i
          if (r0 + i >= nrows) break;
          const float x = n > 0 ? __uint_as_float(o[i]) * ctl.alpha[r0 + i] : 0.f;
          if (whole) a.o[ctl.to[r0 + i] + me] = __float2bfloat16(x);
          else a.part_o[(part * a.rows + r0 + i) * kD + me] = x;
        }
      }
      tc_fence_before();
      group_sync();   // (the next piece writes what is read above)
    }
    if (!a.by_segment && threadIdx.x == 0) a.notes[blockIdx.x] = note;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssueWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

cudaError_t launch_fp4_tile(const PagedArgs& a, const Fp4Args& f, int ctas, cudaStream_t s) {
  static std::atomic<uint64_t> set_up{0};
  int dev = 0;
  bool todo = false;
  cudaError_t e = needs_setup(set_up, &dev, &todo);
  if (e != cudaSuccess) return e;
  if (todo) {
    e = cudaFuncSetAttribute(fp4_tile_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileSmem);
    if (e != cudaSuccess) return e;
    // the register re-split inside the kernel assumes the launch allocation
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, fp4_tile_kernel)) != cudaSuccess) return e;
    if (static_cast<uint32_t>(fa.numRegs) < kRegsLaunch) return cudaErrorInvalidConfiguration;
    mark_done(set_up, dev);
  }
  return launch_pdl(fp4_tile_kernel, dim3(ctas), dim3(kTileThreads), kTileSmem, s, a, f);
}

}  // namespace attn
