// Decode step against a paged key/value cache held in 4 bits.
//
// What it computes: the decode step of attn_paged.cu (query row t of sequence b
// at position len_b - n_q + t attends the cached keys j < len_b, j <= its
// position when causal; O = softmax(c q K^T) V, L = logsumexp) on keys and values
// K = descale_k s c, V = descale_v s c (attn_fp4.cuh).
//
// Bound: HBM, 9 d / 8 bytes a key (144 at d = 128, where bf16 has 512); but 2 d
// values a key have to be unpacked meanwhile, 42 a clock and SM at the copy
// rate, so the path from the packed bytes to the matrix unit decides:
//   * the products are 16 x 8 x 16 warp MMAs in fp16 with the keys (and the
//     columns of V) as the 16, and the query rows as the 8: S^T = K Q^T and
//     O^T = V^T P^T.  Up to 8 rows no lane works on padding, and what is unpacked
//     is the MMA's A operand as it stands: lane (g, t) = (lane / 4, lane % 4) takes
//     the quarter row t of keys g and g + 8 (of 16 bytes at d = 128, whose scales
//     are its own), since the sum over d may go in any order;
//   * two values a conversion (cvt.f16x2.e2m1x2; measured 50 a clock and SM,
//     shifts and masks 30), one multiplication by the scale, both exact;
//   * V^T wants two keys in a register: the codes of two keys are interleaved
//     before they are converted, two operations per four pairs;
//   * P^T comes from S^T by movmatrix, without shared memory.
// Q enters as fp16, scaled by a power of two per row so that its largest element
// is in [2^14, 2^15): exact for elements down to 2^-31 of that one.  P, up to 2^7 where a
// maximum is taken, is rounded to fp16 (a relative 2^-11, of p below 2^-21 of the largest
// an absolute 2^-32 of it), the row sums are of the unrounded fp32 values, S, m, l, O are
// fp32.
//
// The keys of all sequences are divided evenly over the CTAs (attn_paged.cuh).
// A slot (one warp up to 32 rows; above, two warps of 32 rows each) streams its own 32-key
// tiles by 16-byte asynchronous copies through its own ring; what is no page
// is filled with zeros.  Value rows past the end of a sequence may hold
// anything: their scores are replaced, their values' scales are taken as zero.
//
// Measured (replayed from a graph; floors at 6.8 TB/s): 64 sequences of 8192 keys, 8 heads, 4
// rows, d = 128, 604 MB in 115 us = 5.2 TB/s; 16 rows 155 us; 32 rows 230 us.  16
// sequences of 4096-8192 keys 31 us, floor 17; one of 517 keys 6.5 us.  At 4 rows 323
// warp instructions for 16 keys take 62 % of the issue slots; at 32 rows 478, and the
// warp MMAs half of the tensor cores' time, with eight warps on an SM.  d = 64: 64
// sequences of 16384 keys, 4 heads, 32 rows 135 us, 33 to 64 rows 280 (every value is
// unpacked once per 32 rows).  512 queries on 16384 keys, 8 heads, d = 128: 347 us, the
// cache unpacked once per 64 rows (attn_fp4_tile.cu).  Spills of the balanced split at d =
// 128: 144 bytes up to 16 rows (168 registers), 72 up to 32 (255), none up to 8.
#include <type_traits>

#include "attn_fp4.cuh"

namespace attn {
using namespace sm103;

namespace {

constexpr float kLn2 = 0.69314718f;
constexpr float kNone = -3e38f;   // a row's maximum before its first key

// NT: blocks of 8 query rows per warp; MT: warps that share a tile.
template <int D, int NT, int MT>
struct Fp4Cfg {
  static constexpr int kWarps = 4 * MT;
  static constexpr int kSlots = kWarps / MT;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kRows = 8 * NT * MT;                  // of a CTA
  static constexpr bool kSharedQ = NT == 4;                  // Q's fragments in shared memory
  static constexpr int kCodeBytes = kFp4Keys * D / 2;        // of a tile's keys (or values)
  static constexpr int kScaleBytes = kFp4Keys * D / kFp4Block;
  static constexpr int kTileBytes = 2 * (kCodeBytes + kScaleBytes);
  static constexpr int kOverhead = fp4_overhead(kRows);
  static constexpr int kCtasPerSm = fp4_ctas_per_sm(8 * NT * MT);
  static constexpr int kRedStride = D + 4;                   // floats; the pad spreads the rows
  static constexpr int kRedBytes = kRows * kRedStride * 4;   // of a slot
  static constexpr int kStages = NT == 1 && D == 128 ? 2 : MT == 2 || D == 64 ? 4 : 3;
  static constexpr int kRingBytes = kSlots * kStages * kTileBytes;
  static constexpr int kQRows = MT == 1 ? 8 * NT * kWarps : kRows;   // with a segment per warp
  static constexpr int kQBytes = kSharedQ ? kRows * D * 2 : 0;
  static constexpr int kSmem = kRingBytes + 2 * kRedBytes + kQBytes;
  static_assert(kCtasPerSm * (kSmem + 1024 + 2560) <= 228 * 1024, "shared memory of an SM");
  // (a warp to itself needs no `red`, and has Q there)
  static_assert(!kSharedQ || kQRows * D * 2 <= 2 * kRedBytes + kQBytes, "Q of all warps");
};

template <int D, int NT, int MT>
struct Fp4Shared {
  float m[Fp4Cfg<D, NT, MT>::kSlots][Fp4Cfg<D, NT, MT>::kRows];   // maximum taken, log2 units
  float l[Fp4Cfg<D, NT, MT>::kSlots][Fp4Cfg<D, NT, MT>::kRows];
  float c2[Fp4Cfg<D, NT, MT>::kQRows];   // (kSharedQ)
  float L[Fp4Cfg<D, NT, MT>::kRows];     // of the CTA's rows, for the cluster
};

// 16 bytes to shared memory, asynchronously; zeros where nothing is `there`.
__device__ __forceinline__ void copy16_sized(uint32_t dst, const uint8_t* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(there ? 16 : 0)
               : "memory");
}

__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void copies_wait_but() {   // all groups but the last N have landed
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void cluster_ld2(uint32_t addr, float* x) {
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
               : "=f"(x[0]), "=f"(x[1])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {   // an 8 x 8 matrix of 16 bits
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// N words of shared memory.  (Plain loads, so that the compiler may move them
// between the products, but not across the waits for the copies.)
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
  if constexpr (N == 4) {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    w[0] = x.x;
    w[1] = x.y;
    w[2] = x.z;
    w[3] = x.w;
  } else if constexpr (N == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    w[0] = x.x;
    w[1] = x.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// How the segments are given out.
//   kSplit    the balanced split; what it cuts is merged by a second kernel
//   kCluster  a segment per cluster of a.cluster CTAs (of one, perhaps), merged in
//             shared memory
//   kSolo     a segment per warp, which has nobody to merge with
enum Fp4Mode { kSplit, kCluster, kSolo };

template <int D, int NT, int MT, Fp4Mode MODE>
__global__ void __launch_bounds__(Fp4Cfg<D, NT, MT>::kThreads, Fp4Cfg<D, NT, MT>::kCtasPerSm)
    fp4_decode_kernel(const PagedArgs a, const Fp4Args f) {
  using C = Fp4Cfg<D, NT, MT>;
  constexpr int ST = C::kStages, KT = kFp4Keys, kSlots = C::kSlots;
  constexpr int kSteps = D / 16;            // MMA steps along d, and 16-column groups of V
  constexpr int kKeyWords = D / 32;         // 32-bit words of a lane's quarter key row
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Fp4Shared<D, NT, MT> sh;
  float* red = reinterpret_cast<float*>(smem + C::kRingBytes);   // [2][kRows][kRedStride]
  uint2* sq = reinterpret_cast<uint2*>(smem + C::kRingBytes + (MODE == kSolo ? 0 : 2 * C::kRedBytes));

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slot = warp / MT, mt = warp % MT;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + slot * ST * C::kTileBytes;
  grid_dep_wait();
  grid_dep_launch();
  PagedShare share{};
  if constexpr (MODE == kSplit)
    share = paged_share<KT, C::kOverhead, kFp4MinUnits>(a, blockIdx.x, gridDim.x);
  MergeNote note{-1, 0, 0, 0};
  const bool small_pages = a.page_shift < 5;   // 16 keys: a tile lies in two

  // ---- the copies: tile u of this slot is tile t0 + slot + kSlots u of the
  // piece (of a segment of its own: tile u); lane l holds the pages of tile 32 *
  // (batch) + l
  constexpr int kStep = MODE == kSolo ? 1 : kSlots;
  const int first_tile = MODE == kSolo ? 0 : slot;
  int page_of[2] = {0, 0};
  auto slot_tiles = [&](const PagedPiece& p) {
    const int n = p.t1 - p.t0 - first_tile;
    return n > 0 ? (n + kStep - 1) / kStep : 0;
  };
  auto load_pages = [&](const PagedPiece& p, int u0, int nu) {
    const int u = u0 + lane;
    if (u < nu) {
      const int key = (p.t0 + first_tile + kStep * u) * KT;
      const int32_t* row = a.table + p.b * a.table_stride;
      page_of[0] = checked_page(row[key >> a.page_shift], a.num_pages, a.status);
      page_of[1] = !small_pages || key + 16 >= p.len
                       ? page_of[0]
                       : checked_page(row[(key >> a.page_shift) + 1], a.num_pages, a.status);
    }
  };
  // A lane's sources: 16-byte pieces of the tile's key and value codes, and (the
  // slot's first warp) one of its scales, of keys or values.
  constexpr int kCopies = C::kCodeBytes / (MT * 512);    // of codes, per tensor
  constexpr int kScalePieces = C::kScaleBytes / 16;      // per tensor
  const int me = mt * 32 + lane;
  const bool of_values = lane >= kScalePieces;
  const int scale_piece = lane & (kScalePieces - 1);
  const bool scales = mt == 0 && lane < 2 * kScalePieces;
  const uint32_t to_codes = smem_u32(ring) + me * 16;
  const uint32_t to_scales = smem_u32(ring) + 2 * C::kCodeBytes + lane * 16;
  const int64_t scale_page = of_values ? f.v.scale_page : f.k.scale_page;
  const uint8_t *from_k = nullptr, *from_v = nullptr, *from_s = nullptr;
  // and where it reads: see the products
  const int kg = (g >> 1) + 4 * (g & 1);
  const uint8_t* at_k = ring + kg * (D / 2) + t * (D / 8);
  const uint8_t* at_v = ring + C::kCodeBytes + t * (D / 2) + g * (D / 16);
  const uint8_t* at_ks = ring + 2 * C::kCodeBytes + kg * (D / kFp4Block) + t * (D / 64);
  const uint8_t* at_vs = ring + 2 * C::kCodeBytes + C::kScaleBytes +
                         t * (D / kFp4Block) + (D == 128 ? g : g >> 1);
  auto sources = [&](const PagedPiece& p) {
    const int64_t head = p.h / a.blocks;
    from_k = f.k.codes + head * f.k.code_head + me * 16;
    from_v = f.v.codes + head * f.v.code_head + me * 16;
    from_s = (of_values ? f.v.scales + head * f.v.scale_head : f.k.scales + head * f.k.scale_head) +
             scale_piece * 16;
  };
  auto issue = [&](const PagedPiece& p, int u, uint32_t stage) {   // stage: its offset
    int pg0 = __shfl_sync(0xffffffffu, page_of[0], u & 31);
    const bool in0 = pg0 < a.num_pages;
    pg0 = in0 ? pg0 : 0;
    const uint8_t *k0, *v0, *s0, *k1, *v1;
    bool in1 = in0, s_in = in0;
    if (!small_pages) {
      const uint32_t row = (p.t0 + first_tile + kStep * u) * KT & ((1 << a.page_shift) - 1);
      k0 = k1 = page_at(from_k, pg0, f.k.code_page) + row * (D / 2);
      v0 = v1 = page_at(from_v, pg0, f.v.code_page) + row * (D / 2);
      s0 = page_at(from_s, pg0, scale_page) + row * (D / kFp4Block);
    } else {   // the two halves of a tile lie apart
      int pg1 = __shfl_sync(0xffffffffu, page_of[1], u & 31);
      in1 = pg1 < a.num_pages;
      pg1 = in1 ? pg1 : 0;
      k0 = page_at(from_k, pg0, f.k.code_page);
      v0 = page_at(from_v, pg0, f.v.code_page);
      k1 = page_at(from_k, pg1, f.k.code_page) - C::kCodeBytes / 2;
      v1 = page_at(from_v, pg1, f.v.code_page) - C::kCodeBytes / 2;
      const bool upper = scale_piece >= kScalePieces / 2;
      s_in = upper ? in1 : in0;
      s0 = page_at(from_s, upper ? pg1 : pg0, scale_page) - (upper ? C::kScaleBytes / 2 : 0);
    }
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      constexpr int kHalf = C::kCodeBytes / 2;
      const bool second = MT * 512 <= kHalf ? i * MT * 512 >= kHalf : mt * 512 >= kHalf;
      const bool in = second ? in1 : in0;
      copy16_sized(to_codes + stage + i * MT * 512, (second ? k1 : k0) + i * MT * 512, in);
      copy16_sized(to_codes + stage + C::kCodeBytes + i * MT * 512,
                   (second ? v1 : v0) + i * MT * 512, in);
    }
    if (scales) copy16_sized(to_scales + stage, s0, s_in);
  };
  // every warp of the slot: its copies of the tile have landed, and it is done
  // with the tile before
  auto slot_sync = [&] {
    if constexpr (MT == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(slot + 1), "n"(32 * MT) : "memory");
  };

  // What a piece begins with, on its way early: its rows of Q (raw), its pages,
  // its first tiles.
  constexpr bool kOwnQ = C::kSharedQ && MODE == kSolo;   // NT blocks, one after another
  constexpr int kQBlocks = C::kSharedQ ? 1 : NT;   // of 8 rows that this warp loads
  uint32_t qw[kQBlocks][D / 8];
  auto fetch_q = [&](const PagedPiece& p, int block) {   // (kSharedQ: this one)
    const int row0 = segment_row(a, p.h), nrows = segment_rows(a, p.h);
#pragma unroll
    for (int n = 0; n < kQBlocks; ++n) {
      const int r = (C::kSharedQ ? block : mt * NT + n) * 8 + g;
      const bool live = r < nrows;
      const int h = (row0 + r) / a.n_q, qt = row0 + r - h * a.n_q;
      const uint4* qr = reinterpret_cast<const uint4*>(
          a.q + p.b * a.stride_b + h * a.stride_h + static_cast<int64_t>(qt) * a.stride_n +
          t * (D / 4));
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 x = live ? qr[i] : make_uint4(0u, 0u, 0u, 0u);
        qw[n][4 * i] = x.x;
        qw[n][4 * i + 1] = x.y;
        qw[n][4 * i + 2] = x.z;
        qw[n][4 * i + 3] = x.w;
      }
    }
  };
  auto fetch = [&](const PagedPiece& p) {
    const int nu = slot_tiles(p);
    if constexpr (!C::kSharedQ) fetch_q(p, 0);
    if (nu > 0) load_pages(p, 0, nu);
    sources(p);
    for (int u = 0; u < ST - 1; ++u) {
      if (u < nu) issue(p, u, u * C::kTileBytes);
      copies_commit();
    }
  };

  const int rank = MODE == kCluster ? static_cast<int>(cluster_rank()) : 0;
  PagedPiece p;
  if constexpr (MODE == kSplit) {
    p = paged_piece<KT, C::kOverhead>(a, share, share.b, 0, share.s);
  } else {
    const int segment = MODE == kSolo ? blockIdx.x * kSlots + slot : blockIdx.x / a.cluster;
    const int b = segment / a.heads;
    p.valid = false;
    if (b < a.B) p = paged_part<KT>(a, b, segment - b * a.heads, rank, MODE == kSolo ? 1 : a.cluster);
  }
  if (p.valid) fetch(p);
  while (p.valid) {   // (the same pieces in every warp)
    const int nu = slot_tiles(p);
    // Q^T fragments: row r = 8 n + g, columns of quarter t, as fp16 times 2^e
    const int row0 = segment_row(a, p.h), nrows = segment_rows(a, p.h);
    float c2[NT][2];                // what turns a score into log2 units, rows 2t, 2t + 1
    uint32_t qb[kQBlocks][kSteps][2];
    if constexpr (C::kSharedQ) {   // (late: the registers are O's until then)
      // the CTA's blocks, one a warp; of a segment of its own: all of them
      uint2* to = sq + (kOwnQ ? warp * NT * kSteps * 32 : 0);
#pragma unroll 1
      for (int n = kOwnQ ? 0 : warp; n < (kOwnQ ? NT : warp + 1); ++n) {
        fetch_q(p, n);
        int e;
        half_rows<D / 8>(qw[0], &e);
        const float c = score_factor(a.scale_log2 * f.k_descale, e);
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
          to[(n * kSteps + i) * 32 + lane] = make_uint2(qw[0][2 * i], qw[0][2 * i + 1]);
        if (t == 0) sh.c2[(kOwnQ ? warp * NT : 0) * 8 + n * 8 + g] = c;
      }
      if constexpr (kOwnQ) __syncwarp();
      else __syncthreads();
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          c2[n][i] = sh.c2[((kOwnQ ? warp : mt) * NT + n) * 8 + 2 * t + i];
    } else {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        int e;
        half_rows<D / 8>(qw[n], &e);
        const float c = score_factor(a.scale_log2 * f.k_descale, e);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          qb[n][i][0] = qw[n][2 * i];
          qb[n][i][1] = qw[n][2 * i + 1];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) c2[n][i] = __shfl_sync(0xffffffffu, c, 4 * (2 * t + i));
      }
    }
    auto limit = [&](int n, int i) {   // keys below it are allowed, row 2t + i of block n
      const int r = (mt * NT + n) * 8 + 2 * t + i, qt = (row0 + r) % a.n_q;
      return r >= nrows ? 0 : (a.causal ? min(p.len, p.len - a.n_q + qt + 1) : p.len);
    };
    const int open = a.causal ? p.len - a.n_q + 1 : p.len;   // every row is allowed keys below it
    float m[NT][2], l[NT][2];
    float o[kSteps][NT][4];         // columns (D / 8) g + 2 i, + 1; rows 2t, 2t + 1
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[n][i] = kNone;
        l[n][i] = 0.f;
      }
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;

    uint32_t stage = 0, ahead = (ST - 1) * C::kTileBytes;   // of tile u; of tile u + ST - 1
    for (int u = 0; u < nu; ++u) {
      copies_wait_but<ST - 2>();
      slot_sync();
      if (u + ST - 1 < nu) {   // into the stage that the tile before this one has left
        if (((u + ST - 1) & 31) == 0) load_pages(p, u + ST - 1, nu);
        issue(p, u + ST - 1, ahead);
      }
      copies_commit();
      const uint8_t *kc = at_k + stage, *vc = at_v + stage, *ks = at_ks + stage, *vs = at_vs + stage;
      const int k0 = (p.t0 + first_tile + kStep * u) * KT;
      if (k0 + KT > p.len) {   // value rows past the end: their scales are zero
        const int from = (p.len - k0) * (D / kFp4Block) + lane;
        uint8_t* to = ring + stage + 2 * C::kCodeBytes + C::kScaleBytes;
        for (int i = from; i < C::kScaleBytes; i += 32) to[i] = 0;
        __syncwarp();
      }
      stage = stage == (ST - 1) * C::kTileBytes ? 0 : stage + C::kTileBytes;
      ahead = ahead == (ST - 1) * C::kTileBytes ? 0 : ahead + C::kTileBytes;

      // S^T: row m of 16 keys is key m / 2 % 4 + 4 (m % 2) + 8 (m / 8), so that V's
      // pairs below are keys t, t + 4 and t + 8, t + 12
      float sc[2][NT][4];
      uint32_t w[2][2][kKeyWords], unit[2][2][D / 64];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
          sc[half][n][0] = sc[half][n][1] = sc[half][n][2] = sc[half][n][3] = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          constexpr int kRow = D / 2, kScaleRow = D / kFp4Block;
          load_words<kKeyWords>(kc + (16 * half + 8 * i) * kRow, w[half][i]);
          if constexpr (D == 128) {
            const uint32_t s = e4m3_to_half(*reinterpret_cast<const uint16_t*>(
                ks + (16 * half + 8 * i) * kScaleRow));
            unit[half][i][0] = __byte_perm(s, 0, 0x1010);
            unit[half][i][1] = __byte_perm(s, 0, 0x3232);
          } else {
            unit[half][i][0] =
                e4m3_to_half(ks[(16 * half + 8 * i) * kScaleRow] * 0x0101u);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kKeyWords; ++j) {
        uint32_t x[2][2][4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          e2m1_to_half(w[half][0][j], x[half][0]);
          e2m1_to_half(w[half][1][j], x[half][1]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {   // two steps of 16 columns a word
          uint32_t ka[2][4];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            ka[half][0] = mul_half2(x[half][0][2 * i], unit[half][0][j / 2]);
            ka[half][1] = mul_half2(x[half][1][2 * i], unit[half][1][j / 2]);
            ka[half][2] = mul_half2(x[half][0][2 * i + 1], unit[half][0][j / 2]);
            ka[half][3] = mul_half2(x[half][1][2 * i + 1], unit[half][1][j / 2]);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            uint2 q;
            if constexpr (C::kSharedQ) q = sq[(((kOwnQ ? warp : mt) * NT + n) * kSteps + 2 * j + i) * 32 + lane];
            else q = make_uint2(qb[n][2 * j + i][0], qb[n][2 * j + i][1]);
            mma16816_half(sc[0][n], ka[0], q.x, q.y);
            mma16816_half(sc[1][n], ka[1], q.x, q.y);
          }
        }
      }
      if (k0 + KT > open) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int end = limit(n, i) - k0 - kg;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              if (16 * half >= end) sc[half][n][i] = -INFINITY;
              if (16 * half + 8 >= end) sc[half][n][2 + i] = -INFINITY;
            }
          }
      }
      // The maximum that the scores are taken against follows only where P would pass
      // 2^kPLazy.  (Rounded up: of scores so large that fp32 has no halves P stays there.)
      bool over = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float top = fmaxf(fmaxf(sc[0][n][i], sc[0][n][2 + i]), fmaxf(sc[1][n][i], sc[1][n][2 + i]));
          over = over || __fmaf_ru(top, c2[n][i], -kPLazy) > m[n][i];
        }
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float top = fmaxf(fmaxf(sc[0][n][i], sc[0][n][2 + i]), fmaxf(sc[1][n][i], sc[1][n][2 + i]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            const float mn = fmaxf(m[n][i], fmaf(top, c2[n][i], -kPTop));
            const float alpha = ex2_approx(m[n][i] - mn);
            m[n][i] = mn;
            l[n][i] *= alpha;
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
              o[k][n][i] *= alpha;
              o[k][n][2 + i] *= alpha;
            }
          }
      }
      // P^T = 2^(S c - m c) as fp16 B fragments; row sums from the same fp32 values
      uint32_t pb[2][NT][2];
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float p0 = ex2_approx(fmaf(sc[half][n][2 * i], c2[n][0], -m[n][0]));
            const float p1 = ex2_approx(fmaf(sc[half][n][2 * i + 1], c2[n][1], -m[n][1]));
            l[n][0] += p0;
            l[n][1] += p1;
            pb[half][n][i] = transpose8(pack_half2(p0, p1));
          }
      // O^T += V^T P^T: lane g has columns (D / 8) g ...; MMA row g is column 2 i, row
      // g + 8 column 2 i + 1 of them
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t w[4][D / 64], s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          load_words<D / 64>(vc + (16 * half + 4 * j) * (D / 2), w[j]);
          s[j] = vs[(16 * half + 4 * j) * (D / kFp4Block)];
        }
        const uint32_t unit[2] = {e4m3_to_half(__byte_perm(s[0], s[1], 0x0040)),
                                  e4m3_to_half(__byte_perm(s[2], s[3], 0x0040))};
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          uint32_t x[2][2][4];   // [pair of keys][column 2 i or 2 i + 1][i]
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t w0 = w[2 * k][j], w1 = w[2 * k + 1][j];
            e2m1_to_half((w0 & 0x0f0f0f0fu) | ((w1 << 4) & 0xf0f0f0f0u), x[k][0]);
            e2m1_to_half(((w0 >> 4) & 0x0f0f0f0fu) | (w1 & 0xf0f0f0f0u), x[k][1]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t va[4] = {mul_half2(x[0][0][i], unit[0]), mul_half2(x[0][1][i], unit[0]),
                                    mul_half2(x[1][0][i], unit[1]), mul_half2(x[1][1][i], unit[1])};
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma16816_half(o[4 * j + i][n], va, pb[half][n][0], pb[half][n][1]);
          }
        }
      }
    }
    copies_wait_but<0>();
    PagedPiece next = p;
    next.valid = false;
    if constexpr (MODE == kSplit) {
      next = paged_next<KT, C::kOverhead>(a, share, p);
      slot_sync();   // the ring is free
      if (next.valid) fetch(next);
    }

    // the sums over the lanes of equal t
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], 4);
        l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], 8);
        l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], 16);
        // no keys; a row of NaN scores has seen some
        if (l[n][i] == 0.f) m[n][i] = -INFINITY;
        else if (l[n][i] != l[n][i]) m[n][i] = 0.f;
      }
    if constexpr (MODE == kSolo) {   // straight from the registers, 2 or 1 16-byte words a row
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = n * 8 + 2 * t + i;
          if (r >= nrows) continue;
          const int h = (row0 + r) / a.n_q, qt = row0 + r - h * a.n_q;
          const float w = l[n][i] == 0.f ? 0.f : f.v_descale / l[n][i];
          uint4* to = reinterpret_cast<uint4*>(a.o + p.b * a.stride_b + h * a.stride_h +
                                               static_cast<int64_t>(qt) * a.stride_n + (D / 8) * g);
          uint32_t x[kSteps];
#pragma unroll
          for (int k = 0; k < kSteps; ++k) x[k] = pack_bf16x2(o[k][n][i] * w, o[k][n][2 + i] * w);
#pragma unroll
          for (int k = 0; k < kSteps / 4; ++k)
            to[k] = make_uint4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
          if (g == 0)
            a.lse[static_cast<int64_t>(p.b) * a.all_rows + row0 + r] =
                l[n][i] == 0.f ? -INFINITY : fmaf(m[n][i], kLn2, logf(l[n][i]));
        }
    } else {
    // ---- the slots' states merged: m, l per row, then O through shared memory
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (g == 0) {
          sh.m[slot][(mt * NT + n) * 8 + 2 * t + i] = m[n][i];
          sh.l[slot][(mt * NT + n) * 8 + 2 * t + i] = l[n][i];
        }
      }
    __syncthreads();
    auto total = [&](int r, float* top) {
      float mx = -INFINITY, lt = 0.f;
#pragma unroll
      for (int w = 0; w < kSlots; ++w) mx = fmaxf(mx, sh.m[w][r]);
#pragma unroll
      for (int w = 0; w < kSlots; ++w) {
        const float mw = sh.m[w][r];
        if (mw != -INFINITY) lt += sh.l[w][r] * ex2_approx(mw - mx);
      }
      *top = mx;
      return lt;
    };
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx;
        const float lt = total((mt * NT + n) * 8 + 2 * t + i, &mx);
        // this slot's weight, with descale / l folded in
        const float w = m[n][i] == -INFINITY ? 0.f : ex2_approx(m[n][i] - mx) * (f.v_descale / lt);
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          o[k][n][i] *= w;
          o[k][n][2 + i] *= w;
        }
      }
    const bool whole = p.whole();
    if constexpr (MODE == kSplit) {
      if (p.t0 == 0 && !whole) note = paged_note<C::kOverhead>(share, p);
      if (a.by_segment && p.t0 == 0 && threadIdx.x == 0)
        a.notes[p.b * a.heads + p.h] = whole ? MergeNote{p.b, p.h, 0, -1} : note;
    }
    const int64_t part = 2 * static_cast<int64_t>(blockIdx.x) + (p.s < share.lo ? 0 : 1);
    // slots 0, 1 write, 2, 3 add, ...: the sum has a fixed order.  Column (D / 8) g +
    // 2 i + b of a row lies at 16 i + 2 g + b
    for (int w = 0; w < kSlots; w += 2) {
      if (slot == w || slot == w + 1) {
        float* to = red + (slot - w) * C::kRows * C::kRedStride;
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float2* at = reinterpret_cast<float2*>(
                  to + ((mt * NT + n) * 8 + 2 * t + i) * C::kRedStride + 16 * k + 2 * g);
              float2 x = make_float2(o[k][n][i], o[k][n][2 + i]);
              if (w > 0) {
                const float2 y = *at;
                x.x += y.x;
                x.y += y.y;
              }
              *at = x;
            }
      }
      __syncthreads();
    }
    for (int e = threadIdx.x; e < nrows * (D / 4); e += C::kThreads) {
      const int r = e / (D / 4), c = 4 * (e - r * (D / 4));
      const int gg = c / (D / 8), k = c % (D / 8) / 2;
      float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < (kSlots > 1 ? 2 : 1); ++w) {
        const float* from = red + (w * C::kRows + r) * C::kRedStride + 2 * gg;
        const float2 y = *reinterpret_cast<const float2*>(from + 16 * k);
        const float2 z = *reinterpret_cast<const float2*>(from + 16 * k + 16);
        x[0] += y.x;
        x[1] += y.y;
        x[2] += z.x;
        x[3] += z.y;
      }
      float mx, L = 0.f;
      if (c == 0) {
        const float lt = total(r, &mx);
        L = lt == 0.f ? -INFINITY : fmaf(mx, kLn2, logf(lt));
      }
      if (MODE == kCluster && a.cluster > 1) {   // for the others (this thread's own place)
        *reinterpret_cast<float2*>(&red[r * C::kRedStride + 2 * gg + 16 * k]) = make_float2(x[0], x[1]);
        *reinterpret_cast<float2*>(&red[r * C::kRedStride + 2 * gg + 16 * k + 16]) =
            make_float2(x[2], x[3]);
        if (c == 0) sh.L[r] = L;
      } else if (MODE == kCluster || whole) {
        const int h = (row0 + r) / a.n_q, qt = row0 + r - h * a.n_q;
        *reinterpret_cast<uint2*>(a.o + p.b * a.stride_b + h * a.stride_h +
                                  static_cast<int64_t>(qt) * a.stride_n + c) =
            make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
        if (c == 0) a.lse[static_cast<int64_t>(p.b) * a.all_rows + row0 + r] = L;
      } else {
        *reinterpret_cast<float4*>(a.part_o + (part * a.rows + r) * D + c) =
            make_float4(x[0], x[1], x[2], x[3]);
        if (c == 0) a.part_l[part * a.rows + r] = L;
      }
    }
    if constexpr (MODE == kCluster) {
      if (a.cluster > 1) {   // each CTA of the cluster writes a part of the items
        cluster_sync();
        for (int e = rank * C::kThreads + threadIdx.x; e < nrows * (D / 4);
             e += a.cluster * C::kThreads) {
          const int r = e / (D / 4), c = 4 * (e - r * (D / 4));
          const float* at = &red[r * C::kRedStride + 2 * (c / (D / 8)) + 16 * (c % (D / 8) / 2)];
          float top = -INFINITY, sum = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
          for (int k = 0; k < a.cluster; ++k)
            top = fmaxf(top, cluster_ld(cluster_addr(&sh.L[r], k)));
          top = merge_base(top);
          for (int k = 0; k < a.cluster; ++k) {
            const float w = __expf(cluster_ld(cluster_addr(&sh.L[r], k)) - top);
            float y[4];
            cluster_ld2(cluster_addr(at, k), y);
            cluster_ld2(cluster_addr(at + 16, k), y + 2);
            sum += w;
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = fmaf(w, y[i], x[i]);
          }
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          const int h = (row0 + r) / a.n_q, qt = row0 + r - h * a.n_q;
          *reinterpret_cast<uint2*>(a.o + p.b * a.stride_b + h * a.stride_h +
                                    static_cast<int64_t>(qt) * a.stride_n + c) =
              make_uint2(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv));
          if (c == 0)
            a.lse[static_cast<int64_t>(p.b) * a.all_rows + row0 + r] =
                sum == 0.f ? -INFINITY : top + logf(sum);
        }
        cluster_sync();   // the others have read this CTA's rows
      }
    }
    __syncthreads();   // red, m and l are free
    }
    p = next;
  }
  if (MODE == kSplit && !a.by_segment && threadIdx.x == 0) a.notes[blockIdx.x] = note;
}

template <int D, int NT, int MT, Fp4Mode MODE>
cudaError_t launch_mode(const PagedArgs& a, const Fp4Args& f, int ctas, cudaStream_t s) {
  using C = Fp4Cfg<D, NT, MT>;
  static std::atomic<uint64_t> set_up{0};
  int dev = 0;
  bool todo = false;
  cudaError_t e = needs_setup(set_up, &dev, &todo);
  if (e != cudaSuccess) return e;
  auto kernel = fp4_decode_kernel<D, NT, MT, MODE>;
  if (todo) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    mark_done(set_up, dev);
  }
  const unsigned segments = static_cast<unsigned>(a.B * a.heads);
  if (MODE == kCluster)
    return launch_clusters(kernel, dim3(segments * a.cluster), dim3(C::kThreads), C::kSmem,
                           a.cluster, s, a, f);
  const unsigned grid = MODE == kSolo ? (segments + C::kSlots - 1) / C::kSlots : ctas;
  return launch_pdl(kernel, dim3(grid), dim3(C::kThreads), C::kSmem, s, a, f);
}

template <int D, int NT, int MT>
cudaError_t launch_rows(const PagedArgs& a, const Fp4Args& f, int ctas, cudaStream_t s) {
  if (a.cluster > 0) return launch_mode<D, NT, MT, kCluster>(a, f, ctas, s);
  if constexpr (MT == 1)
    if (a.cluster < 0) return launch_mode<D, NT, MT, kSolo>(a, f, ctas, s);
  if constexpr (!fp4_in_tiles(8 * NT * MT, D)) return launch_mode<D, NT, MT, kSplit>(a, f, ctas, s);
  return cudaErrorInvalidValue;   // (launch_fp4_tile's)
}

template <int D>
cudaError_t launch_width(const PagedArgs& a, const Fp4Args& f, int ctas, cudaStream_t s) {
  if (a.rows <= 8) return launch_rows<D, 1, 1>(a, f, ctas, s);
  if (a.rows <= 16) return launch_rows<D, 2, 1>(a, f, ctas, s);
  if (a.rows <= 32) return launch_rows<D, 4, 1>(a, f, ctas, s);
  return launch_rows<D, 4, 2>(a, f, ctas, s);
}

}  // namespace

cudaError_t launch_fp4_decode(const PagedArgs& a, const Fp4Args& f, int ctas, cudaStream_t s) {
  return a.d == 64 ? launch_width<64>(a, f, ctas, s) : launch_width<128>(a, f, ctas, s);
}

}  // namespace attn
