// The attention weight that cached keys receive from the few query rows of a decode
// step (up to 32 of a key/value head; more: attn_weights_tile.cu).
//
// What it computes: for key j of sequence b and key/value head h
//   W[j] = sum_r exp(c q_r k_j - L_r),
// r over the head's query rows that attend j (those of attn_paged.cu), L_r their
// logsumexp, which the decode step has left; W is added to what the key has
// gathered, or replaces it.  With L known there is no softmax to carry along and
// nothing to merge: one pass over the keys, each by one warp.
//
// Bound: HBM, 2 d + 8 bytes a key (9 d / 16 + 8 in 4 bits).
//   * 16 x 8 x 16 warp MMAs, 16 keys by 8 rows, S^T = K Q^T: no lane idle at 8
//     rows.  K's fragments come straight from global memory into registers (the
//     sum over d may go in any order, so lane (g, t) takes 16-byte pieces of its
//     keys), the next keys' while these are worked on;
//   * Q's fragments lie in shared memory in the order in which a warp reads them;
//   * the sum over a key's rows is each lane's own until the last row, then two
//     shuffles.
// Keys in 4 bits are unpacked as in attn_fp4.cu (exactly, to fp16).
// Measured: 16 sequences of 2048-8192 keys, 32 heads over 8, d = 128, 173 MB in 30 us
// = 5.8 TB/s; 16 of 8192 277 MB in 45 us, of a cache in 4 bits 84 MB in 29 us (floor 12):
// the unpacking, for 4 rows.
#include "attn_fp4.cuh"

namespace attn {
using namespace sm103;

namespace {

constexpr int kWeightWarps = 8;
constexpr int kWeightThreads = 32 * kWeightWarps;

struct RowInfo {
  float c2, l2;   // score -> log2 units; L in them (+inf where the row gives nothing)
  int lim;        // keys below it are attended
  int pad;
};

__device__ __forceinline__ void mma16816_bf16(float* c, const uint32_t* a, uint32_t b0,
                                              uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// What lane (g, t) holds of a key: a quarter of its row.
template <int D, bool PACKED>
struct KeyPart {
  uint32_t w[PACKED ? D / 32 : D / 8];
  uint32_t scale;
};

// Zeros where there is no page.
template <int D, bool PACKED>
__device__ __forceinline__ void load_part(const PagedArgs& a, const WeightArgs& f, int64_t page,
                                          int head, int row, int t, KeyPart<D, PACKED>& x) {
  const bool there = page < a.num_pages;
  if constexpr (PACKED) {
    const uint8_t* from = f.cache.codes + page * f.cache.code_page + head * f.cache.code_head +
                          row * (D / 2) + t * (D / 8);
    const uint8_t* unit = f.cache.scales + page * f.cache.scale_page + head * f.cache.scale_head +
                          row * (D / kFp4Block) + t * (D / 64);
    if constexpr (D == 128) {
      const uint4 y =
          there ? __ldcs(reinterpret_cast<const uint4*>(from)) : make_uint4(0u, 0u, 0u, 0u);
      x.w[0] = y.x;
      x.w[1] = y.y;
      x.w[2] = y.z;
      x.w[3] = y.w;
      x.scale = there ? *reinterpret_cast<const uint16_t*>(unit) : 0u;
    } else {
      const uint2 y = there ? __ldcs(reinterpret_cast<const uint2*>(from)) : make_uint2(0u, 0u);
      x.w[0] = y.x;
      x.w[1] = y.y;
      x.scale = there ? *unit * 0x0101u : 0u;
    }
  } else {
    // piece k: 16 bytes, 8 columns, the four lanes' side by side
    const __nv_bfloat16* from =
        f.k + page * f.stride_page + head * f.stride_head + row * f.stride_row + 8 * t;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
      const uint4 y = there ? __ldcs(reinterpret_cast<const uint4*>(from + 32 * k))
                            : make_uint4(0u, 0u, 0u, 0u);
      x.w[4 * k] = y.x;
      x.w[4 * k + 1] = y.y;
      x.w[4 * k + 2] = y.z;
      x.w[4 * k + 3] = y.w;
    }
  }
}

// The part as MMA operands: step s takes its columns 4 s ... 4 s + 3, two registers.
template <int D, bool PACKED>
__device__ __forceinline__ void operands(const KeyPart<D, PACKED>& x, uint32_t (*b)[2]) {
  if constexpr (PACKED) {
    const uint32_t s = e4m3_to_half(x.scale);
    const uint32_t unit[2] = {__byte_perm(s, 0, 0x1010), __byte_perm(s, 0, 0x3232)};
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      uint32_t y[4];
      e2m1_to_half(x.w[j], y);
#pragma unroll
      for (int k = 0; k < 4; ++k) b[2 * j + k / 2][k & 1] = mul_half2(y[k], unit[j / 2]);
    }
  } else {
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      b[s][0] = x.w[2 * s];
      b[s][1] = x.w[2 * s + 1];
    }
  }
}

// The quarter of a row of Q that goes with it (zeros if not `live`), and what turns a
// score into log2 units.
template <int D, bool PACKED>
__device__ __forceinline__ float load_query(const PagedArgs& a, const WeightArgs& f, int b, int at,
                                            bool live, int t, uint32_t* w) {
  const int h = at / a.n_q, qt = at - h * a.n_q;
  const __nv_bfloat16* qr =
      a.q + b * a.stride_b + h * a.stride_h + static_cast<int64_t>(qt) * a.stride_n;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const uint4 y = live ? *reinterpret_cast<const uint4*>(
                               qr + (PACKED ? t * (D / 4) + 8 * i : 32 * i + 8 * t))
                         : make_uint4(0u, 0u, 0u, 0u);
    w[4 * i] = y.x;
    w[4 * i + 1] = y.y;
    w[4 * i + 2] = y.z;
    w[4 * i + 3] = y.w;
  }
  if constexpr (PACKED) {
    int e = 0;
    half_rows<D / 8>(w, &e);
    return score_factor(a.scale_log2 * f.k_descale, e);
  }
  return a.scale_log2;
}

__device__ __forceinline__ RowInfo row_info(const PagedArgs& a, int len,
                                            int at, float L, float c2) {
  RowInfo info;
  info.c2 = c2;
  info.l2 = L == -INFINITY ? INFINITY : L * kLog2Of;
  info.lim = L == -INFINITY ? 0 : (a.causal ? min(len, len - a.n_q + at % a.n_q + 1) : len);
  info.pad = 0;
  return info;
}

template <int D, bool PACKED>
__global__ void __launch_bounds__(kWeightThreads, 2)
    key_weights_kernel(const PagedArgs a, const WeightArgs f) {
  constexpr int kSteps = D / 16, kWords = D / 8;
  constexpr int kParts = PACKED ? 4 : 2;   // keys of a lane at a time, 8 apart
  extern __shared__ __align__(16) uint8_t smem[];
  RowInfo* rows = reinterpret_cast<RowInfo*>(smem);       // [f.pass_rows]
  uint2* qf = reinterpret_cast<uint2*>(smem + f.pass_rows * sizeof(RowInfo));   // [rows / 8][kSteps][32]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  grid_dep_wait();
  grid_dep_launch();
  const PagedShare share =
      paged_share<kWeightKeys, kWeightOverhead, kWeightMinUnits>(a, blockIdx.x, gridDim.x);

  int page_of[2] = {0, 0};
  const bool small_pages = a.page_shift < 5;
  auto load_pages = [&](const PagedPiece& p, int u0, int nu) {
    const int u = u0 + lane;
    if (u < nu) {
      const int key = (p.t0 + warp + kWeightWarps * u) * kWeightKeys;
      const int32_t* row = a.table + p.b * a.table_stride;
      page_of[0] = checked_page(row[key >> a.page_shift], a.num_pages, a.status);
      page_of[1] = !small_pages || key + 16 >= p.len
                       ? page_of[0]
                       : checked_page(row[(key >> a.page_shift) + 1], a.num_pages, a.status);
    }
  };
  // the warp's keys from 8 v on (part v % 4 of its tile v / 4)
  auto load = [&](const PagedPiece& p, int v, KeyPart<D, PACKED>* x) {
    const int u = v >> 2;
    const int pg0 = __shfl_sync(0xffffffffu, page_of[0], u & 31);
    const int pg1 = __shfl_sync(0xffffffffu, page_of[1], u & 31);
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      const int part = (v & 3) + i;
      const int row = ((p.t0 + warp + kWeightWarps * u) * kWeightKeys + 8 * part) &
                      ((1 << a.page_shift) - 1);
      load_part<D, PACKED>(a, f, small_pages && part >= 2 ? pg1 : pg0, p.h, row + g, t, x[i]);
    }
  };

  for (PagedPiece p = paged_piece<kWeightKeys, kWeightOverhead>(a, share, share.b, 0, share.s);
       p.valid; p = paged_next<kWeightKeys, kWeightOverhead>(a, share, p)) {
    const int tiles = p.t1 - p.t0 - warp;
    const int nv = tiles > 0 ? (tiles + kWeightWarps - 1) / kWeightWarps * 4 : 0;
    const int blocks = (a.head_rows + 7) / 8;
    __syncthreads();   // the rows before are no longer in use
    bool dead = false;
    for (int n = warp; n < blocks; n += kWeightWarps) {
      const int r = 8 * n + g, at = p.h * a.head_rows + r;
      const float L = r < a.head_rows ? f.lse[static_cast<int64_t>(p.b) * a.all_rows + at] : -INFINITY;
      dead = dead || L == -INFINITY;
      uint32_t w[kWords];
      const float c2 = load_query<D, PACKED>(a, f, p.b, at, r < a.head_rows, t, w);
      if (t == 0) rows[r] = row_info(a, p.len, at, L, c2);
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
        qf[(n * kSteps + s) * 32 + lane] = make_uint2(w[2 * s], w[2 * s + 1]);
    }
    // a row that gives nothing may hold anything, and an infinite key makes NaN of zeros as
    // well: where there is one, what a row gives is chosen by its limit
    const bool some_dead = __syncthreads_or(dead) != 0;
    if (nv > 0) load_pages(p, 0, nv >> 2);
    KeyPart<D, PACKED> next[kParts];
    if (nv > 0) load(p, 0, next);
    for (int v = 0; v < nv; v += kParts) {
      KeyPart<D, PACKED> now[kParts];
#pragma unroll
      for (int i = 0; i < kParts; ++i) now[i] = next[i];
      if (v + kParts < nv) {
        if (((v + kParts) & 127) == 0) load_pages(p, (v + kParts) >> 2, nv >> 2);
        load(p, v + kParts, next);
      }
      const int k0 = (p.t0 + warp + kWeightWarps * (v >> 2)) * kWeightKeys + 8 * (v & 3);
      const bool masked = some_dead || k0 + 8 * kParts > (a.causal ? p.len - a.n_q + 1 : p.len);
      float* to = f.weights + p.b * f.stride_b + p.h * f.stride_h + k0;
      // lanes t = 0, 1 have keys g, g + 8 of 16 to write
      const int mine = g + 8 * (t & 1);
#pragma unroll
      for (int i = 0; i < kParts; i += 2) {
        float before = 0.f, sum[2] = {0.f, 0.f};
        const bool writes = t < 2 && k0 + mine + 8 * i < p.len;
        if (f.add && writes) before = to[mine + 8 * i];
        uint32_t kb[2][kSteps][2];
        operands<D, PACKED>(now[i], kb[0]);
        operands<D, PACKED>(now[i + 1], kb[1]);
        for (int n = 0; n < blocks; ++n) {
          float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < kSteps; ++s) {
            const uint2 q = qf[(n * kSteps + s) * 32 + lane];
            const uint32_t ka[4] = {kb[0][s][0], kb[1][s][0], kb[0][s][1], kb[1][s][1]};
            if constexpr (PACKED) mma16816_half(c, ka, q.x, q.y);
            else mma16816_bf16(c, ka, q.x, q.y);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const RowInfo info = rows[8 * n + 2 * t + j];
#pragma unroll
            for (int e = 0; e < 2; ++e) {   // keys g, g + 8
              float x = ex2_approx(fmaf(c[2 * e + j], info.c2, -info.l2));
              if (masked && k0 + 8 * i + 8 * e + g >= info.lim) x = 0.f;
              sum[e] += x;
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
          sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
        }
        if (writes) to[mine + 8 * i] = before + (t == 0 ? sum[0] : sum[1]);
      }
    }
  }
}

template <int D, bool PACKED>
cudaError_t launch_kind(const PagedArgs& a, const WeightArgs& f, int ctas, cudaStream_t s) {
  // (up to kWeightTileRows rows: less than the shared memory every kernel may have)
  const size_t bytes = f.pass_rows * (sizeof(RowInfo) + D * 2);
  return launch_pdl(key_weights_kernel<D, PACKED>, dim3(ctas), dim3(kWeightThreads), bytes, s, a, f);
}

}  // namespace

cudaError_t launch_key_weights(const PagedArgs& a, WeightArgs f, int ctas, cudaStream_t s) {
  f.pass_rows = (a.head_rows + 7) / 8 * 8;
  if (f.k == nullptr)
    return a.d == 64 ? launch_kind<64, true>(a, f, ctas, s) : launch_kind<128, true>(a, f, ctas, s);
  return a.d == 64 ? launch_kind<64, false>(a, f, ctas, s) : launch_kind<128, false>(a, f, ctas, s);
}

}  // namespace attn
