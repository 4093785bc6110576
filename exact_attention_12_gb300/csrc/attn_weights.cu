// The attention weight that cached keys receive from query rows.
//
// What it computes: for key j of sequence b and key/value head h
//   W[j] = sum_r exp(c q_r k_j - L_r),
// r over the head's query rows that attend j (those of attn_paged.cu), L_r their
// logsumexp, which the decode step has left; W is added to what the key has
// gathered, or replaces it.  With L known there is no softmax to carry along and
// nothing to merge: one pass over the keys, each by one warp.
//
// Bound: HBM for the few rows of a decode step, 2 d + 8 bytes a key (9 d / 16 + 8
// in 4 bits); for the hundred rows of an observation window the exponentials,
// 16 a clock and SM, and the products as much.
//   * S^T = K Q^T by 16 x 8 x 16 warp MMAs, 16 keys by 8 rows: K's fragments come
//     straight from global memory into registers (the sum over d may go in
//     any order, so lane (g, t) takes 16-byte pieces of keys g and g + 8), the next
//     group's while this one is worked on, and stay there for all rows;
//   * Q's fragments lie in shared memory in the order in which a warp reads them,
//     up to 256 rows at a time;
//   * the sum over a key's rows is each lane's own until the last row, then
//     two shuffles.
// Keys in 4 bits are unpacked as in attn_fp4.cu (exactly, to fp16).
#include "attn_fp4.cuh"

namespace attn {
using namespace sm103;

namespace {

constexpr int kWeightWarps = 8;
constexpr int kWeightThreads = 32 * kWeightWarps;
constexpr int kWeightRows = 256;        // query rows of one pass at most

struct RowInfo {
  float c2, l2;   // score -> log2 units; L in them (+inf where the row gives nothing)
  int lim;        // keys below it are attended
  int pad;
};

__device__ __forceinline__ void mma16816_bf16(float* c, const uint32_t* a, uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// What a lane holds of 16 keys: its pieces of keys g and g + 8.
template <int D, bool PACKED>
struct KeyPieces {
  static constexpr int kWords = PACKED ? D / 32 : D / 8;
  uint32_t w[2][kWords];
  uint32_t scale[PACKED ? 2 : 1];
};

template <int D, bool PACKED>
__global__ void __launch_bounds__(kWeightThreads, 2)
    key_weights_kernel(const PagedArgs a, const WeightArgs f) {
  constexpr int kSteps = D / 16;
  constexpr int G = PACKED ? 2 : 1;   // groups of 16 keys that are loaded together
  extern __shared__ __align__(16) uint8_t smem[];
  RowInfo* rows = reinterpret_cast<RowInfo*>(smem);                        // [f.pass_rows]
  uint2* qf = reinterpret_cast<uint2*>(smem + f.pass_rows * sizeof(RowInfo));   // [rows/8][kSteps][32]
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
  // 16 keys (group v of the warp's: half v % 2 of tile v / 2); zeros where no page is
  auto load = [&](const PagedPiece& p, int v, KeyPieces<D, PACKED>& x) {
    const int u = v >> 1, half = v & 1;
    const int pg0 = __shfl_sync(0xffffffffu, page_of[0], u & 31);
    const int pg1 = __shfl_sync(0xffffffffu, page_of[1], u & 31);
    const int64_t page = small_pages && half ? pg1 : pg0;
    const bool there = page < a.num_pages;
    const int row = ((p.t0 + warp + kWeightWarps * u) * kWeightKeys + 16 * half) &
                    ((1 << a.page_shift) - 1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = row + g + 8 * i;
      if constexpr (PACKED) {
        const uint8_t* from = f.cache.codes + page * f.cache.code_page +
                              p.h * f.cache.code_head + r * (D / 2) + t * (D / 8);
        const uint8_t* unit = f.cache.scales + page * f.cache.scale_page +
                              p.h * f.cache.scale_head + r * (D / kFp4Block) + t * (D / 64);
        if constexpr (D == 128) {
          const uint4 y = there ? __ldcs(reinterpret_cast<const uint4*>(from))
                                : make_uint4(0u, 0u, 0u, 0u);
          x.w[i][0] = y.x;
          x.w[i][1] = y.y;
          x.w[i][2] = y.z;
          x.w[i][3] = y.w;
          x.scale[i] = there ? *reinterpret_cast<const uint16_t*>(unit) : 0u;
        } else {
          const uint2 y = there ? __ldcs(reinterpret_cast<const uint2*>(from)) : make_uint2(0u, 0u);
          x.w[i][0] = y.x;
          x.w[i][1] = y.y;
          x.scale[i] = there ? *unit * 0x0101u : 0u;
        }
      } else {
        // piece k of a row: 16 bytes, 8 columns, the four lanes' side by side
        const __nv_bfloat16* from = f.k + page * f.stride_page + p.h * f.stride_head +
                                    r * f.stride_row + 8 * t;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          const uint4 y = there ? __ldcs(reinterpret_cast<const uint4*>(from + 32 * k))
                                : make_uint4(0u, 0u, 0u, 0u);
          x.w[i][4 * k] = y.x;
          x.w[i][4 * k + 1] = y.y;
          x.w[i][4 * k + 2] = y.z;
          x.w[i][4 * k + 3] = y.w;
        }
      }
    }
  };
  // A fragments: step s takes columns 4 s ... 4 s + 3 of a lane's pieces
  auto fragments = [&](const KeyPieces<D, PACKED>& x, uint32_t (*ka)[4]) {
    if constexpr (PACKED) {
      uint32_t unit[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t s = e4m3_to_half(x.scale[i]);
        unit[i][0] = __byte_perm(s, 0, 0x1010);
        unit[i][1] = __byte_perm(s, 0, 0x3232);
      }
#pragma unroll
      for (int j = 0; j < KeyPieces<D, PACKED>::kWords; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t y[4];
          e2m1_to_half(x.w[i][j], y);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            ka[2 * j + k / 2][i + 2 * (k & 1)] = mul_half2(y[k], unit[i][j / 2]);
        }
    } else {
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        ka[s][0] = x.w[0][2 * s];
        ka[s][1] = x.w[1][2 * s];
        ka[s][2] = x.w[0][2 * s + 1];
        ka[s][3] = x.w[1][2 * s + 1];
      }
    }
  };

  for (PagedPiece p = paged_piece<kWeightKeys, kWeightOverhead>(a, share, share.b, 0, share.s);
       p.valid; p = paged_next<kWeightKeys, kWeightOverhead>(a, share, p)) {
    const int tiles = p.t1 - p.t0 - warp;
    const int nu = tiles > 0 ? (tiles + kWeightWarps - 1) / kWeightWarps : 0;
    for (int r0 = 0; r0 < a.head_rows; r0 += f.pass_rows) {   // (one pass but for very many rows)
      const int nrows = min(a.head_rows - r0, f.pass_rows), blocks = (nrows + 7) / 8;
      __syncthreads();   // the rows before are no longer in use
      for (int n = warp; n < blocks; n += kWeightWarps) {
        const int r = 8 * n + g, at = p.h * a.head_rows + r0 + r;
        const bool live = r < nrows;
        const int h = at / a.n_q, qt = at - h * a.n_q;
        const __nv_bfloat16* qr =
            a.q + p.b * a.stride_b + h * a.stride_h + static_cast<int64_t>(qt) * a.stride_n;
        uint32_t w[D / 8];
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
        float c2 = a.scale_log2;
        if constexpr (PACKED) {
          int e = 0;
          half_rows<D / 8>(w, &e);
          c2 = score_factor(a.scale_log2 * f.k_descale, e);
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
          qf[(n * kSteps + s) * 32 + lane] = make_uint2(w[2 * s], w[2 * s + 1]);
        if (t == 0) {
          const float L = live ? f.lse[static_cast<int64_t>(p.b) * a.all_rows + at] : -INFINITY;
          RowInfo& info = rows[r];
          info.c2 = c2;
          info.l2 = L == -INFINITY ? INFINITY : L * kLog2Of;
          info.lim = !live || L == -INFINITY
                         ? 0
                         : (a.causal ? min(p.len, p.len - a.n_q + qt + 1) : p.len);
        }
      }
      __syncthreads();
      const bool ragged = (nrows & 7) != 0;
      if (nu > 0) load_pages(p, 0, nu);
      KeyPieces<D, PACKED> next[G];
#pragma unroll
      for (int i = 0; i < G; ++i)
        if (nu > 0) load(p, i, next[i]);
      for (int v0 = 0; v0 < 2 * nu; v0 += G) {
        KeyPieces<D, PACKED> now[G];
#pragma unroll
        for (int i = 0; i < G; ++i) now[i] = next[i];
        if (v0 + G < 2 * nu) {
          if (((v0 + G) & 63) == 0) load_pages(p, (v0 + G) >> 1, nu);
#pragma unroll
          for (int i = 0; i < G; ++i) load(p, v0 + G + i, next[i]);
        }
#pragma unroll
        for (int i = 0; i < G; ++i) {
          const int v = v0 + i;
          const int k0 = (p.t0 + warp + kWeightWarps * (v >> 1)) * kWeightKeys + 16 * (v & 1);
          if (k0 >= p.len) continue;
          // lanes t = 0, 1 have keys g, g + 8 to write
          const int mine = k0 + g + 8 * (t & 1);
          const bool writes = t < 2 && mine < p.len;
          float* to = f.weights + p.b * f.stride_b + p.h * f.stride_h + mine;
          float before = 0.f;
          if (writes && (f.add || r0 > 0)) before = *to;
          uint32_t ka[kSteps][4];
          fragments(now[i], ka);
          const bool masked = ragged || k0 + 16 > (a.causal ? p.len - a.n_q + 1 : p.len);
          float sum[2] = {0.f, 0.f};
          for (int n = 0; n < blocks; ++n) {
            float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
              const uint2 b = qf[(n * kSteps + s) * 32 + lane];
              if constexpr (PACKED) mma16816_half(c, ka[s], b.x, b.y);
              else mma16816_bf16(c, ka[s], b.x, b.y);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const RowInfo info = rows[8 * n + 2 * t + j];
              float p0 = ex2_approx(fmaf(c[j], info.c2, -info.l2));
              float p1 = ex2_approx(fmaf(c[2 + j], info.c2, -info.l2));
              if (masked) {
                if (k0 + g >= info.lim) p0 = 0.f;
                if (k0 + g + 8 >= info.lim) p1 = 0.f;
              }
              sum[0] += p0;
              sum[1] += p1;
            }
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 1);
            sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 2);
          }
          if (writes) *to = before + (t == 0 ? sum[0] : sum[1]);
        }
      }
    }
  }
}

template <int D, bool PACKED>
cudaError_t launch_kind(const PagedArgs& a, const WeightArgs& f, int ctas, cudaStream_t s) {
  const size_t bytes = f.pass_rows * (sizeof(RowInfo) + D * 2);
  static std::atomic<uint64_t> set_up{0};
  int dev = 0;
  bool todo = false;
  cudaError_t e = needs_setup(set_up, &dev, &todo);
  if (e != cudaSuccess) return e;
  if (todo) {
    e = cudaFuncSetAttribute(key_weights_kernel<D, PACKED>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kWeightRows * (sizeof(RowInfo) + D * 2));
    if (e != cudaSuccess) return e;
    mark_done(set_up, dev);
  }
  return launch_pdl(key_weights_kernel<D, PACKED>, dim3(ctas), dim3(kWeightThreads), bytes, s, a, f);
}

}  // namespace

cudaError_t launch_key_weights(const PagedArgs& a, WeightArgs f, int ctas, cudaStream_t s) {
  const int rows = (a.head_rows + 7) / 8 * 8;
  f.pass_rows = rows < kWeightRows ? rows : kWeightRows;
  if (f.k == nullptr)
    return a.d == 64 ? launch_kind<64, true>(a, f, ctas, s) : launch_kind<128, true>(a, f, ctas, s);
  return a.d == 64 ? launch_kind<64, false>(a, f, ctas, s) : launch_kind<128, false>(a, f, ctas, s);
}

}  // namespace attn
