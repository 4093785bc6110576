// Caches in 4 bits: the format, its conversions, and the argument blocks of the
// kernels that store, load and read them (attn_fp4.cu, attn_fp4_store.cu,
// attn_weights.cu).
//
// A value is x = descale * s * c: c one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign
// (E2M1: two exponent bits, one of mantissa), s an E4M3 number that 16
// consecutive columns share, descale one fp32 factor of the tensor.  s * c has
// 4 + 2 significant bits and lies between 2^-10 and 2688: it is exact in fp16
// (and bf16), so the products of attention take the cache's values as they
// are, and descale is folded into the score scale and into O.
#pragma once
#include <cuda_fp16.h>

#include "attn_paged.cuh"

namespace attn {

constexpr int kFp4Block = 16;   // columns that share a scale

// One tensor of the cache: a head's rows of a page follow one another.
struct Fp4Cache {
  uint8_t* codes;                  // [num_pages][H_kv][page_size][d / 2]
  uint8_t* scales;                 // [num_pages][H_kv][page_size][d / 16]
  int64_t code_page, code_head;    // bytes between pages, between heads
  int64_t scale_page, scale_head;
};

struct Fp4Args {
  Fp4Cache k, v;
  float k_descale, v_descale;
};

// Storing the newest tokens of each sequence, and loading them back.
struct Fp4CopyArgs {
  int B, H, n, d;
  const int32_t* lens;             // [B] cache lengths
  const int32_t* counts;           // [B] tokens of each sequence among the n; null: n
  const int32_t* table;
  int64_t table_stride;
  int cap, page_shift, num_pages;
  __nv_bfloat16 *k, *v;            // [B][H][n][d]
  int64_t stride_b, stride_h, stride_n;
  Fp4Args cache;
  int* status;
};

// The attention weight of each key (attn_weights.cu).
struct WeightArgs {
  const __nv_bfloat16* k;          // null: the cache in 4 bits
  int64_t stride_page, stride_head, stride_row;
  Fp4Cache cache;
  float k_descale;
  const float* lse;                // [B][H][n_q]
  float* weights;
  int64_t stride_b, stride_h;      // of the weights
  int add;
  int pass_rows;                   // query rows of a pass, set by the launcher
  int ring;                        // key tiles in shared memory, set by the launcher
  int stall;                       // kStallWeightsSum: see attn_debug_stall
};
// Many rows (attn_weights_tile.cu); tk: the cache of bf16, boxes of min(128, page) rows.
cudaError_t launch_key_weights_tile(const CUtensorMap& tk, const PagedArgs& a, const WeightArgs& f,
                                    int ctas, cudaStream_t s);
// Rows of a head above which it is taken: 8 sequences of 8192 keys, 4 heads, 24 rows
// 18.3 us with it, 16.9 without; 40 rows 18.8 and 20.2; 128 rows 18.5 and 37.2.
constexpr int kWeightTileRows = 32;
// A segment's cost beside its 128-key tiles, 2 / 1 / 6: 64 sequences of 0-8192 keys, 64
// rows 108 / 115 / 103 us; 200 of 0-1000 77 / 83 / 68; two of 16384, 128 rows 18.5 / 19.3 /
// 17.5.
constexpr int kWeightTileOverhead = 2;
cudaError_t launch_key_weights(const PagedArgs& a, WeightArgs f, int ctas, cudaStream_t s);

// Up to kWeightTileRows rows, in tiles of 32 keys.  A segment's cost beside them, 8 / 2 /
// 20: 64 sequences of 0-8192 keys, 4 rows 93 / 101 / 92 us, one of 517 keys 7.3 / 8.5 / 6.9.
// Units a CTA takes at least, 16 / 4 / 48: one of 517 keys 7.3 / 5.4 / 11.8, one of 4096
// 7.1 / 6.0 / 12.2, long caches the same.
constexpr int kWeightKeys = 32;
constexpr int kWeightOverhead = 8;
constexpr int kWeightMinUnits = 16;

constexpr float kLog2Of = 1.4426950408889634f;   // log2(e)

// Decode: P is 2^(S c - m), m the row's maximum less kPTop, taken again only when a
// score passes m by more than kPLazy: P reaches 2^15 (fp16's end is 2^16), so what fp16
// cannot hold begins 2^32 below the maximum, not 2^25, and costs nothing.
constexpr float kPTop = 7.f;
constexpr float kPLazy = kPTop + 8.f;

cudaError_t launch_fp4_store(const Fp4CopyArgs& a, cudaStream_t s);
cudaError_t launch_fp4_load(const Fp4CopyArgs& a, cudaStream_t s);
cudaError_t launch_fp4_decode(const PagedArgs& a, const Fp4Args& f, int ctas, cudaStream_t s);

// Decode: key tiles of 32, and the constants of the split, in such tiles.  Swept on
// whole steps (us; H = 32, 8 key/value heads, d = 128 unless said).
// A segment's cost beside its tiles, 8 / 20 above 16 rows: 64 sequences of 0-16384
// keys, 32 rows 286 / 245.
constexpr int kFp4Keys = 32;
constexpr int fp4_overhead(int rows) { return rows <= 16 ? 8 : 20; }
// Units a CTA takes at least, 6 / 2 / 18 (room for 32768 keys): one sequence of 517 keys
// 8.7 / 8.0 / 12.2, 4 of 4096 12.6 / 12.6 / 15.5.
constexpr int kFp4MinUnits = 6;
// Tiles (at full caches) from which on a segment takes more than one CTA: 100 keys
// one CTA 4.5, two 6.2; 517 keys one 8.0, eight 6.4.
constexpr int kFp4ClusterFrom = 8;
// Tiles of a cluster's CTA at most: one sequence of 4096 keys, eight CTAs 8.8, the
// balanced split 9.3; 8192 keys 11.8 and 10.7; 64 rows, 16 sequences of 1000-2000
// keys 20.3 and 17.1.
constexpr int fp4_cluster_tiles(int rows) { return rows <= 32 ? 24 : 12; }
// Where there are more segments than CTAs at a time: tiles of a warp that has a
// segment to itself (300 sequences of 300-600 keys a warp each 38.9, a CTA 45.8,
// split 58.8; 200 of 600-1200 keys 68.2, 51.7, 60.8), and of a CTA (200 sequences
// of 0-2000 keys 61.1, split 70.3).
constexpr int kFp4SoloTiles = 24;
constexpr int kFp4ManyTiles = 64;

// Above 32 rows, d = 128, the balanced split goes to attn_fp4_tile.cu (which is written for
// 128 columns, TMEM's lanes of O^T): tiles of 128 keys, and its own constants in such
// tiles.  64 sequences of 16384 keys, 4 heads, 36 rows
// 299 us, attn_fp4.cu 469; 64 rows 303 and 474; 32 rows, with two tiles of 32 rows at a
// time, 269 and 230.
cudaError_t launch_fp4_tile(const PagedArgs& a, const Fp4Args& f, int ctas, cudaStream_t s);
// A segment's cost beside its tiles, 4 / 1 / 10: 64 sequences of 0-16384 keys, 64 rows 175 /
// 204 / 176, 200 of 0-4000 166 / 191 / 171.  Units a CTA takes at least, 5 / 2 / 15: one of
// 2000 keys, 64 rows 16.9 / 12.8 / 31.1, 64 of 0-16384 the same.
constexpr int kFp4TileOverhead = 4;
constexpr int kFp4TileMinUnits = 5;
constexpr bool fp4_in_tiles(int rows, int d) { return rows > 32 && d == 128; }

// CTAs of the decode kernel per SM at `rows` query rows of a segment: 16 warps of
// up to 8 rows, 12 of 16, 8 of 32.
constexpr int fp4_ctas_per_sm(int rows) {
  return rows <= 8 ? 4 : rows <= 16 ? 3 : rows <= 32 ? 2 : 1;
}

// ------------------------------------------------------------- conversions --

// Four bytes of codes: r[i] the two values of byte i (the low four bits first) as
// fp16.
__device__ __forceinline__ void e2m1_to_half(uint32_t w, uint32_t* r) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

// Two E4M3 numbers (the low byte first) as fp16.
__device__ __forceinline__ uint32_t e4m3_to_half(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}

__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// c += a b, 16 x 8 x 16, fp16 inputs, fp32 accumulators
__device__ __forceinline__ void mma16816_half(float* c, const uint32_t* a, uint32_t b0,
                                              uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// base + page * step, the step in 32 bits (the host sees to that).
__device__ __forceinline__ const uint8_t* page_at(const uint8_t* base, int page, int64_t step) {
  return base + static_cast<uint64_t>(static_cast<uint32_t>(page)) * static_cast<uint32_t>(step);
}

// e with top 2^e in [2^14, 2^15); 0 for an infinite top.
__device__ __forceinline__ int row_exponent(float top) {
  const int ef = static_cast<int>(__float_as_uint(top) >> 23);
  return ef == 255 ? 0 : min(141 - ef, 127);
}

// A row of Q, W words of bf16 pairs in each of the four lanes of equal lane / 4,
// as fp16 pairs times 2^e, with the row's largest element in [2^14, 2^15)
// (an infinite row: as it is).
template <int W>
__device__ __forceinline__ void half_rows(uint32_t* w, int* e) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < W; ++i)
    top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[i] << 16)),
                           fabsf(__uint_as_float(w[i] & 0xffff0000u))));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  *e = row_exponent(top);
  const float up = ldexpf(1.f, *e);
#pragma unroll
  for (int i = 0; i < W; ++i)
    w[i] = pack_half2(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xffff0000u) * up);
}

// What turns a product with such a row into log2 units: `factor` 2^-e, never 0 or
// infinite (a masked score stays -inf, a score of 0 stays 0).
__device__ __forceinline__ float score_factor(float factor, int e) {
  return fminf(fmaxf(ldexpf(factor, -e), 1.2e-38f), 3.0e38f);
}

}  // namespace attn
