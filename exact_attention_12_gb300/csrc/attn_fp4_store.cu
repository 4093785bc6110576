// Storing keys and values in a paged cache of 4 bits, and loading them back.
//
// What it computes (attn_fp4.cuh has the format): of each 16 columns x,
//   s = the E4M3 number nearest to max |x| / (6 descale), at most 448,
//   c = the E2M1 number nearest to x / (s descale), at most 6,
// ties to the even code; where s is 0 the codes are 0, where an x is NaN s is
// NaN and so are the 16 values.  Both are exactly the nearest: the quotient is
// taken with an approximate reciprocal, converted a little below and a little
// above, and where the two differ (a few in 2^19) the sign of x - border * descale
// decides, which one fused multiply-add gives exactly.
//
// Bound: HBM, 2.56 bytes an element.  A thread takes one block of 16 columns,
// 32 bytes in, 9 out; the rows of a page follow one another, so both sides
// are contiguous over a warp.
#include "attn_fp4.cuh"

namespace attn {
using namespace sm103;

namespace {

constexpr int kFp4Threads = 256;
constexpr float kBelow = 1.f - 0x1p-19f, kAbove = 1.f + 0x1p-19f;

__device__ __forceinline__ uint32_t e4m3_of(float x) {   // nearest, at most 448
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xffu;
}

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(e4m3_to_half(code) & 0xffffu)));
}

// Eight values as codes, the first in the low four bits; nearest, at most 6.
__device__ __forceinline__ uint32_t e2m1_of(const uint64_t* x) {   // four packed pairs
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t.reg .f32 l, h;\n\t"
      "mov.b64 {l, h}, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 a, h, l;\n\t"
      "mov.b64 {l, h}, %2;\n\tcvt.rn.satfinite.e2m1x2.f32 b, h, l;\n\t"
      "mov.b64 {l, h}, %3;\n\tcvt.rn.satfinite.e2m1x2.f32 c, h, l;\n\t"
      "mov.b64 {l, h}, %4;\n\tcvt.rn.satfinite.e2m1x2.f32 d, h, l;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "l"(x[0]), "l"(x[1]), "l"(x[2]), "l"(x[3]));
  return r;
}

__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float reciprocal(float x) {   // off by an ulp or so
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float e2m1_value(uint32_t magnitude) {   // of the low three bits
  return magnitude < 2 ? 0.5f * magnitude
                       : __uint_as_float((126u + (magnitude >> 1)) << 23 | (magnitude & 1u) << 22);
}

// Which of two neighbouring codes (their values times `unit`) is nearer to
// x >= 0 in units of descale; the even one if both are as near.
template <typename Value>
__device__ __forceinline__ uint32_t nearer(uint32_t low, uint32_t high, float x, float unit,
                                           float descale, const Value& value) {
  const float border = 0.5f * (value(low) + value(high)) * unit;   // 8 significant bits at most
  const float side = fmaf(-border, descale, x);
  return side < 0.f || (side == 0.f && (low & 1u) == 0) ? low : high;
}

// The scale's code of a block whose largest |x| is `top`.
__device__ __forceinline__ uint32_t block_scale(float top, float descale, float inv6) {
  const float t = top * inv6;
  const uint32_t low = e4m3_of(t * kBelow), high = e4m3_of(t * kAbove);
  if (low == high) return low;
  return nearer(low, high, top, 6.f, descale, [](uint32_t c) { return e4m3_value(c); });
}

// The blocks of a sequence's tokens: block i of `items` is columns 16 (i mod d / 16)
// of token i / (d / 16) (head * n + t).
struct Place {
  int h, t, blk;
  int page, row;     // where the token lies; page < 0: nowhere
  bool valid, live;  // there is such a block; the sequence has such a token
};

template <int D>
__device__ __forceinline__ Place place(const Fp4CopyArgs& a, int b, int64_t i, int len, int count) {
  constexpr int kBlocks = D / kFp4Block;
  Place p{};
  p.valid = i < static_cast<int64_t>(a.H) * a.n * kBlocks;
  p.page = -1;
  if (!p.valid) return p;
  p.blk = static_cast<int>(i % kBlocks);
  const uint32_t r = static_cast<uint32_t>(i / kBlocks);
  p.h = static_cast<int>(r / static_cast<uint32_t>(a.n));
  p.t = static_cast<int>(r - static_cast<uint32_t>(p.h) * a.n);
  const int pos = len - count + p.t;
  p.live = p.t < count && pos >= 0;
  if (!p.live) return p;
  const int page = a.table[b * a.table_stride + (pos >> a.page_shift)];
  if (static_cast<unsigned>(page) < static_cast<unsigned>(a.num_pages)) p.page = page;
  else checked_page(page, a.num_pages, a.status);   // (records it)
  p.row = pos & ((1 << a.page_shift) - 1);
  return p;
}

__device__ __forceinline__ int cache_len(const Fp4CopyArgs& a, int b) {
  return min(max(a.lens[b], 0), a.cap);
}

__device__ __forceinline__ int token_count(const Fp4CopyArgs& a, int b) {
  return a.counts == nullptr ? a.n : min(max(a.counts[b], 0), a.n);
}

// A block's codes and the code of its scale.
__device__ __forceinline__ uint2 quantised(const uint32_t* w, float descale, float inv6,
                                           uint32_t* scale) {
  uint64_t x[8];
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xffff0000u);
    top = max_nan(top, max_nan(fabsf(lo), fabsf(hi)));
    x[i] = f2_pack(lo, hi);
  }
  *scale = 0x7fu;   // NaN
  if (top != top) return make_uint2(0u, 0u);
  *scale = block_scale(top, descale, inv6);
  if (*scale == 0) return make_uint2(0u, 0u);
  const float unit = e4m3_value(*scale), inv = reciprocal(unit * descale);
  const uint64_t inv2 = f2_pack(inv, inv), below = f2_pack(kBelow, kBelow),
                 above = f2_pack(kAbove, kAbove);
  uint64_t low[8], high[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t t = f2_mul(x[i], inv2);
    low[i] = f2_mul(t, below);
    high[i] = f2_mul(t, above);
  }
  uint32_t codes[2] = {e2m1_of(low), e2m1_of(low + 4)};
  const uint32_t other[2] = {e2m1_of(high), e2m1_of(high + 4)};
  if (codes[0] != other[0] || codes[1] != other[1]) {   // a value next to a border
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int s = 4 * (i & 7);
      const uint32_t l = (codes[i >> 3] >> s) & 15u, g = (other[i >> 3] >> s) & 15u;
      if (l == g) continue;
      float lo, hi;
      f2_unpack(x[i >> 1], lo, hi);
      const uint32_t m = nearer(l & 7u, g & 7u, fabsf(i & 1 ? hi : lo), unit, descale,
                                [](uint32_t c) { return e2m1_value(c); });
      codes[i >> 3] = (codes[i >> 3] & ~(15u << s)) | ((l & 8u) | m) << s;
    }
  }
  return make_uint2(codes[0], codes[1]);
}

// N: blocks of a thread.
template <int D, int N>
__global__ void __launch_bounds__(kFp4Threads) fp4_store_kernel(const Fp4CopyArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const bool values = blockIdx.z != 0;
  const Fp4Cache& c = values ? a.cache.v : a.cache.k;
  const float descale = values ? a.cache.v_descale : a.cache.k_descale;
  const float inv6 = 1.f / (6.f * descale);
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    const int len = cache_len(a, b), count = token_count(a, b);
    Place p[N];
    uint4 w[N][2];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      p[k] = place<D>(a, b, (static_cast<int64_t>(blockIdx.x) * N + k) * kFp4Threads + threadIdx.x,
                      len, count);
      if (p[k].live) {
        const uint4* src = reinterpret_cast<const uint4*>(
            (values ? a.v : a.k) + b * a.stride_b + p[k].h * a.stride_h + p[k].t * a.stride_n +
            kFp4Block * p[k].blk);
        w[k][0] = __ldcs(src);
        w[k][1] = __ldcs(src + 1);
      }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if (p[k].page < 0) continue;
      const uint32_t x[8] = {w[k][0].x, w[k][0].y, w[k][0].z, w[k][0].w,
                             w[k][1].x, w[k][1].y, w[k][1].z, w[k][1].w};
      uint32_t scale;
      const uint2 codes = quantised(x, descale, inv6, &scale);
      *reinterpret_cast<uint2*>(c.codes + p[k].page * c.code_page + p[k].h * c.code_head +
                                p[k].row * (D / 2) + 8 * p[k].blk) = codes;
      c.scales[p[k].page * c.scale_page + p[k].h * c.scale_head + p[k].row * (D / kFp4Block) +
               p[k].blk] = static_cast<uint8_t>(scale);
    }
  }
}

template <int D, int N>
__global__ void __launch_bounds__(kFp4Threads) fp4_load_kernel(const Fp4CopyArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const bool values = blockIdx.z != 0;
  const Fp4Cache& c = values ? a.cache.v : a.cache.k;
  const float descale = values ? a.cache.v_descale : a.cache.k_descale;
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    const int len = cache_len(a, b), count = token_count(a, b);
    Place p[N];
    uint2 codes[N];
    uint32_t scale[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      p[k] = place<D>(a, b, (static_cast<int64_t>(blockIdx.x) * N + k) * kFp4Threads + threadIdx.x,
                      len, count);
      codes[k] = make_uint2(0u, 0u);
      scale[k] = 0;
      if (p[k].page >= 0) {
        codes[k] = __ldcs(reinterpret_cast<const uint2*>(
            c.codes + p[k].page * c.code_page + p[k].h * c.code_head + p[k].row * (D / 2) +
            8 * p[k].blk));
        scale[k] = c.scales[p[k].page * c.scale_page + p[k].h * c.scale_head +
                            p[k].row * (D / kFp4Block) + p[k].blk];
      }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if (!p[k].valid) continue;
      // (two roundings of 2^-24 before the one to bf16)
      const float unit = e4m3_value(scale[k]) * descale;
      const uint64_t unit2 = f2_pack(unit, unit);
      uint32_t h[8], out[8];
      e2m1_to_half(codes[k].x, h);
      e2m1_to_half(codes[k].y, h + 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        float lo, hi;
        f2_unpack(f2_mul(f2_pack(x.x, x.y), unit2), lo, hi);
        out[i] = pack_bf16x2(lo, hi);
      }
      uint4* dst = reinterpret_cast<uint4*>((values ? a.v : a.k) + b * a.stride_b +
                                            p[k].h * a.stride_h + p[k].t * a.stride_n +
                                            kFp4Block * p[k].blk);
      __stcs(dst, make_uint4(out[0], out[1], out[2], out[3]));
      __stcs(dst + 1, make_uint4(out[4], out[5], out[6], out[7]));
    }
  }
}

// Four blocks a thread where that leaves enough CTAs: their loads are on the way
// together.
constexpr int kFp4Many = 4;

int64_t items_of(const Fp4CopyArgs& a) {
  return static_cast<int64_t>(a.H) * a.n * (a.d / kFp4Block);
}

bool many(const Fp4CopyArgs& a) { return items_of(a) * a.B >= kFp4Many * kFp4Threads * 512ll; }

dim3 copy_grid(const Fp4CopyArgs& a) {
  const int64_t per = (many(a) ? kFp4Many : 1) * kFp4Threads;
  return dim3(static_cast<unsigned>((items_of(a) + per - 1) / per),
              static_cast<unsigned>(a.B < 65535 ? a.B : 65535), 2);
}

}  // namespace

cudaError_t launch_fp4_store(const Fp4CopyArgs& a, cudaStream_t s) {
  auto kernel = many(a) ? (a.d == 64 ? fp4_store_kernel<64, kFp4Many> : fp4_store_kernel<128, kFp4Many>)
                        : (a.d == 64 ? fp4_store_kernel<64, 1> : fp4_store_kernel<128, 1>);
  return launch_pdl(kernel, copy_grid(a), dim3(kFp4Threads), 0, s, a);
}

cudaError_t launch_fp4_load(const Fp4CopyArgs& a, cudaStream_t s) {
  auto kernel = many(a) ? (a.d == 64 ? fp4_load_kernel<64, kFp4Many> : fp4_load_kernel<128, kFp4Many>)
                        : (a.d == 64 ? fp4_load_kernel<64, 1> : fp4_load_kernel<128, 1>);
  return launch_pdl(kernel, copy_grid(a), dim3(kFp4Threads), 0, s, a);
}

}  // namespace attn
