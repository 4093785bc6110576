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

__device__ __forceinline__ uint32_t e2m1_pair(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 x;\n\t.reg .b16 y;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 x, %1, %2;\n\t"
      "mov.b16 y, {x, 0};\n\t"
      "cvt.u32.u16 %0, y;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r & 0xffu;
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

// One thread's block: which one, or none.
struct Place {
  int b, h, t, blk;
  int page, row;       // where the token lies; page < 0: nowhere
  bool valid, live;    // there is such a block; the sequence has such a token
};

template <int D>
__device__ __forceinline__ Place place(const Fp4CopyArgs& a, int b, bool report) {
  constexpr int kBlocks = D / kFp4Block;
  Place p{};
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kFp4Threads + threadIdx.x;
  p.valid = i < static_cast<int64_t>(a.H) * a.n * kBlocks;
  if (!p.valid) return p;
  p.b = b;
  p.blk = static_cast<int>(i % kBlocks);
  const uint32_t r = static_cast<uint32_t>(i / kBlocks);
  p.h = static_cast<int>(r / static_cast<uint32_t>(a.n));
  p.t = static_cast<int>(r - static_cast<uint32_t>(p.h) * a.n);
  const int len = min(max(a.lens[b], 0), a.cap);
  const int count = a.counts == nullptr ? a.n : min(max(a.counts[b], 0), a.n);
  const int pos = len - count + p.t;
  p.live = p.t < count && pos >= 0;
  p.page = -1;
  if (!p.live) return p;
  const int page = a.table[b * a.table_stride + (pos >> a.page_shift)];
  if (static_cast<unsigned>(page) < static_cast<unsigned>(a.num_pages)) p.page = page;
  else if (report) checked_page(page, a.num_pages, a.status);
  p.row = pos & ((1 << a.page_shift) - 1);
  return p;
}

template <int D>
__global__ void __launch_bounds__(kFp4Threads) fp4_store_kernel(const Fp4CopyArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const bool values = blockIdx.z != 0;
  const Fp4Cache& c = values ? a.cache.v : a.cache.k;
  const float descale = values ? a.cache.v_descale : a.cache.k_descale;
  const float inv6 = 1.f / (6.f * descale);
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    const Place p = place<D>(a, b, true);
    if (!p.valid || !p.live || p.page < 0) continue;
    const uint4* src = reinterpret_cast<const uint4*>(
        (values ? a.v : a.k) + p.b * a.stride_b + p.h * a.stride_h + p.t * a.stride_n +
        kFp4Block * p.blk);
    const uint4 w0 = __ldcs(src), w1 = __ldcs(src + 1);
    const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
    float x[16], top = 0.f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      nan = nan || x[2 * i] != x[2 * i] || x[2 * i + 1] != x[2 * i + 1];
      top = fmaxf(top, fmaxf(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
    }
    uint32_t scale = 0x7fu;   // NaN
    uint64_t codes = 0;
    if (!nan) {
      scale = block_scale(top, descale, inv6);
      if (scale != 0) {
        const float unit = e4m3_value(scale), inv = 1.f / (unit * descale);
        uint64_t low = 0, high = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float t0 = x[2 * i] * inv, t1 = x[2 * i + 1] * inv;
          low |= static_cast<uint64_t>(e2m1_pair(t0 * kBelow, t1 * kBelow)) << (8 * i);
          high |= static_cast<uint64_t>(e2m1_pair(t0 * kAbove, t1 * kAbove)) << (8 * i);
        }
        if (low != high) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint32_t l = (low >> (4 * i)) & 15u, g = (high >> (4 * i)) & 15u;
            if (l == g) continue;
            const uint64_t at = static_cast<uint64_t>(15) << (4 * i);
            const uint32_t m = nearer(l & 7u, g & 7u, fabsf(x[i]), unit, descale,
                                      [](uint32_t c) { return e2m1_value(c); });
            low = (low & ~at) | static_cast<uint64_t>((l & 8u) | m) << (4 * i);
          }
        }
        codes = low;
      }
    }
    *reinterpret_cast<uint64_t*>(c.codes + p.page * c.code_page + p.h * c.code_head +
                                 p.row * (D / 2) + 8 * p.blk) = codes;
    c.scales[p.page * c.scale_page + p.h * c.scale_head + p.row * (D / kFp4Block) + p.blk] =
        static_cast<uint8_t>(scale);
  }
}

template <int D>
__global__ void __launch_bounds__(kFp4Threads) fp4_load_kernel(const Fp4CopyArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const bool values = blockIdx.z != 0;
  const Fp4Cache& c = values ? a.cache.v : a.cache.k;
  const float descale = values ? a.cache.v_descale : a.cache.k_descale;
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    const Place p = place<D>(a, b, true);
    if (!p.valid) continue;
    uint32_t out[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (p.page >= 0) {
      const uint2 codes = __ldcs(reinterpret_cast<const uint2*>(
          c.codes + p.page * c.code_page + p.h * c.code_head + p.row * (D / 2) + 8 * p.blk));
      const float unit =
          e4m3_value(c.scales[p.page * c.scale_page + p.h * c.scale_head +
                              p.row * (D / kFp4Block) + p.blk]);
      uint32_t h[8];
      e2m1_to_half(codes.x, h);
      e2m1_to_half(codes.y, h + 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) {   // s * c is exact, so this rounds in fp32 and to bf16
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        out[i] = pack_bf16x2(x.x * unit * descale, x.y * unit * descale);
      }
    }
    uint4* dst = reinterpret_cast<uint4*>((values ? a.v : a.k) + p.b * a.stride_b +
                                          p.h * a.stride_h + p.t * a.stride_n +
                                          kFp4Block * p.blk);
    __stcs(dst, make_uint4(out[0], out[1], out[2], out[3]));
    __stcs(dst + 1, make_uint4(out[4], out[5], out[6], out[7]));
  }
}

dim3 copy_grid(const Fp4CopyArgs& a) {
  const int64_t items = static_cast<int64_t>(a.H) * a.n * (a.d / kFp4Block);
  return dim3(static_cast<unsigned>((items + kFp4Threads - 1) / kFp4Threads),
              static_cast<unsigned>(a.B < 65535 ? a.B : 65535), 2);
}

}  // namespace

cudaError_t launch_fp4_store(const Fp4CopyArgs& a, cudaStream_t s) {
  return launch_pdl(a.d == 64 ? fp4_store_kernel<64> : fp4_store_kernel<128>, copy_grid(a),
                    dim3(kFp4Threads), 0, s, a);
}

cudaError_t launch_fp4_load(const Fp4CopyArgs& a, cudaStream_t s) {
  return launch_pdl(a.d == 64 ? fp4_load_kernel<64> : fp4_load_kernel<128>, copy_grid(a),
                    dim3(kFp4Threads), 0, s, a);
}

}  // namespace attn
