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
// Bound: HBM, 2.56 bytes an element.  A thread takes 8 columns, 16 bytes in and 4
// out, so that each access of a warp is one run of bytes; two lanes share a
// scale.
// Measured: 8 prompts of 1000-8192 tokens, 8 heads, d = 128: the store, 140 MB read and 39
// written, 51 us (at the copy rate 26; its instructions take 70 % of the issue slots);
// the load, 39 MB read and 268 written, 41 us, which L2 has a part in.  64 tokens: 2.6
// us each.
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

__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b) {   // of bf16 pairs
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
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

__device__ __forceinline__ int cache_len(const Fp4CopyArgs& a, int b) {
  return min(max(a.lens[b], 0), a.cap);
}

__device__ __forceinline__ int token_count(const Fp4CopyArgs& a, int b) {
  return a.counts == nullptr ? a.n : min(max(a.counts[b], 0), a.n);
}

// A CTA takes 2^tile_shift tokens of a sequence, one thread 8 columns of one token,
// of every (kRows >> tile_shift)-th head; kRows rows at once.
template <int D>
struct Lanes {
  static constexpr int kParts = D / 8, kRows = kFp4Threads / kParts;
  int t, h, step, part;   // token, first head, heads between, which 8 columns
  __device__ explicit Lanes(int tile_shift) {
    const int row = threadIdx.x / kParts;
    part = threadIdx.x % kParts;
    t = (blockIdx.x << tile_shift) + (row & ((1 << tile_shift) - 1));
    h = row >> tile_shift;
    step = kRows >> tile_shift;
  }
};

// The page of a token's position, -1 where the table names none.
__device__ __forceinline__ int token_page(const Fp4CopyArgs& a, int b, int pos) {
  const int page = a.table[b * a.table_stride + (pos >> a.page_shift)];
  if (static_cast<unsigned>(page) < static_cast<unsigned>(a.num_pages)) return page;
  checked_page(page, a.num_pages, a.status);   // (records it)
  return -1;
}

// The codes of 8 columns and the code of the scale that they share with the
// neighbouring lane's (which is here too).
__device__ __forceinline__ uint32_t quantised(const uint4& w, float descale, float inv6,
                                              uint32_t* scale) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
  // |x| of two columns at once, NaN above all
  uint32_t two = max_nan2(max_nan2(v[0] & 0x7fff7fffu, v[1] & 0x7fff7fffu),
                          max_nan2(v[2] & 0x7fff7fffu, v[3] & 0x7fff7fffu));
  two = max_nan2(two, __shfl_xor_sync(0xffffffffu, two, 1));
  const float top = max_nan(__uint_as_float(two << 16), __uint_as_float(two & 0xffff0000u));
  *scale = 0x7fu;   // NaN
  if (top != top) return 0u;
  *scale = block_scale(top, descale, inv6);
  if (*scale == 0) return 0u;
  const float unit = e4m3_value(*scale), inv = reciprocal(unit * descale);
  const uint64_t inv2 = f2_pack(inv, inv), below = f2_pack(kBelow, kBelow),
                 above = f2_pack(kAbove, kAbove);
  uint64_t low[4], high[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t t =
        f2_mul(f2_pack(__uint_as_float(v[i] << 16), __uint_as_float(v[i] & 0xffff0000u)), inv2);
    low[i] = f2_mul(t, below);
    high[i] = f2_mul(t, above);
  }
  uint32_t codes = e2m1_of(low);
  for (uint32_t differ = codes ^ e2m1_of(high); differ != 0;) {   // values next to a border
    const int i = (__ffs(differ) - 1) >> 2, s = 4 * i;
    const uint32_t l = (codes >> s) & 15u, g = l ^ ((differ >> s) & 15u);
    const uint32_t word = i & 4 ? (i & 2 ? v[3] : v[2]) : (i & 2 ? v[1] : v[0]);
    const float x = __uint_as_float((i & 1 ? word : word << 16) & 0x7fff0000u);
    const uint32_t m =
        nearer(l & 7u, g & 7u, x, unit, descale, [](uint32_t c) { return e2m1_value(c); });
    codes = (codes & ~(15u << s)) | ((l & 8u) | m) << s;
    differ &= ~(15u << s);
  }
  return codes;
}

// Heads whose loads are on the way together, 4 / 2 / 8: 8 prompts stored and loaded 92 /
// 100 / 92 us, 64 tokens 4.9 / 4.5 / 5.5.
constexpr int kAtOnce = 4;

template <int D>
__global__ void __launch_bounds__(kFp4Threads) fp4_store_kernel(const Fp4CopyArgs a, int tile_shift) {
  grid_dep_wait();
  grid_dep_launch();
  const bool values = blockIdx.z != 0;
  const Fp4Cache& c = values ? a.cache.v : a.cache.k;
  const float descale = values ? a.cache.v_descale : a.cache.k_descale;
  const float inv6 = 1.f / (6.f * descale);
  const Lanes<D> me(tile_shift);
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    const int count = token_count(a, b), pos = cache_len(a, b) - count + me.t;
    if (static_cast<int>(blockIdx.x) << tile_shift >= count) continue;
    const bool live = me.t < count && pos >= 0;
    const __nv_bfloat16* src =
        (values ? a.v : a.k) + b * a.stride_b + me.t * a.stride_n + 8 * me.part;
    const int row = pos & ((1 << a.page_shift) - 1);
    uint8_t *codes_to = nullptr, *scales_to = nullptr;
    for (int base = 0; base < a.H; base += kAtOnce * me.step) {   // (all lanes: two share a scale)
      uint4 w[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int h = base + me.h + k * me.step;
        w[k] = make_uint4(0u, 0u, 0u, 0u);
        if (live && h < a.H) w[k] = __ldcs(reinterpret_cast<const uint4*>(src + h * a.stride_h));
      }
      if (live && base == 0) {
        const int page = token_page(a, b, pos);
        if (page >= 0) {
          codes_to = c.codes + page * c.code_page + row * (D / 2) + 4 * me.part;
          scales_to = c.scales + page * c.scale_page + row * (D / kFp4Block) + me.part / 2;
        }
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int h = base + me.h + k * me.step;
        uint32_t scale;
        const uint32_t codes = quantised(w[k], descale, inv6, &scale);
        if (codes_to == nullptr || h >= a.H) continue;
        *reinterpret_cast<uint32_t*>(codes_to + h * c.code_head) = codes;
        if ((me.part & 1) == 0) scales_to[h * c.scale_head] = static_cast<uint8_t>(scale);
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kFp4Threads) fp4_load_kernel(const Fp4CopyArgs a, int tile_shift) {
  grid_dep_wait();
  grid_dep_launch();
  const bool values = blockIdx.z != 0;
  const Fp4Cache& c = values ? a.cache.v : a.cache.k;
  const float descale = values ? a.cache.v_descale : a.cache.k_descale;
  const Lanes<D> me(tile_shift);
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    const int count = token_count(a, b), pos = cache_len(a, b) - count + me.t;
    if (me.t >= a.n) continue;
    __nv_bfloat16* dst =
        (values ? a.v : a.k) + b * a.stride_b + me.t * a.stride_n + 8 * me.part;
    const int page = me.t < count && pos >= 0 ? token_page(a, b, pos) : -1;
    const int row = pos & ((1 << a.page_shift) - 1);
    const uint8_t* codes_at = c.codes + max(page, 0) * c.code_page + row * (D / 2) + 4 * me.part;
    const uint8_t* scales_at =
        c.scales + max(page, 0) * c.scale_page + row * (D / kFp4Block) + me.part / 2;
    for (int h0 = me.h; h0 < a.H; h0 += kAtOnce * me.step) {
      uint32_t codes[kAtOnce], scale[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int h = h0 + k * me.step;
        codes[k] = scale[k] = 0;
        if (page >= 0 && h < a.H) {
          codes[k] = __ldcs(reinterpret_cast<const uint32_t*>(codes_at + h * c.code_head));
          scale[k] = scales_at[h * c.scale_head];
        }
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int h = h0 + k * me.step;
        if (h >= a.H) break;
        // (two roundings of 2^-24 before the one to bf16)
        const float unit = e4m3_value(scale[k]) * descale;
        const uint64_t unit2 = f2_pack(unit, unit);
        uint32_t x[4], out[4];
        e2m1_to_half(codes[k], x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&x[i]));
          float lo, hi;
          f2_unpack(f2_mul(f2_pack(y.x, y.y), unit2), lo, hi);
          out[i] = pack_bf16x2(lo, hi);
        }
        __stcs(reinterpret_cast<uint4*>(dst + h * a.stride_h),
               make_uint4(out[0], out[1], out[2], out[3]));
      }
    }
  }
}

// Tokens of a CTA: as many as it has rows, fewer where there are fewer (its other
// rows then take other heads).
template <int D>
int tile_of(const Fp4CopyArgs& a) {
  int s = 0;
  while ((1 << s) < a.n && (2 << s) <= Lanes<D>::kRows) ++s;
  return s;
}

template <int D>
cudaError_t launch_copy(void (*kernel)(const Fp4CopyArgs, int), const Fp4CopyArgs& a,
                        cudaStream_t s) {
  const int shift = tile_of<D>(a);
  const dim3 grid(static_cast<unsigned>((a.n + (1 << shift) - 1) >> shift),
                  static_cast<unsigned>(a.B < 65535 ? a.B : 65535), 2);
  return launch_pdl(kernel, grid, dim3(kFp4Threads), 0, s, a, shift);
}

}  // namespace

cudaError_t launch_fp4_store(const Fp4CopyArgs& a, cudaStream_t s) {
  return a.d == 64 ? launch_copy<64>(fp4_store_kernel<64>, a, s)
                   : launch_copy<128>(fp4_store_kernel<128>, a, s);
}

cudaError_t launch_fp4_load(const Fp4CopyArgs& a, cudaStream_t s) {
  return a.d == 64 ? launch_copy<64>(fp4_load_kernel<64>, a, s)
                   : launch_copy<128>(fp4_load_kernel<128>, a, s);
}

}  // namespace attn
