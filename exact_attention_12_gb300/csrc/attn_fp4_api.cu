// Host side of the calls on caches in 4 bits (attn_pages_store_fp4,
// attn_pages_load_fp4, attn_decode_fp4) and of attn_key_weights: argument checks,
// workspace layout, launches.
#include <algorithm>
#include <cmath>
#include <cstdio>

#include "attn.h"
#include "attn_fp4.cuh"

namespace {

using attn::PagedArgs;

constexpr size_t kHeaderBytes = 256;
constexpr uint64_t kTimeoutNs = 2000000000ull;

attn_status fail(attn_status s, const char* msg) {
  return static_cast<attn_status>(attn::record_error(s, msg));
}

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    sms = 148;
  return sms;
}

int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

int kv_heads(const attn_params* p) { return p->H_kv == 0 ? p->H : p->H_kv; }

bool good_strides(std::initializer_list<int64_t> strides, int d) {
  int64_t last = 0;
  for (int64_t s : strides) {
    if (s <= 0 || s % 8 != 0) return false;
    last = s;
  }
  return last >= d;   // the row stride comes last
}

attn_status check_pages(const attn_params* p, const attn_pages* g) {
  if (p == nullptr || g == nullptr) return fail(ATTN_ERR_INVALID_ARG, "params or pages is NULL");
  if (p->B < 0 || p->H < 0 || p->N < 0 || p->H_kv < 0)
    return fail(ATTN_ERR_INVALID_ARG, "negative shape");
  if (p->reserved != 0 || p->reserved2 != 0)
    return fail(ATTN_ERR_INVALID_ARG, "reserved field must be 0");
  if (p->d != 64 && p->d != 128) return fail(ATTN_ERR_UNSUPPORTED, "d must be 64 or 128");
  if (p->key_lens == nullptr && p->B > 0)
    return fail(ATTN_ERR_INVALID_ARG, "key_lens (cache lengths) is NULL");
  if (g->max_pages < 0 || g->num_pages < 0 || g->table_stride < g->max_pages)
    return fail(ATTN_ERR_INVALID_ARG, "pages: negative size, or table_stride < max_pages");
  if (g->page_size < 16 || g->page_size > 32768 || (g->page_size & (g->page_size - 1)) != 0)
    return fail(ATTN_ERR_INVALID_ARG, "page_size must be a power of two, 16 to 32768");
  const int64_t cap = static_cast<int64_t>(g->max_pages) * g->page_size;
  if (cap > (int64_t{1} << 30)) return fail(ATTN_ERR_UNSUPPORTED, "more than 2^30 keys per row");
  if (cap > 0 && p->B > 0 && g->table == nullptr)
    return fail(ATTN_ERR_INVALID_ARG, "page table is NULL");
  if (g->shared_len != 0) return fail(ATTN_ERR_UNSUPPORTED, "shared_len must be 0 here");
  return ATTN_OK;
}

// A cache in 4 bits; one of no pages or heads may be anywhere.
attn_status check_cache(const attn_fp4* c, int heads, int num_pages) {
  if (c == nullptr) return fail(ATTN_ERR_INVALID_ARG, "cache is NULL");
  if (c->reserved != 0) return fail(ATTN_ERR_INVALID_ARG, "cache: reserved field must be 0");
  if (!(c->descale >= 0x1p-100f && c->descale <= 0x1p100f))
    return fail(ATTN_ERR_INVALID_ARG, "cache: descale must be between 2^-100 and 2^100");
  const void* ptrs[2] = {c->codes, c->scales};
  for (const void* ptr : ptrs)
    if ((num_pages > 0 && heads > 0 && ptr == nullptr) || (reinterpret_cast<uintptr_t>(ptr) & 15u) != 0)
      return fail(ATTN_ERR_INVALID_ARG, "cache: codes and scales must be 16-byte aligned");
  const int64_t steps[4] = {c->code_page, c->code_head, c->scale_page, c->scale_head};
  for (int64_t s : steps)
    if (s <= 0 || s % 16 != 0)
      return fail(ATTN_ERR_INVALID_ARG, "cache: strides must be positive multiples of 16 bytes");
  if (c->code_page >> 32 != 0 || c->scale_page >> 32 != 0)
    return fail(ATTN_ERR_UNSUPPORTED, "cache: pages must be less than 2^32 bytes apart");
  return ATTN_OK;
}

// (what is written to)
attn_status check_apart(const attn_fp4* c, const attn_params* p, const attn_pages* g) {
  const int64_t row = static_cast<int64_t>(g->page_size) * p->d;
  if (attn::apart({{g->num_pages, c->code_page}, {p->H_kv, c->code_head}}, row / 2) &&
      attn::apart({{g->num_pages, c->scale_page}, {p->H_kv, c->scale_head}}, row / attn::kFp4Block))
    return ATTN_OK;
  return fail(ATTN_ERR_INVALID_ARG, "cache: heads and pages must lie apart");
}

attn::Fp4Cache cache_of(const attn_fp4* c) {
  return attn::Fp4Cache{static_cast<uint8_t*>(c->codes), static_cast<uint8_t*>(c->scales),
                        c->code_page, c->code_head, c->scale_page, c->scale_head};
}

attn_status check_ptrs(std::initializer_list<const void*> ptrs, uintptr_t align) {
  for (const void* ptr : ptrs) {
    if (ptr == nullptr) return fail(ATTN_ERR_INVALID_ARG, "tensor argument is NULL");
    if ((reinterpret_cast<uintptr_t>(ptr) & (align - 1)) != 0)
      return fail(ATTN_ERR_INVALID_ARG, "tensor argument is misaligned");
  }
  return ATTN_OK;
}

attn_status check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (ws == nullptr) return fail(ATTN_ERR_WORKSPACE, "workspace is NULL");
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
    return fail(ATTN_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (ws_bytes < need) {
    char msg[96];
    snprintf(msg, sizeof(msg), "workspace too small: %zu < %zu bytes", ws_bytes, need);
    return fail(ATTN_ERR_WORKSPACE, msg);
  }
  return ATTN_OK;
}

attn_status launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return ATTN_OK;
  char msg[256];
  snprintf(msg, sizeof(msg), "%s: %s", what, cudaGetErrorString(e));
  return fail(ATTN_ERR_CUDA, msg);
}

// ---------------------------------------------------- steps with query rows --

attn_status check_step(const attn_params* p, int32_t n_q, const attn_pages* g, int keys,
                       int overhead, int max_rows) {
  attn_status st = check_pages(p, g);
  if (st != ATTN_OK) return st;
  if (p->dtype != ATTN_BF16)
    return fail(p->dtype == ATTN_FP32 || p->dtype == ATTN_FP8_E4M3 ? ATTN_ERR_UNSUPPORTED
                                                                   : ATTN_ERR_INVALID_ARG,
                "queries must be bf16");
  if (!std::isfinite(p->scale) || !(p->scale > 0.f))
    return fail(ATTN_ERR_INVALID_ARG, "scale must be positive and finite");
  if (p->dropout_p != 0.f || p->block_mask != nullptr)
    return fail(ATTN_ERR_UNSUPPORTED, "decode takes no dropout and no block mask");
  if (n_q < 1) return fail(ATTN_ERR_INVALID_ARG, "n_q must be >= 1");
  const int H_kv = kv_heads(p);
  if (p->H > 0 && (H_kv < 1 || p->H % H_kv != 0))
    return fail(ATTN_ERR_INVALID_ARG, "H_kv must divide H");
  if (static_cast<int64_t>(p->H) * n_q > 32768 ||
      static_cast<int64_t>(p->B) * p->H * n_q > (1 << 30))
    return fail(ATTN_ERR_UNSUPPORTED, "more than 32768 query rows per sequence or 2^30 in all");
  const int64_t cap = static_cast<int64_t>(g->max_pages) * g->page_size;
  if (cap != p->N) return fail(ATTN_ERR_INVALID_ARG, "N must be max_pages * page_size");
  const int64_t blocks =
      H_kv > 0 ? (static_cast<int64_t>(p->H / H_kv) * n_q + max_rows - 1) / max_rows * H_kv : 0;
  if (p->B * blocks * (cap / keys + overhead + 1) >= (int64_t{1} << 31))
    return fail(ATTN_ERR_UNSUPPORTED,
                "B * H_kv * N / 32 (times H / H_kv * n_q / 64) must stay below 2^31");
  if (!good_strides({p->stride_b, p->stride_h, p->stride_n}, p->d))
    return fail(ATTN_ERR_INVALID_ARG, "strides must be positive multiples of 8, stride_n >= d");
  return ATTN_OK;
}

bool empty(const attn_params* p) { return p->B == 0 || p->H == 0; }

struct Layout {
  size_t notes = 0, part_o = 0, part_l = 0, total = 0;
  int ctas = 0, n_notes = 0;
  bool by_segment = false, tiled = false;
  int cluster = 0;   // CTAs of a segment's cluster; 0: the balanced split; -1: a warp a segment
  int heads = 0, blocks = 1, rows = 0, head_rows = 0;
};

Layout decode_layout(const attn_params* p, int32_t n_q, const attn_pages* g) {
  Layout L;
  const int64_t sms = sm_count();
  const int H_kv = kv_heads(p);
  L.head_rows = H_kv > 0 ? p->H / H_kv * n_q : n_q;
  L.blocks = (L.head_rows + attn::kDecMaxRows - 1) / attn::kDecMaxRows;
  L.rows = L.blocks > 0 ? (L.head_rows + L.blocks - 1) / L.blocks : 0;
  L.heads = H_kv * L.blocks;
  int64_t most = attn::fp4_ctas_per_sm(L.rows) * sms;   // CTAs at a time
  const int64_t tiles = (static_cast<int64_t>(p->N) + attn::kFp4Keys - 1) / attn::kFp4Keys;
  const int64_t segments = static_cast<int64_t>(p->B) * L.heads;
  // Short caches need no balance: a cluster per segment, of as many CTAs as the GPU
  // holds at once and as have a tile for each of their warps, if that leaves each
  // few tiles; a warp per segment where there are more segments than that.
  int c = tiles < attn::kFp4ClusterFrom ? 1 : 8;
  while (c > 1 && (4 * segments * c > 3 * most || 2 * c > tiles)) c /= 2;
  if (segments > most) {
    if (L.rows <= 32 && tiles <= attn::kFp4SoloTiles) L.cluster = -1;
    else if (tiles <= attn::kFp4ManyTiles) L.cluster = 1;
  } else if (tiles <= c * attn::fp4_cluster_tiles(L.rows)) {
    L.cluster = c;
  }
  // the balanced split: CTAs that have the smallest share worth one at full caches
  int64_t want = segments * (tiles + attn::fp4_overhead(L.rows)) / attn::kFp4MinUnits;
  L.tiled = L.cluster == 0 && attn::fp4_in_tiles(L.rows, p->d);
  if (L.tiled) {
    most = sms;
    want = segments * ((static_cast<int64_t>(p->N) + attn::kTile - 1) / attn::kTile +
                       attn::kFp4TileOverhead) / attn::kFp4TileMinUnits;
  }
  L.ctas = static_cast<int>(most < want ? most : want);
  if (L.ctas < 1) L.ctas = 1;
  L.by_segment = segments <= L.ctas;
  L.n_notes = L.by_segment ? static_cast<int>(segments) : L.ctas;
  size_t off = kHeaderBytes;
  L.notes = off;
  off = round_up(off + static_cast<size_t>(L.n_notes) * sizeof(attn::MergeNote), 256);
  L.part_o = off;
  off = round_up(off + 2 * static_cast<size_t>(L.ctas) * L.rows * p->d * sizeof(float), 256);
  L.part_l = off;
  off = round_up(off + 2 * static_cast<size_t>(L.ctas) * L.rows * sizeof(float), 256);
  L.total = off;
  return L;
}

PagedArgs args_of(const attn_params* p, int32_t n_q, const attn_pages* g, const void* q, void* ws) {
  PagedArgs a{};
  a.B = p->B;
  a.H = p->H;
  a.heads = kv_heads(p);
  a.blocks = 1;
  a.n_q = n_q;
  a.head_rows = a.rows = p->H / kv_heads(p) * n_q;
  a.all_rows = p->H * n_q;
  a.causal = p->causal != 0;
  a.d = p->d;
  a.key_lens = p->key_lens;
  a.table = g->table;
  a.table_stride = g->table_stride;
  a.cap = p->N;
  a.page_shift = log2_of(g->page_size);
  a.num_pages = g->num_pages;
  a.scale = p->scale;
  a.scale_log2 = p->scale * attn::kLog2Of;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.stride_b = p->stride_b;
  a.stride_h = p->stride_h;
  a.stride_n = p->stride_n;
  a.status = static_cast<int*>(ws);
  return a;
}

// ------------------------------------------------------------ store and load --

attn_status copy(const attn_params* p, const attn_pages* g, const int32_t* counts, const void* k,
                 const void* v, const attn_fp4* kc, const attn_fp4* vc, void* ws, size_t ws_bytes,
                 void* stream, bool store) {
  attn_status st = check_pages(p, g);
  if (st != ATTN_OK || (st = check_cache(kc, p->H_kv, g->num_pages)) != ATTN_OK ||
      (st = check_cache(vc, p->H_kv, g->num_pages)) != ATTN_OK)
    return st;
  if (store && ((st = check_apart(kc, p, g)) != ATTN_OK || (st = check_apart(vc, p, g)) != ATTN_OK))
    return st;
  if (p->N > (1 << 30)) return fail(ATTN_ERR_UNSUPPORTED, "more than 2^30 tokens");
  if (!good_strides({p->kv_stride_b, p->kv_stride_h, p->kv_stride_n}, p->d))
    return fail(ATTN_ERR_INVALID_ARG, "kv strides must be positive multiples of 8, the last >= d");
  if ((st = check_ws(ws, ws_bytes, kHeaderBytes)) != ATTN_OK) return st;
  if (p->B == 0 || p->H_kv == 0 || p->N == 0) return ATTN_OK;
  if ((st = check_ptrs({k, v}, 16)) != ATTN_OK) return st;
  attn::Fp4CopyArgs a{};
  a.B = p->B;
  a.H = p->H_kv;
  a.n = p->N;
  a.d = p->d;
  a.lens = p->key_lens;
  a.counts = counts;
  a.table = g->table;
  a.table_stride = g->table_stride;
  a.cap = g->max_pages * g->page_size;
  a.page_shift = log2_of(g->page_size);
  a.num_pages = g->num_pages;
  a.k = static_cast<__nv_bfloat16*>(const_cast<void*>(k));
  a.v = static_cast<__nv_bfloat16*>(const_cast<void*>(v));
  a.stride_b = p->kv_stride_b;
  a.stride_h = p->kv_stride_h;
  a.stride_n = p->kv_stride_n;
  a.cache = attn::Fp4Args{cache_of(kc), cache_of(vc), kc->descale, vc->descale};
  a.status = static_cast<int*>(ws);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launched(store ? attn::launch_fp4_store(a, s) : attn::launch_fp4_load(a, s),
                  store ? "store launch" : "load launch");
}

}  // namespace

namespace attn {

bool apart(std::initializer_list<Axis> axes, int64_t extent) {
  Axis live[kMaxAxes];
  int n = 0;
  for (const Axis& x : axes)
    if (x.size > 1 && n < kMaxAxes) live[n++] = x;
  std::sort(live, live + n, [](const Axis& x, const Axis& y) { return x.stride < y.stride; });
  __int128 span = extent;
  for (int i = 0; i < n; ++i) {
    if (live[i].stride < span) return false;
    span += static_cast<__int128>(live[i].size - 1) * live[i].stride;
  }
  return true;
}

}  // namespace attn

extern "C" {

attn_status attn_pages_store_fp4(const attn_params* p, const attn_pages* pages,
                                 const int32_t* counts, const void* k, const void* v,
                                 const attn_fp4* k_cache, const attn_fp4* v_cache, void* ws,
                                 size_t ws_bytes, void* stream) {
  return copy(p, pages, counts, k, v, k_cache, v_cache, ws, ws_bytes, stream, true);
}

attn_status attn_pages_load_fp4(const attn_params* p, const attn_pages* pages,
                                const int32_t* counts, const attn_fp4* k_cache,
                                const attn_fp4* v_cache, void* k, void* v, void* ws,
                                size_t ws_bytes, void* stream) {
  return copy(p, pages, counts, k, v, k_cache, v_cache, ws, ws_bytes, stream, false);
}

size_t attn_decode_fp4_workspace_size(const attn_params* p, int32_t n_q, const attn_pages* pages) {
  if (check_step(p, n_q, pages, attn::kFp4Keys, attn::fp4_overhead(attn::kDecMaxRows),
                 attn::kDecMaxRows) != ATTN_OK)
    return 0;
  return decode_layout(p, n_q, pages).total;
}

attn_status attn_decode_fp4(const attn_params* p, int32_t n_q, const attn_pages* pages,
                            const void* q, const attn_fp4* k, const attn_fp4* v, void* o,
                            float* lse, void* ws, size_t ws_bytes, void* stream) {
  attn_status st =
      check_step(p, n_q, pages, attn::kFp4Keys, attn::fp4_overhead(attn::kDecMaxRows),
                 attn::kDecMaxRows);
  if (st != ATTN_OK || (st = check_cache(k, kv_heads(p), pages->num_pages)) != ATTN_OK ||
      (st = check_cache(v, kv_heads(p), pages->num_pages)) != ATTN_OK)
    return st;
  const Layout L = decode_layout(p, n_q, pages);
  if ((st = check_ws(ws, ws_bytes, L.total)) != ATTN_OK) return st;
  if (empty(p)) return ATTN_OK;
  if ((st = check_ptrs({q, o}, 16)) != ATTN_OK || (st = check_ptrs({lse}, 4)) != ATTN_OK) return st;
  char* w = static_cast<char*>(ws);
  PagedArgs a = args_of(p, n_q, pages, q, ws);
  a.heads = L.heads;
  a.blocks = L.blocks;
  a.rows = L.rows;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.notes = reinterpret_cast<attn::MergeNote*>(w + L.notes);
  a.by_segment = L.by_segment;
  a.part_o = reinterpret_cast<float*>(w + L.part_o);
  a.part_l = reinterpret_cast<float*>(w + L.part_l);
  a.ctas = L.ctas;
  a.cluster = L.cluster;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  attn::Fp4Args f{cache_of(k), cache_of(v), k->descale, v->descale};
  if (pages->num_pages == 0)   // no cache to point at, and none is read
    f.k.codes = f.k.scales = f.v.codes = f.v.scales =
        static_cast<uint8_t*>(const_cast<void*>(q));
  if (L.tiled) {
    a.timeout_ns = kTimeoutNs;
    a.stall = attn::take_stall(attn::kStallFp4Values, &a.timeout_ns);
  }
  if ((st = launched(L.tiled ? attn::launch_fp4_tile(a, f, L.ctas, s)
                             : attn::launch_fp4_decode(a, f, L.ctas, s),
                     "4-bit decode launch")) != ATTN_OK)
    return st;
  if (L.cluster != 0 || L.ctas == 1) return ATTN_OK;   // merged already; one CTA cuts nothing
  return launched(attn::launch_paged_merge(a, L.n_notes, L.ctas, s), "4-bit decode merge launch");
}

attn_status attn_key_weights(const attn_params* p, int32_t n_q, const attn_pages* pages,
                             const void* q, const void* k, const attn_fp4* k_cache,
                             const float* lse, float* weights, int64_t weight_stride_b,
                             int64_t weight_stride_h, int32_t add, void* ws, size_t ws_bytes,
                             void* stream) {
  // (a segment takes all its rows, in one piece)
  attn_status st = check_step(p, n_q, pages, attn::kWeightKeys, attn::kWeightOverhead, 32768);
  if (st != ATTN_OK) return st;
  if (k_cache != nullptr) {
    if (k != nullptr) return fail(ATTN_ERR_INVALID_ARG, "give k or k_cache, not both");
    if ((st = check_cache(k_cache, kv_heads(p), pages->num_pages)) != ATTN_OK) return st;
  } else if (!good_strides({p->kv_stride_b, p->kv_stride_h, p->kv_stride_n}, p->d)) {
    return fail(ATTN_ERR_INVALID_ARG, "kv strides must be positive multiples of 8, the last >= d");
  }
  if (weight_stride_b < 0 || weight_stride_h < 0 ||
      !attn::apart({{p->B, weight_stride_b}, {kv_heads(p), weight_stride_h}}, p->N))
    return fail(ATTN_ERR_INVALID_ARG, "weights: the N entries of sequences and heads must lie apart");
  if ((st = check_ws(ws, ws_bytes, kHeaderBytes)) != ATTN_OK) return st;
  if (empty(p) || p->N == 0) return ATTN_OK;
  if (k_cache == nullptr && pages->num_pages == 0) k = q;   // no cache to point at
  if ((st = check_ptrs({q, k_cache != nullptr ? q : k}, 16)) != ATTN_OK ||
      (st = check_ptrs({lse, weights}, 4)) != ATTN_OK)
    return st;
  const PagedArgs a = args_of(p, n_q, pages, q, ws);
  attn::WeightArgs f{};
  if (k_cache != nullptr) {
    f.cache = cache_of(k_cache);
    f.k_descale = k_cache->descale;
  } else {
    f.k = static_cast<const __nv_bfloat16*>(k);
    f.stride_page = p->kv_stride_b;
    f.stride_head = p->kv_stride_h;
    f.stride_row = p->kv_stride_n;
  }
  f.lse = lse;
  f.weights = weights;
  f.stride_b = weight_stride_b;
  f.stride_h = weight_stride_h;
  f.add = add != 0;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool many = a.head_rows > attn::kWeightTileRows;
  const int keys = many ? attn::kTile : attn::kWeightKeys;
  const int overhead = many ? attn::kWeightTileOverhead : attn::kWeightOverhead;
  const int64_t tiles = (static_cast<int64_t>(p->N) + keys - 1) / keys;
  const int64_t want = static_cast<int64_t>(a.B) * a.heads * (tiles + overhead) /
                       (many ? 1 : attn::kWeightMinUnits);
  const int64_t most = (many ? 1 : 2) * sm_count();
  const int ctas = static_cast<int>(want < 1 ? 1 : (want < most ? want : most));
  if (!many) return launched(attn::launch_key_weights(a, f, ctas, s), "key weights launch");
  CUtensorMap tk{};
  if (k_cache == nullptr) {
    st = static_cast<attn_status>(attn::encode_pages(
        &tk, k, pages->num_pages < 1 ? 1 : pages->num_pages, kv_heads(p), pages->page_size, p->d,
        p->kv_stride_b, p->kv_stride_h, p->kv_stride_n,
        pages->page_size < attn::kTile ? pages->page_size : attn::kTile));
    if (st != ATTN_OK) return st;
  }
  PagedArgs b = a;
  b.timeout_ns = kTimeoutNs;
  f.stall = attn::take_stall(attn::kStallWeightsSum, &b.timeout_ns);
  return launched(attn::launch_key_weights_tile(tk, b, f, ctas, s), "key weights launch");
}

}  // extern "C"
