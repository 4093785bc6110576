// Host side of the paged decode steps (attn_decode_paged, attn_decode_latent
// in include/attn.h): argument checks, workspace layout, launches.
#include <cmath>
#include <cstdio>

#include "attn.h"
#include "attn_paged.cuh"

namespace {

using attn::PagedArgs;

constexpr size_t kHeaderBytes = 256;
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr float kLog2e = 1.4426950408889634f;

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

attn_status validate(const attn_params* p, int32_t n_q, const attn_pages* g, bool latent) {
  if (p == nullptr || g == nullptr) return fail(ATTN_ERR_INVALID_ARG, "params or pages is NULL");
  if (p->B < 0 || p->H < 0 || p->N < 0) return fail(ATTN_ERR_INVALID_ARG, "negative shape");
  if (p->reserved != 0 || p->reserved2 != 0)
    return fail(ATTN_ERR_INVALID_ARG, "reserved field must be 0");
  if (p->dtype != ATTN_BF16)
    return fail(p->dtype == ATTN_FP32 || p->dtype == ATTN_FP8_E4M3 ? ATTN_ERR_UNSUPPORTED
                                                                   : ATTN_ERR_INVALID_ARG,
                "paged decode is implemented for bf16");
  if (latent ? (p->d != 256 && p->d != 512) : (p->d != 64 && p->d != 128))
    return fail(ATTN_ERR_UNSUPPORTED, latent ? "latent decode: d must be 256 or 512"
                                             : "paged decode: d must be 64 or 128");
  if (!std::isfinite(p->scale) || !(p->scale > 0.f))
    return fail(ATTN_ERR_INVALID_ARG, "scale must be positive and finite");
  if (p->dropout_p != 0.f || p->block_mask != nullptr)
    return fail(ATTN_ERR_UNSUPPORTED, "decode takes no dropout and no block mask");
  if (p->key_lens == nullptr && p->B > 0)
    return fail(ATTN_ERR_INVALID_ARG, "decode needs key_lens (cache lengths)");
  if (n_q < 1) return fail(ATTN_ERR_INVALID_ARG, "n_q must be >= 1");
  const int H_kv = latent ? 1 : (p->H_kv == 0 ? p->H : p->H_kv);
  if (latent ? (p->H_kv != 0 && p->H_kv != 1)
             : (p->H_kv < 0 || (p->H > 0 && (H_kv < 1 || p->H % H_kv != 0))))
    return fail(ATTN_ERR_INVALID_ARG, latent ? "latent decode: H_kv must be 0 or 1"
                                             : "H_kv must divide H");
  if (static_cast<int64_t>(p->H) * n_q > 32768 ||
      static_cast<int64_t>(p->B) * p->H * n_q > (1 << 30))
    return fail(ATTN_ERR_UNSUPPORTED, "more than 32768 query rows per sequence or 2^30 in all");
  // pages
  if (g->max_pages < 0 || g->num_pages < 0 || g->table_stride < g->max_pages)
    return fail(ATTN_ERR_INVALID_ARG, "pages: negative size, or table_stride < max_pages");
  if (g->page_size < 16 || g->page_size > 32768 || (g->page_size & (g->page_size - 1)) != 0)
    return fail(ATTN_ERR_INVALID_ARG, "page_size must be a power of two, 16 to 32768");
  const int64_t cap = static_cast<int64_t>(g->max_pages) * g->page_size;
  if (cap > (int64_t{1} << 30)) return fail(ATTN_ERR_UNSUPPORTED, "more than 2^30 keys per row");
  if (cap != p->N) return fail(ATTN_ERR_INVALID_ARG, "N must be max_pages * page_size");
  if (cap > 0 && p->B > 0 && g->table == nullptr)
    return fail(ATTN_ERR_INVALID_ARG, "page table is NULL");
  if (g->shared_len < 0 || g->shared_len > cap || g->shared_len % g->page_size != 0)
    return fail(ATTN_ERR_INVALID_ARG, "shared_len must be a multiple of page_size, at most N");
  const int64_t blocks = latent ? 1 : H_kv > 0 ? (static_cast<int64_t>(p->H / H_kv) * n_q + 63) / 64 * H_kv : 0;
  if (p->B * blocks * (cap / (latent ? attn::kLatentKeys : attn::kPagedKeys) +
                                    attn::kPagedOverhead + 1) >= (int64_t{1} << 31))
    return fail(ATTN_ERR_UNSUPPORTED, "B * H_kv * N / 32 (times H / H_kv * n_q / 64) must stay below 2^31");
  if (latent && g->shared_len != 0)
    return fail(ATTN_ERR_UNSUPPORTED, "latent decode takes no shared prefix");
  // strides
  const int cols = latent ? p->d + attn::kLatentRope : p->d;
  const int64_t st[6] = {p->stride_b,    p->stride_h, p->stride_n, p->kv_stride_b,
                         p->kv_stride_n, latent ? 8 : p->kv_stride_h};
  for (int64_t s : st)
    if (s <= 0 || s % 8 != 0)
      return fail(ATTN_ERR_INVALID_ARG, "strides must be positive multiples of 8 elements");
  if (p->kv_stride_n < cols || p->stride_n < cols)
    return fail(ATTN_ERR_INVALID_ARG, "rows overlap: stride_n is below the row's columns");
  return ATTN_OK;
}

attn_status check_ptrs(std::initializer_list<const void*> ptrs) {
  for (const void* ptr : ptrs) {
    if (ptr == nullptr) return fail(ATTN_ERR_INVALID_ARG, "tensor argument is NULL");
    if ((reinterpret_cast<uintptr_t>(ptr) & 15u) != 0)
      return fail(ATTN_ERR_INVALID_ARG, "tensor argument is not 16-byte aligned");
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

int kv_heads(const attn_params* p) { return p->H_kv == 0 ? p->H : p->H_kv; }

bool empty(const attn_params* p) { return p->B == 0 || p->H == 0; }

struct Layout {
  size_t notes = 0, part_o = 0, part_l = 0, pre_o = 0, pre_l = 0, total = 0;
  int ctas = 0;                            // of the decode kernel (latent: per row group)
  int n_notes = 0;                         // of merges: one per segment or per CTA
  bool by_segment = false;
  int cluster = 0;
  int heads = 0, blocks = 1, rows = 0;     // segments per sequence and key/value head, rows of one
  int head_rows = 0;                       // rows of a key/value head
  int first = 0, splits = 0, tiles = 0;    // the shared prefix
};

int64_t segments_of(const attn_params* p, const Layout& L) {
  return static_cast<int64_t>(p->B) * L.heads;
}

Layout layout(const attn_params* p, int32_t n_q, const attn_pages* g, bool latent) {
  Layout L;
  const int64_t sms = sm_count();
  const int64_t rows_all = static_cast<int64_t>(p->B) * p->H * n_q;
  const int H_kv = p->H_kv == 0 ? p->H : p->H_kv;
  int64_t most;   // CTAs that have the smallest share worth a CTA at full caches
  if (latent) {
    const int64_t groups = (static_cast<int64_t>(p->H) * n_q + attn::kLatentRows - 1) / attn::kLatentRows;
    L.heads = 1;
    L.head_rows = p->H * n_q;
    L.rows = static_cast<int>(groups * attn::kLatentRows);
    most = groups > 0 ? sms / groups : 1;
  } else {
    // more than 64 rows of a key/value head: in equal blocks, each of which
    // reads the keys
    L.head_rows = H_kv > 0 ? p->H / H_kv * n_q : n_q;
    L.blocks = (L.head_rows + attn::kDecMaxRows - 1) / attn::kDecMaxRows;
    L.rows = L.blocks > 0 ? (L.head_rows + L.blocks - 1) / L.blocks : 0;
    L.heads = H_kv * L.blocks;
    most = L.rows > 32 ? sms : 2 * sms;
    // the prefix apart: only where two sequences share it
    L.first = p->B > 1 ? g->shared_len : 0;
  }
  const int keys = latent ? attn::kLatentKeys : attn::kPagedKeys;
  const int64_t tiles = (static_cast<int64_t>(p->N) - L.first + keys - 1) / keys;
  const int64_t units = static_cast<int64_t>(p->B) * L.heads *
                        (tiles + (latent ? attn::kLatentOverhead : attn::kPagedOverhead));
  const int64_t want = units / (latent ? attn::kLatentMinUnits : attn::kPagedMinUnits);
  const int64_t room = most;
  if (most > want) most = want;
  L.ctas = static_cast<int>(most < 1 ? 1 : most);
  if (L.first > 0) {
    // pieces of the prefix: as many as fill the SMs once, two key tiles each
    // at least, 16 at most
    L.tiles = (L.first + attn::kTile - 1) / attn::kTile;
    const int64_t stack = static_cast<int64_t>(p->B) * L.head_rows;
    const int64_t units2 = (stack + 2 * attn::kTile - 1) / (2 * attn::kTile) * H_kv;
    int64_t k = units2 > 0 ? sms / units2 : 1;
    if (k > L.tiles / 2) k = L.tiles / 2;
    if (k > 16) k = 16;
    L.splits = k < 1 ? 1 : static_cast<int>(k);
  }
  // short caches: a cluster per segment, of as many CTAs as the GPU holds at
  // once and as have a tile for each slot (latent: a tile), if that leaves each
  // few tiles; a slot of a CTA per segment where more find no place
  const int64_t segments = segments_of(p, L);
  {
    int c = 8;
    while (c > 1 && (segments * c > room || c > (tiles + (latent ? 0 : 2)) / (latent ? 1 : 3))) c /= 2;
    const int64_t each = latent   ? attn::kLatentClusterTiles
                         : c == 1 ? attn::kPagedSoloTiles
                                  : attn::kPagedClusterTiles;
    if (tiles <= c * each) L.cluster = c;
  }
  L.by_segment = L.first > 0 || segments <= L.ctas;
  L.n_notes = L.by_segment ? static_cast<int>(segments) : L.ctas;
  size_t off = kHeaderBytes;
  L.notes = off;
  off = round_up(off + static_cast<size_t>(L.n_notes) * sizeof(attn::MergeNote), 256);
  L.part_o = off;
  off = round_up(off + 2 * static_cast<size_t>(L.ctas) * L.rows * p->d * sizeof(float), 256);
  L.part_l = off;
  off = round_up(off + 2 * static_cast<size_t>(L.ctas) * L.rows * sizeof(float), 256);
  if (L.splits > 0) {
    L.pre_o = off;
    off = round_up(off + static_cast<size_t>(L.splits + 1) * rows_all * p->d * sizeof(float), 256);
    L.pre_l = off;
    off = round_up(off + static_cast<size_t>(L.splits + 1) * rows_all * sizeof(float), 256);
  }
  L.total = off;
  return L;
}

PagedArgs args_of(const attn_params* p, int32_t n_q, const attn_pages* g, const Layout& L,
                  const void* q, void* o, float* lse, void* ws) {
  char* w = static_cast<char*>(ws);
  PagedArgs a{};
  a.B = p->B;
  a.H = p->H;
  a.heads = L.heads;
  a.blocks = L.blocks;
  a.head_rows = L.head_rows;
  a.n_q = n_q;
  a.rows = L.rows;
  a.all_rows = p->H * n_q;
  a.causal = p->causal != 0;
  a.d = p->d;
  a.key_lens = p->key_lens;
  a.table = g->table;
  a.table_stride = g->table_stride;
  a.cap = p->N;
  a.page_shift = log2_of(g->page_size);
  a.num_pages = g->num_pages;
  a.first = L.first;
  a.scale = p->scale;
  a.scale_log2 = p->scale * kLog2e;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.stride_b = p->stride_b;
  a.stride_h = p->stride_h;
  a.stride_n = p->stride_n;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.notes = reinterpret_cast<attn::MergeNote*>(w + L.notes);
  a.by_segment = L.by_segment;
  a.cluster = L.cluster;
  a.part_o = reinterpret_cast<float*>(w + L.part_o);
  a.part_l = reinterpret_cast<float*>(w + L.part_l);
  a.pre_splits = L.splits;
  a.pre_o = reinterpret_cast<float*>(w + L.pre_o);
  a.pre_l = reinterpret_cast<float*>(w + L.pre_l);
  a.ctas = L.ctas;
  a.status = reinterpret_cast<int*>(w);
  a.timeout_ns = kTimeoutNs;
  return a;
}

attn_status launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return ATTN_OK;
  char msg[256];
  snprintf(msg, sizeof(msg), "%s: %s", what, cudaGetErrorString(e));
  return fail(ATTN_ERR_CUDA, msg);
}

// The tensor map of a cache without pages is read past its end only (a table may
// name pages all the same); it needs some extent.
int at_least_1(int n) { return n < 1 ? 1 : n; }

int box_rows(const attn_pages* g, int keys) { return g->page_size < keys ? g->page_size : keys; }

}  // namespace

extern "C" {

size_t attn_decode_paged_workspace_size(const attn_params* p, int32_t n_q,
                                        const attn_pages* pages) {
  if (validate(p, n_q, pages, false) != ATTN_OK) return 0;
  return layout(p, n_q, pages, false).total;
}

attn_status attn_decode_paged(const attn_params* p, int32_t n_q, const attn_pages* pages,
                              const void* q, const void* k, const void* v, void* o, float* lse,
                              void* ws, size_t ws_bytes, void* stream) {
  attn_status st = validate(p, n_q, pages, false);
  if (st != ATTN_OK) return st;
  const Layout L = layout(p, n_q, pages, false);
  if ((st = check_ws(ws, ws_bytes, L.total)) != ATTN_OK) return st;
  if (empty(p)) return ATTN_OK;
  if (pages->num_pages == 0) k = v = q;   // no cache to point at, and none is read
  if ((st = check_ptrs({q, k, v, o, lse})) != ATTN_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  PagedArgs a = args_of(p, n_q, pages, L, q, o, lse, ws);
  const auto map = [&](CUtensorMap* m, const void* ptr, int keys) {
    return static_cast<attn_status>(attn::encode_pages(
        m, ptr, at_least_1(pages->num_pages), kv_heads(p), pages->page_size, p->d, p->kv_stride_b,
        p->kv_stride_h, p->kv_stride_n, box_rows(pages, keys)));
  };
  CUtensorMap tk, tv;
  if (L.first > 0) {
    if ((st = map(&tk, k, attn::kTile)) != ATTN_OK || (st = map(&tv, v, attn::kTile)) != ATTN_OK)
      return st;
    attn::PrefixArgs f{};
    f.B = p->B;
    f.H = p->H;
    f.H_kv = kv_heads(p);
    f.group = p->H / f.H_kv;
    f.n_q = n_q;
    f.causal = a.causal;
    f.d = p->d;
    f.key_lens = p->key_lens;
    f.table = pages->table;
    f.table_stride = pages->table_stride;
    f.cap = a.cap;
    f.page_shift = a.page_shift;
    f.num_pages = pages->num_pages;
    f.shared_len = L.first;
    f.splits = L.splits;
    f.tiles = L.tiles;
    f.rows = p->B * L.head_rows;
    f.scale = a.scale;
    f.scale_log2 = a.scale_log2;
    f.q = a.q;
    f.stride_b = a.stride_b;
    f.stride_h = a.stride_h;
    f.stride_n = a.stride_n;
    f.pre_o = a.pre_o;
    f.pre_l = a.pre_l;
    f.status = a.status;
    f.timeout_ns = a.timeout_ns;
    f.stall = attn::take_stall(attn::kStallPrefixSoftmax, &f.timeout_ns);
    if ((st = launched(attn::launch_prefix(tk, tv, f, s), "shared prefix launch")) != ATTN_OK)
      return st;
  }
  if ((st = map(&tk, k, attn::kPagedKeys)) != ATTN_OK ||
      (st = map(&tv, v, attn::kPagedKeys)) != ATTN_OK)
    return st;
  a.stall = attn::take_stall(attn::kStallPagedTile, &a.timeout_ns);
  if ((st = launched(attn::launch_paged(tk, tv, a, L.ctas, s), "paged decode launch")) != ATTN_OK)
    return st;
  if (L.cluster > 0) return ATTN_OK;   // merged already
  if (L.first > 0) return launched(attn::launch_paged_finish(a, L.ctas, s), "shared prefix merge launch");
  if (L.ctas == 1) return ATTN_OK;   // one CTA cuts nothing
  return launched(attn::launch_paged_merge(a, L.n_notes, L.ctas, s), "paged merge launch");
}

size_t attn_decode_latent_workspace_size(const attn_params* p, int32_t n_q,
                                         const attn_pages* pages) {
  if (validate(p, n_q, pages, true) != ATTN_OK) return 0;
  return layout(p, n_q, pages, true).total;
}

attn_status attn_decode_latent(const attn_params* p, int32_t n_q, const attn_pages* pages,
                               const void* q, const void* c, void* o, float* lse, void* ws,
                               size_t ws_bytes, void* stream) {
  attn_status st = validate(p, n_q, pages, true);
  if (st != ATTN_OK) return st;
  const Layout L = layout(p, n_q, pages, true);
  if ((st = check_ws(ws, ws_bytes, L.total)) != ATTN_OK) return st;
  if (empty(p)) return ATTN_OK;
  if (pages->num_pages == 0) c = q;   // no cache to point at, and none is read
  if ((st = check_ptrs({q, c, o, lse})) != ATTN_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  PagedArgs a = args_of(p, n_q, pages, L, q, o, lse, ws);
  a.pages = static_cast<const __nv_bfloat16*>(c);
  a.stride_page = p->kv_stride_b;
  a.dense = p->kv_stride_n == p->d + attn::kLatentRope;
  CUtensorMap tc;
  st = static_cast<attn_status>(attn::encode_pages(
      &tc, c, at_least_1(pages->num_pages), 1, pages->page_size, p->d + attn::kLatentRope,
      p->kv_stride_b, p->kv_stride_b, p->kv_stride_n, box_rows(pages, attn::kLatentKeys)));
  if (st != ATTN_OK) return st;
  a.stall = attn::take_stall(attn::kStallLatentSoftmax, &a.timeout_ns);
  if ((st = launched(attn::launch_latent(tc, a, L.ctas, s), "latent decode launch")) != ATTN_OK)
    return st;
  if (L.ctas == 1 || L.cluster > 0) return ATTN_OK;
  // the merge writes o, which is contiguous
  a.stride_n = p->d;
  a.stride_h = static_cast<int64_t>(n_q) * p->d;
  a.stride_b = static_cast<int64_t>(p->H) * n_q * p->d;
  return launched(attn::launch_paged_merge(a, L.n_notes, L.ctas, s), "latent merge launch");
}

}  // extern "C"
