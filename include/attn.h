/*
 * exact_attention_12_gb300 — fused exact scaled dot-product attention for
 * NVIDIA GB300 (sm_103a).  C interface.
 *
 * The operation (FlashAttention: Fast and Memory-Efficient Exact Attention
 * with IO-Awareness, Dao et al. 2022, as summarised on the pages
 * "FlashAttention: Cơ chế Attention chính xác, nhanh và tối ưu bộ nhớ với
 * nhận thức IO" (xyznot.com, "Phương pháp"), "3.3 Hiểu sâu cơ chế
 * Self-Attention" (§3 Scaled Dot-Product Attention, §10 Causal Mask, §12
 * FlashAttention) and the azimuth.plus FlashAttention explainer
 * ("الخوارزمية خطوة بخطوة", the step-by-step algorithm)):
 *
 *   S = scale * Q K^T, with S_ij = -inf where key j is not allowed for query i
 *   L_i = logsumexp_j S_ij               (natural log, fp32)
 *   P = exp(S - L),  P~ = P * Z / (1 - p')  (Z: Philox dropout keep mask)
 *   O = P~ V
 *
 * Allowed(i, j) = (!causal || j <= i) && j < key_lens[b] &&
 *                 block_mask[i / 128][j / 128] != 0.
 * A row with no allowed key gets O_i = 0 and L_i = -inf.
 *
 * Backward (chain rule of the above; the pages state only that S and P are
 * recomputed from Q, K, V and the stored statistics):
 *   D = rowsum(dO * O),  dV = P~^T dO,  dP = (dO V^T) * Z / (1 - p'),
 *   dS = P * (dP - D),   dQ = scale * dS K,  dK = scale * dS^T Q.
 *
 * Dropout keep mask: Philox4x32-10 (Salmon et al., SC'11) at counter
 * (floor(j / 8), i, b * H + h, philox_offset) under key (low 32 bits of
 * philox_seed, high 32 bits) gives four 32-bit words; word (j mod 8) / 2
 * holds the 16-bit uniform u of element (b, h, i, j) in its low half when j
 * is even, its high half when j is odd.  The element is dropped iff u < T,
 * T = min(2^16 - 1, floor(dropout_p * 2^16)) computed in fp64 from the float
 * dropout_p: the drop rate is exactly p' = T / 2^16 (within 2^-16 of
 * dropout_p) and kept probabilities are scaled by 1 / (1 - p'), so P~ =
 * P * Z / (1 - p').  The backward call regenerates the same mask.
 *
 * Layout: Q, K, V, O, dO, dQ, dK, dV are logical [B, H, N, d] arrays with
 * unit stride along d and the element strides stride_b, stride_h, stride_n
 * (shared by all eight tensors).  lse is a contiguous fp32 [B, H, N].
 * Every device pointer must be 16-byte aligned; strides must be multiples
 * of 8 elements (bf16) or 4 elements (fp32).
 *
 * Ownership: the caller allocates and owns every buffer, including the
 * workspace `ws` (device memory, at least attn_workspace_size() bytes).  The
 * library allocates nothing and keeps no state between calls.  The first
 * 256 bytes of a workspace hold a device status word and the forward's work
 * counter, and must be zero before the workspace is first used; every
 * forward leaves the counter at zero when it completes, and attn_check()
 * reads and clears the status word.
 *
 * Streams: every call only enqueues work on `stream` (a cudaStream_t; NULL is
 * the legacy default stream) and returns.  Argument errors are detected on
 * the host before anything is enqueued.  Launch failures return
 * ATTN_ERR_CUDA.  A kernel that stops making progress gives up after a
 * bounded wait and records ATTN_ERR_TIMEOUT in the workspace status word,
 * which attn_check() returns.
 *
 * CUDA graphs: attn_fwd, attn_bwd, the decode steps and the calls on paged
 * caches (attn_decode_paged, _latent and _fp4, attn_key_weights, attn_pages_*)
 * neither synchronise nor allocate, and every launch argument (tensor maps
 * included) is passed by value, so the calls can be captured into a CUDA graph
 * and replayed.  Make
 * one uncaptured call of each kind first: it sets the kernels' attributes.
 * The forward and backward kernels and those on paged caches are launched
 * with programmatic stream serialisation; each waits for the preceding work in
 * the stream to complete before it reads or writes global memory.  One does not
 * wait for the kernel directly before it: with a shared prefix the paged decode
 * kernel starts on its own keys as soon as every CTA of the prefix kernel has
 * passed that wait, so everything before the call is complete, and waits for the
 * prefix kernel before it merges and before it ends.
 *
 * Thread safety: calls on different workspaces may run concurrently; two
 * calls in flight on the same workspace race.
 */
#ifndef EXACT_ATTENTION_12_GB300_ATTN_H
#define EXACT_ATTENTION_12_GB300_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  ATTN_OK = 0,
  ATTN_ERR_INVALID_ARG = 1,   /* bad shape, stride, pointer, scale, p, ... */
  ATTN_ERR_UNSUPPORTED = 2,   /* valid but not implemented (e.g. fp32 bwd) */
  ATTN_ERR_CUDA = 3,          /* a CUDA runtime/driver call failed */
  ATTN_ERR_TIMEOUT = 4,       /* a kernel wait gave up (device status) */
  ATTN_ERR_WORKSPACE = 5,     /* workspace missing, misaligned or too small */
  ATTN_ERR_PAGE = 6,          /* a page table or list in device memory held an
                                 index outside its range (device status) */
  ATTN_ERR_FULL = 7           /* a cache had no free page left (device status) */
} attn_status;

typedef enum { ATTN_BF16 = 0, ATTN_FP32 = 1, ATTN_FP8_E4M3 = 2 } attn_dtype;

typedef struct attn_params {
  int32_t B, H, N, d;        /* batch, heads, sequence length, head dim.
                                d in {64, 128}.  B, H or N = 0: no work. */
  int32_t dtype;             /* attn_dtype.  bf16: forward and backward;
                                fp32: forward only, on the tensor cores in
                                TF32 (the scores as three TF32 products of
                                the operands' high and low parts, P V as
                                one), fp32 o; fp8 (E4M3 q, k, v with the
                                de-scale factors below, bf16 o): forward
                                only, d = 128, no dropout. */
  float scale;               /* score scale, e.g. 1/sqrt(d); finite */
  int32_t causal;            /* nonzero: keep j <= i (top-left aligned) */
  float dropout_p;           /* drop probability in [0, 1); 0 = no dropout */
  uint64_t philox_seed;      /* Philox key */
  uint64_t philox_offset;    /* Philox counter word 3; must be < 2^32 */
  const int32_t* key_lens;   /* device [B]: keys j >= key_lens[b] masked;
                                NULL = all N keys valid.  Values are
                                clamped to [0, N]. */
  const uint8_t* block_mask; /* device uint8 [nb][nb], nb = ceil(N / 128),
                                row-major; nonzero = 128x128 block kept;
                                NULL = dense.  bf16 only. */
  int64_t block_mask_head_stride; /* bytes between the masks of consecutive
                                (b * H + h); 0 = one mask for all heads */
  int64_t stride_b, stride_h, stride_n; /* element strides of q, o, dout,
                                dq (and of k, v, dk, dv when the kv_stride
                                fields are 0) */
  /* Grouped-query attention ("3.3 Hiểu sâu cơ chế Self-Attention", §9.2
   * MQA and §9.3 GQA): the query heads are split into H_kv groups of H / H_kv
   * consecutive heads that share one key/value head, so query head h reads
   * key/value head h / (H / H_kv).  k, v, dk and dv are [B, H_kv, N, d]; dk
   * and dv of a shared head are the sums over its group.  H_kv = H (or 0) is
   * ordinary multi-head attention, H_kv = 1 multi-query attention. */
  int32_t H_kv;              /* key/value heads, dividing H; 0 = H */
  int32_t reserved;          /* must be 0 */
  int64_t kv_stride_b, kv_stride_h, kv_stride_n; /* element strides of k, v,
                                dk, dv; all three 0 = the strides above
                                (then H_kv must equal H) */
  /* FP8 inputs (dtype ATTN_FP8_E4M3).  The FlashAttention explainer
   * (azimuth.plus, timeline entry "FlashAttention-3") names FP8 as the
   * Hopper successor's step to higher throughput; the format is E4M3 of the
   * OCP 8-bit floating point specification (bias 7, largest value 448, no
   * infinities).  The attention is that of the real values
   *   Q = q_descale * q,  K = k_descale * k,  V = v_descale * v,
   * so the scores are scale * q_descale * k_descale * (q k^T).  The kernel
   * rounds the probabilities to E4M3 for the P V product (the row sums
   * that normalise O are taken before rounding), so O carries an error of
   * at most 2^-4 * sum_j P_ij |V_jc| + 2^-10 * max_j P_ij * sum_j |V_jc|
   * beyond the bf16 rounding of O; L is exact up to fp32 arithmetic.
   * o is bf16 [B, H, N, d] with the query strides.  Strides are in
   * elements and must be multiples of 16.  0 means 1 for each factor;
   * ignored for the other dtypes. */
  float q_descale, k_descale, v_descale;
  int32_t reserved2;         /* must be 0 */
} attn_params;

/* Bytes of device workspace a forward (for_backward = 0) or backward
 * (for_backward != 0) call needs.  Returns 0 if the parameters are invalid
 * (the call itself then reports why). */
size_t attn_workspace_size(const attn_params* p, int for_backward);

/* Forward: O [B,H,N,d] (same dtype as q; bf16 for fp8 inputs) and lse
 * [B,H,N] fp32.  For fp8 the workspace also holds a transposed copy of v
 * ([B, H_kv, d, N] padded to a multiple of 128 keys), written by the call;
 * for fp32 it holds the high and low TF32 parts of q and k and a transposed
 * copy of v, written by the call. */
attn_status attn_fwd(const attn_params* p, const void* q, const void* k,
                     const void* v, void* o, float* lse, void* ws,
                     size_t ws_bytes, void* stream);

/* Backward (bf16): needs o and lse from attn_fwd with the same parameters
 * (dropout seed and offset included).  Writes dq [B,H,N,d] and dk, dv
 * [B,H_kv,N,d] bf16. */
attn_status attn_bwd(const attn_params* p, const void* q, const void* k,
                     const void* v, const void* o, const float* lse,
                     const void* dout, void* dq, void* dk, void* dv, void* ws,
                     size_t ws_bytes, void* stream);

/* The three stages attn_bwd runs, callable one by one on the same workspace
 * (for callers that schedule or time them separately):
 *   attn_bwd_preprocess  D = rowsum(dO * O) and L * log2(e) into the
 *                        workspace (rows padded to a multiple of 128);
 *                        zeroes the workspace's fp32 dQ accumulator.
 *   attn_bwd_main        the fused recomputing backward: dK, dV written,
 *                        dQ accumulated into the workspace.  Reads what the
 *                        preprocess of the same call sequence wrote.
 *   attn_bwd_dq          dQ = scale * accumulator, converted to bf16.
 * Arguments mean the same as for attn_bwd; the workspace must be the same
 * and at least attn_workspace_size(p, 1) bytes. */
attn_status attn_bwd_preprocess(const attn_params* p, const void* o,
                                const float* lse, const void* dout, void* ws,
                                size_t ws_bytes, void* stream);
attn_status attn_bwd_main(const attn_params* p, const void* q, const void* k,
                          const void* v, const void* dout, void* dk, void* dv,
                          void* ws, size_t ws_bytes, void* stream);
attn_status attn_bwd_dq(const attn_params* p, void* dq, void* ws,
                        size_t ws_bytes, void* stream);

/* Backward without a caller workspace.  The pages have no counterpart: this
 * is an interface for callers that cannot allocate device memory (a plug-in
 * inside a host application that owns all device allocations, a runtime with
 * a fixed device-memory budget, a latency-critical loop where cudaMalloc
 * could synchronise the device).  Arguments and results are those of
 * attn_bwd; the scratch attn_bwd would take from `ws` comes from a 64 MiB
 * array built into the library, which every GPU that loads the library holds
 * until the process exits.
 *   - Problems needing more than 64 MiB of scratch (attn_workspace_size(p, 1))
 *     are rejected with ATTN_ERR_WORKSPACE before anything is enqueued.
 *   - Nothing is allocated: no cudaMalloc, cudaFree or allocating library call.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current and caches it; make that
 *     first call before any stream capture.
 *   - All calls share the one array and it keeps the previous call's
 *     contents: calls that overlap on the GPU (other streams, other host
 *     threads) race with each other.  The call clears the status words and
 *     rewrites everything else it reads.
 *   - A device-side time-out is recorded in the built-in array's status
 *     words: attn_check(NULL, stream) reports it (and clears it).  The next
 *     attn_bwd_noalloc call clears it too, so check before the next call. */
attn_status attn_bwd_noalloc(const attn_params* p, const void* q,
                             const void* k, const void* v, const void* o,
                             const float* lse, const void* dout, void* dq,
                             void* dk, void* dv, void* stream);

/* Decode step: the newest n_q query positions of each sequence against its
 * key/value cache.  The pages' pass is the training forward; this is the
 * same attention at generation time, where each new token attends the keys
 * cached so far (the KV cache of "3.3 Hiểu sâu cơ chế Self-Attention", §9).
 *   p->N          cache capacity: k and v are [B, H_kv, N, d] (key/value
 *                 strides and grouping as in attn_params)
 *   p->key_lens   required, device [B]: cached keys per sequence, clamped to
 *                 [0, N].  Query row t of sequence b is the token at position
 *                 key_lens[b] - n_q + t.
 *   p->causal     nonzero: query t attends keys j <= its position; otherwise
 *                 every cached key
 *   q, o          [B, H, n_q, d] with the query strides (stride_n steps over
 *                 the n_q rows); bf16
 *   lse           fp32 [B, H, n_q] (natural log; -inf for a row with no key)
 * 1 <= n_q and (H / H_kv) * n_q <= 64; dropout_p must be 0 and block_mask
 * NULL (ATTN_ERR_UNSUPPORTED otherwise).  The cache is split into chunks
 * processed in parallel and merged by the logsumexp rule; the workspace
 * (attn_decode_workspace_size bytes, the same 256-byte header rules as
 * above) holds the per-chunk partial results. */
size_t attn_decode_workspace_size(const attn_params* p, int32_t n_q);
attn_status attn_decode(const attn_params* p, int32_t n_q, const void* q, const void* k,
                        const void* v, void* o, float* lse, void* ws, size_t ws_bytes,
                        void* stream);

/* ------------------------------------------------------------------------
 * Paged key/value caches.  A serving program keeps the caches of many
 * sequences in pages of equal size that are handed out as sequences grow, so
 * that no sequence needs a contiguous, full-length buffer (the KV cache of
 * "3.3 Hiểu sâu cơ chế Self-Attention", §9, has no pages; these calls have
 * no counterpart there).
 *
 * Key j of sequence b lies in row j mod page_size of page
 * table[b * table_stride + j / page_size].  Only the entries that hold cached
 * keys, ceil(len / page_size) of a row, are read.  An entry outside
 * [0, num_pages) is never followed: its page reads as zeros and the
 * workspace's status becomes ATTN_ERR_PAGE, which attn_check reports. */
typedef struct attn_pages {
  const int32_t* table;      /* device [B][table_stride] */
  int64_t table_stride;      /* entries between the rows of two sequences */
  int32_t max_pages;         /* entries of a row that may be used */
  int32_t page_size;         /* keys per page: a power of two, 16 to 32768 */
  int32_t num_pages;         /* pages in the cache */
  int32_t shared_len;        /* leading keys that all sequences share (below); 0: none */
} attn_pages;

/* Decode step against a paged cache: attn_decode with
 *   k, v    [num_pages, H_kv, page_size, d] bf16, where kv_stride_b is the
 *           stride between pages (all three key/value strides are required)
 *   p->N    must be max_pages * page_size
 * and the same query rows, masks and outputs.  rows = (H / H_kv) * n_q is not
 * limited to 64 here; the cache is read once per 64 of these rows.  Limits
 * (ATTN_ERR_UNSUPPORTED beyond): H * n_q <= 32768, B * H * n_q <= 2^30, p->N <=
 * 2^30, and B * H_kv * ceil(rows / 64) * (p->N / 32 + 9) < 2^31.
 * Rows of a page past the end of its sequence are not used, whatever they
 * hold.  A key that a query row may not attend (causal, n_q > 1) may hold
 * anything too, but its value must be finite unless no row of its sequence
 * attends it: a probability of 0 times infinity or NaN is NaN.  A cache of no
 * pages is one too: k and v may be NULL then.
 *
 * How the work is given out goes by max_pages, not by the lengths, which are on
 * the device: where all sequences are short, a table that is no wider than the
 * longest needs is faster (64 sequences of 50 to 200 keys: 13 us, with room for
 * 20000 keys 19 us).
 *
 * shared_len > 0: the first shared_len / page_size entries of the table rows,
 * as far as each sequence reaches, name the same pages (a fork of one prompt, a
 * common system prompt); those of the longest sequence are read.  Their keys are attended once for all sequences, the
 * rest per sequence, and the two are merged by the logsumexp rule; the result
 * is that of shared_len = 0 up to rounding.  It pays where the prefix would be
 * read often, from about B * H_kv = 32 on (16384 shared keys: 32 sequences, 8
 * key/value heads 30 us instead of 158; 2 sequences, one head 25 instead of 13,
 * since a prefix is cut into 16 pieces at most).  shared_len must be a multiple
 * of page_size and at most p->N.  A cache_lens[b] below shared_len is allowed:
 * that sequence attends its own first keys only; the keys and values of the
 * shared pages that other sequences use must then be finite. */
size_t attn_decode_paged_workspace_size(const attn_params* p, int32_t n_q,
                                        const attn_pages* pages);
attn_status attn_decode_paged(const attn_params* p, int32_t n_q, const attn_pages* pages,
                              const void* q, const void* k, const void* v, void* o, float* lse,
                              void* ws, size_t ws_bytes, void* stream);

/* Decode step of latent attention, absorbed form: every cached token is one
 * vector of d + 64 columns that is the key of all heads as it stands and
 * whose first d columns are their value,
 *   S = scale * q c^T,  O = softmax(S) c[:, 0:d],  L = logsumexp(S)
 * (the per-head up-projections of keys and values are folded into q and into
 * what follows O; the last 64 columns carry the position).
 *   p->d    value columns: 256 or 512;  p->N = max_pages * page_size;
 *           p->H_kv 0 or 1
 *   q       [B, H, n_q, d + 64] bf16 with the query strides
 *   c       [num_pages, page_size, d + 64] bf16; kv_stride_b between pages,
 *           kv_stride_n between tokens (kv_stride_h is ignored)
 *   o       [B, H, n_q, d] bf16, contiguous;  lse fp32 [B, H, n_q]
 * key_lens, causal and the query positions are those of attn_decode, what is
 * said of max_pages and of values that some rows may not attend holds here too.
 * Limits (ATTN_ERR_UNSUPPORTED beyond): H * n_q <= 32768, B * H * n_q <= 2^30,
 * p->N <= 2^30, B * (p->N / 64 + 9) < 2^31.  pages->shared_len must be 0. */
size_t attn_decode_latent_workspace_size(const attn_params* p, int32_t n_q,
                                         const attn_pages* pages);
attn_status attn_decode_latent(const attn_params* p, int32_t n_q, const attn_pages* pages,
                               const void* q, const void* c, void* o, float* lse, void* ws,
                               size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Paged caches in 4 bits.  Every 16 columns of a key (or value) share a scale:
 *   x = descale * s * c,
 * c in {0, 0.5, 1, 1.5, 2, 3, 4, 6} with a sign (E2M1; a byte holds two, the
 * column of even index in its low four bits), s an E4M3 number (the OCP 8-bit
 * format, as in attn_fwd), descale one factor of the tensor.  9 d / 16 bytes a
 * key where bf16 has 2 d.  Codes and scales are two buffers of pages: codes
 * [num_pages][H_kv][page_size][d / 2], scales [num_pages][H_kv][page_size][d / 16];
 * a head's rows of a page follow one another without gaps, pages and heads may
 * be apart (what is written to must not overlap).  attn_pages_copy, _fork, _compact
 * and _evict take them as pools.  (The pages about attention have no counterpart.) */
typedef struct attn_fp4 {
  void* codes;               /* 16-byte aligned, as is scales */
  void* scales;
  int64_t code_page, code_head;    /* bytes between pages (below 2^32) and between */
  int64_t scale_page, scale_head;  /* heads, multiples of 16 */
  float descale;             /* 2^-100 to 2^100 */
  int32_t reserved;          /* must be 0 */
} attn_fp4;

/* Stores new keys and values: token t of sequence b, t < counts[b], becomes the
 * cached key (and value) at position key_lens[b] - counts[b] + t, that is, the
 * cache has grown already (attn_pages_extend) and these are its newest tokens.
 *   p->B, p->H_kv, p->d (64 or 128);  p->N = n, the tokens k and v have room for;
 *   p->key_lens  the cache lengths, clamped to [0, max_pages * page_size]
 *   counts       device [B], clamped to [0, n]; NULL: n for every sequence
 *   k, v         [B, H_kv, n, d] bf16 with the kv strides
 * s is the E4M3 number nearest to max |x| / (6 descale) of its columns (at most
 * 448), c the nearest to x / (s descale) (at most 6), ties to the even code.  A
 * NaN makes its 16 columns NaN; infinities become the largest value.
 * Tokens whose position is negative are left out; an entry of the table outside
 * the cache is recorded (ATTN_ERR_PAGE) and its tokens are left out.  Fields of
 * p that are not named are ignored; n <= 2^30.  ws: 256 bytes. */
attn_status attn_pages_store_fp4(const attn_params* p, const attn_pages* pages,
                                 const int32_t* counts, const void* k, const void* v,
                                 const attn_fp4* k_cache, const attn_fp4* v_cache, void* ws,
                                 size_t ws_bytes, void* stream);

/* The way back: k and v [B, H_kv, n, d] receive, as bf16, what the cache holds of
 * the tokens that attn_pages_store_fp4 would store; zeros where there is none. */
attn_status attn_pages_load_fp4(const attn_params* p, const attn_pages* pages,
                                const int32_t* counts, const attn_fp4* k_cache,
                                const attn_fp4* v_cache, void* k, void* v, void* ws,
                                size_t ws_bytes, void* stream);

/* attn_decode_paged on such a cache (the kv strides of p are ignored, shared_len
 * must be 0): what it says of rows, masks, lengths and of values that are not
 * attended holds here.  Q and P enter the products in fp16, Q scaled by a power
 * of two per row, P to be 2^7 where a row's maximum is taken: keys 2^32 below it
 * begin to be lost.  Keys and values as they are.  S, L and O in fp32, O rounded
 * to bf16.  Scores (scale q k) stay below 2^27 in magnitude; fp32 tells larger ones
 * apart by 16 and more, which P does not reach.  Limits as there, the last one
 * being B * H_kv * ceil(rows / 64) * (p->N / 32 + 21) < 2^31. */
size_t attn_decode_fp4_workspace_size(const attn_params* p, int32_t n_q, const attn_pages* pages);
attn_status attn_decode_fp4(const attn_params* p, int32_t n_q, const attn_pages* pages,
                            const void* q, const attn_fp4* k, const attn_fp4* v, void* o,
                            float* lse, void* ws, size_t ws_bytes, void* stream);

/* The attention weight that query rows give each cached key:
 *   W[b, h, j] = sum over the query heads of key/value head h and the n_q rows of
 *                exp(scale q k_j - lse)   over the rows that attend key j,
 * added to weights[b, h, j] (add != 0) or written there, for j < key_lens[b];
 * further entries stay as they are.  Rows, masks and positions as in
 * attn_decode_paged, whose lse [B, H, n_q] this takes; a row with lse = -inf gives
 * nothing, whatever its queries and the keys hold.  Summed in fp32 in an order that
 * does not depend on timing.  Limits as there, rows in one piece: the last one is
 * B * H_kv * (p->N / 32 + 9) < 2^31.
 *   k         [num_pages, H_kv, page_size, d] bf16 with the kv strides, or NULL and
 *   k_cache   a cache in 4 bits (then NULL otherwise)
 *   weights   fp32, weight_stride_b and weight_stride_h entries between sequences
 *             and heads; the max_pages * page_size entries of each lie apart
 * ws: 256 bytes. */
attn_status attn_key_weights(const attn_params* p, int32_t n_q, const attn_pages* pages,
                             const void* q, const void* k, const attn_fp4* k_cache,
                             const float* lse, float* weights, int64_t weight_stride_b,
                             int64_t weight_stride_h, int32_t add, void* ws, size_t ws_bytes,
                             void* stream);

/* Upkeep of a paged cache, on the device: no call synchronises or reads
 * anything back.  The state is a table of pages, a length per sequence (row)
 * and a reference count per page; a page with count 0 is free.  A row holds
 * ceil(len / page_size) pages, its further entries mean nothing.  Lists are
 * int32 device arrays.  What a list or the state holds wrongly is skipped and
 * recorded in the workspace's status (ATTN_ERR_PAGE; ATTN_ERR_FULL where a
 * cache has too few free pages), which attn_check reports. */
typedef struct attn_page_table {
  int32_t* table;            /* [rows][table_stride] */
  int64_t table_stride;
  int32_t* lens;             /* [rows] */
  int32_t* refs;             /* [num_pages] */
  int32_t rows, max_pages, page_size, num_pages;
} attn_page_table;

/* One buffer of pages (keys or values of one layer, latent vectors, ...): a
 * page's page_bytes are contiguous.  base 16-byte aligned (NULL where the cache
 * has no pages), both sizes multiples of 16. */
typedef struct attn_pool {
  void* base;
  int64_t page_stride, page_bytes;
} attn_pool;

/* Workspace of every call below for lists of up to n entries (the header
 * rules of the other calls apply); attn_pages_copy needs 256 bytes. */
size_t attn_pages_workspace_size(const attn_page_table* t, int32_t n);

/* Page dst[i] of every pool becomes a copy of page src[i].  Where a dst is
 * also another pair's src or dst, what it and the copies of it hold is
 * unspecified. */
attn_status attn_pages_copy(const attn_pool* pools, int32_t n_pools, int32_t num_pages,
                            const int32_t* src, const int32_t* dst, int32_t n, void* ws,
                            size_t ws_bytes, void* stream);

/* Sequence seqs[i] grows to new_lens[i] keys (not below its length): the
 * pages it needs are the lowest free ones, in the list's order.  A sequence
 * for which too few are left stays as it was, and so do those after it that
 * need pages.  Of a row that is named twice the first entry counts. */
attn_status attn_pages_extend(const attn_page_table* t, const int32_t* seqs,
                              const int32_t* new_lens, int32_t n, void* ws, size_t ws_bytes,
                              void* stream);

/* Row children[i], which must be empty (length 0), becomes a copy of sequence
 * parents[i]: full pages are shared (their counts grow), a part-filled last
 * page is copied, in every pool, to the lowest free page.  new_pages[i]
 * (device, output) is that page, -1 if none was needed, -2 if the fork was
 * not made, because of its rows, of a page of the parent that is free or
 * outside the cache, or for want of a free page.  Of a child that is named twice the first entry counts; all
 * entries see the state before the call. */
attn_status attn_pages_fork(const attn_page_table* t, const attn_pool* pools, int32_t n_pools,
                            const int32_t* parents, const int32_t* children, int32_t n,
                            int32_t* new_pages, void* ws, size_t ws_bytes, void* stream);

/* The sequences give back their pages: counts fall, the entries they held
 * become -1, the lengths 0.  Freeing an empty row does nothing. */
attn_status attn_pages_free(const attn_page_table* t, const int32_t* seqs, int32_t n, void* ws,
                            size_t ws_bytes, void* stream);

/* Moves the pages in use to the places [0, pages in use): those behind, in
 * ascending order, to the free ones before, in ascending order, in every
 * pool; tables and counts follow.  moved[p] (device [num_pages], output) is
 * where page p now is, -1 for a page that was free (an entry that names one
 * becomes -1 and is recorded, one outside the cache stays as it is). */
attn_status attn_pages_compact(const attn_page_table* t, const attn_pool* pools, int32_t n_pools,
                               int32_t* moved, void* ws, size_t ws_bytes, void* stream);

/* A buffer of pages by its rows: row r of head h in page g is row_bytes bytes at
 * base + g * page_stride + h * head_stride + r * row_stride (bytes).  Everything a
 * multiple of 4; rows, heads and pages apart. */
typedef struct attn_rows {
  void* base;
  int64_t page_stride, head_stride, row_stride;
  int32_t row_bytes, reserved;     /* reserved must be 0 */
} attn_rows;

/* Eviction by gathered attention weight: sequence seqs[i] shrinks to new_lens[i]
 * keys, every head by its own weights.  A head keeps its last
 * min(recent, new_lens[i]) keys and, of those before them, the ones with the
 * largest weights (of equal ones those in front; NaN counts as the largest); they keep
 * their order and move to the front, in every pool.  The weights move along (a -0 as 0,
 * a NaN as some NaN), those behind the new length become 0.  Pages that are no longer needed are given
 * back as in attn_pages_free.  A sequence that is not longer than new_lens[i] stays
 * as it is.
 *   weights    fp32 [rows][heads][width], weight_stride_row and weight_stride_head
 *              entries between rows and heads, the max_pages * page_size entries of
 *              each lie apart; width >= max_pages * page_size
 *   slots      device int32 [n][heads][width], output: slots[i][h][j] is where the
 *              key that is now in place j was before; -1 from the new length on,
 *              -2 throughout where a sequence was refused
 * Refused and recorded (ATTN_ERR_PAGE): a sequence outside the table, or named
 * before in the list; a negative new length; a length or page outside the cache, a
 * page that is free; a page that would be written to but is shared with another
 * sequence (of a fork; pages_copy to pages of its own first).  Pages behind the new
 * length may be shared.  All pools together at most 32768 bytes a row, 16 pools. */
size_t attn_pages_evict_workspace_size(const attn_page_table* t, int32_t heads, int32_t n,
                                       const attn_rows* pools, int32_t n_pools);
attn_status attn_pages_evict(const attn_page_table* t, const attn_rows* pools, int32_t n_pools,
                             int32_t heads, float* weights, int64_t weight_stride_row,
                             int64_t weight_stride_head, int32_t width, const int32_t* seqs,
                             const int32_t* new_lens, int32_t n, int32_t recent, int32_t* slots,
                             void* ws, size_t ws_bytes, void* stream);

/* Diagnostic: runs the kernels' time-out path on purpose.  Enqueues one warp
 * that waits on a barrier nothing arrives at, giving up after `limit_ns`
 * (clamped to [1 ms, 2 s]); it records ATTN_ERR_TIMEOUT in the workspace's
 * status words exactly as a stalled attention kernel would, so a following
 * attn_check returns ATTN_ERR_TIMEOUT.  `ws` needs 256 bytes. */
attn_status attn_selftest_timeout(void* ws, uint64_t limit_ns, void* stream);

/* Test hook for the time-out path of the attention kernels themselves (the
 * pages have no counterpart: this checks this library's failure detection).
 * Arms a one-shot stall for the next launch of the named kernel made by a
 * call on the calling host thread:
 *   ATTN_STALL_FWD_SOFTMAX  the forward (attn_fwd, bf16 or fp8): in every CTA,
 *                           softmax warp 0 withholds its "P ready" arrive for
 *                           its first key tile;
 *   ATTN_STALL_BWD_COMPUTE  the backward main kernel (attn_bwd, attn_bwd_main,
 *                           attn_bwd_noalloc): in every CTA, compute warp 0
 *                           withholds its "P ready" arrive for its first
 *                           query tile;
 *   ATTN_STALL_PAGED_TILE   the paged decode kernel (attn_decode_paged): in
 *                           every CTA, the first key tile is not copied;
 *   ATTN_STALL_PREFIX_SOFTMAX  the shared prefix's kernel (attn_decode_paged
 *                           with shared_len > 0 and two sequences or more), as
 *                           the forward's;
 *   ATTN_STALL_LATENT_SOFTMAX  attn_decode_latent, as the forward's;
 *   ATTN_STALL_EVICT_READ   attn_pages_evict: a head's first keys that move are
 *                           never reported as read (the cache's state is then
 *                           undefined);
 *   ATTN_STALL_WEIGHTS_SUM  attn_key_weights with many rows of a head: a warp
 *                           never gives its first scores back;
 *   ATTN_STALL_FP4_VALUES   attn_decode_fp4 with more than 32 rows of a head, d =
 *                           128, long caches: the first values never arrive.
 * The wait on that barrier then runs out; every wait of that launch
 * gives up after `limit_ns` (clamped to [1 ms, 2 s]).  The kernel drains its
 * copies and MMAs, frees its tensor memory and returns, and the status words
 * of the call's workspace hold ATTN_ERR_TIMEOUT and the wait site, which
 * attn_check reports.  That call's outputs are undefined; later calls are
 * unaffected.  Nothing faults, traps or hangs.  ATTN_STALL_NONE disarms;
 * other values give ATTN_ERR_INVALID_ARG. */
typedef enum {
  ATTN_STALL_NONE = 0,
  ATTN_STALL_FWD_SOFTMAX = 1,
  ATTN_STALL_BWD_COMPUTE = 2,
  ATTN_STALL_PAGED_TILE = 3,
  ATTN_STALL_PREFIX_SOFTMAX = 4,
  ATTN_STALL_LATENT_SOFTMAX = 5,
  ATTN_STALL_EVICT_READ = 8,
  ATTN_STALL_WEIGHTS_SUM = 9,
  ATTN_STALL_FP4_VALUES = 10
} attn_stall;
attn_status attn_debug_stall(int32_t which, uint64_t limit_ns);

/* Synchronises `stream`, returns the workspace's device status (ATTN_OK or
 * ATTN_ERR_TIMEOUT, ATTN_ERR_PAGE or ATTN_ERR_FULL) and clears it.  ws = NULL: the status of
 * attn_bwd_noalloc's built-in scratch on the current device. */
attn_status attn_check(void* ws, void* stream);

/* Static description of a status code. */
const char* attn_status_string(attn_status s);

/* Detail message of the last non-OK status returned on the calling thread. */
const char* attn_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* EXACT_ATTENTION_12_GB300_ATTN_H */
