"""Python binding of eviction from paged caches by gathered attention weight:
argument marshalling only."""

import struct

import torch

from ._abi import lib
from .fp4 import _cache
from .paged import _PAGES, _PARAMS, _bf16, _call, _empty, _f32, _i32, _list, _strides, _table, _table_args

_ROWS = struct.Struct("@P3q2i").pack   # attn_rows as bytes
_MOST = 2 ** 31 - 1   # what the library's 32-bit counts hold


def _weights(weights, rows, heads, keys, index):
    shape = weights.shape
    if weights.dtype is not _f32 or weights.get_device() != index or len(shape) != 3 \
            or shape[0] != rows or shape[1] != heads or shape[2] < keys \
            or (weights.stride(2) != 1 and shape[2] > 1):
        raise ValueError("weights must be fp32 [sequences, H_kv, at least max_pages * page_size] "
                         "on the tensors' device, contiguous along the last axis")
    step, head, _ = weights.stride()
    return weights.data_ptr(), step, head


def attention_key_weights(q, k_pages, page_table, cache_lens, lse, weights, *, k_scales=None,
                          k_descale=1.0, scale=None, causal=True, add=True, ws=None):
    """Adds to `weights` what attention weight the query rows give each cached key
    (see attn_key_weights in include/attn.h).

    q: [B, H, n_q, d] bf16 and lse fp32 [B, H, n_q], the query rows of a decode step
    and the logsumexps that it returned (a step of many rows: an observation
    window); k_pages: bf16 [num_pages, H_kv, page_size, d], or the codes of a cache
    in 4 bits with k_scales and k_descale; page_table, cache_lens, scale, causal as in
    that step; weights: fp32 [B, H_kv, max_pages * page_size or more]: entry [b, h, j]
    of each cached key j grows by the sum of its probabilities over the rows of
    head group h (add=False: becomes that sum).  Returns weights.
    """
    shape, index = q.shape, q.get_device()
    if q.dtype is not _bf16 or len(shape) != 4:
        raise TypeError("q must be bf16 [B, H, n_q, d]")
    B, H, n_q, d = shape
    dense = q.is_contiguous()
    qs = ((H or 1) * n_q * d, n_q * d, d) if dense else _strides(q)[:3]
    cache = keys = 0
    ks = (0, 0, 0)
    if k_scales is not None:
        cache, pages = _cache(k_pages, k_scales, k_descale, index, "keys")
    else:
        pages = k_pages.shape
        if k_pages.dtype is not _bf16 or k_pages.get_device() != index:
            raise TypeError("k_pages must be bf16 on q's device, or codes with k_scales")
        if len(pages) != 4:
            raise ValueError("k_pages must be [num_pages, H_kv, page_size, d]")
        keys = k_pages.data_ptr()
        ks = ((pages[1] or 1) * pages[2] * d, pages[2] * d, d) if k_pages.is_contiguous() \
            else _strides(k_pages)[:3]
    num_pages, H_kv, page_size, cols = pages
    if cols != d or H_kv < (1 if H else 0) or (H_kv and H % H_kv):
        raise ValueError("the keys must have q's d and an H_kv that divides its H")
    if lse.shape != shape[:3] or not lse.is_contiguous() or lse.dtype is not _f32 \
            or lse.get_device() != index:
        raise ValueError("lse must be a contiguous fp32 [B, H, n_q] on q's device")
    table, row, width, lens = _table(page_table, cache_lens, B, index, page_size)
    w = _weights(weights, B, H_kv, width * page_size, index)
    p = _PARAMS(B, H, width * page_size, d, 0, d ** -0.5 if scale is None else scale,
                1 if causal else 0, 0.0, 0, 0, lens, 0, 0, *qs, H_kv, 0, *ks, 0.0, 0.0, 0.0, 0)
    g = _PAGES(table, row, width, page_size, num_pages, 0)
    _call(lib().attn_key_weights, None, (),
          (p, n_q, g, q.data_ptr(), keys, cache, lse.data_ptr(), *w, 1 if add else 0), q.device,
          ws, "attn_key_weights")
    return weights


def pages_evict(pools, page_table, cache_lens, refs, weights, seqs, new_lens, *, recent=0,
                page_size, ws=None):
    """Sequence seqs[i] shrinks to new_lens[i] keys: every head keeps its last
    `recent` keys and of the others those with the largest weights, in their
    order (see attn_pages_evict).

    pools: buffers [num_pages, H_kv, page_size, ...] (keys, values; of a cache in 4
    bits codes and scales); weights: fp32 [rows, H_kv, max_pages * page_size or
    more], which move along with the keys (those behind the new length become 0);
    page_table, cache_lens, refs as in pages_extend; all in place.  Returns slots,
    int32 [n, H_kv, weights' last axis]: where the key now in place j was before, -1
    from the new length on; -2 throughout where the sequence was refused, because a page
    to be written is shared or the state is wrong (reported by check()).
    """
    t = _table_args(page_table, cache_lens, refs, page_size)
    index, P = refs.get_device(), refs.shape[0]
    if weights.dim() != 3:
        raise ValueError("weights must be [rows, H_kv, keys]")
    heads = weights.shape[1]
    w = _weights(weights, page_table.shape[0], heads, page_table.shape[1] * page_size, index)
    if weights.shape[2] > _MOST:
        raise ValueError("weights: more than 2^31 - 1 keys")
    recent = max(-1, min(recent, _MOST))   # (as many as there are; a negative one is refused)
    lead, rows = (P, heads, page_size), b""
    for x in pools:
        shape, n = x.shape, x.element_size()   # n: bytes of a row
        if x.get_device() != index or len(shape) < 4 or shape[:3] != lead:
            raise ValueError("pools must be [num_pages, H_kv, page_size, ...] on the table's device")
        if x.is_contiguous():
            for size in shape[3:]:
                n *= size
            steps = heads * page_size * n, page_size * n, n
        else:
            s, item = _strides(x), n
            for size, step in zip(reversed(shape[3:]), reversed(s[3:])):
                if size != 1 and step * item != n:
                    raise ValueError("a pool's row must be one contiguous block of memory")
                n *= size
            steps = s[0] * item, s[1] * item, s[2] * item
        rows += _ROWS(x.data_ptr(), *steps, n, 0)
    a, n = _list(seqs, refs.device, "seqs")
    b, m = _list(new_lens, refs.device, "new_lens")
    if n != m:
        raise ValueError("seqs and new_lens must have the same length")
    slots = _empty((n, heads, weights.shape[2]), dtype=_i32, device=refs.device)
    c = lib()
    _call(c.attn_pages_evict, c.attn_pages_evict_workspace_size, (t, heads, n, rows, len(pools)),
          (t, rows, len(pools), heads, *w, weights.shape[2], a, b, n, recent, slots.data_ptr()),
          refs.device, ws, "attn_pages_evict")
    return slots
