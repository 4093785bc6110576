"""Python binding of the calls on caches in 4 bits: argument marshalling only.

A cache in 4 bits is two tensors for the keys and two for the values: codes
uint8 [num_pages, H_kv, page_size, d / 2] (two E2M1 codes a byte, the even column
in the low four bits) and scales float8_e4m3fn [num_pages, H_kv, page_size,
d / 16], with one factor, `descale`, for each tensor: the values are
descale * scale * code (see attn_fp4 in include/attn.h).  A head's rows of a page
must follow one another; pages and heads may be apart.
"""

import struct

import torch

from .api import _FP8
from ._abi import lib
from .paged import _PAGES, _PARAMS, _bf16, _call, _empty, _empty_like, _i32, _lse, _strides, _table

_FP4 = struct.Struct("@PP4qfi").pack   # attn_fp4 as bytes
_u8 = torch.uint8


def _cache(codes, scales, descale, index, what):
    """attn_fp4 of a cache tensor, and its (num_pages, H_kv, page_size, d)."""
    if codes.dtype is not _u8 or scales.dtype is not _FP8 \
            or not index == codes.get_device() == scales.get_device():
        raise TypeError(f"{what}: codes must be uint8 and scales float8_e4m3fn, on one device")
    if codes.ndim != 4 or scales.ndim != 4:
        raise ValueError(f"{what}: codes and scales must have four dimensions")
    P, H, size, n = scales.shape
    if codes.shape != (P, H, size, 8 * n):
        raise ValueError(f"{what}: codes must be [num_pages, H_kv, page_size, d / 2], scales "
                         "[num_pages, H_kv, page_size, d / 16]")
    if codes.is_contiguous() and scales.is_contiguous():
        # (a cache without heads has no strides to speak of)
        head = size * n
        page = (H or 1) * head
        return _FP4(codes.data_ptr(), scales.data_ptr(), 8 * page, 8 * head, page, head, descale,
                    0), (P, H, size, 16 * n)
    cs, ss = _strides(codes), _strides(scales)
    if (cs[2], ss[2]) != (8 * n, n) and size > 1:
        raise ValueError(f"{what}: a head's rows of a page must follow one another")
    return _FP4(codes.data_ptr(), scales.data_ptr(), cs[0], cs[1], ss[0], ss[1], descale,
                0), (P, H, size, 16 * n)


def _both(k_codes, k_scales, v_codes, v_scales, k_descale, v_descale, index):
    k, shape = _cache(k_codes, k_scales, k_descale, index, "keys")
    v, other = _cache(v_codes, v_scales, v_descale, index, "values")
    if shape != other:
        raise ValueError("keys and values must have the same shape")
    return k, v, shape


def attention_decode_fp4(q, k_codes, k_scales, v_codes, v_scales, page_table, cache_lens, *,
                         k_descale=1.0, v_descale=1.0, scale=None, causal=True, out=None,
                         lse=None, ws=None):
    """The decode step of attention_decode_paged against a cache in 4 bits (see
    attn_decode_fp4 in include/attn.h).

    q: [B, H, n_q, d] bf16, H_kv dividing H; the cache as the module describes;
    page_table, cache_lens as in attention_decode_paged.  Returns (o, lse) with
    o like q and lse fp32 [B, H, n_q].  A page index outside the cache is reported
    by check().
    """
    shape, index, device = q.shape, q.get_device(), q.device
    k, v, (num_pages, H_kv, page_size, d) = _both(k_codes, k_scales, v_codes, v_scales, k_descale,
                                                  v_descale, index)
    if q.dtype is not _bf16:
        raise TypeError("q must be bf16")
    if len(shape) != 4 or shape[3] != d:
        raise ValueError("q must be [B, H, n_q, d] with the cache's d")
    B, H, n_q, _ = shape
    if H_kv < (1 if H else 0) or (H_kv and H % H_kv):
        raise ValueError("H_kv must divide q's H")
    dense = q.is_contiguous()
    qs = ((H or 1) * n_q * d, n_q * d, d) if dense else _strides(q)[:3]
    if out is None:
        out = _empty_like(q) if dense else torch.empty_strided(shape, q.stride(), dtype=_bf16,
                                                               device=device)
    elif out.shape != shape or _strides(out) != _strides(q) or out.dtype is not _bf16 \
            or out.get_device() != index:
        raise ValueError("out must be like q")
    lse = _lse(lse, shape, device)
    table, row, width, lens = _table(page_table, cache_lens, B, index, page_size)
    p = _PARAMS(B, H, width * page_size, d, 0, d ** -0.5 if scale is None else scale,
                1 if causal else 0, 0.0, 0, 0, lens, 0, 0, *qs, H_kv, 0, 0, 0, 0, 0.0, 0.0, 0.0, 0)
    g = _PAGES(table, row, width, page_size, num_pages, 0)
    c = lib()
    _call(c.attn_decode_fp4, c.attn_decode_fp4_workspace_size, (p, n_q, g),
          (p, n_q, g, q.data_ptr(), k, v, out.data_ptr(), lse.data_ptr()), device, ws,
          "attn_decode_fp4")
    return out, lse


def _copy_args(B, n, strides, cache, page_table, cache_lens, counts, index):
    """attn_params, attn_pages and the counts' pointer of a store or load."""
    num_pages, H_kv, page_size, d = cache
    if counts is not None and (counts.dtype is not _i32 or counts.get_device() != index
                               or counts.shape != (B,) or not counts.is_contiguous()):
        raise ValueError("counts must be a contiguous int32 [B] on the tensors' device")
    table, row, width, lens = _table(page_table, cache_lens, B, index, page_size)
    p = _PARAMS(B, H_kv, n, d, 0, 1.0, 0, 0.0, 0, 0, lens, 0, 0, d, d, d, H_kv, 0, *strides,
                0.0, 0.0, 0.0, 0)
    return p, _PAGES(table, row, width, page_size, num_pages, 0), \
        0 if counts is None else counts.data_ptr()


def pages_store_fp4(k, v, k_codes, k_scales, v_codes, v_scales, page_table, cache_lens, *,
                    k_descale=1.0, v_descale=1.0, counts=None, ws=None):
    """Stores the newest tokens of each sequence in a cache of 4 bits (see
    attn_pages_store_fp4).

    k, v: [B, H_kv, n, d] bf16 with like strides; token t < counts[b] (None: n)
    becomes the cached key and value at position cache_lens[b] - counts[b] + t: the
    lengths are those after pages_extend.  descale: about the largest value over
    2688 (6 * 448, the format's largest); a block of 16 columns keeps its relative
    precision down to 2^-14 of that.
    """
    shape, index = k.shape, k.get_device()
    kc, vc, cache = _both(k_codes, k_scales, v_codes, v_scales, k_descale, v_descale, index)
    if not (k.dtype is v.dtype is _bf16) or v.get_device() != index:
        raise TypeError("k and v must be bf16 on one device")
    _, H_kv, _, d = cache
    if len(shape) != 4 or shape != v.shape or shape[1] != H_kv or shape[3] != d:
        raise ValueError("k and v must be [B, H_kv, n, d] with the cache's H_kv and d")
    B, _, n, _ = shape
    if k.is_contiguous() and v.is_contiguous():
        strides = (H_kv or 1) * (n or 1) * d, (n or 1) * d, d
    else:
        strides = _strides(k)[:3]
        if strides != _strides(v)[:3]:
            raise ValueError("k and v must share strides")
    p, g, m = _copy_args(B, n, strides, cache, page_table, cache_lens, counts, index)
    _call(lib().attn_pages_store_fp4, None, (), (p, g, m, k.data_ptr(), v.data_ptr(), kc, vc),
          k.device, ws, "attn_pages_store_fp4")


def pages_load_fp4(k_codes, k_scales, v_codes, v_scales, page_table, cache_lens, n, *,
                   k_descale=1.0, v_descale=1.0, counts=None, ws=None):
    """The newest tokens of each sequence out of a cache of 4 bits: (k, v), bf16
    [B, H_kv, n, d], token t < counts[b] (None: n) that of position cache_lens[b] -
    counts[b] + t, zeros elsewhere.  With counts = cache_lens: whole sequences."""
    index = k_codes.get_device()
    kc, vc, cache = _both(k_codes, k_scales, v_codes, v_scales, k_descale, v_descale, index)
    _, H_kv, _, d = cache
    B = page_table.shape[0]
    k = _empty((B, H_kv, n, d), dtype=_bf16, device=k_codes.device)
    v = _empty_like(k)
    p, g, m = _copy_args(B, n, ((H_kv or 1) * (n or 1) * d, (n or 1) * d, d), cache, page_table,
                         cache_lens, counts, index)
    _call(lib().attn_pages_load_fp4, None, (), (p, g, m, kc, vc, k.data_ptr(), v.data_ptr()),
          k_codes.device, ws, "attn_pages_load_fp4")
    return k, v
