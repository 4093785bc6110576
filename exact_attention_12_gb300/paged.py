"""Python binding of the paged-cache calls: argument marshalling only.

As in api.py every step of the computation runs in the CUDA library, on the
current stream of the tensors' device.  A decode step on a short cache takes
a few microseconds on the device, so the calls here do little per call: one
structure is filled and one library function called, and the workspace's size
is asked for only when the one at hand is too small.
"""

import math
import struct

import torch

from . import _abi
from ._abi import check_status, lib
from .api import _workspaces, workspace

# The C structures (attn_params, attn_pages, attn_page_table) as bytes, which
# ctypes passes as a pointer: a third of the time of filling a ctypes.Structure.
_PARAMS = struct.Struct("@5ifif2Q2P4q2i3q3fi").pack
_PAGES = struct.Struct("@Pq4i").pack
_TABLE = struct.Struct("@PqPP4i").pack

_ROPE = 64   # columns of a latent vector beside its d_v value columns


_empty, _empty_like, _bf16, _f32, _i32 = (torch.empty, torch.empty_like, torch.bfloat16,
                                          torch.float32, torch.int32)


def _public_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


# the current stream's handle without the stream object around it (2 us), and
# the current device without a look at whether CUDA is initialised
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_stream)
_current = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(fn, size_fn, size_args, args, device, ws, what):
    """fn(*args, ws pointer, bytes, stream) on `device`, with the caller's
    workspace or the device's shared one, which grows (to what `size_fn` says)
    when the call finds it too small."""
    index = device.index
    if index is None or device.type != "cuda":
        raise ValueError(f"{what}: tensors must be on a CUDA device")
    if _current() != index:
        with torch.cuda.device(device):
            return _call(fn, size_fn, size_args, args, device, ws, what)
    stream = _stream(index)
    if ws is None:
        w = _workspaces.get(("cuda", index))   # (what workspace() would look up)
        if w is None:
            w = workspace(device, 256)
        st = fn(*args, w.data_ptr(), w.numel(), stream)
        if st == _abi.ATTN_ERR_WORKSPACE:
            need = size_fn(*size_args) if size_fn else 256
            if need == 0:
                check_status(_abi.ATTN_ERR_INVALID_ARG, what)
            w = workspace(device, need)
            st = fn(*args, w.data_ptr(), w.numel(), stream)
    else:
        if ws.device != device or not ws.is_contiguous():
            raise ValueError(f"{what}: ws must be contiguous, on the tensors' device")
        st = fn(*args, ws.data_ptr(), ws.numel() * ws.element_size(), stream)
    if st:
        check_status(st, what)


def _int32(t, index, dim, what):
    if t.dtype is not _i32 or t.get_device() != index or t.ndim != dim \
            or not (t.is_contiguous() or t.stride(-1) == 1):
        raise ValueError(f"{what} must be a {dim}-dimensional int32 tensor on the tensors' device, "
                         "contiguous along its last axis")


def _table(table, cache_lens, B, index, page_size):
    """Pointers, row stride and width of a page table with B rows."""
    _int32(table, index, 2, "page_table")
    _int32(cache_lens, index, 1, "cache_lens")
    rows, width = table.shape
    if rows != B or cache_lens.shape[0] != B:
        raise ValueError("page_table and cache_lens must have a row per sequence")
    if width * page_size > 1 << 30:
        raise ValueError("page_table: more than 2^30 keys per row")
    return table.data_ptr(), (table.stride(0) if rows > 1 else width), width, cache_lens.data_ptr()


def _strides(t):
    """Strides of a tensor; an axis of one element or none, over which nothing
    strides, has the value it has in a contiguous tensor."""
    shape = t.shape
    if not t.is_contiguous():
        s = list(t.stride())
        if s[-1] != 1 and shape[-1] > 1:
            raise ValueError("the last axis must be contiguous")
    else:
        s = [1] * len(shape)
        for i in range(len(shape) - 2, -1, -1):
            s[i] = s[i + 1] * (shape[i + 1] or 1)
        return s
    inner = shape[-1]
    for i in range(len(shape) - 2, -1, -1):
        if shape[i] <= 1:
            s[i] = inner
        inner = max(inner, s[i] * shape[i])
    return s


def attention_decode_paged(q, k_pages, v_pages, page_table, cache_lens, *, scale=None, causal=True,
                           shared_len=0, out=None, lse=None, ws=None):
    """The decode step of attention_decode against a paged cache (see
    attn_decode_paged in include/attn.h).

    q: [B, H, n_q, d] bf16; k_pages, v_pages: [num_pages, H_kv, page_size, d]
    bf16, with like strides, H_kv dividing H and page_size a power of two from
    16 on; page_table: int32 [B, max_pages]: key j of sequence b is row
    j % page_size of page page_table[b, j // page_size]; cache_lens: int32 [B].
    shared_len: a multiple of page_size; the first shared_len keys of all
    sequences (of a shorter one, all it has) lie in the same pages and are
    attended once for the whole batch, which pays from about B * H_kv = 32 on.
    A table no wider than the longest sequence needs (page_table[:, :most]) is
    faster where all are short.  Returns (o, lse) with o like
    q and lse fp32 [B, H, n_q].  A page index outside the cache is reported by
    check().
    """
    shape, pages, index = q.shape, k_pages.shape, q.get_device()
    if not (q.dtype is k_pages.dtype is v_pages.dtype is _bf16) \
            or not index == k_pages.get_device() == v_pages.get_device():
        raise TypeError("q, k_pages and v_pages must be bf16 on one device")
    if len(shape) != 4 or len(pages) != 4 or pages != v_pages.shape or pages[3] != shape[3]:
        raise ValueError("q must be [B, H, n_q, d], k_pages and v_pages "
                         "[num_pages, H_kv, page_size, d]")
    B, H, n_q, d = shape
    num_pages, H_kv, page_size, _ = pages
    if H_kv < (1 if H else 0) or (H_kv and H % H_kv):
        raise ValueError("H_kv must divide q's H")
    if k_pages.is_contiguous() and v_pages.is_contiguous():
        ks = ((H_kv or 1) * page_size * d, page_size * d, d)
    else:
        ks = _strides(k_pages)
        if ks != _strides(v_pages):
            raise ValueError("k_pages and v_pages must share strides")
    device = q.device
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
                1 if causal else 0, 0.0, 0, 0, lens, 0, 0, *qs, H_kv, 0, *ks[:3], 0.0, 0.0, 0.0, 0)
    g = _PAGES(table, row, width, page_size, num_pages, shared_len)
    c = lib()
    _call(c.attn_decode_paged, c.attn_decode_paged_workspace_size, (p, n_q, g),
          (p, n_q, g, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), out.data_ptr(),
           lse.data_ptr()), device, ws, "attn_decode_paged")
    return out, lse


def attention_decode_latent(q, c_pages, page_table, cache_lens, *, scale, d_v=512, causal=True,
                            out=None, lse=None, ws=None):
    """The decode step of latent attention in its absorbed form, against a
    paged cache of latent vectors (see attn_decode_latent in include/attn.h).

    q: [B, H, n_q, d_v + 64] bf16; c_pages: [num_pages, page_size, d_v + 64]
    bf16: a cached vector is the key of every head, its first d_v columns (256
    or 512) the value; page_table, cache_lens as in attention_decode_paged.
    `scale` has no default: it belongs to the heads' width before the
    projections were folded in.  Returns (o, lse): o [B, H, n_q, d_v] bf16,
    contiguous, and lse fp32 [B, H, n_q].
    """
    device, shape, pages, cols = q.device, q.shape, c_pages.shape, d_v + _ROPE
    index = q.get_device()
    if not (q.dtype is c_pages.dtype is _bf16) or c_pages.get_device() != index:
        raise TypeError("q and c_pages must be bf16 on one device")
    if len(shape) != 4 or len(pages) != 3 or shape[3] != cols or pages[2] != cols:
        raise ValueError(f"q must be [B, H, n_q, d_v + {_ROPE}], c_pages "
                         f"[num_pages, page_size, d_v + {_ROPE}]")
    B, H, n_q, _ = shape
    num_pages, page_size, _ = pages
    if out is None:
        out = _empty((B, H, n_q, d_v), dtype=_bf16, device=device)
    elif out.shape != (B, H, n_q, d_v) or not out.is_contiguous() or out.dtype is not _bf16 \
            or out.get_device() != index:
        raise ValueError("out must be a contiguous bf16 [B, H, n_q, d_v] on q's device")
    lse = _lse(lse, shape, device)
    cs, qs = _strides(c_pages), _strides(q)
    table, row, width, lens = _table(page_table, cache_lens, B, index, page_size)
    p = _PARAMS(B, H, width * page_size, d_v, 0, scale, 1 if causal else 0, 0.0, 0, 0, lens, 0, 0,
                *qs[:3], 1, 0, cs[0], cs[0], cs[1], 0.0, 0.0, 0.0, 0)
    g = _PAGES(table, row, width, page_size, num_pages, 0)
    c = lib()
    _call(c.attn_decode_latent, c.attn_decode_latent_workspace_size, (p, n_q, g),
          (p, n_q, g, q.data_ptr(), c_pages.data_ptr(), out.data_ptr(), lse.data_ptr()), device,
          ws, "attn_decode_latent")
    return out, lse


def _lse(lse, shape, device):
    if lse is None:
        return _empty(shape[:3], dtype=_f32, device=device)
    if lse.shape != shape[:3] or not lse.is_contiguous() or lse.dtype is not _f32 \
            or lse.device != device:
        raise ValueError("lse must be a contiguous fp32 [B, H, n_q] on q's device")
    return lse


# ------------------------------------------------------------------- upkeep --

def _table_args(page_table, cache_lens, refs, page_size):
    index = refs.get_device()
    _int32(refs, index, 1, "refs")
    rows = page_table.shape[0]
    table, row, width, lens = _table(page_table, cache_lens, rows, index, page_size)
    return _TABLE(table, row, lens, refs.data_ptr(), rows, width, page_size, refs.shape[0])


def _pool_args(pools, num_pages, device):
    """attn_pool of each page buffer [num_pages, ...]: a page's elements must
    fill one contiguous block, in whatever order its axes have."""
    got = []
    for t in pools:
        shape = t.shape
        if t.device != device or len(shape) < 2 or shape[0] != num_pages:
            raise ValueError("pools must be tensors [num_pages, ...] on the table's device")
        item = t.element_size()
        page = math.prod(shape[1:])
        if t.is_contiguous():
            step = page
        else:
            n = 1   # the page's axes in the order of their strides
            for stride, size in sorted(zip(t.stride()[1:], shape[1:])):
                if size != 1 and stride != n:
                    raise ValueError("a page must be one contiguous block of memory")
                n *= size
            step = t.stride(0) if num_pages > 1 else page
        got += (t.data_ptr(), step * item, page * item)
    return struct.pack(f"@{len(got)}q", *got)   # attn_pool: three 64-bit words


def _list(t, device, what):
    _int32(t, -1 if device.type == "cpu" else device.index, 1, what)
    return t.data_ptr(), t.shape[0]


def pages_copy(pools, src, dst, *, ws=None):
    """Page dst[i] of every page buffer in `pools` ([num_pages, ...] tensors)
    becomes a copy of page src[i]; src, dst: int32 on the device, dst without
    repeats and apart from src."""
    if not pools:
        return
    dev, num_pages = pools[0].device, pools[0].shape[0]
    arr = _pool_args(pools, num_pages, dev)
    s, n = _list(src, dev, "src")
    d, m = _list(dst, dev, "dst")
    if n != m:
        raise ValueError("src and dst must have the same length")
    _call(lib().attn_pages_copy, None, (), (arr, len(pools), num_pages, s, d, n), dev, ws,
          "attn_pages_copy")


def pages_extend(page_table, cache_lens, refs, seqs, new_lens, *, page_size, ws=None):
    """Sequence seqs[i] grows to new_lens[i] keys, taking the lowest free pages
    (see attn_pages_extend).  page_table int32 [rows, max_pages], cache_lens
    int32 [rows], refs int32 [num_pages], in place."""
    t = _table_args(page_table, cache_lens, refs, page_size)
    s, n = _list(seqs, refs.device, "seqs")
    d, m = _list(new_lens, refs.device, "new_lens")
    if n != m:
        raise ValueError("seqs and new_lens must have the same length")
    c = lib()
    _call(c.attn_pages_extend, c.attn_pages_workspace_size, (t, n), (t, s, d, n), refs.device, ws,
          "attn_pages_extend")


def pages_fork(pools, page_table, cache_lens, refs, parents, children, *, page_size, ws=None):
    """Row children[i] (empty) becomes a copy of sequence parents[i]: full
    pages shared, a part-filled last page copied in every buffer of `pools`
    (see attn_pages_fork).  Returns the new pages, int32 like parents: -1 where
    none was needed, -2 where the fork was not made."""
    t = _table_args(page_table, cache_lens, refs, page_size)
    arr = _pool_args(pools, refs.shape[0], refs.device)
    a, n = _list(parents, refs.device, "parents")
    b, m = _list(children, refs.device, "children")
    if n != m:
        raise ValueError("parents and children must have the same length")
    new = torch.empty_like(parents)
    c = lib()
    _call(c.attn_pages_fork, c.attn_pages_workspace_size, (t, n),
          (t, arr, len(pools), a, b, n, new.data_ptr()), refs.device, ws, "attn_pages_fork")
    return new


def pages_free(page_table, cache_lens, refs, seqs, *, page_size, ws=None):
    """The sequences `seqs` give back their pages (see attn_pages_free)."""
    t = _table_args(page_table, cache_lens, refs, page_size)
    s, n = _list(seqs, refs.device, "seqs")
    _call(lib().attn_pages_free, None, (), (t, s, n), refs.device, ws,
          "attn_pages_free")


def pages_compact(pools, page_table, cache_lens, refs, *, page_size, ws=None):
    """Moves the pages in use to the front of the buffers `pools`, tables and
    counts with them (see attn_pages_compact).  Returns where each page now is,
    int32 [num_pages], -1 for a free one."""
    t = _table_args(page_table, cache_lens, refs, page_size)
    arr = _pool_args(pools, refs.shape[0], refs.device)
    moved = torch.empty_like(refs)
    c = lib()
    _call(c.attn_pages_compact, c.attn_pages_workspace_size, (t, 0),
          (t, arr, len(pools), moved.data_ptr()), refs.device, ws, "attn_pages_compact")
    return moved
