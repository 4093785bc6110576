"""What the calls on compact caches promise beside ordinary results, as far as it shows
without a GPU: what they refuse before anything is launched."""

import ctypes

import pytest
import torch

from tests.test_fp4_cpu import FAKE, _Seen, _step, _tensors, lib  # noqa: F401


def _table(**kw):
    from exact_attention_12_gb300 import _abi
    t = _abi.AttnPageTable()
    t.table = t.lens = t.refs = FAKE
    t.table_stride = t.max_pages = 4
    t.rows, t.page_size, t.num_pages = 2, 16, 8
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def _evict(lib, t, weights=FAKE, row=128, head=64, width=64, slots=FAKE, n=1, pools=(), heads=2):  # noqa: F811
    from exact_attention_12_gb300 import _abi
    rows = (_abi.AttnRows * max(1, len(pools)))(*pools)
    return lib.attn_pages_evict(ctypes.byref(t), rows, len(pools), heads, weights, row, head, width,
                                FAKE, FAKE, n, 0, slots, FAKE, 1 << 30, None)


@pytest.mark.parametrize("kw", [dict(max_pages=0, table_stride=0, table=None), dict(num_pages=0), dict()])
def test_an_eviction_without_slots_is_refused(lib, kw):  # noqa: F811
    # (a table without pages as well: every call writes slots as far as `width`)
    assert _evict(lib, _table(**kw), slots=None) == 1 and b"NULL" in lib.attn_last_error()


# What several sequences and heads would write to, row and head entries apart; 64 entries each,
# 3 sequences, 2 heads.
APART = [(128, 64), (64, 192), (1000, 64), (500, 3000), (129, 64), (64, 193)]
SHARED = [(64, 64), (127, 64), (64, 191), (100, 100), (64, 128), (1 << 62, 63)]


@pytest.mark.parametrize("row,head,ok", [(*x, True) for x in APART] + [(*x, False) for x in SHARED])
def test_weights_of_one_place_are_refused(lib, row, head, ok):  # noqa: F811
    p, g, c, _ = _step(lib, B=3, N=64, max_pages=4, table_stride=4)
    # (without a workspace: what passes the checks of the weights is refused there)
    st = lib.attn_key_weights(ctypes.byref(p), 1, ctypes.byref(g), FAKE, None, ctypes.byref(c), FAKE, FAKE,
                              row, head, 1, None, 0, None)
    assert st == (5 if ok else 1) and (ok or b"apart" in lib.attn_last_error())
    assert _evict(lib, _table(rows=3), row=row, head=head, n=0) == (0 if ok else 1)
    assert ok or b"apart" in lib.attn_last_error()


# Page, head and row steps of pools with 3 pages, 2 heads, 16 rows of 128 bytes.
POOLS = [((4096, 2048, 128), True), ((4096, 128, 256), True), ((128, 6144, 384), True),
         ((5000, 2108, 132), True), ((1 << 40, 1 << 33, 1 << 20), True),
         # (16 rows 132 apart take 15 * 132 + 128 = 2108)
         ((5000, 2100, 132), False), ((128, 128, 128), False), ((4096, 1024, 128), False), ((2048, 4096, 128), False),
         ((4096, 128, 128), False), ((4096, 2048, 256), False), ((256, 4096, 256), False)]


@pytest.mark.parametrize("steps,ok", POOLS)
def test_pools_whose_rows_share_memory_are_refused(lib, steps, ok):  # noqa: F811
    from exact_attention_12_gb300 import _abi
    pool = _abi.AttnRows(FAKE, *steps, 128, 0)
    t = _table(num_pages=3)
    assert _evict(lib, t, pools=(pool,), n=0) == (0 if ok else 1)
    assert ok or b"apart" in lib.attn_last_error()
    size = lib.attn_pages_evict_workspace_size(ctypes.byref(t), 2, 1, ctypes.byref(pool), 1)
    assert (size > 256) is ok


# Page and head bytes of codes and scales: 4 pages, 2 heads of 16 keys with 32 and 4 bytes.
CACHES = [(dict(), True), (dict(code_page=512, code_head=2048, scale_page=64, scale_head=256), True),
          (dict(code_page=512), False), (dict(code_head=496), False), (dict(code_page=1008), False),
          (dict(scale_head=48), False), (dict(scale_page=64), False), (dict(code_page=512, code_head=2032), False)]


@pytest.mark.parametrize("kw,ok", CACHES)
@pytest.mark.parametrize("which", ["keys", "values"])
def test_a_store_into_places_of_one_another_is_refused(lib, kw, ok, which):  # noqa: F811
    p, g, c, _ = _step(lib, **kw)
    good = _step(lib)[2]
    pair = (c, good) if which == "keys" else (good, c)
    # (without a workspace: what passes the checks of the cache is refused there)
    st = lib.attn_pages_store_fp4(ctypes.byref(p), ctypes.byref(g), None, FAKE, FAKE,
                                  *(ctypes.byref(x) for x in pair), None, 0, None)
    assert st == (5 if ok else 1) and (ok or b"apart" in lib.attn_last_error())
    # reading is free to
    assert lib.attn_pages_load_fp4(ctypes.byref(p), ctypes.byref(g), None, *(ctypes.byref(x) for x in pair),
                                   FAKE, FAKE, None, 0, None) == 5


# ---------------------------------------------------------------- binding --

@pytest.mark.parametrize("recent,want", [(0, 0), (7, 7), (2 ** 31, 2 ** 31 - 1), (2 ** 32, 2 ** 31 - 1),
                                         (2 ** 32 + 3, 2 ** 31 - 1), (2 ** 64, 2 ** 31 - 1), (-2 ** 32, -1),
                                         (-2 ** 31 - 1, -1)])
def test_recent_is_not_taken_modulo_32_bits(lib, monkeypatch, recent, want):  # noqa: F811
    import exact_attention_12_gb300 as ea
    seen, x = _Seen(monkeypatch), _tensors()
    ea.pages_evict((x["kc"],), x["t"], x["lens"], x["refs"], x["w"], x["lens"][:1], x["lens"][:1],
                   recent=recent, page_size=16)
    assert ctypes.c_int32(seen.calls[0][1][11]).value == want


def test_weights_wider_than_32_bits_count_are_refused(lib, monkeypatch):  # noqa: F811
    import exact_attention_12_gb300 as ea
    seen, x = _Seen(monkeypatch), _tensors()
    call = lambda width: ea.pages_evict(  # noqa: E731
        (), x["t"], x["lens"], x["refs"], torch.empty(2, 2, width, device="meta"), x["lens"][:0],
        x["lens"][:0], page_size=16)
    call(2 ** 31 - 1)
    for width in (2 ** 31, 2 ** 32 + 64):
        with pytest.raises(ValueError):
            call(width)
    assert len(seen.calls) == 1
