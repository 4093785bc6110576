"""What the calls on compact caches promise beside ordinary results, as far as it shows
without a GPU: what they refuse before anything is launched."""

import ctypes

import pytest

from tests.test_fp4_cpu import FAKE, lib  # noqa: F401


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
