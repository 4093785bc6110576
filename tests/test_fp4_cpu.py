"""The cache format in 4 bits and the calls around it, as far as it shows without a
GPU: the definitions themselves, the argument checks, the binding."""

import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import eviction, fp4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ------------------------------------------------------------ definitions --

def test_scales_are_torchs_e4m3():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(fp4.SCALES, want, equal_nan=True)


@pytest.mark.parametrize("descale", [1.0, 2.0 ** -9, 24.0 / 2688, 0.3])
def test_codes_are_the_nearest(descale):
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.normal(size=(40, 64)) * 3).to(torch.bfloat16).double().numpy()
    codes, scales = fp4.encode(x, descale)
    y = fp4.decode(codes, scales, descale)
    unit = np.repeat(fp4.SCALES[scales], 16, -1) * float(np.float32(descale))
    # no other code of the block's scale is nearer
    others = np.abs(x[..., None] - unit[..., None] * np.concatenate([fp4.LEVELS, -fp4.LEVELS]))
    assert np.all(np.abs(x - y) <= others.min(-1) * (1 + 1e-12) + 1e-300)
    # and what was stored is stored as itself
    again, s2 = fp4.encode(y, descale)
    full = np.abs(y.reshape(40, -1, 16)).max(-1) == 6 * unit.reshape(40, -1, 16)[..., 0]
    same = (again == codes).reshape(40, 4, 8).all(-1) | ~full
    assert same.all() and full.any() and np.array_equal(s2[full], scales[full])


def test_ties_go_to_the_even_code():
    x = np.zeros((1, 16))
    x[0, :9] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5]
    codes, scales = fp4.encode(x, 1.0)
    got = np.stack([codes & 15, codes >> 4], -1).reshape(1, 16)
    assert fp4.SCALES[scales[0, 0]] == 1
    assert got[0, :9].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 14]
    # a scale half way between two: 6 * 17 / 16 is as far from 1 as from 9 / 8
    _, s = fp4.encode(np.full((1, 16), 6 * 17 / 16), 1.0)
    assert s[0, 0] % 2 == 0 and fp4.SCALES[s[0, 0]] == 1


def test_largest_smallest_and_not_numbers():
    x = np.zeros((6, 16))
    x[0] = 1e30                 # saturates
    x[1, 3] = np.inf
    x[2, 5] = np.nan
    x[3] = 2.0 ** -40           # below the smallest scale
    x[4] = 6 * 2.0 ** -9        # the smallest scale
    codes, scales = fp4.encode(x, 1.0)
    y = fp4.decode(codes, scales, 1.0)
    assert np.all(y[0] == 2688) and y[1, 3] == 2688 and np.all(y[1, :3] == 0)
    assert np.isnan(y[2]).all()
    assert np.all(y[3] == 0) and np.all(codes[3] == 0)
    assert np.all(y[4] == 6 * 2.0 ** -9) and np.all(y[5] == 0)


def test_what_a_head_keeps():
    w = np.array([3.0, 1, 2, 2, 2, 9, 0, 0])
    assert eviction.kept(w, 8, 4, 2).tolist() == [0, 5, 6, 7]
    assert eviction.kept(w, 8, 5, 2).tolist() == [0, 2, 5, 6, 7]     # of equal ones the first
    assert eviction.kept(w, 8, 3, 8).tolist() == [5, 6, 7]
    assert eviction.kept(w, 8, 0, 2).tolist() == []
    w[1] = np.nan
    assert eviction.kept(w, 8, 2, 0).tolist() == [1, 5]


# -------------------------------------------------------- argument checks --

@pytest.fixture(scope="module")
def lib():
    from exact_attention_12_gb300 import _abi, build
    build.build()
    return _abi.lib()


@pytest.mark.parametrize("name,size", [("attn_fp4", 56), ("attn_rows", 40)])
def test_struct_layouts(lib, name, size, tmp_path):
    from exact_attention_12_gb300 import _abi, eviction as ev, fp4 as binding
    mirror = {"attn_fp4": _abi.AttnFp4, "attn_rows": _abi.AttnRows}[name]
    packed = {"attn_fp4": lambda: binding._FP4(*[0] * 6, 0.0, 0),
              "attn_rows": lambda: ev._ROWS(*[0] * 6)}[name]()
    src = tmp_path / "layout.c"
    fields = [f[0] for f in mirror._fields_]
    src.write_text("\n".join(
        ["#include <stddef.h>", "#include <stdio.h>", '#include "attn.h"', "int main(void) {",
         f'printf("%zu\\n", sizeof({name}));'] +
        [f'printf("%zu\\n", offsetof({name}, {f}));' for f in fields] + ["return 0; }"]))
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                           str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)], text=True).split()]
    assert got[0] == ctypes.sizeof(mirror) == len(packed) == size
    assert got[1:] == [getattr(mirror, f).offset for f in fields]


FAKE = 0x10000


def _step(lib, **kw):
    """A decode step's arguments; kw changes fields by name."""
    from exact_attention_12_gb300 import _abi
    d = kw.pop("d", 64)
    p, g, c = _abi.AttnParams(), _abi.AttnPages(), _abi.AttnFp4()
    p.B, p.H, p.H_kv, p.N, p.d, p.scale = 1, 4, 2, 32, d, 1.0
    p.stride_b, p.stride_h, p.stride_n = 4 * d, d, d
    p.kv_stride_b, p.kv_stride_h, p.kv_stride_n = 64 * d, 16 * d, d
    p.key_lens = g.table = FAKE
    g.table_stride = g.max_pages = 2
    g.page_size, g.num_pages = 16, 4
    c.codes = c.scales = FAKE
    c.code_head, c.scale_head = 16 * d // 2, 16 * d // 16
    c.code_page, c.scale_page, c.descale = 2 * c.code_head, 2 * c.scale_head, 1.0
    other = {}
    for k, v in kw.items():
        for s in (p, g, c):
            if k in (f[0] for f in s._fields_):
                setattr(s, k, v)
                break
        else:
            other[k] = v
    return p, g, c, other


BAD = [(dict(d=96), 2), (dict(B=-1), 1), (dict(H_kv=3), 1), (dict(scale=0.0), 1),
       (dict(scale=float("nan")), 1), (dict(n_q=0), 1), (dict(key_lens=None), 1),
       (dict(table=None), 1), (dict(page_size=24), 1), (dict(page_size=8), 1),
       (dict(shared_len=16), 2), (dict(N=48), 1), (dict(table_stride=1), 1), (dict(stride_n=60), 1),
       (dict(stride_h=12), 1), (dict(n_q=16384), 2), (dict(dtype=1), 2), (dict(dtype=9), 1),
       (dict(dropout_p=0.5), 2), (dict(reserved2=1), 1)]
BAD_CACHE = [(dict(descale=0.0), 1), (dict(descale=-1.0), 1), (dict(descale=float("nan")), 1),
             (dict(descale=float("inf")), 1), (dict(descale=2.0 ** -120), 1), (dict(codes=None), 1),
             (dict(scales=FAKE + 8), 1), (dict(code_page=24), 1), (dict(scale_head=0), 1),
             (dict(code_page=1 << 33), 2)]


@pytest.mark.parametrize("kw,status", BAD + BAD_CACHE)
def test_decode_refuses(lib, kw, status):
    p, g, c, o = _step(lib, **kw)
    n_q = o.get("n_q", 1)
    st = lib.attn_decode_fp4(ctypes.byref(p), n_q, ctypes.byref(g), FAKE, ctypes.byref(c),
                             ctypes.byref(c), FAKE, FAKE, FAKE, 1 << 30, None)
    assert st == status, lib.attn_last_error()
    if (kw, status) in BAD:
        assert lib.attn_decode_fp4_workspace_size(ctypes.byref(p), n_q, ctypes.byref(g)) == 0


@pytest.mark.parametrize("kw,status", BAD + BAD_CACHE + [(dict(k=FAKE), 1), (dict(stride_w=-1), 1)])
def test_key_weights_refuse(lib, kw, status):
    p, g, c, o = _step(lib, **kw)
    st = lib.attn_key_weights(ctypes.byref(p), o.get("n_q", 1), ctypes.byref(g), FAKE, o.get("k"),
                              ctypes.byref(c), FAKE, FAKE, o.get("stride_w", 64), 32, 1, FAKE, 256,
                              None)
    assert st == status, lib.attn_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(d=32), 2), (dict(B=-1), 1), (dict(N=-1), 1), (dict(kv_stride_n=60), 1),
    (dict(kv_stride_h=0), 1), (dict(key_lens=None), 1), (dict(page_size=17), 1)] + BAD_CACHE)
@pytest.mark.parametrize("call", ["store", "load"])
def test_store_and_load_refuse(lib, call, kw, status):
    p, g, c, _ = _step(lib, **kw)
    c = ctypes.byref(c)
    kv = (FAKE, FAKE)
    args = (*kv, c, c) if call == "store" else (c, c, *kv)
    st = getattr(lib, f"attn_pages_{call}_fp4")(ctypes.byref(p), ctypes.byref(g), None, *args, FAKE,
                                                256, None)
    assert st == status, lib.attn_last_error()


def test_a_small_or_missing_workspace_is_refused(lib):
    p, g, c, _ = _step(lib)
    need = lib.attn_decode_fp4_workspace_size(ctypes.byref(p), 1, ctypes.byref(g))
    for ws, n in ((None, need), (FAKE + 16, need), (FAKE, need - 1)):
        assert lib.attn_decode_fp4(ctypes.byref(p), 1, ctypes.byref(g), FAKE, ctypes.byref(c),
                                   ctypes.byref(c), FAKE, FAKE, ws, n, None) == 5
        assert lib.attn_pages_store_fp4(ctypes.byref(p), ctypes.byref(g), None, FAKE, FAKE,
                                        ctypes.byref(c), ctypes.byref(c), ws, min(n, 255), None) == 5


def _evict(lib, pools=1, heads=2, width=64, n=1, recent=0, ws=FAKE, ws_bytes=1 << 30, **kw):
    from exact_attention_12_gb300 import _abi
    t, r = _abi.AttnPageTable(), _abi.AttnRows()
    t.table = t.lens = t.refs = FAKE
    t.table_stride = t.max_pages = 4
    t.rows, t.page_size, t.num_pages = 2, 16, 8
    r.base, r.page_stride, r.head_stride, r.row_stride, r.row_bytes = FAKE, 4096, 2048, 128, 128
    for k, v in kw.items():
        setattr(t if k in (f[0] for f in t._fields_) else r, k, v)
    rows = (_abi.AttnRows * max(1, pools))(*[r] * pools)
    size = lib.attn_pages_evict_workspace_size(ctypes.byref(t), heads, n, rows, pools)
    st = lib.attn_pages_evict(ctypes.byref(t), rows, pools, heads, FAKE, 128, 64, width, FAKE, FAKE,
                              n, recent, FAKE, ws, ws_bytes, None)
    return st, size


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(page_size=20), 1), (dict(table_stride=3), 1), (dict(table=None), 1),
    (dict(refs=None), 1), (dict(heads=-1), 1), (dict(n=-1), 1), (dict(pools=17), 2),
    (dict(row_bytes=130), 1), (dict(row_bytes=0), 1), (dict(row_stride=64), 1),
    (dict(head_stride=2), 1), (dict(base=FAKE + 2), 1), (dict(reserved=1), 1),
    (dict(row_bytes=32772, row_stride=32772), 2), (dict(recent=-1), 1), (dict(width=63), 1),
    (dict(ws=None), 5), (dict(ws=FAKE + 4), 5), (dict(ws_bytes=64), 5), (dict(heads=1 << 20), 2)])
def test_evict_refuses(lib, kw, status):
    st, size = _evict(lib, **kw)
    assert st == status, lib.attn_last_error()
    assert _evict(lib, n=0)[0] == 0 and _evict(lib, heads=0)[0] == 0 and _evict(lib)[1] > 256


@pytest.mark.parametrize("kw", [dict(page_stride=0), dict(page_stride=124), dict(head_stride=0)])
def test_evict_refuses_pools_that_overlap(lib, kw):
    assert _evict(lib, **kw)[0] == 1
    one = dict(num_pages=1) if "page_stride" in kw else dict(heads=1)
    assert _evict(lib, **{**kw, **one, "n": 0})[0] == 0     # nothing to be apart from


@pytest.mark.parametrize("row,head", [(0, 64), (128, 0), (63, 64), (128, 63), (0, 0)])
def test_weights_that_overlap_are_refused(lib, row, head):
    # (what expand() gives: several would add to one entry)
    from exact_attention_12_gb300 import _abi
    p, g, c, _ = _step(lib, B=2, N=64, max_pages=4, table_stride=4)
    call = lambda: lib.attn_key_weights(  # noqa: E731
        ctypes.byref(p), 1, ctypes.byref(g), FAKE, None, ctypes.byref(c), FAKE, FAKE, row, head, 1, FAKE,
        256, None)
    assert call() == 1 and b"apart" in lib.attn_last_error()
    p.B = 0     # passes every check, and enqueues nothing, where only one is left
    assert call() == (1 if head < 64 else 0)
    t = _abi.AttnPageTable()
    t.table = t.lens = t.refs = FAKE
    t.table_stride = t.max_pages = 4
    t.rows, t.page_size, t.num_pages = 2, 16, 8
    call = lambda: lib.attn_pages_evict(  # noqa: E731
        ctypes.byref(t), None, 0, 2, FAKE, row, head, 64, FAKE, FAKE, 0, 0, FAKE, FAKE, 1 << 20, None)
    assert call() == 1 and b"strides" in lib.attn_last_error()
    t.rows = 1
    assert call() == (1 if head < 64 else 0)


def test_the_waits_can_be_stalled(lib):
    from exact_attention_12_gb300 import _abi
    for which in (_abi.ATTN_STALL_EVICT_READ, _abi.ATTN_STALL_WEIGHTS_SUM, _abi.ATTN_STALL_FP4_VALUES,
                  _abi.ATTN_STALL_NONE):
        assert lib.attn_debug_stall(which, 1) == _abi.ATTN_OK


# ---------------------------------------------------------------- binding --

class _Seen:
    """Stands in for the library call; the C checks see the arguments."""

    def __init__(self, monkeypatch):
        from exact_attention_12_gb300 import eviction as ev, fp4 as binding
        self.calls = []
        for m in (ev, binding):
            monkeypatch.setattr(m, "_call", self)

    def __call__(self, fn, size_fn, size_args, args, device, ws, what):
        self.calls.append((what, args))
        if size_fn is not None:
            assert size_fn(*size_args) >= 256


def _tensors(B=2, H=4, H_kv=2, d=64, P=5, page=16, n=3):
    i32 = dict(dtype=torch.int32)
    return dict(
        q=torch.zeros(B, H, 1, d, dtype=torch.bfloat16), kc=torch.zeros(P, H_kv, page, d // 2, dtype=torch.uint8),
        ks=torch.zeros(P, H_kv, page, d // 16).to(torch.float8_e4m3fn), t=torch.zeros(B, n, **i32),
        lens=torch.zeros(B, **i32), refs=torch.zeros(P, **i32), lse=torch.zeros(B, H, 1),
        w=torch.zeros(B, H_kv, n * page), k=torch.zeros(B, H_kv, 2, d, dtype=torch.bfloat16))


@pytest.mark.parametrize("kw", [dict(), dict(B=0), dict(H=0, H_kv=0), dict(P=0), dict(n=0), dict(d=128)])
def test_the_binding_reaches_the_library(lib, monkeypatch, kw):
    import exact_attention_12_gb300 as ea
    seen, x = _Seen(monkeypatch), _tensors(**kw)
    cache = (x["kc"], x["ks"], x["kc"], x["ks"], x["t"], x["lens"])
    ea.attention_decode_fp4(x["q"], *cache)
    ea.pages_store_fp4(x["k"], x["k"], *cache)
    k, v = ea.pages_load_fp4(*cache, 7)
    assert k.shape == v.shape == (x["t"].shape[0], x["kc"].shape[1], 7, x["q"].shape[3])
    ea.attention_key_weights(x["q"], x["kc"], x["t"], x["lens"], x["lse"], x["w"], k_scales=x["ks"])
    ea.pages_evict((x["kc"], x["ks"]), x["t"], x["lens"], x["refs"], x["w"], x["lens"][:1],
                   x["lens"][:1], page_size=16)
    assert len(seen.calls) == 5


def test_the_binding_refuses(monkeypatch):
    import exact_attention_12_gb300 as ea
    _Seen(monkeypatch)
    x = _tensors()
    q, kc, ks, t, lens, w, lse = (x[k] for k in ("q", "kc", "ks", "t", "lens", "w", "lse"))
    dec = ea.attention_decode_fp4
    with pytest.raises(TypeError):
        dec(q.float(), kc, ks, kc, ks, t, lens)
    with pytest.raises(TypeError):
        dec(q, kc, ks.float(), kc, ks, t, lens)
    with pytest.raises(ValueError):
        dec(q, kc[..., :16], ks, kc, ks, t, lens)
    with pytest.raises(ValueError):
        dec(q, kc, ks, kc[:4], ks[:4], t, lens)
    with pytest.raises(ValueError):
        dec(q[:, :3], kc, ks, kc, ks, t, lens)
    with pytest.raises(ValueError):
        dec(q, kc, ks, kc, ks, t[:1], lens)
    with pytest.raises(ValueError):   # rows of a page apart
        wide = torch.zeros(5, 2, 16, 40, dtype=torch.uint8)[..., :32]
        dec(q, wide, ks, kc, ks, t, lens)
    with pytest.raises(ValueError):
        ea.pages_store_fp4(x["k"], x["k"][:, :, :1], kc, ks, kc, ks, t, lens)
    with pytest.raises(ValueError):
        ea.pages_store_fp4(x["k"], x["k"], kc, ks, kc, ks, t, lens, counts=lens.long())
    kw = ea.attention_key_weights
    with pytest.raises(ValueError):
        kw(q, kc, t, lens, lse, w[:, :, :40], k_scales=ks)
    with pytest.raises(ValueError):
        kw(q, kc, t, lens, lse[:, :2], w, k_scales=ks)
    with pytest.raises(TypeError):
        kw(q, kc, t, lens, lse, w)
    with pytest.raises(ValueError):
        ea.pages_evict((kc.transpose(1, 2),), t, lens, x["refs"], w, lens, lens, page_size=16)
    with pytest.raises(ValueError):
        ea.pages_evict((kc,), t, lens, x["refs"], w, lens, lens[:1], page_size=16)
    with pytest.raises(ValueError):
        ea.pages_evict((kc[..., ::2],), t, lens, x["refs"], w, lens, lens, page_size=16)
