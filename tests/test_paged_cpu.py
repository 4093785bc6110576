"""The paged-cache calls' host side, without a GPU: struct layouts, argument
checks of the C interface and of the Python binding, and the definitions they
are tested against.  Every refusal comes before anything touches a device."""

import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import attention, paged

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def abi():
    from exact_attention_12_gb300 import build, _abi
    if not os.path.exists(build.LIB_PATH):
        build.build()
    return _abi


@pytest.mark.parametrize("cls,name", [("AttnPages", "attn_pages"),
                                      ("AttnPageTable", "attn_page_table"),
                                      ("AttnPool", "attn_pool")])
def test_struct_layouts(abi, tmp_path, cls, name):
    c = getattr(abi, cls)
    names = [f[0] for f in c._fields_]
    src = tmp_path / "layout.c"
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "attn.h"', 'int main(void) {',
             f'  printf("size %zu\\n", sizeof({name}));']
    lines += [f'  printf("{n} %zu\\n", offsetof({name}, {n}));' for n in names]
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                           str(exe)])
    got = dict(x.split() for x in subprocess.check_output([str(exe)], text=True).splitlines())
    assert int(got["size"]) == ctypes.sizeof(c)
    for n in names:
        assert int(got[n]) == getattr(c, n).offset, n


@pytest.mark.parametrize("fmt,cls", [("_PARAMS", "AttnParams"), ("_PAGES", "AttnPages"),
                                     ("_TABLE", "AttnPageTable")])
def test_packed_structures_are_the_declared_ones(abi, fmt, cls):
    # the binding packs the structures as bytes: the same as the ctypes mirror filled in order
    from exact_attention_12_gb300 import paged as binding
    c = getattr(abi, cls)
    values = [float(i + 1) if t is ctypes.c_float else i + 1 for i, (_, t) in enumerate(c._fields_)]
    got = getattr(binding, fmt)(*values)
    assert len(got) == ctypes.sizeof(c)
    s = c.from_buffer_copy(got)
    assert [getattr(s, n) for n, _ in c._fields_] == values


def _decode(abi, latent=False, **kw):
    p, g = abi.AttnParams(), abi.AttnPages()
    d = 512 if latent else 64
    cols = d + 64 if latent else d
    p.B, p.H, p.N, p.d, p.scale = 2, 4, 256, d, 0.125
    p.stride_b, p.stride_h, p.stride_n = 4 * cols, cols, cols
    p.H_kv = 1 if latent else 2
    p.kv_stride_b, p.kv_stride_h, p.kv_stride_n = 2 * 32 * cols, 32 * cols, cols
    p.key_lens = 0x1000
    g.table, g.table_stride, g.max_pages, g.page_size, g.num_pages = 0x1000, 8, 8, 32, 20
    n_q = kw.pop("n_q", 1)
    for k, v in kw.items():
        setattr(g if hasattr(g, k) else p, k, v)
    return p, g, n_q


def _status(abi, p, g, n_q, latent=False, ws=0x1000, nb=1 << 40, ptr=0x1000):
    """The call with host-only stand-ins for pointers; it must not launch."""
    lib, f = abi.lib(), ctypes.c_void_p(ptr)
    pp, gp = ctypes.byref(p), ctypes.byref(g)
    if latent:
        return lib.attn_decode_latent(pp, n_q, gp, f, f, f, f, ws, nb, None)
    return lib.attn_decode_paged(pp, n_q, gp, f, f, f, f, f, ws, nb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=96), 2), (dict(dtype=1), 2), (dict(dtype=9), 1), (dict(scale=0.0), 1),
    (dict(scale=float("nan")), 1), (dict(dropout_p=0.1), 2), (dict(block_mask=0x1000), 2),
    (dict(key_lens=None), 1), (dict(n_q=0), 1), (dict(H_kv=3), 1), (dict(n_q=9000), 2),
    (dict(B=-1), 1), (dict(reserved=1), 1), (dict(N=255), 1), (dict(table=None), 1),
    (dict(page_size=24, N=192), 1), (dict(page_size=8, N=64), 1), (dict(page_size=0, N=0), 1),
    (dict(max_pages=-1), 1), (dict(num_pages=-1), 1), (dict(table_stride=7), 1),
    (dict(shared_len=16), 1), (dict(shared_len=-32), 1), (dict(shared_len=288), 1),
    (dict(stride_n=60), 1), (dict(stride_n=56), 1), (dict(kv_stride_n=56), 1),
    (dict(kv_stride_h=0), 1), (dict(kv_stride_b=-64), 1), (dict(stride_h=4), 1),
    (dict(max_pages=1 << 16, table_stride=1 << 16, page_size=32768, N=0), 2),
    (dict(B=1 << 29, n_q=2), 2), (dict(B=1 << 20, max_pages=1 << 15, table_stride=1 << 15,
                                       N=1 << 20), 2),
])
def test_paged_decode_refusals(abi, kw, status):
    p, g, n_q = _decode(abi, **kw)
    assert abi.lib().attn_decode_paged_workspace_size(ctypes.byref(p), n_q, ctypes.byref(g)) == 0
    assert _status(abi, p, g, n_q) == status, abi.lib().attn_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(d=128), 2), (dict(H_kv=2), 1), (dict(shared_len=32), 2), (dict(n_q=20000), 2),
    (dict(kv_stride_n=512), 1), (dict(stride_n=512), 1), (dict(page_size=48, N=384), 1),
    (dict(key_lens=None), 1), (dict(dtype=2), 2),
])
def test_latent_decode_refusals(abi, kw, status):
    p, g, n_q = _decode(abi, latent=True, **kw)
    assert abi.lib().attn_decode_latent_workspace_size(ctypes.byref(p), n_q, ctypes.byref(g)) == 0
    assert _status(abi, p, g, n_q, latent=True) == status, abi.lib().attn_last_error()


@pytest.mark.parametrize("latent", [False, True])
def test_pointers_and_workspace_are_checked(abi, latent):
    lib = abi.lib()
    p, g, n_q = _decode(abi, latent=latent)
    size = lib.attn_decode_latent_workspace_size if latent else lib.attn_decode_paged_workspace_size
    need = size(ctypes.byref(p), n_q, ctypes.byref(g))
    assert need > 256
    assert _status(abi, p, g, n_q, latent, nb=need - 1) == abi.ATTN_ERR_WORKSPACE
    assert _status(abi, p, g, n_q, latent, ws=None) == abi.ATTN_ERR_WORKSPACE
    assert _status(abi, p, g, n_q, latent, ws=0x1010) == abi.ATTN_ERR_WORKSPACE
    assert _status(abi, p, g, n_q, latent, nb=need, ptr=0x1008) == abi.ATTN_ERR_INVALID_ARG
    assert _status(abi, p, g, n_q, latent, nb=need, ptr=None) == abi.ATTN_ERR_INVALID_ARG
    # the workspace does not grow with the caches beyond the CTAs' partials
    p2, g2, _ = _decode(abi, latent=latent, max_pages=4096, table_stride=4096, N=4096 * 32)
    p3, g3, _ = _decode(abi, latent=latent, max_pages=8192, table_stride=8192, N=8192 * 32)
    assert size(ctypes.byref(p2), n_q, ctypes.byref(g2)) == size(ctypes.byref(p3), n_q,
                                                                 ctypes.byref(g3))
    p.B = 0   # nothing to do
    assert _status(abi, p, g, n_q, latent, nb=1 << 20, ptr=None) == abi.ATTN_OK


@pytest.mark.parametrize("latent", [False, True])
@pytest.mark.parametrize("none", [dict(H=0), dict(B=0, key_lens=None, table=None), dict(B=0, H=0)])
def test_no_heads_or_no_sequences(abi, latent, none):
    # nothing to do, whatever the pointers are; the sizes divide by nothing
    p, g, n_q = _decode(abi, latent=latent, **none)
    lib = abi.lib()
    size = lib.attn_decode_latent_workspace_size if latent else lib.attn_decode_paged_workspace_size
    assert size(ctypes.byref(p), n_q, ctypes.byref(g)) >= 256
    assert _status(abi, p, g, n_q, latent, nb=1 << 20, ptr=None) == abi.ATTN_OK


def _table(abi, **kw):
    t = abi.AttnPageTable(0x1000, 8, 0x1000, 0x1000, 4, 8, 16, 20)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(max_pages=9), dict(page_size=0),
                                dict(page_size=1 << 28), dict(num_pages=-1), dict(table=None),
                                dict(lens=None), dict(refs=None)])
def test_page_table_refusals(abi, kw):
    lib, t = abi.lib(), _table(abi, **kw)
    tp, f, big = ctypes.byref(t), 0x1000, 1 << 40
    assert lib.attn_pages_workspace_size(tp, 1) == 0
    assert lib.attn_pages_extend(tp, f, f, 1, f, big, None) == abi.ATTN_ERR_INVALID_ARG
    assert lib.attn_pages_free(tp, f, 1, f, big, None) == abi.ATTN_ERR_INVALID_ARG
    assert lib.attn_pages_fork(tp, None, 0, f, f, 1, f, f, big, None) == abi.ATTN_ERR_INVALID_ARG
    assert lib.attn_pages_compact(tp, None, 0, f, f, big, None) == abi.ATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("pool", [(None, 64, 64), (0x1008, 64, 64), (0x1000, 64, 0),
                                  (0x1000, 72, 64), (0x1000, 64, 40), (0x1000, 32, 64)])
def test_pool_refusals(abi, pool):
    lib, t = abi.lib(), _table(abi)
    tp, f, big = ctypes.byref(t), 0x1000, 1 << 40
    arr = (abi.AttnPool * 1)(abi.AttnPool(*pool))
    assert lib.attn_pages_copy(arr, 1, 4, f, f, 1, f, big, None) == abi.ATTN_ERR_INVALID_ARG
    assert lib.attn_pages_fork(tp, arr, 1, f, f, 1, f, f, big, None) == abi.ATTN_ERR_INVALID_ARG
    assert lib.attn_pages_compact(tp, arr, 1, f, f, big, None) == abi.ATTN_ERR_INVALID_ARG


def test_page_list_and_workspace_refusals(abi):
    lib, t = abi.lib(), _table(abi)
    tp, f, big = ctypes.byref(t), 0x1000, 1 << 40
    need = lib.attn_pages_workspace_size(tp, 3)
    assert need >= 256 + 4 * (4 + 2 * 3 + 20)
    assert lib.attn_pages_extend(tp, f, f, 3, f, need - 1, None) == abi.ATTN_ERR_WORKSPACE
    assert lib.attn_pages_extend(tp, f, f, 3, None, big, None) == abi.ATTN_ERR_WORKSPACE
    assert lib.attn_pages_extend(tp, f, f, 3, 0x1010, big, None) == abi.ATTN_ERR_WORKSPACE
    assert lib.attn_pages_extend(tp, None, f, 3, f, big, None) == abi.ATTN_ERR_INVALID_ARG
    assert lib.attn_pages_extend(tp, f, f, -1, f, big, None) == abi.ATTN_ERR_INVALID_ARG
    assert lib.attn_pages_fork(tp, None, 0, f, f, 1, None, f, big, None) == abi.ATTN_ERR_INVALID_ARG
    assert lib.attn_pages_fork(tp, None, -1, f, f, 1, f, f, big, None) == abi.ATTN_ERR_INVALID_ARG
    assert lib.attn_pages_compact(tp, None, 0, None, f, big, None) == abi.ATTN_ERR_INVALID_ARG
    for st in (lib.attn_pages_extend(tp, None, None, 0, f, big, None),
               lib.attn_pages_free(tp, None, 0, f, big, None),
               lib.attn_pages_fork(tp, None, 0, None, None, 0, None, f, big, None),
               lib.attn_pages_copy(None, 0, 4, f, f, 0, f, big, None)):
        assert st == abi.ATTN_OK   # nothing to do


def test_binding_refusals():
    import exact_attention_12_gb300 as ea
    bf = torch.bfloat16
    q, k = torch.zeros(2, 4, 1, 64, dtype=bf), torch.zeros(5, 2, 16, 64, dtype=bf)
    t, n = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    ok = dict(q=q, k_pages=k, v_pages=k, page_table=t, cache_lens=n)
    for kw, err in [(dict(q=q.float()), TypeError), (dict(q=q[0]), ValueError),
                    (dict(v_pages=k[:, :1]), ValueError),
                    (dict(k_pages=k[..., :32], v_pages=k[..., :32]), ValueError),
                    (dict(q=q[:, :3]), ValueError), (dict(page_table=t.long()), ValueError),
                    (dict(page_table=t[:1]), ValueError), (dict(cache_lens=n[:1]), ValueError),
                    (dict(page_table=t.repeat(1, 2)[:, ::2]), ValueError),
                    (dict(page_table=t.repeat(1, 1 << 25)), ValueError),
                    (dict(v_pages=k.transpose(1, 2).contiguous().transpose(1, 2)), ValueError),
                    (dict(out=q.float()), ValueError), (dict(lse=torch.zeros(2, 4)), ValueError),
                    (dict(), ValueError)]:   # the last: not on a GPU
        with pytest.raises(err):
            ea.attention_decode_paged(**{**ok, **kw})
    c, qc = torch.zeros(5, 16, 576, dtype=bf), torch.zeros(2, 4, 1, 576, dtype=bf)
    for kw in (dict(q=q), dict(c_pages=c[..., :512]), dict(d_v=256), dict(out=qc), dict()):
        with pytest.raises(ValueError):
            ea.attention_decode_latent(**{**dict(q=qc, c_pages=c, page_table=t, cache_lens=n,
                                                 scale=0.1), **kw})
    r, s = torch.zeros(5, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        ea.pages_fork([k[:4]], t, n, r, s, s, page_size=16)     # a pool of another size
    with pytest.raises(ValueError):
        ea.pages_fork([k[..., :32]], t, n, r, s, s, page_size=16)   # pages with holes
    with pytest.raises(ValueError):
        ea.pages_fork([k], t, n, r, s, s[:1], page_size=16)
    with pytest.raises(ValueError):
        ea.pages_extend(t, n, r, s, s.long(), page_size=16)
    with pytest.raises(ValueError):
        ea.pages_free(t, n[:1], r, s, page_size=16)
    with pytest.raises(ValueError):
        ea.pages_copy([k], s, s[:1])


def test_the_paged_definition_is_the_contiguous_one():
    rng = np.random.default_rng(0)
    B, H, H_kv, n_q, d, size = 2, 4, 2, 3, 8, 4
    k, v = rng.normal(size=(2, 7, H_kv, size, d))
    q = rng.normal(size=(B, H, n_q, d))
    table, lens = np.array([[3, 0, 6], [5, 3, 1]]), [10, 2]
    for causal in (True, False):
        O, L, A = paged.paged_decode(q, k, v, table, lens, 0.3, causal)
        K, V = (np.stack([np.concatenate([x[p] for p in row], axis=1) for row in table])
                for x in (k, v))
        want = attention.decode_forward(q, K, V, 0.3, lens, causal)
        assert np.allclose(O, want[0], atol=1e-12) and np.allclose(L, want[1], atol=1e-12)
        assert (A >= np.abs(O) - 1e-12).all()
    c = rng.normal(size=(7, size, d))
    O, L, _ = paged.latent_decode(q, c, table, lens, 0.3, 5)
    K = np.stack([np.concatenate([c[p] for p in row]) for row in table])[:, None]
    O2, L2 = attention.decode_forward(q, K, K, 0.3, lens)
    assert np.allclose(O, O2[..., :5], atol=1e-12) and np.allclose(L, L2, atol=1e-12)
