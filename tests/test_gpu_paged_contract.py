"""What the paged-cache calls promise beyond ordinary results: waits that run
out, wrong state, caches and batches of nothing."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import paged as oracle
from tests.helpers import np64
from tests.test_gpu_paged import WIDE, _hold, _poison, _run, _table, ea  # noqa: F401
from tests.test_gpu_pages import Cache, _i

pytestmark = pytest.mark.gpu


# ------------------------------------------------------- waits that run out --

def _used_workspace():
    """A workspace whose header is zero and whose rest holds another call's data."""
    g = torch.Generator().manual_seed(1)
    ws = torch.randint(-2 ** 31, 2 ** 31, (1 << 24,), generator=g, dtype=torch.int64).to(torch.int32)
    ws[:64] = 0
    return ws.cuda()


def _stalled(stall, sites, call, want):
    """The call with one of its kernels stalled, then twice as it is."""
    from exact_attention_12_gb300 import _abi
    lib, ws = _abi.lib(), _used_workspace()
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert lib.attn_debug_stall(stall, 20_000_000) == _abi.ATTN_OK
    call(ws)
    assert lib.attn_check(ws.data_ptr(), stream) == _abi.ATTN_ERR_TIMEOUT
    msg = lib.attn_last_error().decode()
    assert int(msg.rsplit("wait site", 1)[1]) in sites, msg
    assert lib.attn_check(ws.data_ptr(), stream) == _abi.ATTN_OK   # read and cleared
    for _ in range(2):
        o, lse = call(ws)
        assert lib.attn_check(ws.data_ptr(), stream) == _abi.ATTN_OK
        _hold(o, lse, want)


# The balanced split with a merge per segment and per CTA, one CTA's 64 rows, a
# cluster per segment, a slot per segment; with a prefix, stalled in either
# kernel: its own merge, and the decode kernel's
@pytest.mark.parametrize("kernel,lens,H,H_kv,shared,room", [
    ("paged", [9000, 40, 0, 700], 4, 1, 0, WIDE), ("paged", [300, 0, 41] * 30, 8, 4, 0, WIDE),
    ("paged", [700, 900], 64, 1, 0, WIDE), ("paged", [300, 1, 33], 4, 2, 0, 0),
    ("paged", [40, 0, 77] * 30, 8, 4, 0, 0)] + [
    (kernel, *case) for kernel in ("paged", "prefix") for case in (
        ([5000, 4100, 1100], 4, 2, 1024, WIDE), ([1100, 1024, 1050], 4, 2, 1024, 0),
        ([300] * 90, 8, 4, 256, 0))])
def test_a_stalled_paged_step_ends_and_reports(ea, kernel, lens, H, H_kv, shared, room):
    from exact_attention_12_gb300 import _abi
    rng, g = np.random.default_rng(3), torch.Generator().manual_seed(3)
    table, P = _table(rng, lens, 16, shared=shared, room=room)
    k, v = (_poison(torch.randn(P, H_kv, 16, 64, generator=g).to(torch.bfloat16), table, lens, 16)
            for _ in range(2))
    q = torch.randn(len(lens), H, 1, 64, generator=g).to(torch.bfloat16)
    args = [x.cuda() for x in (q, k, v, torch.from_numpy(table),
                               torch.tensor(lens, dtype=torch.int32))]
    stall, sites = {"paged": (_abi.ATTN_STALL_PAGED_TILE, (60, 61)),
                    "prefix": (_abi.ATTN_STALL_PREFIX_SOFTMAX, range(62, 70))}[kernel]
    _stalled(stall, sites,
             lambda ws: ea.attention_decode_paged(*args, shared_len=shared, ws=ws),
             oracle.paged_decode(np64(q), np64(k), np64(v), table, lens, 0.125))


@pytest.mark.parametrize("lens,H,room", [([5000, 40, 0, 700], 16, WIDE), ([5000, 700], 128, WIDE),
                                         ([130, 0, 65] * 60, 8, WIDE), ([200, 1, 64], 40, 0)])
def test_a_stalled_latent_step_ends_and_reports(ea, lens, H, room):
    from exact_attention_12_gb300 import _abi
    rng, g = np.random.default_rng(4), torch.Generator().manual_seed(4)
    table, P = _table(rng, lens, 32, room=room)
    c = _poison(torch.randn(P, 32, 320, generator=g).to(torch.bfloat16), table, lens, 32)
    q = torch.randn(len(lens), H, 1, 320, generator=g).to(torch.bfloat16)
    args = [x.cuda() for x in (q, c, torch.from_numpy(table), torch.tensor(lens, dtype=torch.int32))]
    _stalled(_abi.ATTN_STALL_LATENT_SOFTMAX, range(70, 77),
             lambda ws: ea.attention_decode_latent(*args, scale=0.05, d_v=256, ws=ws),
             oracle.latent_decode(np64(q), np64(c), table, lens, 0.05, 256))


# ------------------------------------------------------------ rows of a CTA --

# 33 to 63 rows of a key/value head take four row tiles, the last of which may
# have none; 65 are a block of 33 and one of 32
@pytest.mark.parametrize("H,n_q", [(33, 1), (40, 1), (47, 1), (48, 1), (49, 1), (65, 1), (5, 7),
                                   (97, 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shared", [0, 64])
@pytest.mark.parametrize("room", [0, WIDE])
def test_row_tiles_without_rows(ea, H, n_q, d, shared, room):
    _run(ea, [shared + n for n in (300, 1, 170)], H, 1, n_q, d, 32, True, shared, seed=H, room=room)


# --------------------------------------------------------------- the prefix --

@pytest.mark.parametrize("lens", [[0, 300, 257], [100, 300, 90, 513], [0, 0, 90, 30], [64, 256, 256],
                                  [0] * 40 + [270] + [0] * 40 + [400]])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("room", [0, WIDE])
def test_a_prefix_is_read_where_a_sequence_holds_it(ea, lens, causal, room):
    """The first rows of a batch may be empty (padding, ended sequences) or end
    inside the prefix: their unused entries name nothing."""
    shared, page = 256, 32
    rng, g = np.random.default_rng(2), torch.Generator().manual_seed(2)
    table, P = _table(rng, lens, page, shared=shared, room=room)
    for b, n in enumerate(lens):
        table[b, -(-n // page):] = -1
    k, v = (_poison(torch.randn(P, 2, page, 64, generator=g).to(torch.bfloat16), table, lens, page)
            for _ in range(2))
    q = torch.randn(len(lens), 4, 2, 64, generator=g).to(torch.bfloat16)
    o, lse = ea.attention_decode_paged(q.cuda(), k.cuda(), v.cuda(), torch.from_numpy(table).cuda(),
                                       torch.tensor(lens, dtype=torch.int32).cuda(), causal=causal,
                                       shared_len=shared)
    ea.check()
    _hold(o, lse, oracle.paged_decode(np64(q), np64(k), np64(v), table, lens, 0.125, causal))


# --------------------------------------------------------------- wrong state --

def _reported(ea):
    from exact_attention_12_gb300 import _abi
    with pytest.raises(_abi.AttnError) as e:
        ea.check()
    assert e.value.status == _abi.ATTN_ERR_PAGE


def test_compact_reports_entries_that_name_no_page_in_use(ea):
    for wrong in ("free", 20, -1):
        c = Cache(np.random.default_rng(4), 6, 4, 20, 16, [20, 60, 5, 33])
        if wrong == "free":
            wrong = c.twin.refs.index(0)
        was = c.twin.table[1][2]
        c.table[1, 2] = wrong
        moved = ea.pages_compact(c.pools, *c.state, page_size=16)
        assert moved.cpu().tolist() == c.twin.compact(c.plain)
        _reported(ea)
        # the page that the entry had named moved with the others; the entry is as documented
        assert c.twin.table[1][2] == moved[was].item()
        c.twin.table[1][2] = wrong if not 0 <= wrong < 20 else -1
        c.same()


@pytest.mark.parametrize("at", [0, 2, 3])   # a full page, the last full one, the part-filled one
@pytest.mark.parametrize("wrong", ["free", "the lowest free", 30, -1, 1 << 30])
def test_forks_of_a_parent_with_a_wrong_page_are_not_made(ea, at, wrong):
    """Such a page has no count to raise, and one that is free may be handed out as new
    in the same call."""
    c = Cache(np.random.default_rng(5), 9, 5, 30, 16, [20, 60, 5, 33])
    unused = [p for p, r in enumerate(c.twin.refs) if r == 0]
    name = {"free": unused[3], "the lowest free": unused[0]}.get(wrong, wrong)
    c.table[1, at], c.twin.table[1][at] = name, name
    par, kid = [0, 1, 3, 1, 2], [4, 5, 6, 7, 8]
    new = ea.pages_fork(c.pools, *c.state, _i(par), _i(kid), page_size=16)
    want = c.twin.fork(par, kid, c.plain)
    assert want[1] == want[3] == -2 and new.cpu().tolist() == want
    _reported(ea)
    c.same()


def test_forks_of_a_parent_with_a_wrong_length_are_not_made(ea):
    for n in (-1, -16, 81, 1 << 30):
        c = Cache(np.random.default_rng(6), 6, 5, 30, 16, [20, 60])
        c.lens[1], c.twin.lens[1] = n, n
        new = ea.pages_fork(c.pools, *c.state, _i([0, 1]), _i([4, 5]), page_size=16)
        assert new.cpu().tolist() == c.twin.fork([0, 1], [4, 5], c.plain) and new[1] == -2
        _reported(ea)
        c.same()


# ------------------------------------------------------------------ nothing --

def test_caches_without_pages(ea):
    """As a serving program has them before it has decided how many pages there are."""
    i32 = dict(dtype=torch.int32, device="cuda")
    k, c = (torch.zeros(0, *s, dtype=torch.bfloat16, device="cuda") for s in ((2, 16, 64), (16, 320)))
    q, qc = (torch.ones(3, 4, 2, d, dtype=torch.bfloat16, device="cuda") for d in (64, 320))
    for width, len_ in ((0, 0), (4, 0), (2000, 0), (4, 40), (2000, 40)):
        t, n = torch.zeros(3, width, **i32), torch.full((3,), len_, **i32)
        for shared in (0, 32):
            if shared > width * 16:
                continue
            o, lse = ea.attention_decode_paged(q, k, k, t, n, shared_len=shared)
            assert torch.all(o == 0)   # keys that are named read as zeros
            _empty_or_named(ea, lse, len_)
        o, lse = ea.attention_decode_latent(qc, c, t, n, scale=0.1, d_v=256)
        assert torch.all(o == 0)
        _empty_or_named(ea, lse, len_)
    t, n, refs = torch.full((3, 4), -1, **i32), torch.zeros(3, **i32), torch.zeros(0, **i32)
    none = torch.zeros(0, **i32)
    pools = (k, c)
    assert ea.pages_compact(pools, t, n, refs, page_size=16).numel() == 0
    assert ea.pages_fork(pools, t, n, refs, none, none, page_size=16).numel() == 0
    assert ea.pages_fork(pools, t, n, refs, _i([0]), _i([2]), page_size=16).tolist() == [-1]
    ea.pages_copy(pools, none, none)
    ea.pages_free(t, n, refs, _i([0, 1]), page_size=16)
    ea.pages_extend(t, n, refs, _i([0]), _i([0]), page_size=16)
    ea.check()
    assert torch.all(t == -1) and torch.all(n == 0)
    n[1] = 20
    ea.pages_compact(pools, t, n, refs, page_size=16)
    _reported(ea)


def _empty_or_named(ea, lse, len_):
    if len_ == 0:
        assert torch.all(torch.isneginf(lse))
        ea.check()
    else:
        want = torch.tensor([[len_ - 1, len_]], dtype=torch.float64).log()   # scores of 0, causal
        assert (lse.cpu() - want).abs().max() <= 1e-5
        _reported(ea)


@pytest.mark.parametrize("H_kv", [0, 2])
def test_no_heads(ea, H_kv):
    i32 = dict(dtype=torch.int32, device="cuda")
    t, n = torch.zeros(3, 4, **i32), torch.full((3,), 20, **i32)
    k = torch.zeros(5, H_kv, 16, 64, dtype=torch.bfloat16, device="cuda")
    for n_q in (1, 2):
        o, lse = ea.attention_decode_paged(k.new_zeros(3, 0, n_q, 64), k, k, t, n)
        assert o.shape == (3, 0, n_q, 64) and lse.shape == (3, 0, n_q)
        o, lse = ea.attention_decode_latent(k.new_zeros(3, 0, n_q, 320), k.new_zeros(5, 16, 320), t,
                                            n, scale=0.1, d_v=256)
        assert o.shape == (3, 0, n_q, 256) and lse.shape == (3, 0, n_q)
    if H_kv == 0:   # heads that no key/value head serves
        with pytest.raises(ValueError):
            ea.attention_decode_paged(k.new_zeros(3, 4, 1, 64), k, k, t, n)
    ea.check()


# ------------------------------------------------------------------- status --

def test_check_sees_what_was_recorded_before_the_workspace_grew(ea):
    from exact_attention_12_gb300 import _abi
    k = torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16, device="cuda")
    t, n = _i([0, 9]).view(1, 2), _i([32])
    dev = q.device

    def grow():
        before = ea.workspace(dev, 256)
        assert ea.workspace(dev, before.numel() + 1).data_ptr() != before.data_ptr()

    def page():
        _reported(ea)
        ea.check()   # read and cleared

    ea.attention_decode_paged(q, k, k, t, n)
    grow()
    page()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ea.attention_decode_paged(q, k, k, t, n)
    grow()
    graph.replay()
    page()
    ea.attention_decode_paged(q, k, k, t, n)
    with pytest.raises(_abi.AttnError):
        ea.check(device="cuda")
    assert ea.workspace("cuda", 256).data_ptr() == ea.workspace(dev, 256).data_ptr()
    ea.check()
