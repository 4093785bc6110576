"""The attention weight of cached keys (attention_key_weights) and eviction by it
(pages_evict) against their definitions, and a run of the calls on compact caches
together, as a serving loop makes them.

Tolerances.  A weight is a sum of exp(S - L): S is a sum of d exact products in
fp32, off by at most (d + 8) 2^-24 T with T = c sum |q_c k_c|, the fused
multiply-add before the exponential by 2^-24 of |S| + |L| <= 2 T + |L|, ex2.approx
by 2^-22, the sum over R rows by R 2^-24: relative
((d + 8) T + 2 T + |L| + 4 + R) 2^-24 in all.  Eviction is whole numbers and copies:
equal.
"""

import ctypes

import numpy as np
import pytest
import torch

from oracle import eviction as oracle, fp4, paged
from tests.helpers import L_MAX_ABS, np64
from tests.test_gpu_fp4 import E4M3, _cache, _on_gpu
from tests.test_gpu_pages import Cache, _i
from tests.test_gpu_paged import WIDE, _pages, _table, ea  # noqa: F401

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------- weights --

def _weights(ea, lens, H, H_kv, n_q, d, page, packed=False, causal=True, add=True, seed=0,
             layout="hnd", room=0):
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    table, P = _table(rng, lens, page, room=room)
    q = torch.randn(len(lens), H, n_q, d, generator=g).to(torch.bfloat16)
    kw = dict(scale=d ** -0.5, causal=causal)
    if packed:
        codes, scales = _cache(rng, table, lens, P, H_kv, page, d)
        keys = fp4.decode(codes, scales, 2.0 ** -7)
        c, s = _on_gpu(codes, scales, layout)
        dev, kw2 = c, dict(k_scales=s, k_descale=2.0 ** -7)
        kw["scale"] *= 0.3
    else:
        k, dev = _pages(g, (P, H_kv, page, d), table, lens, layout)
        keys, kw2 = np64(k), {}
    t, ln = torch.from_numpy(table).cuda(), _i(lens)
    _, L, _ = paged.paged_decode(np64(q), keys, np.zeros(keys.shape[:3] + (1,)), table, lens,
                                 kw["scale"], causal)
    lse = torch.from_numpy(L).float()
    before = torch.rand(len(lens), H_kv, table.shape[1] * page + 5, generator=g)
    w = before.cuda()
    got = ea.attention_key_weights(q.cuda(), dev, t, ln, lse.cuda(), w, add=add, **kw, **kw2)
    torch.cuda.synchronize()
    ea.check()
    assert got is w
    want, T = oracle.key_weights(np64(q), keys, table, lens, np64(lse), kw["scale"], causal)
    R = H // H_kv * n_q
    big = np.abs(np.where(np.isfinite(L), L, 0)).max() if L.size else 0
    rel = ((d + 10) * T + big + 4 + R) * 2.0 ** -24
    w, before = np64(w), np64(before)
    for b, n in enumerate(lens):
        base = before[b, :, :n] if add else 0.0
        err = np.abs(w[b, :, :n] - base - want[b])
        assert np.all(err <= rel * want[b] + 2.0 ** -23 * (base + want[b]) + 1e-37), (b, err.max())
        assert np.array_equal(w[b, :, n:], before[b, :, n:])     # left as they were
    return w


@pytest.mark.parametrize("H,H_kv,n_q", [(2, 2, 1), (8, 1, 1), (9, 1, 1), (8, 2, 4), (17, 1, 1), (8, 1, 5),
                                         (16, 2, 33), (8, 1, 80)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("packed", [False, True])
def test_rows_and_widths(ea, H, H_kv, n_q, d, packed):  # noqa: F811
    # (8 x 80 rows of a head: more than one pass)
    _weights(ea, [300, 1, 33, 0, 129], H, H_kv, n_q, d, 16, packed, seed=H + n_q)


@pytest.mark.parametrize("page", [16, 32, 256])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("add", [True, False])
@pytest.mark.parametrize("packed", [False, True])
def test_pages_masks_and_sums(ea, page, causal, add, packed):  # noqa: F811
    _weights(ea, [0, 1, 15, 16, 17, 31, 32, 33, 512, 513, 700], 4, 2, 3, 64, page, packed, causal,
             add, seed=page)


@pytest.mark.parametrize("packed,layout", [(False, "nhd"), (False, "padded"), (True, "nhd"), (True, "apart")])
def test_layouts(ea, packed, layout):  # noqa: F811
    _weights(ea, [200, 77], 8, 4, 1, 128, 32, packed, seed=3, layout=layout)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("n_q", [1, 40])
def test_long_and_wide(ea, packed, n_q):  # noqa: F811
    _weights(ea, [9001, 40, 2500], 2, 1, n_q, 64, 64, packed, seed=5, room=WIDE)


def test_rows_that_attend_nothing_give_nothing(ea):  # noqa: F811
    # lse = -inf; and the weights of all rows add up to their number
    g = torch.Generator().manual_seed(2)
    k = torch.randn(4, 1, 16, 64, generator=g).to(torch.bfloat16).cuda()
    q = torch.randn(1, 4, 1, 64, generator=g).to(torch.bfloat16).cuda()
    t, n = _i([[0, 1, 2, 3]]), _i([60])
    _, lse = ea.attention_decode_paged(q, k, k, t, n)
    w = torch.zeros(1, 1, 64, device="cuda")
    ea.attention_key_weights(q, k, t, n, lse, w)
    assert abs(w.sum().item() - 4) <= 4 * 2 * L_MAX_ABS and torch.all(w[..., 60:] == 0)
    lse[0, 1] = float("-inf")
    ea.attention_key_weights(q, k, t, n, lse, w, add=False)
    assert abs(w.sum().item() - 3) <= 3 * 2 * L_MAX_ABS
    again = torch.zeros_like(w)
    for _ in range(3):    # the same every time
        ea.attention_key_weights(q, k, t, n, lse, again, add=False)
        assert torch.equal(again, w)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("H", [9, 40, 130])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_minus_infinity_give_nothing_whatever_they_hold(ea, packed, H, d):  # noqa: F811
    # rows that pad a batch: no logsumexp, and a q that nobody has written
    g = torch.Generator().manual_seed(H)
    rng = np.random.default_rng(H)
    codes, scales = (torch.from_numpy(x).cuda() for x in
                     _cache(rng, np.arange(12).reshape(1, 12), [700], 12, 1, 64, d))
    keys = torch.randn(12, 1, 64, d, generator=g).to(torch.bfloat16).cuda()
    kw = dict(k_scales=scales.view(E4M3), k_descale=2.0 ** -7) if packed else {}
    q = torch.randn(1, H, 1, d, generator=g).to(torch.bfloat16)
    lse = torch.randn(1, H, 1, generator=g) + 5
    odd, some = q.clone(), lse.clone()
    for h, x in ((1, float("nan")), (H // 2, float("inf")), (H - 1, -float("inf"))):
        odd[0, h], some[0, h], q[0, h] = x, -float("inf"), 0
    t, n = _i([list(range(12))]), _i([700])
    got = [ea.attention_key_weights(x.cuda(), codes if packed else keys, t, n, some.cuda(),
                                    torch.zeros(1, 1, 768, device="cuda"), scale=0.01, **kw) for x in (q, odd)]
    ea.check()
    assert torch.isfinite(got[0]).all() and got[0][0, 0, :700].min() > 0
    assert torch.equal(*got)


def test_a_bad_page_of_keys_is_reported(ea):  # noqa: F811
    from exact_attention_12_gb300 import AttnError
    k = torch.ones(2, 1, 16, 64, device="cuda", dtype=torch.bfloat16)
    q = torch.zeros(1, 1, 1, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(1, 1, 48, device="cuda")
    ea.attention_key_weights(q, k, _i([[0, 9, 1]]), _i([48]), torch.zeros(1, 1, 1, device="cuda"), w)
    with pytest.raises(AttnError):
        ea.check()
    assert torch.all(w == 1)    # exp(0 - 0), the missing page's keys being zero


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("n_q", [10, 70])
def test_a_stalled_sum_of_many_rows_ends_and_reports(ea, packed, n_q):  # noqa: F811
    from exact_attention_12_gb300 import _abi
    lib = _abi.lib()
    z = dict(device="cuda")
    P = 640      # tiles enough for every CTA's ring to come round
    k = torch.zeros(P, 1, 128, 32 if packed else 64, dtype=torch.uint8 if packed else torch.bfloat16, **z)
    kw = dict(k_scales=torch.zeros(P, 1, 128, 4, **z).to(E4M3)) if packed else {}
    t, n = torch.arange(P, dtype=torch.int32, **z).view(1, P), _i([P * 128])
    q = torch.zeros(1, 8, n_q, 64, dtype=torch.bfloat16, **z)
    w, lse = torch.zeros(1, 1, P * 128, **z), torch.zeros(1, 8, n_q, **z)
    ws = torch.zeros(256, dtype=torch.uint8, **z)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert lib.attn_debug_stall(_abi.ATTN_STALL_WEIGHTS_SUM, 20_000_000) == _abi.ATTN_OK
    ea.attention_key_weights(q, k, t, n, lse, w, causal=False, ws=ws, **kw)
    assert lib.attn_check(ws.data_ptr(), stream) == _abi.ATTN_ERR_TIMEOUT
    assert int(lib.attn_last_error().decode().rsplit("wait site", 1)[1]) in range(85, 89)
    for _ in range(2):
        ea.attention_key_weights(q, k, t, n, lse, w, causal=False, ws=ws, add=False, **kw)
        assert lib.attn_check(ws.data_ptr(), stream) == _abi.ATTN_OK
        assert torch.all(w == 8 * n_q)      # exp(0 - 0) of every row


def test_weights_of_nothing(ea):  # noqa: F811
    z = dict(device="cuda", dtype=torch.bfloat16)
    k, w = torch.zeros(3, 2, 16, 64, **z), torch.ones(1, 2, 32, device="cuda")
    t, n, lse = _i([[0, 1]]), _i([0]), torch.zeros(1, 4, 1, device="cuda")
    ea.attention_key_weights(torch.zeros(1, 4, 1, 64, **z), k, t, n, lse, w)
    ea.attention_key_weights(torch.zeros(1, 4, 1, 64, **z), k[:0], t, n, lse, w)
    ea.attention_key_weights(torch.zeros(0, 4, 1, 64, **z), k, t[:0], n[:0], lse[:0], w[:0])
    ea.attention_key_weights(torch.zeros(1, 4, 1, 64, **z), k, t[:, :0], n, lse, w)
    ea.check()
    assert torch.all(w == 1)


# ---------------------------------------------------------------- eviction --

def _spread(rng, shape):
    """Weights as they gather: a few large, many alike, zeros."""
    w = np.exp(2 * rng.normal(size=shape)).astype(np.float32)
    return np.where(w < 0.4, np.round(w * 8) / 8, w).astype(np.float32)


def _raw(x):
    return x.view(torch.uint8) if x.element_size() == 1 else x.view(torch.int16)


class Evicting:
    """Device state, weights and pools, with their twins."""

    def __init__(self, seed, lens, size, H=2, rows=None, most=None, spare=3, room=0, kind="bf16", d=64,
                 weights=None):
        self.rng = rng = np.random.default_rng(seed)
        rows = len(lens) if rows is None else rows
        most = max(1, max(-(-n // size) for n in lens)) + 1 if most is None else most
        P = sum(-(-n // size) for n in lens) + spare
        self.c = Cache(rng, rows, most, P, size, lens, pools=())
        g = torch.Generator().manual_seed(seed)
        width = most * size + room
        self.w = _spread(rng, (rows, H, width)) if weights is None else weights
        self.wd = torch.from_numpy(self.w.copy()).cuda()
        if kind == "bf16":
            self.pools = [torch.randn(P, H, size, d, generator=g).to(torch.bfloat16).cuda()
                          for _ in range(2)]
        elif kind == "fp4":
            self.pools = [torch.randint(0, 256, (P, H, size, n), generator=g, dtype=torch.uint8).cuda()
                          for n in (d // 2, d // 16) * 2]
            self.pools[1], self.pools[3] = self.pools[1].view(E4M3), self.pools[3].view(E4M3)
        elif kind == "odd":      # 12, 20 and 4 bytes a row; heads behind the rows
            self.pools = [torch.randn(P, H, size, 3, generator=g).cuda(),
                          torch.randn(P, size, H, 5, generator=g).cuda().transpose(1, 2),
                          torch.randint(0, 99, (P, H, size, 1), generator=g, dtype=torch.int32).cuda()]
        self.plain = [x.cpu().clone() if x.element_size() > 1 else x.view(torch.uint8).cpu().clone()
                      for x in self.pools]

    def evict(self, ea, seqs, new_lens, recent, status=0, ws=None):
        from exact_attention_12_gb300 import AttnError
        c = self.c
        slots = ea.pages_evict(self.pools, *c.state, self.wd, _i(seqs), _i(new_lens), recent=recent,
                               page_size=c.size, ws=ws)
        torch.cuda.synchronize()
        if status:
            with pytest.raises(AttnError) as e:
                ea.check(ws=ws)
            assert e.value.status == status
        ea.check(ws=ws)
        plain = [x.numpy() if x.dtype != torch.bfloat16 else x.view(torch.int16).numpy()
                 for x in self.plain]
        want = oracle.evict(c.twin, plain, self.w, seqs, new_lens, recent)
        assert np.array_equal(slots.cpu().numpy(), want)
        self.same()
        return slots

    def same(self):
        self.c.same()
        assert np.array_equal(self.wd.cpu().numpy(), self.w, equal_nan=True)
        for a, b in zip(self.pools, self.plain):
            a = a.view(torch.uint8) if a.element_size() == 1 else a
            assert torch.equal(a.cpu(), b)


@pytest.mark.parametrize("kind", ["bf16", "fp4", "odd"])
@pytest.mark.parametrize("size", [16, 64])
@pytest.mark.parametrize("recent", [0, 1, 40, 100000])
def test_lengths(ea, kind, size, recent):  # noqa: F811
    e = Evicting(size + recent, [1, 15, 16, 17, 100, 333, 1000, 0, 64], size, H=3, kind=kind)
    e.evict(ea, list(range(9)), [0, 3, 16, 16, 50, 300, 17, 5, 63], recent)


@pytest.mark.parametrize("old,new", [(5000, 4999), (5000, 2500), (5000, 1), (4096, 4095), (9000, 8000)])
@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_long_sequences(ea, old, new, kind):  # noqa: F811
    # one sequence: a cluster per head; many chunks that wait for one another
    e = Evicting(old + new, [old], 32, H=2, kind=kind)
    e.evict(ea, [0], [new], 100)


def test_very_long(ea):  # noqa: F811
    # more weights than a CTA's shared memory holds, in one CTA per head and in clusters
    for lens, H in (([50000] * 40, 4), ([400000], 1)):
        rng = np.random.default_rng(1)
        e = Evicting(3, lens, 1024, H=H, kind="odd", weights=_spread(rng, (len(lens), H, max(lens) + 2000 & ~1023)),
                     most=(max(lens) + 2000 & ~1023) // 1024)
        e.evict(ea, list(range(len(lens))), [n // 3 for n in lens], 500)


def test_many_sequences_out_of_order(ea):  # noqa: F811
    rng = np.random.default_rng(4)
    lens = [int(x) for x in rng.integers(0, 600, 70)]
    e = Evicting(4, lens, 16, H=8, rows=80)
    seqs = [int(x) for x in rng.permutation(70)[:50]]
    e.evict(ea, seqs, [int(rng.integers(0, 400)) for _ in seqs], 30)


def test_again_and_again(ea):  # noqa: F811
    e = Evicting(5, [500, 400], 16, H=2)
    for n in (450, 449, 300, 300, 17, 16, 1, 0):
        e.evict(ea, [1, 0], [n, n], 10)


@pytest.mark.parametrize("weights", ["equal", "zero", "special", "ascending", "descending"])
def test_weights_of_all_kinds(ea, weights):  # noqa: F811
    rng = np.random.default_rng(6)
    w = {"equal": np.full((1, 2, 720), 0.7), "zero": np.zeros((1, 2, 720)),
         "special": rng.choice([np.nan, np.inf, -np.inf, -1.0, -0.0, 0.0, 1e-45, 3e38, -np.nan], (1, 2, 720)),
         "ascending": np.arange(1440.0).reshape(1, 2, 720),
         "descending": -np.arange(1440.0).reshape(1, 2, 720)}[weights].astype(np.float32)
    e = Evicting(6, [700], 16, H=2, weights=w, most=45)
    e.evict(ea, [0], [333], 20)


def test_what_is_refused(ea):  # noqa: F811
    e = Evicting(7, [100, 100, 100, 100, 100, 100], 16, rows=7, spare=4)
    c = e.c
    # a shared page that would be written (1), one behind the new length (2), a free
    # page (3), one outside the cache (4), a wrong length (6)
    for s, j, value in ((4, 3, 1 << 20),):
        c.table[s, j] = value
        c.twin.table[s][j] = value
    for s, j, refs in ((1, 2, 2), (2, 6, 2), (3, 1, 0)):
        pg = c.twin.table[s][j]
        c.refs[pg] = refs
        c.twin.refs[pg] = refs
    c.lens[6] = 10 ** 6
    c.twin.lens[6] = 10 ** 6
    slots = e.evict(ea, [0, 1, 2, 3, 4, 5, 6, 7, -1, 0], [50, 50, 50, 50, 50, -1, 50, 50, 50, 20], 5,
                    status=6)
    refused = [(x == -2).all().item() for x in slots]
    assert refused == [False, True, False, True, True, True, True, True, True, True]
    # a sequence that stays may share all it has
    e.evict(ea, [1], [100], 5)


def test_nothing_to_evict(ea):  # noqa: F811
    e = Evicting(8, [100, 0], 16)
    e.evict(ea, [], [], 5)
    e.evict(ea, [0, 1], [100, 0], 5)
    e.evict(ea, [1, 0], [7, 1000], 5)
    none = [x[:, :0] for x in e.pools]
    slots = ea.pages_evict(none, *e.c.state, e.wd[:, :0], _i([0]), _i([3]), page_size=16)
    assert slots.shape == (1, 0, e.w.shape[2])
    e.same()
    e.pools, e.plain = [], []      # tables and weights alone
    e.evict(ea, [0], [33], 5)


def test_a_stalled_eviction_ends_and_reports(ea):  # noqa: F811
    from exact_attention_12_gb300 import _abi
    lib = _abi.lib()
    e = Evicting(9, [3000], 16)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert lib.attn_debug_stall(_abi.ATTN_STALL_EVICT_READ, 20_000_000) == _abi.ATTN_OK
    ea.pages_evict(e.pools, *e.c.state, e.wd, _i([0]), _i([1500]), page_size=16, ws=ws)
    assert lib.attn_check(ws.data_ptr(), stream) == _abi.ATTN_ERR_TIMEOUT
    assert int(lib.attn_last_error().decode().rsplit("wait site", 1)[1]) == 81
    assert lib.attn_check(ws.data_ptr(), stream) == _abi.ATTN_OK
    # the workspace serves the next call
    Evicting(10, [3000], 16).evict(ea, [0], [1500], 30, ws=ws)


def test_a_captured_eviction(ea):  # noqa: F811
    e = Evicting(11, [900, 300], 16)
    start = [x.clone() for x in (*e.c.state, e.wd, *e.pools)]
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    seqs, new = _i([0, 1]), _i([400, 200])
    run = lambda: ea.pages_evict(e.pools, *e.c.state, e.wd, seqs, new, recent=20, page_size=16, ws=ws)  # noqa: E731
    want = run()
    after = [x.clone() for x in (*e.c.state, e.wd, *e.pools)]

    def reset():
        for x, y in zip((*e.c.state, e.wd, *e.pools), start):
            x.copy_(y)

    reset()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        slots = run()
    for _ in range(3):
        reset()
        graph.replay()
        assert torch.equal(slots, want)
        for x, y in zip((*e.c.state, e.wd, *e.pools), after):
            assert torch.equal(x, y)
    ea.check(ws=ws)


# --------------------------------------------------------------- a whole run --

@pytest.mark.parametrize("packed", [False, True])
def test_a_serving_loop(ea, packed):  # noqa: F811
    """Sequences grow by a prompt and then token by token; every step attends, adds up
    the keys' weights, and evicts what is over the budget.  The twins hold plain
    lists of the keys that each head still has."""
    B, H, H_kv, d, size, P, budget, recent = 3, 4, 2, 64, 16, 60, 48, 8
    g = torch.Generator().manual_seed(12)
    table, lens, refs = _i([[-1] * 12] * B), _i([0] * B), _i([0] * P)
    if packed:
        pools = [torch.zeros(P, H_kv, size, n, dtype=torch.uint8, device="cuda") for n in (d // 2, d // 16) * 2]
        pools[1], pools[3] = pools[1].view(E4M3), pools[3].view(E4M3)
    else:
        pools = [torch.zeros(P, H_kv, size, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    factors = dict(k_descale=0.005, v_descale=0.004)
    w = torch.zeros(B, H_kv, 12 * size, device="cuda")
    keys = [[[] for _ in range(H_kv)] for _ in range(B)]    # (k, v, weight) per head
    n_now = [0] * B
    seqs = _i(range(B))
    for step in range(25):
        n = [50, 20, 33] if step == 0 else [1, 1, 1]
        most = max(n)
        k, v = (torch.randn(B, H_kv, most, d, generator=g).to(torch.bfloat16) for _ in range(2))
        n_now = [a + b for a, b in zip(n_now, n)]
        ea.pages_extend(table, lens, refs, seqs, _i(n_now), page_size=size)
        if packed:
            ea.pages_store_fp4(k.cuda(), v.cuda(), *pools, table, lens, counts=_i(n), **factors)
            kd, vd = (fp4.decode(*fp4.encode(np64(x), D), D)
                      for x, D in ((k, factors["k_descale"]), (v, factors["v_descale"])))
        else:
            kd, vd = np64(k), np64(v)
            rows = table.tolist()
            for b in range(B):
                for j in range(n[b]):
                    pos = n_now[b] - n[b] + j
                    for pool, x in zip(pools, (k, v)):
                        pool[rows[b][pos // size], :, pos % size] = x[b, :, j].cuda()
        for b in range(B):
            for h in range(H_kv):
                keys[b][h] += [[kd[b, h, j], vd[b, h, j], 0.0] for j in range(n[b])]
        q = torch.randn(B, H, 1, d, generator=g).to(torch.bfloat16)
        if packed:
            o, lse = ea.attention_decode_fp4(q.cuda(), *pools, table, lens, **factors)
            ea.attention_key_weights(q.cuda(), pools[0], table, lens, lse, w, k_scales=pools[1],
                                     k_descale=factors["k_descale"])
        else:
            o, lse = ea.attention_decode_paged(q.cuda(), *pools, table, lens)
            ea.attention_key_weights(q.cuda(), pools[0], table, lens, lse, w)
        got_w = np64(w)
        for b in range(B):
            for h in range(H):
                mine = keys[b][h // (H // H_kv)]
                kk, vv = (np.array([x[i] for x in mine]) for i in (0, 1))
                s = kk @ np64(q)[b, h, 0] * d ** -0.5
                p = np.exp(s - s.max())
                p /= p.sum()
                bound = 1.01 * ((2.0 ** -8 + 2 * L_MAX_ABS) * (p @ np.abs(vv)) + 2.0 ** -8 * np.abs(p @ vv)) + 1e-6
                assert np.all(np.abs(np64(o)[b, h, 0] - p @ vv) <= bound)
                for x, y in zip(mine, p):
                    x[2] += y
            for h in range(H_kv):
                assert np.allclose(got_w[b, h, :n_now[b]], [x[2] for x in keys[b][h]], rtol=4 * L_MAX_ABS, atol=1e-6)
                assert np.all(got_w[b, h, n_now[b]:] == 0)
        # evict a few at a time, by the device's own weights
        slots = ea.pages_evict(pools, table, lens, refs, w, seqs, _i([budget] * B), recent=recent,
                               page_size=size)
        new = [min(x, budget) for x in n_now]
        for b in range(B):
            for h in range(H_kv):
                want = oracle.kept(got_w[b, h].astype(np.float32), n_now[b], new[b], recent) \
                    if new[b] < n_now[b] else np.arange(new[b])
                assert slots[b, h, :new[b]].tolist() == want.tolist()
                keys[b][h] = [keys[b][h][j] for j in want]
        n_now = new
        assert lens.tolist() == n_now
        held = sum(-(-x // size) for x in n_now)
        assert int((refs > 0).sum()) == held
    ea.check()


@pytest.mark.parametrize("H", [4, 40])
def test_pages_further_apart_than_32_bits(ea, H):  # noqa: F811
    # the same calls on pages next to one another and on pages (of codes, scales and
    # bf16 keys) 2.5 GiB apart give the same bits
    page, P, apart = 64, 6, 5 << 29
    big = torch.zeros(P * apart + (1 << 20), dtype=torch.uint8, device="cuda")
    shapes = [(P, 1, page, 64), (P, 1, page, 8)] * 2 + [(P, 1, page, 256)]
    far = [big[i << 17:].as_strided(s, (apart, page * s[3], s[3], 1)) for i, s in enumerate(shapes)]
    near = [torch.zeros(s, dtype=torch.uint8, device="cuda") for s in shapes]
    g = torch.Generator().manual_seed(H)
    k, v = (torch.randn(1, 1, 300, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(1, H, 1, 128, generator=g).to(torch.bfloat16).cuda()
    keys = torch.randn(P, 1, page, 128, generator=g).to(torch.bfloat16).cuda()
    table = torch.full((1, 320), -1, dtype=torch.int32, device="cuda")
    table[0, :5] = _i([5, 0, 3, 1, 4])
    out = []
    for pools in (near, far):
        t, lens, refs = table.clone(), _i([300]), _i([1, 1, 0, 1, 1, 1])
        pools[4].copy_(keys.view(torch.uint8))
        cache = [pools[0], pools[1].view(E4M3), pools[2], pools[3].view(E4M3)]
        wide = pools[4].view(torch.bfloat16)
        kw = dict(k_descale=2.0 ** -9, v_descale=2.0 ** -9)
        w = torch.zeros(1, 1, 320 * page, device="cuda")
        ea.pages_store_fp4(k, v, *cache, t, lens, **kw)
        back = ea.pages_load_fp4(*cache, t, lens, 300, **kw)
        step = ea.attention_decode_fp4(q, *cache, t, lens, **kw)
        ea.attention_key_weights(q, cache[0], t, lens, step[1], w, k_scales=cache[1], k_descale=2.0 ** -9)
        first = w.clone()
        ea.attention_key_weights(q, wide, t, lens, step[1], w)
        second = w.clone()
        slots = ea.pages_evict([*cache, wide], t, lens, refs, w, _i([0]), _i([100]), recent=10,
                               page_size=page)
        ea.check()
        out.append([*back, *step, first, second, slots, w, t, lens, refs,
                    *(x.view(torch.uint8)[[5, 0]] for x in pools)])
    for a, b in zip(*out):
        assert torch.equal(a, b)
    assert out[0][0].abs().sum() > 0 and out[0][4].sum() > 0


@pytest.mark.parametrize("packed", [False, True])
def test_a_captured_step_of_many_rows(ea, packed):  # noqa: F811
    # decode (4 bits), the weights of 48 rows a head and an eviction in one graph, replayed
    # with other queries and lengths on a stream of its own
    page, P, B, d = 32, 90, 2, 128
    rng, g = np.random.default_rng(3), torch.Generator().manual_seed(3)
    table = torch.full((B, 600), -1, dtype=torch.int32)
    table[:, :40] = torch.from_numpy(rng.permutation(P)[:80].reshape(B, 40).astype(np.int32))
    codes = [torch.from_numpy(rng.integers(0, 256, (P, 1, page, d // 2), dtype=np.uint8)).cuda() for _ in range(2)]
    scales = [torch.from_numpy(rng.integers(0x20, 0x50, (P, 1, page, d // 16), dtype=np.uint8)).cuda().view(E4M3)
              for _ in range(2)]
    cache = (codes[0], scales[0], codes[1], scales[1])
    keys = torch.randn(P, 1, page, d, generator=g).to(torch.bfloat16).cuda()
    pools = [*cache, keys]
    start = [x.clone() for x in pools]
    q = torch.zeros(B, 12, 4, d, dtype=torch.bfloat16, device="cuda")
    t, lens, refs = table.cuda(), _i([0, 0]), _i([0] * P)
    w, new, seqs = torch.zeros(B, 1, 600 * page, device="cuda"), _i([0, 0]), _i([0, 1])
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")

    def set_up(n, m, seed):
        for x, y in zip(pools, start):
            x.copy_(y)
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(seed)) * 0.3)
        lens.copy_(_i(n))
        new.copy_(_i(m))
        t.copy_(table)
        for b in range(B):
            t[b, -(-n[b] // page):] = -1
        refs.zero_()
        refs[t[t >= 0].long()] = 1
        w.zero_()

    def step():
        o, lse = ea.attention_decode_fp4(q, *cache, t, lens, scale=0.02, k_descale=0.01, ws=ws)
        ea.attention_key_weights(q, codes[0] if packed else keys, t, lens, lse, w, scale=0.02, ws=ws,
                                 **(dict(k_scales=scales[0], k_descale=0.01) if packed else {}))
        seen = w.clone()
        return o, lse, seen, ea.pages_evict(pools, t, lens, refs, w, seqs, new, recent=7, page_size=page, ws=ws)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        set_up([1000, 3], [500, 3], 0)
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = step()
        for n, m, seed in (([1000, 77], [333, 20], 1), ([1, 1280], [5, 64], 2), ([0, 640], [0, 0], 3)):
            set_up(n, m, seed)
            graph.replay()
            first = [x.clone() for x in (*got, t, lens, refs, w, *pools)]
            set_up(n, m, seed)
            again = [*step(), t, lens, refs, w, *pools]
            for a, b in zip(first, again):
                assert torch.equal(a.view(torch.uint8) if a.dtype is E4M3 else a,
                                   b.view(torch.uint8) if b.dtype is E4M3 else b)
            assert lens.tolist() == [min(x, y) for x, y in zip(n, m)]
            stream.synchronize()
            ea.check(ws=ws)
