"""Decode steps against paged caches (attn_decode_paged with and without a
shared prefix, attn_decode_latent) against the fp64 definitions.

Tolerances.  L: the bar of every L here (L_MAX_ABS), which covers the fp32
scores.  O: P is rounded to bf16, a relative 2^-8 of each term, and so is O;
with scores off by at most L_MAX_ABS and L by as much, P is off by a relative
2 L_MAX_ABS more: |O - O*| <= (2^-8 + 2 L_MAX_ABS) sum_j P_j |V_j| + 2^-8 |O|,
with a hundredth on top for the products of these.
"""

import numpy as np
import pytest
import torch

from oracle import paged as oracle
from tests.helpers import L_MAX_ABS, max_abs, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ea():
    import exact_attention_12_gb300 as ea
    from exact_attention_12_gb300 import build
    build.build()
    return ea


# A table with room for many more keys than are cached: short caches then go
# through the balanced split of the keys instead of clusters.
WIDE = 20000


def _table(rng, lens, page, spare=2, shared=0, room=0):
    """A random table for these lengths, and `room` keys: unused entries are
    far out of range."""
    most = max(1, shared // page, room // page, max(-(-n // page) for n in lens)) + 1
    P = sum(-(-n // page) for n in lens) + shared // page + spare
    free = list(rng.permutation(P))
    pre = [free.pop() for _ in range(shared // page)]
    t = np.full((len(lens), most), 1 << 29, dtype=np.int32)
    for b, n in enumerate(lens):
        for j in range(-(-n // page)):
            t[b, j] = pre[j] if j < len(pre) else free.pop()
        t[b, :len(pre)] = pre
    return t, P


def _poison(pages, table, lens, page):
    """NaN in every row that no sequence has cached."""
    keep = torch.zeros(pages.shape[0], page, dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range(-(-n // page)):
            keep[table[b, j], :min(page, n - j * page)] = True
    dead = (~keep).view(keep.shape[0], *([1] * (pages.dim() - 3)), page, 1)
    return pages.masked_fill(dead, float("nan"))


def _pages(g, shape, table, lens, layout="hnd"):
    x = torch.randn(shape, generator=g).to(torch.bfloat16)
    x = _poison(x, table, lens, shape[-2])
    if layout == "nhd":   # [P, page, H_kv, d] in memory
        return x, x.cuda().transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "padded":   # pages apart, rows wider than d
        big = torch.full((shape[0], shape[1], shape[2] + 1, shape[3] + 8), float("nan"),
                         dtype=torch.bfloat16, device="cuda")
        view = big[:, :, :shape[2], :shape[3]]
        view.copy_(x)
        return x, view
    return x, x.cuda()


def _hold(o, lse, want, what=""):
    O, L, A = want
    got = np64(o.cpu())
    bound = 1.01 * ((2.0 ** -8 + 2 * L_MAX_ABS) * A + 2.0 ** -8 * np.abs(O)) + 1e-30
    assert np.isfinite(got).all(), what
    worst = np.max(np.abs(got - O) / bound) if O.size else 0.0
    assert worst <= 1.0, (what, worst)
    assert max_abs(lse.cpu().numpy(), L) <= L_MAX_ABS, what


def _run(ea, lens, H, H_kv, n_q, d, page, causal=True, shared=0, seed=0, layout="hnd", scale=None,
         room=0):
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    table, P = _table(rng, lens, page, shared=shared, room=room)
    shape = (P, H_kv, page, d)
    k, kd = _pages(g, shape, table, lens, layout)
    v, vd = _pages(g, shape, table, lens, layout)
    q = torch.randn(B, H, n_q, d, generator=g).to(torch.bfloat16)
    scale = d ** -0.5 if scale is None else scale
    o, lse = ea.attention_decode_paged(q.cuda(), kd, vd, torch.from_numpy(table).cuda(),
                                       torch.tensor(lens, dtype=torch.int32).cuda(), scale=scale,
                                       causal=causal, shared_len=shared)
    torch.cuda.synchronize()
    ea.check()
    want = oracle.paged_decode(np64(q), np64(k), np64(v), table, lens, scale, causal)
    _hold(o, lse, want)
    return o, lse


# rows per key/value head: 1, 4, 16, 24, 40, 64 -- each row-tile count -- and
# 65, 100, 128, 200, in blocks
@pytest.mark.parametrize("H,H_kv,n_q", [(2, 2, 1), (8, 2, 1), (16, 1, 1), (6, 2, 8), (10, 2, 8),
                                         (64, 1, 1), (65, 1, 1), (40, 2, 5), (128, 1, 1), (8, 1, 25)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("room", [0, WIDE])
def test_rows_and_widths(ea, H, H_kv, n_q, d, room):
    _run(ea, [300, 1, 33, 0, 129], H, H_kv, n_q, d, 16, seed=H + d, room=room)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 512])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("room", [0, WIDE])
def test_page_sizes(ea, page, causal, room):
    _run(ea, [0, 1, 15, 16, 17, 31, 32, 33, 512, 513, 700], 4, 2, 3, 64, page, causal, seed=page,
         room=room)


@pytest.mark.parametrize("layout", ["nhd", "padded"])
def test_layouts(ea, layout):
    _run(ea, [200, 77], 8, 4, 1, 128, 32, layout=layout, seed=3)


@pytest.mark.parametrize("room", [0, WIDE])
def test_empty_sequences(ea, room):
    o, lse = _run(ea, [0, 0, 0], 4, 2, 2, 64, 16, room=room)
    assert torch.all(o == 0) and torch.all(torch.isneginf(lse))


def test_no_sequences(ea):
    i32 = dict(dtype=torch.int32, device="cuda")
    k = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    t, n = torch.zeros(0, 4, **i32), torch.zeros(0, **i32)
    o, lse = ea.attention_decode_paged(k.new_zeros(0, 4, 1, 64), k, k, t, n)
    assert o.shape == (0, 4, 1, 64) and lse.shape == (0, 4, 1)
    o, lse = ea.attention_decode_latent(k.new_zeros(0, 4, 2, 320), k.new_zeros(3, 16, 320), t, n,
                                        scale=0.1, d_v=256)
    assert o.shape == (0, 4, 2, 256) and lse.shape == (0, 4, 2)
    ea.check()


def test_one_long_sequence_over_all_ctas(ea):
    _run(ea, [9001], 4, 1, 1, 128, 64, seed=9)


@pytest.mark.parametrize("lens,H,H_kv,n_q,d,shared", [
    ([20000], 2, 1, 1, 64, 0), ([6001, 5999], 64, 1, 1, 128, 0), ([9000, 40], 4, 1, 3, 64, 0),
    ([5000, 4100], 4, 2, 2, 64, 1024), ([2100, 2048], 33, 1, 1, 128, 2048)])
def test_few_sequences_in_many_pieces(ea, lens, H, H_kv, n_q, d, shared):
    # sixteen threads share a merge's items, in rounds, a thread's pieces two at a time
    _run(ea, lens, H, H_kv, n_q, d, 32, True, shared, seed=12, room=WIDE)


def test_many_short_and_one_long(ea):
    _run(ea, [5] * 130 + [4000] + [0] * 70, 4, 2, 1, 64, 16, seed=10)


@pytest.mark.parametrize("H,n_q", [(4, 1), (12, 2), (20, 5), (40, 7)])
@pytest.mark.parametrize("shared", [0, 48])
def test_many_short_sequences(ea, H, n_q, shared):
    # more segments than the GPU holds CTAs, few tiles each: one slot of a CTA per segment
    rng = np.random.default_rng(H)
    lens = [int(shared + x) for x in rng.integers(0, 200, 81)]
    lens[3], lens[80] = shared, shared + 200
    _run(ea, lens, H, 4, n_q, 64, 16, True, shared, seed=H)


def test_large_scores(ea):
    # scores to +-100: the running maximum has to hold
    _run(ea, [500, 64], 4, 2, 2, 64, 32, scale=4.0, seed=11)


@pytest.mark.parametrize("B,H,H_kv,n_q,d,page,shared", [
    (2, 2, 2, 1, 64, 16, 16), (5, 8, 2, 1, 128, 16, 1040), (3, 4, 1, 5, 64, 64, 128),
    (40, 16, 2, 1, 128, 32, 512), (3, 48, 2, 4, 64, 32, 256), (70, 8, 1, 2, 64, 256, 256), (9, 32, 1, 2, 128, 128, 2048)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("room", [0, WIDE])
def test_shared_prefix(ea, B, H, H_kv, n_q, d, page, shared, causal, room):
    rng = np.random.default_rng(B)
    lens = [int(shared + x) for x in rng.integers(n_q, 150, B)]
    _run(ea, lens, H, H_kv, n_q, d, page, causal, shared, seed=B + d, room=room)


@pytest.mark.parametrize("room", [0, WIDE])
def test_shared_prefix_is_all_there_is(ea, room):
    # nothing of their own; and the newest queries reach back into the prefix
    _run(ea, [256, 256, 257, 300], 4, 2, 3, 64, 64, True, 256, seed=5, room=room)


@pytest.mark.parametrize("lens", [[100, 300, 0, 513], [100, 90, 1, 0]])
@pytest.mark.parametrize("room", [0, WIDE])
def test_sequences_shorter_than_the_prefix(ea, lens, room):
    # a sequence that ends inside the prefix attends its own keys; where all do, the rows
    # behind the longest hold NaN
    _run(ea, lens, 4, 2, 2, 128, 64, True, 512, seed=6, room=room)


def test_shared_equals_unshared(ea):
    rng = np.random.default_rng(1)
    g = torch.Generator().manual_seed(1)
    lens = [700, 801, 640]
    table, P = _table(rng, lens, 64, shared=640)
    k, v = (torch.randn(P, 2, 64, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(3, 8, 1, 128, generator=g).to(torch.bfloat16).cuda()
    t, n = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    a = ea.attention_decode_paged(q, k, v, t, n)
    b = ea.attention_decode_paged(q, k, v, t, n, shared_len=640)
    assert (a[0].float() - b[0].float()).abs().max() <= 2 * (2.0 ** -8 + 1e-3) * 4
    assert (a[1] - b[1]).abs().max() <= L_MAX_ABS


def _run_latent(ea, lens, H, n_q, d_v, page, causal=True, seed=0, scale=0.04, padded=False, room=0):
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    table, P = _table(rng, lens, page, room=room)
    D = d_v + 64
    c = _poison(torch.randn(P, page, D, generator=g).to(torch.bfloat16), table, lens, page)
    cd = c.cuda()
    if padded:
        big = torch.full((P, page + 2, D + 16), float("nan"), dtype=torch.bfloat16, device="cuda")
        big[:, :page, :D] = cd
        cd = big[:, :page, :D]
    q = torch.randn(len(lens), H, n_q, D, generator=g).to(torch.bfloat16)
    o, lse = ea.attention_decode_latent(q.cuda(), cd, torch.from_numpy(table).cuda(),
                                        torch.tensor(lens, dtype=torch.int32).cuda(), scale=scale,
                                        d_v=d_v, causal=causal)
    torch.cuda.synchronize()
    ea.check()
    _hold(o, lse, oracle.latent_decode(np64(q), np64(c), table, lens, scale, d_v, causal))
    return o, lse


@pytest.mark.parametrize("H,n_q", [(1, 1), (16, 1), (20, 2), (33, 1), (64, 1), (65, 1), (128, 1),
                                   (24, 8)])
@pytest.mark.parametrize("d_v", [256, 512])
@pytest.mark.parametrize("room", [0, WIDE])
def test_latent_rows(ea, H, n_q, d_v, room):
    _run_latent(ea, [130, 0, 1, 64], H, n_q, d_v, 32, seed=H, room=room)


@pytest.mark.parametrize("page", [16, 32, 64, 256])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("room", [0, WIDE])
def test_latent_pages(ea, page, causal, room):
    _run_latent(ea, [0, 1, 15, 16, 17, 63, 64, 65, 400], 8, 3, 512, page, causal, seed=page, room=room)


def test_latent_long_and_ragged(ea):
    _run_latent(ea, [5000, 3, 700, 0, 0, 90], 16, 1, 512, 64, seed=2)


@pytest.mark.parametrize("lens,H,d_v", [([20000], 5, 256), ([15000, 3], 16, 512), ([7000], 64, 256)])
def test_latent_few_sequences_in_many_pieces(ea, lens, H, d_v):
    _run_latent(ea, lens, H, 1, d_v, 64, seed=13, room=WIDE)


@pytest.mark.parametrize("room", [0, WIDE])
def test_latent_padded_pages_and_large_scores(ea, room):
    _run_latent(ea, [300, 129], 16, 1, 512, 16, seed=4, scale=1.0, padded=True, room=room)


def test_q_views(ea):
    # q as a slice of a wider projection, heads and queries in the other order
    g = torch.Generator().manual_seed(8)
    lens, page = [90, 40], 16
    table, P = _table(np.random.default_rng(8), lens, page)
    k, v = (torch.randn(P, 2, page, 64, generator=g).to(torch.bfloat16) for _ in range(2))
    wide = torch.randn(2, 3, 4, 96, generator=g).to(torch.bfloat16)
    q = wide[..., 16:80].transpose(1, 2)
    o, lse = ea.attention_decode_paged(wide.cuda()[..., 16:80].transpose(1, 2), k.cuda(), v.cuda(),
                                       torch.from_numpy(table).cuda(),
                                       torch.tensor(lens, dtype=torch.int32).cuda())
    _hold(o, lse, oracle.paged_decode(np64(q), np64(k), np64(v), table, lens, 0.125))


def test_caches_beyond_32_bit_offsets(ea):
    # pages whose elements lie past 2^31; all but the used ones hold whatever was there
    g = torch.Generator().manual_seed(9)
    P, page = 270000, 64
    pool = torch.empty(P, 1, page, 128, dtype=torch.bfloat16, device="cuda")   # 4.4 GB
    used = [P - 1, 0, P - 2, 262144, 131072, P // 2]
    x = torch.randn(6, 1, page, 128, generator=g).to(torch.bfloat16)
    pool[torch.tensor(used).cuda()] = x.cuda()
    table = torch.tensor([used[:3], used[3:]], dtype=torch.int32)
    small = np.array([[0, 1, 2], [3, 4, 5]])
    lens = torch.tensor([150, 192], dtype=torch.int32)
    q = torch.randn(2, 4, 1, 128, generator=g).to(torch.bfloat16)
    for shared in (0, 64):
        if shared:
            table[1, 0], small[1, 0] = table[0, 0], 0
        o, lse = ea.attention_decode_paged(q.cuda(), pool, pool, table.cuda(), lens.cuda(),
                                           shared_len=shared)
        ea.check()
        _hold(o, lse, oracle.paged_decode(np64(q), np64(x), np64(x), small, lens, 128 ** -0.5))
    ea.pages_copy([pool], torch.tensor([P - 1], dtype=torch.int32).cuda(),
                  torch.tensor([P - 9], dtype=torch.int32).cuda())
    assert torch.equal(pool[P - 9].cpu(), x[0])
    c = pool.view(-1)[:P * page * 128 // (page * 576) * page * 576].view(-1, page, 576)
    used = [c.shape[0] - 1, 7, c.shape[0] - 3]
    y = torch.randn(3, page, 576, generator=g).to(torch.bfloat16)
    c[torch.tensor(used).cuda()] = y.cuda()
    qc = torch.randn(1, 16, 1, 576, generator=g).to(torch.bfloat16)
    o, lse = ea.attention_decode_latent(qc.cuda(), c, torch.tensor([used], dtype=torch.int32).cuda(),
                                        torch.tensor([170], dtype=torch.int32).cuda(), scale=0.04)
    ea.check()
    _hold(o, lse, oracle.latent_decode(np64(qc), np64(y), [[0, 1, 2]], [170], 0.04, 512))


def test_bad_page_is_reported_and_reads_as_zeros(ea):
    from exact_attention_12_gb300 import _abi
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(4, 1, 16, 64, generator=g).to(torch.bfloat16) for _ in range(2))
    c = torch.randn(4, 16, 320, generator=g).to(torch.bfloat16)
    q = torch.randn(2, 2, 1, 64, generator=g).to(torch.bfloat16)
    qc = torch.randn(2, 2, 1, 320, generator=g).to(torch.bfloat16)
    lens = torch.tensor([40, 40], dtype=torch.int32)
    for bad in (4, -1, 1 << 30):
        table = torch.tensor([[0, 1, 2], [3, bad, 2]], dtype=torch.int32)
        zero = table.clone().numpy()
        zero[1, 1] = 4
        z = [np.concatenate([np64(x), np.zeros((1,) + x.shape[1:])]) for x in (k, v, c)]
        for shared in (0, 16):
            t = table if not shared else torch.tensor([[bad, 1, 2], [bad, 0, 2]], dtype=torch.int32)
            tz = t.clone().numpy()
            tz[(tz < 0) | (tz > 3)] = 4
            o, lse = ea.attention_decode_paged(q.cuda(), k.cuda(), v.cuda(), t.cuda(), lens.cuda(),
                                               shared_len=shared)
            with pytest.raises(_abi.AttnError) as e:
                ea.check()
            assert e.value.status == _abi.ATTN_ERR_PAGE
            _hold(o, lse, oracle.paged_decode(np64(q), z[0], z[1], tz, [40, 40], 0.125))
        o, lse = ea.attention_decode_latent(qc.cuda(), c.cuda(), table.cuda(), lens.cuda(),
                                            scale=0.05, d_v=256)
        with pytest.raises(_abi.AttnError) as e:
            ea.check()
        assert e.value.status == _abi.ATTN_ERR_PAGE
        _hold(o, lse, oracle.latent_decode(np64(qc), z[2], zero, [40, 40], 0.05, 256))
        ea.check()


def _nan_rows(call, q, b, h, t):
    """A NaN in one query row shows in all of that row's results and nowhere else."""
    o, lse = call(q)
    bad = q.clone()
    bad[b, h, t, 3] = float("nan")
    o2, lse2 = call(bad)
    hit = torch.zeros(q.shape[:3], dtype=torch.bool, device="cuda")
    hit[b, h, t] = True
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    assert torch.isnan(o2[hit]).all() and torch.isnan(lse2[hit]).all()
    assert torch.equal(o2[~hit], o[~hit]) and torch.equal(lse2[~hit], lse[~hit])


# one CTA per segment and cut ones, clusters, many short sequences; with a prefix each
@pytest.mark.parametrize("lens,room", [([200, 1500, 40], WIDE), ([200, 300, 40], 0),
                                       ([40 + i for i in range(90)], 0)])
@pytest.mark.parametrize("shared", [0, 32])
@pytest.mark.parametrize("n_q", [1, 5])
def test_a_nan_query_is_not_hidden(ea, lens, room, shared, n_q):
    rng, g = np.random.default_rng(7), torch.Generator().manual_seed(7)
    table, P = _table(rng, lens, 16, shared=shared, room=room)
    k, v = (torch.randn(P, 4, 16, 64, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(len(lens), 16, n_q, 64, generator=g).to(torch.bfloat16).cuda()
    t, n = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    for b in range(min(3, len(lens))):
        _nan_rows(lambda x: ea.attention_decode_paged(x, k, v, t, n, shared_len=shared), q, b, 5,
                  n_q - 1)
    ea.check()


@pytest.mark.parametrize("lens,room,H", [([200, 1500, 40], WIDE, 8), ([200, 1500, 40], WIDE, 128),
                                         ([200, 250, 40], 0, 8), ([200, 250, 40], 0, 70)])
def test_a_nan_latent_query_is_not_hidden(ea, lens, room, H):
    rng, g = np.random.default_rng(8), torch.Generator().manual_seed(8)
    table, P = _table(rng, lens, 16, room=room)
    c = torch.randn(P, 16, 576, generator=g).to(torch.bfloat16).cuda()
    q = torch.randn(len(lens), H, 2, 576, generator=g).to(torch.bfloat16).cuda()
    t, n = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    for b in range(3):
        _nan_rows(lambda x: ea.attention_decode_latent(x, c, t, n, scale=0.04), q, b, H - 3, 1)
    ea.check()


@pytest.mark.parametrize("room", [0, WIDE])
def test_replayed_graph_follows_lengths_and_tables(ea, room):
    """Captured once, replayed with other lengths, pages and queries."""
    g = torch.Generator().manual_seed(4)
    B, page, most = 4, 32, 12
    P = B * most
    k, v = (torch.randn(P, 2, page, 64, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    c = torch.randn(P, page, 576, generator=g).to(torch.bfloat16).cuda()
    q = torch.zeros(B, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    qc = torch.zeros(B, 8, 1, 576, dtype=torch.bfloat16, device="cuda")
    table = torch.full((B, max(most, room // page)), -1, dtype=torch.int32).cuda()
    table[:, :most] = torch.arange(P).view(B, most)
    lens = torch.full((B,), page * most, dtype=torch.int32).cuda()

    def step():
        return (ea.attention_decode_paged(q, k, v, table, lens),
                ea.attention_decode_paged(q, k, v, table, lens, shared_len=64),
                ea.attention_decode_latent(qc, c, table, lens, scale=0.04))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        out = step()
    for seed, n in ((5, [384, 1, 65, 200]), (6, [64, 0, 383, 100])):
        r = torch.Generator().manual_seed(seed)
        t = torch.randperm(P, generator=r).to(torch.int32).view(B, most)
        t[:, :2] = t[0, :2].clone()
        q.copy_(torch.randn(q.shape, generator=r))
        qc.copy_(torch.randn(qc.shape, generator=r))
        table[:, :most] = t.cuda()
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        ea.check()
        want = oracle.paged_decode(np64(q), np64(k), np64(v), t.numpy(), n, 0.125)
        _hold(*out[0], want)
        _hold(*out[1], want)
        _hold(*out[2], oracle.latent_decode(np64(qc), np64(c), t.numpy(), n, 0.04, 512))
        eager = step()
        for a, b in zip(out, eager):   # the same split, the same order of sums
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_streams_with_their_own_workspaces(ea):
    g = torch.Generator().manual_seed(12)
    cases = []
    for i, lens in enumerate(([900, 33, 512], [64, 1500])):
        table, P = _table(np.random.default_rng(i), lens, 32)
        k, v = (torch.randn(P, 2, 32, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
        q = torch.randn(len(lens), 8, 1, 128, generator=g).to(torch.bfloat16).cuda()
        cases.append((q, k, v, torch.from_numpy(table).cuda(),
                      torch.tensor(lens, dtype=torch.int32).cuda()))
    alone = [ea.attention_decode_paged(*x) for x in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    spaces = [torch.zeros(1 << 24, dtype=torch.uint8, device="cuda") for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (x, s, w) in enumerate(zip(cases, streams, spaces)):
            with torch.cuda.stream(s):
                got[i].append(ea.attention_decode_paged(*x, ws=w))
    torch.cuda.synchronize()
    for w in spaces:
        ea.check(ws=w)
    for want, runs in zip(alone, got):
        for o, lse in runs:
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
