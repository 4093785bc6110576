"""Upkeep of a paged cache (attn_pages_*) against plain Python lists, and a
run of the paged calls together, as a serving loop makes them.  Everything
here is whole numbers and copies: results are equal, not near."""

import numpy as np
import pytest
import torch

from oracle import paged as oracle
from tests.helpers import np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ea():
    import exact_attention_12_gb300 as ea
    from exact_attention_12_gb300 import build
    build.build()
    return ea


class Cache:
    """Device state and its list twin."""

    def __init__(self, rng, rows, most, P, size, lens, pools=((2, 64),), sharing=False):
        perm = iter(rng.permutation(P))
        table = np.full((rows, most), -7, dtype=np.int32)
        refs = np.zeros(P, dtype=np.int32)
        for s, n in enumerate(lens):
            for j in range(-(-n // size)):
                table[s, j] = next(perm)
                refs[table[s, j]] += 1
        full = list(lens) + [0] * (rows - len(lens))
        self.size = size
        self.table = torch.from_numpy(table).cuda()
        self.lens = torch.tensor(full, dtype=torch.int32).cuda()
        self.refs = torch.from_numpy(refs).cuda()
        g = torch.Generator().manual_seed(P)
        self.pools = [torch.randn(P, h, size, d, generator=g).to(torch.bfloat16).cuda()
                      for h, d in pools]
        self.twin = oracle.PageTable(table, full, refs, size)
        self.plain = [p.cpu().clone() for p in self.pools]

    @property
    def state(self):
        return self.table, self.lens, self.refs

    def same(self):
        torch.cuda.synchronize()
        assert self.table.cpu().tolist() == self.twin.table
        assert self.lens.cpu().tolist() == self.twin.lens
        assert self.refs.cpu().tolist() == self.twin.refs
        for a, b in zip(self.pools, self.plain):
            assert torch.equal(a.cpu(), b)


def _i(x):
    return torch.tensor(list(x), dtype=torch.int32).cuda()


@pytest.mark.parametrize("size", [1, 16, 48, 256])
@pytest.mark.parametrize("P", [40, 9000])
def test_extend_fork_free_compact(ea, size, P):
    rng = np.random.default_rng(size)
    c = Cache(rng, 12, 9, P, size, [0, 1, size, size + 1, 3 * size, 4 * size - 1],
              pools=((1, 64), (2, 64)))
    ea.pages_extend(*c.state, _i([3, 0, 7]), _i([2 * size, size + 1, 5]), page_size=size)
    c.twin.extend([3, 0, 7], [2 * size, size + 1, 5])
    ea.check()
    c.same()
    new = ea.pages_fork(c.pools, *c.state, _i([5, 4, 3, 11]), _i([8, 9, 10, 6]), page_size=size)
    assert new.cpu().tolist() == c.twin.fork([5, 4, 3, 11], [8, 9, 10, 6], c.plain)
    ea.check()
    c.same()
    ea.pages_free(*c.state, _i([2, 9, 2, 1, 11]), page_size=size)   # one twice, one empty
    c.twin.free([2, 9, 1, 11])
    ea.check()
    c.same()
    moved = ea.pages_compact(c.pools, *c.state, page_size=size)
    assert moved.cpu().tolist() == c.twin.compact(c.plain)
    ea.check()
    c.same()
    used = sum(r != 0 for r in c.twin.refs)
    assert all(c.twin.refs[:used]) and not any(c.twin.refs[used:])


def test_compact_of_full_empty_and_compact_caches(ea):
    for lens in ([], [32, 32], [64]):
        c = Cache(np.random.default_rng(1), 3, 2, 4, 16, [min(n, 32) for n in lens])
        moved = ea.pages_compact(c.pools, *c.state, page_size=16)
        assert moved.cpu().tolist() == c.twin.compact(c.plain)
        again = ea.pages_compact(c.pools, *c.state, page_size=16)
        assert again.cpu().tolist() == c.twin.compact(c.plain)
        c.same()


def test_large_cache_many_forks(ea):
    rng = np.random.default_rng(2)
    lens = [int(x) for x in rng.integers(0, 200, 300)]
    c = Cache(rng, 2500, 13, 30000, 16, lens, pools=((1, 64),))
    par = [int(x) for x in rng.integers(0, 300, 2100)]
    kids = [int(x) for x in 300 + rng.permutation(2200)[:2100]]
    new = ea.pages_fork(c.pools, *c.state, _i(par), _i(kids), page_size=16)
    assert new.cpu().tolist() == c.twin.fork(par, kids, c.plain)
    gone = [int(x) for x in rng.permutation(2500)[:1500]]
    ea.pages_free(*c.state, _i(gone), page_size=16)
    c.twin.free(gone)
    moved = ea.pages_compact(c.pools, *c.state, page_size=16)
    assert moved.cpu().tolist() == c.twin.compact(c.plain)
    grow = [int(x) for x in rng.permutation(2500)[:1200]]
    to = [min(13 * 16, c.twin.lens[s] + int(rng.integers(0, 60))) for s in grow]
    ea.pages_extend(*c.state, _i(grow), _i(to), page_size=16)
    c.twin.extend(grow, to)
    ea.check()
    c.same()


@pytest.mark.parametrize("P", [32768, 32769, 70001])
def test_more_pages_than_a_plan_looks_at_together(ea, P):
    rng = np.random.default_rng(P)
    lens = [P // 7] * 3 + [0, P // 9, 77]
    c = Cache(rng, 8, P // 5, P, 1, lens, pools=((1, 8),))
    ea.pages_free(*c.state, _i([1]), page_size=1)
    c.twin.free([1])
    for rows, to in (([3, 6], [P // 11, 5]), ([7], [P // 6])):
        ea.pages_extend(*c.state, _i(rows), _i(to), page_size=1)
        c.twin.extend(rows, to)
    moved = ea.pages_compact(c.pools, *c.state, page_size=1)
    assert moved.cpu().tolist() == c.twin.compact(c.plain)
    ea.check()
    c.same()


def test_a_full_cache_is_reported_and_left_whole(ea):
    from exact_attention_12_gb300 import _abi
    c = Cache(np.random.default_rng(3), 8, 4, 6, 16, [20, 17])   # 4 of 6 pages taken
    ea.pages_extend(*c.state, _i([2, 3, 0]), _i([33, 8, 30]), page_size=16)   # 3, 1, 0 pages
    c.twin.extend([2, 3, 0], [33, 8, 30])
    with pytest.raises(_abi.AttnError) as e:
        ea.check()
    assert e.value.status == _abi.ATTN_ERR_FULL
    c.same()
    new = ea.pages_fork(c.pools, *c.state, _i([0, 1, 1]), _i([4, 5, 6]), page_size=16)
    assert new.cpu().tolist() == c.twin.fork([0, 1, 1], [4, 5, 6], c.plain) and -2 in new.tolist()
    with pytest.raises(_abi.AttnError) as e:
        ea.check()
    assert e.value.status == _abi.ATTN_ERR_FULL
    c.same()


def test_wrong_lists_are_skipped_and_reported(ea):
    from exact_attention_12_gb300 import _abi
    c = Cache(np.random.default_rng(4), 6, 3, 20, 16, [20, 40, 5])

    def reported():
        with pytest.raises(_abi.AttnError) as e:
            ea.check()
        assert e.value.status == _abi.ATTN_ERR_PAGE
        c.same()

    ea.pages_free(*c.state, _i([-1, 6, 1 << 30]), page_size=16)
    reported()
    # a row out of range, shrinking, past the row's end, named twice (the first counts)
    seqs, to = [9, 1, 0, 2, 2], [5, 39, 49, 30, 48]
    ea.pages_extend(*c.state, _i(seqs), _i(to), page_size=16)
    c.twin.extend(seqs, to)
    reported()
    # a child that is not empty, rows out of range, a child named twice, a child as a parent
    par, kid = [0, 0, -3, 0, 1, 3], [1, 77, 4, 3, 3, 5]
    new = ea.pages_fork(c.pools, *c.state, _i(par), _i(kid), page_size=16)
    assert new.cpu().tolist() == c.twin.fork(par, kid, c.plain)
    reported()
    ea.pages_copy(c.pools, _i([0, 20, -1]), _i([-5, 1, 2]))
    reported()
    # a table that names pages that do not exist, or free ones
    t, n, r = (x.clone() for x in c.state)
    t[0, 0], t[1, 0] = 20, int((r == 0).nonzero()[0])
    before = r.clone()
    ea.pages_free(t, n, r, _i([0]), page_size=16)
    with pytest.raises(_abi.AttnError):
        ea.check()
    assert (r <= before).all() and r.min() >= 0
    ea.pages_free(t, n, r, _i([1]), page_size=16)
    with pytest.raises(_abi.AttnError):
        ea.check()
    assert r.min() >= 0


@pytest.mark.parametrize("shape", [(2, 16, 64), (1, 16, 8), (5, 48, 72)])
def test_copy(ea, shape):
    P = 50
    g = torch.Generator().manual_seed(1)
    pools = [torch.randn(P, *shape, generator=g).to(t).cuda() for t in (torch.bfloat16, torch.float32)]
    # pages apart from each other, and a permuted page
    big = torch.randn(P, 2, *shape, generator=g).to(torch.bfloat16).cuda()
    pools += [big[:, 1], torch.randn(P, *shape, generator=g).to(torch.bfloat16).cuda().transpose(1, 2)]
    other = big[:, 0].clone()
    perm = torch.randperm(P, generator=g)
    src, dst = perm[:20], perm[20:40]
    want = [p.clone() for p in pools]
    for w in want:
        w[dst.cuda()] = w[src.cuda()]
    ea.pages_copy(pools, src.to(torch.int32).cuda(), dst.to(torch.int32).cuda())
    ea.check()
    for p, w in zip(pools, want):
        assert torch.equal(p, w)
    assert torch.equal(big[:, 0], other)


def test_more_pools_than_one_launch_takes(ea):
    c = Cache(np.random.default_rng(5), 6, 3, 20, 16, [20, 40, 5], pools=((1, 8),) * 70)
    new = ea.pages_fork(c.pools, *c.state, _i([0, 1]), _i([3, 4]), page_size=16)
    assert new.cpu().tolist() == c.twin.fork([0, 1], [3, 4], c.plain)
    ea.pages_free(*c.state, _i([0, 2]), page_size=16)
    c.twin.free([0, 2])
    moved = ea.pages_compact(c.pools, *c.state, page_size=16)
    assert moved.cpu().tolist() == c.twin.compact(c.plain)
    ea.check()
    c.same()


def test_no_pools_and_empty_lists(ea):
    c = Cache(np.random.default_rng(6), 4, 3, 20, 16, [20, 40])
    c.pools, c.plain = [], []
    none = _i([])
    ea.pages_extend(*c.state, none, none, page_size=16)
    ea.pages_free(*c.state, none, page_size=16)
    assert ea.pages_fork([], *c.state, none, none, page_size=16).numel() == 0
    new = ea.pages_fork([], *c.state, _i([0]), _i([3]), page_size=16)
    assert new.cpu().tolist() == c.twin.fork([0], [3])
    moved = ea.pages_compact([], *c.state, page_size=16)
    assert moved.cpu().tolist() == c.twin.compact()
    ea.check()
    c.same()


def test_a_serving_loop(ea):
    """Prompts into pages, forks of one of them decoding on with the prompt as
    their shared prefix, sequences ending, the cache closing up, decoding
    going on: each step's attention against the fp64 definition over the
    twin's own cache."""
    from tests.test_gpu_paged import _hold
    rng = np.random.default_rng(7)
    size, H, H_kv, d, P, rows, most = 16, 4, 2, 64, 64, 8, 10
    c = Cache(rng, rows, most, P, size, [], pools=((H_kv, d), (H_kv, d)))
    g = torch.Generator().manual_seed(7)

    def write(seqs, news):
        """New tokens' keys and values at the ends of the sequences."""
        old = list(c.twin.lens)
        to = [old[s] + n for s, n in zip(seqs, news)]
        ea.pages_extend(*c.state, _i(seqs), _i(to), page_size=size)
        c.twin.extend(seqs, to)
        for s, n in zip(seqs, news):
            pos = torch.arange(old[s], old[s] + n)
            kv = torch.randn(2, n, H_kv, d, generator=g).to(torch.bfloat16)
            page = torch.tensor(c.twin.table[s])[pos // size]
            for pool, plain, x in zip(c.pools, c.plain, kv):
                pool[page.cuda(), :, (pos % size).cuda()] = x.cuda()
                plain[page, :, pos % size] = x

    def decode(seqs, n_q, shared=0):
        table = c.table[_i(seqs).long()].contiguous()
        lens = c.lens[_i(seqs).long()].contiguous()
        q = torch.randn(len(seqs), H, n_q, d, generator=g).to(torch.bfloat16)
        o, lse = ea.attention_decode_paged(q.cuda(), *c.pools, table, lens, shared_len=shared)
        want = oracle.paged_decode(np64(q), *(np64(p) for p in c.plain),
                                   [c.twin.table[s] for s in seqs], [c.twin.lens[s] for s in seqs],
                                   d ** -0.5)
        _hold(o, lse, want)

    write([0, 1, 2], [50, 7, 33])
    decode([0, 1, 2], 1)
    ea.pages_fork(c.pools, *c.state, _i([0, 0, 0]), _i([3, 4, 5]), page_size=size)
    c.twin.fork([0, 0, 0], [3, 4, 5], c.plain)
    for step in range(3):
        write([0, 3, 4, 5, 1], [1, 2, 1, 3, 1])
        decode([0, 3, 4, 5], 2, shared=48)
        decode([1, 2, 5], 1)
        c.same()
    ea.pages_free(*c.state, _i([0, 4, 2]), page_size=size)
    c.twin.free([0, 4, 2])
    ea.pages_compact(c.pools, *c.state, page_size=size)
    c.twin.compact(c.plain)
    c.same()
    write([3, 5, 0], [20, 1, 17])
    decode([3, 5], 1, shared=48)
    decode([0, 1, 3, 5], 3)
    ea.check()
    c.same()


def test_upkeep_replayed_from_a_graph(ea):
    c = Cache(np.random.default_rng(8), 8, 4, 24, 16, [20, 40, 5])
    par, kid, gone = _i([0, 1]), _i([4, 5]), _i([2])
    start = [x.clone() for x in c.state] + [p.clone() for p in c.pools]

    def step():
        new = ea.pages_fork(c.pools, *c.state, par, kid, page_size=16)
        ea.pages_free(*c.state, gone, page_size=16)
        return new, ea.pages_compact(c.pools, *c.state, page_size=16)

    def reset():
        for x, y in zip(list(c.state) + c.pools, start):
            x.copy_(y)

    step()
    torch.cuda.synchronize()
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        new, moved = step()
    for p, k, f in (([0, 1], [4, 5], [2]), ([2, 2], [7, 3], [1])):
        reset()
        par.copy_(_i(p))
        kid.copy_(_i(k))
        gone.copy_(_i(f))
        twin = oracle.PageTable(start[0].tolist(), start[1].tolist(), start[2].tolist(), 16)
        plain = [x.cpu().clone() for x in start[3:]]
        want_new = twin.fork(p, k, plain)
        twin.free(f)
        want_moved = twin.compact(plain)
        graph.replay()
        torch.cuda.synchronize()
        ea.check()
        assert new.tolist() == want_new and moved.tolist() == want_moved
        c.twin, c.plain = twin, plain
        c.same()
