"""What the calls on compact caches promise beside ordinary results: limits, odd
weights and keys, what a caller may leave in places that nothing attends."""

import numpy as np
import pytest
import torch

from oracle import fp4, paged as oracle
from tests.helpers import L_MAX_ABS, np64
from tests.test_gpu_eviction import Evicting
from tests.test_gpu_fp4 import E4M3, _cache, _on_gpu
from tests.test_gpu_pages import _i
from tests.test_gpu_paged import WIDE, _table, ea  # noqa: F401

pytestmark = pytest.mark.gpu


def test_weights_as_wide_as_32_bits_count(ea):  # noqa: F811
    # slots are written up to the last entry, and nowhere else
    width, size = 2 ** 31 - 1, 16
    w = torch.zeros(1, 1, width, device="cuda")
    w[0, 0, :40] = torch.arange(40.0)
    for new, status in ((9, 0), (40, 0), (-1, 6)):
        table, lens, refs = _i([[2, 0, 1]]), _i([40]), _i([1, 1, 1])
        slots = ea.pages_evict((), table, lens, refs, w.clone(), _i([0]), _i([new]), page_size=size)[0, 0]
        if status:
            with pytest.raises(ea.AttnError):
                ea.check()
            assert int(slots.max()) == int(slots.min()) == -2
            continue
        ea.check()
        assert slots[:new].tolist() == list(range(40 - new, 40))
        assert int(slots[new:].max()) == int(slots[new:].min()) == -1
        del slots


# ------------------------------------------------------------- key weights --

def _keys(packed, d, H_kv, seed, pages=12, page=64):
    """Keys of a paged cache, and what says so to attention_key_weights."""
    g = torch.Generator().manual_seed(seed)
    if not packed:
        return torch.randn(pages, H_kv, page, d, generator=g).to(torch.bfloat16).cuda(), {}
    codes = torch.randint(0, 256, (pages, H_kv, page, d // 2), generator=g, dtype=torch.uint8).cuda()
    scales = torch.randint(0x20, 0x58, (pages, H_kv, page, d // 16), generator=g, dtype=torch.uint8).cuda()
    return codes, dict(k_scales=scales.view(E4M3), k_descale=2.0 ** -7)


# rows a head: a full block of 8 and of 128, two of them, and more than a pass of 512
@pytest.mark.parametrize("rows", [8, 32, 128, 256, 640])
@pytest.mark.parametrize("d", [64, 128])
def test_a_dead_row_gives_nothing_to_an_infinite_key(ea, rows, d):  # noqa: F811
    # every live row scores the key with -inf: its weight is 0.  A row of no logsumexp
    # is not to turn that into 0 * inf
    keys, _ = _keys(False, d, 1, rows)
    q = torch.randn(1, rows, 1, d, generator=torch.Generator().manual_seed(d)).to(torch.bfloat16)
    q[..., 5] = -q[..., 5].abs() - 1
    lse = torch.full((1, rows, 1), 6.0)
    lse[0, [1, rows - 1]] = float("-inf")
    t, n = _i([list(range(12))]), _i([700])
    run = lambda: ea.attention_key_weights(q.cuda(), keys, t, n, lse.cuda(),  # noqa: E731
                                           torch.zeros(1, 1, 768, device="cuda"), scale=0.02)[0, 0]
    want = run()
    odd = [3, 130, 611, 699]
    for j in odd:
        keys[j // 64, 0, j % 64, 5] = float("inf")
    got = run()
    ea.check()
    assert torch.isfinite(want).all() and want[:700].min() > 0
    want[odd] = 0
    assert torch.equal(got, want)


@pytest.mark.parametrize("rows", [8, 32, 128, 256, 640])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("packed", [False, True])
def test_a_head_of_dead_rows_gives_nothing_to_any_key(ea, rows, d, packed):  # noqa: F811
    # (a place of a padded batch: neither its queries nor its keys need be numbers)
    keys, kw = _keys(packed, d, 2, rows)
    if packed:
        kw["k_scales"].view(torch.uint8)[2, 0, :9] = 0x7f
    else:
        keys[2, 0, :9] = float("nan")
        keys[3, 0, 4, 7] = float("inf")
    q = torch.randn(1, 2 * rows, 1, d, generator=torch.Generator().manual_seed(d)).to(torch.bfloat16)
    q[0, 2] = float("nan")
    lse = torch.full((1, 2 * rows, 1), 6.0)
    lse[0, :rows] = float("-inf")
    t, n = _i([list(range(12))]), _i([700])
    start = torch.rand(1, 2, 768, device="cuda")
    w = ea.attention_key_weights(q.cuda(), keys, t, n, lse.cuda(), start.clone(), scale=0.02, **kw)
    ea.check()
    assert torch.equal(w[0, 0], start[0, 0])
    assert torch.isfinite(w[0, 1]).all() and (w[0, 1, :700] > start[0, 1, :700]).all()
    w = ea.attention_key_weights(q.cuda(), keys, t, n, lse.cuda(), start.clone(), scale=0.02, add=False, **kw)
    assert torch.all(w[0, 0, :700] == 0) and torch.equal(w[0, :, 700:], start[0, :, 700:])


@pytest.mark.parametrize("rows", [4, 40, 130, 600])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_bad_pages_of_keys_read_as_zeros_and_are_reported(ea, rows, d, packed, page):  # noqa: F811
    keys, kw = _keys(packed, d, 1, rows, pages=768 // page + 1, page=page)
    P = keys.shape[0]
    for x in (keys, *(y for y in kw.values() if torch.is_tensor(y))):
        x[P - 1].view(torch.uint8).zero_()
    q = torch.randn(2, rows, 1, d, generator=torch.Generator().manual_seed(d)).to(torch.bfloat16).cuda()
    lse = torch.full((2, rows, 1), 6.0, device="cuda")
    table = torch.tensor([list(range(P - 1))] * 2, dtype=torch.int32)
    bad, zero = table.clone(), table.clone()
    for b, j, value in ((0, 0, -1), (0, (P - 1) // 2, 2 ** 31 - 1), (1, P - 2, P + 5)):
        bad[b, j], zero[b, j] = value, P - 1
    n = _i([730, 768])
    got = []
    for t, pages, fails in ((zero, P, False), (bad, P - 1, True)):
        got.append(ea.attention_key_weights(
            q, keys[:pages], t.cuda(), n, lse, torch.zeros(2, 1, 768, device="cuda"), scale=0.02,
            **{k: x[:pages] if torch.is_tensor(x) else x for k, x in kw.items()}))
        if fails:
            with pytest.raises(ea.AttnError) as e:
                ea.check()
            assert e.value.status == 6
        ea.check()
    assert torch.equal(*got) and got[0][0, 0, :730].min() > 0


# ---------------------------------------------------------------- eviction --

def test_hundreds_of_sequences(ea):  # noqa: F811
    # (more than the moves keep at hand)
    rng = np.random.default_rng(14)
    lens = [int(x) for x in rng.integers(0, 70, 320)]
    e = Evicting(14, lens, 16, rows=330)
    seqs = [int(x) for x in rng.permutation(320)[:300]]
    e.evict(ea, seqs, [int(rng.integers(0, 60)) for _ in seqs], 6)
    e.evict(ea, list(range(320)), [int(x) for x in rng.integers(0, 30, 320)], 0)


# rows of 3, 8 and 32 KB: chunks of 8, 4 and one key
@pytest.mark.parametrize("d", [770, 2048, 8192])
def test_wide_rows(ea, d):  # noqa: F811
    e = Evicting(d, [400, 33, 90], 16, d=d)
    e.evict(ea, [2, 0, 1], [50, 213, 32], 9)
    e.evict(ea, [0, 1], [1, 31], 0)


# ------------------------------------------------------------ 4-bit decode --

# rows a head in one to four blocks of 8, two warps a tile, tcgen05 (a long table, d = 128)
ROWS = [(1, 64, 0), (8, 128, 0), (16, 64, 0), (16, 128, WIDE), (32, 128, 0), (32, 64, WIDE), (40, 128, 0),
        (40, 64, WIDE), (40, 128, WIDE), (64, 128, WIDE)]


@pytest.mark.parametrize("gap", [20, 26, 28.5, 31])
@pytest.mark.parametrize("rows,d,room", ROWS)
def test_small_probabilities_count(ea, rows, d, room, gap):  # noqa: F811
    """Every 32nd key has a score `gap` log2 units above the others, and a value of 0 where
    theirs is 1: O is what the small probabilities add up to.  P has 11 bits down to 2^-21
    of the row's largest, below that an absolute 2^-32 of it; L_MAX_ABS for the scores and
    for L; O rounded to bf16."""
    page, n = 64, 2048
    P = n // page
    codes = torch.full((P, 1, page, d // 2), 0x22, dtype=torch.uint8, device="cuda")    # ones
    codes[:, :, ::32] = 0
    scales = torch.full((P, 1, page, d // 16), 0x38, dtype=torch.uint8, device="cuda").view(E4M3)
    q = torch.full((1, rows, 1, d), -1.0, dtype=torch.bfloat16, device="cuda")
    table = torch.full((1, P + room // page), -1, dtype=torch.int32, device="cuda")
    table[0, :P] = torch.arange(P)
    o, lse = ea.attention_decode_fp4(q, codes, scales, codes, scales, table, _i([n]),
                                     scale=gap * float(np.log(2)) / d)
    ea.check()
    tail = 31 * 2.0 ** -gap
    want = tail / (1 + tail)
    bound = 1.01 * ((2.0 ** -11 + 2 * L_MAX_ABS + 2.0 ** -8) * want + 31 * 2.0 ** -32)
    assert (o.double() - want).abs().max().item() <= bound
    assert (lse.double() - np.log(n / 32 * (1 + tail))).abs().max().item() <= L_MAX_ABS


@pytest.mark.parametrize("rows,d,room", ROWS)
@pytest.mark.parametrize("scale", [1e3, 1e5, 5e5])
def test_scores_of_a_hundred_million(ea, rows, d, room, scale):  # noqa: F811
    # (up to 2^27: a key is attended alone, the next score being far below)
    n, page = 1024, 64
    rng = np.random.default_rng(rows)
    table, P = _table(rng, [n], page, room=room)
    (kc, ks), (vc, vs) = (_cache(rng, table, [n], P, 1, page, d) for _ in range(2))
    ks[...] = 0x38
    q = torch.randn(1, rows, 1, d, generator=torch.Generator().manual_seed(rows)).to(torch.bfloat16)
    o, lse = ea.attention_decode_fp4(q.cuda(), *_on_gpu(kc, ks), *_on_gpu(vc, vs),
                                     torch.from_numpy(table).cuda(), _i([n]), scale=scale)
    ea.check()
    k, v = (oracle.gather(fp4.decode(c, s, 1.0), table[0], n)[0] for c, s in ((kc, ks), (vc, vs)))
    s = np64(q)[0, :, 0] @ k.T * scale
    first, second = np.sort(s)[:, -1], np.sort(s)[:, -2]
    assert 30 * scale < first.min() and first.max() < 2.0 ** 27
    # S is a sum of d exact products, truncated rather than rounded
    off = 2 * (d + 8) * 2.0 ** -24 * scale * (np.abs(np64(q)[0, :, 0]) @ np.abs(k).T).max()
    alone = first - second > 40 + 2 * off
    assert alone.mean() > 0.7
    want = v[s.argmax(1)]
    # P and the sum are the same number, P rounded to fp16; O to bf16
    far = np.abs(np64(o)[0, :, 0] - want) / (np.abs(want) + 1e-30)
    assert far[alone].max() <= 1.01 * (2.0 ** -11 + 2.0 ** -8)
    assert np.all(np.abs(np64(lse)[0, :, 0] - first) <= off + 2.0 ** -21 * first + 1)
