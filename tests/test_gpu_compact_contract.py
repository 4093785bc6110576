"""What the calls on compact caches promise beside ordinary results: limits, odd
weights and keys, what a caller may leave in places that nothing attends."""

import numpy as np
import pytest
import torch

from tests.test_gpu_fp4 import E4M3
from tests.test_gpu_pages import _i
from tests.test_gpu_paged import ea  # noqa: F401

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
