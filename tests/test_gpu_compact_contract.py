"""What the calls on compact caches promise beside ordinary results: limits, odd
weights and keys, what a caller may leave in places that nothing attends."""

import numpy as np
import pytest
import torch

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
