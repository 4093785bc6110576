"""A seeded random sweep of the paged decode steps: sizes, head layouts, page
sizes, lengths (0 and 1 among them), shared prefixes and spare table width
drawn together, each case against the fp64 definitions with the tolerances of
test_gpu_paged."""

import numpy as np
import pytest

from tests.test_gpu_paged import WIDE, _run, _run_latent, ea  # noqa: F401

pytestmark = pytest.mark.gpu


def _lens(rng, B, most):
    kind = rng.integers(4)
    if kind == 0:
        return [most] * B
    n = rng.integers(0, most + 1, B)
    if kind == 1:
        n[rng.random(B) < 0.5] = rng.integers(0, 3)
    if kind == 2:
        n[rng.integers(B)] = most
    return [int(x) for x in n]


@pytest.mark.parametrize("seed", range(48))
def test_paged(ea, seed):
    rng = np.random.default_rng(1000 + seed)
    H_kv = int(rng.choice([1, 2, 3]))
    group = int(rng.choice([1, 2, 4, 5, 8]))
    n_q = int(rng.choice([1, 1, 2, 3, 7]))
    page = int(rng.choice([16, 32, 64, 128, 256]))
    B = int(rng.choice([1, 2, 3, 9, 40, 160]))
    most = int(rng.choice([1, 40, 130, 700, 1500])) if B < 40 else int(rng.choice([3, 50, 200]))
    shared = page * int(rng.integers(0, 5)) if seed % 2 else 0
    lens = [x + shared for x in _lens(rng, B, most)]
    if shared and rng.random() < 0.3:
        lens[int(rng.integers(B))] = int(rng.integers(0, shared + 1))
    _run(ea, lens, H_kv * group, H_kv, n_q, int(rng.choice([64, 128])), page,
         bool(rng.random() < 0.7), shared, seed=seed,
         layout=str(rng.choice(["hnd", "nhd", "padded"])), room=int(rng.choice([0, 0, WIDE])))


@pytest.mark.parametrize("seed", range(32))
def test_latent(ea, seed):
    rng = np.random.default_rng(2000 + seed)
    B = int(rng.choice([1, 2, 5, 20]))
    most = int(rng.choice([1, 63, 64, 65, 300, 900])) if B < 20 else int(rng.choice([5, 70, 130]))
    _run_latent(ea, _lens(rng, B, most), int(rng.choice([1, 8, 16, 48, 64, 96, 128])),
                int(rng.choice([1, 1, 2, 3])), int(rng.choice([256, 512])),
                int(rng.choice([16, 32, 64, 128])), bool(rng.random() < 0.7), seed=seed,
                padded=bool(rng.random() < 0.3), room=int(rng.choice([0, WIDE])))
