"""Ragged prefills over the 8-bit cache whose jobs of few and of many query rows follow one another
within a CTA, so that a half of it computes nothing for long stretches of its tiles.

Bounds: tests/gpu_kv8.py.  The K exponents of neighbouring blocks differ by up to 2^10, so a tile
weighed in another tile's scales is far outside them.
"""
import numpy as np
import pytest
import torch

from tests.gpu_kv8 import check
from tests.test_gpu_kv8 import Store, _attend, _bf16, _fill, _tables, csa2  # noqa: F401

pytestmark = pytest.mark.gpu

RAGGED = [
    # lens, new, H, Hkv, D, window
    ([2300 + 631 * (i % 7) for i in range(20)], [(300, 20, 600, 150)[i % 4] for i in range(20)], 8, 8, 64, 0),
    ([2000 + 577 * (i % 8) for i in range(20)], [(300, 20, 600, 150)[i % 4] for i in range(20)], 8, 4, 128, 0),
    ([4000 + 577 * (i % 5) for i in range(30)], [(30, 100, 256, 17)[i % 4] for i in range(30)], 8, 8, 64, 3000),
    # thousands of queries ahead of the first token: whole jobs that see nothing
    ([1500, 2600, 700] * 4, [9000, 2600, 5000] * 4, 4, 4, 32, 0),
]


@pytest.mark.parametrize("lens,new,H,Hkv,D,window", RAGGED)
def test_halves_that_sit_out(csa2, lens, new, H, Hkv, D, window):  # noqa: F811
    rng = np.random.default_rng(len(lens) + D)
    pages = sum(-(-n // 128) for n in lens) + 2
    st = Store(csa2, pages, Hkv, D)
    table = _tables(rng, lens, pages)
    _fill(rng, st, lens, table, spread=8)
    q = _bf16(rng.normal(size=(sum(new), H, D)) * 2.0 ** rng.integers(-2, 4, size=(1, H, 1)))
    for _ in range(3):
        out, lse, status = _attend(csa2, st, lens, new, table, q, window, D ** -0.5)
        assert status == csa2.OK
        assert check(st, lens, new, table, q, window, D ** -0.5, out, lse) == sum(new)
