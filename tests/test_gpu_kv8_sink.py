"""Attention with one key far above tens of thousands of others, whose small weights add up: they must
not be rounded away one by one.

Sequences of 65,536 tokens over the same pages, so that a CTA meets a whole sequence.  The first key
has a logit of L * ln 2 and a zero value, the others 0 and values of 0.5 to 2; out is their mean times
65,535 / 2^L (or so).  Bounds (tests/gpu_kv8.py): a small weight is off by at most 2^-26 of the largest
in the decode kernel (2^-29 of it is the least it can round to 0) and 2^-28 in the prefill kernel.
"""
import math

import numpy as np
import pytest
import torch

from oracle import kv8_ref as R
from tests.gpu_kv8 import check
from tests.test_gpu_kv8 import Store, _attend, _bf16, csa2  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,G,least", [(1, 8, 2.0 ** -26), (1, 16, 2.0 ** -26), (3, 8, 2.0 ** -28)])
def test_many_small_weights_beside_a_large_one(csa2, n, G, least):  # noqa: F811
    N, S, Hkv, D = 65536, 24, 8, 64
    st = Store(csa2, N // 128, Hkv, D, fill=0)
    for e in st.exp:
        e.fill_(127)
    g = torch.Generator(device="cuda").manual_seed(1)
    some = torch.from_numpy(R.e4m3_encode([0.5, 1.0, 1.5, 2.0])).cuda()
    st.dev[1].copy_(some[torch.randint(0, 4, st.dev[1].shape, generator=g, device="cuda")])
    st.dev[1][0, :, 0] = 0
    st.dev[0][0, :, 0, 0] = int(R.e4m3_encode([16.0])[0])
    table = np.tile(np.arange(N // 128, dtype=np.int32), (S, 1))
    L = np.linspace(14, 27, G)                                   # 2^-14 to 2^-27 of the largest weight
    q = np.zeros((S * n, Hkv * G, D))
    q[:, :, 0] = np.tile(L / 16, Hkv)
    q = _bf16(q)
    out, lse, status = _attend(csa2, st, [N] * S, None, table, q, 0, math.log(2), per=n)
    assert status == csa2.OK
    assert check(st, [N] * S, [n] * S, table, q, 0, math.log(2), out, lse, least=least) == S * n
