"""Amplitudes of the rotation at the ends of their range: refused where fp32 would lose them (CPU),
and the same keys from a large batch as from small ones (GPU)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import kv8_ref as R
from tests.test_gpu_kv8 import Store, _bf16, _i32
from tests.test_kv8_host import csa2  # noqa: F401


def test_amplitudes_that_fp32_does_not_hold_are_refused(csa2):  # noqa: F811
    f = (ctypes.c_double * 32)()

    def ask(amplitude):
        return csa2.lib().csa2_rope_frequencies(ctypes.byref(csa2.make_rope(64, amplitude=amplitude)), f)
    for a in (2.0 ** -126, 1e-30, 1.0, 999999.0):
        assert ask(a) == csa2.OK
    for a in (2.0 ** -127, 1e-40, 1e-46, 5e-324, 0.0, -1.0, 1e6, float("inf"), float("nan")):
        assert ask(a) == csa2.ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("amplitude,size", [(2.0 ** -126, 2.0 ** 120), (1e-30, 1.0), (1e-20, 1e20), (1.3, 1.0),
                                            (9e5, 1.0)])
@pytest.mark.parametrize("chunk", [640, 32])
def test_keys_of_far_amplitudes_do_not_depend_on_the_batch(csa2, amplitude, size, chunk):  # noqa: F811
    """640 tokens of 16 heads in one call share angles in a CTA; 32 at a time do not."""
    rng = np.random.default_rng(21)
    H, D, n = 16, 64, 640
    st = Store(csa2, 5, H, D)
    table = np.arange(5, dtype=np.int32)[None]
    x = _bf16(rng.normal(size=(n, H, D)) * size)
    rope = dict(rot_dim=D, amplitude=amplitude)
    for t in range(0, n, chunk):
        seqs = csa2.make_seqs(None, _i32([t + chunk]), chunk, block_table=_i32(table))
        csa2.kv8_append(x[t:t + chunk], x[t:t + chunk], st.cache, seqs, None, st.ws,
                        rope=csa2.make_rope(**rope))
    assert csa2.status_fetch(st.ws) == csa2.OK
    (kc, _), (ke, _) = st.host()
    x64 = x.double().cpu().numpy()
    codes, exps = np.zeros((5, H, 128, D), np.uint8), np.zeros((5, H, 8), np.uint8)
    exact = R.append(codes, exps, R.rope(x64, np.arange(n), **rope), [0, n], [n], table)
    # a value on the border of two exponents may fall to either side of it
    assert np.abs(ke.astype(int) - exps).max() <= 1 and (ke == exps).mean() > 0.99
    got = R.VALUES[kc] * np.repeat(2.0 ** (ke.astype(int) - exps), 16, 2)[..., None]
    # half a step of the code, and 2^-20 of the block's largest for the rotation (448 in its scale;
    # its product of two turns has twice the error of one); a step more where the exponent differs
    far = np.abs(got - exact) - (np.abs(exact) * 2.0 ** -4 + 2.0 ** -9 + 2.0 ** -20 * 2 * 448)
    assert far.max() <= 0, far.max()
