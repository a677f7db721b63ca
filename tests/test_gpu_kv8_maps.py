"""Appends whose q_seq contradicts tok_start inside a 16-token block: what is reported as skipped is
not stored, and nothing is dropped without a report."""
import numpy as np
import pytest
import torch

from oracle import kv8_ref as R
from tests.test_gpu_kv8 import Store, _bf16, _i32, csa2  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wrong", [7, -1, 1, -2])
@pytest.mark.parametrize("at", [0, 2, 5])
def test_a_token_that_names_another_sequence_keeps_its_block_out(csa2, wrong, at):  # noqa: F811
    st = Store(csa2, 3, 1, 16, fill=0)
    x = torch.ones(6, 1, 16, device="cuda", dtype=torch.bfloat16)
    q_seq = [0] * 6
    q_seq[at] = wrong
    before = st.host()
    seqs = csa2.make_seqs(None, _i32([6, 2]), q_seq=_i32(q_seq), block_table=_i32([[2, -1], [1, -1]]))
    csa2.kv8_append(x, x, st.cache, seqs, _i32([0, 6, 6]), st.ws)
    assert csa2.status_fetch(st.ws) == csa2.ERR_INVALID_ARG
    after = st.host()
    assert all(np.array_equal(a, b) for u, v in zip(before, after) for a, b in zip(u, v))


@pytest.mark.parametrize("T,H", [(400, 1), (400, 40)])            # windows of 1 and of 16 tokens
@pytest.mark.parametrize("at", [3, 16, 33, 37, 399])
def test_only_that_block_is_left_out(csa2, T, H, at):  # noqa: F811
    rng = np.random.default_rng(at)
    st = Store(csa2, 4, H, 16)
    x = _bf16(rng.normal(size=(T, H, 16)))
    table, first = [[3, 1, 0, 2]], 5                              # 5 tokens stored before
    codes, exps = st.host()
    q_seq = [0] * T
    q_seq[at] = -1
    seqs = csa2.make_seqs(None, _i32([first + T]), q_seq=_i32(q_seq), block_table=_i32(table))
    csa2.kv8_append(x, x, st.cache, seqs, _i32([0, T]), st.ws)
    assert csa2.status_fetch(st.ws) == csa2.ERR_INVALID_ARG
    v = x.double().cpu().numpy()
    block = (first + at) // 16 * 16
    lo, hi = max(0, block - first), min(T, block + 16 - first)
    got_c, got_e = st.host()
    for kv in range(2):
        kept_c, kept_e = codes[kv].copy(), exps[kv].copy()
        for a, b in ((0, lo), (hi, T)):
            if a < b:
                R.append(kept_c, kept_e, v[a:b], [0, b - a], [first + b], table)
        np.testing.assert_array_equal(got_c[kv], kept_c)
        np.testing.assert_array_equal(got_e[kv], kept_e)


@pytest.mark.parametrize("start", [[-5, 6, 6], [-1, 6, 6], [-(2 ** 31), 6, 6]])
@pytest.mark.parametrize("length", [6, 11, 16])
def test_rows_that_start_before_the_first_are_refused(csa2, start, length):  # noqa: F811
    st = Store(csa2, 3, 1, 16, fill=0)
    x = torch.ones(6, 1, 16, device="cuda", dtype=torch.bfloat16)
    before = st.host()
    seqs = csa2.make_seqs(None, _i32([length, 2]), q_seq=_i32([0] * 6), block_table=_i32([[2, -1], [1, -1]]))
    csa2.kv8_append(x, x, st.cache, seqs, _i32(start), st.ws)
    assert csa2.status_fetch(st.ws) == csa2.ERR_INVALID_ARG
    after = st.host()
    assert all(np.array_equal(a, b) for u, v in zip(before, after) for a, b in zip(u, v))
