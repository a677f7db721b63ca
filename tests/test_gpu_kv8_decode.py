"""The decode kernel in its main use: one or a few tokens per sequence, q of exactly the batch's
size, both of its row counts, 5 to 16 query rows per KV head, 128 channels, serving steps.

The library picks the kernel from the mean of query rows per KV head (rows of q / sequences, rounded
up, times H / H_kv): up to 8 and up to 16 the decode kernel, above the prefill kernel.  Each case
names the one it is for, and the workspace's size, which depends on it, says that it is the one.
Bounds: tests/gpu_kv8.py.
"""
import numpy as np
import pytest
import torch

from oracle import kv8_ref as R
from tests.gpu_kv8 import check
from tests.test_gpu_kv8 import Server, Store, _attend, _bf16, _check_attn, _fill, _tables, csa2  # noqa: F401

pytestmark = pytest.mark.gpu


def _rows(csa2, num_q, num_seqs, H, Hkv, D):  # noqa: F811
    """The kernel's rows per job, from the workspace: partials of 2 * rows * 520 bytes for each of
    its CTAs (three per SM of 8 rows, two of 16, one of 256)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    need = csa2.kv8_attn_workspace(num_q, num_seqs, H, Hkv, D)
    up = lambda n: -(-n // 256) * 256  # noqa: E731
    for rows, per in ((8, 3), (16, 2), (256, 1)):
        ctas = min(1024, sms * per)
        size = 256 + up(ctas * 20) + up(ctas * 2 * rows * 8) + ctas * 2 * rows * 512
        if rows == 256:
            size += up(num_q * H * 256) + num_q * H * 4
        if size == need:
            return rows
    raise AssertionError(need)


DECODES = [
    # rows, lens, new, H, Hkv, D, window
    (8, [1], [1], 8, 1, 128, 0),
    (8, [127], [1], 8, 1, 128, 0),
    (8, [129], [1], 16, 2, 128, 0),
    (8, [5000], [1], 16, 2, 128, 0),
    (8, [5000], [1], 5, 1, 128, 700),
    (8, [1, 300, 2000, 64, 129, 700], [1] * 6, 32, 4, 128, 0),
    (8, [1, 300, 2000, 64, 129, 700], [1] * 6, 14, 2, 128, 100),
    (8, [900, 40, 3000], [2, 2, 2], 8, 2, 128, 0),
    (8, [900, 40, 3000, 77], [8, 1, 3, 4], 2, 1, 128, 64),      # means of 4 tokens, up to 8
    (8, [2500, 0, 1300, 2], [0, 0, 1, 3], 6, 1, 96, 0),         # idle, empty, more queries than tokens
    (16, [127], [1], 16, 1, 128, 0),
    (16, [5000, 1, 130], [1] * 3, 32, 2, 128, 0),
    (16, [5000, 1, 130], [1] * 3, 22, 2, 128, 129),
    (16, [700, 3000], [4, 4], 8, 2, 128, 0),
    (16, [700, 3000, 12, 128], [13, 1, 12, 38], 1, 1, 128, 0),
    (16, [40000], [2], 8, 1, 128, 0),
]


@pytest.mark.parametrize("rows,lens,new,H,Hkv,D,window", DECODES)
def test_decode_kernel_matches_the_definition(csa2, rows, lens, new, H, Hkv, D, window):  # noqa: F811
    T = sum(new)
    assert _rows(csa2, T, len(lens), H, Hkv, D) == rows
    rng = np.random.default_rng(sum(lens) + H)
    pages = sum(-(-n // 128) for n in lens) + 2
    st = Store(csa2, pages, Hkv, D)
    table = _tables(rng, lens, pages)
    _fill(rng, st, lens, table, spread=8)
    q = _bf16(rng.normal(size=(T, H, D)) * 2.0 ** rng.integers(-3, 4, size=(1, H, 1)))
    out, lse, status = _attend(csa2, st, lens, new, table, q, window, D ** -0.5)
    assert status == csa2.OK
    assert check(st, lens, new, table, q, window, D ** -0.5, out, lse) == T
    again, lse2, _ = _attend(csa2, st, lens, new, table, q, window, D ** -0.5)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("S,per,H,Hkv", [(64, 1, 64, 8), (300, 1, 8, 1), (40, 2, 32, 4), (700, 1, 48, 4)])
def test_decode_batches_of_ragged_lengths(csa2, S, per, H, Hkv):  # noqa: F811
    """More jobs than CTAs and fewer, over pages that the sequences share."""
    rng = np.random.default_rng(S)
    lens = [int(v) for v in np.exp(rng.uniform(np.log(per), np.log(9000), S))]
    st = Store(csa2, 71, Hkv, 128)
    order = rng.permutation(71).astype(np.int32)
    table = np.stack([np.roll(order, s)[:71] for s in range(S)])
    _fill(rng, st, [71 * 128], order[None], spread=6)
    q = _bf16(rng.normal(size=(S * per, H, 128)) * 2.0)
    out, lse, status = _attend(csa2, st, lens, None, table, q, 0, 128 ** -0.5, per=per)
    assert status == csa2.OK
    assert check(st, lens, [per] * S, table, q, 0, 128 ** -0.5, out, lse) == S * per


def _decode_steps(seed, S, H, Hkv, D, n):
    rng = np.random.default_rng(seed)
    for _ in range(n):
        yield [1] * S, *(_bf16(rng.normal(size=(S, h, D))) for h in (H, Hkv, Hkv))


@pytest.mark.parametrize("H,Hkv,D,rows", [(16, 2, 128, 8), (32, 2, 64, 16)])
@pytest.mark.parametrize("captured", [False, True])
def test_serving_steps_of_single_tokens(csa2, H, Hkv, D, rows, captured):  # noqa: F811
    """Steps of one token for each of 5 requests, with no spare rows: plan, rotation, append and the
    decode kernel together, eager and as one graph; the first requests end up past a page."""
    S = 5
    assert _rows(csa2, S, S, H, Hkv, D) == rows
    srv = Server(csa2, S, S, H, Hkv, D, 12, 0)
    big = Server(csa2, S, 140 * S, H, Hkv, D, 12, 0)              # fills the prompts
    for a in ("table", "free", "old", "new", "used", "st"):
        setattr(srv, a, getattr(big, a))
    srv.seqs = csa2.make_seqs(None, srv.plan["seq_len"], q_seq=srv.plan["q_seq"], block_table=srv.table)
    rng = np.random.default_rng(3)
    prompt = [126, 127, 140, 1, 15]
    lens, kept = [0] * S, [[[] for _ in range(S)] for _ in "kv"]
    f = dict(scaling="parts", factor=4.0)
    graph = None

    def note(new, k, v):
        t = 0
        for s, n in enumerate(new):
            pos = np.arange(lens[s], lens[s] + n)
            kept[0][s].append(R.rope(k[t:t + n].double().cpu().numpy(), pos, D, **f))
            kept[1][s].append(v[t:t + n].double().cpu().numpy())
            lens[s] += n
            t += n

    q, k, v = (_bf16(rng.normal(size=(sum(prompt), h, D))) for h in (H, Hkv, Hkv))
    big.feed(prompt, q, k, v)
    big.calls()
    note(prompt, k, v)
    big.advance()
    if captured:
        srv.new.zero_()
        srv.calls()                                               # nothing is stored
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            srv.calls()
    for new, q, k, v in _decode_steps(4, S, H, Hkv, D, 5):
        srv.feed(new, q, k, v)
        graph.replay() if captured else srv.calls()
        assert [csa2.status_fetch(w) for w in srv.ws + big.ws] == [csa2.OK] * 6
        note(new, k, v)
        assert srv.plan["seq_len"].tolist() == lens
        table = srv.table.cpu().numpy()
        (kc, vc), (ke, ve) = srv.st.host()
        for s in range(S):
            for had, c, e in ((kept[0][s], kc, ke), (kept[1][s], vc, ve)):
                want = np.concatenate(had)
                got = R.sequence(c, e, table[s, :-(-lens[s] // 128)], lens[s])
                for b in range(0, lens[s], 16):
                    w, g = want[b:b + 16], got[b:b + 16]
                    top = np.abs(w).max(axis=(0, 2), keepdims=True)
                    # half a step of the code twice (a growing scale moves older codes)
                    assert np.all(np.abs(g - w) <= 2 * (np.abs(w) * 2.0 ** -4 + top / 224 * 2.0 ** -10) + 1e-6)
        # V has block exponents of its own here: the bound of tests/gpu_kv8.py
        check(srv.st, lens, new, table, srv.q, 0, srv.scale, srv.out, srv.lse)
        srv.advance()
