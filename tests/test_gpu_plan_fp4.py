"""The page plan ahead of the FP4 cache, one entry per token: its rows as csa2_quant_append's dst_row,
its q_seq and q_pos for the indexer and csa2_sparse_attn, over two steps of ragged prefills and
decodes.  Codes and indices are equal to the definitions; attention is within the FP4 path's
tolerance (max-abs 2e-2, rel-L2 1e-2)."""
import math

import numpy as np
import pytest
import torch

from oracle import csa2_ref as R
from tests import oracle_harness as OH

pytestmark = pytest.mark.gpu

S, D, H, H_I, d_I, TOPK, WINDOW = 3, 128, 16, 4, 64, 64, 128


class Fp4:
    """Pages of the FP4 cache and of the indexer's keys, and the requests' lengths."""

    def __init__(self, csa2, pages=9):
        self.csa2 = csa2
        z = lambda *s, dtype=torch.uint8: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
        self.codes, self.scales = z(pages * 128, D // 2), z(pages * 128, D // 16)
        self.idx_k = z(pages * 128, d_I, dtype=torch.bfloat16)
        self.table = torch.full((S, 4), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(pages, device="cuda").to(torch.int32)
        self.old, self.used = z(S, dtype=torch.int32), z(1, dtype=torch.int32)
        self.ws = csa2.workspace(csa2.quant_append_workspace())

    def step(self, new, spare, x, kI):
        c = self.csa2
        T = sum(new)
        out = c.plan_outputs(S, T + spare)
        ws = c.workspace(c.plan_pages_workspace())
        c.plan_pages(self.old, torch.tensor(new, dtype=torch.int32, device="cuda"), self.table, self.free,
                     self.used, out, ws)
        assert c.status_fetch(ws) == c.OK
        c.quant_append(x, out["rows"][:T], self.codes, self.scales, self.ws, kI, self.idx_k)
        assert c.status_fetch(self.ws) == c.OK
        self.old, self.used = out["seq_len"].clone(), out["free_used"].clone()
        return out


def _bf16(rng, *shape):
    return torch.from_numpy(rng.normal(size=shape).astype(np.float32)).cuda().to(torch.bfloat16)


@pytest.mark.parametrize("spare", [0, 5])
def test_plan_feeds_the_fp4_cache(spare):
    from fp4_kv_cache_03_b200 import csa2
    rng = np.random.default_rng(5)
    torch.manual_seed(5)
    m = Fp4(csa2)
    kept_x, kept_k = [[] for _ in range(S)], [[] for _ in range(S)]
    for new in ([200, 0, 130], [1, 37, 1], [1, 1, 1]):
        T = sum(new)
        x = torch.from_numpy(rng.normal(size=(T, D)).astype(np.float32)).cuda()
        kI = torch.from_numpy(rng.integers(-4, 5, size=(T, d_I)).astype(np.float32)).cuda().to(torch.bfloat16)
        out = m.step(new, spare, x, kI)
        t = 0
        for s, n in enumerate(new):
            kept_x[s].append(x[t:t + n].cpu().numpy())
            kept_k[s].append(kI[t:t + n].float().cpu().numpy())
            t += n
        seq, pos, rows = out["q_seq"][:T].contiguous(), out["q_pos"][:T].contiguous(), out["rows"][:T]
        seqs = csa2.make_seqs(None, out["seq_len"], q_per_seq=0, q_seq=seq, block_table=m.table)
        assert torch.equal(csa2.cache_rows(seqs, seq, pos.int()), rows)
        for s in range(S):
            if not sum(len(v) for v in kept_x[s]):
                continue
            n = int(out["seq_len"][s])
            r = csa2.cache_rows(seqs, torch.full((n,), s, dtype=torch.int32, device="cuda"),
                                torch.arange(n, dtype=torch.int32, device="cuda"))
            codes, scales = R.quantize_rows(np.concatenate(kept_x[s]))
            np.testing.assert_array_equal(m.codes[r].cpu().numpy(), codes)
            np.testing.assert_array_equal(m.scales[r].cpu().numpy(), scales)
        # indexer and attention of the step's tokens
        qI = torch.from_numpy(rng.integers(-4, 5, size=(T, H_I, d_I)).astype(np.float32)).cuda().to(torch.bfloat16)
        w = torch.from_numpy(rng.integers(1, 5, size=(T, H_I)).astype(np.float32)).cuda()
        idx = torch.full((T, TOPK), -7, dtype=torch.int32, device="cuda")
        ws_i = csa2.workspace(csa2.index_full_workspace(T, 512, TOPK))
        csa2.index_full(qI, w, m.idx_k, seqs, TOPK, idx, ws_i, 512, q_visible=(pos + 1).int())
        q = _bf16(rng, T, H, D)
        lens = [int(v) for v in out["seq_len"]]
        swa_start = np.concatenate([[0], np.cumsum(lens)[:-1]])
        swa = _bf16(rng, sum(lens), D)
        got, lse = torch.zeros(T, H, D, device="cuda"), torch.zeros(T, H, device="cuda")
        ws_a = csa2.workspace(csa2.sparse_attn_workspace(T, H, D, TOPK, WINDOW))
        csa2.sparse_attn(q, m.codes, m.scales, seqs, idx, swa, torch.from_numpy(swa_start).cuda(), pos, WINDOW,
                         1.0 / math.sqrt(D), got, ws_a, lse=lse)
        assert csa2.status_fetch(ws_i) == csa2.OK and csa2.status_fetch(ws_a) == csa2.OK
        for i in range(0, T, 1 if T < 50 else 23):
            s, p = int(seq[i]), int(pos[i])
            keys = np.concatenate(kept_k[s])[:p + 1]
            sc = R.index_scores(qI[i].float().cpu().numpy(), w[i].cpu().numpy(), keys)
            want = R.topk_ascending(sc, TOPK)
            np.testing.assert_array_equal(idx[i].cpu().numpy(), want)
            sel = R.dequantize_rows(*R.quantize_rows(np.concatenate(kept_x[s])[want[want >= 0]]))
            win = swa[int(swa_start[s]) + R.window_positions(p, WINDOW)].float().cpu().numpy()
            ref, _ = R.sparse_attention(q[i].float().cpu().numpy(), sel, win, 1.0 / math.sqrt(D))
            ok, mx, rl2 = OH.attn_close(got[i].cpu().numpy(), ref)
            assert ok, (i, mx, rl2)


def test_spare_tokens_are_reported_by_the_fp4_calls():
    """What the header says of the maps' -1: each of these calls records an error for them and does
    the others' work."""
    from fp4_kv_cache_03_b200 import csa2
    rng = np.random.default_rng(6)
    torch.manual_seed(6)
    m = Fp4(csa2)
    x = torch.from_numpy(rng.normal(size=(6, D)).astype(np.float32)).cuda()
    kI = torch.ones(6, d_I, device="cuda", dtype=torch.bfloat16)
    out = m.step([2, 1, 3], 2, x, kI)
    codes = m.codes.clone()
    m.codes.zero_()
    more = torch.cat([x, x[:2]])
    csa2.quant_append(more, out["rows"], m.codes, m.scales, m.ws)
    assert csa2.status_fetch(m.ws) == csa2.ERR_CAPACITY and torch.equal(m.codes, codes)
    seqs = csa2.make_seqs(None, out["seq_len"], q_per_seq=0, q_seq=out["q_seq"], block_table=m.table)
    idx = torch.full((8, TOPK), -7, dtype=torch.int32, device="cuda")
    ws = csa2.workspace(csa2.index_full_workspace(8, 512, TOPK))
    csa2.index_full(torch.ones(8, H_I, d_I, device="cuda", dtype=torch.bfloat16), torch.ones(8, H_I, device="cuda"),
                    m.idx_k, seqs, TOPK, idx, ws, 512)
    assert csa2.status_fetch(ws) == csa2.ERR_INVALID_ARG
    assert bool((idx[6:] == -1).all()) and bool((idx[:6, 0] == 0).all())
