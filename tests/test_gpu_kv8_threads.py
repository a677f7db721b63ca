"""The page plan and the append from several host threads at once, with shapes that take different
amounts of shared memory: each call is launched with what it needs.  The library's functions are
called without the binding, so that the threads spend their time in them."""
import ctypes
import sys
import threading

import pytest
import torch

from tests.test_gpu_kv8 import csa2  # noqa: F401

pytestmark = pytest.mark.gpu


def _i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32, device="cuda")


def _together(fn, calls, n):
    """fn(*args) n times for each of ``calls`` in a thread of its own; the statuses other than 0."""
    bad, ready = [], threading.Barrier(len(calls))

    def work(args):
        torch.cuda.set_device(0)
        ready.wait()
        for _ in range(n):
            st = fn(*args)
            if st:
                bad.append(st)

    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        threads = [threading.Thread(target=work, args=(c,)) for c in calls]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    torch.cuda.synchronize()
    return bad


def test_plans_of_different_sizes_in_several_threads(csa2):  # noqa: F811
    sides = []
    for S in (16384, 4000, 16384, 4000):
        t = [_i32(S), _i32(S), _i32(S, 1), _i32(1), _i32(1)]
        t[1][-1] = 1
        out = csa2.plan_outputs(S, 1)
        sides.append((S, t, out, csa2.workspace(csa2.plan_pages_workspace()), torch.cuda.Stream()))
    torch.cuda.synchronize()
    calls = []
    for S, (old, new, table, free, used), out, ws, stream in sides:
        p = lambda x: ctypes.c_void_p(x.data_ptr())  # noqa: E731
        calls.append((S, p(old), p(new), 1, p(table), 1, p(free), 1, p(used), p(out["free_used"]),
                      p(out["seq_len"]), p(out["tok_start"]), p(out["q_seq"]), p(out["q_pos"]),
                      p(out["rows"]), p(ws), ws.numel(), ctypes.c_void_p(stream.cuda_stream)))
    assert not _together(csa2.lib().csa2_plan_pages, calls, 10000)
    for S, _, out, ws, _ in sides:
        assert csa2.status_fetch(ws) == csa2.OK
        assert out["q_seq"].tolist() == [S - 1] and out["seq_len"][-1] == 1


def test_appends_of_different_sizes_in_several_threads(csa2):  # noqa: F811
    sides, rope = [], csa2.make_rope(128)
    for T in (40000, 20000, 40000, 20000):               # windows of 64 and of 33 tokens
        pages = -(-T // 128)
        dev = [torch.zeros(pages, 1, 128, 128, dtype=torch.uint8, device="cuda") for _ in "kv"]
        exp = [torch.zeros(pages, 1, 8, dtype=torch.uint8, device="cuda") for _ in "kv"]
        table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
        seqs = csa2.make_seqs(None, torch.full((1,), T, dtype=torch.int32, device="cuda"), T, block_table=table)
        x = torch.ones(T, 1, 128, device="cuda", dtype=torch.bfloat16)
        sides.append((T, csa2.make_kv8(*dev, *exp), seqs, x, csa2.workspace(csa2.kv8_append_workspace()),
                      torch.cuda.Stream(), exp))
    torch.cuda.synchronize()
    calls = [(ctypes.c_void_p(x.data_ptr()), 128, ctypes.c_void_p(x.data_ptr()), 128, T, cache, seqs, None,
              ctypes.byref(rope), ctypes.c_void_p(ws.data_ptr()), ws.numel(),
              ctypes.c_void_p(stream.cuda_stream)) for T, cache, seqs, x, ws, stream, _ in sides]
    assert not _together(csa2.lib().csa2_kv8_append, calls, 5000)
    for T, _, _, _, ws, _, exp in sides:
        assert csa2.status_fetch(ws) == csa2.OK
        assert bool((exp[1].flatten()[:T // 16] == 127 - 8).all())      # 1 is 256 * 2^-8
