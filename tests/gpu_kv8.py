"""Attention over the 8-bit cache from its definition, in 64 bits on the GPU, and the bound that its
outputs are held to: for batches that the loops of oracle/kv8_ref.py would take minutes for.
"""
import torch


def _cache(st, kv, pages, n, h):
    """Codes as values and exponents of the first n tokens of a sequence, KV head h."""
    c = st.dev[kv][pages, h].view(torch.float8_e4m3fn).double().reshape(-1, st.D)[:n]
    e = (st.exp[kv][pages, h].double() - 127).clamp(-60, 60).repeat_interleave(16, 1).reshape(-1)[:n]
    return c, e


def check(st, lens, new, table, q, window, scale, out, lse, least=2.0 ** -22):
    """Every row of out and lse against the definition; returns the rows checked.  The bound is
      d    = scale * (D * 2^-23 * max_j sum|q k| + 2^-17 * max|q| * max_j sum|k|) + 2^-18 * (|lse| + 70)
      lse    d + 2^-20 |lse|
      out    2^-8 |out| + (2^-11 + 2 d) * sum p |v| + least * max_j(p_j 2^e_j) * sum |code|:
    fp32 sums, Q's second term, the fp32 exponent, one rounding to bf16, and weights w 2^e that are
    off by at most 2^-11 of themselves (2^-14 from 2^-10 of the largest on in the decode kernel) and
    ``least`` of the row's largest."""
    t = 0
    D, G = st.D, q.shape[1] // st.H
    for s, (n_len, n) in enumerate(zip(lens, new)):
        pages = torch.as_tensor(table[s, :-(-n_len // 128)], device="cuda").long()
        pos = torch.arange(n_len - n, n_len, device="cuda").repeat_interleave(G)[:, None]
        j = torch.arange(n_len, device="cuda")[None]
        hidden = (j > pos) | (j <= pos - window) if window else j > pos
        empty = hidden.all(1) if n_len else torch.ones_like(pos[:, 0], dtype=torch.bool)
        for h in range(st.H if n else 0):
            heads = slice(h * G, h * G + G)
            go = out[t:t + n, heads].double().reshape(n * G, D)
            gl = lse[t:t + n, heads].double().reshape(n * G)
            assert torch.equal(gl == -torch.inf, empty), (s, h)
            assert not go[empty].any()
            if bool(empty.all()):
                continue
            qs = q[t:t + n, heads].double().reshape(n * G, D)
            (kc, ke), (vc, ve) = _cache(st, 0, pages, n_len, h), _cache(st, 1, pages, n_len, h)
            k, v = kc * torch.exp2(ke)[:, None], vc * torch.exp2(ve)[:, None]
            see = (~hidden).double()
            # what nobody sees may hold NaN codes
            seen = (~hidden).any(0)
            k[~seen], v[~seen], vc[~seen] = 0, 0, 0
            x = (qs @ k.T * scale).masked_fill_(hidden, -torch.inf)
            wl = torch.logsumexp(x, 1)
            p = torch.softmax(x, 1).nan_to_num_(0.0)
            terms = ((qs.abs() @ k.abs().T) * see).amax(1)
            small = qs.abs().amax(1) * (see * k.abs().sum(1)).amax(1)
            d = scale * (D * 2.0 ** -23 * terms + 2.0 ** -17 * small) + 2.0 ** -18 * (wl.abs() + 70)
            err = (gl - wl).abs() - d - 2.0 ** -20 * wl.abs()
            assert bool((err <= 0)[~empty].all()), (s, h, float(err[~empty].max()))
            want = p @ v
            tol = (want.abs() * 2.0 ** -8 + (2.0 ** -11 + 2 * d)[:, None] * (p @ v.abs())
                   + least * (p * torch.exp2(ve)).amax(1)[:, None] * (see @ vc.abs()))
            bad = ((go - want).abs() - tol)[~empty]
            assert bool((bad <= 0).all()), (s, h, float(bad.max()))
        t += n
    return t
