"""The division of attention over the 8-bit cache among CTAs, replayed on the host: which key tiles
each half of a prefill job sees, in the order in which its CTA takes them.  For the choice of test
cases; shares no code with the kernels.
"""
PAGE, ROWS = 128, 256


def shares(total, ctas):
    """Equal contiguous parts of ``total`` tiles."""
    ctas = max(1, min(ctas, total))
    each, more = divmod(total, ctas)
    cut = [each * c + more * c // ctas for c in range(ctas + 1)]
    return list(zip(cut, cut[1:]))


def jobs(lens, new, G, Hkv, window):
    """(first key tile, key tiles, [(lo, hi) of half 0, of half 1]) in the order of the walk."""
    QT = ROWS // G
    out = []
    for n_len, n in zip(lens, new):
        for i in range(0, n, QT):
            p0, nq = n_len - n + i, min(QT, n - i)
            seen = lambda p: max(0, p - window + 1) // PAGE if window else 0
            first = seen(p0)
            count = max(1, -(-max(0, p0 + nq) // PAGE) - first)
            halves = []
            for x in range(2):
                rows = (min(nq * G, 128), max(0, nq * G - 128))[x]
                a = p0 + x * 128 // G
                b = p0 + (min(nq * G, 128) - 1, nq * G - 1)[x] // G
                halves.append((seen(a), b // PAGE + 1 if rows and b >= 0 else 0))
            out += [(first, count, halves)] * Hkv
    return out


def idle_runs(lens, new, H, Hkv, window, ctas=148):
    """The longest distance, in tiles of a CTA, between two tiles that a half of it computes (from
    one before the first)."""
    work = jobs(lens, new, H // Hkv, Hkv, window)
    flat = [(j, k) for j, (_, count, _) in enumerate(work) for k in range(count)]
    most = 0
    for begin, end in shares(len(flat), ctas):
        latest = [-1, -1]
        for g, (j, k) in enumerate(flat[begin:end]):
            first, _, halves = work[j]
            for x, (lo, hi) in enumerate(halves):
                if lo <= first + k < hi:
                    most = max(most, g - latest[x])
                    latest[x] = g
    return most
