"""The convolution's map from grid slots to tokens, restated in Python (CPU):
slot i of a launch with WT-token tiles is sequence s and tile i - s for the
largest s with tile(cu[s]) + s <= i, found by probing 64 sequences at a time.
Every token is covered exactly once for well-formed packings, and no token
outside the tensor is ever named for malformed ones."""
import random

import pytest


def tile(cu, nstates, total, WT, slot):
    cl = lambda v: min(max(v, 0), total)  # noqa: E731
    lo, n = 0, nstates
    while n > 1:
        step = (n + 63) // 64
        ok = [lane * step < n and cl(cu[min(lo + lane * step, nstates)]) // WT + lo + lane * step <= slot
              for lane in range(64)]
        cnt = max(1, sum(ok))
        end = lo + n
        lo += (cnt - 1) * step
        n = min(step, end - lo)
    assert 0 <= lo < nstates
    start = cl(cu[lo])
    end = max(start, cl(cu[lo + 1]))
    t = slot - lo
    return lo, start, end, max(t * WT, start), min(t * WT + WT, end)


def slots(total, nstates, WT):
    return (total + WT - 1) // WT + nstates


@pytest.mark.parametrize("WT", [8, 32, 64])
def test_every_token_is_covered_once(WT):
    rnd = random.Random(WT)
    for _ in range(40):
        nseq = rnd.choice((1, 2, 5, 63, 64, 65, 200, 4100))
        lens = [rnd.choice((0, 0, 1, 2, 3, WT - 1, WT, WT + 1, rnd.randint(0, 5 * WT)))
                if rnd.random() < 0.5 or nseq < 300 else rnd.randint(0, 2) for _ in range(nseq)]
        lead, tail = rnd.choice((0, 0, 3, WT)), rnd.choice((0, 0, 5, 2 * WT))
        cu = [lead]
        for n in lens:
            cu.append(cu[-1] + n)
        total = cu[-1] + tail
        seen = {}
        for i in range(slots(total, nseq, WT)):
            s, start, end, lo, hi = tile(cu, nseq, total, WT, i)
            for t in range(lo, hi):
                assert t not in seen
                seen[t] = s
                assert cu[s] <= t < cu[s + 1] and (start, end) == (cu[s], cu[s + 1])
        assert sorted(seen) == list(range(cu[0], cu[-1]))


def test_malformed_packings_stay_inside():
    rnd = random.Random(3)
    big = 2 ** 31 - 1
    for _ in range(200):
        nseq, total, WT = rnd.choice((1, 2, 7, 64, 65, 130)), rnd.randint(1, 500), rnd.choice((8, 32, 64))
        cu = [rnd.choice((rnd.randint(-10, 600), -big - 1, big)) for _ in range(nseq + 1)]
        for i in range(slots(total, nseq, WT)):
            s, start, end, lo, hi = tile(cu, nseq, total, WT, i)
            if lo < hi:
                assert 0 <= start <= lo < hi <= end <= total
