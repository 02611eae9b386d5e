"""The convolution's map from grid slots to tokens (tests/test_conv_tiles.py) at the tile
sizes that its launches have, read from the source (CPU): four runs of 16 or 4 tokens
forward, of 64 or 16 steps less K - 1 backward.  Most are no powers of two."""
import os
import random
import re

import pytest

from tests.test_conv_tiles import slots, tile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = open(os.path.join(ROOT, "state_space_model_ssd_amd", "csrc", "ssd_conv.hip")).read()


def constant(name):
    return int(re.search(rf"\b{name} = (\d+)", SOURCE).group(1))


def tile_sizes():
    waves = constant("kConvThreads") // 64
    out = {constant(n) * waves for n in ("kConvFwdLong", "kConvFwdShort")}
    out |= {(constant(n) - (K - 1)) * waves for n in ("kConvBwdLong", "kConvBwdShort") for K in (2, 3, 4)}
    return sorted(out)


def test_sizes_of_the_launches():
    assert tile_sizes() == [16, 52, 56, 60, 64, 244, 248, 252]


@pytest.mark.parametrize("WT", tile_sizes())
def test_every_token_is_covered_once_at_the_launches_sizes(WT):
    rnd = random.Random(WT)
    for _ in range(12):
        nseq = rnd.choice((1, 2, 5, 63, 64, 65, 200, 4100))
        lens = [rnd.choice((0, 0, 1, 2, 3, WT - 1, WT, WT + 1, rnd.randint(0, 3 * WT)))
                if nseq < 300 else rnd.randint(0, 2) for _ in range(nseq)]
        lead, tail = rnd.choice((0, 0, 3, WT)), rnd.choice((0, 0, 5, 2 * WT))
        cu = [lead]
        for n in lens:
            cu.append(cu[-1] + n)
        total, next_token = cu[-1] + tail, {}
        for i in range(slots(total, nseq, WT)):
            s, start, end, lo, hi = tile(cu, nseq, total, WT, i)
            if lo >= hi:
                continue
            assert (start, end) == (cu[s], cu[s + 1]) and start <= lo and hi <= end and hi - lo <= WT
            assert next_token.get(s, start) == lo          # the sequence's tiles in order, no gap
            next_token[s] = hi
        assert next_token == {s: cu[s + 1] for s in range(nseq) if lens[s] > 0}


@pytest.mark.parametrize("WT", tile_sizes())
def test_malformed_packings_stay_inside_at_the_launches_sizes(WT):
    rnd = random.Random(WT)
    big = 2 ** 31 - 1
    for _ in range(60):
        nseq, total = rnd.choice((1, 2, 7, 64, 65, 130)), rnd.randint(1, 900)
        cu = [rnd.choice((rnd.randint(-10, 1000), -big - 1, big)) for _ in range(nseq + 1)]
        for i in range(slots(total, nseq, WT)):
            s, start, end, lo, hi = tile(cu, nseq, total, WT, i)
            if lo < hi:
                assert 0 <= start <= lo < hi <= end <= total
