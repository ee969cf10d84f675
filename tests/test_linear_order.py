"""The scales of the few-token FP8 product between its epilogue warps, on the host.

One warp writes the scales of a block of inputs to a row of a small table, all
four meet at a barrier, then each reads the row.  Nothing but the next block's
barrier holds the writer back, so a row may be written again only behind the
barrier that follows its reading, also where a thread block goes on to another
tile.
"""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(__file__), "..", "serving_router_sigmoid_gb300", "csrc", "k_fp8lin.cu")
# the row of a block of inputs: k counts within a tile, n accumulators from the start
ROWS = {"k & 3": lambda k, n: k & 3, "acc.slot": lambda k, n: n & 1}


def rows_of_the_kernel():
    with open(SOURCE) as f:
        found = set(re.findall(r"sm\.sc\[([^\]]+)\]", f.read()))
    assert len(found) == 1, found
    return ROWS[found.pop()]


def stale(blocks, tiles, row, seed):
    """Whether a warp reads scales of another block of inputs."""
    r, table, met, at = random.Random(seed), {}, [0] * 4, [0] * 4

    def warp(w):
        for tile in range(tiles):
            for k in range(blocks):
                i = row(k, tile * blocks + k)
                if w == 0:
                    table[i] = (tile, k)
                met[w] += 1
                while min(met) < met[w]:
                    yield None
                for _ in range(r.choice([0, 0, 1, 4])):
                    yield None
                yield table[i] != (tile, k)
    warps = {w: warp(w) for w in range(4)}
    while warps:
        w = r.choice(list(warps))
        try:
            if next(warps[w]):
                return True
        except StopIteration:
            del warps[w]
            met[w] = 1 << 30
    return False


@pytest.mark.parametrize("blocks", [1, 2, 3, 4, 5, 9])
def test_scales_are_read_before_they_are_written_again(blocks):
    row = rows_of_the_kernel()
    assert not any(stale(blocks, 6, row, s) for s in range(200))


def test_the_model_sees_a_row_written_too_early():
    assert any(stale(5, 6, ROWS["k & 3"], s) for s in range(200))
    assert not any(stale(4, 6, ROWS["k & 3"], s) for s in range(200))
