"""cos and sin of moe_rope_append by themselves: queries of (1, 0) pairs give them.

The angle is position times the pair's turns, a fraction of 2^64, exactly; the
reference takes it from there in integers and 64 bits.  With a the distance to
the nearest quarter turn, in half turns, the kernel's angle is off by at most
2^-33 (the integer's rounding) and 2^-24 a (its conversion to fp32), in half
turns; the derivative of one of cos and sin is the other; and sincospif is
within 2 ulp, 2^-22 of the value.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import serving_router_sigmoid_gb300 as m
    torch.cuda.set_device(0)
    return m


def exact(turns, pos):
    """cos, sin and the distance from a quarter turn, in 64 bits."""
    part = turns[None, :] * pos[:, None]  # int64, modulo 2^64
    quarter = ((part + (1 << 61)) >> 62) & 3
    rest = (part - (quarter << 62)).double() * 2.0**-63
    c, s = (rest * math.pi).cos(), (rest * math.pi).sin()
    odd, far = (quarter & 1).bool(), 1.0 - 2.0 * (quarter >> 1).double()
    return torch.where(odd, -s, c) * far, torch.where(odd, c, s) * far, rest.abs()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot,base", [(64, 10000.0), (128, 500000.0), (34, 10000.0)])
@pytest.mark.parametrize("start,step", [(0, 1), (100000, 7), (2**26, 12347), (2**31 - 40001, 2), (-5000, 1)])
def test_angles(moe, rot, base, inter, start, step):
    n = 20000
    rope = moe.Rope(rot, base=base, interleaved=inter)
    pos = torch.arange(n, device="cuda") * step + start
    pos = torch.where(pos < 2**31, pos, pos - 2**31)
    q = torch.zeros((n, 1, rot), device="cuda")
    (q.view(n, rot // 2, 2)[:, :, 0] if inter else q[:, 0, :rot // 2]).fill_(1.0)
    cache = torch.zeros((1, 16, 1, rot), dtype=torch.bfloat16, device="cuda")
    slots = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    got = rope.append(q, q, None, pos.int(), slots, cache, None)[:, 0]
    c, s = (got[:, 0::2], got[:, 1::2]) if inter else (got[:, :rot // 2], got[:, rot // 2:])
    wc, ws, a = exact(rope.turns, pos)
    angle = math.pi * (2.0**-33 + a * 2.0**-24)
    for g, w, other in ((c, wc, ws), (s, ws, wc)):
        bound = angle * other.abs() + w.abs() * 2.0**-22 + 2.0**-60
        off = (g.double() - w).abs()
        assert (off <= bound).all(), (int((off > bound).sum()), float((off / bound).max()))
