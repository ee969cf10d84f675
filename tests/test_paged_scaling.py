"""Frequencies scaled by parts, linear in the pair's index, and an amplitude of
the caller's own."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def moe():
    import serving_router_sigmoid_gb300 as m
    return m


def turns(moe, rot, base, factor, original, fast, slow, scaling=4):
    from serving_router_sigmoid_gb300._paged import MoeRopeDesc
    out, amp = (ctypes.c_uint64 * (rot // 2))(), ctypes.c_float(0)
    rc = moe.library().moe_rope_turns(ctypes.byref(MoeRopeDesc(rot, base, scaling, factor, original, fast, slow)), out,
                                      ctypes.byref(amp))
    return rc, [v / 2.0**64 for v in out], amp.value


@pytest.mark.parametrize("rot,base,factor,original,fast,slow", [
    (128, 10000.0, 8.0, 16384, 32.0, 1.0), (64, 10000.0, 40.0, 4096, 32.0, 1.0), (128, 1e6, 4.0, 32768, 32.0, 1.0),
    (128, 10000.0, 4.0, 8, 32.0, 1.0), (64, 10000.0, 2.0, 2**30, 32.0, 1.0), (16, 500000.0, 16.0, 8192, 4.0, 1.0)])
def test_linear_in_the_index(moe, rot, base, factor, original, fast, slow):
    rc, got, amp = turns(moe, rot, base, factor, original, fast, slow)
    assert rc == 0 and abs(amp - (0.1 * math.log(factor) + 1)) < 1e-6
    th = [base ** (-2 * i / rot) for i in range(rot // 2)]
    in_len = [original * t / (2 * math.pi) for t in th + [base ** (-2 * i / rot) for i in range(rot // 2, rot)]]
    # the bounds by counting: indices 0..rot-1, whose pairs turn less and less
    low = max([i for i, n in enumerate(in_len) if n >= fast], default=0)
    high = min([i for i, n in enumerate(in_len) if n <= slow], default=rot - 1)
    for i, (t, g) in enumerate(zip(th, got)):
        part = min(1.0, max(0.0, (i - low) / (high - low))) if high > low else float(i > low)
        want = t * (1 - part + part / factor) / (2 * math.pi)
        assert abs(g - want) <= want * 2.0**-48 + 2.0**-63, (i, low, high)


def test_both_ramps_agree_at_their_ends_and_differ_between(moe):
    a, b = (turns(moe, 128, 10000.0, 8.0, 16384, 32.0, 1.0, s)[1] for s in (3, 4))
    assert a[0] == b[0] and a[-1] == b[-1]
    assert max(abs(x / y - 1) for x, y in zip(a, b)) > 0.1


def test_refusals(moe):
    for bad in (dict(slow=0.0), dict(slow=-1.0), dict(base=1.0), dict(base=0.5), dict(original=0), dict(fast=1.0),
                dict(factor=0.5), dict(scaling=5)):
        kw = dict(rot=64, base=10000.0, factor=2.0, original=4096, fast=32.0, slow=1.0)
        kw.update(bad)
        assert turns(moe, **kw)[0] == moe.MOE_ERR_INVALID_ARG, bad


@pytest.mark.gpu
@pytest.mark.parametrize("scaling", ["none", "parts", "parts_by_index"])
def test_an_amplitude_of_ones_own(moe, scaling):
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn((40, 2, 64), generator=g, device="cuda")
    cache = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    pos, slots = torch.arange(40, dtype=torch.int32, device="cuda") + 5000, torch.arange(40, device="cuda")
    kw = dict(scaling=scaling, factor=8.0, original_len=1024)
    own, one, two = moe.Rope(64, **kw), moe.Rope(64, amplitude=1.0, **kw), moe.Rope(64, amplitude=2.0, **kw)
    assert own.amplitude == pytest.approx(1.0 if scaling == "none" else 0.1 * math.log(8) + 1, rel=1e-6)
    a, b, c = (r.append(q, q, None, pos, slots, cache, None) for r in (own, one, two))
    assert torch.equal(c, 2 * b)  # a power of two: the same roundings
    if scaling == "none":
        assert torch.equal(a, b)
    # lengths of pairs: the amplitude's factor, five roundings of fp32
    lengths = [(t.double().view(40, 2, 2, 32).square().sum(2)).sqrt() for t in (q, a)]
    assert ((lengths[1] / lengths[0] / own.amplitude - 1).abs() < 5 * 2.0**-23).all()
