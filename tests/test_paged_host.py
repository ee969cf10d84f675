"""Host side of the paged-cache operators: rotary frequencies against the
formula, and refusals that answer before the GPU is touched."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def moe():
    import serving_router_sigmoid_gb300 as m
    return m


def turns(moe, rot, base=10000.0, scaling=0, factor=1.0, original=4096, fast=32.0, slow=1.0):
    from serving_router_sigmoid_gb300._paged import MoeRopeDesc
    out, amp = (ctypes.c_uint64 * max(1, rot // 2))(), ctypes.c_float(0)
    rc = moe.library().moe_rope_turns(ctypes.byref(MoeRopeDesc(rot, base, scaling, factor, original, fast, slow)), out,
                                      ctypes.byref(amp))
    return rc, [v / 2.0**64 for v in out], amp.value


@pytest.mark.parametrize("rot", [2, 6, 64, 128, 512])
def test_frequencies_follow_the_formula(moe, rot):
    th = [10000.0 ** (-2 * i / rot) for i in range(rot // 2)]
    rc, got, amp = turns(moe, rot)
    assert rc == 0 and amp == 1.0
    # a turn fraction in 64 bits of a frequency in 53: 2^-52 relative, 2^-64 absolute
    for t, g in zip(th, got):
        assert abs(g - t / (2 * math.pi)) <= t * 2.0**-52 + 2.0**-63
    rc, got, amp = turns(moe, rot, scaling=1, factor=4.0)
    for t, g in zip(th, got):
        assert abs(g - t / 4 / (2 * math.pi)) <= t * 2.0**-52 + 2.0**-63
    if rot > 2:
        rc, got, amp = turns(moe, rot, scaling=2, factor=4.0)
        b = 10000.0 * 4.0 ** (rot / (rot - 2))
        for i, g in enumerate(got):
            t = b ** (-2 * i / rot)
            assert abs(g - t / (2 * math.pi)) <= t * 2.0**-48 + 2.0**-63  # two powers: 2^-49 of the base's error
        # by design the lowest frequency is divided by the factor
        assert abs(got[-1] * 4 / (th[-1] / (2 * math.pi)) - 1) < 1e-9


def test_scaling_by_parts(moe):
    rc, got, amp = turns(moe, 128, scaling=3, factor=8.0, original=16384)
    assert rc == 0 and abs(amp - (0.1 * math.log(8) + 1)) < 1e-6
    for i, g in enumerate(got):
        t = 10000.0 ** (-2 * i / 128)
        r = 16384 * t / (2 * math.pi)
        keep = min(1, max(0, (r - 1) / 31))
        want = t * (keep + (1 - keep) / 8) / (2 * math.pi)
        assert abs(g - want) <= want * 2.0**-48 + 2.0**-63
    assert got[0] == turns(moe, 128)[1][0]  # the fastest pair keeps its frequency


def test_rope_refusals(moe):
    for bad in (dict(rot=0), dict(rot=3), dict(rot=514)):
        assert turns(moe, **bad)[0] == moe.MOE_ERR_SHAPE
    for bad in (dict(base=0.0), dict(base=float("nan")), dict(scaling=9), dict(scaling=1, factor=0.5),
                dict(scaling=3, factor=2.0, original=0), dict(scaling=3, factor=2.0, fast=1.0, slow=1.0)):
        assert turns(moe, 64, **bad)[0] == moe.MOE_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        moe.Rope(64, scaling="cubic")


def test_null_and_bad_sizes_answer_on_the_host(moe):
    lib = moe.library()
    plan = lambda n, page, room=0: lib.moe_kv_plan(None, None, n, None, 0, None, page, None, 0, 0, room, None,  # noqa: E731
                                                   None, None, None, None, None)
    assert plan(-1, 16) == moe.MOE_ERR_SHAPE and plan(8193, 16) == moe.MOE_ERR_SHAPE
    assert plan(1, 0) == moe.MOE_ERR_SHAPE and plan(1, 16, -1) == moe.MOE_ERR_SHAPE
    assert plan(1, 16) == moe.MOE_ERR_INVALID_ARG
    assert lib.moe_rope_append(None, None) == moe.MOE_ERR_INVALID_ARG
    assert lib.moe_block_norm(None, None) == moe.MOE_ERR_INVALID_ARG
    assert lib.moe_attn_decode(None, None, None) == moe.MOE_ERR_INVALID_ARG
    assert lib.moe_attn_destroy(None) == moe.MOE_OK
    from serving_router_sigmoid_gb300._paged import MoeAttnDesc
    h = ctypes.c_void_p()
    for bad in ((0, 8, 2, 64, 64), (8193, 8, 2, 64, 64), (1, 8, 3, 64, 64), (1, 8, 2, 60, 64), (1, 8, 2, 64, 264),
                (1, 2048, 2, 64, 64)):
        assert lib.moe_attn_create(ctypes.byref(MoeAttnDesc(*bad)), ctypes.byref(h)) == moe.MOE_ERR_SHAPE


def test_cpu_tensors_are_refused(moe):
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        moe.block_norm(x, x)
    with pytest.raises(ValueError):
        moe.KvPlan(1, 1, 16, device="cpu")
