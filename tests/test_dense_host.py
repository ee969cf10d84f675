"""Host side of the FP8 products and the latent attention: refusals that answer
before the GPU is touched."""
import ctypes
import math

import pytest
import torch

A = 1 << 20  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def moe():
    import serving_router_sigmoid_gb300 as m
    return m


def quant(moe, x=A, act=0, xs=256, n=4, dim=256, x8=2 * A, os=256, scale=3 * A):
    return moe.library().moe_quant_act_fp8(x, act, xs, n, dim, x8, os, scale, None)


def linear(moe, n=4, inner=256, outer=100, kind=2, x8=A, xs=2 * A, w8=3 * A, ws=4 * A, out=5 * A, x_st=256, w_st=256, o_st=100):
    from serving_router_sigmoid_gb300._latent import _LINEAR_ARGS
    return moe.library().moe_fp8_linear(_LINEAR_ARGS.pack(n, inner, outer, kind, x8, xs, w8, ws, out, x_st, w_st, o_st), None)


def prompt(moe, n=2, heads=4, nq=8, nk=8, nope=128, rope=64, v=128, act=2, causal=1, scale=0.1, qst=A, kst=2 * A, q=3 * A,
           k=4 * A, kr=5 * A, val=6 * A, out=7 * A, lse=8 * A, q_t=768, q_h=192, k_t=512, k_h=128, r_t=64, v_t=512, v_h=128,
           o_t=512, o_h=128):
    from serving_router_sigmoid_gb300._latent import _PROMPT_ARGS
    return moe.library().moe_latent_prompt(
        _PROMPT_ARGS.pack(n, heads, nq, nk, nope, rope, v, act, causal, scale, qst, kst, q, k, kr, val, out, lse, q_t, q_h,
                          k_t, k_h, r_t, v_t, v_h, o_t, o_h), None)


def test_quantiser(moe):
    for bad in (dict(n=-1), dict(dim=0), dict(dim=8), dict(dim=40), dict(dim=65552), dict(xs=-16), dict(os=240),
                dict(xs=1 << 41)):
        assert quant(moe, **bad) == moe.MOE_ERR_SHAPE, bad
    for bad in (dict(act=3), dict(act=-1), dict(x=0), dict(x8=0), dict(scale=0), dict(x=A + 8), dict(x8=A + 1), dict(xs=258),
                dict(act=1, xs=260), dict(os=264), dict(x8=A), dict(scale=A + 4), dict(scale=2 * A + 128)):
        assert quant(moe, **bad) == moe.MOE_ERR_INVALID_ARG, bad
    assert quant(moe, n=0, x=0, x8=0, scale=0) == moe.MOE_OK


def test_linear(moe):
    for bad in (dict(n=-1), dict(n=(1 << 24) + 1), dict(inner=0), dict(inner=24), dict(inner=65552), dict(outer=0),
                dict(outer=(1 << 20) + 1), dict(x_st=240), dict(w_st=240), dict(o_st=99), dict(x_st=1 << 38),
                dict(n=1 << 21, outer=1 << 20, o_st=1 << 20)):
        assert linear(moe, **bad) == moe.MOE_ERR_SHAPE, bad
    for bad in (dict(kind=3), dict(x8=0), dict(xs=0), dict(w8=0), dict(ws=0), dict(out=0), dict(x8=A + 8), dict(w8=A + 4),
                dict(x_st=264), dict(w_st=260), dict(out=5 * A + 1), dict(xs=2 * A + 2), dict(out=A + 512), dict(out=2 * A + 16),
                dict(out=3 * A + 256), dict(out=4 * A), dict(o_st=(1 << 38) - 1, out=0)):
        assert linear(moe, **bad) == moe.MOE_ERR_INVALID_ARG, bad
    assert linear(moe, n=0, x8=0) == moe.MOE_OK
    assert moe.library().moe_fp8_linear(None, None) == moe.MOE_ERR_INVALID_ARG


def test_prompt(moe):
    for bad in (dict(n=-1), dict(n=8193), dict(heads=0), dict(heads=1025), dict(nq=-1), dict(nk=2**31 - 200), dict(nope=0),
                dict(nope=120), dict(rope=80), dict(rope=8), dict(nope=208), dict(v=0), dict(v=272), dict(v=100)):
        assert prompt(moe, **bad) == moe.MOE_ERR_SHAPE, bad
    for bad in (dict(act=0), dict(act=3), dict(scale=math.inf), dict(scale=math.nan), dict(scale=2.0**121), dict(scale=-2.0**121),
                dict(qst=0), dict(kst=0), dict(q=0), dict(k=0), dict(kr=0), dict(val=0), dict(out=0), dict(q=3 * A + 8),
                dict(k=4 * A + 2), dict(kr=5 * A + 4), dict(val=6 * A + 8), dict(out=7 * A + 1), dict(lse=8 * A + 2),
                dict(q_t=772), dict(k_h=4), dict(r_t=-64), dict(v_t=1 << 37), dict(o_t=-1), dict(q_t=0), dict(k_t=0), dict(v_t=0),
                dict(r_t=0), dict(out=3 * A), dict(out=4 * A + 64), dict(out=6 * A), dict(lse=5 * A), dict(lse=A), dict(lse=7 * A),
                dict(out=2 * A), dict(o_t=0), dict(o_h=0), dict(o_h=127), dict(o_t=256), dict(o_t=128, o_h=1000)):
        assert prompt(moe, **bad) == moe.MOE_ERR_INVALID_ARG, bad
    assert prompt(moe, n=0, q=0) == moe.MOE_OK and prompt(moe, nq=0, q=0) == moe.MOE_OK
    assert moe.library().moe_latent_prompt(None, None) == moe.MOE_ERR_INVALID_ARG


def test_spans_beyond_the_address_space(moe):
    """Strides times rows that pass 64 bits neither wrap around nor meet by it."""
    far = (1 << 37) - 8
    assert prompt(moe, nq=2**31 - 300, q_t=far, out=A // 2) == moe.MOE_ERR_INVALID_ARG  # out runs over the others
    assert prompt(moe, nq=2**31 - 300, q_t=512, q_h=far, out=3 * A + (1 << 30)) == moe.MOE_ERR_INVALID_ARG
    assert linear(moe, n=1 << 20, o_st=(1 << 38) - 1, kind=0, out=A // 2) == moe.MOE_ERR_INVALID_ARG


def test_handles(moe):
    from serving_router_sigmoid_gb300._latent import _LATENT_ARGS, MoeLatentDesc
    lib, h = moe.library(), ctypes.c_void_p()
    for bad in ((0, 64, 512, 64), (8193, 64, 512, 64), (1, 0, 512, 64), (1, 1025, 512, 64), (1, 64, 0, 64), (1, 64, 500, 64),
                (1, 64, 576, 64), (1, 64, 512, 72), (1, 64, 512, 80), (1, 64, 512, -16)):
        assert lib.moe_latent_create(ctypes.byref(MoeLatentDesc(*bad)), ctypes.byref(h)) == moe.MOE_ERR_SHAPE, bad
        assert not h.value
    assert lib.moe_latent_create(None, ctypes.byref(h)) == moe.MOE_ERR_INVALID_ARG
    assert lib.moe_latent_destroy(None) == moe.MOE_OK
    args = _LATENT_ARGS.pack(1, 2, 2, 16, 1, 0.1, 1.0, A, A, 1, 1, A, A, A, A, 0, 576, 0, 512, 0, 576)
    assert lib.moe_latent_decode(None, args, None) == moe.MOE_ERR_INVALID_ARG
    assert lib.moe_dense_status(None, None) == moe.MOE_ERR_INVALID_ARG


def test_structs_have_the_headers_sizes():
    from serving_router_sigmoid_gb300._latent import _LATENT_ARGS, _LINEAR_ARGS, _PROMPT_ARGS
    # fields one after another, pointers and 64-bit numbers on 8 bytes
    assert _LINEAR_ARGS.size == 4 * 4 + 5 * 8 + 3 * 8
    assert _LATENT_ARGS.size == (5 + 2) * 4 + 4 + 2 * 8 + 2 * 8 + 4 * 8 + 6 * 8
    assert _PROMPT_ARGS.size == (9 + 1) * 4 + 8 * 8 + 9 * 8


def test_cpu_tensors_are_refused(moe):
    x, i = torch.zeros(4, 256), torch.zeros(2, dtype=torch.int32)
    h = torch.zeros(4, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        moe.quant_act_fp8(x)
    with pytest.raises(ValueError):
        moe.fp8_linear(x.to(torch.float8_e4m3fn), torch.ones(4, 2), x.to(torch.float8_e4m3fn), torch.ones(1, 2))
    with pytest.raises(ValueError):
        moe.latent_prompt(h, h, None, h, i, i, 0.1)
    with pytest.raises(ValueError):
        moe.LatentAttention(1, 4, device="cpu")
