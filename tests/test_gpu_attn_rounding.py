"""16-bit outputs of moe_attn_decode are the rounded results, not the results of
16-bit weights: how many differ from the correctly rounded 64-bit ones.

Queries and keys are small whole numbers, so that the products q . k are exact
and a weight carries the errors of its exponent (s * fac and s - m: 2^-23 rms at
these sizes) and of the exponential (2^-22 at most).  An output's error against
S = sqrt(sum (p v)^2), rms: 2^-22.8 and 2^-23 of those, half an ulp for each
step's rounded add of a warp's dozen steps (2^-23), and what the tensor cores cut
off a step's sum of three terms (2^-22.4): 2^-21.3, of which the mean size is
0.8.  With bf16 caches E = 2^-21 S bounds it.  In f16 form (f16, E4M3) every
product goes into the running sum, which loses half an ulp towards zero at each
of two terms a tile: with at most 64 tiles a warp 2 * 64 * 2/3 * 2^-24 S, below
E = 2^-17 S.  (Weights of one term: 2^-9.8 S and 2^-12.8 S; of two bf16 terms:
2^-19.5 S.)  An output whose error is e falls on another side of a rounding
boundary with the chance e / ulp, so that sum E / ulp outputs differ at most, and
four standard deviations of that count.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

F16, BF16, E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def moe():
    import serving_router_sigmoid_gb300 as m
    torch.cuda.set_device(0)
    return m


def ulps(x, dtype):
    """Distance of neighbouring values of the type at x."""
    bits, least = (10, -14) if dtype is F16 else (7, -126)
    return torch.exp2(torch.frexp(x.abs().clamp(min=2.0**least))[1].double() - 1 - bits)


@pytest.mark.parametrize("act,cache,tail", [(BF16, BF16, -21), (F16, F16, -17), (F16, E4M3, -17), (BF16, E4M3, -17)])
@pytest.mark.parametrize("dim,kv,group", [(128, 8, 8), (64, 8, 4), (128, 4, 16), (256, 4, 8)])
def test_outputs_are_rounded_once(moe, act, cache, tail, dim, kv, group):
    n, length, page = 64, 512, 16
    g = torch.Generator(device="cuda").manual_seed(dim + group)
    whole = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").float()  # noqa: E731
    q, k = whole(n, kv * group, dim).to(act), whole(n * length // page, page, kv, dim).to(cache)
    v = torch.randn((n * length // page, page, kv, dim), generator=g, device="cuda").to(cache)
    table = torch.arange(n * length // page, dtype=torch.int32, device="cuda").view(n, -1)
    scale = 2.0 ** -(3 + dim.bit_length() / 2 // 1)
    out, _ = moe.PagedAttention(n, kv * group, kv, dim).decode(
        q, k, v, table, torch.full((n,), length, dtype=torch.int32, device="cuda"), scale=scale)
    allowed = differ = 0.0
    for b in range(n):
        rows = slice(b * length // page, (b + 1) * length // page)
        kd, vd = (t[rows].flatten(0, 1).float().double() for t in (k, v))
        s = torch.einsum("hgd,lhd->hgl", q[b].double().unflatten(0, (kv, group)), kd) * scale
        p = torch.softmax(s, -1)
        want = torch.einsum("hgl,lhd->hgd", p, vd).flatten(0, 1)
        size = torch.einsum("hgl,lhd->hgd", p.square(), vd.square()).flatten(0, 1).sqrt()
        allowed += float((size * 2.0**tail / ulps(want, act)).clamp(max=1).sum())
        differ += float((out[b] != want.to(act)).sum())
    assert differ <= allowed + 4 * math.sqrt(allowed), (differ, allowed, out.numel())
