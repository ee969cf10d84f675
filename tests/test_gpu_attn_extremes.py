"""moe_attn_decode where one token's logit stands far above all others: the
output is that token's value row and the log-sum-exp its logit.

Queries and keys are powers of two, one dimension at a time, so that logits are
exact; the gaps are beyond what an exponential in fp32 can show.  out = (w v) /
w: exact in a 16-bit type that holds v, three half-ulps in fp32 (the product,
the reciprocal, its product).  lse = (m + log2 w) ln 2: the factors log2 e and
ln 2 and three products and a sum, each half an ulp: 2^-21 of it.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, F16, BF16, E4M3 = torch.float32, torch.float16, torch.bfloat16, torch.float8_e4m3fn
PAGE = 16


@pytest.fixture(scope="module")
def moe():
    import serving_router_sigmoid_gb300 as m
    torch.cuda.set_device(0)
    return m


def decode(moe, q, k, v, length, scale):
    """One request a row of q [n, dim], one head; k, v [n * length, dim]."""
    n, dim = q.shape
    rows = -(-length // PAGE)
    table = torch.arange(n * rows, dtype=torch.int32, device="cuda").view(n, rows)

    def paged(t):
        full = torch.full((n, rows * PAGE, dim), 0.0, device="cuda").to(t.dtype)
        full.view(torch.uint8).fill_(0x7F)  # NaN, or near it, beyond the request
        full.view(torch.uint8)[:, :length] = t.view(n, length, dim).view(torch.uint8)
        return full.view(n * rows, PAGE, 1, dim)

    out, lse = moe.PagedAttention(n, 1, 1, dim).decode(
        q[:, None], paged(k), paged(v), table, torch.full((n,), length, dtype=torch.int32, device="cuda"), scale=scale)
    return out[:, 0], lse[:, 0]


def check(moe, act, cache, length, winner, q_row, keys, scale, dim=64):
    """q_row, keys: the numbers in the dimension that n requests use (one each)."""
    n = len(winner)
    g = torch.Generator(device="cuda").manual_seed(length)
    at = torch.randint(0, dim, (n,), generator=g, device="cuda")
    q, k = torch.zeros((n, dim), device="cuda"), torch.zeros((n, length, dim), device="cuda")
    q[torch.arange(n), at] = q_row
    k.scatter_(2, at[:, None, None].expand(n, length, 1), keys[:, :, None])
    q, k = q.to(act), k.to(cache)
    v = torch.randn((n, length, dim), generator=g, device="cuda").to(cache)
    logits = (q[torch.arange(n), at].double()[:, None] * keys.to(cache).double()) * scale
    best = logits.amax(1)
    assert torch.equal(logits.argmax(1), winner)
    assert ((best[:, None] - logits).scatter(1, winner[:, None], 1e9).amin(1) > 200).all()
    out, lse = decode(moe, q, k.flatten(0, 1), v.flatten(0, 1), length, scale)
    want = v[torch.arange(n), winner].double()
    assert ((out.double() - want).abs() <= (want.abs() * 3 * 2.0**-24 if act is F32 else 0)).all()
    assert ((lse.double() - best).abs() <= best.abs() * 2.0**-21).all(), (lse, best)


@pytest.mark.parametrize("act,cache", [(F32, F16), (F32, BF16), (F32, E4M3), (F16, F16), (F16, E4M3), (BF16, BF16),
                                       (BF16, E4M3)])
@pytest.mark.parametrize("length", [2, 17, 300, 5000])
def test_the_winner_takes_all(moe, act, cache, length):
    """Logits of +-2^9 and below, the winner first, last or anywhere."""
    n = 12
    g = torch.Generator(device="cuda").manual_seed(length)
    winner = torch.randint(0, length, (n,), generator=g, device="cuda")
    winner[0], winner[1] = 0, length - 1
    keys = -torch.exp2(torch.randint(0, 4, (n, length), generator=g, device="cuda").float())
    keys[torch.arange(n), winner] = 4.0
    check(moe, act, cache, length, winner, torch.full((n,), 256.0, device="cuda"), keys, 0.5)


@pytest.mark.parametrize("act,cache,k_size", [(F32, BF16, 2.0**63), (BF16, BF16, 2.0**63), (F32, F16, 2.0**10),
                                              (F32, E4M3, 2.0**6), (BF16, E4M3, 2.0**6)])
@pytest.mark.parametrize("length", [2, 300, 5000])
def test_logits_near_the_end_of_fp32(moe, act, cache, k_size, length):
    """All logits between -2.5e38 and -1.7e38 (in units of log 2 down to -3.1e38), or as far above 0."""
    n = 8
    winner = torch.arange(n, device="cuda") * (length - 1) // (n - 1)
    for sign, most, least in ((-1.0, 1.0, 1.25), (1.0, 1.25, 1.0)):
        keys = torch.full((n, length), least, device="cuda")
        keys[torch.arange(n), winner] = most
        check(moe, act, cache, length, winner, torch.full((n,), sign * 2.0**126 / k_size, device="cuda"), keys * k_size, 2.0)


@pytest.mark.parametrize("length", [2, 300])
def test_the_largest_queries(moe, length):
    """Queries of the type's largest value on keys so small that the logits are ordinary."""
    n = 4
    winner = torch.arange(n, device="cuda") * (length - 1) // (n - 1)
    for act, top in ((F32, 3.4028234e38), (BF16, 3.3895314e38)):
        keys = torch.full((n, length), -2.0**-119, device="cuda")
        keys[torch.arange(n), winner] = 2.0**-119
        check(moe, act, BF16, length, winner, torch.full((n,), top, device="cuda"), keys, 0.5)
