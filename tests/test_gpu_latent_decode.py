"""LatentAttention.decode against the definition in 64 bits.

Errors: a logit is a sum of latent + rope exact products in fp32, off by less than
2^-20 S with S = scale * k_scale * sum |q c| (a unit of 2^-23 for each of some 36
tensor-core steps, typically far less); its weight by that, relatively.  Weights
enter the second product rounded to the type: half a step u each, 2^-8 (bf16),
2^-11 (f16; below 2^-21 of the largest, half of 2^-31 absolutely), their sum is
taken before the rounding.  With P = sum p |c|: |error| <= u |out| + (u + 2^-19 S +
2^-18) P (fp32 sums, exponentials and joins in 2^-18), plus the smallest
subnormal's half; lse is off by less than 2^-19 (S + |lse| + 1).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

HALF = {torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8}
E4 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def moe():
    import serving_router_sigmoid_gb300 as m
    return m


def normal(g, shape, dt, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dt)


def setup(lens, heads, latent, rope, dt, cache_dt, page, seed=0, std=1.0, spare=3, extra=0):
    """A cache whose rows nobody may read are NaN, the requests' pages in any order."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, dim = len(lens), latent + rope
    held = [-(-max(x, 0) // page) for x in lens]
    pages = sum(held) + spare
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((n, max(held + [0]) + 2), -1, dtype=torch.int32, device="cuda")
    cache = torch.full((pages, page, 1, dim + extra), math.nan, device="cuda").to(cache_dt)
    at = 0
    for b, x in enumerate(lens):
        table[b, :held[b]] = ids[at:at + held[b]]
        rows = normal(g, (max(x, 0), dim), cache_dt, std).view(torch.uint8)
        for p in range(held[b]):
            part = rows[p * page:(p + 1) * page]
            cache[int(ids[at + p])].view(torch.uint8)[:part.shape[0], 0, :part.shape[1]] = part
        at += held[b]
    q = normal(g, (n, heads, dim), dt)
    return q, cache[..., :dim], table, torch.tensor(lens, dtype=torch.int32, device="cuda")


def rows_of(cache, table, b, n):
    page, pages = cache.shape[1], cache.shape[0]
    j = torch.arange(n, device="cuda")
    ids = table[b].long()[j // page]
    ok = (ids >= 0) & (ids < pages)
    flat = cache.view(torch.uint8)[ids[ok], (j % page)[ok], 0].view(cache.dtype)
    return flat.double()


def check(out, lse, q, cache, table, lens, latent, scale, k_scale=1.0):
    u = HALF[q.dtype]
    cols = table.shape[1] * cache.shape[1]
    for b, n in enumerate(lens.tolist()):
        n = min(n, cols)
        c = rows_of(cache, table, b, n) if n > 0 else torch.zeros((0, cache.shape[-1]), device="cuda").double()
        if c.shape[0] == 0:
            assert bool((out[b] == 0).all()) and bool((lse[b] == -math.inf).all())
            continue
        c = c * k_scale
        qd = q[b].double()
        s = qd @ c.T * scale
        top = (qd.abs() @ c.abs().T * abs(scale)).amax(-1, keepdim=True)
        p = torch.softmax(s, -1)
        ref, total = p @ c[:, :latent], p @ c[:, :latent].abs()
        off = (out[b].double() - ref).abs()
        room = u * ref.abs() + (u + 2.0**-19 * top + 2.0**-18) * total * (1 + u) + 2.0**-25
        assert bool((off <= room).all()), (b, n, float((off / room).max()))
        want = torch.logsumexp(s, -1)
        assert bool(((lse[b].double() - want).abs() <= 2.0**-19 * (top[:, 0] + want.abs() + 1)).all()), (b, n)


CASES = [
    # lens, heads, latent, rope, page
    ([1], 64, 512, 64, 16), ([777], 64, 512, 64, 16), ([64], 64, 512, 64, 64), ([65, 1, 63, 0, 128], 64, 512, 64, 16),
    ([5, 300, 129], 1, 512, 64, 1), ([1000, 3], 16, 512, 64, 48), ([40, 500], 20, 256, 64, 7), ([2000], 128, 512, 64, 64),
    ([130, 0, 900], 96, 512, 32, 128), ([257, 66], 4, 128, 16, 32), ([100] * 40, 8, 64, 0, 16), ([333, 1, 2], 65, 384, 48, 24),
    ([5000, 17, 300, 1], 33, 512, 64, 64), ([70, 200], 200, 320, 64, 16), ([9000, 9001], 48, 448, 0, 256), ([0, 0], 64, 512, 64, 16),
]


@pytest.mark.parametrize("lens,heads,latent,rope,page", CASES)
@pytest.mark.parametrize("dt,cache_dt", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16),
                                         (torch.bfloat16, E4), (torch.float16, E4)])
def test_against_64_bits(moe, lens, heads, latent, rope, page, dt, cache_dt):
    q, cache, table, n = setup(lens, heads, latent, rope, dt, cache_dt, page, seed=len(lens) + heads)
    attn = moe.LatentAttention(len(lens), heads, latent, rope)
    k = 0.75 if cache_dt is E4 else 1.0
    scale = 1 / math.sqrt(128 + rope)
    out, lse = attn.decode(q, cache, table, n, scale, k_scale=k)
    check(out, lse, q, cache, table, n, latent, scale, k)
    assert moe.dense_status() == 0


def test_many_ragged_requests(moe):
    g = torch.Generator().manual_seed(1)
    lens = [int(x) for x in torch.randint(0, 700, (150,), generator=g)]
    q, cache, table, n = setup(lens, 24, 512, 64, torch.bfloat16, torch.bfloat16, 32, seed=2)
    out, lse = moe.LatentAttention(200, 24).decode(q, cache, table, n, 0.08)
    check(out, lse, q, cache, table, n, 512, 0.08)


def test_pages_that_are_none_are_not_seen(moe):
    q, cache, table, n = setup([200, 90, 64, 640], 64, 512, 64, torch.bfloat16, torch.bfloat16, 16, seed=3)
    table[0, 3], table[0, 12], table[1, :], table[2, 0], table[3, 4:8] = -1, cache.shape[0], -7, 2**31 - 1, -1
    table[3, 0:4] = -1  # the first tile of 64 holds nothing
    out, lse = moe.LatentAttention(4, 64).decode(q, cache, table, n, 0.07)
    check(out, lse, q, cache, table, n, 512, 0.07)


def test_lengths_beyond_the_table_and_negative(moe):
    q, cache, table, n = setup([100, 50, 16], 64, 512, 64, torch.float16, torch.float16, 16, seed=4)
    n = torch.tensor([10**6, -3, 16], dtype=torch.int32, device="cuda")
    table = table[:, :6].contiguous()
    out, lse = moe.LatentAttention(3, 64).decode(q, cache, table, n, 0.07)
    check(out, lse, q, cache, table, n, 512, 0.07)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_far_apart_logits(moe, dt):
    """A late token far above all before it (the sums are rescaled), and far below."""
    q, cache, table, n = setup([700, 700], 64, 512, 64, dt, dt, 64, seed=5, std=0.05)
    for b, sign in ((0, 1.0), (1, -1.0)):
        for j in (100, 333, 640):
            cache[int(table[b, j // 64]), j % 64, 0] = (q[b, j % 64].float() * sign * (1 + j / 700)).to(dt)
    out, lse = moe.LatentAttention(2, 64).decode(q, cache, table, n, 0.25)
    check(out, lse, q, cache, table, n, 512, 0.25)
    for scale in (0.0, -0.25):
        out, lse = moe.LatentAttention(2, 64).decode(q, cache, table, n, scale)
        check(out, lse, q, cache, table, n, 512, scale)


def test_small_weights_count(moe):
    """One token with e^12 times the weight of each of 60000 others (f16 weights)."""
    n = 60000
    q, cache, table, lens = setup([n], 16, 512, 64, torch.float16, torch.float16, 64, seed=6)
    q[:] = 0
    q[:, :, 0] = 1.0
    flat = cache.view(-1, 576)
    flat[:, 0] = 0
    cache[int(table[0, 10]), 5, 0, 0] = 12.0
    out, lse = moe.LatentAttention(1, 16).decode(q, cache, table, lens, 1.0)
    check(out, lse, q, cache, table, lens, 512, 1.0)


def test_strides_and_guards(moe):
    q, cache, table, n = setup([130, 70, 9], 40, 512, 64, torch.bfloat16, torch.bfloat16, 16, seed=7, extra=24)
    wide = torch.full((3, 40, 640), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:, :, 32:608] = q
    room = torch.full((5, 42, 520), 3.0, dtype=torch.bfloat16, device="cuda")
    lroom = torch.full((4, 40), 5.0, device="cuda")
    far = torch.full((3, table.shape[1] + 9), -1, dtype=torch.int32, device="cuda")
    far[:, :table.shape[1]] = table
    attn = moe.LatentAttention(8, 40)
    o, l = attn.decode(wide[:, :, 32:608], cache[:, :, 0], far[:, :table.shape[1]], n, 0.1, out=room[1:4, 1:41, 3:515],
                       lse=lroom[:3])
    check(o, l, q, cache, table, n, 512, 0.1)
    room[1:4, 1:41, 3:515] = 3.0
    assert bool((room == 3).all()) and bool((lroom[3] == 5).all())
    # heads before tokens, as a transposed view
    qt = q.transpose(0, 1).contiguous().transpose(0, 1)
    o2, _ = attn.decode(qt, cache, table, n, 0.1)
    check(o2, l, q, cache, table, n, 512, 0.1)


def test_repeats_graph_and_streams(moe):
    q, cache, table, n = setup([3000, 100, 900, 0, 64], 64, 512, 64, torch.bfloat16, torch.bfloat16, 64, seed=8)
    attn = moe.LatentAttention(5, 64)
    want = attn.decode(q, cache, table, n, 0.07)
    for _ in range(30):
        got = attn.decode(q, cache, table, n, 0.07)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = attn.decode(q, cache, table, n, 0.07, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = attn.decode(q, cache, table, n, 0.07)
    for lens in ([1, 64, 65, 2, 900], [3000, 0, 0, 0, 0], [2999, 100, 1, 0, 64]):  # the lengths are read at replay
        m = torch.tensor(lens, dtype=torch.int32, device="cuda")
        m = torch.minimum(m, torch.tensor([3000, 100, 900, 0, 64], device="cuda").int())
        n.copy_(m)
        graph.replay()
        check(out, lse, q, cache, table, n, 512, 0.07)
    del graph


def test_two_handles_on_two_streams(moe):
    q, cache, table, n = setup([2500, 2000, 300], 64, 512, 64, torch.bfloat16, E4, 64, seed=9)
    a, b = moe.LatentAttention(3, 64), moe.LatentAttention(3, 64)
    want = a.decode(q, cache, table, n, 0.07)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (sa, sb):
        s.wait_stream(torch.cuda.current_stream())
    got = [h.decode(q, cache, table, n, 0.07, stream=s) for _ in range(5) for h, s in ((a, sa), (b, sb))]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) and torch.equal(l, want[1]) for o, l in got)


def test_offsets_beyond_32_bits(moe):
    """Pages at byte offsets beyond 2^32."""
    page, pages, dim = 64, 62000, 576  # 4.6 GB of bf16
    cache = torch.zeros((pages, page, 1, dim), dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[61999, 3, 58300, 61000]], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for p in table[0].tolist():
        cache[p] = normal(g, (page, 1, dim), torch.bfloat16)
    q, n = normal(g, (1, 64, dim), torch.bfloat16), torch.tensor([250], dtype=torch.int32, device="cuda")
    out, lse = moe.LatentAttention(1, 64).decode(q, cache, table, n, 0.07)
    check(out, lse, q, cache, table, n, 512, 0.07)


@pytest.mark.parametrize("n,heads", [(1, 64), (3, 64), (5, 40), (6, 128), (11, 64), (13, 100), (30, 64)])
def test_joins_of_many_pieces(moe, n, heads):
    """Few and more requests, each over several blocks."""
    lens = [1400 + 97 * i % 900 for i in range(n)]
    q, cache, table, ln = setup(lens, heads, 512, 64, torch.bfloat16, torch.bfloat16, 64, seed=n)
    attn = moe.LatentAttention(n, heads)
    out, lse = attn.decode(q, cache, table, ln, 0.07)
    check(out, lse, q, cache, table, ln, 512, 0.07)
    again = attn.decode(q, cache, table, ln, 0.07)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
