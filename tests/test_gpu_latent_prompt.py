"""latent_prompt against the definition in 64 bits.

The bound is that of one attention row: a logit is off by less than 2^-20 S, S =
|scale| sum |q k|; weights enter the second product rounded to the type, half a
step u each, 2^-8 (bf16) or 2^-11 (f16; below 2^-21 of the largest, half of 2^-31
absolutely), their sum is taken before the rounding.  With P = sum p |v|: |error| <=
u |out| + (u + 2^-19 S + 2^-18) P plus half the smallest subnormal; lse is off by
less than 2^-19 (S + |lse| + 1).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

HALF = {torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8}


@pytest.fixture(scope="module")
def moe():
    import serving_router_sigmoid_gb300 as m
    return m


def starts(lens):
    return torch.tensor([0] + list(lens), device="cuda").cumsum(0).int()


def setup(nq, nk, heads, nope, rope, v, dt, seed=0, spare=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *s: (torch.randn(s, generator=g, device="cuda") * std).to(dt)  # noqa: E731
    tq, tk = sum(nq) + spare, sum(nk) + spare
    kv, row = new(tk, heads, nope + v), new(tk, 512 + rope)
    q = new(tq, heads, nope + rope)
    if spare:  # rows of no request
        q[sum(nq):], kv[sum(nk):], row[sum(nk):] = math.nan, math.nan, math.nan
    return q, kv[..., :nope], row[:, 512:] if rope else None, kv[..., nope:], starts(nq), starts(nk)


def check(out, lse, q, k, kr, v, q_start, kv_start, scale, causal):
    u = HALF[q.dtype]
    qs, ks = q_start.tolist(), kv_start.tolist()
    for b in range(len(qs) - 1):
        nq, nk = qs[b + 1] - qs[b], ks[b + 1] - ks[b]
        if nq <= 0:
            continue
        at, kt = slice(qs[b], qs[b + 1]), slice(ks[b], ks[b + 1])
        seen = torch.ones((nq, max(nk, 0)), dtype=torch.bool, device="cuda")
        if causal:
            seen = seen.tril(nk - nq)
        for h in range(q.shape[1]):
            key = k[kt, h].double()
            if kr is not None:
                key = torch.cat([key, kr[kt].double()], 1)
            qd, val = q[at, h].double(), v[kt, h].double()
            s = (qd @ key.T * scale).masked_fill(~seen, -math.inf)
            top = (qd.abs() @ key.abs().T * abs(scale)).masked_fill(~seen, 0).sum(-1 if nk == 0 else 1, keepdim=True) * 0
            if nk:
                top = (qd.abs() @ key.abs().T * abs(scale)).masked_fill(~seen, 0).amax(-1, keepdim=True)
            live = seen.any(-1)
            p = torch.softmax(s, -1).nan_to_num(0)
            ref, total = p @ val, p @ val.abs()
            o, ls = out[at, h].double(), lse[at, h].double()
            assert bool((o[~live] == 0).all()) and bool((ls[~live] == -math.inf).all())
            off = (o - ref).abs()
            room = u * ref.abs() + (u + 2.0**-19 * top + 2.0**-18) * total * (1 + u) + 2.0**-25
            assert bool((off <= room).all()), (b, h, float((off / room).max()))
            want = torch.logsumexp(s[live], -1)
            assert bool(((ls[live] - want).abs() <= 2.0**-19 * (top[live, 0] + want.abs() + 1)).all()), (b, h)


DIMS = [(128, 64, 128), (192, 64, 256), (64, 32, 64), (96, 64, 80), (64, 64, 192), (16, 0, 16), (240, 16, 240), (112, 48, 144)]
RAGGED = [
    ([1], [1]), ([128], [128]), ([129], [129]), ([1, 2, 3], [1, 200, 64]), ([300, 5, 0, 77], [300, 133, 9, 500]),
    ([257], [1000]), ([64, 1], [64, 640]), ([20, 130], [5, 64]), ([3, 4], [0, 4]), ([127, 255, 1], [256, 255, 127]),
]


@pytest.mark.parametrize("nope,rope,v", DIMS)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_head_sizes(moe, nope, rope, v, dt):
    a = setup([70, 200], [70, 333], 3, nope, rope, v, dt, seed=nope + v, spare=5)
    for causal in (True, False):
        out, lse = moe.latent_prompt(*a, 1 / math.sqrt(nope + rope), causal=causal)
        check(out, lse, *a, 1 / math.sqrt(nope + rope), causal)
    assert moe.dense_status() == 0


@pytest.mark.parametrize("nq,nk", RAGGED)
@pytest.mark.parametrize("causal", [True, False])
def test_ragged_lengths(moe, nq, nk, causal):
    a = setup(nq, nk, 2, 128, 64, 128, torch.bfloat16, seed=sum(nq), spare=3)
    out, lse = moe.latent_prompt(*a, 0.07, causal=causal)
    check(out, lse, *a, 0.07, causal)
    assert moe.dense_status() == 0


def test_longer_prompt_and_many_heads(moe):
    a = setup([1500], [2600], 5, 128, 64, 128, torch.bfloat16, seed=1)
    out, lse = moe.latent_prompt(*a, 0.07)
    check(out, lse, *a, 0.07, True)
    a = setup([150], [150], 130, 64, 64, 64, torch.float16, seed=2)
    out, lse = moe.latent_prompt(*a, 0.09)
    check(out, lse, *a, 0.09, True)


def test_many_requests(moe):
    g = torch.Generator().manual_seed(3)
    nk = [int(x) for x in torch.randint(0, 90, (300,), generator=g)]
    nq = [int(torch.randint(0, x + 1, (1,), generator=g)) for x in nk]
    a = setup(nq, nk, 2, 64, 32, 64, torch.bfloat16, seed=4)
    out, lse = moe.latent_prompt(*a, 0.1)
    check(out, lse, *a, 0.1, True)


@pytest.mark.parametrize("nope,rope,v", [(128, 64, 128), (192, 64, 256), (64, 64, 192)])
def test_many_work_items_a_block(moe, nope, rope, v):
    """More (request, queries, head) items than SMs, of one and of several tiles."""
    a = setup([600, 90, 300, 1, 0, 257], [900, 90, 700, 400, 5, 257], 48, nope, rope, v, torch.bfloat16, seed=nope)
    for causal in (True, False):
        out, lse = moe.latent_prompt(*a, 0.07, causal=causal)
        check(out, lse, *a, 0.07, causal)
        assert moe.dense_status() == 0


def test_rows_of_no_request_stay(moe):
    q, k, kr, v, qs, ks = setup([40, 30], [60, 45], 4, 128, 64, 128, torch.bfloat16, seed=5, spare=20)
    out = torch.full((90, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((90, 4), 7.0, device="cuda")
    qs2, ks2 = qs + 10, ks + 15  # rows before the first request too
    moe.latent_prompt(q, k, kr, v, qs2, ks2, 0.07, out=out, lse=lse)
    assert bool((out[:10] == 7).all()) and bool((out[80:] == 7).all())
    assert bool((lse[:10] == 7).all()) and bool((lse[80:] == 7).all())
    got = (out.clone(), lse.clone())
    q, k, kr, v, _, _ = setup([40, 30], [60, 45], 4, 128, 64, 128, torch.bfloat16, seed=5, spare=20)
    q[70:], k[105:], v[105:], kr[105:] = 1.0, 1.0, 1.0, 1.0
    out.fill_(7.0)
    moe.latent_prompt(q, k, kr, v, qs2, ks2, 0.07, out=out, lse=lse)
    assert bool(out[10:80].isfinite().all()) and got[0].shape == out.shape
    check(out, lse, q, k, kr, v, qs2, ks2, 0.07, True)


def test_neighbours_do_not_leak(moe):
    """Infinities and NaN in another request's rows change nothing."""
    a = setup([50, 60, 70], [100, 60, 130], 3, 128, 64, 128, torch.bfloat16, seed=6)
    want, wl = moe.latent_prompt(*a, 0.07)
    q, k, kr, v, qs, ks = a
    for t, s in ((q, qs), (k, ks), (kr, ks), (v, ks)):
        t[:int(s[1])] = math.nan
        t[int(s[2]):] = math.inf
    got, gl = moe.latent_prompt(*a, 0.07)
    at = slice(50, 110)
    assert torch.equal(got[at], want[at]) and torch.equal(gl[at], wl[at])


def test_bounds_beyond_the_rows_are_cut(moe):
    q, k, kr, v, qs, ks = setup([30, 40], [50, 60], 2, 128, 64, 128, torch.bfloat16, seed=7)
    want, _ = moe.latent_prompt(q, k, kr, v, qs, ks, 0.07)
    qs2, ks2 = qs.clone(), ks.clone()
    qs2[-1], ks2[-1] = 70, 10**6
    got, _ = moe.latent_prompt(q, k, kr, v, qs2, ks2, 0.07, causal=False)
    ref, _ = moe.latent_prompt(q, k, kr, v, qs, ks, 0.07, causal=False)
    assert torch.equal(got, ref)
    qs2 = torch.tensor([-5, 30, 10**9], dtype=torch.int32, device="cuda")
    got, _ = moe.latent_prompt(q, k, kr, v, qs2, ks, 0.07, causal=False)
    assert torch.equal(got, ref)
    falling = torch.tensor([0, 60, 20], dtype=torch.int32, device="cuda")  # no rows of the second request
    out = torch.full_like(got, 5.0)
    moe.latent_prompt(q, k, kr, v, falling, ks, 0.07, out=out)
    assert bool((out[60:] == 5).all())
    assert want.shape == got.shape


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_far_apart_logits(moe, dt):
    q, k, kr, v, qs, ks = setup([400], [400], 2, 128, 64, 128, dt, seed=8, std=0.2)
    for j in (130, 260, 390):  # late keys far above all before them
        k[j] = q[395, :, :128] * (10 + j / 40)
    out, lse = moe.latent_prompt(q, k, kr, v, qs, ks, 1.0)
    check(out, lse, q, k, kr, v, qs, ks, 1.0, True)
    for scale in (0.0, -1.0):
        out, lse = moe.latent_prompt(q, k, kr, v, qs, ks, scale)
        check(out, lse, q, k, kr, v, qs, ks, scale, True)


def test_strides(moe):
    q, k, kr, v, qs, ks = a = setup([90], [140], 4, 128, 64, 128, torch.float16, seed=9)
    want, wl = moe.latent_prompt(*a, 0.07)
    by_head = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    wide = torch.full((90, 6, 200), 3.0, dtype=torch.float16, device="cuda")
    got, gl = moe.latent_prompt(by_head(q), by_head(k), kr.contiguous(), by_head(v), qs, ks, 0.07, out=wide[:, 1:5, 7:135])
    assert torch.equal(got, want) and torch.equal(gl, wl)
    wide[:, 1:5, 7:135] = 3.0
    assert bool((wide == 3).all())
    # one key row for all heads
    one = k[:, :1].expand(-1, 4, -1)
    got, _ = moe.latent_prompt(q, one, kr, v, qs, ks, 0.07)
    ref, _ = moe.latent_prompt(q, one.contiguous(), kr, v, qs, ks, 0.07)
    assert torch.equal(got, ref)


def test_repeats_graph_and_streams(moe):
    a = setup([200, 100, 300], [200, 400, 300], 4, 128, 64, 128, torch.bfloat16, seed=10)
    q, k, kr, v, qs, ks = a
    want, wl = moe.latent_prompt(*a, 0.07)
    for _ in range(20):
        got, gl = moe.latent_prompt(*a, 0.07)
        assert torch.equal(got, want) and torch.equal(gl, wl)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (sa, sb):
        s.wait_stream(torch.cuda.current_stream())
    got = [moe.latent_prompt(*a, 0.07, stream=s) for _ in range(4) for s in (sa, sb)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o, _ in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = moe.latent_prompt(*a, 0.07)
    for nq, nk in (([600, 0, 0], [900, 0, 0]), ([10, 20, 30], [10, 700, 30])):  # the bounds are read at replay
        qs.copy_(starts(nq))
        ks.copy_(starts(nk))
        graph.replay()
        check(out, lse, *a, 0.07, True)


def some(a, out, lse, step=31):
    """Inputs and outputs of a few heads, for the check."""
    q, k, kr, v, qs, ks = a
    h = slice(None, None, step)
    return out[:, h], lse[:, h], q[:, h], k[:, h], kr, v[:, h], qs, ks


# with so many heads a block holds 256 queries as two streams, where heads are narrow
@pytest.mark.parametrize("nope,rope,v", [(128, 64, 128), (64, 32, 64), (96, 64, 80), (16, 0, 16), (112, 48, 112), (128, 16, 128)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_head_sizes_of_many_heads(moe, nope, rope, v, dt):
    a = setup([70, 200], [70, 333], 160, nope, rope, v, dt, seed=nope + v, spare=5)
    for causal in (True, False):
        out, lse = moe.latent_prompt(*a, 1 / math.sqrt(nope + rope), causal=causal)
        check(*some(a, out, lse), 1 / math.sqrt(nope + rope), causal)
    assert moe.dense_status() == 0


@pytest.mark.parametrize("nq,nk", RAGGED)
@pytest.mark.parametrize("causal", [True, False])
def test_ragged_lengths_of_many_heads(moe, nq, nk, causal):
    a = setup(nq, nk, 160, 128, 64, 128, torch.bfloat16, seed=sum(nq), spare=3)
    out, lse = moe.latent_prompt(*a, 0.07, causal=causal)
    check(*some(a, out, lse), 0.07, causal)
    assert moe.dense_status() == 0


@pytest.mark.parametrize("nope,rope,v", [(208, 48, 64), (240, 16, 16), (192, 64, 128)])
def test_wide_keys_and_narrow_values(moe, nope, rope, v):
    a = setup([70, 200], [70, 333], 3, nope, rope, v, torch.bfloat16, seed=nope + v, spare=5)
    for causal in (True, False):
        out, lse = moe.latent_prompt(*a, 1 / math.sqrt(nope + rope), causal=causal)
        check(out, lse, *a, 1 / math.sqrt(nope + rope), causal)


def test_neighbours_of_many_heads(moe):
    """Infinities and NaN in other rows change nothing, rows of no request stay."""
    a = setup([50, 300, 70], [100, 300, 130], 160, 128, 64, 128, torch.bfloat16, seed=6)
    q, k, kr, v, qs, ks = a
    want, wl = moe.latent_prompt(*a, 0.07)
    for t, s in ((q, qs), (k, ks), (kr, ks), (v, ks)):
        t[:int(s[1])] = math.nan
        t[int(s[2]):] = math.inf
    out, lse = torch.full_like(want, 7.0), torch.full_like(wl, 7.0)
    moe.latent_prompt(q, k, kr, v, qs[1:3].contiguous(), ks[1:3].contiguous(), 0.07, out=out, lse=lse)
    at = slice(50, 350)
    assert torch.equal(out[at], want[at]) and torch.equal(lse[at], wl[at])
    for t in (out, lse):
        assert bool((t[:50] == 7).all()) and bool((t[350:] == 7).all())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_far_apart_logits_of_many_heads(moe, dt):
    a = setup([300], [900], 160, 64, 32, 64, dt, seed=12, std=3.0)
    out, lse = moe.latent_prompt(*a, 0.3)
    check(*some(a, out, lse), 0.3, True)


def test_offsets_beyond_32_bits(moe):
    """Tokens 2^23 elements apart: rows beyond 2^31 elements of every tensor."""
    heads, step = 2, 1 << 23
    a = setup([150, 130], [170, 150], heads, 128, 64, 128, torch.bfloat16, seed=13)
    q, k, kr, v, qs, ks = a
    want, wl = moe.latent_prompt(*a, 0.07)
    big, room = (torch.empty(330 * step, dtype=torch.bfloat16, device="cuda") for _ in range(2))  # 5.5 GB each

    def far(t, at):
        shape = t.shape
        inner = (shape[2], 1) if t.dim() == 3 else (1,)
        f = torch.as_strided(big, shape, (step,) + inner, at)
        f.copy_(t)
        return f
    out = torch.as_strided(room, want.shape, (step, 128, 1), 64)
    got, gl = moe.latent_prompt(far(q, 0), far(k, 4096), far(kr, 8192), far(v, 12288), qs, ks, 0.07, out=out)
    assert torch.equal(got, want) and torch.equal(gl, wl)
    check(got, gl, *a, 0.07, True)


# two streams: more tiles of keys in the ring than one, or just one (the last)
@pytest.mark.parametrize("nope,rope,v", [(128, 0, 128), (64, 64, 128), (64, 32, 64), (64, 0, 64), (128, 64, 64), (128, 64, 128)])
@pytest.mark.parametrize("nq,nk", [
    ([256] * 11, [384, 256] * 5 + [384]),                       # (2, 3) and (1, 2) tiles, five items a block
    ([256] + [0] * 500 + [256, 256] + [0] * 900 + [256] * 2, [256] + [9] * 500 + [384, 384] + [0] * 900 + [384] * 2),
    ([256, 128, 200, 256, 300, 256, 40], [512, 128, 333, 384, 300, 640, 384]),
])
def test_streams_that_run_apart(moe, nope, rope, v, nq, nk):
    """Several items a block, logits that grow towards the diagonal (O is scaled in both halves of each tile),
    searches past many empty requests."""
    q, k, kr, val, qs, ks = setup(nq, nk, 64, nope, rope, v, torch.bfloat16, seed=nope + v + len(nq), spare=2)
    scale = 0.07
    q[..., 0] = 4.0
    k[:-2, :, 0] = torch.cat([torch.arange(n, device="cuda") for n in nk])[:, None] * (0.125 / (4 * scale))
    a = (q, k, kr, val, qs, ks)
    out, lse = moe.latent_prompt(*a, scale)
    assert moe.dense_status() == 0
    check(*some(a, out, lse, 21), scale, True)
    for _ in range(20):
        again, al = moe.latent_prompt(*a, scale)
        assert torch.equal(again[:sum(nq)], out[:sum(nq)]) and torch.equal(al[:sum(nq)], lse[:sum(nq)])
    assert moe.dense_status() == 0


@pytest.mark.parametrize("nope,rope,v", [(64, 32, 64), (128, 0, 128), (64, 0, 16), (128, 64, 64), (192, 64, 256)])
@pytest.mark.parametrize("gap", [0, 70])
def test_many_items_of_one_tile(moe, nope, rope, v, gap):
    """One stream, dozens of items a block, each of one tile with rows behind its last key; `gap` requests
    without queries between those that have some."""
    g = torch.Generator().manual_seed(gap)
    nk = [int(x) for x in torch.randint(1, 128, (100,), generator=g)]
    nq = [min(1 + i % 3, n) for i, n in enumerate(nk)]
    nq = [x for n in nq for x in [n] + [0] * gap]
    nk = [x for n in nk for x in [n] + [0] * gap]
    a = setup(nq, nk, 64, nope, rope, v, torch.bfloat16, seed=nope + gap, spare=1)
    for causal in (True, False):
        out, lse = moe.latent_prompt(*a, 0.1, causal=causal)
        assert moe.dense_status() == 0
        check(*some(a, out, lse), 0.1, causal)
        for _ in range(20):
            again, _ = moe.latent_prompt(*a, 0.1, causal=causal)
            assert torch.equal(again[:sum(nq)], out[:sum(nq)])
    assert moe.dense_status() == 0


# with a long request among them the short ones, too, are items of two streams
@pytest.mark.parametrize("nq,nk", RAGGED)
@pytest.mark.parametrize("nope,rope,v", [(128, 64, 128), (64, 0, 64)])
def test_short_requests_beside_a_long_one(moe, nope, rope, v, nq, nk):
    nq, nk = nq[:1] + [700] + nq[1:], nk[:1] + [830] + nk[1:]
    a = setup(nq, nk, 160, nope, rope, v, torch.bfloat16, seed=sum(nq), spare=3)
    for causal in (True, False):
        out, lse = moe.latent_prompt(*a, 0.07, causal=causal)
        check(*some(a, out, lse), 0.07, causal)
    assert moe.dense_status() == 0


@pytest.mark.parametrize("nope,rope,v", [(128, 64, 128), (128, 0, 128), (64, 32, 64)])
def test_two_streams_past_many_empty_requests(moe, nope, rope, v):
    nq = ([1280] * 8 + [0] * 70) * 4  # 131 on average
    nk = ([1280, 1400] * 4 + [0, 9] * 35) * 4
    a = setup(nq, nk, 2, nope, rope, v, torch.bfloat16, seed=nope, spare=1)
    out, lse = moe.latent_prompt(*a, 0.07)
    check(out, lse, *a, 0.07, True)
    for _ in range(10):
        again, _ = moe.latent_prompt(*a, 0.07)
        assert torch.equal(again[:sum(nq)], out[:sum(nq)])
    assert moe.dense_status() == 0


@pytest.mark.parametrize("nope,rope,v", [(240, 16, 240), (208, 48, 256), (208, 16, 144), (240, 0, 256)])
def test_rings_shorter_than_a_tile(moe, nope, rope, v):
    """Keys of five chunks beside wide values: a tile of both is more than the ring holds."""
    a = setup([150, 600, 40, 300], [900, 700, 40, 1300], 40, nope, rope, v, torch.bfloat16, seed=nope + v, spare=2)
    for causal in (True, False):
        out, lse = moe.latent_prompt(*a, 0.06, causal=causal)
        check(*some(a, out, lse, 13), 0.06, causal)
        for _ in range(20):
            again, _ = moe.latent_prompt(*a, 0.06, causal=causal)
            assert torch.equal(again[:-2], out[:-2])
    assert moe.dense_status() == 0


@pytest.mark.parametrize("nope,rope,v", [(64, 0, 64), (128, 64, 128), (48, 16, 80)])
def test_items_of_one_stream_between_those_of_two(moe, nope, rope, v):
    """Requests of up to 128 queries, whose second stream has no tile, behind long keys; and requests whose first
    128 queries see none."""
    nq = [100, 512, 128, 256, 400, 1, 600, 128, 300, 256] * 3
    nk = [900, 512, 700, 128, 272, 1500, 600, 128, 172, 130] * 3
    a = setup(nq, nk, 48, nope, rope, v, torch.bfloat16, seed=nope, spare=2)
    for causal in (True, False):
        out, lse = moe.latent_prompt(*a, 0.08, causal=causal)
        check(*some(a, out, lse, 17), 0.08, causal)
        for _ in range(20):
            again, _ = moe.latent_prompt(*a, 0.08, causal=causal)
            assert torch.equal(again[:-2], out[:-2])
    assert moe.dense_status() == 0
