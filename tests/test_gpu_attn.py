"""moe_attn_decode against the definition in 64 bits.

Bounds, fixed from the arithmetic before the first run.  A logit is a sum of
k_dim products in fp32 (the tensor cores may truncate: one ulp an addition):
es = scale * max_j sum |q k_j| * (k_dim + 8) * 2^-23.  A weight exp(s - m) is
then off by 2 es + 8 * 2^-24 relative, and rounded once for the product with v:
2^-8 where q and out are 16-bit types, 2^-20 where they are fp32 (which the
kernel holds in several terms).  The sum over the tokens adds an ulp every 8 of
them.  All of it times sum p |v|; then half an ulp of the output's type.
"""
import math
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

F32, F16, BF16, E4M3 = torch.float32, torch.float16, torch.bfloat16, torch.float8_e4m3fn
HALF_ULP = {F32: (2.0**-24, 0.0), F16: (2.0**-11, 2.0**-25), BF16: (2.0**-8, 0.0)}
LENGTHS = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 100, 257, 1000, 2049]


@pytest.fixture(scope="module")
def moe():
    import serving_router_sigmoid_gb300 as m
    torch.cuda.set_device(0)
    return m


def rows_of(cache, pages, at):
    """cache[pages, at] as fp64 (by bytes for 8-bit types)."""
    if cache.dtype is E4M3:
        return cache.view(torch.uint8)[pages, at].view(E4M3).float().double()
    return cache[pages, at].double()


def put(cache, pages, at, rows):
    if cache.dtype is E4M3:
        cache.view(torch.uint8)[pages, at] = rows.view(torch.uint8)
    else:
        cache[pages, at] = rows


class Batch:
    """Requests with their rows in a paged cache whose every other row is NaN."""

    def __init__(self, lens, heads, kv, dim, act, cache, page, v_dim=None, by_head=False, seed=0, spare_cols=2,
                 q_std=1.0, pages=None, low=0):
        g = torch.Generator(device="cuda").manual_seed(seed + 17)
        r = random.Random(seed)
        self.lens, self.heads, self.kv, self.dim, self.page = lens, heads, kv, dim, page
        self.v_dim = dim if v_dim is None else v_dim
        need = [-(-n // page) for n in lens]
        self.n_pages = pages or sum(need) + 3
        free = list(range(low, self.n_pages))
        r.shuffle(free)
        cols = max(need, default=0) + spare_cols
        # entries beyond a request's pages are junk that must not be read
        table = [[free.pop() for _ in range(m)] + [r.choice([-1, 2**31 - 1, -2**31, 12345678]) for _ in range(cols - m)]
                 for m in need]
        self.table = torch.tensor(table, dtype=torch.int32).view(len(lens), cols).cuda()

        def filled(d):
            shape = (self.n_pages, kv, page, d) if by_head else (self.n_pages, page, kv, d)
            if pages:
                c = torch.empty(shape, dtype=cache, device="cuda")  # too large to fill
            elif cache is E4M3:
                c = torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda").view(E4M3)
            else:
                c = torch.full(shape, float("nan"), dtype=cache, device="cuda")
            return c.transpose(1, 2) if by_head else c

        self.k, self.v = filled(dim), filled(self.v_dim)
        for b, n in enumerate(lens):
            at = torch.arange(n, device="cuda")
            pg = self.table[b, at // page].long()
            for c, d in ((self.k, dim), (self.v, self.v_dim)):
                put(c, pg, at % page, torch.randn((n, kv, d), generator=g, device="cuda").to(cache))
        self.q = (torch.randn((len(lens), heads, dim), generator=g, device="cuda") * q_std).to(act)
        self.seq = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def check(self, got, lse, scale=None, window=0, ks=1.0, vs=1.0):
        scale = 1 / math.sqrt(self.dim) if scale is None else scale
        rel, ab = HALF_ULP[got.dtype]
        up = 2.0**-20 if got.dtype is F32 else 2.0**-8
        assert got.shape == (len(self.lens), self.heads, self.v_dim) and lse.dtype is F32
        for b, n in enumerate(self.lens):
            o = got[b].double()
            first = max(0, n - window) if window else 0
            if n - first <= 0:
                assert (o == 0).all() and (lse[b] == -math.inf).all()
                continue
            at = torch.arange(first, n, device="cuda")
            pg = self.table[b, at // self.page].long()
            k, v = rows_of(self.k, pg, at % self.page) * ks, rows_of(self.v, pg, at % self.page) * vs
            q = self.q[b].double().unflatten(0, (self.kv, -1))
            s = torch.einsum("hgd,lhd->hgl", q, k) * scale
            es = abs(scale) * torch.einsum("hgd,lhd->hgl", q.abs(), k.abs()).amax(-1) * (self.dim + 8) * 2.0**-23
            es = es.flatten()
            p = torch.softmax(s, -1)
            want = torch.einsum("hgl,lhd->hgd", p, v).flatten(0, 1)
            big = torch.einsum("hgl,lhd->hgd", p, v.abs()).flatten(0, 1)
            bound = big * (2 * es[:, None] + 8 * 2.0**-24 + up + (n - first + 64) / 8 * 2.0**-23)
            bound = bound * (1 + rel) + want.abs() * rel + ab
            off = (o - want).abs()
            assert (off <= bound).all(), (b, n, float((off - bound).max()), float(off.max()))
            wl = torch.logsumexp(s, -1).flatten()
            bl = 2 * es + (8 + (n - first + 64) / 8) * 2.0**-23 + wl.abs() * 2.0**-22
            assert ((lse[b].double() - wl).abs() <= bl).all(), (b, n, float((lse[b].double() - wl).abs().max()))


def run(moe, batch, attn=None, **kw):
    attn = attn or moe.PagedAttention(max(1, len(batch.lens)), batch.heads, batch.kv, batch.dim, batch.v_dim)
    scales = {k: kw[a] for k, a in (("ks", "k_scale"), ("vs", "v_scale")) if a in kw}
    out, lse = attn.decode(batch.q, batch.k, batch.v, batch.table, batch.seq, **kw)
    batch.check(out, lse, kw.get("scale"), kw.get("window", 0), **scales)
    again, lse2 = attn.decode(batch.q, batch.k, batch.v, batch.table, batch.seq, **kw)
    assert torch.equal(out, again) and torch.equal(lse, lse2)  # whatever block finishes first
    return out, lse


@pytest.mark.parametrize("act", [F32, F16, BF16])
@pytest.mark.parametrize("cache", [F16, BF16, E4M3])
@pytest.mark.parametrize("dim,kv,group", [(64, 2, 1), (64, 1, 12), (128, 2, 8), (128, 1, 16), (256, 1, 4), (256, 1, 9)])
def test_types(moe, act, cache, dim, kv, group):
    kw = dict(k_scale=0.7, v_scale=1.3) if cache is E4M3 else {}
    run(moe, Batch(LENGTHS, kv * group, kv, dim, act, cache, 16, seed=dim + group), **kw)


@pytest.mark.parametrize("page", [1, 3, 7, 16, 24, 48, 64, 256])
@pytest.mark.parametrize("by_head", [False, True])
def test_pages_and_layouts(moe, page, by_head):
    run(moe, Batch(LENGTHS, 8, 2, 128, BF16, BF16, page, by_head=by_head, seed=page))
    run(moe, Batch(LENGTHS, 8, 2, 64, F16, E4M3, page, by_head=by_head, seed=page), window=37)


@pytest.mark.parametrize("dim,v_dim", [(8, 8), (16, 40), (40, 16), (72, 72), (80, 80), (96, 96), (112, 64), (136, 128),
                                       (192, 128), (200, 248), (64, 256)])
def test_head_sizes(moe, dim, v_dim):
    run(moe, Batch(LENGTHS, 6, 2, dim, BF16, BF16, 16, v_dim=v_dim, seed=dim))
    run(moe, Batch(LENGTHS, 6, 2, dim, F32, F16, 16, v_dim=v_dim, seed=dim))
    if dim % 16 == 0 and v_dim % 16 == 0:
        run(moe, Batch(LENGTHS, 6, 2, dim, BF16, E4M3, 16, v_dim=v_dim, seed=dim))


@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 8, 9, 15, 16, 17, 20, 24, 32, 40])
def test_groups(moe, group):
    run(moe, Batch([5, 300, 0, 64], 2 * group, 2, 64, BF16, BF16, 16, seed=group))
    run(moe, Batch([5, 300, 0, 64], 3 * group, 3, 128, F32, BF16, 16, seed=group))


@pytest.mark.parametrize("window", [1, 15, 16, 17, 100, 1000, 100000])
def test_windows(moe, window):
    run(moe, Batch(LENGTHS, 8, 2, 128, BF16, BF16, 16, seed=window), window=window)
    run(moe, Batch(LENGTHS, 8, 8, 64, F32, F16, 7, seed=window), window=window)


@pytest.mark.parametrize("lens", [[1], [40], [777], [5000], [70001], [131072, 1], [9, 30000, 0, 17, 12000, 1, 1, 64]])
def test_long_requests_are_split_and_joined(moe, lens):
    run(moe, Batch(lens, 32, 4, 128, BF16, BF16, 64, seed=lens[0]))
    run(moe, Batch(lens, 8, 8, 64, F16, E4M3, 16, seed=lens[0]), k_scale=0.5)


def test_many_short_requests(moe):
    r = random.Random(3)
    run(moe, Batch([r.randrange(0, 40) for _ in range(1500)], 8, 2, 64, BF16, BF16, 16, seed=8))


def test_sharp_flat_and_growing_logits(moe):
    for std, scale in ((30.0, None), (1.0, 0.0), (1.0, -3.0), (200.0, 1.0)):
        run(moe, Batch([1, 64, 1000, 5000], 8, 2, 64, F32, BF16, 16, q_std=std, seed=2), scale=scale)
    # every logit above the last one: the running maximum moves at each step
    b = Batch([4096], 8, 1, 64, F32, F16, 16, seed=4)
    ramp = torch.linspace(-40, 40, 4096, device="cuda").half()
    at = torch.arange(4096, device="cuda")
    b.k[b.table[0, at // 16].long(), at % 16] = ramp[:, None, None].expand(4096, 1, 64).contiguous() / 8
    b.q.fill_(1.0)
    run(moe, b, scale=1.0)
    b.k[b.table[0, at // 16].long(), at % 16] = -ramp[:, None, None].expand(4096, 1, 64).contiguous() / 8
    run(moe, b, scale=1.0)


def test_extreme_values(moe):
    """The types' largest values in q, and logits far beyond exp's range."""
    b = Batch([3, 100], 4, 1, 64, F32, BF16, 16, seed=1)
    b.q[0] *= 1e6
    run(moe, b)
    b = Batch([3, 100], 4, 1, 64, BF16, F16, 16, seed=1)
    b.q[1] *= 1e30
    run(moe, b, scale=1e-30)
    b = Batch([3, 100], 4, 1, 64, F32, E4M3, 16, seed=1)
    b.q[1] *= 1e-30
    run(moe, b, scale=1e30)


def test_pages_nobody_holds_are_not_seen(moe):
    """A table entry of -1 (or beyond the cache) inside a request: its tokens count as masked."""
    b = Batch([100, 64], 8, 2, 128, BF16, BF16, 16, seed=9)
    hole = Batch([100, 64], 8, 2, 128, BF16, BF16, 16, seed=9)
    b.table[0, 2], b.table[1, :] = -1, b.n_pages
    out, lse = moe.PagedAttention(2, 8, 2, 128).decode(b.q, b.k, b.v, b.table, b.seq)
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()
    # the same request without that page's tokens
    hole.table[0] = torch.cat([hole.table[0, :2], hole.table[0, 3:], hole.table[0, 2:3]])
    hole.lens, hole.seq = [84, 0], torch.tensor([84, 0], dtype=torch.int32, device="cuda")
    hole.check(out, lse)


def test_lengths_beyond_the_table_are_cut(moe):
    b = Batch([64, 30], 4, 2, 64, BF16, BF16, 16, spare_cols=0, seed=3)
    seq = torch.tensor([1000, -7], dtype=torch.int32, device="cuda")
    out, lse = moe.PagedAttention(2, 4, 2, 64).decode(b.q, b.k, b.v, b.table, seq)
    b.lens = [64, 0]
    b.check(out, lse)


def test_offsets_beyond_32_bits(moe):
    """The rows of a request lie beyond 2^31 elements (and 2^32 bytes) of the cache."""
    pages = 2**31 // (64 * 8 * 128) + 40
    b = Batch([600, 64], 16, 8, 128, BF16, BF16, 64, pages=pages, low=pages - 30, seed=6)
    run(moe, b)
    del b
    torch.cuda.empty_cache()


def test_strided_queries_outputs_and_table(moe):
    b = Batch([100, 7, 300], 8, 2, 64, BF16, BF16, 16, seed=5)
    wide = torch.zeros((3, 8, 100), dtype=BF16, device="cuda")
    wide[:, :, 3:67] = b.q
    b.q = wide[:, :, 3:67]
    out = torch.full((3, 8, 70), 7.0, dtype=BF16, device="cuda")
    lse = torch.empty((3, 8), device="cuda")
    table = torch.full((3, b.table.shape[1] + 5), 9, dtype=torch.int32, device="cuda")
    table[:, :b.table.shape[1]] = b.table
    b.table = table[:, :b.table.shape[1]]
    moe.PagedAttention(3, 8, 2, 64).decode(b.q, b.k, b.v, b.table, b.seq, out=out[:, :, 1:65], lse=lse)
    b.check(out[:, :, 1:65], lse)
    assert (out[:, :, :1] == 7).all() and (out[:, :, 65:] == 7).all()


def test_one_handle_many_batches_streams_and_graphs(moe):
    attn = moe.PagedAttention(40, 16, 2, 128)
    batches = [Batch(lens, 16, 2, 128, BF16, BF16, 16, seed=i) for i, lens in enumerate(
        ([3000], [1] * 40, [500, 20000], [0], [64] * 17))]
    for b in batches + batches[::-1]:
        run(moe, b, attn)
    s, b = torch.cuda.Stream(), batches[2]
    want, _ = run(moe, b, attn)
    torch.cuda.synchronize()
    got, _ = attn.decode(b.q, b.k, b.v, b.table, b.seq, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out, lse, g = torch.empty_like(want), torch.empty((2, 16), device="cuda"), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        attn.decode(b.q, b.k, b.v, b.table, b.seq, out=out, lse=lse)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    b.lens, b.seq[1] = [500, 12345], 12345  # other lengths, same graph
    g.replay()
    torch.cuda.synchronize()
    b.check(out, lse)
    attn.decode(b.q[:0], b.k, b.v, b.table, b.seq)  # no request
    attn.close()


def test_refusals(moe):
    b = Batch([20, 30], 8, 2, 64, BF16, BF16, 16, seed=1)
    attn = moe.PagedAttention(2, 8, 2, 64)
    attn.decode(b.q, b.k, b.v, b.table, b.seq)
    for bad in (dict(q=b.q.cpu()), dict(q=b.q[:, :4]), dict(q=b.q.double()), dict(k_cache=b.k.float()),
                dict(v_cache=b.v.half()), dict(v_cache=b.v[:1]), dict(block_table=b.table[:1]),
                dict(block_table=b.table.long()), dict(seq_len=b.seq.long()), dict(seq_len=b.seq[:1]),
                dict(out=b.q[:1]), dict(lse=torch.empty((2, 8), dtype=F16, device="cuda"))):
        a = dict(q=b.q, k_cache=b.k, v_cache=b.v, block_table=b.table, seq_len=b.seq)
        a.update(bad)
        with pytest.raises(ValueError):
            attn.decode(**a)
    odd = torch.zeros((4, 16, 2, 68), dtype=BF16, device="cuda")[..., :64]  # rows off 16 bytes
    for bad in (dict(window=-1), dict(scale=float("nan")), dict(k_scale=2.0), dict(k_cache=odd)):
        a = dict(q=b.q, k_cache=b.k[:4], v_cache=b.v[:4], block_table=b.table, seq_len=b.seq)
        a.update(bad)
        with pytest.raises(moe.MoeError):
            attn.decode(**a)
    with pytest.raises(moe.MoeError):  # more requests than the handle holds
        big = Batch([1, 1, 1], 8, 2, 64, BF16, BF16, 16)
        attn.decode(big.q, big.k, big.v, big.table, big.seq)
    with pytest.raises(moe.MoeError):  # 8-bit rows need multiples of 16
        c = Batch([20], 2, 1, 72, BF16, E4M3, 16)
        moe.PagedAttention(1, 2, 1, 72).decode(c.q, c.k, c.v, c.table, c.seq)
    for bad in ((0, 8, 2, 64), (9000, 8, 2, 64), (1, 9, 2, 64), (1, 8, 2, 68), (1, 8, 2, 264), (1, 8, 0, 64)):
        with pytest.raises(moe.MoeError):
            moe.PagedAttention(*bad)


@pytest.mark.parametrize("cache", [F16, BF16, E4M3])
@pytest.mark.parametrize("dim", [64, 256])
def test_long_fp32_sums_keep_fp32_accuracy(moe, cache, dim):
    """Rounding errors of fp32 sums do not grow with the tokens of a warp: relative L2
    2e-6 (logits up to 16 in units of log 2 carry half an ulp, 5e-7, in fp32; the
    sums' own roundings stay below that)."""
    b = Batch([8192] * 12, 16, 8, dim, F32, cache, 64, q_std=2.0, seed=dim)
    out, _ = moe.PagedAttention(12, 16, 8, dim).decode(b.q, b.k, b.v, b.table, b.seq)
    at = torch.arange(8192, device="cuda")
    for i in (0, 5, 11):
        pg = b.table[i, at // 64].long()
        k, v = rows_of(b.k, pg, at % 64), rows_of(b.v, pg, at % 64)
        s = torch.einsum("hgd,lhd->hgl", b.q[i].double().unflatten(0, (8, -1)), k) / math.sqrt(dim)
        want = torch.einsum("hgl,lhd->hgd", torch.softmax(s, -1), v).flatten(0, 1)
        assert float((out[i].double() - want).norm() / want.norm()) < 2e-6


def test_refuses_other_ranks(moe):
    b = Batch([20, 30], 8, 2, 64, BF16, BF16, 16, seed=1)
    attn = moe.PagedAttention(2, 8, 2, 64)
    for bad in (dict(q=b.q[0]), dict(q=b.q[0, 0, 0]), dict(k_cache=b.k[0]), dict(v_cache=b.v[0]),
                dict(v_cache=b.v[0, 0, 0, 0]), dict(block_table=b.table[0]), dict(seq_len=b.seq[0]), dict(out=b.q[0]),
                dict(lse=torch.empty(2, device="cuda"))):
        a = dict(q=b.q, k_cache=b.k, v_cache=b.v, block_table=b.table, seq_len=b.seq)
        a.update(bad)
        with pytest.raises(ValueError):
            attn.decode(**a)
