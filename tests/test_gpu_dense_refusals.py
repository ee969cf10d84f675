"""Calls that the FP8 products and the latent attention refuse, as ValueError in
the binding or MoeError from the library, and the edges that they take."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

E4 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def moe():
    import serving_router_sigmoid_gb300 as m
    torch.cuda.set_device(0)
    return m


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def refused(moe, call, *a, **k):
    with pytest.raises((ValueError, moe.MoeError)):
        call(*a, **k)


def test_quantiser(moe):
    x = torch.randn((6, 256), device="cuda")
    for bad in (x[0], x[None], x.double(), x.int(), x[:, :24].contiguous(), x[:, ::2], x[:, 1:129], x.T,
                torch.randn((2, 65552), device="cuda")):
        refused(moe, moe.quant_act_fp8, bad)
    codes = torch.empty((6, 256), dtype=E4, device="cuda")
    for bad in (dict(x8=codes[:5]), dict(x8=codes.view(torch.int8)), dict(x8=codes[:, ::2]), dict(x8=x.view(E4)[:, :256]),
                dict(x8=codes[:1].expand(6, 256)), dict(scale=torch.empty((6, 3), device="cuda")),
                dict(scale=torch.empty((6, 2), device="cuda").double()), dict(scale=torch.empty((2, 6), device="cuda").T),
                dict(scale=x.view(-1)[4:16].view(6, 2)), dict(x8=codes, scale=codes.view(torch.float32).view(-1)[:12].view(6, 2)),
                dict(x8=codes.cpu())):
        refused(moe, moe.quant_act_fp8, x, **bad)
    x8, s = moe.quant_act_fp8(x[:1].expand(6, 256), x8=codes.view(torch.uint8))  # one row many times is fine
    assert torch.equal(x8[5], x8[0]) and torch.equal(s[5], s[0])


@pytest.mark.parametrize("dt", [torch.float32, torch.float16, torch.bfloat16])
def test_quantiser_of_nan_and_infinity(moe, dt):
    """As the formula: a NaN goes to its group's scale and codes, an infinity makes the scale one."""
    x = torch.randn((5, 300), device="cuda")[:, :288].to(dt).contiguous()
    clean8, clean = moe.quant_act_fp8(x)
    x[1, 130], x[2, 3], x[2, 9], x[3, 280], x[4, 270] = math.nan, math.inf, -math.inf, -math.inf, math.nan
    x[4, 271] = math.inf
    x8, s = moe.quant_act_fp8(x)
    f = torch.nn.functional.pad(x.float(), (0, 96)).view(5, 3, 128)
    want = (f.abs().amax(-1).double() / 448).float().clamp(min=1e-12)
    assert torch.equal(s.isnan(), want.isnan()) and torch.equal(s.nan_to_num(-1), want.nan_to_num(-1))
    codes = (f / want[..., None]).flatten(1)[:, :288]
    assert torch.equal(x8.float().isnan(), codes.isnan())
    fine = want.isfinite().repeat_interleave(128, 1)[:, :288]
    assert torch.equal(x8.view(torch.uint8)[fine], clean8.view(torch.uint8)[fine]) and int(fine.sum()) == 5 * 288 - 128 * 2 - 32 * 2
    at_inf = want.isinf().repeat_interleave(128, 1)[:, :288] & x.float().isfinite()
    assert bool((x8.float()[at_inf] == 0).all())


def test_linear(moe):
    x8, xs = moe.quant_act_fp8(torch.randn((6, 256), device="cuda"))
    w8, ws = torch.randn((200, 256), device="cuda").to(E4), torch.ones((2, 2), device="cuda")
    want = moe.fp8_linear(x8, xs, w8, ws)
    for bad in ((x8[0], xs, w8, ws), (x8.float(), xs, w8, ws), (x8[:, :128], xs, w8, ws), (x8, xs[:5], w8, ws),
                (x8, xs.double(), w8, ws), (x8, xs.T.contiguous().T, w8, ws), (x8, xs, w8.T, ws), (x8, xs, w8.half(), ws),
                (x8, xs, w8, ws[:1]), (x8, xs, w8, ws.half()), (x8, xs, w8.cpu(), ws), (x8[:, 8:136], xs[:, :1], w8[:, :128], ws[:, :1].contiguous())):
        refused(moe, moe.fp8_linear, *bad)
    out = torch.empty((6, 200), device="cuda")
    for bad in (dict(dtype=torch.float64), dict(out=out.double()), dict(out=out[:5]), dict(out=out.T.contiguous().T),
                dict(out=out[:1].expand(6, 200)), dict(out=w8.view(-1)[:4800].view(torch.float32).view(6, 200)),
                dict(out=out.cpu())):
        refused(moe, moe.fp8_linear, x8, xs, w8, ws, **bad)
    assert torch.equal(moe.fp8_linear(x8.view(torch.uint8), xs, w8.view(torch.uint8), ws), want)  # codes as bytes
    assert torch.equal(moe.fp8_linear(x8[:0], xs[:0], w8, ws), want[:0])


def test_linear_of_nan_codes(moe):
    """A NaN code or scale shows in its row, and in no other."""
    x8, xs = moe.quant_act_fp8(torch.randn((70, 512), device="cuda"))
    w8, ws = torch.randn((300, 512), device="cuda").to(E4), torch.ones((3, 4), device="cuda")
    for n in (5, 70):
        a, s = x8[:n].clone(), xs[:n].clone()
        want = moe.fp8_linear(a, s, w8, ws)
        a[3, 100], s[1, 2] = math.nan, math.nan
        got = moe.fp8_linear(a, s, w8, ws)
        bad = torch.zeros(n, dtype=torch.bool, device="cuda")
        bad[[1, 3]] = True
        assert bool(got[bad].isnan().all()) and torch.equal(got[~bad], want[~bad])


def test_decode(moe):
    n, h = 2, 4
    q = torch.randn((n, h, 576), device="cuda").half()
    cache = torch.randn((6, 16, 1, 576), device="cuda").half()
    table, lens = i32(0, 1, 2, 3).view(2, 2), i32(20, 30)
    attn = moe.LatentAttention(2, h)
    want, wl = attn.decode(q, cache, table, lens, 0.1)
    for bad in ((q.float(), cache, table, lens), (q[:, :3], cache, table, lens), (q[..., :512], cache, table, lens),
                (q[0], cache, table, lens), (q.bfloat16(), cache, table, lens), (q, cache.float(), table, lens),
                (q, cache[..., :512], table, lens), (q, cache.expand(-1, -1, 2, -1), table, lens), (q, cache[0, 0], table, lens),
                (q, cache, table.long(), lens), (q, cache, table[:1], lens), (q, cache, table.T, lens), (q, cache, table[0], lens),
                (q, cache, table, lens.long()), (q, cache, table, lens[:1]), (q, cache, table, lens.view(2, 1)),
                (q.cpu(), cache, table, lens), (q, cache.cpu(), table, lens), (q, cache, table, lens.cpu()),
                (torch.randn((3, h, 576), device="cuda").half(), cache, i32(*range(6)).view(3, 2), i32(1, 1, 1))):
        refused(moe, attn.decode, *bad, 0.1)
    for scale in (math.inf, math.nan, 2.0**121, 1e39, None, "1"):
        refused(moe, attn.decode, q, cache, table, lens, scale)
    for bad in (dict(k_scale=0.5), dict(k_scale=0), dict(k_scale=None), dict(out=want.float()), dict(out=want[:1]), dict(out=want[:1].expand(2, -1, -1)),
                dict(out=want[:, :1].expand(-1, h, -1)), dict(out=q[..., :512]), dict(out=cache.view(-1)[:n * h * 512].view(n, h, 512)),
                dict(lse=wl.double()), dict(lse=wl[:1]), dict(lse=q.view(torch.float32).view(-1)[:8].view(2, 4)),
                dict(out=want, lse=want.view(torch.float32).view(-1)[:8].view(2, 4))):
        refused(moe, attn.decode, q, cache, table, lens, 0.1, **bad)
    e4 = cache.to(E4)
    for k in (0.0, -1.0, math.inf, math.nan):
        refused(moe, attn.decode, q, e4, table, lens, 0.1, k_scale=k)
    refused(moe, attn.decode, q, e4, table, lens, 2.0**100, k_scale=2.0**30)
    off = torch.zeros(cache.numel() + 8, dtype=torch.float16, device="cuda")
    refused(moe, attn.decode, q, off[1:1 + cache.numel()].view(cache.shape), table, lens, 0.1)
    refused(moe, attn.decode, off[4:4 + q.numel()].view(q.shape), cache, table, lens, 0.1)
    big = torch.empty((1, 2**31 // 16), dtype=torch.int32, device="cuda")
    refused(moe, attn.decode, q[:1], cache, big, lens, 0.1)
    del big
    got, _ = attn.decode(q[:0], cache, table, lens, 0.1)  # no requests
    assert got.shape == (0, h, 512)
    got, gl = attn.decode(q, cache[:0], table, lens, 0.1)  # no pages
    assert bool((got == 0).all()) and bool((gl == -math.inf).all())
    got, gl = attn.decode(q, cache, table[:, :0], lens, 0.1)  # no table
    assert bool((got == 0).all()) and bool((gl == -math.inf).all())
    # q of one head row for all, cache pages that overlap: read only
    one = q[:, :1].expand(-1, h, -1)
    got, _ = attn.decode(one, cache, table, lens, 0.1)
    assert torch.equal(got, attn.decode(one.contiguous(), cache, table, lens, 0.1)[0])
    slide = torch.as_strided(cache, (6, 16, 1, 576), (576, 576, 576, 1))
    got, _ = attn.decode(q, slide, table, lens, 0.1)
    assert torch.equal(got, attn.decode(q, slide.contiguous(), table, lens, 0.1)[0])
    attn.close()
    attn.close()


def test_decode_takes_negative_and_zero_scales(moe):
    import test_gpu_latent_decode as t
    for dt in (torch.float16, torch.bfloat16):
        q, cache, table, lens = t.setup([70, 5, 2000], 8, 512, 64, dt, dt, 16, seed=1)
        attn = moe.LatentAttention(3, 8)
        for scale in (-0.07, 0.0):
            out, lse = attn.decode(q, cache, table, lens, scale)
            t.check(out, lse, q, cache, table, lens, 512, scale)


def test_prompt_takes_negative_and_zero_scales(moe):
    import test_gpu_latent_prompt as t
    for dims in ((128, 64, 128), (192, 64, 256)):
        a = t.setup([140, 3], [300, 3], 2, *dims, torch.bfloat16, seed=2)
        for scale in (-0.07, 0.0):
            for causal in (True, False):
                out, lse = moe.latent_prompt(*a, scale, causal=causal)
                t.check(out, lse, *a, scale, causal)


def test_prompt(moe):
    nq, h = 10, 4
    q, k = torch.randn((nq, h, 192), device="cuda").half(), torch.randn((nq, h, 128), device="cuda").half()
    r, v = torch.randn((nq, 64), device="cuda").half(), torch.randn((nq, h, 128), device="cuda").half()
    s = i32(0, 4, 10)
    want, wl = moe.latent_prompt(q, k, r, v, s, s, 0.1)
    for bad in ((q.float(), k, r, v, s, s), (q.bfloat16(), k, r, v, s, s), (q, k.bfloat16(), r, v, s, s), (q, k, r.float(), v, s, s),
                (q, k, r, v.float(), s, s), (q[..., :128], k, r, v, s, s), (q, k, None, v, s, s), (q, k, r[:9], v, s, s),
                (q, k, r, v[:9], s, s), (q, k[:, :3], r, v, s, s), (q, k, r, v[:, :2], s, s), (q[0], k, r, v, s, s),
                (q, k[0], r, v, s, s), (q, k, r[0], v, s, s), (q, k, r[:, None], v, s, s), (q, k, r, v, s.long(), s), (q, k, r, v, s, s[:2]),
                (q, k, r, v, s[None], s), (q, k, r, v, s[::2], s), (q, k, r, v, s[:0], s[:0]), (q.cpu(), k, r, v, s, s),
                (q, k, r, v, s, s.cpu()), (q, k, r[:1].expand(nq, 64), v, s, s), (q, k[:1].expand(nq, h, 128), r, v, s, s),
                (q[:1].expand(nq, h, 192), k, r, v, s, s), (q.transpose(1, 2).contiguous().transpose(1, 2), k, r, v, s, s)):
        refused(moe, moe.latent_prompt, *bad, 0.1)
    for scale in (math.inf, math.nan, 2.0**121, -1e39, None, "x"):
        refused(moe, moe.latent_prompt, q, k, r, v, s, s, scale)
    for bad in (dict(out=want.float()), dict(out=want[:9]), dict(out=want[:1].expand(nq, h, 128)),
                dict(out=want[:, :1].expand(nq, h, 128)), dict(out=q[..., :128]), dict(out=k), dict(out=v),
                dict(out=want.transpose(1, 2).contiguous().transpose(1, 2)), dict(lse=wl.double()), dict(lse=wl[:9]),
                dict(out=want, lse=want.view(torch.float32).view(-1)[:40].view(nq, h)), dict(lse=r.view(torch.float32).view(-1)[:40].view(nq, h))):
        refused(moe, moe.latent_prompt, q, k, r, v, s, s, 0.1, **bad)
    for at in range(4):  # rows that start off 16 bytes
        t = [q, k, r, v]
        off = torch.zeros(t[at].numel() + 8, dtype=torch.float16, device="cuda")
        t[at] = off[1:1 + t[at].numel()].view(t[at].shape)
        refused(moe, moe.latent_prompt, *t, s, s, 0.1)
    for nope, rope, vd in ((120, 64, 128), (128, 72, 128), (208, 64, 128), (128, 64, 272), (128, 8, 128), (128, 64, 100)):
        new = lambda *shape: torch.zeros(shape, dtype=torch.float16, device="cuda")  # noqa: E731
        refused(moe, moe.latent_prompt, new(nq, h, nope + rope), new(nq, h, nope), new(nq, rope), new(nq, h, vd), s, s, 0.1)
    got, gl = moe.latent_prompt(q[:0], k, r, v, s, s, 0.1)
    assert got.shape == (0, h, 128) and gl.shape == (0, h)
    got, gl = moe.latent_prompt(q, k[:0], r[:0], v[:0], s, s, 0.1)  # no keys at all
    assert bool((got == 0).all()) and bool((gl == -math.inf).all())
    got, gl = torch.full_like(want, 3.0), torch.full_like(wl, 5.0)
    moe.latent_prompt(q, k, r, v, s[:1], s[:1], 0.1, out=got, lse=gl)  # no requests: nothing is written
    assert bool((got == 3).all()) and bool((gl == 5).all())
    one = moe.latent_prompt(q[:1], k[:1], r[:1], v[:1], i32(0, 1), i32(0, 1), 0.1)  # one token sees itself
    assert torch.equal(one[0], v[:1])


def test_sizes_of_a_handle(moe):
    for bad in ((0, 4), (8193, 4), (1, 0), (1, 1025), (1, 4, 500), (1, 4, 576), (1, 4, 0), (1, 4, 512, 72), (1, 4, 512, 80)):
        refused(moe, moe.LatentAttention, *bad)
    attn = moe.LatentAttention(8192, 1024)  # the largest workspace
    q = torch.randn((3, 1024, 576), device="cuda").bfloat16()
    cache, table, lens = torch.randn((5, 64, 1, 576), device="cuda").bfloat16(), i32(0, 1, 2, 3, 4, -1).view(3, 2), i32(128, 100, 60)
    import test_gpu_latent_decode as t
    out, lse = attn.decode(q, cache, table, lens, 0.07)
    t.check(out, lse, q, cache, table, lens, 512, 0.07)


def test_the_largest_batch(moe):
    """Thousands of requests, most of them one token or none, over the same pages."""
    import test_gpu_latent_decode as t
    g = torch.Generator(device="cuda").manual_seed(6)
    n = 8192
    cache = t.normal(g, (40, 16, 1, 128), torch.float16)
    table = torch.randint(0, 40, (n, 3), generator=g, device="cuda").to(torch.int32)
    lens = torch.randint(0, 4, (n,), generator=g, device="cuda").to(torch.int32)
    lens[::500] = 48
    q = t.normal(g, (n, 2, 128), torch.float16)
    out, lse = moe.LatentAttention(n, 2, 64, 64).decode(q, cache, table, lens, 0.1)
    some = torch.cat([torch.arange(0, n, 500), torch.arange(5, n, 331)]).cuda()
    t.check(out[some], lse[some], q[some], cache, table[some], lens[some], 64, 0.1)
    none = lens == 0
    assert bool((out[none] == 0).all()) and bool((lse[none] == -math.inf).all())
    assert moe.dense_status() == 0


def test_two_calls_at_once(moe):
    """Calls without a handle on two streams share nothing."""
    import test_gpu_latent_prompt as t
    a, b = t.setup([300, 40], [300, 500], 4, 128, 64, 128, torch.bfloat16, seed=3), t.setup([200], [900], 8, 192, 64, 256, torch.float16, seed=4)
    x = torch.randn((500, 1024), device="cuda")
    w8, ws = torch.randn((640, 1024), device="cuda").to(E4), torch.ones((5, 8), device="cuda")

    def calls(stream):
        x8, xs = moe.quant_act_fp8(x, stream=stream)
        few = moe.fp8_linear(x8[:20], xs[:20], w8, ws, stream=stream)
        return [*moe.latent_prompt(*a, 0.07, stream=stream), x8.view(torch.uint8), xs, few,
                moe.fp8_linear(x8, xs, w8, ws, stream=stream), *moe.latent_prompt(*b, 0.06, stream=stream)]
    want = calls(None)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    got = [calls(s) for _ in range(5) for s in (sa, sb)]
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for g in got for p, q in zip(g, want))
    assert moe.dense_status() == 0
