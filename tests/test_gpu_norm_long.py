"""moe_block_norm over many rows: the kernel that goes through rows with copies in
flight (from 8 rows an SM), at each number of pieces a thread and of copies, and
the one with a block a row that fetches its weights late.

The definition in 64 bits and its bounds as for small batches: sums of at most 64
sequential squares a thread and a tree, so 64 half-ulps of fp32 for each norm and
for r, the error of r in its norm, and half an ulp of the stored type.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
HALF_ULP = {F32: (2.0**-24, 0.0), F16: (2.0**-11, 2.0**-25), BF16: (2.0**-8, 0.0)}
EPS, H = 1e-5, 64 * 2.0**-24


@pytest.fixture(scope="module")
def moe():
    import serving_router_sigmoid_gb300 as m
    torch.cuda.set_device(0)
    return m


def near(got, want, err, what):
    rel, ab = HALF_ULP[got.dtype]
    off = (got.double() - want).abs() - (err * (1 + rel) + want.abs() * rel + ab)
    assert not (off > 0).any(), (what, int((off > 0).sum()), float(off.max()), (off > 0).nonzero()[0].tolist())


def check(moe, n, dim, dt, post=True, pre=True, gate="full", y=True, alias=False, act="sigmoid", pad=0):
    g = torch.Generator(device="cuda").manual_seed(n + dim)
    new = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    wide = lambda std: (new(n, dim + pad) * std).to(dt)[:, :dim]  # noqa: E731
    x, yy = wide(3.0), wide(1.0) if y else None
    x[n // 2] *= 4  # no two rows look alike
    wp, wn = 1 + 0.1 * new(dim) if post and y else None, 1 + 0.1 * new(dim) if pre else None
    shape = {None: None, "token": (n, 1), "channel": (1, dim), "full": (n, dim)}[gate if y else None]
    gt = None if shape is None else new(*shape).to(dt)
    u = torch.zeros((n, dim), dtype=torch.float64, device="cuda") if yy is None else yy.double()
    if wp is not None:
        u = u / (u.square().mean(-1, keepdim=True) + EPS).sqrt() * wp.double()
    if gt is not None:
        u = u * (torch.sigmoid(gt.double()) if act == "sigmoid" else gt.double())
    r = 1.5 * x.double() - 0.5 * u
    er = H * ((1.5 * x.double()).abs() + (0.5 * u).abs())
    f = 1 / (r.square().mean(-1, keepdim=True) + EPS).sqrt()
    w = 1.0 if wn is None else wn.double()
    nn = r * f * w
    en = er * f * (w if wn is None else w.abs()) + nn.abs() * (H + er.norm(dim=-1, keepdim=True) / r.norm(dim=-1, keepdim=True))
    normed = yy if alias else torch.full((n, dim), 7.0, dtype=dt, device="cuda") if pre else None
    out, got = moe.block_norm(x, yy, w_post=wp, gate=gt, w_pre=wn, alpha=1.5, beta=-0.5, eps=EPS, gate_act=act,
                              out=x if alias else None, normed=normed)
    what = (n, dim, dt, post, pre, gate, y, alias)
    near(out, r, er, what)
    if normed is not None:
        near(got, nn, en, what)
    else:
        assert got is None


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


LONG = [(F32, 5632), (F32, 6144), (BF16, 5632), (F16, 6144), (BF16, 8192), (BF16, 9216), (F16, 12288), (BF16, 14336),
        (F16, 16384), (BF16, 16384)]
ROWS = [(F32, 2304), (F32, 4096), (F32, 5120), (F32, 8192), (F32, 16384), (BF16, 4352), (F16, 5120)]


@pytest.mark.parametrize("dt,dim", LONG + ROWS)
def test_forms(moe, dt, dim):
    """Every form of the call, and batches around the eight rows an SM and with an uneven last round."""
    n = 8 * sms()
    for rows in (n - 1, n, n + 1, 2048):
        check(moe, rows, dim, dt)
    for kw in (dict(gate=None), dict(gate="token"), dict(gate="channel"), dict(post=False), dict(pre=False),
               dict(post=False, pre=False, gate=None), dict(post=False, gate=None), dict(pre=False, gate="token"),
               dict(y=False), dict(y=False, pre=False), dict(act="none"), dict(gate="token", act="none")):
        check(moe, n + 37, dim, dt, **kw)


@pytest.mark.parametrize("dt,dim", LONG + ROWS)
def test_aliases_and_strides(moe, dt, dim):
    n = 8 * sms() + 101
    check(moe, n, dim, dt, alias=True)
    check(moe, n, dim, dt, alias=True, post=False, gate=None)
    check(moe, n, dim, dt, pad=16)


@pytest.mark.parametrize("dt,dim", LONG + ROWS)
def test_medium_batches(moe, dt, dim):
    """A block a row, weights early or late."""
    for n in (sms(), sms() + 1, 2 * sms() - 4, 4 * sms(), 4 * sms() + 1, 1000):
        check(moe, n, dim, dt, gate="full" if n % 2 else "token")
    check(moe, 300, dim, dt, alias=True)
    check(moe, 300, dim, dt, y=False)


@pytest.mark.parametrize("dt,dim", [(F32, 6143), (BF16, 6146), (F16, 8199)])
def test_rows_off_16_bytes(moe, dt, dim):
    check(moe, 8 * sms() + 3, dim, dt)
    check(moe, 300, dim, dt, post=False, gate="channel")


def test_the_same_bits_again(moe):
    """A row's result does not depend on the batch around it."""
    for dt, dim in ((F32, 6144), (BF16, 8192), (F16, 16384)):
        n = 9 * sms()
        g = torch.Generator(device="cuda").manual_seed(1)
        x, y, gt = (torch.randn((n, dim), generator=g, device="cuda").to(dt) for _ in range(3))
        w = torch.randn(dim, generator=g, device="cuda")
        first = moe.block_norm(x, y, w_post=w, gate=gt, w_pre=w)
        for _ in range(5):
            again = moe.block_norm(x, y, w_post=w, gate=gt, w_pre=w)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
