"""moe_block_norm against the definition in 64 bits.

Bounds from the arithmetic: a sum of dim squares in fp32 over at most 64
sequential terms and a tree is within 80 half-ulps, its rsqrt within half of
that and 2 ulp; a sigmoid is within 6; the products and the sum of r add 6: 64
half-ulps (2^-24) of |alpha x| + |beta g u| for r, the same again for the norm
of r, whose own error enters times the norm's factor.  Then half an ulp of the
stored type.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
HALF_ULP = {F32: (2.0**-24, 0.0), F16: (2.0**-11, 2.0**-25), BF16: (2.0**-8, 0.0)}
EPS = 1e-5


@pytest.fixture(scope="module")
def moe():
    import serving_router_sigmoid_gb300 as m
    torch.cuda.set_device(0)
    return m


def reference(x, y, w_post, gate, w_pre, alpha, beta, sigmoid, eps=EPS):
    """out, normed and the bounds of their fp32 errors, in 64 bits."""
    d = lambda t: None if t is None else t.double().cpu()  # noqa: E731
    x, y, w_post, gate, w_pre = map(d, (x, y, w_post, gate, w_pre))
    u = torch.zeros_like(x) if y is None else y
    if w_post is not None:
        u = u / (u.square().mean(-1, keepdim=True) + eps).sqrt() * w_post
    if gate is not None:
        u = u * (torch.sigmoid(gate) if sigmoid else gate)
    r = alpha * x + beta * u
    er = 64 * 2.0**-24 * ((alpha * x).abs() + (beta * u).abs())
    f = 1 / (r.square().mean(-1, keepdim=True) + eps).sqrt()
    w = 1.0 if w_pre is None else w_pre
    n = r * f * w
    # the error of r in the factor: its relative size in the row's norm
    rel = er.square().sum(-1, keepdim=True).sqrt() / (r.square().sum(-1, keepdim=True).sqrt() + 1e-300)
    return r, er, n, er * f * abs(w) + n.abs() * (64 * 2.0**-24 + rel)


def near(got, want, err):
    rel, ab = HALF_ULP[got.dtype]
    got = got.double().cpu()
    bound = err * (1 + rel) + want.abs() * rel + ab
    bad = (got - want).abs() > bound
    assert not bad.any(), (int(bad.sum()), float(((got - want).abs() - bound).max()))


def check(moe, n, dim, dt=F32, post=True, pre=True, gate=None, act="sigmoid", y=True, alpha=1.0, beta=0.5, pad=0,
          alias=False, scale=1.0, zero_row=False, norm=None):
    g = torch.Generator().manual_seed(n * 7 + dim)
    new = lambda shape: torch.randn(shape, generator=g)  # noqa: E731
    x = (new((n, dim + pad)) * 3 * scale).to(dt).cuda()[:, :dim]
    yy = (new((n, dim + pad)) * scale).to(dt).cuda()[:, :dim] if y else None
    if zero_row:
        x[0] = 0
        if y:
            yy[0] = 0
    wp, wn = ((1 + 0.1 * new(dim)).cuda() if f else None for f in (post, pre))
    gt = None if gate is None else new({"token": (n, 1), "channel": (1, dim), "full": (n, dim), "one": (1, 1)}[gate]).to(
        dt).cuda()
    r, er, nn, en = reference(x, yy, wp, gt, wn, alpha, beta, act == "sigmoid")
    kw = dict(out=x, normed=yy) if alias else {}
    out, normed = moe.block_norm(x, yy, w_post=wp, gate=gt, w_pre=wn, alpha=alpha, beta=beta, eps=EPS, gate_act=act,
                                 norm=norm, **kw)
    near(out, r, er)
    if pre or norm or alias:
        near(normed, nn, en)
    else:
        assert normed is None


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("dim", [1, 2, 31, 64, 100, 256, 1000, 2049, 4096, 6144, 8192, 8200, 12289, 16384])
def test_sizes_and_types(moe, dt, dim):
    check(moe, 3, dim, dt)
    check(moe, 3, dim, dt, gate="full")


@pytest.mark.parametrize("gate", [None, "token", "channel", "full", "one"])
@pytest.mark.parametrize("act", ["sigmoid", "none"])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
def test_forms(moe, gate, act, post, pre):
    check(moe, 5, 512, F32, post, pre, gate, act)
    check(moe, 5, 130, BF16, post, pre, gate, act, alpha=0.7, beta=-1.3)


@pytest.mark.parametrize("n", [0, 1, 2, 151, 153, 2048])
def test_token_counts(moe, n):
    check(moe, n, 768, BF16, gate="full")
    check(moe, n, 256, F32)


def test_plain_norm_views_and_aliases(moe):
    check(moe, 6, 640, F32, post=False, y=False, gate=None)
    check(moe, 6, 640, F32, post=False, pre=False, y=False, norm=True)
    check(moe, 6, 640, F32, pad=5)
    check(moe, 6, 640, BF16, pad=8, gate="full")
    check(moe, 6, 640, F32, alias=True)
    check(moe, 6, 6144, F16, alias=True)
    check(moe, 6, 641, F16, alias=True)


def test_zero_rows_tiny_and_large_values(moe):
    check(moe, 4, 384, F32, zero_row=True)
    check(moe, 4, 384, F32, scale=1e-6)
    check(moe, 4, 384, F32, scale=1e12)


def test_the_block_that_the_layer_computes(moe):
    """x + y and its norm are what moe_block_forward's residual block does."""
    x, y = torch.randn((8, 6144), device="cuda"), torch.randn((8, 6144), device="cuda")
    out, normed = moe.block_norm(x, y, w_pre=torch.ones(6144, device="cuda"))
    assert torch.equal(out, x + y)
    s, _ = moe.block_norm(x, y, stream=torch.cuda.current_stream())
    assert torch.equal(s, out)


def test_refusals(moe):
    x, w = torch.randn((4, 64), device="cuda"), torch.ones(64, device="cuda")
    moe.block_norm(x, x.clone(), w_post=w)
    for bad in (dict(x=x.cpu()), dict(x=x.double()), dict(x=x[0]), dict(y=x.half()), dict(y=x[:2]), dict(w_post=w[:8]),
                dict(w_pre=w.half()), dict(gate=x[:, :8]), dict(gate=x.half()), dict(gate_act="tanh"),
                dict(out=x[:1]), dict(x=x.t()[:, :4]), dict(w_pre=w, norm=False)):
        a = dict(x=x, y=x.clone())
        a.update(bad)
        with pytest.raises(ValueError):
            moe.block_norm(**a)
    for bad in (dict(eps=-1.0), dict(alpha=float("inf")), dict(y=None, w_post=w)):
        a = dict(x=x, y=x.clone())
        a.update(bad)
        with pytest.raises(moe.MoeError):
            moe.block_norm(**a)
    with pytest.raises(moe.MoeError):
        moe.block_norm(torch.ones((1, 20000), device="cuda"))
