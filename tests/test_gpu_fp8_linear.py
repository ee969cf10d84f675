"""quant_act_fp8 and fp8_linear against their definitions.

Codes and scales of the quantiser are those of the formula in fp32, bit for bit
(maximum, two IEEE divisions, one rounding to E4M3).

A product's error: the exact value is a sum over blocks b of 128 of x_scale *
w_scale * (a sum of 128 exact products).  In fp32, with A the sum of the absolute
values of all products: adding up a block costs at most one unit of 2^-23 of it
for each of its 4 tensor-core steps (or 128 / 32 lane sums and 5 shuffles), the
scale product and its application 2 x 2^-24, the sum over nb blocks nb x 2^-24,
sums of split contractions a few more.  So |error| <= (nb + 16) 2^-22 A holds with
room, plus half a step of the output type: 2^-8 (bf16), 2^-11 (f16), 2^-24 (f32)
of the value, and half the smallest subnormal for f16.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0**-24, torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8}
TINY = {torch.float32: 0.0, torch.float16: 2.0**-25, torch.bfloat16: 0.0}


@pytest.fixture(scope="module")
def moe():
    import serving_router_sigmoid_gb300 as m
    return m


def groups(x):
    n, dim = x.shape
    return torch.nn.functional.pad(x, (0, -dim % 128)).view(n, -1, 128)


def by_formula(x):
    g = groups(x.float())
    # torch multiplies by the reciprocal of a number; a quotient of 53 bits rounds to the IEEE one of 24
    s = (g.abs().amax(-1).double() / 448).float().clamp(min=1e-12)
    return (g / s[..., None]).clamp(-448, 448).flatten(1)[:, :x.shape[1]].to(torch.float8_e4m3fn), s


@pytest.mark.parametrize("dt", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,dim", [(1, 16), (1, 6144), (3, 128), (5, 144), (33, 576), (7, 1040), (300, 2048), (2, 65536)])
def test_codes_are_the_formulas(moe, dt, n, dim):
    g = torch.Generator(device="cuda").manual_seed(n + dim)
    x = (torch.randn((n, dim), generator=g, device="cuda") * torch.randn(dim, generator=g, device="cuda").exp()).to(dt)
    x[0, :16] = 0
    if n > 2:
        x[1] = 0                      # the scale's floor
        x[2, :8] = 1e-7               # small numbers next to larger ones
    x8, s = moe.quant_act_fp8(x)
    want, ws = by_formula(x)
    assert torch.equal(s, ws)
    assert torch.equal(x8.view(torch.uint8), want.view(torch.uint8))


def test_ties_and_every_code(moe):
    codes = torch.arange(256, dtype=torch.int32, device="cuda").to(torch.uint8)
    vals = codes.view(torch.float8_e4m3fn).float()
    vals = vals[vals.isfinite()]                     # 254 numbers
    pos = vals[vals >= 0].unique()
    mid = (pos[1:] + pos[:-1]) / 2                   # every tie between neighbours, exact in fp32
    row = torch.cat([vals, mid, -mid])
    row = torch.nn.functional.pad(row, (0, -row.numel() % 127)).view(-1, 127)
    x = torch.cat([torch.full((row.shape[0], 1), 448.0, device="cuda"), row], 1)  # scale 1 in every group
    x8, s = moe.quant_act_fp8(x)
    assert torch.equal(s, torch.ones_like(s))
    assert torch.equal(x8.view(torch.uint8), x.to(torch.float8_e4m3fn).view(torch.uint8))


def test_quant_strides_outputs_and_stream(moe):
    big = torch.randn((40, 1024), device="cuda")
    x = big[::2, 256:256 + 400]
    buf = torch.full((20, 512), 7, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scale = torch.empty((20, 4), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, sc = moe.quant_act_fp8(x, x8=buf[:, 32:432], scale=scale, stream=s)
    s.synchronize()
    want, ws = by_formula(x)
    assert sc is scale and torch.equal(scale, ws)
    assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
    raw = buf.view(torch.uint8)
    assert bool((raw[:, :32] == 7).all()) and bool((raw[:, 432:] == 7).all())
    e8, es = moe.quant_act_fp8(torch.empty((0, 256), device="cuda"))
    assert e8.shape == (0, 256) and es.shape == (0, 2)


def operands(n, inner, outer, seed, wide=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    nb, ob = -(-inner // 128), -(-outer // 128)
    x8 = (new(n, inner) * (300 if wide else 60)).clamp(-448, 448).to(torch.float8_e4m3fn)
    w8 = (new(outer, inner) * (300 if wide else 60)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return x8, new(n, nb).exp() * 1e-3, w8, new(ob, nb).exp() * 1e-4


def definition(x8, xs, w8, ws):
    """The value and the sum of absolute products, in 64 bits."""
    n, inner = x8.shape
    x = x8.double() * xs.double().repeat_interleave(128, 1)[:, :inner]
    w = w8.double() * ws.double().repeat_interleave(128, 0)[:w8.shape[0]].repeat_interleave(128, 1)[:, :inner]
    return x @ w.T, x.abs() @ w.abs().T


def check(out, x8, xs, w8, ws):
    ref, total = definition(x8, xs, w8, ws)
    off = (out.double() - ref).abs()
    room = HALF[out.dtype] * ref.abs() + TINY[out.dtype] + (xs.shape[1] + 16) * 2.0**-22 * total * (1 + HALF[out.dtype])
    assert bool((off <= room).all()), float((off / room.clamp(min=1e-300)).max())


SHAPES = [(1, 16, 1), (1, 128, 128), (1, 6144, 576), (2, 144, 40), (3, 1040, 129), (5, 2048, 1000), (8, 6144, 512),
          (15, 576, 300), (16, 512, 2048), (17, 640, 77), (31, 2048, 129), (32, 1040, 640), (33, 256, 1024), (64, 6144, 576),
          (65, 1040, 200), (100, 128, 4000), (128, 2048, 384), (129, 576, 257), (200, 8192, 128), (255, 1552, 520),
          (300, 4096, 1536), (513, 272, 1281), (1000, 2048, 640)]


@pytest.mark.parametrize("n,inner,outer", SHAPES)
def test_linear_against_64_bits(moe, n, inner, outer):
    ops = operands(n, inner, outer, n + inner + outer, wide=outer % 2 == 0)
    for dt in HALF:
        check(moe.fp8_linear(*ops, dtype=dt), *ops)
    assert moe.dense_status() == 0


def test_linear_all_sums_exact(moe):
    """Codes +-1 with scales of one: whole numbers, exact in fp32."""
    for n, inner, outer in ((4, 8192, 384), (40, 8192, 384), (160, 8192, 384)):
        g = torch.Generator(device="cuda").manual_seed(n)
        x = torch.randint(0, 2, (n, inner), generator=g, device="cuda").float() * 2 - 1
        w = torch.randint(0, 2, (outer, inner), generator=g, device="cuda").float() * 2 - 1
        one = lambda r: torch.ones((r, inner // 128), device="cuda")  # noqa: E731
        out = moe.fp8_linear(x.to(torch.float8_e4m3fn), one(n), w.to(torch.float8_e4m3fn).view(torch.uint8), one(3),
                             dtype=torch.float32)
        assert torch.equal(out, (x.double() @ w.double().T).float())


@pytest.mark.parametrize("n", [3, 40, 200])
def test_linear_strides_guard_and_repeat(moe, n):
    inner, outer = 400, 333
    x8, xs, w8, ws = operands(n, inner, outer, 5)
    xb = torch.zeros((n, 512), dtype=torch.uint8, device="cuda")
    wb = torch.full((outer, 464), 0x7F, dtype=torch.uint8, device="cuda")  # NaN between the rows
    xb[:, 16:416], wb[:, 32:432] = x8.view(torch.uint8), w8.view(torch.uint8)
    xb[:, :16], xb[:, 416:] = 0x7F, 0x7F
    room = torch.full((n + 2, outer + 5), 9.0, dtype=torch.bfloat16, device="cuda")
    out = moe.fp8_linear(xb[:, 16:416].view(torch.float8_e4m3fn), xs, wb[:, 32:432], ws, out=room[1:-1, 2:-3])
    check(out, x8, xs, w8, ws)
    assert bool((room[0] == 9).all()) and bool((room[-1] == 9).all())
    assert bool((room[:, :2] == 9).all()) and bool((room[:, -3:] == 9).all())
    again = moe.fp8_linear(x8, xs, w8, ws)
    for _ in range(20):
        assert torch.equal(moe.fp8_linear(x8, xs, w8, ws), again)


def test_linear_rows_do_not_depend_on_the_batch_codes(moe):
    """A NaN code stays in its row and its column."""
    x8, xs, w8, ws = operands(50, 512, 300, 3)
    x8.view(torch.uint8)[7, 100] = 0x7F
    w8.view(torch.uint8)[131, 5] = 0xFF
    bad = moe.fp8_linear(x8, xs, w8, ws).isnan()
    want = torch.zeros_like(bad)
    want[7], want[:, 131] = True, True
    assert torch.equal(bad, want)


def test_linear_empty_streams_and_graph(moe):
    x8, xs, w8, ws = operands(48, 1024, 500, 9)
    assert moe.fp8_linear(x8[:0], xs[:0], w8, ws).shape == (0, 500)
    want = moe.fp8_linear(x8, xs, w8, ws)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (a, b):
        s.wait_stream(torch.cuda.current_stream())
    got = [moe.fp8_linear(x8, xs, w8, ws, stream=s) for _ in range(4) for s in (a, b)]  # two streams at once
    torch.cuda.synchronize()
    assert all(torch.equal(t, want) for t in got)
    x = torch.zeros((48, 1024), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, s = moe.quant_act_fp8(x)
        out = moe.fp8_linear(q, s, w8, ws, dtype=torch.float32)
    for seed in (1, 2):
        x.copy_(torch.randn((48, 1024), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
        graph.replay()
        check(out, *by_formula(x), w8, ws)


def test_int32_offsets_are_passed(moe):
    """A matrix and an output beyond 2^31 elements."""
    inner, outer = 16, 140_000
    x8, xs, w8, ws = operands(70, inner, outer, 4)
    big = torch.zeros((outer, 16384), dtype=torch.uint8, device="cuda")  # 2.3 GB
    big[:, :16] = w8.view(torch.uint8)
    want = moe.fp8_linear(x8, xs, w8, ws)
    check(want, x8, xs, w8, ws)
    assert torch.equal(moe.fp8_linear(x8, xs, big[:, :16], ws), want)
    assert torch.equal(moe.fp8_linear(x8[:5], xs[:5], big[:, :16], ws), moe.fp8_linear(x8[:5], xs[:5], w8, ws))
    n = 16500
    x8, xs, w8, ws = operands(n, inner, outer, 4)
    out = moe.fp8_linear(x8, xs, w8, ws)
    check(out[-130:], x8[-130:], xs[-130:], w8, ws)


def test_quant_offsets_beyond_32_bits(moe):
    step = 1 << 30
    x = torch.randn((5, 272), device="cuda").half()
    big, codes = (torch.empty(4 * step + 512, dtype=t, device="cuda") for t in (torch.float16, torch.uint8))
    xf, cf = (torch.as_strided(b, (5, 272), (step, 1)) for b in (big, codes))
    xf.copy_(x)
    want, ws = moe.quant_act_fp8(x)
    got, s = moe.quant_act_fp8(xf, x8=cf)
    assert torch.equal(got, want.view(torch.uint8)) and torch.equal(s, ws)


def test_as_many_blocks_as_find_room(moe):
    """Tile counts around what clusters of every size hold at once, with contractions to split."""
    for n, inner, outer in ((128, 1152, 1024), (128, 1152, 1920), (130, 1152, 1920), (128, 1152, 2944), (200, 640, 3584),
                            (128, 1152, 6144), (128, 256, 9728), (20, 1152, 5888), (20, 1152, 6144), (40, 1152, 19456)):
        x8, xs, w8, ws = operands(n, inner, outer, n + outer)
        check(moe.fp8_linear(x8, xs, w8, ws, dtype=torch.float32), x8, xs, w8, ws)
    assert moe.dense_status() == 0


@pytest.mark.parametrize("inner", [128, 640, 1152, 1040, 256])
@pytest.mark.parametrize("n", [5, 16, 32])
def test_few_tokens_of_many_tiles(moe, n, inner):
    """More tiles of 128 rows than blocks run at once, scales of neighbouring blocks of rows 2^20 apart."""
    outer = 80_000
    x8, xs, w8, ws = operands(n, inner, outer, n + inner)
    ws *= torch.where(torch.arange(ws.shape[0], device="cuda") * 7 % 5 < 2, 2.0**-20, 1.0)[:, None]
    out = moe.fp8_linear(x8, xs, w8, ws, dtype=torch.float32)
    check(out, x8, xs, w8, ws)
    for _ in range(50):
        assert torch.equal(moe.fp8_linear(x8, xs, w8, ws, dtype=torch.float32), out)
    assert moe.dense_status() == 0


def test_quant_as_many_rows_as_are_counted(moe):
    """2^31 - 2 rows: the last launch begins where one step more passes 31 bits (codes and scales 43 GB)."""
    n = 2**31 - 2
    row = torch.randn((1, 16), device="cuda").half()
    want, ws = by_formula(row)
    x8 = torch.full((n, 16), 0x55, dtype=torch.uint8, device="cuda")
    x8, s = moe.quant_act_fp8(row.expand(n, 16), x8=x8)
    step = 1 << 27
    for t in range(0, n, step):
        assert bool((x8[t:t + step].view(torch.int64) == want.view(torch.int64)).all())
        assert bool((s[t:t + step] == ws).all())
    torch.cuda.synchronize()
