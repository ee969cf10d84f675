"""moe_rope_append against the definition in 64 bits.

Bounds, per element of a rotated pair (a, b), fixed from the arithmetic: cos
and sin come from sincospif (within 2 ulp) of an angle within 2^-32 of a half
turn, times the amplitude; a c - b s has two products and a sum: together at
most 8 half-ulps of fp32, 8 * 2^-24 * amplitude * (|a| + |b|), and for 2^-32 pi
another 2^-26 of it.  Then one rounding to the stored type: half an ulp, 2^-8
relative for bf16, 2^-11 for f16 (or 2^-25 absolute below its normals), 2^-4
for e4m3 (or 2^-10 absolute, in units of the scale).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

F32, F16, BF16, E4M3 = torch.float32, torch.float16, torch.bfloat16, torch.float8_e4m3fn
HALF_ULP = {F32: (2.0**-24, 0.0), F16: (2.0**-11, 2.0**-25), BF16: (2.0**-8, 0.0), E4M3: (2.0**-4, 2.0**-10)}


@pytest.fixture(scope="module")
def moe():
    import serving_router_sigmoid_gb300 as m
    torch.cuda.set_device(0)
    return m


def theta(rot, base, scaling, factor, original, fast, slow):
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    th = base ** (-2 * i / rot)
    if scaling == "linear":
        th = th / factor
    if scaling == "parts":
        keep = ((original * th / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        th = th * keep + th / factor * (1 - keep)
    return th, (0.1 * math.log(factor) + 1 if scaling == "parts" else 1.0)


def turned(x, pos, th, amp, at, inter):
    """Rotated x [n, heads, dim] in 64 bits and, per element, |a| + |b| (0 where it passes through)."""
    x = x.double().cpu().clone()
    size, half = torch.zeros_like(x), th.numel()
    ang = (pos.double()[:, None] * th)[:, None]
    c, s = ang.cos() * amp, ang.sin() * amp
    i = at + torch.arange(half) * (2 if inter else 1)
    j = i + (1 if inter else half)
    a, b = x[..., i].clone(), x[..., j].clone()
    x[..., i], x[..., j] = a * c - b * s, a * s + b * c
    size[..., i] = size[..., j] = (a.abs() + b.abs()) * amp
    return x, size


def near(got, want, size, scale=1.0):
    rel, ab = HALF_ULP[got.dtype]
    got = got.cpu().to(torch.float32).double() * scale
    if rel == 2.0**-4:
        want = want.clamp(-448 * scale, 448 * scale)
    bound = size * (8 * 2.0**-24 + 2.0**-26) * (1 + rel) + want.abs() * rel + ab * scale
    if scale != 1.0:
        bound = bound + want.abs() * 2.0**-23  # the division by the scale
    bad = ((got - want).abs() > bound)
    assert not bad.any(), (int(bad.sum()), float(((got - want).abs() - bound).max()))


def check(moe, n, heads, kv, dim, rot, at=0, inter=False, act=F32, cache=BF16, page=16, v_dim=None, start=0,
          scaling="none", factor=4.0, original=512, view=True, by_head=False, drop=(), odd=0, scale=None, inplace=False):
    g = torch.Generator().manual_seed(n * 31 + dim)
    vd = dim if v_dim is None else v_dim
    width = heads * dim + kv * dim + kv * vd + odd
    x = (torch.randn((n, width), generator=g) * 2).to(act).cuda()
    q = x[:, :heads * dim].unflatten(1, (heads, dim))
    k = x[:, heads * dim:(heads + kv) * dim].unflatten(1, (kv, dim))
    v = x[:, (heads + kv) * dim:width - odd].unflatten(1, (kv, vd)) if vd else None
    if not view:
        q, k, v = q.contiguous(), k.contiguous(), None if v is None else v.contiguous()
    pages = n // page + 2
    ids = torch.randperm(pages * page, generator=g)[:n]
    slots = ids.clone()
    for t in drop:
        slots[t % n] = -1 if t % 2 else pages * page + t
    pos = torch.arange(n) + start
    sk, sv = scale or (1.0, 1.0)

    def fresh(d):
        shape = (pages, kv, page, d) if by_head else (pages, page, kv, d)
        c = torch.randn(shape, generator=g).to(cache).cuda()
        return c.transpose(1, 2) if by_head else c

    kc, vc = fresh(dim), fresh(vd) if vd else None
    k0, v0 = kc.cpu().float().double(), None if vc is None else vc.cpu().float().double()
    rope = moe.Rope(rot, base=10000.0, interleaved=inter, rot_offset=at, scaling=scaling, factor=factor,
                    original_len=original)
    th, amp = theta(rot, 10000.0, scaling, factor, original, 32.0, 1.0)
    qw, qs = turned(q, pos, th, amp, at, inter)
    kw, ks = turned(k, pos, th, amp, at, inter)
    vw = None if v is None else v.double().cpu()
    got = rope.append(q, k, v, pos.int().cuda(), slots.cuda(), kc, vc, q_out=q if inplace else None, k_scale=sk,
                      v_scale=sv)
    near(got, qw, qs)
    live = (slots >= 0) & (slots < pages * page)
    for c, rows, size, old, s in ((kc, kw, ks, k0, sk), (vc, vw, None, v0, sv)):
        if c is None:
            continue
        flat = c.contiguous().flatten(0, 1)
        flat = flat.cpu()
        near(flat.view(torch.uint8)[slots[live]].view(c.dtype) if c.dtype is E4M3 else flat[slots[live]], rows[live],
             torch.zeros_like(rows[live]) if size is None else size[live], s)
        rest = torch.ones(pages * page, dtype=torch.bool)
        rest[slots[live]] = False
        assert torch.equal(flat.float().double()[rest], old.flatten(0, 1)[rest])  # nothing else is written


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("act,cache", [(F32, BF16), (F32, F16), (F32, E4M3), (BF16, BF16), (BF16, E4M3), (F16, F16),
                                       (F16, E4M3), (BF16, F16)])
def test_types(moe, act, cache, inter):
    check(moe, 37, 8, 2, 128, 128, inter=inter, act=act, cache=cache)
    check(moe, 5, 4, 4, 64, 32, at=32, inter=inter, act=act, cache=cache, page=7)


@pytest.mark.parametrize("dim,rot,at", [(64, 64, 0), (80, 32, 48), (96, 96, 0), (96, 48, 8), (128, 64, 64), (192, 64, 128),
                                        (256, 256, 0), (256, 32, 0), (512, 512, 0), (576 - 64, 64, 448)])
@pytest.mark.parametrize("inter", [False, True])
def test_parts_of_a_head(moe, dim, rot, at, inter):
    check(moe, 19, 5, 1, dim, rot, at=at, inter=inter, act=BF16, cache=BF16)


@pytest.mark.parametrize("dim,rot,at,vd", [(7, 2, 3, 5), (10, 10, 0, 1), (36, 12, 5, 36), (100, 50, 50, 33), (128, 126, 1, 128)])
@pytest.mark.parametrize("inter", [False, True])
def test_odd_sizes(moe, dim, rot, at, vd, inter):
    for act, cache in ((F32, BF16), (BF16, E4M3), (F16, F16)):
        check(moe, 11, 3, 3, dim, rot, at=at, inter=inter, act=act, cache=cache, v_dim=vd)


@pytest.mark.parametrize("n", [1, 2, 607, 609, 1300, 5000])
def test_token_counts(moe, n):
    check(moe, n, 4, 2, 64, 64, act=BF16, cache=BF16, page=48)


def test_views_alignment_layouts(moe):
    check(moe, 9, 4, 2, 64, 64, act=F32, odd=1)                       # rows off 16 bytes
    check(moe, 9, 4, 2, 64, 64, act=BF16, odd=8, by_head=True)
    check(moe, 9, 4, 2, 64, 64, act=F16, cache=F16, view=False, by_head=True, page=3)
    check(moe, 9, 4, 2, 64, 64, act=F32, inplace=True)
    check(moe, 9, 4, 2, 64, 64, act=BF16, inter=True, inplace=True)


def test_dropped_tokens_and_no_values(moe):
    check(moe, 23, 4, 2, 64, 64, act=BF16, drop=(1, 2, 8, 22))
    check(moe, 23, 4, 2, 33, 32, act=BF16, drop=(0, 5))
    check(moe, 23, 16, 1, 192, 64, at=128, inter=True, act=BF16, v_dim=0)


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "parts"])
@pytest.mark.parametrize("start", [0, 131000, 5000000, 2**27])
def test_scalings_at_long_positions(moe, scaling, start):
    check(moe, 33, 4, 1, 128, 128, act=F32, start=start, scaling=scaling, factor=8.0, original=16384)


def test_scaled_codes_and_saturation(moe):
    check(moe, 40, 4, 2, 64, 64, act=F32, cache=E4M3, scale=(0.0225, 0.004))
    check(moe, 40, 4, 2, 64, 64, act=BF16, cache=E4M3, scale=(0.03, 7.0), inter=True)
    check(moe, 10, 2, 2, 20, 10, act=F32, cache=E4M3, scale=(0.0225, 0.004))


def test_side_stream(moe):
    rope, s = moe.Rope(64), torch.cuda.Stream()
    x = torch.randn((50, 4, 64), device="cuda")
    kc, vc = (torch.zeros((4, 16, 4, 64), dtype=BF16, device="cuda") for _ in range(2))
    pos, slots = torch.arange(50, dtype=torch.int32, device="cuda"), torch.arange(50, device="cuda")
    want = rope.append(x, x, x, pos, slots, kc, vc)
    k1 = kc.clone()
    kc.zero_()
    s.wait_stream(torch.cuda.current_stream())
    got = rope.append(x, x, x, pos, slots, kc, vc, stream=s)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(kc, k1)


def test_refusals(moe):
    rope = moe.Rope(64)
    x = torch.randn((4, 2, 64), device="cuda")
    kc, vc = (torch.zeros((2, 16, 2, 64), dtype=BF16, device="cuda") for _ in range(2))
    pos, slots = torch.arange(4, dtype=torch.int32, device="cuda"), torch.arange(4, device="cuda")
    rope.append(x, x, x, pos, slots, kc, vc)
    for bad in (dict(q=x.cpu()), dict(q=x.double()), dict(k=x[:, :, :32]), dict(v=x.half()), dict(positions=slots),
                dict(slots=pos), dict(positions=pos[:3]), dict(k_cache=kc.float()), dict(v_cache=None),
                dict(v_cache=vc[:1]), dict(q=x.transpose(1, 2)), dict(q_out=x.half())):
        a = dict(q=x, k=x, v=x, positions=pos, slots=slots, k_cache=kc, v_cache=vc)
        a.update(bad)
        with pytest.raises(ValueError):
            rope.append(**a)
    for bad in (dict(k_scale=2.0), dict(v_scale=float("nan"))):
        with pytest.raises(moe.MoeError):
            rope.append(x, x, x, pos, slots, kc, vc, **bad)
    with pytest.raises(moe.MoeError):  # a rotated part longer than the head
        moe.Rope(128).append(x, x, x, pos, slots, kc, vc)


def test_refuses_other_ranks(moe):
    rope = moe.Rope(64)
    x = torch.randn((4, 2, 64), device="cuda")
    kc, vc = (torch.zeros((2, 16, 2, 64), dtype=BF16, device="cuda") for _ in range(2))
    pos, slots = torch.arange(4, dtype=torch.int32, device="cuda"), torch.arange(4, device="cuda")
    for bad in (dict(q=x[0]), dict(k=x[0]), dict(v=x[0]), dict(q_out=x[0]), dict(positions=pos[0]), dict(slots=slots[0]),
                dict(k_cache=kc[0]), dict(v_cache=vc[0]), dict(v_cache=vc[0, 0, 0, 0])):
        a = dict(q=x, k=x, v=x, positions=pos, slots=slots, k_cache=kc, v_cache=vc)
        a.update(bad)
        with pytest.raises(ValueError):
            rope.append(**a)


def test_one_object_in_two_threads(moe):
    """A Rope keeps nothing of a call: threads on streams of their own share it."""
    from concurrent.futures import ThreadPoolExecutor
    rope = moe.Rope(64)

    def work(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            x = torch.randn((5 + seed, 2, 64), device="cuda", generator=g)
            kc, vc = (torch.zeros((2, 16, 2, 64), dtype=BF16, device="cuda") for _ in range(2))
            n = x.shape[0]
            pos, slots = torch.arange(n, dtype=torch.int32, device="cuda"), torch.arange(n, device="cuda")
            first = rope.append(x, x, x, pos, slots, kc, vc)
            same = torch.ones((), dtype=torch.bool, device="cuda")
            for _ in range(200):
                same &= (rope.append(x, x, x, pos, slots, kc, vc) == first).all()
            s.synchronize()
            return bool(same) and torch.equal(vc.view(-1, 2, 64)[:n], x.to(BF16))

    with ThreadPoolExecutor(4) as pool:
        assert all(pool.map(work, range(4)))
