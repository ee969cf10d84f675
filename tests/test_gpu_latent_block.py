"""The example block (examples/latent_block.py): its operators as they follow
each other, against 64 bits, and in a CUDA graph against the same calls with a
synchronisation after each.

The FP8 products and the attention are held to the bounds of their own tests, each
at its own inputs.  Steps are also held to the expanded form of the attention in
64 bits, from the cached rows and the queries before absorption: absorbing rounds
each of a query's latent numbers by 2^-8 and its sum of products runs in fp32, so
a logit moves by less than D = (2^-8 + 2^-12) S, S its sum of absolute products
with absolute expansions; weights then move by a factor e^(2 D) at most, the latent
output and the expanded one round by 2^-8 each, weights by 2^-8 (and once more in
the cached rows' place for the queries' rotary part: rounded after its turn, within
the 2^-8 of S): |error| <= (e^(2 D) (1 + 2^-8)^3 - 1) P with P the absolute form of the output.
"""
import math
import os
import sys

import pytest
import torch

ROOT = os.path.abspath(os.path.join(os.path.dirname(__file__), ".."))
sys.path.insert(0, os.path.join(ROOT, "examples"))

import test_gpu_fp8_linear as products  # noqa: E402
import test_gpu_latent_decode as decode  # noqa: E402
import test_gpu_latent_prompt as prompts  # noqa: E402

pytestmark = pytest.mark.gpu

BF, E4 = torch.bfloat16, torch.float8_e4m3fn
LENGTHS = [17, 1, 0, 200, 16]


@pytest.fixture(scope="module")
def ex():
    import latent_block
    torch.cuda.set_device(0)
    torch.backends.cuda.matmul.allow_tf32 = False
    return latent_block


def begin(ex, cache, seed=3):
    block = ex.Block(len(LENGTHS), pages=64, cache=cache)
    g = torch.Generator(device="cuda").manual_seed(seed)
    lengths = torch.tensor(LENGTHS, dtype=torch.int32, device="cuda")
    x = torch.randn((sum(LENGTHS), block.cfg.D), generator=g, device="cuda")
    return block, lengths, x, torch.randn((len(LENGTHS), block.cfg.D), generator=g, device="cuda")


def turn(x, pos, base):
    half = x.shape[-1] // 2
    th = base ** (-torch.arange(half, dtype=torch.float64, device=x.device) / half)
    z = torch.polar(torch.ones_like(th * pos[:, None].double()), th * pos[:, None].double())[:, None]
    r = torch.view_as_complex(x.unflatten(-1, (half, 2)).contiguous()) * z
    return torch.view_as_real(r).flatten(-2)


def cached(block, b, n):
    return decode.rows_of(block.cache, block.table, b, n) * block.k_scale


@pytest.mark.parametrize("cache", [BF, E4])
def test_block_against_64_bits(ex, cache):
    import serving_router_sigmoid_gb300 as moe
    block, lengths, px, x = begin(ex, cache)
    w = block.w
    got = block.prompt(px, lengths)
    starts = block.plan.q_start
    assert starts.tolist() == [0, 17, 18, 18, 218, 234]
    prompts.check(got.attention, got.lse, got.q, got.kv[..., :ex.NOPE], got.row[:, ex.LATENT:], got.kv[..., ex.NOPE:], starts,
                  starts, ex.SCALE, True)
    products.check(got.kv.flatten(1), *moe.quant_act_fp8(got.row[:, :ex.LATENT].contiguous()), *w.kv_b)
    products.check(got.projected, *moe.quant_act_fp8(got.attention.flatten(1)), *w.o)
    # the rows of the cache are those the prompt computed with, rounded to the cache's type
    at = 0
    for b, n in enumerate(LENGTHS):
        want = (got.row[at:at + n].double() / block.k_scale).float().to(cache).double() * block.k_scale
        held, lat = cached(block, b, n), slice(0, ex.LATENT)
        assert torch.equal(held[:, lat], want[:, lat])
        # the turned part is rounded once in the cache, twice here: a step of the cache's type apart at most
        step = 0.0 if cache == BF else 2.0**-3
        assert bool(((held - want).abs() <= step * torch.maximum(held.abs(), want.abs()) + step * 2.0**-6 * block.k_scale).all())
        at += n
    for step in range(20):  # across page ends
        got = block.step(x)
        lens = lengths + step + 1
        decode.check(got.latent, got.lse, got.q, block.cache, block.table, lens, ex.LATENT, ex.SCALE, block.k_scale)
        products.check(got.projected, *moe.quant_act_fp8(got.attention.flatten(1)), *w.o)
        kb, vb = w.k_b.double(), w.v_b.double()
        for b, n in enumerate(lens.tolist()):
            c = cached(block, b, n)
            lat, rot = c[:, :ex.LATENT], c[:, ex.LATENT:]
            qn = got.heads[b, :, :ex.NOPE].double()
            qr = turn(got.heads[b:b + 1, :, ex.NOPE:].double(), (lens[b:b + 1] - 1), ex.BASE)[0]
            keys = torch.einsum("hdl,jl->jhd", kb, lat)
            s = (torch.einsum("hd,jhd->hj", qn, keys) + qr @ rot.T) * ex.SCALE
            size = (torch.einsum("hl,jl->hj", torch.einsum("hd,hdl->hl", qn.abs(), kb.abs()), lat.abs()) +
                    qr.abs() @ rot.abs().T * 2) * ex.SCALE
            p = torch.softmax(s, -1)
            ref = torch.einsum("hj,jl,hvl->hv", p, lat, vb)
            total = torch.einsum("hj,jl,hvl->hv", p, lat.abs(), vb.abs())
            d = (2.0**-8 + 2.0**-12) * size.amax(-1, keepdim=True)
            room = (torch.exp(2 * d) * (1 + 2.0**-8) ** 3 - 1) * total
            off = (got.attention[b].double() - ref).abs()
            assert bool((off <= room).all()), (step, b, float((off / room).max()))
            # the bound is loose for sums of many signs; in the norm the two forms are close
            assert float(off.norm() / ref.norm()) < 0.05
        assert torch.equal(got.experts, block.layer.forward(got.expert_input))
        assert torch.equal(got.out, got.residual + got.experts)
        assert block.plan.info[2].item() == 0 and block.past.tolist() == lens.tolist()
        x = got.out
    assert block.layer.device_status() == 0 and moe.dense_status() == 0
    used = block.table[block.table >= 0].tolist()
    assert len(used) == len(set(used)) == int(block.head)  # no page is held twice
    block.layer.close()
    block.attn.close()


def test_a_step_continues_a_prompt(ex):
    """The last token of a prompt, expanded, against the same token as a step, absorbed."""
    block, lengths, px, _ = begin(ex, BF, seed=4)
    whole = block.prompt(px, lengths)
    other, _, _, _ = begin(ex, BF, seed=4)
    b, n = 3, LENGTHS[3]
    at = sum(LENGTHS[:b])
    keep = torch.ones(sum(LENGTHS), dtype=torch.bool, device="cuda")
    keep[at + n - 1] = False
    short = lengths.clone()
    short[b] -= 1
    other.prompt(px[keep], short)
    x = torch.zeros((len(LENGTHS), block.cfg.D), device="cuda")
    x[b] = px[at + n - 1]
    a, e = other.step(x).attention[b].double(), whole.attention[at + n - 1].double()
    # keys and values come from codes here, off by up to 2^-4 each, 2.6 % in the mean square: the same for a sum of them,
    # once by the values and once by logits of about unit size
    assert float((a - e).norm() / e.norm()) < 0.1


@pytest.mark.parametrize("cache", [BF, E4])
def test_overlapped_launches_see_the_outputs_before_them(ex, cache, monkeypatch):
    import serving_router_sigmoid_gb300 as moe
    block, lengths, px, x0 = begin(ex, cache)
    state = [block.cache, block.table, block.past, block.head]
    zero = [t.clone() for t in state]

    def reset():
        for t, z in zip(state, zero):
            t.view(torch.uint8).copy_(z.view(torch.uint8))

    def run():
        parts, x = [block.prompt(px, lengths)], x0
        for _ in range(3):
            parts.append(block.step(x))
            x = parts[-1].out
        return [t for p in parts for t in vars(p).values()]

    with monkeypatch.context() as m:
        for owner, name in ((moe, "block_norm"), (moe, "quant_act_fp8"), (moe, "fp8_linear"), (moe, "latent_prompt"),
                            (moe.LatentAttention, "decode"), (moe.Rope, "append"), (moe.KvPlan, "update"),
                            (moe.MoeLayer, "forward")):
            def waits(*a, call=getattr(owner, name), **k):
                torch.cuda.synchronize()
                r = call(*a, **k)
                torch.cuda.synchronize()
                return r
            m.setattr(owner, name, waits)
        want = [t.clone() for t in run()] + [t.clone() for t in state]
    assert all(bool(torch.isfinite(t.float()).all()) for t in want[:-4] if t.dim() > 2)
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(10):
        reset()
        for t in got:
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got + state, want))
    assert moe.dense_status() == 0
    del graph


@pytest.mark.parametrize("how", ["del", "close"])
def test_a_handle_dropped_in_a_capture(ex, how):
    import serving_router_sigmoid_gb300 as moe
    x = torch.randn(64, 64, device="cuda")
    gone = moe.LatentAttention(2, 8)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = x + 1
        if how == "close":
            gone.close()
        del gone
        y = y * 2
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, (x + 1) * 2)
    assert len(moe._parked) == 1
    moe.LatentAttention(1, 1).close()  # the next one to close takes it along
    assert not moe._parked


def test_example_runs(ex, monkeypatch, capsys):
    for cache in ("bf16", "e4m3"):
        monkeypatch.setattr(sys, "argv", ["latent_block.py", "--requests", "2", "--steps", "3", "--cache", cache])
        ex.main()
        out = capsys.readouterr().out
        assert "step 2: lengths [8, 15]" in out and math.isfinite(float(out.split("|x| ")[-1].split(",")[0]))
