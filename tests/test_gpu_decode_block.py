"""The example block (examples/decode_block.py) over a prompt and several
decode steps, against the same steps in 64 bits on unpaged keys and values.

Keys and values are rounded to bf16 in the cache, so the reference rounds its
own; a key that falls on the other side of a rounding moves a logit by 2^-8 of
one product at most, which for 64 dimensions and few such keys stays below 1e-3
relative in the attention's output.  Beyond the attention everything is fp32
(the MoE layer is compared at its own input, by the layer itself).
"""
import os
import sys

import pytest
import torch

ROOT = os.path.abspath(os.path.join(os.path.dirname(__file__), ".."))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def norm(x, w, eps):
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w


def turn(x, pos, base):
    half = x.shape[-1] // 2
    th = base ** (-torch.arange(half, dtype=torch.float64, device=x.device) / half)
    z = torch.polar(torch.ones_like(th * pos[:, None].double()), th * pos[:, None].double())[:, None]
    r = torch.view_as_complex(x.unflatten(-1, (half, 2)).contiguous()) * z
    return torch.view_as_real(r).flatten(-2)


def test_steps_against_64_bits():
    import decode_block as ex
    torch.backends.cuda.matmul.allow_tf32 = False
    n = 5
    block = ex.Block(n, pages=64)
    w, d = block.w, block.cfg.D
    g = torch.Generator(device="cuda").manual_seed(3)
    lengths = torch.tensor([17, 1, 0, 33, 16], dtype=torch.int32, device="cuda")
    prompt = torch.randn((67, d), generator=g, device="cuda")
    block.prompt(prompt, lengths)
    keys, values = [[] for _ in range(n)], [[] for _ in range(n)]

    def qkv(x, pos):
        q, k, v = (norm(x.double(), w.pre.double(), ex.EPS) @ w.qkv.double()).split(
            [ex.HEADS * ex.DIM, ex.KV_HEADS * ex.DIM, ex.KV_HEADS * ex.DIM], dim=1)
        q, k, v = (t.unflatten(1, (-1, ex.DIM)) for t in (q, k, v))
        return turn(q, pos, ex.BASE), turn(k, pos, ex.BASE).bfloat16().double(), v.bfloat16().double()

    at = 0
    for b, m in enumerate(lengths.tolist()):
        _, k, v = qkv(prompt[at:at + m], torch.arange(m, device="cuda"))
        keys[b] += list(k)
        values[b] += list(v)
        at += m
    x = torch.randn((n, d), generator=g, device="cuda")
    for step in range(20):  # across page ends
        got = block.step(x)
        q, k, v = qkv(x, lengths + step)
        att = []
        for b in range(n):
            keys[b].append(k[b])
            values[b].append(v[b])
            ks, vs = torch.stack(keys[b]), torch.stack(values[b])
            s = torch.einsum("hgd,lhd->hgl", q[b].unflatten(0, (ex.KV_HEADS, -1)), ks) / ex.DIM**0.5
            att.append(torch.einsum("hgl,lhd->hgd", torch.softmax(s, -1), vs).flatten(0, 1))
        att = torch.stack(att)
        assert float((got.attention - att).norm() / att.norm()) < 1e-3
        y = got.attention.double().flatten(1) @ w.out.double()
        r = x.double() + torch.sigmoid(w.gate.double()) * norm(y, w.post.double(), ex.EPS)
        assert float((got.residual - r).norm() / r.norm()) < 1e-5
        h = norm(r, w.moe.double(), ex.EPS)
        assert float((got.expert_input - h).norm() / h.norm()) < 1e-5
        assert torch.equal(got.experts, block.layer.forward(got.expert_input))
        assert torch.equal(got.out, got.residual + got.experts)
        assert block.plan.info[2].item() == 0 and block.past.tolist() == (lengths + step + 1).tolist()
        x = got.out
    assert block.layer.device_status() == 0
    used = block.table[block.table >= 0].tolist()
    assert len(used) == len(set(used)) == int(block.head)  # no page is held twice
    block.layer.close()
