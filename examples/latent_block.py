#!/usr/bin/env python
"""Prompts and decode steps of one transformer block with a latent cache, FP8
matrices and routed experts.

    python examples/latent_block.py [--requests N] [--steps K] [--cache bf16|e4m3]

The cache holds one row a token that all heads share: a normed latent and a
rotary part.  The calls of a block, as they follow each other in a serving loop:

    plan      pages, positions and slots of the new tokens       KvPlan.update
    norm      the block's input norm                             block_norm
    q         FP8: to the query latent, norm, FP8: to the heads  quant_act_fp8, fp8_linear, block_norm
    row       FP8: to the latent row, norm of its latent         quant_act_fp8, fp8_linear, block_norm
    rope      rotary positions, the row into the cache           Rope.append
    attend    prompts: keys and values expanded a head (FP8)     fp8_linear, latent_prompt
              steps: the key expansion absorbed into q           torch, LatentAttention.decode, torch
    project   FP8: back to the residual stream                   quant_act_fp8, fp8_linear
    join      norm after attention, gate, residual, norm         block_norm
    experts   the routed-MoE layer                               MoeLayer.forward
    join      residual add                                       block_norm

The residual stream is fp32 (what the MoE layer takes), the attention bf16.
Weights are random.
"""
import argparse
import os
import sys
from types import SimpleNamespace

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import serving_router_sigmoid_gb300 as moe  # noqa: E402
import synth  # noqa: E402

HEADS, NOPE, ROPE, V, LATENT, Q_LATENT, PAGE = 8, 64, 32, 64, 128, 192, 16
BASE, EPS = 10000.0, 1e-5
SCALE = (NOPE + ROPE) ** -0.5


def fp8_matrix(w):
    """A matrix [O, I] as a checkpoint holds it: E4M3 codes and one scale a 128 x 128 block."""
    o, i = w.shape
    blocks = torch.nn.functional.pad(w, (0, -i % 128, 0, -o % 128)).unflatten(1, (-1, 128)).unflatten(0, (-1, 128))
    scale = blocks.abs().amax((1, 3)) / 448
    codes = (blocks / scale[:, None, :, None]).to(torch.float8_e4m3fn).flatten(2).flatten(0, 1)[:o, :i]
    return codes.contiguous(), scale.contiguous()


def widened(w8, scale):
    return w8.float() * scale.repeat_interleave(128, 0).repeat_interleave(128, 1)[:w8.shape[0], :w8.shape[1]]


def linear(x, w, dtype=torch.bfloat16):
    return moe.fp8_linear(*moe.quant_act_fp8(x), *w, dtype=dtype)


class Block:
    """The block's weights and handles, and the state of its requests."""

    def __init__(self, requests, pages=256, max_new=1024, cache=torch.bfloat16, config="tiny", seed=0, device="cuda"):
        cfg = self.cfg = synth.CONFIGS[config]
        g = torch.Generator(device=device).manual_seed(seed)
        new = lambda *shape: torch.randn(shape, generator=g, device=device)  # noqa: E731
        matrix = lambda o, i: fp8_matrix(new(o, i) / i**0.5)  # noqa: E731
        near1 = lambda n: 1 + 0.1 * new(n)  # noqa: E731
        d = cfg.D
        self.w = SimpleNamespace(
            q_a=matrix(Q_LATENT, d), q_b=matrix(HEADS * (NOPE + ROPE), Q_LATENT), kv_a=matrix(LATENT + ROPE, d),
            kv_b=matrix(HEADS * (NOPE + V), LATENT), o=matrix(d, HEADS * V), pre=near1(d), q_norm=near1(Q_LATENT),
            kv_norm=near1(LATENT), post=near1(d), moe=near1(d), gate=new(1, d))
        # for steps: the expansions of keys and values a head, [heads, nope or v, latent]
        kv_b = widened(*self.w.kv_b).bfloat16().unflatten(0, (HEADS, NOPE + V))
        self.w.k_b, self.w.v_b = kv_b[:, :NOPE].contiguous(), kv_b[:, NOPE:].contiguous()
        experts = []
        for e in range(cfg.E + cfg.n_shared):
            packed = [moe.pack_int4(w.to(device)) for w in synth.expert_fp32(cfg, e)]
            experts.append(tuple(t for pair in packed for t in pair))
        self.layer = moe.MoeLayer(cfg.D, cfg.I, cfg.E, cfg.K, cfg.n_shared, cfg.routed_scale, max_new,
                                  synth.router_weight(cfg).to(device), synth.router_bias(cfg).to(device), experts)
        # rotary parts: behind the latent (rows, absorbed queries), behind the plain part (queries of prompts)
        self.rope, self.rope_q = (moe.Rope(ROPE, base=BASE, interleaved=True, rot_offset=at, device=device)
                                  for at in (LATENT, NOPE))
        self.attn = moe.LatentAttention(requests, HEADS, LATENT, ROPE, device=device)
        self.plan = moe.KvPlan(requests, max_new, PAGE, device=device)
        self.cache = torch.zeros((pages, PAGE, 1, LATENT + ROPE), device=device).to(cache)
        self.k_scale = 1.0 if cache == torch.bfloat16 else 1 / 16  # E4M3: codes hold row / k_scale, up to 448
        # the serving state: a list of free pages and its head, a page table, the lengths so far
        self.free = torch.randperm(pages, generator=g, device=device).to(torch.int32)
        self.head = torch.zeros(1, dtype=torch.int32, device=device)
        self.table = torch.full((requests, pages), -1, dtype=torch.int32, device=device)
        self.past = torch.zeros(requests, dtype=torch.int32, device=device)
        self.one = torch.ones(requests, dtype=torch.int32, device=device)
        self.nowhere = torch.full((max_new,), -1, dtype=torch.int64, device=device)

    def allocate(self, new_len):
        """Pages and slots for new_len tokens a request; the lengths move on."""
        self.plan.update(self.past, new_len, self.free, self.head, self.table)
        self.head.copy_(self.plan.info[1:2])
        self.past.copy_(self.plan.seq_len)
        return self.plan

    def project(self, x):
        """The input norm, the queries [n, heads, nope + rope] and the cache rows
        [n, latent + rope], both before their rotary positions."""
        _, h = moe.block_norm(x, w_pre=self.w.pre, eps=EPS)
        h8 = moe.quant_act_fp8(h)  # once for both products
        _, qa = moe.block_norm(moe.fp8_linear(*h8, *self.w.q_a), w_pre=self.w.q_norm, eps=EPS)
        q = linear(qa, self.w.q_b).unflatten(1, (HEADS, NOPE + ROPE))
        raw = moe.fp8_linear(*h8, *self.w.kv_a)
        row = torch.empty_like(raw)
        moe.block_norm(raw[:, :LATENT], w_pre=self.w.kv_norm, eps=EPS, normed=row[:, :LATENT])
        row[:, LATENT:] = raw[:, LATENT:]
        return q, row

    def finish(self, x, a):
        """From the attention's output [n, heads, v] to the block's."""
        y = linear(a.flatten(1), self.w.o, dtype=torch.float32)
        r, h = moe.block_norm(x, y, w_post=self.w.post, gate=self.w.gate, w_pre=self.w.moe, eps=EPS)
        m = self.layer.forward(h)
        out, _ = moe.block_norm(r, m)
        return SimpleNamespace(projected=y, residual=r, expert_input=h, experts=m, out=out)

    def prompt(self, x, lengths):
        """Whole prompts of new requests: x [sum(lengths), D] -> the block's output and its parts."""
        plan = self.allocate(lengths)
        q, row = self.project(x)
        # the rows are queries of their own here: their turned form comes back, too
        row = self.rope.append(row[:, None], row[:, None], None, plan.positions, plan.slots, self.cache, None,
                               k_scale=self.k_scale)[:, 0]
        q = self.rope_q.append(q, q[:, :1], None, plan.positions, self.nowhere, self.cache[..., :NOPE + ROPE], None)
        kv = linear(row[:, :LATENT], self.w.kv_b).unflatten(1, (HEADS, NOPE + V))
        a, lse = moe.latent_prompt(q, kv[..., :NOPE], row[:, LATENT:], kv[..., NOPE:], plan.q_start, plan.q_start, SCALE)
        return SimpleNamespace(q=q, row=row, kv=kv, attention=a, lse=lse, **vars(self.finish(x, a)))

    def step(self, x):
        """One new token a request: x [requests, D] -> the block's output and its parts."""
        plan = self.allocate(self.one)
        heads, row = self.project(x)
        q = heads.new_empty((x.shape[0], HEADS, LATENT + ROPE))
        q[..., :LATENT] = torch.einsum("nhd,hdl->nhl", heads[..., :NOPE], self.w.k_b)
        q[..., LATENT:] = heads[..., NOPE:]
        q = self.rope.append(q, row[:, None], None, plan.positions, plan.slots, self.cache, None, k_scale=self.k_scale)
        c, lse = self.attn.decode(q, self.cache, self.table, plan.seq_len, SCALE, k_scale=self.k_scale)
        a = torch.einsum("nhl,hvl->nhv", c, self.w.v_b)
        return SimpleNamespace(heads=heads, q=q, row=row, latent=c, lse=lse, attention=a, **vars(self.finish(x, a)))


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    a = ap.parse_args()
    block = Block(a.requests, cache=torch.bfloat16 if a.cache == "bf16" else torch.float8_e4m3fn)
    g = torch.Generator(device="cuda").manual_seed(1)
    lengths = torch.arange(5, 5 + 7 * a.requests, 7, dtype=torch.int32, device="cuda")
    x = block.prompt(torch.randn((int(lengths.sum()), block.cfg.D), generator=g, device="cuda"), lengths).out
    x = x[lengths.cumsum(0) - 1]  # each request's last token
    for i in range(a.steps):
        x = block.step(x).out
        flags = int(block.plan.info[2])
        print(f"step {i}: lengths {block.past.tolist()}, |x| {float(x.norm()):.4f}, plan flags {flags}")
        if flags:
            raise SystemExit("out of pages")
    if block.layer.device_status() or moe.dense_status():
        raise SystemExit("a kernel flagged an error")


if __name__ == "__main__":
    main()
