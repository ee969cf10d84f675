#!/usr/bin/env python
"""Decode steps of one transformer block with routed experts on a paged cache.

    python examples/decode_block.py [--requests N] [--steps K]

One block, as its calls follow each other in a serving loop:

    plan     pages, positions and slots of the new tokens    KvPlan.update
    norm     the block's input norm                          block_norm
    q, k, v  one projection                                  torch
    rope     rotary positions, k and v into the cache        Rope.append
    attend   one new token a request over its pages          PagedAttention.decode
    project  back to the residual stream                     torch
    join     norm after attention, gate, residual, norm      block_norm
    experts  the routed-MoE layer                            MoeLayer.forward
    join     residual add                                    block_norm

The activations are fp32 (what the MoE layer takes), the cache bf16.  Weights
are random; prompts are written to the cache by the same plan and append calls.
"""
import argparse
import os
import sys
from types import SimpleNamespace

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import serving_router_sigmoid_gb300 as moe  # noqa: E402
import synth  # noqa: E402

HEADS, KV_HEADS, DIM, PAGE = 8, 2, 64, 16
BASE, EPS = 10000.0, 1e-5


class Block:
    """The block's weights and handles, and the state of its requests."""

    def __init__(self, requests, pages=256, max_new=4096, config="tiny", seed=0, device="cuda"):
        cfg = self.cfg = synth.CONFIGS[config]
        g = torch.Generator(device=device).manual_seed(seed)
        new = lambda *shape: torch.randn(shape, generator=g, device=device)  # noqa: E731
        d, width = cfg.D, (HEADS + 2 * KV_HEADS) * DIM
        self.w = SimpleNamespace(qkv=new(d, width) / d**0.5, out=new(HEADS * DIM, d) / (HEADS * DIM) ** 0.5,
                                 pre=1 + 0.1 * new(d), post=1 + 0.1 * new(d), moe=1 + 0.1 * new(d), gate=new(1, d))
        experts = []
        for e in range(cfg.E + cfg.n_shared):
            packed = [moe.pack_int4(w.to(device)) for w in synth.expert_fp32(cfg, e)]
            experts.append(tuple(t for pair in packed for t in pair))
        self.layer = moe.MoeLayer(cfg.D, cfg.I, cfg.E, cfg.K, cfg.n_shared, cfg.routed_scale, requests,
                                  synth.router_weight(cfg).to(device), synth.router_bias(cfg).to(device), experts)
        self.rope = moe.Rope(DIM, base=BASE, interleaved=True, device=device)
        self.attn = moe.PagedAttention(requests, HEADS, KV_HEADS, DIM, device=device)
        self.plan = moe.KvPlan(requests, max_new, PAGE, device=device)
        self.k_cache, self.v_cache = (torch.zeros((pages, PAGE, KV_HEADS, DIM), dtype=torch.bfloat16, device=device)
                                      for _ in range(2))
        # the serving state: a list of free pages and its head, a page table, the lengths so far
        self.free = torch.randperm(pages, generator=g, device=device).to(torch.int32)
        self.head = torch.zeros(1, dtype=torch.int32, device=device)
        self.table = torch.full((requests, pages), -1, dtype=torch.int32, device=device)
        self.past = torch.zeros(requests, dtype=torch.int32, device=device)
        self.one = torch.ones(requests, dtype=torch.int32, device=device)

    def allocate(self, new_len):
        """Pages and slots for new_len tokens a request; the lengths move on."""
        self.plan.update(self.past, new_len, self.free, self.head, self.table)
        self.head.copy_(self.plan.info[1:2])
        self.past.copy_(self.plan.seq_len)
        return self.plan

    def project(self, x):
        """The input norm and q, k, v as views of one projection."""
        _, h = moe.block_norm(x, w_pre=self.w.pre, eps=EPS)
        qkv = h @ self.w.qkv
        q, k, v = qkv.split([HEADS * DIM, KV_HEADS * DIM, KV_HEADS * DIM], dim=1)
        return q.unflatten(1, (HEADS, DIM)), k.unflatten(1, (KV_HEADS, DIM)), v.unflatten(1, (KV_HEADS, DIM))

    def prompt(self, x, lengths):
        """The prompts' keys and values into the cache; x [sum(lengths), D]."""
        plan = self.allocate(lengths)
        q, k, v = self.project(x)
        self.rope.append(q, k, v, plan.positions, plan.slots, self.k_cache, self.v_cache)

    def step(self, x):
        """One new token a request: x [requests, D] -> the block's output and its parts."""
        plan = self.allocate(self.one)
        q, k, v = self.project(x)
        q = self.rope.append(q, k, v, plan.positions, plan.slots, self.k_cache, self.v_cache)
        a, _ = self.attn.decode(q, self.k_cache, self.v_cache, self.table, plan.seq_len)
        y = a.flatten(1) @ self.w.out
        r, h = moe.block_norm(x, y, w_post=self.w.post, gate=self.w.gate, w_pre=self.w.moe, eps=EPS)
        m = self.layer.forward(h)
        out, _ = moe.block_norm(r, m)
        return SimpleNamespace(attention=a, residual=r, expert_input=h, experts=m, out=out)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    block = Block(a.requests)
    g = torch.Generator(device="cuda").manual_seed(1)
    lengths = torch.arange(5, 5 + 7 * a.requests, 7, dtype=torch.int32, device="cuda")
    block.prompt(torch.randn((int(lengths.sum()), block.cfg.D), generator=g, device="cuda"), lengths)
    x = torch.randn((a.requests, block.cfg.D), generator=g, device="cuda")
    for i in range(a.steps):
        x = block.step(x).out
        flags = int(block.plan.info[2])
        print(f"step {i}: lengths {block.past.tolist()}, |x| {float(x.norm()):.4f}, plan flags {flags}")
        if flags:
            raise SystemExit("out of pages")
    if block.layer.device_status():
        raise SystemExit("the MoE layer flagged an error")


if __name__ == "__main__":
    main()
